// Attention of one new token per sequence over a paged key/value cache.
//
//     o = sum_j p_j v_j / sum_j p_j,   p_j = exp(scale q.k_j - m)
//
// for the query heads of one K/V head at a time. It is bound by HBM: every
// key and value is read once (2 d elements a key and K/V head) for 4 G d
// operations, G query heads a K/V head, so the matrix work is far below what
// even the warp-level matrix instructions give, and what counts is that every
// SM has loads in flight all the time, whatever the sequences' lengths.
//
// Work split. A unit is (sequence, K/V head, block of up to 8 NT query heads),
// cut into steps of kStep keys; the steps of ALL units, laid end to end, are
// shared out evenly over all WARPS of the grid (kWarps a block, one block an
// SM), so ragged lengths balance to one step, one long sequence fills the chip
// and many short ones cost no block-wide hand-over. A warp's range covers the
// end of one unit, whole units, and the start of another. Whole units are
// finished in registers. A unit that ends in a later warp than it began in
// leaves partial results (normalised O and log-sum-exp, fp32): one from the
// warp that ends it, and one a block from the warps that are still inside it
// when their ranges end, joined in shared memory once, at the block's end.
// fa_paged_join adds a unit's parts in order. A block leaves at most 2 kWarps
// parts whatever the lengths, so the workspace does not grow with them.
//
// A warp has a ring of kStages (K, V) steps of its own that its lanes fill
// with 16-byte cp.async, and it runs on across unit boundaries: there is no
// block barrier before the end. Each lane looks up the page of one key of the
// next step while the present one is computed, and the rows' offsets go round
// by shuffle: any page size and page order costs the same (one page looked up
// for 16 keys, where page_size is a multiple of 16, was no faster). A key that
// is hidden or has no page is zero-filled and its score set to -inf, never
// read, so what lies there cannot reach the result. Keys and values are marked
// to leave L2 first: parts, tables and what the next kernels read stay there.
// Without the mark a batch of 16 takes 60.6 us for 59.9, one of 256 short
// sequences 38.8 for 36.0. Keys that are read again lose a little by it:
// 16 sequences with 32768 keys in shared pages take 207 us for 200 without, 128
// query heads on one K/V head (blocks of 16, each reading the keys) 70.0 for 68.3.
//
// Products (mma.sync m16n8k16, fp32 accumulators): S^T = K Q^T with the keys
// as rows and 8 query heads as columns, then O^T += V^T P^T. The C fragment of
// S^T transposed 8x8 block by block (movmatrix) is the B fragment of P^T, and
// a thread's two columns (heads) are the same in S^T and O^T, so running
// maxima, sums and rescaling never leave the thread. A head's reference
// maximum moves only when a score exceeds it by more than 8 (log2 units),
// found by one vote a step; p is at most 2^8 and O / sum is exact whatever the
// reference. e4m3 keys and values are widened exactly to f16 (one conversion
// for two) and multiplied there; q, whose bf16 range f16 lacks, is scaled by a
// power of two per head first, which is exact but for elements 2^-31 below the
// head's largest (its largest lies in [2^14, 2^15) then, where f16's smallest
// step, 2^-24, is the last bit of a bf16 value 2^-31 below).
//
// Roundings. bf16 values want bf16 probabilities, off by up to 2^-8 each; as
// the matrix pipe is idle most of the time, P enters the product as two bf16
// parts (p rounded, and the rest rounded: 2^-16), which costs 0.5 % of the
// time and leaves O with the rounding of its result alone; O is divided by the
// exact sum. For e4m3 P is f16 (2^-11, an eighth of a bf16 result's own
// rounding), and O is divided by the sum of the rounded probabilities. f16 ends
// at 2^-24, so p is taken 2^7 larger there: keys above 2^-32 of the reference key
// count, where many of them between that and 2^-25 would be lost to O. A second
// f16 part takes 2 to 9 % longer (16 heads a K/V head, 8 sequences of 16384 keys:
// 37.7 us for 34.5; the batch of 32 below 56.0 for 54.3). lse takes the exact
// sum.
//
// Measured (device time, both kernels): one sequence of 131072 tokens, 8 K/V
// heads, d 128 89 us (537 MB: 6.1 TB/s), 16 of 2048 to 8192 tokens 57.5 us
// (336 MB: 5.8 TB/s), 256 of 20 to 300 tokens 36 us (171 MB: 4.8 TB/s), e4m3
// 32 of 9 to 8192 tokens 54.3 us (269 MB: 5.0 TB/s; all 8192 long, 89 us for 537
// MB), 777 tokens 12 heads d 64 8.9 us. Beyond 16 heads a K/V head keys are read
// again for every 16: 32 and 128 heads on one K/V head, 4 sequences of 32768
// keys, 30 and 70 us where the bytes once want 10; d 256, 32 heads, 66 us (46
// e4m3), where the 16-head kernels spill 76 to 252 bytes a thread. Of a long call 4
// us pass before the first key arrives (lengths, page numbers, keys: three
// trips to memory), and 5 to 9 between the first and the last SM's end: under
// full load a fifth of the SMs get a tenth less bandwidth.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cstdint>

#include "cp_async.cuh"
#include "sm100_ptx.cuh"

namespace fa {

constexpr int kPdBlocks = 148;             // one block an SM
// Warps of a block, at most, by head dim and 8-head products a unit.
constexpr int pd_warps_most(int d, int nt) { return d == 128 && nt == 1 ? 12 : 8; }

// A row's bytes decide how the ring is cut: two or three stages a warp of 4 to
// 16 KB, 96 to 128 KB on the way an SM. Rows of 128 bytes or less take 32 keys
// a step (e4m3 d 128: 16-key steps 64.7 us, 32-key steps 60.6 us on the batch
// of 32), and e4m3 at d 128 with up to 8 heads 12 warps of two stages instead
// of 8 of three (91.6 and 95.4 us, all sequences 8192 long; 16 warps of 16-key
// steps 99.7). 512-byte rows take 6 warps of two stages (16 heads a K/V head:
// 119 us; 4 warps of three stages 137).
template <int D, int E, int NT>
struct PdCfg {
    static constexpr int kRow = D * E;                                    // bytes of a K or V row
    static constexpr int kStep = kRow <= 128 ? 32 : 16;                   // keys of a step
    static constexpr int kGroups = kStep / 16;
    static constexpr int kStage = 2 * kStep * kRow;                       // K and V of a step
    static constexpr int kWarps = kRow >= 512 ? 6 : (D == 128 && E == 1 && NT == 1) ? 12 : 8;
    static constexpr int kThreads = 32 * kWarps;
    static constexpr int kStages = kWarps == 12 || kWarps == 6 ? 2 : kRow >= 128 ? 3 : 6;
    static constexpr int kHeads = 8 * NT;
    static constexpr int kPitch = D + 4;                                  // of the merge buffer
    static constexpr int kRing = kWarps * kStages * kStage;
    static constexpr int kMerge = kWarps * kHeads * kPitch * 4;           // in the ring's place
    static constexpr int kStat = 3 * kWarps * kHeads * 4;                 // m, l, lr
    // log2 of a factor in every p: a score is at most 8 above the reference, so p
    // in f16 (2^-24 to 2^16) then reaches up to 2^15
    static constexpr float kLift = E == 1 ? 7.f : 0.f;
    static constexpr int kSmem = kRing + kStat + kWarps * kStages * 4;
    static_assert(kWarps <= pd_warps_most(D, NT), "parts of a block");
    static_assert(kMerge <= kRing, "the merge buffer reuses the ring");
    static_assert(kSmem <= 226 * 1024, "shared memory per block");
};

struct PdParams {
    const __nv_bfloat16* q;
    int64_t q_sb, q_sh;
    const uint8_t *kc, *vc;
    int64_t c_sp, c_sh, c_st;              // page, head, token strides in bytes
    const int32_t* table;
    int64_t table_stride;
    int width, num_pages, page_size;
    uint32_t page_mul, page_shift;         // key / page_size = (2 key * page_mul) >> 32 >> page_shift
    const int32_t* kv_len;
    __nv_bfloat16* o;
    float* lse;
    // Parts: slot (block * 2 + 0) * kWarps + w is that of the unit warp w ended,
    // slot (block * 2 + 1) * kWarps + w that of the warps from w on which are
    // inside one unit at their ends.
    float* part_o;                         // [blocks][2][kWarps][kHeads][D]
    float* part_lse;                       // [blocks][2][kWarps][kHeads], log2 units
    int2* split;                           // [B][units]: first and last warp, or (-1, -1)
    int B, H, H_kv, G, hblk;               // hblk: head blocks of a K/V head
    float scale_log2, o_mul;
};

__device__ __forceinline__ void ldsm4(uint32_t addr, uint32_t (&r)[4]) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr)
                 : "memory");
}
__device__ __forceinline__ void ldsm4_t(uint32_t addr, uint32_t (&r)[4]) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr)
                 : "memory");
}
__device__ __forceinline__ uint32_t transpose8x8(uint32_t a) {
    uint32_t d;
    asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(d) : "r"(a));
    return d;
}
// D += A B, 16 x 8 x 16; E 2: bf16 operands, E 1: f16.
template <int E>
__device__ __forceinline__ void mma16816(float (&c)[4], const uint32_t (&a)[4], uint32_t b0,
                                         uint32_t b1) {
    if constexpr (E == 2)
        asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
            "{%8,%9}, {%0,%1,%2,%3};"
            : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
            : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
    else
        asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
            "{%8,%9}, {%0,%1,%2,%3};"
            : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
            : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
// Four e4m3 codes to two f16 pairs, exactly: bytes 0 and 1, bytes 2 and 3.
__device__ __forceinline__ void widen_e4m3(uint32_t v, uint32_t& lo, uint32_t& hi) {
    asm("{\n\t.reg .b16 a, b;\n\tmov.b32 {a, b}, %2;\n\t"
        "cvt.rn.f16x2.e4m3x2 %0, a;\n\tcvt.rn.f16x2.e4m3x2 %1, b;\n\t}"
        : "=r"(lo), "=r"(hi)
        : "r"(v));
}
__device__ __forceinline__ uint32_t pack_f16x2(float lo, float hi) {
    __half2 v = __floats2half2_rn(lo, hi);
    return *reinterpret_cast<uint32_t*>(&v);
}

// Byte of 16-byte chunk c of row r in a stage: rows of 128 bytes or more XOR
// the chunk with the row (mod 8), 64-byte rows with half the row (mod 4), so
// that the eight rows of an ldmatrix block fall into different banks.
template <int kRow>
__device__ __forceinline__ uint32_t stage_at(int r, int c) {
    if constexpr (kRow >= 128) return (uint32_t)(r * kRow + ((c ^ (r & 7)) << 4));
    else return (uint32_t)(r * kRow + ((c ^ ((r >> 1) & 3)) << 4));
}

// Steps of a sequence of length len: its keys' and one more without keys. That
// one stands for what a unit costs besides its keys (its query, its statistics
// and its row), about a step's time, so that ranges of many short units are
// not longer in time than others; and an empty sequence has a step to write
// its row from.
template <int kStep>
__device__ __forceinline__ int steps_of(int len) {
    return (len + kStep - 1) / kStep + 1;
}

// a / b for a >= 0, b > 0, by the 32-bit divider where both fit it.
__device__ __forceinline__ int64_t div_pos(int64_t a, int64_t b) {
    if (((uint64_t)(a | b) >> 32) == 0) return (int64_t)((uint32_t)a / (uint32_t)b);
    return a / b;
}

__device__ __forceinline__ int seq_len(const PdParams& p, int b) {
    const int64_t most = min((int64_t)p.width * p.page_size, (int64_t)INT32_MAX - 4096);
    return (int)max((int64_t)0, min((int64_t)p.kv_len[b], most));
}

// A place in the line of steps: all sequences for the first unit index (K/V
// head and block of query heads), then all for the next. Keys of the same
// tokens are then read for all heads at about the same time, which matters
// where a token's heads lie side by side (e4m3, 32 sequences of 8192 tokens in
// token-major pages: 104 us with each sequence's heads in turn, 100 so). The
// next sequence's length is fetched one sequence ahead.
struct PdCursor {
    int b, unit, step, n, len, next_len;
};

__device__ __forceinline__ int pd_peek(const PdParams& p, int b) {
    return seq_len(p, b + 1 < p.B ? b + 1 : 0);
}

template <int kStep>
__device__ __forceinline__ void pd_next(const PdParams& p, PdCursor& c) {
    if (++c.step < c.n) return;
    c.step = 0;
    if (++c.b == p.B) {
        c.b = 0;
        ++c.unit;
    }
    c.len = c.next_len;
    c.n = steps_of<kStep>(c.len);
    c.next_len = pd_peek(p, c.b);
}

template <int D, int E, int NT>
__global__ void __launch_bounds__(PdCfg<D, E, NT>::kThreads, 1)
    fa_paged_decode_kernel(const PdParams p) {
    using C = PdCfg<D, E, NT>;
    extern __shared__ __align__(128) uint8_t smem[];
    float* st_m = reinterpret_cast<float*>(smem + C::kRing);              // [warp][kHeads]
    float* st_l = st_m + C::kWarps * C::kHeads;
    float* st_lr = st_l + C::kWarps * C::kHeads;
    uint32_t* seen = reinterpret_cast<uint32_t*>(st_lr + C::kWarps * C::kHeads);
    __shared__ int64_t s_open[C::kWarps];
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int units = p.H_kv * p.hblk;
    pdl_launch_dependents();
    pdl_wait_prerequisites();

    // ---------------------------------------------------------- the range
    // Steps before each sequence, in every warp by itself (no block barrier
    // stands before the first load): a lane sums a slice of the sequences.
    const int slice = (p.B + 31) >> 5;
    const int b_lo = min(p.B, lane * slice), b_hi = min(p.B, b_lo + slice);
    int64_t mine = 0;
    int b_len = 0;                                           // of the slice's last sequence
    for (int b = b_lo; b < b_hi; ++b) {
        b_len = seq_len(p, b);
        mine += steps_of<C::kStep>(b_len);
    }
    int64_t incl = mine;
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
        const int64_t up = __shfl_up_sync(0xffffffffu, incl, off);
        if (lane >= off) incl += up;
    }
    const int64_t total = __shfl_sync(0xffffffffu, incl, 31), all = total * units;
    // With fewer steps than warps, the first `busy` warps take one step each,
    // spread over the blocks: a unit's parts then lie in consecutive workers,
    // none of them without work.
    const int per = (int)min((int64_t)C::kWarps, div_pos(all + kPdBlocks - 1, kPdBlocks));
    const int busy = (int)min(all, (int64_t)kPdBlocks * per);
    if ((int)blockIdx.x * per >= busy) return;               // uniform in the block
    const int worker = (int)blockIdx.x * per + warp;
    const bool works = warp < per && worker < busy;
    const int64_t quota = div_pos(all, busy), extra = all - quota * busy;
    const int64_t count = works ? quota + (worker < extra ? 1 : 0) : 0;
    const int64_t t_lo = worker * quota + min((int64_t)worker, extra);
    PdCursor cur{};
    if (works) {                                             // uniform in the warp
        cur.unit = (int)div_pos(t_lo, total);
        const int64_t want = t_lo - cur.unit * total;        // in steps of one unit a sequence
        int64_t at = incl - mine;
        const bool owner = at <= want && want < incl;        // one lane
        int b = b_lo, n = 1;
        if (owner) {
            if (slice > 1)
                for (;; ++b) {
                    b_len = seq_len(p, b);
                    if (want < at + steps_of<C::kStep>(b_len)) break;
                    at += steps_of<C::kStep>(b_len);
                }
            n = steps_of<C::kStep>(b_len);
        }
        const int who = __ffs(__ballot_sync(0xffffffffu, owner)) - 1;
        cur.b = __shfl_sync(0xffffffffu, b, who);
        cur.len = __shfl_sync(0xffffffffu, b_len, who);
        cur.n = __shfl_sync(0xffffffffu, n, who);
        cur.step = (int)(want - __shfl_sync(0xffffffffu, at, who));
        cur.next_len = pd_peek(p, cur.b);
    }

    // ---------------------------------------------------------- loading
    const uint32_t ring = smem_u32(smem) + (uint32_t)(warp * C::kStages * C::kStage);
    uint32_t* my_seen = seen + warp * C::kStages;
    PdCursor put = cur;
    int64_t put_i = 0;
    int64_t put_head = (put.unit / p.hblk) * p.c_sh;         // of the unit's K/V head
    constexpr uint32_t kLanesIn = C::kStep == 32 ? 0xffffffffu : 0xffffu;
    const int lane_key = lane & (C::kStep - 1);              // a lane looks up its key's page
    int entry = -1, slot_in_page = 0;
    auto lookup = [&]() {
        const int key = put.step * C::kStep + lane_key;
        const int pg = (int)(__umulhi(2u * (uint32_t)key, p.page_mul) >> p.page_shift);
        slot_in_page = key - pg * p.page_size;
        entry = -1;
        if (put_i < count && key < put.len) entry = p.table[put.b * p.table_stride + pg];
    };
    constexpr int kChunks = C::kRow / 16;                    // of a row
    constexpr int kRowsAt = 32 / kChunks;                    // rows of one warp-wide copy
    const int my_row = lane / kChunks, my_chunk = lane % kChunks;
    const int64_t v_off = p.vc - p.kc;
    const uint64_t once = policy_evict_first();              // keys and values are read once
    auto issue = [&](int slot) {
        if (put_i < count) {
            const bool ok = entry >= 0 && entry < p.num_pages;
            const int64_t off =
                ok ? entry * p.c_sp + put_head + slot_in_page * p.c_st : 0;
            const uint32_t kd = ring + (uint32_t)(slot * C::kStage), vd = kd + C::kStep * C::kRow;
            const uint32_t mask = __ballot_sync(0xffffffffu, ok) & kLanesIn;
            if (mask != 0) {
                const uint8_t* base = p.kc + my_chunk * 16;
#pragma unroll
                for (int i = 0; i < C::kStep / kRowsAt; ++i) {
                    const int r = i * kRowsAt + my_row;
                    const bool in = (mask >> r) & 1u;
                    const uint8_t* from = (in ? base : p.kc) + __shfl_sync(0xffffffffu, off, r);
                    const uint32_t at = stage_at<C::kRow>(r, my_chunk);
                    cp_async16(kd + at, from, in, once);
                    cp_async16(vd + at, from + v_off, in, once);
                }
            }
            if (lane == 0) my_seen[slot] = mask;
            ++put_i;
            const int was = put.unit;
            pd_next<C::kStep>(p, put);
            if (put.unit != was) put_head = (put.unit / p.hblk) * p.c_sh;
            lookup();
        }
        cp_async_commit();
    };
    // ---------------------------------------------------------- state
    uint32_t qf[D / 16][NT][2];
    float o[D / 16][NT][4];
    float m[NT][2], l[NT][2], lr[NT][2], sc[NT][2];
    const int qr = lane >> 2, qc = lane & 3;
    // The unit's queries as they lie in memory: requested before the last
    // unit's results are written, so that the two latencies overlap.
    auto load_q = [&]() {
        const int hkv = cur.unit / p.hblk, hb = cur.unit - hkv * p.hblk;
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
            const int g = hb * C::kHeads + nt * 8 + qr;      // head of the group
            const bool in = g < p.G;
            const __nv_bfloat16* src = p.q + cur.b * p.q_sb + (int64_t)(hkv * p.G + (in ? g : 0)) * p.q_sh;
#pragma unroll
            for (int kk = 0; kk < D / 16; ++kk) {
                if constexpr (E == 2) {
#pragma unroll
                    for (int j = 0; j < 2; ++j)
                        qf[kk][nt][j] = in ? *reinterpret_cast<const uint32_t*>(
                                                 src + kk * 16 + j * 8 + 2 * qc) : 0u;
                } else {                                     // 4 qc .. 4 qc + 3 of each 16,
                    const uint2 u = in ? *reinterpret_cast<const uint2*>(src + kk * 16 + 4 * qc)
                                       : make_uint2(0u, 0u); // as the keys' bytes come
                    qf[kk][nt][0] = u.x;
                    qf[kk][nt][1] = u.y;
                }
            }
        }
    };
    auto begin_unit = [&]() {
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
            sc[nt][0] = sc[nt][1] = p.scale_log2;
            if constexpr (E == 1) {
                // f16 q, scaled to a largest magnitude in [2^14, 2^15): both scales
                // stay normal numbers whatever the head's magnitude
                float amax = 0.f;
#pragma unroll
                for (int kk = 0; kk < D / 16; ++kk)
#pragma unroll
                    for (int j = 0; j < 2; ++j)
                        amax = fmaxf(amax, fmaxf(fabsf(__uint_as_float(qf[kk][nt][j] << 16)),
                                                 fabsf(__uint_as_float(qf[kk][nt][j] & 0xffff0000u))));
                amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 1));
                amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 2));
                int ex = (int)(__float_as_uint(amax) >> 23) - 127;
                ex = max(-112, min(127, ex));                // infinities stay infinite
                const float down = __uint_as_float((uint32_t)(127 + 14 - ex) << 23);
#pragma unroll
                for (int kk = 0; kk < D / 16; ++kk)
#pragma unroll
                    for (int j = 0; j < 2; ++j) {
                        const uint32_t w = qf[kk][nt][j];
                        qf[kk][nt][j] = pack_f16x2(__uint_as_float(w << 16) * down,
                                                   __uint_as_float(w & 0xffff0000u) * down);
                    }
#pragma unroll
                for (int j = 0; j < 2; ++j) {                // of this thread's two columns
                    const int e2 = __shfl_sync(0xffffffffu, ex, (2 * qc + j) * 4);
                    sc[nt][j] = p.scale_log2 * __uint_as_float((uint32_t)(127 - 14 + e2) << 23);
                }
            }
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                m[nt][j] = -INFINITY;
                l[nt][j] = lr[nt][j] = 0.f;
            }
#pragma unroll
            for (int mt = 0; mt < D / 16; ++mt)
#pragma unroll
                for (int j = 0; j < 4; ++j) o[mt][nt][j] = 0.f;
        }
    };
    bool from_start = cur.step == 0;                         // this warp has the unit's step 0
    lookup();
    if (works) load_q();
    for (int s = 0; s < C::kStages - 1; ++s) issue(s);
    if (works) begin_unit();

    // ---------------------------------------------------------- one step
    const int kr = lane & 15, kcol = lane >> 4;              // ldmatrix rows: K
    const int vg = lane >> 3, vi = lane & 7;                 // and V (transposed)
    auto compute = [&](int slot) {
        const uint32_t mask = my_seen[slot];
        if (mask == 0) return;
        const uint32_t kb = ring + (uint32_t)(slot * C::kStage), vb = kb + C::kStep * C::kRow;
        float x[C::kGroups][NT][4];
        bool move = false;
#pragma unroll
        for (int g = 0; g < C::kGroups; ++g) {
            float s[2][NT][4];                               // two chains of products
#pragma unroll
            for (int h = 0; h < 2; ++h)
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                    for (int j = 0; j < 4; ++j) s[h][nt][j] = 0.f;
            if constexpr (E == 2) {
#pragma unroll
                for (int kk = 0; kk < D / 16; ++kk) {
                    uint32_t a[4];
                    ldsm4(kb + stage_at<C::kRow>(g * 16 + kr, kk * 2 + kcol), a);
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt)
                        mma16816<E>(s[kk & 1][nt], a, qf[kk][nt][0], qf[kk][nt][1]);
                }
            } else {
#pragma unroll
                for (int k2 = 0; k2 < D / 32; ++k2) {
                    uint32_t r[4];
                    ldsm4(kb + stage_at<C::kRow>(g * 16 + kr, k2 * 2 + kcol), r);
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        uint32_t a[4];
                        widen_e4m3(r[2 * h], a[0], a[2]);
                        widen_e4m3(r[2 * h + 1], a[1], a[3]);
#pragma unroll
                        for (int nt = 0; nt < NT; ++nt)
                            mma16816<E>(s[h][nt], a, qf[2 * k2 + h][nt][0], qf[2 * k2 + h][nt][1]);
                    }
                }
            }
            const bool in0 = (mask >> (g * 16 + qr)) & 1u, in1 = (mask >> (g * 16 + qr + 8)) & 1u;
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const float v = (s[0][nt][j] + s[1][nt][j]) * sc[nt][j & 1];
                    x[g][nt][j] = (j < 2 ? in0 : in1) ? v : -INFINITY;
                    move |= x[g][nt][j] > m[nt][j & 1] + 8.f;
                }
        }
        if (__any_sync(0xffffffffu, move)) {
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    float t = fmaxf(x[0][nt][j], x[0][nt][j + 2]);
                    if constexpr (C::kGroups == 2)
                        t = fmaxf(t, fmaxf(x[C::kGroups - 1][nt][j], x[C::kGroups - 1][nt][j + 2]));
                    t = fmaxf(t, __shfl_xor_sync(0xffffffffu, t, 4));
                    t = fmaxf(t, __shfl_xor_sync(0xffffffffu, t, 8));
                    t = fmaxf(t, __shfl_xor_sync(0xffffffffu, t, 16));
                    const float mn = fmaxf(m[nt][j], t);
                    const float alpha = mn == -INFINITY ? 1.f : fast_exp2(m[nt][j] - mn);
                    m[nt][j] = mn;
                    l[nt][j] *= alpha;
                    if (E == 1) lr[nt][j] *= alpha;
#pragma unroll
                    for (int mt = 0; mt < D / 16; ++mt) {
                        o[mt][nt][j] *= alpha;
                        o[mt][nt][j + 2] *= alpha;
                    }
                }
        }
        uint32_t pb[C::kGroups][NT][2], pl[C::kGroups][NT][2];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
            const float m0 = (m[nt][0] == -INFINITY ? 0.f : m[nt][0]) - C::kLift;
            const float m1 = (m[nt][1] == -INFINITY ? 0.f : m[nt][1]) - C::kLift;
#pragma unroll
            for (int gh = 0; gh < 2 * C::kGroups; ++gh) {    // keys qr, then qr + 8, of a group
                const int g = gh >> 1, h = gh & 1;
                const float p0 = fast_exp2(x[g][nt][2 * h] - m0);
                const float p1 = fast_exp2(x[g][nt][2 * h + 1] - m1);
                l[nt][0] += p0;
                l[nt][1] += p1;
                uint32_t u;
                if constexpr (E == 2) {
                    u = pack_bf16x2(p0, p1);
                    pl[g][nt][h] = transpose8x8(
                        pack_bf16x2(p0 - __uint_as_float(u << 16),
                                    p1 - __uint_as_float(u & 0xffff0000u)));
                } else {
                    u = pack_f16x2(p0, p1);
                    const float2 f = __half22float2(*reinterpret_cast<__half2*>(&u));
                    lr[nt][0] += f.x;
                    lr[nt][1] += f.y;
                }
                pb[g][nt][h] = transpose8x8(u);
            }
        }
#pragma unroll
        for (int g = 0; g < C::kGroups; ++g) {
            if constexpr (E == 2) {
#pragma unroll
                for (int mt = 0; mt < D / 16; ++mt) {
                    uint32_t a[4];
                    ldsm4_t(vb + stage_at<C::kRow>(g * 16 + (vg >> 1) * 8 + vi, 2 * mt + (vg & 1)), a);
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt) {
                        mma16816<E>(o[mt][nt], a, pb[g][nt][0], pb[g][nt][1]);
                        mma16816<E>(o[mt][nt], a, pl[g][nt][0], pl[g][nt][1]);
                    }
                }
            } else {
                // a transposed 16-bit block gives, for head-dim pair 2 qr, 2 qr + 1
                // (bytes) and keys 2 qc, 2 qc + 1: rows qr and qr + 8 of the
                // product's A are head dims 2 qr and 2 qr + 1
#pragma unroll
                for (int m2 = 0; m2 < D / 32; ++m2) {
                    uint32_t r[4];
                    ldsm4_t(vb + stage_at<C::kRow>(g * 16 + (vg & 1) * 8 + vi, 2 * m2 + (vg >> 1)), r);
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        uint32_t a[4];
                        widen_e4m3(__byte_perm(r[2 * h], 0u, 0x3120), a[0], a[1]);
                        widen_e4m3(__byte_perm(r[2 * h + 1], 0u, 0x3120), a[2], a[3]);
#pragma unroll
                        for (int nt = 0; nt < NT; ++nt)
                            mma16816<E>(o[2 * m2 + h][nt], a, pb[g][nt][0], pb[g][nt][1]);
                    }
                }
            }
        }
    };

    // ---------------------------------------------------------- a unit's end in this warp
    auto add_lanes = [&]() {                                 // sums over the 8 lanes of a column
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int j = 0; j < 2; ++j)
#pragma unroll
                for (int off = 4; off < 32; off <<= 1) {
                    l[nt][j] += __shfl_xor_sync(0xffffffffu, l[nt][j], off);
                    if (E == 1) lr[nt][j] += __shfl_xor_sync(0xffffffffu, lr[nt][j], off);
                    else lr[nt][j] = l[nt][j];
                }
    };
    // log2-sum-exp of exact sum `sum` with reference m: -inf for no key at all
    auto lse2 = [](float sum, float ref) {
        return sum == 0.f ? -INFINITY : (ref == -INFINITY ? 0.f : ref) + (log2f(sum) - C::kLift);
    };
    // whole: the unit's row; otherwise this warp's part, into slot kind (0: the
    // unit ends here, 1: it goes on)
    auto finish = [&](int b, int unit, bool whole, int kind) {
        add_lanes();
        const int hkv = unit / p.hblk, hb = unit - hkv * p.hblk;
        if (whole) {
            if (lane == 0) p.split[(int64_t)b * units + unit] = make_int2(-1, -1);
            const int64_t row0 = (int64_t)b * p.H + hkv * p.G + hb * C::kHeads;
            const int heads = p.G - hb * C::kHeads;          // live ones of this block of heads
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
                float inv[2];
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    inv[j] = lr[nt][j] == 0.f ? 0.f : p.o_mul / lr[nt][j];   // no visible key: 0
                    const int h = nt * 8 + 2 * qc + j;
                    if (qr == 0 && h < heads)
                        p.lse[row0 + h] = lse2(l[nt][j], m[nt][j]) * 0.6931471805599453f;
                }
#pragma unroll
                for (int mt = 0; mt < D / 16; ++mt) {
                    const float(&f)[4] = o[mt][nt];
                    if constexpr (E == 2) {
                        // 8 x 8 blocks transposed: head qr, two neighbouring columns
#pragma unroll
                        for (int h8 = 0; h8 < 2; ++h8) {
                            const uint32_t u = transpose8x8(
                                pack_bf16x2(f[2 * h8] * inv[0], f[2 * h8 + 1] * inv[1]));
                            if (nt * 8 + qr < heads)
                                *reinterpret_cast<uint32_t*>(p.o + (row0 + nt * 8 + qr) * D +
                                                             mt * 16 + h8 * 8 + 2 * qc) = u;
                        }
                    } else {
#pragma unroll
                        for (int j = 0; j < 2; ++j)
                            if (nt * 8 + 2 * qc + j < heads)
                                *reinterpret_cast<uint32_t*>(
                                    p.o + (row0 + nt * 8 + 2 * qc + j) * D + mt * 16 + 2 * qr) =
                                    pack_bf16x2(f[j] * inv[j], f[j + 2] * inv[j]);
                    }
                }
            }
        } else {
            const int64_t row0 =
                ((int64_t)(blockIdx.x * 2 + kind) * C::kWarps + warp) * C::kHeads;
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    const int64_t row = row0 + nt * 8 + 2 * qc + j;
                    const float inv = lr[nt][j] == 0.f ? 0.f : p.o_mul / lr[nt][j];
                    if (qr == 0) p.part_lse[row] = lse2(l[nt][j], m[nt][j]);
#pragma unroll
                    for (int mt = 0; mt < D / 16; ++mt) {
                        float* dst = p.part_o + row * D + mt * 16;
                        if constexpr (E == 2) {
                            dst[qr] = o[mt][nt][j] * inv;
                            dst[qr + 8] = o[mt][nt][j + 2] * inv;
                        } else {
                            *reinterpret_cast<float2*>(dst + 2 * qr) =
                                make_float2(o[mt][nt][j] * inv, o[mt][nt][j + 2] * inv);
                        }
                    }
                }
        }
    };

    // ---------------------------------------------------------- the loop
    int get = 0, fill = C::kStages - 1;
    bool grouped = false;            // ends inside a unit that a neighbour is inside of, too
    for (int64_t i = 0; i < count; ++i) {
        cp_async_wait<C::kStages - 2>();
        __syncwarp();           // stage `get` is in, and every lane is done with stage `fill`
        issue(fill);
        compute(get);
        get = get + 1 == C::kStages ? 0 : get + 1;
        fill = fill + 1 == C::kStages ? 0 : fill + 1;
        const bool ends = cur.step + 1 == cur.n, more = i + 1 < count;
        if (!ends && more) {
            ++cur.step;
            continue;
        }
        const int b = cur.b, unit = cur.unit;
        if (!ends) {
            // The range ends inside the unit. The warp before it in the block
            // is inside it unless it starts here; the one after it is unless
            // it ends there.
            const int64_t last = t_lo + i + (cur.n - 1 - cur.step);      // the unit's last step
            const int64_t next_end = t_lo + count + quota + (worker + 1 < extra ? 1 : 0);
            grouped = (!from_start && warp > 0) || (last >= next_end && warp + 1 < per);
            if (lane == 0 && from_start) {                   // the warp that has the last step
                const int64_t wide = extra * (quota + 1);    // steps of the longer ranges
                const int end = (int)(last < wide ? div_pos(last, quota + 1)
                                                  : extra + div_pos(last - wide, quota));
                p.split[(int64_t)b * units + unit] =
                    make_int2((int)blockIdx.x * C::kWarps + warp,
                              end / per * C::kWarps + end % per);
            }
            if (grouped) break;
        }
        if (more) {
            pd_next<C::kStep>(p, cur);
            load_q();
        }
        finish(b, unit, ends && from_start, ends ? 0 : 1);
        from_start = true;
        if (more) begin_unit();
    }
    cp_async_wait<0>();

    // ---------------------------------------------------------- parts of groups
    if (grouped) {
        add_lanes();
        if (qr == 0) {
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    const int h = warp * C::kHeads + nt * 8 + 2 * qc + j;
                    st_m[h] = m[nt][j];
                    st_l[h] = l[nt][j];
                    st_lr[h] = lr[nt][j];
                }
        }
    }
    if (lane == 0) s_open[warp] = grouped ? (int64_t)cur.b * units + cur.unit : -1;
    if (!__syncthreads_or(grouped)) return;                  // rings are done with, too
    // Warps that follow one another inside one unit form a group; its common
    // reference is the largest of theirs.
    int first = warp, past = warp + 1;
    if (grouped) {
        while (first > 0 && s_open[first - 1] == s_open[warp]) --first;
        while (past < C::kWarps && s_open[past] == s_open[warp]) ++past;
        float* mine_o = reinterpret_cast<float*>(smem) + warp * C::kHeads * C::kPitch;
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                const int h = nt * 8 + 2 * qc + j;
                float ref = -INFINITY;
                for (int w = first; w < past; ++w) ref = fmaxf(ref, st_m[w * C::kHeads + h]);
                const float a = m[nt][j] == -INFINITY ? 0.f : fast_exp2(m[nt][j] - ref);
#pragma unroll
                for (int mt = 0; mt < D / 16; ++mt) {
                    float* row = mine_o + h * C::kPitch + mt * 16;
                    if constexpr (E == 2) {
                        row[qr] = o[mt][nt][j] * a;
                        row[qr + 8] = o[mt][nt][j + 2] * a;
                    } else {
                        *reinterpret_cast<float2*>(row + 2 * qr) =
                            make_float2(o[mt][nt][j] * a, o[mt][nt][j + 2] * a);
                    }
                }
            }
    }
    __syncthreads();
    for (int w0 = 0; w0 < C::kWarps;) {
        const int64_t unit = s_open[w0];
        int w1 = w0 + 1;
        while (w1 < C::kWarps && s_open[w1] == unit) ++w1;
        if (unit >= 0) {
            const int64_t row0 = ((int64_t)(blockIdx.x * 2 + 1) * C::kWarps + w0) * C::kHeads;
            for (int e = tid; e < C::kHeads * (D / 4); e += C::kThreads) {
                const int h = e / (D / 4), col = (e - h * (D / 4)) * 4;
                float ref = -INFINITY, sum = 0.f, exact = 0.f;
                for (int w = w0; w < w1; ++w) ref = fmaxf(ref, st_m[w * C::kHeads + h]);
                float4 t = make_float4(0.f, 0.f, 0.f, 0.f);
                for (int w = w0; w < w1; ++w) {
                    const int sh = w * C::kHeads + h;
                    // a warp without a finite score has sums of 0, or NaN to pass on
                    const float a = st_m[sh] == -INFINITY ? 1.f : fast_exp2(st_m[sh] - ref);
                    sum += a * st_lr[sh];
                    exact += a * st_l[sh];
                    const float4 v = *reinterpret_cast<const float4*>(
                        reinterpret_cast<const float*>(smem) + sh * C::kPitch + col);
                    t.x += v.x;
                    t.y += v.y;
                    t.z += v.z;
                    t.w += v.w;
                }
                const float inv = sum == 0.f ? 0.f : p.o_mul / sum;
                *reinterpret_cast<float4*>(p.part_o + (row0 + h) * D + col) =
                    make_float4(t.x * inv, t.y * inv, t.z * inv, t.w * inv);
                if (col == 0) p.part_lse[row0 + h] = lse2(exact, ref);
            }
        }
        w0 = w1;
    }
}

// Joins the parts of the units that more than one warp worked on. Parts in the
// order of the keys: one of each block that the unit does not end in, one of
// the block that it ends in unless it ends in the first warp inside it there,
// and the last. It is all latency, so a row (sequence, query head) has kAt
// parts loaded side by side, D / 4 lanes (a float4 each) a part, and their
// loads do not wait for the log-sum-exps. kAt = 8, a block a row, where units
// are few and have many parts (up to one a block: with one warp a row, parts
// one after another, the join took 8 us of the 95 of a 131072-key sequence;
// so, 3 us); kAt = 1, rows side by side in a block, from kPdJoinUnits units on,
// which have at most four parts on average (256 sequences of 20 to 300 tokens,
// 8 K/V heads: 36 us in all, with kAt = 8 49; one sequence of 131072 tokens, 8
// units: 89, with kAt = 1 91; 8 units of 16 heads, 32768 keys: 30 and 35).
constexpr int kPdJoinUnits = 64;

template <int D, int kAt>
struct PdJoinCfg {
    static constexpr int kLanes = D / 4;                     // of a part
    static constexpr int kRows = kAt == 1 ? 128 / kLanes : 1;            // of a block
    static constexpr int kThreads = kLanes * kAt * kRows;
};

template <int D, int kAt>
__global__ void __launch_bounds__(PdJoinCfg<D, kAt>::kThreads)
    fa_paged_join(const PdParams p, int heads, int warps) {
    pdl_launch_dependents();
    pdl_wait_prerequisites();
    using C = PdJoinCfg<D, kAt>;
    constexpr int kLanes = C::kLanes;
    constexpr int kMost = 4;                                 // kept in registers a lane
    __shared__ float4 s_acc[C::kThreads];
    __shared__ float s_m[kAt], s_w[kAt];
    const int64_t row = (int64_t)blockIdx.x * C::kRows + (kAt == 1 ? (int)threadIdx.x / kLanes : 0);
    if (row >= (int64_t)p.B * p.H) return;
    const int b = (int)(row / p.H), h = (int)(row - (int64_t)b * p.H);
    const int hkv = h / p.G, g = h - hkv * p.G, hb = g / heads;
    const int2 sp = p.split[((int64_t)b * p.H_kv + hkv) * p.hblk + hb];
    if (sp.x < 0) return;
    const int hh = g - hb * heads;
    const int blk0 = sp.x / warps, w0 = sp.x - blk0 * warps;
    const int blk1 = sp.y / warps, w1 = sp.y - blk1 * warps;
    const int inside = blk1 - blk0 + (w1 > (blk0 == blk1 ? w0 : 0) ? 1 : 0);
    const int parts = inside + 1;
    auto at = [&](int i) {
        const int slot = i < inside ? ((blk0 + i) * 2 + 1) * warps + (i == 0 ? w0 : 0)
                                    : blk1 * 2 * warps + w1;
        return slot * heads + hh;
    };
    const int mine = kAt == 1 ? 0 : (int)threadIdx.x / kLanes, c = (int)threadIdx.x % kLanes;
    float m = -INFINITY, wsum = 0.f;
    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int i0 = mine; i0 < parts; i0 += kAt * kMost) {
        float ls[kMost];
        float4 v[kMost];
#pragma unroll
        for (int u = 0; u < kMost; ++u) {
            const int i = i0 + u * kAt;
            ls[u] = -INFINITY;
            if (i < parts) {
                const int r = at(i);
                ls[u] = p.part_lse[r];
                v[u] = *reinterpret_cast<const float4*>(p.part_o + (int64_t)r * D + c * 4);
            }
        }
        float mx = m;
#pragma unroll
        for (int u = 0; u < kMost; ++u) mx = fmaxf(mx, ls[u]);
        const float ref = mx == -INFINITY ? 0.f : mx;        // no finite part: zeros, or NaN
        const float keep = m == -INFINITY ? 1.f : exp2f(m - ref);
        wsum *= keep;
        acc.x *= keep;
        acc.y *= keep;
        acc.z *= keep;
        acc.w *= keep;
        m = mx;
#pragma unroll
        for (int u = 0; u < kMost; ++u) {
            if (ls[u] == -INFINITY) continue;
            const float w = exp2f(ls[u] - ref);
            wsum += w;
            acc.x = fmaf(w, v[u].x, acc.x);
            acc.y = fmaf(w, v[u].y, acc.y);
            acc.z = fmaf(w, v[u].z, acc.z);
            acc.w = fmaf(w, v[u].w, acc.w);
        }
    }
    float ref = m == -INFINITY ? 0.f : m, sum = wsum;
    float4 t = acc;
    if constexpr (kAt > 1) {
        s_acc[threadIdx.x] = acc;
        if (c == 0) {
            s_m[mine] = m;
            s_w[mine] = wsum;
        }
        __syncthreads();
        if (mine != 0) return;
#pragma unroll
        for (int k = 0; k < kAt; ++k) m = fmaxf(m, s_m[k]);
        ref = m == -INFINITY ? 0.f : m;
        t = make_float4(0.f, 0.f, 0.f, 0.f);
        sum = 0.f;
#pragma unroll
        for (int k = 0; k < kAt; ++k) {
            const float w = s_m[k] == -INFINITY ? 1.f : exp2f(s_m[k] - ref);   // 1: of 0, or NaN
            const float4 a = s_acc[k * kLanes + c];
            sum = fmaf(w, s_w[k], sum);
            t.x = fmaf(w, a.x, t.x);
            t.y = fmaf(w, a.y, t.y);
            t.z = fmaf(w, a.z, t.z);
            t.w = fmaf(w, a.w, t.w);
        }
    }
    const float inv = sum == 0.f ? 0.f : 1.f / sum;
    *reinterpret_cast<uint2*>(p.o + row * D + c * 4) =
        make_uint2(pack_bf16x2(t.x * inv, t.y * inv), pack_bf16x2(t.z * inv, t.w * inv));
    if (c == 0)
        p.lse[row] = sum == 0.f ? -INFINITY : (ref + log2f(sum)) * 0.6931471805599453f;
}

}  // namespace fa
