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
// cut into tiles of kKeys keys; the tiles of ALL units, laid end to end, are
// shared out evenly over the blocks (one an SM), so ragged lengths balance to
// one tile and a single long sequence fills the chip. A block's range covers
// the end of one unit, whole units, and the start of another: only the first
// and the last can be shared with other blocks, so a block leaves at most two
// partial results (normalised O and log-sum-exp in fp32), whatever the
// lengths, and fa_paged_join merges a unit's parts in block order.
//
// Inside a block every warp works alone on 16 keys of each tile, with a ring
// of kStages (K, V) stages of its own that its lanes fill with 16-byte
// cp.async: no block barrier in the loop. Each lane looks up the page of one
// key (table entries are fetched one tile ahead) and the row's offset goes
// round by shuffle, so any page size and page order costs the same; a key
// that is hidden or has no page is zero-filled and its score set to -inf,
// never read, so what lies there cannot reach the result. Rings continue
// across unit boundaries.
//
// Products (mma.sync m16n8k16, fp32 accumulators): S^T = K Q^T with the keys
// as rows and 8 query heads as columns, then O^T += V^T P^T. The C fragment of
// S^T transposed 8x8 block by block (movmatrix) is the B fragment of P^T, and
// a thread's two columns (heads) are the same in S^T and O^T, so running
// maxima, sums and rescaling never leave the thread. A head's reference
// maximum moves only when a score exceeds it by more than 8 (log2 units),
// found by one vote a tile; p is at most 2^8 and O / sum is exact whatever the
// reference. e4m3 keys and values are widened exactly to f16 (one conversion
// for two) and multiplied there; q, whose bf16 range f16 lacks, is scaled by a
// power of two per head first, which is exact but for elements 2^-31 below the
// head's largest. P is rounded to the values' type (bf16, or f16 for e4m3):
// at most half a step, 2^-8 (2^-11) relative, and O is divided by the sum of the rounded
// probabilities, lse by the exact one, as in the decoding tile over a
// contiguous cache.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cstdint>

#include "sm100_ptx.cuh"

namespace fa {

constexpr int kPdBlocks = 148;             // one block an SM
constexpr int kPdPitch = 132;              // floats of a head's row in the merge buffer

template <int D, int E, int NT>
struct PdCfg {
    static constexpr int kRow = D * E;                                    // bytes of a K or V row
    static constexpr int kStage = 2 * 16 * kRow;                          // K and V of 16 keys
    static constexpr int kWarps = kRow >= 512 ? 4 : 8;
    static constexpr int kThreads = 32 * kWarps;
    static constexpr int kKeys = 16 * kWarps;                             // keys of a tile
    static constexpr int kStages = kRow >= 256 ? 3 : kRow == 128 ? 6 : 8;
    static constexpr int kHeads = 8 * NT;
    static constexpr int kCols = D < 128 ? D : 128;                       // of one merge pass
    static constexpr int kRing = kWarps * kStages * kStage;
    static constexpr int kMerge = kWarps * 8 * kPdPitch * 4;
    static constexpr int kStat = 3 * kWarps * kHeads * 4;                 // m, l, lr
    static constexpr int kSmem = kRing + kMerge + kStat + kWarps * kStages * 4;
    static_assert(kSmem <= 227 * 1024, "shared memory per block");
};

struct PdParams {
    const __nv_bfloat16* q;
    int64_t q_sb, q_sh;
    const uint8_t *kc, *vc;
    int64_t c_sp, c_sh, c_st;              // page, head, token strides in bytes
    const int32_t* table;
    int64_t table_stride;
    int width, num_pages, page_size;
    const int32_t* kv_len;
    __nv_bfloat16* o;
    float* lse;
    float* part_o;                         // [blocks][2][kHeads][D]
    float* part_lse;                       // [blocks][2][kHeads], log2 units
    int2* split;                           // [B][units]: first and last block, or (-1, -1)
    int B, H, H_kv, G, hblk;               // hblk: head blocks of a K/V head
    float scale_log2, o_mul;
};

__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src, bool in) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst),
                 "l"(src), "r"(in ? 16 : 0)
                 : "memory");
}
__device__ __forceinline__ void cp_async_commit() {
    asm volatile("cp.async.commit_group;" ::: "memory");
}
template <int N>
__device__ __forceinline__ void cp_async_wait() {
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}
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

// Tiles of the sequence of length len (an empty one has one, so that its row
// is written).
template <int kKeys>
__device__ __forceinline__ int tiles_of(int len) {
    return len <= 0 ? 1 : (len + kKeys - 1) / kKeys;
}

__device__ __forceinline__ int seq_len(const PdParams& p, int b) {
    const int64_t most = min((int64_t)p.width * p.page_size, (int64_t)INT32_MAX - 4096);
    return (int)max((int64_t)0, min((int64_t)p.kv_len[b], most));
}

// A place in the line of tiles.
struct PdCursor {
    int b, unit, tile, n, len;
};

template <int kKeys>
__device__ __forceinline__ void pd_next(const PdParams& p, PdCursor& c, int units) {
    if (++c.tile < c.n) return;
    c.tile = 0;
    if (++c.unit < units) return;
    c.unit = 0;
    if (++c.b < p.B) {
        c.len = seq_len(p, c.b);
        c.n = tiles_of<kKeys>(c.len);
    }
}

template <int D, int E, int NT>
__global__ void __launch_bounds__(PdCfg<D, E, NT>::kThreads, 1)
    fa_paged_decode_kernel(const PdParams p) {
    using C = PdCfg<D, E, NT>;
    extern __shared__ __align__(128) uint8_t smem[];
    float* merge = reinterpret_cast<float*>(smem + C::kRing);             // [warp][8][kPdPitch]
    float* st_m = reinterpret_cast<float*>(smem + C::kRing + C::kMerge);  // [warp][kHeads]
    float* st_l = st_m + C::kWarps * C::kHeads;
    float* st_lr = st_l + C::kWarps * C::kHeads;
    uint32_t* seen = reinterpret_cast<uint32_t*>(st_lr + C::kWarps * C::kHeads);
    __shared__ int64_t s_scan[C::kWarps];
    __shared__ int64_t s_at;
    __shared__ int s_b;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int units = p.H_kv * p.hblk;
    pdl_launch_dependents();

    // ---------------------------------------------------------- the range
    // Tiles before each sequence: every thread sums a slice of them.
    const int slice = (p.B + C::kThreads - 1) / C::kThreads;
    const int b_lo = min(p.B, tid * slice), b_hi = min(p.B, b_lo + slice);
    int64_t mine = 0;
    for (int b = b_lo; b < b_hi; ++b) mine += tiles_of<C::kKeys>(seq_len(p, b));
    int64_t incl = mine;
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
        const int64_t up = __shfl_up_sync(0xffffffffu, incl, off);
        if (lane >= off) incl += up;
    }
    if (lane == 31) s_scan[warp] = incl;
    __syncthreads();
    int64_t before = incl - mine, total = 0;
#pragma unroll
    for (int w = 0; w < C::kWarps; ++w) {
        if (w < warp) before += s_scan[w];
        total += s_scan[w];
    }
    const int64_t all = total * units;
    // with fewer tiles than blocks, the first `busy` blocks take one each: a
    // unit's parts then lie in consecutive blocks, none of them empty
    const int64_t busy = min(all, (int64_t)kPdBlocks);
    if ((int64_t)blockIdx.x >= busy) return;                 // uniform in the block
    const int64_t t_lo = (int64_t)blockIdx.x * all / busy;
    const int64_t t_hi = (int64_t)(blockIdx.x + 1) * all / busy;
    const int64_t seq_tile = t_lo / units;                   // in tiles of one unit per sequence
    if (before <= seq_tile && seq_tile < before + mine) {    // one thread
        int b = b_lo;
        for (;; ++b) {
            const int n = tiles_of<C::kKeys>(seq_len(p, b));
            if (seq_tile < before + n) break;
            before += n;
        }
        s_b = b;
        s_at = before;
    }
    __syncthreads();
    PdCursor cur;
    cur.b = s_b;
    cur.len = seq_len(p, cur.b);
    cur.n = tiles_of<C::kKeys>(cur.len);
    int64_t unit_start;                                      // line index of the unit's tile 0
    {
        const int64_t in_seq = t_lo - s_at * units;
        cur.unit = (int)(in_seq / cur.n);
        cur.tile = (int)(in_seq - (int64_t)cur.unit * cur.n);
        unit_start = t_lo - cur.tile;
    }
    const int64_t count = t_hi - t_lo;

    // ---------------------------------------------------------- loading
    const uint32_t ring = smem_u32(smem) + (uint32_t)(warp * C::kStages * C::kStage);
    uint32_t* my_seen = seen + warp * C::kStages;
    PdCursor put = cur;
    int64_t put_i = 0;
    int entry = -1;                                          // page of this lane's next key
    auto lookup = [&]() {
        const int key = put.tile * C::kKeys + warp * 16 + (lane & 15);
        entry = -1;
        if (put_i < count && key < put.len)
            entry = p.table[put.b * p.table_stride + key / p.page_size];
    };
    constexpr int kChunks = C::kRow / 16;                    // of a row
    constexpr int kRowsAt = 32 / kChunks;                    // rows of one warp-wide copy
    auto issue = [&](int slot) {
        if (put_i < count) {
            const int key = put.tile * C::kKeys + warp * 16 + (lane & 15);
            const bool ok = entry >= 0 && entry < p.num_pages;
            const int64_t off = ok ? entry * p.c_sp + (put.unit / p.hblk) * p.c_sh +
                                         (key % p.page_size) * p.c_st
                                   : 0;
            const uint32_t mask = __ballot_sync(0xffffffffu, ok) & 0xffffu;
            if (lane == 0) my_seen[slot] = mask;
            if (mask != 0) {
                const uint32_t kd = ring + (uint32_t)(slot * C::kStage), vd = kd + 16 * C::kRow;
                const int c = lane % kChunks;
#pragma unroll
                for (int i = 0; i < 16 / kRowsAt; ++i) {
                    const int r = i * kRowsAt + lane / kChunks;
                    const int64_t ro = __shfl_sync(0xffffffffu, off, r) + c * 16;
                    const bool in = (mask >> r) & 1u;
                    const uint32_t at = stage_at<C::kRow>(r, c);
                    cp_async16(kd + at, p.kc + ro, in);
                    cp_async16(vd + at, p.vc + ro, in);
                }
            }
            ++put_i;
            pd_next<C::kKeys>(p, put, units);
            lookup();
        }
        cp_async_commit();
    };
    lookup();
    for (int s = 0; s < C::kStages - 1; ++s) issue(s);

    // ---------------------------------------------------------- state
    uint32_t qf[D / 16][NT][2];
    float o[D / 16][NT][4];
    float m[NT][2], l[NT][2], lr[NT][2], sc[NT][2];
    const int qr = lane >> 2, qc = lane & 3;
    auto begin_unit = [&]() {
        const int hkv = cur.unit / p.hblk, hb = cur.unit - hkv * p.hblk;
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
            const int g = hb * C::kHeads + nt * 8 + qr;      // head of the group
            const bool in = g < p.G;
            const __nv_bfloat16* src = p.q + cur.b * p.q_sb + (int64_t)(hkv * p.G + (in ? g : 0)) * p.q_sh;
            if constexpr (E == 2) {
#pragma unroll
                for (int kk = 0; kk < D / 16; ++kk)
#pragma unroll
                    for (int j = 0; j < 2; ++j)
                        qf[kk][nt][j] = in ? *reinterpret_cast<const uint32_t*>(
                                                 src + kk * 16 + j * 8 + 2 * qc) : 0u;
                sc[nt][0] = sc[nt][1] = p.scale_log2;
            } else {
                // f16 q, scaled to a largest magnitude in [1, 2): element order
                // 4 qc .. 4 qc + 3 of each 16, as the keys' bytes come
                float amax = 0.f;
#pragma unroll
                for (int kk = 0; kk < D / 16; ++kk) {
                    const uint2 u = in ? *reinterpret_cast<const uint2*>(src + kk * 16 + 4 * qc)
                                       : make_uint2(0u, 0u);
                    qf[kk][nt][0] = u.x;
                    qf[kk][nt][1] = u.y;
#pragma unroll
                    for (int j = 0; j < 2; ++j) {
                        const uint32_t w = j ? u.y : u.x;
                        amax = fmaxf(amax, fmaxf(fabsf(__uint_as_float(w << 16)),
                                                 fabsf(__uint_as_float(w & 0xffff0000u))));
                    }
                }
                amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 1));
                amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 2));
                int ex = (int)(__float_as_uint(amax) >> 23) - 127;
                if (amax == 0.f || ex > 127) ex = 0;         // zeros; infinities stay infinite
                ex = max(-100, min(100, ex));
                const float down = __uint_as_float((uint32_t)(127 - ex) << 23);
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
                    sc[nt][j] = p.scale_log2 * __uint_as_float((uint32_t)(127 + e2) << 23);
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
    bool from_start = cur.tile == 0;                         // this block has the unit's tile 0
    begin_unit();

    // ---------------------------------------------------------- one stage
    const int kr = lane & 15, kcol = lane >> 4;              // ldmatrix rows: K
    const int vg = lane >> 3, vi = lane & 7;                 // and V (transposed)
    auto compute = [&](int slot) {
        const uint32_t mask = my_seen[slot];
        if (mask == 0) return;
        const uint32_t kb = ring + (uint32_t)(slot * C::kStage), vb = kb + 16 * C::kRow;
        float s[2][NT][4];
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
                ldsm4(kb + stage_at<C::kRow>(kr, kk * 2 + kcol), a);
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
                    mma16816<E>(s[kk & 1][nt], a, qf[kk][nt][0], qf[kk][nt][1]);
            }
        } else {
#pragma unroll
            for (int k2 = 0; k2 < D / 32; ++k2) {
                uint32_t r[4];
                ldsm4(kb + stage_at<C::kRow>(kr, k2 * 2 + kcol), r);
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
        const bool in0 = (mask >> qr) & 1u, in1 = (mask >> (qr + 8)) & 1u;
        float x[NT][4];
        bool move = false;
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const float v = (s[0][nt][j] + s[1][nt][j]) * sc[nt][j & 1];
                x[nt][j] = (j < 2 ? in0 : in1) ? v : -INFINITY;
                move |= x[nt][j] > m[nt][j & 1] + 8.f;
            }
        if (__any_sync(0xffffffffu, move)) {
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    float t = fmaxf(x[nt][j], x[nt][j + 2]);
                    t = fmaxf(t, __shfl_xor_sync(0xffffffffu, t, 4));
                    t = fmaxf(t, __shfl_xor_sync(0xffffffffu, t, 8));
                    t = fmaxf(t, __shfl_xor_sync(0xffffffffu, t, 16));
                    const float mn = fmaxf(m[nt][j], t);
                    const float alpha = mn == -INFINITY ? 1.f : fast_exp2(m[nt][j] - mn);
                    m[nt][j] = mn;
                    l[nt][j] *= alpha;
                    lr[nt][j] *= alpha;
#pragma unroll
                    for (int mt = 0; mt < D / 16; ++mt) {
                        o[mt][nt][j] *= alpha;
                        o[mt][nt][j + 2] *= alpha;
                    }
                }
        }
        uint32_t pb[NT][2];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
            const float m0 = m[nt][0] == -INFINITY ? 0.f : m[nt][0];
            const float m1 = m[nt][1] == -INFINITY ? 0.f : m[nt][1];
#pragma unroll
            for (int h = 0; h < 2; ++h) {                    // keys qr, then qr + 8
                const float p0 = fast_exp2(x[nt][2 * h] - m0), p1 = fast_exp2(x[nt][2 * h + 1] - m1);
                l[nt][0] += p0;
                l[nt][1] += p1;
                uint32_t u;
                if constexpr (E == 2) {
                    u = pack_bf16x2(p0, p1);
                    lr[nt][0] = add_bf16_lo(u, lr[nt][0]);
                    lr[nt][1] = add_bf16_hi(u, lr[nt][1]);
                } else {
                    u = pack_f16x2(p0, p1);
                    const float2 f = __half22float2(*reinterpret_cast<__half2*>(&u));
                    lr[nt][0] += f.x;
                    lr[nt][1] += f.y;
                }
                pb[nt][h] = transpose8x8(u);
            }
        }
        if constexpr (E == 2) {
#pragma unroll
            for (int mt = 0; mt < D / 16; ++mt) {
                uint32_t a[4];
                ldsm4_t(vb + stage_at<C::kRow>((vg >> 1) * 8 + vi, 2 * mt + (vg & 1)), a);
#pragma unroll
                for (int nt = 0; nt < NT; ++nt) mma16816<E>(o[mt][nt], a, pb[nt][0], pb[nt][1]);
            }
        } else {
            // a transposed 16-bit block gives, for head-dim pair 2 qr, 2 qr + 1
            // (bytes) and keys 2 qc, 2 qc + 1: rows qr and qr + 8 of the
            // product's A are head dims 2 qr and 2 qr + 1
#pragma unroll
            for (int m2 = 0; m2 < D / 32; ++m2) {
                uint32_t r[4];
                ldsm4_t(vb + stage_at<C::kRow>((vg & 1) * 8 + vi, 2 * m2 + (vg >> 1)), r);
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    uint32_t a[4];
                    widen_e4m3(__byte_perm(r[2 * h], 0u, 0x3120), a[0], a[1]);
                    widen_e4m3(__byte_perm(r[2 * h + 1], 0u, 0x3120), a[2], a[3]);
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt)
                        mma16816<E>(o[2 * m2 + h][nt], a, pb[nt][0], pb[nt][1]);
                }
            }
        }
    };

    // ---------------------------------------------------------- end of a unit's part
    auto end_unit = [&](bool to_end, int64_t line) {
        // per-warp statistics, then the common reference of the block
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int j = 0; j < 2; ++j) {
#pragma unroll
                for (int off = 4; off < 32; off <<= 1) {
                    l[nt][j] += __shfl_xor_sync(0xffffffffu, l[nt][j], off);
                    lr[nt][j] += __shfl_xor_sync(0xffffffffu, lr[nt][j], off);
                }
                if (qr == 0) {
                    const int h = warp * C::kHeads + nt * 8 + 2 * qc + j;
                    st_m[h] = m[nt][j];
                    st_l[h] = l[nt][j];
                    st_lr[h] = lr[nt][j];
                }
            }
        __syncthreads();
        const bool whole = from_start && to_end;
        const int hkv = cur.unit / p.hblk, hb = cur.unit - hkv * p.hblk;
        const int64_t slot = (int64_t)blockIdx.x * 2 + (from_start ? 1 : 0);
        if (tid == 0 && from_start) {
            int2 sp = make_int2(-1, -1);
            if (!to_end) {
                const int64_t last = line + (cur.n - 1 - cur.tile);       // the unit's last tile
                sp = make_int2((int)blockIdx.x, (int)(((last + 1) * busy - 1) / all));
            }
            p.split[(int64_t)cur.b * units + cur.unit] = sp;
        }
        auto reference = [&](int h) {
            float r = -INFINITY;
#pragma unroll
            for (int w = 0; w < C::kWarps; ++w) r = fmaxf(r, st_m[w * C::kHeads + h]);
            return r;
        };
        auto weighted = [&](const float* st, int h, float ref) {
            float t = 0.f;
#pragma unroll
            for (int w = 0; w < C::kWarps; ++w) {
                const float mw = st_m[w * C::kHeads + h];
                // a warp without a finite score has sums of 0, or NaN to pass on
                t += (mw == -INFINITY ? 1.f : fast_exp2(mw - ref)) * st[w * C::kHeads + h];
            }
            return t;
        };
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
            float a[2];
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                const float ref = reference(nt * 8 + 2 * qc + j);
                a[j] = m[nt][j] == -INFINITY ? 0.f : fast_exp2(m[nt][j] - ref);
            }
#pragma unroll
            for (int d0 = 0; d0 < D; d0 += C::kCols) {
                float* mine_m = merge + warp * 8 * kPdPitch;
#pragma unroll
                for (int t = 0; t < C::kCols / 16; ++t) {
                    const int mt = d0 / 16 + t;
#pragma unroll
                    for (int j = 0; j < 2; ++j) {
                        float* row = mine_m + (2 * qc + j) * kPdPitch + t * 16;
                        if constexpr (E == 2) {
                            row[qr] = o[mt][nt][j] * a[j];
                            row[qr + 8] = o[mt][nt][j + 2] * a[j];
                        } else {
                            *reinterpret_cast<float2*>(row + 2 * qr) =
                                make_float2(o[mt][nt][j] * a[j], o[mt][nt][j + 2] * a[j]);
                        }
                    }
                }
                __syncthreads();
                for (int e = tid; e < 8 * C::kCols / 4; e += C::kThreads) {
                    const int hh = e / (C::kCols / 4), col = (e - hh * (C::kCols / 4)) * 4;
                    const int h = nt * 8 + hh, g = hb * C::kHeads + h;
                    if (g >= p.G) continue;
                    float4 t = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
                    for (int w = 0; w < C::kWarps; ++w) {
                        const float4 v = *reinterpret_cast<const float4*>(
                            merge + (w * 8 + hh) * kPdPitch + col);
                        t.x += v.x;
                        t.y += v.y;
                        t.z += v.z;
                        t.w += v.w;
                    }
                    const float ref = reference(h);
                    const float sum = weighted(st_lr, h, ref);
                    const float inv = sum == 0.f ? 0.f : p.o_mul / sum;   // no visible key: 0
                    t.x *= inv;
                    t.y *= inv;
                    t.z *= inv;
                    t.w *= inv;
                    const bool stat = d0 == 0 && col == 0;
                    float ls = -INFINITY;
                    if (stat) {
                        const float exact = weighted(st_l, h, ref);
                        if (exact != 0.f) ls = (ref == -INFINITY ? 0.f : ref) + log2f(exact);
                    }
                    if (whole) {
                        const int64_t row = (int64_t)cur.b * p.H + hkv * p.G + g;
                        *reinterpret_cast<uint2*>(p.o + row * D + d0 + col) =
                            make_uint2(pack_bf16x2(t.x, t.y), pack_bf16x2(t.z, t.w));
                        if (stat) p.lse[row] = ls * 0.6931471805599453f;
                    } else {
                        const int64_t row = slot * C::kHeads + h;
                        *reinterpret_cast<float4*>(p.part_o + row * D + d0 + col) = t;
                        if (stat) p.part_lse[row] = ls;
                    }
                }
                __syncthreads();                             // the buffer is free again
            }
        }
    };

    // ---------------------------------------------------------- the loop
    int get = 0, fill = C::kStages - 1;
    for (int64_t i = 0; i < count; ++i) {
        cp_async_wait<C::kStages - 2>();
        __syncwarp();           // stage `get` is in, and every lane is done with stage `fill`
        issue(fill);
        compute(get);
        get = get + 1 == C::kStages ? 0 : get + 1;
        fill = fill + 1 == C::kStages ? 0 : fill + 1;
        const bool last_tile = cur.tile + 1 == cur.n;
        if (last_tile || i + 1 == count) {
            end_unit(last_tile, t_lo + i);
            from_start = true;
            if (i + 1 < count) {
                pd_next<C::kKeys>(p, cur, units);
                begin_unit();
            }
        } else {
            ++cur.tile;
        }
    }
    cp_async_wait<0>();
}

// Joins the parts of the units that more than one block worked on: one warp a
// row (sequence, query head), D / 32 columns a lane, parts in block order.
constexpr int kPdJoinWarps = 4;

template <int D>
__global__ void __launch_bounds__(32 * kPdJoinWarps)
    fa_paged_join(const PdParams p, int heads) {
    pdl_wait_prerequisites();
    constexpr int kPer = D / 32;
    const int64_t row = (int64_t)blockIdx.x * kPdJoinWarps + (threadIdx.x >> 5);
    const int lane = threadIdx.x & 31;
    if (row >= (int64_t)p.B * p.H) return;
    const int b = (int)(row / p.H), h = (int)(row - (int64_t)b * p.H);
    const int hkv = h / p.G, g = h - hkv * p.G, hb = g / heads;
    const int2 sp = p.split[((int64_t)b * p.H_kv + hkv) * p.hblk + hb];
    if (sp.x < 0) return;
    const int hh = g - hb * heads, parts = sp.y - sp.x + 1;
    // part i: block sp.x + i, whose first part of the two it is unless the
    // unit began there
    auto at = [&](int i) { return ((int64_t)(sp.x + i) * 2 + (i == 0 ? 1 : 0)) * heads + hh; };
    float mx = -INFINITY;
    for (int i = lane; i < parts; i += 32) mx = fmaxf(mx, p.part_lse[at(i)]);
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, off));
    float acc[kPer], wsum = 0.f;
#pragma unroll
    for (int c = 0; c < kPer; ++c) acc[c] = 0.f;
    if (mx == -INFINITY) mx = 0.f;                           // no finite part: zeros, or NaN
    for (int i0 = 0; i0 < parts; i0 += 32) {
        const float ls = i0 + lane < parts ? p.part_lse[at(i0 + lane)] : -INFINITY;
        const float wl = ls == -INFINITY ? 0.f : exp2f(ls - mx);
        wsum += wl;
        const int cnt = min(32, parts - i0);
#pragma unroll 4
        for (int i = 0; i < cnt; ++i) {
            const float w = __shfl_sync(0xffffffffu, wl, i);
            const float* src = p.part_o + at(i0 + i) * D + lane * kPer;
#pragma unroll
            for (int c = 0; c < kPer; c += 2) {
                const float2 v = *reinterpret_cast<const float2*>(src + c);
                acc[c] = fmaf(w, v.x, acc[c]);
                acc[c + 1] = fmaf(w, v.y, acc[c + 1]);
            }
        }
    }
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) wsum += __shfl_xor_sync(0xffffffffu, wsum, off);
    const float inv = wsum == 0.f ? 0.f : 1.f / wsum;
#pragma unroll
    for (int c = 0; c < kPer; c += 2)
        *reinterpret_cast<uint32_t*>(p.o + row * D + lane * kPer + c) =
            pack_bf16x2(acc[c] * inv, acc[c + 1] * inv);
    if (lane == 0)
        p.lse[row] = wsum == 0.f ? -INFINITY : (mx + log2f(wsum)) * 0.6931471805599453f;
}

}  // namespace fa
