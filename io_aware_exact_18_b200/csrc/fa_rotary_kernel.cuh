// Per-head norm and rotary position of queries and keys, and the append of
// keys and values to a paged cache, in one pass; and the backward pass.
//
// A row is one head of one token, d bf16 elements. Row x at position p:
//     y = x r w,  r = 1 / sqrt(mean x^2 + eps)             (or y = x)
//     a' = s (a cos t - b sin t),  b' = s (b cos t + a sin t),  t = p f_i
// over the pairs (a, b) of y. Both steps are linear in x once r is known, so
// with per-element coefficients A_e = w_e s cos t and B_e = -+ w_partner s sin t
//     out_e = r (A_e x_e + B_e x_partner),
// two multiply-adds an element whatever the norm. A and B depend on the token
// alone, not on the head.
//
// What bounds it: HBM, 2 bytes read and 2 written an element (backward with
// the norm: 4 and 2), and next to it the instructions that a 16-byte chunk
// takes. So a thread owns two chunks (8 elements each) of the rows of ONE
// token, keeps their A and B in registers and walks over the heads. In the
// half layout they are the two chunks whose elements pair up (rotary_dim is a
// multiple of 16, so whole chunks do), or two of those that are not turned;
// interleaved, pairs stay in a chunk and any two do. No element crosses lanes
// then, and fp32 is multiplied in pairs (2 to 5 % faster than one by one). With
// one chunk a thread, the partner's coming by shuffle and unpacked again, a chunk
// took 124 instructions where this takes 94. A row's d / 16 lanes lie in one
// warp, so the sum of squares is a shuffle reduction.
//
// Angles: f_i / 2 pi, taken in fp64 (off by 2^-55 turns for f up to 1), becomes a
// 64-bit fixed-point fraction of a turn, and its product with the position,
// modulo 2^64, the angle's fraction of a turn; whole turns fall off the top and
// the product adds no error. So the angle is off by the position times 2^-55
// turns, 2^-24 at the last 32-bit position (2^-25.1 found for base 10000) and
// within the rounding to fp32 for sincospi (2^-25 turns, 2e-7 rad) up to 2^30. fp32
// products would be off by 0.01 rad at position 10^5. A block's angles are
// computed once, cooperatively, into shared memory: a few sincospi a thread
// for all its heads.
#pragma once

#include <cuda_bf16.h>
#include <cstdint>

#include "cp_async.cuh"
#include "sm100_ptx.cuh"

namespace fa {

constexpr int kRotThreads = 128;
constexpr int kRotUnroll = 4;        // rows of a batch
constexpr int kRotBlocksPerSm = 4;
constexpr int kRotFill = 2 * 148;    // blocks of a launch, if the heads of a tile can be split

struct RotRows {                     // one [B, heads, N, d] view, strides in elements
    uint8_t* ptr;
    int64_t sb, sh, sn;
};

struct RotParams {
    RotRows q, k, v, qo, ko;         // v: append only; ko: dense output only
    const int32_t* pos;
    int64_t pos_sb, pos_sn;
    const double* freqs;
    const void *wq, *wk;             // null: ones
    int w32;
    int rot;
    float cs_scale, sin_sign, eps;
    int B, H, H_kv, N;
    int64_t tokens;                  // B * N
    int tt_shift;                    // log2 of the tokens of a tile
    int pair_shift;                  // log2 of rot / 2, rounded up
    int splits;                      // blocks that share a tile's heads (forward)
    // append
    uint8_t *kc, *vc;
    int64_t c_sp, c_sh, c_st;        // page, head, token strides in elements
    const int32_t* table;
    int64_t table_stride;
    const int32_t* seq;
    int num_seqs, width, num_pages, page_size;
    float k_inv, v_inv;              // 1 / descale
};

template <int D>
struct RotCfg {
    static constexpr int kLanes = D / 16;                    // lanes of a row, two chunks each
    static constexpr int kSlots = kRotThreads / kLanes;      // rows a block holds at once
    static constexpr int kTable = kSlots * D / 2;            // (cos, sin) of kSlots tokens
};

// Pairs of fp32 in one 64-bit register: sm_100 multiplies and adds them two at
// a time (each half rounded like the scalar instruction).
using f2 = uint64_t;
__device__ __forceinline__ f2 f2_make(float lo, float hi) {
    f2 r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(lo), "f"(hi));
    return r;
}
__device__ __forceinline__ float2 f2_get(f2 v) {
    float2 r;
    asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(v));
    return r;
}
__device__ __forceinline__ f2 f2_mul(f2 a, f2 b) {
    f2 r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
__device__ __forceinline__ f2 f2_fma(f2 a, f2 b, f2 c) {
    f2 r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
    return r;
}
__device__ __forceinline__ float f2_sum(f2 v) {
    const float2 t = f2_get(v);
    return t.x + t.y;
}

__device__ __forceinline__ f2 bf2(uint32_t v) {          // a bf16 pair, widened
    return f2_make(__uint_as_float(v << 16), __uint_as_float(v & 0xffff0000u));
}
__device__ __forceinline__ void unpack8(const uint4& u, f2 (&x)[4]) {
    x[0] = bf2(u.x);
    x[1] = bf2(u.y);
    x[2] = bf2(u.z);
    x[3] = bf2(u.w);
}
__device__ __forceinline__ uint32_t pack2(f2 v) {
    const float2 t = f2_get(v);
    return pack_bf16x2(t.x, t.y);
}
__device__ __forceinline__ uint4 pack8(const f2 (&x)[4]) {
    return make_uint4(pack2(x[0]), pack2(x[1]), pack2(x[2]), pack2(x[3]));
}

// Norm weights of the 8 elements of chunk c.
__device__ __forceinline__ void norm_weights(const void* w, int w32, int c, f2 (&x)[4]) {
    if (w == nullptr) {
#pragma unroll
        for (int j = 0; j < 4; ++j) x[j] = f2_make(1.f, 1.f);
    } else if (w32) {
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const float* src = static_cast<const float*>(w) + c * 8 + 2 * j;
            x[j] = f2_make(src[0], src[1]);
        }
    } else {
        const __nv_bfloat16* src = static_cast<const __nv_bfloat16*>(w) + c * 8;
#pragma unroll
        for (int j = 0; j < 4; ++j)
            x[j] = f2_make(__bfloat162float(src[2 * j]), __bfloat162float(src[2 * j + 1]));
    }
}

// Token `tok` of the batch, as (b, n). Tokens number less than 2^31.
struct RotToken {
    int64_t b, n;
};
__device__ __forceinline__ RotToken rot_token(const RotParams& p, int64_t tok) {
    const uint32_t b = (uint32_t)tok / (uint32_t)p.N;
    return RotToken{(int64_t)b, tok - (int64_t)b * p.N};
}

// A thread's pair among the angles, and its fraction of a turn a position.
struct RotPair {
    int i;                           // rot / 2 and more: none
    uint64_t frac;
};
__device__ __forceinline__ RotPair rot_pair(const RotParams& p, int tid) {
    RotPair r{tid & ((1 << p.pair_shift) - 1), 0};
    if (r.i < p.rot >> 1) {
        const double turn = p.freqs[r.i] * 0.15915494309189533577;
        r.frac = (uint64_t)((turn - floor(turn)) * 18446744073709551616.0);
    }
    return r;
}

// (s cos, s sin) of a tile's n tokens into shared memory. A thread stays with
// its pair and takes kRotAngles tokens at a time, whose chains (position,
// product, sincospi) then overlap. position(t) is token t's; all threads call
// it together.
constexpr int kRotAngles = 4;
template <class Position>
__device__ __forceinline__ void rotary_table(float2* cs, const RotParams& p, const RotPair& pair,
                                             int n, int tid, Position&& position) {
    const int half = p.rot >> 1, step = kRotThreads >> p.pair_shift, mine = tid >> p.pair_shift;
    for (int t = 0; t < n; t += step * kRotAngles) {
        int32_t pos[kRotAngles];
#pragma unroll
        for (int k = 0; k < kRotAngles; ++k) pos[k] = position(min(t + mine + k * step, n - 1));
        float c[kRotAngles], s[kRotAngles];
#pragma unroll
        for (int k = 0; k < kRotAngles; ++k) {
            // the upper half as a signed number: [-1/2, 1/2) turns times 2^32
            const int32_t part = (int32_t)(((uint64_t)(int64_t)pos[k] * pair.frac) >> 32);
            sincospif((float)part * 4.656612873077393e-10f, &s[k], &c[k]);   // 2 turns
        }
#pragma unroll
        for (int k = 0; k < kRotAngles; ++k)
            if (pair.i < half && t + mine + k * step < n)
                cs[(t + mine + k * step) * half + pair.i] =
                    make_float2(c[k] * p.cs_scale, s[k] * p.cs_scale * p.sin_sign);
    }
}

// A lane's two chunks, whether each is turned, and its first pair of the table.
// In one instruction a row's lanes touch neighbouring chunks wherever the layout
// leaves the choice: with a lane's two chunks side by side, each 32-byte sector
// is asked for twice, halves at a time (B4 H32 H_kv8 N4096 d128, interleaved:
// the backward pass, which reads past L1, takes 143 us for 95, the forward 58.7
// for 57.4).
struct LaneRole {
    int c0, c1;
    bool turned0, turned1;
    int pair0, pair1;
};

template <int kLanes, bool kInter>
__device__ __forceinline__ LaneRole lane_role(int l, int rot) {
    LaneRole r;
    if constexpr (kInter) {                                  // pairs stay in a chunk
        r.c0 = l;
        r.c1 = l + kLanes;
        r.turned0 = r.c0 < rot >> 3;
        r.turned1 = r.c1 < rot >> 3;
        r.pair0 = 4 * r.c0;
        r.pair1 = 4 * r.c1;
    } else {                                                 // a chunk and its partner
        const int both = rot >> 4;                           // such lanes
        r.turned0 = r.turned1 = l < both;
        r.c0 = r.turned0 ? l : l + both;
        r.c1 = r.c0 + (r.turned0 ? both : kLanes - both);
        r.pair0 = r.pair1 = 8 * l;
    }
    return r;
}

// Coefficients of the turned pairs: y0 = a0 x0 + b0 p0 and y1 = a1 x1 + b1 p1
// for a lane's chunks x0, x1 and their partners' elements p0, p1.
struct LaneAngles {
    f2 a0[4], b0[4], a1[4], b1[4];
};

template <bool kInter>
__device__ __forceinline__ void lane_angles(const float2* cs, const LaneRole& r, LaneAngles& t) {
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        t.a0[j] = t.a1[j] = f2_make(1.f, 1.f);
        t.b0[j] = t.b1[j] = f2_make(0.f, 0.f);
    }
    if constexpr (kInter) {                                  // one pair in two elements
        if (r.turned0) {
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const float2 u = cs[r.pair0 + j];
                t.a0[j] = f2_make(u.x, u.x);
                t.b0[j] = f2_make(-u.y, u.y);
            }
        }
        if (r.turned1) {
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const float2 v = cs[r.pair1 + j];
                t.a1[j] = f2_make(v.x, v.x);
                t.b1[j] = f2_make(-v.y, v.y);
            }
        }
    } else if (r.turned0) {                                  // two pairs, half of each
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const float4 u = *reinterpret_cast<const float4*>(cs + r.pair0 + 2 * j);
            t.a0[j] = t.a1[j] = f2_make(u.x, u.z);
            t.b0[j] = f2_make(-u.y, -u.w);
            t.b1[j] = f2_make(u.y, u.w);
        }
    }
}

// a x + b p for a lane's chunk x and its partners' elements p. In interleaved
// pairs p is x with its halves swapped, which costs as many moves as the
// products in pairs save: there they are taken one by one.
template <bool kInter>
__device__ __forceinline__ f2 turn2(f2 a, f2 x, f2 b, f2 p) {
    if constexpr (!kInter) return f2_fma(a, x, f2_mul(b, p));
    const float2 ca = f2_get(a), cb = f2_get(b), u = f2_get(x), v = f2_get(p);
    return f2_make(fmaf(ca.x, u.x, cb.x * v.x), fmaf(ca.y, u.y, cb.y * v.y));
}

// The partners' elements. Where part of the head is turned, chunks that are not
// get zeros, so that an infinity there is not multiplied by a zero coefficient.
// (The selects are 16 instructions a row. A branch around the products instead
// is slower here, 61.4 us for 60.5 in the normed case below: the rows of
// a batch are then computed one after another. The backward pass, which has one
// row at a time, gains 2 % from it.)
template <bool kInter>
__device__ __forceinline__ void lane_partners(const f2 (&x0)[4], const f2 (&x1)[4],
                                              bool zero0, bool zero1, f2 (&p0)[4], f2 (&p1)[4]) {
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        if constexpr (kInter) {
            const float2 u = f2_get(x0[j]), v = f2_get(x1[j]);
            p0[j] = f2_make(u.y, u.x);
            p1[j] = f2_make(v.y, v.x);
        } else {
            p0[j] = x1[j];
            p1[j] = x0[j];
        }
        if (zero0) p0[j] = 0ull;
        if (zero1) p1[j] = 0ull;
    }
}

template <int kLanes>
__device__ __forceinline__ float row_sum(float v) {
#pragma unroll
    for (int off = kLanes / 2; off > 0; off >>= 1) v += __shfl_xor_sync(0xffffffffu, v, off);
    return v;
}

enum RotStore { kDense = 0, kPageBf16 = 1, kPageE4m3 = 2 };

// Eight fp32 values as e4m3 codes.
__device__ __forceinline__ uint2 codes8(const f2 (&y)[4]) {
    const float2 a = f2_get(y[0]), b = f2_get(y[1]), d = f2_get(y[2]), e = f2_get(y[3]);
    return make_uint2(pack_e4m3x4(a.x, a.y, b.x, b.y), pack_e4m3x4(d.x, d.y, e.x, e.y));
}

// The coefficients times the norm's weights (the partners' for b) and `mul`.
template <int D, bool kNorm, bool kInter>
__device__ __forceinline__ void coefficients(const float2* cs, const LaneRole& role, const void* w,
                                             int w32, float mul, LaneAngles& t) {
    lane_angles<kInter>(cs, role, t);
    const f2 mm = f2_make(mul, mul);
    f2 w0[4], w1[4], v0[4], v1[4];
    if constexpr (kNorm) {
        norm_weights(w, w32, role.c0, w0);
        norm_weights(w, w32, role.c1, w1);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            w0[j] = f2_mul(w0[j], mm);
            w1[j] = f2_mul(w1[j], mm);
        }
    } else {
#pragma unroll
        for (int j = 0; j < 4; ++j) w0[j] = w1[j] = mm;
    }
    // (where nothing is turned b is zero, and stays so beside an infinite weight)
    lane_partners<kInter>(w0, w1, kNorm && !role.turned0, kNorm && !role.turned1, v0, v1);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        t.a0[j] = f2_mul(t.a0[j], w0[j]);
        t.b0[j] = f2_mul(t.b0[j], v0[j]);
        t.a1[j] = f2_mul(t.a1[j], w1[j]);
        t.b1[j] = f2_mul(t.b1[j], v1[j]);
    }
}

// Block (token tile, head split). Virtual heads: the H of q, the H_kv of k
// and, appending, the H_kv of v; a split takes an even share of them, and a
// thread goes through its own in batches of kRotUnroll rows (two chunks each)
// kept on the way in registers, the first batch while the angles are computed.
// What decides the speed is the bytes on the way: batches of two, three and
// four rows took 75, 67 and 61 us (B1 H32 H_kv8 N16384 d128 with the norm,
// 51 us at the copy rate; the same walk that only copies the rows, 59 us).
// Tried, and no faster: the work shared out evenly
// over one round of blocks (62 us; 1024 tiles over 592 places are two rounds
// for the work of 1.7), more splits (65 us with two: each computes the angles
// again), and rows fetched by cp.async up to eight ahead (63 us: the
// bookkeeping of single rows costs more instructions than the loads on the way
// give back).
template <int D, bool kNorm, bool kInter, int kStore>
__global__ void __launch_bounds__(kRotThreads, kRotBlocksPerSm) fa_qk_rotary_fwd(const RotParams p) {
    using C = RotCfg<D>;
    __shared__ __align__(16) float2 cs[C::kTable];
    pdl_launch_dependents();
    pdl_wait_prerequisites();
    const int tid = threadIdx.x;
    const int tt = 1 << p.tt_shift;
    const uint32_t tile = blockIdx.x / (uint32_t)p.splits;
    const int split = (int)(blockIdx.x - tile * p.splits);
    const int64_t tok0 = (int64_t)tile * tt;
    const int heads = p.H + p.H_kv + (kStore != kDense ? p.H_kv : 0);
    const int lo = (int)((int64_t)heads * split / p.splits);
    const int hi = (int)((int64_t)heads * (split + 1) / p.splits);
    const int slot = tid / C::kLanes;
    const int ts = slot & (tt - 1), h_off = slot >> p.tt_shift, h_step = C::kSlots >> p.tt_shift;
    const LaneRole role = lane_role<C::kLanes, kInter>(tid % C::kLanes, p.rot);
    const bool alone0 = p.rot < D && !role.turned0;          // no partners: multiplied by 1
    const bool alone1 = kInter ? p.rot < D && !role.turned1 : alone0;
    const bool live = tok0 + ts < p.tokens;
    const RotToken t0 = rot_token(p, tok0);
    RotToken at{t0.b, t0.n + ts};
    if (at.n >= p.N) at = rot_token(p, live ? tok0 + ts : 0);

    // A batch: heads h0 + i h_step + h_off, i < kRotUnroll, below end, of one
    // input (0 q, 1 k, 2 v). Past the last head the last is loaded again, and
    // past the last token the first: those rows are computed and not stored.
    auto load = [&](int input, int h0, int h_end, uint4 (&u)[kRotUnroll][2]) {
        const RotRows& r = input == 0 ? p.q : input == 1 ? p.k : p.v;
        const uint8_t* src = r.ptr + (at.b * r.sb + at.n * r.sn) * 2;
        const int64_t sh = r.sh * 2;
#pragma unroll
        for (int i = 0; i < kRotUnroll; ++i) {
            const uint8_t* row = src + min(h0 + i * h_step + h_off, h_end - 1) * sh;
            u[i][0] = *reinterpret_cast<const uint4*>(row + role.c0 * 16);
            u[i][1] = *reinterpret_cast<const uint4*>(row + role.c1 * 16);
        }
    };
    int input = lo < p.H ? 0 : lo < p.H + p.H_kv ? 1 : 2;
    int before = input == 0 ? 0 : input == 1 ? p.H : p.H + p.H_kv;        // virtual heads
    uint4 u[kRotUnroll][2];
    load(input, lo - before, min(hi - before, input == 0 ? p.H : p.H_kv), u);
    if (input < 2)
        rotary_table(cs, p, rot_pair(p, tid), (int)min((int64_t)tt, p.tokens - tok0), tid, [&](int t) {
            RotToken a{t0.b, t0.n + t};
            if (a.n >= p.N) a = rot_token(p, tok0 + t);
            return p.pos[a.b * p.pos_sb + a.n * p.pos_sn];
        });
    __syncthreads();

    bool write = live, stored = live;
    uint8_t *k_out = nullptr, *v_out = nullptr;
    int64_t out_sh = 0;
    constexpr int kElem = kStore == kPageE4m3 ? 1 : 2;
    if constexpr (kStore != kDense) {
        // the token's slot in the cache, every index checked
        int32_t pos = -1;
        if (live) pos = p.pos[at.b * p.pos_sb + at.n * p.pos_sn];
        write = pos >= 0;
        stored = false;
        if (write) {
            const int64_t row = p.seq != nullptr ? p.seq[at.b] : at.b;
            const int pg = pos / p.page_size;
            if (row >= 0 && row < p.num_seqs && pg < p.width) {
                const int page = p.table[row * p.table_stride + pg];
                if (page >= 0 && page < p.num_pages) {
                    stored = true;
                    const int64_t off = (page * p.c_sp + (pos - pg * p.page_size) * p.c_st) * kElem;
                    k_out = p.kc + off;
                    v_out = p.vc + off;
                }
            }
        }
        out_sh = p.c_sh * kElem;
    } else {
        k_out = p.ko.ptr + (at.b * p.ko.sb + at.n * p.ko.sn) * 2;
        out_sh = p.ko.sh * 2;
    }

    for (bool loaded = true; input < (kStore == kDense ? 2 : 3); ++input) {
        const int size = input == 0 ? p.H : p.H_kv;
        const int h_lo = max(lo - before, 0), h_hi = min(hi - before, size);
        before += size;
        if (h_lo >= h_hi) continue;
        LaneAngles t;
        if (input < 2)
            coefficients<D, kNorm, kInter>(cs + ts * (p.rot >> 1), role, input == 0 ? p.wq : p.wk,
                                           p.w32, kStore == kPageE4m3 && input == 1 ? p.k_inv : 1.f,
                                           t);
        const bool keep = input == 0 ? write : stored;
        const int64_t sh = input == 0 ? p.qo.sh * 2 : out_sh;
        uint8_t* row = (input == 0 ? p.qo.ptr + (at.b * p.qo.sb + at.n * p.qo.sn) * 2
                        : input == 1 ? k_out : v_out) + (h_lo + h_off) * sh;
        const bool codes = kStore == kPageE4m3 && input != 0;            // uniform
        for (int h0 = h_lo; h0 < h_hi; h0 += h_step * kRotUnroll) {
            if (!loaded) load(input, h0, h_hi, u);
            loaded = false;
#pragma unroll
            for (int i = 0; i < kRotUnroll; ++i) {
                if (h0 + i * h_step >= h_hi) break;          // uniform in the block
                const bool here = keep && h0 + i * h_step + h_off < h_hi;
                f2 x0[4], x1[4], y0[4], y1[4];
                unpack8(u[i][0], x0);
                unpack8(u[i][1], x1);
                if (kStore != kDense && input == 2) {
                    const f2 inv = f2_make(p.v_inv, p.v_inv);
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        y0[j] = f2_mul(inv, x0[j]);
                        y1[j] = f2_mul(inv, x1[j]);
                    }
                } else {
                    f2 p0[4], p1[4];
                    lane_partners<kInter>(x0, x1, alone0, alone1, p0, p1);
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        y0[j] = f2_fma(t.a0[j], x0[j], f2_mul(t.b0[j], p0[j]));
                        y1[j] = f2_fma(t.a1[j], x1[j], f2_mul(t.b1[j], p1[j]));
                    }
                    if constexpr (kNorm) {
                        f2 s2 = f2_mul(x0[0], x0[0]), s3 = f2_mul(x1[0], x1[0]);
#pragma unroll
                        for (int j = 1; j < 4; ++j) {
                            s2 = f2_fma(x0[j], x0[j], s2);
                            s3 = f2_fma(x1[j], x1[j], s3);
                        }
                        const float r = rsqrtf(
                            fmaf(row_sum<C::kLanes>(f2_sum(s2) + f2_sum(s3)), 1.f / D, p.eps));
                        const f2 rr = f2_make(r, r);
#pragma unroll
                        for (int j = 0; j < 4; ++j) {
                            y0[j] = f2_mul(y0[j], rr);
                            y1[j] = f2_mul(y1[j], rr);
                        }
                    }
                }
                if (here) {
                    if (codes) {
                        *reinterpret_cast<uint2*>(row + role.c0 * 8) = codes8(y0);
                        *reinterpret_cast<uint2*>(row + role.c1 * 8) = codes8(y1);
                    // Values, and what is not turned, pass through bit for bit. (One
                    // chain of branches: with the values' inside the other's, a prompt
                    // of 8192 into bf16 pages, normed, takes 38.5 us for 37.8.)
                    } else if (kStore != kDense && input == 2) {
                        *reinterpret_cast<uint4*>(row + role.c0 * 16) = u[i][0];
                        *reinterpret_cast<uint4*>(row + role.c1 * 16) = u[i][1];
                    } else {
                        *reinterpret_cast<uint4*>(row + role.c0 * 16) =
                            !kNorm && alone0 ? u[i][0] : pack8(y0);
                        *reinterpret_cast<uint4*>(row + role.c1 * 16) =
                            !kNorm && alone1 ? u[i][1] : pack8(y1);
                    }
                }
                row += h_step * sh;
            }
        }
    }
}

// ---------------------------------------------------------------- backward
// With g the output gradient turned back (the rotation's transpose, times s)
// and r as in the forward:
//     dw_e  += g_e n_e,   dx_e = r (g_e w_e - n_e mean(g w n)),   n = x r.
// x is read again (the forward keeps nothing), both row sums are reduced in
// the same shuffles, and dw is kept in registers over everything a thread
// sees: its chunks are fixed. Blocks [0, q_blocks) have q's rows, the others
// k's, kRotBwdBlocks at most in all (three an SM; four, with the weights read
// from shared memory to make room, take 40.3 us for 37.5 at B2 H16 N4096 d128
// and the same at B4 H32 H_kv8). dw leaves as that many partial rows, which
// fa_rotary_dw adds in a fixed order: no atomics.
// A side's work is its token tiles times its heads, laid end to end in steps of
// the heads that a block takes at once and shared out evenly. A thread has
// kRotBwdDepth - 1 rows of g and x under way by cp.async into slots of its own
// in shared memory, across tiles; no other thread reads them, so no barrier is
// needed but around the angles. (With two rows in registers instead 52 us for
// 41 at B2 H16 N4096 d128, and 123 for 103 at B4 H32 H_kv8.) The next tile's
// positions are loaded a tile ahead: with their wait in the way it took 41 us
// for 38, and 103 for 95.
constexpr int kRotBwdBlocks = 3 * 148;
constexpr int kRotBwdDepth = 5;

struct RotBwdSide {                  // q's or k's
    RotRows g, x, out;               // output gradient, forward input, gradient
    const void* w;
    int heads;
    uint32_t per_tile;               // steps of a tile's heads
    int64_t steps;                   // of all tiles
};

struct RotBwdParams {
    RotParams f;                     // tokens, positions, frequencies
    RotBwdSide side[2];
    int q_blocks;
    float* part;                     // [blocks][D]
};

// A place in the line of steps: token tile and step within it.
struct RotCursor {
    uint32_t tile, s;
    __device__ __forceinline__ bool next(uint32_t per_tile) {            // true: a new tile
        if (++s < per_tile) return false;
        s = 0;
        ++tile;
        return true;
    }
};

template <int D, bool kInter>
__global__ void __launch_bounds__(kRotThreads, kRotBwdBlocks / 148)
    fa_qk_rotary_bwd_norm(const RotBwdParams bp) {
    using C = RotCfg<D>;
    const RotParams& p = bp.f;
    __shared__ __align__(16) uint4 ring[kRotBwdDepth][4][kRotThreads];   // g, g, x, x
    __shared__ __align__(16) float2 cs[C::kTable];           // then the dw reduction, 8 KB both
    static_assert(C::kTable * 2 == C::kSlots * D, "the reduction reuses the table");
    pdl_launch_dependents();
    pdl_wait_prerequisites();
    const int tid = threadIdx.x;
    const int tt = 1 << p.tt_shift;
    const int slot = tid / C::kLanes;
    const int ts = slot & (tt - 1), h_off = slot >> p.tt_shift, h_step = C::kSlots >> p.tt_shift;
    const LaneRole role = lane_role<C::kLanes, kInter>(tid % C::kLanes, p.rot);
    const bool alone0 = p.rot < D && !role.turned0;          // as in the forward
    const bool alone1 = p.rot < D && !role.turned1;
    const bool for_k = (int)blockIdx.x >= bp.q_blocks;
    const RotBwdSide& sd = bp.side[for_k ? 1 : 0];
    const int64_t blk = blockIdx.x - (for_k ? bp.q_blocks : 0);
    const int64_t blks = for_k ? gridDim.x - bp.q_blocks : bp.q_blocks;
    const uint32_t first = (uint32_t)(blk * sd.steps / blks);
    const int count = (int)((uint32_t)((blk + 1) * sd.steps / blks) - first);
    f2 w0[4], w1[4], dw0[4], dw1[4];
    norm_weights(sd.w, p.w32, role.c0, w0);
    norm_weights(sd.w, p.w32, role.c1, w1);
#pragma unroll
    for (int j = 0; j < 4; ++j) dw0[j] = dw1[j] = f2_make(0.f, 0.f);

    // past a tile's last token the batch's first stands in, unused
    auto token_at = [&](uint32_t tile, int t) {
        const int64_t tok = ((int64_t)tile << p.tt_shift) + t;
        return rot_token(p, tok < p.tokens ? tok : 0);
    };
    // Every warp holds its tile's positions, lane t that of token t (a tile has
    // kSlots tokens at most), loaded while it works on the tile before.
    static_assert(C::kSlots <= 32);
    auto position_of = [&](uint32_t tile) {
        const RotToken at = token_at(tile, tid & (tt - 1));
        return p.pos[at.b * p.pos_sb + at.n * p.pos_sn];
    };
    RotCursor put{first / sd.per_tile, first % sd.per_tile};
    RotCursor get = put;
    int put_i = 0;
    const uint8_t *g_in = nullptr, *x_in = nullptr;
    auto enter = [&]() {
        const RotToken at = token_at(put.tile, ts);
        g_in = sd.g.ptr + (at.b * sd.g.sb + at.n * sd.g.sn) * 2;
        x_in = sd.x.ptr + (at.b * sd.x.sb + at.n * sd.x.sn) * 2;
    };
    const RotPair pair = rot_pair(p, tid);
    int32_t position = 0;
    if (count > 0) {
        position = position_of(get.tile);
        enter();
    }
    auto issue = [&](int at_slot) {
        if (put_i < count) {
            const int h = min((int)put.s * h_step + h_off, sd.heads - 1);
            const uint8_t *gr = g_in + h * sd.g.sh * 2, *xr = x_in + h * sd.x.sh * 2;
            cp_async16(smem_u32(&ring[at_slot][0][tid]), gr + role.c0 * 16, true);
            cp_async16(smem_u32(&ring[at_slot][1][tid]), gr + role.c1 * 16, true);
            cp_async16(smem_u32(&ring[at_slot][2][tid]), xr + role.c0 * 16, true);
            cp_async16(smem_u32(&ring[at_slot][3][tid]), xr + role.c1 * 16, true);
            ++put_i;
            if (put.next(sd.per_tile) && put_i < count) enter();
        }
        cp_async_commit();
    };
    for (int i = 0; i < kRotBwdDepth - 1; ++i) issue(i);

    bool fresh = true, live = false;
    LaneAngles t;
    uint8_t* out = nullptr;
    for (int i = 0, from = 0; i < count; ++i) {
        if (fresh) {
            const RotToken at = token_at(get.tile, ts);
            const int64_t tok0 = (int64_t)get.tile << p.tt_shift;
            live = tok0 + ts < p.tokens;
            out = sd.out.ptr + (at.b * sd.out.sb + at.n * sd.out.sn) * 2;
            if (i > 0) __syncthreads();                      // the last tile's angles are read
            rotary_table(cs, p, pair, (int)min((int64_t)tt, p.tokens - tok0), tid,
                         [&](int t) { return __shfl_sync(0xffffffffu, position, t); });
            __syncthreads();
            position = position_of(get.tile + 1);
            lane_angles<kInter>(cs + ts * (p.rot >> 1), role, t);
        }
        issue(from == 0 ? kRotBwdDepth - 1 : from - 1);      // where the row before this lay
        const int h = (int)get.s * h_step + h_off;
        cp_async_wait<kRotBwdDepth - 1>();
        {
            f2 x0[4], x1[4], g0[4], g1[4];
            unpack8(ring[from][0][tid], g0);
            unpack8(ring[from][1][tid], g1);
            unpack8(ring[from][2][tid], x0);
            unpack8(ring[from][3][tid], x1);
            f2 s2 = 0ull, s3 = 0ull, d2 = 0ull, d3 = 0ull;
            f2 y0[4], y1[4];                                 // g w, then dx
            f2 p0[4], p1[4];
            lane_partners<kInter>(g0, g1, false, false, p0, p1);
            if (!alone0) {
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    g0[j] = turn2<kInter>(t.a0[j], g0[j], t.b0[j], p0[j]);
                    if (!kInter) g1[j] = turn2<kInter>(t.a1[j], g1[j], t.b1[j], p1[j]);
                }
            }
            if (kInter && !alone1) {
#pragma unroll
                for (int j = 0; j < 4; ++j) g1[j] = turn2<kInter>(t.a1[j], g1[j], t.b1[j], p1[j]);
            }
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                y0[j] = f2_mul(g0[j], w0[j]);
                y1[j] = f2_mul(g1[j], w1[j]);
                s2 = f2_fma(x0[j], x0[j], s2);
                s3 = f2_fma(x1[j], x1[j], s3);
                d2 = f2_fma(y0[j], x0[j], d2);
                d3 = f2_fma(y1[j], x1[j], d3);
            }
            float ss = f2_sum(s2) + f2_sum(s3), dot = f2_sum(d2) + f2_sum(d3);
#pragma unroll
            for (int off = C::kLanes / 2; off > 0; off >>= 1) {
                ss += __shfl_xor_sync(0xffffffffu, ss, off);
                dot += __shfl_xor_sync(0xffffffffu, dot, off);
            }
            const float r = rsqrtf(fmaf(ss, 1.f / D, p.eps));
            // mean(g w n), then r: each of the size of what it stands for, where r^3
            // would leave fp32's normal numbers for rows of rms 2^42 or 2^-43
            const float k = -(r * dot * (1.f / D)) * r;
            if (live && h < sd.heads) {
                const f2 rr = f2_make(r, r), kk = f2_make(k, k);
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const f2 n0 = f2_mul(x0[j], rr), n1 = f2_mul(x1[j], rr);
                    dw0[j] = f2_fma(g0[j], n0, dw0[j]);
                    dw1[j] = f2_fma(g1[j], n1, dw1[j]);
                    y0[j] = f2_fma(y0[j], rr, f2_mul(n0, kk));
                    y1[j] = f2_fma(y1[j], rr, f2_mul(n1, kk));
                }
                uint8_t* row = out + h * sd.out.sh * 2;
                *reinterpret_cast<uint4*>(row + role.c0 * 16) = pack8(y0);
                *reinterpret_cast<uint4*>(row + role.c1 * 16) = pack8(y1);
            }
        }
        from = from + 1 == kRotBwdDepth ? 0 : from + 1;
        fresh = get.next(sd.per_tile);
    }
    cp_async_wait<0>();

    float* red = reinterpret_cast<float*>(cs);               // [kSlots][D]
    __syncthreads();
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        *reinterpret_cast<float2*>(red + slot * D + role.c0 * 8 + 2 * j) = f2_get(dw0[j]);
        *reinterpret_cast<float2*>(red + slot * D + role.c1 * 8 + 2 * j) = f2_get(dw1[j]);
    }
    __syncthreads();
    for (int j = tid; j < D; j += kRotThreads) {
        float s = 0.f;
        for (int r = 0; r < C::kSlots; ++r) s += red[r * D + j];
        bp.part[(int64_t)blockIdx.x * D + j] = s;
    }
}

// dw[j] = sum over the side's blocks of part[block][j]: 32 columns a block, 32
// rows of threads, in fp64 and a fixed order. blockIdx.y 0: q, 1: k.
template <int D>
__global__ void __launch_bounds__(1024)
    fa_rotary_dw(const float* part, int blocks, int q_blocks, float* dwq, float* dwk) {
    pdl_launch_dependents();
    pdl_wait_prerequisites();
    __shared__ double red[32][33];
    const int j = blockIdx.x * 32 + threadIdx.x;
    const int lo = blockIdx.y ? q_blocks : 0, hi = blockIdx.y ? blocks : q_blocks;
    constexpr int kEach = (kRotBwdBlocks + 31) / 32;         // one side's blocks over 32 rows
    float v[kEach];                                          // loaded together
#pragma unroll
    for (int i = 0; i < kEach; ++i) {
        const int r = lo + (int)threadIdx.y + 32 * i;
        v[i] = r < hi ? part[(int64_t)r * D + j] : 0.f;
    }
    double s = 0.0;
#pragma unroll
    for (int i = 0; i < kEach; ++i) s += (double)v[i];
    red[threadIdx.y][threadIdx.x] = s;
    __syncthreads();
    s = red[threadIdx.x][threadIdx.y];                       // warp y: column y
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) s += __shfl_xor_sync(0xffffffffu, s, off);
    if (threadIdx.x == 0) (blockIdx.y ? dwk : dwq)[blockIdx.x * 32 + threadIdx.y] = (float)s;
}

}  // namespace fa
