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
// the norm: 4 and 2). So a thread owns one 16-byte chunk (8 elements) of the
// rows of ONE token, keeps A and B (16 registers) for that token and walks
// over the heads, four loads in flight. A half-layout chunk's partner is the
// chunk r/16 lanes away (rotary_dim is a multiple of 16), fetched by shuffle;
// interleaved partners sit in the chunk itself. A row's d / 8 lanes lie in
// one warp, so the sum of squares is a shuffle reduction.
//
// Angles: p f_i is formed in fp64 in turns (f_i / 2 pi), reduced to
// [-1/2, 1/2] there and only then rounded to fp32 (an error of at most 2^-25
// turns, 2e-7 rad, at any position); fp32 products would be off by 0.01 rad
// at position 10^5. A block's angles are computed once, cooperatively, into
// shared memory: one sincospi a thread for every 10 or so chunks.
#pragma once

#include <cuda_bf16.h>
#include <cstdint>

#include "sm100_ptx.cuh"

namespace fa {

constexpr int kRotThreads = 256;
constexpr int kRotUnroll = 4;        // heads whose loads a thread keeps in flight

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
    int tt_shift;                    // log2 of the tokens of a block
    int splits;                      // blocks that share a token tile's heads
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
    static constexpr int kLanes = D / 8;                     // lanes of a row
    static constexpr int kSlots = kRotThreads / kLanes;      // rows a block holds at once
    static constexpr int kTable = kSlots * D / 2;            // (cos, sin) of kSlots tokens
};

__device__ __forceinline__ float bf_lo(uint32_t v) { return __uint_as_float(v << 16); }
__device__ __forceinline__ float bf_hi(uint32_t v) { return __uint_as_float(v & 0xffff0000u); }

__device__ __forceinline__ void unpack8(const uint4& u, float (&x)[8]) {
    x[0] = bf_lo(u.x); x[1] = bf_hi(u.x);
    x[2] = bf_lo(u.y); x[3] = bf_hi(u.y);
    x[4] = bf_lo(u.z); x[5] = bf_hi(u.z);
    x[6] = bf_lo(u.w); x[7] = bf_hi(u.w);
}

__device__ __forceinline__ uint4 pack8(const float (&x)[8]) {
    return make_uint4(pack_bf16x2(x[0], x[1]), pack_bf16x2(x[2], x[3]), pack_bf16x2(x[4], x[5]),
                      pack_bf16x2(x[6], x[7]));
}

__device__ __forceinline__ float norm_weight(const void* w, int w32, int i) {
    if (w == nullptr) return 1.f;
    return w32 ? static_cast<const float*>(w)[i]
               : __bfloat162float(static_cast<const __nv_bfloat16*>(w)[i]);
}

// (s cos, s sin) of the block's tokens into shared memory. With `pad`, tokens
// outside the batch or at negative positions give position 0 (never used).
__device__ __forceinline__ void rotary_table(float2* cs, const RotParams& p, int64_t tok0, int tt,
                                             int tid) {
    const int half = p.rot >> 1;
    for (int e = tid; e < tt * half; e += kRotThreads) {
        const int t = e / half, i = e - t * half;
        const int64_t tok = tok0 + t;
        float c = 0.f, s = 0.f;
        if (tok < p.tokens) {
            const int64_t b = tok / p.N, n = tok - b * p.N;
            const int32_t pos = p.pos[b * p.pos_sb + n * p.pos_sn];
            double turns = (double)pos * p.freqs[i] * 0.15915494309189533577;
            turns -= rint(turns);
            sincospif(2.f * (float)turns, &s, &c);
        }
        cs[e] = make_float2(c * p.cs_scale, s * p.cs_scale * p.sin_sign);
    }
}

// Where a chunk stands in the rotation: whether it is turned, the lane of its
// partner chunk (half layout) and its first pair.
struct ChunkRole {
    bool turned, second;
    int partner, pair0;
};

template <int D, bool kInter>
__device__ __forceinline__ ChunkRole chunk_role(int c, int lane, int rot) {
    ChunkRole r;
    const int e0 = c * 8, half = rot >> 1;
    r.turned = e0 < rot;
    r.partner = lane;
    if constexpr (kInter) {
        r.second = false;
        r.pair0 = e0 >> 1;
    } else {
        r.second = r.turned && e0 >= half;
        r.pair0 = r.second ? e0 - half : e0;
        if (r.turned) r.partner = r.second ? lane - (half >> 3) : lane + (half >> 3);
    }
    return r;
}

// cos and signed sin of a chunk's elements: out_e = c_e y_e + s_e y_partner.
template <bool kInter>
__device__ __forceinline__ void chunk_angles(const float2* cs, const ChunkRole& r, float (&co)[8],
                                             float (&si)[8]) {
#pragma unroll
    for (int e = 0; e < 8; ++e) {
        co[e] = 1.f;
        si[e] = 0.f;
    }
    if (!r.turned) return;
    if constexpr (kInter) {
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const float2 t = cs[r.pair0 + j];
            co[2 * j] = co[2 * j + 1] = t.x;
            si[2 * j] = -t.y;
            si[2 * j + 1] = t.y;
        }
    } else {
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            const float2 t = cs[r.pair0 + e];
            co[e] = t.x;
            si[e] = r.second ? t.y : -t.y;
        }
    }
}

// The partners of a chunk's 8 elements. Elements that are not turned get 0,
// so that an infinity there is not multiplied by a zero coefficient.
template <bool kInter>
__device__ __forceinline__ void chunk_partners(const uint4& u, const ChunkRole& r,
                                               float (&xp)[8]) {
    if constexpr (kInter) {
        float x[8];
        unpack8(u, x);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            xp[2 * j] = r.turned ? x[2 * j + 1] : 0.f;
            xp[2 * j + 1] = r.turned ? x[2 * j] : 0.f;
        }
    } else {
        uint4 o;
        o.x = __shfl_sync(0xffffffffu, u.x, r.partner);
        o.y = __shfl_sync(0xffffffffu, u.y, r.partner);
        o.z = __shfl_sync(0xffffffffu, u.z, r.partner);
        o.w = __shfl_sync(0xffffffffu, u.w, r.partner);
        if (!r.turned) o = make_uint4(0u, 0u, 0u, 0u);
        unpack8(o, xp);
    }
}

template <int kLanes>
__device__ __forceinline__ float row_sum(float v) {
#pragma unroll
    for (int off = kLanes / 2; off > 0; off >>= 1) v += __shfl_xor_sync(0xffffffffu, v, off);
    return v;
}

enum RotStore { kDense = 0, kPageBf16 = 1, kPageE4m3 = 2 };

// Eight fp32 values to a cache row chunk (8 codes or 8 bf16 at element c * 8).
template <bool kE4m3>
__device__ __forceinline__ void store_chunk(uint8_t* row, int c, const float (&y)[8]) {
    if constexpr (kE4m3)
        *reinterpret_cast<uint2*>(row + c * 8) = make_uint2(
            pack_e4m3x4(y[0], y[1], y[2], y[3]), pack_e4m3x4(y[4], y[5], y[6], y[7]));
    else
        *reinterpret_cast<uint4*>(row + c * 16) = pack8(y);
}

// Heads [h_lo, h_hi) of one input for this thread's token: load, norm, turn,
// store. `in` and `out` point at head 0 of the token; strides in bytes. `mul`
// (1 / descale of an e4m3 store) is part of A and B already.
template <int D, bool kNorm, bool kInter, bool kE4m3>
__device__ __forceinline__ void turn_heads(const uint8_t* in, int64_t in_sh, uint8_t* out,
                                           int64_t out_sh, int h_lo, int h_hi, int h_off,
                                           int h_step, bool live, bool store, int c,
                                           const ChunkRole& role, const float (&A)[8],
                                           const float (&Bc)[8], float eps) {
    for (int h0 = h_lo; h0 < h_hi; h0 += h_step * kRotUnroll) {
        uint4 u[kRotUnroll];
#pragma unroll
        for (int i = 0; i < kRotUnroll; ++i) {
            const int h = h0 + i * h_step + h_off;
            u[i] = make_uint4(0u, 0u, 0u, 0u);
            if (live && h < h_hi)
                u[i] = *reinterpret_cast<const uint4*>(in + h * in_sh + c * 16);
        }
#pragma unroll
        for (int i = 0; i < kRotUnroll; ++i) {
            if (h0 + i * h_step >= h_hi) break;              // uniform in the block
            const int h = h0 + i * h_step + h_off;
            float x[8], xp[8], y[8];
            unpack8(u[i], x);
            chunk_partners<kInter>(u[i], role, xp);
            float r = 1.f;
            if constexpr (kNorm) {
                float ss = 0.f;
#pragma unroll
                for (int e = 0; e < 8; ++e) ss = fmaf(x[e], x[e], ss);
                ss = row_sum<D / 8>(ss);
                r = rsqrtf(fmaf(ss, 1.f / D, eps));
            }
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                y[e] = fmaf(A[e], x[e], Bc[e] * xp[e]);
                if constexpr (kNorm) y[e] *= r;
            }
            if (!(store && h < h_hi)) continue;
            if (!kNorm && !kE4m3 && !role.turned)            // passes through bit for bit
                *reinterpret_cast<uint4*>(out + h * out_sh + c * 16) = u[i];
            else
                store_chunk<kE4m3>(out + h * out_sh, c, y);
        }
    }
}

// A and B of one chunk: angles times the norm's weights (the partner's for B).
template <int D, bool kNorm, bool kInter>
__device__ __forceinline__ void coefficients(const float2* cs, const ChunkRole& role, int c,
                                             int rot, const void* w, int w32, float mul,
                                             float (&A)[8], float (&Bc)[8]) {
    chunk_angles<kInter>(cs, role, A, Bc);
#pragma unroll
    for (int e = 0; e < 8; ++e) {
        float wa = mul, wb = mul;
        if constexpr (kNorm) {
            const int i = c * 8 + e;
            int j = i;
            if (role.turned) {
                if constexpr (kInter) j = i ^ 1;
                else j = role.second ? i - (rot >> 1) : i + (rot >> 1);
            }
            wa *= norm_weight(w, w32, i);
            wb *= norm_weight(w, w32, j);
        }
        A[e] *= wa;
        Bc[e] *= wb;
    }
}

// Block (token tile, head split). Virtual heads: the H of q, the H_kv of k
// and, appending, the H_kv of v; a split takes an even share of them.
template <int D, bool kNorm, bool kInter, int kStore>
__global__ void __launch_bounds__(kRotThreads) fa_qk_rotary_fwd(const RotParams p) {
    using C = RotCfg<D>;
    __shared__ __align__(16) float2 cs[C::kTable];
    const int tid = threadIdx.x, lane = tid & 31;
    const int tt = 1 << p.tt_shift;
    const int64_t tile = blockIdx.x / (unsigned)p.splits;
    const int split = (int)(blockIdx.x - tile * p.splits);
    const int64_t tok0 = tile * tt;
    const int heads = p.H + p.H_kv + (kStore != kDense ? p.H_kv : 0);
    const int lo = (int)((int64_t)heads * split / p.splits);
    const int hi = (int)((int64_t)heads * (split + 1) / p.splits);
    if (lo < p.H + p.H_kv) rotary_table(cs, p, tok0, tt, tid);
    __syncthreads();

    const int c = tid % C::kLanes, slot = tid / C::kLanes;
    const int ts = slot & (tt - 1), h_off = slot >> p.tt_shift, h_step = C::kSlots >> p.tt_shift;
    const int64_t tok = tok0 + ts;
    const bool live = tok < p.tokens;
    const int64_t b = live ? tok / p.N : 0, n = live ? tok - b * p.N : 0;
    const ChunkRole role = chunk_role<D, kInter>(c, lane, p.rot);
    const float2* my_cs = cs + ts * (p.rot >> 1);

    bool write = live, stored = live;
    uint8_t *kdst = nullptr, *vdst = nullptr;
    int64_t dst_sh = 0;
    constexpr int kElem = kStore == kPageE4m3 ? 1 : 2;
    if constexpr (kStore != kDense) {
        // the token's slot in the cache, every index checked
        int32_t pos = -1;
        if (live) pos = p.pos[b * p.pos_sb + n * p.pos_sn];
        write = pos >= 0;
        stored = false;
        if (write) {
            const int64_t row = p.seq != nullptr ? p.seq[b] : b;
            const int pg = pos / p.page_size;
            if (row >= 0 && row < p.num_seqs && pg < p.width) {
                const int page = p.table[row * p.table_stride + pg];
                if (page >= 0 && page < p.num_pages) {
                    stored = true;
                    const int64_t off = (page * p.c_sp + (pos - pg * p.page_size) * p.c_st) * kElem;
                    kdst = p.kc + off;
                    vdst = p.vc + off;
                }
            }
        }
        dst_sh = p.c_sh * kElem;
    } else {
        kdst = p.ko.ptr + (b * p.ko.sb + n * p.ko.sn) * 2;
        dst_sh = p.ko.sh * 2;
    }

    float A[8], Bc[8];
    if (lo < p.H) {
        coefficients<D, kNorm, kInter>(my_cs, role, c, p.rot, p.wq, p.w32, 1.f, A, Bc);
        turn_heads<D, kNorm, kInter, false>(
            p.q.ptr + (b * p.q.sb + n * p.q.sn) * 2, p.q.sh * 2,
            p.qo.ptr + (b * p.qo.sb + n * p.qo.sn) * 2, p.qo.sh * 2, lo, min(hi, p.H), h_off,
            h_step, live, write, c, role, A, Bc, p.eps);
    }
    const int k_lo = max(lo - p.H, 0), k_hi = min(hi - p.H, p.H_kv);
    if (k_lo < k_hi) {
        coefficients<D, kNorm, kInter>(my_cs, role, c, p.rot, p.wk, p.w32,
                                       kStore == kPageE4m3 ? p.k_inv : 1.f, A, Bc);
        turn_heads<D, kNorm, kInter, kStore == kPageE4m3>(
            p.k.ptr + (b * p.k.sb + n * p.k.sn) * 2, p.k.sh * 2, kdst, dst_sh, k_lo, k_hi, h_off,
            h_step, live, stored, c, role, A, Bc, p.eps);
    }
    if constexpr (kStore != kDense) {
        const int v_lo = max(lo - p.H - p.H_kv, 0), v_hi = hi - p.H - p.H_kv;
        const uint8_t* vin = p.v.ptr + (b * p.v.sb + n * p.v.sn) * 2;
        for (int h0 = v_lo; h0 < v_hi; h0 += h_step * kRotUnroll) {
            uint4 u[kRotUnroll];
#pragma unroll
            for (int i = 0; i < kRotUnroll; ++i) {
                const int h = h0 + i * h_step + h_off;
                if (stored && h < v_hi)
                    u[i] = *reinterpret_cast<const uint4*>(vin + h * p.v.sh * 2 + c * 16);
            }
#pragma unroll
            for (int i = 0; i < kRotUnroll; ++i) {
                const int h = h0 + i * h_step + h_off;
                if (!(stored && h < v_hi)) continue;
                if constexpr (kStore == kPageE4m3) {
                    float y[8];
                    unpack8(u[i], y);
#pragma unroll
                    for (int e = 0; e < 8; ++e) y[e] *= p.v_inv;
                    store_chunk<true>(vdst + h * dst_sh, c, y);
                } else {
                    *reinterpret_cast<uint4*>(vdst + h * dst_sh + c * 16) = u[i];
                }
            }
        }
    }
}

// ---------------------------------------------------------------- backward
// With g the output gradient turned back (the rotation's transpose, times s)
// and r as in the forward:
//     dw_e  += g_e x_e r,        dx_e = r (g_e w_e - x_e r^2 mean(g w x)).
// x is read again (the forward keeps nothing), both row sums are reduced in
// the same shuffles, and dw is kept in registers over everything a thread
// sees: its chunk is fixed. The grid is at most kRotBwdBlocks blocks that
// take (token tile, head split) items in turn, so dw leaves as that many
// partial rows, which fa_rotary_dw adds in block order: no atomics.
constexpr int kRotBwdBlocks = 4 * 148;
constexpr int kRotBwdUnroll = 2;

struct RotBwdParams {
    RotParams f;                     // q, k: the forward's inputs; qo, ko: the outputs dq, dk
    RotRows dq_out, dk_out;
    float* part;                     // [blocks][2 D]
    int64_t items;                   // token tiles * splits
};

template <int D, bool kInter>
__device__ __forceinline__ void turn_back_heads(const uint8_t* gin, int64_t g_sh,
                                                const uint8_t* xin, int64_t x_sh, uint8_t* out,
                                                int64_t out_sh, int h_lo, int h_hi, int h_off,
                                                int h_step, bool live, int c,
                                                const ChunkRole& role, const float (&co)[8],
                                                const float (&si)[8], const void* wp, int w32,
                                                float eps, float (&dw)[8]) {
    float w[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) w[e] = norm_weight(wp, w32, c * 8 + e);
    for (int h0 = h_lo; h0 < h_hi; h0 += h_step * kRotBwdUnroll) {
        uint4 gu[kRotBwdUnroll], xu[kRotBwdUnroll];
#pragma unroll
        for (int i = 0; i < kRotBwdUnroll; ++i) {
            const int h = h0 + i * h_step + h_off;
            gu[i] = xu[i] = make_uint4(0u, 0u, 0u, 0u);
            if (live && h < h_hi) {
                gu[i] = *reinterpret_cast<const uint4*>(gin + h * g_sh + c * 16);
                xu[i] = *reinterpret_cast<const uint4*>(xin + h * x_sh + c * 16);
            }
        }
#pragma unroll
        for (int i = 0; i < kRotBwdUnroll; ++i) {
            if (h0 + i * h_step >= h_hi) break;              // uniform in the block
            const int h = h0 + i * h_step + h_off;
            float x[8], g[8], gp[8];
            unpack8(xu[i], x);
            unpack8(gu[i], g);
            chunk_partners<kInter>(gu[i], role, gp);
            float ss = 0.f, dot = 0.f;
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                g[e] = fmaf(co[e], g[e], si[e] * gp[e]);
                ss = fmaf(x[e], x[e], ss);
                dot = fmaf(g[e] * w[e], x[e], dot);
            }
#pragma unroll
            for (int off = D / 16; off > 0; off >>= 1) {
                ss += __shfl_xor_sync(0xffffffffu, ss, off);
                dot += __shfl_xor_sync(0xffffffffu, dot, off);
            }
            const float r = rsqrtf(fmaf(ss, 1.f / D, eps));
            const float k = r * r * dot * (1.f / D);
            if (live && h < h_hi) {                          // others hold zeros or no row
                float y[8];
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    dw[e] = fmaf(g[e], x[e] * r, dw[e]);
                    y[e] = r * fmaf(g[e], w[e], -x[e] * k);
                }
                *reinterpret_cast<uint4*>(out + h * out_sh + c * 16) = pack8(y);
            }
        }
    }
}

template <int D, bool kInter>
__global__ void __launch_bounds__(kRotThreads) fa_qk_rotary_bwd_norm(const RotBwdParams bp) {
    using C = RotCfg<D>;
    const RotParams& p = bp.f;
    __shared__ __align__(16) float2 cs[C::kTable];           // then the dw reduction, 8 KB both
    static_assert(C::kTable * 2 == C::kSlots * D, "the reduction reuses the table");
    pdl_launch_dependents();
    const int tid = threadIdx.x, lane = tid & 31;
    const int tt = 1 << p.tt_shift;
    const int c = tid % C::kLanes, slot = tid / C::kLanes;
    const int ts = slot & (tt - 1), h_off = slot >> p.tt_shift, h_step = C::kSlots >> p.tt_shift;
    const ChunkRole role = chunk_role<D, kInter>(c, lane, p.rot);
    const int heads = p.H + p.H_kv;
    float dwq[8], dwk[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) dwq[e] = dwk[e] = 0.f;

    for (int64_t item = blockIdx.x; item < bp.items; item += gridDim.x) {
        const int64_t tile = item / p.splits;
        const int split = (int)(item - tile * p.splits);
        const int64_t tok0 = tile * tt;
        const int lo = (int)((int64_t)heads * split / p.splits);
        const int hi = (int)((int64_t)heads * (split + 1) / p.splits);
        __syncthreads();                                     // the last item's table is read
        rotary_table(cs, p, tok0, tt, tid);
        __syncthreads();
        const int64_t tok = tok0 + ts;
        const bool live = tok < p.tokens;
        const int64_t b = live ? tok / p.N : 0, n = live ? tok - b * p.N : 0;
        float co[8], si[8];
        chunk_angles<kInter>(cs + ts * (p.rot >> 1), role, co, si);
        if (lo < p.H)
            turn_back_heads<D, kInter>(
                bp.dq_out.ptr + (b * bp.dq_out.sb + n * bp.dq_out.sn) * 2, bp.dq_out.sh * 2,
                p.q.ptr + (b * p.q.sb + n * p.q.sn) * 2, p.q.sh * 2,
                p.qo.ptr + (b * p.qo.sb + n * p.qo.sn) * 2, p.qo.sh * 2, lo, min(hi, p.H), h_off,
                h_step, live, c, role, co, si, p.wq, p.w32, p.eps, dwq);
        const int k_lo = max(lo - p.H, 0), k_hi = hi - p.H;
        if (k_lo < k_hi)
            turn_back_heads<D, kInter>(
                bp.dk_out.ptr + (b * bp.dk_out.sb + n * bp.dk_out.sn) * 2, bp.dk_out.sh * 2,
                p.k.ptr + (b * p.k.sb + n * p.k.sn) * 2, p.k.sh * 2,
                p.ko.ptr + (b * p.ko.sb + n * p.ko.sn) * 2, p.ko.sh * 2, k_lo, k_hi, h_off,
                h_step, live, c, role, co, si, p.wk, p.w32, p.eps, dwk);
    }

    float* red = reinterpret_cast<float*>(cs);               // [kSlots][D]
    auto reduce = [&](const float (&dw)[8], float* dst) {
        __syncthreads();
#pragma unroll
        for (int e = 0; e < 8; e += 4)
            *reinterpret_cast<float4*>(red + slot * D + c * 8 + e) =
                make_float4(dw[e], dw[e + 1], dw[e + 2], dw[e + 3]);
        __syncthreads();
        for (int j = tid; j < D; j += kRotThreads) {
            float s = 0.f;
            for (int r = 0; r < C::kSlots; ++r) s += red[r * D + j];
            dst[j] = s;
        }
    };
    reduce(dwq, bp.part + (int64_t)blockIdx.x * 2 * D);
    reduce(dwk, bp.part + (int64_t)blockIdx.x * 2 * D + D);
}

// dw[j] = sum over blocks of part[block][j], j < 2 D: 32 columns a block, 32
// rows of threads, in fp64 and a fixed order.
template <int D>
__global__ void __launch_bounds__(1024)
    fa_rotary_dw(const float* part, int blocks, float* dwq, float* dwk) {
    pdl_wait_prerequisites();
    __shared__ double red[32][33];
    const int j = blockIdx.x * 32 + threadIdx.x;
    double s = 0.0;
    for (int r = threadIdx.y; r < blocks; r += 32) s += (double)part[(int64_t)r * 2 * D + j];
    red[threadIdx.y][threadIdx.x] = s;
    __syncthreads();
    if (threadIdx.y == 0) {
        double t = 0.0;
#pragma unroll
        for (int r = 0; r < 32; ++r) t += red[r][threadIdx.x];
        (j < D ? dwq[j] : dwk[j - D]) = (float)t;
    }
}

}  // namespace fa
