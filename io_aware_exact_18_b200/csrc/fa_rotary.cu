// Host side of fa_rotary.h: argument checks and launches.
#include <cuda_runtime.h>

#include <cmath>

#include "fa_host.h"
#include "fa_rotary_launch.h"

namespace fa {

int rotary_check(const fa_rotary_t& r, int d) {
    if (d != 64 && d != 128 && d != 256) return FA_ERR_UNSUPPORTED;
    if (r.rotary_dim < 0 || r.rotary_dim > d || r.rotary_dim % 16 != 0) return FA_ERR_INVALID_ARG;
    if ((r.interleaved | 1) != 1 || (r.norm | 1) != 1 || (r.weight_f32 | 1) != 1)
        return FA_ERR_INVALID_ARG;
    if (!std::isfinite(r.rotary_scale)) return FA_ERR_INVALID_ARG;
    if (r.norm && (!std::isfinite(r.norm_eps) || r.norm_eps < 0.f)) return FA_ERR_INVALID_ARG;
    const uintptr_t wmask = r.weight_f32 ? 3u : 1u;
    if (r.norm && ((addr(r.q_weight) | addr(r.k_weight)) & wmask) != 0) return FA_ERR_INVALID_ARG;
    if (r.rotary_dim > 0 && (r.freqs == nullptr || (addr(r.freqs) & 7u) != 0))
        return FA_ERR_INVALID_ARG;
    return FA_OK;
}

namespace {

// B, H, H_kv, N within what the kernels index: every product fits 63 bits and
// the grid 31.
int sizes_check(int B, int H, int H_kv, int N) {
    if (B < 0 || H < 0 || H_kv < 0 || N < 0) return FA_ERR_INVALID_ARG;
    if (H > 65536 || H_kv > 65536) return FA_ERR_INVALID_ARG;
    // rows (and so units of work) are counted in 31 bits
    if ((double)B * N * ((double)H + H_kv) > INT32_MAX) return FA_ERR_INVALID_ARG;
    if ((int64_t)B * N > INT32_MAX) return FA_ERR_INVALID_ARG;
    return FA_OK;
}

// Every view usable, every output with rows of its own, apart from the inputs
// (or exactly the one it may replace) and from the other outputs.
int views_check(const View* in, int n_in, const View* out, int n_out, const int* replaces) {
    for (int i = 0; i < n_in; ++i)
        if (in[i].H != 0 && !view_ok(in[i])) return FA_ERR_INVALID_ARG;
    for (int o = 0; o < n_out; ++o) {
        if (out[o].H == 0) continue;
        if (!view_ok(out[o]) || !rows_distinct(out[o])) return FA_ERR_INVALID_ARG;
        for (int i = 0; i < n_in; ++i) {
            if (in[i].H == 0 || (i == replaces[o] && same_view(in[i], out[o]))) continue;
            if (!views_apart(in[i], out[o])) return FA_ERR_INVALID_ARG;
        }
        for (int u = 0; u < o; ++u)
            if (out[u].H != 0 && !views_apart(out[u], out[o])) return FA_ERR_INVALID_ARG;
    }
    return FA_OK;
}

struct WriteSpan {
    const void* p;
    size_t n;
};
WriteSpan write_span(const View& v) { return WriteSpan{v.t.ptr, view_bytes(v)}; }

// The n spans that a call writes against positions, frequencies and weights.
bool spans_apart(const fa_rotary_t& r, const int32_t* pos, int64_t sb, int64_t sn, int B, int N,
                 int d, const WriteSpan* out, int n) {
    const ReadSpan reads[4] = {
        positions_span(pos, sb, sn, B, N), freqs_span(r), weight_span(r, r.q_weight, d),
        weight_span(r, r.k_weight, d)};
    for (const ReadSpan& x : reads)
        for (int o = 0; o < n; ++o)
            if (bytes_meet(out[o].p, out[o].n, x.p, x.n)) return false;
    return true;
}

template <int D, bool kNorm, bool kInter>
int launch_fwd_d(const RotParams& p, unsigned blocks, cudaStream_t s) {
    return launch_dependent(fa_qk_rotary_fwd<D, kNorm, kInter, kDense>, blocks, kRotThreads, 0, s, p);
}

template <int D>
int launch_fwd(RotParams p, bool norm, bool inter, cudaStream_t s) {
    const unsigned n = rot_grid(&p, RotCfg<D>::kSlots, p.H + p.H_kv);
    if (norm)
        return inter ? launch_fwd_d<D, true, true>(p, n, s) : launch_fwd_d<D, true, false>(p, n, s);
    return inter ? launch_fwd_d<D, false, true>(p, n, s) : launch_fwd_d<D, false, false>(p, n, s);
}

int launch_fwd_any(const RotParams& p, int d, bool norm, bool inter, cudaStream_t s) {
    return d == 64    ? launch_fwd<64>(p, norm, inter, s)
           : d == 128 ? launch_fwd<128>(p, norm, inter, s)
                      : launch_fwd<256>(p, norm, inter, s);
}

int fwd(const fa_qk_rotary_t& a, void* stream) {
    int rc = rotary_check(a.rotary, a.d);
    if (rc == FA_OK) rc = sizes_check(a.B, a.H, a.H_kv, a.N);
    if (rc != FA_OK) return rc;
    if (a.B == 0 || a.N == 0 || a.H + a.H_kv == 0) return FA_OK;
    if (!positions_ok(a.positions, a.pos_stride_b, a.pos_stride_n, a.B, a.N))
        return FA_ERR_INVALID_ARG;       // read whatever rotary_dim is
    const View in[2] = {{a.q, a.B, a.H, a.N, a.d}, {a.k, a.B, a.H_kv, a.N, a.d}};
    const View out[2] = {{a.q_out, a.B, a.H, a.N, a.d}, {a.k_out, a.B, a.H_kv, a.N, a.d}};
    const int replaces[2] = {0, 1};
    rc = views_check(in, 2, out, 2, replaces);
    if (rc != FA_OK) return rc;
    const WriteSpan writes[2] = {write_span(out[0]), write_span(out[1])};
    if (!spans_apart(a.rotary, a.positions, a.pos_stride_b, a.pos_stride_n, a.B, a.N, a.d, writes, 2))
        return FA_ERR_INVALID_ARG;
    rc = device_ready();
    if (rc != FA_OK) return rc;
    RotParams p{};
    p.q = rot_rows(a.q);
    p.k = rot_rows(a.k);
    p.qo = rot_rows(a.q_out);
    p.ko = rot_rows(a.k_out);
    rot_fill(&p, a.rotary, a.positions, a.pos_stride_b, a.pos_stride_n, a.B, a.H, a.H_kv, a.N);
    return launch_fwd_any(p, a.d, a.rotary.norm, a.rotary.interleaved,
                          static_cast<cudaStream_t>(stream));
}

int slots_of(int d) { return d == 64 ? RotCfg<64>::kSlots : d == 128 ? RotCfg<128>::kSlots
                                                                     : RotCfg<256>::kSlots; }

// Steps and blocks of the backward with the norm, q's and k's blocks in
// proportion to their heads.
int bwd_blocks(RotBwdParams* bp, int slots) {
    const int64_t tiles = rot_tiles(&bp->f, slots);
    const int H = bp->side[0].heads, H_kv = bp->side[1].heads;
    int64_t n[2] = {0, 0};
    for (int i = 0; i < 2; ++i) {
        RotBwdSide& sd = bp->side[i];
        if (sd.heads == 0) continue;
        sd.per_tile = (uint32_t)rot_steps(bp->f, slots, sd.heads);
        sd.steps = tiles * sd.per_tile;
        const int64_t share = (int64_t)kRotBwdBlocks * sd.heads / (H + H_kv);
        n[i] = std::max<int64_t>(1, std::min<int64_t>(sd.steps, share));
    }
    bp->q_blocks = (int)n[0];
    return (int)(n[0] + n[1]);
}

int bwd_blocks_of(int B, int H, int H_kv, int N, int d) {
    RotBwdParams bp{};
    bp.f.tokens = (int64_t)B * N;
    bp.side[0].heads = H;
    bp.side[1].heads = H_kv;
    return bwd_blocks(&bp, slots_of(d));
}

template <int D>
int launch_bwd(RotBwdParams bp, bool inter, float* dwq, float* dwk, cudaStream_t s) {
    const int blocks = bwd_blocks(&bp, RotCfg<D>::kSlots);
    const int rc = launch_dependent(
        inter ? fa_qk_rotary_bwd_norm<D, true> : fa_qk_rotary_bwd_norm<D, false>, blocks,
        kRotThreads, 0, s, bp);
    if (rc != FA_OK) return rc;
    return launch_dependent(fa_rotary_dw<D>, dim3(D / 32, 2), dim3(32, 32), 0, s,
                            (const float*)bp.part, blocks, bp.q_blocks, dwq, dwk);
}

int bwd(const fa_qk_rotary_bwd_t& a, void* ws, size_t ws_bytes, void* stream) {
    int rc = rotary_check(a.rotary, a.d);
    if (rc == FA_OK) rc = sizes_check(a.B, a.H, a.H_kv, a.N);
    if (rc != FA_OK) return rc;
    const bool norm = a.rotary.norm != 0;
    if (norm && (!a.dq_weight || !a.dk_weight ||
                 ((addr(a.dq_weight) | addr(a.dk_weight)) & 3u) != 0 ||
                 bytes_meet(a.dq_weight, 4 * a.d, a.dk_weight, 4 * a.d)))
        return FA_ERR_INVALID_ARG;
    if (!norm && (a.dq_weight || a.dk_weight)) return FA_ERR_INVALID_ARG;
    const bool empty = a.B == 0 || a.N == 0 || a.H + a.H_kv == 0;
    if (empty && !norm) return FA_OK;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    if (empty) {                      // no rows: the weights' gradients are zero
        rc = device_ready();
        if (rc != FA_OK) return rc;
        return cudaMemsetAsync(a.dq_weight, 0, 4 * a.d, s) == cudaSuccess &&
                       cudaMemsetAsync(a.dk_weight, 0, 4 * a.d, s) == cudaSuccess
                   ? FA_OK
                   : FA_ERR_LAUNCH;
    }
    if (!positions_ok(a.positions, a.pos_stride_b, a.pos_stride_n, a.B, a.N))
        return FA_ERR_INVALID_ARG;       // read whatever rotary_dim is
    const View in[4] = {{a.dq_out, a.B, a.H, a.N, a.d}, {a.dk_out, a.B, a.H_kv, a.N, a.d},
                        {a.q, a.B, a.H, a.N, a.d}, {a.k, a.B, a.H_kv, a.N, a.d}};
    const View out[2] = {{a.dq, a.B, a.H, a.N, a.d}, {a.dk, a.B, a.H_kv, a.N, a.d}};
    const int replaces[2] = {0, 1};
    rc = views_check(in, norm ? 4 : 2, out, 2, replaces);
    if (rc != FA_OK) return rc;
    const size_t need =
        norm ? (size_t)bwd_blocks_of(a.B, a.H, a.H_kv, a.N, a.d) * a.d * 4 : 0;
    const size_t dw_bytes = norm ? 4 * (size_t)a.d : 0;
    const WriteSpan writes[5] = {{ws, need}, {a.dq_weight, dw_bytes}, {a.dk_weight, dw_bytes},
                                 write_span(out[0]), write_span(out[1])};
    if (!spans_apart(a.rotary, a.positions, a.pos_stride_b, a.pos_stride_n, a.B, a.N, a.d, writes, 5))
        return FA_ERR_INVALID_ARG;
    if (norm) {
        if (ws == nullptr || (addr(ws) & 15u) != 0 || ws_bytes < need) return FA_ERR_INVALID_ARG;
        const WriteSpan* w = writes;
        for (int i = 0; i < 3; ++i) {
            for (const View& v : in)
                if (bytes_meet(w[i].p, w[i].n, v.t.ptr, view_bytes(v))) return FA_ERR_INVALID_ARG;
            for (const View& v : out)
                if (bytes_meet(w[i].p, w[i].n, v.t.ptr, view_bytes(v))) return FA_ERR_INVALID_ARG;
            if (i > 0 && bytes_meet(ws, need, w[i].p, w[i].n)) return FA_ERR_INVALID_ARG;
        }
    }
    rc = device_ready();
    if (rc != FA_OK) return rc;
    RotParams p{};
    rot_fill(&p, a.rotary, a.positions, a.pos_stride_b, a.pos_stride_n, a.B, a.H, a.H_kv, a.N);
    p.sin_sign = -1.f;                // the transpose of a rotation turns back
    p.qo = rot_rows(a.dq);
    p.ko = rot_rows(a.dk);
    if (!norm) {                      // dx = g: the forward with the angles negated
        p.q = rot_rows(a.dq_out);
        p.k = rot_rows(a.dk_out);
        return launch_fwd_any(p, a.d, false, a.rotary.interleaved, s);
    }
    RotBwdParams bp{};
    bp.f = p;
    bp.side[0] = RotBwdSide{rot_rows(a.dq_out), rot_rows(a.q), p.qo, p.wq, a.H, 0, 0};
    bp.side[1] = RotBwdSide{rot_rows(a.dk_out), rot_rows(a.k), p.ko, p.wk, a.H_kv, 0, 0};
    bp.part = static_cast<float*>(ws);
    const bool inter = a.rotary.interleaved != 0;
    if (a.d == 64) return launch_bwd<64>(bp, inter, a.dq_weight, a.dk_weight, s);
    if (a.d == 128) return launch_bwd<128>(bp, inter, a.dq_weight, a.dk_weight, s);
    return launch_bwd<256>(bp, inter, a.dq_weight, a.dk_weight, s);
}

}  // namespace
}  // namespace fa

#define FA_EXPORT __attribute__((visibility("default")))

extern "C" {

FA_EXPORT int fa_qk_rotary(const fa_qk_rotary_t* args, void* stream) {
    return args == nullptr ? FA_ERR_INVALID_ARG : fa::fwd(*args, stream);
}

FA_EXPORT int fa_qk_rotary_bwd(const fa_qk_rotary_bwd_t* args, void* workspace,
                               size_t workspace_bytes, void* stream) {
    return args == nullptr ? FA_ERR_INVALID_ARG
                           : fa::bwd(*args, workspace, workspace_bytes, stream);
}

FA_EXPORT size_t fa_qk_rotary_bwd_workspace_bytes(int B, int H, int H_kv, int N, int d, int norm) {
    if ((d != 64 && d != 128 && d != 256) || fa::sizes_check(B, H, H_kv, N) != FA_OK || !norm ||
        B == 0 || N == 0 || H + H_kv == 0)
        return 0;
    return (size_t)fa::bwd_blocks_of(B, H, H_kv, N, d) * (size_t)d * 4;
}

}  // extern "C"
