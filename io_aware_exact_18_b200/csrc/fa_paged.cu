// Host side of fa_paged.h: argument checks and launches.
#include <cuda_runtime.h>

#include <cmath>

#include "fa_host.h"
#include "fa_page_copy_kernel.cuh"
#include "fa_paged.h"
#include "fa_paged_decode_kernel.cuh"
#include "fa_rotary_launch.h"

namespace fa {
namespace {

// Whether two row sets of one layout, `delta` elements apart, share one: rows of
// `row` elements at sums of i_a s_a, 0 <= i_a < n_a, the strides ascending and
// each stepping over the whole extent of the axes below. On each axis from the
// widest only the two multiples around delta can bring the rest within reach.
bool rows_meet(int64_t delta, const int64_t* s, const int64_t* n, int axes, int64_t row) {
    if (axes == 0) return delta < row && -delta < row;
    const int64_t st = s[axes - 1], most = n[axes - 1] - 1;
    if (most == 0) return rows_meet(delta, s, n, axes - 1, row);
    const int64_t below = delta / st - (delta % st < 0 ? 1 : 0);         // floor
    for (int64_t i = below; i <= below + 1; ++i)
        if (i >= -most && i <= most && rows_meet(delta - i * st, s, n, axes - 1, row)) return true;
    return false;
}

// The cache's own arguments; *bytes: from its first to past its last byte,
// the same for K and V. A call that writes it needs K and V apart.
int cache_check(const fa_paged_cache_t& c, bool writes, size_t* bytes) {
    if (c.d != 64 && c.d != 128 && c.d != 256) return FA_ERR_UNSUPPORTED;
    if (c.elem != 1 && c.elem != 2) return FA_ERR_UNSUPPORTED;
    if (c.num_pages < 0 || c.page_size < 1 || c.page_size > 65536 || c.H_kv < 0 || c.H_kv > 65536)
        return FA_ERR_INVALID_ARG;
    if (!std::isfinite(c.k_descale) || !std::isfinite(c.v_descale) || !(c.k_descale > 0.f) ||
        !(c.v_descale > 0.f) || (c.elem == 2 && (c.k_descale != 1.f || c.v_descale != 1.f)))
        return FA_ERR_INVALID_ARG;
    *bytes = 0;
    if (c.num_pages == 0 || c.H_kv == 0) return FA_OK;
    if (!c.k || !c.v || ((addr(c.k) | addr(c.v)) & 15u) != 0) return FA_ERR_INVALID_ARG;
    // strides: multiples of 16 bytes, each axis stepping over the ones below
    int64_t s[3] = {c.stride_page, c.stride_head, c.stride_token};
    int64_t n[3] = {c.num_pages, c.H_kv, c.page_size};
    for (int i = 0; i < 3; ++i) {
        if (n[i] == 1) s[i] = 0;
        if (s[i] < 0 || (s[i] * c.elem) % 16 != 0 || (double)s[i] * (double)n[i] > 1.0e18)
            return FA_ERR_INVALID_ARG;
    }
    for (int i = 0; i < 3; ++i)
        for (int j = i + 1; j < 3; ++j)
            if (s[j] < s[i]) {
                std::swap(s[i], s[j]);
                std::swap(n[i], n[j]);
            }
    int64_t extent = c.d;
    for (int i = 0; i < 3; ++i) {
        if (n[i] == 1) continue;
        if (s[i] < extent) return FA_ERR_INVALID_ARG;
        extent += s[i] * (n[i] - 1);
    }
    *bytes = (size_t)extent * c.elem;
    const int64_t apart = (int64_t)(addr(c.v) - addr(c.k)) / c.elem;
    if (apart == 0 || (writes && bytes_meet(c.k, *bytes, c.v, *bytes) &&
                       rows_meet(apart, s, n, 3, c.d)))
        return FA_ERR_INVALID_ARG;
    return FA_OK;
}

int table_check(const fa_block_table_t& t) {
    if (t.num_seqs < 0 || t.pages_per_seq < 0 || t.stride < 0) return FA_ERR_INVALID_ARG;
    if (t.num_seqs == 0 || t.pages_per_seq == 0) return FA_OK;
    if (!t.pages || (addr(t.pages) & 3u) != 0) return FA_ERR_INVALID_ARG;
    if (t.num_seqs > 1 && (double)t.stride * t.num_seqs > 1.0e18) return FA_ERR_INVALID_ARG;
    return FA_OK;
}

bool meets_cache(const fa_paged_cache_t& c, size_t bytes, const void* p, size_t n) {
    return bytes_meet(c.k, bytes, p, n) || bytes_meet(c.v, bytes, p, n);
}

// ------------------------------------------------------------------ append
template <int D, bool kNorm, bool kInter>
int launch_append_d(const RotParams& p, unsigned blocks, int elem, cudaStream_t s) {
    return launch_dependent(elem == 1 ? fa_qk_rotary_fwd<D, kNorm, kInter, kPageE4m3>
                                      : fa_qk_rotary_fwd<D, kNorm, kInter, kPageBf16>,
                            blocks, kRotThreads, 0, s, p);
}

template <int D>
int launch_append(RotParams p, int elem, bool norm, bool inter, cudaStream_t s) {
    const unsigned n = rot_grid(&p, RotCfg<D>::kSlots, p.H + 2 * p.H_kv);
    if (norm)
        return inter ? launch_append_d<D, true, true>(p, n, elem, s)
                     : launch_append_d<D, true, false>(p, n, elem, s);
    return inter ? launch_append_d<D, false, true>(p, n, elem, s)
                 : launch_append_d<D, false, false>(p, n, elem, s);
}

int append(const fa_paged_append_t& a, void* stream) {
    const fa_paged_cache_t& c = a.cache;
    size_t cbytes = 0;
    int rc = cache_check(c, true, &cbytes);
    if (rc == FA_OK) rc = rotary_check(a.rotary, c.d);
    if (rc == FA_OK) rc = table_check(a.table);
    if (rc != FA_OK) return rc;
    if (a.B < 0 || a.H < 0 || a.N < 0 || (int64_t)a.B * a.N > INT32_MAX || a.H > 65536 ||
        (double)a.B * a.N * ((double)a.H + 2.0 * c.H_kv) > INT32_MAX)   // rows in 31 bits
        return FA_ERR_INVALID_ARG;
    // Codes are x / descale; the product with the rounded reciprocal is off by
    // 2^-23 of it, far below the 2^-4 of the e4m3 rounding that follows. A
    // reciprocal that is infinite would make NaN of zeros.
    const float k_inv = 1.f / c.k_descale, v_inv = 1.f / c.v_descale;
    if (!std::isfinite(k_inv) || !std::isfinite(v_inv)) return FA_ERR_INVALID_ARG;
    if ((a.q.ptr == nullptr) != (a.q_out.ptr == nullptr)) return FA_ERR_INVALID_ARG;
    const int H = a.q.ptr == nullptr ? 0 : a.H;
    if (a.B == 0 || a.N == 0 || H + c.H_kv == 0) return FA_OK;
    if (!positions_ok(a.positions, a.pos_stride_b, a.pos_stride_n, a.B, a.N))
        return FA_ERR_INVALID_ARG;
    if ((addr(a.seq) & 3u) != 0) return FA_ERR_INVALID_ARG;
    const View k{a.k, a.B, c.H_kv, a.N, c.d}, v{a.v, a.B, c.H_kv, a.N, c.d};
    const View q{a.q, a.B, H, a.N, c.d}, qo{a.q_out, a.B, H, a.N, c.d};
    if (c.H_kv > 0 && (!view_ok(k) || !view_ok(v))) return FA_ERR_INVALID_ARG;
    if (H > 0) {
        if (!view_ok(q) || !view_ok(qo) || !rows_distinct(qo)) return FA_ERR_INVALID_ARG;
        if (!same_view(q, qo) && !views_apart(q, qo)) return FA_ERR_INVALID_ARG;
        if (c.H_kv > 0 && (!views_apart(k, qo) || !views_apart(v, qo))) return FA_ERR_INVALID_ARG;
    }
    for (const View& x : {k, v, q, qo})
        if (x.H > 0 && meets_cache(c, cbytes, x.t.ptr, view_bytes(x))) return FA_ERR_INVALID_ARG;
    const int64_t table_ints = a.table.num_seqs == 0 || a.table.pages_per_seq == 0
                                   ? 0
                                   : (a.table.num_seqs - 1) * a.table.stride + a.table.pages_per_seq;
    const ReadSpan reads[6] = {
        {a.table.pages, (size_t)table_ints * 4}, {a.seq, a.seq ? (size_t)a.B * 4 : 0},
        positions_span(a.positions, a.pos_stride_b, a.pos_stride_n, a.B, a.N),
        freqs_span(a.rotary), weight_span(a.rotary, a.rotary.q_weight, c.d),
        weight_span(a.rotary, a.rotary.k_weight, c.d)};
    for (const ReadSpan& r : reads)
        if (meets_cache(c, cbytes, r.p, r.n) ||
            (H > 0 && bytes_meet(a.q_out.ptr, view_bytes(qo), r.p, r.n)))
            return FA_ERR_INVALID_ARG;
    rc = device_ready();
    if (rc != FA_OK) return rc;
    RotParams p{};
    rot_fill(&p, a.rotary, a.positions, a.pos_stride_b, a.pos_stride_n, a.B, H, c.H_kv, a.N);
    p.q = rot_rows(a.q);
    p.k = rot_rows(a.k);
    p.v = rot_rows(a.v);
    p.qo = rot_rows(a.q_out);
    p.kc = static_cast<uint8_t*>(c.k);
    p.vc = static_cast<uint8_t*>(c.v);
    p.c_sp = c.stride_page;
    p.c_sh = c.stride_head;
    p.c_st = c.stride_token;
    p.table = a.table.pages;
    p.table_stride = a.table.stride;
    p.seq = a.seq;
    p.num_seqs = a.table.num_seqs;
    p.width = a.table.pages_per_seq;
    p.num_pages = c.num_pages;
    p.page_size = c.page_size;
    p.k_inv = k_inv;
    p.v_inv = v_inv;
    const bool norm = a.rotary.norm != 0, inter = a.rotary.interleaved != 0;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    return c.d == 64    ? launch_append<64>(p, c.elem, norm, inter, s)
           : c.d == 128 ? launch_append<128>(p, c.elem, norm, inter, s)
                        : launch_append<256>(p, c.elem, norm, inter, s);
}

// ------------------------------------------------------------------ decode
// Query heads of a unit: one 8-column product up to 8 heads a K/V head, two
// up to 16 and beyond (blocks of 16 heads, which read K and V again).
int head_tiles(int group) { return group <= 8 ? 1 : 2; }

struct PdPlan {
    int G, nt, hblk;
    size_t o_bytes, lse_bytes, split_bytes;
    size_t total() const { return o_bytes + lse_bytes + split_bytes; }
};

size_t up256(size_t n) { return (n + 255) & ~size_t(255); }

PdPlan pd_plan(int B, int H, int H_kv, int d) {
    PdPlan pl;
    pl.G = H / H_kv;
    pl.nt = head_tiles(pl.G);
    pl.hblk = (pl.G + 8 * pl.nt - 1) / (8 * pl.nt);
    const size_t rows = (size_t)kPdBlocks * 2 * pd_warps_most(d, pl.nt) * 8 * pl.nt;
    pl.o_bytes = rows * d * 4;
    pl.lse_bytes = up256(rows * 4);
    pl.split_bytes = up256((size_t)B * H_kv * pl.hblk * 8);
    return pl;
}

template <int D, int kAt>
int launch_join(const PdParams& p, int heads, int warps, cudaStream_t s) {
    using C = PdJoinCfg<D, kAt>;
    return launch_dependent(fa_paged_join<D, kAt>,
                            (unsigned)(((int64_t)p.B * p.H + C::kRows - 1) / C::kRows),
                            C::kThreads, 0, s, p, heads, warps);
}

template <int D, int E, int NT>
int launch_decode(const PdParams& p, cudaStream_t s) {
    using C = PdCfg<D, E, NT>;
    auto kern = fa_paged_decode_kernel<D, E, NT>;
    // once per device: a benign race sets the same value twice
    static bool ready[64];
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return FA_ERR_LAUNCH;
    if (!__atomic_load_n(&ready[dev], __ATOMIC_ACQUIRE)) {
        if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, C::kSmem) !=
            cudaSuccess)
            return FA_ERR_LAUNCH;
        __atomic_store_n(&ready[dev], true, __ATOMIC_RELEASE);
    }
    const int rc = launch_dependent(kern, kPdBlocks, C::kThreads, C::kSmem, s, p);
    if (rc != FA_OK) return rc;
    if ((int64_t)p.B * p.H_kv * p.hblk >= kPdJoinUnits)
        return launch_join<D, 1>(p, C::kHeads, C::kWarps, s);
    return launch_join<D, 8>(p, C::kHeads, C::kWarps, s);
}

template <int D>
int launch_decode_d(const PdParams& p, int elem, int nt, cudaStream_t s) {
    if (elem == 2) return nt == 1 ? launch_decode<D, 2, 1>(p, s) : launch_decode<D, 2, 2>(p, s);
    return nt == 1 ? launch_decode<D, 1, 1>(p, s) : launch_decode<D, 1, 2>(p, s);
}

int decode(const fa_paged_decode_t& a, void* ws, size_t ws_bytes, void* stream) {
    const fa_paged_cache_t& c = a.cache;
    size_t cbytes = 0;
    int rc = cache_check(c, false, &cbytes);
    if (rc == FA_OK) rc = table_check(a.table);
    if (rc != FA_OK) return rc;
    if (a.B < 0 || a.H < 0 || (int64_t)a.B * a.H > INT32_MAX / 64) return FA_ERR_INVALID_ARG;
    if (a.H > 0 && (c.H_kv < 1 || c.H_kv > a.H || a.H % c.H_kv != 0)) return FA_ERR_INVALID_ARG;
    if (!std::isfinite(a.scale) || !(a.scale > 0.f)) return FA_ERR_INVALID_ARG;
    if (a.B == 0 || a.H == 0) return FA_OK;
    if (a.table.num_seqs < a.B) return FA_ERR_INVALID_ARG;
    if (!a.q || !a.o || !a.lse || !a.kv_len) return FA_ERR_INVALID_ARG;
    if (((addr(a.q) | addr(a.o)) & 15u) != 0 || ((addr(a.lse) | addr(a.kv_len)) & 3u) != 0)
        return FA_ERR_INVALID_ARG;
    const View q{{const_cast<void*>(a.q), a.q_stride_b, a.q_stride_h, 0}, a.B, a.H, 1, c.d};
    if (!view_ok(q)) return FA_ERR_INVALID_ARG;
    const PdPlan pl = pd_plan(a.B, a.H, c.H_kv, c.d);
    const size_t rows = (size_t)a.B * a.H, ob = rows * c.d * 2, lb = rows * 4, need = pl.total();
    if (ws == nullptr || (addr(ws) & 15u) != 0 || ws_bytes < need) return FA_ERR_INVALID_ARG;
    struct Buf { const void* p; size_t n; };
    const Buf outs[3] = {{a.o, ob}, {a.lse, lb}, {ws, need}};
    const Buf ins[3] = {{a.q, view_bytes(q)}, {a.kv_len, (size_t)a.B * 4},
                        {a.table.pages, a.table.pages_per_seq == 0
                                            ? 0
                                            : ((size_t)(a.B - 1) * a.table.stride +
                                               a.table.pages_per_seq) * 4}};
    for (int i = 0; i < 3; ++i) {
        if (meets_cache(c, cbytes, outs[i].p, outs[i].n)) return FA_ERR_INVALID_ARG;
        for (int j = 0; j < 3; ++j)
            if (bytes_meet(outs[i].p, outs[i].n, ins[j].p, ins[j].n)) return FA_ERR_INVALID_ARG;
        for (int j = 0; j < i; ++j)
            if (bytes_meet(outs[i].p, outs[i].n, outs[j].p, outs[j].n)) return FA_ERR_INVALID_ARG;
    }
    rc = device_ready();
    if (rc != FA_OK) return rc;
    PdParams p{};
    p.q = static_cast<const __nv_bfloat16*>(a.q);
    p.q_sb = a.B > 1 ? a.q_stride_b : 0;
    p.q_sh = a.H > 1 ? a.q_stride_h : 0;
    p.kc = static_cast<const uint8_t*>(c.k);
    p.vc = static_cast<const uint8_t*>(c.v);
    p.c_sp = c.num_pages > 1 ? c.stride_page * c.elem : 0;
    p.c_sh = c.H_kv > 1 ? c.stride_head * c.elem : 0;
    p.c_st = c.page_size > 1 ? c.stride_token * c.elem : 0;
    p.table = a.table.pages;
    p.table_stride = a.table.stride;
    p.width = a.table.pages_per_seq;
    p.num_pages = c.num_pages;
    p.page_size = c.page_size;
    // key / page_size = (2 key * m) >> 32 >> s for keys below 2^31, with s =
    // ceil(log2 page_size) and m = ceil(2^(31 + s) / page_size) < 2^32: the
    // excess of m is below page_size / 2^(31 + s), so key times it stays below
    // one unit of 1 / page_size.
    uint32_t lg = 0;
    while ((1ll << lg) < c.page_size) ++lg;
    p.page_mul = (uint32_t)(((1ull << (31 + lg)) + c.page_size - 1) / c.page_size);
    p.page_shift = lg;
    p.kv_len = a.kv_len;
    p.o = static_cast<__nv_bfloat16*>(a.o);
    p.lse = a.lse;
    uint8_t* w = static_cast<uint8_t*>(ws);
    p.part_o = reinterpret_cast<float*>(w);
    p.part_lse = reinterpret_cast<float*>(w + pl.o_bytes);
    p.split = reinterpret_cast<int2*>(w + pl.o_bytes + pl.lse_bytes);
    p.B = a.B;
    p.H = a.H;
    p.H_kv = c.H_kv;
    p.G = pl.G;
    p.hblk = pl.hblk;
    p.scale_log2 = (float)((double)a.scale * c.k_descale * 1.4426950408889634);
    p.o_mul = c.v_descale;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    if (c.d == 64) return launch_decode_d<64>(p, c.elem, pl.nt, s);
    if (c.d == 128) return launch_decode_d<128>(p, c.elem, pl.nt, s);
    return launch_decode_d<256>(p, c.elem, pl.nt, s);
}

// ------------------------------------------------------------------ copies
int copy(const fa_paged_cache_t& c, const int32_t* src, const int32_t* dst, int n, void* stream) {
    size_t cbytes = 0;
    int rc = cache_check(c, true, &cbytes);
    if (rc != FA_OK) return rc;
    if (n < 0 || n > INT32_MAX / 128) return FA_ERR_INVALID_ARG;
    if (n == 0 || cbytes == 0) return FA_OK;
    if (!src || !dst || ((addr(src) | addr(dst)) & 3u) != 0) return FA_ERR_INVALID_ARG;
    if (meets_cache(c, cbytes, src, 4 * (size_t)n) || meets_cache(c, cbytes, dst, 4 * (size_t)n))
        return FA_ERR_INVALID_ARG;
    const int64_t row_vecs = (int64_t)c.d * c.elem / 16;
    const int64_t vecs = row_vecs * c.H_kv * c.page_size;
    if (vecs > INT32_MAX / 2) return FA_ERR_INVALID_ARG;
    CopyParams p{};
    p.k = static_cast<uint8_t*>(c.k);
    p.v = static_cast<uint8_t*>(c.v);
    p.page = c.num_pages > 1 ? c.stride_page * c.elem : 0;
    p.head = c.H_kv > 1 ? c.stride_head * c.elem : 0;
    p.token = c.page_size > 1 ? c.stride_token * c.elem : 0;
    p.src = src;
    p.dst = dst;
    p.n = n;
    p.num_pages = c.num_pages;
    p.vecs = (int)vecs;
    p.row_vecs = (int)row_vecs;
    p.tokens = c.page_size;
    p.per = (int)std::max<int64_t>(1, kCopyVecs / vecs);
    p.segs = (int)((vecs + kCopyVecs - 1) / kCopyVecs);
    const int64_t blocks = ((int64_t)n + p.per - 1) / p.per * p.segs;
    if (blocks > INT32_MAX) return FA_ERR_INVALID_ARG;
    // rows of a page side by side, heads outermost or tokens outermost
    const int64_t row = (int64_t)c.d * c.elem;
    const bool heads_out = (c.page_size == 1 || p.token == row) &&
                           (c.H_kv == 1 || p.head == row * c.page_size);
    const bool tokens_out = (c.H_kv == 1 || p.head == row) &&
                            (c.page_size == 1 || p.token == row * c.H_kv);
    rc = device_ready();
    if (rc != FA_OK) return rc;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    const dim3 grid((unsigned)blocks, 2);
    return launch_dependent(heads_out || tokens_out ? fa_page_copy<true> : fa_page_copy<false>,
                            grid, kCopyThreads, 0, s, p);
}

}  // namespace
}  // namespace fa

#define FA_EXPORT __attribute__((visibility("default")))

extern "C" {

FA_EXPORT int fa_paged_append(const fa_paged_append_t* args, void* stream) {
    return args == nullptr ? FA_ERR_INVALID_ARG : fa::append(*args, stream);
}

FA_EXPORT int fa_paged_decode(const fa_paged_decode_t* args, void* workspace,
                              size_t workspace_bytes, void* stream) {
    return args == nullptr ? FA_ERR_INVALID_ARG
                           : fa::decode(*args, workspace, workspace_bytes, stream);
}

FA_EXPORT size_t fa_paged_decode_workspace_bytes(int B, int H, int H_kv, int d) {
    if (B < 1 || H < 1 || H_kv < 1 || H % H_kv != 0 || (d != 64 && d != 128 && d != 256) ||
        (int64_t)B * H > INT32_MAX / 64)
        return 0;
    return fa::pd_plan(B, H, H_kv, d).total();
}

FA_EXPORT int fa_copy_pages(const fa_paged_cache_t* cache, const int32_t* src, const int32_t* dst,
                            int n, void* stream) {
    return cache == nullptr ? FA_ERR_INVALID_ARG : fa::copy(*cache, src, dst, n, stream);
}

}  // extern "C"
