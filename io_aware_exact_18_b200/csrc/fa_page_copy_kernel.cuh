// Whole-page copies within a paged cache: 2 page bytes of HBM traffic a page,
// nothing to compute. A block moves kCopyVecs 16-byte pieces of K or of V,
// eight loads in flight a thread: a share of one large page, or several small
// pages. Pages whose rows lie dense (either order of heads and tokens) are
// copied as flat memory; others row by row with their strides. 2000 pages of
// 32 KB each of K and V: 42.1 us, 6.2 TB/s read and written, 0.95 of the copy
// rate; a handful of pages, 2.9 us.
#pragma once

#include <cstdint>

#include "sm100_ptx.cuh"

namespace fa {

constexpr int kCopyThreads = 256;
constexpr int kCopyUnroll = 8;
constexpr int kCopyVecs = kCopyThreads * kCopyUnroll;    // 32 KB a block

struct CopyParams {
    uint8_t *k, *v;
    int64_t page, head, token;       // strides in bytes
    const int32_t *src, *dst;
    int n, num_pages;
    int vecs;                        // 16-byte pieces of one page of K (or V)
    int row_vecs, tokens;            // of one row; page_size
    int per;                         // pages a block covers (vecs < kCopyVecs), else 1
    int segs;                        // blocks that share a page, else 1
};

template <bool kFlat>
__global__ void __launch_bounds__(kCopyThreads) fa_page_copy(const CopyParams p) {
    pdl_launch_dependents();
    pdl_wait_prerequisites();
    uint8_t* base = blockIdx.y ? p.v : p.k;
    const int seg = (int)(blockIdx.x % (unsigned)p.segs);
    const int64_t first = (int64_t)(blockIdx.x / (unsigned)p.segs) * p.per;
    const int here = (int)min((int64_t)p.per, p.n - first);
    const int v_lo = seg * kCopyVecs;
    const int total = p.segs > 1 ? min(p.vecs, v_lo + kCopyVecs) : here * p.vecs;
    uint4 val[kCopyUnroll];
    uint8_t* to[kCopyUnroll];
#pragma unroll
    for (int u = 0; u < kCopyUnroll; ++u) {
        const int i = v_lo + u * kCopyThreads + (int)threadIdx.x;
        to[u] = nullptr;
        if (i >= total) continue;
        const int pair = i / p.vecs, v = i - pair * p.vecs;
        const int s = p.src[first + pair], d = p.dst[first + pair];
        if (s < 0 || s >= p.num_pages || d < 0 || d >= p.num_pages || s == d) continue;
        int64_t in_page;
        if constexpr (kFlat) {
            in_page = (int64_t)v * 16;
        } else {
            const int row = v / p.row_vecs, c = v - row * p.row_vecs;
            const int h = row / p.tokens, t = row - h * p.tokens;
            in_page = h * p.head + t * p.token + c * 16;
        }
        to[u] = base + d * p.page + in_page;
        val[u] = *reinterpret_cast<const uint4*>(base + s * p.page + in_page);
    }
#pragma unroll
    for (int u = 0; u < kCopyUnroll; ++u)
        if (to[u] != nullptr) *reinterpret_cast<uint4*>(to[u]) = val[u];
}

}  // namespace fa
