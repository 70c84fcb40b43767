// Launch parameters shared by fa_rotary.cu and fa_paged.cu.
#pragma once

#include <algorithm>

#include "fa_host.h"
#include "fa_rotary_kernel.cuh"

namespace fa {

inline RotRows rot_rows(const fa_heads_t& t) {
    return RotRows{static_cast<uint8_t*>(t.ptr), t.stride_b, t.stride_h, t.stride_n};
}

inline void rot_fill(RotParams* p, const fa_rotary_t& r, const int32_t* pos, int64_t pos_sb,
                     int64_t pos_sn, int B, int H, int H_kv, int N) {
    p->pos = pos;
    p->pos_sb = pos_sb;
    p->pos_sn = pos_sn;
    p->freqs = r.freqs;
    p->wq = r.q_weight;
    p->wk = r.k_weight;
    p->w32 = r.weight_f32;
    p->rot = r.rotary_dim;
    p->cs_scale = r.rotary_scale;
    p->sin_sign = 1.f;
    p->eps = r.norm_eps;
    p->B = B;
    p->H = H;
    p->H_kv = H_kv;
    p->N = N;
    p->tokens = (int64_t)B * N;
}

// How the rows go to blocks. A block holds `slots` rows at a time; it takes
// as many tokens as it has slots (fewer where the batch has fewer tokens, the
// slots then spread over heads), so that a thread's angles serve all its
// heads. The heads of a token tile are split over blocks only until there are
// kRotFill blocks (4 an SM): each split computes the tile's angles again.
constexpr int64_t kRotFill = 4 * 148;

inline int64_t rot_tiling(RotParams* p, int slots, int heads) {
    int shift = 0;
    while ((1 << shift) < slots && ((int64_t)1 << shift) < p->tokens) ++shift;
    p->tt_shift = shift;
    const int64_t tiles = (p->tokens + (1ll << shift) - 1) >> shift;
    const int step = slots >> shift;                         // heads a block takes at once
    const int64_t most = (heads + step - 1) / step;
    p->splits = (int)std::max<int64_t>(1, std::min<int64_t>(most, (kRotFill + tiles - 1) / tiles));
    return tiles * p->splits;
}

// Positions: a device array that stays inside 63 bits of address.
inline bool positions_ok(const int32_t* pos, int64_t sb, int64_t sn, int64_t B, int64_t N) {
    return pos != nullptr && (addr(pos) & 3u) == 0 && sb >= 0 && sn >= 0 &&
           (double)sb * (double)B + (double)sn * (double)N < 1.0e18;
}

}  // namespace fa
