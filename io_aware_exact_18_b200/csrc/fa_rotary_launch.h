// Launch parameters shared by fa_rotary.cu and fa_paged.cu.
#pragma once

#include <algorithm>

#include "fa_host.h"
#include "fa_launch.h"
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
    p->pair_shift = 0;
    while ((1 << p->pair_shift) < r.rotary_dim / 2) ++p->pair_shift;
    p->cs_scale = r.rotary_scale;
    p->sin_sign = 1.f;
    p->eps = r.norm_eps;
    p->B = B;
    p->H = H;
    p->H_kv = H_kv;
    p->N = N;
    p->tokens = (int64_t)B * N;
}

// Tokens of a tile, and the tiles: a block holds `slots` rows at a time; it
// takes as many tokens as it has slots (fewer where the batch has fewer, the
// slots then spread over heads), so that a thread's angles serve all its
// heads.
inline int64_t rot_tiles(RotParams* p, int slots) {
    int shift = 0;
    while ((1 << shift) < slots && ((int64_t)1 << shift) < p->tokens) ++shift;
    p->tt_shift = shift;
    return (p->tokens + (1ll << shift) - 1) >> shift;
}

// Steps of `heads` heads in a tile: as many heads as a block takes at once.
inline int rot_steps(const RotParams& p, int slots, int heads) {
    const int step = slots >> p.tt_shift;
    return (heads + step - 1) / step;
}

// The grid of a forward or an append: token tiles, their heads split over
// blocks (each of which computes the tile's angles) up to kRotFill blocks.
inline unsigned rot_grid(RotParams* p, int slots, int heads) {
    const int64_t tiles = rot_tiles(p, slots);
    p->splits = (int)std::max<int64_t>(1, std::min<int64_t>(rot_steps(*p, slots, heads),
                                                            (kRotFill + tiles - 1) / tiles));
    return (unsigned)(tiles * p->splits);
}

// Positions: a device array that stays inside 63 bits of address.
inline bool positions_ok(const int32_t* pos, int64_t sb, int64_t sn, int64_t B, int64_t N) {
    return pos != nullptr && (addr(pos) & 3u) == 0 && sb >= 0 && sn >= 0 &&
           (double)sb * (double)B + (double)sn * (double)N < 1.0e18;
}

}  // namespace fa
