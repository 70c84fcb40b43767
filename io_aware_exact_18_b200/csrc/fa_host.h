// Host helpers shared by the library's translation units.
#pragma once

#include <cstddef>
#include <cstdint>

#include "fa_rotary.h"

namespace fa {

// Capability check of the current device: FA_OK, or the status to return.
int device_ready();

// ---------------------------------------------------------------- views
inline uintptr_t addr(const void* p) { return reinterpret_cast<uintptr_t>(p); }

inline bool bytes_meet(const void* a, size_t na, const void* b, size_t nb) {
    return na != 0 && nb != 0 && addr(a) < addr(b) + nb && addr(b) < addr(a) + na;
}

// A [B, heads, N, d] bf16 view with its sizes.
struct View {
    fa_heads_t t;
    int64_t B, H, N;
    int d;
};

// Bytes from the first to past the last element of a view (strides >= 0, 0 if
// empty). Overflow is excluded by view_ok.
inline size_t view_bytes(const View& v) {
    if (v.B == 0 || v.H == 0 || v.N == 0) return 0;
    return 2 * (size_t)((v.B > 1 ? (v.B - 1) * v.t.stride_b : 0) +
                        (v.H > 1 ? (v.H - 1) * v.t.stride_h : 0) +
                        (v.N > 1 ? (v.N - 1) * v.t.stride_n : 0) + v.d);
}

inline bool stride_ok(int64_t s, int64_t n) {
    // a multiple of 16 bytes whose extent stays far inside 63 bits; the stride
    // of an axis with one entry is never used
    return n <= 1 || (s >= 0 && (s & 7) == 0 && (double)s * (double)(n - 1) < 1.0e18);
}

inline bool view_ok(const View& v) {
    return v.t.ptr != nullptr && (addr(v.t.ptr) & 15u) == 0 && stride_ok(v.t.stride_b, v.B) &&
           stride_ok(v.t.stride_h, v.H) && stride_ok(v.t.stride_n, v.N);
}

// An output may not place two rows at one address: sorting the three axes by
// stride, each must step over the whole extent of the ones below it.
inline bool rows_distinct(const View& v) {
    int64_t s[3] = {v.t.stride_b, v.t.stride_h, v.t.stride_n}, n[3] = {v.B, v.H, v.N};
    for (int i = 0; i < 3; ++i)
        for (int j = i + 1; j < 3; ++j)
            if (s[j] < s[i]) {
                const int64_t a = s[i], b = n[i];
                s[i] = s[j]; n[i] = n[j];
                s[j] = a; n[j] = b;
            }
    int64_t extent = v.d;
    for (int i = 0; i < 3; ++i) {
        if (n[i] <= 1) continue;
        if (s[i] < extent) return false;
        extent += s[i] * (n[i] - 1);
    }
    return true;
}

// Whether the two views share no element. Beyond disjoint address ranges this
// knows one case: head ranges of the same token-major buffer (equal batch and
// token strides, each token's heads within one token stride, apart).
inline bool views_apart(const View& a, const View& b) {
    const size_t na = view_bytes(a), nb = view_bytes(b);
    if (!bytes_meet(a.t.ptr, na, b.t.ptr, nb)) return true;
    if (a.B != b.B || a.N != b.N) return false;
    if ((a.B > 1 && a.t.stride_b != b.t.stride_b) || (a.N > 1 && a.t.stride_n != b.t.stride_n))
        return false;
    const int64_t fa = (a.H > 1 ? (a.H - 1) * a.t.stride_h : 0) + a.d;
    const int64_t fb = (b.H > 1 ? (b.H - 1) * b.t.stride_h : 0) + b.d;
    const bool a_first = addr(a.t.ptr) < addr(b.t.ptr);
    const int64_t gap = (int64_t)((a_first ? addr(b.t.ptr) - addr(a.t.ptr)
                                           : addr(a.t.ptr) - addr(b.t.ptr)) / 2);
    const int64_t low = a_first ? fa : fb, span = gap + (a_first ? fb : fa);
    if (gap < low) return false;
    // the tokens' spans must not run into one another either
    if (a.N > 1 && a.t.stride_n < span) return false;
    const int64_t batch = (a.N > 1 ? (a.N - 1) * a.t.stride_n : 0) + span;
    return a.B <= 1 || a.t.stride_b >= batch;
}

inline bool same_view(const View& a, const View& b) {
    return a.t.ptr == b.t.ptr && (a.B <= 1 || a.t.stride_b == b.t.stride_b) &&
           (a.H <= 1 || a.t.stride_h == b.t.stride_h) &&
           (a.N <= 1 || a.t.stride_n == b.t.stride_n) && a.H == b.H;
}

// What a call reads besides its views: nothing it writes may meet them.
struct ReadSpan {
    const void* p;
    size_t n;
};
inline ReadSpan positions_span(const int32_t* pos, int64_t sb, int64_t sn, int64_t B, int64_t N) {
    return ReadSpan{pos, pos == nullptr ? 0 : 4 * (size_t)((B - 1) * sb + (N - 1) * sn + 1)};
}
inline ReadSpan freqs_span(const fa_rotary_t& r) {
    return ReadSpan{r.freqs, (size_t)r.rotary_dim / 2 * 8};
}
inline ReadSpan weight_span(const fa_rotary_t& r, const void* w, int d) {
    return ReadSpan{w, r.norm && w != nullptr ? (size_t)d * (r.weight_f32 ? 4 : 2) : 0};
}

// Sizes, positions and rotary arguments of the three entry points that turn
// heads (FA_OK, or the status to return).
int rotary_check(const fa_rotary_t& r, int d);

}  // namespace fa
