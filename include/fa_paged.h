/*
 * fa_paged.h -- a key/value cache in pages: writing new tokens into it, one
 * new token's attention over it, and copies of its pages.
 *
 * The cache holds K and V as num_pages pages of page_size tokens; a block
 * table row lists the pages of one sequence in order, so key j of sequence s
 * lies in page block_table[s][j / page_size], slot j % page_size. Conventions
 * are those of fa.h and fa_rotary.h (caller-owned device pointers, status
 * codes, errors before any CUDA call, asynchronous, deterministic, sm_100
 * only; no bounded waits, so the device status word is not used), with:
 *   - Table entries, positions and lengths live on the device and are checked
 *     there: an entry outside [0, num_pages) names no page. What would be
 *     written to such a page is dropped, and its keys are hidden.
 *   - All offsets are 64-bit.
 */
#ifndef FA_PAGED_H_
#define FA_PAGED_H_

#include <stddef.h>
#include <stdint.h>

#include "fa.h"
#include "fa_rotary.h"

#ifdef __cplusplus
extern "C" {
#endif

/*
 * The pages. Element j of head h, slot t, page p lies at p * stride_page +
 * h * stride_head + t * stride_token + j elements from k (and from v): both
 * [pages, H_kv, page_size, d] and [pages, page_size, H_kv, d] orders fit.
 * Pointers are 16-byte aligned and strides multiples of 16 bytes, > 0 where
 * the extent is above 1. Distinct rows must not overlap; K and V may lie in one
 * buffer, and share no element where a call writes them. page_size is any
 * number from 1 to 65536, d is 64, 128 or 256.
 * elem 2: bf16. elem 1: e4m3 codes that stand for descale * code
 * (k_descale, v_descale finite and > 0; both must be 1 for bf16).
 */
typedef struct {
    void *k, *v;
    int64_t stride_page, stride_head, stride_token;
    int32_t num_pages, page_size, H_kv, d, elem;
    float k_descale, v_descale;
    int32_t reserved;
} fa_paged_cache_t;

/* Page lists: int32 [num_seqs, pages_per_seq], rows stride elements apart. */
typedef struct {
    const int32_t *pages;
    int64_t stride;
    int32_t num_seqs, pages_per_seq;
} fa_block_table_t;

typedef struct {
    fa_paged_cache_t cache;
    fa_block_table_t table;
    fa_heads_t k, v;          /* in: bf16 [B, H_kv, N, d] */
    fa_heads_t q, q_out;      /* in and out: bf16 [B, H, N, d]; both pointers NULL: no queries */
    const int32_t *positions; /* device int32, as in fa_qk_rotary_t */
    int64_t pos_stride_b, pos_stride_n;
    const int32_t *seq;       /* device int32 [B]: table row of batch row b; NULL: row b */
    fa_rotary_t rotary;       /* rotary_dim 0 and norm 0: keys are stored as they come */
    int32_t B, H, N, reserved;
} fa_paged_append_t;

/*
 * Writes new tokens into the cache: k normed and turned as in fa_qk_rotary,
 * then stored (bf16 or e4m3, rounded once, e4m3 saturating at 448) at its
 * sequence's position, v stored as it is, and q normed and turned into q_out,
 * in one pass. e4m3 descales must have finite reciprocals (above 2^-128).
 * Token (b, n) goes to key positions[b][n] of table row seq[b].
 * A token with a negative position is padding: nothing of it is written, in
 * the cache or q_out. One whose sequence, page slot or page does not exist is
 * dropped from the cache (its q_out row is written). Two tokens of one call
 * must not go to the same slot. Slots that no token goes to are left as they
 * were. q_out may be q itself.
 */
int fa_paged_append(const fa_paged_append_t *args, void *stream);

typedef struct {
    fa_paged_cache_t cache;
    fa_block_table_t table;   /* row b: sequence b; num_seqs >= B */
    const void *q;            /* bf16 [B, H, d] view, 16-byte aligned, strides multiples of 8 */
    int64_t q_stride_b, q_stride_h;
    void *o;                  /* out, bf16 [B, H, d] contiguous */
    float *lse;               /* out, fp32 [B, H]: natural log, scale included */
    const int32_t *kv_len;    /* device int32 [B], clamped to [0, pages_per_seq * page_size] */
    int32_t B, H;             /* H a multiple of cache.H_kv */
    float scale;
    int32_t reserved;
} fa_paged_decode_t;

/*
 * Attention of one new token per sequence over its first kv_len[b] keys:
 * o = softmax(scale q K^T) V and lse, as fa_fwd_splitkv gives for Nq = 1 over
 * a contiguous cache. Query head h reads K/V head h / (H / H_kv). A sequence
 * with no visible key gets O = 0 and lse = -inf. The tiles of all sequences
 * are shared out evenly over the SMs, whatever the lengths; parts of a
 * sequence are joined by a second kernel by their log-sum-exp. Slots that are
 * not visible are never used in arithmetic: they may hold NaN. NaN and
 * infinities in visible keys, values or queries reach what they enter and
 * nothing else (the rows that read the key or hold the query, the value's
 * element of those rows); an infinity may give NaN there.
 * workspace: device memory owned by the caller, 16-byte aligned, at least
 * fa_paged_decode_workspace_bytes(B, H, H_kv, d) bytes (whatever the
 * lengths), overlapping nothing else, with no initialisation; two calls in
 * flight at once must not share it.
 */
int fa_paged_decode(const fa_paged_decode_t *args, void *workspace, size_t workspace_bytes,
                    void *stream);

/* Workspace bytes of fa_paged_decode; 0 if invalid or nothing to do. */
size_t fa_paged_decode_workspace_bytes(int B, int H, int H_kv, int d);

/*
 * Copies whole pages within the cache: page src[i] to page dst[i], all heads,
 * K and V, for i < n (device int32 arrays). It serves copy-on-write when
 * sequences fork and moves of live pages when a pool is compacted. A page may
 * be the source of several copies; no destination may appear twice or also be
 * a source (a pair with src[i] == dst[i] is allowed and changes nothing). A
 * pair with a page outside [0, num_pages) is skipped. n <= 2^31 / 128.
 */
int fa_copy_pages(const fa_paged_cache_t *cache, const int32_t *src, const int32_t *dst, int n,
                  void *stream);

#ifdef __cplusplus
}
#endif

#endif /* FA_PAGED_H_ */
