/*
 * bsmt_serving.h: the part of libbsmt's C ABI that prepares q and k and serves
 * from a cache: rotary positions, a paged cache of keys and values in 8 bits,
 * and attention over it. The conventions of bsmt.h hold for every entry point
 * here (status codes and messages, caller-owned memory, streams, the device
 * status word, no exceptions). The pages behind the library have no
 * counterpart of these calls.
 */
#ifndef BSMT_SERVING_H
#define BSMT_SERVING_H

#include "bsmt.h"

#ifdef __cplusplus
extern "C" {
#endif

/* ------------------------------------------------------- rotary positions
 * Rotary positions with several axes (time, height, width for images and
 * video; one axis for text), applied to q and k before attention. Pair i of
 * a head's first 2 * num_pairs elements, (a, b) = (x[i], x[i + num_pairs])
 * or, interleaved, (x[2i], x[2i + 1]), turns by the angle
 * t_i = pos[axis[i]] * inv_freq[i]:
 *   a' = a cos t_i - b sin t_i,   b' = a sin t_i + b cos t_i.
 * Elements behind the pairs pass through. With inverse != 0 the angle is
 * -t_i: the gradient of the map, which is orthogonal. The angle is reduced
 * modulo a turn in 64-bit integer arithmetic, so positions of any int32
 * value, negative ones too, keep full accuracy. */
#define BSMT_MAX_ROTARY_PAIRS 128
enum { BSMT_BF16 = 0, BSMT_FP32 = 1 };

typedef struct bsmt_rotary_spec {
    int32_t head_dim;
    int32_t num_pairs;    /* 1 .. BSMT_MAX_ROTARY_PAIRS, 2 * num_pairs <= head_dim */
    int32_t num_axes;     /* 1 .. 127 */
    int32_t interleaved;  /* 0: pairs (i, i + num_pairs); 1: pairs (2i, 2i + 1) */
    double inv_freq[BSMT_MAX_ROTARY_PAIRS];  /* radians a position; finite */
    int8_t axis[BSMT_MAX_ROTARY_PAIRS];      /* 0 .. num_axes - 1 */
} bsmt_rotary_spec;

/* Fills a spec with sections[a] >= 0 consecutive pairs for axis a. inv_freq is
 * base^(-i / pairs) over all pairs in one ladder, or with per_axis != 0
 * base^(-j / sections[a]) over each axis's own. base > 0. Host-only. */
bsmt_status bsmt_rotary_sections(int32_t head_dim, const int32_t* sections, int32_t num_sections, double base,
                                 int32_t per_axis, int32_t interleaved, bsmt_rotary_spec* out);

/* One tensor [B, heads, T, head_dim] in device memory, its innermost
 * dimension contiguous, the other strides any (in elements; batch, head,
 * token). `out` may be `in` with the same strides, and must not overlap it
 * otherwise. */
typedef struct bsmt_rotary_tensor {
    const void* in;
    void* out;
    int64_t in_strides[3];
    int64_t out_strides[3];
    int32_t heads;
} bsmt_rotary_tensor;

/* Turns one or two tensors (q and k: their heads may differ in number) that
 * share B, T and positions.
 *   dtype      BSMT_BF16 or BSMT_FP32, of every tensor. The arithmetic is
 *              fp32; the result is rounded once.
 *   positions  device int32, element (axis, b, t) at axis * position_strides[0]
 *              + b * position_strides[1] + t * position_strides[2]
 * Rows that are 16-byte aligned (pointers and strides) with num_pairs a
 * multiple of 8 move in 16-byte pieces; others element by element. */
bsmt_status bsmt_rotary(const bsmt_rotary_spec* spec, int32_t dtype, int64_t B, int64_t T, const int32_t* positions,
                        const int64_t position_strides[3], int32_t inverse, const bsmt_rotary_tensor* tensors,
                        int32_t num_tensors, void* stream);

/* ------------------------------------------------- paged cache in 8 bits
 * Keys and values of many sequences, held as 8-bit codes in pages of
 * page_size tokens. A value is code * scale, with one scale for each
 * (layer, page, kv head) of k and of v, always a power of two as the library
 * writes it: the smallest 2^e (e >= -120) with amax <= top * 2^e, top = 448
 * (e4m3) or 127 (int8). Every step but the rounding to a code is then exact.
 *
 *   k, v        codes [num_layers, num_pages, num_kv_heads, page_size, head_dim]
 *   k_scale, v_scale  float [num_layers, num_pages, num_kv_heads]
 *   page_table  int32 [max_seqs, max_pages]: the pages of each sequence
 *               (a slot of the table), in order; entries behind its length
 *               are not read
 *   seq_lens    int32 [max_seqs]: tokens of each sequence (0: an empty slot)
 *   ref_counts  int32 [num_pages]: sequences that hold the page (0: free)
 * All contiguous device memory owned by the caller; k, v and ref_counts
 * 16-byte aligned. An empty cache has seq_lens and ref_counts all 0. The
 * layers share table, lengths and counts.
 *
 * Conditions that the calls below keep: a page is in use exactly when its
 * count is the number of table rows that hold it, and a page that several
 * sequences share is full. Lists of sequences (device int32) may hold -1:
 * an entry to be passed over, so that a padded batch of fixed size can be
 * captured into a CUDA graph once. Pages are handed out lowest first, in
 * the order of the list, so a call's result does not depend on timing.
 *
 * Offsets (cu_seqlens) begin at 0; where they do not, the tokens in front of
 * the first belong to no sequence, and the call reports
 * BSMT_ERR_DEVICE_PRECONDITION.
 *
 * Calls on one cache must not overlap in time, except reads (gather,
 * attention) with reads. head_dim is 64 or 128, page_size 16, 32, 64 or 128,
 * max_seqs at most 2^18, max_pages * page_size below 2^31 - 256
 * (BSMT_ERR_UNSUPPORTED otherwise). */
enum { BSMT_CACHE_E4M3 = 0, BSMT_CACHE_INT8 = 1 };

typedef struct bsmt_kv_cache {
    void* k;
    void* v;
    float* k_scale;
    float* v_scale;
    int32_t* page_table;
    int32_t* seq_lens;
    int32_t* ref_counts;
    int32_t num_layers, num_pages, num_kv_heads, page_size, head_dim;
    int32_t max_seqs, max_pages;
    int32_t dtype; /* BSMT_CACHE_* */
} bsmt_kv_cache;

/* Workspace bytes of bsmt_cache_extend, bsmt_cache_fork (n entries) and
 * bsmt_cache_compact (n = 0). Only num_pages is read. Host-only. The
 * workspace is caller-owned device memory, 256-byte aligned, not zeroed,
 * reusable once the stream has passed the call. */
bsmt_status bsmt_cache_workspace_bytes(const bsmt_kv_cache* cache, int64_t n, int64_t* bytes);

/* Grows n sequences: seqs[i] by counts[i] >= 0 tokens (counts NULL: by 1
 * each). Writes the old length to starts[i] (-1 for an entry that is passed
 * over), takes pages for the new tokens and sets the new length; the new
 * tokens' codes are written by bsmt_cache_write. All or nothing: with too few
 * free pages or places in a table row (BSMT_ERR_DEVICE_CAPACITY), a sequence
 * listed twice, a negative count, or a partial last page that others hold
 * too (BSMT_ERR_DEVICE_PRECONDITION), or a sequence, length or page out of
 * range (BSMT_ERR_DEVICE_BOUNDS), nothing changes and every start is -1, so
 * that a bsmt_cache_write of the same step writes nothing. */
bsmt_status bsmt_cache_extend(const bsmt_kv_cache* cache, const int32_t* seqs, const int32_t* counts, int64_t n,
                              int32_t* starts, void* workspace, int64_t workspace_bytes, void* stream);

/* Quantises keys and values into the pages: token t of the call, with
 * cu_seqlens[i] <= t < cu_seqlens[i + 1], goes to position
 * starts[i] + t - cu_seqlens[i] of sequence seqs[i], in layer `layer`.
 *   k, v        device bf16, element (t, head, d) at t * strides[0] + head * strides[1] + d;
 *               16-byte aligned, strides multiples of 8 elements
 *   cu_seqlens  device int32 [n + 1], from 0, not decreasing, at most T; NULL:
 *               one token each (T = n). Tokens at or past the last offset are
 *               not read.
 * A page's scale comes from its first write (at row 0) and grows when later
 * tokens need a larger one; the codes that the page holds before them are
 * then rounded anew to the larger scale. So tokens are written once, in
 * order; writing the same call again gives the same cache. Infinities are
 * stored as the largest code; NaN stays NaN in e4m3, and is stored as 0 in
 * int8, which has none, with BSMT_ERR_DEVICE_PRECONDITION. Neither takes
 * part in the scale. An entry with seqs[i] or starts[i] = -1 is passed over.
 * Positions past the sequence's length and pages out of range are not written
 * (BSMT_ERR_DEVICE_BOUNDS), pages held by another sequence too or by none
 * are not written (BSMT_ERR_DEVICE_PRECONDITION). A sequence may be listed
 * once in a call: two entries that meet in a page would race for its scale
 * (bsmt_cache_extend refuses such a list). */
bsmt_status bsmt_cache_write(const bsmt_kv_cache* cache, int32_t layer, const int32_t* seqs, const int32_t* starts,
                             int64_t n, const int32_t* cu_seqlens, const void* k, const void* v, int64_t T,
                             const int64_t k_strides[2], const int64_t v_strides[2], void* stream);

/* The reverse: k and v, device bf16 [T, num_kv_heads, head_dim] contiguous and
 * 16-byte aligned, of the positions starts[i] + t - cu_seqlens[i] (starts
 * NULL: from 0), for instance to run bsmt_flex_attention_fwd_packed over a
 * prompt's cached part. code * scale is exact in bf16 (while in its range).
 * Rows of entries with seqs[i] or starts[i] = -1, rows past the last offset
 * and rows of positions or pages out of range (BSMT_ERR_DEVICE_BOUNDS) are 0,
 * and so are rows in front of the first offset. */
bsmt_status bsmt_cache_gather(const bsmt_kv_cache* cache, int32_t layer, const int32_t* seqs, const int32_t* starts,
                              int64_t n, const int32_t* cu_seqlens, int64_t T, void* k, void* v, void* stream);

/* Forks n sequences: dst[i], an empty slot, becomes a copy of src[i]. Full
 * pages are shared (their counts grow); a partial last page is copied, in
 * every layer, to a page taken for the child. A parent may be listed many
 * times, a child once. All or nothing as bsmt_cache_extend; a child that is
 * not empty or listed twice is BSMT_ERR_DEVICE_PRECONDITION. (A number out of
 * range among a parent's full pages is copied as it stands and reported.) */
bsmt_status bsmt_cache_fork(const bsmt_kv_cache* cache, const int32_t* src, const int32_t* dst, int64_t n,
                            void* workspace, int64_t workspace_bytes, void* stream);

/* Empties n sequences: their pages' counts fall by one (at 0 the page is
 * free), their table entries become -1, their lengths 0. Emptying an empty
 * slot, or one twice, does nothing. Entries out of range are passed over and
 * reported (BSMT_ERR_DEVICE_BOUNDS); a page that is free already keeps its
 * count of 0 (BSMT_ERR_DEVICE_PRECONDITION). */
bsmt_status bsmt_cache_free(const bsmt_kv_cache* cache, const int32_t* seqs, int64_t n, void* stream);

/* Moves the pages in use to the front of the pool, [0, live): those at or
 * behind `live` go, in order, to the free places before it, codes, scales
 * and counts in every layer, and the table's entries follow. Writes live, the
 * number of pages in use, to live[0] (device int32): a caller can then give
 * back the pool's end. */
bsmt_status bsmt_cache_compact(const bsmt_kv_cache* cache, int32_t* live, void* workspace, int64_t workspace_bytes,
                               void* stream);

/* Attention of each sequence's newest tokens over its cached keys and values:
 *   out[t, hq, :] = softmax_j(mod(scale * q[t, hq] . k_j) masked) @ v
 * where query t of sequence seqs[i] (cu_seqlens_q[i] <= t < cu_seqlens_q[i+1])
 * has position q_idx = seq_lens - (cu_seqlens_q[i+1] - t): the queries are the
 * sequence's last tokens, already extended and written, and j runs over its
 * positions kv_idx in [0, seq_lens).
 *   q     device bf16 [T, Hq, head_dim], contiguous, 16-byte aligned
 *   cu_seqlens_q  device int32 [n + 1], from 0, not decreasing, at most T;
 *         NULL: one query each (T = n)
 *   mask_spec  a mask program over (q_idx, kv_idx) (NULL: none). Pages that no
 *         query of the sequence sees are not read, so a window with sink
 *         tokens costs the window. DOCUMENT is BSMT_ERR_UNSUPPORTED: a
 *         sequence is one document.
 *   score, scale, enable_gqa  as for bsmt_flex_attention_fwd; Hkv is the cache's
 *   out   device bf16 [T, Hq, head_dim], 16-byte aligned
 *   lse   device float [Hq, T]
 *   workspace  caller-owned device memory, 256-byte aligned, of
 *         bsmt_paged_attention_workspace_bytes bytes; written and read back by
 *         the call, need not be zeroed. Calls that share one must not overlap.
 * Rows that see no key (an empty sequence, a mask that leaves nothing, an
 * entry with seqs[i] = -1, tokens outside the offsets) get out = 0 and
 * lse = -inf. A page out of range counts as keys of value 0 and is reported
 * (BSMT_ERR_DEVICE_BOUNDS), as is a sequence out of range. Codes behind a
 * sequence's end and NaN codes that the mask hides do not reach the result.
 * V scales may differ by up to 2^100 within a sequence. Made for few queries
 * a sequence (a row is one query of one head of a kv head's group; rows are
 * taken 8 or 16 at a time, with a head_dim of 64 also 32, and each such tile
 * reads the keys again, from L2 mostly); the result does not depend on timing. */
bsmt_status bsmt_paged_attention_workspace_bytes(int64_t D, int64_t* bytes);
bsmt_status bsmt_paged_attention(const void* q, int64_t T, int64_t Hq, const bsmt_kv_cache* cache, int32_t layer,
                                 const int32_t* seqs, int64_t n, const int32_t* cu_seqlens_q,
                                 const bsmt_mask_spec* mask_spec, const bsmt_score_spec* score, float scale,
                                 int32_t enable_gqa, void* out, float* lse, void* workspace, int64_t workspace_bytes,
                                 void* stream);

#ifdef __cplusplus
}
#endif
#endif /* BSMT_SERVING_H */
