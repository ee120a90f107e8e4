/*
 * attn_cache.h -- C ABI of libattn, serving operators: rotary positions, a paged
 * key/value cache, and exact attention of new (drafted) tokens over that cache.
 *
 * Conventions are those of attn.h: every pointer inside the structs below that is
 * not marked HOST is a DEVICE pointer owned by the caller; calls are asynchronous on
 * `stream`; argument errors are returned before anything is launched; what only the
 * device can see (a slot or page number out of range, an inconsistent length) makes
 * the kernel leave that sequence or row alone and record ATTN_ERR_INVALID_ARG in the
 * device error word (attn_get_device_status).  Nothing here allocates beyond that
 * word, keeps a pointer, or reads the device back, so every call can be captured
 * into a graph once the library has been used on the device.
 */
#ifndef LIBATTN_ATTN_CACHE_H
#define LIBATTN_ATTN_CACHE_H

#include "attn.h"

#ifdef __cplusplus
extern "C" {
#endif

/* ------------------------------------------------------------ rotary positions
 * Pair i of the first `dim` values of a head, at position p, turns by p * f_i:
 *     (a, b) -> amplitude * (a cos - b sin, b cos + a sin).
 * The pairs are (i, i + dim/2), or (2i, 2i + 1) when `interleaved`.  The frequency is
 * given in turns per position as a 64-bit fixed-point fraction, turns[i] =
 * round(f_i / (2 pi) * 2^64): p * turns[i] modulo 2^64 is then the exact fraction of
 * a turn at any int32 position, however far.  The values behind `dim` pass through. */
typedef struct {
  const uint64_t* turns; /* [dim / 2] */
  int dim;               /* rotated values of a head: a multiple of 16, <= d */
  int interleaved;
  float amplitude; /* finite, > 0 */
} attn_rope_plan_t;

typedef enum { ATTN_BF16 = 0, ATTN_FP16 = 1, ATTN_FP32 = 2 } attn_type_t;

/* Rows of one tensor: head h of token n of batch b starts at element b * batch +
 * n * token + h * head (strides in elements, multiples of 16 bytes; a row is
 * contiguous).  src and dst are 16-byte aligned; they may be the same tensor, and
 * must not overlap otherwise. */
typedef struct {
  const void* src;
  void* dst;
  int heads;
  int64_t src_batch, src_token, src_head;
  int64_t dst_batch, dst_token, dst_head;
} attn_rows_t;

/*
 * Rotates `count` (1 or 2: q, or q and k) tensors of the same tokens in one launch.
 * inverse != 0: by the negative angles, which is the gradient (the amplitude stays).
 * Dense: B x N tokens.  Packed: cu_seqlens int32[B+1], N tokens in all; B <= 1024.
 * positions: int32 per token (b * N + n), any value; NULL: the token's index in its
 * sequence.  Packed tokens outside [cu_seqlens[0], cu_seqlens[B]) are left alone when
 * positions is NULL.
 * d: a multiple of 16, at most 256.
 */
ATTN_API attn_status_t attn_rope(const attn_rope_plan_t* plan, int inverse, attn_type_t type,
                                 const attn_rows_t* tensors, int count, int d, int B, int N,
                                 const int32_t* cu_seqlens, const int32_t* positions,
                                 attn_stream_t stream);

/* --------------------------------------------------------------- the paged cache
 * k, v: [layers, pages, page_size, heads, d], contiguous, 16-byte aligned, bf16 or (e4m3
 * != 0) E4M3 holding the real values divided by k_scale / v_scale.  Token p of slot s
 * lies in page page_table[s][p / page_size], row p % page_size, in every layer.
 * refs[page] counts the slots that hold a page; 0 means free.  A slot of lens[s]
 * tokens holds exactly ceil(lens[s] / page_size) pages; entries behind those are not
 * read.  Slots share full pages (attn_cache_fork copies one that is not full).
 * Tokens in a shared page are shared: fork a slot when its tokens have been appended.  A slot that
 * attn_cache_compact cuts back inside a shared page keeps it; attn_cache_alloc gives it a page of its
 * own, the tokens copied, before it grows.
 * page_size: a power of two from 16 to 1024; d 64 or 128; slots <= 8192.
 * Page operations (alloc, free, fork, copy, compact) that share a cache must not run
 * at the same time: issue them on one stream. */
typedef struct {
  void* k;
  void* v;
  int32_t* page_table; /* [slots, max_pages] */
  int32_t* lens;       /* [slots] */
  int32_t* refs;       /* [pages] */
  int layers, pages, page_size, heads, d;
  int slots, max_pages;
  int e4m3;
  float k_scale, v_scale;
} attn_cache_t;

/*
 * Grows slot slots[i] to new_lens[i] >= lens tokens, i < n <= 8192.  Pages are handed out
 * in order of i, lowest page number first; request i is granted (granted[i] = 1) iff
 * it needs no page or the pages needed by requests 0..i do not exceed the free ones.  A slot
 * that grows inside a page which another slot holds too needs one more, in place of that page, whose
 * tokens are copied in every layer.  One not granted changes nothing.  A slot named twice, a shorter length or one
 * beyond max_pages: not granted (the first of two counts), error recorded.
 */
ATTN_API attn_status_t attn_cache_alloc(const attn_cache_t* cache, const int32_t* slots,
                                        const int32_t* new_lens, int n, int32_t* granted,
                                        attn_stream_t stream);

/* Empties the slots: their pages lose a reference, their table entries become -1, lens 0.
 * A slot that is empty, or named again, is a no-op.  Here, and where attn_cache_compact releases pages, a page
 * number out of range is taken from the table like the others, error recorded. */
ATTN_API attn_status_t attn_cache_free(const attn_cache_t* cache, const int32_t* slots, int n,
                                       attn_stream_t stream);

/*
 * Forks slot src[i] into the empty slot dst[i], i < n <= 8192: full pages are shared
 * (refs + 1), the tokens of a last page that is not full are copied, in every layer, to
 * a new page (handed out as by attn_cache_alloc).  granted as there; a destination
 * that holds tokens, equals its source or is named twice is refused, error recorded, and so is a source
 * with a page out of range (whose copy's page counts as needed in this call).
 * workspace: attn_cache_fork_workspace_size(n) bytes, 16-byte aligned.
 */
ATTN_API attn_status_t attn_cache_fork(const attn_cache_t* cache, const int32_t* src,
                                       const int32_t* dst, int n, int32_t* granted,
                                       void* workspace, size_t workspace_bytes,
                                       attn_stream_t stream);
ATTN_API size_t attn_cache_fork_workspace_size(int n);

/* Copies page src[i] to page dst[i] in every layer, i < n, whatever holds them.  Of a
 * destination named twice the last copy counts.  A source that another copy writes is
 * refused (that copy is left out, error recorded). */
ATTN_API attn_status_t attn_cache_copy(const attn_cache_t* cache, const int32_t* src,
                                       const int32_t* dst, int n, attn_stream_t stream);

/*
 * Keeps the accepted path of each sequence's drafted tokens.  The last n_b = cu_q[b+1] -
 * cu_q[b] tokens of slot slots[b] (NULL: slot b) are drafted; path[b][0..accepted[b])
 * names, strictly increasing, which of them stay.  In every layer they move together
 * behind the context, lens becomes context + accepted[b], and pages behind the new end
 * lose a reference.  A sequence whose path is not valid, or whose tokens would move into a
 * page that another slot holds too, is left alone, error recorded, and so is the second
 * of two sequences with the same slot.  B <= 1024.
 */
ATTN_API attn_status_t attn_cache_compact(const attn_cache_t* cache, const int32_t* cu_q,
                                          const int32_t* path, int path_width,
                                          const int32_t* accepted, const int32_t* slots, int B,
                                          attn_stream_t stream);

/*
 * Writes new tokens into the cache and rotates their queries, in one launch.  Token t of
 * sequence b (cu_q int32[B+1], T tokens packed, B <= 1024) belongs at position lens -
 * n_b + t of its slot: alloc first, then append.  plan NULL: nothing is rotated.
 * positions: int32[T], the rotary position (a drafted token's depth behind its context);
 * NULL: the token's place in the cache.  q, k: rows of bf16 (batch strides unused); q->dst
 * receives the rotated queries (q may be NULL); k->dst and v->dst are not used.  Rotated keys
 * and values are rounded once, to the cache's type (E4M3: divided by the scale, saturated).  Of a
 * token that has no row in the cache (error recorded) the query is left alone too; of two
 * sequences with one slot the second is refused so.
 */
ATTN_API attn_status_t attn_rope_append(const attn_cache_t* cache, int layer,
                                        const attn_rope_plan_t* plan, const attn_rows_t* q,
                                        const attn_rows_t* k, const attn_rows_t* v, int B, int T,
                                        const int32_t* cu_q, const int32_t* slots,
                                        const int32_t* positions, attn_stream_t stream);

/*
 * Exact attention of each sequence's last n_b tokens over its slot of the cache, those
 * tokens included (append first).  q, o: [T, Hq, d] bf16, contiguous, packed by cu_q
 * int32[B+1], B <= 1024; lse: [Hq, T] fp32.  Query head h reads cache head h / (Hq /
 * heads); Hq / heads at most 128.  Every token sees the whole context (the tokens before
 * the last n_b).  Among the drafted tokens, token t sees token j iff mask[t][j] != 0
 * (mask: one byte each, [T, mask_width], t counted over the batch, j within its sequence;
 * n_b <= mask_width <= 256), or j <= t when mask is NULL.  A token that sees nothing gets
 * O = 0 and LSE = -inf; one that sees a score which is not a number gets NaN in both.  n_b = 0 is fine; rows outside [cu_q[0], cu_q[B]) are left alone.
 * What pages hold behind a sequence's end never counts; a key that no token of its sequence
 * sees may hold anything, but values of a sequence's own tokens must be finite.  A cu_q
 * that decreases or leaves [0, T] makes the whole call do nothing (error recorded).
 * Rows that would read a page out of range are left alone (error recorded).
 * An E4M3 cache is read as it is.  Queries keep 2^-17 of their row's largest value (the sum of two
 * E4M3 terms).  A probability keeps 2^-8 of itself, as in a bf16 cache, down to 2^-20 of its row's
 * largest one, and 2^-28 of that below (the sum of three E5M2 terms).
 * Unsupported: (B + T Hq / heads / 256) heads items of (max_pages page_size / 128) key tiles each that might
 * come to more than about 3e8 tiles.
 * workspace: attn_tree_workspace_size(d) bytes (42 MB for d 128, 21 for 64, whatever the call), 256-byte
 * aligned; calls that run at the same time need one each.  Results do not depend on timing: the same call is bitwise
 * repeatable.
 */
ATTN_API attn_status_t attn_tree_fwd(const attn_cache_t* cache, int layer, const void* q, void* o,
                                     float* lse, int Hq, int B, int T, const int32_t* cu_q,
                                     const int32_t* slots, const uint8_t* mask, int mask_width,
                                     float scale, void* workspace, size_t workspace_bytes,
                                     attn_stream_t stream);
ATTN_API size_t attn_tree_workspace_size(int d);

#ifdef __cplusplus
}
#endif
#endif /* LIBATTN_ATTN_CACHE_H */
