/*
 * samspec_kv.h -- C ABI of libsamspec.so, second part: the paged key/value
 * cache of the target model and the attention of a verification pass.
 *
 * samspec.h drafts tokens and verifies them against the target's logits; the
 * entry points here serve the target's own pass between the two.  "SAM投机推理：
 * 长序列强化学习训练加速利器" §2.1 compares a normal and a verification form of
 * paged attention; the pages describe neither, so the formulas stand below.
 * The conventions of samspec.h hold: d_ pointers are device pointers, the
 * caller owns all memory, calls are asynchronous on `stream` and return
 * SAMSPEC_OK or a negative code before any launch, conditions found on the
 * device are status words, one per sequence, and nothing traps.
 */
#ifndef SAMSPEC_KV_H_
#define SAMSPEC_KV_H_

#include "samspec.h"

#ifdef __cplusplus
extern "C" {
#endif

/* element type of the cache besides SAMSPEC_BF16 */
#define SAMSPEC_F16 2

/* status words besides those of samspec.h */
#define SAMSPEC_ST_PAGE 10 /* a sequence's page table or counts do not fit the pool */
#define SAMSPEC_ST_ROW 11  /* a row outside the cache, named twice in one call, or  */
                           /* not empty where it has to be                          */

/* =========================================================================
 * Paged key/value cache of the target model: what a verification pass writes
 * and reads, and what follows its outcome.
 *
 * `kv_cache` describes tensors that the caller holds (device pointers):
 *   k, v       [layers, n_pages, kv_heads, page, head_dim] of dtype (BF16 or
 *              F16), 16-byte aligned
 *   table      [seqs, max_pages] int32: the pages of each sequence in order;
 *              token t lies in slot t % page of page table[t / page]
 *   lens       [seqs] int32: committed tokens
 *   held       [seqs] int32: pages held (the first entries of the table row);
 *              held * page >= lens
 *   refs       [n_pages] int32: how many table rows hold the page
 *   free_bits  [ceil(n_pages / 32)]: bit p % 32 of word p / 32 is set exactly
 *              where refs[p] is 0
 * An empty cache has lens, held and refs 0, free_bits set for every page below
 * n_pages, and any table.  Sequences that share pages (kv_fork) never write
 * to them: kv_reserve copies a shared page before it is appended to.
 * Limits: page 16, 32, 64 or 128; head_dim 64 or 128; 1 <= kv_heads <= 1024;
 * 1 <= layers; seqs, max_pages <= 2^20; max_pages * page < 2^30; n_pages *
 * layers and n_pages * kv_heads * page < 2^31.
 *
 * Calls name n sequences by d_rows [n] (NULL: 0 .. n-1), each at most once;
 * d_status [n] (may be NULL) receives ST_OK or why a sequence was left as it
 * was (ST_ROW, ST_PAGE, ST_CAPACITY, ST_BADDRAFT), while the others proceed.
 * Every call is asynchronous on `stream`, allocates nothing and may be
 * captured in a graph.  Calls on one cache are ordered by their stream.
 * ========================================================================= */
typedef struct kv_cache {
  void* k;
  void* v;
  int32_t* table;
  int32_t* lens;
  int32_t* held;
  int32_t* refs;
  uint32_t* free_bits;
  int32_t dtype, layers, n_pages, page, kv_heads, head_dim, seqs, max_pages;
} kv_cache;

/* Room for n_tok[i] more tokens behind lens[row i] (d_n_tok NULL: N for all;
 * 0 <= n_tok[i] <= N).  Pages are taken lowest number first, in the order of
 * the call's sequences and of their positions; a sequence whose share of the
 * free pages is gone, or whose table row is too short, gets ST_CAPACITY (so
 * does each later one that needs more pages than are left after those before
 * it).  Where the last page is partly filled and held by others too, its
 * filled slots are copied to a page of the sequence's own, in all layers
 * (whatever n_tok[i] is, 0 included).
 * Workspace: kv_reserve_workspace_bytes bytes, 16-byte aligned, any content,
 * not shared by two calls in flight.  Two launches. */
size_t kv_reserve_workspace_bytes(const kv_cache* cache, int32_t n);
int kv_reserve(const kv_cache* cache, const int32_t* d_rows, int32_t n, int32_t N,
               const int32_t* d_n_tok, int32_t* d_status, void* d_workspace, size_t ws_bytes,
               samspec_stream_t stream);

/* Sequence d_dst[i] (empty, holding no page) becomes a copy of d_src[i]'s
 * committed tokens by sharing their pages.  d_dst are distinct and none of
 * them is a source; a source may be named many times.  One launch. */
int kv_fork(const kv_cache* cache, const int32_t* d_src, const int32_t* d_dst, int32_t n,
            int32_t* d_status, samspec_stream_t stream);

/* What follows verification.  A sequence's N new tokens (or nodes of its draft
 * tree, node 0 first) lie in slots lens .. lens + N - 1.  With a =
 * d_accept_len[i] (-1 .. N - 1, as spec_verify and spec_verify_tree write it)
 * slot lens + 1 + t receives the key and value of slot lens + d_path[i, t]
 * for t < a, in all layers; lens grows by 1 + a, and pages wholly behind it
 * are released.  d_path [n, N] (N <= 32) as spec_verify_tree writes it:
 * strictly increasing node numbers; NULL: a chain, nothing moves.  a = -1
 * keeps no new token.  With a path the pages written have to be the
 * sequence's alone (ST_CAPACITY; kv_reserve sees to it), and d_status must be
 * given.  One launch without a path, two with one. */
int kv_commit(const kv_cache* cache, const int32_t* d_rows, int32_t n, int32_t N,
              const int32_t* d_accept_len, const int32_t* d_path, int32_t* d_status,
              samspec_stream_t stream);

/* Cuts sequences to min(lens, d_new_len[i]) tokens (NULL: 0) and releases the
 * pages behind, reserved ones among them.  One launch. */
int kv_truncate(const kv_cache* cache, const int32_t* d_rows, int32_t n,
                const int32_t* d_new_len, int32_t* d_status, samspec_stream_t stream);

/* The plan of one pass over n sequences with up to N new tokens each: read by
 * kv_append and kv_attend of every layer.  Sequence i has n_tok[i] of them
 * (NULL: N), a chain, or (d_first_child / d_next_sibling [n, N], N <= 32, as
 * for spec_verify_tree, n_tok ignored) a tree of N nodes: token j sees the
 * committed tokens and, of the new ones, 0 .. j of a chain, or node j and its
 * ancestors.  Its position is lens + j, or lens + depth.  d_group [n] (may be
 * NULL): consecutive sequences of the same number form a group; the pages
 * that the table rows of all its sequences begin with are read once for the
 * whole group (sequences without tokens, or with a status, count for nothing in
 * it).  Grouping changes no result beyond rounding.  Slots must have
 * been reserved (ST_CAPACITY).  d_plan: kv_plan_bytes bytes, 256-byte
 * aligned, any content; it starts with the n status words, and holds the
 * workspace of kv_attend: one kv_attend at a time may use a plan (grouped:
 * non-zero where d_group is given, which takes more of it).  kv_attend is
 * given the same plan_bytes, n, N and q_heads as kv_plan, and it and kv_append
 * a cache of the same sizes (but for layers and n_pages) and table.  A plan holds until
 * the cache's lengths or tables change.  Limits: n <= 2^20, N <= 2^16, q_heads
 * a multiple of kv_heads, at most 64 times as many, n * N * q_heads < 2^30
 * (with groups 2^29), and what the units of work may cost below 2^31: units *
 * ((max_pages * page / 128 + 2) * 2 + 5) * kv_heads, by the table's width,
 * however short the sequences are.  A unit is up to 2 * floor(128 / rep) tokens
 * of a sequence, rep = q_heads / kv_heads; with groups ceil(n * N / those) + n
 * units more count.  (Tables of a million tokens and 8 key heads: 16,000
 * sequences of one unit each, 8,000 with groups.)  A grouped plan holds two fp32
 * results of every query row besides, 2 * n * N * q_heads * (4 * head_dim + 8)
 * bytes: 1 GB for 8 sequences of 4000 tokens and 32 heads of 128. */
size_t kv_plan_bytes(const kv_cache* cache, int32_t n, int32_t N, int32_t q_heads,
                     int32_t grouped);
int kv_plan(const kv_cache* cache, const int32_t* d_rows, int32_t n, int32_t N, int32_t q_heads,
            const int32_t* d_n_tok, const int32_t* d_first_child, const int32_t* d_next_sibling,
            const int32_t* d_group, void* d_plan, size_t plan_bytes, samspec_stream_t stream);

/* Puts the new tokens' keys and values into their slots of one layer and turns
 * queries and keys to their positions: pair j of the first `rot` elements of
 * a head is rotated by position * d_inv_freq[j] radians (fp64 [rot / 2]; the
 * angle is reduced exactly, whatever the position) and scaled by mscale.
 * layout: pairs (j, j + rot / 2) for SAMSPEC_ROPE_HALF, (2j, 2j + 1) for
 * SAMSPEC_ROPE_INTERLEAVED.  rot = 0: no rotation.  d_q [n, N, q_heads,
 * head_dim] -> d_q_out (contiguous; may be d_q; both may be NULL), d_k and
 * d_v [n, N, kv_heads, head_dim]; *_stride: elements from one token to the
 * next (tokens of consecutive sequences follow one another; a multiple of 8).
 * All of the cache's dtype, 16-byte aligned.  Tokens beyond n_tok, or of a
 * sequence with a status, write nothing to the cache and zeros to d_q_out.
 * One launch. */
#define SAMSPEC_ROPE_HALF 0
#define SAMSPEC_ROPE_INTERLEAVED 1
int kv_append(const kv_cache* cache, int32_t layer, const void* d_plan, int32_t n, int32_t N,
              int32_t q_heads, const void* d_q, int64_t q_stride, void* d_q_out, const void* d_k,
              int64_t k_stride, const void* d_v, int64_t v_stride, const double* d_inv_freq,
              int32_t rot, int32_t layout, float mscale, samspec_stream_t stream);

/* Attention of the pass on one layer: d_out [n, N, q_heads, head_dim]
 * (contiguous, 32-byte aligned, the cache's dtype) = softmax(scale * q k^T) v over the keys that
 * each token sees (query head h reads key head h / (q_heads / kv_heads)),
 * scale positive and finite.
 * Scores, softmax and sums in fp32; the probabilities are rounded to the
 * cache's dtype for the product with v.  Keys and values outside a token's
 * sight never reach it, whatever they hold (infinities and NaN included).  A
 * query all of whose scores are -infinity gets zeros.
 * Tokens beyond n_tok, or of a sequence with a status, get zeros. */
int kv_attend(const kv_cache* cache, int32_t layer, void* d_plan, size_t plan_bytes, int32_t n,
              int32_t N, int32_t q_heads, const void* d_q, int64_t q_stride, float scale,
              void* d_out, samspec_stream_t stream);

/* Test hook of kv_attend's bounded waits, as samspec_set_wait_limit_ns is of
 * the verification kernels': every on-chip wait gives up after `ns`
 * nanoseconds (0: the default 2 s).  A kernel whose wait runs out sets
 * ST_TIMEOUT in the plan's status of the sequences that it was working on (their outputs
 * are undefined), waits for its copies and matrix products in flight (all of
 * them, whichever wait ran out; up to 2 s each) and returns; the context stays
 * usable.  Process-wide, for launches
 * after the call.  Returns the previous limit. */
uint64_t kv_set_wait_limit_ns(uint64_t ns);

#ifdef __cplusplus
}
#endif

#endif /* SAMSPEC_KV_H_ */
