/*
 * hstu_cache.h -- C ABI of the paged 4-bit history cache (B200, sm_100a).
 *
 * Serving keeps every user's history cached between requests and computes only
 * the new rows: new history events, and candidates scored against the cached
 * history (HSTU notes "Actions Speak Louder than Words", section 2.6,
 * M-FALCON with cached keys and values).  Four operations:
 *
 *   hstu_cache_plan    pages, slots and lengths of a step, on the device
 *   hstu_cache_append  K/V rows quantised to 4 bits into their slots
 *   hstu_cache_read    rows of given slots back as bf16
 *   hstu_cache_attend  SLA HSTU attention of the new rows over the cache
 *
 * Rows in 4 bits.  A row x of d values (one token, one head, K or V) is held
 * as d codes 0..15 with a step s and a minimum m, both bf16:
 *     m = min x,  s = bf16((max x - min x) / 15), taken as 0 below 2^-126,
 *     code_i = round((x_i - m) * (1 / s)) in 0..15  (0 for s = 0),
 *     x_i ~ m + s code_i,
 * each step of it rounded to fp32, ties to even.  (The keys and values of an
 * HSTU layer are SiLU outputs: nearly all of a row's range lies above zero, so
 * a minimum per row uses all 16 codes where a symmetric grid would use half.)
 * A row that holds a NaN or an infinity, or whose range passes fp32's, is held
 * as NaN (m and s NaN, codes 0).
 *
 * Pages.  A page holds page_size (16, 32 or 64) tokens of every head; head h
 * of page p is the block of page_size * (d + 8) bytes at
 * pages + p * page_stride + h * page_size * (d + 8):
 *   K codes   [page_size][d / 2]  32-bit word w of a token has its dims
 *             8w .. 8w + 7, nibble n (bits 4n..4n+3) being dim
 *             8w + 2 (n mod 4) + n / 4
 *   V codes   [d / 2][page_size]  byte (i, .) has dims 2i (low nibble) and
 *             2i + 1 of one token, each group of four tokens in the order
 *             0, 2, 1, 3
 *   K pairs   [page_size] (s, m) bf16 each
 *   V pairs   [page_size] (s, m)
 * (so that a tensor-core fragment's two adjacent values come out of one word
 * by one shift and one and-or, for K along d and for V along the tokens).
 *
 * Conventions are those of hstu_sla.h: device pointers, caller-owned buffers,
 * asynchronous on `stream`, HSTU_SLA_* return codes, no traps.  One set of
 * tables serves every layer of a model (the layers' histories have the same
 * lengths); each layer has its own pages.  Calls that use one set of tables are
 * ordered by the caller: plan, then the layers' appends and attends.
 */
#ifndef HSTU_CACHE_H_
#define HSTU_CACHE_H_

#include "hstu_sla.h"

#ifdef __cplusplus
extern "C" {
#endif

/* The tables of a cache of B sequences (user slots) and num_pages pages; all
 * pointers are device int32, 4-byte aligned.
 *   status       [1] 0, or the HSTU_SLA_ERR_* code of the first failed call
 *                since the last plan: plan sets it afresh, the other calls do
 *                nothing while it is set and set it on bad input
 *   free_count   [1] pages on the free stack
 *   lengths      [B] tokens cached per sequence
 *   free_pages   [num_pages] the stack; entries [0, free_count) are free
 *   block_table  [B][max_pages] page of a sequence's tokens
 *                [i page_size, (i + 1) page_size) at entry i */
typedef struct {
  int32_t B;          /* 1 .. 2^30 */
  int32_t max_pages;  /* per sequence, 1 .. 2^19 */
  int32_t num_pages;  /* >= 1 */
  int32_t page_size;  /* 16, 32 or 64 */
  int32_t* status;
  int32_t* free_count;
  int32_t* lengths;
  int32_t* free_pages;
  int32_t* block_table;
} hstu_cache_tables;

/* Workspace of hstu_cache_plan: 256-byte aligned, contents need not be
 * initialised.  0: the call needs none (NULL will do), or the arguments are
 * invalid. */
size_t hstu_cache_plan_workspace_bytes(int32_t B, int64_t total_tokens);

/* One step's plan.  Sequence b brings the rows [seq_offsets[b],
 * seq_offsets[b + 1]) of the step's batch, the last num_targets[b] of them
 * candidates (NULL = none), which are not cached.  In the order of the
 * sequences: a sequence with release[b] != 0 (NULL = none) first gives all its
 * pages back (they go on top of the free stack, entry by entry) and its length
 * becomes 0; then every sequence takes the pages its new history rows need off
 * the top of the stack, one by one; its block-table entries and length are
 * written.  slots[t] (device int64 [total_tokens]) is
 * page * page_size + place of row t, and -1 for a candidate and for rows
 * behind the last sequence (seq_offsets[B] may be below total_tokens).
 * Block-table entries past a sequence's pages and stack entries past
 * free_count are left as they were.
 *
 * If the pages do not suffice (HSTU_SLA_ERR_NO_PAGES), or a sequence would
 * outgrow max_pages, or an input is out of range (HSTU_SLA_ERR_BAD_INPUT),
 * status says so, every slot is -1 and the tables stay as they were. */
int hstu_cache_plan(const hstu_cache_tables* t, const int32_t* seq_offsets,
                    const int32_t* num_targets, const int32_t* release, int64_t total_tokens,
                    int64_t* slots, void* workspace, size_t workspace_bytes,
                    hstu_stream_t stream);

/* Slots of the last tokens of each sequence: row t of sequence b, the r-th of
 * its n_b = seq_offsets[b + 1] - seq_offsets[b] rows, is the token at position
 * lengths[b] - n_b + r; rows behind the last sequence get -1.  A sequence with
 * n_b > lengths[b], offsets, lengths or page ids out of range set status
 * (HSTU_SLA_ERR_BAD_INPUT); the rows in question get -1, the others theirs or -1. */
int hstu_cache_slot_map(const hstu_cache_tables* t, const int32_t* seq_offsets,
                        int64_t total_tokens, int64_t* slots, hstu_stream_t stream);

/* The pages of one layer and rows that go into or come out of them.  k and v:
 * device bf16 [T, H, d] as in hstu_sla.h (row strides in elements, multiples
 * of 8; base pointers 16-byte aligned). */
typedef struct {
  int32_t H;
  int32_t d;             /* 32, 64 or 128 */
  int64_t T;             /* rows */
  const int64_t* slots;  /* device [T]; -1 (any negative) = no row */
  void* pages;           /* device bytes, 16-byte aligned */
  int64_t page_stride;   /* bytes between pages, a multiple of 16 */
  void* k;               /* read by append, written by read */
  void* v;
  int64_t k_row_stride;
  int64_t v_row_stride;
} hstu_cache_rows;

/* Quantise row t of k and v into slot slots[t].  A row whose slot lies
 * beyond the pages sets status (HSTU_SLA_ERR_BAD_INPUT) and is not written; the
 * call's other rows then may or may not be.  Slots are distinct (two rows of one
 * slot leave either, or a mix). */
int hstu_cache_append(const hstu_cache_tables* t, const hstu_cache_rows* r,
                      hstu_stream_t stream);

/* Row t of k and v becomes what slot slots[t] holds, m + s code rounded to
 * bf16, and zeros for a negative slot.  A slot beyond the pages sets status; what
 * the call writes is then unspecified. */
int hstu_cache_read(const hstu_cache_tables* t, const hstu_cache_rows* r, hstu_stream_t stream);

/* SLA HSTU attention of the new rows over the cached histories.  After plan
 * and append, sequence b has Lh = lengths[b] cached tokens; of its n rows
 * [seq_offsets[b], seq_offsets[b + 1]) the last num_targets[b] are candidates
 * and the others are its last history tokens, at positions
 * Lh - (n - num_targets[b]) .. Lh - 1.  With hstu_sla.h's mask,
 *     out_i = (1/N) sum_j M(i,j) SiLU(alpha q_i . k_j) v_j
 * over the cached k_j, v_j (m + s code), a history row's own pair
 * among them; a candidate's own pair uses its row of k and v.  A row that sees
 * nothing is zero.  Rows of out behind seq_offsets[B] are left as they were.
 *
 * What a row does not see does not reach it, whatever it holds: other
 * candidates' rows, masked tokens, the unused places of a page.
 *
 * A row of q that holds a NaN or an infinity gives a NaN row (if it sees a key).
 * Sums are held in fp32 and scaled inside by up to 2^24: finite inputs stay
 * finite while |alpha| max|q| and the steps s are below 2^100 and the sums are.
 * Fewer bits than fp32 have, as in hstu_sla_fwd: SiLU over the cached keys, which
 * takes tanh from the GPU's instruction (relative error about 2^-11), and its product
 * with a key's step of V, an operand of the second matrix product: f16 scaled by a
 * power of two per row in the kernel of few rows (off by up to 2^-11 of itself, and by
 * 2^-29 of the largest for what is more than 2^18 below that), bf16 in the one of many
 * rows (up to 2^-8).  The result is rounded to bf16 once, at the end.
 *
 * There is no relative attention bias here (hstu_sla_fwd's rab_pos, rab_time): a model
 * that has one is scored from the whole history.
 *
 * A sequence whose offsets, targets, length or page ids are out of range, or
 * which has more than max_new rows, sets status (HSTU_SLA_ERR_BAD_INPUT), also in a
 * call with max_new or total_tokens 0; out's rows are then unspecified.  (Page ids are
 * checked where they are read.)  2^29 blocks (B H times max_new in 128s, or in 8s for
 * few rows) are the most there can be: beyond, HSTU_SLA_ERR_UNSUPPORTED. */
typedef struct {
  int32_t H;
  int32_t d;                   /* 32, 64 or 128 */
  int64_t total_tokens;        /* rows of q, k, v, out; >= seq_offsets[B] */
  int32_t max_new;             /* >= every sequence's rows (device-checked); it and the
                                  tables' max_pages choose the kernel, the splits and the
                                  workspace, so a tight bound is a quicker call */
  const int32_t* seq_offsets;  /* device [B + 1] */
  const int32_t* num_targets;  /* device [B] or NULL */
  int32_t contextual_len, K1, K2;
  float alpha, N;
  const void* q;               /* device bf16 [T, H, d] */
  const void* k;               /* candidates' rows; may be NULL without num_targets */
  const void* v;
  int64_t q_row_stride, k_row_stride, v_row_stride;
  const void* pages;           /* as in hstu_cache_rows */
  int64_t page_stride;
  void* out;                   /* device bf16 [T, H, d] */
  int64_t out_row_stride;
} hstu_cache_attend_params;

/* Workspace of a call with these sizes (the blocks' partial sums): 256-byte
 * aligned, contents need not be initialised; calls that may overlap need one
 * each.  0: the call needs none (NULL will do), or the arguments are invalid
 * (the call itself says so). */
size_t hstu_cache_attend_workspace_bytes(const hstu_cache_tables* t,
                                         const hstu_cache_attend_params* p);

int hstu_cache_attend(const hstu_cache_tables* t, const hstu_cache_attend_params* p,
                      void* workspace, size_t workspace_bytes, hstu_stream_t stream);

/* Synchronises `stream` and returns the tables' status, or HSTU_SLA_ERR_CUDA. */
int hstu_cache_get_error(const hstu_cache_tables* t, hstu_stream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* HSTU_CACHE_H_ */
