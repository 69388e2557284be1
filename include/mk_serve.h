/*
 * mk_serve -- serving operators around the decode step of mk.h: pages of a
 * K/V cache, decode attention for a batch that shares a prefix, token
 * probabilities, and the verification of drafted tokens.
 *
 * Conventions (beside those of mk.h):
 *  - Every call is asynchronous and ordered on `stream` (cudaStream_t as
 *    void*; NULL = legacy default stream) unless it says otherwise.  It runs
 *    on the current device, which must hold every device pointer.  No call
 *    allocates memory or synchronises, so all of them can be captured into
 *    CUDA graphs.
 *  - `workspace` is device scratch of at least the size that the matching
 *    *_workspace_bytes call returns, 256-byte aligned, with any contents.  A
 *    call uses it until its work on the stream has finished: calls that may
 *    overlap on the GPU (two streams, two graphs) need a workspace each.
 *  - Device-side problems (a page number, a length or a list entry out of
 *    range) never make a kernel read or write outside the caller's buffers:
 *    the entry is skipped or clamped as each call says, and the first code is
 *    kept in a status word (device int32; the caller sets it to 0 and reads
 *    it when it likes; NULL where none is wanted).
 */
#ifndef MK_SERVE_H
#define MK_SERVE_H

#include "mk.h"

#ifdef __cplusplus
extern "C" {
#endif

/* ------------------------------------------------------------------ cache pages */
/*
 * A pool of K/V pages.  The layout is the one of mk_kv_cache with the pages in
 * the place of the sequences, so an engine's cache is a pool of max_batch
 * pages ("slots") of max_seq positions.
 */
typedef struct {
  void *k;            /* device [n_layers][n_pages][n_kv_heads][page][head_dim], 16-byte aligned */
  void *v;            /* same layout */
  int32_t n_layers;
  int32_t n_pages;    /* 1 .. 2^20 */
  int32_t n_kv_heads;
  int32_t page;       /* positions per page, 1 .. 2^24 */
  int32_t head_dim;
  int32_t elem_bytes; /* 1, 2 or 4; head_dim * elem_bytes must be a multiple of 16 */
  /* n_layers * n_kv_heads * ceil(page / rows of 8 KB) is below 2^30 */
} mk_kv_pool;

/*
 * The bookkeeping of a paged cache: int32 words on the device,
 *   [0] pages free, [1] status (first MK_ERR_* code), [2], [3] zero,
 *   length of each sequence          [n_seqs]
 *   references to each page          [n_pages]  (0: free)
 *   free pages, a stack              [n_pages]  (the first [0] words; the top is the last of them)
 *   pages of each sequence           [n_seqs][max_pages]  (-1: none)
 * Sequence s of length n holds ceil(n / page) pages, position p in the page
 * at p / page.  Pages may be shared between sequences; a shared page is never
 * written by growth (mk_kv_resize copies it first).
 */
typedef struct {
  int32_t *words;    /* device, mk_kv_state_words() of them */
  int32_t n_seqs;    /* 1 .. 2^20 */
  int32_t max_pages; /* pages a sequence can hold; max_pages * page < 2^31 */
  int32_t n_pages;   /* as the pool's */
} mk_kv_state;

/* Words of a bookkeeping buffer (0 for a non-positive size). */
int64_t mk_kv_state_words(int32_t n_seqs, int32_t max_pages, int32_t n_pages);

/* Every page free (page 0 on top of the stack), every sequence empty, status 0.
 * Errors: MK_ERR_INVALID_ARG, MK_ERR_LAUNCH, MK_ERR_CUDA. */
int mk_kv_init(const mk_kv_state *st, void *stream);

/* Scratch of mk_kv_resize / mk_kv_fork / mk_kv_compact / mk_kv_copy (lists of up to n entries). */
int64_t mk_kv_workspace_bytes(int32_t n_pages, int32_t n);

/*
 * mk_kv_resize: set the length of sequence seqs[i] to lens[i], for i < n.
 *  1. Every page past a sequence's new length is given back (one reference
 *     less); the pages that are then free go onto the stack in ascending order.
 *  2. Sequences that grow take pages from the top of the stack, entry by
 *     entry.  A sequence that grows inside a page which others hold too first
 *     gets a copy of that page's rows in a page of its own (of several that
 *     grow on one page, the last holder in list order keeps it).
 * A length of 0 frees the sequence.  New rows hold what their page held.
 *  - seqs, lens: device int32 [n], 1 <= n <= 1024.
 *  - An entry out of range (sequence, length over max_pages * page) and a
 *    sequence's second entry are skipped: MK_ERR_DEVICE_INPUT.  An entry that
 *    the free pages do not cover keeps its length: MK_ERR_OUT_OF_MEMORY; later
 *    entries may still fit.
 *  - Errors: MK_ERR_INVALID_ARG, MK_ERR_LAUNCH, MK_ERR_CUDA.
 */
int mk_kv_resize(const mk_kv_pool *pool, const mk_kv_state *st, const int32_t *seqs,
                 const int32_t *lens, int32_t n, void *workspace, void *stream);

/*
 * mk_kv_fork: sequence children[i] becomes a copy of sequence parents[i], for
 * i < n.  Full pages are shared (one reference more); the rows of a last page
 * that is not full are copied into a page from the free stack, in list order.
 *  - parents, children: device int32 [n], 1 <= n <= 1024.  Parents are read as
 *    they were before the call.
 *  - An entry is skipped with MK_ERR_DEVICE_INPUT when it is out of range, its
 *    child is not empty, is its parent, or was an earlier entry's child; with
 *    MK_ERR_OUT_OF_MEMORY when it needs a page and none is left.
 */
int mk_kv_fork(const mk_kv_pool *pool, const mk_kv_state *st, const int32_t *parents,
               const int32_t *children, int32_t n, void *workspace, void *stream);

/*
 * mk_kv_compact: with n pages in use, move the k-th page in use among those
 * numbered n and up into the k-th free page below n, for all k, and change
 * every sequence's page numbers to match.  The pages n and up are then free,
 * page n on top of the stack.
 */
int mk_kv_compact(const mk_kv_pool *pool, const mk_kv_state *st, void *workspace, void *stream);

/*
 * mk_kv_copy: copy rows between pages of two pools (or of one pool), all
 * layers and heads, K and V.  Entry i copies rows [src_row, src_row + rows)
 * of src_page to the rows from dst_row of dst_page.  The pools agree in
 * n_layers, n_kv_heads, head_dim and elem_bytes; their page sizes may differ.
 *  - items: device int32 [n][5] = src_page, src_row, dst_page, dst_row, rows;
 *    1 <= n <= 16384.
 *  - Copies are independent.  An entry is skipped with MK_ERR_DEVICE_INPUT when
 *    it is out of range, or when its destination meets an earlier entry's
 *    destination or any entry's source (whether or not that entry is itself
 *    skipped for such a meeting).  rows = 0 copies nothing.
 *  - status: device int32 or NULL.
 *  - Two pools that overlap in memory without being the same:
 *    MK_ERR_INVALID_ARG.
 */
int mk_kv_copy(const mk_kv_pool *src, const mk_kv_pool *dst, const int32_t *items, int32_t n,
               int32_t *status, void *workspace, void *stream);

/* ------------------------------------------------------------------ shared-prefix attention */
enum { MK_DTYPE_BF16 = 0, MK_DTYPE_F16 = 1, MK_DTYPE_F32 = 2 };

/*
 * One layer's decode attention for a batch whose sequences start with the same
 * prefix.  Query t (of n_tokens) of sequence b sees the positions
 * [0, lens[b] - (n_tokens - 1 - t)): the last n_tokens positions are the
 * queries' own, each seeing itself and what is before it.  Positions below
 * *prefix_len are read from prefix_pages, once for the whole batch; the
 * others from the sequence's row of `table`, whose entry j holds the positions
 * [j * page, (j + 1) * page) (entries wholly inside the prefix are not read).
 *   out = sum_j p_j v_j,  p = softmax_j(scale * q . k_j)
 * with 32-bit sums; head h reads K/V head h / (n_q_heads / n_kv_heads).
 *  - A query that sees nothing gets zeros (and a log-sum-exp of -infinity).
 *    A sequence with lens[b] < 0 is unused: its rows of out / lse are left as
 *    they are.  Values in masked positions, infinities and NaN too, have no
 *    influence.
 *  - A page number out of range is read as page 0, a length past the pages of
 *    its list is cut to them: MK_ERR_DEVICE_INPUT in *status.
 *  - MK_ERR_TIMEOUT in *status: a wait inside the kernel gave up after a second
 *    (every one is bounded); the results are then undefined.
 *  - Results do not depend on timing: the same call gives the same bits.
 *  - Scores, maxima and sums are 32-bit.  The weights p go to the matrix
 *    instructions in the type of q: as one number each (off by 2^-8 of it for
 *    bf16, 2^-11 for fp16, like out's own rounding) for a prefix whose pages have
 *    room for 1024 positions or more, as two (2^-16, 2^-22) for other prefixes and
 *    for a sequence's own positions.  fp16 weights less than 2^-21 of the row's
 *    largest are off by up to 2^-32 of that.
 *  - Each page list has room for fewer than 2^31 - 64 positions, and n_kv_heads *
 *    (batch * n_tokens * group / 16 + batch) * (the room of both lists / 16 + 6)
 *    stays below 2^31: MK_ERR_INVALID_ARG.
 */
typedef struct {
  int32_t batch;              /* 1 .. 1024; batch * n_tokens <= 1024 */
  int32_t n_tokens;           /* queries per sequence, 1 .. 16 */
  int32_t n_q_heads;
  int32_t n_kv_heads;         /* n_q_heads a multiple of it, by at most 16 */
  int32_t head_dim;           /* 64 or 128 */
  int32_t dtype;              /* MK_DTYPE_BF16 or MK_DTYPE_F16: q, k, v and out */
  int32_t page;               /* positions per page */
  int32_t n_pages;            /* pages in k / v */
  int32_t n_prefix_pages;     /* entries of prefix_pages (0: no prefix) */
  int32_t table_width;        /* entries per row of table */
  float scale;                /* finite, usually head_dim^-0.5 */
  const void *q;              /* device [batch][n_tokens][n_q_heads][head_dim], strides below */
  const void *k;              /* device [n_pages][n_kv_heads][page][head_dim], strides below */
  const void *v;              /* same strides as k */
  void *out;                  /* as q, strides below */
  float *lse;                 /* device [batch][n_tokens][n_q_heads] contiguous, or NULL */
  const int32_t *prefix_pages;/* device [n_prefix_pages] */
  const int32_t *prefix_len;  /* device, one word (may be NULL without prefix pages) */
  const int32_t *table;       /* device [batch][table_width] */
  const int32_t *lens;        /* device [batch], prefix included */
  int32_t *status;            /* device, or NULL */
  /* strides in elements, multiples of 8 (the last dimension is contiguous; pointers 16-byte aligned) */
  int64_t q_batch_stride;
  int64_t q_token_stride;
  int64_t q_head_stride;
  int64_t out_batch_stride;
  int64_t out_token_stride;
  int64_t out_head_stride;
  int64_t page_stride;
  int64_t kv_head_stride;
  int64_t row_stride;
} mk_attn_shared_args;

/* Scratch of mk_attn_shared for these sizes (0 for sizes it refuses). */
int64_t mk_attn_shared_workspace_bytes(const mk_attn_shared_args *a);

/* Errors: MK_ERR_INVALID_ARG (NULL, misaligned, inconsistent),
 * MK_ERR_UNSUPPORTED_SHAPE (head_dim, group size, batch, n_tokens or dtype outside the above),
 * MK_ERR_LAUNCH, MK_ERR_CUDA. */
int mk_attn_shared(const mk_attn_shared_args *a, void *workspace, void *stream);

/* ------------------------------------------------------------------ token probabilities */
/*
 * mk_token_probs: probs[i][j] = exp((z_ij - max_i) / T_i) / sum over j, for the
 * n rows z of logits, in 32 bits.  T_i = 0 gives the greedy choice: 1 at the
 * first of the largest logits, 0 elsewhere.
 *  - logits: device [n][vocab], rows logits_stride elements apart, of `dtype`
 *    (MK_DTYPE_*).  probs: device float [n][vocab], rows probs_stride apart;
 *    may be the logits themselves when those are float with the same stride.
 *  - temperature: device float [n], or NULL (all 1).
 *  - A logit of -infinity is a token that cannot come.  A row without a finite
 *    largest logit, with a NaN, or with a temperature that is negative or not
 *    finite has no distribution: its probabilities are all 0.
 *  - n <= 2^24, vocab < 2^30.  Errors: MK_ERR_INVALID_ARG, MK_ERR_LAUNCH, MK_ERR_CUDA.
 */
int mk_token_probs(const void *logits, int32_t dtype, int64_t logits_stride, const float *temperature,
                   float *probs, int64_t probs_stride, int32_t n, int32_t vocab, void *stream);

/* ------------------------------------------------------------------ verification of drafted tokens */
/*
 * mk_verify: decide how many of each sequence's drafted tokens stand, and
 * sample the token after them, so that the output is distributed as if sampled
 * from the target.  For sequence b with n = n_drafted[b] tokens x_0 .. x_{n-1}:
 *   token j stands if all before it do and u_j * q_j(x_j) < p_j(x_j);
 *   a = the number that stand; the next token is the first i with
 *   sum_{k <= i} r_k > u_max_drafted * sum_k r_k, where r = max(p_a - q_a, 0)
 *   (p_a if that is 0 everywhere) for a < n and r = p_n for a = n.
 * Products and sums are in 64 bits.
 *  - target: device float [batch][max_drafted + 1][vocab] probabilities p, with
 *    the strides given (elements).  They need not sum to 1; values that are
 *    not above 0 or not finite count as 0.
 *  - draft: device float [batch][max_drafted][vocab] probabilities q, or NULL
 *    for a drafter without any (q_j is then 1 at x_j and 0 elsewhere).
 *  - tokens: device int32 [batch][max_drafted]; n_drafted: device int32
 *    [batch], or NULL (all max_drafted).  Counts outside [0, max_drafted] are
 *    clamped, a token outside the vocabulary does not stand:
 *    MK_ERR_DEVICE_INPUT in *status (device int32, or NULL).
 *  - u: device float [batch][max_drafted + 1] in [0, 1).
 *  - out_tokens: device int32 [batch][max_drafted + 1]: the tokens that stand,
 *    the sampled one, then -1.  A row r that is 0 everywhere has no token: -1.
 *  - n_accepted: device int32 [batch]: a.
 *  - batch <= 65535, max_drafted 0 .. 64, vocab < 2^30.  A vocabulary above
 *    104857600 is MK_ERR_UNSUPPORTED_SHAPE (a block keeps the running sums of its
 *    part of a row on chip).
 *  - Errors: MK_ERR_INVALID_ARG, MK_ERR_UNSUPPORTED_SHAPE, MK_ERR_LAUNCH, MK_ERR_CUDA.
 */
typedef struct {
  int32_t batch;
  int32_t max_drafted;
  int32_t vocab;
  const float *target;
  const float *draft;
  const int32_t *tokens;
  const int32_t *n_drafted;
  const float *u;
  int32_t *out_tokens;
  int32_t *n_accepted;
  int32_t *status;
  int64_t target_batch_stride;
  int64_t target_row_stride;
  int64_t draft_batch_stride;
  int64_t draft_row_stride;
} mk_verify_args;

int mk_verify(const mk_verify_args *a, void *stream);

/* ------------------------------------------------------------------ with an engine */
/*
 * mk_speculate: check drafted tokens of one sequence with an engine, and sample
 * the token after those that stand: mk_prefill of the n_tokens given tokens
 * with every row's logits kept, mk_token_probs of those rows, mk_verify.
 *  - tokens: device int32 [n_tokens]: the sequence's last token, at position
 *    pos0, then n_tokens - 1 drafted ones; 1 <= n_tokens <= 16.  (n_tokens = 1
 *    samples the next token.)  Their K/V rows are written; those of tokens that
 *    do not stand are overwritten by the call that continues at
 *    pos0 + accepted + 1.
 *  - draft_probs: device float [n_tokens - 1][vocab] probabilities of the
 *    drafter, or NULL.  temperature: device float, one word, or NULL (1); 0 is
 *    greedy.  u: device float [n_tokens] in [0, 1), the last for the sampling.
 *  - out_tokens: device int32 [n_tokens] as mk_verify's; n_accepted: device
 *    int32, one word.
 *  - As for mk_prefill: a plan that runs as one launch a step; a batched plan
 *    takes all tokens in one launch, a batch-1 plan one launch a token.  The
 *    first call after mk_plan allocates scratch (not while capturing).
 *  - Errors: MK_ERR_INVALID_ARG, MK_ERR_NOT_PLANNED, MK_ERR_OUT_OF_MEMORY,
 *    MK_ERR_LAUNCH, MK_ERR_CUDA; device-side ones by mk_get_status.
 */
int mk_speculate(mk_handle *h, int32_t seq, const int32_t *tokens, int32_t n_tokens, int32_t pos0,
                 const float *draft_probs, const float *temperature, const float *u,
                 int32_t *out_tokens, int32_t *n_accepted, void *stream);

/*
 * mk_decode_step_shared: mk_decode_step for sequences that share their first
 * prefix_len positions, whose keys and values are read, once for the batch,
 * from sequence prefix_seq's rows of the cache (the kernels of mk_attn_shared in
 * the place of the attention instructions, on the step's 32-bit q and output).
 * Sequence b holds only its own rows prefix_len .. positions[b].
 *  - Needs a plan with exec_mode MK_EXEC_PER_OP (one launch per instruction
 *    class), MK_ERR_INVALID_ARG otherwise.  0 <= prefix_len <= max_seq; a
 *    position below prefix_len is reported as MK_ERR_DEVICE_INPUT.
 *  - The other arguments and errors as for mk_decode_step.  The first call
 *    after mk_plan allocates scratch (not while capturing).  Steps of both
 *    kinds may follow one another.
 */
int mk_decode_step_shared(mk_handle *h, const int32_t *tokens, const int32_t *positions,
                          int32_t prefix_seq, int32_t prefix_len, float *logits_out,
                          int32_t *next_tokens_out, void *stream);

#ifdef __cplusplus
}
#endif
#endif /* MK_SERVE_H */
