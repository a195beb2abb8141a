/*
 * gdn.h -- C ABI of libgdn.so: the Gated DeltaNet tail-replay state rebuild
 * on one GB300 (sm_103a).
 *
 * Conventions shared by every call
 * --------------------------------
 * State layout.  A recurrent state S is fp32, d_v x d_k, row-major, and one
 * token updates it as
 *     S_t = alpha_t S_{t-1} (I - beta_t k_t k_t^T) + beta_t v_t k_t^T,   alpha_t = exp(g_t),
 * which is Eq. (1) of "Tail-Replay: Escaping the Curse of Linear Attention in
 * Prefix Caching for Hybrid LLMs" (section 2) written on the transposed state
 * (T_t = alpha_t (I - beta_t k_t k_t^T) is symmetric, so T_t S^T = (S T_t)^T).
 * The readout is o_t = S_t (scale * q_t) with the updated state.
 *
 * Token-major inputs.  q, k: [total_tokens][h_k][d_k]; v and O: [total_tokens]
 * [h_v][d_v]; g and beta: fp32 [total_tokens][h_v].  Sequences (replay tails)
 * are packed back to back; cu_seqlens (int32, DEVICE memory, n_seqs + 1
 * entries, non-decreasing, cu_seqlens[n_seqs] <= total_tokens) gives each
 * one's token range.  A range that breaks this (negative, past total_tokens,
 * or starting before an earlier offset) is skipped, its state left untouched,
 * and reported as GDN_ERR_SHAPE through gdn_get_status.  v-head h reads q/k
 * head h / (h_v / h_k) (consecutive v-heads share a key head).  States: fp32 [n_seqs][h_v][d_v][d_k].
 *
 * Ownership and memory.  Every pointer except the host arrays of gdn_compose
 * is a DEVICE pointer owned by the caller; the library never frees or keeps
 * them.  Calls that need scratch memory take it from a per-device pool that
 * the library grows on first need with cudaMallocAsync on the caller's
 * stream (stream-ordered) and keeps until process exit.
 *
 * Asynchrony and errors.  Every call only enqueues work on `stream` (a
 * cudaStream_t; NULL = the legacy default stream) and returns 0 (GDN_OK) or a
 * negative GDN_ERR_* code without launching anything.  No exception crosses
 * the ABI.  gdn_last_error() gives a thread-local message for the last
 * failure.  Errors found on the device (malformed cu_seqlens) are recorded in
 * a sticky per-device status word that gdn_get_status() returns and clears.
 *
 * Alignment.  q, k, v, O, S0, S_out, T and S_local base pointers must be
 * 16-byte aligned; g, beta and cu_seqlens 4-byte aligned (else GDN_ERR_ALIGN).
 */
#ifndef GDN_H_
#define GDN_H_

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

#define GDN_ABI_VERSION 1

/* return codes */
#define GDN_OK 0
#define GDN_ERR_ARG (-1)         /* null pointer, negative size, bad flag */
#define GDN_ERR_SHAPE (-2)       /* inconsistent sizes (h_v % h_k, token ranges) */
#define GDN_ERR_ALIGN (-3)       /* a base pointer breaks the alignment rule */
#define GDN_ERR_UNSUPPORTED (-4) /* a head size or dtype the library has no kernel for */
#define GDN_ERR_CUDA (-5)        /* a CUDA runtime call failed (message in gdn_last_error) */
#define GDN_ERR_TIMEOUT (-6)     /* a bounded device-side wait gave up */
#define GDN_ERR_NOMEM (-7)       /* the scratch pool could not grow */

/* storage type of q, k, v and O (g, beta and every state are always fp32) */
#define GDN_F32 0
#define GDN_BF16 1

/* flags */
#define GDN_QK_L2NORM 1u   /* normalise q and k per (token, head): x / sqrt(sum x^2 + 1e-6) */
#define GDN_STATE_ONLY 2u  /* rebuild the state only; O_out may be NULL and is not written */
#define GDN_PRECISE 4u     /* bf16 inputs: take the fp32-accurate path (as fp32 inputs do) */
/* Scalar-decay recurrence family (Mamba-2), which "LinearKV: One Cached State
 * Suffices for Position-Independent Caching in Hybrid LLMs" (composition passage)
 * sets beside GDN: the per-token transition is the scalar alpha_t instead of
 * alpha_t (I - beta_t k_t k_t^T), i.e. S_t = alpha_t S_{t-1} + beta_t v_t k_t^T
 * (beta_t scales the input; same readout), so a chunk's transition is
 * (prod alpha_t) I.  Accepted by gdn_replay, gdn_replay_noalloc and
 * gdn_chunk_operator (whose T_out is then that scaled identity).  A decay that
 * is the head's alone, the same in every token, is gdn_linear_attn's, in less
 * than half gdn_replay's time. */
#define GDN_SCALAR_DECAY 8u
#define GDN_HEAD_DECAY 16u /* gdn_decode: one decay per v-head, S_t = lambda_h S_{t-1} + v_t k_t^T */
#define GDN_KEEP_STATE 32u /* gdn_decode: outputs only, the states stay as they are */

typedef struct {
  int32_t n_seqs;       /* packed sequences (replay tails, or chunks for gdn_chunk_operator) */
  int32_t total_tokens; /* rows of q, k, v, g, beta, O */
  int32_t h_k;          /* q/k heads */
  int32_t h_v;          /* v heads, a multiple of h_k */
  int32_t d_k;          /* key/query head dim: a multiple of 8, at most 128 */
  int32_t d_v;          /* value head dim: a multiple of 8, at most 128 */
  int32_t dtype;        /* GDN_F32 or GDN_BF16 */
  uint32_t flags;       /* GDN_QK_L2NORM | GDN_STATE_ONLY | GDN_PRECISE | GDN_SCALAR_DECAY */
  float scale;          /* multiplies q in the readout (1.0 when unsure) */
} gdn_dims;

/*
 * gdn_replay -- rebuild each sequence's recurrent state by replaying its tail.
 * Source: "Tail-Replay: ..." section 3, Eq. (2): the state at the start of
 * the tail is S0 (zero when S0 == NULL, the method's zero-initialised
 * replay), Eq. (1) is applied to every tail token, the final state is
 * written to S_out and, unless GDN_STATE_ONLY, every token's readout to O_out.
 *   q, k, v      inputs in `dims->dtype`, layouts above
 *   g, beta      fp32 [total_tokens][h_v]; g = log(alpha) <= 0
 *   cu_seqlens   int32 device [n_seqs + 1]
 *   S0           fp32 [n_seqs][h_v][d_v][d_k] or NULL
 *   O_out        [total_tokens][h_v][d_v] in `dims->dtype`; NULL iff GDN_STATE_ONLY.
 *                Rows outside every sequence's range are not written.
 *   S_out        fp32 [n_seqs][h_v][d_v][d_k]; may alias S0 (in-place update)
 * Computation: chunks of 64 tokens, fp32 state carried between chunks.  bf16
 * inputs with 128-dim heads run on the tcgen05 tensor cores; with several tails
 * their sequential scans start longest first (a small kernel ranks the tails by
 * length on the stream before the chunk kernels).  GDN_STATE_ONLY calls of that
 * kind with few enough (tail, head) pairs to give every 32-row slice of every
 * state its own SM carry the state through each chunk's d_k x d_k operator,
 * built ahead of the carry, so that the chunk-to-chunk chain is one product per
 * chunk; the result is the same state to rounding.  fp32 inputs,
 * other head sizes and GDN_PRECISE take the fp32-accurate path: fp32 data,
 * every contraction as three tf32 products (about 21 significant bits), in two
 * passes with pool scratch of (ceil(total_tokens / 64) + n_seqs) * h_v * 34048
 * bytes (gdn_workspace_bytes gives the amount); its second pass runs on the
 * tcgen05 tensor cores for state-only calls with 128-dim heads, on warp-level
 * tensor cores otherwise.
 */
int gdn_replay(const gdn_dims* dims, const void* q, const void* k, const void* v, const float* g,
               const float* beta, const int32_t* cu_seqlens, const float* S0, void* O_out, float* S_out,
               void* stream);

/*
 * gdn_replay_noalloc -- gdn_replay without any device allocation.
 * The pages have no counterpart to this call; it exists for callers of this
 * library that cannot allocate device memory when they call it, for example a
 * serving process that reserves almost all of the GPU's memory at start-up
 * (for its cache) and forbids allocations afterwards, or a caller whose
 * process-wide policy routes every device allocation through its own
 * allocator.  gdn_replay takes its scratch from a pool that can grow; this
 * variant instead uses one static device array of 96 MiB that every GPU that
 * loads the library holds until the process exits.
 *   Arguments, layouts, results and error codes are those of gdn_replay.
 *   Limit: the tensor-core path needs (ceil(total_tokens / 64) + n_seqs) * h_v
 *   * 41984 bytes of scratch, plus 4 * n_seqs bytes when n_seqs > 1
 *   (gdn_workspace_bytes gives the exact figure; a 3277-token tail at 32
 *   v-heads needs 67.9 MiB); a larger problem is rejected with GDN_ERR_NOMEM
 *   before anything is launched.  fp32 inputs and GDN_PRECISE need no scratch.
 *   Every call looks up the static array's device address (cudaGetSymbolAddress,
 *   with the caller's current device); the first lookup on a device can load
 *   the library's device code, so make the first call before any stream
 *   capture.
 *   All calls share the one array: calls that overlap on the GPU (on two
 *   streams, or from two threads) race with each other and must be serialised
 *   by the caller.  Every byte a call reads from the array is written by the
 *   same call first, so nothing needs clearing between calls.
 */
int gdn_replay_noalloc(const gdn_dims* dims, const void* q, const void* k, const void* v, const float* g,
                       const float* beta, const int32_t* cu_seqlens, const float* S0, void* O_out, float* S_out,
                       void* stream);

/*
 * gdn_chunk_operator -- the affine operator of isolated chunks.
 * Source: "LinearKV: One Cached State Suffices for Position-Independent
 * Caching in Hybrid LLMs", composition passage: a chunk maps an entering
 * state to T_C S_in + S_local (transposed-state form), T_C the product of its
 * per-token transitions T_t = alpha_t (I - beta_t k_t k_t^T), latest on the
 * left, and S_local the state it reaches from an empty start.
 *   Each of the n_seqs ranges of cu_seqlens is one chunk (any length).  When
 *   cu_seqlens == NULL, n_seqs must be 1 and the chunk is all total_tokens.
 *   T_out       fp32 [n_seqs][h_v][d_k][d_k], T_C row-major, so that
 *               S_out = S_in T_C^T + S_local in this ABI's state layout
 *   Slocal_out  fp32 [n_seqs][h_v][d_v][d_k]
 * q is not needed; dims->scale and GDN_STATE_ONLY are ignored.  Computed at
 * fp32 accuracy whatever the input dtype, in two passes: the chunk-shared
 * quantities ((I + A)^{-1}, gates, norms) once per (64-token piece, v-head)
 * into pool scratch of (ceil(total_tokens / 64) + n_seqs) * h_v * 34048 bytes,
 * then the 128-row slices of the augmented state [S; P] (P seeded with the
 * identity, fed zero values; P = T_C^T after the chunk).  With d_k = d_v = 128
 * the second pass runs on the tensor cores (every contraction as three tf32
 * products); other head sizes take the fp32 CUDA-core path.
 */
int gdn_chunk_operator(const gdn_dims* dims, const void* k, const float* g, const float* beta, const void* v,
                       const int32_t* cu_seqlens, float* T_out, float* Slocal_out, void* stream);

/*
 * gdn_compose -- apply K chunk operators back to back.
 * Source: "LinearKV: ..." composition passage: the closed form
 * S_K = T_{C_K}...T_{C_2} S_local_1 + ... + T_{C_K} S_local_{K-1} + S_local_K
 * (transposed-state form), extended by T_{C_K}...T_{C_1} S_in when an
 * entering state is given.  Evaluated as S <- S T_j^T + S_local_j, j = 1..K.
 *   dims        uses h_v, d_k, d_v only (one state per v-head)
 *   K           number of chunks, 0 <= K <= 256
 *   T, Slocal   HOST arrays of K device pointers; T[j] fp32 [h_v][d_k][d_k],
 *               Slocal[j] fp32 [h_v][d_v][d_k]
 *   S_in        fp32 [h_v][d_v][d_k] or NULL (empty entering state)
 *   S_out       fp32 [h_v][d_v][d_k]; must not alias any input
 * With d_k = d_v = 128 the tensor cores do the products (T and S each split
 * into a tf32 part and an exact fp32 remainder; three products per step,
 * fp32 accuracy).  When the T[j] sit at one non-negative stride that is a
 * multiple of 512 bytes (e.g. the K slices of one [K][h_v][d_k][d_k] array)
 * each step's T arrives by tensor copies shared across the four CTAs of a
 * head; other pointer arrays take a slower path that copies T row by row.
 * Both give the same results up to fp32 rounding order.
 */
int gdn_compose(const gdn_dims* dims, int32_t K, const float* const* T, const float* const* Slocal,
                const float* S_in, float* S_out, void* stream);

/*
 * gdn_linear_attn -- linear attention with a decay for each head, over packed prompts.
 * Source: the scalar-transition family that "LinearKV: One Cached State Suffices
 * for Position-Independent Caching in Hybrid LLMs" (composition passage) sets
 * beside the delta rule, with a transition that belongs to the head alone:
 *     S_t = lambda_h S_{t-1} + v_t k_t^T,   o_t = S_t (scale * q_t),   lambda_h = exp(log_decay[h]).
 *   dims        as gdn_replay's; the only flag taken is GDN_STATE_ONLY (q and k are used as given);
 *               at most 2^31 - 1024 tokens
 *   q, k, v     inputs in `dims->dtype`, layouts above (q may be NULL with GDN_STATE_ONLY)
 *   log_decay   fp32 device [h_v], <= 0 (0: no decay; -inf: each token's state is its own)
 *   cu_seqlens  int32 device [n_seqs + 1]; malformed ranges are skipped and reported as in gdn_replay
 *   S0          fp32 [n_seqs][h_v][d_v][d_k] or NULL (zero); a sequence of no tokens returns it
 *   O_out       [total_tokens][h_v][d_v] in `dims->dtype`, NULL with GDN_STATE_ONLY (and where there
 *               are no tokens); rows outside every sequence's range are not written
 *   S_out       fp32 [n_seqs][h_v][d_v][d_k]; may alias S0
 * The state is carried in fp32 whatever the inputs' type, and is within 4e-7 of its norm over 32,768
 * tokens.  fp32 outputs are within 3e-7.  For bf16 outputs the state (as the operand of S q) and the
 * decayed scores are rounded once each to bf16, as the output itself is: together 2.4e-3 of the norm,
 * where the output's own rounding alone is 1.7e-3.  More exact are q, k and v widened to fp32, and
 * gdn_replay with GDN_SCALAR_DECAY, without GDN_QK_L2NORM, with beta = 1 and g = log_decay in every token:
 * the same recurrence at 1.7e-3 (its states within 1e-5, with GDN_PRECISE 3e-7), in more than twice the time.
 * An infinite or NaN value makes its row of the state, and that row's outputs, infinite or NaN from its
 * token on (a key its column of the state and every output, a query its own outputs), and no earlier
 * output.  With bf16 inputs a decay may hold partial sums 2^60 times as large as the outputs: they are
 * finite while |sum (q.k) v| stays below 2^67.
 * Scratch, from the library's pool and returned to it in stream order: a plan of the call when it has
 * several sequences, and the states between the segments of prompts that are cut to fill the GPU (at
 * most two states of d_v d_k floats per SM; nothing for a single short prompt).  The call can be
 * captured into a graph and replayed with new contents.  O_out overlaps no input.
 */
int gdn_linear_attn(const gdn_dims* dims, const void* q, const void* k, const void* v, const float* log_decay,
                    const int32_t* cu_seqlens, const float* S0, void* O_out, float* S_out, void* stream);

/*
 * gdn_decode -- the recurrent form: one token, or a short window of tokens, for
 * each of n_seqs requests whose states live in a pool.
 * Source: "Tail-Replay: ..." section 2, Eq. (1), token by token (delta rule; with
 * GDN_SCALAR_DECAY or GDN_HEAD_DECAY the scalar-transition families), readout with
 * the updated state as in gdn_replay.
 *   dims        n_seqs requests; total_tokens = n_seqs * window: request i's tokens are rows
 *               [i * window, (i + 1) * window) of q, k, v, g, beta and O; at most 2^31 - 1024 of them
 *   n_slots     states in the pool
 *   g, beta     fp32 [total_tokens][h_v]; with GDN_HEAD_DECAY g is the log decay [h_v] and beta NULL
 *   slots       int32 device [n_seqs]: each request's state in the pool; NULL: request i has state i.
 *               A negative slot is padding: nothing of that request is read or written.
 *   counts      int32 device [n_seqs]: how many of the window's tokens count, 0 to window; NULL: all.
 *               The rows behind them are not read, and their outputs are left as they were.
 *   S_pool      fp32 [n_slots][h_v][d_v][d_k], updated in place (read only with GDN_KEEP_STATE)
 *   O_out       [total_tokens][h_v][d_v] in `dims->dtype`; NULL iff GDN_STATE_ONLY
 * Flags: GDN_QK_L2NORM, GDN_STATE_ONLY, GDN_SCALAR_DECAY, GDN_HEAD_DECAY, GDN_KEEP_STATE.
 * Speculative decoding runs a window with GDN_KEEP_STATE (the output of every position, the states
 * untouched), verifies the drafts (gdn_verify_draft) and then runs the same window with
 * GDN_STATE_ONLY and the verification's counts: a recurrent state cannot be cut back like a
 * key-value cache, so it is advanced by exactly the tokens that stand.
 * A slot past the pool, a count outside the window, or a slot that an earlier request of the call
 * already updates: that request is skipped and GDN_ERR_SHAPE reported through gdn_get_status.
 * No scratch memory; the call can be captured into a graph and replayed with new contents.  O_out overlaps
 * no input.
 */
int gdn_decode(const gdn_dims* dims, int32_t n_slots, const void* q, const void* k, const void* v, const float* g,
               const float* beta, const int32_t* slots, const int32_t* counts, float* S_pool, void* O_out,
               void* stream);

typedef struct {
  int32_t n_seqs;        /* requests */
  int32_t n_draft;       /* drafted tokens per request (the most, with draft_lens), at most 2^31 - 1024 */
  int32_t vocab;         /* entries of a probability row, at most 524288 */
  int32_t dtype;         /* of target and draft: GDN_F32 or GDN_BF16 */
  int64_t target_stride; /* elements between consecutive rows of target, at least vocab */
  int64_t draft_stride;  /* the same of draft (ignored when draft is NULL) */
} gdn_verify_dims;

/*
 * gdn_verify_draft -- drafted tokens against the target's probabilities, from given
 * random numbers (speculative sampling: the emitted tokens follow the target's distribution).
 * The pages have no counterpart; the call decides how many tokens of a window gdn_decode commits.
 *   target      [n_seqs][n_draft + 1][vocab] probabilities: row j is the target's distribution of the
 *               token at draft position j, row n_draft (or a request's draft length) that behind the drafts
 *   draft       [n_seqs][n_draft][vocab], the distributions the drafts were drawn from, or NULL when
 *               the drafts were chosen outright (each with probability 1)
 *   drafted     int32 [n_seqs][n_draft]
 *   draft_lens  int32 [n_seqs], each request's drafts, 0 to n_draft; NULL: n_draft each.  Negative:
 *               padding, nothing of that request is written, and what it holds does not matter.
 *   uniforms    fp32 [n_seqs][n_draft + 1] in [0, 1): the first n_draft for the drafts, the last one
 *               for the sampled token
 * Request by request: draft j is accepted while u_j * q_j(x_j) < p_j(x_j), in exact arithmetic.  Behind
 * the a accepted ones a token is sampled from the distribution max(p_a - q_a, 0) when draft a was
 * rejected (p_a itself where that is zero throughout), from p_a when every draft was accepted: the
 * lowest index whose inclusive sum of weights exceeds floor(u * sum) (one product in fp64; a u outside
 * [0, 1) takes the first or the last weight), the weights whole multiples of 2^-44 (each probability
 * clamped to [0, 1] and rounded down; NaN counts as 0), so that the order of summation cannot change the
 * token.
 *   counts_out  int32 [n_seqs]: a + 1, the emitted tokens -- and, in a window of the last token
 *               followed by the drafts, the tokens that gdn_decode is to commit
 *   tokens_out  int32 [n_seqs][n_draft + 1]: the accepted drafts, the sampled token, then -1.  Where
 *               the row to sample from is zero throughout, the sampled token is -1.
 * A draft length above n_draft: the request is skipped and GDN_ERR_SHAPE reported through
 * gdn_get_status.  A drafted token outside the vocabulary is rejected and reported the same way.
 * No scratch memory; the call can be captured into a graph.
 */
int gdn_verify_draft(const gdn_verify_dims* dims, const void* target, const void* draft, const int32_t* drafted,
                     const int32_t* draft_lens, const float* uniforms, int32_t* counts_out, int32_t* tokens_out,
                     void* stream);

typedef struct {
  int32_t n_seqs;        /* requests */
  int32_t total_tokens;  /* rows of q, k, v and O: the requests' new tokens */
  int32_t max_q;         /* most new tokens of one request, at least 1 */
  int32_t h_q;           /* query heads, a multiple of h_kv, at most 128 to one: head h reads key head h / (h_q / h_kv) */
  int32_t h_kv;          /* key and value heads */
  int32_t d;             /* head dim of queries, keys and values: a multiple of 8, at most 128 */
  int32_t page_size;     /* tokens of a page, a power of two */
  int32_t n_pages;       /* pages of the cache */
  int32_t table_width;   /* entries of a request's row of the page table, of at most 2^31 - 1024 tokens together */
  int32_t dtype;         /* of q, k, v, the pages and O: GDN_F32 or GDN_BF16 */
  int32_t window;        /* gdn_paged_attn: a token sees the last `window` tokens, itself among them; 0: all */
  float scale;           /* gdn_paged_attn: multiplies q.k */
  int64_t table_stride;  /* elements between the rows of the page table, at least table_width */
  int64_t q_stride, k_stride, v_stride; /* elements between the tokens of q, and of the new k and v (a token's heads
                                           lie one after another) */
  int64_t k_page, k_token, k_head; /* elements between the pages, a page's tokens and a token's heads of k_pages */
  int64_t v_page, v_token, v_head; /* the same of v_pages */
} gdn_paged_dims;

#define GDN_MAX_AXES 4
typedef struct {
  int32_t rotary_dim; /* values of a head that are rotated (the first ones): even, at most d; 0: none */
  int32_t neighbours; /* 0: values i and i + rotary_dim / 2 turn together; 1: values 2 i and 2 i + 1 */
  int32_t n_axes;     /* rows of positions, 1 to GDN_MAX_AXES */
  int32_t sections[GDN_MAX_AXES]; /* consecutive pairs that turn by each axis, rotary_dim / 2 in all (not read for one axis) */
} gdn_rotary;

/*
 * gdn_kv_append -- new keys and values into a paged cache, rotated by their positions on the way.
 * The attention layers between a hybrid model's recurrent ones; the pages name their cache (its
 * copy beside the replay is "Tail-Replay: ..." section 3) and give no kernel.
 *   k, v          [total_tokens][h_kv][d] in `dims->dtype`, k_stride and v_stride apart
 *   page_table    int32 device [n_seqs][table_width]: position p of request i lies in page page_table[i][p /
 *                 page_size], slot p % page_size.  Entries behind a request's length are not read.
 *   kv_lens       int32 device [n_seqs]: tokens in the cache once the call's are in it; new token t of n takes
 *                 position kv_lens - n + t, and one whose position is below zero has no place (nothing is written
 *                 for it).  Negative: padding, nothing of that request is read or written.
 *   cu_seqlens    int32 device [n_seqs + 1], or NULL: every request has total_tokens / n_seqs new tokens
 *   k_pages, v_pages  the cache; written at the new tokens' places alone
 *   q, q_out      queries to rotate by the same positions, [total_tokens][h_q][d] q_stride apart, into
 *                 [total_tokens][h_q][d] without gaps; both NULL: none.  q_out may be q where q has no gaps.
 *   rotary        NULL: k and q are copied as they are
 *   inv_freq      fp32 device [rotary_dim / 2]: pair i turns by the angle position * inv_freq[i]
 *   positions     int32 device [n_axes][total_tokens], or NULL (one axis): a token's place in the cache
 * A pair (a, b) becomes (a cos - b sin, b cos + a sin).  Angles are reduced to a part of a turn in integers of 2^-64, so
 * that far positions lose nothing; the rest is fp32 and rounded once to `dtype`.
 * A malformed range (as in gdn_replay), one of more than max_q tokens, a kv_lens past the table, or a page
 * outside the cache: the request (for a page, the tokens of that page) is skipped and GDN_ERR_SHAPE reported through
 * gdn_get_status.  No scratch memory; the call can be captured into a graph and replayed with new contents.  The pages overlap
 * neither q, k, v nor q_out; two tokens of a call never have the same place.
 * Alignment: 16 bytes for q, k, v, the pages, q_out and each of the strides.
 */
int gdn_kv_append(const gdn_paged_dims* dims, const gdn_rotary* rotary, const void* q, const void* k, const void* v,
                  const float* inv_freq, const int32_t* positions, const int32_t* page_table, const int32_t* kv_lens,
                  const int32_t* cu_seqlens, void* k_pages, void* v_pages, void* q_out, void* stream);

/*
 * gdn_paged_attn -- attention of each request's new tokens over its paged cache: one token, a window of
 * drafts, or a chunk of a prompt.
 *     o_t = sum_j p_tj v_j,   p_tj = exp(scale q_t.k_j - lse_t),   lse_t = log sum_j exp(scale q_t.k_j)
 * over the keys j that token t sees: with kv_lens tokens in the cache, the n new ones the last of them
 * (gdn_kv_append has put them there), token t of n has position p = kv_lens - n + t and sees 0 <= j <= p, and
 * with a window only j > p - window.
 *   q, page_table, kv_lens, cu_seqlens, the pages: as in gdn_kv_append
 *   O_out         [total_tokens][h_q][d] in `dims->dtype`, without gaps
 *   lse_out       fp32 [total_tokens][h_q], or NULL
 * A token that sees no key (its position is below zero) has output 0 and lse -inf.  Rows outside every range, and
 * those of padding (kv_lens negative), are left as they were.  What lies in the cache behind a request's length is
 * not read, and an infinite or NaN key or value reaches only the tokens that see it.
 * Sums are fp32.  bf16: the weights p are rounded once to bf16 as operands of the sum over values, as the output
 * itself is: together 2.4e-3 of an output's norm, where its own rounding alone is 1.7e-3; lse has neither.
 * Malformed ranges and lengths are reported as by gdn_kv_append, the request's rows left as they were; with a page
 * outside the cache the request's outputs are unspecified.
 * Scratch, from the library's pool and returned to it in stream order: partial results of requests that are shared
 * between SMs, at most two tiles of d floats for each row per SM.  The call can be captured into a graph and
 * replayed with new contents.  O_out and lse_out overlap no input.
 */
int gdn_paged_attn(const gdn_paged_dims* dims, const void* q, const void* k_pages, const void* v_pages,
                   const int32_t* page_table, const int32_t* kv_lens, const int32_t* cu_seqlens, void* O_out,
                   float* lse_out, void* stream);

typedef struct {
  int32_t n_seqs;  /* requests */
  int32_t beams;   /* beams of a request, at most 64 */
  int32_t best;    /* continuations that are selected, at most 64 */
  int32_t vocab;   /* entries of a row of logits, at most 524288 */
  int32_t dtype;   /* of the logits: GDN_F32 or GDN_BF16 */
  int64_t stride;  /* elements between consecutive rows of logits, at least vocab */
} gdn_beam_dims;

/*
 * gdn_beam_select -- the best continuations of each request over its beams and the vocabulary.
 * The pages have no counterpart; beside gdn_verify_draft, the other way to a request's next tokens.
 *     total(b, v) = scores[b] + logits[b][v] - log sum_w exp(logits[b][w])
 *   logits      [n_seqs][beams][vocab] in `dims->dtype`, rows `stride` apart
 *   scores      fp32 [n_seqs][beams], the beams' totals so far; -inf: the beam is dead
 *   scores_out, parents_out, tokens_out   fp32, int32, int32 [n_seqs][best]: the `best` largest totals, their
 *               beams and tokens, largest first; equal totals in the order of their beams, a beam's by
 *               (larger logit, lower token)
 * A logit of -inf is never selected, nor is NaN; a row with a NaN or +inf, like a dead beam, has no continuation.
 * Where there are fewer than `best`, the rest is -inf, -1, -1.  Totals are compared in fp64: the logits' and scores'
 * numbers as they are, the log sum within 1e-7 of itself; scores_out is rounded once.
 * Scratch, from the library's pool and returned to it in stream order: 12 + 8 * best bytes for each 8,192 entries
 * of a row (each 2,048 for few rows).  The call can be captured into a graph.  Outputs overlap no input.
 */
int gdn_beam_select(const gdn_beam_dims* dims, const void* logits, const float* scores, float* scores_out,
                    int32_t* parents_out, int32_t* tokens_out, void* stream);

typedef struct {
  int32_t n_seqs;   /* requests */
  int32_t beams;    /* beams of a request, at most 64 */
  int32_t n_slots;  /* rows of the pool */
  int32_t layers;   /* pools of the same slots, one after another (one for each layer); 0: slots_out alone */
  int64_t row_bytes, slot_stride, layer_stride; /* bytes of a row, between rows, between layers: multiples of 16 */
} gdn_reorder_dims;

/*
 * gdn_beam_reorder -- the rows of a pool (gdn_decode's states; pages of a key-value cache) follow their beams.
 * The pages have no counterpart; the call stands between gdn_beam_select and the next gdn_decode.
 *   slots       int32 device [n_seqs][beams]: the row of each beam so far.  A negative first slot: padding, its
 *               request's slots_out are -1, nothing of it moves, and what else it holds does not matter.
 *   parents     int32 device [n_seqs][beams]: the beam that each new beam continues, or negative: none (the new beam
 *               gets a slot, whose row stays as it is)
 *   pool        any rows of row_bytes, updated in place
 *   slots_out   int32 device [n_seqs][beams]: the rows of the new beams, a permutation of the request's slots.  The
 *               first child of a beam keeps its row; the k-th of the other new beams takes the row of the k-th beam
 *               without children, and its parent's row is copied there.
 * A slot outside the pool or named twice (by the request, or by an earlier one), or a parent that is no beam: the
 * request is skipped, its slots_out are -1, and GDN_ERR_SHAPE is reported through gdn_get_status.  No scratch memory;
 * the call can be captured into a graph and replayed with new contents.  slots_out overlaps no input.  The pool is
 * 16-byte aligned.
 */
int gdn_beam_reorder(const gdn_reorder_dims* dims, const int32_t* slots, const int32_t* parents, void* pool,
                     int32_t* slots_out, void* stream);

/*
 * gdn_get_status -- synchronise `stream`, then return and clear the sticky
 * device status of the current device: GDN_OK, GDN_ERR_SHAPE (a malformed
 * cu_seqlens was skipped), GDN_ERR_TIMEOUT, or GDN_ERR_CUDA when the stream
 * itself reports an error.
 */
int gdn_get_status(void* stream);

/* Thread-local message of the last failed call ("" if none). */
const char* gdn_last_error(void);

/* Bytes of scratch the library's pool needs for a gdn_replay of this problem (0 if none). */
size_t gdn_workspace_bytes(const gdn_dims* dims);

/*
 * gdn_set_stage_event -- measurement hook (no counterpart on the pages).
 * `event` is a cudaEvent_t created by the caller.  The next gdn_replay or
 * gdn_replay_noalloc call made by this thread on the tensor-core path records
 * it on its stream between its two kernels (chunk prep, then scan), so that
 * the caller can time each kernel with its own events before and after the
 * call; the hook is then cleared.  Other calls ignore it.
 */
void gdn_set_stage_event(void* event);

/*
 * gdn_set_wait_limit_ns -- test hook for the device-side timeout path (no
 * counterpart on the pages).  Every wait inside the tensor-core kernels is
 * bounded (2 s by default): a wait that runs out makes the kernel stop issuing
 * work, let what it has already issued finish, and report GDN_ERR_TIMEOUT
 * through gdn_get_status, leaving the context usable.  The next gdn_compose
 * call made by this thread uses `ns` as that bound (0: a wait gives up unless
 * its event has already happened, so the call reports a timeout); the hook is
 * then cleared.  Results of a call that timed out are unspecified.
 */
void gdn_set_wait_limit_ns(uint64_t ns);

/* GDN_ABI_VERSION of the loaded library. */
int gdn_abi_version(void);

#ifdef __cplusplus
}
#endif

#endif /* GDN_H_ */
