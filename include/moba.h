/*
 * moba.h - C ABI of the B200 (sm_100a) MoBA hot path.
 *
 * MoBA (Mixture of Block Attention), as defined in "Optimizing Mixture of
 * Block Attention" (Xiao, Guo, Mazaheri, Han; summarised on the lowest.today
 * pages, Italian and German): keys are split into blocks of B tokens, each
 * block is represented by its mean key (centroid), every query scores the
 * causally visible centroids with q . k~_j, keeps its own block plus the
 * best-scoring earlier blocks (k blocks in all), and exact softmax attention
 * with scale 1/sqrt(d) runs over the selected tokens only.
 *
 * Conventions shared by every entry point
 * ---------------------------------------
 *  Tokens are packed ("varlen"): sequences s = 0..batch-1 occupy tokens
 *  [cu_seqlens[s], cu_seqlens[s+1]).  cu_seqlens is int32 [batch + 1] in
 *  DEVICE memory, non-decreasing, cu_seqlens[0] = 0, cu_seqlens[batch] = T.
 *  Blocks, causality and the key convolution restart at every sequence.
 *
 *  q, out, dout, dq:  bf16 [T, h_q,  d] row-major (d contiguous).
 *  k, v, dk, dv:      bf16 [T, h_kv, d] row-major.
 *  lse:               fp32 [T, h_q], natural log of sum exp(q.k/sqrt(d)).
 *  sel_idx:           int32 [T, h_q, topk]: the selected blocks of each
 *                     query, block numbers relative to the query's sequence,
 *                     sorted ascending, the query's own block last among the
 *                     valid entries, unused slots -1.
 *  Query head h reads KV head h / (h_q / h_kv) (grouped-query attention).
 *
 *  Every pointer is a device pointer owned by the caller, 16-byte aligned
 *  (the workspace: 256-byte aligned).  The library allocates no memory, keeps
 *  no state between calls (apart from the optional per-thread stage-timing
 *  table of moba_set_stage_events, a cached driver entry point used to build
 *  TMA tensor maps on the host, and the static device scratch of
 *  moba_build_index_noalloc) and never synchronises: each call only enqueues
 *  kernels on `stream` (a cudaStream_t; NULL = legacy default stream) and
 *  returns.  Argument errors are reported synchronously by the return code;
 *  data-dependent errors found on the device (bad cu_seqlens, out-of-range
 *  sel_idx entries) are recorded in the workspace's status word and read
 *  with moba_check_status().  No call ever traps the device.
 *
 *  Supported sizes: d in {64, 128}; B in {16, 32, 64, 128}; 1 <= topk <= 64;
 *  h_q a multiple of h_kv; T * h_q * max(d, topk) < 2^31.  T = 0 is valid:
 *  the call returns MOBA_OK after checking the shape, launches nothing and
 *  leaves the workspace (and its status word) untouched.
 */
#ifndef MOBA_H_
#define MOBA_H_

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

/* Problem shape.  All fields are plain host values. */
typedef struct moba_shape {
  int32_t total_tokens; /* T = cu_seqlens[batch] */
  int32_t batch;        /* number of packed sequences, >= 1 */
  int32_t h_q;          /* query heads */
  int32_t h_kv;         /* key/value heads; divides h_q */
  int32_t head_dim;     /* d: 64 or 128 */
  int32_t block_size;   /* B: 16, 32, 64 or 128 */
  int32_t topk;         /* k: selected blocks per query, own block included */
} moba_shape;

/* Return codes. */
#define MOBA_OK 0
#define MOBA_EINVAL (-1)     /* null pointer, unsupported size, bad shape */
#define MOBA_EALIGN (-2)     /* pointer not 16-byte (workspace: 256-byte) aligned */
#define MOBA_EWORKSPACE (-3) /* workspace smaller than the *_workspace_size() */
#define MOBA_ELAUNCH (-4)    /* a kernel launch failed (CUDA error) */
#define MOBA_EDEVICE (-5)    /* moba_check_status(): the device flagged bad input */

/* Device status bits reported by moba_check_status(). */
#define MOBA_STATUS_BAD_SEQLENS 1 /* cu_seqlens not monotone or not ending at T */
#define MOBA_STATUS_BAD_SEL_IDX 2 /* a sel_idx entry outside [-1, own block]; skipped */
#define MOBA_STATUS_INDEX_OVERFLOW 4
#define MOBA_STATUS_TIMEOUT 8     /* a bounded device wait gave up; outputs of that call are invalid */

/* Kernel-path bits reported by moba_check_path(): which kernel families the
 * last call on a workspace ran (each kernel's first thread sets its bit). */
#define MOBA_PATH_ROUTE_TCGEN05 1 /* routing scores on the tcgen05 tensor cores */
#define MOBA_PATH_FWD_TCGEN05 2   /* forward attention on the tcgen05 tensor cores */
#define MOBA_PATH_BWD_TCGEN05 4   /* backward attention on the tcgen05 tensor cores */
#define MOBA_PATH_EXACT_ROWS 8    /* rows far above the softmax reference recomputed exactly */

/* Bytes of device workspace moba_forward / moba_key_conv_centroid need for
 * `shape` (0 for an invalid shape).  The caller allocates it; its contents
 * need no initialisation and are scratch after the call, except the status
 * word read by moba_check_status(). */
size_t moba_fwd_workspace_size(const moba_shape* shape);

/* Bytes of device workspace moba_backward / moba_build_index need. */
size_t moba_bwd_workspace_size(const moba_shape* shape);

/*
 * Key convolution (optional) and block centroids: the first two steps of
 * the forward, exposed on their own.
 *
 * Follows "Optimizing Mixture of Block Attention", section "Progettazione
 * della Convoluzione delle Chiavi (Appendice B)", "Forma Formale":
 *   k'_t = k_t + SiLU(sum_{l=0}^{W-1} w_l (.) k_{t-l})
 * depthwise (one filter per channel), causal with zero padding before the
 * sequence start, no bias; k' is rounded to bf16 (nearest even).  And section
 * "Architettura del Modello Statistico" 1: centroid of block j = mean of its
 * keys (k' when the conv is on; a partial last block averages its real
 * tokens).
 *
 *  k         bf16 [T, h_kv, d]   input keys
 *  conv_w    fp32 [h_kv, d, conv_width], tap l multiplies k_{t-l}; NULL and
 *            conv_width = 0 for no convolution; conv_width <= 8
 *  k_out     bf16 [T, h_kv, d]   k' (ignored when conv_width = 0); must not
 *            alias k
 *  centroid  fp32 [h_kv, nblk, d] where block j of sequence s is row
 *            blk_off[s] + j, blk_off[s] = sum_{s'<s} ceil(L_s'/B), and
 *            nblk = T / B + batch is the row capacity (unused rows untouched)
 */
int moba_key_conv_centroid(const void* k, const float* conv_w, int conv_width, const int32_t* cu_seqlens,
                           const moba_shape* shape, void* k_out, float* centroid, void* workspace,
                           size_t workspace_bytes, void* stream);

/*
 * MoBA forward: (key conv) -> centroids -> routing + top-k -> block index ->
 * gather-and-densify sparse attention -> normalisation.
 *
 * Routing: "Optimizing Mixture of Block Attention", section "Architettura del
 * Modello Statistico" 1 (s_j = q . k~_j) and "Definizione del Compito"
 * (top-k blocks); a query at local position p (block b = p / B) scores blocks
 * j < b, keeps the topk-1 best (exact ties: lower j) and always its own block.
 * Attention: "Definizione del Compito", O = softmax(Q K^T / sqrt(d)) V over
 * the selected tokens, causal inside the own block.
 *
 *  q, k, v           inputs (see conventions)
 *  conv_w, conv_width optional key convolution, as in moba_key_conv_centroid;
 *                    when on, k_conv_out (bf16 [T, h_kv, d]) receives k',
 *                    which routing and attention use and which the backward
 *                    must be given as its k
 *  out               bf16 [T, h_q, d]
 *  lse               fp32 [T, h_q]
 *  sel_idx           int32 [T, h_q, topk] (output)
 *  workspace         >= moba_fwd_workspace_size(shape) bytes
 */
int moba_forward(const void* q, const void* k, const void* v, const int32_t* cu_seqlens,
                 const moba_shape* shape, const float* conv_w, int conv_width, void* k_conv_out, void* out,
                 float* lse, int32_t* sel_idx, void* workspace, size_t workspace_bytes, void* stream);

/*
 * Block index: inverts sel_idx (query -> blocks) into per-(KV head, block)
 * query lists, the key-block-major varlen layout of "Optimizing Mixture of
 * Block Attention", section "Progettazione del Kernel FlashMoBA", "Tre Kernel
 * Fusi" 1 (stage 3) used by the forward and the backward.
 *
 *  blk_ptr   int32 [h_kv * nblk + 1]: bucket (kvh, gb) = kvh * nblk + gb
 *            holds entries blk_ptr[b] .. blk_ptr[b+1]-1; nblk = T / B + batch
 *  blk_rows  int32 [T * h_q * topk] capacity: query row ids t * h_q + h of
 *            every valid pick (own block included); order inside a bucket
 *            is unspecified
 */
int moba_build_index(const int32_t* sel_idx, const int32_t* cu_seqlens, const moba_shape* shape,
                     int32_t* blk_ptr, int32_t* blk_rows, void* workspace, size_t workspace_bytes,
                     void* stream);

/*
 * Allocation-free moba_build_index.  The paper has no counterpart: this entry
 * point exists for callers that cannot provide device scratch memory, such
 * as code running inside a host framework that owns all device memory and
 * forbids side allocations, or latency-critical paths that must not call
 * cudaMalloc because it can synchronise the device.
 *
 * Same inputs and outputs as moba_build_index, without the workspace: its
 * scratch lives in a static device array of MOBA_NOALLOC_SCRATCH_BYTES
 * compiled into the library, which every GPU that loads the library keeps
 * until the process exits.  The call allocates and frees nothing.  blk_ptr
 * is identical to moba_build_index's and every bucket holds the same row
 * ids, but the order of the ids inside a bucket may differ between the two
 * entry points and from call to call (consumers only sum over a bucket).
 *
 *  - Runs on the current device; `stream` must belong to it.  Every call
 *    looks up the array's device address on the current device
 *    (cudaGetSymbolAddress, a host-side query), so a device reset never
 *    leaves a stale address behind.  The first call on a device also makes
 *    the runtime set the array up in that device's context: make it before
 *    any stream capture.
 *  - Every call on a device shares the one array, and the array keeps what the
 *    last call left in it (this call clears what must start at zero).  Calls
 *    whose work overlaps on the GPU (other streams, other host threads) race
 *    on it and give wrong results: serialise them.
 *  - The scratch holds 4 * (h_kv * (T / B + batch)) * 2 bytes of counters and
 *    cursors plus 3 * 4 * (batch + 1) bytes of sequence plan (each part rounded
 *    up to 256 bytes, plus 256); a shape that needs more than
 *    MOBA_NOALLOC_SCRATCH_BYTES returns MOBA_EWORKSPACE and launches nothing.
 *  - Device-side input errors (bad cu_seqlens or sel_idx) are skipped, as in
 *    moba_build_index; the status word is not readable from outside here.
 */
#define MOBA_NOALLOC_SCRATCH_BYTES (8u << 20)
int moba_build_index_noalloc(const int32_t* sel_idx, const int32_t* cu_seqlens, const moba_shape* shape,
                             int32_t* blk_ptr, int32_t* blk_rows, void* stream);

/*
 * MoBA backward with the selection held fixed ("Optimizing Mixture of Block
 * Attention", section "Progettazione del Kernel FlashMoBA", "Tre Kernel
 * Fusi" 3: recompute per key block, dQ by atomic accumulation in fp32).
 *
 *  q, k, v, out, lse, sel_idx   as given to / returned by moba_forward (k is
 *                               k' when the forward used the key conv)
 *  dout              bf16 [T, h_q, d]
 *  dq                bf16 [T, h_q, d]  (output)
 *  dk, dv            bf16 [T, h_kv, d] (output; summed over the query heads
 *                    of each group).  The gradient stops at k': the key
 *                    convolution's own backward is not part of this call.
 *  workspace         >= moba_bwd_workspace_size(shape) bytes
 *  fwd_workspace     optional (NULL: rebuild the block index from sel_idx).
 *                    The workspace of the moba_forward call that produced
 *                    sel_idx, same shape, untouched since: its block index
 *                    is reused instead of being rebuilt.  Read only.
 */
int moba_backward(const void* q, const void* k, const void* v, const void* out, const float* lse,
                  const void* dout, const int32_t* sel_idx, const int32_t* cu_seqlens, const moba_shape* shape,
                  void* dq, void* dk, void* dv, void* workspace, size_t workspace_bytes,
                  const void* fwd_workspace, void* stream);

/*
 * Optional stage timing for benchmarks.  While a table is installed on the
 * calling host thread, moba_forward and moba_backward record events[2*i]
 * (a cudaEvent_t) on their stream before stage i and events[2*i+1] after it,
 * for every i with 2*i+1 < n_events; NULL entries are skipped.  The stages:
 * forward plan, key conv + centroids, routing, block index, attention,
 * normalisation (+ exact re-computation of flagged rows); backward plan,
 * block index, preprocessing, attention, dQ conversion; key-conv backward
 * (moba_key_conv_backward).  The table is read,
 * never written; the caller keeps it (and the events) alive while installed.
 * Pass (NULL, 0) to remove it.  Results are unaffected.
 */
#define MOBA_STAGE_FWD_PLAN 0
#define MOBA_STAGE_FWD_CENTROID 1
#define MOBA_STAGE_FWD_ROUTE 2
#define MOBA_STAGE_FWD_INDEX 3
#define MOBA_STAGE_FWD_ATTN 4
#define MOBA_STAGE_FWD_FINALIZE 5
#define MOBA_STAGE_BWD_PLAN 6
#define MOBA_STAGE_BWD_INDEX 7
#define MOBA_STAGE_BWD_PRE 8
#define MOBA_STAGE_BWD_ATTN 9
#define MOBA_STAGE_BWD_DQ 10
#define MOBA_STAGE_CONV_BWD 11
#define MOBA_NUM_STAGES 12
int moba_set_stage_events(void* const* events, int n_events);

/*
 * Backward of the key convolution, for training with it: from dK' (the
 * gradient moba_backward returns for k', which the attention used) to the
 * gradient of the original keys and of the conv weights.  Differentiates
 * "Optimizing Mixture of Block Attention", section "Progettazione della
 * Convoluzione delle Chiavi (Appendice B)", "Forma Formale", with
 * x_t = sum_l w_l (.) k_{t-l} and g_t = dK'_t (.) SiLU'(x_t):
 *   dK_t = dK'_t + sum_l w_l (.) g_{t+l}   (t + l inside the sequence)
 *   dW_l = sum_t g_t (.) k_{t-l}
 * The bf16 rounding of k' is treated as the identity.
 *
 *  k, conv_w, conv_width, cu_seqlens   as given to moba_forward (1 <= width <= 8)
 *  dk_conv   bf16 [T, h_kv, d]  dK' (e.g. moba_backward's dk)
 *  dk        bf16 [T, h_kv, d]  output; must alias neither k nor dk_conv
 *  dw        fp32 [h_kv, d, conv_width]  output (overwritten, not accumulated)
 *  workspace >= moba_bwd_workspace_size(shape) bytes
 */
int moba_key_conv_backward(const void* k, const float* conv_w, int conv_width, const int32_t* cu_seqlens,
                           const moba_shape* shape, const void* dk_conv, void* dk, float* dw, void* workspace,
                           size_t workspace_bytes, void* stream);

/*
 * ---------------------------------------------------------------------------
 * Serving from a paged 8-bit cache
 * ---------------------------------------------------------------------------
 * MoBA for generation: keys and values of many requests ("rows") are held in
 * pages of one MoBA block (B tokens), complete blocks in 8 bits.  Four calls,
 * one after the other on one stream, serve a step (one token per request,
 * several, or whole prompts):
 *   moba_cache_tables     gives pages to the rows that grow, takes back those
 *                         of finished rows, and lists the new tokens;
 *   moba_cache_append     writes their keys and values (key conv included);
 *   moba_cache_route      picks each new query's blocks from the centroids;
 *   moba_cache_attention  attends to the picked blocks, or to all of them.
 * Nothing is read back to the host, so a step can be captured into a graph.
 * A step of no tokens (total_new = 0) needs no token arrays, and only
 * moba_cache_tables a workspace; one that is given has its status cleared.
 *
 * A loop: with lengths in new_len, moba_cache_tables(c, new_len, NULL, NULL,
 * plan, ...), moba_cache_append(c, plan, k, v, conv_w, ...), moba_cache_route(c,
 * plan, q, h_q, topk, sel, ...), moba_cache_attention(c, plan, q, h_q, sel, topk,
 * out, lse, ...); then, where drafts were rejected, their number is taken off
 * the token counts in row_state.
 *
 * The buffers (device memory of the caller, 16-byte aligned; contents set by
 * moba_cache_reset and the calls above).  Element order is row-major.
 *  k, v          8 bits [n_pages, h_kv, B, d]: complete blocks.  kind 0: e4m3,
 *                kind 1: int8; the value held is x8 * scale
 *  k_scale, v_scale  fp32 [n_pages, h_kv]: max(amax * r, 2^-126) over the
 *                block's B x d values, r = the fp32 nearest 1/448 (e4m3) or
 *                1/127 (int8)
 *  cent          bf16 [2, n_pages, h_kv, d]: the mean of a complete block's
 *                bf16 keys as hi + lo (hi = bf16(c), lo = bf16(c - hi))
 *  tail_k, tail_v  bf16 [rows, 2, h_kv, B, d]: the tokens of a row's last two
 *                blocks, block j in bank j mod 2.  A partial block is read
 *                from here.  Because both are kept, a row's length may be
 *                set back (rejected drafts: lower the token count of its
 *                row_state, its pages stay) to B tokens less than the longest
 *                it has had since the row was empty, however often; with a
 *                key conv of width 2 or more to set_back tokens less
 *  hist          bf16 [rows, 16, h_kv, d]: the last raw keys, position p at
 *                p mod 16 (NULL allowed when conv_width <= 1).  Of a step's
 *                tokens the last conv_width - 1 + set_back go there
 *  block_table   int32 [rows, max_blocks]: the page of each block of a row;
 *                entries from the row's page count on are stale
 *  row_state     int32 [rows, 2]: tokens held, pages held
 *  free_pages    int32 [n_pages]: ring of free pages; ring: int64 [2], the
 *                ring's first entry and its end (both count up; mod n_pages)
 *
 * h_q (at most 65535), head_dim, block_size, topk and conv_width have the
 * limits of the other calls; max_blocks * B, n_pages * B and T * h_q * max(d, topk) are < 2^31.
 * Offsets into the pages are 64 bits wide.  max_blocks should be no larger than
 * the longest request needs: the host divides the work of attention and routing
 * by it, so the same requests take longer under a table many times as wide as
 * they are long, and need more workspace.
 */
#define MOBA_CACHE_E4M3 0
#define MOBA_CACHE_INT8 1

/* Further bits of the device status word (moba_check_status). */
#define MOBA_STATUS_NO_PAGES 16   /* a row was refused: no free pages, or more than max_blocks blocks */
#define MOBA_STATUS_BAD_TABLE 32  /* a row state, page number or plan entry out of range; skipped */
#define MOBA_STATUS_NONFINITE 64  /* a NaN or infinite key or value was stored as 0 */

typedef struct moba_cache {
  int32_t rows;       /* requests the cache has room for */
  int32_t n_pages;
  int32_t max_blocks; /* width of the block table */
  int32_t h_kv;
  int32_t head_dim;   /* 64 or 128 */
  int32_t block_size; /* 16, 32, 64 or 128 */
  int32_t kind;       /* MOBA_CACHE_E4M3 or MOBA_CACHE_INT8 */
  int32_t conv_width; /* 0 (no key conv) .. 8 */
  int32_t set_back;   /* with a key conv: tokens a row's length may be set back by, 0 .. 17 - conv_width */
  void* k;
  void* v;
  float* k_scale;
  float* v_scale;
  void* cent;
  void* tail_k;
  void* tail_v;
  void* hist;
  int32_t* block_table;
  int32_t* row_state;
  int32_t* free_pages;
  int64_t* ring;
} moba_cache;

/* The new tokens of a step, packed row after row: written by
 * moba_cache_tables, read by the other calls.  total_new (host value) is the
 * capacity T of the token arrays; entries behind cu_new[rows] are padding
 * (row, position and slot -1). */
typedef struct moba_cache_plan {
  int32_t total_new;
  int32_t* cu_new;    /* [rows + 1] first new token of each row */
  int32_t* token_row; /* [T] */
  int32_t* token_pos; /* [T] position in the row; -1: the row was refused */
  int32_t* slot_map;  /* [T] page * B + position mod B; -1: not stored */
} moba_cache_plan;

/* Bytes of device workspace that any of the calls below needs for a step of
 * total_new tokens and h_q query heads (0: invalid; a smaller step may need
 * more, as its rows are cut into more parts).  As elsewhere it needs
 * no initialisation, its first word is the status word, and calls whose work
 * can overlap on the GPU need a workspace each. */
size_t moba_cache_workspace_size(const moba_cache* cache, int total_new, int h_q);

/* Empties the cache: no tokens, every page free, tails and history zero. */
int moba_cache_reset(const moba_cache* cache, void* stream);

/*
 * Block tables and slot maps.  new_len: int32 [rows], the tokens each row is
 * about to get; a negative number gives the row's pages back and empties it
 * (they can be taken from the next call on).
 *
 * Row r needs max(0, ceil((L + n) / B) - pages held) pages.  They are taken
 * from the ring in row order.  A row is served if all pages needed by rows up
 * to and including it are there; one that is not served (also: more than
 * max_blocks blocks; more than T tokens up to and including it) keeps its
 * state, its tokens get position and slot -1, and MOBA_STATUS_NO_PAGES is set
 * (BAD_SEQLENS for the tokens beyond T, which are not listed).
 *
 * row_state_out, ring_out: where the state after the step goes; the cache's
 * own buffers for the usual step in place (then NULL may be given), others to
 * plan a step that can be planned again.  Block table and ring entries are
 * written in place; planning a step again writes the same ones.
 */
int moba_cache_tables(const moba_cache* cache, const int32_t* new_len, int32_t* row_state_out, int64_t* ring_out,
                      const moba_cache_plan* plan, void* workspace, size_t workspace_bytes, void* stream);

/*
 * Writes the new tokens.  row_state is the state after moba_cache_tables.
 *  k, v     bf16 [T, h_kv, d]; conv_w fp32 [h_kv, d, conv_width] (NULL at 0)
 * Keys pass through the key conv (k' = bf16(k + SiLU(sum_l w_l (.) k_{t-l})),
 * summed in 64 bits, with the raw keys before the step from hist).  A block
 * that becomes complete is rounded to 8 bits from its bf16 tokens, once:
 * x / scale to the nearest value, ties to even.  NaN and infinities are
 * stored as 0 (MOBA_STATUS_NONFINITE).  Tokens with slot -1 are skipped.
 */
int moba_cache_append(const moba_cache* cache, const moba_cache_plan* plan, const void* k, const void* v,
                      const float* conv_w, void* workspace, size_t workspace_bytes, void* stream);

/*
 * Routing of the new queries over the cached centroids: as in moba_forward,
 * the topk - 1 earlier blocks with the largest q . (hi + lo) and the own
 * block.  Scores are compared exactly (as if summed in 64 bits; a NaN score
 * counts as -infinity); equal scores keep the lower block.
 *  q        bf16 [T, h_q, d];  sel_idx int32 [T, h_q, topk] (output, ascending,
 *           own block last, then -1).  Rows of tokens with position -1 are all
 *           -1; rows of padding tokens stay as they were.
 */
int moba_cache_route(const moba_cache* cache, const moba_cache_plan* plan, const void* q, int h_q, int topk,
                     int32_t* sel_idx, void* workspace, size_t workspace_bytes, void* stream);

/*
 * Attention of the new queries over the cache: softmax(q . k / sqrt(d)) v over
 * the tokens at positions <= the query's, of the blocks listed in sel_idx
 * (moba_cache_route's; ascending, an entry that is not above the one before it
 * or is beyond the own block is skipped with MOBA_STATUS_BAD_SEL_IDX), or of
 * all blocks when sel_idx is NULL (topk is then ignored).
 *  out bf16 [T, h_q, d];  lse fp32 [T, h_q].  A query that sees no token
 *  (position -1, or no valid entry) gets out 0 and lse -infinity; rows of
 *  padding tokens stay as they were.
 */
int moba_cache_attention(const moba_cache* cache, const moba_cache_plan* plan, const void* q, int h_q,
                         const int32_t* sel_idx, int topk, void* out, float* lse, void* workspace,
                         size_t workspace_bytes, void* stream);

/* Synchronises `stream`, then reads the status word the last call on this
 * workspace left.  *device_status receives the MOBA_STATUS_* bits (0 = ok).
 * Returns MOBA_OK, MOBA_EDEVICE if any bit is set, or MOBA_ELAUNCH if the
 * stream reported a CUDA error. */
int moba_check_status(const void* workspace, void* stream, int32_t* device_status);

/* Synchronises `stream`, then reads which kernel families the last call on
 * this workspace ran (MOBA_PATH_* bits; forward workspace: routing, forward
 * attention, exact rows; backward workspace: backward attention).  Returns
 * MOBA_OK or MOBA_ELAUNCH if the stream reported a CUDA error.  Every shape
 * the library accepts runs the tcgen05 kernels: there is no other attention
 * or routing path. */
int moba_check_path(const void* workspace, void* stream, int32_t* path_bits);

/*
 * Self-test of the bounded device waits (the pages have no counterpart).
 * Every tensor-core kernel of this library waits on mbarriers for TMA copies,
 * MMA completions and hand-offs between warps; each such wait gives up after
 * a wall-clock limit, records MOBA_STATUS_TIMEOUT and lets the kernel return,
 * so a lost completion cannot hang the GPU.  This entry point runs that path
 * on purpose: one CTA waits, with limit `limit_ns` (1 ns .. 10 s), on an
 * mbarrier that is never completed (no copy or MMA is in flight), then sets
 * MOBA_STATUS_TIMEOUT in the status word of `workspace` (>= 256 bytes,
 * 256-byte aligned; only its first 8 bytes are written) and exits.  Read the
 * result with moba_check_status(); the device stays usable afterwards.
 */
int moba_selftest_bounded_wait(unsigned long long limit_ns, void* workspace, size_t workspace_bytes, void* stream);

/* Static description of a return code. */
const char* moba_status_string(int code);

#ifdef __cplusplus
}
#endif

#endif /* MOBA_H_ */
