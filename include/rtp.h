/*
 * rtp.h -- C ABI of the B200 (sm_100a) head-wise sparse attention layer.
 *
 * The layer is the one described for RTPurbo in "Full Attention Strikes Back:
 * Transferring Full Attention into Sparse within Hundred Training Steps"
 * (arXiv 2605.16928): only a few KV heads ("retrieval heads") keep the whole
 * context; the others ("local heads") attend to attention sinks plus a sliding
 * window (atlas.scime.ai summary, "Approach").  Retrieval heads choose tokens
 * with a 16-dimensional pre-RoPE indexer (abstract, observation (2)) and keep
 * a query-dependent top-p set instead of a fixed top-k (abstract, observation
 * (3); atlas "Approach": "query-adaptive top-p threshold"), then run exact
 * attention over the kept rows.
 *
 * Conventions for every entry point
 *   - Pointers are DEVICE pointers unless the comment says "host".  The caller
 *     owns all memory; the library never allocates, frees or keeps a pointer
 *     after the call returns.
 *   - `stream` is a cudaStream_t passed as void* (NULL = legacy default
 *     stream).  All device work is enqueued on it; nothing synchronises.
 *   - The return value is an rtp_status.  Errors that the host can see (null
 *     pointers, bad shapes, small workspace, a failed launch) return at once
 *     with nothing enqueued and a message in rtp_last_error().
 *   - Errors only the device can see (a sequence length or a position outside
 *     the cache) never trap: the kernels skip the offending sequence/row and
 *     OR an RTP_DEV_* bit into *cache->status, which the caller reads back
 *     when it wants (it is never cleared by the library).
 *   - Device buffers must be 16-byte aligned (torch and cudaMalloc allocations
 *     are); a misaligned pointer returns RTP_ERR_INVALID.
 *   - Layouts are dense row-major in the order written, e.g. K [B][Hkv][Lmax][D]
 *     means element (b, h, j, d) sits at ((b*Hkv + h)*Lmax + j)*D + d.
 *   - Element type of q, k, v, out and of the caches is cfg->dtype (bf16 or
 *     fp32); the indexer projections are always fp32; accumulation is fp32.
 */
#ifndef RTP_H_
#define RTP_H_

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

/* Host-visible status codes. */
typedef enum rtp_status {
  RTP_OK = 0,
  RTP_ERR_INVALID = 1,   /* null pointer or scalar argument out of range */
  RTP_ERR_SHAPE = 2,     /* unsupported head_dim / group size / sizes */
  RTP_ERR_DTYPE = 3,     /* dtype not RTP_BF16 or RTP_FP32 */
  RTP_ERR_WORKSPACE = 4, /* workspace NULL, too small or not 256-byte aligned */
  RTP_ERR_CUDA = 5       /* a CUDA runtime call or kernel launch failed */
} rtp_status;

/* Device-side status bits OR-ed into *cache->status. */
#define RTP_DEV_SEQ_LEN  0x1  /* decode: seq_len[b] < 1 or > max_seq_len; sequence b skipped */
#define RTP_DEV_POSITION 0x2  /* append/prefill: a position outside [0, max_ctx); rows skipped */
#define RTP_DEV_TIMEOUT  0x4  /* decode or prefill: a bounded in-kernel wait gave up; that call's output is invalid */
#define RTP_DEV_BLOCKS   0x8  /* paged cache: out of free blocks, or a block or slot outside the pool */

typedef enum rtp_dtype { RTP_BF16 = 0, RTP_FP32 = 1 } rtp_dtype;

/* One attention layer.
 *   batch         B, sequences per call
 *   n_q_heads     Hq;  n_kv_heads Hkv;  G = Hq / Hkv query heads share a KV head
 *                 (GQA; q head hq reads KV head hq / G).  Supported G: 1, 2, 4, 8.
 *   head_dim      D: 64 or 128
 *   idx_dim       d, the indexer width: 16 (abstract, observation (2)), or 4, 8
 *                 or 32 for the pages' indexer-dimension ablation
 *                 (atlas.scime.ai summary, "Surprising findings": dimension 4).
 *                 Scores are q~ . k~ / sqrt(d), with 1/sqrt(d) rounded to fp32.
 *   max_ctx       Lmax, cache capacity per sequence (positions [0, Lmax));
 *                 at most 2^23
 *   n_sink        S >= 0: positions [0, S) are always attended (sinks)
 *   window        W >= 1: the last W positions up to and including the query
 *                 position are always attended (sliding window)
 *   top_p         p in (0, 1]: retrieval heads keep the smallest set of tokens
 *                 whose indexer softmax mass reaches p (>= p), ties to the lower
 *                 token index; p = 1 keeps every token
 *   rope_base     rotary base (10000 for Qwen3); rotate-half convention
 *   retrieval_mask bit h set => KV head h is a retrieval head.  Retrieval
 *                 heads are ranked r = 0..R-1 in increasing h; R <= 64
 *   dtype         rtp_dtype of q, k, v, out and the caches
 *   local_cap     0: every KV head keeps the whole context in the cache.
 *                 > 0 (ring mode, at least `window`): local heads keep only
 *                 the S sinks and a ring of local_cap window rows, so the cache
 *                 holds the full context only for retrieval heads (abstract:
 *                 the full KV cache is kept for retrieval heads only).  A
 *                 prefill chunk of T tokens then needs local_cap >= T + W - 1.
 *                 Ignored (whole context kept) when S + local_cap >= max_ctx.
 *   top_k         0: top-p selection.  k > 0: static top-k, the pages' fixed-
 *                 budget baseline (atlas.scime.ai summary, "Key results" and
 *                 "Baselines": static top-k): retrieval query heads keep the k
 *                 highest indexer scores (ties to the lower index; every token
 *                 when k >= the context), united with sinks and window as for
 *                 top-p.  Decode only: rtp_prefill_attn returns RTP_ERR_SHAPE.
 */
typedef struct rtp_layer_cfg {
  int batch;
  int n_q_heads;
  int n_kv_heads;
  int head_dim;
  int idx_dim;
  int max_ctx;
  int n_sink;
  int window;
  float top_p;
  float rope_base;
  uint64_t retrieval_mask;
  int dtype;
  int local_cap;
  int top_k;
} rtp_layer_cfg;

/* The layer's cache (device memory owned by the caller; sizes from
 * rtp_cache_bytes):
 *   k       [B][Hkv][Lmax][D]  keys after RoPE at their own position
 *   v       [B][Hkv][Lmax][D]  values
 *           In ring mode (cfg->local_cap > 0) k and v are [B][rows][D]: per
 *           sequence the KV heads follow one another in order h = 0..Hkv-1,
 *           a retrieval head taking Lmax rows (position j in row j) and a local
 *           head S + local_cap rows (position j < S in row j, position j >= S
 *           in row S + (j - S) mod local_cap).
 *   kidx    [B][R][Lk][d]      d-dim indexer keys k~ = W_k k_pre, one row per
 *                              token for each retrieval KV head (pre-RoPE);
 *                              Lk = Lmax, except Lmax rounded up to even when a
 *                              row is 8 bytes (bf16, d = 4), so that every
 *                              (b, r) block starts on a 16-byte boundary
 *   status  one int of device-side error bits (see RTP_DEV_*), zeroed by the
 *           caller before first use
 */
typedef struct rtp_cache {
  void* k;
  void* v;
  void* kidx;
  int* status;
} rtp_cache;

/* Host.  Bytes of each cache buffer for cfg.  Any output pointer may be NULL. */
int rtp_cache_bytes(const rtp_layer_cfg* cfg, size_t* k_bytes, size_t* v_bytes,
                    size_t* kidx_bytes);

/* Host.  Scratch bytes rtp_decode_attn needs for cfg (any max_seq_len <= max_ctx). */
int rtp_decode_workspace_bytes(const rtp_layer_cfg* cfg, size_t* bytes);

/* Host.  Scratch bytes rtp_prefill_attn needs for cfg and chunk length T. */
int rtp_prefill_workspace_bytes(const rtp_layer_cfg* cfg, int T, size_t* bytes);

/* Append T tokens per sequence to the cache.
 *
 * For every sequence b, token t and KV head h, at position pos = start_pos[b] + t:
 *   k[b][h][pos] = RoPE(k_pre[b][t][h], pos)            (stored in dtype)
 *   v[b][h][pos] = v_in[b][t][h]
 *   kidx[b][r][pos] = W_k^(r) k_pre[b][t][h]              (retrieval head h of rank r;
 *                                                         fp32 accumulation, stored in dtype)
 * The indexer key is taken BEFORE RoPE, as the pages' "pre-RoPE" projection
 * says (atlas.scime.ai summary, "Approach" and its one-line summary).
 *
 *   k_pre, v_in  [B][T][Hkv][D] dtype, device
 *   start_pos    [B] int32, device
 *   w_k          [R][d][D] fp32, device (may be NULL when R = 0)
 * Rows with pos outside [0, max_ctx) are skipped and set RTP_DEV_POSITION.
 */
int rtp_append_kv(const rtp_layer_cfg* cfg, const rtp_cache* cache, const void* k_pre,
                  const void* v_in, const int* start_pos, int T, const float* w_k,
                  void* stream);

/* One decode step: the query of sequence b sits at position seq_len[b] - 1 (the
 * token just appended with rtp_append_kv) and sees positions [0, seq_len[b]).
 *
 * Local KV heads: exact attention over sinks [0, S) and window
 * [seq_len-W, seq_len) (atlas.scime.ai summary, "Approach").
 * Retrieval KV heads, for each of their G query heads separately:
 *   q~ = W_q^(r) q_pre (fp32), s_j = q~ . kidx_j / sqrt(d) for every cached j
 *   (fp32; for a bf16 layer on tensor cores from q~'s bf16 high and low parts,
 *   the fp32 score to about 2^-17 of the score),
 *   P = softmax(s); keep the smallest set, ordered by (P desc, j asc), whose
 *   mass reaches top_p (abstract, observations (2)-(3)); attend exactly over
 *   that set united with the sinks and the window.
 * Attention: softmax(RoPE(q, pos) . k_j / sqrt(D)) over the attended rows.
 *
 *   q_pre        [B][Hq][D] dtype, device, pre-RoPE queries
 *   seq_len      [B] int32, device, 1 <= seq_len[b] <= max_seq_len
 *   max_seq_len  host int, an upper bound on seq_len (sizes the grid);
 *                0 means cfg->max_ctx
 *   w_q          [R][d][D] fp32, device
 *   out          [B][Hq][D] dtype, device
 *   sel_bitmask  optional (NULL to skip) [B][R*G][ceil(max_ctx/32)] uint32: bit
 *                j of head (b, r*G+g) is set iff token j is in that query head's
 *                top-p set (before the sinks/window union).  Words covering
 *                positions >= max_seq_len are not written.
 *   sel_count    optional [B][R*G] int32: size of each top-p set
 *   workspace    >= rtp_decode_workspace_bytes, 256-byte aligned, device; its
 *                contents need no initialisation and are clobbered
 * A sequence with an invalid seq_len is skipped (its out rows untouched) and
 * sets RTP_DEV_SEQ_LEN.
 * q_pre, w_q and seq_len are read before the kernels wait for the work already
 * on the stream (only the cache reads wait): they must not be written by a
 * kernel that may still be running when this call's kernels start, such as an
 * earlier kernel launched with programmatic dependent launch.
 * The bounded waits inside the call (on the asynchronous copies of the
 * indexer keys, of the scores and of the sink/window rows) give up after about
 * 0.4 s; the call's output is then invalid and RTP_DEV_TIMEOUT is set.
 */
int rtp_decode_attn(const rtp_layer_cfg* cfg, const rtp_cache* cache, const void* q_pre,
                    const int* seq_len, int max_seq_len, const float* w_q, void* out,
                    uint32_t* sel_bitmask, int* sel_count, void* workspace,
                    size_t workspace_bytes, void* stream);

/* Attention mass recall of a decode step's retrieval heads, a diagnostic the
 * method is evaluated by (atlas.scime.ai summary, "Experimental setup",
 * metrics): for each sequence b and retrieval query head r*G+g, the share of
 * the full causal attention's softmax mass, softmax(RoPE(q, L-1) . k_j /
 * sqrt(D)) over every j in [0, L), L = seq_len[b], that the rows the decode
 * step attended carry: the top-p set of sel_bitmask united with the sinks
 * [0, S) and the window [L-W, L).  fp32 arithmetic; a full-attention pass
 * over the retrieval heads' keys, so it costs about a dense decode step.
 *
 *   q_pre, seq_len, max_seq_len  as for the rtp_decode_attn call that wrote
 *                sel_bitmask (same cache contents)
 *   sel_bitmask  [B][R*G][ceil(max_ctx/32)] uint32, device, as rtp_decode_attn
 *                writes it
 *   recall       [B][R*G] float, device, in [0, 1]
 *   workspace    device, 256-byte aligned, contents clobbered; a workspace of
 *                rtp_decode_workspace_bytes bytes is always large enough
 * A sequence with an invalid seq_len is skipped (its recall entries untouched).
 * With no retrieval heads the call does nothing.
 */
int rtp_decode_recall(const rtp_layer_cfg* cfg, const rtp_cache* cache, const void* q_pre,
                      const int* seq_len, int max_seq_len, const uint32_t* sel_bitmask,
                      float* recall, void* workspace, size_t workspace_bytes, void* stream);

/* Size of the fixed device scratch array behind rtp_decode_attn_noalloc. */
#define RTP_NOALLOC_SCRATCH_BYTES (32u << 20)

/* rtp_decode_attn without a caller workspace, for callers that cannot
 * allocate device memory: plug-ins inside a host framework that owns the
 * device memory pool, latency-critical callers that cannot accept
 * cudaMalloc's implicit synchronisation, plain C callers holding only their
 * input and output buffers.  (The paper has no counterpart; this is an
 * interface convenience.)
 *
 * Arguments, results and errors are those of rtp_decode_attn minus
 * `workspace`/`workspace_bytes`: the scratch lives in one library-owned
 * device array of RTP_NOALLOC_SCRATCH_BYTES (32 MiB), reserved on every GPU
 * that loads the library until the process exits.  The call allocates
 * nothing.
 *   - Configurations needing more scratch than that (rtp_decode_workspace_bytes
 *     > RTP_NOALLOC_SCRATCH_BYTES) return RTP_ERR_WORKSPACE, nothing enqueued.
 *   - All calls share the array and it keeps the last call's contents; the
 *     kernels clear what must start at zero.  Calls whose device work
 *     overlaps (several streams or threads) race on it: serialise them.
 *   - The first call on each device looks up the array's device address with
 *     that device current and caches it; make that first call before any
 *     stream capture.  The cached address is not looked up again: do not use
 *     this entry point after a cudaDeviceReset in the same process.
 */
int rtp_decode_attn_noalloc(const rtp_layer_cfg* cfg, const rtp_cache* cache, const void* q_pre,
                            const int* seq_len, int max_seq_len, const float* w_q, void* out,
                            uint32_t* sel_bitmask, int* sel_count, void* stream);

/* One causal prefill chunk: query row t of sequence b sits at position
 * i = start_pos[b] + t and sees positions [0, i].  The chunk's keys and values
 * must already be in the cache (rtp_append_kv with the same start_pos and T).
 * Per row the layer computes exactly what rtp_decode_attn computes for a
 * query at position i (top-p over the indexer scores of [0, i] for retrieval
 * query heads; sinks and window [i-W+1, i] for every head).  The indexer
 * scores are computed on tensor cores from q~ split into a bf16 high part and
 * a bf16 low part accumulated in fp32 (the fp32 score to about 2^-17 of the
 * score), with exactly the arithmetic rtp_decode_attn uses for a bf16 layer:
 * a row's top-p set equals the decode step's at that position, bit for bit.
 * The attention itself runs on tensor cores in bf16 with fp32 accumulation
 * (atlas.scime.ai summary, "Approach"; abstract, observations (2)-(3)).
 * cfg->dtype must be RTP_BF16.
 *
 *   q_pre        [B][T][Hq][D] bf16, device
 *   start_pos    [B] int32, device; 0 <= start_pos[b] and start_pos[b] + T <= max_ctx
 *                (else the sequence is skipped and RTP_DEV_POSITION is set)
 *   w_q          [R][d][D] fp32, device
 *   out          [B][T][Hq][D] bf16, device
 *   sel_bitmask  optional [B][R*G][T][ceil(max_ctx/32)] uint32: row (b, r*G+g, t)
 *                has bit j set iff token j is in that row's top-p set; words
 *                past position i of the row are not written
 *   sel_tau      optional [B][R*G][T] float: score of the last kept token
 *                (-inf when p = 1 keeps every token)
 *   sel_jcut     optional [B][R*G][T] int32: tokens with score == sel_tau are kept
 *                iff their index <= sel_jcut (so membership is
 *                s_j > tau || (s_j == tau && j <= jcut))
 *   sel_count    optional [B][R*G][T] int32: size of the row's top-p set
 *   workspace    >= rtp_prefill_workspace_bytes(cfg, T), 256-byte aligned.  It
 *                holds a per-row top-p bitmask for a block of rows at a time;
 *                the block is sized so the workspace stays under 1 GiB, and
 *                longer chunks run block by block.
 * Ring mode (cfg->local_cap > 0) needs local_cap >= T + W - 1, else
 * RTP_ERR_SHAPE.
 */
int rtp_prefill_attn(const rtp_layer_cfg* cfg, const rtp_cache* cache, const void* q_pre,
                     const int* start_pos, int T, const float* w_q, void* out,
                     uint32_t* sel_bitmask, float* sel_tau, int* sel_jcut, int* sel_count,
                     void* workspace, size_t workspace_bytes, void* stream);

/* ---------------------------------------------------------------------------
 * The paged 8-bit cache: K and V of many requests in one pool of blocks.
 *
 * A block holds block_size consecutive positions of one request, for every KV
 * head, as e4m3 values with one fp32 scale per (block, KV head) for K and one
 * for V: half the bytes of a bf16 cache that keeps every position of every head
 * (a ring, rtp_layer_cfg.local_cap, keeps fewer of local heads' and may be
 * smaller).  Scales are powers of two, so a
 * stored value times its scale is exact in bf16 and fp32, and a block whose
 * scale grows keeps its values (only what falls below e4m3's smallest step is
 * rounded again).  A request's blocks may lie anywhere in the pool; its row of
 * the block table names them in order.  A step of a serving loop is
 *     rtp_page_plan                       (once)
 *     rtp_append_q8, rtp_attn_q8          (each layer)
 * with the step's new tokens of all requests packed one after another:
 * request b's tokens are rows [cu[b], cu[b + 1]) of every packed array.
 *
 * The layer is rtp_layer_cfg's: retrieval KV heads attend to the whole
 * context, local ones to sinks and window.  There is no indexer on this cache
 * and no ring: cfg->top_p must be 1, cfg->top_k and cfg->local_cap 0
 * (RTP_ERR_SHAPE otherwise); cfg->idx_dim is not used.  cfg->max_ctx bounds a
 * request's positions, and a row of the block table has
 * ceil(max_ctx / block_size) entries.
 */

/* Pool of blocks (device memory owned by the caller).
 *   k, v              [n_blocks][Hkv][block_size][D] e4m3
 *   k_scale, v_scale  [n_blocks][Hkv] fp32, powers of two of at least 2^-64
 *                     (smaller ones are read as 2^-64); the entries of a block
 *                     that was never appended to are not read
 *   status            one int of RTP_DEV_* bits, as in rtp_cache
 *   n_blocks          n_blocks * Hkv * block_size < 2^31
 *   block_size        16, 32, 64 or 128 positions
 * rtp_append_q8 never stores a NaN in v (see there), and rtp_attn_q8 relies on
 * that for rows below a request's length; other rows may hold anything.
 */
typedef struct rtp_q8_cache {
  void* k;
  void* v;
  float* k_scale;
  float* v_scale;
  int* status;
  int n_blocks;
  int block_size;
} rtp_q8_cache;

/* Rotary axes.  The rotary pair k (dims k and k + D/2) of a token turns by
 * pos[axis[k]][token] * rope_base^(-2k/D): one axis for text, three (time,
 * height, width) for pictures and video, the pairs shared out between them.
 * A NULL rtp_rope_axes means one axis.  Positions are any int32. */
typedef struct rtp_rope_axes {
  int n_axes;             /* 1 .. 4 */
  unsigned char axis[64]; /* of each pair k < D/2, below n_axes */
} rtp_rope_axes;

/* Host.  Bytes of each of k and v, and of each scale array. */
int rtp_q8_cache_bytes(const rtp_layer_cfg* cfg, int n_blocks, int block_size, size_t* kv_bytes,
                       size_t* scale_bytes);

/* Block tables and slot map of one step, from the requests' lengths.
 *
 * Request b holds ctx_len[b] cached positions in its first
 * have = ceil(ctx_len[b] / block_size) table entries.
 *   new_len[b] >= 0: it brings that many tokens.  It takes the
 *     need = ceil((ctx_len[b] + new_len[b]) / block_size) - have blocks that
 *     they lack from the top of the stack of free blocks, in request order:
 *     table entry have + i is free_list[top - 1 - before[b] - i], before[b]
 *     the need of the requests ahead of it.  seq_len[b] = ctx_len[b] +
 *     new_len[b].
 *   new_len[b] < 0: it has ended.  Its blocks go on top of the stack, in table
 *     order, before any is taken; seq_len[b] = 0.  Its table row stays as it
 *     is and means nothing any more.
 * `top` is n_free plus the blocks of ended requests.  Requests must not share
 * blocks.
 *
 * A request's length may fall between steps (a draft's tokens were rejected).  The plan
 * knows its blocks by ctx_len alone: where ceil(length / block_size) falls too, table
 * entries from there on are no longer its own and would be lost.  The caller gives them
 * back before the next plan, by one in which they are a request of their own that ends:
 * batch rows of a table that begin with those entries, ctx_len[b] = block_size times
 * their number (max_ctx where that is less), new_len[b] = -1, max_tokens = 0.
 *
 * A request that cannot be served is refused: it takes no block, seq_len[b] =
 * ctx_len[b], its tokens get slot -1 (so rtp_append_q8 skips them), the others
 * are served as if it were there.  That is where before[b] + need > top
 * (RTP_DEV_BLOCKS), ctx_len[b] + new_len[b] > max_ctx or
 * its packed tokens pass max_tokens (RTP_DEV_POSITION).  ctx_len[b] outside [0, max_ctx]
 * counts as 0 cached and no new tokens (RTP_DEV_SEQ_LEN).
 * rtp_attn_q8 knows nothing of refusals: a refused request keeps its rows in cu_new,
 * so its outputs there are made as if its newest cached tokens were the new ones (or
 * left as they were, where it has fewer of them), and mean nothing.  Where *status has one of these bits, its rows are those with slot -1
 * ahead of cu_new[B]; the caller drops them, or plans the step again without it.
 *
 *   ctx_len, new_len  [B] int32, device
 *   block_table       [B][ceil(max_ctx / block_size)] int32, device, in/out
 *   free_list         [free_cap] int32, device, in/out: entries [0, n_free) are the stack
 *   n_free            one int32, device, in [0, free_cap]
 *   seq_len           [B] int32, device, out; may be ctx_len
 *   cu_new            [B + 1] int32, device, out: first packed row of each request, then their number
 *   slot_map          [max_tokens] int64, device, out: block * block_size + offset of each packed
 *                     token; -1 for refused ones and for rows past the last token
 *   positions         [max_tokens] int32, device, out: position of each packed token (0 past the last)
 *   n_free_out        one int32, device, out; may be n_free
 * A block number below 0 met in the table or the stack gives its tokens slot -1, and a
 * block that the stack has no room for is dropped (both RTP_DEV_BLOCKS).
 * cfg gives batch (at most 4096 here) and max_ctx. */
int rtp_page_plan(const rtp_layer_cfg* cfg, int block_size, const int* ctx_len, const int* new_len,
                  int* block_table, int* free_list, int free_cap, const int* n_free, int* seq_len,
                  int* cu_new, int64_t* slot_map, int* positions, int max_tokens, int* n_free_out,
                  int* status, void* stream);

/* Append packed tokens to the pool.
 *
 * For packed token t with slot_map[t] = block * block_size + o >= 0, KV head h:
 *   k row (block, h, o) = e4m3(RoPE(k_pre[t][h], pos[.][t]) / k_scale[block][h])
 *   v row (block, h, o) = e4m3(v_in[t][h] / v_scale[block][h])
 * to nearest, ties to even, from the rotation in 64 bits (one rounding).  The
 * scale of a (block, head) becomes the least power of two, at least 2^-64, with
 * |x| <= 448 scale for every value this call stores there, and not below its
 * former one if the block held rows before (o > 0 for the call's first token
 * in it); where it grows, those rows are rounded again to the new scale.
 * A (token, head) row with a value that is not finite (in K, as rotated, or V) is stored
 * as K all NaN and V all 0 and does not count for the scales: queries that see
 * it answer NaN, no other query is touched.
 *
 *   k_pre, v_in  [n_tokens][Hkv][D] dtype, device; token t's [Hkv][D] slice
 *                starts at element t * k_stride (v_stride) and is dense, so the
 *                fused projection's output can be passed as it is.  Strides are
 *                multiples of 16 bytes, at least Hkv * D; 0 means Hkv * D
 *   slot_map     [n_tokens] int64, device; negative: the token is skipped
 *   pos          [n_axes][n_tokens] int32, device
 *   rope         host, or NULL for one axis
 * Tokens of one block have to be consecutive, in ascending slots (as
 * rtp_page_plan gives them): a block named by two separate runs, or a slot
 * named twice, ends up with unspecified values.  Slots past the pool are
 * skipped (RTP_DEV_BLOCKS). */
int rtp_append_q8(const rtp_layer_cfg* cfg, const rtp_q8_cache* cache, const void* k_pre,
                  int64_t k_stride, const void* v_in, int64_t v_stride, const int64_t* slot_map,
                  const int* pos, const rtp_rope_axes* rope, int n_tokens, void* stream);

/* Host.  Scratch bytes of rtp_attn_q8 for calls of up to n_tokens packed
 * queries, max_q of one request and max_seq_len positions (0: cfg->max_ctx).
 * batch * n_kv_heads * (ceil(max_seq_len / 32) + 16) * c has to stay below 2^31
 * (RTP_ERR_SHAPE, here and in rtp_attn_q8); c = ceil(max_q G / 8) for fp32
 * layers, at most 2 for bf16 ones. */
int rtp_attn_q8_workspace_bytes(const rtp_layer_cfg* cfg, int block_size, int n_tokens, int max_q,
                                int max_seq_len, size_t* bytes);

/* Attention of packed queries over the paged cache.
 *
 * Request b's n = cu_q[b + 1] - cu_q[b] queries are the last n of its
 * seq_len[b] cached positions: query row t sits at i = seq_len[b] - n + t and
 * sees positions [0, i]; local KV heads see of them the sinks [0, S) and the
 * window [i - W + 1, i].
 *   out = softmax(RoPE(q, pos) . k_j / sqrt(D)) v_j    k_j, v_j as stored, times their scales
 * One token a request (decode), a few, or chunks, in any mix.  Arithmetic is
 * on tensor cores with fp32 accumulation; queries (scaled by a power of two a
 * row) and softmax weights enter them as fp16.  Queries enter as two fp16 parts
 * (22 bits) where max_q * G <= 8, and for fp32 layers, whose weights do so too.
 * Value scales of any size may lie beside one another.  Where max_q * G > 32, in
 * bf16, requests of more than 32 query rows (n G) a KV head, and a batch of one,
 * lose bits of query rows below 2^-64 and want scores q . k / sqrt(D) of less
 * than 2^23: larger ones may answer NaN.  Blocks may be shared between requests.
 * v holds no NaN at cached positions (rtp_append_q8 writes none): a weight of 0
 * does not hide one.
 *
 *   q_pre        [n_tokens][Hq][D] dtype, device, pre-RoPE; rows q_stride
 *                elements apart (multiple of 16 bytes, at least Hq * D; 0 means Hq * D)
 *   cu_q         [B + 1] int32, device, ascending from 0; rows from cu_q[B] on are left as they were in `out`
 *   seq_len      [B] int32, device
 *   block_table  [B][ceil(max_ctx / block_size)] int32, device
 *   pos          [n_axes][n_tokens] int32, device
 *   max_q        host: bound on a request's queries
 *   max_seq_len  host: bound on seq_len (0: cfg->max_ctx)
 *   out          [n_tokens][Hq][D] dtype, device, dense
 *   workspace    >= rtp_attn_q8_workspace_bytes, 256-byte aligned, device; needs
 *                no initialisation, clobbered; calls that may overlap need one each
 * A request with seq_len[b] < n, or above max_seq_len, is skipped, its rows left as
 * they were (RTP_DEV_SEQ_LEN); so is one with n < 0, n > max_q or rows past
 * n_tokens (RTP_DEV_POSITION).  Positions whose block number lies outside the pool
 * count as not there (RTP_DEV_BLOCKS); a query that sees none gets 0. */
int rtp_attn_q8(const rtp_layer_cfg* cfg, const rtp_q8_cache* cache, const void* q_pre,
                int64_t q_stride, const int* cu_q, const int* seq_len, const int* block_table,
                const int* pos, const rtp_rope_axes* rope, int n_tokens, int max_q, int max_seq_len,
                void* out, void* workspace, size_t workspace_bytes, void* stream);

/* Kernel stages, for rtp_trace_stage. */
typedef enum rtp_stage {
  RTP_STAGE_APPEND = 0,         /* rtp_append_kv: RoPE + cache + indexer-key store */
  RTP_STAGE_DECODE_SCORE = 1,   /* decode: indexer scores over the d-dim key cache */
  RTP_STAGE_DECODE_SELECT = 2,  /* decode: exact top-p selection, bitmask, kept-row attention */
  RTP_STAGE_DECODE_LOCAL = 3,   /* decode: sink/window attention of every KV head (beside the selection), final merge */
  RTP_STAGE_PREFILL_INDEX = 4,  /* prefill: per-row exact top-p selection */
  RTP_STAGE_PREFILL_ATTN = 5,   /* prefill: masked causal attention */
  RTP_STAGE_PAGE_PLAN = 6,      /* rtp_page_plan */
  RTP_STAGE_APPEND_Q8 = 7,      /* rtp_append_q8 */
  RTP_STAGE_ATTN_Q8 = 8,        /* rtp_attn_q8 (all of its kernels) */
  RTP_STAGE_COUNT = 9
} rtp_stage;

/* Host.  Optional instrumentation (no work is skipped or added).  Arms a
 * one-shot trace: the next kernel of `stage` launched by an rtp_* call on this
 * host thread is bracketed by cudaEventRecord(start_event) and
 * cudaEventRecord(stop_event) on its launch stream.  Events are cudaEvent_t
 * passed as void*, created and owned by the caller (with timing enabled to
 * read cudaEventElapsedTime).  A stage launched several times by one call
 * (prefill chunks longer than one row block) records around its first launch.
 * NULL events disarm the stage.  Returns RTP_ERR_INVALID for an unknown stage. */
int rtp_trace_stage(int stage, void* start_event, void* stop_event);

/* Host.  Test hook for the bounded waits of rtp_decode_attn (no counterpart
 * in the paper).  Arms the next rtp_decode_attn call on this host thread to
 * wait for completion flags that never reach the awaited value, giving up
 * after `polls` polls (about 100 ns each): the call then sets RTP_DEV_TIMEOUT,
 * its output is invalid, and the GPU stays usable.  polls <= 0 disarms.
 * Returns RTP_OK. */
int rtp_debug_wait_expiry(int polls);

/* Host.  Message for the last non-OK return on this thread ("" if none). */
const char* rtp_last_error(void);

/* Host.  Library version string. */
const char* rtp_version(void);

#ifdef __cplusplus
}
#endif

#endif /* RTP_H_ */
