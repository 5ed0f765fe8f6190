/*
 * nsa.h -- C ABI of the B200 (sm_100a) Native Sparse Attention / MoBA
 * forward library (libnsa_b200.so).
 *
 * Operations (the sources print no equations; each operation is the plain
 * reading of their prose with the constants of the workload statement):
 *   - nsa_compress_kv: token compression, "Zhang Xiaojun EP94 notes" §五 branch
 *     one; lchairun.cn NSA article, compression paragraph.
 *   - nsa_prefill / nsa_decode: the three-branch NSA forward, EP94 notes §五
 *     (compressed, selected and sliding-window branches, gating) and §六 (GQA
 *     group-shared selection); lchairun.cn NSA article, selection, window and
 *     gate paragraphs (decode is bound by KV bytes moved).
 *   - moba_prefill: MoBA, EP94 notes §九/§十/§十六 (mean-pooled block keys,
 *     parameter-free per-head top-k, block 512, top-3); LateTalk ep.103 (the
 *     query's own block is always attended).
 *
 * Conventions for every call:
 *   - Tensors are plain device pointers, contiguous, row-major, in the layout
 *     given per argument ("bshd": [batch, tokens, heads, head_dim]). The caller
 *     allocates and owns all of them; the library never allocates or frees
 *     device memory and never synchronises, except nsa_check.
 *   - `stream` is a cudaStream_t passed as void* (NULL = legacy default
 *     stream). All work is enqueued asynchronously on it.
 *   - Arguments are validated on the host before anything is launched; on an
 *     error nothing is written and a status other than NSA_OK is returned,
 *     with a message in nsa_last_error_detail().
 *   - Launch failures return NSA_ERR_CUDA. Faults found on the device (a
 *     bounded wait that gave up, a sequence length, append position, page
 *     number or token offset out of range) set a
 *     per-device error word that nsa_check reports.
 *   - Thread safety: calls on different streams may run concurrently; the
 *     error-detail string is thread-local.
 */
#ifndef NSA_B200_H_
#define NSA_B200_H_

#include <stddef.h>
#include <stdint.h>

#if defined(__GNUC__)
#define NSA_API __attribute__((visibility("default")))
#else
#define NSA_API
#endif

#ifdef __cplusplus
extern "C" {
#endif

typedef enum {
  NSA_OK = 0,
  NSA_ERR_INVALID_ARGUMENT = 1, /* bad pointer, shape, size or mode          */
  NSA_ERR_UNSUPPORTED = 2,      /* valid but not implemented (e.g. head dim) */
  NSA_ERR_WORKSPACE_TOO_SMALL = 3,
  NSA_ERR_CUDA = 4,             /* a CUDA runtime call or launch failed      */
  NSA_ERR_DEVICE_TIMEOUT = 5    /* a bounded device-side wait gave up        */
} nsa_status;

typedef enum { NSA_DTYPE_F32 = 0, NSA_DTYPE_BF16 = 1 } nsa_dtype;

/* Operation ids for nsa_workspace_size. */
typedef enum {
  NSA_OP_COMPRESS = 0,
  NSA_OP_PREFILL = 1,
  NSA_OP_DECODE = 2,
  NSA_OP_MOBA_PREFILL = 3,
  NSA_OP_PREFILL_BACKWARD = 4,
  NSA_OP_DECODE_Q8 = 5,
  NSA_OP_PREFILL_Q8 = 6
} nsa_op;

/* Problem description shared by all calls.
 *   B, T       batch and tokens (prefill: every sequence has T tokens; decode:
 *              T is the KV-cache capacity, the live length comes from seq_lens;
 *              MoBA: tokens per sequence).
 *   Hq, Hkv    query heads and KV heads; Hq % Hkv == 0; query head h reads KV
 *              head h / (Hq / Hkv) (consecutive heads form a GQA group).
 *   d          head dimension: 64 or 128.
 *   cmp_block, cmp_stride   compression length l and stride s (l >= s >= 1).
 *   sel_block  selection block size (NSA: 64); MoBA block size m (512).
 *   top_n      NSA: blocks kept per (token, KV head), block 0 included;
 *              MoBA: blocks kept per (token, head), the own block included.
 *   window     sliding-window length w (>= 1).
 *   softmax_scale  0 selects 1/sqrt(d).
 *   gate_mode  0: g = sigmoid(q . Wg) per branch (Wg [d,3], order cmp, slc,
 *              win, raw unscaled q); 1: g = fixed_gates for every query.
 *   dtype      element type of q, k, v, compressed k/v and out.
 *   top_p      0: keep top_n blocks. In (0, 1]: adaptive selection (lchairun
 *              NSA article, adaptive sparsification): block 0, then the other
 *              blocks by score (ties to the lower index) up to the first prefix
 *              whose score sum reaches top_p times the sum over all candidate
 *              blocks, at most top_n blocks; unused sel_idx slots hold -1.
 *   sel_mode   block scores the NSA selection ranks: 0 the compressed-branch
 *              probability mass on each block, summed over the GQA group
 *              (EP94 notes §五); 1 the Quest-style block bound of the pages'
 *              selection ablation (EP94 notes §八): with kmin, kmax the
 *              element-wise min and max of the block's keys up to the query,
 *              sum over the group's heads of sum_e max(q_e kmin_e, q_e kmax_e).
 *              Mode 1 needs top_p == 0. Prefill (bf16, d = 128, 16 heads per
 *              KV head, selection block 64) takes it from a block-bounds
 *              table built inside the call; decode takes that table from the
 *              caller through nsa_decode_quest (nsa_decode computes the bounds
 *              from the keys, on the CUDA-core path).
 * MoBA uses B, T, Hq, Hkv, d, sel_block, top_n, softmax_scale and dtype. */
typedef struct {
  int B, T, Hq, Hkv, d;
  int cmp_block, cmp_stride;
  int sel_block, top_n, window;
  float softmax_scale;
  int gate_mode;
  float fixed_gates[3];
  nsa_dtype dtype;
  float top_p;
  int sel_mode;
} nsa_params;

/* Bytes of caller-provided device workspace `op` needs for `p` (0 is
 * possible). The workspace must be 256-byte aligned. */
NSA_API nsa_status nsa_workspace_size(const nsa_params* p, int op, size_t* bytes);

/* Number of compressed blocks for T tokens: floor((T - l) / s) + 1, or 0 when
 * T < l. Compressed block i covers tokens [i*s, i*s + l - 1]. */
NSA_API int nsa_num_cmp_blocks(int T, int cmp_block, int cmp_stride);

/* Token compression (EP94 notes §五 branch one).
 *   k, v       [B, T, Hkv, d] dtype.
 *   w_cmp      [cmp_block] fp32 weights shared by keys and values.
 *   k_cmp, v_cmp  [B, Nc, Hkv, d] dtype outputs, Nc = nsa_num_cmp_blocks(T):
 *              k_cmp[b,i,g,:] = sum_j w_cmp[j] * k[b, i*s + j, g, :]
 *              (accumulated in fp64, rounded once to dtype, nearest-even). */
NSA_API nsa_status nsa_compress_kv(const nsa_params* p, const void* k, const void* v,
                           const float* w_cmp, void* k_cmp, void* v_cmp, void* stream);

/* NSA causal prefill (EP94 notes §五, §六).
 *   q          [B, T, Hq, d]; k, v [B, T, Hkv, d]; k_cmp, v_cmp [B, Nc, Hkv, d]
 *              (from nsa_compress_kv).
 *   w_gate     [d, 3] fp32 (ignored when gate_mode == 1; may then be NULL).
 *   out        [B, T, Hq, d] dtype.
 *   sel_idx    [B, T, Hkv, top_n] int32 or NULL: the selected blocks of each
 *              (token, KV head), ascending, block 0 first, -1 padded when
 *              fewer than top_n blocks exist.
 *   workspace  device scratch of nsa_workspace_size(NSA_OP_PREFILL) bytes. */
NSA_API nsa_status nsa_prefill(const nsa_params* p, const void* q, const void* k, const void* v,
                       const void* k_cmp, const void* v_cmp, const float* w_gate, void* out,
                       int32_t* sel_idx, void* workspace, size_t ws_bytes, void* stream);

/* NSA prefill backward: gradients of L = sum(dout * out) of nsa_prefill
 * (EP94 notes §五: the compressed branch carries the gradient that trains the
 * selection; lchairun.cn NSA article, the paragraph on trainability). The
 * selected blocks are constants of the backward (the top-n choice is
 * discrete); gradients flow through the gates, the three attentions and the
 * compression, whose storage rounding is taken as the identity.
 *   q, k, v, k_cmp, v_cmp, w_gate  as passed to nsa_prefill; k_cmp, v_cmp are
 *              nsa_compress_kv(k, v, w_cmp).
 *   w_cmp      [cmp_block] fp32, the compression weights.
 *   sel_idx    [B, T, Hkv, top_n] int32: the forward's selected blocks (as
 *              nsa_prefill writes them); entries < 0, repeated, or past the
 *              row's own block are ignored.
 *   dout       [B, T, Hq, d] dtype.
 *   dq         [B, T, Hq, d] fp32 output.
 *   dk, dv     [B, T, Hkv, d] fp32 outputs (overwritten).
 *   dw_cmp     [cmp_block] fp32 output.
 *   dw_gate    [d, 3] fp32 output; zeros when gate_mode == 1 (may be NULL then).
 *   workspace  device scratch of nsa_workspace_size(NSA_OP_PREFILL_BACKWARD)
 *              bytes (caller-owned; contents need not be initialised).
 * Runs on CUDA cores in fp32; dk, dv and the compressed-branch gradients are
 * summed with atomics, so their last bits can vary between runs. top_n > 64
 * returns NSA_ERR_UNSUPPORTED. */
NSA_API nsa_status nsa_prefill_backward(const nsa_params* p, const void* q, const void* k,
                                const void* v, const void* k_cmp, const void* v_cmp,
                                const float* w_cmp, const float* w_gate, const int32_t* sel_idx,
                                const void* dout, float* dq, float* dk, float* dv, float* dw_cmp,
                                float* dw_gate, void* workspace, size_t ws_bytes, void* stream);

/* NSA single-token decode over a KV cache (EP94 notes §六; lchairun.cn NSA
 * article: decode moves the group's one shared KV subset).
 *   q          [B, Hq, d]: the query of the token at position seq_lens[b]-1.
 *   k_cache, v_cache  [B, T, Hkv, d] (T = capacity); positions < seq_lens[b]
 *              are live and include the current token.
 *   seq_lens   [B] int32 device array, 1 <= seq_lens[b] <= T (violations set
 *              the device error word and zero that sequence's output).
 *   k_cmp, v_cmp  [B, Nc(T), Hkv, d]; entries of blocks ending before
 *              seq_lens[b] are read.
 *   w_gate, out [B, Hq, d], sel_idx [B, Hkv, top_n], workspace: as prefill. */
NSA_API nsa_status nsa_decode(const nsa_params* p, const void* q, const void* k_cache,
                      const void* v_cache, const int32_t* seq_lens, const void* k_cmp,
                      const void* v_cmp, const float* w_gate, void* out, int32_t* sel_idx,
                      void* workspace, size_t ws_bytes, void* stream);

/* Streaming decode: appends one token per sequence to the caches (lchairun NSA
 * article: decode reads the compressed cache, which gains one block every s
 * tokens, plus the selected and most recent tokens; EP94 notes §五).
 *   k_new, v_new      [B, Hkv, d] dtype: the new token's keys and values.
 *   pos               [B] int32, device: where to write, the sequence's length
 *                     before the append (0 <= pos < T).
 *   k_cache, v_cache  [B, T, Hkv, d] dtype, written at [b, pos[b]].
 *   w_cmp             [cmp_block] fp32 (the weights given to nsa_compress_kv).
 *   k_cmp, v_cmp      [B, Nc, Hkv, d] dtype. When pos + 1 completes compressed
 *                     block i = (pos + 1 - l) / s (pos + 1 >= l and
 *                     (pos + 1 - l) % s == 0), entry i is written exactly as
 *                     nsa_compress_kv computes it; no other entry is touched.
 *   A position outside [0, T) writes nothing for that sequence and sets the
 *   device error word (nsa_check then returns NSA_ERR_INVALID_ARGUMENT). The
 *   caller passes seq_lens = pos + 1 to the next nsa_decode. */
NSA_API nsa_status nsa_append_kv(const nsa_params* p, const void* k_new, const void* v_new,
                                 const int32_t* pos, void* k_cache, void* v_cache,
                                 const float* w_cmp, void* k_cmp, void* v_cmp, void* stream);

/* Quest-style block bounds beside a KV cache, for nsa_decode_quest (EP94 notes
 * §八: the selection ablation's Quest-style block score).
 *   k_cache    [B, T, Hkv, d] dtype.
 *   seq_lens   [B] int32, device, 1 <= seq_lens[b] <= T.
 *   k_bounds   [B, nblk, Hkv, 2, d] dtype, nblk = ceil(T / sel_block):
 *              k_bounds[b, j, g, 0, :] is the element-wise maximum and
 *              k_bounds[b, j, g, 1, :] the minimum of the keys of selection
 *              block j among the first seq_lens[b] tokens (the block holding
 *              the last token covers the tokens so far). Entries of blocks at
 *              or past seq_lens[b] are not written. Uses B, T, Hkv, d,
 *              sel_block and dtype of p.
 *   A length outside [1, T] writes nothing for that sequence and sets the
 *   device error word (nsa_check: NSA_ERR_INVALID_ARGUMENT). */
NSA_API nsa_status nsa_block_bounds(const nsa_params* p, const void* k_cache,
                                    const int32_t* seq_lens, void* k_bounds, void* stream);

/* Keeps k_bounds current after nsa_append_kv wrote token pos[b] (0 <= pos[b]
 * < T): block pos[b] / sel_block then covers keys up to pos[b] (a block's
 * first token restarts its extremes).
 *   k_new      [B, Hkv, d] dtype (the appended keys); pos [B] int32, device. */
NSA_API nsa_status nsa_append_bounds(const nsa_params* p, const void* k_new, const int32_t* pos,
                                     void* k_bounds, void* stream);

/* NSA decode that ranks blocks by the Quest-style bound (p->sel_mode must be
 * 1; EP94 notes §八): for the query's group, sum over its heads of
 * sum_e max(q_e kmin_e, q_e kmax_e), with kmin / kmax read from k_bounds as
 * nsa_block_bounds / nsa_append_bounds keep them; block 0 and the n - 1 best
 * others (ties to the lower index) are kept, the three branches and gates are
 * nsa_decode's. Arguments as nsa_decode plus k_bounds; the workspace is
 * nsa_workspace_size(NSA_OP_DECODE). On shapes other than the bf16, d = 128,
 * 16 heads per KV head, selection block 64 fast path, the CUDA-core path
 * computes the bounds from the keys (k_bounds unused). */
NSA_API nsa_status nsa_decode_quest(const nsa_params* p, const void* q, const void* k_cache,
                                    const void* v_cache, const int32_t* seq_lens,
                                    const void* k_cmp, const void* v_cmp, const void* k_bounds,
                                    const float* w_gate, void* out, int32_t* sel_idx,
                                    void* workspace, size_t ws_bytes, void* stream);

/* nsa_decode without a workspace argument, for callers that cannot allocate
 * device memory: code that runs while a stream capture is in progress
 * (cudaMalloc is not permitted during a global-mode capture), real-time or
 * callback threads that must not block in an allocator, and hosts whose device
 * memory is owned by another runtime's pool. Nothing here states whether the
 * call itself can be captured into a graph.
 * The sources describe no such call; it has no counterpart in the method.
 *   Same arguments and results as nsa_decode, minus workspace / ws_bytes. The
 *   scratch is a static 64 MiB device array in this library, held on every GPU
 *   that loads it until the process exits. Shapes whose decode scratch
 *   (nsa_workspace_size(NSA_OP_DECODE)) exceeds 64 MiB are rejected with
 *   NSA_ERR_UNSUPPORTED before anything runs (32 sequences of 65536 tokens
 *   with 4 KV heads need about 39 MB).
 *   The first call on each device looks the scratch's address up (once, with
 *   that device current); make that first call before any stream capture.
 *   All calls share the one scratch: calls that overlap on the GPU (different
 *   streams, no ordering) race and corrupt each other's results. Nothing in
 *   it must start at zero: every call writes each scratch byte it reads.
 *   No device memory is allocated or freed, by this call or any library
 *   routine it uses. */
NSA_API nsa_status nsa_decode_noalloc(const nsa_params* p, const void* q, const void* k_cache,
                                      const void* v_cache, const int32_t* seq_lens,
                                      const void* k_cmp, const void* v_cmp, const float* w_gate,
                                      void* out, int32_t* sel_idx, void* stream);

/* MoBA causal prefill (EP94 notes §九/§十).
 *   q [B, T, Hq, d]; k, v [B, T, Hkv, d]; out [B, T, Hq, d].
 *   Block m = sel_block; each (token t, head h) keeps its own block t/m and the
 *   top_n - 1 earlier blocks by q . mean(K_block) (ties to the lower index),
 *   then one causal softmax over the kept tokens.
 *   sel_idx    [B, T, Hq, top_n] int32 or NULL (ascending, -1 padded). */
NSA_API nsa_status moba_prefill(const nsa_params* p, const void* q, const void* k, const void* v,
                        void* out, int32_t* sel_idx, void* workspace, size_t ws_bytes,
                        void* stream);

/* ---- 8-bit paged KV cache ------------------------------------------------
 *
 * K and V in e4m3 codes (1 sign, 4 exponent, 3 mantissa bits; largest 448),
 * in pages of sel_block tokens with one scale for each page and KV head: a
 * component is code * scale. The page is the NSA selection block, so the block
 * numbers that nsa_decode and nsa_decode_quest select address its pages. The
 * sources describe no 8-bit or paged cache; it has no counterpart there.
 *
 *   k_pages, v_pages  [num_pages, Hkv, sel_block, d] e4m3 bytes, 16-byte
 *              aligned (one head's page is contiguous).
 *   k_scale, v_scale  [num_pages, Hkv] fp32, positive; powers of two where
 *              nsa_append_q8 continues a page (it writes no others).
 *   page_table [B, ceil(T / sel_block)] int32: token x of sequence b is slot
 *              x % sel_block of page page_table[b, x / sel_block]. Entries of
 *              pages without a token that a call reads or writes are not
 *              used: those behind a sequence's end and, with NSA_KEYS_WINDOW,
 *              before the first query's window, whose pages may be gone. Sequences may share
 *              pages that none of them appends to.
 * All in device memory. Of nsa_params the calls use B, T (tokens a sequence
 * can have), Hq, Hkv, d, sel_block (16, 32, 64 or 128), dtype (of q, k, v and
 * outputs) and, for attention, softmax_scale, window and top_n. */
typedef struct {
  void* k_pages;
  void* v_pages;
  float* k_scale;
  float* v_scale;
  const int32_t* page_table;
  int num_pages;
} nsa_q8_cache;

/* Position rotation of the first `dim` components x of a key or query at
 * position t: for each of the dim / 2 pairs i, (x_a, x_b) becomes
 * (x_a cos - x_b sin, x_b cos + x_a sin) with cos = table[t, 0, i], sin =
 * table[t, 1, i]. NSA_ROPE_HALF: a = i, b = i + dim / 2. NSA_ROPE_PAIRS:
 * a = 2 i, b = 2 i + 1. Computed in fp32.
 *   table      [len, 2, dim / 2] fp32, device, 16-byte aligned.
 *   dim        a multiple of 16, at most d. */
typedef enum { NSA_ROPE_HALF = 0, NSA_ROPE_PAIRS = 1 } nsa_rope_style;
typedef struct {
  const float* table;
  int len;
  int dim;
  int style;
} nsa_rope;

/* Appends new tokens to the 8-bit cache; keys are rotated by their position on
 * the way, and so are the queries of the same tokens.
 *   k_new, v_new  [N, Hkv, d] dtype.
 *   pos        [B] int32, device: the sequence's length before the append; its
 *              i-th new token is written at position pos[b] + i.
 *   cu_new     [B + 1] int32, device, ascending, or NULL: the new tokens of
 *              sequence b are rows cu_new[b] .. cu_new[b + 1] - 1 (none is
 *              fine); rows outside are ignored. NULL: one token per sequence,
 *              row b (N == B).
 *   rope       NULL: no rotation.
 *   q, q_out   [N, Hq, d] dtype, or both NULL: the rotated queries (q_out == q
 *              is allowed).
 *   k_out, v_out  [N, Hkv, d] dtype, or both NULL: the new tokens as the cache
 *              holds them (rotated, quantised), rounded to dtype.
 * Per (page, head) of K and of V: with a the largest finite magnitude the call
 * writes there, need = the smallest power of two >= 2^-126 with a <= 448 need.
 * The scale becomes need when the call writes the page's first slot, else
 * max(scale, need). When it changes, the codes of the page's other slots are
 * re-coded so that they stand for the same values (exact but for those that
 * fall below e4m3's normal range; in a page that the call begins, values of
 * stale slots beyond the new range become NaN). A component's code is
 * x / scale rounded once from the fp32 x, to nearest even; NaN and infinities
 * become NaN. So a page filled by several calls holds what one call's scale
 * gives, up to the re-coded small values.
 *   A sequence whose positions leave [0, T) or the rotation table is not
 *   written (device error word; nsa_check: NSA_ERR_INVALID_ARGUMENT); so are a
 *   page whose number is outside [0, num_pages) and a sequence whose offsets
 *   are out of order. Two sequences must not append to one page. */
NSA_API nsa_status nsa_append_q8(const nsa_params* p, const nsa_q8_cache* cache,
                                 const void* k_new, const void* v_new, int N, const int32_t* pos,
                                 const int32_t* cu_new, const nsa_rope* rope, const void* q,
                                 void* q_out, void* k_out, void* v_out, void* stream);

/* Keys that a query at position t of its sequence attends to, of [0, t]:
 * NSA_KEYS_ALL: all; NSA_KEYS_WINDOW: the last `window` (its own included);
 * NSA_KEYS_BLOCKS (nsa_decode_q8): those in the listed blocks. */
typedef enum { NSA_KEYS_ALL = 0, NSA_KEYS_WINDOW = 1, NSA_KEYS_BLOCKS = 2 } nsa_keys;

/* Single-token attention over the 8-bit cache: softmax(scale q . k) v of one
 * query per sequence over its keys. The codes are read once for every 16 heads of
 * a KV head.
 *   q          [B, Hq, d] dtype: the query at position seq_lens[b] - 1.
 *   seq_lens   [B] int32, device, 0 <= seq_lens[b] <= T (0: no keys).
 *   keys       nsa_keys.
 *   sel_idx    [B, Hkv, top_n] int32 (NSA_KEYS_BLOCKS; else ignored): block
 *              numbers as nsa_decode writes them, in any order; negative
 *              entries and those at or past the length are ignored, a repeated
 *              one counts once.
 *   out        [B, Hq, d] dtype.
 *   lse        [B, Hq] fp32 or NULL: natural logarithm of the sum of
 *              exp(scale q . k), to join with other branches' outputs.
 * A query without keys gives 0 and -inf. A length outside [0, T] does too and
 * sets the device error word; the tokens of a page whose number is outside
 * [0, num_pages) are left out, and set it. NaN components of keys and values
 * reach the queries that attend to them and no others; a query with a NaN or an
 * infinite component gives NaN where it has keys.
 * Sums are fp32; a weight, times its page's value scale, is an fp16 number (two
 * for fp32 queries) in units that follow the row's largest product of a weight and
 * a value, so that a scale set by tokens that a query does not see changes nothing.
 * Besides its relative rounding, a weight has an error of up to 2^-35 of the row's
 * largest where the value scales are alike, and up to 2^-23 (fp32 queries: 2^-27)
 * where they lie up to 2^12 (2^8) apart. Beyond, it is up to 2^-33 (2^-21 beside
 * codes near e4m3's smallest) of the largest product of a weight and a component
 * that the row sees, for each key in out. Values below 1e-30 may count as zero.
 *   workspace  nsa_workspace_size(NSA_OP_DECODE_Q8) bytes; calls that may
 *              overlap on the GPU need one each. */
NSA_API nsa_status nsa_decode_q8(const nsa_params* p, const nsa_q8_cache* cache, const void* q,
                                 const int32_t* seq_lens, int keys, const int32_t* sel_idx,
                                 void* out, float* lse, void* workspace, size_t ws_bytes,
                                 void* stream);

/* Causal attention of chunks of queries over the 8-bit cache, which already
 * holds the chunks' own keys and values (chunked prompts, draft tokens).
 *   q          [N, Hq, d] dtype, N <= B * T.
 *   cu_q       [B + 1] int32, device, ascending, or NULL (one query per
 *              sequence, N == B): sequence b's n queries are rows cu_q[b] ..
 *              cu_q[b + 1] - 1, the i-th at position seq_lens[b] - n + i.
 *              Rows outside are not written.
 *   seq_lens   [B] int32, device: tokens in the cache, n <= seq_lens[b] <= T.
 *   keys       NSA_KEYS_ALL or NSA_KEYS_WINDOW.
 *   out, lse   [N, Hq, d] dtype, [N, Hq] fp32 or NULL.
 *   workspace  nsa_workspace_size(NSA_OP_PREFILL_Q8) bytes.
 * Errors and NaN as nsa_decode_q8; a sequence whose offsets are out of order
 * is not written. */
NSA_API nsa_status nsa_prefill_q8(const nsa_params* p, const nsa_q8_cache* cache, const void* q,
                                  int N, const int32_t* cu_q, const int32_t* seq_lens, int keys,
                                  void* out, float* lse, void* workspace, size_t ws_bytes,
                                  void* stream);

/* Synchronise `stream`, then read and clear this device's error word:
 * NSA_ERR_DEVICE_TIMEOUT if a bounded wait gave up, NSA_ERR_INVALID_ARGUMENT
 * if a kernel met an out-of-range sequence length, append position, page
 * number or token offset, else NSA_OK (or
 * NSA_ERR_CUDA if the synchronisation itself failed). */
NSA_API nsa_status nsa_check(void* stream);

/* Test hook for the failure path: launches one kernel that waits for *flag
 * (device int) to become nonzero for at most max_iters polls, then sets the
 * error word and returns. Nothing sets the flag in the test, so nsa_check must
 * report NSA_ERR_DEVICE_TIMEOUT while the context stays usable. */
NSA_API nsa_status nsa_debug_bounded_wait(const int32_t* flag, int max_iters, void* stream);

/* Kernel trace (timing aid). While enabled, every kernel this library
 * launches is bracketed by two CUDA events recorded on its stream; records
 * accumulate until the next nsa_trace_enable call. Enabling clears the
 * record; at most `capacity` launches are kept (later ones are counted but
 * not timed). Events are created at enable time, so the traced region itself
 * creates none. Not for concurrent use from several host threads. */
NSA_API nsa_status nsa_trace_enable(int on, int capacity);

/* Restrict event brackets to kernels whose name starts with `prefix` (NULL or
 * "" = every kernel). Every launch is still counted. Events between kernels
 * delay the next launch slightly, so timing only the kernel of interest keeps
 * the rest of the timeline undisturbed. */
NSA_API nsa_status nsa_trace_set_filter(const char* prefix);

/* Number of launches since the trace was enabled (including untimed ones). */
NSA_API int nsa_trace_count(void);

/* Number of launches bracketed with events (see nsa_trace_set_filter). */
NSA_API int nsa_trace_timed(void);

/* Name and device duration (ms) of timed launch i (0 <= i < nsa_trace_timed();
 * synchronises on its stop event). NSA_ERR_INVALID_ARGUMENT when out of range. */
NSA_API nsa_status nsa_trace_get(int i, const char** name, float* ms);

/* Static description of a status code. */
NSA_API const char* nsa_status_string(nsa_status s);

/* Detail of the last error returned on this host thread ("" if none). */
NSA_API const char* nsa_last_error_detail(void);

#ifdef __cplusplus
}
#endif

#endif /* NSA_B200_H_ */
