/*
 * csa2.h -- C ABI of the CSA2 compressed-sparse-attention layer step (sm_103a).
 *
 * What the step computes follows "DeepSeek-V4.1 架构解析" (DeepSeek-V4.1
 * architecture analysis, blog.yuzhonghai.cloud), §02 "CSA2" and §03
 * "precision and state rebuild", with the 4:1 ratio also given by the
 * DeepSeek V4 review (wmrh.cn), §2.1-§2.2.  Where the pages leave a step open
 * this header fixes one reading; every such reading is marked READING.
 *
 * ---------------------------------------------------------------------------
 * Conventions (all entry points)
 *   - Every tensor pointer is caller-owned DEVICE memory unless stated.  The
 *     library allocates nothing and never synchronises the stream.
 *   - `stream` is a cudaStream_t passed as void* (NULL = legacy default stream).
 *   - Every call returns CSA2_OK or an error code.  Arguments are validated on
 *     the host before anything is launched; on error nothing is launched and
 *     csa2_last_error() returns a message (thread-local, valid until the
 *     calling thread's next call).
 *   - Values held in device memory (page-table entries, entry counts, token
 *     positions, indices) cannot be checked on the host without a sync.  The
 *     kernels check them and skip an out-of-range access instead of making it;
 *     they then raise a flag in a device status word, which
 *     csa2_get_status() reads (and clears) after the caller syncs.
 *   - bf16 tensors are passed as uint16_t* (IEEE bfloat16 bit patterns).
 *   - All row-major; innermost dimension last.  Device pointers must be
 *     16-byte aligned.
 *
 * Shapes (names follow the pages):
 *   B   sequences;  Tq query tokens per sequence (1 for decode)
 *   d   latent width (64 or 512); r rotated channels at its end (even, <= d)
 *   Hq  attention query heads (1 .. 128; 64 in the pages' model)
 *   Hi, Di  indexer heads and head width (Hi <= 16, Di in {32, 64, 128})
 *   K   Top-K (1 .. 2048; 512 in the pages' model)
 *   W   sliding-window length in raw tokens (1 .. 1024; 128 in the pages)
 *
 * Data layout in HBM:
 *   KV page pool:    64 compressed entries per page.
 *     kv_codes  uint8 [n_pages][64][d/2]   E2M1 codes, channel 2i in the low
 *                                          nibble of byte i, 2i+1 in the high
 *     kv_scales uint8 [n_pages][64][d/16]  E4M3 scale codes, one per 16 channels
 *   (dims.kv_format = CSA2_KV_FP8, the V4-style main KV kept for comparison:
 *     kv_codes  uint8 [n_pages][64][d]     E4M3 codes
 *     kv_scales fp32  [n_pages][64]        one scale per entry, R5's rule;
 *     516 bytes per 512-d entry against MXFP4's 288.)
 *     idx_k     [n_pages][64][Di]          indexer keys (bf16 or fp32)
 *   page_table int32 [B][max_pages]: physical page of logical page p of
 *     sequence b; entry j of sequence b lives in page page_table[b][j/64],
 *     slot j%64.
 *   Window buffers:  swa_codes uint8 [B][swa_cap][d] (E4M3),
 *     swa_scales fp32 [B][swa_cap]; row i of sequence b is raw token
 *     swa_pos0[b] + i.
 *
 * READINGS fixed by this library (the pages leave these open):
 *   R1 compression: c_j = W * [h_4j; h_4j+1; h_4j+2; h_4j+3] (token-major
 *      concatenation, no bias); W is bf16 [d][4H]; a partial group makes no
 *      entry.
 *   R2 RMSNorm over all d channels: x = c / sqrt(mean(c^2) + eps) * gamma.
 *   R3 RoPE on the last r channels, rotate-half pairs (i, i + r/2),
 *      angle = p * base^(-2i/r), at p = 4j+3 (the entry's last token).
 *   R4 MXFP4: per 16 channels, scale = E4M3_rne_satfinite(amax / 6), codes =
 *      E2M1_rne_satfinite(x / scale) (fp32 IEEE division; ties to the even
 *      code; the sign bit is kept, so -0 is code 0x8); a scale that rounds
 *      to 0 makes all 16 codes +0.  Dequantised values e2m1 * e4m3 are exact
 *      in bf16 and in fp16.
 *   R5 FP8 window: per raw token, scale = amax / 448 (fp32, stored fp32),
 *      codes = E4M3_rne_satfinite(x / scale); scale 0 gives zero codes; the
 *      attention operand is bf16_rne(fp32(e4m3 * scale)).
 *   R6 index score s_j = sum_h w_h * ReLU(q_h . k_j), fp32 accumulation.
 *   R7 causality: entry j is visible to the token at raw position t iff
 *      4j + 3 <= t, i.e. j < min(n_entries, floor((t+1)/4)).
 *   R8 Top-K: the K highest scores (equal scores -> lower index; scores that
 *      are zero compare equal whatever their sign; NaN scores are not
 *      supported); if fewer than K entries are visible, all of them.  Output
 *      is the set in ascending index order, padded with -1, plus its count.
 *   R9 block pool: block b = entries 8b..8b+7; block score = max over its
 *      visible entries; the n_pool_blocks (2048) best blocks by (score desc,
 *      id asc), all visible blocks if fewer; output ascending, -1 padded.
 *   R10 Reindex scores the visible positions of the pooled blocks with its
 *      own indexer query against the shared indexer keys and keeps the Top-K
 *      (ties -> lower entry index).  Reuse copies the indices unchanged.
 *   R11 attention: K = V = the dequantised latent (one shared KV head); one
 *      softmax over {selected entries} U {window rows at raw positions
 *      max(0, t-W+1) .. t that the window buffer holds}, logits
 *      q . k * softmax_scale (1/sqrt(d) in the pages' model), no sink; a
 *      key in both sets counts twice.  O is fp32, lse (natural log) optional.
 *      Operand range: the products run on fp16 tensor-core operands with fp32
 *      accumulation.  Every bf16 value keeps all its bits there: each head of
 *      Q is scaled by a power of two that puts its largest magnitude in
 *      [2^14, 2^15) (values below 2^-31 of that largest one lose bits), and a
 *      window row whose scale lies outside [2^-8, 2^7] is dequantised with
 *      the scale times 2^-f (f = floor(log2 scale), clamped to [-100, 100]),
 *      its logits and softmax weights corrected by the same power.  MXFP4
 *      values (<= 2688 in magnitude, >= 2^-10) need none.  Logits must stay
 *      finite in fp32.  Softmax weights are rounded to fp16 for the product with
 *      the values (2^-11 of each at most, and 2^-25 of the largest below its normal
 *      range); their sum takes them unrounded.  A NaN in a head of Q or in a key that
 *      the token sees makes O and lse NaN there, and nowhere else.
 *   R12 the indexer key of a new entry (Full layer with compression) is
 *      W_idx * [h_4j; ..; h_4j+3], rounded to the indexer dtype.
 *   R13 SWA Bounded Replay (csa2_swa_replay): a rebuilt window row is the
 *      replayed token's own latent RoPE_t(RMSNorm(W_swa h_t)) at its raw
 *      position t, packed as R5; the rebuilt window starts at the first
 *      replayed token.
 *   R14 attention over the whole cache (csa2_dense_attn): R11's attention with
 *      every visible entry in the place of a selection, and O in bf16.  Logits
 *      l = cap * tanh(softmax_scale * q . k / cap) (cap = 0: no cap), minus
 *      slopes[h] * |t - p| with p the raw position of the key (an entry's: of
 *      its last token).  A key is visible to the token at raw position t if
 *        - entry: its last token lies at or before t; tokens of the prefix (t <
 *          prefix_len) see every entry whose last token lies below prefix_len
 *          instead.  The last token of entry j is at entry_pos where the call
 *          gets it (an evicted cache's entries lie in any order, R16), else at
 *          4 (j + shift) + 3, shift the number of entries evicted so far;
 *        - window row: raw position in max(0, t-W+1) .. t, held by the buffer
 *          (the window stays causal in the prefix too);
 *        - and, with a document mask, all of its tokens lie at or after
 *          doc_start.
 *      A token that sees nothing gets O = 0 and lse = -inf; a NaN in a key
 *      reaches the tokens that see the key, and no other.  Products run on
 *      fp16 tensor-core operands with R11's powers of two, P rounded to fp16
 *      (at d = 512, in units of 2^-7 of a reference that is the row's maximum
 *      or up to 2^8 below it), everything else in fp32; O is rounded once.
 *   R15 accumulated weight: weight_out[j] = decay * weight_in[j] + the sum over
 *      the call's query tokens and heads of exp(l - lse), l as in R14, lse as
 *      csa2_dense_attn wrote it; rows whose lse is infinite add nothing.
 *   R16 eviction: of n > keep entries those stay whose position is among the
 *      first n_sink of the sequence or the newest n_recent, then the ones of
 *      highest weight (equal weights -> lower index; -0 equals +0), keep in
 *      all.  Survivors below index keep stay where they are; those above, in
 *      index order, fill the holes below keep, in index order.  So an entry's
 *      index no longer gives its position: entry_pos does.
 *   R17 pages (csa2_page_plan): a sequence of L tokens of which `shift` entries
 *      were evicted has e = floor(L/4) - shift entries and holds ceil(e/64) pages.
 *      A step changes L by n_new (negative: drafts that were rejected, or the end
 *      of the sequence).  The free list is a stack.  First every page that is no
 *      longer needed goes onto it, in the order of sequences and then of pages;
 *      then sequences that need more pop them, in the same order.  A sequence
 *      waits (all of its state stays as it was) if its pages and those of all
 *      sequences before it that need some are more than there are; who needs
 *      none never waits.
 *   R18 FP8 rows (csa2_pack_fp8_blocks): per 128 columns, a = max(amax, 2^-100),
 *      scale = a / 448 and codes = E4M3_rne_satfinite(x * (448 / a)), each step
 *      rounded to fp32.  The last block of a row may be shorter.  A block with an
 *      infinity dequantises to NaN, a NaN stays one by itself.
 *   R19 product (csa2_matmul_fp8): C[m][n] = sum over blocks kb of
 *      (a_scales[m][kb] * b_scales[n/128][kb]) * (sum of the block's code products);
 *      the product of the scales (so it has to be a normal fp32 value, or 0), every
 *      block's sum and the sum over blocks are held in fp32, in an order that M, N
 *      and K fix; C is rounded once.
 *   R20 rotary positions (csa2_rope): pair i of the r rotated channels turns by
 *      p * theta_i, theta_i = base^(-2i/r) as in R3; scaled for long contexts:
 *      LINEAR theta_i / factor; NTK base * factor^(r/(r-2)) in the place of base;
 *      YARN theta_i (1 - g_i) + theta_i / factor * g_i with g_i = clamp((i - lo) /
 *      max(hi - lo, 0.001), 0, 1), lo = max(0, floor(c(beta_fast))), hi =
 *      min(r - 1, ceil(c(beta_slow))), c(n) = r ln(original_len / (2 pi n)) /
 *      (2 ln base).  HALF pairs channels (i, i + r/2), INTERLEAVED (2i, 2i + 1).  The
 *      frequencies are fp64: the angle at position p is known to p 2^-50 radians
 *      (below fp32's own rounding up to p = 2^26).
 *   R21 drafted trees: node i of a sequence continues node parent[i] < i, or the
 *      committed text (-1); -2 marks a place without a node.  It stands at raw
 *      position ctx_len + depth.  csa2_tree_attn is R11 with the window rows of
 *      positions from ctx_len on taken from the node's own ancestors (itself
 *      among them), and O in bf16.  A place without a node gets O = 0, lse = -inf
 *      (its selection is not looked at).
 * ---------------------------------------------------------------------------
 */
#ifndef CSA2_H
#define CSA2_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

/* status codes */
#define CSA2_OK 0
#define CSA2_ERR_INVALID_ARG 1 /* a pointer, size or alignment is wrong      */
#define CSA2_ERR_UNSUPPORTED 2 /* a valid shape this build has no kernel for */
#define CSA2_ERR_CUDA 3        /* a launch failed; see csa2_last_error()     */
#define CSA2_ERR_WORKSPACE 4   /* workspace NULL or smaller than required    */
#define CSA2_ERR_DEVICE_DATA 5 /* csa2_get_status: a kernel met bad device data */

/* element types of the indexer query / key */
#define CSA2_F32 0
#define CSA2_BF16 1

/* main-KV formats (dims.kv_format) */
#define CSA2_KV_MXFP4 0 /* E2M1 codes + E4M3 scale per 16 channels (V4.1, the pages' format) */
#define CSA2_KV_FP8 1   /* E4M3 codes + fp32 scale per entry (V4-style, for the A/B)       */

/* layer modes (static per layer) */
#define CSA2_MODE_FULL 0    /* compute KV (optional), score all, Top-K   */
#define CSA2_MODE_REINDEX 1 /* rescore the Full layer's pool, Top-K      */
#define CSA2_MODE_REUSE 2   /* take the previous layer's indices         */

/* status-word bits set by kernels that met bad device-resident data */
#define CSA2_STATUS_BAD_PAGE 1u     /* page-table entry outside [0, n_pages)  */
#define CSA2_STATUS_BAD_INDEX 2u    /* an index outside the visible entries   */
#define CSA2_STATUS_BAD_COUNT 4u    /* a count or position out of range       */
#define CSA2_STATUS_TIMEOUT 8u      /* a bounded on-chip wait gave up; outputs of that launch are invalid */

/* ABI version of this header (bumped on any incompatible change). */
#define CSA2_ABI_VERSION 2

int csa2_abi_version(void);

/* Number of kernels this library has launched in this process (all devices,
 * all threads).  Used to count launches inside a timed region. */
uint64_t csa2_launch_count(void);

/* Message of the last error of the calling thread ("" if none). */
const char* csa2_last_error(void);

/* Reads and clears the device status word (CSA2_STATUS_* bits) for the
 * current device.  Blocks until the stream's prior work is done.  Returns
 * CSA2_OK, or CSA2_ERR_CUDA if the copy failed; *bits receives the flags. */
int csa2_get_status(uint32_t* bits, void* stream);

/* Shapes shared by the entry points. */
typedef struct csa2_dims {
  int32_t B;             /* sequences                                      */
  int32_t Tq;            /* query tokens per sequence                      */
  int32_t d;             /* latent width: 64 or 512                        */
  int32_t r;             /* rotated channels at the end of the latent      */
  int32_t Hq;            /* attention query heads                          */
  int32_t Hi;            /* indexer heads                                  */
  int32_t Di;            /* indexer head width                             */
  int32_t idx_dtype;     /* CSA2_BF16 or CSA2_F32 (indexer q and k)        */
  int32_t K;             /* Top-K                                          */
  int32_t W;             /* window length in raw tokens                    */
  int32_t max_pages;     /* row length of the page table                   */
  int32_t n_pool_blocks; /* hierarchical pool: blocks kept (2048)          */
  int32_t pool_block;    /* hierarchical pool: entries per block (8)       */
  int32_t swa_cap;       /* rows per sequence in the window buffers        */
  int32_t kv_format;     /* CSA2_KV_MXFP4 (0) or CSA2_KV_FP8 (FP8 needs d = 512) */
} csa2_dims;

/* The shared compressed cache of one layer group. */
typedef struct csa2_cache {
  uint8_t* kv_codes;         /* [n_pages][64][d/2] (FP8: [n_pages][64][d])   */
  uint8_t* kv_scales;        /* [n_pages][64][d/16] (FP8: fp32 [n_pages][64]) */
  void* idx_k;               /* [n_pages][64][Di], idx_dtype                 */
  const int32_t* page_table; /* [B][max_pages]                               */
  const int32_t* n_entries;  /* [B] entries present (device)                 */
  int64_t n_pages;           /* physical pages in the pool                   */
} csa2_cache;

/* The sliding window of one layer. */
typedef struct csa2_window {
  uint8_t* codes;            /* [B][swa_cap][d] E4M3                         */
  float* scales;             /* [B][swa_cap]                                 */
  const int32_t* pos0;       /* [B] raw position of row 0 (device)           */
} csa2_window;

/* ---- a3: MXFP4 pack of a given fp32 array (bit-exact contract, R4) -------
 * x fp32 [n_rows][d] -> codes uint8 [n_rows][d/2], scales uint8 [n_rows][d/16].
 * d: multiple of 16, <= 4096.  n_rows may be 0 (no launch). */
int csa2_pack_mxfp4_f32(const float* x, int64_t n_rows, int32_t d, uint8_t* codes,
                        uint8_t* scales, void* stream);

/* Dequantise MXFP4 rows to bf16 (exact, R4).  out uint16 [n_rows][d]. */
int csa2_unpack_mxfp4_bf16(const uint8_t* codes, const uint8_t* scales, int64_t n_rows,
                           int32_t d, uint16_t* out, void* stream);

/* ---- a10: FP8 window pack (bit-exact contract, R5) ------------------------
 * x fp32 [n_rows][d] -> codes uint8 [n_rows][d], scales fp32 [n_rows].
 * d: multiple of 16, <= 4096. */
int csa2_pack_swa_fp8(const float* x, int64_t n_rows, int32_t d, uint8_t* codes,
                      float* scales, void* stream);

/* ---- a2+a3 on a given latent: RMSNorm, RoPE, MXFP4, paged store ----------
 * latent fp32 [B][n_max][d]; rows i < n_rows[b] of sequence b become entries
 * first_entry[b] + i (R2, R3 at position 4(first_entry[b]+i)+3, R4) and are
 * written into the page pool through page_table.  gamma fp32 [d].
 * first_entry, n_rows: int32 [B], device.  d in {64, 512}; r even, <= d. */
int csa2_norm_rope_pack(const float* latent, int32_t B, int32_t n_max, int32_t d, int32_t r,
                        const float* gamma, float eps, float rope_base,
                        const int32_t* first_entry, const int32_t* n_rows,
                        const int32_t* page_table, int32_t max_pages, int64_t n_pages,
                        uint8_t* kv_codes, uint8_t* kv_scales, void* stream);

/* The same for the FP8 main-KV format (dims.kv_format = CSA2_KV_FP8): after
 * RMSNorm and RoPE each entry row is packed by R5's rule (scale = amax / 448,
 * stored fp32; codes = E4M3_rne_satfinite(x / scale)) into kv_codes uint8
 * [n_pages][64][d] and kv_scales fp32 [n_pages][64].  The V4 review and the
 * V4.1 analysis (§03) describe V4's main KV as FP8; this format exists to
 * compare the two on the same path.  d = 512 only. */
int csa2_norm_rope_pack_fp8(const float* latent, int32_t B, int32_t n_max, int32_t d, int32_t r,
                            const float* gamma, float eps, float rope_base,
                            const int32_t* first_entry, const int32_t* n_rows,
                            const int32_t* page_table, int32_t max_pages, int64_t n_pages,
                            uint8_t* kv_codes, float* kv_scales, void* stream);

/* ---- a1-a4: compress new tokens into the paged cache ----------------------
 * hidden bf16 [B][T][H] (the new tokens of every sequence, token 0 at raw
 * position 4*first_entry[b]); W bf16 [d][4H]; gamma fp32 [d]; W_idx bf16
 * [Di][4H] or NULL; idx_k receives the new indexer keys (R12) when W_idx is
 * given.  Entries first_entry[b] .. first_entry[b] + T/4 - 1 are written.
 * Needs csa2_compress_workspace_size() bytes of workspace.
 * H: multiple of 64 (so 4H is a multiple of 256); d in {64, 512}. */
size_t csa2_compress_workspace_size(int32_t B, int32_t T, int32_t H, int32_t d, int32_t Di);
int csa2_compress_pack(const uint16_t* hidden, int32_t B, int32_t T, int32_t H,
                       const uint16_t* W, const float* gamma, float eps, float rope_base,
                       const uint16_t* W_idx, const int32_t* first_entry,
                       const csa2_dims* dims, const csa2_cache* cache,
                       void* ws, size_t ws_bytes, void* stream);

/* ---- a1-a4 for several layers from one hidden state --------------------------
 * "DeepSeek-V4.1 架构解析" §01 (causal encoder-decoder): every decoder layer
 * projects its KV from the same hidden state (the last encoder layer's) with
 * its own compression weights.  One GEMM over the layers' stacked weights,
 * then each layer's RMSNorm, RoPE, MXFP4 pack and paged store (R1-R4, R12)
 * into its own cache.
 * hidden bf16 [B][T][H] as for csa2_compress_pack; W_all bf16 [L][d + Di][4H]
 * (layer l: rows 0..d-1 its W, rows d..d+Di-1 its W_idx); Di = 0 (no indexer
 * keys written) or dims->Di; gamma_all fp32 [L][d]; caches: host array of L
 * caches sharing dims (page tables, entry counts and pools may differ).
 * Entries first_entry[b] .. first_entry[b] + T/4 - 1 of every layer's cache
 * are written.  Needs csa2_compress_layers_workspace_size() bytes of workspace.
 * H: multiple of 64; d in {64, 512}; L >= 1. */
size_t csa2_compress_layers_workspace_size(int32_t B, int32_t T, int32_t H, int32_t L, int32_t d, int32_t Di);
int csa2_compress_layers(const uint16_t* hidden, int32_t B, int32_t T, int32_t H, int32_t L,
                         const uint16_t* W_all, int32_t Di, const float* gamma_all, float eps,
                         float rope_base, const int32_t* first_entry, const csa2_dims* dims,
                         const csa2_cache* caches, void* ws, size_t ws_bytes, void* stream);

/* ---- SWA Bounded Replay: a layer's window rebuilt from its last tokens -------
 * "DeepSeek-V4.1 架构解析" §03 (SWA Bounded Replay): the window KV is not kept
 * in the persistent cache; a layer rebuilds it by replaying only the last
 * n_win (128) raw tokens, and tokens early in the replay see a shorter
 * window than the exact state would give them.
 * READING R13: the window row of raw token t is that token's own latent,
 * x_t = RoPE_t(RMSNorm(W_swa h_t)): W_swa bf16 [d][H] without bias, R2's
 * RMSNorm with gain gamma, R3's rotation at t itself (not at an entry
 * position), then R5's FP8 pack.  With the window buffer's first row at the
 * first replayed position, R11 gives a replayed token at p the rows
 * max(first replayed position, p - W + 1) .. p.
 * hidden bf16 [B][n_tok][H]: this layer's hidden states of the replayed
 * tokens, row i of sequence b at raw position tok_pos0[b] + i (tok_pos0 int32
 * [B], device); gamma fp32 [d].  Row i of sequence b is written to window
 * row tok_pos0[b] + i - win->pos0[b]; a row outside [0, dims->swa_cap), or at
 * a negative raw position, is not written and raises CSA2_STATUS_BAD_COUNT.
 * Uses dims->B, d, r and swa_cap (the struct is validated as for every entry
 * point).  Needs csa2_swa_replay_workspace_size() bytes of workspace.
 * H: multiple of 64; d in {64, 512}. */
size_t csa2_swa_replay_workspace_size(int32_t B, int32_t n_tok, int32_t H, int32_t d);
int csa2_swa_replay(const uint16_t* hidden, int32_t B, int32_t n_tok, int32_t H, const uint16_t* W_swa,
                    const float* gamma, float eps, float rope_base, const int32_t* tok_pos0,
                    const csa2_dims* dims, const csa2_window* win, void* ws, size_t ws_bytes,
                    void* stream);

/* ---- a5: index scores of every visible entry (R6, R7) ----------------------
 * idx_q [B][Tq][Hi][Di] (idx_dtype), w fp32 [B][Tq][Hi], q_pos int32 [B][Tq].
 * scores fp32 [B*Tq][score_stride]: column j < n_vis(row) receives s_j;
 * other columns are not written.  blockmax (NULL or fp32
 * [B*Tq][bm_stride]): column b < ceil(n_vis/pool_block) receives the block
 * maximum (R9).  score_stride >= max visible entries of any row. */
int csa2_index_scores(const csa2_dims* dims, const csa2_cache* cache, const void* idx_q,
                      const float* w, const int32_t* q_pos, float* scores,
                      int64_t score_stride, float* blockmax, int64_t bm_stride, void* stream);

/* ---- a6: Top-K of a given fp32 array (bit-exact contract, R8) -------------
 * scores fp32 [rows][stride]; n_valid int32 [rows] (device) or NULL (all
 * `stride` columns valid).  out_idx int32 [rows][k] ascending, -1 padded;
 * out_cnt int32 [rows].  k in 1..4096; stride < 2^31.  With a workspace of
 * csa2_topk_workspace_size() bytes each row is spread over many CTAs (for few,
 * long rows); with ws == NULL one CTA handles each row.  Same result. */
size_t csa2_topk_workspace_size(int64_t rows, int64_t stride, int32_t k);
int csa2_topk_f32(const float* scores, int64_t rows, int64_t stride, const int32_t* n_valid,
                  int32_t k, int32_t* out_idx, int32_t* out_cnt, void* ws, size_t ws_bytes,
                  void* stream);

/* ---- a7: block pool of a given fp32 score array (bit-exact contract, R9) --
 * scores fp32 [rows][stride], n_valid int32 [rows] entries valid per row.
 * out_pool int32 [rows][n_pool_blocks] ascending block ids, -1 padded;
 * out_pool_cnt int32 [rows]; out_blockmax (NULL or fp32 [rows][ceil(stride/block)]). */
int csa2_block_pool_f32(const float* scores, int64_t rows, int64_t stride, const int32_t* n_valid,
                        int32_t block, int32_t n_pool_blocks, int32_t* out_pool,
                        int32_t* out_pool_cnt, float* out_blockmax, void* ws, size_t ws_bytes,
                        void* stream);

/* ---- a5+a6 (+a7) Full, or a8 Reindex: indexer and Top-K in one call -------
 * Full (pool == NULL): scores every visible entry, keeps Top-K into out_idx /
 * out_cnt; if out_pool != NULL also builds the hierarchical pool (R9).
 * Reindex (pool != NULL, pool_cnt int32 [B*Tq]): scores only the pooled
 * positions (R10).  Scratch: csa2_index_topk_workspace_size() bytes. */
size_t csa2_index_topk_workspace_size(const csa2_dims* dims, int32_t max_entries);
int csa2_index_topk(const csa2_dims* dims, const csa2_cache* cache, const void* idx_q,
                    const float* w, const int32_t* q_pos, const int32_t* pool,
                    const int32_t* pool_cnt, int32_t* out_idx, int32_t* out_cnt,
                    int32_t* out_pool, int32_t* out_pool_cnt, int32_t max_entries,
                    void* ws, size_t ws_bytes, void* stream);

/* ---- csa2_index_topk without a caller workspace ---------------------------
 * No counterpart in the paper: a convenience for callers that cannot
 * allocate device memory (for example code that runs while a CUDA graph is
 * being captured, or a serving thread that must never wait on the
 * allocator).  Same arguments and results as csa2_index_topk, but the scratch
 * lives in one fixed 8 MiB array inside the library
 * (csa2_index_topk_noalloc_capacity() bytes), held by every GPU that loads
 * the library until the process exits.  Shapes whose
 * csa2_index_topk_workspace_size() exceeds it are rejected with
 * CSA2_ERR_WORKSPACE.  The first call in a CUDA context looks the array's
 * device address up (cudaGetSymbolAddress) with that context current and
 * caches it for that context; a context re-created by cudaDeviceReset is
 * looked up again.  Make the first call in a context before any stream
 * capture.  The call clears the part of the array that
 * must start at zero.  All calls share the one array: calls that can overlap
 * on the GPU (different streams without ordering between them) race and give
 * wrong results; order them on one stream.  Allocates nothing. */
size_t csa2_index_topk_noalloc_capacity(void);
int csa2_index_topk_noalloc(const csa2_dims* dims, const csa2_cache* cache, const void* idx_q,
                            const float* w, const int32_t* q_pos, const int32_t* pool,
                            const int32_t* pool_cnt, int32_t* out_idx, int32_t* out_cnt,
                            int32_t* out_pool, int32_t* out_pool_cnt, int32_t max_entries,
                            void* stream);

/* ---- a11: gathered sparse MQA attention + FP8 window (R11) ----------------
 * Q bf16 [B][Tq][Hq][d] (already rotated at its own position); idx int32
 * [B][Tq][K] (-1 padded) with cnt int32 [B][Tq]; O fp32 [B][Tq][Hq][d];
 * lse fp32 [B][Tq][Hq] or NULL.  d must be 512 or 64. */
int csa2_sparse_attn(const csa2_dims* dims, const csa2_cache* cache, const csa2_window* win,
                     const uint16_t* Q, const int32_t* q_pos, const int32_t* idx,
                     const int32_t* cnt, float softmax_scale, float* O, float* lse,
                     void* stream);

/* ---- the query side of a step: pages, FP8 projections, rotary positions, trees ----
 * What a step needs around csa2_layer: pages and positions for its tokens, the
 * projections that give the queries, their rotation, and attention for tokens
 * that were drafted as a tree. */

/* Pages of a pool and who holds them; all arrays are read and written. */
typedef struct csa2_page_pool {
  int32_t* page_table;       /* [B][max_pages]: the array behind csa2_cache.page_table */
  int32_t* held;             /* [B] pages that a sequence holds: its first `held` places */
  int32_t* free_pages;       /* [n_pages]: a stack, its bottom first         */
  int32_t* n_free;           /* [1] pages on the stack                       */
  int64_t n_pages;           /* pages of the pool (below 2^31)               */
} csa2_page_pool;

/* Block tables, positions and slots of a step (R17).  seq_len int32 [B] raw tokens
 * before the step, n_new int32 [B] tokens that it adds (negative: takes away),
 * shift int32 [B] entries evicted so far or NULL.  Writes the pool, and per sequence
 * seq_len_out [B] (may be seq_len), n_entries [B] and first_entry [B] (the first
 * entry that the step writes; n_entries where it writes none), granted [B] (1, or 0
 * where the sequence waits; NULL: not wanted), q_pos [B][Tq] (raw positions of the
 * new tokens, -1 behind them; NULL: not wanted) and slots int64 [B][max_new] (64 page
 * + place of every new entry in the pool, -1 behind them; NULL: not wanted).
 * Table places at or behind a sequence's pages, and stack places at or behind
 * n_free, keep whatever they held.  A sequence whose state is impossible (a
 * negative length, fewer pages held than its entries need, more pages than
 * max_pages, more new tokens than Tq where q_pos is wanted or new entries than
 * max_new where slots are) waits and raises CSA2_STATUS_BAD_COUNT; a pool whose
 * counts cannot be (n_free outside 0 .. n_pages, more released than it lacks)
 * makes every sequence wait.  A page id outside the pool is passed on, gets no slot
 * and raises CSA2_STATUS_BAD_PAGE.  After csa2_evict the pages behind the kept
 * entries come back with the next call (shift says so).  A page belongs to one
 * sequence or to the free list.  Counts and tables may be the ones that csa2_cache
 * points to.  dims: B, Tq, max_pages are used.  Needs csa2_page_plan_workspace_size() bytes of workspace, which calls that
 * can overlap must not share. */
size_t csa2_page_plan_workspace_size(const csa2_dims* dims);
int csa2_page_plan(const csa2_dims* dims, const csa2_page_pool* pool, const int32_t* seq_len,
                   const int32_t* n_new, const int32_t* shift, int32_t max_new, int32_t* seq_len_out,
                   int32_t* n_entries, int32_t* first_entry, int32_t* q_pos, int64_t* slots,
                   int32_t* granted, void* ws, size_t ws_bytes, void* stream);

/* Rows to FP8 (R18): x bf16 or fp32 (dtype CSA2_BF16 or CSA2_F32) [n_rows][K], rows
 * row_stride elements apart (a multiple of 16 bytes) -> codes uint8 [n_rows][K],
 * scales fp32 [n_rows][ceil(K/128)].  K: a multiple of 16. */
int csa2_pack_fp8_blocks(const void* x, int32_t dtype, int64_t row_stride, int64_t n_rows, int32_t K,
                         uint8_t* codes, float* scales, void* stream);

/* C = A Bw^T of FP8 rows (R19): A E4M3 [M][K] with a_scales fp32 [M][ceil(K/128)] as
 * csa2_pack_fp8_blocks writes them, Bw E4M3 [N][K] (weights, one row per output) with
 * b_scales fp32 [ceil(N/128)][ceil(K/128)], C [M][N] bf16 or fp32 (c_dtype).  K: a
 * multiple of 16; M and N any.  Needs csa2_matmul_fp8_workspace_size() bytes of
 * workspace (0: ws may be NULL), which calls that can overlap must not share.  A size
 * belongs to its very shape: fewer rows of A can need more of it (4,096 x 4,096 x 7,168
 * needs none, 32 x 4,096 x 7,168 some), as K is split where there are few tiles.
 * CSA2_MATMUL_FP8_WORKSPACE_MAX bytes are enough for every shape, so that a program
 * with several can keep one workspace of that size. */
#define CSA2_MATMUL_FP8_WORKSPACE_MAX 9961472
size_t csa2_matmul_fp8_workspace_size(int32_t M, int32_t N, int32_t K);
int csa2_matmul_fp8(const uint8_t* A, const float* a_scales, const uint8_t* Bw, const float* b_scales,
                    int32_t M, int32_t N, int32_t K, void* C, int32_t c_dtype, void* ws, size_t ws_bytes,
                    void* stream);

/* frequencies of csa2_rope (R20) */
#define CSA2_ROPE_PLAIN 0
#define CSA2_ROPE_LINEAR 1
#define CSA2_ROPE_NTK 2
#define CSA2_ROPE_YARN 3
/* pairs of csa2_rope */
#define CSA2_ROPE_HALF 0
#define CSA2_ROPE_INTERLEAVED 1

typedef struct csa2_rope_spec {
  int32_t scaling;           /* CSA2_ROPE_PLAIN .. CSA2_ROPE_YARN            */
  int32_t original_len;      /* YARN: context length before the scaling      */
  double base;               /* above 1 (10000 in R3)                        */
  double factor;             /* all but PLAIN: how many times longer, >= 1   */
  float beta_fast, beta_slow;/* YARN: turns (32 and 1 are usual)             */
} csa2_rope_spec;

/* The table that csa2_rope reads, made once for a model: table uint64 [r/2] (device)
 * receives theta_i / 2 pi in turns per position, as 0.64 fixed point.  r: even, <= 2048. */
int csa2_rope_table(const csa2_rope_spec* spec, int32_t r, uint64_t* table, void* stream);

/* y = x with channels start .. start + r - 1 of every head rotated to its token's
 * position (R20) and multiplied by amplitude (1, or YARN's attention factor); the
 * other channels are copied.  x and y: bf16 or fp32, [n_tokens][heads][d] with the
 * given strides in elements, channels contiguous; fastest where rows are 16-byte
 * aligned and 8 divides d (HALF: start and r / 2 too).  y may be x (same
 * type and strides: only the rotated channels are touched); otherwise they must not
 * overlap, and no two rows of y either.  positions int32 [n_tokens] (negative ones turn backwards).  inverse != 0
 * turns by -p: back, and also the gradient (the transpose) of the rotation. */
int csa2_rope(const void* x, int32_t x_dtype, int64_t x_token_stride, int64_t x_head_stride, void* y,
              int32_t y_dtype, int64_t y_token_stride, int64_t y_head_stride, int64_t n_tokens,
              int32_t heads, int32_t d, int32_t start, int32_t r, int32_t layout, int32_t inverse,
              float amplitude, const int32_t* positions, const uint64_t* table, void* stream);

/* A tree of drafted tokens per sequence (R21). */
typedef struct csa2_tree {
  const uint8_t* codes;      /* [B][Tq][d] E4M3: the nodes' window rows (csa2_pack_swa_fp8) */
  const float* scales;       /* [B][Tq]                                      */
  const int32_t* ctx_len;    /* [B] committed raw tokens                     */
  const int32_t* path;       /* [B][Tq][max_depth] as csa2_tree_plan writes it */
  int32_t max_depth;         /* row length of path                           */
} csa2_tree;

/* Positions and paths of the trees: parent int32 [B][Tq], ctx_len int32 [B] ->
 * q_pos [B][Tq] (-1 where there is no node) and path [B][Tq][max_depth] (the node's
 * ancestor at every depth, itself last, -1 behind it).  A parent at or behind its
 * child, or one that is no node, raises CSA2_STATUS_BAD_INDEX, a node deeper than
 * max_depth or past position 2^31 - 1 and a negative ctx_len CSA2_STATUS_BAD_COUNT;
 * these are no nodes then.  Tq <= 1024.  dims: B, Tq are used. */
int csa2_tree_plan(const csa2_dims* dims, const int32_t* parent, const int32_t* ctx_len,
                   int32_t max_depth, int32_t* q_pos, int32_t* path, void* stream);

/* csa2_sparse_attn for drafted trees (R21): q_pos and tree->path as csa2_tree_plan
 * wrote them, win the committed rows (unused, and may be NULL, where swa_cap or W is
 * 0), idx and cnt the selection of every node, O bf16 [B][Tq][Hq][d], lse fp32
 * [B][Tq][Hq] or NULL.  A path that does not reach the token's position raises
 * CSA2_STATUS_BAD_INDEX, and that key is left out. */
int csa2_tree_attn(const csa2_dims* dims, const csa2_cache* cache, const csa2_window* win,
                   const csa2_tree* tree, const uint16_t* Q, const int32_t* q_pos, const int32_t* idx,
                   const int32_t* cnt, float softmax_scale, uint16_t* O, float* lse, void* stream);

/* ---- a bounded cache: attention over all of it, weights, eviction ------------
 * A cache that never grows past a fixed size needs no selection: every entry it
 * holds is attended to, the weight each entry receives is added up, and when
 * the cache is full the entries of least weight leave.
 *
 * State of such a cache, beside csa2_cache (weight and entry_pos lie like the
 * pages, one value per slot; shift has one per sequence).  A cache that no
 * entry was evicted from may go without (NULL, or NULL members): entry j's
 * position is then 4 (j + shift) + 3 and shift is 0.
 *
 * Entries of such a cache are appended by csa2_compress_pack_bounded alone.
 * csa2_compress_pack, csa2_compress_layers and csa2_layer with hidden != NULL
 * rotate a new entry at 4 e + 3 with e its index, and write neither entry_pos
 * nor weight: once entries were evicted they must not be used on it (csa2_cache
 * does not show that, so they cannot refuse). */
typedef struct csa2_bounded {
  int32_t* entry_pos;        /* [n_pages][64] raw position of the entry's last token */
  float* weight;             /* [n_pages][64] accumulated weight (R15)          */
  int32_t* shift;            /* [B] entries evicted so far                      */
} csa2_bounded;

/* Changes to the logits and to what is visible (R14); NULL or zeros: none. */
typedef struct csa2_score_mods {
  float logit_cap;           /* 2^-126 .. 2^127: l = cap * tanh(l / cap); 0: none */
  const float* slopes;       /* fp32 [Hq]: l -= slopes[h] * |t - p|             */
  const int32_t* doc_start;  /* [B][Tq] raw position where the token's document starts */
  const int32_t* prefix_len; /* [B] tokens below it see every entry that ends below it (R14); one that
                                the prefix ends in the middle of, and the window, stay causal */
} csa2_score_mods;

/* Attention over every visible entry and the window (R14).  Q bf16
 * [B][Tq][Hq][d], q_pos int32 [B][Tq] raw positions (after an eviction too), O
 * bf16 [B][Tq][Hq][d], lse fp32 [B][Tq][Hq] or NULL.  max_entries bounds every
 * n_entries[b] (more: CSA2_STATUS_BAD_COUNT, and only max_entries are read).
 * dims: B, Tq, d, Hq, W, max_pages, swa_cap are used; d = 512 or 64, MXFP4 main
 * KV only.  A page-table entry out of range hides its entries and raises
 * CSA2_STATUS_BAD_PAGE.  bounded: entry_pos and shift are read (NULL: see
 * above).  Needs csa2_dense_attn_workspace_size() bytes of workspace, which
 * calls that can overlap must not share. */
size_t csa2_dense_attn_workspace_size(const csa2_dims* dims, int32_t max_entries);
int csa2_dense_attn(const csa2_dims* dims, const csa2_cache* cache, const csa2_bounded* bounded,
                    const csa2_window* win, const csa2_score_mods* mods, const uint16_t* Q,
                    const int32_t* q_pos, float softmax_scale, int32_t max_entries, uint16_t* O,
                    float* lse, void* ws, size_t ws_bytes, void* stream);

/* The weight that every entry received from the call's query tokens (R15):
 * Q, q_pos, softmax_scale and mods as given to csa2_dense_attn, lse as it wrote
 * them.  weight_in fp32 [n_pages][64] (NULL: zeros), weight_out fp32
 * [n_pages][64] (may be weight_in): written for the n_entries[b] entries of
 * every sequence (but those behind a bad page), whether a token of the call saw
 * them or not; other slots are left as they were.  A call without query tokens
 * (Tq = 0) launches nothing and leaves weight_out as it was: no decay, and no
 * copy of weight_in.  Sequences must not share pages.  decay in 0..1.  Sums run
 * in a fixed order.  Needs csa2_entry_weights_workspace_size() bytes of
 * workspace, which calls that can overlap must not share. */
size_t csa2_entry_weights_workspace_size(const csa2_dims* dims, int32_t max_entries);
int csa2_entry_weights(const csa2_dims* dims, const csa2_cache* cache, const csa2_bounded* bounded,
                       const csa2_score_mods* mods, const uint16_t* Q, const int32_t* q_pos,
                       const float* lse, float softmax_scale, float decay, const float* weight_in,
                       float* weight_out, int32_t max_entries, void* ws, size_t ws_bytes,
                       void* stream);

/* Cuts every sequence of more than `keep` entries to `keep` (R16): moves codes,
 * scales, indexer keys (unless cache->idx_k is NULL), weights and positions
 * inside the sequence's own pages, sets n_entries[b] = keep and adds the number
 * evicted to shift[b].  n_entries is the array that cache->n_entries points to,
 * writable.  Slots at index >= keep keep their bytes; pages that lie wholly
 * there are free for reuse once the call is done.  keep >= 1, n_sink +
 * n_recent <= keep.  A sequence whose n_entries is negative, above max_entries
 * or past its page table, or whose shift is negative, stays as it is and raises
 * CSA2_STATUS_BAD_COUNT; one that would be cut but has a page-table entry out
 * of range stays as it is and raises CSA2_STATUS_BAD_PAGE (with max_entries <=
 * keep the call returns at once and looks at no count and no page).  Sequences
 * must not share pages.  NaN weights are not supported.  dims: B, d, Di,
 * idx_dtype, max_pages, kv_format are used.  Needs csa2_evict_workspace_size()
 * bytes of workspace, which calls that can overlap must not share.
 *
 * After an eviction csa2_index_topk, csa2_sparse_attn and the other calls that
 * know nothing of shift take q_pos[b][i] - 4 shift[b] in the place of q_pos
 * (their visible count is then min(n_entries, floor((t+1)/4) - shift)) and
 * win->pos0[b] - 4 shift[b] in the place of pos0, with keep >= W / 4.  They go
 * by index, so they are right for query tokens that see all that the eviction
 * left, q_pos[b][i] >= 4 (keep + shift[b]) - 1 (evict, append, then ask); an
 * older token would be shown entries of its future.  csa2_dense_attn and
 * csa2_entry_weights go by entry_pos and take any token. */
size_t csa2_evict_workspace_size(const csa2_dims* dims, int32_t max_entries);
int csa2_evict(const csa2_dims* dims, const csa2_cache* cache, const csa2_bounded* bounded,
               int32_t* n_entries, int32_t keep, int32_t n_sink, int32_t n_recent,
               int32_t max_entries, void* ws, size_t ws_bytes, void* stream);

/* csa2_compress_pack into a bounded cache: entry first_entry[b] + i (an index)
 * is rotated at position 4 (first_entry[b] + shift[b] + i) + 3, which entry_pos
 * receives, and starts with weight 0.  An entry whose shift is negative or whose
 * position passes 2^31 - 1 is not written and raises CSA2_STATUS_BAD_COUNT.
 * Workspace as for csa2_compress_pack. */
int csa2_compress_pack_bounded(const uint16_t* hidden, int32_t B, int32_t T, int32_t H,
                               const uint16_t* W, const float* gamma, float eps, float rope_base,
                               const uint16_t* W_idx, const int32_t* first_entry,
                               const csa2_dims* dims, const csa2_cache* cache,
                               const csa2_bounded* bounded, void* ws, size_t ws_bytes,
                               void* stream);

/* ---- one layer step in any mode -------------------------------------------
 * FULL    : [compress new tokens if hidden != NULL] [pack window rows of the
 *           new tokens if swa_new != NULL] -> index + Top-K (+ pool if
 *           hierarchical) -> attention.
 * REINDEX : [pack window rows] -> pooled rescoring (pool/pool_cnt read) ->
 *           attention.
 * REUSE   : [pack window rows] -> idx_out/cnt_out = idx_in/cnt_in (copied
 *           unless the same buffers) -> attention.
 * swa_new fp32 [B][Tq][d]: window latent of the query tokens, written to
 * window row q_pos - pos0.  Scratch: csa2_layer_workspace_size() bytes. */
typedef struct csa2_layer_args {
  int32_t mode;              /* CSA2_MODE_*                                  */
  int32_t hierarchical;      /* FULL: also build the pool                    */
  csa2_dims dims;
  csa2_cache cache;
  csa2_window window;
  const int32_t* q_pos;      /* [B][Tq]                                      */
  int32_t max_entries;       /* upper bound of any n_entries[b]              */
  /* FULL only, optional compression of the new tokens (hidden == NULL: none) */
  const uint16_t* hidden;    /* bf16 [B][T][H]                               */
  int32_t T, H;
  const uint16_t* W_c;       /* bf16 [d][4H]                                 */
  const uint16_t* W_idx;     /* bf16 [Di][4H] or NULL                        */
  const float* gamma;        /* fp32 [d]                                     */
  float eps, rope_base;
  const int32_t* first_entry;/* [B]                                          */
  /* optional window rows of the query tokens (NULL: none) */
  const float* swa_new;      /* fp32 [B][Tq][d]                              */
  /* indexer query (FULL, REINDEX) */
  const void* idx_q;         /* [B][Tq][Hi][Di]                              */
  const float* idx_w;        /* [B][Tq][Hi]                                  */
  /* attention */
  const uint16_t* Q;         /* bf16 [B][Tq][Hq][d]                          */
  float softmax_scale;
  /* indices */
  const int32_t* idx_in;     /* REUSE: [B][Tq][K]                            */
  const int32_t* cnt_in;     /* REUSE: [B][Tq]                               */
  int32_t* idx_out;          /* [B][Tq][K]                                   */
  int32_t* cnt_out;          /* [B][Tq]                                      */
  int32_t* pool;             /* [B][Tq][n_pool_blocks]: FULL+hier writes, REINDEX reads */
  int32_t* pool_cnt;         /* [B][Tq]                                      */
  /* outputs */
  float* O;                  /* [B][Tq][Hq][d]                               */
  float* lse;                /* [B][Tq][Hq] or NULL                          */
} csa2_layer_args;

size_t csa2_layer_workspace_size(const csa2_layer_args* a);
int csa2_layer(const csa2_layer_args* a, void* ws, size_t ws_bytes, void* stream);

#ifdef __cplusplus
}
#endif
#endif /* CSA2_H */
