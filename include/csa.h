/*
 * csa.h -- C ABI of the GB300 (sm_103a) compressed sparse attention decode
 * library, libcsa.so.
 *
 * One decode step of DSV4-style Compressed Sparse Attention (CSA), as the
 * project's pages describe it:
 *   1. lightning-indexer logits of each query token against every compressed
 *      KV entry            -> csa_indexer_logits
 *   2. top-k over the causally visible entries  -> csa_topk
 *   3. gather of the selected FP8/BF16 latents together with the SWA window
 *                          -> fused into step 4 (csa_gather_swa is the
 *                             standalone packed gather)
 *   4. one sink-merged attention pass  -> csa_sink_attention_decode
 * and the heavily-compressed (HCA) variant that attends to every visible entry
 * with no indexer -> hca_sink_attention_decode. csa_decode_step runs 1, 2, 4.
 *
 * Beside the step: queries and latents are prepared by csa_head_norm_rope and
 * csa_head_norm_rope_e4m3, caches are filled by csa_cache_append and read back by
 * csa_cache_read, and the *_fp4 calls run the attention and the step over caches
 * of 4-bit records. Speculative decoding runs the attention and the step over a
 * tree of drafted tokens (csa_tree_attention_decode, hca_tree_attention_decode,
 * csa_tree_decode_step), accepts a path of it (csa_verify_drafts) and puts that
 * path's records into the caches (csa_cache_commit).
 *
 * Conventions for every call
 *  - Pointers are DEVICE pointers unless stated; the caller owns all memory.
 *    The library allocates no device memory (csa_pipeline_create makes a
 *    small host object, two streams and events) and keeps no state beyond
 *    per-process caches of kernel attributes, device properties and TMA
 *    descriptors.
 *  - Calls are asynchronous on `stream`; none synchronises the device (the
 *    diagnostics and csa_pipeline_wait/sync/destroy block the host).
 *    Argument errors are detected on the host before any launch and returned
 *    as codes; launch failures return CSA_ERR_CUDA (cudaGetLastError).
 *  - Status word: every compute call takes `status`, a caller-owned int32 in
 *    device memory (4-byte aligned; NULL = do not record). Problems found
 *    inside a kernel are recorded there, the first one winning (atomic
 *    compare-and-swap from CSA_OK): an index or position that would address
 *    memory outside a cache (the access is skipped: CSA_ERR_BAD_INDEX) and a
 *    bounded wait that expired (the kernel winds down: CSA_ERR_TIMEOUT).
 *    Kernels never trap. The word is read without stalling the stream by
 *    csa_check_device_status ("ROADMAP -- Stage E", section E4: no
 *    synchronisation on the decode path; return codes instead). Calls that
 *    share a word share its first-error-wins slot; give concurrent streams
 *    their own words.
 *  - Shapes fixed by the method: H = 128 query heads, latent D = 512 = 448
 *    FP8 E4M3 "nope" dims + 64 BF16 rope dims, indexer Hi = 64 heads x Di = 128
 *    FP8 dims. Tensors are dense row-major in the order of their index lists.
 *  - Every pointer must be 16-byte aligned.
 *
 * Latent record (one compressed entry or one SWA token), CSA_RECORD_BYTES:
 *   bytes [0,448)   nope dims, FP8 E4M3
 *   bytes [448,576) rope dims, BF16
 *   bytes [576,592) 4 fp32 dequantisation multipliers; multiplier i covers
 *                   nope dims [128i, min(128i+128, 448))
 * (pages: "DSV4 Audit", section B1 -- FP8 nope + BF16 rope, fed to attention
 * without a BF16 dequantised copy; "ROADMAP -- Stage E", section E1 -- FP8
 * entries with the inverse scale stored alongside.)
 */
#ifndef CSA_H_
#define CSA_H_

#include <stddef.h>
#include <stdint.h>
#include <cuda_runtime_api.h>

#ifdef __cplusplus
extern "C" {
#endif

#if defined(__GNUC__)
#define CSA_API __attribute__((visibility("default")))
#else
#define CSA_API
#endif

#define CSA_HEADS 128
#define CSA_LATENT_DIM 512
#define CSA_NOPE_DIM 448
#define CSA_ROPE_DIM 64
#define CSA_SCALE_BLOCK 128
#define CSA_RECORD_BYTES 592
#define CSA_INDEXER_HEADS 64
#define CSA_INDEXER_DIM 128
#define CSA_MAX_TOKENS_PER_SEQ 128 /* T: query tokens per sequence and step */
#define CSA_MAX_TOPK 2048
#define CSA_MAX_SWA_WINDOW 512 /* W */

typedef enum {
    CSA_OK = 0,
    CSA_ERR_INVALID_ARG = 1, /* null/misaligned pointer, size out of range */
    CSA_ERR_UNSUPPORTED = 2, /* a shape outside what the kernels implement */
    CSA_ERR_WORKSPACE = 3,   /* workspace missing or smaller than required */
    CSA_ERR_CUDA = 4,        /* a CUDA runtime call or launch failed */
    CSA_ERR_TIMEOUT = 5,     /* (device word) a bounded wait in a kernel expired */
    CSA_ERR_BAD_INDEX = 6    /* (device word) an index/position outside a cache */
} csa_status_t;

/* A cache of latent records (compressed entries). Logical entry c of sequence
 * b (0 <= c < seq_capacity) is record
 *     b * seq_stride + c                                     if block_table == NULL
 *     block_table[b*max_pages + c/page_records]*page_records + c%page_records
 * ("DSV4 Inference Kernel" README, Architecture: classical paged cache of
 * 128-token pages, i.e. 32 CSA entries or 1 HCA entry per page).
 * Records outside [0, n_records) are never read. */
typedef struct {
    const void *base;           /* device, n_records * CSA_RECORD_BYTES bytes */
    int64_t n_records;          /* records addressable from base */
    int64_t seq_stride;         /* contiguous mode: records between sequences */
    const int32_t *block_table; /* device [B, max_pages] or NULL */
    int32_t page_records;       /* paged mode: records per page (> 0) */
    int32_t max_pages;          /* paged mode: block-table row length */
    int32_t seq_capacity;       /* logical entries per sequence (Ncap) */
} csa_cache_desc;

/* Element types of tensors that a call reads in more than one type. */
typedef enum { CSA_BF16 = 0, CSA_FP16 = 1, CSA_FP32 = 2 } csa_dtype_t;

/* Formats of latent records. CSA_FORMAT_FP8 is the record above; a 4-bit
 * record, CSA_FP4_RECORD_BYTES, is
 *   bytes [0,224)   nope dims, E2M1, dim 2i in the low nibble of byte i
 *   bytes [224,352) rope dims, BF16
 *   bytes [352,380) 28 E4M3 block scales, scale i covers nope dims [16i, 16i+16)
 *   byte  380       power-of-two multiplier of the record, 2^(byte - 127)
 *                   (255: infinite, see csa_cache_append)
 *   bytes [381,384) zero
 * and nope dim d stands for e2m1(code d) * e4m3(scale d/16) * 2^(byte-127).
 * The product of an E2M1 and an E4M3 value has at most 6 significant bits and
 * the power of two changes none of them, so every 4-bit latent is a BF16
 * value exactly: the tensor cores read it without a further rounding. */
typedef enum { CSA_FORMAT_FP8 = 0, CSA_FORMAT_FP4 = 1 } csa_format_t;
#define CSA_FP4_RECORD_BYTES 384

typedef enum {
    CSA_OP_INDEXER = 0,
    CSA_OP_TOPK = 1,
    CSA_OP_ATTENTION = 2,     /* csa_sink_attention_decode, `k` = top-k */
    CSA_OP_HCA_ATTENTION = 3, /* hca_sink_attention_decode, `k` ignored */
    CSA_OP_DECODE_STEP = 4,   /* csa_decode_step */
    CSA_OP_TREE_ATTENTION = 5,     /* csa_tree_attention_decode, T = N */
    CSA_OP_HCA_TREE_ATTENTION = 6, /* hca_tree_attention_decode, T = N, `k` ignored */
    CSA_OP_TREE_STEP = 7,          /* csa_tree_decode_step, T = N */
    CSA_OP_VERIFY = 8              /* csa_verify_drafts, T = N, Ncap = V, `k` ignored: 0 so far */
} csa_op_t;

/* Workspace bytes that `op` needs for these sizes (0 if none). A workspace
 * passed to a call must be at least this large and 256-byte aligned; its
 * contents need no initialisation and are scratch between calls. */
CSA_API size_t csa_workspace_bytes(csa_op_t op, int B, int T, int Ncap, int k);

/* Step 1 -- lightning-indexer logits ("DSV4 Audit", section B2: weighted-ReLU
 * MQA logits of every query token against every compressed entry, FP8 keys).
 *   logits[b,t,c] = sum_h w_idx[b,t,h] *
 *                   max(0, q_idx_scale[b,t,h] * k_idx_scale[b,c] *
 *                          sum_d e4m3(q_idx[b,t,h,d]) * e4m3(k_idx[b,c,d]))
 * for c < n_vis(b,t), and -inf for n_vis(b,t) <= c < Ncap, where
 *   n_vis(b,t) = min(floor(q_pos[b,t] / m), n_comp[b], Ncap)
 * ("DSV4 Audit", section A3 item 1: a query sees only the compressed blocks
 * strictly before its own incomplete block; q_pos is the 0-based position).
 *   q_idx       [B,T,64,128] e4m3 codes     q_idx_scale [B,T,64] fp32 (> 0)
 *   w_idx       [B,T,64] fp32               k_idx [B,Ncap,128] e4m3 codes
 *   k_idx_scale [B,Ncap] fp32 (> 0)          q_pos [B,T] int32, n_comp [B] int32
 *   logits      [B,T,Ncap] fp32 (written in full)
 * Requires 1 <= T <= CSA_MAX_TOKENS_PER_SEQ, Ncap >= 1, m >= 1. Accumulation
 * is fp32. Up to 4 tokens of a sequence share one read of its keys; larger T
 * (a prefill-style step, "ROADMAP -- Stage E" section E8) runs as groups of
 * up to 4 tokens (the largest of 4, 3, 2, 1 dividing T), each reading the
 * keys again. */
CSA_API csa_status_t csa_indexer_logits(const uint8_t *q_idx, const float *q_idx_scale, const float *w_idx,
                                const uint8_t *k_idx, const float *k_idx_scale,
                                const int32_t *q_pos, const int32_t *n_comp,
                                int B, int T, int Ncap, int m, float *logits, int32_t *status,
                                cudaStream_t stream);

/* Step 2 -- top-k of the indexer logits over the visible entries ("DSV4
 * Audit", section B2 and "ROADMAP -- Stage E", section E7: top-k per query
 * token with warp-level reductions and no global lock).
 * For each (b,t): the min(k, n_vis) entries c < n_vis with the largest
 * logits, ties going to the lower index, written to topk_idx[b,t,0..cnt) in
 * ascending index order, the rest of the row set to -1; topk_cnt[b,t] = cnt.
 *   logits [B,T,Ncap] fp32 (entries >= n_vis are not read), topk_idx [B,T,k]
 *   int32, topk_cnt [B,T] int32. Requires 1 <= k <= min(Ncap, CSA_MAX_TOPK).
 * The workspace may be NULL when csa_workspace_bytes(CSA_OP_TOPK, ...) is 0;
 * rows of more than 32768 entries with ceil(Ncap / 32768) * k <= 32768 are
 * selected in two stages and keep the slices' candidate indices there
 * (4 * B * T * ceil(Ncap / 32768) * (k + 1) bytes). */
CSA_API csa_status_t csa_topk(const float *logits, const int32_t *q_pos, const int32_t *n_comp,
                      int B, int T, int Ncap, int m, int k, int32_t *topk_idx, int32_t *topk_cnt,
                      void *workspace, size_t workspace_bytes, int32_t *status, cudaStream_t stream);

/* Step 3, standalone -- packed candidate records ("DSV4 Audit", section A3:
 * the query attends to [top-k compressed entries] ++ [SWA window]; a token in
 * both is kept twice; "ROADMAP -- Stage E", section E1: gathers straight from
 * the FP8 cache, block-table strided).
 * For each (b,t) with p = q_pos[b,t]: kv_out[b,t,i] = comp entry
 * topk_idx[b,t,i] for i < topk_cnt[b,t], followed by the SWA records of
 * positions max(0,p-W+1) .. p (oldest first), position j read from
 * swa_ring[b, j mod R]; kv_cnt[b,t] = number written. Slots past kv_cnt are
 * not written. Byte-exact copies, no dequantisation.
 *   swa_ring [B,R,592] bytes, kv_out [B,T,k+W,592] bytes, kv_cnt [B,T] int32.
 * Requires 1 <= W <= R and q_pos >= 0. The caller keeps the ring holding the
 * window of every query token (R >= W + T - 1 for consecutive tokens). */
CSA_API csa_status_t csa_gather_swa(csa_cache_desc comp, const void *swa_ring, int R, int W,
                            const int32_t *topk_idx, const int32_t *topk_cnt, const int32_t *q_pos,
                            int B, int T, int k, void *kv_out, int32_t *kv_cnt, int32_t *status,
                            cudaStream_t stream);

/* Step 4 -- sink-merged attention over [top-k entries] ++ [SWA window]
 * ("DSV4 Inference Kernel" README, Architecture: one 512-d latent per entry
 * shared by all 128 heads as key and value; sink weights merge the sparse and
 * SWA terms). With x_j the dequantised candidate latents (nope code times
 * its block multiplier, rope as BF16), for every head h:
 *   z_j   = softmax_scale * sum_d q[b,t,h,d] * x_j[d]
 *   M     = max(sink[h], max_j z_j)
 *   den   = exp(sink[h] - M) + sum_j exp(z_j - M)
 *   out   = sum_j exp(z_j - M) x_j / den       (BF16)
 *   lse   = M + ln(den)                         (fp32)
 * No candidates: out = 0 and lse = sink[h].
 *   q [B,T,128,512] bf16, sink [128] fp32, out [B,T,128,512] bf16,
 *   lse [B,T,128] fp32; other arguments as in csa_gather_swa.
 * The candidates are read straight from the caches (no packed copy). */
CSA_API csa_status_t csa_sink_attention_decode(const void *q, const float *sink, float softmax_scale,
                                       csa_cache_desc comp, const void *swa_ring, int R, int W,
                                       const int32_t *topk_idx, const int32_t *topk_cnt,
                                       const int32_t *q_pos, int B, int T, int k,
                                       void *out, float *lse, void *workspace, size_t workspace_bytes,
                                       int32_t *status, cudaStream_t stream);

/* HCA variant ("DSV4 Inference Kernel" README, Architecture, m' = 128;
 * "ROADMAP -- Stage E", section E1, gather of all compressed entries):
 * step 4 with the candidates = every visible entry c < n_vis(b,t) (computed
 * with m = m_hca as in csa_indexer_logits) ++ the SWA window. No indexer. */
CSA_API csa_status_t hca_sink_attention_decode(const void *q, const float *sink, float softmax_scale,
                                       csa_cache_desc comp, const int32_t *n_comp,
                                       const void *swa_ring, int R, int W, const int32_t *q_pos,
                                       int B, int T, int m_hca, void *out, float *lse,
                                       void *workspace, size_t workspace_bytes, int32_t *status,
                                       cudaStream_t stream);

/* Output epilogue of the attention ("DSV4 Audit" section A4: the attention
 * output is turned back by RoPE(-t) at the query position t, which makes the
 * absolute positions carried by the summed latents relative; "ROADMAP --
 * Stage E" section E6: the output may leave the attention as FP4 E2M1 with a
 * per-128-element block amax, packed inside the same launch). Used by the
 * _ex entry points; NULL there means plain BF16 output.
 *   inverse_rope   nonzero: the rope dims of every head's output, pair i =
 *                  dims (448 + 2i, 449 + 2i), i < 32, are turned back by
 *                  a = t * rope_theta^(-2i/64) radians, t = q_pos[b,t]:
 *                    x' = x cos a + y sin a,   y' = -x sin a + y cos a
 *                  (the pages fix no RoPE convention; this pairing and
 *                  frequency schedule are this library's reading)
 *   rope_theta     RoPE base, > 1 (e.g. 10000); read only with inverse_rope
 *   out_fp4        NULL: BF16 output in `out`. Otherwise device
 *                  [B,T,128,256] bytes, 16-byte aligned: the E2M1 codes of
 *                  the 512 output dims (after the rotation), dim 2i in the
 *                  low nibble of byte i; `out` is not written and may be NULL
 *   out_fp4_scale  with out_fp4: device [B,T,128,4] fp32, 16-byte aligned:
 *                  s = amax / 6 of output dims [128 j, 128 j + 128) (1 when
 *                  they are all zero); code = the E2M1 value nearest to
 *                  value / s (ties to even, saturating at 6), so that
 *                  value ~ e2m1(code) * s */
typedef struct {
    int32_t inverse_rope;
    float rope_theta;
    uint8_t *out_fp4;
    float *out_fp4_scale;
} csa_attention_epilogue;

/* csa_sink_attention_decode / hca_sink_attention_decode with an output
 * epilogue (see csa_attention_epilogue); identical to them when `epilogue`
 * is NULL or asks for neither step. Same workspace sizes. A bad epilogue
 * (theta <= 1 with inverse_rope, out_fp4 without out_fp4_scale, misaligned
 * pointers) returns CSA_ERR_INVALID_ARG before any launch. */
CSA_API csa_status_t csa_sink_attention_decode_ex(const void *q, const float *sink, float softmax_scale,
                                                  csa_cache_desc comp, const void *swa_ring, int R, int W,
                                                  const int32_t *topk_idx, const int32_t *topk_cnt,
                                                  const int32_t *q_pos, int B, int T, int k, void *out, float *lse,
                                                  const csa_attention_epilogue *epilogue, void *workspace,
                                                  size_t workspace_bytes, int32_t *status, cudaStream_t stream);
CSA_API csa_status_t hca_sink_attention_decode_ex(const void *q, const float *sink, float softmax_scale,
                                                  csa_cache_desc comp, const int32_t *n_comp, const void *swa_ring,
                                                  int R, int W, const int32_t *q_pos, int B, int T, int m_hca,
                                                  void *out, float *lse, const csa_attention_epilogue *epilogue,
                                                  void *workspace, size_t workspace_bytes, int32_t *status,
                                                  cudaStream_t stream);

/* Allocation-free variant of csa_sink_attention_decode (the pages have no
 * counterpart; it exists for callers of this library that cannot allocate
 * device memory on the decode path -- e.g. a serving runtime whose device
 * memory is all reserved by its own pool at start-up, a plugin whose host
 * framework owns every device allocation, or latency-critical host code that
 * cannot afford cudaMalloc's implicit synchronisation -- and so cannot pass a
 * workspace). Same arguments and results as csa_sink_attention_decode minus
 * the workspace: the split partials live in a static 16 MiB device array that
 * every device which loads the library holds until the process exits.
 *  - No cudaMalloc, cudaFree or allocating library call is made.
 *  - The first call on a device (with that device current) looks up the
 *    array's device address once (cudaGetSymbolAddress) and caches it; make
 *    that first call before any stream capture.
 *  - Sizes whose partials exceed the array return CSA_ERR_UNSUPPORTED (use
 *    csa_sink_attention_decode with a workspace instead); every size with
 *    csa_workspace_bytes(CSA_OP_ATTENTION, B, T, Ncap, k) <= 16 MiB fits.
 *  - Argument checks and their status codes are those of
 *    csa_sink_attention_decode; `status` is the caller's status word.
 *  - Every call shares the array and leaves its contents behind; nothing in it
 *    needs to start at zero. Calls that overlap on the GPU (concurrent streams)
 *    race on the array: serialise them. */
CSA_API csa_status_t csa_sink_attention_decode_noalloc(const void *q, const float *sink, float softmax_scale,
                                                       csa_cache_desc comp, const void *swa_ring, int R, int W,
                                                       const int32_t *topk_idx, const int32_t *topk_cnt,
                                                       const int32_t *q_pos, int B, int T, int k, void *out,
                                                       float *lse, int32_t *status, cudaStream_t stream);

/* One CSA decode step: csa_indexer_logits -> csa_topk ->
 * csa_sink_attention_decode on one stream. Logits, indices and attention
 * scratch live in the workspace (csa_workspace_bytes(CSA_OP_DECODE_STEP,...)).
 * The indexer keys are contiguous per sequence ([B,Ncap,...]); comp may be
 * paged. Arguments keep the meaning given above. topk_idx/topk_cnt may be
 * NULL; if given ([B,T,k] / [B,T]) they receive the selection. */
CSA_API csa_status_t csa_decode_step(const uint8_t *q_idx, const float *q_idx_scale, const float *w_idx,
                             const uint8_t *k_idx, const float *k_idx_scale,
                             const void *q, const float *sink, float softmax_scale,
                             csa_cache_desc comp, const void *swa_ring, int R, int W,
                             const int32_t *q_pos, const int32_t *n_comp,
                             int B, int T, int Ncap, int m, int k,
                             void *out, float *lse, int32_t *topk_idx, int32_t *topk_cnt,
                             void *workspace, size_t workspace_bytes, int32_t *status, cudaStream_t stream);

/* csa_decode_step with the attention's output epilogue
 * (csa_attention_epilogue; NULL = csa_decode_step): the step's last kernel
 * writes the inverse-RoPE'd and/or E2M1 output ("ROADMAP -- Stage E",
 * section E6: the quantised output leaves the attention in the same launch).
 * With E2M1 output `out` may be NULL. Checks as csa_decode_step plus those of
 * csa_sink_attention_decode_ex, all before the first launch. */
CSA_API csa_status_t csa_decode_step_ex(const uint8_t *q_idx, const float *q_idx_scale, const float *w_idx,
                                        const uint8_t *k_idx, const float *k_idx_scale, const void *q,
                                        const float *sink, float softmax_scale, csa_cache_desc comp,
                                        const void *swa_ring, int R, int W, const int32_t *q_pos,
                                        const int32_t *n_comp, int B, int T, int Ncap, int m, int k, void *out,
                                        float *lse, int32_t *topk_idx, int32_t *topk_cnt,
                                        const csa_attention_epilogue *epilogue, void *workspace,
                                        size_t workspace_bytes, int32_t *status, cudaStream_t stream);

/* Normalisation and rotation of one head (csa_head_norm_rope,
 * csa_head_norm_rope_e4m3, csa_cache_append). With x the D values of a head:
 *   norm       nonzero: y_d = x_d * (sum_d x_d^2 / D + eps)^(-1/2) * weight[d]
 *              zero: y = x (weight must then be NULL)
 *   eps        >= 0, finite; read only with norm
 *   weight     device fp32 [D], 16-byte aligned, or NULL for all ones
 *   rope_dim   the last rope_dim values are turned as pairs i = (D - rope_dim +
 *              2i, D - rope_dim + 2i + 1) by a = p * rope_theta^(-2i/rope_dim)
 *              radians, p the token's position:
 *                x' = x cos a - y sin a,   y' = x sin a + y cos a
 *              (the rotation that csa_attention_epilogue turns back);
 *              0: no rotation
 *   rope_theta > 1, finite; read only with rope_dim > 0
 * Sums and the rotation are fp32, the angle is reduced to one turn in 64-bit
 * fixed point (positions far beyond 2^24 keep it), and the result is rounded
 * once, to the output's type. */
typedef struct {
    int32_t norm;
    float eps;
    const float *weight;
    int32_t rope_dim;
    float rope_theta;
} csa_norm_rope;

/* RMS norm of every head and the position rotation in one pass over the
 * heads: the attention's queries (H = 128, D = 512), or its latents before
 * they are cached (H = 1).
 *   x     element (b, t, h, d) at x[b*x_seq_stride + t*x_token_stride +
 *         h*x_head_stride + d] of type x_dtype (strides in elements, >= 0;
 *         base and strides multiples of 16 bytes): a slice of a wider
 *         projection needs no copy
 *   pos   [B,T] int32; a token with pos < 0 is padding: it is not read and its
 *         rows of the output are left as they were
 *   out   [B,T,H,D] BF16, dense. It may be x itself when x is dense BF16; any
 *         other overlap with x is not allowed.
 * Requires B, T, H >= 1, B*T <= 2^24, B*T*H < 2^31 - 2^20, D a multiple of 8 up to
 * 512 and rope_dim a multiple of 8 up to min(D, 256). The status word is
 * accepted as by every compute call; nothing is recorded in it. */
CSA_API csa_status_t csa_head_norm_rope(const void *x, csa_dtype_t x_dtype, int64_t x_seq_stride,
                                        int64_t x_token_stride, int64_t x_head_stride, const int32_t *pos, int B,
                                        int T, int H, int D, const csa_norm_rope *how, void *out, int32_t *status,
                                        cudaStream_t stream);

/* The same pass with E4M3 output, the form that csa_indexer_logits reads its
 * queries in (H = 64, D = 128): scale[b,t,h] = amax_d |y_d| / 448 (1 when all
 * are zero), codes[b,t,h,d] = e4m3(y_d / scale), ties as in csa_cache_append.
 *   codes [B,T,H,D] bytes, scale [B,T,H] fp32; neither may overlap x. */
CSA_API csa_status_t csa_head_norm_rope_e4m3(const void *x, csa_dtype_t x_dtype, int64_t x_seq_stride,
                                             int64_t x_token_stride, int64_t x_head_stride, const int32_t *pos,
                                             int B, int T, int H, int D, const csa_norm_rope *how, uint8_t *codes,
                                             float *scale, int32_t *status, cudaStream_t stream);

/* Indexer keys of the entries that csa_cache_append writes: 128 values each,
 * rotated like the latent (the last 64 of them, at the same position; not
 * normalised) and stored as csa_indexer_logits reads them.
 *   key         element (b, t, d) at key[b*seq_stride + t*token_stride + d], of
 *               the latents' type (same rules for strides and alignment)
 *   k_idx       [B,Ncap,128] e4m3 codes, k_idx_scale [B,Ncap] fp32
 *               (amax / 448, 1 when all are zero)
 * Entries at or past Ncap are not stored (CSA_ERR_BAD_INDEX). */
typedef struct {
    const void *key;
    int64_t seq_stride, token_stride;
    uint8_t *k_idx;
    float *k_idx_scale;
    int32_t Ncap;
} csa_index_append;

/* Appends latents to a cache, normalised and rotated on the way: token t of
 * sequence b (t < count[b]) becomes entry e = first[b] + t of its sequence,
 * at position p = e * pos_stride (1 for tokens; tokens per entry for
 * compressed entries).
 *   cache  the records, contiguous or paged, of format fmt; base is written
 *   ring   nonzero: the record is entry e mod seq_capacity (the sliding
 *          window's ring, a contiguous cache with seq_stride =
 *          seq_capacity = R), and of more than seq_capacity tokens only the last
 *          seq_capacity are kept
 *   x      element (b, t, d), d < 512, at x[b*x_seq_stride + t*x_token_stride + d]
 *          of type x_dtype (strides in elements; base and strides multiples
 *          of 16 bytes)
 *   first  [B] int32, >= 0
 *   count  [B] int32 in [0, T], or NULL for T tokens of every sequence
 *   how    D = 512; rope_dim 64 or 0
 *   idx    NULL, or the entries' indexer keys, stored by the same launch
 *          (not with ring)
 * Records: rope dims are rounded to BF16. FP8: multiplier = amax / 448 of each
 * 128-dim block (1 when it is all zero), code = e4m3(y / multiplier). 4 bits:
 * with amax over the 448 nope dims, E = the smallest whole number with amax <=
 * 6 * 448 * 2^E (at least -111; 0 when all are zero), the block scale s =
 * e4m3(max |y| of the block / 6 * 2^-E), code = e2m1(y / (s * 2^E)), ties to
 * even in both, codes 0 where s is 0. The 4-bit quotients are decided as if
 * computed exactly from the fp32 y; those of E4M3 codes are y * 448 / amax, exact
 * for 16-bit inputs that are not normalised, else within two fp32 roundings. An
 * infinite or NaN nope dim makes its FP8 block or its 4-bit record read back as
 * NaN in every nope dim.
 * An entry outside the cache is not stored (CSA_ERR_BAD_INDEX, also for
 * first < 0 or a count outside [0, T], which is then clamped). Every other
 * record is left as it was. Sequences of one call must not share a page that
 * it writes. Requires B, T >= 1, B*T <= 2^24, 1 <= pos_stride <= 65536. */
CSA_API csa_status_t csa_cache_append(csa_cache_desc cache, csa_format_t fmt, int ring, const void *x,
                                      csa_dtype_t x_dtype, int64_t x_seq_stride, int64_t x_token_stride,
                                      const int32_t *first, const int32_t *count, int B, int T, int pos_stride,
                                      const csa_norm_rope *how, const csa_index_append *idx, int32_t *status,
                                      cudaStream_t stream);

/* Reads entries back as BF16 latents: out[b,t,0..512) = the values of entry
 * first[b] + t of sequence b for t < count[b] (with ring: of entry
 * (first[b] + t) mod seq_capacity, for the last seq_capacity of these t). FP8
 * values are rounded to BF16 (code x multiplier), 4-bit values are exact. Rows
 * of out that no entry belongs to, or whose entry lies outside the cache
 * (CSA_ERR_BAD_INDEX), are left as they were. Arguments as in csa_cache_append;
 * out [B,T,512] BF16. */
CSA_API csa_status_t csa_cache_read(csa_cache_desc cache, csa_format_t fmt, int ring, const int32_t *first,
                                    const int32_t *count, int B, int T, void *out, int32_t *status,
                                    cudaStream_t stream);

/* The sink-merged attention over caches of 4-bit records: formulas, arguments,
 * output epilogue, workspace (csa_workspace_bytes of CSA_OP_ATTENTION,
 * CSA_OP_HCA_ATTENTION and CSA_OP_DECODE_STEP) and error behaviour of
 * csa_sink_attention_decode_ex, hca_sink_attention_decode_ex and
 * csa_decode_step_ex, but comp and swa_ring hold records of
 * CSA_FP4_RECORD_BYTES bytes (swa_ring [B,R,384]). The latents enter the tensor
 * cores without a rounding; the softmax weights are rounded to BF16, and the
 * partial outputs of a query that is split over several CTAs to FP16 in units of
 * a power of two for each 32 dims. lse of a query without candidates is the sink.
 * With E2M1 output, a block of 128 output dims with a NaN has a NaN multiplier. */
CSA_API csa_status_t csa_sink_attention_decode_fp4(const void *q, const float *sink, float softmax_scale,
                                                   csa_cache_desc comp, const void *swa_ring, int R, int W,
                                                   const int32_t *topk_idx, const int32_t *topk_cnt,
                                                   const int32_t *q_pos, int B, int T, int k, void *out, float *lse,
                                                   const csa_attention_epilogue *epilogue, void *workspace,
                                                   size_t workspace_bytes, int32_t *status, cudaStream_t stream);
CSA_API csa_status_t hca_sink_attention_decode_fp4(const void *q, const float *sink, float softmax_scale,
                                                   csa_cache_desc comp, const int32_t *n_comp, const void *swa_ring,
                                                   int R, int W, const int32_t *q_pos, int B, int T, int m_hca,
                                                   void *out, float *lse, const csa_attention_epilogue *epilogue,
                                                   void *workspace, size_t workspace_bytes, int32_t *status,
                                                   cudaStream_t stream);
CSA_API csa_status_t csa_decode_step_fp4(const uint8_t *q_idx, const float *q_idx_scale, const float *w_idx,
                                         const uint8_t *k_idx, const float *k_idx_scale, const void *q,
                                         const float *sink, float softmax_scale, csa_cache_desc comp,
                                         const void *swa_ring, int R, int W, const int32_t *q_pos,
                                         const int32_t *n_comp, int B, int T, int Ncap, int m, int k, void *out,
                                         float *lse, int32_t *topk_idx, int32_t *topk_cnt,
                                         const csa_attention_epilogue *epilogue, void *workspace,
                                         size_t workspace_bytes, int32_t *status, cudaStream_t stream);

/* ---- Speculative decoding: a tree of drafted tokens in one step.
 *
 * A tree of N tokens a sequence is an array of parents: parent[b,i] < i is the
 * token that token i follows, -1 the last committed token (one that is in the
 * sequence's window ring). Token i stands at position q_pos[b,i] = position of its
 * parent + 1 (siblings share one); q_pos[b,i] < 0 marks padding: the token is not
 * computed and its rows of the outputs are left as they were.
 *   records  [B,N, record bytes] the drafted tokens' latents, records of the cache's
 *            format (csa_cache_append with B sequences of N entries makes them)
 *   parent   [B,N] int32. An entry outside [-1, i) is taken as -1
 *            (CSA_ERR_BAD_INDEX) */
typedef struct {
    const void *records;
    const int32_t *parent;
} csa_draft_tree;

/* The sink-merged attention of a tree's tokens: formulas, arguments, epilogue and
 * error behaviour of csa_sink_attention_decode_ex, hca_sink_attention_decode_ex
 * and csa_decode_step_ex, over caches of either format `fmt` (comp, swa_ring and
 * tree->records hold records of it), but the window of token i at position p is
 * itself, its ancestors a_1, a_2, .. in the tree and, before them, the
 * committed tokens: the W positions p, p - 1, .. (none below 0), of which the
 * first come from tree->records and, from the last committed token's on, from the
 * ring. The ring has to hold the W - 1 committed positions before a root token
 * (R >= W); no token of the tree is read from it. For every token the selected or
 * visible compressed entries are those of its position q_pos among the stored ones, as
 * without a tree (csa_indexer_logits' n_vis). An entry that the tree's own tokens complete
 * is not among them: tokens behind a compression boundary have it in their window, token by
 * token, but not also as an entry, which decoding one token at a time would give them, and
 * their logits differ by that. The caller of a chain can append such entries (and their
 * keys, and raise n_comp) before the call; branches of a tree would need different entries
 * at one index, which these calls do not have. After the commit the entries that the accepted
 * tokens complete are appended as always (csa_cache_append).
 * FP8 latents enter the scores as two BF16 numbers (2^-17 of a latent is lost) and the
 * output rounded to BF16, 4-bit ones are exact; weights and partial outputs are
 * rounded as in the *_fp4 calls, and as there, a NaN or infinite latent reaches the
 * rows that select it and no others. Requires N <= CSA_MAX_TOKENS_PER_SEQ;
 * workspaces: CSA_OP_TREE_ATTENTION, CSA_OP_HCA_TREE_ATTENTION, CSA_OP_TREE_STEP. */
CSA_API csa_status_t csa_tree_attention_decode(const void *q, const float *sink, float softmax_scale,
                                               csa_cache_desc comp, csa_format_t fmt, const void *swa_ring, int R,
                                               int W, const csa_draft_tree *tree, const int32_t *topk_idx,
                                               const int32_t *topk_cnt, const int32_t *q_pos, int B, int N, int k,
                                               void *out, float *lse, const csa_attention_epilogue *epilogue,
                                               void *workspace, size_t workspace_bytes, int32_t *status,
                                               cudaStream_t stream);
CSA_API csa_status_t hca_tree_attention_decode(const void *q, const float *sink, float softmax_scale,
                                               csa_cache_desc comp, csa_format_t fmt, const int32_t *n_comp,
                                               const void *swa_ring, int R, int W, const csa_draft_tree *tree,
                                               const int32_t *q_pos, int B, int N, int m_hca, void *out, float *lse,
                                               const csa_attention_epilogue *epilogue, void *workspace,
                                               size_t workspace_bytes, int32_t *status, cudaStream_t stream);
CSA_API csa_status_t csa_tree_decode_step(const uint8_t *q_idx, const float *q_idx_scale, const float *w_idx,
                                          const uint8_t *k_idx, const float *k_idx_scale, const void *q,
                                          const float *sink, float softmax_scale, csa_cache_desc comp,
                                          csa_format_t fmt, const void *swa_ring, int R, int W,
                                          const csa_draft_tree *tree, const int32_t *q_pos, const int32_t *n_comp,
                                          int B, int N, int Ncap, int m, int k, void *out, float *lse,
                                          int32_t *topk_idx, int32_t *topk_cnt,
                                          const csa_attention_epilogue *epilogue, void *workspace,
                                          size_t workspace_bytes, int32_t *status, cudaStream_t stream);

/* Verification of a tree's drafted tokens against the target's distribution, given
 * the random numbers: what is emitted is distributed as if drawn from the target
 * whose logits are passed (of a tree's attention, see above for what these know).
 * Token 0 is the sequence's newest known token (the last one emitted), the others
 * are drafts. With z = logits[b,j,.], t = temperature[b] and
 *   p_j(v) = exp(z_v / t) / sum_w exp(z_w / t),   q_j(v) = draft_probs[b,j,v]
 * the walk starts at j = 0 with r = p_0, R = 1 and goes through the children i of
 * j (those with parent[b,i] = j) in ascending order. With x = token[b,i]:
 *   accept  if uniform[b,i] * q_j(x) * R < r(x): j becomes i, r = p_i, R = 1;
 *   reject  else: r = max(r - R q_j, 0) for every v, R = sum_v r(v).
 * Without draft_probs (drafts that are no draws: the best tokens, looked-up text)
 * q_j(x) is 1 and a rejection sets r(x) = 0 instead. When no child of j is left,
 * next_token[b] = the v with the largest r(v) / noise[b,v] among r(v) > 0, the lowest
 * on ties: for noise of exponential variates a draw from r. (If rounding left no
 * r(v) > 0, r is p_j again.) t <= 0 or NaN is greedy: a child is accepted if its
 * token is the largest logit's (the lowest on ties), which also is next_token.
 *   logits       element (b, i, v) at logits[b*seq_stride + i*token_stride + v], of
 *                type logits_dtype; strides in elements, >= 0. -inf masks a token. A
 *                row whose largest logit is not finite (all are -inf, one is +inf or
 *                NaN) has no distribution: if the walk reaches it, it ends there
 *                and next_token is -1
 *   draft_probs  NULL, or [B,N,V] of type draft_dtype, dense: row i is the
 *                distribution that the children of i were drawn from (of rows that the
 *                walk does not reach no more than the children's own elements is read,
 *                of rows without children nothing counts)
 *   token        [B,N] int32; parent [B,N] int32 (see csa_draft_tree; token 0's is not
 *                used, and tokens that token 0 does not lead to are never reached:
 *                padding has parent -1, and any entry outside [-1,i) is taken as -1 here
 *                without being reported). A draft outside [0,V) is never
 *                accepted and takes nothing from r (CSA_ERR_BAD_INDEX if it is tried)
 *   uniform      [B,N] fp32 in [0,1)      noise [B,V] fp32, > 0
 *   temperature  [B] fp32, or NULL for 1
 *   path         [B,N] int32: the accepted tokens' numbers from 0 on, -1 behind them
 *   accepted     [B] int32 in [1,N]: how many these are
 *   next_token   [B] int32
 * After CSA_ERR_TIMEOUT every sequence has its result, or the part of its path that had
 * been walked and next_token -1. Weights, sums and quotients are fp32. Requires B >= 1, 1 <= N <=
 * CSA_MAX_TOKENS_PER_SEQ, B*N <= 65535, 1 <= V <= 2^24. Pointers need the alignment
 * of their elements only (rows that all begin on 16 bytes are read in wider loads). */
CSA_API csa_status_t csa_verify_drafts(const void *logits, csa_dtype_t logits_dtype, int64_t seq_stride,
                                       int64_t token_stride, const void *draft_probs, csa_dtype_t draft_dtype,
                                       const int32_t *token, const int32_t *parent, const float *uniform,
                                       const float *noise, const float *temperature, int B, int N, int V,
                                       int32_t *path, int32_t *accepted, int32_t *next_token, void *workspace,
                                       size_t workspace_bytes, int32_t *status, cudaStream_t stream);

/* Puts records into a cache byte for byte: record select[b,t] of sequence b
 * (t < count[b]) becomes entry first[b] + t of its sequence. After
 * csa_verify_drafts, select is its path, count its accepted, first the number of
 * committed tokens.
 *   cache, fmt, ring, first, count   as in csa_cache_append (base is written; of more
 *            than seq_capacity tokens only the last are kept in a ring)
 *   records  [B,N, record bytes], not part of the cache
 *   select   [B,T] int32 in [0,N) (entries behind count are not read), or NULL for t. As
 *            every pointer of this call it begins on 16 bytes, and so has a path that
 *            csa_verify_drafts (which asks for 4) writes for it
 * An entry outside the cache or a select outside [0,N) is not stored
 * (CSA_ERR_BAD_INDEX); every other record of the cache is left as it was. Sequences of one
 * call must not share a page that it writes. Requires
 * B, T, N >= 1, B*T <= 2^24, and T <= N without select. */
CSA_API csa_status_t csa_cache_commit(csa_cache_desc cache, csa_format_t fmt, int ring, const void *records, int N,
                                      const int32_t *select, const int32_t *first, const int32_t *count, int B,
                                      int T, int32_t *status, cudaStream_t stream);

/* Host-I/O decode pipeline (the pages have no counterpart; it serves callers
 * whose query-side inputs arrive in, and whose results go back to, host
 * memory). csa_decode_step_host runs csa_decode_step on per-step copies of
 * the query-side inputs taken from host memory and copies out/lse back to
 * host memory. Each step uses one of `depth` staging slots in device memory,
 * so the host->device copy of step i+1 and the device->host copy of step i-1
 * run on two copy streams while step i's kernels run on the compute stream;
 * nothing blocks the host until csa_pipeline_wait / csa_pipeline_sync
 * ("ROADMAP -- Stage E", section E4: no synchronisation on the decode path).
 * Results are identical to csa_decode_step on the same inputs.
 *
 * csa_pipeline_staging_bytes: device bytes of the staging area for these
 * sizes (depth slots of q_idx, q_idx_scale, w_idx, q, q_pos, out, lse, each
 * 256-byte aligned); 0 if an argument is out of range. */
typedef struct csa_pipeline_s *csa_pipeline_t;
#define CSA_PIPELINE_MAX_DEPTH 4

CSA_API size_t csa_pipeline_staging_bytes(int B, int T, int depth);

/* Creates a pipeline for B sequences x T tokens on the current device.
 *   staging   device memory of >= csa_pipeline_staging_bytes(B, T, depth)
 *             bytes, 256-byte aligned, owned by the caller and untouched by
 *             anything else while the pipeline lives
 *   depth     2..CSA_PIPELINE_MAX_DEPTH staging slots
 *   compute   the caller's stream for the kernels (0 = legacy default)
 * Allocates the host-side object and creates two non-blocking copy streams
 * and 3 x depth events on the current device (no device memory). Returns
 * CSA_ERR_INVALID_ARG for a null handle or staging, a misaligned or short
 * staging area, or sizes out of range; CSA_ERR_CUDA if a stream or event
 * cannot be created (nothing is left behind). */
CSA_API csa_status_t csa_pipeline_create(csa_pipeline_t *pipeline, int B, int T, int depth, void *staging,
                                         size_t staging_bytes, cudaStream_t compute);

/* Enqueues one decode step. Pointers prefixed h_ are HOST memory with the
 * layouts of csa_decode_step (q_idx [B,T,64,128] e4m3 codes, q_idx_scale and
 * w_idx [B,T,64] fp32, q [B,T,128,512] bf16, q_pos [B,T] int32; out
 * [B,T,128,512] bf16, lse [B,T,128] fp32); page-locked host memory lets the
 * copies run asynchronously and overlap (pageable memory works, serialised).
 * The other arguments are the device-resident layer state and sizes of
 * csa_decode_step (B and T are the pipeline's). The host inputs must stay
 * unchanged and the host outputs unread until csa_pipeline_wait(step) (or
 * csa_pipeline_sync) returns. *step_out (may be NULL) receives the step's
 * ordinal, 0 for the first step of the pipeline. Arguments are checked before
 * anything is enqueued; CSA_ERR_INVALID_ARG also when the current device is
 * not the pipeline's. */
CSA_API csa_status_t csa_decode_step_host(csa_pipeline_t pipeline, const uint8_t *h_q_idx,
                                          const float *h_q_idx_scale, const float *h_w_idx, const void *h_q,
                                          const int32_t *h_q_pos, const uint8_t *k_idx, const float *k_idx_scale,
                                          const float *sink, float softmax_scale, csa_cache_desc comp,
                                          const void *swa_ring, int R, int W, const int32_t *n_comp, int Ncap,
                                          int m, int k, void *h_out, float *h_lse, void *workspace,
                                          size_t workspace_bytes, int32_t *status, int64_t *step_out);

/* Blocks the host until step `step` (an ordinal returned by
 * csa_decode_step_host) has its results in host memory and its host inputs
 * are no longer read. CSA_ERR_INVALID_ARG for a step not yet enqueued;
 * CSA_ERR_CUDA if a copy or kernel failed. */
CSA_API csa_status_t csa_pipeline_wait(csa_pipeline_t pipeline, int64_t step);

/* Blocks the host until every enqueued step has completed. */
CSA_API csa_status_t csa_pipeline_sync(csa_pipeline_t pipeline);

/* Waits for every enqueued step, then releases the streams, events and host
 * object (not the staging memory, which the caller owns). NULL is a no-op. */
CSA_API csa_status_t csa_pipeline_destroy(csa_pipeline_t pipeline);

/* Reads and clears a status word without synchronising ("ROADMAP -- Stage
 * E", section E4: no synchronisation on the decode path; errors come back as
 * codes). Enqueues on `stream` a copy of *status (device) into *host_status
 * (host memory; page-locked memory keeps the copy asynchronous, pageable
 * memory makes the runtime stage it) followed by a reset of *status to
 * CSA_OK. The value in *host_status is valid once the stream has passed this
 * point (an event recorded after the call, or a synchronisation chosen by
 * the caller): CSA_OK, or the first CSA_ERR_TIMEOUT / CSA_ERR_BAD_INDEX that
 * a kernel recorded in the word since the previous reset. Work enqueued on
 * the stream after this call records into a clean word. Legal inside CUDA
 * graph capture. CSA_ERR_INVALID_ARG for a null or misaligned pointer,
 * CSA_ERR_CUDA if the copy or the reset cannot be enqueued. */
CSA_API csa_status_t csa_check_device_status(int32_t *status, int32_t *host_status, cudaStream_t stream);

/* Blocking convenience for tests and diagnostics: csa_check_device_status
 * into a local, then cudaStreamSynchronize(stream), then *host_code = the
 * value read. Not for the decode path. */
CSA_API csa_status_t csa_read_device_error(int32_t *status, int32_t *host_code, cudaStream_t stream);

/* Diagnostic: sets the time limit of the bounded waits inside the tensor-core
 * kernels (indexer and attention) and the verification for launches made after this call, in
 * nanoseconds of GPU global time; 0 restores the default of one second. A
 * wait that reaches the limit records CSA_ERR_TIMEOUT in the status word and
 * the kernel winds down: it drains its own copies and MMAs already in flight
 * (those waits keep the one-second limit), frees its tensor memory and exits.
 * Exists so that tests can drive the timeout path without hanging or faulting
 * anything; process-wide, not for the decode path. */
CSA_API void csa_debug_set_wait_limit_ns(uint64_t ns);

/* Static description of a status code. */
CSA_API const char *csa_status_string(csa_status_t status);

/* Number of kernels this process has launched through the library (all
 * devices, all streams; a host-side counter incremented at every launch). */
CSA_API uint64_t csa_kernel_launches(void);

/* Library ABI version (major * 100 + minor). */
CSA_API int csa_version(void);

#ifdef __cplusplus
}
#endif

#endif /* CSA_H_ */
