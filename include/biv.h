/*
 * libbiv -- batch-invariant transformer forward for one GB300 (sm_103a).
 *
 * Every call computes each output row from that row's own inputs (and its own
 * sequence's KV cache or SSM state) with one fixed reduction order, so a
 * token's logprob does not change with batch size, batch mix, prefill vs
 * chunked prefill vs decode, eager vs CUDA-Graph replay, or rollout vs
 * trainer recompute.  The requirement and the rules that achieve it (one
 * computation path, one quantisation rule, one tie-break, one accumulation
 * order per op) come from "Finish RL Training Faster: Bitwise-Consistent,
 * High-Performance, Agent-Driven", sections "零差异需要一个精确的比较对象" and
 * "让训练前向使用推理的数值", and from "No More Train-Inference Mismatch:
 * Bitwise Consistent On-Policy Reinforcement Learning with vLLM and
 * TorchTitan", section "方法细节".
 *
 * Conventions for every entry point:
 *  - All tensor pointers are DEVICE pointers owned by the caller; the library
 *    never allocates, frees or synchronises (except biv_poll_error), and only
 *    launches kernels on the given stream.  Weights may be updated in place
 *    between calls (captured graphs keep reading the same addresses).
 *  - bf16 tensors are passed as uint16_t* (raw bfloat16 payloads); FP8 tensors
 *    as uint8_t* (OCP E4M3FN codes).  Row-major; *_stride arguments are in
 *    ELEMENTS between consecutive rows.
 *  - Pointers used with 16-byte vector or TMA access must be 16-byte aligned
 *    and row strides must keep rows 16-byte aligned; the host check returns
 *    BIV_ERR_INVALID otherwise, without launching anything.
 *  - Zero-sized work (rows == 0, T == 0 ...) returns BIV_OK and launches nothing.
 *  - On error the status is returned and biv_last_error() describes it.
 *  - mode BIV_MODE_FAST switches the split-K / split-KV choice to one that
 *    depends on the batch (the non-invariant comparator); results then change
 *    with batch size.  BIV_MODE_INVARIANT never lets the batch enter a
 *    reduction.
 */
#ifndef BIV_H
#define BIV_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef struct CUstream_st* biv_stream_t; /* a cudaStream_t; NULL = legacy default stream */

typedef enum {
  BIV_OK = 0,
  BIV_ERR_INVALID = 1,     /* bad argument: nothing was launched */
  BIV_ERR_UNSUPPORTED = 2, /* valid but not implemented shape/dtype combination */
  BIV_ERR_WORKSPACE = 3,   /* workspace pointer NULL or smaller than required */
  BIV_ERR_CUDA = 4,        /* a CUDA runtime/driver call or launch failed */
  BIV_ERR_TIMEOUT = 5      /* a device-side wait gave up (see biv_poll_error) */
} biv_status;

typedef enum { BIV_MODE_INVARIANT = 0, BIV_MODE_FAST = 1 } biv_mode;
typedef enum { BIV_BF16 = 0, BIV_F32 = 1, BIV_E4M3 = 2 } biv_dtype;

/* Chunk partials that a bf16 biv_gemm left in its workspace: the output
 * element (row, col) is RN(((p[0] + p[1]) + p[2]) + ...) with p[c] =
 * p + c*chunk_stride + row*ld + col, rounded once to the GEMM's output type;
 * chunks == 0 means the call wrote C itself. */
typedef struct {
  const float* p;
  int chunks;
  int64_t ld;
  int64_t chunk_stride;
} biv_partials;


/* Library version (major*10000 + minor*100 + patch). */
int biv_version(void);

/* Thread-local description of the last error on this thread; never NULL. */
const char* biv_last_error(void);

/* Number of SMs of the current device (0 if no device). */
int biv_device_sm_count(void);

/* Reads and clears the device error word that bounded device-side waits set
 * when they give up.  Synchronises the given stream.  *code receives the word
 * (0 = no timeout).  Returns BIV_ERR_TIMEOUT when the word was non-zero. */
biv_status biv_poll_error(biv_stream_t stream, int* code);

/* Test hook for the timeout path: launches one CTA that waits on an mbarrier
 * nothing will ever arrive on, for at most `limit_ns` nanoseconds, then sets
 * the device error word and returns.  Never hangs, never traps. */
biv_status biv_selftest_timeout(uint64_t limit_ns, biv_stream_t stream);

/* ---------------------------------------------------------------- embed --
 * h[t, :] = table[ids[t], :]   ids int32 [T] (0 <= id < vocab, checked on the
 * device: an out-of-range id writes a zero row and sets the error word);
 * table bf16 [vocab, d]; h bf16 [T, d] with row stride h_stride. */
biv_status biv_embed(const int32_t* ids, const uint16_t* table, int vocab, int T, int d,
                     uint16_t* h, int64_t h_stride, biv_stream_t stream);

/* ------------------------------------------------------------ RMSNorm ----
 * Fused residual add + RMSNorm ("No More Train-Inference Mismatch", section
 * "方法细节": fused RMSNorm with residual).  With residual != NULL:
 *   r' = bf16(x + r) (written back to residual), y = bf16(r' * inv * w);
 * with residual == NULL: y = bf16(x * inv * w); inv = 1/sqrt(mean(v^2) + eps)
 * where v is r' (or x), summed in FP32 in a fixed tree that depends on d
 * only.  x, residual, y bf16 [rows, d] with their own row strides; w bf16 [d].
 * d must be a multiple of 8 and <= 8192; y may alias x. */
biv_status biv_add_rmsnorm(const uint16_t* x, int64_t x_stride, uint16_t* residual,
                           int64_t r_stride, const uint16_t* w, uint16_t* y, int64_t y_stride,
                           int rows, int d, float eps, biv_stream_t stream);

/* The same, with x given as the chunk partials of the GEMM that produced it
 * (biv_gemm with defer_fold): x = the GEMM's rounded output, formed here
 * instead of by the GEMM's fold kernel, so the result is the same bit for
 * bit and one launch and one round trip of x are saved.  The partials stay
 * the caller's (the GEMM workspace) and are only read.  BIV_ERR_INVALID on
 * x NULL or chunks outside 1..8, a partial base not 16-byte aligned, or
 * ld / chunk_stride not multiples of 4. */
biv_status biv_add_rmsnorm_partials(const biv_partials* x, uint16_t* residual, int64_t r_stride,
                                    const uint16_t* w, uint16_t* y, int64_t y_stride, int rows,
                                    int d, float eps, biv_stream_t stream);

/* ------------------------------------------------------------ SiLU-mul ----
 * y = bf16(silu(g) * u), silu(g) = g / (1 + exp(-g)) in FP32, for
 * gate_up = [g | u] bf16 [rows, 2I] ("No More Train-Inference Mismatch",
 * section "方法细节": fused SiLU MLP).  y bf16 [rows, I].  I % 8 == 0. */
biv_status biv_silu_mul(const uint16_t* gate_up, int64_t gu_stride, uint16_t* y,
                        int64_t y_stride, int rows, int I, biv_stream_t stream);

/* The same, with gate_up given as the chunk partials of the GEMM that
 * produced it (biv_gemm with defer_fold; partial columns [0, I) are g and
 * [I, 2I) are u): folded here to the GEMM's bf16 output, so y is the same bit
 * for bit.  BIV_ERR_INVALID on chunks outside 1..8, a partial base not
 * 16-byte aligned, or ld / chunk_stride not multiples of 4 or ld < 2I. */
biv_status biv_silu_mul_partials(const biv_partials* gate_up, uint16_t* y, int64_t y_stride,
                                 int rows, int I, biv_stream_t stream);

/* --------------------------------------------------------- RoPE table ----
 * cos_sin float32 [2, max_pos, D/2]: cos then sin of pos * theta^(-2i/D),
 * computed in double precision on the device and rounded to FP32. */
biv_status biv_rope_table(double theta, int D, int max_pos, float* cos_sin,
                          biv_stream_t stream);

/* ---------------------------------------------------- QK-norm + RoPE ----
 * In place on the q and k heads of a packed qkv buffer [T, (Hq+2Hkv)*D]:
 * q at columns [0, Hq*D), k at [Hq*D, (Hq+Hkv)*D).  For each (token, head):
 * optional per-head RMSNorm with gain q_w / k_w bf16 [D] (NULL = skip, the
 * norm output rounded to bf16), then rotate-half RoPE with pairs
 * (i, i+D/2) at position pos[t] (int32 [T], 0 <= pos < max_pos), FP32
 * arithmetic, bf16 result.  D in {64, 80, 128}. */
biv_status biv_qk_norm_rope(uint16_t* qkv, int64_t row_stride, int T, int Hq, int Hkv, int D,
                            const uint16_t* q_w, const uint16_t* k_w, const float* cos_sin,
                            int max_pos, const int32_t* pos, float eps, biv_stream_t stream);

/* ------------------------------------------------------- KV cache store --
 * Paged KV cache, page size `page` tokens: slot s = page_id*page + offset.
 * k, v rows: bf16 [T, Hkv, D] at k + t*row_stride, v + t*row_stride.
 * slot int64 [T] (slot < 0 = skip the row).
 *
 * biv_kv_store_bf16: k_cache/v_cache bf16 [pages, page, Hkv, D].
 * biv_kv_fp8_quant ("Finish RL Training Faster", section
 *   "让训练前向使用推理的数值": the cache stays FP8 and every path makes the same
 *   round trip): per (token, kv head), separately for K and V,
 *   s = amax/448 (IEEE division; 1 when amax = 0),
 *   code = e4m3_rne_satfinite(x / s); codes uint8 [pages, page, Hkv, D],
 *   scales float32 [pages, page, Hkv]. */
biv_status biv_kv_store_bf16(const uint16_t* k, const uint16_t* v, int64_t row_stride,
                             const int64_t* slot, int T, int Hkv, int D, uint16_t* k_cache,
                             uint16_t* v_cache, biv_stream_t stream);
biv_status biv_kv_fp8_quant(const uint16_t* k, const uint16_t* v, int64_t row_stride,
                            const int64_t* slot, int T, int Hkv, int D, uint8_t* k_codes,
                            uint8_t* v_codes, float* k_scales, float* v_scales,
                            biv_stream_t stream);

/* QKV finalize: biv_qk_norm_rope followed by biv_kv_store_bf16 (kv_dtype
 * BIV_BF16) or biv_kv_fp8_quant (BIV_E4M3) of the k and v heads, in one
 * pass with the same per-element operations, so the same bits.  When
 * qkv_partials is non-NULL with chunks > 0, the packed qkv [T, (Hq+2Hkv)*D]
 * is first formed from the QKV GEMM's chunk partials (biv_gemm with
 * defer_fold) and written to qkv; otherwise qkv holds it already.  After the
 * call qkv holds roped q and k and the plain v; k/v of rows with slot >= 0
 * are in the cache (bf16 [slots, Hkv, D], or e4m3 codes with per-(token,
 * head) scales).  Sizes and the error behaviour are those of the separate
 * ops (D in {64, 80, 128}; an out-of-range position is reported through
 * biv_poll_error and read as 0); BIV_ERR_INVALID also on partials with
 * more than 8 chunks. */
biv_status biv_qkv_finalize(uint16_t* qkv, int64_t row_stride, const biv_partials* qkv_partials,
                            int T, int Hq, int Hkv, int D, const uint16_t* q_w, const uint16_t* k_w,
                            const float* cos_sin, int max_pos, const int32_t* pos, float eps,
                            const int64_t* slot, int kv_dtype, void* k_cache, void* v_cache,
                            float* k_scale, float* v_scale, biv_stream_t stream);

/* Gather + dequantise: for each sequence i, tokens [0, ctx_len[i]) of its
 * pages (block_table int32 [nseq, max_pages]) are written as
 * bf16(float(code) * s) to out bf16 [sum ctx, Hkv, D] starting at row
 * out_row0[i] (int64 [nseq]).  Same formula as the attention loader. */
biv_status biv_kv_fp8_gather(const uint8_t* codes, const float* scales,
                             const int32_t* block_table, int max_pages, const int32_t* ctx_len,
                             const int64_t* out_row0, int nseq, int Hkv, int D, int page,
                             uint16_t* out, biv_stream_t stream);

/* ----------------------------------------------------------- attention --
 * One paged GQA attention kernel for prefill, chunked prefill and decode rows
 * ("Finish RL Training Faster", section "让训练前向使用推理的数值": every path
 * gathers, dequantises and enters the same attention operator).
 * Row t (a token of sequence row_seq[t] at absolute position row_pos[t])
 * attends to keys at positions <= row_pos[t] of its sequence, read from the
 * paged cache through block_table.  Keys are visited in 64-token tiles aligned
 * to absolute positions, grouped into splits of kv_split tokens (a model
 * constant); each split keeps an online softmax (FP32), P enters P.V as
 * three bf16 parts hi + mid + lo that add up to the FP32 p exactly, and the
 * splits are merged in ascending order in FP32.  With topk_idx != NULL (sparse attention) the
 * keys of row t are the positions topk_idx[t, 0..topk) (ascending, -1 =
 * none) and splits run over that list.
 * qblocks int32 [nqblocks, 2] = (first row, row count): rows of a block must
 * belong to one sequence (sparse: one row per block).  The grouping into
 * blocks does not change any result bit.  Output bf16 [T, Hq, D]. */
typedef struct {
  const uint16_t* q;        /* [T, Hq, D] rows at q + t*q_stride */
  int64_t q_stride;
  uint16_t* out;            /* [T, Hq, D] rows at out + t*out_stride */
  int64_t out_stride;
  int T, Hq, Hkv, D;        /* D in {64, 80, 128}; Hq % Hkv == 0 */
  const int32_t* row_seq;   /* [T] */
  const int32_t* row_pos;   /* [T] */
  const int32_t* qblocks;   /* [nqblocks, 2] */
  int nqblocks;
  int max_rows_per_block;   /* host bound on the row count of any block */
  int kv_dtype;             /* BIV_BF16 or BIV_E4M3 */
  const void* k_cache;      /* [pages, page, Hkv, D] bf16 or e4m3 */
  const void* v_cache;
  const float* k_scale;     /* [pages, page, Hkv] (E4M3 only) */
  const float* v_scale;
  const int32_t* block_table; /* [nseq, max_pages]: page indices, 0 <= page < 2^31 / 64
                                 (the thread loader raises the device error word on a
                                 negative or larger entry, reads zeros for that page's
                                 keys and leaves the outputs that see them undefined) */
  int max_pages;
  int page;                 /* must be 64 */
  int kv_split;             /* tokens per split, multiple of 64 (INVARIANT: model constant) */
  int max_ctx;              /* host bound: max over rows of row_pos+1 (dense) */
  const int32_t* topk_idx;  /* optional [T, topk] */
  int64_t topk_stride;
  int topk;
  float scale;              /* softmax scale, usually 1/sqrt(D) */
  int mode;                 /* biv_mode; FAST picks kv_split from the batch */
  int num_pages;            /* pages the cache arrays hold (bf16 caches: lets the
                               kernel fetch whole pages by TMA); 0 = unknown */
} biv_attn_desc;

biv_status biv_attention_workspace(const biv_attn_desc* desc, size_t* bytes);
biv_status biv_attention(const biv_attn_desc* desc, void* workspace, size_t workspace_bytes,
                         biv_stream_t stream);

/* Allocation-free variant of biv_attention (the paper has no counterpart: it
 * exists for callers that cannot call cudaMalloc, e.g. code running inside
 * another runtime's memory budget or a hook that must not allocate).  Same
 * arguments and results as biv_attention, but the split partials go to a
 * fixed 64 MiB device array inside the library instead of a caller
 * workspace.  Every GPU that loads the library holds that array until the
 * process exits.  The first call in a CUDA context looks the array's address
 * up (with that context's device current) and caches it for that context;
 * make that first call before any stream capture, and again after a device
 * reset (a new context gets a fresh lookup on its first call).  A call whose scratch need (biv_attention_workspace)
 * exceeds 64 MiB returns BIV_ERR_WORKSPACE and launches nothing.  All calls
 * share the one array: calls whose work can overlap on the GPU (different
 * streams, no ordering between them) race and must not be issued.  Nothing
 * in the array needs to start at zero. */
biv_status biv_attention_noalloc(const biv_attn_desc* desc, biv_stream_t stream);

/* ---------------------------------------------------------------- GEMM --
 * C[M, N] = A[M, K] . B[N, K]^T on the tcgen05 tensor cores, FP32
 * accumulation in TMEM ("Finish RL Training Faster", section
 * "让训练前向使用推理的数值": one batch-invariant GEMM schedule with a fixed K
 * split).  A and B are K-major (row-major with K contiguous).  INVARIANT
 * mode, whatever M is:
 *  - bf16 x bf16 -> bf16 or f32 (c_dtype): with KB = ceil(K/64), K is cut
 *    into chunks of max(8, ceil(KB/8)) blocks of 64 (at most 8 chunks, the
 *    last may be shorter); each chunk P_c is accumulated in FP32 from zero in
 *    ascending K steps of 16; the output is the left fold r = P_0,
 *    r = r + P_1, ... in FP32, rounded once to c_dtype.
 *  - e4m3 x e4m3 -> bf16 with block scales: per 128-wide K block kb,
 *    acc += (sa[m,kb]*sb[g][n/128,kb]) * (FP8 products summed over the
 *    block), promoted to FP32 every block, blocks in ascending order.
 * Grouped (MoE) when groups > 1: rows [off[g], off[g+1]) of A use weight
 * group g (B rows g*N .. g*N+N-1, sb + g*ceil(N/128)*ceil(K/128)).
 * K % 8 == 0 (bf16) / K % 16 == 0 (e4m3); lda, ldb keep rows 16-byte
 * aligned; ldc keeps rows 16-byte aligned for vector stores.
 * FAST mode (bf16): no K chunks when M fills the GPU, a K split sized to the
 * GPU when it does not (results depend on M; the comparator).
 * Workspace (bf16, when biv_gemm_workspace reports > 0: few output tiles,
 * where the chunks of one tile run on different SMs and a second kernel
 * folds them): device memory, 16-byte aligned, owned by the caller, no
 * initial value needed.  Calls that can overlap on the GPU need separate
 * workspaces.
 * Returns BIV_ERR_WORKSPACE when the workspace is missing or too small. */
typedef struct {
  int M, N, K;
  int a_dtype, b_dtype, c_dtype;
  const void* A; int64_t lda;
  const void* B; int64_t ldb;
  void* C; int64_t ldc;
  const float* sa; int64_t ld_sa;   /* FP8: [M, ld_sa >= ceil(K/128)] */
  const float* sb;                  /* FP8: [groups, ceil(N/128), ceil(K/128)] */
  const int32_t* group_offsets;     /* optional device [groups+1] */
  int groups;                       /* 0/1 = plain */
  int mode;                         /* biv_mode */
  int defer_fold;                   /* 1: when the call leaves chunk partials in the
                                       workspace (biv_gemm_partials says so), skip the
                                       fold: a consumer op reads them; C is not written */
  int b_early;                      /* bf16.  0: B may be the output of the call just before.
                                       1: the first tiles of B are loaded while calls ahead in
                                       the stream may still run (a decode step of 64 sequences
                                       through 28 layers: 2.39 ms, without 2.45).  Only for a B
                                       with another call of this library between its last
                                       writer and this call, one that launches work and is no
                                       GEMM (those let their successor start before they have
                                       waited themselves): the weights of a forward that begins
                                       with biv_embed, say */
} biv_gemm_desc;

/* Fills *out with the partials layout of a call (chunks = 0 when the plan
 * folds inside the GEMM).  Pure host computation, no launch. */
biv_status biv_gemm_partials(const biv_gemm_desc* desc, const void* workspace, biv_partials* out);

biv_status biv_gemm_workspace(const biv_gemm_desc* desc, size_t* bytes);
biv_status biv_gemm(const biv_gemm_desc* desc, void* workspace, size_t workspace_bytes,
                    biv_stream_t stream);

/* Per-token activation quantisation for the FP8 GEMM: groups of 128 along K,
 * s = amax/448 (1 when amax = 0), code = e4m3_rne_satfinite(x/s).
 * x bf16 [rows, K]; codes uint8 [rows, K] (row stride K); scales float32
 * [rows, ceil(K/128)].  K % 16 == 0. */
biv_status biv_act_quant_fp8(const uint16_t* x, int64_t x_stride, int rows, int K,
                             uint8_t* codes, float* scales, biv_stream_t stream);

/* biv_silu_mul followed by biv_act_quant_fp8 of its result, in one pass:
 * gate_up = [g | u] bf16 [rows, 2I] (row stride gu_stride >= 2I); codes
 * uint8 [rows, I] and scales float32 [rows, ceil(I/128)] are bit for bit what
 * the two calls write (the bf16 activation is not stored).  I % 16 == 0. */
biv_status biv_silu_mul_quant_fp8(const uint16_t* gate_up, int64_t gu_stride, int rows, int I,
                                  uint8_t* codes, float* scales, biv_stream_t stream);

/* -------------------------------------------------------------- Top-K ---
 * Sparse-attention selection ("Finish RL Training Faster", section
 * "让训练前向使用推理的数值": fixed tie-break and fixed position order): per row
 * r, among indices j < valid_len[r] with scores[r, j] > -inf, the k largest
 * scores, equal scores resolved toward the LOWER index; the chosen indices
 * are written to idx int32 [rows, k] in ASCENDING index order, padded with
 * -1.  -0.0 and +0.0 compare equal; a NaN score is never chosen.
 * 0 < k <= n <= 32768, ld >= n. */
biv_status biv_topk(const float* scores, int64_t ld, const int32_t* valid_len, int rows, int n,
                    int k, int32_t* idx, biv_stream_t stream);

/* MoE router: per row, the k largest of E logits (ties -> lower expert id),
 * written in rank order (logit descending, id ascending) to idx int32
 * [rows, k]; w float32 [rows, k] = softmax probability of each chosen expert
 * over all E (not renormalised).  E <= 1024, k <= 32. */
biv_status biv_router_topk(const float* logits, int64_t ld, int rows, int E, int k, int32_t* idx,
                           float* w, biv_stream_t stream);

/* Deterministic dispatch: experts idx int32 [T, k] -> offsets int32 [E+1]
 * (rows of expert e = [offsets[e], offsets[e+1])) and perm int32 [T*k]
 * (entry t*k+s of expert e placed at offsets[e] + rank of (t, s) among that
 * expert's entries in ascending (t, s) order); src_row int32 [T, k] is the
 * inverse (row of entry (t, s) in the grouped layout).  T*k <= 1<<20. */
biv_status biv_moe_dispatch(const int32_t* idx, int T, int k, int E, int32_t* offsets,
                            int32_t* perm, int32_t* src_row, biv_stream_t stream);

/* Row gather for grouped GEMM inputs: dst[i, :] = src[perm[i] / k_div, :] for
 * byte rows of `row_bytes` (multiple of 16), i < n. */
biv_status biv_gather_rows(const void* src, int64_t src_stride_bytes, const int32_t* perm,
                           int k_div, int n, int row_bytes, void* dst, int64_t dst_stride_bytes,
                           biv_stream_t stream);

/* FP32 fixed-slot combine ("Finish RL Training Faster", section
 * "让训练前向使用推理的数值": expert outputs merged in FP32 in slot order):
 * out[t] = bf16( sum_{s=0..k-1, in order} w[t,s]*float(y_row(t,s)) + float(shared[t]) )
 * with y_row(t,s) = y[src_row[t*k+s]] when src_row != NULL, else y[t*k+s];
 * y bf16 [*, d], shared bf16 [T, d] or NULL, out bf16 [T, d]. */
biv_status biv_moe_combine(const uint16_t* y, const int32_t* src_row, const float* w,
                           const uint16_t* shared, uint16_t* out, int T, int k, int d,
                           biv_stream_t stream);

/* ------------------------------------------------------------ log-prob --
 * lp[t] = z[t, target[t]] - (m + log sum_v exp(z[t, v] - m)), m = max_v z,
 * in FP32 with a reduction order that depends on V only (the logprob of
 * every sampled token, "Finish RL Training Faster", section
 * "零差异需要一个精确的比较对象").  logits float32 [T, V] rows at ld. */
biv_status biv_logprob(const float* logits, int64_t ld, const int32_t* target, int T, int V,
                       float* lp, biv_stream_t stream);

/* LM head with the log-softmax gather in its epilogue: lp[t] = z[t, target[t]]
 * - logsumexp_v z[t, v] for z = h . W^T, without writing the FP32 logits
 * (same source as biv_logprob).  The GEMM is biv_gemm's bf16 schedule (K
 * chunks in INVARIANT mode), folded in the CTA on 256-column tiles for every
 * M.  Its epilogue reduces each row's logits in groups of 128 columns
 * (group g = columns [128g, 128g+128) of V) to m_g = max z and
 * s_g = sum exp(z - m_g), summed as four interleaved chains (column mod 4,
 * ascending) added as (c0 + c1) + (c2 + c3); a second kernel forms
 * M = max_g m_g and S = sum_g s_g * exp(m_g - M) (lane l of a warp takes
 * groups l, l+32, ... in order, then a xor tree) and lp = z_t - (M + log S).
 * Every step depends on V and the row only, so a row's lp has the same bits
 * in every batch.
 * h bf16 [M, K] rows at ldh; W bf16 [V, K] rows at ldw (K-major, 16-byte
 * aligned rows); target int32 [M]; lp float32 [M].  V % 4 == 0, K % 8 == 0.
 * A target outside [0, V) gives lp = NaN and the device error code 2.
 * Workspace: device memory of biv_lm_head_logprob_workspace(M, V) bytes,
 * 16-byte aligned, owned by the caller, no initial value needed; calls that
 * can overlap on the GPU need separate workspaces. */
biv_status biv_lm_head_logprob_workspace(int M, int V, size_t* bytes);
biv_status biv_lm_head_logprob(const uint16_t* h, int64_t ldh, const uint16_t* W, int64_t ldw,
                               int M, int V, int K, const int32_t* target, int mode, float* lp,
                               void* workspace, size_t workspace_bytes, biv_stream_t stream);

/* ------------------------------------------------------------- SSD scan --
 * Mamba-2 SSD over chunks of `chunk` positions aligned to absolute positions
 * ("Finish RL Training Faster", section "一致性有多个层面": decode replays the
 * prefill chunk order).  For each sequence i, rows [row0[i], row0[i]+n[i])
 * of x/dt/B/C are its next n[i] tokens, starting at absolute position pos0[i].
 * Per sequence the library keeps, in caller memory:
 *   state  float32 [nseq, H, P, N]: the state at the start of the open chunk;
 *   buf_x  bf16 [nseq, chunk, H, P], buf_B/buf_C bf16 [nseq, chunk, N],
 *   buf_dt float32 [nseq, chunk, H]: the open chunk's rows so far.
 * Every output row y_t is computed from its chunk's start state and the
 * chunk's rows <= t with one code path, so prefill, chunked prefill and
 * token-by-token decode give the same bits.  When a chunk closes its end
 * state replaces `state`.  Set state to zero for a new sequence (pos0 = 0).
 * H*P, N: P in {64}, N in {128}; chunk in {64, 128, 256}. */
typedef struct {
  const uint16_t* x; int64_t x_stride;   /* [rows, H, P] */
  const float* dt;   int64_t dt_stride;  /* [rows, H] (after softplus) */
  const float* A;                        /* [H], negative */
  const uint16_t* B; int64_t B_stride;   /* [rows, N] */
  const uint16_t* C; int64_t C_stride;   /* [rows, N] */
  const float* D;                        /* [H] */
  uint16_t* y; int64_t y_stride;         /* [rows, H, P] */
  int H, P, N, chunk;
  int nseq;
  const int32_t* row0;                   /* [nseq] */
  const int32_t* n;                      /* [nseq] */
  const int32_t* pos0;                   /* [nseq] */
  int max_n;                             /* host bound on n[i] */
  float* state;
  uint16_t* buf_x;
  uint16_t* buf_B;
  uint16_t* buf_C;
  float* buf_dt;
  void* workspace;                       /* optional, biv_ssd_workspace bytes, 16-byte aligned */
  size_t workspace_bytes;
} biv_ssd_desc;

/* Workspace of the parallel path (0 when no sequence has more than 4 new rows,
 * where one CTA per (sequence, head) runs the chunk).  With a large enough
 * workspace a call with many new rows runs every (sequence, chunk, head) in
 * parallel and hands states on chunk to chunk; without one it runs the
 * per-(sequence, head) path.  Both evaluate every row with the same FP32
 * operations in the same order, so the choice changes no bit.  The workspace
 * needs no initial value. */
biv_status biv_ssd_workspace(const biv_ssd_desc* desc, size_t* bytes);
biv_status biv_ssd_scan(const biv_ssd_desc* desc, biv_stream_t stream);

/* ------------------------------------------------- Mamba-2 mixer steps --
 * The steps of a Mamba-2 layer around biv_ssd_scan ("Finish RL Training
 * Faster", section "两组结果，要连同分母一起读": the Mamba-2 hybrid; section
 * "一致性有多个层面": decode replays the prefill order bit for bit).
 *
 * biv_causal_conv1d: depthwise causal convolution of width 4 over the
 * `channels` xBC columns of the in-projection output u (columns col_x ..),
 * then SiLU, rounded to bf16 into out [T, channels]:
 *   out[t, c] = bf16(silu(acc)), acc = b[c]; acc = acc + w[c, j] * x[t-3+j, c]
 *   for j = 0..3 in FP32, product and sum each rounded (no fma);
 * and, over the `heads` dt columns (col_dt ..), dt_out[t, h] =
 * softplus(dt_raw + dt_bias[h]) in FP32 (x > 20 gives x).  Rows of sequence
 * i (0 <= i < nseq) are rows row0[i] .. row0[i]+n[i]-1 of this call, at
 * consecutive positions from pos0[i]; row_seq / row_pos give each row's i
 * and position.  Inputs before a sequence's first row in the call come from
 * state [nseq, 3, channels] bf16 (the three inputs that preceded it; zero for
 * a new sequence, pos0 = 0), so prefill, chunked prefill and decode give the
 * same bits.  After the call state[i] holds the last three inputs of every
 * sequence with n[i] > 0.  conv_w bf16 [channels, 4], conv_b bf16
 * [channels], dt_bias fp32 [heads].  channels and heads multiples of 8;
 * u, out rows and state 16-byte aligned.  A row whose (row_seq, row_pos) is
 * not one of its sequence's rows is reported through biv_poll_error and
 * written as zeros. */
typedef struct {
  const uint16_t* u; int64_t u_stride;
  int col_x, col_dt, channels, heads, width;   /* width must be 4 */
  const uint16_t* conv_w; const uint16_t* conv_b; const float* dt_bias;
  uint16_t* out; int64_t out_stride;
  float* dt_out; int64_t dt_stride;
  int T;
  const int32_t* row_seq; const int32_t* row_pos;
  int nseq;
  const int32_t* row0; const int32_t* n; const int32_t* pos0;
  uint16_t* state;
} biv_conv_desc;
biv_status biv_causal_conv1d(const biv_conv_desc* desc, biv_stream_t stream);

/* Gated RMSNorm of the Mamba-2 output: g = y * silu(z) in FP32 (not
 * rounded), out = bf16((g * inv) * w), inv = 1/sqrt(mean(g^2) + eps), the
 * same per-row reduction tree as biv_add_rmsnorm.  y, z, out bf16 rows of d
 * (d a multiple of 8, at most 8192), w bf16 [d]. */
biv_status biv_gated_rmsnorm(const uint16_t* y, int64_t y_stride, const uint16_t* z,
                             int64_t z_stride, const uint16_t* w, uint16_t* out,
                             int64_t out_stride, int rows, int d, float eps, biv_stream_t stream);

/* NVFP4 weights to bf16 ("Finish RL Training Faster", section
 * "两组结果，要连同分母一起读": NVFP4 weights): out[n, k] = e2m1(code[n, k])
 * * e4m3(scales[n, k/16]), global scale 1.  codes uint8 [N, K/2] packed two
 * per byte (element 2i in the low nibble of byte i), scales uint8 [N, K/16]
 * (e4m3), out bf16 [N, K]; the product is exact in bf16.  K a multiple of
 * 16, codes and out 16-byte aligned. */
biv_status biv_nvfp4_dequant(const uint8_t* codes, const uint8_t* scales, int N, int K,
                             uint16_t* out, biv_stream_t stream);

/* GEMM with NVFP4 weights (W4A16): C[M, N] = A[M, K] . W^T with W = the
 * biv_nvfp4_dequant of (codes, scales), every output bit equal to biv_gemm
 * on that bf16 W (same K-chunk schedule, same tcgen05 MMAs; "Finish RL
 * Training Faster", section "两组结果，要连同分母一起读": NVFP4 weights, and
 * section "让训练前向使用推理的数值": one schedule for every batch).  When
 * the bf16 plan would spread a few output tiles' K chunks over the SMs
 * (decode-sized M), the kernel streams the packed codes and scales by TMA
 * and decodes them in shared memory: 0.5625 bytes of HBM per weight instead
 * of 2 (K a multiple of 256).  Otherwise (many rows: compute-bound; or
 * another K) the weights are decoded once into the workspace and the bf16
 * GEMM runs.  A bf16 [M, K] row-major
 * (lda >= K); codes/scales as for biv_nvfp4_dequant; C bf16 or f32 (c_dtype)
 * [M, ldc].  K a multiple of 16; every pointer 16-byte aligned.  Workspace:
 * biv_gemm_nvfp4_workspace bytes (0 possible), caller-owned, 16-byte
 * aligned, no initial value; BIV_ERR_WORKSPACE when missing or too small. */
biv_status biv_gemm_nvfp4_workspace(int M, int N, int K, int c_dtype, int mode, size_t* bytes);
biv_status biv_gemm_nvfp4(const uint16_t* A, int64_t lda, const uint8_t* codes,
                          const uint8_t* scales, int M, int N, int K, void* C, int64_t ldc,
                          int c_dtype, int mode, void* workspace, size_t workspace_bytes,
                          biv_stream_t stream);

/* ------------------------------------------------------------ backward --
 * Backward of the fused forward ops for a trainer that runs the inference
 * ops' own backward ("No More Train-Inference Mismatch", section "方法细节"),
 * the FP8 KV round trip passing gradients straight through ("Finish RL
 * Training Faster", section "让训练前向使用推理的数值").  FP32 on the CUDA
 * cores; every reduction has one order fixed by the shapes (per-row trees,
 * ascending loops), so results repeat bit for bit, and a row's dx / dz / dq
 * depends on that row (and, for dq, its keys) only.
 *
 * RMSNorm of x (bf16 rows of d, gain w bf16 [d]): dy, dx float32 rows;
 * dx = inv*(w*dy) - x*(inv^3*sum(x*w*dy)/d), inv = 1/sqrt(mean(x^2)+eps);
 * dw float32 [d] = sum over rows in ascending order of dy*x*inv.  Workspace:
 * rows*d*4 bytes (caller-owned, no initial value). */
biv_status biv_rmsnorm_backward(const uint16_t* x, int64_t x_stride, const uint16_t* w,
                                const float* dy, int64_t dy_stride, float* dx, int64_t dx_stride,
                                float* dw, int rows, int d, float eps, void* workspace,
                                size_t workspace_bytes, biv_stream_t stream);

/* SiLU-mul: gate_up bf16 [rows, 2I] ([gate | up]), dy float32 [rows, I] ->
 * dgate_up float32 [rows, 2I]: dgate = dy*up*s*(1+gate*(1-s)), dup =
 * dy*gate*s, s = 1/(1+exp(-gate)). */
biv_status biv_silu_mul_backward(const uint16_t* gate_up, int64_t gate_up_stride, const float* dy,
                                 int64_t dy_stride, float* dgate_up, int64_t dgate_up_stride,
                                 int rows, int I, biv_stream_t stream);

/* logprob: logits float32 [T, V] (ld), target int32 [T], dlp float32 [T] ->
 * dz float32 [T, V] (ldz) = dlp*(onehot(target) - exp(z - lse)); lse from a
 * per-row max and sum in a fixed order.  A target outside [0, V) is reported
 * through biv_poll_error. */
biv_status biv_logprob_backward(const float* logits, int64_t ld, const int32_t* target,
                                const float* dlp, int T, int V, float* dz, int64_t ldz,
                                biv_stream_t stream);

/* Causal GQA attention of one sequence: q, dout bf16 [Tq, Hq, D]; k, v bf16
 * [Tk, Hkv, D] (the cache's dequantised values: an FP8 round trip passes dk,
 * dv through unchanged); key j is visible to row i iff k_pos[j] <= q_pos[i].
 * dq float32 [Tq, Hq, D], dk, dv float32 [Tk, Hkv, D]: with p = softmax(s),
 * s = q.k*scale, D_i = dout_i . o_i, ds = p*(dout.v - D): dq = sum_j ds k
 * scale (keys ascending), dk = sum ds q scale and dv = sum p dout (rows
 * ascending, q heads of the group ascending).  D <= 128.  workspace float32
 * [2*Tq*Hq] (row statistics, no initial value). */
typedef struct {
  const uint16_t* q; const uint16_t* k; const uint16_t* v; const uint16_t* dout;
  float* dq; float* dk; float* dv;
  int Tq, Tk, Hq, Hkv, D;
  const int32_t* q_pos; const int32_t* k_pos;
  float scale;
  float* workspace;
} biv_attn_bwd_desc;
biv_status biv_attention_backward(const biv_attn_bwd_desc* desc, biv_stream_t stream);

/* --------------------------------------------------------- policy loss --
 * The trainer's loss on the recomputed logprobs ("No More Train-Inference
 * Mismatch", section "方法细节": the trainer's forward and backward around the
 * imported ops; GRPO without importance correction, "Finish RL Training
 * Faster", section "两组结果，要连同分母一起读"): a clipped policy loss with a KL
 * term, and its gradient in the same call.
 *
 * Rows t = 0..T-1 are tokens; sequence s holds rows [seq_start[s],
 * seq_start[s+1]).  A row counts when it lies in a sequence and its mask byte
 * is not 0.  With A the advantage (of the row or of its sequence), x clamped
 * to [-20, 20] written clamp(x):
 *   r  = exp(clamp(lp - old_lp)),  u = -A r,  c = -A min(max(r, 1-clip_lo), 1+clip_hi)
 *   pg = max(u, c);  dual_clip > 0 and A < 0:  pg = min(pg, -A dual_clip)
 *   e  = clamp(ref_lp - lp),  kl = exp(e) - e - 1   (the k3 estimator)
 *   loss = sum_t w_t (pg + kl_coef kl - ent_coef H)
 *   dlp  = w ((u is taken ? u : 0) + kl_coef (1 - exp(e)))
 * where u is taken when u >= c, the dual bound does not act and |lp - old_lp|
 * < 20, and the KL part is 0 at |ref_lp - lp| >= 20 (the clamps' derivative); u's
 * part is 0 at lp = -inf too, where no old_lp stands beside it.
 * w_t by `reduce`: TOKEN_MEAN 1/N, N counted rows; SEQ_MEAN 1/(S n_s), S
 * sequences that have counted rows, n_s their number; SUM 1/norm.
 * A row that does not count has weight 0: what its lp, logits and target hold
 * does not matter, and its dlp, lp, entropy and dz are written as zeros; with no counted
 * row at all (T = 0 too) loss, statistics and gradients are zeros.
 *
 * stats float32 [8]: loss, sum w pg, sum w kl, sum w H, then over counted rows
 * the share where u is not taken by clipping, mean of exp(d) - 1 - d (d =
 * clamp(lp - old_lp)), max |lp - old_lp|, and their number.  Blocks of 1024
 * rows are summed in one fixed order, blocks ascending (32 lanes, then a xor
 * tree): every call repeats its bits, and a row's gradient depends on that row
 * and its weight only.
 * seq_start outside [0, T] or not ascending is reported through
 * biv_poll_error (results are then unspecified; no access leaves [0, T)).
 * Outputs must not overlap inputs (dz over the logits excepted, see below).
 * Workspace: biv_policy_loss_workspace bytes, 16-byte aligned, caller-owned,
 * no initial value; calls that can overlap on the GPU need separate ones. */
typedef enum { BIV_LOSS_TOKEN_MEAN = 0, BIV_LOSS_SEQ_MEAN = 1, BIV_LOSS_SUM = 2 } biv_loss_reduce;
typedef struct {
  int T, nseq;
  const int32_t* seq_start;  /* [nseq + 1], ascending, within [0, T] */
  const uint8_t* mask;       /* [T]; NULL: every row of a sequence counts */
  const float* old_lp;       /* [T] logprobs of the policy that sampled; NULL: lp itself (r = 1) */
  const float* ref_lp;       /* [T] reference logprobs; may be NULL when kl_coef is 0 */
  const float* adv;          /* [T] when adv_per_row, else [nseq] (NULL when nseq is 0) */
  int adv_per_row;
  float clip_lo, clip_hi;    /* 0 <= clip_lo <= 1, 0 <= clip_hi */
  float dual_clip;           /* 0: off; else > 1 */
  float kl_coef, ent_coef;   /* in [-1000, 1000] */
  int reduce;                /* biv_loss_reduce */
  float norm;                /* SUM only: > 0 */
  float* stats;              /* [8] */
  void* workspace;
  size_t workspace_bytes;
} biv_policy_desc;
biv_status biv_policy_loss_workspace(int T, int nseq, size_t* bytes);

/* From per-token logprobs (biv_lm_head_logprob's or biv_logprob's output):
 * lp float32 [T] -> dlp float32 [T] (NULL: statistics only), ready for
 * biv_logprob_backward.  ent_coef must be 0 (the entropy needs the logits). */
biv_status biv_policy_loss(const biv_policy_desc* desc, const float* lp, float* dlp,
                           biv_stream_t stream);

/* From the logits, in one pass over them: z [T, V] rows at ld (z_dtype
 * BIV_F32 or BIV_BF16), x = z inv_temp, target int32 [T]:
 *   lp = x[target] - lse, p = exp(x - lse), H = lse - sum_v p_v x_v
 *   dz_v = inv_temp (dlp ([v = target] - p_v) + w ent_coef p_v (log p_v + H))
 * lp, entropy float32 [T]; dz [T, V] rows at ldz (dz_dtype BIV_F32 or
 * BIV_BF16, one rounding; NULL: no gradient).  dz may be z itself (same
 * pointer, type and stride), and must not overlap it otherwise.  A logit of
 * -1e30 or less (-inf, a type's lowest value) is masked: p = 0 and dz = 0; a
 * row of masked logits alone gives NaN, as a NaN or +inf among them does; where
 * the target is masked, dlp is 0 (its lp is -inf, or the low value's).  A counted
 * row whose target is outside [0, V) gives lp = NaN and the device error code
 * 2; other rows' results and what lies around dz stay as they are.
 * Each row's bits depend on V and the row only: 4 KB groups of logits are
 * reduced to (max, sum, entropy sum) by one warp and merged in one order,
 * however the row is spread over CTAs.  They are not the bits of
 * biv_lm_head_logprob or biv_logprob, whose sums run in another order: lp
 * agrees with theirs to rounding, so with a rollout's logprobs as old_lp the
 * ratio of an unchanged policy is 1 to rounding only and the gap's statistics
 * are not exactly 0.  Where they have to be, take biv_policy_loss on the recompute's
 * own lp, then biv_logprob_backward; or old_lp from this call.
 * 1 <= V <= 262144, 0.01 <= inv_temp <= 100.  Rows that keep 16 bytes'
 * alignment load and store fastest; any element alignment works. */
biv_status biv_policy_loss_logits(const biv_policy_desc* desc, const void* z, int64_t ld,
                                  int z_dtype, const int32_t* target, int V, float inv_temp,
                                  float* lp, float* entropy, void* dz, int64_t ldz, int dz_dtype,
                                  biv_stream_t stream);

/* ------------------------------------------- cross entropy of the LM head --
 * The trainer's loss and gradient at the LM head without the [T, V] logits ("No
 * More Train-Inference Mismatch", section "方法细节": the trainer's forward and
 * backward around the imported ops).  h bf16 [T, K] rows at ldh, W bf16 [V, K]
 * rows at ldw (16-byte aligned rows, K % 8 == 0), target int32 [T], any V >= 1.
 *
 * biv_lm_head_loss: z = h . W^T as in biv_lm_head_logprob,
 *   lse = logsumexp_v z_v,  lp = z[target] - lse     (lp has biv_lm_head_logprob's bits)
 *   c_t = weight_t / N (TOKEN_MEAN, N the sum of the counted rows' weights) or weight_t / norm (SUM)
 *   loss = sum_t c_t (-lp_t + z_coef lse_t^2)
 * A row whose target is ignore_index or whose weight is 0 does not count: its
 * lp, lse, dlp and dlse are written as zeros, whatever its h holds; weight NULL:
 * all weights are 1; without a counted row loss and statistics are zeros.  A
 * counted row with another target outside [0, V) gives lp = NaN and the device
 * error code 2.  Outputs: lp, lse float32 [T]; dlp = dloss/dlp = -c and dlse =
 * dloss/dlse = 2 z_coef c lse float32 [T] (each may be NULL), ready for
 * biv_lm_head_backward; stats float32 [4]: loss, sum c nll, sum c lse^2, N.
 * A row's bits depend on the row, W and N only; the sums run in one order fixed
 * by T.  The logits' accumulators truncate, as biv_lm_head_logprob's do: a bias that
 * a mean over rows keeps (the loss of 4096 x 151936 x 2048 is off by 3.6e-7 of
 * itself).  Workspace: biv_lm_head_loss_workspace bytes, 16-byte aligned,
 * caller-owned, no initial value; calls that can overlap on the GPU need
 * separate ones. */
typedef struct {
  int T, V, K;
  const uint16_t* h; int64_t ldh;
  const uint16_t* W; int64_t ldw;
  const int32_t* target;
  const float* weight;       /* [T] or NULL */
  int ignore_index;          /* usually -100 */
  float z_coef;              /* in [0, 1000] */
  int reduce;                /* BIV_LOSS_TOKEN_MEAN or BIV_LOSS_SUM */
  float norm;                /* SUM only: > 0 */
  float* lp; float* lse;     /* [T] */
  float* dlp; float* dlse;   /* [T] or NULL */
  float* stats;              /* [4] */
  void* workspace;
  size_t workspace_bytes;
} biv_lm_loss_desc;
biv_status biv_lm_head_loss_workspace(int T, int V, size_t* bytes);
biv_status biv_lm_head_loss(const biv_lm_loss_desc* desc, biv_stream_t stream);

/* Gradient of any loss of lp and lse (biv_lm_head_loss, or biv_policy_loss's dlp):
 * with p = exp(h . W^T - lse),
 *   dz = dlp ([v = target] - p) + dlse p,   dh = dz . W,   dW = dz^T . h (or dW += it).
 * lse as the forward wrote it; dlse may be NULL.  A row with dlp = dlse = 0 has
 * no gradient: its dh is written as zeros, and what its h, lse and target hold
 * does not matter; it costs no products.  A row with another target outside
 * [0, V) is treated the same and raises the device error code 2.
 * dh [T, K] rows at lddh, dW [V, K] rows at lddw, each BIV_BF16 or BIV_F32, each
 * may be NULL; they must not overlap the inputs or each other.  accumulate = 1
 * adds to dW what it holds (in FP32, one rounding).
 * The logits are formed again in chunks of at most 8192 columns and never stored;
 * dz of a few chunks is, in the workspace.  dz enters the products as bf16, for a
 * FP32 gradient as two bf16 parts, which leave 2.7e-6 of the p terms in the mean
 * square; accumulators of 768 K elements are then off by about 1e-6 of a sum.  The
 * term of a row's own target is added in FP32.  dh is the sum of its chunks' FP32
 * products in ascending order: a row's dh depends on the row, V, K and the
 * gradients' types only.  dW adds the p terms of the counted rows in ascending
 * order, then those of the rows whose target a row of W is, in an order fixed by
 * the targets.  Every call repeats its bits.
 * T <= 2^20, V < 2^24, K <= 65536.  Workspace: biv_lm_head_backward_workspace
 * bytes (the sizes and gradient types of the call), 256-byte aligned,
 * caller-owned, no initial value.  With T' and K' = T and K rounded up to 256 it
 * is at most the sum of
 *   dz: 192 MiB, or 48 KiB T' (three chunks) where that is more, but no more than
 *     dz of all chunks; with a FP32 gradient twice as much
 *   sums of dh: 192 MiB, or 4 T' K' where that is more
 *   rows: T' (3 K' + 64) + 1 MiB.
 * That is far below the T x V FP32 logits of a trainer's micro-batch (4096 x
 * 151936 x 2048: 245 of 2,374 MiB), but may be above those of few rows (200 x
 * 151936 x 2048: 99 of 116 MiB, 13 x 151936 x 256: 86 of 7.5).  Calls that can
 * overlap on the GPU need separate ones. */
typedef struct {
  int T, V, K;
  const uint16_t* h; int64_t ldh;
  const uint16_t* W; int64_t ldw;
  const int32_t* target;
  const float* lse;
  const float* dlp;
  const float* dlse;         /* [T] or NULL */
  void* dh; int64_t lddh; int dh_dtype;
  void* dW; int64_t lddw; int dw_dtype;
  int accumulate;
  void* workspace;
  size_t workspace_bytes;
} biv_lm_grad_desc;
biv_status biv_lm_head_backward_workspace(int T, int V, int K, int dh_dtype, int dw_dtype,
                                          size_t* bytes);
biv_status biv_lm_head_backward(const biv_lm_grad_desc* desc, biv_stream_t stream);

/* ------------------------------------------------- activations in 8 bits --
 * What a trainer holds between its forward and its backward, in 8 bits ("No
 * More Train-Inference Mismatch", section "方法细节": fused RMSNorm with residual
 * and SiLU MLP, and their backward).  A row is quantised as by biv_act_quant_fp8
 * ("Finish RL Training Faster", section "让训练前向使用推理的数值": one quantisation
 * rule): per 128 consecutive elements s = amax / 448 (1 when amax is 0), code =
 * e4m3_rne_satfinite(v / s); codes uint8 rows without gaps, scales float32
 * [rows, ceil(width / 128)].  16-byte aligned rows; d and I multiples of 16.
 *
 * biv_add_rmsnorm_fp8: biv_add_rmsnorm with 8-bit outputs beside or in place of
 * the bf16 one.  r' = bf16(x + residual) goes to residual_out (NULL: back to
 * residual; without a residual r' = x and nothing is written), v = r' * inv * w,
 *   y = bf16(v)        (r', inv and y have biv_add_rmsnorm's bits)
 *   codes, scales of v (in FP32: one rounding; biv_add_rmsnorm and then
 *                       biv_act_quant_fp8 round twice), an FP8 GEMM's A
 *   keep, keep_scales of r' (what biv_act_quant_fp8 of r' writes), inv float32
 *                      [rows]: what the backward reads
 * y, codes, keep and inv may be NULL, but not both y and codes; codes and keep
 * each come with their scales.  y may alias x, residual_out residual.
 * d <= 8192.  A row's bits depend on the row only.  A row with an infinite or
 * NaN element gives NaN in that row (its kept codes hold NaN where the element
 * is not finite, or v / s is not). */
typedef struct {
  const uint16_t* x; int64_t x_stride;
  uint16_t* residual; int64_t r_stride;       /* or NULL */
  uint16_t* residual_out; int64_t ro_stride;  /* or NULL */
  const uint16_t* w;
  uint16_t* y; int64_t y_stride;
  uint8_t* codes; float* scales;
  uint8_t* keep; float* keep_scales;
  float* inv;
  int rows, d;
  float eps;
} biv_norm_fp8_desc;
biv_status biv_add_rmsnorm_fp8(const biv_norm_fp8_desc* desc, biv_stream_t stream);

/* Backward of it from the kept rows: with x' = code * (s * inv), inv as the forward
 * wrote it and dy the gradient of v,
 *   dx = inv*(w*dy - x'*(sum(w*dy*x')/d)) (+ dres),
 *   dw float32 [d] = sum over rows of dy*x' (added to dw when accumulate is 1).
 * dres: the gradient that reaches r' past the norm, of dx's type, or NULL.  dy
 * BIV_F32 or BIV_BF16, dx likewise.  dx may be dres, or dy where types and strides
 * agree.  dw is summed in an order fixed by rows, d and the types.  Workspace:
 * biv_rmsnorm_backward_fp8_workspace bytes, 16-byte aligned, no initial value. */
typedef struct {
  const uint8_t* keep; const float* keep_scales; const float* inv;
  const uint16_t* w;
  const void* dy; int64_t dy_stride; int dy_dtype;
  const void* dres; int64_t dres_stride;
  void* dx; int64_t dx_stride; int dx_dtype;
  float* dw;
  int accumulate;
  int rows, d;
  void* workspace;
  size_t workspace_bytes;
} biv_norm_bwd_fp8_desc;
biv_status biv_rmsnorm_backward_fp8_workspace(int rows, int d, size_t* bytes);
biv_status biv_rmsnorm_backward_fp8(const biv_norm_bwd_fp8_desc* desc, biv_stream_t stream);

/* biv_silu_mul (y bf16 [rows, I], its bits; NULL: not written) that also keeps
 * its input gate_up bf16 [rows, 2I] in 8 bits: keep uint8 [rows, 2I], keep_scales
 * float32 [rows, 2 ceil(I / 128)]; gate and up are quantised apart, each half's
 * groups start at its first column. */
biv_status biv_silu_mul_keep_fp8(const uint16_t* gate_up, int64_t gu_stride, uint16_t* y,
                                 int64_t y_stride, uint8_t* keep, float* keep_scales, int rows, int I,
                                 biv_stream_t stream);

/* Backward of it from the kept rows (gate, up = code * s), dy BIV_F32 or BIV_BF16
 * rows of I.  dgate_up rows of 2I: BIV_F32, by biv_silu_mul_backward's operations
 * (its bits where bf16 holds gate and up); BIV_BF16, the same with a sigmoid that is
 * off by 1 ulp of FP32 at most, or by 2^-126 where it is below that, before the
 * rounding to bf16.  y (bf16 rows of I, or NULL) gets silu(gate) * up of the kept
 * values, by the same sigmoid, which the gradient of the product behind it reads. */
biv_status biv_silu_mul_backward_fp8(const uint8_t* keep, const float* keep_scales, const void* dy,
                                     int64_t dy_stride, int dy_dtype, void* dgate_up,
                                     int64_t dgate_up_stride, int dgate_up_dtype, uint16_t* y,
                                     int64_t y_stride, int rows, int I, biv_stream_t stream);

/* ------------------------------------------------------ optimizer step --
 * AdamW over many tensors at once, writing the model's own weights in
 * place (captured graphs keep their addresses; BF16 weights that the forward
 * reads, "Finish RL Training Faster", section "让训练前向使用推理的数值").  Per
 * element, in FP32:
 *   g = grad * coef;  m = b1 m + (1-b1) g;  v = b2 v + ((1-b2) g) g
 *   w = w (1 - lr wd) - (lr / (1-b1^t)) m / (sqrt(v) / sqrt(1-b2^t) + eps)
 * (each operation rounded once, in the order written: m and v, and with 8 bits their
 * codes and scales, have these bits.  w has but for its root and quotient, each an
 * approximation corrected once, which may miss the nearest value where two all but tie)
 * with t the step's number, lr = *lr * lr_scale and wd of the tensor.
 *
 * A biv_opt_tensor describes one tensor of numel elements, all arrays dense:
 *   param  BIV_F32: the weight; BIV_BF16 with master (float32): the master is
 *          updated and param gets its nearest bf16; BIV_BF16 without master:
 *          w is the bf16 weight, rounded back to bf16.
 *   grad   BIV_F32 or BIV_BF16.
 *   state  BIV_F32: m, v float32.  BIV_E4M3: blocks of 128 consecutive
 *          elements (the last one shorter); with a = max(amax|m|, 2^-100) of
 *          the block, m holds e4m3 codes of m (448 (1/a)) and m_scale a (1/448),
 *          each operation rounded once; v and v_scale hold sqrt(v) the same way
 *          (the root halves the exponent range that the codes have to cover),
 *          and a positive root never gets code 0.  m_scale, v_scale float32 [ceil(numel / 128)].
 * rounding (8-bit states and bf16 weights without a master): NEAREST (ties to
 * even), or STOCHASTIC: the magnitude goes up with a chance equal to the part
 * cut off, from 16 bits of a hash of (seed, t, element), so that steps below
 * half a grid spacing still move the value on average; a rerun repeats it.
 * Without a clip a NaN or infinite gradient is not caught: its weight becomes NaN
 * in either rounding, m and v NaN or infinite.  With 8-bit states an infinite m
 * makes its block's scale infinite, and at the next step the block's 128 weights
 * NaN; an infinite v with a finite m (a square beyond FP32) makes all positive v
 * of the block infinite, whose weights then only decay, and its zeros NaN.
 *
 * biv_opt_plan (host only, no launch) checks a HOST array of n tensors and
 * fills first_chunk, rng_base and vec; *chunks receives the launch size and
 * *kinds which combinations of types occur (each is a launch of its own).  The
 * caller then copies the array to the device (by a memory copy: the kernels
 * read it before earlier kernels of the stream are done).  It refuses null pointers,
 * misaligned elements, unsupported type combinations and tensors whose written
 * ranges overlap. */
typedef enum { BIV_ROUND_NEAREST = 0, BIV_ROUND_STOCHASTIC = 1 } biv_rounding;
typedef struct {
  void* param;
  float* master;
  const void* grad;
  void* m;
  void* v;
  float* m_scale;
  float* v_scale;
  int64_t numel;
  int64_t first_chunk;       /* filled by biv_opt_plan */
  int64_t rng_base;          /* filled by biv_opt_plan */
  float lr_scale, weight_decay;
  int32_t param_dtype, grad_dtype, state_dtype;
  int32_t vec;               /* filled by biv_opt_plan */
} biv_opt_tensor;
biv_status biv_opt_plan(biv_opt_tensor* host_tensors, int n, int64_t* chunks, int* kinds);

/* Global L2 norm of all gradients: out (float32 [4]) [0] = norm, [1] = min(1,
 * max_norm / (norm + 1e-6)) (1 when max_norm is 0); [2] must be 0 before the
 * first call and is 0 again after each, [3] is not used.  FP32 sums that carry their rounding
 * errors along, in one order fixed by the tensors' sizes; a norm beyond about
 * 1.8e19 is not finite.  tensors:
 * device copy of the planned array.  Workspace: biv_grad_norm_workspace bytes,
 * 16-byte aligned, caller-owned, no initial value. */
biv_status biv_grad_norm_workspace(int64_t chunks, size_t* bytes);
biv_status biv_grad_norm(const biv_opt_tensor* tensors, int n, int64_t chunks, float max_norm,
                         float* out, void* workspace, size_t workspace_bytes, biv_stream_t stream);

/* One AdamW step.  lr (float32 [1]), step (int32 [2]) and clip (float32 [4],
 * biv_grad_norm's out, or NULL for coef = 1) are device memory read by the
 * kernel, so a captured step replays with new values.  step[0] counts the
 * steps taken (0 for new states): the call uses t = step[0] + 1 and stores it;
 * step[1] must be 0 between calls and is 0 again after each; calls that share
 * it, or tensors, must not overlap on the GPU.  With clip given
 * and its norm not finite the whole call changes nothing, step included; so does
 * a call of no chunk (no tensor has an element).  The next call of the stream may
 * read the new weights. */
typedef struct {
  const biv_opt_tensor* tensors;   /* device */
  int n;
  int kinds;                       /* biv_opt_plan's */
  int64_t chunks;
  const float* lr;
  const float* clip;
  int32_t* step;
  double beta1, beta2;             /* 0 <= beta < 1 */
  float eps;                       /* >= 1e-30 */
  int rounding;                    /* biv_rounding */
  uint64_t seed;
} biv_adamw_desc;
biv_status biv_adamw(const biv_adamw_desc* desc, biv_stream_t stream);

#ifdef __cplusplus
}
#endif
#endif /* BIV_H */
