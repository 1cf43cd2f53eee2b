/*
 * moe.h -- C ABI of libmoe, a single-GPU (MI355X / gfx950) implementation of
 * the mixture-of-experts layer of a Basalt-style local inference engine:
 * router logits, softmax top-k gating, token-to-expert bucketing, block-
 * quantized (NVFP4, Q6_K-style, Q8_0, IQ3-style) SwiGLU expert FFNs with the dequantization
 * fused into the matmuls, the gate-weighted combine, and the per-step expert
 * usage histogram that decides which experts stay resident; of the same
 * layer's attention over a paged key/value cache; and of the norms and
 * microscaled dense projections around both.
 *
 * What the pages fix, and where:
 *   - each token uses a few experts chosen from many; the busiest experts stay
 *     in GPU memory and the rest may live in system RAM and be streamed on
 *     demand -- basalt.jgulfo.com, section "Expert tiers"; aiopssre.com
 *     ("What Basalt changes in a Blackwell local inference stack"), section
 *     "Experts can move without becoming free";
 *   - routed experts are NVIDIA NVFP4, packs also carry GGUF Q6_K tensors --
 *     basalt.jgulfo.com, sections "Models", "Quick start" and the engine notes
 *     under "All the numbers";
 *   - 1 to 8 concurrent request slots, so decode batches of 1..8 tokens --
 *     aiopssre.com, section "Concurrency divides context unless you pay for
 *     more cache"; devotd.net (en), section "--parallel slots and KV cache
 *     allocation";
 *   - Q8_0 is the 8-bit GGUF format the pages measure quality against and
 *     keep for Basalt's dense projections -- basalt.jgulfo.com, "All the
 *     numbers" (the quality table and the engine notes); here it is offered
 *     as a down-projection format of the experts;
 *   - community packs run IQ3 GGUF files -- basalt.jgulfo.com, "Community";
 *     their grids are not on the pages, so MOE_FMT_IQ3G keeps the IQ3
 *     structure (grid indices per 4 weights, sign bits, small scales) with a
 *     grid defined here (below), offered as a down-projection format;
 *   - the pages' packs also carry IQ1_M tensors (basalt.jgulfo.com,
 *     "Models"), a codebook format of under two bits per weight whose grid
 *     the pages do not give either, so MOE_FMT_IQ1G keeps that structure
 *     (a ternary grid vector per 8 weights, small scales) with a grid
 *     defined here (below), offered as a down-projection format.
 * The pages give no formula.  The arithmetic below is the plainest reading;
 * each entry point states it.
 *
 * Conventions (all entry points):
 *   - Pointers are DEVICE pointers unless marked "host".  Every buffer is
 *     owned by the caller; the library allocates nothing per call and frees
 *     nothing it was given.
 *   - Calls are asynchronous and ordered on the given stream.  T == 0 returns
 *     MOE_OK without launching anything.
 *   - Arguments are validated on the host before any launch; an invalid or
 *     unsupported argument returns an error status and launches nothing (no
 *     clamping, no truncation).  A failed launch returns MOE_ERR_HIP.  The
 *     message of the last failure on the calling thread is moe_last_error().
 *     Device-side faults surface at the caller's next synchronization.
 *   - Calls on different streams may run concurrently if they write
 *     different buffers.
 *   - bf16 values are passed as uint16_t bit patterns.
 *
 * Supported shapes: 1 <= k <= min(E, 64), E <= 1024, H % 128 == 0,
 * 128 <= H <= 8192, I % 128 == 0 (NVFP4, Q8_0) or I % 256 == 0 (Q6_K, IQ3G, IQ1G),
 * I <= 8192.  The attention side states its own (moe_kv_cache, moe_qkv_desc).
 */
#ifndef MOE_H
#define MOE_H

#include <stddef.h>
#include <stdint.h>

#include <hip/hip_runtime_api.h>

#ifdef __cplusplus
extern "C" {
#endif

#define MOE_ABI_VERSION 2

typedef enum moe_status {
  MOE_OK = 0,
  MOE_ERR_INVALID_ARG = -1,  /* null pointer, negative size, k > E, ... */
  MOE_ERR_UNSUPPORTED = -2,  /* shape or format outside the supported set */
  MOE_ERR_WORKSPACE = -3,    /* workspace or bucket buffer too small */
  MOE_ERR_BUDGET = -4,       /* tier: HBM budget below the working set */
  MOE_ERR_HIP = -5,          /* a HIP runtime call or launch failed */
  MOE_ERR_HOST_ALLOC = -6    /* tier: host metadata allocation failed */
} moe_status;

/* Weight formats. */
#define MOE_FMT_NVFP4 1  /* E2M1 codes, E4M3 scale per 16 along K, fp32 per-tensor scale */
#define MOE_FMT_Q6K 2    /* 256-element superblocks: 16 x int8 sub-scales, fp16 scale, 6-bit codes */
#define MOE_FMT_Q8_0 3   /* 32-element blocks: fp16 scale, 32 int8 codes (down projection only) */
#define MOE_FMT_IQ3G 4   /* 256-element superblocks: fp16 scale, 4-bit odd multipliers per 32,
                            8-bit grid index per 4, sign bits (down projection only) */
#define MOE_FMT_IQ1G 5   /* 256-element superblocks: fp16 scale, 4-bit odd multipliers per 32,
                            10-bit ternary grid index per 8 (down projection only) */

/* Element types of the expert-output buffer y. */
#define MOE_DTYPE_F32 0
#define MOE_DTYPE_BF16 1

/* Library version of this header (MOE_ABI_VERSION). */
int moe_abi_version(void);

/* Expert-FFN kernel family (moe_layer_desc.ffn_mode, read by each
 * moe_expert_ffn call; there is no process-wide state):
 *   MOE_FFN_AUTO -- dequant-fused GEMV for decode-sized batches, MFMA grouped
 *                   GEMM once experts average >= 16 tokens (default);
 *   MOE_FFN_GEMV / MOE_FFN_GEMM -- force one family (any size; results agree
 *                   within the stated tolerance).  The grouped GEMM needs
 *                   H % 256 == 0, T*H < 2^32 and T*k*I < 2^32; AUTO uses the
 *                   GEMV otherwise, and a forced GEMM call fails with
 *                   MOE_ERR_UNSUPPORTED.
 * Any other value is rejected with MOE_ERR_INVALID_ARG by every call that
 * takes the layer. */
#define MOE_FFN_AUTO 0
#define MOE_FFN_GEMV 1
#define MOE_FFN_GEMM 2

/* Message of the last failing call on this thread ("" if none).  Host
 * string owned by the library, valid until the next failing call. */
const char* moe_last_error(void);

/* ------------------------------------------------------------------------ */
/* Expert weights                                                            */
/* ------------------------------------------------------------------------ */

/*
 * Canonical input layouts (what moe_pack_experts reads):
 *   NVFP4 matrix W[N][K]: codes u8 [N][K/2], element k of row n in nibble
 *     (k & 1) of byte k/2 (even element low); E2M1 code: bit 3 sign, bits 2..1
 *     exponent (bias 1), bit 0 mantissa.  scales u8 [N][K/16]: E4M3 (fn) scale
 *     of elements 16b..16b+15.  One fp32 per-tensor scale ts.
 *     w[n][k] = e2m1(code) * e4m3(scale) * ts.
 *   Q6_K-style matrix W[N][K]: row n is K/256 superblocks of 210 bytes:
 *     ql[128] (low 4 bits of element i: nibble i&1 of byte i/2), qh[64]
 *     (high 2 bits of element i: bits 2*(i&3) of byte i/4), sc int8[16]
 *     (sub-block i/16), d fp16 little-endian[2];
 *     w = d * sc[i/16] * (q - 32), q = low | high << 4 in 0..63.
 *   Q8_0 matrix W[N][K]: row n is K/32 blocks of 34 bytes: d fp16
 *     little-endian[2], then the int8 codes q[32] of elements 32b..32b+31;
 *     w = d * q.
 *   IQ3G matrix W[N][K] (3.19 bits per weight): row n is K/256 superblocks of
 *     102 bytes: d fp16 little-endian[2]; s[4], the 4-bit multiplier s_j of
 *     sub-block j (elements 32j..32j+31) in byte j/2 (low nibble for even j);
 *     idx[64], the grid entry of elements 4g..4g+3; sgn[32], bit i%8 of byte
 *     i/8 set when element i is negative;
 *     w = d * (2 s_j + 1) * grid[idx[i/4]][i%4] * (sgn ? -1 : 1),
 *     grid = the 256 smallest vectors of four positive odd integers <= 15,
 *     ordered by squared norm, then lexicographically (entry 0 = (1,1,1,1);
 *     every magnitude is at most 9).
 *   IQ1G matrix W[N][K] (1.44 bits per weight): row n is K/256 superblocks of
 *     46 bytes: d fp16 little-endian[2]; s[4], the 4-bit multiplier s_j of
 *     sub-block j (elements 32j..32j+31) in byte j/2 (low nibble for even j);
 *     qs[32], the low 8 bits of the grid entry of elements 8g..8g+7; qh[8],
 *     its high 2 bits at bits 2(g%4), 2(g%4)+1 of byte g/4;
 *     w = d * (2 s_j + 1) * grid[idx[i/8]][i%8],
 *     grid = the 1024 vectors of eight values in {-1, 0, +1} with the fewest
 *     nonzero values, ordered by that count, then lexicographically
 *     (-1 < 0 < +1, value 0 the most significant; entry 0 = all zero).
 *   Gate and up are [I][H] (K = H); down is [H][I] (K = I).
 *
 * The GPU kernels read a packed "blob" per expert (a device-friendly
 * re-arrangement of the same bytes, 16-byte granules transposed so that one
 * wavefront load covers consecutive rows).  moe_expert_blob_bytes gives its
 * size; moe_pack_experts writes it.  With Q6_K, Q8_0, IQ3G or IQ1G down weights the blob
 * ends with a 256-byte section holding one int32 computed by the pack from
 * the expert's block scales: the power of two by which the grouped GEMM
 * scales that expert's fp16 down weights (so none can overflow fp16, for any
 * scales; the product is scaled back in fp32).
 */

/* One entry of the device-resident expert table (24 bytes). */
typedef struct moe_expert_ref {
  const void* blob;   /* device pointer to the packed expert (256-byte aligned) */
  float ts_gate;      /* NVFP4 per-tensor scales */
  float ts_up;
  float ts_down;      /* ignored when the down projection is Q6_K, Q8_0, IQ3G or IQ1G */
  uint32_t reserved;  /* 0 (not read by the library) */
} moe_expert_ref;

/* Bytes of one packed expert blob (a multiple of 256); 0 if unsupported. */
size_t moe_expert_blob_bytes(int32_t H, int32_t I, int32_t fmt_gate_up, int32_t fmt_down);

/* Pack E experts from the canonical layouts (device arrays stacked over
 * experts: gate_q [E][I][H/2], gate_s [E][I][H/16], up likewise, down_q
 * [E][H][I/2] and down_s [E][H][I/16] for NVFP4, down_q [E][H][I/256*210]
 * for Q6_K, [E][H][I/32*34] for Q8_0, [E][H][I/256*102] for IQ3G or
 * [E][H][I/256*46] for IQ1G, down_s == NULL for those four) into
 * E blobs at blobs + e * blob_stride.
 * blob_stride >= moe_expert_blob_bytes(...) and a multiple of 256. */
moe_status moe_pack_experts(int32_t E, int32_t H, int32_t I, int32_t fmt_gate_up,
                            int32_t fmt_down, const uint8_t* gate_q, const uint8_t* gate_s,
                            const uint8_t* up_q, const uint8_t* up_s, const uint8_t* down_q,
                            const uint8_t* down_s, void* blobs, size_t blob_stride,
                            hipStream_t stream);

/* ------------------------------------------------------------------------ */
/* Layer description and bucket buffers                                      */
/* ------------------------------------------------------------------------ */

/* Host struct holding device pointers; read during each call only. */
typedef struct moe_layer_desc {
  int32_t E;            /* experts */
  int32_t k;            /* experts per token */
  int32_t H;            /* hidden size */
  int32_t I;            /* expert intermediate size */
  int32_t fmt_gate_up;  /* MOE_FMT_NVFP4 */
  int32_t fmt_down;     /* MOE_FMT_NVFP4, MOE_FMT_Q6K, MOE_FMT_Q8_0, MOE_FMT_IQ3G or MOE_FMT_IQ1G */
  int32_t renormalize;  /* 1: softmax renormalised over the selected k; 0: full softmax */
  int32_t ffn_mode;     /* MOE_FFN_AUTO (0), MOE_FFN_GEMV or MOE_FFN_GEMM */
  const moe_expert_ref* experts;  /* device [E] */
  const float* w_router;          /* device fp32 [E][H] */
  const float* router_bias;       /* device fp32 [E], or NULL (no bias) */
} moe_layer_desc;

/* Per-step bucket results (device pointers into one caller buffer). */
typedef struct moe_buckets {
  uint32_t* counts;     /* [E]   assignments per expert */
  int32_t* offsets;     /* [E+1] exclusive prefix sum of counts */
  int32_t* sorted_asg;  /* [T*k] assignments a = t*k + j ordered by (expert, a) */
  int32_t* asg_pos;     /* [T*k] position of assignment a in sorted_asg */
  int32_t* active;      /* [E]   experts with counts > 0, ascending (first n_active) */
  int32_t* n_active;    /* [1] */
  int64_t T_max;        /* capacity in tokens */
  int32_t E;
  int32_t k;
} moe_buckets;

/* Bytes needed for the bucket buffers of (E, T_max, k). */
size_t moe_buckets_bytes(int32_t E, int64_t T_max, int32_t k);

/* Point the fields of *out into the caller's device buffer buf (bytes long,
 * 256-byte aligned).  Host-only bookkeeping: launches nothing. */
moe_status moe_buckets_carve(void* buf, size_t bytes, int32_t E, int64_t T_max, int32_t k,
                             moe_buckets* out);

/* Device workspace bytes for moe_bucket and moe_expert_ffn on up to T_max
 * tokens of layer L (covers both calls; one buffer may serve both). */
size_t moe_workspace_bytes(const moe_layer_desc* L, int64_t T_max);

/* ------------------------------------------------------------------------ */
/* The layer's steps                                                         */
/* ------------------------------------------------------------------------ */

/* Router and top-k gating.  The pages' model routes every token to a small
 * subset of its many experts (basalt.jgulfo.com, "Expert tiers"; aiopssre.com,
 * "Experts can move without becoming free"); how the subset is scored is not
 * given, so this is the plainest reading: a linear router, top-k on its
 * logits, softmax weights.
 *   logits[t][e] = fp32( sum_h x[t][h] * w_router[e][h] + bias[e] ), the sum
 *     taken in double precision in one fixed order -- 64 interleaved partial
 *     sums (partial j adds h = j, j+64, ... ascending), combined pairwise
 *     p[j] += p[j+w] for w = 32, 16, ..., 1, then the bias -- and rounded to
 *     fp32 once, so the logits (and hence the selected experts) are
 *     reproducible bit for bit.
 *   topk_idx[t][0..k) = the k experts first in the order (logit desc, expert
 *     index asc): ties go to the lower index.
 *   topk_w[t][j] = exp(l_j - l_0) / sum_{i<k} exp(l_i - l_0) (renormalize=1),
 *     or the full softmax probability of expert idx[t][j] (renormalize=0).
 * x: bf16 [T][H]; logits: fp32 [T][E]; topk_idx: int32 [T][k];
 * topk_w: fp32 [T][k].  All caller-allocated. */
moe_status moe_route(const moe_layer_desc* L, const uint16_t* x, int64_t T, float* logits,
                     int32_t* topk_idx, float* topk_w, hipStream_t stream);

/* Token-to-expert bucketing: a stable counting sort of the T*k assignments by
 * expert (deterministic; no dependence on atomic ordering), so that each
 * selected expert runs once per step over all the tokens that chose it and
 * experts nobody chose are not touched (the sparse selection of
 * basalt.jgulfo.com, "Expert tiers").  Fills every
 * field of *b for this step.  b->T_max >= T, b->E == L->E, b->k == L->k.
 * ws: device workspace of at least moe_workspace_bytes(L, T) bytes. */
moe_status moe_bucket(const moe_layer_desc* L, const int32_t* topk_idx, int64_t T,
                      const moe_buckets* b, void* ws, size_t ws_bytes, hipStream_t stream);

/* Gating step in one call: moe_route, then moe_bucket, then (when hist is
 * not NULL) moe_expert_hist, with the same arguments and the same results
 * bit for bit.  For E <= 256, T <= 64 and T*k <= 256 (decode-sized steps) top-k,
 * bucketing and the histogram update run as one single-workgroup kernel
 * after the router logits, two launches instead of four.
 * hist: uint32 [E] or NULL; shifts as for moe_expert_hist (checked only when
 * hist is not NULL).  ws: as for moe_bucket. */
moe_status moe_route_bucket(const moe_layer_desc* L, const uint16_t* x, int64_t T,
                            float* logits, int32_t* topk_idx, float* topk_w, const moe_buckets* b,
                            void* ws, size_t ws_bytes, uint32_t* hist, int32_t decay_shift,
                            int32_t unit_shift, hipStream_t stream);

/* Expert FFNs with fused dequantization (SwiGLU).  The routed experts are
 * stored block-quantized -- NVFP4 in the pages' packs, with GGUF Q6_K tensors
 * in the DQ6_K packs (basalt.jgulfo.com, "Models" and "Quick start"); the
 * weights are decoded inside the matmuls, never materialised:
 *   for each assignment a of expert e (token t = a / k), at sorted position
 *   p = b->asg_pos[a]:
 *     g = x[t] . dq(Wg_e)^T,  u = x[t] . dq(Wu_e)^T,  h = silu(g) * u,
 *     y[p] = h . dq(Wd_e)^T,  silu(z) = z / (1 + exp(-z)),
 *   accumulated in fp32.  y: [T*k][H] of y_dtype (MOE_DTYPE_F32 or _BF16),
 *   rows in sorted order.  Decode-sized batches run as dequant-fused GEMV;
 *   larger ones as an MFMA grouped GEMM over experts, which multiplies an
 *   fp16 copy of x scaled per token row by a power of two (exact for every
 *   value above 2^-29 of the row's largest magnitude).  h between the two
 *   projections is rounded to 16 bits (bf16 in the GEMV; scaled fp16 in the
 *   GEMM, redone in bf16 if it would overflow).  The GEMM rounds Q6_K and
 *   Q8_0 down weights once to fp16 after scaling each expert's weights by a
 *   power of two fixed at pack time (see the blob), so any scales are in
 *   range; the GEMV decodes them exactly.
 * ws: at least moe_workspace_bytes(L, T) bytes. */
moe_status moe_expert_ffn(const moe_layer_desc* L, const uint16_t* x, int64_t T,
                          const moe_buckets* b, void* y, int32_t y_dtype, void* ws,
                          size_t ws_bytes, hipStream_t stream);

/* moe_expert_ffn for callers that cannot allocate device memory (code under
 * HIP graph capture, tight serving loops, harnesses that forbid hipMalloc):
 * the same computation, kernels and results (bit for bit) as moe_expert_ffn,
 * with the workspace taken from a static buffer inside the library instead
 * of a caller argument.  The caller still passes x, the buckets and y.
 *   - The buffer is MOE_NOALLOC_WORKSPACE_BYTES (32 MiB) per GPU, part of the
 *     library's code object: each GPU the library runs on holds it until the
 *     process ends.  Its device address is looked up on the first call made
 *     with that device current; the call itself allocates nothing (no
 *     hipMalloc, no hipFree, no allocating library routine).
 *   - A call whose workspace (moe_workspace_bytes covers it) would exceed the
 *     buffer returns MOE_ERR_WORKSPACE before any launch.  At the decode
 *     layer's shape (E 128, k 8, H 2048, I 768) that is above about 2,000
 *     tokens.
 *   - Every call on one GPU shares that GPU's buffer, which keeps the last
 *     call's contents (nothing in it needs to start at zero): calls that
 *     overlap on one GPU -- on different streams, or from different threads --
 *     race and must not be issued.  Calls on different GPUs do not interact. */
#define MOE_NOALLOC_WORKSPACE_BYTES ((size_t)32 << 20)
moe_status moe_expert_ffn_noalloc(const moe_layer_desc* L, const uint16_t* x, int64_t T,
                                  const moe_buckets* b, void* y, int32_t y_dtype,
                                  hipStream_t stream);

/* moe_route_bucket followed by moe_expert_ffn (the layer's routing and its
 * routed experts: basalt.jgulfo.com, "Expert tiers"), with the same arguments
 * and the same outputs bit for bit (logits, top-k, buckets, histogram, y).  For
 * batches of up to 4 tokens (with E <= 256, the GEMV family, NVFP4 gate/up
 * with H <= 2048) it takes one launch fewer: every
 * workgroup of the gate/up kernel repeats the batch's top-k and bucketing
 * in its own LDS from the router logits and finds its expert there, and one
 * of them writes the gating outputs.  Otherwise it makes the two calls.
 * ws: at least moe_workspace_bytes(L, T) bytes (serves both steps). */
moe_status moe_route_ffn(const moe_layer_desc* L, const uint16_t* x, int64_t T, float* logits,
                         int32_t* topk_idx, float* topk_w, const moe_buckets* b, uint32_t* hist,
                         int32_t decay_shift, int32_t unit_shift, void* y, int32_t y_dtype,
                         void* ws, size_t ws_bytes, hipStream_t stream);

/* The whole layer step: moe_route_ffn then moe_combine (same arguments,
 * routing outputs, buckets and histogram bit for bit; out within the bf16
 * rounding of the combine).  For decode batches of 2 to 8 tokens on the
 * GEMV family the down projection and the combine run as one kernel that
 * writes out straight from h: y is then not written (the caller still
 * passes it, for the other sizes), and out sums each token's k gate-weighted
 * expert rows in a fixed order (slots j = w mod 8 for each w, then w
 * ascending) -- the mixture of the experts a token uses (basalt.jgulfo.com,
 * "Expert tiers").  residual: bf16 [T][H] or NULL; out: bf16 [T][H] (may
 * alias residual).  ws: at least moe_workspace_bytes(L, T) bytes. */
moe_status moe_layer_forward(const moe_layer_desc* L, const uint16_t* x, int64_t T,
                             const uint16_t* residual, uint16_t* out, float* logits,
                             int32_t* topk_idx, float* topk_w, const moe_buckets* b,
                             uint32_t* hist, int32_t decay_shift, int32_t unit_shift, void* y,
                             int32_t y_dtype, void* ws, size_t ws_bytes, hipStream_t stream);

/* Gate-weighted combine: each token's output is its selected experts'
 * outputs weighted by the gates (the mixture the pages' model computes from
 * the few experts a token uses: basalt.jgulfo.com, "Expert tiers"), written
 * as a gather so that the result does not depend on scheduling:
 *   out[t] = bf16_rne( residual[t] + sum_{j=0..k-1} topk_w[t][j] * y[asg_pos[t*k+j]] ),
 *   in fp32 with j ascending.  residual: bf16 [T][H] or NULL; out: bf16 [T][H]
 *   (may alias residual). */
moe_status moe_combine(const moe_layer_desc* L, const void* y, int32_t y_dtype,
                       const moe_buckets* b, const float* topk_w, int64_t T,
                       const uint16_t* residual, uint16_t* out, hipStream_t stream);

/* Expert-usage histogram deciding residency: the pages keep the most-routed
 * experts in GPU memory and let the placement follow usage as the
 * conversation changes (basalt.jgulfo.com, "Expert tiers" and the FAQ).  The
 * running count is this reading: an exponentially decaying integer count,
 * unsigned 32-bit arithmetic:
 *   hist[e] = hist[e] - (hist[e] >> decay_shift) + (counts[e] << unit_shift).
 * hist: uint32 [E], read and written.  0 <= decay_shift, unit_shift < 32. */
moe_status moe_expert_hist(const moe_layer_desc* L, const moe_buckets* b, uint32_t* hist,
                           int32_t decay_shift, int32_t unit_shift, hipStream_t stream);

/* ------------------------------------------------------------------------ */
/* The layer's attention side: key/value cache and attention                 */
/* ------------------------------------------------------------------------ */
/*
 * The pages' engine keeps a key/value cache for its 1 to 8 request slots beside
 * the experts and lets its precision be chosen, because the two share GPU
 * memory (aiopssre.com, "Concurrency divides context unless you pay for more
 * cache"; devotd.net (en), "--parallel slots and KV cache allocation"); the
 * pages give no layout.  Here the cache is paged and holds 16-bit values
 * (MOE_FMT_BF16) or the block formats of the experts, NVFP4 (4.5 bits per
 * value) and Q8_0 (8.5 bits per value), with blocks along the head size D.
 *
 * Page of page_tokens tokens (P below): for each key/value head in turn, four
 * sections one after the other (o: token within the page, d: element):
 *   NVFP4  K codes  u8 [P][D/2]       element d of token o in nibble d & 1
 *          K scales E4M3 [P][D/16]
 *          V codes  u8 [P/4][16][4][D/32]: token o, element d in byte
 *                   (d % (D/16)) / 2 of [o/4][d/(D/16)][o%4], nibble d & 1
 *          V scales E4M3 [D/16][P]
 *   Q8_0   K codes  int8 [P][D];       K scales fp16 [P][D/32]
 *          V codes  int8 [P/4][D][4]   token o, element d at [o/4][d][o%4]
 *          V scales fp16 [D/32][P]
 *   BF16   K [P][D];  V [P/4][D][4]    (no scales)
 * Quantisation of a bf16 value x in a block whose largest magnitude is A, in
 * fp32, divisions and conversions rounded to nearest even:
 *   NVFP4  S = e4m3(min(A / (6 ts), 448)), code = e2m1(x / (S ts)) (0 when
 *          S = 0), value code * S * ts; ts = k_scale or v_scale of the cache.
 *   Q8_0   d = fp16(min(A, 65024) / 127), q = rint(x / d) within +-127 (0 when
 *          d = 0), value q * d (65024 = 512 * 127, so every value fits fp16).
 * A block that holds an infinity or a NaN gets a NaN scale, so all its values
 * read as NaN.
 */
#define MOE_FMT_BF16 6  /* 16-bit cache values, as they are */

/* Host struct: a layer's cache.  pool is device memory, 256-byte aligned, of
 * n_pages * moe_kv_page_bytes(...) bytes; it needs no particular contents. */
typedef struct moe_kv_cache {
  int32_t fmt;          /* MOE_FMT_NVFP4, MOE_FMT_Q8_0 or MOE_FMT_BF16 */
  int32_t n_kv;         /* key/value heads, 1..1024 */
  int32_t D;            /* head size: 64, 128 or 256 */
  int32_t page_tokens;  /* 32, 64, 128 or 256 */
  int32_t n_pages;      /* pages in the pool, >= 1 */
  float k_scale;        /* NVFP4 per-tensor scales, finite and > 0 (not read */
  float v_scale;        /*   for the other formats) */
  void* pool;
} moe_kv_cache;

/* Bytes of one page (a multiple of 256); 0 if unsupported. */
size_t moe_kv_page_bytes(int32_t fmt, int32_t n_kv, int32_t D, int32_t page_tokens);

/* Host struct holding device pointers: the sequences (request slots) of a
 * step.  Sequence b has the packed rows row_start[b] .. row_start[b+1]-1 of
 * the step's row arrays (none, one, or many), which are the last of its
 * kv_len[b] tokens: row row_start[b] + i of n rows is token
 * kv_len[b] - n + i.  Token j lies in page page_table[b][j / page_tokens].
 * The arrays live on the device, so their contents are checked there: rows
 * outside 0..T are not touched (those of the same sequence inside are answered
 * as ever), a row before its sequence's first token
 * (kv_len[b] < n) stores nothing and sees nothing, and a page outside
 * 0..n_pages-1 (or a token past max_pages pages) is neither read nor written:
 * whatever should have been read from it is NaN in the results. */
typedef struct moe_seq_batch {
  int32_t n_seq;              /* sequences, 0..65535 */
  int32_t max_pages;          /* row length of page_table */
  const int32_t* row_start;   /* [n_seq + 1], ascending */
  const int32_t* kv_len;      /* [n_seq] */
  const int32_t* page_table;  /* [n_seq][max_pages] */
} moe_seq_batch;

/* Host struct: what happens to a step's queries and keys before they are used. */
typedef struct moe_qkv_desc {
  int32_t n_q;             /* query heads, a multiple of n_kv, <= 1024 */
  float eps;               /* of the norms, finite and >= 0 */
  const float* q_norm;     /* device fp32 [D]: norm weights of the query heads, or NULL: no norm */
  const float* k_norm;     /* the same for the key heads */
  int32_t rot_dim;         /* rotated elements of a head, a multiple of 16 up to D; 0: none */
  int32_t interleaved;     /* 1: pairs (2i, 2i+1); 0: pairs (i, i + rot_dim/2) */
  const double* inv_freq;  /* device fp64 [rot_dim/2]: radians per position (moe_rope_freqs) */
  float rope_scale;        /* factor of the cosines and sines (1, or moe_rope_freqs's) */
} moe_qkv_desc;

/* Frequencies of rotary positions, f_i = base^(-2i/rot_dim), stretched for
 * contexts longer than the orig_len tokens a model was trained on by `factor`
 * >= 1.  Host call, launches nothing; freqs: host fp64 [rot_dim/2].
 *   MOE_ROPE_PLAIN   f_i (factor ignored)
 *   MOE_ROPE_LINEAR  f_i / factor
 *   MOE_ROPE_BASE    base * factor^(rot_dim/(rot_dim-2)) in place of base: the
 *                    slowest pair is stretched by factor, the fastest not at all
 *   MOE_ROPE_PARTS   by the turns t_i = orig_len f_i / 2 pi a pair makes over
 *                    orig_len: f_i kept where t_i >= turns_hi, f_i / factor
 *                    where t_i <= turns_lo, linear in the pair's index between
 *                    (interpolation by parts); *scale = 0.1 ln(factor) + 1.
 * scale: the value for rope_scale (1 for the other kinds). */
#define MOE_ROPE_PLAIN 0
#define MOE_ROPE_LINEAR 1
#define MOE_ROPE_BASE 2
#define MOE_ROPE_PARTS 3
moe_status moe_rope_freqs(int32_t kind, int32_t rot_dim, double base, double factor,
                          double orig_len, double turns_lo, double turns_hi, double* freqs,
                          float* scale);

/* Norms of queries and keys per head, their rotation by position, and the
 * cache's new tokens, in one pass over the projections' output:
 *   qkv: bf16 rows of n_q query heads, n_kv key heads and n_kv value heads, D
 *   each, qkv_stride elements apart.  For a query or key head x at position p:
 *     z = x / sqrt(mean(x^2) + eps) * w     (with a norm weight w; else z = x)
 *     (u, v) of pair i -> (u c - v s, v c + u s), c, s = rope_scale * cos, sin
 *     of p * inv_freq[i],
 *   keys in fp64, rounded to fp32 and then to bf16, so that the codes in the
 *   cache do not depend on the order of a sum; queries, which meet the matrix
 *   units anyway, in fp32 (sine and cosine from fp64), rounded to bf16 once.
 *   q_out: bf16 [T] rows of n_q * D, q_stride apart; k_out: the same with
 *   n_kv * D, or NULL (for moe_attn_prompt, whose values may stay in qkv).
 *   q_out and k_out may be the query and key parts of qkv itself (the same
 *   addresses and stride); other overlaps are refused.
 *   Keys and values go into the cache at the rows' tokens.  Rows at or behind
 *   row_start[n_seq] are left as they are.  pos: device int32 [T], the rows'
 *   rotary positions, or NULL: the token's index in its sequence.  The page
 *   table decides where tokens go: two tokens of a call must not share a place.
 * Strides: multiples of 8 elements, the row's width or more; pointers 16-byte
 * aligned. */
moe_status moe_kv_append(const moe_kv_cache* c, const moe_qkv_desc* p, const moe_seq_batch* s,
                         const uint16_t* qkv, int64_t qkv_stride, int64_t T, const int32_t* pos,
                         uint16_t* q_out, int64_t q_stride, uint16_t* k_out, int64_t k_stride,
                         hipStream_t stream);

/* The cache read back as bf16 rows (rounded once where the format's values
 * need it), for prompt chunks that attend to a cached prefix.  Token j of
 * sequence b, first[b] <= j < kv_len[b], goes to row out_start[b] + j -
 * first[b] of k_out and v_out (n_kv * D wide), as long as there is such a token
 * (0 <= j) and row (0 <= row < R) and the row is below out_start[b+1].  first:
 * device int32 [n_seq], or NULL: 0.  out_start: device int32 [n_seq + 1],
 * ascending.  k_out or v_out may be NULL; they must not overlap.  row_start of
 * the batch is not read. */
moe_status moe_kv_read(const moe_kv_cache* c, const moe_seq_batch* s, const int32_t* first,
                       const int32_t* out_start, int64_t R, uint16_t* k_out, int64_t k_stride,
                       uint16_t* v_out, int64_t v_stride, hipStream_t stream);

/* Attention of a step's rows over the cache (their own tokens included): one
 * row per sequence in a decode step, a few in a verification batch; any number
 * is right.  Query head h uses key/value head h / (n_q / n_kv):
 *   s_j = scale * q . k_j over the tokens j at or before the row's own,
 *   out = sum_j softmax(s)_j v_j,
 * sums and softmax in fp32; out bf16, zero for a row that sees no token.  The
 * keys, values and softmax weights meet the matrix units as fp16 (block
 * formats; the query rows scaled by a power of two each; a weight below 2^-32
 * of the largest counts as none) or bf16 (16-bit cache).  What a row does not
 * see has no influence on it, also if it is NaN or infinite.
 * q, out: bf16 [T] rows of n_q * D (out may be q, with the same stride; other
 * overlaps are refused).  max_len: the longest
 * kv_len expected; it decides how the work is split, never the result's
 * validity (0: max_pages * page_tokens).  ws: moe_attn_workspace_bytes of the
 * same cache, heads and n_seq, with this T and max_len or larger ones; nothing
 * in it needs to start at zero.  Calls that may overlap need workspaces of
 * their own. */
size_t moe_attn_workspace_bytes(const moe_kv_cache* c, int32_t n_q, int32_t n_seq, int64_t T,
                                int64_t max_len);
moe_status moe_attn_decode(const moe_kv_cache* c, const moe_seq_batch* s, int32_t n_q,
                           const uint16_t* q, int64_t q_stride, int64_t T, int64_t max_len,
                           float scale, uint16_t* out, int64_t out_stride, void* ws,
                           size_t ws_bytes, hipStream_t stream);

/* The same attention for steps with many rows of a sequence: a prompt's chunks
 * behind what is cached of it, alone or beside other slots' decode steps, long
 * verification batches.  Arguments, types, results for rows that see nothing, bad
 * pages and rows outside the sequences as for moe_attn_decode; the two differ in how
 * they cut the work: here a cached token is decoded once for all rows of a tile
 * of 256 (row, head) pairs (heads of 256: 128).  Operands as there: keys
 * and values of MOE_FMT_Q8_0, code times scale, are rounded once to fp16 (2^-11
 * of one), those of MOE_FMT_NVFP4 are fp16 values as they are.
 * Which is faster: moe_attn_decode for a few rows a sequence (32 query and 4
 * key/value heads of 128: up to some 128 behind 8192 tokens) and behind short
 * caches; this call for more of them behind a long cache, alone or among decode
 * rows; moe_kv_read and moe_attn_prompt, where there is memory for the 16-bit
 * keys and values, for thousands of rows of a sequence.
 * ws: moe_attn_chunk_workspace_bytes of the same cache, heads and n_seq, with
 * this T and max_len or larger ones. */
size_t moe_attn_chunk_workspace_bytes(const moe_kv_cache* c, int32_t n_q, int32_t n_seq, int64_t T,
                                      int64_t max_len);
moe_status moe_attn_chunk(const moe_kv_cache* c, const moe_seq_batch* s, int32_t n_q,
                          const uint16_t* q, int64_t q_stride, int64_t T, int64_t max_len,
                          float scale, uint16_t* out, int64_t out_stride, void* ws,
                          size_t ws_bytes, hipStream_t stream);

/* Causal attention over whole prompts (or chunks of them), packed: sequence b
 * has the query rows q_start[b] .. q_start[b+1]-1 and the key and value rows
 * kv_start[b] .. kv_start[b+1]-1, the queries being the last of the keys'
 * positions: query i of n sees keys j <= L - n + i of L.  The same formula,
 * rounding and empty rows as moe_attn_decode, with bf16 operands.
 * q_start, kv_start: device int32 [n_seq + 1], ascending; kv_start NULL: the
 * queries' own.  q: bf16 [T] rows of n_q * D; k, v: bf16 [Tk] rows of n_kv * D;
 * out: bf16 [T] rows of n_q * D (may be q, with the same stride; other overlaps
 * are refused).  k_stride and
 * v_stride: at most 2^24.  Rows outside
 * the sequences are left as they are; indices are held inside T and Tk: of a
 * sequence with rows outside 0..T those inside are answered, one with keys
 * outside 0..Tk has NaN rows. */
moe_status moe_attn_prompt(int32_t n_q, int32_t n_kv, int32_t D, int32_t n_seq,
                           const int32_t* q_start, const int32_t* kv_start, int64_t T, int64_t Tk,
                           const uint16_t* q, int64_t q_stride, const uint16_t* k,
                           int64_t k_stride, const uint16_t* v, int64_t v_stride, float scale,
                           uint16_t* out, int64_t out_stride, hipStream_t stream);

/* ------------------------------------------------------------------------ */
/* Around the attention and the experts: norms and dense projections         */
/* ------------------------------------------------------------------------ */
/*
 * The pages keep a pack's dense projections in a format of their own beside the
 * experts' (basalt.jgulfo.com, "All the numbers", the engine notes); the pages
 * give no formula.  Here they are 4-bit microscaled matrices, which the matrix
 * units take as they are, and the rows that meet them are 4- or 8-bit
 * microscaled: along a row, each 32 values have one scale, a power of two.
 *   MOE_FMT_MXFP4  E2M1 codes, element 2i in the low half of byte i
 *   MOE_FMT_MXFP8  E4M3 codes, one a byte
 * Rows of K elements: codes u8 [T][K/2] or [T][K], scales u8 [T][K/32], dense;
 * value = code * 2^(s - 127), s = 255 (NaN) making its 32 values NaN.
 * Quantisation of the 32 bf16 values of a block whose largest magnitude is A:
 *   s = max(floor(log2 A) - (2 or 8), -127) + 127, code = the nearest of
 *   x / 2^(s - 127), ties to the even code, held to +-6 or +-448
 * (the block format of the Open Compute Project's microscaling specification);
 * A = 0 gives s = 0, an infinity or a NaN in the block s = 255 and codes 0.
 *
 * Shapes: K and H multiples of 128; H up to 16384, K up to 32768, N 1..2^20,
 * T up to 2^20.  Strides: multiples of 8 elements, the row's width or more;
 * pointers 16-byte aligned.
 */
#define MOE_FMT_MXFP4 7
#define MOE_FMT_MXFP8 8

/* The residual's addition and the root-mean-square norm, in one pass over the
 * rows:
 *   h = bf16(x + residual)  (x without a residual),
 *   z = bf16(h / sqrt(mean(h^2) + eps) * weight),
 * the sum of squares and the products in fp64 (so that codes do not depend on
 * the order of a sum), rounded to fp32 and then to bf16; the additions in fp32.
 * x, residual (or NULL): bf16 [T][H]; weight: fp32 [H].
 * sum: h, bf16 [T][H], or NULL; out: z, bf16 [T][H], or NULL; codes, scales: z
 * in fmt (MOE_FMT_MXFP4 or _MXFP8), or NULL with fmt 0: what moe_mx_quant makes
 * of out.  sum and out may each be x or residual (the same address and stride);
 * other overlaps are refused.  At least one output is given. */
moe_status moe_add_norm(int32_t H, int64_t T, const uint16_t* x, int64_t x_stride,
                        const uint16_t* residual, int64_t residual_stride, const float* weight,
                        float eps, uint16_t* sum, int64_t sum_stride, uint16_t* out,
                        int64_t out_stride, int32_t fmt, uint8_t* codes, uint8_t* scales,
                        hipStream_t stream);

/* bf16 rows [T][K] in fmt (MOE_FMT_MXFP4 or MOE_FMT_MXFP8). */
moe_status moe_mx_quant(int32_t fmt, int32_t K, int64_t T, const uint16_t* x, int64_t x_stride,
                        uint8_t* codes, uint8_t* scales, hipStream_t stream);

/* A dense projection's weights W[N][K] in MOE_FMT_MXFP4, packed once at load
 * from codes u8 [N][K/2] and scales u8 [N][K/32] (moe_mx_quant makes them from
 * bf16 rows) into `packed`, moe_mx_matrix_bytes(N, K) bytes, 256-byte aligned.
 * Host struct holding device pointers. */
typedef struct moe_mx_matrix {
  int32_t N, K;
  const void* packed;
  const float* bias;  /* fp32 [N], or NULL */
} moe_mx_matrix;

/* Bytes of a packed matrix (a multiple of 256); 0 if unsupported. */
size_t moe_mx_matrix_bytes(int32_t N, int32_t K);
moe_status moe_mx_pack(int32_t N, int32_t K, const uint8_t* codes, const uint8_t* scales,
                       void* packed, hipStream_t stream);

/* y[t][n] = sum_k a[t][k] W[n][k] + bias[n], rows a in fmt as codes and scales;
 * y: [T] rows of N, y_stride apart, of y_dtype (MOE_DTYPE_F32 or _BF16).  The
 * products meet the matrix units as codes and are summed in fp32; with
 * MOE_FMT_MXFP8 rows the units cut each product to a multiple of 2^-13 of the
 * power of two of the largest one among its 8 neighbours (elements 8i..8i+7) on
 * the way (a few 1e-6 of the result, norm over norm, for normal rows).  The
 * result is rounded once.  A NaN scale makes the outputs that meet it NaN.  The
 * order of the sums depends on T, N and K, not on scheduling. */
moe_status moe_mx_linear(const moe_mx_matrix* w, int32_t fmt, const uint8_t* codes,
                         const uint8_t* scales, int64_t T, void* y, int64_t y_stride,
                         int32_t y_dtype, hipStream_t stream);

/* moe_mx_quant of bf16 rows x [T][K], then moe_mx_linear, with the same results
 * bit for bit; a few rows are quantised inside the product's launch.  ws:
 * moe_mx_workspace_bytes of this fmt and K, with this T or a larger one; nothing
 * in it needs to start at zero.  Calls that may overlap need workspaces of
 * their own. */
size_t moe_mx_workspace_bytes(int32_t fmt, int32_t K, int64_t T);
moe_status moe_mx_linear_rows(const moe_mx_matrix* w, int32_t fmt, const uint16_t* x,
                              int64_t x_stride, int64_t T, void* y, int64_t y_stride,
                              int32_t y_dtype, void* ws, size_t ws_bytes, hipStream_t stream);

/* ------------------------------------------------------------------------ */
/* Optional cold-expert tier: pinned host RAM -> HBM slots                   */
/* ------------------------------------------------------------------------ */
/*
 * Experts that do not fit the GPU memory budget stay in system RAM and are
 * copied in when a token routes to them (aiopssre.com, "Experts can move
 * without becoming free"); the most-routed experts are the ones kept in GPU
 * memory, with system RAM as the last tier (basalt.jgulfo.com, "Expert
 * tiers"); the resident set follows the usage histogram, so it moves as usage
 * changes (basalt.jgulfo.com, FAQ).  One GPU only: no peer-GPU tier.
 *
 * Per layer l: R resident slots (experts chosen by moe_tier_rebalance) in the
 * caller's HBM pool, plus S staging slots shared by all layers.  Before the
 * experts of layer l run, moe_tier_prepare copies the step's active list to
 * the host (the one host synchronization per layer), copies every active
 * expert that is not resident from pinned host memory into a staging slot on
 * the copy stream, writes the layer's device expert table (moe_expert_ref [E])
 * and makes the compute stream wait for those copies.  moe_expert_ffn then
 * reads every expert through that table, so a tiered step computes exactly
 * (bit for bit) what the same step computes with every expert resident.
 * Entries of inactive, non-resident experts are set to blob = NULL.
 *
 * Copies: when every host blob is mapped for the device (hipHostMalloc
 * memory is), one kernel on the copy stream moves a call's experts and the
 * table, reading the pinned memory directly (expert-sized pieces then move at
 * the large-transfer rate); otherwise one runtime copy per expert is issued.
 *
 * Ownership: host blobs (pinned, e.g. hipHostMalloc), the HBM pool, the
 * device tables and both streams belong to the caller and must outlive the
 * tier.  The tier owns host metadata, a few pinned bytes for the active
 * list, the table staging and the copy list, two events and the device state
 * of moe_tier_prepare_async (allocated at create, freed by destroy).  A tier
 * is not thread-safe.
 */
typedef struct moe_tier_desc {
  int32_t L;                      /* layers */
  int32_t E;                      /* experts per layer */
  int32_t resident_per_layer;     /* R (0 <= R <= E) */
  int32_t staging_slots;          /* S: most misses one layer step may have (<= E) */
  size_t expert_bytes;            /* moe_expert_blob_bytes(...) of every expert */
  const void* const* host_blobs;  /* host array [L*E]: pinned host address of blob (l, e) */
  const moe_expert_ref* scales;   /* host array [L*E]: ts_gate/ts_up/ts_down of (l, e); blob ignored */
  void* hbm_pool;                 /* device, 256-aligned, >= (L*R + S) * expert_bytes */
  size_t hbm_pool_bytes;
  hipStream_t copy_stream;        /* side stream for the H2D copies */
} moe_tier_desc;

typedef struct moe_tier_stats {
  uint64_t hits;          /* active experts found resident */
  uint64_t misses;        /* active experts copied from host */
  uint64_t h2d_bytes;     /* bytes copied host -> HBM (misses and promotions) */
  uint64_t promotions;    /* experts moved into a resident slot by rebalance */
  uint64_t prepares;
  uint64_t rebalances;
} moe_tier_stats;

typedef struct moe_tier moe_tier;

/* Validates (budget: MOE_ERR_BUDGET if the pool is below (L*R + S) slots)
 * and creates the tier with no expert resident. */
moe_status moe_tier_create(const moe_tier_desc* desc, moe_tier** out);

/* After moe_bucket of layer `layer` on `compute`: stage this step's missing
 * experts and fill table_dev (device moe_expert_ref [E]).  Blocks the host
 * until the active list of this step is known (one event wait).  Returns
 * MOE_ERR_BUDGET if the step has more misses than staging slots. */
moe_status moe_tier_prepare(moe_tier* t, int32_t layer, const moe_buckets* b,
                            moe_expert_ref* table_dev, hipStream_t compute);

/* The same on the device, with no host synchronization: two launches on
 * `compute`, a planning kernel (reads the step's active list and the tier's
 * device copy of the layer's resident slots, assigns the misses staging slots
 * in active-list order, writes table_dev and the copy list) and the copy
 * kernel, which reads the pinned host blobs directly.  So a caller can
 * enqueue many layers ahead, or capture them in a graph (with
 * moe_tier_rebalance, which synchronizes, outside it).  Results equal those
 * of moe_tier_prepare bit for bit.  The tier's device state (base tables,
 * blob addresses, copy list, counters: about 36 bytes per expert of every
 * layer) is allocated once by moe_tier_create, when the host blobs are mapped
 * for the device; otherwise this call returns MOE_ERR_UNSUPPORTED.  Staging
 * must hold every possible miss: MOE_ERR_BUDGET, before any launch, if
 * min(E, b->T_max * b->k) > S.  Hit and miss counts are kept on the device and
 * added by moe_tier_stats_get (synchronize `compute` before reading them).
 * This call and moe_tier_prepare share the staging slots: do not interleave
 * them on different streams. */
moe_status moe_tier_prepare_async(moe_tier* t, int32_t layer, const moe_buckets* b,
                                  moe_expert_ref* table_dev, hipStream_t compute);

/* Make the R most used experts of `layer` (hist_dev: device uint32 [E], as
 * updated by moe_expert_hist; ties to the lower index) resident, copying the
 * newcomers into freed slots.  Synchronizes `compute` (reads the histogram). */
moe_status moe_tier_rebalance(moe_tier* t, int32_t layer, const uint32_t* hist_dev,
                              hipStream_t compute);

/* Host copy of the counters; resident expert list of a layer (host int32 [R],
 * -1 for an empty slot) when resident_out is not NULL. */
moe_status moe_tier_stats_get(const moe_tier* t, moe_tier_stats* out, int32_t layer,
                              int32_t* resident_out);

/* Releases host metadata and events (not the caller's buffers). */
void moe_tier_destroy(moe_tier* t);

#ifdef __cplusplus
}
#endif

#endif /* MOE_H */
