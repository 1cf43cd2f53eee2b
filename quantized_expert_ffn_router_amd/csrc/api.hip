// api.hip -- the extern "C" entry points of libmoe: argument validation
// (before any launch), error reporting and kernel dispatch.
#include <math.h>
#include <stdarg.h>
#include <stdio.h>
#include <string.h>

#include <algorithm>
#include <mutex>
#include <utility>

#include "attn_common.h"
#include "gemv_common.h"
#include "mx.h"

// Workspace of moe_expert_ffn_noalloc: one copy per GPU, held until the
// process ends.  Host code never passes this name to a kernel or a copy (on
// the host it is only a stand-in for the symbol); it uses the device address
// that hipGetSymbolAddress returns for the current device (scratch_ptr).
constexpr size_t kScratchBytes = MOE_NOALLOC_WORKSPACE_BYTES;
static __device__ __align__(256) uint8_t scratch[kScratchBytes];

namespace {

thread_local char g_err[512] = "";

moe_status fail(moe_status st, const char* fmt, ...) {
  va_list ap;
  va_start(ap, fmt);
  vsnprintf(g_err, sizeof(g_err), fmt, ap);
  va_end(ap);
  return st;
}

moe_status hip_status(const char* where, hipError_t e) {
  if (e == hipSuccess) return MOE_OK;
  return fail(MOE_ERR_HIP, "%s: %s", where, hipGetErrorString(e));
}

#define CHECK_PTR(p, where) \
  if (!(p)) return fail(MOE_ERR_INVALID_ARG, "%s: %s is NULL", where, #p)

moe_status check_shape(int E, int k, int H, int I, int fmt_gu, int fmt_down, const char* where) {
  if (E < 1 || k < 1 || H < 1 || I < 1)
    return fail(MOE_ERR_INVALID_ARG, "%s: E=%d k=%d H=%d I=%d must be positive", where, E, k, H, I);
  if (k > E) return fail(MOE_ERR_INVALID_ARG, "%s: k=%d > E=%d", where, k, E);
  if (E > 1024) return fail(MOE_ERR_UNSUPPORTED, "%s: E=%d > 1024", where, E);
  if (k > 64) return fail(MOE_ERR_UNSUPPORTED, "%s: k=%d > 64", where, k);
  if (H % 128 != 0 || H > 8192)
    return fail(MOE_ERR_UNSUPPORTED, "%s: H=%d must be a multiple of 128 and <= 8192", where, H);
  if (fmt_gu != MOE_FMT_NVFP4)
    return fail(MOE_ERR_UNSUPPORTED, "%s: gate/up format %d (only NVFP4)", where, fmt_gu);
  if (fmt_down == MOE_FMT_NVFP4 || fmt_down == MOE_FMT_Q8_0) {
    if (I % 128 != 0 || I > 8192)
      return fail(MOE_ERR_UNSUPPORTED, "%s: I=%d must be a multiple of 128 and <= 8192", where, I);
  } else if (fmt_down == MOE_FMT_Q6K || fmt_down == MOE_FMT_IQ3G || fmt_down == MOE_FMT_IQ1G) {
    if (I % 256 != 0 || I > 8192)
      return fail(MOE_ERR_UNSUPPORTED,
                  "%s: I=%d must be a multiple of 256 and <= 8192 for %s", where, I,
                  fmt_down == MOE_FMT_Q6K ? "Q6_K" : (fmt_down == MOE_FMT_IQ3G ? "IQ3G" : "IQ1G"));
  } else {
    return fail(MOE_ERR_UNSUPPORTED, "%s: down format %d", where, fmt_down);
  }
  return MOE_OK;
}

moe_status check_layer(const moe_layer_desc* L, const char* where) {
  CHECK_PTR(L, where);
  moe_status st = check_shape(L->E, L->k, L->H, L->I, L->fmt_gate_up, L->fmt_down, where);
  if (st != MOE_OK) return st;
  if (L->renormalize != 0 && L->renormalize != 1)
    return fail(MOE_ERR_INVALID_ARG, "%s: renormalize=%d must be 0 or 1", where, L->renormalize);
  if (L->ffn_mode != MOE_FFN_AUTO && L->ffn_mode != MOE_FFN_GEMV && L->ffn_mode != MOE_FFN_GEMM)
    return fail(MOE_ERR_INVALID_ARG, "%s: ffn_mode=%d", where, L->ffn_mode);
  return MOE_OK;
}

moe_status check_buckets(const moe_layer_desc* L, const moe_buckets* b, int64_t T,
                         const char* where) {
  CHECK_PTR(b, where);
  if (b->E != L->E || b->k != L->k)
    return fail(MOE_ERR_INVALID_ARG, "%s: buckets carved for E=%d k=%d, layer has E=%d k=%d", where,
                b->E, b->k, L->E, L->k);
  if (T > b->T_max)
    return fail(MOE_ERR_WORKSPACE, "%s: T=%lld exceeds bucket capacity %lld", where, (long long)T,
                (long long)b->T_max);
  if (!b->counts || !b->offsets || !b->sorted_asg || !b->asg_pos || !b->active || !b->n_active)
    return fail(MOE_ERR_INVALID_ARG, "%s: bucket field is NULL (use moe_buckets_carve)", where);
  return MOE_OK;
}

constexpr int64_t kMaxT = (int64_t)1 << 24;

moe_status check_T(int64_t T, int k, const char* where) {
  if (T < 0) return fail(MOE_ERR_INVALID_ARG, "%s: T=%lld < 0", where, (long long)T);
  if (T > kMaxT || T * k > INT32_MAX)
    return fail(MOE_ERR_UNSUPPORTED, "%s: T=%lld too large", where, (long long)T);
  return MOE_OK;
}

// Workspace of moe_expert_ffn: h (bf16 [T*k][I], both paths), then for the
// grouped GEMM an fp16 copy of x ([T][H]), its row scales ([T]) and the tile list.
struct FfnWs {
  size_t h, xh, xscale, tiles, total;
};
FfnWs ffn_ws_layout(const moe_layer_desc* L, int64_t T) {
  const size_t A = (size_t)T * L->k;
  FfnWs w;
  w.h = 0;
  w.xh = moe::align_up(A * (size_t)L->I * sizeof(uint16_t));
  w.xscale = w.xh + moe::align_up((size_t)T * L->H * sizeof(uint16_t));
  w.tiles = w.xscale + moe::align_up((size_t)T * sizeof(float));
  w.total = w.tiles + moe::gemm_tiles_bytes(L->E, (int64_t)A);
  return w;
}
size_t ffn_ws(const moe_layer_desc* L, int64_t T) { return ffn_ws_layout(L, T).total; }

// The grouped GEMM needs 256-column down tiles and 32-bit element offsets
// of the token rows (x: T*H values) and of h (T*k*I values).
bool gemm_fits(const moe_layer_desc* L, int64_t T) {
  return L->H % 256 == 0 && (uint64_t)T * (uint64_t)L->H <= UINT32_MAX &&
         (uint64_t)T * (uint64_t)L->k * (uint64_t)L->I <= UINT32_MAX;
}

// Grouped GEMM once experts average >= 16 tokens (and the batch is not a
// decode step); dequant-fused GEMV otherwise.
// Batches of 2 to 8 tokens run the down projection and the combine as one
// kernel in moe_layer_forward (graph-replayed steps: batch 8 39.0 against
// 41.8 us, batch 4 27.7 against 29.5; at batch 1 its 32 workgroups pull
// each CU's 221 KB of expert rows too slowly, 20.0 against 19.2 us, and at
// batch 16 the experts that several tokens share are read once per token).
constexpr int64_t kDownCombineMinT = 2, kDownCombineMaxT = 8;

bool use_gemm(const moe_layer_desc* L, int64_t T) {
  if (L->ffn_mode == MOE_FFN_GEMV) return false;
  if (L->ffn_mode == MOE_FFN_GEMM) return true;
  return T > 64 && T * L->k >= 16 * (int64_t)L->E && gemm_fits(L, T);
}

}  // namespace

namespace moe {
moe_status tier_fail(moe_status st, const char* fmt, ...) {
  va_list ap;
  va_start(ap, fmt);
  vsnprintf(g_err, sizeof(g_err), fmt, ap);
  va_end(ap);
  return st;
}
}  // namespace moe

extern "C" {

int moe_abi_version(void) { return MOE_ABI_VERSION; }

const char* moe_last_error(void) { return g_err; }

size_t moe_expert_blob_bytes(int32_t H, int32_t I, int32_t fmt_gate_up, int32_t fmt_down) {
  if (check_shape(1, 1, H, I, fmt_gate_up, fmt_down, "moe_expert_blob_bytes") != MOE_OK) return 0;
  return moe::blob_layout(H, I, fmt_down).total;
}

moe_status moe_pack_experts(int32_t E, int32_t H, int32_t I, int32_t fmt_gate_up,
                            int32_t fmt_down, const uint8_t* gate_q, const uint8_t* gate_s,
                            const uint8_t* up_q, const uint8_t* up_s, const uint8_t* down_q,
                            const uint8_t* down_s, void* blobs, size_t blob_stride,
                            hipStream_t stream) {
  const char* W = "moe_pack_experts";
  moe_status st = check_shape(E, 1, H, I, fmt_gate_up, fmt_down, W);
  if (st != MOE_OK) return st;
  CHECK_PTR(gate_q, W); CHECK_PTR(gate_s, W); CHECK_PTR(up_q, W); CHECK_PTR(up_s, W);
  CHECK_PTR(down_q, W); CHECK_PTR(blobs, W);
  if (fmt_down == MOE_FMT_NVFP4) CHECK_PTR(down_s, W);
  const moe::BlobLayout lay = moe::blob_layout(H, I, fmt_down);
  if (blob_stride < lay.total || blob_stride % moe::kAlign != 0)
    return fail(MOE_ERR_INVALID_ARG, "%s: blob_stride %zu must be >= %zu and a multiple of 256", W,
                blob_stride, lay.total);
  uint8_t* d = (uint8_t*)blobs;
  const size_t gu_q = (size_t)I * H / 2, gu_s = (size_t)I * H / 16;
  hipError_t e;
  // gate / up: N = I rows, K = H
  e = moe::launch_pack_granules(gate_q, E, gu_q, I, H / 32, 16, H / 2, 1, 16, 0, d + lay.gate_q, blob_stride, stream);
  if (e == hipSuccess) e = moe::launch_pack_granules(gate_s, E, gu_s, I, H / 128, 8, H / 16, 1, 8, 0, d + lay.gate_s, blob_stride, stream);
  if (e == hipSuccess) e = moe::launch_pack_granules(up_q, E, gu_q, I, H / 32, 16, H / 2, 1, 16, 0, d + lay.up_q, blob_stride, stream);
  if (e == hipSuccess) e = moe::launch_pack_granules(up_s, E, gu_s, I, H / 128, 8, H / 16, 1, 8, 0, d + lay.up_s, blob_stride, stream);
  if (e != hipSuccess) return hip_status(W, e);
  if (fmt_down == MOE_FMT_NVFP4) {
    // down: N = H rows, K = I
    e = moe::launch_pack_granules(down_q, E, (size_t)H * I / 2, H, I / 32, 16, I / 2, 1, 16, 0, d + lay.down_q, blob_stride, stream);
    if (e == hipSuccess) e = moe::launch_pack_granules(down_s, E, (size_t)H * I / 16, H, I / 128, 8, I / 16, 1, 8, 0, d + lay.down_s, blob_stride, stream);
  } else if (fmt_down == MOE_FMT_Q8_0) {
    // 34-byte blocks: codes in two 16-byte granules per block, the 4 scales of
    // a 128-element group gathered into one 8-byte granule
    const size_t row = (size_t)(I / 32) * 34, ex = (size_t)H * row;
    e = moe::launch_pack_granules(down_q, E, ex, H, I / 16, 16, row, 2, 34, 2, d + lay.down_q, blob_stride, stream);
    if (e == hipSuccess) e = moe::launch_pack_granules(down_q, E, ex, H, I / 128, 2, row, 1, 34, 0, d + lay.down_s, blob_stride, stream, 4);
    if (e == hipSuccess) e = moe::launch_down_exponent(down_q, E, H, I, fmt_down, d + lay.down_meta, blob_stride, stream);
  } else if (fmt_down == MOE_FMT_IQ3G) {
    // 102-byte superblocks: grid indices in 16-byte granules of 64 elements,
    // sign bits in 16-byte granules of 128 elements, and d with the 4-bit
    // multipliers (6 bytes) in an 8-byte granule per superblock
    const size_t row = (size_t)(I / 256) * moe::kIq3gBlockBytes, ex = (size_t)H * row;
    e = moe::launch_pack_granules(down_q, E, ex, H, I / 64, 16, row, 4, moe::kIq3gBlockBytes, 6, d + lay.down_q, blob_stride, stream);
    if (e == hipSuccess) e = moe::launch_pack_granules(down_q, E, ex, H, I / 128, 16, row, 2, moe::kIq3gBlockBytes, 70, d + lay.down_s, blob_stride, stream);
    if (e == hipSuccess) e = moe::launch_pack_granules(down_q, E, ex, H, I / 256, 6, row, 1, moe::kIq3gBlockBytes, 0, d + lay.down_sc, blob_stride, stream, 1, 2);
    if (e == hipSuccess) e = moe::launch_down_exponent(down_q, E, H, I, fmt_down, d + lay.down_meta, blob_stride, stream);
  } else if (fmt_down == MOE_FMT_IQ1G) {
    // 46-byte superblocks: index low bytes in 16-byte granules of 128
    // elements, their 2-bit high parts in 4-byte granules of 128 elements,
    // and d with the 4-bit multipliers (6 bytes) in an 8-byte granule per
    // superblock
    const size_t row = (size_t)(I / 256) * moe::kIq1gBlockBytes, ex = (size_t)H * row;
    e = moe::launch_pack_granules(down_q, E, ex, H, I / 128, 16, row, 2, moe::kIq1gBlockBytes, 6, d + lay.down_q, blob_stride, stream);
    if (e == hipSuccess) e = moe::launch_pack_granules(down_q, E, ex, H, I / 128, 4, row, 2, moe::kIq1gBlockBytes, 38, d + lay.down_s, blob_stride, stream);
    if (e == hipSuccess) e = moe::launch_pack_granules(down_q, E, ex, H, I / 256, 6, row, 1, moe::kIq1gBlockBytes, 0, d + lay.down_sc, blob_stride, stream, 1, 2);
    if (e == hipSuccess) e = moe::launch_down_exponent(down_q, E, H, I, fmt_down, d + lay.down_meta, blob_stride, stream);
  } else {
    const size_t row = (size_t)(I / 256) * 210, ex = (size_t)H * row;
    e = moe::launch_pack_granules(down_q, E, ex, H, I / 32, 16, row, 8, 210, 0, d + lay.down_ql, blob_stride, stream);
    if (e == hipSuccess) e = moe::launch_pack_granules(down_q, E, ex, H, I / 64, 16, row, 4, 210, 128, d + lay.down_qh, blob_stride, stream);
    if (e == hipSuccess) e = moe::launch_pack_granules(down_q, E, ex, H, I / 256, 16, row, 1, 210, 192, d + lay.down_sc, blob_stride, stream);
    if (e == hipSuccess) e = moe::launch_pack_granules(down_q, E, ex, H, I / 256, 2, row, 1, 210, 208, d + lay.down_d, blob_stride, stream);
    if (e == hipSuccess) e = moe::launch_down_exponent(down_q, E, H, I, fmt_down, d + lay.down_meta, blob_stride, stream);
  }
  return hip_status(W, e);
}

size_t moe_buckets_bytes(int32_t E, int64_t T_max, int32_t k) {
  if (E < 1 || k < 1 || T_max < 0) return 0;
  size_t A = (size_t)T_max * k;
  return moe::align_up((size_t)E * 4) + moe::align_up((size_t)(E + 1) * 4) +
         moe::align_up(A * 4) * 2 + moe::align_up((size_t)E * 4) + moe::align_up(4);
}

moe_status moe_buckets_carve(void* buf, size_t bytes, int32_t E, int64_t T_max, int32_t k,
                             moe_buckets* out) {
  const char* W = "moe_buckets_carve";
  CHECK_PTR(buf, W);
  CHECK_PTR(out, W);
  if (E < 1 || k < 1 || T_max < 0)
    return fail(MOE_ERR_INVALID_ARG, "%s: E=%d k=%d T_max=%lld", W, E, k, (long long)T_max);
  if ((uintptr_t)buf % moe::kAlign != 0)
    return fail(MOE_ERR_INVALID_ARG, "%s: buffer not 256-byte aligned", W);
  size_t need = moe_buckets_bytes(E, T_max, k);
  if (bytes < need) return fail(MOE_ERR_WORKSPACE, "%s: %zu bytes < %zu needed", W, bytes, need);
  size_t A = (size_t)T_max * k;
  char* p = (char*)buf;
  out->counts = (uint32_t*)p; p += moe::align_up((size_t)E * 4);
  out->offsets = (int32_t*)p; p += moe::align_up((size_t)(E + 1) * 4);
  out->sorted_asg = (int32_t*)p; p += moe::align_up(A * 4);
  out->asg_pos = (int32_t*)p; p += moe::align_up(A * 4);
  out->active = (int32_t*)p; p += moe::align_up((size_t)E * 4);
  out->n_active = (int32_t*)p;
  out->T_max = T_max;
  out->E = E;
  out->k = k;
  return MOE_OK;
}

size_t moe_workspace_bytes(const moe_layer_desc* L, int64_t T_max) {
  if (check_layer(L, "moe_workspace_bytes") != MOE_OK || T_max < 0) return 0;
  size_t a = moe::bucket_ws_bytes(L->E, T_max * L->k);
  size_t b = ffn_ws(L, T_max);
  size_t w = a > b ? a : b;
  return w ? w : moe::kAlign;
}

moe_status moe_route(const moe_layer_desc* L, const uint16_t* x, int64_t T, float* logits,
                     int32_t* topk_idx, float* topk_w, hipStream_t stream) {
  const char* W = "moe_route";
  moe_status st = check_layer(L, W);
  if (st != MOE_OK) return st;
  if ((st = check_T(T, L->k, W)) != MOE_OK) return st;
  if (T == 0) return MOE_OK;
  CHECK_PTR(x, W); CHECK_PTR(logits, W); CHECK_PTR(topk_idx, W); CHECK_PTR(topk_w, W);
  CHECK_PTR(L->w_router, W);
  hipError_t e = moe::launch_router(x, T, L->H, L->w_router, L->router_bias, L->E, logits, stream);
  if (e == hipSuccess) e = moe::launch_topk(logits, T, L->E, L->k, L->renormalize, topk_idx, topk_w, stream);
  return hip_status(W, e);
}

moe_status moe_bucket(const moe_layer_desc* L, const int32_t* topk_idx, int64_t T,
                      const moe_buckets* b, void* ws, size_t ws_bytes, hipStream_t stream) {
  const char* W = "moe_bucket";
  moe_status st = check_layer(L, W);
  if (st != MOE_OK) return st;
  if ((st = check_T(T, L->k, W)) != MOE_OK) return st;
  if ((st = check_buckets(L, b, T, W)) != MOE_OK) return st;
  if (T == 0) return MOE_OK;
  CHECK_PTR(topk_idx, W);
  size_t need = moe::bucket_ws_bytes(L->E, T * L->k);
  if (need > 0) {
    CHECK_PTR(ws, W);
    if (ws_bytes < need) return fail(MOE_ERR_WORKSPACE, "%s: workspace %zu < %zu", W, ws_bytes, need);
  }
  return hip_status(W, moe::launch_bucket(topk_idx, T * L->k, L->E, b, ws, stream));
}

}  // extern "C"

namespace {

// Argument checks shared by moe_expert_ffn and moe_expert_ffn_noalloc.
moe_status ffn_check(const char* W, const moe_layer_desc* L, const uint16_t* x, int64_t T,
                     const moe_buckets* b, const void* y, int32_t y_dtype) {
  moe_status st = check_layer(L, W);
  if (st != MOE_OK) return st;
  if ((st = check_T(T, L->k, W)) != MOE_OK) return st;
  if ((st = check_buckets(L, b, T, W)) != MOE_OK) return st;
  if (y_dtype != MOE_DTYPE_F32 && y_dtype != MOE_DTYPE_BF16)
    return fail(MOE_ERR_INVALID_ARG, "%s: y_dtype=%d", W, y_dtype);
  if (T == 0) return MOE_OK;
  CHECK_PTR(x, W); CHECK_PTR(y, W); CHECK_PTR(L->experts, W);
  if (use_gemm(L, T) && !gemm_fits(L, T))
    return fail(MOE_ERR_UNSUPPORTED, "%s: grouped GEMM needs H %% 256 == 0, T*H and T*k*I < 2^32",
                W);
  return MOE_OK;
}

// The GEMV family's gate/up into h (bf16 [T*k][I], sorted order): 32-row
// slices for up to 16 tokens (it redoes the weight decode per token, which
// costs more than it saves once experts hold many tokens), else 64-row blocks.
hipError_t gemv_gateup_launch(const moe_layer_desc* L, const uint16_t* x, int64_t T,
                              const moe_buckets* b, int max_slots, uint16_t* h,
                              hipStream_t stream) {
  return (T <= 16 && moe::gemv_gateup32_fits(L))
             ? moe::launch_gemv_gateup32(L, x, b, max_slots, h, stream)
             : moe::launch_gemv_gateup(L, x, b, max_slots, h, stream);
}

// The FFN's launches (checks done, T > 0, ws holds ffn_ws(L, T) bytes).
moe_status ffn_launch(const char* W, const moe_layer_desc* L, const uint16_t* x, int64_t T,
                      const moe_buckets* b, void* y, int32_t y_dtype, void* ws,
                      hipStream_t stream) {
  if (use_gemm(L, T)) {
    const FfnWs w = ffn_ws_layout(L, T);
    char* c = (char*)ws;
    return hip_status(W, moe::launch_gemm_ffn(L, x, T, b, (uint16_t*)(c + w.h),
                                               (uint16_t*)(c + w.xh), (float*)(c + w.xscale),
                                               c + w.tiles, y, y_dtype, stream));
  }
  // Worst-case number of active experts; workgroups past n_active exit.
  const int max_slots = (int)((T * L->k < L->E) ? T * L->k : L->E);
  uint16_t* h = (uint16_t*)ws;  // bf16 [T*k][I], sorted order
  hipError_t e = gemv_gateup_launch(L, x, T, b, max_slots, h, stream);
  if (e == hipSuccess) e = moe::launch_gemv_down(L, h, b, max_slots, y, y_dtype, stream);
  return hip_status(W, e);
}

// Device address of `scratch` on each device, looked up on the first
// moe_expert_ffn_noalloc call made with that device current.
constexpr int kMaxDevices = 64;
std::once_flag g_scratch_once[kMaxDevices];
void* g_scratch_ptr[kMaxDevices];
hipError_t g_scratch_err[kMaxDevices];

moe_status scratch_ptr(const char* W, void** out) {
  int dev = 0;
  hipError_t e = hipGetDevice(&dev);
  if (e != hipSuccess) return hip_status(W, e);
  if (dev < 0 || dev >= kMaxDevices)
    return fail(MOE_ERR_UNSUPPORTED, "%s: device %d beyond %d", W, dev, kMaxDevices);
  std::call_once(g_scratch_once[dev], [dev] {
    void* p = nullptr;
    g_scratch_err[dev] = hipGetSymbolAddress(&p, HIP_SYMBOL(scratch));
    g_scratch_ptr[dev] = p;
  });
  if (g_scratch_err[dev] != hipSuccess) return hip_status(W, g_scratch_err[dev]);
  if (!g_scratch_ptr[dev]) return fail(MOE_ERR_HIP, "%s: no device address for the scratch", W);
  *out = g_scratch_ptr[dev];
  return MOE_OK;
}

}  // namespace

extern "C" {

moe_status moe_expert_ffn(const moe_layer_desc* L, const uint16_t* x, int64_t T,
                          const moe_buckets* b, void* y, int32_t y_dtype, void* ws,
                          size_t ws_bytes, hipStream_t stream) {
  const char* W = "moe_expert_ffn";
  moe_status st = ffn_check(W, L, x, T, b, y, y_dtype);
  if (st != MOE_OK || T == 0) return st;
  CHECK_PTR(ws, W);
  const size_t need = ffn_ws(L, T);
  if (ws_bytes < need) return fail(MOE_ERR_WORKSPACE, "%s: workspace %zu < %zu", W, ws_bytes, need);
  return ffn_launch(W, L, x, T, b, y, y_dtype, ws, stream);
}

moe_status moe_expert_ffn_noalloc(const moe_layer_desc* L, const uint16_t* x, int64_t T,
                                  const moe_buckets* b, void* y, int32_t y_dtype,
                                  hipStream_t stream) {
  const char* W = "moe_expert_ffn_noalloc";
  moe_status st = ffn_check(W, L, x, T, b, y, y_dtype);
  if (st != MOE_OK || T == 0) return st;
  const size_t need = ffn_ws(L, T);
  if (need > kScratchBytes)
    return fail(MOE_ERR_WORKSPACE,
                "%s: this call needs %zu bytes of workspace, above the library's static %zu "
                "(use moe_expert_ffn with a caller workspace)",
                W, need, kScratchBytes);
  void* ws = nullptr;
  if ((st = scratch_ptr(W, &ws)) != MOE_OK) return st;
  return ffn_launch(W, L, x, T, b, y, y_dtype, ws, stream);
}

moe_status moe_combine(const moe_layer_desc* L, const void* y, int32_t y_dtype,
                       const moe_buckets* b, const float* topk_w, int64_t T,
                       const uint16_t* residual, uint16_t* out, hipStream_t stream) {
  const char* W = "moe_combine";
  moe_status st = check_layer(L, W);
  if (st != MOE_OK) return st;
  if ((st = check_T(T, L->k, W)) != MOE_OK) return st;
  if ((st = check_buckets(L, b, T, W)) != MOE_OK) return st;
  if (y_dtype != MOE_DTYPE_F32 && y_dtype != MOE_DTYPE_BF16)
    return fail(MOE_ERR_INVALID_ARG, "%s: y_dtype=%d", W, y_dtype);
  if (T == 0) return MOE_OK;
  CHECK_PTR(y, W); CHECK_PTR(topk_w, W); CHECK_PTR(out, W);
  return hip_status(W, moe::launch_combine(y, y_dtype, b->asg_pos, topk_w, T, L->k, L->H, residual,
                                           out, stream));
}

moe_status moe_route_bucket(const moe_layer_desc* L, const uint16_t* x, int64_t T,
                            float* logits, int32_t* topk_idx, float* topk_w, const moe_buckets* b,
                            void* ws, size_t ws_bytes, uint32_t* hist, int32_t decay_shift,
                            int32_t unit_shift, hipStream_t stream) {
  const char* W = "moe_route_bucket";
  moe_status st = check_layer(L, W);
  if (st != MOE_OK) return st;
  if ((st = check_T(T, L->k, W)) != MOE_OK) return st;
  if ((st = check_buckets(L, b, T, W)) != MOE_OK) return st;
  if (hist && (decay_shift < 0 || decay_shift > 31 || unit_shift < 0 || unit_shift > 31))
    return fail(MOE_ERR_INVALID_ARG, "%s: shifts (%d, %d) must be in [0, 31]", W, decay_shift,
                unit_shift);
  if (T == 0) return MOE_OK;
  CHECK_PTR(x, W); CHECK_PTR(logits, W); CHECK_PTR(topk_idx, W); CHECK_PTR(topk_w, W);
  CHECK_PTR(L->w_router, W);
  const size_t need = moe::bucket_ws_bytes(L->E, T * L->k);
  if (need > 0) {
    CHECK_PTR(ws, W);
    if (ws_bytes < need) return fail(MOE_ERR_WORKSPACE, "%s: workspace %zu < %zu", W, ws_bytes, need);
  }
  hipError_t e = moe::launch_router(x, T, L->H, L->w_router, L->router_bias, L->E, logits, stream);
  if (e != hipSuccess) return hip_status(W, e);
  if (moe::gate_fused_fits(T, L->E, L->k))
    return hip_status(W, moe::launch_gate_fused(logits, T, L->E, L->k, L->renormalize, topk_idx,
                                                 topk_w, b, hist, decay_shift, unit_shift, stream));
  e = moe::launch_topk(logits, T, L->E, L->k, L->renormalize, topk_idx, topk_w, stream);
  if (e == hipSuccess) e = moe::launch_bucket(topk_idx, T * L->k, L->E, b, ws, stream);
  if (e == hipSuccess && hist)
    e = moe::launch_hist(b->counts, L->E, hist, decay_shift, unit_shift, stream);
  return hip_status(W, e);
}

moe_status moe_route_ffn(const moe_layer_desc* L, const uint16_t* x, int64_t T, float* logits,
                         int32_t* topk_idx, float* topk_w, const moe_buckets* b, uint32_t* hist,
                         int32_t decay_shift, int32_t unit_shift, void* y, int32_t y_dtype,
                         void* ws, size_t ws_bytes, hipStream_t stream) {
  const char* W = "moe_route_ffn";
  moe_status st = ffn_check(W, L, x, T, b, y, y_dtype);
  if (st != MOE_OK) return st;
  if (hist && (decay_shift < 0 || decay_shift > 31 || unit_shift < 0 || unit_shift > 31))
    return fail(MOE_ERR_INVALID_ARG, "%s: shifts (%d, %d) must be in [0, 31]", W, decay_shift,
                unit_shift);
  if (T == 0) return MOE_OK;
  CHECK_PTR(logits, W); CHECK_PTR(topk_idx, W); CHECK_PTR(topk_w, W); CHECK_PTR(ws, W);
  CHECK_PTR(L->w_router, W);
  const size_t need = ffn_ws(L, T);
  if (ws_bytes < need) return fail(MOE_ERR_WORKSPACE, "%s: workspace %zu < %zu", W, ws_bytes, need);
  if (use_gemm(L, T) || !moe::gemv_gate_gateup32_fits(L, T)) {  // the two calls
    st = moe_route_bucket(L, x, T, logits, topk_idx, topk_w, b, ws, ws_bytes, hist, decay_shift,
                          unit_shift, stream);
    if (st != MOE_OK) return st;
    return ffn_launch(W, L, x, T, b, y, y_dtype, ws, stream);
  }
  const int max_slots = (int)((T * L->k < L->E) ? T * L->k : L->E);
  uint16_t* h = (uint16_t*)ws;  // bf16 [T*k][I], sorted order
  hipError_t e = moe::launch_router(x, T, L->H, L->w_router, L->router_bias, L->E, logits, stream);
  if (e == hipSuccess)
    e = moe::launch_gemv_gate_gateup32(L, x, T, logits, topk_idx, topk_w, b, hist, decay_shift,
                                       unit_shift, max_slots, h, stream);
  if (e == hipSuccess) e = moe::launch_gemv_down(L, h, b, max_slots, y, y_dtype, stream);
  return hip_status(W, e);
}

moe_status moe_layer_forward(const moe_layer_desc* L, const uint16_t* x, int64_t T,
                             const uint16_t* residual, uint16_t* out, float* logits,
                             int32_t* topk_idx, float* topk_w, const moe_buckets* b,
                             uint32_t* hist, int32_t decay_shift, int32_t unit_shift, void* y,
                             int32_t y_dtype, void* ws, size_t ws_bytes, hipStream_t stream) {
  const char* W = "moe_layer_forward";
  moe_status st = ffn_check(W, L, x, T, b, y, y_dtype);
  if (st != MOE_OK) return st;
  if (hist && (decay_shift < 0 || decay_shift > 31 || unit_shift < 0 || unit_shift > 31))
    return fail(MOE_ERR_INVALID_ARG, "%s: shifts (%d, %d) must be in [0, 31]", W, decay_shift,
                unit_shift);
  if (T == 0) return MOE_OK;
  CHECK_PTR(out, W); CHECK_PTR(logits, W); CHECK_PTR(topk_idx, W); CHECK_PTR(topk_w, W);
  CHECK_PTR(ws, W); CHECK_PTR(L->w_router, W);
  const size_t need = ffn_ws(L, T);
  if (ws_bytes < need) return fail(MOE_ERR_WORKSPACE, "%s: workspace %zu < %zu", W, ws_bytes, need);
  if (use_gemm(L, T) || T < kDownCombineMinT || T > kDownCombineMaxT) {  // the two calls
    st = moe_route_ffn(L, x, T, logits, topk_idx, topk_w, b, hist, decay_shift, unit_shift, y,
                       y_dtype, ws, ws_bytes, stream);
    if (st != MOE_OK) return st;
    return moe_combine(L, y, y_dtype, b, topk_w, T, residual, out, stream);
  }
  const int max_slots = (int)((T * L->k < L->E) ? T * L->k : L->E);
  uint16_t* h = (uint16_t*)ws;  // bf16 [T*k][I], sorted order
  hipError_t e;
  if (moe::gemv_gate_gateup32_fits(L, T)) {
    e = moe::launch_router(x, T, L->H, L->w_router, L->router_bias, L->E, logits, stream);
    if (e == hipSuccess)
      e = moe::launch_gemv_gate_gateup32(L, x, T, logits, topk_idx, topk_w, b, hist, decay_shift,
                                         unit_shift, max_slots, h, stream);
  } else {
    st = moe_route_bucket(L, x, T, logits, topk_idx, topk_w, b, ws, ws_bytes, hist, decay_shift,
                          unit_shift, stream);
    if (st != MOE_OK) return st;
    e = gemv_gateup_launch(L, x, T, b, max_slots, h, stream);
  }
  if (e == hipSuccess)
    e = moe::launch_gemv_down_combine(L, h, T, topk_idx, b->asg_pos, topk_w, residual, out,
                                      stream);
  return hip_status(W, e);
}

moe_status moe_expert_hist(const moe_layer_desc* L, const moe_buckets* b, uint32_t* hist,
                           int32_t decay_shift, int32_t unit_shift, hipStream_t stream) {
  const char* W = "moe_expert_hist";
  moe_status st = check_layer(L, W);
  if (st != MOE_OK) return st;
  CHECK_PTR(b, W);
  if (b->E != L->E) return fail(MOE_ERR_INVALID_ARG, "%s: buckets carved for E=%d", W, b->E);
  CHECK_PTR(b->counts, W);
  CHECK_PTR(hist, W);
  if (decay_shift < 0 || decay_shift > 31 || unit_shift < 0 || unit_shift > 31)
    return fail(MOE_ERR_INVALID_ARG, "%s: shifts (%d, %d) must be in [0, 31]", W, decay_shift,
                unit_shift);
  return hip_status(W, moe::launch_hist(b->counts, L->E, hist, decay_shift, unit_shift, stream));
}

}  // extern "C"

// ---------------------------------------------------------------- attention side

namespace {

moe_status check_head(int D, const char* where) {
  if (D != 64 && D != 128 && D != 256)
    return fail(MOE_ERR_UNSUPPORTED, "%s: D=%d (64, 128 or 256)", where, D);
  return MOE_OK;
}

moe_status check_cache_shape(int fmt, int n_kv, int D, int P, const char* where) {
  if (fmt != MOE_FMT_NVFP4 && fmt != MOE_FMT_Q8_0 && fmt != MOE_FMT_BF16)
    return fail(MOE_ERR_UNSUPPORTED, "%s: cache format %d", where, fmt);
  if (n_kv < 1 || n_kv > 1024)
    return fail(MOE_ERR_UNSUPPORTED, "%s: n_kv=%d must be in 1..1024", where, n_kv);
  if (P != 32 && P != 64 && P != 128 && P != 256)
    return fail(MOE_ERR_UNSUPPORTED, "%s: page_tokens=%d (32, 64, 128 or 256)", where, P);
  return check_head(D, where);
}

moe_status check_aligned(const void* p, const char* name, const char* where) {
  if ((uintptr_t)p % 16 != 0)
    return fail(MOE_ERR_INVALID_ARG, "%s: %s is not 16-byte aligned", where, name);
  return MOE_OK;
}

moe_status check_rows(const void* p, int64_t stride, int64_t width, const char* name,
                      const char* where) {
  if (!p) return fail(MOE_ERR_INVALID_ARG, "%s: %s is NULL", where, name);
  if (stride < width || stride % 8 != 0)
    return fail(MOE_ERR_INVALID_ARG,
                "%s: %s stride %lld must be a multiple of 8 and at least %lld", where, name,
                (long long)stride, (long long)width);
  return check_aligned(p, name, where);
}

struct RowBlock {  // n rows of `width` 16-bit elements, stride apart
  const void* p;
  int64_t stride, width, n;
};

bool share_elements(RowBlock a, RowBlock b) {
  if (a.n < 1 || b.n < 1) return false;
  if ((uintptr_t)a.p > (uintptr_t)b.p) std::swap(a, b);
  const int64_t at = (int64_t)(((uintptr_t)b.p - (uintptr_t)a.p) / 2);  // of b's first row, from a's
  if ((__int128)at >= (__int128)(a.n - 1) * a.stride + a.width) return false;
  // rows inside one another's range: side by side at the same stride, or not known to be apart
  if (a.stride != b.stride) return true;
  const int64_t d = at % a.stride;
  return d < a.width || b.width > a.stride - d;
}

// An output's rows are not those of an input, except in the input's own place.
moe_status check_apart(RowBlock out, RowBlock in, bool in_place, const char* out_name,
                       const char* in_name, const char* where) {
  if (in_place && out.p == in.p && (out.stride == in.stride || out.n == 1)) return MOE_OK;
  if (!share_elements(out, in)) return MOE_OK;
  return fail(MOE_ERR_INVALID_ARG, "%s: %s overlaps %s%s", where, out_name, in_name,
              in_place ? " other than at its address and stride" : "");
}

moe_status check_cache(const moe_kv_cache* c, const char* where) {
  CHECK_PTR(c, where);
  moe_status st = check_cache_shape(c->fmt, c->n_kv, c->D, c->page_tokens, where);
  if (st != MOE_OK) return st;
  if (c->n_pages < 1) return fail(MOE_ERR_INVALID_ARG, "%s: n_pages=%d", where, c->n_pages);
  if (c->fmt == MOE_FMT_NVFP4 &&
      !(c->k_scale > 0.0f && isfinite(c->k_scale) && c->v_scale > 0.0f && isfinite(c->v_scale)))
    return fail(MOE_ERR_INVALID_ARG, "%s: k_scale=%g v_scale=%g must be finite and > 0", where,
                (double)c->k_scale, (double)c->v_scale);
  if (!c->pool) return fail(MOE_ERR_INVALID_ARG, "%s: pool is NULL", where);
  if ((uintptr_t)c->pool % moe::kAlign != 0)
    return fail(MOE_ERR_INVALID_ARG, "%s: pool not 256-byte aligned", where);
  return MOE_OK;
}

moe_status check_seqs(const moe_seq_batch* s, bool rows, const char* where) {
  CHECK_PTR(s, where);
  if (s->n_seq < 0 || s->n_seq > 65535)
    return fail(s->n_seq < 0 ? MOE_ERR_INVALID_ARG : MOE_ERR_UNSUPPORTED,
                "%s: n_seq=%d must be in 0..65535", where, s->n_seq);
  if (s->n_seq == 0) return MOE_OK;
  if (s->max_pages < 1) return fail(MOE_ERR_INVALID_ARG, "%s: max_pages=%d", where, s->max_pages);
  if (rows && !s->row_start) return fail(MOE_ERR_INVALID_ARG, "%s: row_start is NULL", where);
  if (!s->kv_len) return fail(MOE_ERR_INVALID_ARG, "%s: kv_len is NULL", where);
  if (!s->page_table) return fail(MOE_ERR_INVALID_ARG, "%s: page_table is NULL", where);
  return MOE_OK;
}

// Query heads against key/value heads, and the launch sizes they give.
moe_status check_heads(int n_q, int n_kv, int64_t T, int64_t n_seq, const char* where) {
  if (n_q < 1 || n_q > 1024 || n_kv < 1 || n_q % n_kv != 0)
    return fail(n_q > 1024 ? MOE_ERR_UNSUPPORTED : MOE_ERR_INVALID_ARG,
                "%s: n_q=%d must be a multiple of n_kv=%d, at most 1024", where, n_q, n_kv);
  if (T < 0) return fail(MOE_ERR_INVALID_ARG, "%s: T=%lld < 0", where, (long long)T);
  if (T > kMaxT || T * n_q > ((int64_t)1 << 26) || n_seq * n_q > ((int64_t)1 << 22))
    return fail(MOE_ERR_UNSUPPORTED, "%s: T=%lld, n_seq=%lld with n_q=%d is too large", where,
                (long long)T, (long long)n_seq, n_q);
  return MOE_OK;
}

moe_status check_scale(float scale, const char* where) {
  if (!(scale > 0.0f && isfinite(scale)))
    return fail(MOE_ERR_INVALID_ARG, "%s: scale=%g must be finite and > 0", where, (double)scale);
  return MOE_OK;
}

// The arguments that a workspace's size goes by.
moe_status check_attn_sizes(const moe_kv_cache* c, int n_q, int n_seq, int64_t T, int64_t max_len,
                                   const char* where) {
  if (!c) return fail(MOE_ERR_INVALID_ARG, "%s: c is NULL", where);
  moe_status st = check_cache_shape(c->fmt, c->n_kv, c->D, c->page_tokens, where);
  if (st != MOE_OK) return st;
  if ((st = check_heads(n_q, c->n_kv, T, n_seq, where)) != MOE_OK) return st;
  if (n_seq < 0 || max_len < 0)
    return fail(MOE_ERR_INVALID_ARG, "%s: n_seq=%d max_len=%lld", where, n_seq, (long long)max_len);
  return MOE_OK;
}

}  // namespace

extern "C" {

size_t moe_kv_page_bytes(int32_t fmt, int32_t n_kv, int32_t D, int32_t page_tokens) {
  if (check_cache_shape(fmt, n_kv, D, page_tokens, "moe_kv_page_bytes") != MOE_OK) return 0;
  return (size_t)n_kv * moe::kv_layout(fmt, D, page_tokens).head;
}

moe_status moe_rope_freqs(int32_t kind, int32_t rot_dim, double base, double factor,
                          double orig_len, double turns_lo, double turns_hi, double* freqs,
                          float* scale) {
  const char* W = "moe_rope_freqs";
  const double kTwoPi = 6.283185307179586;
  if (kind < MOE_ROPE_PLAIN || kind > MOE_ROPE_PARTS)
    return fail(MOE_ERR_INVALID_ARG, "%s: kind=%d", W, kind);
  if (rot_dim < 16 || rot_dim > 256 || rot_dim % 16 != 0)
    return fail(MOE_ERR_UNSUPPORTED, "%s: rot_dim=%d must be a multiple of 16 in 16..256", W, rot_dim);
  if (!(base > 1.0 && isfinite(base))) return fail(MOE_ERR_INVALID_ARG, "%s: base=%g", W, base);
  if (kind != MOE_ROPE_PLAIN && !(factor >= 1.0 && isfinite(factor)))
    return fail(MOE_ERR_INVALID_ARG, "%s: factor=%g must be >= 1", W, factor);
  if (kind == MOE_ROPE_PARTS && !(orig_len > 0.0 && turns_lo > 0.0 && turns_hi > turns_lo && isfinite(orig_len) && isfinite(turns_hi)))
    return fail(MOE_ERR_INVALID_ARG, "%s: orig_len=%g, turns %g..%g", W, orig_len, turns_lo, turns_hi);
  CHECK_PTR(freqs, W);
  CHECK_PTR(scale, W);
  const int half = rot_dim / 2;
  if (kind == MOE_ROPE_BASE) base *= pow(factor, rot_dim / (rot_dim - 2.0));
  // the pair index whose frequency makes `turns` turns over orig_len
  const auto index_of = [&](double turns) {
    return rot_dim * log(orig_len / (turns * kTwoPi)) / (2.0 * log(base));
  };
  double lo = 0.0, hi = 0.0;
  if (kind == MOE_ROPE_PARTS) {
    lo = index_of(turns_hi);
    hi = index_of(turns_lo);
  }
  for (int i = 0; i < half; ++i) {
    const double f = pow(base, -2.0 * i / rot_dim);
    if (kind == MOE_ROPE_LINEAR) {
      freqs[i] = f / factor;
    } else if (kind == MOE_ROPE_PARTS) {
      double r = (i - lo) / (hi - lo);  // 0: kept, 1: stretched
      r = r < 0.0 ? 0.0 : r > 1.0 ? 1.0 : r;
      freqs[i] = f * (1.0 - r) + f / factor * r;
    } else {
      freqs[i] = f;
    }
  }
  *scale = kind == MOE_ROPE_PARTS ? (float)(0.1 * log(factor) + 1.0) : 1.0f;
  return MOE_OK;
}

moe_status moe_kv_append(const moe_kv_cache* c, const moe_qkv_desc* p, const moe_seq_batch* s,
                         const uint16_t* qkv, int64_t qkv_stride, int64_t T, const int32_t* pos,
                         uint16_t* q_out, int64_t q_stride, uint16_t* k_out, int64_t k_stride,
                         hipStream_t stream) {
  const char* W = "moe_kv_append";
  moe_status st = check_cache(c, W);
  if (st != MOE_OK) return st;
  CHECK_PTR(p, W);
  if ((st = check_seqs(s, true, W)) != MOE_OK) return st;
  if ((st = check_heads(p->n_q, c->n_kv, T, s->n_seq, W)) != MOE_OK) return st;
  if (!(p->eps >= 0.0f && isfinite(p->eps)))
    return fail(MOE_ERR_INVALID_ARG, "%s: eps=%g", W, (double)p->eps);
  if (p->rot_dim < 0 || p->rot_dim > c->D || p->rot_dim % 16 != 0)
    return fail(MOE_ERR_UNSUPPORTED, "%s: rot_dim=%d must be a multiple of 16 in 0..%d", W,
                p->rot_dim, c->D);
  if (p->interleaved != 0 && p->interleaved != 1)
    return fail(MOE_ERR_INVALID_ARG, "%s: interleaved=%d must be 0 or 1", W, p->interleaved);
  if (p->rot_dim > 0 && (!p->inv_freq || !isfinite(p->rope_scale)))
    return fail(MOE_ERR_INVALID_ARG, "%s: inv_freq is NULL or rope_scale=%g", W,
                (double)p->rope_scale);
  if (T == 0 || s->n_seq == 0) return MOE_OK;
  const int64_t D = c->D, qw = p->n_q * D, kw = c->n_kv * D;
  if ((st = check_rows(qkv, qkv_stride, qw + 2 * kw, "qkv", W)) != MOE_OK) return st;
  if ((st = check_rows(q_out, q_stride, qw, "q_out", W)) != MOE_OK) return st;
  if (k_out && (st = check_rows(k_out, k_stride, kw, "k_out", W)) != MOE_OK) return st;
  if ((st = check_aligned(p->q_norm, "q_norm", W)) != MOE_OK) return st;
  if ((st = check_aligned(p->k_norm, "k_norm", W)) != MOE_OK) return st;
  const RowBlock in{qkv, qkv_stride, qw + 2 * kw, T}, qo{q_out, q_stride, qw, T}, ko{k_out, k_stride, kw, T};
  if ((st = check_apart(qo, in, true, "q_out", "qkv", W)) != MOE_OK) return st;
  if (k_out) {
    if (k_out != qkv + qw || (k_stride != qkv_stride && T > 1))  // (the keys' own place)
      if ((st = check_apart(ko, in, false, "k_out", "qkv", W)) != MOE_OK) return st;
    if ((st = check_apart(ko, qo, false, "k_out", "q_out", W)) != MOE_OK) return st;
  }
  return hip_status(W, moe::launch_kv_append(c, p, s, qkv, qkv_stride, T, pos, q_out, q_stride,
                                             k_out, k_stride, stream));
}

moe_status moe_kv_read(const moe_kv_cache* c, const moe_seq_batch* s, const int32_t* first,
                       const int32_t* out_start, int64_t R, uint16_t* k_out, int64_t k_stride,
                       uint16_t* v_out, int64_t v_stride, hipStream_t stream) {
  const char* W = "moe_kv_read";
  moe_status st = check_cache(c, W);
  if (st != MOE_OK) return st;
  if ((st = check_seqs(s, false, W)) != MOE_OK) return st;
  if (R < 0) return fail(MOE_ERR_INVALID_ARG, "%s: R=%lld < 0", W, (long long)R);
  if (R > (int64_t)1 << 28)
    return fail(MOE_ERR_UNSUPPORTED, "%s: R=%lld too large", W, (long long)R);
  if (R == 0 || s->n_seq == 0 || (!k_out && !v_out)) return MOE_OK;
  CHECK_PTR(out_start, W);
  const int64_t kw = (int64_t)c->n_kv * c->D;
  if (k_out && (st = check_rows(k_out, k_stride, kw, "k_out", W)) != MOE_OK) return st;
  if (v_out && (st = check_rows(v_out, v_stride, kw, "v_out", W)) != MOE_OK) return st;
  if (k_out && v_out &&
      (st = check_apart({k_out, k_stride, kw, R}, {v_out, v_stride, kw, R}, false, "k_out", "v_out", W)) != MOE_OK)
    return st;
  return hip_status(W, moe::launch_kv_read(c, s, first, out_start, R, k_out, k_stride, v_out,
                                           v_stride, stream));
}

size_t moe_attn_workspace_bytes(const moe_kv_cache* c, int32_t n_q, int32_t n_seq, int64_t T,
                                int64_t max_len) {
  if (check_attn_sizes(c, n_q, n_seq, T, max_len, "moe_attn_workspace_bytes") != MOE_OK) return 0;
  // max_len 0 stands for the page table's capacity, which is not known here:
  // the longest cache gives the largest split.  Fewer rows can need more (they
  // are split finer); beyond kSplitPairs there are no splits.
  size_t most = 0;
  for (int64_t t = 1; t <= T && t * n_q <= moe::kSplitPairs; ++t)
    most = std::max(most, moe::attn_decode_ws_bytes(c->fmt, c->n_kv, c->D, n_q, n_seq, t,
                                                    max_len ? max_len : INT32_MAX));
  return most;
}

moe_status moe_attn_decode(const moe_kv_cache* c, const moe_seq_batch* s, int32_t n_q,
                           const uint16_t* q, int64_t q_stride, int64_t T, int64_t max_len,
                           float scale, uint16_t* out, int64_t out_stride, void* ws,
                           size_t ws_bytes, hipStream_t stream) {
  const char* W = "moe_attn_decode";
  moe_status st = check_cache(c, W);
  if (st != MOE_OK) return st;
  if ((st = check_seqs(s, true, W)) != MOE_OK) return st;
  if ((st = check_heads(n_q, c->n_kv, T, s->n_seq, W)) != MOE_OK) return st;
  if ((st = check_scale(scale, W)) != MOE_OK) return st;
  if (max_len < 0) return fail(MOE_ERR_INVALID_ARG, "%s: max_len=%lld < 0", W, (long long)max_len);
  if (T == 0 || s->n_seq == 0) return MOE_OK;
  const int64_t qw = (int64_t)n_q * c->D;
  if ((st = check_rows(q, q_stride, qw, "q", W)) != MOE_OK) return st;
  if ((st = check_rows(out, out_stride, qw, "out", W)) != MOE_OK) return st;
  if (max_len == 0) max_len = (int64_t)s->max_pages * c->page_tokens;
  const size_t need = moe::attn_decode_ws_bytes(c->fmt, c->n_kv, c->D, n_q, s->n_seq, T, max_len);
  if (need > 0) {
    CHECK_PTR(ws, W);
    if (ws_bytes < need) return fail(MOE_ERR_WORKSPACE, "%s: workspace %zu < %zu", W, ws_bytes, need);
    if ((st = check_aligned(ws, "ws", W)) != MOE_OK) return st;
  }
  if ((st = check_apart({out, out_stride, qw, T}, {q, q_stride, qw, T}, true, "out", "q", W)) != MOE_OK) return st;
  return hip_status(W, moe::launch_attn_decode(c, s, n_q, q, q_stride, T, max_len, scale, out,
                                               out_stride, ws, stream));
}

size_t moe_attn_chunk_workspace_bytes(const moe_kv_cache* c, int32_t n_q, int32_t n_seq, int64_t T,
                                      int64_t max_len) {
  if (check_attn_sizes(c, n_q, n_seq, T, max_len, "moe_attn_chunk_workspace_bytes") != MOE_OK) return 0;
  // (as above: the longest cache gives the largest split, and fewer rows can need more)
  size_t most = 0;
  for (int64_t t = 1; t <= T && t * n_q <= moe::kChunkPairs; ++t)
    most = std::max(most, moe::attn_chunk_ws_bytes(c->n_kv, c->D, n_q, n_seq, t, max_len ? max_len : INT32_MAX));
  return most;
}

moe_status moe_attn_chunk(const moe_kv_cache* c, const moe_seq_batch* s, int32_t n_q,
                          const uint16_t* q, int64_t q_stride, int64_t T, int64_t max_len,
                          float scale, uint16_t* out, int64_t out_stride, void* ws,
                          size_t ws_bytes, hipStream_t stream) {
  const char* W = "moe_attn_chunk";
  moe_status st = check_cache(c, W);
  if (st != MOE_OK) return st;
  if ((st = check_seqs(s, true, W)) != MOE_OK) return st;
  if ((st = check_heads(n_q, c->n_kv, T, s->n_seq, W)) != MOE_OK) return st;
  if ((st = check_scale(scale, W)) != MOE_OK) return st;
  if (max_len < 0) return fail(MOE_ERR_INVALID_ARG, "%s: max_len=%lld < 0", W, (long long)max_len);
  if (T == 0 || s->n_seq == 0) return MOE_OK;
  const int64_t qw = (int64_t)n_q * c->D;
  if ((st = check_rows(q, q_stride, qw, "q", W)) != MOE_OK) return st;
  if ((st = check_rows(out, out_stride, qw, "out", W)) != MOE_OK) return st;
  if (max_len == 0) max_len = (int64_t)s->max_pages * c->page_tokens;
  const size_t need = moe::attn_chunk_ws_bytes(c->n_kv, c->D, n_q, s->n_seq, T, max_len);
  if (need > 0) {
    CHECK_PTR(ws, W);
    if (ws_bytes < need) return fail(MOE_ERR_WORKSPACE, "%s: workspace %zu < %zu", W, ws_bytes, need);
    if ((st = check_aligned(ws, "ws", W)) != MOE_OK) return st;
  }
  if ((st = check_apart({out, out_stride, qw, T}, {q, q_stride, qw, T}, true, "out", "q", W)) != MOE_OK) return st;
  return hip_status(W, moe::launch_attn_chunk(c, s, n_q, q, q_stride, T, max_len, scale, out,
                                              out_stride, ws, stream));
}

moe_status moe_attn_prompt(int32_t n_q, int32_t n_kv, int32_t D, int32_t n_seq,
                           const int32_t* q_start, const int32_t* kv_start, int64_t T, int64_t Tk,
                           const uint16_t* q, int64_t q_stride, const uint16_t* k,
                           int64_t k_stride, const uint16_t* v, int64_t v_stride, float scale,
                           uint16_t* out, int64_t out_stride, hipStream_t stream) {
  const char* W = "moe_attn_prompt";
  moe_status st = check_head(D, W);
  if (st != MOE_OK) return st;
  if (n_seq < 0 || n_seq > 65535)
    return fail(n_seq < 0 ? MOE_ERR_INVALID_ARG : MOE_ERR_UNSUPPORTED,
                "%s: n_seq=%d must be in 0..65535", W, n_seq);
  if ((st = check_heads(n_q, n_kv, T, n_seq, W)) != MOE_OK) return st;
  if ((st = check_scale(scale, W)) != MOE_OK) return st;
  if (Tk < 0) return fail(MOE_ERR_INVALID_ARG, "%s: Tk=%lld < 0", W, (long long)Tk);
  if (!kv_start && Tk < T)
    return fail(MOE_ERR_INVALID_ARG, "%s: Tk=%lld < T=%lld without kv_start", W, (long long)Tk,
                (long long)T);
  if (T == 0 || n_seq == 0) return MOE_OK;
  CHECK_PTR(q_start, W);
  const int64_t qw = (int64_t)n_q * D, kw = (int64_t)n_kv * D;
  if ((st = check_rows(q, q_stride, qw, "q", W)) != MOE_OK) return st;
  if ((st = check_rows(out, out_stride, qw, "out", W)) != MOE_OK) return st;
  if (Tk > 0) {
    if ((st = check_rows(k, k_stride, kw, "k", W)) != MOE_OK) return st;
    if ((st = check_rows(v, v_stride, kw, "v", W)) != MOE_OK) return st;
    // a tile of 64 rows is read with 32-bit byte offsets
    if (k_stride > (1 << 24) || v_stride > (1 << 24))
      return fail(MOE_ERR_UNSUPPORTED, "%s: k and v strides are at most 2^24 elements", W);
  }
  const RowBlock o{out, out_stride, qw, T};
  if ((st = check_apart(o, {q, q_stride, qw, T}, true, "out", "q", W)) != MOE_OK) return st;
  if (Tk > 0) {
    if ((st = check_apart(o, {k, k_stride, kw, Tk}, false, "out", "k", W)) != MOE_OK) return st;
    if ((st = check_apart(o, {v, v_stride, kw, Tk}, false, "out", "v", W)) != MOE_OK) return st;
  }
  return hip_status(W, moe::launch_attn_prompt(n_q, n_kv, D, n_seq, q_start, kv_start, T, Tk, q,
                                               q_stride, k, k_stride, v, v_stride, scale, out,
                                               out_stride, stream));
}

}  // extern "C"

// ---------------------------------------------------------------------------
// Norms and dense projections
// ---------------------------------------------------------------------------

namespace {

moe_status check_mx_fmt(int fmt, const char* where) {
  if (fmt != MOE_FMT_MXFP4 && fmt != MOE_FMT_MXFP8)
    return fail(MOE_ERR_UNSUPPORTED, "%s: row format %d (MXFP4 or MXFP8)", where, fmt);
  return MOE_OK;
}

moe_status check_width(int n, int most, const char* name, const char* where) {
  if (n < 1 || n % 128 != 0 || n > most)
    return fail(n < 1 ? MOE_ERR_INVALID_ARG : MOE_ERR_UNSUPPORTED,
                "%s: %s=%d must be a multiple of 128 in 128..%d", where, name, n, most);
  return MOE_OK;
}

moe_status check_matrix(int N, int K, const char* where) {
  if (N < 1 || N > (1 << 20))
    return fail(N < 1 ? MOE_ERR_INVALID_ARG : MOE_ERR_UNSUPPORTED, "%s: N=%d must be in 1..2^20", where, N);
  return check_width(K, 32768, "K", where);
}

moe_status check_count(int64_t T, const char* where) {
  if (T < 0) return fail(MOE_ERR_INVALID_ARG, "%s: T=%lld < 0", where, (long long)T);
  if (T > (1 << 20)) return fail(MOE_ERR_UNSUPPORTED, "%s: T=%lld > 2^20", where, (long long)T);
  return MOE_OK;
}

// T rows of `bytes` bytes each, one after the other.
RowBlock dense(const void* p, int64_t bytes, int64_t T) { return RowBlock{p, bytes / 2, bytes / 2, T}; }
int64_t code_bytes(int fmt, int64_t K) { return fmt == MOE_FMT_MXFP4 ? K / 2 : K; }

moe_status check_codes(const uint8_t* codes, const uint8_t* scales, const char* where) {
  CHECK_PTR(codes, where);
  CHECK_PTR(scales, where);
  moe_status st = check_aligned(codes, "codes", where);
  return st != MOE_OK ? st : check_aligned(scales, "scales", where);
}

struct Named {
  RowBlock rows;
  const char* name;
};
// `out` shares no element with any of these (in_place: but may be one of them).
template <size_t N>
moe_status check_all_apart(Named out, const Named (&in)[N], bool in_place, const char* where) {
  if (!out.rows.p) return MOE_OK;
  for (const Named& i : in) {
    if (!i.rows.p) continue;
    const moe_status st = check_apart(out.rows, i.rows, in_place, out.name, i.name, where);
    if (st != MOE_OK) return st;
  }
  return MOE_OK;
}

moe_status check_product(const moe_mx_matrix* w, int fmt, int64_t T, const char* where) {
  CHECK_PTR(w, where);
  moe_status st = check_matrix(w->N, w->K, where);
  if (st != MOE_OK) return st;
  if ((st = check_mx_fmt(fmt, where)) != MOE_OK) return st;
  if ((st = check_count(T, where)) != MOE_OK) return st;
  CHECK_PTR(w->packed, where);
  if ((uintptr_t)w->packed % moe::kAlign != 0)
    return fail(MOE_ERR_INVALID_ARG, "%s: packed not 256-byte aligned", where);
  return check_aligned(w->bias, "bias", where);
}

// The outputs of a product, in 16-bit elements.
moe_status check_result(const moe_mx_matrix* w, int64_t T, const void* y, int64_t y_stride, int y_dtype,
                        Named* out, const char* where) {
  if (y_dtype != MOE_DTYPE_F32 && y_dtype != MOE_DTYPE_BF16)
    return fail(MOE_ERR_INVALID_ARG, "%s: y_dtype=%d", where, y_dtype);
  const moe_status st = check_rows(y, y_stride, w->N, "y", where);
  if (st != MOE_OK) return st;
  const int64_t e = y_dtype == MOE_DTYPE_F32 ? 2 : 1;
  *out = Named{RowBlock{y, y_stride * e, w->N * e, T}, "y"};
  const Named weights[] = {{dense(w->packed, (int64_t)moe::mx_layout(w->N, w->K).total, 1), "the weights"},
                           {dense(w->bias, 4 * (int64_t)w->N, 1), "bias"}};
  return check_all_apart(*out, weights, false, where);
}

}  // namespace

extern "C" {

moe_status moe_add_norm(int32_t H, int64_t T, const uint16_t* x, int64_t x_stride,
                        const uint16_t* residual, int64_t residual_stride, const float* weight,
                        float eps, uint16_t* sum, int64_t sum_stride, uint16_t* out,
                        int64_t out_stride, int32_t fmt, uint8_t* codes, uint8_t* scales,
                        hipStream_t stream) {
  const char* W = "moe_add_norm";
  moe_status st = check_width(H, 16384, "H", W);
  if (st != MOE_OK) return st;
  if ((st = check_count(T, W)) != MOE_OK) return st;
  if (!(eps >= 0.0f && isfinite(eps))) return fail(MOE_ERR_INVALID_ARG, "%s: eps=%g", W, (double)eps);
  if (fmt != 0 && (st = check_mx_fmt(fmt, W)) != MOE_OK) return st;
  if (fmt == 0 && (codes || scales)) return fail(MOE_ERR_INVALID_ARG, "%s: codes or scales without a format", W);
  if (!sum && !out && fmt == 0) return fail(MOE_ERR_INVALID_ARG, "%s: no output", W);
  if (T == 0) return MOE_OK;
  if ((st = check_rows(x, x_stride, H, "x", W)) != MOE_OK) return st;
  if (residual && (st = check_rows(residual, residual_stride, H, "residual", W)) != MOE_OK) return st;
  if (sum && (st = check_rows(sum, sum_stride, H, "sum", W)) != MOE_OK) return st;
  if (out && (st = check_rows(out, out_stride, H, "out", W)) != MOE_OK) return st;
  CHECK_PTR(weight, W);
  if ((st = check_aligned(weight, "weight", W)) != MOE_OK) return st;
  if (fmt != 0 && (st = check_codes(codes, scales, W)) != MOE_OK) return st;
  const Named in[] = {{{x, x_stride, H, T}, "x"}, {{residual, residual_stride, H, T}, "residual"}};
  const Named w{dense(weight, 4 * (int64_t)H, 1), "weight"};
  const Named s{{sum, sum_stride, H, T}, "sum"}, o{{out, out_stride, H, T}, "out"};
  const Named c{dense(codes, code_bytes(fmt, H), T), "codes"}, f{dense(scales, H / 32, T), "scales"};
  const Named after_sum[] = {w}, after_out[] = {w, s}, after_codes[] = {in[0], in[1], w, s, o},
              after_scales[] = {in[0], in[1], w, s, o, c};
  if ((st = check_all_apart(s, in, true, W)) != MOE_OK) return st;
  if ((st = check_all_apart(s, after_sum, false, W)) != MOE_OK) return st;
  if ((st = check_all_apart(o, in, true, W)) != MOE_OK) return st;
  if ((st = check_all_apart(o, after_out, false, W)) != MOE_OK) return st;
  if ((st = check_all_apart(c, after_codes, false, W)) != MOE_OK) return st;
  if ((st = check_all_apart(f, after_scales, false, W)) != MOE_OK) return st;
  return hip_status(W, moe::launch_add_norm(H, T, x, x_stride, residual, residual_stride, weight, eps, sum,
                                            sum_stride, out, out_stride, fmt, codes, scales, stream));
}

moe_status moe_mx_quant(int32_t fmt, int32_t K, int64_t T, const uint16_t* x, int64_t x_stride,
                        uint8_t* codes, uint8_t* scales, hipStream_t stream) {
  const char* W = "moe_mx_quant";
  moe_status st = check_mx_fmt(fmt, W);
  if (st != MOE_OK) return st;
  if ((st = check_width(K, 32768, "K", W)) != MOE_OK) return st;
  if ((st = check_count(T, W)) != MOE_OK) return st;
  if (T == 0) return MOE_OK;
  if ((st = check_rows(x, x_stride, K, "x", W)) != MOE_OK) return st;
  if ((st = check_codes(codes, scales, W)) != MOE_OK) return st;
  const Named in[] = {{{x, x_stride, K, T}, "x"}};
  const Named c[] = {{dense(codes, code_bytes(fmt, K), T), "codes"}};
  const Named f{dense(scales, K / 32, T), "scales"};
  if ((st = check_all_apart(c[0], in, false, W)) != MOE_OK) return st;
  if ((st = check_all_apart(f, in, false, W)) != MOE_OK) return st;
  if ((st = check_all_apart(f, c, false, W)) != MOE_OK) return st;
  return hip_status(W, moe::launch_mx_quant(fmt, K, T, x, x_stride, codes, scales, stream));
}

size_t moe_mx_matrix_bytes(int32_t N, int32_t K) {
  if (check_matrix(N, K, "moe_mx_matrix_bytes") != MOE_OK) return 0;
  return moe::mx_layout(N, K).total;
}

moe_status moe_mx_pack(int32_t N, int32_t K, const uint8_t* codes, const uint8_t* scales,
                       void* packed, hipStream_t stream) {
  const char* W = "moe_mx_pack";
  moe_status st = check_matrix(N, K, W);
  if (st != MOE_OK) return st;
  if ((st = check_codes(codes, scales, W)) != MOE_OK) return st;
  CHECK_PTR(packed, W);
  if ((uintptr_t)packed % moe::kAlign != 0)
    return fail(MOE_ERR_INVALID_ARG, "%s: packed not 256-byte aligned", W);
  const Named in[] = {{dense(codes, K / 2, N), "codes"}, {dense(scales, K / 32, N), "scales"}};
  const Named p{dense(packed, (int64_t)moe::mx_layout(N, K).total, 1), "packed"};
  if ((st = check_all_apart(p, in, false, W)) != MOE_OK) return st;
  return hip_status(W, moe::launch_mx_pack(N, K, codes, scales, packed, stream));
}

moe_status moe_mx_linear(const moe_mx_matrix* w, int32_t fmt, const uint8_t* codes,
                         const uint8_t* scales, int64_t T, void* y, int64_t y_stride,
                         int32_t y_dtype, hipStream_t stream) {
  const char* W = "moe_mx_linear";
  moe_status st = check_product(w, fmt, T, W);
  if (st != MOE_OK) return st;
  if (T == 0) return MOE_OK;
  if ((st = check_codes(codes, scales, W)) != MOE_OK) return st;
  Named out;
  if ((st = check_result(w, T, y, y_stride, y_dtype, &out, W)) != MOE_OK) return st;
  const Named in[] = {{dense(codes, code_bytes(fmt, w->K), T), "codes"}, {dense(scales, w->K / 32, T), "scales"}};
  if ((st = check_all_apart(out, in, false, W)) != MOE_OK) return st;
  return hip_status(W, moe::launch_mx_linear(w, fmt, nullptr, 0, codes, scales, T, y, y_stride, y_dtype, stream));
}

size_t moe_mx_workspace_bytes(int32_t fmt, int32_t K, int64_t T) {
  const char* W = "moe_mx_workspace_bytes";
  if (check_mx_fmt(fmt, W) != MOE_OK || check_width(K, 32768, "K", W) != MOE_OK || check_count(T, W) != MOE_OK)
    return 0;
  return moe::align_up((size_t)T * code_bytes(fmt, K)) + moe::align_up((size_t)T * (K / 32));
}

moe_status moe_mx_linear_rows(const moe_mx_matrix* w, int32_t fmt, const uint16_t* x,
                              int64_t x_stride, int64_t T, void* y, int64_t y_stride,
                              int32_t y_dtype, void* ws, size_t ws_bytes, hipStream_t stream) {
  const char* W = "moe_mx_linear_rows";
  moe_status st = check_product(w, fmt, T, W);
  if (st != MOE_OK) return st;
  if (T == 0) return MOE_OK;
  if ((st = check_rows(x, x_stride, w->K, "x", W)) != MOE_OK) return st;
  Named out;
  if ((st = check_result(w, T, y, y_stride, y_dtype, &out, W)) != MOE_OK) return st;
  const size_t need = moe_mx_workspace_bytes(fmt, w->K, T);
  CHECK_PTR(ws, W);
  if (ws_bytes < need) return fail(MOE_ERR_WORKSPACE, "%s: workspace %zu < %zu", W, ws_bytes, need);
  if ((st = check_aligned(ws, "ws", W)) != MOE_OK) return st;
  const Named in[] = {{{x, x_stride, w->K, T}, "x"}, {dense(ws, (int64_t)need, 1), "ws"}};
  if ((st = check_all_apart(out, in, false, W)) != MOE_OK) return st;
  if (moe::mx_linear_takes_rows(w->N, w->K, T))
    return hip_status(W, moe::launch_mx_linear(w, fmt, x, x_stride, nullptr, nullptr, T, y, y_stride, y_dtype, stream));
  const Named rows[] = {in[0]};
  if ((st = check_all_apart(in[1], rows, false, W)) != MOE_OK) return st;
  uint8_t* const codes = (uint8_t*)ws;
  uint8_t* const scales = codes + moe::align_up((size_t)T * code_bytes(fmt, w->K));
  const hipError_t e = moe::launch_mx_quant(fmt, w->K, T, x, x_stride, codes, scales, stream);
  if (e != hipSuccess) return hip_status(W, e);
  return hip_status(W, moe::launch_mx_linear(w, fmt, nullptr, 0, codes, scales, T, y, y_stride, y_dtype, stream));
}

}  // extern "C"
