// attn_common.h -- pieces shared by the key/value cache and attention kernels.
//
// The pages' engine keeps a key/value cache per request slot and trades its
// precision against the experts' memory (aiopssre.com, "Concurrency divides
// context unless you pay for more cache").  The cache layout is chosen for the
// reader: one (page, head) block is contiguous, keys are rows of D values (a
// lane of the score product takes a quarter of one token's row), values are
// laid out in quads of tokens (a lane of the output product takes D/16 elements
// of four tokens), so every fragment of a 16-token step is one vector load.
#pragma once

#include <type_traits>

#include "gate_common.h"
#include "pairs.h"

namespace moe {

constexpr float kNone = -3.0e38f;  // running maximum before any token
constexpr float kGrow = 8.0f;      // log2 headroom before the accumulators are rescaled

// The cache's codes and scales as fp16, two at a time.
typedef _Float16 v2h __attribute__((ext_vector_type(2)));
__device__ __forceinline__ v2h fp4_pair(uint32_t w, int k) {  // byte k: two E2M1 codes
  switch (k) {
    case 0: return __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(w, 1.0f, 0);
    case 1: return __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(w, 1.0f, 1);
    case 2: return __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(w, 1.0f, 2);
    default: return __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(w, 1.0f, 3);
  }
}
__device__ __forceinline__ v2h fp8_pair(uint32_t w, int k) {  // half-word k: two E4M3 scales
  return k ? __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(w, 1.0f, true)
           : __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(w, 1.0f, false);
}
// int8 codes 2k, 2k + 1 of a word whose sign bits are flipped: byte b + 128 under
// the exponent byte of 1024 is 1024 + 128 + b in fp16, exactly; one packed
// subtraction leaves b.
__device__ __forceinline__ v2h i8_pair(uint32_t biased, int k) {
  const uint32_t w = __builtin_amdgcn_perm(0x64646464u, biased, k ? 0x07030702u : 0x05010400u);
  const v2h c = {(_Float16)1152.0f, (_Float16)1152.0f};
  return __builtin_bit_cast(v2h, w) - c;
}
__device__ __forceinline__ uint32_t bits(v2h v) { return __builtin_bit_cast(uint32_t, v); }
__device__ __forceinline__ v2h halves(uint32_t w) { return __builtin_bit_cast(v2h, w); }

// Byte offsets inside one (page, head) block; head = bytes of the block.
struct KvLayout {
  uint32_t ks, vq, vs, head;
};

__host__ __device__ constexpr KvLayout kv_layout(int fmt, int D, int P) {
  const uint32_t codes = fmt == MOE_FMT_NVFP4 ? (uint32_t)(P * D / 2)
                         : fmt == MOE_FMT_Q8_0 ? (uint32_t)(P * D)
                                               : (uint32_t)(2 * P * D);
  const uint32_t scales = fmt == MOE_FMT_BF16 ? 0u : (uint32_t)(P * D / 16);
  return KvLayout{codes, codes + scales, 2 * codes + scales, 2 * (codes + scales)};
}

// A step's sequences as the kernels take them (device pointers).
struct SeqView {
  const int32_t* row_start;
  const int32_t* kv_len;
  const int32_t* page_table;
  int n_seq, max_pages, n_pages, log2P;
};

// Sequence of packed row t, with its first row, row count and length; b = -1
// when the row belongs to none.  Every lane of the wave takes part and gets the
// same answer.  Up to 64 sequences cost one round of loads.
struct RowSeq {
  int b, r0, len;
  int64_t rows;
};
// Wave-wide sum, in the order of wave_incl_scan.
__device__ __forceinline__ float wave_sum(float v) {
  const auto add = [&](auto CTRL, auto ROWS) {
    v += __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(v), CTRL(), ROWS(), 0xf, ROWS() == 0xf));
  };
  using std::integral_constant;
  add(integral_constant<int, 0x111>(), integral_constant<int, 0xf>());
  add(integral_constant<int, 0x112>(), integral_constant<int, 0xf>());
  add(integral_constant<int, 0x114>(), integral_constant<int, 0xf>());
  add(integral_constant<int, 0x118>(), integral_constant<int, 0xf>());
  add(integral_constant<int, 0x142>(), integral_constant<int, 0xa>());
  add(integral_constant<int, 0x143>(), integral_constant<int, 0xc>());
  return __int_as_float(__builtin_amdgcn_readlane(__float_as_int(v), 63));
}

// Values whose loads are to be on their way together: the compiler would put one
// whose use is behind a branch there, a round trip later.
__device__ __forceinline__ void loaded(int& a, int& b, int& c, int& d) {
#if defined(__HIP_DEVICE_COMPILE__)
  asm volatile("" : "+v"(a), "+v"(b), "+v"(c), "+v"(d));
#endif
}
// also: another such value of the caller's.
__device__ __forceinline__ RowSeq find_row(const SeqView& s, int64_t t, int* also = nullptr) {
  RowSeq r{-1, 0, 0, 0};
  for (int i0 = 0; i0 < s.n_seq; i0 += 64) {
    const int i = min(i0 + lane_id(), s.n_seq - 1);
    int start = s.row_start[i], end = s.row_start[i + 1], len = s.kv_len[i];
    int none = 0;
    loaded(end, start, len, also ? *also : none);
    const uint64_t behind = __ballot(i0 + lane_id() < s.n_seq && (int64_t)end > t);
    if (!behind) continue;
    const int l = __ffsll((unsigned long long)behind) - 1;
    r.r0 = __builtin_amdgcn_readlane(start, l);
    r.rows = (int64_t)__builtin_amdgcn_readlane(end, l) - r.r0;
    r.len = __builtin_amdgcn_readlane(len, l);
    if (r.r0 <= t) r.b = i0 + l;
    break;
  }
  return r;
}

// The unit-th aligned quad of tokens that rows inside 0..T belong to, over all
// sequences: its sequence (b = -1: there are not so many), the first and last
// such row of the sequence, and the row of the quad's first token (which may lie
// before the first row).
__device__ __forceinline__ RowSeq find_quad(const SeqView& s, int64_t T, int unit, int64_t* first,
                                            int64_t* last, int64_t* row) {
  RowSeq r{-1, 0, 0, 0};
  int before = 0;
  for (int i0 = 0; i0 < s.n_seq; i0 += 64) {
    const int i = min(i0 + lane_id(), s.n_seq - 1);
    const int start = s.row_start[i], end = s.row_start[i + 1], len = s.kv_len[i];
    const int64_t lo = max(start, 0), hi = min((int64_t)end, T);
    const int64_t tok = (int64_t)len - ((int64_t)end - start) + (lo - start);
    const int sum = wave_incl_scan(
        i0 + lane_id() < s.n_seq && hi > lo ? (int)(((tok + hi - lo - 1) >> 2) - (tok >> 2)) + 1 : 0);
    const uint64_t past = __ballot(before + sum > unit);
    if (!past) {
      before += __builtin_amdgcn_readlane(sum, 63);
      continue;
    }
    const int l = __ffsll((unsigned long long)past) - 1;
    if (l > 0) before += __builtin_amdgcn_readlane(sum, l - 1);
    r.r0 = __builtin_amdgcn_readlane(start, l);
    const int e = __builtin_amdgcn_readlane(end, l);
    r.rows = (int64_t)e - r.r0;
    r.len = __builtin_amdgcn_readlane(len, l);
    r.b = i0 + l;
    *first = max(r.r0, 0);
    *last = min((int64_t)e, T) - 1;
    const int64_t t0 = r.len - r.rows + (*first - r.r0);  // token of the first row
    *row = *first + (((t0 >> 2) + unit - before) << 2) - t0;
    break;
  }
  return r;
}

// Page of token j of sequence b, or -1 when the table or the pool has none.
__device__ __forceinline__ int page_of(const SeqView& s, int b, int64_t j) {
  const int64_t n = j >> s.log2P;
  if (j < 0 || n >= s.max_pages) return -1;
  const int p = s.page_table[(int64_t)b * s.max_pages + n];
  return (unsigned)p < (unsigned)s.n_pages ? p : -1;
}

}  // namespace moe

namespace moe {

hipError_t launch_kv_append(const moe_kv_cache* c, const moe_qkv_desc* p, const moe_seq_batch* s,
                            const uint16_t* qkv, int64_t qkv_stride, int64_t T, const int32_t* pos,
                            uint16_t* q_out, int64_t q_stride, uint16_t* k_out, int64_t k_stride,
                            hipStream_t stream);
hipError_t launch_kv_read(const moe_kv_cache* c, const moe_seq_batch* s, const int32_t* first,
                          const int32_t* out_start, int64_t R, uint16_t* k_out, int64_t k_stride,
                          uint16_t* v_out, int64_t v_stride, hipStream_t stream);
// Most (row, query head) pairs of a step whose sequences are split in moe_attn_decode.
constexpr int64_t kSplitPairs = 1 << 14;
size_t attn_decode_ws_bytes(int fmt, int n_kv, int D, int n_q, int n_seq, int64_t T, int64_t max_len);
hipError_t launch_attn_decode(const moe_kv_cache* c, const moe_seq_batch* s, int n_q,
                              const uint16_t* q, int64_t q_stride, int64_t T, int64_t max_len,
                              float scale, uint16_t* out, int64_t out_stride, void* ws,
                              hipStream_t stream);
// The same in moe_attn_chunk, whose tiles of rows are larger.
constexpr int64_t kChunkPairs = 1 << 16;
size_t attn_chunk_ws_bytes(int n_kv, int D, int n_q, int n_seq, int64_t T, int64_t max_len);
hipError_t launch_attn_chunk(const moe_kv_cache* c, const moe_seq_batch* s, int n_q,
                             const uint16_t* q, int64_t q_stride, int64_t T, int64_t max_len,
                             float scale, uint16_t* out, int64_t out_stride, void* ws,
                             hipStream_t stream);
hipError_t launch_attn_prompt(int n_q, int n_kv, int D, int n_seq, const int32_t* q_start,
                              const int32_t* kv_start, int64_t T, int64_t Tk, const uint16_t* q,
                              int64_t q_stride, const uint16_t* k, int64_t k_stride,
                              const uint16_t* v, int64_t v_stride, float scale, uint16_t* out,
                              int64_t out_stride, hipStream_t stream);

}  // namespace moe
