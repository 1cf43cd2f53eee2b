// mx.h -- microscaled values: what the norm, the quantiser and the product share.
//
// A block of 32 values along a row has one scale 2^(s - 127), s a byte; its values
// are E2M1 (MOE_FMT_MXFP4) or E4M3 (MOE_FMT_MXFP8) codes.  s puts the block's
// largest magnitude A into the format's highest binade, s - 127 = floor(log2 A) -
// (2 or 8), so a code's value before scaling is below 8 or 512; what is beyond 6 or
// 448 is held to that.  Powers of two make every product with a scale exact: the
// codes are the only rounding.
#pragma once

#include "pairs.h"

namespace moe {

constexpr int kMxBlock = 32;   // values of a scale
constexpr int kMxStep = 128;   // elements of K that a matrix instruction takes: 4 blocks
constexpr int kMxTile = 16;    // rows of a tile of the packed matrix

// Packed matrix [N][K]: the 4-bit codes as tiles of 16 rows by 128 elements, 1 KB
// each, [N/16][K/128][4 blocks][16 rows][16 bytes], so that a wave's load of 16
// bytes a lane is one tile and a matrix instruction's operand; behind them the scales
// [N/16][K/128][16 rows][4 bytes].  Rows from N to the next multiple of 16 are zero.
struct MxLayout {
  int64_t tiles, steps;
  size_t scales, total;
};
inline MxLayout mx_layout(int64_t N, int64_t K) {
  MxLayout l;
  l.tiles = (N + kMxTile - 1) / kMxTile;
  l.steps = K / kMxStep;
  l.scales = (size_t)l.tiles * l.steps * 1024;
  l.total = align_up(l.scales + (size_t)l.tiles * l.steps * 64);
  return l;
}

template <int FMT>
constexpr int mx_bytes(int n) { return FMT == MOE_FMT_MXFP4 ? n / 2 : n; }

// Scale byte of a block whose largest magnitude has these bits (bf16 without its
// sign): 255, NaN, where the block holds an infinity or a NaN.
template <int FMT>
__device__ __forceinline__ uint32_t mx_scale(uint32_t top) {
  constexpr int drop = FMT == MOE_FMT_MXFP4 ? 2 : 8;
  return top >= 0x7f80u ? 255u : (uint32_t)max((int)(top >> 7) - drop, 0);
}
// The largest magnitude of 8 bf16 values, as bits.
__device__ __forceinline__ uint32_t mx_top(uint4 x) {
  typedef uint16_t v2us __attribute__((ext_vector_type(2)));
  const auto pair = [](uint32_t a, uint32_t b) {
    return __builtin_bit_cast(uint32_t, __builtin_elementwise_max(__builtin_bit_cast(v2us, a), __builtin_bit_cast(v2us, b)));
  };
  constexpr uint32_t mag = 0x7fff7fffu;
  const uint32_t m = pair(pair(x.x & mag, x.y & mag), pair(x.z & mag, x.w & mag));
  return max(m & 0xffffu, m >> 16);
}
// Codes of 8 bf16 values: one word of E2M1 or two of E4M3, to nearest even.  The
// conversions divide by the scale; the 4-bit one holds what is too large to 6 by itself,
// for the 8-bit one, which would make a NaN of it, the magnitudes are held to 448 times the
// scale first (as bits, which order as the values do).
template <int FMT>
__device__ __forceinline__ uint2 mx_codes(uint4 x, uint32_t s) {
  typedef __bf16 v2b __attribute__((ext_vector_type(2)));
  typedef short v2s __attribute__((ext_vector_type(2)));
  typedef uint16_t v2us __attribute__((ext_vector_type(2)));
  const float scale = __uint_as_float(s ? s << 23 : 0x00400000u);  // 2^(s - 127)
  const uint32_t w[4] = {x.x, x.y, x.z, x.w};
  uint2 q = make_uint2(0u, 0u);
  if constexpr (FMT == MOE_FMT_MXFP4) {
    q.x = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(q.x, __builtin_bit_cast(v2b, w[0]), scale, 0);
    q.x = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(q.x, __builtin_bit_cast(v2b, w[1]), scale, 1);
    q.x = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(q.x, __builtin_bit_cast(v2b, w[2]), scale, 2);
    q.x = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(q.x, __builtin_bit_cast(v2b, w[3]), scale, 3);
  } else {
    const uint16_t most = (uint16_t)((s + 8) << 7 | 0x60u);  // 1.75 * 2^(s + 8 - 127)
    v2b v[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const v2us m = __builtin_elementwise_min(__builtin_bit_cast(v2us, w[i] & 0x7fff7fffu), v2us{most, most});
      v[i] = __builtin_bit_cast(v2b, __builtin_bit_cast(uint32_t, m) | (w[i] & 0x80008000u));
    }
    v2s a = {0, 0}, b = {0, 0};
    a = __builtin_amdgcn_cvt_scalef32_pk_fp8_bf16(a, v[0], scale, false);
    a = __builtin_amdgcn_cvt_scalef32_pk_fp8_bf16(a, v[1], scale, true);
    b = __builtin_amdgcn_cvt_scalef32_pk_fp8_bf16(b, v[2], scale, false);
    b = __builtin_amdgcn_cvt_scalef32_pk_fp8_bf16(b, v[3], scale, true);
    q = make_uint2(__builtin_bit_cast(uint32_t, a), __builtin_bit_cast(uint32_t, b));
  }
  return s == 255u ? make_uint2(0u, 0u) : q;  // (whatever an infinity or a NaN has made)
}

// Maximum over each 4 neighbouring lanes (a block whose lanes hold 8 values each).
__device__ __forceinline__ uint32_t quad_max(uint32_t v) {
  v = max(v, (uint32_t)__builtin_amdgcn_update_dpp((int)v, (int)v, 0xb1, 0xf, 0xf, true));
  return max(v, (uint32_t)__builtin_amdgcn_update_dpp((int)v, (int)v, 0x4e, 0xf, 0xf, true));
}

// Launchers: arguments are validated before.
hipError_t launch_add_norm(int H, int64_t T, const uint16_t* x, int64_t x_stride,
                           const uint16_t* residual, int64_t residual_stride, const float* weight,
                           float eps, uint16_t* sum, int64_t sum_stride, uint16_t* out,
                           int64_t out_stride, int fmt, uint8_t* codes, uint8_t* scales,
                           hipStream_t stream);
hipError_t launch_mx_quant(int fmt, int K, int64_t T, const uint16_t* x, int64_t x_stride,
                           uint8_t* codes, uint8_t* scales, hipStream_t stream);
hipError_t launch_mx_pack(int N, int K, const uint8_t* codes, const uint8_t* scales, void* packed,
                          hipStream_t stream);
// Whether a product of T rows quantises its 16-bit rows itself (else they have to be
// quantised first).
bool mx_linear_takes_rows(int64_t N, int64_t K, int64_t T);
// x: 16-bit rows, or NULL: codes and scales.
hipError_t launch_mx_linear(const moe_mx_matrix* w, int fmt, const uint16_t* x, int64_t x_stride,
                            const uint8_t* codes, const uint8_t* scales, int64_t T, void* y,
                            int64_t y_stride, int y_dtype, hipStream_t stream);

}  // namespace moe
