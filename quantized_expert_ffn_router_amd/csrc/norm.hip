// norm.hip -- the residual's addition and the root-mean-square norm in front of a
// layer's projections and of its experts, and rows in the microscaled formats.
//
// One pass: a row is read once into registers, its squares are summed, and the sum,
// the normed row and the row's codes are written from there.  With
//   h = bf16(x + residual),  z = bf16(fp32(h / sqrt(mean(h^2) + eps) * w))
// squares of bf16 values are exact in fp32 but may lie outside its range, and the
// codes must not hang on the order of a sum, so the norm is in fp64 (as many fp64 as
// plain fp32 operations run per cycle here); the codes are those of z.
//
// Bound by memory: 16384 rows of 2048 with a residual, both 16-bit outputs and 8-bit codes
// 54 to 57 us (5.3 to 5.6 TB/s, above a large copy's 4.9), 16384 rows of 4096 into 8 bits 36 to
// 38 us (5.4); over the same buffers again and again, which the last cache holds in part, 4-bit
// codes 50 against 56 and 26 against 30, the sum and codes alone 34 (4 bits) and 36.  8 rows are
// a launch, 2.9 and 2.3 us in a graph.  A row to a workgroup's waves, as many as hold it 16 or
// 32 bytes a lane: no loop over rows, in which the loads of the next row would take the
// registers that the widened values need (155 us, with spills).
#include <algorithm>

#include "mx.h"

namespace moe {

namespace {

template <int CTRL>
__device__ __forceinline__ double dpp(double v) {
  const uint64_t u = __builtin_bit_cast(uint64_t, v);
  const int lo = (int)u, hi = (int)(u >> 32);
  const uint32_t l = __builtin_amdgcn_update_dpp(lo, lo, CTRL, 0xf, 0xf, true);
  const uint32_t h = __builtin_amdgcn_update_dpp(hi, hi, CTRL, 0xf, 0xf, true);
  return __builtin_bit_cast(double, ((uint64_t)h << 32) | l);
}
__device__ __forceinline__ double wave_sum(double v) {
  v += dpp<0xb1>(v);   // lane ^ 1
  v += dpp<0x4e>(v);   // lane ^ 2
  v += dpp<0x141>(v);  // mirrored in 8
  v += dpp<0x140>(v);  // mirrored in 16
  v += __shfl_xor(v, 16);
  return v + __shfl_xor(v, 32);
}

struct NormArgs {
  const uint16_t* x;
  const uint16_t* residual;
  const float* weight;
  uint16_t* sum;
  uint16_t* out;
  uint8_t* codes;
  uint8_t* scales;
  int64_t x_stride, residual_stride, sum_stride, out_stride, T;
  double inv_n, eps;
  int H, waves, rows;  // waves of a row, rows of a workgroup
};

// A value where it is: not widened ahead of its use, where it would take twice the
// registers, and not rounded past fp32 in one go, which takes ten instructions.
__device__ __forceinline__ float as_is(float v) {
#if defined(__HIP_DEVICE_COMPILE__)
  asm("" : "+v"(v));
#endif
  return v;
}

// A workgroup: `rows` rows of `waves` waves each, C chunks of 512 elements a wave, 8
// elements of each a lane.  (16384 rows of 2048: 55 us with four waves a row, 56 to 58
// with two or one, 61 where a workgroup goes over several rows, the next one's loads
// on their way.)
template <int FMT, int C>
__global__ __launch_bounds__(1024) void k_add_norm(NormArgs a) {
  __shared__ double part[16];
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = lane_id();
  const int r = wave / a.waves, w = wave % a.waves;
  const int64_t t = (int64_t)blockIdx.x * a.rows + r;
  const auto place = [&](int c) { return (c * a.waves + w) * 512 + lane * 8; };
  uint4 h[C], y[C];
  float4 g[C][2];
#pragma unroll
  for (int c = 0; c < C; ++c) {
    const int i = place(c);
    const bool in = i < a.H && t < a.T;
    h[c] = y[c] = make_uint4(0, 0, 0, 0);
    g[c][0] = g[c][1] = make_float4(0.f, 0.f, 0.f, 0.f);
    if (in) {
      h[c] = *reinterpret_cast<const uint4*>(a.x + t * a.x_stride + i);
      if (a.residual) y[c] = *reinterpret_cast<const uint4*>(a.residual + t * a.residual_stride + i);
      g[c][0] = *reinterpret_cast<const float4*>(a.weight + i);
      g[c][1] = *reinterpret_cast<const float4*>(a.weight + i + 4);
    }
  }
  double ss = 0.0;
#pragma unroll
  for (int c = 0; c < C; ++c) {
    uint32_t u[4] = {h[c].x, h[c].y, h[c].z, h[c].w};
    const uint32_t v[4] = {y[c].x, y[c].y, y[c].z, y[c].w};
    if (a.residual) {
#pragma unroll
      for (int k = 0; k < 4; ++k) u[k] = bf16_pair(lo16(u[k]) + lo16(v[k]), hi16(u[k]) + hi16(v[k]));
    }
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const double p = lo16(u[k]), q = hi16(u[k]);
      ss = fma(p, p, ss);
      ss = fma(q, q, ss);
    }
    h[c] = make_uint4(u[0], u[1], u[2], u[3]);
  }
  ss = wave_sum(ss);
  if (a.waves > 1) {
    if (lane == 0) part[wave] = ss;
    __syncthreads();
    ss = 0.0;
    for (int k = 0; k < a.waves; ++k) ss += part[r * a.waves + k];
  }
  if (t >= a.T) return;
  const double inv = rsqrt(ss * a.inv_n + a.eps);
#pragma unroll
  for (int c = 0; c < C; ++c) {
    const int i = place(c);
    if (i >= a.H) continue;
    const uint32_t u[4] = {h[c].x, h[c].y, h[c].z, h[c].w};
    const float gw[8] = {g[c][0].x, g[c][0].y, g[c][0].z, g[c][0].w, g[c][1].x, g[c][1].y, g[c][1].z, g[c][1].w};
    uint32_t z[4];
#pragma unroll
    for (int k = 0; k < 4; ++k)
      z[k] = bf16_pair(as_is((float)((double)as_is(lo16(u[k])) * inv * (double)as_is(gw[2 * k]))),
                       as_is((float)((double)as_is(hi16(u[k])) * inv * (double)as_is(gw[2 * k + 1]))));
    const uint4 zz = make_uint4(z[0], z[1], z[2], z[3]);
    if (a.sum) *reinterpret_cast<uint4*>(a.sum + t * a.sum_stride + i) = h[c];
    if (a.out) *reinterpret_cast<uint4*>(a.out + t * a.out_stride + i) = zz;
    if constexpr (FMT != 0) {
      const uint32_t s = mx_scale<FMT>(quad_max(mx_top(zz)));
      const uint2 q = mx_codes<FMT>(zz, s);
      uint8_t* d = a.codes + t * mx_bytes<FMT>(a.H) + mx_bytes<FMT>(i);
      if constexpr (FMT == MOE_FMT_MXFP4) *reinterpret_cast<uint32_t*>(d) = q.x;
      else *reinterpret_cast<uint2*>(d) = q;
      if (!(lane & 3)) a.scales[t * (a.H / kMxBlock) + i / kMxBlock] = (uint8_t)s;
    }
  }
}

// One wave: C chunks of 512 elements of one row.
template <int FMT, int C>
__global__ __launch_bounds__(256) void k_mx_quant(const uint16_t* x, int64_t x_stride, int64_t T,
                                                  int K, int segs, uint8_t* codes, uint8_t* scales) {
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = lane_id();
  const uint32_t id = blockIdx.x * 4 + wave;
  const int64_t t = id / (uint32_t)segs;
  const int i0 = (int)(id % (uint32_t)segs) * (512 * C) + lane * 8;
  if (t >= T) return;
  uint4 v[C];
#pragma unroll
  for (int c = 0; c < C; ++c)
    v[c] = i0 + 512 * c < K ? *reinterpret_cast<const uint4*>(x + t * x_stride + i0 + 512 * c) : make_uint4(0, 0, 0, 0);
#pragma unroll
  for (int c = 0; c < C; ++c) {
    const int i = i0 + 512 * c;
    if (i >= K) break;
    const uint32_t s = mx_scale<FMT>(quad_max(mx_top(v[c])));
    const uint2 q = mx_codes<FMT>(v[c], s);
    uint8_t* d = codes + t * mx_bytes<FMT>(K) + mx_bytes<FMT>(i);
    if constexpr (FMT == MOE_FMT_MXFP4) *reinterpret_cast<uint32_t*>(d) = q.x;
    else *reinterpret_cast<uint2*>(d) = q;
    if (!(lane & 3)) scales[t * (K / kMxBlock) + i / kMxBlock] = (uint8_t)s;
  }
}

template <int FMT>
void norm(NormArgs a, hipStream_t stream) {
  const int chunks = (a.H + 511) / 512;
  const int C = (chunks + 15) / 16;  // (16 waves a row at most)
  a.waves = (chunks + C - 1) / C;
  a.rows = a.waves >= 4 ? 1 : 4 / a.waves;
  const unsigned grid = (unsigned)((a.T + a.rows - 1) / a.rows), block = 64 * a.waves * a.rows;
  if (C == 1) k_add_norm<FMT, 1><<<grid, block, 0, stream>>>(a);
  else k_add_norm<FMT, 2><<<grid, block, 0, stream>>>(a);
}

template <int FMT>
void quant(int K, int64_t T, const uint16_t* x, int64_t x_stride, uint8_t* codes, uint8_t* scales,
           hipStream_t stream) {
  const int chunks = (K + 511) / 512;
  const bool few = T * chunks <= 8192;
  const int segs = few ? chunks : (chunks + 3) / 4;
  const unsigned grid = (unsigned)((T * segs + 3) / 4);
  if (few) k_mx_quant<FMT, 1><<<grid, 256, 0, stream>>>(x, x_stride, T, K, segs, codes, scales);
  else k_mx_quant<FMT, 4><<<grid, 256, 0, stream>>>(x, x_stride, T, K, segs, codes, scales);
}

}  // namespace

hipError_t launch_add_norm(int H, int64_t T, const uint16_t* x, int64_t x_stride,
                           const uint16_t* residual, int64_t residual_stride, const float* weight,
                           float eps, uint16_t* sum, int64_t sum_stride, uint16_t* out,
                           int64_t out_stride, int fmt, uint8_t* codes, uint8_t* scales,
                           hipStream_t stream) {
  const NormArgs a{x, residual, weight, sum, out, codes, scales, x_stride, residual_stride,
                   sum_stride, out_stride, T, 1.0 / H, (double)eps, H, 0, 0};
  switch (fmt) {
    case MOE_FMT_MXFP4: norm<MOE_FMT_MXFP4>(a, stream); break;
    case MOE_FMT_MXFP8: norm<MOE_FMT_MXFP8>(a, stream); break;
    default: norm<0>(a, stream);
  }
  return hipGetLastError();
}

hipError_t launch_mx_quant(int fmt, int K, int64_t T, const uint16_t* x, int64_t x_stride,
                           uint8_t* codes, uint8_t* scales, hipStream_t stream) {
  if (fmt == MOE_FMT_MXFP4) quant<MOE_FMT_MXFP4>(K, T, x, x_stride, codes, scales, stream);
  else quant<MOE_FMT_MXFP8>(K, T, x, x_stride, codes, scales, stream);
  return hipGetLastError();
}

}  // namespace moe
