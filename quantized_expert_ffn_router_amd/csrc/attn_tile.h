// attn_tile.h -- tiles of 64 keys against a wave's 32 query rows: what the prompt and the
// chunk kernels share.
#pragma once

#include "attn_common.h"

namespace moe {

namespace {

typedef __bf16 v8b __attribute__((ext_vector_type(8)));
typedef _Float16 v8h __attribute__((ext_vector_type(8)));
typedef float v16f __attribute__((ext_vector_type(16)));
typedef uint32_t v4u __attribute__((ext_vector_type(4)));
typedef short v4s __attribute__((ext_vector_type(4)));

constexpr int kBN = 64;  // keys of a tile

// HALF: operands of fp16, not bf16.
template <bool HALF = false>
__device__ __forceinline__ v16f mma(v4u a, v4u b, v16f c) {
  if constexpr (HALF)
    return __builtin_amdgcn_mfma_f32_32x32x16_f16(__builtin_bit_cast(v8h, a), __builtin_bit_cast(v8h, b), c, 0, 0, 0);
  else
    return __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(v8b, a), __builtin_bit_cast(v8b, b), c, 0, 0, 0);
}

// Place of 16-byte chunk `chunk` of row `row` in an LDS tile of D-wide rows:
// chunks are permuted within their row so that neither the row-wise reads of K
// (32 rows, one chunk column) nor the transposed reads of V (4 rows, 4 chunk
// columns) meet twice in a bank.
template <int D>
__device__ __forceinline__ int swz(int row, int chunk) {
  if constexpr (D == 64) return chunk ^ (((row & 1) << 2) | ((row >> 1) & 3));
  else return chunk ^ (((row & 3) << 2) | ((row >> 2) & 3));
}

// Waits until at most N of the wave's loads are on their way (its newest ones).
template <int N>
__device__ __forceinline__ void wait_loads() {
#if defined(__HIP_DEVICE_COMPILE__)
  __builtin_amdgcn_s_waitcnt((N & 15) | ((N >> 4) << 14) | 0x0f70);
#endif
}

// Two softmax weights in the operand type of the second product, rounded to
// nearest even (half a step: 2^-8, fp16 2^-11), and their sum added to l -- of the
// rounded weights, so that rounding does not shift a row's mean.
template <bool HALF>
__device__ __forceinline__ uint32_t weight_pair(float a, float b, float* l) {
  typedef __bf16 v2b __attribute__((ext_vector_type(2)));
  if constexpr (HALF) {
    const v2h w = {(_Float16)a, (_Float16)b}, one = {(_Float16)1.0f, (_Float16)1.0f};
    *l = __builtin_amdgcn_fdot2(w, one, *l, false);
    return __builtin_bit_cast(uint32_t, w);
  }
  const v2b w = {(__bf16)a, (__bf16)b};
  const v2b one = {(__bf16)1.0f, (__bf16)1.0f};
  *l = __builtin_amdgcn_fdot2_f32_bf16(w, one, *l, false);
  return __builtin_bit_cast(uint32_t, w);
}

// What a wave carries for 32 query rows: a lane column is one row, its accumulators and
// statistics the lane's own.
template <int D, bool HALF = false>
struct TileRows {
  static constexpr int KS = D / 16, NJ = D / 32;
  v4u qf[KS];
  v16f o[NJ];
  float m, l;
  int64_t limit;  // this lane's row: last key it sees
  int h;          // half of the wave

  __device__ __forceinline__ void clear() {
#pragma unroll
    for (int j = 0; j < NJ; ++j)
#pragma unroll
      for (int i = 0; i < 16; ++i) o[j][i] = 0.0f;
    m = kNone;
    l = 0.0f;
  }
  __device__ __forceinline__ void mask(v16f (&x)[2], int64_t t0) const {
    const int left = (int)min(max(limit - t0, (int64_t)-1), (int64_t)kBN) - 4 * h;
#pragma unroll
    for (int t = 0; t < 2; ++t)
#pragma unroll
      for (int i = 0; i < 16; ++i)
        if (32 * t + 8 * (i >> 2) + (i & 3) > left) x[t][i] = -__builtin_inff();
  }
  // Largest scaled score of this lane's row.
  __device__ __forceinline__ float top(const v16f (&x)[2], float c) const {
    float mx = x[0][0];
#pragma unroll
    for (int t = 0; t < 2; ++t)
#pragma unroll
      for (int i = 0; i < 16; ++i) mx = fmaxf(mx, x[t][i]);
    return over_halves(mx) * c;
  }
  // The larger of a row's two lanes.
  __device__ __forceinline__ static float over_halves(float mx) {
    const uint32_t u = __float_as_uint(mx);
    const auto w = __builtin_amdgcn_permlane32_swap(u, u, false, false);
    return fmaxf(__uint_as_float(w[0]), __uint_as_float(w[1]));
  }
  // The lane's sum, over both halves of the wave.
  __device__ __forceinline__ void finish() {
    const uint32_t u = __float_as_uint(l);
    const auto s = __builtin_amdgcn_permlane32_swap(u, u, false, false);
    l = __uint_as_float(s[0]) + __uint_as_float(s[1]);
  }
  // Weight v of the tile's 32 per lane; a pair is rounded when its second value
  // is there.
  __device__ __forceinline__ void weight(v16f (&x)[2], float c, v4u (&p)[4], int v) {
    const int t = v >> 4, i = v & 15;
    x[t][i] = __builtin_amdgcn_exp2f(fmaf(x[t][i], c, -m));
    if (i & 1) p[v >> 3][(i & 7) >> 1] = weight_pair<HALF>(x[t][i - 1], x[t][i], &l);
  }
  // The scores y of one tile and the weighted values of the tile before (scores x), as one
  // stream: a matrix instruction, then a piece of the softmax in its shadow, and
  // fragments, key(half, step) and value(step, block), read kAhead steps early.  A weight
  // is ready when its step of the second product begins: 20 of a lane's 32 go
  // with the first product, the rest with the first three quarters of the second.
  // NEXT false: there is no next tile, only the weighted values.  also(I): the caller's
  // own work beside matrix instruction I (a type).
  template <bool NEXT, typename K, typename V, typename A>
  __device__ __forceinline__ void stream(K key, V value, float c, v16f (&x)[2], v16f (&y)[2], A also) {
    constexpr int N1 = 2 * KS, N2 = 4 * NJ, kAhead = 3, kRing = 4;
    v4u f[kRing], p[4];
    const auto fragment = [&](int i) {
      return i < N1 ? key(i / KS, i % KS) : value((i - N1) / NJ, (i - N1) % NJ);
    };
    const auto weights_by = [](int i) {
      return i < 0 ? 0 : i < N1 ? 20 * (i + 1) / N1 : min(32, 20 + 12 * (i - N1 + 1) / (3 * NJ));
    };
    constexpr int I0 = NEXT ? 0 : N1;
#pragma unroll
    for (int i = I0; i < I0 + kAhead; ++i) f[i % kRing] = fragment(i);
    if constexpr (!NEXT) {
#pragma unroll
      for (int v = 0; v < weights_by(N1 - 1); ++v) weight(x, c, p, v);
    }
    each<I0, N1 + N2>([&](auto I) {
      constexpr int i = I();
      if (i + kAhead < N1 + N2) f[(i + kAhead) % kRing] = fragment(i + kAhead);
      if constexpr (i < N1) {
        v16f zero;
#pragma unroll
        for (int k = 0; k < 16; ++k) zero[k] = 0.0f;
        y[i / KS] = mma<HALF>(f[i % kRing], qf[i % KS], i % KS ? y[i / KS] : zero);
      } else {
        constexpr int s = (i - N1) / NJ, j = (i - N1) % NJ;
        o[j] = mma<HALF>(f[i % kRing], p[s], o[j]);
      }
#pragma unroll
      for (int v = weights_by(i - 1); v < weights_by(i); ++v) weight(x, c, p, v);
      also(I);
      __builtin_amdgcn_sched_barrier(0);
    });
  }
};

}  // namespace

}  // namespace moe
