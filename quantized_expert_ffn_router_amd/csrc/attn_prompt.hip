// attn_prompt.hip -- causal attention over packed prompts.
//
// A prompt's attention is the other half of a prefill (basalt.jgulfo.com, "All
// the numbers", quotes prompt rates beside decode rates).  Work is one tile of
// query rows of one head: one pass over the keys the tile sees, with the running
// maximum and sum of the softmax, everything but the keys and values in
// registers:
//   scores^T (64 tokens x 32 rows of a wave) = K Q^T,  out^T (D x 32) += V^T P^T
// as 32x32x16 bf16 matrix instructions.  A lane column is one query row, so the
// softmax statistics are per-lane scalars (one swap between the wave's halves
// per tile), and the score accumulators, rounded to bf16, are the operand of
// the second product as they lie; V's fragments come out of LDS transposed
// (ds_read_b64_tr_b16) with their tokens in the same order.
#include "attn_common.h"

namespace moe {

namespace {

typedef __bf16 v8b __attribute__((ext_vector_type(8)));
typedef float v16f __attribute__((ext_vector_type(16)));
typedef uint32_t v4u __attribute__((ext_vector_type(4)));
typedef short v4s __attribute__((ext_vector_type(4)));

constexpr int kBN = 64;            // keys of a tile
constexpr float kNone = -3.0e38f;  // running maximum before any token
constexpr float kGrow = 8.0f;      // log2 headroom before the accumulators are rescaled

struct PromptArgs {
  const int32_t* q_start;
  const int32_t* kv_start;
  const uint16_t* q;
  const uint16_t* k;
  const uint16_t* v;
  uint16_t* out;
  int64_t q_stride, k_stride, v_stride, out_stride, T, Tk;
  int n_q, G, n_seq;
  float c;  // scale * log2(e)
};

__device__ __forceinline__ v16f mma(v4u a, v4u b, v16f c) {
  return __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(v8b, a),
                                                 __builtin_bit_cast(v8b, b), c, 0, 0, 0);
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

// 64 rows of a K or V head into an LDS tile, straight from global memory: lane
// i of a load fills the 16 bytes at slot i, and reads the chunk that belongs
// there.  Rows past the last one are read as the last one (masked later).
template <int D, int WAVES>
__device__ __forceinline__ void load_tile(uint8_t* lds, const uint16_t* __restrict__ src,
                                          int64_t stride, int64_t t0, int64_t last, int wave,
                                          int lane) {
  constexpr int CPR = D / 8;                    // chunks of a row
  constexpr int LOADS = kBN * CPR / 64 / WAVES;  // loads of a wave
#pragma unroll
  for (int i = 0; i < LOADS; ++i) {
    const int slot = (i * WAVES + wave) * 64 + lane;
    const int row = slot / CPR, chunk = swz<D>(row, slot % CPR);
    const uint16_t* p = src + min(t0 + row, last) * stride + chunk * 8;
    __builtin_amdgcn_global_load_lds(
        (const __attribute__((address_space(1))) void*)p,
        (__attribute__((address_space(3))) void*)(lds + (i * WAVES + wave) * 1024), 16, 0, 0);
  }
}

template <int D, int WAVES>
__global__ __launch_bounds__(64 * WAVES) void k_attn_prompt(PromptArgs a) {
  constexpr int KS = D / 16, NJ = D / 32, BM = 32 * WAVES, TILE = kBN * D * 2;
  extern __shared__ __align__(16) uint8_t lds[];  // two buffers of a K and a V tile
  const int wave = threadIdx.x >> 6, lane = lane_id(), n = lane & 31, h = lane >> 5;

  // row tiles of all sequences, the last ones (the most keys) first
  const int head = (int)(blockIdx.x % a.n_q);
  int64_t total = 0;
  for (int i0 = 0; i0 < a.n_seq; i0 += 64) {
    int64_t m = 0;
    if (i0 + lane < a.n_seq)
      m = (max((int64_t)a.q_start[i0 + lane + 1] - a.q_start[i0 + lane], (int64_t)0) + BM - 1) / BM;
#pragma unroll
    for (int d = 32; d; d >>= 1) m += __shfl_xor(m, d);
    total += m;
  }
  const int64_t want = total - 1 - (int64_t)(blockIdx.x / a.n_q);
  if (want < 0) return;
  int b = -1;
  int64_t base = 0, tile = 0;
  for (int i0 = 0; i0 < a.n_seq; i0 += 64) {
    int64_t m = 0;
    if (i0 + lane < a.n_seq)
      m = (max((int64_t)a.q_start[i0 + lane + 1] - a.q_start[i0 + lane], (int64_t)0) + BM - 1) / BM;
    int64_t sum = m;
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
      const int64_t v = __shfl_up(sum, d);
      if (lane >= d) sum += v;
    }
    const uint64_t past = __ballot(base + sum > want);
    if (past) {
      const int l = __ffsll((unsigned long long)past) - 1;
      b = i0 + l;
      tile = want - (base + __shfl(sum, l) - __shfl(m, l));
      break;
    }
    base += __shfl(sum, 63);
  }
  if (b < 0) return;

  const int64_t r0 = a.q_start[b], rows = (int64_t)a.q_start[b + 1] - r0;
  const int64_t k0 = a.kv_start[b], len = (int64_t)a.kv_start[b + 1] - k0;
  const int64_t i_wg = tile * BM, i_row = i_wg + wave * 32 + n;
  const bool live = i_row < rows && r0 + i_row >= 0 && r0 + i_row < a.T;
  const bool keys = k0 >= 0 && k0 + len <= a.Tk;  // else nothing is read and the rows are NaN
  const int64_t limit = live && keys ? len - rows + i_row : -1;
  const int64_t hi = keys ? len - rows + min(i_wg + BM, rows) - 1 : -1;  // last key of the tile's rows
  const int64_t lo_wave = len - rows + i_wg + wave * 32;  // key that all rows of the wave see
  const int n_tiles = hi < 0 ? 0 : (int)(hi / kBN) + 1;

  const uint16_t* kp = a.k + k0 * a.k_stride + (int64_t)(head / a.G) * D;
  const uint16_t* vp = a.v + k0 * a.v_stride + (int64_t)(head / a.G) * D;
  v4u qf[KS];
  {
    const uint16_t* qp = a.q + (live ? r0 + i_row : 0) * a.q_stride + (int64_t)head * D + 8 * h;
#pragma unroll
    for (int s = 0; s < KS; ++s) qf[s] = *reinterpret_cast<const v4u*>(qp + 16 * s);
  }
  v16f o[NJ];
#pragma unroll
  for (int j = 0; j < NJ; ++j)
#pragma unroll
    for (int i = 0; i < 16; ++i) o[j][i] = 0.0f;
  float m = kNone, l = 0.0f;

  // addresses of this lane's transposed reads: row r + ..., 4 elements
  const int vrow = 4 * h + ((lane & 15) >> 2), vcol = ((lane >> 4) & 1) * 16 + 4 * (lane & 3);

  if (n_tiles > 0) {
    load_tile<D, WAVES>(lds, kp, a.k_stride, 0, len - 1, wave, lane);
    load_tile<D, WAVES>(lds + TILE, vp, a.v_stride, 0, len - 1, wave, lane);
  }
  for (int it = 0; it < n_tiles; ++it) {
    uint8_t* kt = lds + (it & 1) * 2 * TILE;
    uint8_t* vt = kt + TILE;
    __builtin_amdgcn_s_waitcnt(0x0f70);  // vmcnt(0): this wave's part of the tile
    __syncthreads();  // the whole tile has arrived, the other buffer has been read
    if (it + 1 < n_tiles) {
      uint8_t* nx = lds + ((it + 1) & 1) * 2 * TILE;
      load_tile<D, WAVES>(nx, kp, a.k_stride, (int64_t)(it + 1) * kBN, len - 1, wave, lane);
      load_tile<D, WAVES>(nx + TILE, vp, a.v_stride, (int64_t)(it + 1) * kBN, len - 1, wave, lane);
    }
    const int64_t t0 = (int64_t)it * kBN;
    v16f x[2];
#pragma unroll
    for (int t = 0; t < 2; ++t) {
#pragma unroll
      for (int i = 0; i < 16; ++i) x[t][i] = 0.0f;
#pragma unroll
      for (int s = 0; s < KS; ++s) {
        const int row = 32 * t + n;
        const v4u f = *reinterpret_cast<const v4u*>(kt + row * (2 * D) + swz<D>(row, 2 * s + h) * 16);
        x[t] = mma(f, qf[s], x[t]);
      }
    }
    const bool edge = t0 + kBN - 1 > lo_wave;  // some row does not see all of it
    if (edge) {
#pragma unroll
      for (int t = 0; t < 2; ++t)
#pragma unroll
        for (int i = 0; i < 16; ++i)
          if (t0 + 32 * t + 8 * (i >> 2) + 4 * h + (i & 3) > limit) x[t][i] = -__builtin_inff();
    }
    float mx = x[0][0];
#pragma unroll
    for (int t = 0; t < 2; ++t)
#pragma unroll
      for (int i = 0; i < 16; ++i) mx = fmaxf(mx, x[t][i]);
    {
      const uint32_t u = __float_as_uint(mx);
      const auto w = __builtin_amdgcn_permlane32_swap(u, u, false, false);
      mx = fmaxf(__uint_as_float(w[0]), __uint_as_float(w[1])) * a.c;
    }
    if (__any(mx > m + kGrow)) {
      const float mn = fmaxf(m, mx), al = __builtin_amdgcn_exp2f(m - mn);
#pragma unroll
      for (int j = 0; j < NJ; ++j)
#pragma unroll
        for (int i = 0; i < 16; ++i) o[j][i] *= al;
      l *= al;
      m = mn;
    }
    v4u p[4];
#pragma unroll
    for (int t = 0; t < 2; ++t)
#pragma unroll
      for (int i = 0; i < 16; i += 2) {
        const float e0 = __builtin_amdgcn_exp2f(fmaf(x[t][i], a.c, -m));
        const float e1 = __builtin_amdgcn_exp2f(fmaf(x[t][i + 1], a.c, -m));
        l += e0;
        l += e1;
        typedef __bf16 v2b __attribute__((ext_vector_type(2)));
        const v2b w = {(__bf16)e0, (__bf16)e1};
        p[2 * t + (i >> 3)][(i & 7) >> 1] = __builtin_bit_cast(uint32_t, w);
      }
    bool wild = false;
    if (edge) {
      // infinities or NaN among values that some row does not see
      bool any = false;
#pragma unroll 1
      for (int i = lane; i < TILE / 16; i += 64) {
        const v4u f = reinterpret_cast<const v4u*>(vt)[i];
#pragma unroll
        for (int w = 0; w < 4; ++w)
          any |= (f[w] & 0x7f80u) == 0x7f80u || (f[w] & 0x7f800000u) == 0x7f800000u;
      }
      wild = __any(any);
    }
#pragma unroll
    for (int s = 0; s < 4; ++s) {
#pragma unroll
      for (int j = 0; j < NJ; ++j) {
        v4u f;
#pragma unroll
        for (int q = 0; q < 2; ++q) {
          const int row = 16 * s + 8 * q + vrow, col = 32 * j + vcol;
          const uint8_t* ad = vt + row * (2 * D) + swz<D>(row, col >> 3) * 16 + (col & 4) * 2;
          const v4s r = __builtin_amdgcn_ds_read_tr16_b64_v4i16(
              (__attribute__((address_space(3))) v4s*)(ad));
          const uint2 w = __builtin_bit_cast(uint2, r);
          f[2 * q] = w.x; f[2 * q + 1] = w.y;
        }
        if (!wild) {
          o[j] = mma(f, p[s], o[j]);
        } else {
          // A zero weight would not silence them: one token at a time, added
          // only to the rows that see it.
#pragma unroll 1
          for (int tk = 0; tk < 16; ++tk) {
            const bool mine = h == ((tk >> 2) & 1);
            const bool seen = t0 + 16 * s + tk <= limit;
            const int at = 2 * (tk >> 3) + ((tk & 3) >> 1);
            const uint32_t keep = mine ? 0xffffu << (16 * (tk & 1)) : 0u;
            v4u one;
#pragma unroll
            for (int i = 0; i < 4; ++i) one[i] = i == at ? f[i] & keep : 0u;
            v16f z;
#pragma unroll
            for (int i = 0; i < 16; ++i) z[i] = 0.0f;
            z = mma(one, p[s], z);
#pragma unroll
            for (int i = 0; i < 16; ++i) o[j][i] += seen ? z[i] : 0.0f;
          }
        }
      }
    }
  }
  {
    const uint32_t u = __float_as_uint(l);
    const auto w = __builtin_amdgcn_permlane32_swap(u, u, false, false);
    l = __uint_as_float(w[0]) + __uint_as_float(w[1]);
  }
  if (!live) return;
  const float inv = !keys ? __uint_as_float(0x7fc00000u) : limit < 0 ? 0.0f : 1.0f / l;
  uint16_t* d = a.out + (r0 + i_row) * a.out_stride + (int64_t)head * D + 4 * h;
#pragma unroll
  for (int j = 0; j < NJ; ++j)
#pragma unroll
    for (int i = 0; i < 16; i += 4) {
      const uint32_t w0 = (uint32_t)f32_to_bf16_rne(o[j][i] * inv) | ((uint32_t)f32_to_bf16_rne(o[j][i + 1] * inv) << 16);
      const uint32_t w1 = (uint32_t)f32_to_bf16_rne(o[j][i + 2] * inv) | ((uint32_t)f32_to_bf16_rne(o[j][i + 3] * inv) << 16);
      *reinterpret_cast<uint2*>(d + 32 * j + 2 * i) = make_uint2(w0, w1);
    }
}

template <int D, int WAVES>
hipError_t launch(const PromptArgs& a, hipStream_t stream) {
  constexpr int lds = 4 * kBN * D * 2;
  const int64_t tiles = a.T / (32 * WAVES) + a.n_seq;  // at most: one part tile a sequence
  const hipError_t e = hipFuncSetAttribute(reinterpret_cast<const void*>(&k_attn_prompt<D, WAVES>),
                                           hipFuncAttributeMaxDynamicSharedMemorySize, lds);
  if (e != hipSuccess) return e;
  k_attn_prompt<D, WAVES><<<(unsigned)(tiles * a.n_q), 64 * WAVES, lds, stream>>>(a);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_attn_prompt(int n_q, int n_kv, int D, int n_seq, const int32_t* q_start,
                              const int32_t* kv_start, int64_t T, int64_t Tk, const uint16_t* q,
                              int64_t q_stride, const uint16_t* k, int64_t k_stride,
                              const uint16_t* v, int64_t v_stride, float scale, uint16_t* out,
                              int64_t out_stride, hipStream_t stream) {
  const PromptArgs a{q_start, kv_start ? kv_start : q_start, q, k, v, out, q_stride, k_stride,
                     v_stride, out_stride, T, Tk, n_q, n_q / n_kv, n_seq,
                     scale * 1.4426950408889634f};
  switch (D) {
    case 64: return launch<64, 4>(a, stream);
    case 128: return launch<128, 4>(a, stream);
    default: return launch<256, 4>(a, stream);
  }
}

}  // namespace moe
