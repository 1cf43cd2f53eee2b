// kv_cache.hip -- the paged key/value cache: what writes it (norms of queries
// and keys per head, rotary positions, quantisation, in one pass over the
// projections' output) and what reads it back as bf16 rows.
//
// The cache's precision is a choice against the experts' memory
// (aiopssre.com, "Concurrency divides context unless you pay for more cache");
// layout and rounding are stated in moe.h.
#include <type_traits>

#include "attn_common.h"

namespace moe {

namespace {

constexpr int kRows = 4;  // rows (waves) of an append workgroup

// Orders a wave's own LDS writes before its reads (no other wave is involved).
__device__ __forceinline__ void wave_lds_fence() {
  __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
  __builtin_amdgcn_wave_barrier();
}

__device__ __forceinline__ float lo16(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float hi16(uint32_t w) { return __uint_as_float(w & 0xffff0000u); }

// Sum over groups of N lanes (8, 16 or 32): within a row of 16 by lane
// permutations of the adder's operand.
template <int CTRL>
__device__ __forceinline__ float dpp(float v) {
  const int i = __float_as_int(v);
  return __int_as_float(__builtin_amdgcn_update_dpp(i, i, CTRL, 0xf, 0xf, true));
}
template <int CTRL>
__device__ __forceinline__ double dpp(double v) {
  const uint64_t u = __builtin_bit_cast(uint64_t, v);
  const int lo = (int)u, hi = (int)(u >> 32);
  const uint32_t l = __builtin_amdgcn_update_dpp(lo, lo, CTRL, 0xf, 0xf, true);
  const uint32_t h = __builtin_amdgcn_update_dpp(hi, hi, CTRL, 0xf, 0xf, true);
  return __builtin_bit_cast(double, ((uint64_t)h << 32) | l);
}
template <int N, typename T>
__device__ __forceinline__ T group_sum(T v) {
  v += dpp<0xb1>(v);   // lane ^ 1
  v += dpp<0x4e>(v);   // lane ^ 2
  v += dpp<0x141>(v);  // mirrored in 8: the other four
  if constexpr (N >= 16) v += dpp<0x140>(v);  // mirrored in 16: the other eight
  if constexpr (N >= 32) v += __shfl_xor(v, 16);
  return v;
}

// The largest magnitude of 8 bf16 values, as bits (so that an infinity or a
// NaN, 0x7f80 or more, wins).
__device__ __forceinline__ uint32_t top_bits(uint4 x) {
  uint32_t m = 0;
  const uint32_t w[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) m = max(m, max(w[i] & 0x7fffu, (w[i] >> 16) & 0x7fffu));
  return m;
}

// The 8-bit codes and the scale of 8 values of a block of 32 (4 lanes).
__device__ __forceinline__ uint2 q8_codes(uint4 x, uint16_t* scale) {
  uint32_t top = top_bits(x);
  top = max(top, (uint32_t)__shfl_xor((int)top, 1));
  top = max(top, (uint32_t)__shfl_xor((int)top, 2));
  const float v[8] = {lo16(x.x), hi16(x.x), lo16(x.y), hi16(x.y),
                      lo16(x.z), hi16(x.z), lo16(x.w), hi16(x.w)};
  const _Float16 d = top >= 0x7f80u
                         ? __builtin_bit_cast(_Float16, (uint16_t)0x7e00)
                         : (_Float16)(fminf(__uint_as_float(top << 16), 65024.0f) / 127.0f);
  const float df = (float)d;
  uint32_t q[2] = {0, 0};
  if (df > 0.0f) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int c = (int)fminf(fmaxf(rintf(v[i] / df), -127.0f), 127.0f);
      q[i >> 2] |= (uint32_t)(c & 0xff) << (8 * (i & 3));
    }
  }
  *scale = __builtin_bit_cast(uint16_t, d);
  return make_uint2(q[0], q[1]);
}

// Quantises 8 values (elements 8n..8n+7 of token o) of a key or value head and
// stores them; all lanes take part in the block maximum (store: whether this
// lane's head belongs to the cache at all).
template <int FMT, int D>
__device__ __forceinline__ void store_token(uint8_t* __restrict__ blk, const KvLayout lay, int P,
                                            int o, int n, bool is_v, float ts, uint4 x,
                                            bool store) {
  if constexpr (FMT == MOE_FMT_BF16) {
    if (!store) return;
    uint16_t* p = reinterpret_cast<uint16_t*>(blk + (is_v ? lay.vq : 0));
    if (!is_v) {
      *reinterpret_cast<uint4*>(p + o * D + 8 * n) = x;
    } else {
      p += ((o >> 2) * D + 8 * n) * 4 + (o & 3);
      const uint32_t w[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        p[8 * i] = (uint16_t)w[i];
        p[8 * i + 4] = (uint16_t)(w[i] >> 16);
      }
    }
    return;
  }
  if constexpr (FMT == MOE_FMT_Q8_0) {
    uint16_t d;
    const uint2 q = q8_codes(x, &d);
    if (!store) return;
    if (!is_v) {
      *reinterpret_cast<uint2*>(blk + o * D + 8 * n) = q;
      if (!(n & 3)) *reinterpret_cast<uint16_t*>(blk + lay.ks + 2 * (o * (D / 32) + (n >> 2))) = d;
    } else {
      uint8_t* p = blk + lay.vq + ((o >> 2) * D + 8 * n) * 4 + (o & 3);
#pragma unroll
      for (int i = 0; i < 8; ++i) p[4 * i] = (uint8_t)((i < 4 ? q.x : q.y) >> (8 * (i & 3)));
      if (!(n & 3)) *reinterpret_cast<uint16_t*>(blk + lay.vs + 2 * ((n >> 2) * P + o)) = d;
    }
    return;
  }
  uint32_t top = top_bits(x);
  top = max(top, (uint32_t)__shfl_xor((int)top, 1));
  if (!store) return;
  const float amax = __uint_as_float(top << 16);
  const bool bad = top >= 0x7f80u;
  const float v[8] = {lo16(x.x), hi16(x.x), lo16(x.y), hi16(x.y),
                      lo16(x.z), hi16(x.z), lo16(x.w), hi16(x.w)};
  if constexpr (FMT == MOE_FMT_NVFP4) {
    const float a = fminf(amax / (6.0f * ts), 448.0f);
    const uint32_t sb = bad ? 0x7fu : (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(a, a, 0, false) & 0xffu;
    const float den = bad ? 0.0f : e4m3_to_f32(sb) * ts;
    uint32_t q = 0;
    if (den > 0.0f) {
      q = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(q, v[0] / den, v[1] / den, 1.0f, 0);
      q = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(q, v[2] / den, v[3] / den, 1.0f, 1);
      q = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(q, v[4] / den, v[5] / den, 1.0f, 2);
      q = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(q, v[6] / den, v[7] / den, 1.0f, 3);
    }
    if (!is_v) {
      *reinterpret_cast<uint32_t*>(blk + o * (D / 2) + 4 * n) = q;
      if (!(n & 1)) blk[lay.ks + o * (D / 16) + (n >> 1)] = (uint8_t)sb;
    } else {
      uint8_t* p = blk + lay.vq;
      const int quad = (o >> 2) * 16, b = o & 3;
      if constexpr (D == 64) {  // groups of 4 elements
        *reinterpret_cast<uint16_t*>(p + ((quad + 2 * n) * 4 + b) * 2) = (uint16_t)q;
        *reinterpret_cast<uint16_t*>(p + ((quad + 2 * n + 1) * 4 + b) * 2) = (uint16_t)(q >> 16);
      } else if constexpr (D == 128) {
        *reinterpret_cast<uint32_t*>(p + ((quad + n) * 4 + b) * 4) = q;
      } else {
        *reinterpret_cast<uint32_t*>(p + ((quad + (n >> 1)) * 4 + b) * 8 + 4 * (n & 1)) = q;
      }
      if (!(n & 1)) blk[lay.vs + (n >> 1) * P + o] = (uint8_t)sb;
    }
  }
}

// Sine and cosine of an angle in fp64: reduced by multiples of pi/2 held in two
// parts (the products are exact inside the fused operations, so positions up to
// 2^31 lose nothing), then the Taylor series to x^15 and x^16, whose remainders
// are below 2^-54 for |x| <= pi/4.
__device__ __forceinline__ void sin_cos(double a, double* s, double* c) {
  const double n = rint(a * 0.63661977236758134);
  const double x = fma(-n, 6.123233995736766e-17, fma(-n, 1.5707963267948966, a)), z = x * x;
  double p = -1.0 / 1307674368000.0, q = 1.0 / 20922789888000.0;
  p = fma(p, z, 1.0 / 6227020800.0);  q = fma(q, z, -1.0 / 87178291200.0);
  p = fma(p, z, -1.0 / 39916800.0);   q = fma(q, z, 1.0 / 479001600.0);
  p = fma(p, z, 1.0 / 362880.0);      q = fma(q, z, -1.0 / 3628800.0);
  p = fma(p, z, -1.0 / 5040.0);       q = fma(q, z, 1.0 / 40320.0);
  p = fma(p, z, 1.0 / 120.0);         q = fma(q, z, -1.0 / 720.0);
  p = fma(p, z, -1.0 / 6.0);          q = fma(q, z, 1.0 / 24.0);
  p = fma(p * z, x, x);               q = fma(q, z, -0.5);
  q = fma(q, z, 1.0);
  const int k = (int)(long long)n & 3;  // quarter turns
  const double u = k & 1 ? q : p, v = k & 1 ? p : q;
  *s = k & 2 ? -u : u;
  *c = (k + 1) & 2 ? -v : v;
}

struct AppendArgs {
  const uint16_t* qkv;
  uint16_t* q_out;
  uint16_t* k_out;
  const int32_t* pos;
  const float* q_norm;
  const float* k_norm;
  const double* inv_freq;
  uint8_t* pool;
  int64_t qkv_stride, q_stride, k_stride, T;
  SeqView s;
  int n_q, n_kv, rot, interleaved;
  float eps, rope_scale, k_ts, v_ts;
};

// 8 elements of a head: z * w / rms(z), then the rotation of the lane's four
// pairs: (z[i], z[i + 4]) where the lane holds both halves' elements, neighbours
// otherwise.  T: float for queries (a few 2^-24, against the 2^-8 of the
// rounding to bf16), double for keys.  The squares are summed in fp64 for both:
// those of a bf16 value may lie outside fp32.
template <int LPH, int D, typename T>
__device__ __forceinline__ void norm_turn(T (&z)[8], const float (&w)[8], bool normed, float eps,
                                          bool halves, bool turn, const T (&cs)[8]) {
  if (normed) {
    double ss = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) ss = fma((double)z[i], (double)z[i], ss);
    ss = group_sum<LPH>(ss);
    double r = rsqrt(ss / (double)D + (double)eps);
    if (sizeof(T) == 4 && r > 0x1p100) {  // (beyond fp32 for the smallest values)
      r *= 0x1p-64;
#pragma unroll
      for (int i = 0; i < 8; ++i) z[i] *= (T)0x1p64;
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) z[i] = z[i] * (T)r * (T)w[i];
  }
  if (turn) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const T zu = halves ? z[i] : z[2 * i], zv = halves ? z[i + 4] : z[2 * i + 1];
      const T nu = zu * cs[2 * i] - zv * cs[2 * i + 1], nv = zv * cs[2 * i] + zu * cs[2 * i + 1];
      z[halves ? i : 2 * i] = nu;
      z[halves ? i + 4 : 2 * i + 1] = nv;
    }
  }
}

// Buffer accesses of 8 bytes a lane at a byte offset: nothing happens (a load
// gives 0) from `bytes` on.
#if defined(__HIP_DEVICE_COMPILE__)  // (the host pass does not know the builtins)
typedef __amdgpu_buffer_rsrc_t Rsrc;
#else
typedef const void* Rsrc;
#endif
__device__ __forceinline__ Rsrc buffer_of(const uint16_t* p, int bytes) {
#if defined(__HIP_DEVICE_COMPILE__)
  return __builtin_amdgcn_make_buffer_rsrc(const_cast<uint16_t*>(p), 0, bytes, 0x00020000);
#else
  return p;
#endif
}
__device__ __forceinline__ uint2 load_8(Rsrc r, uint32_t at) {
#if defined(__HIP_DEVICE_COMPILE__)
  const auto x = __builtin_amdgcn_raw_buffer_load_b64(r, at, 0, 0);
  return make_uint2(x[0], x[1]);
#else
  return make_uint2(0, 0);
#endif
}
__device__ __forceinline__ void store_8(Rsrc r, uint32_t at, uint2 x) {
#if defined(__HIP_DEVICE_COMPILE__)
  typedef uint32_t v2u __attribute__((ext_vector_type(2)));
  __builtin_amdgcn_raw_buffer_store_b64(v2u{x.x, x.y}, r, at, 0, 0);
#endif
}

// One wave per row, D/8 lanes per head, 64/(D/8) heads at a time: the row's
// queries, then its keys, then its values, the next group's elements on their way
// while one is worked on.  The row's angles are taken once, in fp64 (a far
// position times a frequency needs more than 24 bits), and kept in the wave's
// LDS.  Queries are normed and rotated in fp32.  Keys are in fp64 (as many fp64
// as plain fp32 operations run per cycle here), so that the codes in the cache do
// not hang on the order of a sum: they go through LDS into 8 consecutive elements
// a lane, the unit of quantisation.
// HALVES: the rotation pairs elements of the head's two halves (i, i + rot/2).
//
// QUADS (the formats that keep four tokens' values side by side): the four waves
// take the tokens of one aligned quad of a sequence, so that the quad's values
// are written as whole pieces, put together in LDS; a quad that is not whole in
// this call is written value by value.  16384 rows (bf16 cache) 95 us without, 70
// with it.
//
// Bound by memory, one read and one write of everything: 16384 rows of 40 heads of
// 128 into a bf16 cache 70 us, 5.0 TB/s (a large copy reaches 5.15); 4096 rows
// into NVFP4 19 us, 4.3 TB/s.  A decode step's 8 rows take 4.4 us, the launch and
// one chain of loads.
template <int FMT, int D, bool HALVES>
__global__ __launch_bounds__(64 * kRows) void k_kv_append(AppendArgs a) {
  constexpr int LPH = D / 8, HPW = 64 / LPH;
  constexpr bool QUADS = FMT != MOE_FMT_NVFP4;
  constexpr int VB = FMT == MOE_FMT_BF16 ? 2 : 1;  // bytes of a value
  __shared__ double2 cs_s[kRows][128];
  __shared__ __align__(16) uint16_t k_s[kRows][HPW][D];
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = lane_id();
  int64_t t = (int64_t)blockIdx.x * kRows + wave;  // row
  RowSeq q;
  bool mine = true, whole = false;  // there is such a row; all rows of the quad are there
  if constexpr (QUADS) {
    int64_t first, last;
    q = find_quad(a.s, a.T, blockIdx.x, &first, &last, &t);
    if (q.b < 0) return;
    whole = t >= first && t + 3 <= last;
    t += wave;
    mine = t >= first && t <= last;
  } else if (t >= a.T) {
    return;
  }
  const int n = lane % LPH, g = lane / LPH;
  const int n_q = __builtin_amdgcn_readfirstlane(a.n_q), n_kv = __builtin_amdgcn_readfirstlane(a.n_kv);
  const int q_groups = (n_q + HPW - 1) / HPW, kv_groups = (n_kv + HPW - 1) / HPW;
  const int groups = q_groups + 2 * kv_groups, step = gridDim.y;
  const uint16_t* row = a.qkv + t * a.qkv_stride;
  // places of the lane's 8 elements in a query or key head: 4 pairs
  const bool split = HALVES && n < a.rot / 8;
  const bool turn = HALVES ? split : 8 * n < a.rot;
  const int a0 = split ? 4 * n : 8 * n, b0 = split ? a.rot / 2 + 4 * n : 8 * n + 4;

  // head of this lane in a group (of its kind), -1: none
  const auto head_of = [&](int u) {
    const int k = u < q_groups ? u : u < q_groups + kv_groups ? u - q_groups : u - q_groups - kv_groups;
    const int h = k * HPW + g;
    return h < (u < q_groups ? n_q : n_kv) ? h : -1;
  };
  // Buffer accesses, out of range where there is no head (or row): no access is
  // behind a branch, which would make every wait for a load one for the stores
  // after it, too (16384 rows 70 us, with branches 85).
  constexpr uint32_t kNowhere = 0x80000000u;
  const Rsrc from = buffer_of(row, mine ? (n_q + 2 * n_kv) * D * 2 : 0);
  const auto fetch = [&](int u, uint2& xa, uint2& xb) {
    const int h = u < groups ? head_of(u) : -1;
    const bool v = u >= q_groups + kv_groups;
    const uint32_t at = 2 * (h + (u < q_groups ? 0 : v ? n_q + n_kv : n_q)) * D;
    xa = load_8(from, h < 0 ? kNowhere : at + 2 * (v ? 8 * n : a0));
    xb = load_8(from, h < 0 ? kNowhere : at + 2 * (v ? 8 * n + 4 : b0));
  };
  int u = mine ? blockIdx.y : groups;
  uint2 xa, xb;
  fetch(u, xa, xb);

  if constexpr (!QUADS) {
    q = find_row(a.s, t);
    if (q.b < 0) return;
  }
  const int64_t tok = (int64_t)q.len - q.rows + (t - q.r0);
  const int page = page_of(a.s, q.b, tok);
  const int P = 1 << a.s.log2P, o = (int)(tok & (P - 1));
  const KvLayout lay = kv_layout(FMT, D, P);
  uint8_t* page_p = a.pool + (size_t)max(page, 0) * ((size_t)n_kv * lay.head);

  const double p = (double)(a.pos && mine ? (int64_t)a.pos[t] : tok);
  for (int i = lane; i < a.rot / 2; i += 64) {
    double s, c;
    sin_cos(p * a.inv_freq[i], &s, &c);
    cs_s[wave][i] = make_double2(c * (double)a.rope_scale, s * (double)a.rope_scale);
  }
  wave_lds_fence();
  const auto weights = [&](const float* w, float (&out)[8]) {
    if (w) {
      const float4 wa = *reinterpret_cast<const float4*>(w + a0), wb = *reinterpret_cast<const float4*>(w + b0);
      out[0] = wa.x; out[1] = wa.y; out[2] = wa.z; out[3] = wa.w;
      out[4] = wb.x; out[5] = wb.y; out[6] = wb.z; out[7] = wb.w;
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i) out[i] = 1.0f;
    }
#if defined(__HIP_DEVICE_COMPILE__)
#pragma unroll
    for (int i = 0; i < 8; ++i) asm("" : "+v"(out[i]));  // (waited for here, not in every group)
#endif
  };
  // the cache's part of a group: x, 8 consecutive elements of a lane
  const auto store = [&](int h, bool is_v, uint4 x) {
    store_token<FMT, D>(page_p + (size_t)max(h, 0) * lay.head, lay, P, o, n, is_v,
                        is_v ? a.v_ts : a.k_ts, x, h >= 0 && page >= 0);
  };

  if (u < q_groups) {
    float w[8], cs[8];
    weights(a.q_norm, w);
    if (turn) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const double2 c = cs_s[wave][4 * n + i];
        cs[2 * i] = (float)c.x;
        cs[2 * i + 1] = (float)c.y;
      }
    }
    const Rsrc to = buffer_of(a.q_out + t * a.q_stride, n_q * D * 2);
    for (; u < q_groups; u += step) {
      const int h = head_of(u);
      float z[8] = {lo16(xa.x), hi16(xa.x), lo16(xa.y), hi16(xa.y),
                    lo16(xb.x), hi16(xb.x), lo16(xb.y), hi16(xb.y)};
      fetch(u + step, xa, xb);
      norm_turn<LPH, D>(z, w, a.q_norm != nullptr, a.eps, split, turn, cs);
      const uint32_t at = 2 * h * D;
      store_8(to, h < 0 ? kNowhere : at + 2 * a0, make_uint2(bf16_pair(z[0], z[1]), bf16_pair(z[2], z[3])));
      store_8(to, h < 0 ? kNowhere : at + 2 * b0, make_uint2(bf16_pair(z[4], z[5]), bf16_pair(z[6], z[7])));
    }
  }
  for (; u < q_groups + kv_groups; u += step) {
    const int h = head_of(u);
    double z[8] = {lo16(xa.x), hi16(xa.x), lo16(xa.y), hi16(xa.y),
                   lo16(xb.x), hi16(xb.x), lo16(xb.y), hi16(xb.y)};
    fetch(u + step, xa, xb);
    float w[8];
    double cs[8];
    weights(a.k_norm, w);
    if (turn) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const double2 c = cs_s[wave][4 * n + i];
        cs[2 * i] = c.x;
        cs[2 * i + 1] = c.y;
      }
    }
    norm_turn<LPH, D>(z, w, a.k_norm != nullptr, a.eps, split, turn, cs);
    uint32_t y[4];  // fp64 -> fp32 -> bf16 (the compiler makes one rounding of two conversions)
#pragma unroll
    for (int i = 0; i < 4; ++i)
      y[i] = (uint32_t)f32_to_bf16_rne((float)z[2 * i]) | ((uint32_t)f32_to_bf16_rne((float)z[2 * i + 1]) << 16);
    const uint2 ya = make_uint2(y[0], y[1]), yb = make_uint2(y[2], y[3]);
    if (h >= 0 && a.k_out) {
      uint16_t* k = a.k_out + t * a.k_stride + (size_t)h * D;
      *reinterpret_cast<uint2*>(k + a0) = ya;
      *reinterpret_cast<uint2*>(k + b0) = yb;
    }
    uint16_t* st = k_s[wave][g];
    *reinterpret_cast<uint2*>(st + a0) = ya;
    *reinterpret_cast<uint2*>(st + b0) = yb;
    wave_lds_fence();
    const uint4 x = *reinterpret_cast<const uint4*>(st + 8 * n);
    wave_lds_fence();
    store(h, false, x);
  }
  if (!QUADS || !whole) {
    for (; u < groups; u += step) {
      const int h = head_of(u);
      const uint4 x = make_uint4(xa.x, xa.y, xb.x, xb.y);
      fetch(u + step, xa, xb);
      store(h, true, x);
    }
    return;
  }
  // a whole quad: each wave's token into LDS, then a thread's two elements of all
  // four tokens to their place
  if constexpr (QUADS) {
    uint8_t* const v_s = reinterpret_cast<uint8_t*>(k_s);  // [token][head of the group][D]
    const int tg = threadIdx.x / (D / 2), td = 2 * (threadIdx.x % (D / 2));
    __syncthreads();  // the keys' part has been read
    for (; u < groups; u += step) {
      const int h = head_of(u);
      const uint4 x = make_uint4(xa.x, xa.y, xb.x, xb.y);
      fetch(u + step, xa, xb);
      uint8_t* const mine_s = v_s + ((wave * HPW + g) * D + 8 * n) * VB;
      if constexpr (FMT == MOE_FMT_BF16) {
        *reinterpret_cast<uint4*>(mine_s) = x;
      } else {
        uint16_t d;
        *reinterpret_cast<uint2*>(mine_s) = q8_codes(x, &d);
        if (h >= 0 && page >= 0 && tok >= 0 && !(n & 3))
          *reinterpret_cast<uint16_t*>(page_p + (size_t)h * lay.head + lay.vs + 2 * ((n >> 2) * P + o)) = d;
      }
      __syncthreads();
      const int th = (u - q_groups - kv_groups) * HPW + tg;
      if (th < n_kv && page >= 0) {
        uint8_t* dst = page_p + (size_t)th * lay.head + lay.vq + ((o >> 2) * D + td) * 4 * VB;
        uint32_t w[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const uint8_t* p = v_s + ((i * HPW + tg) * D + td) * VB;
          w[i] = VB == 2 ? *reinterpret_cast<const uint32_t*>(p) : (uint32_t)*reinterpret_cast<const uint16_t*>(p);
        }
        if constexpr (FMT == MOE_FMT_BF16) {
          *reinterpret_cast<uint4*>(dst) = make_uint4(
              __builtin_amdgcn_perm(w[1], w[0], 0x05040100u), __builtin_amdgcn_perm(w[3], w[2], 0x05040100u),
              __builtin_amdgcn_perm(w[1], w[0], 0x07060302u), __builtin_amdgcn_perm(w[3], w[2], 0x07060302u));
        } else {
          const uint32_t l = __builtin_amdgcn_perm(w[1], w[0], 0x05010400u);  // a0 b0 a1 b1
          const uint32_t r = __builtin_amdgcn_perm(w[3], w[2], 0x05010400u);
          *reinterpret_cast<uint2*>(dst) = make_uint2(__builtin_amdgcn_perm(r, l, 0x05040100u),
                                                      __builtin_amdgcn_perm(r, l, 0x07060302u));
        }
      }
      __syncthreads();
    }
  }
}

struct ReadArgs {
  const uint8_t* pool;
  const int32_t* first;
  const int32_t* out_start;
  uint16_t* k_out;
  uint16_t* v_out;
  int64_t k_stride, v_stride, R;
  SeqView s;
  int n_kv;
  float k_ts, v_ts;
};

constexpr uint32_t kNanPair = 0x7fc07fc0u;

__device__ __forceinline__ float e4m3_scale(uint32_t b) {  // (0x7f, 0xff: NaN)
  return (b & 0x7fu) == 0x7fu ? __uint_as_float(0x7fc00000u) : e4m3_to_f32(b);
}

// Eight E2M1 codes of a word times a block's scale and the tensor's, as bf16.
__device__ __forceinline__ uint4 fp4_values(uint32_t q, float s, float ts) {
  typedef float f2 __attribute__((ext_vector_type(2)));
  const f2 p0 = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(q, 1.0f, 0);
  const f2 p1 = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(q, 1.0f, 1);
  const f2 p2 = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(q, 1.0f, 2);
  const f2 p3 = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(q, 1.0f, 3);
  return make_uint4(bf16_pair(p0.x * s * ts, p0.y * s * ts), bf16_pair(p1.x * s * ts, p1.y * s * ts),
                    bf16_pair(p2.x * s * ts, p2.y * s * ts), bf16_pair(p3.x * s * ts, p3.y * s * ts));
}
__device__ __forceinline__ uint32_t i8_values(uint32_t q, int i, float s) {  // bytes i, i + 1
  return bf16_pair((float)(int8_t)(q >> (8 * i)) * s, (float)(int8_t)(q >> (8 * i + 8)) * s);
}

// One wave per 16 aligned tokens of a sequence and head.  What it reads is a
// third of what it writes or less (4 bits): every load of the wave is on its way
// before the first value is worked on, each in the order of the cache, and a
// lane writes consecutive elements of a row.  Bound by what it writes: 57 K tokens
// of 4 heads of 128 out of NVFP4 31 us, 4.8 TB/s.
template <int FMT, int D>
__global__ __launch_bounds__(256) void k_kv_read(ReadArgs a) {
  const int lane = lane_id(), wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int unit = (int)blockIdx.x * 4 + wave, h = blockIdx.y;
  // the sequence that holds this unit: tokens f.. and units of its span, summed
  int before = 0, u = -1, b = -1;
  int64_t f = 0, end = 0, out = 0;  // first token, the one after the last, row of token 0
  for (int i0 = 0; i0 < a.s.n_seq; i0 += 64) {
    const int i = min(i0 + lane, a.s.n_seq - 1);
    int begin = (a.first ? a.first : a.s.kv_len)[i], len = a.s.kv_len[i];
    int o0 = a.out_start[i], o1 = a.out_start[i + 1];
    loaded(begin, len, o0, o1);
    if (!a.first) begin = 0;
    // (tokens before the sequence's first, or whose row lies before row 0, are left out)
    const int64_t at_0 = (int64_t)begin - o0;  // the token of row 0
    const int64_t from = max(max((int64_t)begin, at_0), (int64_t)0);
    const int64_t stop = min((int64_t)len, at_0 + o1);
    const int sum = wave_incl_scan(
        i0 + lane < a.s.n_seq && stop > from ? (int)(((stop - 1) >> 4) - (from >> 4)) + 1 : 0);
    const uint64_t past = __ballot(before + sum > unit);
    if (!past) {
      before += __builtin_amdgcn_readlane(sum, 63);
      continue;
    }
    const int l = __ffsll((unsigned long long)past) - 1;
    if (l > 0) before += __builtin_amdgcn_readlane(sum, l - 1);
    b = i0 + l;
    f = __builtin_amdgcn_readlane((int)from, l);  // (both fit: from < stop <= len)
    end = __builtin_amdgcn_readlane((int)stop, l);
    out = (int64_t)__builtin_amdgcn_readlane(o0, l) - __builtin_amdgcn_readlane(begin, l);
    u = unit - before;
    break;
  }
  if (b < 0) return;
  const int64_t t0 = ((f >> 4) + u) << 4;  // first token of the unit
  const int page = page_of(a.s, b, t0);
  const int P = 1 << a.s.log2P, o = (int)(t0 & (P - 1));
  const KvLayout lay = kv_layout(FMT, D, P);
  const uint8_t* blk = a.pool + (size_t)max(page, 0) * ((size_t)a.n_kv * lay.head) + (size_t)h * lay.head;
  const int64_t row0 = out + t0;
  const auto wanted = [&](int j) {  // token j of the unit
    return t0 + j >= f && t0 + j < end && row0 + j >= 0 && row0 + j < a.R;
  };

  // keys: 8 elements of a token a lane
  constexpr int LPT = D / 8, TPI = 64 / LPT, KI = 16 / TPI;  // lanes of a token, tokens at a time
  const int kn = lane % LPT, kj = lane / LPT;
  uint4 kq[KI];
  uint32_t kscale[KI];
  if (a.k_out) {
#pragma unroll
    for (int i = 0; i < KI; ++i) {
      const int tok = o + i * TPI + kj;
      if constexpr (FMT == MOE_FMT_BF16) {
        kq[i] = *reinterpret_cast<const uint4*>(blk + 2 * (tok * D + 8 * kn));
      } else if constexpr (FMT == MOE_FMT_Q8_0) {
        const uint2 x = *reinterpret_cast<const uint2*>(blk + tok * D + 8 * kn);
        kq[i].x = x.x; kq[i].y = x.y;
        kscale[i] = *reinterpret_cast<const uint16_t*>(blk + lay.ks + 2 * (tok * (D / 32) + (kn >> 2)));
      } else {
        kq[i].x = *reinterpret_cast<const uint32_t*>(blk + tok * (D / 2) + 4 * kn);
        kscale[i] = blk[lay.ks + tok * (D / 16) + (kn >> 1)];
      }
    }
  }
  // values: NVFP4: D/16 elements of one token; the others: 16 bytes, four tokens'
  constexpr int GE = D / 16;                              // elements (NVFP4)
  constexpr int DC = FMT == MOE_FMT_BF16 ? 2 : 4;         // elements of a chunk (others)
  constexpr int VI = FMT == MOE_FMT_NVFP4 ? 4 : D / (16 * DC);
  const uint8_t* vq = blk + lay.vq;
  uint4 vv[VI];
  uint2 vscale[VI];
  if (a.v_out) {
#pragma unroll
    for (int i = 0; i < VI; ++i) {
      if constexpr (FMT == MOE_FMT_NVFP4) {
        const uint8_t* p = vq + ((o / 4 + i) * 64 + lane) * (GE / 2);
        if constexpr (GE == 4) vv[i].x = *reinterpret_cast<const uint16_t*>(p);
        if constexpr (GE == 8) vv[i].x = *reinterpret_cast<const uint32_t*>(p);
        if constexpr (GE == 16) { const uint2 x = *reinterpret_cast<const uint2*>(p); vv[i].x = x.x; vv[i].y = x.y; }
        vscale[i].x = blk[lay.vs + ((lane >> 2) * GE / 16) * P + o + 4 * i + (lane & 3)];
      } else {
        const int c = i * 64 + lane, quad = c / (D / DC), d = c % (D / DC) * DC;
        vv[i] = *reinterpret_cast<const uint4*>(vq + (o / 4 * (D / DC) + c) * 16);
        if constexpr (FMT == MOE_FMT_Q8_0)
          vscale[i] = *reinterpret_cast<const uint2*>(blk + lay.vs + 2 * ((d / 32) * P + o + 4 * quad));
      }
    }
  }

  if (a.k_out) {
#pragma unroll
    for (int i = 0; i < KI; ++i) {
      const int j = i * TPI + kj;
      uint4 x = kq[i];
      if constexpr (FMT == MOE_FMT_NVFP4) x = fp4_values(kq[i].x, e4m3_scale(kscale[i]), a.k_ts);
      if constexpr (FMT == MOE_FMT_Q8_0) {
        const float s = f16_to_f32((uint16_t)kscale[i]);
        x = make_uint4(i8_values(kq[i].x, 0, s), i8_values(kq[i].x, 2, s), i8_values(kq[i].y, 0, s),
                       i8_values(kq[i].y, 2, s));
      }
      if (page < 0) x = make_uint4(kNanPair, kNanPair, kNanPair, kNanPair);
      if (wanted(j))
        *reinterpret_cast<uint4*>(a.k_out + (row0 + j) * a.k_stride + (size_t)h * D + 8 * kn) = x;
    }
  }
  if (!a.v_out) return;
#pragma unroll
  for (int i = 0; i < VI; ++i) {
    if constexpr (FMT == MOE_FMT_NVFP4) {
      const int j = 4 * i + (lane & 3), n = lane >> 2;
      const float s = page < 0 ? __uint_as_float(0x7fc00000u) : e4m3_scale(vscale[i].x);
      const uint4 x = fp4_values(vv[i].x, s, a.v_ts);
      if (!wanted(j)) continue;
      uint16_t* dst = a.v_out + (row0 + j) * a.v_stride + (size_t)h * D + n * GE;
      if constexpr (GE == 4) *reinterpret_cast<uint2*>(dst) = make_uint2(x.x, x.y);
      if constexpr (GE >= 8) *reinterpret_cast<uint4*>(dst) = x;
      if constexpr (GE == 16) *reinterpret_cast<uint4*>(dst + 8) = fp4_values(vv[i].y, s, a.v_ts);
    } else {
      const int c = i * 64 + lane, quad = c / (D / DC), d = c % (D / DC) * DC;
      const uint32_t w[4] = {vv[i].x, vv[i].y, vv[i].z, vv[i].w};
#pragma unroll
      for (int t = 0; t < 4; ++t) {
        const int j = 4 * quad + t;
        uint16_t* dst = a.v_out + (row0 + j) * a.v_stride + (size_t)h * D + d;
        if constexpr (FMT == MOE_FMT_BF16) {  // w: two tokens of an element each
          const uint32_t x = __builtin_amdgcn_perm(w[2 + t / 2], w[t / 2], t & 1 ? 0x07060302u : 0x05040100u);
          if (wanted(j)) *reinterpret_cast<uint32_t*>(dst) = page < 0 ? kNanPair : x;
        } else {  // w: four tokens of an element each
          const float s = page < 0 ? __uint_as_float(0x7fc00000u)
                                   : f16_to_f32((uint16_t)((t < 2 ? vscale[i].x : vscale[i].y) >> (16 * (t & 1))));
          float e[4];
#pragma unroll
          for (int k = 0; k < 4; ++k) e[k] = (float)(int8_t)(w[k] >> (8 * t)) * s;
          if (wanted(j)) *reinterpret_cast<uint2*>(dst) = make_uint2(bf16_pair(e[0], e[1]), bf16_pair(e[2], e[3]));
        }
      }
    }
  }
}

SeqView seq_view(const moe_kv_cache* c, const moe_seq_batch* s) {
  int l2 = 0;
  while ((1 << l2) < c->page_tokens) ++l2;
  return SeqView{s->row_start, s->kv_len, s->page_table, s->n_seq, s->max_pages, c->n_pages, l2};
}

template <typename F>
hipError_t by_format(int fmt, int D, F&& f) {
#define MOE_KV_D(FMT)                                                            \
  switch (D) {                                                                   \
    case 64: return f(std::integral_constant<int, FMT>{}, std::integral_constant<int, 64>{});   \
    case 128: return f(std::integral_constant<int, FMT>{}, std::integral_constant<int, 128>{}); \
    default: return f(std::integral_constant<int, FMT>{}, std::integral_constant<int, 256>{});  \
  }
  switch (fmt) {
    case MOE_FMT_NVFP4: MOE_KV_D(MOE_FMT_NVFP4)
    case MOE_FMT_Q8_0: MOE_KV_D(MOE_FMT_Q8_0)
    default: MOE_KV_D(MOE_FMT_BF16)
  }
#undef MOE_KV_D
}

}  // namespace

hipError_t launch_kv_append(const moe_kv_cache* c, const moe_qkv_desc* p, const moe_seq_batch* s,
                            const uint16_t* qkv, int64_t qkv_stride, int64_t T, const int32_t* pos,
                            uint16_t* q_out, int64_t q_stride, uint16_t* k_out, int64_t k_stride,
                            hipStream_t stream) {
  AppendArgs a{qkv, q_out, k_out, pos, p->q_norm, p->k_norm, p->inv_freq, (uint8_t*)c->pool,
               qkv_stride, q_stride, k_stride, T, seq_view(c, s), p->n_q, c->n_kv, p->rot_dim,
               p->interleaved, p->eps, p->rope_scale, c->k_scale, c->v_scale};
  const int per_wave = 64 / (c->D / 8);
  const int groups = (p->n_q + per_wave - 1) / per_wave + 2 * ((c->n_kv + per_wave - 1) / per_wave);
  // (quads: n rows of a sequence lie in at most n/4 + 2 of them)
  const int64_t wgs = c->fmt == MOE_FMT_NVFP4 ? (T + kRows - 1) / kRows : T / 4 + 2 * (int64_t)s->n_seq;
  // few rows: the heads of a row spread over workgroups (each takes the row's
  // angles again: 6001 rows 17.8 us over 1526 workgroups, 19.7 over 3052)
  int hs = (int)((1024 + wgs - 1) / wgs);
  hs = hs < 1 ? 1 : hs > groups ? groups : hs;
  return by_format(c->fmt, c->D, [&](auto F, auto DD) {
    const dim3 grid((unsigned)wgs, (unsigned)hs);
    if (a.interleaved) k_kv_append<F(), DD(), false><<<grid, 64 * kRows, 0, stream>>>(a);
    else k_kv_append<F(), DD(), true><<<grid, 64 * kRows, 0, stream>>>(a);
    return hipGetLastError();
  });
}

hipError_t launch_kv_read(const moe_kv_cache* c, const moe_seq_batch* s, const int32_t* first,
                          const int32_t* out_start, int64_t R, uint16_t* k_out, int64_t k_stride,
                          uint16_t* v_out, int64_t v_stride, hipStream_t stream) {
  ReadArgs a{(const uint8_t*)c->pool, first, out_start, k_out, v_out, k_stride, v_stride, R,
             seq_view(c, s), c->n_kv, c->k_scale, c->v_scale};
  if (c->fmt != MOE_FMT_NVFP4) a.k_ts = a.v_ts = 1.0f;
  // a span of n tokens touches at most n/16 + 2 units
  const int64_t units = R / 16 + 2 * (int64_t)s->n_seq;
  const int64_t wgs = (units + 3) / 4;
  return by_format(c->fmt, c->D, [&](auto F, auto DD) {
    k_kv_read<F(), DD()><<<dim3((unsigned)wgs, (unsigned)c->n_kv), 256, 0, stream>>>(a);
    return hipGetLastError();
  });
}

}  // namespace moe
