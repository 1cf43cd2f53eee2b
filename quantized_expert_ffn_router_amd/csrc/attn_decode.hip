// attn_decode.hip -- attention of a step's newest rows over the paged cache.
//
// Every cached byte is needed once per (sequence, key/value head) and meets
// only the few query rows of that head's group, so the kernel is bound by
// streaming the cache from HBM, and decodes it in registers on the way
// (aiopssre.com, "Concurrency divides context unless you pay for more cache":
// the cache's size is what limits the context, hence the 4- and 8-bit forms).
//
//   scores^T (16 tokens x 16 query rows) = K Q^T,   out^T (D x 16) += V^T P^T
// as 16x16x32 matrix instructions.  The accumulator of the first has one query
// row per lane column and 4 tokens per lane, which is exactly an operand
// fragment of the second when V's fragment lists its tokens in the same order:
// the softmax weights go from one product to the next without leaving their
// lanes, and a row's maximum needs two lane swaps.
#include <type_traits>

#include "attn_common.h"

namespace moe {

namespace {

typedef _Float16 v2h __attribute__((ext_vector_type(2)));
typedef _Float16 v8h __attribute__((ext_vector_type(8)));
typedef __bf16 v8b __attribute__((ext_vector_type(8)));
typedef float v4f __attribute__((ext_vector_type(4)));
typedef uint32_t v4u __attribute__((ext_vector_type(4)));

constexpr int kWaves = 4;
constexpr float kNone = -3.0e38f;   // running maximum before any token
constexpr float kGrow = 8.0f;       // log2 headroom before the accumulators are rescaled

struct DecodeArgs {
  const uint8_t* pool;
  const uint16_t* q;
  uint16_t* out;
  float* part_o;   // [T * n_q][S][D]
  float2* part_ml; // [T * n_q][S]
  int64_t q_stride, out_stride, T;
  SeqView s;
  int n_q, n_kv, G, S, ztiles;
  float scale_log2, v_ts;
};

// What one tile of 16 query rows (row r = i * G + g: packed row i, head g of
// the group) of a sequence sees, and how its 32-token units are split.
struct TilePlan {
  int64_t hi;  // last token that any row of the tile sees (-1: none)
  int64_t lo;  // last token that all of them see
  int units, per_split, n_split;
};
__device__ __forceinline__ TilePlan tile_plan(int64_t len, int64_t rows, int G, int64_t tile, int S) {
  TilePlan p;
  const int64_t last = min((tile * 16 + 15) / G, rows - 1);
  p.hi = max(len - rows + last, (int64_t)-1);
  p.lo = len - rows + (tile * 16) / G;
  p.units = (int)((p.hi + 32) >> 5);
  const int even = (p.units + S - 1) / S;
  p.per_split = max((even + kWaves - 1) / kWaves * kWaves, kWaves);
  p.n_split = (p.units + p.per_split - 1) / p.per_split;
  return p;
}

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
// int8 codes: byte b + 128 under the exponent byte of 1024 is 1024 + 128 + b
// in fp16, exactly; one packed subtraction leaves b.
__device__ __forceinline__ v2h i8_pair(uint32_t biased, int k) {
  const uint32_t w = __builtin_amdgcn_perm(0x64646464u, biased, k ? 0x07030702u : 0x05010400u);
  const v2h c = {(_Float16)1152.0f, (_Float16)1152.0f};
  return __builtin_bit_cast(v2h, w) - c;
}
__device__ __forceinline__ uint32_t bits(v2h v) { return __builtin_bit_cast(uint32_t, v); }
__device__ __forceinline__ v2h halves(uint32_t w) { return __builtin_bit_cast(v2h, w); }

// max / sum over the four 16-lane groups (a query row's lanes).
__device__ __forceinline__ float groups_max(float v) {
  const uint32_t u = __float_as_uint(v);
  const auto a = __builtin_amdgcn_permlane32_swap(u, u, false, false);
  v = fmaxf(__uint_as_float(a[0]), __uint_as_float(a[1]));
  const uint32_t w = __float_as_uint(v);
  const auto b = __builtin_amdgcn_permlane16_swap(w, w, false, false);
  return fmaxf(__uint_as_float(b[0]), __uint_as_float(b[1]));
}
__device__ __forceinline__ float groups_sum(float v) {
  v += __shfl_xor(v, 32);
  return v + __shfl_xor(v, 16);
}

// The cache bytes of one lane for a unit of 32 tokens (two tiles of 16): a
// quarter of one token's key per tile, D/16 elements of four tokens' values.
template <int FMT, int D>
struct Unit {
  static constexpr int W = FMT == MOE_FMT_NVFP4 ? D / 32 : FMT == MOE_FMT_Q8_0 ? D / 16 : D / 8;
  uint32_t k[2][W], v[2][W];
  uint32_t ks[2];     // NVFP4: D/64 E4M3 bytes; Q8_0: D/128 (at least one) fp16
  uint32_t vs[2][2];  // scales of the 4 tokens: E4M3 bytes in [0], or 4 fp16

  __device__ __forceinline__ static void words(uint32_t* d, const uint8_t* p) {
    if constexpr (W == 2) {
      typedef uint32_t v2u __attribute__((ext_vector_type(2)));
      const v2u x = __builtin_nontemporal_load(reinterpret_cast<const v2u*>(p));
      d[0] = x.x; d[1] = x.y;
    } else {
#pragma unroll
      for (int i = 0; i < W / 4; ++i) {
        const v4u x = __builtin_nontemporal_load(reinterpret_cast<const v4u*>(p) + i);
        d[4 * i] = x.x; d[4 * i + 1] = x.y; d[4 * i + 2] = x.z; d[4 * i + 3] = x.w;
      }
    }
  }

  // blk: the (page, head) block; o: the unit's first token within the page.
  __device__ __forceinline__ void load(const uint8_t* blk, const KvLayout lay, int P, int o, int n,
                                       int g) {
#pragma unroll
    for (int t = 0; t < 2; ++t) {
      const int tok = o + 16 * t + n, quad = ((o + 16 * t) >> 2) + g;
      words(k[t], blk + (tok * 4 + g) * (4 * W));
      words(v[t], blk + lay.vq + (quad * 16 + n) * (4 * W));
      if constexpr (FMT == MOE_FMT_NVFP4) {
        const uint8_t* s = blk + lay.ks + tok * (D / 16) + g * (D / 64);
        if constexpr (D == 64) ks[t] = *s;
        if constexpr (D == 128) ks[t] = *reinterpret_cast<const uint16_t*>(s);
        if constexpr (D == 256) ks[t] = *reinterpret_cast<const uint32_t*>(s);
        vs[t][0] = *reinterpret_cast<const uint32_t*>(blk + lay.vs + (n * D / 256) * P + o + 16 * t + 4 * g);
      } else if constexpr (FMT == MOE_FMT_Q8_0) {
        const uint8_t* s = blk + lay.ks + 2 * (tok * (D / 32) + g * D / 128);
        if constexpr (D == 256) ks[t] = *reinterpret_cast<const uint32_t*>(s);
        else ks[t] = *reinterpret_cast<const uint16_t*>(s);
        const uint2 x = *reinterpret_cast<const uint2*>(blk + lay.vs + 2 * ((n * D / 512) * P + o + 16 * t + 4 * g));
        vs[t][0] = x.x; vs[t][1] = x.y;
      }
    }
  }

  // Key fragment s (elements g * D/4 + 8 s ..) of tile t, as 4 words.
  __device__ __forceinline__ v4u key(int t, int s) const {
    v4u r;
    if constexpr (FMT == MOE_FMT_NVFP4) {
      const v2h sp = fp8_pair(ks[t], s >> 2);
      const v2h sc = (s >> 1) & 1 ? v2h{sp.y, sp.y} : v2h{sp.x, sp.x};
#pragma unroll
      for (int i = 0; i < 4; ++i) r[i] = bits(fp4_pair(k[t][s], i) * sc);
    } else if constexpr (FMT == MOE_FMT_Q8_0) {
      const v2h sp = halves(ks[t]);
      const v2h sc = s >> 2 ? v2h{sp.y, sp.y} : v2h{sp.x, sp.x};
#pragma unroll
      for (int i = 0; i < 4; ++i) r[i] = bits(i8_pair(k[t][2 * s + (i >> 1)] ^ 0x80808080u, i & 1) * sc);
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i) r[i] = k[t][4 * s + i];
    }
    return r;
  }

  // Value fragment of element n * D/16 + j: tokens 4g.. of tile 0, then of
  // tile 1 (the order of the score accumulators).
  __device__ __forceinline__ v4u value(int j) const {
    v4u r;
#pragma unroll
    for (int t = 0; t < 2; ++t) {
#pragma unroll
      for (int h = 0; h < 2; ++h) {  // tokens 2h, 2h + 1
        if constexpr (FMT == MOE_FMT_NVFP4) {
          uint32_t a, b;
          if constexpr (D == 64) {
            a = v[t][h]; b = v[t][h] >> 16;
          } else {
            a = v[t][2 * h * (D / 128) + j / 8]; b = v[t][(2 * h + 1) * (D / 128) + j / 8];
          }
          // element j of both tokens in one byte: even elements from the low
          // nibbles, odd ones from the high nibbles
          const uint32_t w = j & 1 ? ((a >> 4) & 0x0f0f0f0fu) | (b & 0xf0f0f0f0u)
                                   : (a & 0x0f0f0f0fu) | ((b << 4) & 0xf0f0f0f0u);
          r[2 * t + h] = bits(fp4_pair(w, (j & 7) >> 1) * fp8_pair(vs[t][0], h));
        } else if constexpr (FMT == MOE_FMT_Q8_0) {
          r[2 * t + h] = bits(i8_pair(v[t][j] ^ 0x80808080u, h) * halves(vs[t][h]));
        } else {
          r[2 * t + h] = v[t][2 * j + h];
        }
      }
    }
    return r;
  }

  // Zeroes the values of this lane's tokens from the `left`-th of the unit on
  // (left: tokens of the unit that some row sees), whatever they hold.
  __device__ __forceinline__ void cut(int left, int g) {
#pragma unroll
    for (int t = 0; t < 2; ++t) {
      const int n = min(max(left - 16 * t - 4 * g, 0), 4);
      if constexpr (FMT == MOE_FMT_NVFP4) {
        vs[t][0] = n >= 4 ? vs[t][0] : vs[t][0] & ((1u << (8 * n)) - 1u);
      } else {
        const uint32_t m0 = n >= 2 ? ~0u : n == 1 ? 0xffffu : 0u;
        const uint32_t m1 = n >= 4 ? ~0u : n == 3 ? 0xffffu : 0u;
        if constexpr (FMT == MOE_FMT_Q8_0) {
          vs[t][0] &= m0; vs[t][1] &= m1;
        } else {
#pragma unroll
          for (int j = 0; j < D / 16; ++j) { v[t][2 * j] &= m0; v[t][2 * j + 1] &= m1; }
        }
      }
    }
  }

  // Whether any of this lane's values is infinite or NaN (in the block
  // formats a NaN scale says so; an infinite fp16 scale counts too).
  __device__ __forceinline__ bool wild() const {
    bool any = false;
#pragma unroll
    for (int t = 0; t < 2; ++t) {
      if constexpr (FMT == MOE_FMT_NVFP4) {
#pragma unroll
        for (int i = 0; i < 4; ++i) any |= ((vs[t][0] >> (8 * i)) & 0x7fu) == 0x7fu;
      } else if constexpr (FMT == MOE_FMT_Q8_0) {
#pragma unroll
        for (int i = 0; i < 4; ++i)
          any |= ((vs[t][i >> 1] >> (16 * (i & 1))) & 0x7c00u) == 0x7c00u;
      } else {
#pragma unroll
        for (int j = 0; j < W; ++j)
          any |= (v[t][j] & 0x7f80u) == 0x7f80u || (v[t][j] & 0x7f800000u) == 0x7f800000u;
      }
    }
    return any;
  }
};

template <int FMT>
__device__ __forceinline__ v4f mma(v4u a, v4u b, v4f c) {
  if constexpr (FMT == MOE_FMT_BF16)
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(v8b, a),
                                                   __builtin_bit_cast(v8b, b), c, 0, 0, 0);
  else
    return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(v8h, a),
                                                  __builtin_bit_cast(v8h, b), c, 0, 0, 0);
}

// Two softmax weights as a pair of the product's operand type, rounded to
// nearest even: at most half a step of weights between 0 and 2^kGrow.
template <int FMT>
__device__ __forceinline__ uint32_t weight_pair(float a, float b) {
  if constexpr (FMT == MOE_FMT_BF16) {
    typedef __bf16 v2b __attribute__((ext_vector_type(2)));
    const v2b r = {(__bf16)a, (__bf16)b};
    return __builtin_bit_cast(uint32_t, r);
  } else {
    const v2h r = {(_Float16)a, (_Float16)b};
    return bits(r);
  }
}

template <int FMT, int D>
__global__ __launch_bounds__(64 * kWaves) void k_attn_decode(DecodeArgs a) {
  constexpr int KS = D / 32, NJ = D / 16, LD = D + 4;
  __shared__ __align__(16) float o_s[kWaves][16][LD];
  __shared__ float m_s[kWaves][16], l_s[kWaves][16];
  const int wave = threadIdx.x >> 6, lane = lane_id(), n = lane & 15, g = lane >> 4;
  uint32_t id = blockIdx.x;
  const int sp = (int)(id % a.S); id /= a.S;
  const int kvh = (int)(id % a.n_kv); id /= a.n_kv;
  const int zt = (int)(id % a.ztiles);
  const int b = (int)(id / a.ztiles);

  const int64_t r0 = a.s.row_start[b], rows = (int64_t)a.s.row_start[b + 1] - r0;
  const int64_t len = a.s.kv_len[b];
  if (rows <= 0 || r0 < 0) return;
  const int P = 1 << a.s.log2P;
  const KvLayout lay = kv_layout(FMT, D, P);
  const size_t page_bytes = (size_t)a.n_kv * lay.head;
  const uint8_t* heads = a.pool + (size_t)kvh * lay.head;

  for (int64_t tile = zt; tile * 16 < rows * a.G; tile += a.ztiles) {
    if (r0 + tile * 16 / a.G >= a.T) break;
    const TilePlan plan = tile_plan(len, rows, a.G, tile, a.S);
    const int u_begin = sp * plan.per_split, u_end = min(plan.units, u_begin + plan.per_split);
    if (sp > 0 && u_begin >= u_end) continue;  // split 0 also answers rows that see nothing

    // this lane's query row, its last visible token and its fragments
    const int64_t r = tile * 16 + n;
    const int64_t row = r0 + r / a.G;
    const int head = kvh * a.G + (int)(r % a.G);
    const bool live = r < rows * a.G && row < a.T;
    const int64_t limit = live ? len - rows + r / a.G : -1;
    v4u qf[KS];
    const uint16_t* qp = a.q + (live ? row : r0) * a.q_stride + (size_t)(live ? head : kvh * a.G) * D + g * (D / 4);
    float qs = a.scale_log2;
#pragma unroll
    for (int s = 0; s < KS; ++s) qf[s] = *reinterpret_cast<const v4u*>(qp + 8 * s);
    if constexpr (FMT != MOE_FMT_BF16) {
      // bf16 -> fp16, scaled by the power of two that puts the row's largest
      // magnitude into [2^14, 2^15): exact for values above 2^-29 of it
      uint32_t top = 0;
#pragma unroll
      for (int s = 0; s < KS; ++s)
#pragma unroll
        for (int i = 0; i < 4; ++i) top = max(top, max(qf[s][i] & 0x7fffu, (qf[s][i] >> 16) & 0x7fffu));
      top = max(top, (uint32_t)__shfl_xor((int)top, 16));
      top = max(top, (uint32_t)__shfl_xor((int)top, 32));
      const int e = min(max(141 - (int)(top >> 7), -113), 126);
      const float up = __uint_as_float((uint32_t)(127 + e) << 23);
      qs *= __uint_as_float((uint32_t)(127 - e) << 23);
#pragma unroll
      for (int s = 0; s < KS; ++s)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const v2h p = {(_Float16)(__uint_as_float(qf[s][i] << 16) * up),
                         (_Float16)(__uint_as_float(qf[s][i] & 0xffff0000u) * up)};
          qf[s][i] = bits(p);
        }
    }

    v4f o[NJ];
#pragma unroll
    for (int j = 0; j < NJ; ++j) o[j] = v4f{0.f, 0.f, 0.f, 0.f};
    float m = kNone, l = 0.0f;

    for (int u = u_begin + wave; u < u_end; u += kWaves) {
      const int64_t t0 = (int64_t)u * 32;
      const int page = page_of(a.s, b, t0);
      if (page < 0) {  // nothing to read: whoever sees a token of it has no answer
        if (limit >= t0) l = __uint_as_float(0x7fc00000u);
        continue;
      }
      Unit<FMT, D> c;
      c.load(heads + (size_t)page * page_bytes, lay, P, (int)(t0 & (P - 1)), n, g);

      v4f x[2];
#pragma unroll
      for (int t = 0; t < 2; ++t) {
        x[t] = v4f{0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int s = 0; s < KS; ++s) x[t] = mma<FMT>(c.key(t, s), qf[s], x[t]);
      }
      const bool edge = t0 + 31 > plan.lo;  // some row does not see all of it
      float mx = kNone;
#pragma unroll
      for (int t = 0; t < 2; ++t)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          x[t][i] *= qs;
          if (edge && t0 + 16 * t + 4 * g + i > limit) x[t][i] = -__builtin_inff();
          mx = fmaxf(mx, x[t][i]);
        }
      mx = groups_max(mx);
      if (__any(mx > m + kGrow)) {
        const float mn = fmaxf(m, mx), al = __builtin_amdgcn_exp2f(m - mn);
#pragma unroll
        for (int j = 0; j < NJ; ++j)
#pragma unroll
          for (int i = 0; i < 4; ++i) o[j][i] *= al;
        l *= al;
        m = mn;
      }
      v4u p;
#pragma unroll
      for (int t = 0; t < 2; ++t) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          x[t][i] = __builtin_amdgcn_exp2f(x[t][i] - m);
          l += x[t][i];
        }
        p[2 * t] = weight_pair<FMT>(x[t][0], x[t][1]);
        p[2 * t + 1] = weight_pair<FMT>(x[t][2], x[t][3]);
      }
      if (edge) {
        const int64_t left = plan.hi + 1 - t0;
        if (left < 32) c.cut((int)left, g);
        if (__any(c.wild())) {
          // A zero weight would not silence an infinity or a NaN: take the
          // tokens one at a time and add each only to the rows that see it.
          for (int tk = 0; tk < 32; ++tk) {
            const bool mine = g == ((tk & 15) >> 2), seen = t0 + tk <= limit;
            const int w = 2 * (tk >> 4) + ((tk & 3) >> 1);
            const uint32_t keep = mine ? 0xffffu << (16 * (tk & 1)) : 0u;
#pragma unroll
            for (int j = 0; j < NJ; ++j) {
              v4u f = c.value(j);
#pragma unroll
              for (int i = 0; i < 4; ++i) f[i] = i == w ? f[i] & keep : 0u;
              const v4f add = mma<FMT>(f, p, v4f{0.f, 0.f, 0.f, 0.f});
#pragma unroll
              for (int i = 0; i < 4; ++i) o[j][i] += seen ? add[i] : 0.0f;
            }
          }
          continue;
        }
      }
#pragma unroll
      for (int j = 0; j < NJ; ++j) o[j] = mma<FMT>(c.value(j), p, o[j]);
    }
    l = groups_sum(l);

    // join the waves' parts
    __syncthreads();  // a former tile's parts have been read
    if (g == 0) { m_s[wave][n] = m; l_s[wave][n] = l; }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      float* d = &o_s[wave][n][(4 * g + i) * NJ];
#pragma unroll
      for (int j = 0; j < NJ; j += 4)
        *reinterpret_cast<float4*>(d + j) = make_float4(o[j][i], o[j + 1][i], o[j + 2][i], o[j + 3][i]);
    }
    __syncthreads();
    const int qr = threadIdx.x >> 4, d0 = (threadIdx.x & 15) * NJ;
    const int64_t rr = tile * 16 + qr;
    const int64_t orow = r0 + rr / a.G;
    if (rr < rows * a.G && orow < a.T) {
      float M = kNone, L = 0.0f, acc[NJ];
#pragma unroll
      for (int w = 0; w < kWaves; ++w) M = fmaxf(M, m_s[w][qr]);
#pragma unroll
      for (int j = 0; j < NJ; ++j) acc[j] = 0.0f;
#pragma unroll
      for (int w = 0; w < kWaves; ++w) {
        const float f = __builtin_amdgcn_exp2f(m_s[w][qr] - M);
        L += f * l_s[w][qr];
#pragma unroll
        for (int j = 0; j < NJ; ++j) acc[j] += f * o_s[w][qr][d0 + j];
      }
      const int64_t h = kvh * a.G + rr % a.G;
      if (plan.n_split <= 1) {
        const float inv = len - rows + rr / a.G < 0 ? 0.0f : a.v_ts / L;
        uint32_t w[NJ / 2];
#pragma unroll
        for (int j = 0; j < NJ / 2; ++j)
          w[j] = (uint32_t)f32_to_bf16_rne(acc[2 * j] * inv) | ((uint32_t)f32_to_bf16_rne(acc[2 * j + 1] * inv) << 16);
        uint16_t* d = a.out + orow * a.out_stride + h * D + d0;
        if constexpr (NJ == 4) *reinterpret_cast<uint2*>(d) = make_uint2(w[0], w[1]);
        if constexpr (NJ >= 8) *reinterpret_cast<uint4*>(d) = make_uint4(w[0], w[1], w[2], w[3]);
        if constexpr (NJ == 16) *reinterpret_cast<uint4*>(d + 8) = make_uint4(w[4], w[5], w[6], w[7]);
      } else {
        const int64_t at = (orow * a.n_q + h) * a.S + sp;
        if (d0 == 0) a.part_ml[at] = make_float2(M, L);
        float* d = a.part_o + at * D + d0;
#pragma unroll
        for (int j = 0; j < NJ; j += 4)
          *reinterpret_cast<float4*>(d + j) = make_float4(acc[j], acc[j + 1], acc[j + 2], acc[j + 3]);
      }
    }
  }
}

// Joins the splits of one (row, head): weights exp2(m_s - M), in the order of
// the splits, so the result does not depend on scheduling.
template <int D>
__global__ __launch_bounds__(256) void k_attn_join(DecodeArgs a) {
  constexpr int LW = D / 4, NG = 256 / LW;  // lanes of a row, splits at a time
  __shared__ __align__(16) float4 acc_s[NG][LW];
  __shared__ float l_s[NG];
  const int64_t t = blockIdx.x / a.n_q;
  const int h = (int)(blockIdx.x % a.n_q);
  const int b = find_seq(a.s.row_start, a.s.n_seq, t);
  if (b >= a.s.n_seq) return;
  const int64_t r0 = a.s.row_start[b], rows = (int64_t)a.s.row_start[b + 1] - r0;
  if (t < r0 || r0 < 0) return;
  const int64_t tile = ((t - r0) * a.G + h % a.G) / 16;
  const int ns = tile_plan(a.s.kv_len[b], rows, a.G, tile, a.S).n_split;
  if (ns <= 1) return;
  const int64_t at = (t * a.n_q + h) * a.S;
  const int lane = lane_id();
  float M = kNone, L = 0.0f;
  for (int s = lane; s < ns; s += 64) M = fmaxf(M, a.part_ml[at + s].x);
#pragma unroll
  for (int d = 32; d; d >>= 1) M = fmaxf(M, __shfl_xor(M, d));
  const int grp = threadIdx.x / LW, x = threadIdx.x % LW;
  float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
  for (int s = grp; s < ns; s += NG) {
    const float2 ml = a.part_ml[at + s];
    const float f = __builtin_amdgcn_exp2f(ml.x - M);
    const float4 v = *reinterpret_cast<const float4*>(a.part_o + (at + s) * D + 4 * x);
    o.x += f * v.x; o.y += f * v.y; o.z += f * v.z; o.w += f * v.w;
    L += f * ml.y;
  }
  acc_s[grp][x] = o;
  if (x == 0) l_s[grp] = L;
  __syncthreads();
  if (threadIdx.x < LW) {
    o = acc_s[0][x];
    L = l_s[0];
#pragma unroll
    for (int i = 1; i < NG; ++i) {
      const float4 v = acc_s[i][x];
      o.x += v.x; o.y += v.y; o.z += v.z; o.w += v.w;
      L += l_s[i];
    }
    const float inv = a.s.kv_len[b] - rows + (t - r0) < 0 ? 0.0f : a.v_ts / L;
    uint16_t* d = a.out + t * a.out_stride + (int64_t)h * D + 4 * x;
    *reinterpret_cast<uint2*>(d) =
        make_uint2((uint32_t)f32_to_bf16_rne(o.x * inv) | ((uint32_t)f32_to_bf16_rne(o.y * inv) << 16),
                   (uint32_t)f32_to_bf16_rne(o.z * inv) | ((uint32_t)f32_to_bf16_rne(o.w * inv) << 16));
  }
}

struct Split {
  int S, ztiles;
};
// Splits of a sequence's cache: enough workgroups for every CU to hold four
// (the resident number at this register use), none shorter than one round of
// the four waves.
Split split_of(int n_kv, int n_q, int n_seq, int64_t T, int64_t max_len) {
  const int G = n_q / n_kv;
  const int64_t per_seq = (T + n_seq - 1) / n_seq;
  Split r;
  r.ztiles = (int)((per_seq * G + 15) / 16);
  const int64_t base = (int64_t)n_seq * n_kv * r.ztiles;
  int64_t S = (1024 + base - 1) / base;
  const int64_t most = (max_len + 32 * kWaves - 1) / (32 * kWaves);
  if (S > most) S = most;
  if (S > 256) S = 256;
  r.S = S < 1 ? 1 : (int)S;
  return r;
}

}  // namespace

size_t attn_decode_ws_bytes(int n_kv, int D, int n_q, int n_seq, int64_t T, int64_t max_len) {
  if (n_seq < 1 || T < 1) return 0;
  const Split sp = split_of(n_kv, n_q, n_seq, T, max_len);
  if (sp.S == 1) return 0;
  const size_t n = (size_t)T * n_q * sp.S;
  return align_up(n * D * sizeof(float)) + align_up(n * sizeof(float2));
}

hipError_t launch_attn_decode(const moe_kv_cache* c, const moe_seq_batch* s, int n_q,
                              const uint16_t* q, int64_t q_stride, int64_t T, int64_t max_len,
                              float scale, uint16_t* out, int64_t out_stride, void* ws,
                              hipStream_t stream) {
  const Split sp = split_of(c->n_kv, n_q, s->n_seq, T, max_len);
  int l2 = 0;
  while ((1 << l2) < c->page_tokens) ++l2;
  const bool fp4 = c->fmt == MOE_FMT_NVFP4;
  const size_t n = (size_t)T * n_q * sp.S;
  DecodeArgs a{(const uint8_t*)c->pool, q, out, (float*)ws,
               (float2*)((char*)ws + align_up(n * c->D * sizeof(float))), q_stride, out_stride, T,
               SeqView{s->row_start, s->kv_len, s->page_table, s->n_seq, s->max_pages, c->n_pages, l2},
               n_q, c->n_kv, n_q / c->n_kv, sp.S, sp.ztiles,
               scale * 1.4426950408889634f * (fp4 ? c->k_scale : 1.0f), fp4 ? c->v_scale : 1.0f};
  const unsigned grid = (unsigned)((int64_t)sp.S * c->n_kv * sp.ztiles * s->n_seq);
#define MOE_DECODE(FMT)                                                              \
  switch (c->D) {                                                                    \
    case 64: k_attn_decode<FMT, 64><<<grid, 64 * kWaves, 0, stream>>>(a); break;     \
    case 128: k_attn_decode<FMT, 128><<<grid, 64 * kWaves, 0, stream>>>(a); break;   \
    default: k_attn_decode<FMT, 256><<<grid, 64 * kWaves, 0, stream>>>(a);           \
  }
  switch (c->fmt) {
    case MOE_FMT_NVFP4: MOE_DECODE(MOE_FMT_NVFP4) break;
    case MOE_FMT_Q8_0: MOE_DECODE(MOE_FMT_Q8_0) break;
    default: MOE_DECODE(MOE_FMT_BF16)
  }
#undef MOE_DECODE
  hipError_t e = hipGetLastError();
  if (e != hipSuccess || sp.S == 1) return e;
  const unsigned heads = (unsigned)(T * n_q);
  switch (c->D) {
    case 64: k_attn_join<64><<<heads, 256, 0, stream>>>(a); break;
    case 128: k_attn_join<128><<<heads, 256, 0, stream>>>(a); break;
    default: k_attn_join<256><<<heads, 256, 0, stream>>>(a);
  }
  return hipGetLastError();
}

}  // namespace moe
