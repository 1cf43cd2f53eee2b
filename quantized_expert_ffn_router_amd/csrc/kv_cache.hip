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

// fp64 -> fp32 -> bf16, each rounded to nearest even.
__device__ __forceinline__ uint32_t bf16_pair(double a, double b) {
  return (uint32_t)f32_to_bf16_rne((float)a) | ((uint32_t)f32_to_bf16_rne((float)b) << 16);
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
  uint32_t top = top_bits(x);
  top = max(top, (uint32_t)__shfl_xor((int)top, 1));
  if constexpr (FMT == MOE_FMT_Q8_0) top = max(top, (uint32_t)__shfl_xor((int)top, 2));
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
  } else {
    const _Float16 d = bad ? __builtin_bit_cast(_Float16, (uint16_t)0x7e00)
                           : (_Float16)(fminf(amax, 65024.0f) / 127.0f);
    const float df = (float)d;
    uint32_t q[2] = {0, 0};
    if (df > 0.0f) {
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const int c = (int)fminf(fmaxf(rintf(v[i] / df), -127.0f), 127.0f);
        q[i >> 2] |= (uint32_t)(c & 0xff) << (8 * (i & 3));
      }
    }
    const uint16_t db = __builtin_bit_cast(uint16_t, d);
    if (!is_v) {
      *reinterpret_cast<uint2*>(blk + o * D + 8 * n) = make_uint2(q[0], q[1]);
      if (!(n & 3)) *reinterpret_cast<uint16_t*>(blk + lay.ks + 2 * (o * (D / 32) + (n >> 2))) = db;
    } else {
      uint8_t* p = blk + lay.vq + ((o >> 2) * D + 8 * n) * 4 + (o & 3);
#pragma unroll
      for (int i = 0; i < 8; ++i) p[4 * i] = (uint8_t)(q[i >> 2] >> (8 * (i & 3)));
      if (!(n & 3)) *reinterpret_cast<uint16_t*>(blk + lay.vs + 2 * ((n >> 2) * P + o)) = db;
    }
  }
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

// One wave per row, D/8 lanes per head, 64/(D/8) heads at a time.  The row's
// angles are taken once, in fp64 (a far position times a frequency needs more
// than 24 bits), and kept in the wave's LDS.  A lane holds 4 rotation pairs of
// its head (elements a0.., b0..: both halves of a pair, so no lane needs
// another's value), norms and rotates them in fp64 -- on this chip as many
// fp64 as plain fp32 operations run per cycle -- and rounds once.  Keys then go
// through LDS into 8 consecutive elements a lane, the unit of quantisation.
template <int FMT, int D>
__global__ __launch_bounds__(64 * kRows) void k_kv_append(AppendArgs a) {
  constexpr int LPH = D / 8, HPW = 64 / LPH;
  __shared__ double2 cs_s[kRows][128];
  __shared__ __align__(16) uint16_t k_s[kRows][HPW][D];
  const int wave = threadIdx.x >> 6, lane = lane_id();
  const int64_t t = (int64_t)blockIdx.x * kRows + wave;
  if (t >= a.T) return;
  const RowSeq q = find_row(a.s, t);
  if (q.b < 0) return;
  const int64_t tok = (int64_t)q.len - q.rows + (t - q.r0);
  const int page = page_of(a.s, q.b, tok);
  const int P = 1 << a.s.log2P, o = (int)(tok & (P - 1));
  const KvLayout lay = kv_layout(FMT, D, P);
  uint8_t* page_p = a.pool + (size_t)max(page, 0) * ((size_t)a.n_kv * lay.head);

  const double p = (double)(a.pos ? (int64_t)a.pos[t] : tok);
  for (int i = lane; i < a.rot / 2; i += 64) {
    double s, c;
    sincos(p * a.inv_freq[i], &s, &c);
    cs_s[wave][i] = make_double2(c * (double)a.rope_scale, s * (double)a.rope_scale);
  }
  wave_lds_fence();

  const int n = lane % LPH, g = lane / LPH;
  const int NH = a.n_q + 2 * a.n_kv;
  const uint16_t* row = a.qkv + t * a.qkv_stride;
  const bool split = !a.interleaved && n < a.rot / 8;  // holds pairs (i, i + rot/2)
  const bool turn = split || (a.interleaved && 8 * n < a.rot);

  for (int h0 = blockIdx.y * HPW; h0 < NH; h0 += gridDim.y * HPW) {
    const int h = h0 + g;
    const bool live = h < NH, is_q = h < a.n_q, is_v = h >= a.n_q + a.n_kv;
    const bool sp = split && !is_v;
    const int a0 = sp ? 4 * n : 8 * n, b0 = sp ? a.rot / 2 + 4 * n : 8 * n + 4;
    uint2 xa = make_uint2(0, 0), xb = make_uint2(0, 0);
    if (live) {
      xa = *reinterpret_cast<const uint2*>(row + (size_t)h * D + a0);
      xb = *reinterpret_cast<const uint2*>(row + (size_t)h * D + b0);
    }
    if (h0 < a.n_q + a.n_kv) {  // some head of this group is a query or a key
      double z[8] = {lo16(xa.x), hi16(xa.x), lo16(xa.y), hi16(xa.y),
                     lo16(xb.x), hi16(xb.x), lo16(xb.y), hi16(xb.y)};
      const float* w = is_q ? a.q_norm : a.k_norm;
      double ss = 0.0;
#pragma unroll
      for (int i = 0; i < 8; ++i) ss = fma(z[i], z[i], ss);
#pragma unroll
      for (int m = 1; m < LPH; m <<= 1) ss += __shfl_xor(ss, m);
      if (w && !is_v) {
        const double r = rsqrt(ss / D + (double)a.eps);
        const float4 wa = *reinterpret_cast<const float4*>(w + a0);
        const float4 wb = *reinterpret_cast<const float4*>(w + b0);
        const float ww[8] = {wa.x, wa.y, wa.z, wa.w, wb.x, wb.y, wb.z, wb.w};
#pragma unroll
        for (int i = 0; i < 8; ++i) z[i] = z[i] * r * (double)ww[i];
      }
      if (turn && !is_v) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const double2 cs = cs_s[wave][4 * n + i];
          const double zu = sp ? z[i] : z[2 * i], zv = sp ? z[i + 4] : z[2 * i + 1];
          const double nu = zu * cs.x - zv * cs.y, nv = zv * cs.x + zu * cs.y;
          if (sp) { z[i] = nu; z[i + 4] = nv; } else { z[2 * i] = nu; z[2 * i + 1] = nv; }
        }
      }
      if (!is_v) {
        xa = make_uint2(bf16_pair(z[0], z[1]), bf16_pair(z[2], z[3]));
        xb = make_uint2(bf16_pair(z[4], z[5]), bf16_pair(z[6], z[7]));
      }
      if (live && is_q) {
        uint16_t* d = a.q_out + t * a.q_stride + (size_t)h * D;
        *reinterpret_cast<uint2*>(d + a0) = xa;
        *reinterpret_cast<uint2*>(d + b0) = xb;
      } else if (live && !is_v && a.k_out) {
        uint16_t* k = a.k_out + t * a.k_stride + (size_t)(h - a.n_q) * D;
        *reinterpret_cast<uint2*>(k + a0) = xa;
        *reinterpret_cast<uint2*>(k + b0) = xb;
      }
    }
    if (h0 + HPW > a.n_q) {  // some head of this group goes into the cache
      uint16_t* st = k_s[wave][g];
      *reinterpret_cast<uint2*>(st + a0) = xa;
      *reinterpret_cast<uint2*>(st + b0) = xb;
      wave_lds_fence();
      const uint4 x = *reinterpret_cast<const uint4*>(st + 8 * n);
      wave_lds_fence();
      const int kvh = is_v ? h - a.n_q - a.n_kv : max(h - a.n_q, 0);
      store_token<FMT, D>(page_p + (size_t)kvh * lay.head, lay, P, o, n, is_v,
                          is_v ? a.v_ts : a.k_ts, x, live && !is_q && page >= 0);
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

// Tokens first.. of sequence b that are read, in units of 16 aligned tokens.
__device__ __forceinline__ void read_span(const ReadArgs& a, int b, int64_t* f, int64_t* end,
                                          int64_t* units) {
  *f = a.first ? max((int64_t)a.first[b], (int64_t)0) : 0;
  const int64_t room = (int64_t)a.out_start[b + 1] - a.out_start[b];
  *end = min((int64_t)a.s.kv_len[b], *f + room);
  *units = *end > *f ? ((*end - 1) >> 4) - (*f >> 4) + 1 : 0;
}

constexpr uint32_t kNanPair = 0x7fc07fc0u;

// One wave per 16 aligned tokens of a sequence and head: both halves are bound
// by writing bf16 rows, so a lane takes what it writes as one vector: 8
// consecutive elements of a key, D/16 of a value (its quad layout).
template <int FMT, int D>
__global__ __launch_bounds__(256) void k_kv_read(ReadArgs a) {
  const int lane = lane_id();
  const int64_t unit = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6);
  const int h = blockIdx.y;
  // the sequence that holds this unit: a running sum over the sequences
  int64_t base = 0;
  int b = -1;
  int64_t u = 0;
  for (int i0 = 0; i0 < a.s.n_seq; i0 += 64) {
    int64_t f, e, m = 0;
    if (i0 + lane < a.s.n_seq) read_span(a, i0 + lane, &f, &e, &m);
    int64_t sum = m;
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
      const int64_t v = __shfl_up(sum, d);
      if (lane >= d) sum += v;
    }
    const uint64_t past = __ballot(base + sum > unit);
    if (past) {
      const int l = __ffsll((unsigned long long)past) - 1;
      b = i0 + l;
      u = unit - (base + __shfl(sum, l) - __shfl(m, l));
      break;
    }
    base += __shfl(sum, 63);
  }
  if (b < 0) return;
  int64_t f, end, units;
  read_span(a, b, &f, &end, &units);
  const int64_t t0 = ((f >> 4) + u) << 4;  // first token of the unit
  const int page = page_of(a.s, b, t0);
  const int P = 1 << a.s.log2P, o0 = (int)(t0 & (P - 1));
  const KvLayout lay = kv_layout(FMT, D, P);
  const uint8_t* blk = a.pool + (size_t)max(page, 0) * ((size_t)a.n_kv * lay.head) + (size_t)h * lay.head;
  const int64_t row0 = (int64_t)a.out_start[b] + t0 - f;

  if (a.k_out) {
    constexpr int LPT = D / 8, TPI = 64 / LPT;  // lanes per token, tokens at a time
    const int n = lane % LPT;
#pragma unroll
    for (int i = 0; i < 16 / TPI; ++i) {
      const int j = i * TPI + lane / LPT, o = o0 + j;
      const int64_t row = row0 + j;
      if (t0 + j < f || t0 + j >= end || row < 0 || row >= a.R) continue;
      uint4 x;
      if (page < 0) {
        x = make_uint4(kNanPair, kNanPair, kNanPair, kNanPair);
      } else if constexpr (FMT == MOE_FMT_BF16) {
        x = *reinterpret_cast<const uint4*>(blk + 2 * (o * D + 8 * n));
      } else {
        float v[8], s;
        if constexpr (FMT == MOE_FMT_NVFP4) {
          const uint32_t q = *reinterpret_cast<const uint32_t*>(blk + o * (D / 2) + 4 * n);
          const uint32_t sb = blk[lay.ks + o * (D / 16) + (n >> 1)];
          s = (sb & 0x7fu) == 0x7fu ? __uint_as_float(0x7fc00000u) : e4m3_to_f32(sb);
          typedef float f2 __attribute__((ext_vector_type(2)));
          const f2 p0 = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(q, 1.0f, 0);
          const f2 p1 = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(q, 1.0f, 1);
          const f2 p2 = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(q, 1.0f, 2);
          const f2 p3 = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(q, 1.0f, 3);
          v[0] = p0.x; v[1] = p0.y; v[2] = p1.x; v[3] = p1.y;
          v[4] = p2.x; v[5] = p2.y; v[6] = p3.x; v[7] = p3.y;
#pragma unroll
          for (int k = 0; k < 8; ++k) v[k] = v[k] * s * a.k_ts;
        } else {
          const uint2 q = *reinterpret_cast<const uint2*>(blk + o * D + 8 * n);
          s = f16_to_f32(*reinterpret_cast<const uint16_t*>(blk + lay.ks + 2 * (o * (D / 32) + (n >> 2))));
#pragma unroll
          for (int k = 0; k < 8; ++k)
            v[k] = (float)(int8_t)((k < 4 ? q.x : q.y) >> (8 * (k & 3))) * s;
        }
        x.x = (uint32_t)f32_to_bf16_rne(v[0]) | ((uint32_t)f32_to_bf16_rne(v[1]) << 16);
        x.y = (uint32_t)f32_to_bf16_rne(v[2]) | ((uint32_t)f32_to_bf16_rne(v[3]) << 16);
        x.z = (uint32_t)f32_to_bf16_rne(v[4]) | ((uint32_t)f32_to_bf16_rne(v[5]) << 16);
        x.w = (uint32_t)f32_to_bf16_rne(v[6]) | ((uint32_t)f32_to_bf16_rne(v[7]) << 16);
      }
      *reinterpret_cast<uint4*>(a.k_out + row * a.k_stride + (size_t)h * D + 8 * n) = x;
    }
  }
  if (a.v_out) {
    constexpr int GE = D / 16;  // elements of a lane: group n of the quad's token bq
    const int n = lane >> 2, bq = lane & 3;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int j = 4 * i + bq, o = o0 + j;
      const int64_t row = row0 + j;
      if (t0 + j < f || t0 + j >= end || row < 0 || row >= a.R) continue;
      uint32_t x[GE / 2];
      const uint8_t* vq = blk + lay.vq;
      if (page < 0) {
#pragma unroll
        for (int k = 0; k < GE / 2; ++k) x[k] = kNanPair;
      } else {
        uint16_t e[GE];
        if constexpr (FMT == MOE_FMT_BF16) {
          const uint16_t* src = reinterpret_cast<const uint16_t*>(vq) + ((o >> 2) * D + n * GE) * 4 + bq;
#pragma unroll
          for (int k = 0; k < GE; ++k) e[k] = src[4 * k];
        } else if constexpr (FMT == MOE_FMT_Q8_0) {
          const int8_t* src = reinterpret_cast<const int8_t*>(vq) + ((o >> 2) * D + n * GE) * 4 + bq;
          const float s = f16_to_f32(*reinterpret_cast<const uint16_t*>(blk + lay.vs + 2 * ((n * GE / 32) * P + o)));
#pragma unroll
          for (int k = 0; k < GE; ++k) e[k] = f32_to_bf16_rne((float)src[4 * k] * s);
        } else {
          const uint32_t sb = blk[lay.vs + (n * GE / 16) * P + o];
          const float s = (sb & 0x7fu) == 0x7fu ? __uint_as_float(0x7fc00000u) : e4m3_to_f32(sb);
          const uint8_t* src = vq + (((o >> 2) * 16 + n) * 4 + bq) * (GE / 2);
          uint32_t q[2] = {0, 0};
          if constexpr (GE == 4) q[0] = *reinterpret_cast<const uint16_t*>(src);
          if constexpr (GE == 8) q[0] = *reinterpret_cast<const uint32_t*>(src);
          if constexpr (GE == 16) { const uint2 t = *reinterpret_cast<const uint2*>(src); q[0] = t.x; q[1] = t.y; }
#pragma unroll
          for (int k = 0; k < GE; ++k) {
            const uint32_t c = (q[k >> 3] >> (4 * (k & 7))) & 15u;
            const uint32_t ex = (c >> 1) & 3u, m = c & 1u;
            const float mag = ex ? __uint_as_float(((ex + 126u) << 23) | (m << 22)) : 0.5f * (float)m;
            e[k] = f32_to_bf16_rne(((c & 8u) ? -mag : mag) * s * a.v_ts);
          }
        }
#pragma unroll
        for (int k = 0; k < GE / 2; ++k) x[k] = (uint32_t)e[2 * k] | ((uint32_t)e[2 * k + 1] << 16);
      }
      uint16_t* dst = a.v_out + row * a.v_stride + (size_t)h * D + n * GE;
      if constexpr (GE == 4) *reinterpret_cast<uint2*>(dst) = make_uint2(x[0], x[1]);
      if constexpr (GE >= 8) *reinterpret_cast<uint4*>(dst) = make_uint4(x[0], x[1], x[2], x[3]);
      if constexpr (GE == 16) *reinterpret_cast<uint4*>(dst + 8) = make_uint4(x[4], x[5], x[6], x[7]);
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
  const int groups = (p->n_q + 2 * c->n_kv + per_wave - 1) / per_wave;
  const int64_t wgs = (T + kRows - 1) / kRows;
  // few rows: the heads of a row spread over workgroups
  int hs = (int)((2048 + wgs - 1) / wgs);
  hs = hs < 1 ? 1 : hs > groups ? groups : hs;
  return by_format(c->fmt, c->D, [&](auto F, auto DD) {
    k_kv_append<F(), DD()><<<dim3((unsigned)wgs, (unsigned)hs), 64 * kRows, 0, stream>>>(a);
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
