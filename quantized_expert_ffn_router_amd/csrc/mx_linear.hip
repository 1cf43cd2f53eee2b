// mx_linear.hip -- product of microscaled rows with a 4-bit microscaled matrix,
//   y[t][n] = sum_k a[t][k] w[n][k] (+ bias[n]),
// the dense projections around a layer's attention and the scores over a vocabulary.
//
// The matrix units take the codes as they are, with each block's scale beside them
// (mfma_scale 16x16x128 and 32x32x64, 4-bit by 4- or 8-bit): nothing is decoded.
// Sums are fp32, but with 8-bit rows the units first cut each product to a multiple of
// 2^-13 of the power of two of the largest among its 8 neighbours: 4e-6 of the result
// (norm over norm, 2048 normal values), where the 8-bit codes themselves are rounded at
// 2^-4.  The products of 4-bit codes lose nothing.
//
// The weights are the matrix instruction's first operand, so that a lane holds 4
// neighbouring outputs of one row.  8-bit operands come in two halves, of blocks
// (0, 1) and (2, 3) of a 128-element step (16x16x128) or of both blocks of a 64-element
// one: lane group g holds elements 16 g.. of each half, and the scale of block g.
//
// A few rows are bound by reading the weights (5 x 100003 x 2048: 22.3 us, 4.9 TB/s, a large
// copy's rate), and below some 10 MB of them by the launch and the chain of loads, products
// and the waves' sum (1 x 5120 x 2048 3.5 us, 8 x 2048 x 4096 4.4; out of the caches 4.2 and
// 4.7).  Many rows: see there.
#include <algorithm>
#include <type_traits>

#include "mx.h"

namespace moe {

namespace {

typedef int v8i __attribute__((ext_vector_type(8)));
typedef float v4f __attribute__((ext_vector_type(4)));
typedef float v16f __attribute__((ext_vector_type(16)));
typedef uint32_t v4u __attribute__((ext_vector_type(4)));

constexpr int kFp8 = 0, kFp4 = 4;  // operand formats of the instructions
template <int FMT>
constexpr int kOperand = FMT == MOE_FMT_MXFP4 ? kFp4 : kFp8;

#if defined(__HIP_DEVICE_COMPILE__)  // (the host pass does not know the builtins)
typedef __amdgpu_buffer_rsrc_t Rsrc;
#else
typedef const void* Rsrc;
#endif
__device__ __forceinline__ Rsrc buffer_of(const void* p, int64_t bytes) {
#if defined(__HIP_DEVICE_COMPILE__)
  return __builtin_amdgcn_make_buffer_rsrc(const_cast<void*>(p), 0, (int)bytes, 0x00020000);
#else
  return p;
#endif
}
__device__ __forceinline__ v4u load_16(Rsrc r, uint32_t at, uint32_t base) {
#if defined(__HIP_DEVICE_COMPILE__)
  return __builtin_bit_cast(v4u, __builtin_amdgcn_raw_buffer_load_b128(r, at, base, 0));
#else
  return v4u{0, 0, 0, 0};
#endif
}
__device__ __forceinline__ uint32_t load_4(Rsrc r, uint32_t at, uint32_t base) {
#if defined(__HIP_DEVICE_COMPILE__)
  return __builtin_amdgcn_raw_buffer_load_b32(r, at, base, 0);
#else
  return 0;
#endif
}
// N bytes a lane from global memory straight into LDS: lane i's to lds + N i.  Written as
// the instruction itself: with the builtin the compiler, which does not tell the turns of a
// ring of buffers apart at the head of their loop, waits there for every load (256 rows, K
// 4096, 8 bits: 17.7 us, so 14.8).  It has no output but LDS; who reads that waits with
// wait_loads_and_reads and a barrier.
template <int N>
__device__ __forceinline__ void load_lds(Rsrc r, uint8_t* lds, uint32_t at, uint32_t base) {
#if defined(__HIP_DEVICE_COMPILE__)
  static_assert(N == 4 || N == 16, "");
  const uint32_t to = __builtin_amdgcn_readfirstlane((uint32_t)(uintptr_t)(__attribute__((address_space(3))) uint8_t*)lds);
  base = __builtin_amdgcn_readfirstlane(base);
  if constexpr (N == 16)
    asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tbuffer_load_dwordx4 %1, %2, %3 offen lds" ::"s"(to), "v"(at), "s"(r), "s"(base) : "memory", "m0");
  else
    asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tbuffer_load_dword %1, %2, %3 offen lds" ::"s"(to), "v"(at), "s"(r), "s"(base) : "memory", "m0");
#endif
}
// Waits until at most N of the wave's loads are on their way, and for all its LDS reads.
template <int N>
__device__ __forceinline__ void wait_loads_and_reads() {
#if defined(__HIP_DEVICE_COMPILE__)
  __builtin_amdgcn_s_waitcnt((N & 15) | ((N >> 4) << 14) | 0x0070);
#endif
}
struct LinearArgs {
  const uint8_t* w;         // packed codes
  const uint8_t* w_scales;  // packed scales
  const float* bias;
  const uint16_t* x;  // 16-bit rows, or NULL
  const uint8_t* codes;
  const uint8_t* scales;
  void* y;
  int64_t x_stride, y_stride, T;
  int N, K, steps, tiles, f32;
};

// Four neighbouring outputs of a row, from column n on.
__device__ __forceinline__ void store_4(const LinearArgs& a, int64_t t, int n, v4f v) {
  const int64_t at = t * a.y_stride + n;
  if (a.f32) {
    float* d = (float*)a.y + at;
    if (n + 3 < a.N) *reinterpret_cast<float4*>(d) = make_float4(v[0], v[1], v[2], v[3]);
    else
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (n + i < a.N) d[i] = v[i];
  } else {
    uint16_t* d = (uint16_t*)a.y + at;
    const uint32_t lo = bf16_pair(v[0], v[1]), hi = bf16_pair(v[2], v[3]);
    if (n + 3 < a.N) *reinterpret_cast<uint2*>(d) = make_uint2(lo, hi);
    else
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (n + i < a.N) d[i] = (uint16_t)((i < 2 ? lo : hi) >> (16 * (i & 1)));
  }
}

// ------------------------------------------------------------------ few rows

// Up to 16 rows.  A tile of 16 outputs a workgroup at a time, its waves taking KS
// steps of K each (in several passes, if K is longer) and adding up in LDS; the next
// tile's weights are on their way while one is worked on.  The rows' codes stay in
// registers while there is one pass; ROWS: they are made here from 16-bit rows.
template <int FMT, bool ROWS, int KS>
__global__ __launch_bounds__(1024) void k_mx_few(LinearArgs a, int passes) {
  extern __shared__ v4f part[];  // [2][waves][64]
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), waves = blockDim.x >> 6;
  const int lane = lane_id(), r = lane & 15, g = lane >> 4;
  v8i b[KS];
  int bs[KS];

  const auto rows = [&](int pass) {
#pragma unroll
    for (int s = 0; s < KS; ++s) {
      const int ks = (pass * waves + wave) * KS + s;
      const bool in = r < a.T && ks < a.steps;
      v4u q[2] = {v4u{0, 0, 0, 0}, v4u{0, 0, 0, 0}};
      uint32_t sc = 0;
      if constexpr (!ROWS) {
        if (in) {
          const uint8_t* p = a.codes + (int64_t)r * mx_bytes<FMT>(a.K) + mx_bytes<FMT>(ks * kMxStep) + 16 * g;
          q[0] = *reinterpret_cast<const v4u*>(p);
          if constexpr (FMT == MOE_FMT_MXFP8) q[1] = *reinterpret_cast<const v4u*>(p + 64);
          sc = a.scales[(int64_t)r * (a.K / kMxBlock) + ks * 4 + g];
        }
      } else {
        // 32 elements: those of block g, or 16 of each half
        uint4 x[4];
        const uint16_t* p = a.x + (int64_t)r * a.x_stride + ks * kMxStep + (FMT == MOE_FMT_MXFP4 ? 32 : 16) * g;
#pragma unroll
        for (int i = 0; i < 4; ++i)
          x[i] = in ? *reinterpret_cast<const uint4*>(p + 8 * i + (FMT == MOE_FMT_MXFP8 && i > 1 ? 48 : 0))
                    : make_uint4(0, 0, 0, 0);
        if constexpr (FMT == MOE_FMT_MXFP4) {
          sc = mx_scale<FMT>(max(max(mx_top(x[0]), mx_top(x[1])), max(mx_top(x[2]), mx_top(x[3]))));
#pragma unroll
          for (int i = 0; i < 4; ++i) q[0][i] = mx_codes<FMT>(x[i], sc).x;
        } else {
          // a block's other 16 elements are in the neighbouring lane group, and block
          // g's scale in another
          uint32_t s2[2];
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const uint32_t top = max(mx_top(x[2 * h]), mx_top(x[2 * h + 1]));
            const auto m = __builtin_amdgcn_permlane16_swap(top, top, false, false);
            s2[h] = mx_scale<FMT>(max((uint32_t)m[0], (uint32_t)m[1]));
#pragma unroll
            for (int i = 0; i < 2; ++i) {
              const uint2 c = mx_codes<FMT>(x[2 * h + i], s2[h]);
              q[h][2 * i] = c.x;
              q[h][2 * i + 1] = c.y;
            }
          }
          const int from = (g & 1) * 32 + r;
          const uint32_t s0 = __shfl((int)s2[0], from), s1 = __shfl((int)s2[1], from);
          sc = g < 2 ? s0 : s1;
        }
      }
#pragma unroll
      for (int i = 0; i < 8; ++i) b[s][i] = (int)q[i >> 2][i & 3];
      bs[s] = (int)sc;
    }
  };

  v4u w[KS];
  uint32_t ws[KS];
  const auto weights = [&](int tile, int pass) {  // (steps past the last one read as zero)
    const int ks = (pass * waves + wave) * KS;
    const int left = min(max(a.steps - ks, 0), KS);
    const Rsrc c = buffer_of(a.w + ((int64_t)tile * a.steps + ks) * 1024, left * 1024);
    const Rsrc d = buffer_of(a.w_scales + ((int64_t)tile * a.steps + ks) * 64, left * 64);
#pragma unroll
    for (int s = 0; s < KS; ++s) {
      w[s] = load_16(c, s * 1024 + lane * 16, 0);
      ws[s] = load_4(d, s * 64 + r * 4, 0);
    }
  };

  int tile = blockIdx.x, pass = 0, turn = 0;
  weights(tile, 0);
  rows(0);
  v4f o = v4f{0.f, 0.f, 0.f, 0.f};
  while (true) {
    v4u c[KS];
    uint32_t cs[KS];
#pragma unroll
    for (int s = 0; s < KS; ++s) { c[s] = w[s]; cs[s] = ws[s]; }
    const bool last = pass + 1 == passes;
    const int next = last ? tile + (int)gridDim.x : tile;
    if (next < a.tiles) weights(next, last ? 0 : pass + 1);
#pragma unroll
    for (int s = 0; s < KS; ++s) {
      v8i m;
#pragma unroll
      for (int i = 0; i < 8; ++i) m[i] = i < 4 ? (int)c[s][i] : 0;
      o = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(m, b[s], o, kFp4, kOperand<FMT>, 0,
                                                           (int)(cs[s] >> (8 * g)), 0, bs[s]);
    }
    if (last) {
      v4f* const p = part + turn * waves * 64;
      p[wave * 64 + lane] = o;
      __syncthreads();
      if (wave == 0) {
        v4f sum = p[lane];
        for (int k = 1; k < waves; ++k) sum += p[k * 64 + lane];
        const int n = tile * kMxTile + 4 * g;
        if (a.bias)
#pragma unroll
          for (int e = 0; e < 4; ++e) sum[e] += n + e < a.N ? a.bias[n + e] : 0.0f;
        if (r < a.T) store_4(a, r, n, sum);
      }
      turn ^= 1;  // (the other half is free once all have passed this barrier)
      o = v4f{0.f, 0.f, 0.f, 0.f};
    }
    if (next >= a.tiles) break;
    tile = next;
    pass = last ? 0 : pass + 1;
    if (passes > 1) rows(pass);
  }
}

struct Few {
  int ks, waves, passes;
};
// How a product of few rows is cut, by the steps of K and the tiles of N.  (5120 x 2048, 8 bits:
// 16 rows 4.9 us; 17 as two tiles of 16 rows here 5.6, as a tile of 64 below 5.7, and 32 rows
// 7.7 and 5.7; 32 x 20000 x 2048 17.7 and 8.1.)
constexpr int64_t kFewRows = 16;
Few few_of(int steps, int tiles) {
  Few f;
  const int most = 16;
  // two steps of K a wave while the waves of a workgroup reach over all of it, four for many
  // outputs of a longer K (5 x 100003 x 2048 23.0 us, with two 24.3)
  f.ks = steps <= 8 || (steps <= 2 * most && tiles < 1024) ? 2 : 4;
  f.waves = std::min((steps + f.ks - 1) / f.ks, most);
  f.passes = (steps + f.ks * f.waves - 1) / (f.ks * f.waves);
  return f;
}

template <int FMT>
void launch_few(const LinearArgs& a, hipStream_t stream) {
  const Few f = few_of(a.steps, a.tiles);
  // (what runs at once: 16 waves a CU)
  const unsigned grid = (unsigned)std::min(a.tiles, 256 * std::max(16 / f.waves, 1));
  const unsigned block = 64 * f.waves;
  const size_t lds = (size_t)2 * f.waves * 1024;
  if (a.x) k_mx_few<FMT, true, 2><<<grid, block, lds, stream>>>(a, f.passes);
  else if (f.ks == 2) k_mx_few<FMT, false, 2><<<grid, block, lds, stream>>>(a, f.passes);
  else k_mx_few<FMT, false, 4><<<grid, block, lds, stream>>>(a, f.passes);
}

// ------------------------------------------------------------------ many rows

// One workgroup: WT x WN waves, each FT x FN squares of 32 rows by 32 outputs.  Per
// step of 128 elements the rows' and the weights' codes and scales go from global
// memory into one of three LDS buffers, up to three steps ahead.  The waves meet in the
// midst of a step, between its two halves: the operands of the half behind the barrier
// are in registers by then, those of the next step's first half are read beside it, so
// that the matrix units do not wait for LDS.
//
// 16384 x 5120 x 2048 of 8-bit rows 154 to 169 us (2.0 to 2.2 PFLOP/s), of 4-bit rows 138 (2.5);
// 8192 x 2048 x 4096 62 and 45 (2.2 and 3.1), 53 and 39 where rows and results stay in the last
// cache; a bf16 library product reaches 1.2, the instructions themselves, from registers, 4.7
// and 8.2.  32-bit results take longer to store: 236 and 211 us, 75 and 71.  The
// matrix units are half of the time busy at the 2.1 GHz they hold: codes that are all zero
// took 14 % less (power), steps whose loads read nothing a quarter less than that: loads into
// LDS beside the reads of it.  Two groups of waves that take every other step: no gain.
template <int FMT, int WT, int WN, int FT, int FN>
struct Gemm {
  static constexpr int WAVES = WT * WN, BT = WT * FT * 32, BN = WN * FN * 32;
  static constexpr int CB = mx_bytes<FMT>(kMxStep);  // bytes of a row's step
  static constexpr int NA = BT * CB / 1024, NB = BN / 16, NS = (BT + BN) / 64;  // wave loads
  static constexpr int OA = 0, OB = BT * CB, OS = OB + BN * 64, BYTES = OS + (BT + BN) * 4;
  static constexpr int PER = (NA + NB + WAVES - 1) / WAVES + 1;  // loads of a wave
  static_assert(NA % WAVES == 0 && NB % WAVES == 0 && NS <= WAVES, "waves share the loads evenly");

  const LinearArgs& a;
  const uint8_t *rows, *weights, *scales;  // scales: of rows or weights, as this wave loads them
  int64_t row_bytes, weight_bytes, scale_bytes;
  int wave, lane, r, h, wt, wn, scale_step;
  uint32_t at[PER];

  // What the chunks of a row are permuted by in LDS.
  __device__ __forceinline__ static int place(int row) {
    return FMT == MOE_FMT_MXFP8 ? (row >> 1) & 7 : (row >> 2) & 3;
  }
  __device__ __forceinline__ Gemm(const LinearArgs& args, int64_t t0, int tile0, int w) : a(args), wave(w), lane(lane_id()) {
    r = lane & 31;
    h = lane >> 5;
    wt = wave / WN;
    wn = wave % WN;
    const int64_t pitch = mx_bytes<FMT>(a.K), n = min(a.T - t0, (int64_t)BT);
    const int64_t m = min(a.tiles - tile0, BN / 16);
    rows = a.codes + t0 * pitch;
    row_bytes = n * pitch;
    weights = a.w + (int64_t)tile0 * a.steps * 1024;
    weight_bytes = m * a.steps * 1024;
#pragma unroll
    for (int i = 0; i < PER - 1; ++i) {
      const int u = i * WAVES + wave;
      if (i < NA / WAVES) {
        // 8 bits: 8 rows of 8 chunks of 16 bytes, 4 bits: 16 rows of 4.  Neighbouring lanes
        // take chunks of one row, permuted so that 16 rows' reads of a chunk meet all banks.
        // (Lanes of different rows are looked up one by one: 64 x 2048 x 4096 of 8 bits 13.7
        // us, so 9.0; 8192 rows 58, so 53.)
        if constexpr (FMT == MOE_FMT_MXFP8) {
          const int row = u * 8 + (lane >> 3);
          at[i] = (uint32_t)(row * pitch + ((lane & 7) ^ place(row)) * 16);
        } else {
          const int row = u * 16 + (lane >> 2);
          at[i] = (uint32_t)(row * pitch + ((lane & 3) ^ place(row)) * 16);
        }
      } else {
        at[i] = (uint32_t)((u - NA) * a.steps * 1024 + lane * 16);
      }
    }
    const int u = wave % NS, width = a.K / kMxBlock;  // (waves past the last load repeat one)
    const bool of_rows = u < BT / 64;
    scales = of_rows ? a.scales + t0 * width : a.w_scales + (int64_t)tile0 * a.steps * 64;
    scale_bytes = of_rows ? n * width : m * a.steps * 64;
    scale_step = of_rows ? 4 : 64;
    at[PER - 1] = of_rows ? (uint32_t)((u * 64 + lane) * width)
                          : (uint32_t)(((u - BT / 64) * 4 + (lane >> 4)) * a.steps * 64 + (lane & 15) * 4);
  }
  // (Of a step behind the last one nothing is read: its loads are there so that as many are
  // always on their way, without a branch, past which the matrix instructions would move.)
  struct Step {
    Rsrc x, w, s;
    int k;
  };
  __device__ __forceinline__ Step step(int ks) const {
    const bool in = ks < a.steps;
    return Step{buffer_of(rows, in ? row_bytes : 0), buffer_of(weights, in ? weight_bytes : 0),
                buffer_of(scales, in ? scale_bytes : 0), in ? ks : 0};
  }
  // Load i of PER.
  __device__ __forceinline__ void load(const Step& f, uint8_t* lds, int i) const {
    const int u = i * WAVES + wave;
    if (i == PER - 1) load_lds<4>(f.s, lds + OS + (wave % NS) * 256, at[PER - 1], f.k * scale_step);
    else if (i < NA / WAVES) load_lds<16>(f.x, lds + OA + u * 1024, at[i], f.k * CB);
    else load_lds<16>(f.w, lds + OB + (u - NA) * 1024, at[i], f.k * 1024);
  }
  __device__ __forceinline__ void load(uint8_t* lds, int ks) const {
    const Step f = step(ks);
#pragma unroll
    for (int i = 0; i < PER; ++i) load(f, lds, i);
  }
  __device__ __forceinline__ v8i row_part(const uint8_t* lds, int f, int j) const {
    const int row = (wt * FT + f) * 32 + r;
    v4u q[2] = {v4u{0, 0, 0, 0}, v4u{0, 0, 0, 0}};
    if constexpr (FMT == MOE_FMT_MXFP8) {
#pragma unroll
      for (int k = 0; k < 2; ++k)
        q[k] = *reinterpret_cast<const v4u*>(lds + OA + row * 128 + ((4 * j + 2 * k + h) ^ place(row)) * 16);
    } else {
      q[0] = *reinterpret_cast<const v4u*>(lds + OA + row * 64 + ((2 * j + h) ^ place(row)) * 16);
    }
    v8i v;
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = (int)q[i >> 2][i & 3];
    return v;
  }
  __device__ __forceinline__ v8i weight_part(const uint8_t* lds, int f, int j) const {
    const int row = (wn * FN + f) * 32 + r;
    const v4u q = *reinterpret_cast<const v4u*>(lds + OB + (row >> 4) * 1024 + (2 * j + h) * 256 + (row & 15) * 16);
    v8i v;
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = i < 4 ? (int)q[i] : 0;
    return v;
  }
  // The operands of half a step, J: 64 elements of each row and output.
  struct Parts {
    v8i p[FT], q[FN];
  };
  // Part i of FN + FT, in the order of their use.
  __device__ __forceinline__ void part(const uint8_t* lds, int j, Parts& f, int i) const {
    if (i < FN) f.q[i] = weight_part(lds, i, j);
    else f.p[i - FN] = row_part(lds, i - FN, j);
  }
  // The step's scales, as they lie: that of block 2 J + h of a row is byte 2 J of its word
  // shifted by h bytes.
  struct Scales {
    uint32_t p[FT], q[FN];
  };
  __device__ __forceinline__ void scales_of(const uint8_t* lds, Scales& s) const {
#pragma unroll
    for (int n = 0; n < FN; ++n)
      s.q[n] = *reinterpret_cast<const uint32_t*>(lds + OS + (BT + (wn * FN + n) * 32 + r) * 4);
#pragma unroll
    for (int t = 0; t < FT; ++t)
      s.p[t] = *reinterpret_cast<const uint32_t*>(lds + OS + ((wt * FT + t) * 32 + r) * 4);
  }
  __device__ __forceinline__ void shift(Scales& s) const {
#pragma unroll
    for (int n = 0; n < FN; ++n) s.q[n] >>= 8 * h;
#pragma unroll
    for (int t = 0; t < FT; ++t) s.p[t] >>= 8 * h;
  }
  // The FT * FN matrix instructions of half a step; beside them the caller's pieces
  // 0 .. PIECES - 1 (a type each), all but the last instruction's time for them.  Kept in
  // this order: left to the compiler, the loads and the wait for the next scales stood before
  // the instructions (16384 x 5120 x 2048, 8 bits: 168 us, so 165).
  template <int J, int PIECES, typename P>
  __device__ __forceinline__ void product(const Parts& f, const Scales& s, v16f (&o)[FT][FN], P piece) const {
    each<0, FT * FN>([&](auto I) {
      constexpr int i = I(), t = i / FN, n = i % FN, M = FT * FN > 1 ? FT * FN - 1 : 1;
      o[t][n] = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(f.q[n], f.p[t], o[t][n], kFp4, kOperand<FMT>,
                                                                2 * J, (int)s.q[n], 2 * J, (int)s.p[t]);
      if constexpr (i < M) each<PIECES * i / M, PIECES * (i + 1) / M>(piece);
      __builtin_amdgcn_sched_barrier(0);
    });
  }
};

template <int FMT, int WT, int WN, int FT, int FN>
__global__ __launch_bounds__(64 * WT * WN) void k_mx_gemm(LinearArgs a, int tiles_t, int tiles_n) {
  typedef Gemm<FMT, WT, WN, FT, FN> G;
  __shared__ __align__(16) uint8_t b0[G::BYTES], b1[G::BYTES], b2[G::BYTES];
  // Workgroups go to the 8 dies in turn: each die takes a run of tiles, 8 tiles of rows
  // by what is in flight, so that rows and weights are shared in its cache.
  const int total = tiles_t * tiles_n, per = (total + 7) / 8;
  const int id = (int)(blockIdx.x & 7) * per + (int)(blockIdx.x >> 3);
  if ((int)(blockIdx.x >> 3) >= per || id >= total) return;
  const int band = id / (8 * tiles_n), in = id - band * 8 * tiles_n;
  const int high = min(8, tiles_t - band * 8);
  const int tn = in / high, tt = band * 8 + in % high;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int64_t t0 = (int64_t)tt * G::BT;
  const int n0 = tn * G::BN;
  const G m(a, t0, n0 / 16, wave);

  v16f o[FT][FN];  // (from the bias on; past its end, or without one, from 0)
  const Rsrc bias = buffer_of(a.bias, a.bias ? (int64_t)a.N * 4 : 0);
#pragma unroll
  for (int n = 0; n < FN; ++n)
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      const int c = n0 + (m.wn * FN + n) * 32 + 8 * (i >> 2) + 4 * m.h + (i & 3);
      const float v = __uint_as_float(load_4(bias, c * 4, 0));
#pragma unroll
      for (int f = 0; f < FT; ++f) o[f][n][i] = v;
    }
  const int steps = a.steps;
  typename G::Parts f0, f1;
  typename G::Scales sc;
  const auto meet = [&] {
    asm volatile("" ::: "memory");
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
  };
  // Step ks: its first half's operands and its scales are there, or on their way.
  const auto turn = [&](int ks, uint8_t* now, uint8_t* next) {
    const typename G::Step ahead = m.step(ks + 3);
    m.shift(sc);
    m.template product<0, FN + FT>(f0, sc, o, [&](auto i) { m.part(now, 1, f1, i()); });
    wait_loads_and_reads<G::PER>();  // the next step's, of those that are on their way
    meet();
    typename G::Scales after;  // (behind the last step: of nothing that is used)
    m.template product<1, G::PER + 1 + FN + FT>(f1, sc, o, [&](auto i) {
      constexpr int k = i() - G::PER - 1;
      if constexpr (k < -1) m.load(ahead, now, i());
      else if constexpr (k == -1) m.scales_of(next, after);
      else m.part(next, 0, f0, k);
    });
    sc = after;
  };
  m.load(b0, 0);
  m.load(b1, 1);
  m.load(b2, 2);
  wait_loads_and_reads<2 * G::PER>();
  meet();
  m.scales_of(b0, sc);
#pragma unroll
  for (int i = 0; i < FN + FT; ++i) m.part(b0, 0, f0, i);
#pragma unroll 1
  for (int ks = 0; ks < steps; ks += 3) {
    turn(ks, b0, b1);
    if (ks + 1 < steps) turn(ks + 1, b1, b2);
    if (ks + 2 < steps) turn(ks + 2, b2, b0);
  }
  wait_loads_and_reads<0>();

  if (a.f32) {
#pragma unroll
    for (int f = 0; f < FT; ++f) {
      const int64_t t = t0 + (m.wt * FT + f) * 32 + m.r;
      if (t >= a.T) continue;
#pragma unroll
      for (int n = 0; n < FN; ++n)
#pragma unroll
        for (int i = 0; i < 16; i += 4)
          store_4(a, t, n0 + (m.wn * FN + n) * 32 + 2 * i + 4 * m.h, v4f{o[f][n][i], o[f][n][i + 1], o[f][n][i + 2], o[f][n][i + 3]});
    }
    return;
  }
  // 16 bits: 32 rows at a time through LDS, so that a row's outputs are stored together.
  constexpr int PITCH = FN * 64 + 16, LPR = FN * 4;  // lanes of a row, 8 outputs each
  static_assert(G::WAVES / 2 * 32 * PITCH <= G::BYTES, "half of the waves' rows in a buffer");
  __syncthreads();
  uint8_t* const mine = (wave < G::WAVES / 2 ? b0 : b1) + (wave % (G::WAVES / 2)) * 32 * PITCH;
#pragma unroll
  for (int f = 0; f < FT; ++f) {
#pragma unroll
    for (int n = 0; n < FN; ++n)
#pragma unroll
      for (int i = 0; i < 16; i += 4)
        *reinterpret_cast<uint2*>(mine + m.r * PITCH + (n * 32 + 2 * i + 4 * m.h) * 2) =
            make_uint2(bf16_pair(o[f][n][i], o[f][n][i + 1]), bf16_pair(o[f][n][i + 2], o[f][n][i + 3]));
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    __builtin_amdgcn_wave_barrier();
#pragma unroll
    for (int k = 0; k < 32 * LPR / 64; ++k) {
      const int row = (k * 64 + m.lane) / LPR, col = (m.lane % LPR) * 8;
      const uint4 v = *reinterpret_cast<const uint4*>(mine + row * PITCH + col * 2);
      const int64_t t = t0 + (m.wt * FT + f) * 32 + row;
      const int c = n0 + m.wn * FN * 32 + col;
      if (t >= a.T) continue;
      uint16_t* d = (uint16_t*)a.y + t * a.y_stride + c;
      if (c + 7 < a.N) {
        *reinterpret_cast<uint4*>(d) = v;
      } else {
        const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
        for (int e = 0; e < 8; ++e)
          if (c + e < a.N) d[e] = (uint16_t)(w[e >> 1] >> (16 * (e & 1)));
      }
    }
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    __builtin_amdgcn_wave_barrier();
  }
}

template <int FMT, int WT, int WN, int FT, int FN>
void launch_gemm(const LinearArgs& a, hipStream_t stream) {
  typedef Gemm<FMT, WT, WN, FT, FN> G;
  const int tiles_t = (int)((a.T + G::BT - 1) / G::BT), tiles_n = (a.N + G::BN - 1) / G::BN;
  const unsigned grid = (unsigned)(((int64_t)tiles_t * tiles_n + 7) / 8 * 8);
  k_mx_gemm<FMT, WT, WN, FT, FN><<<grid, 64 * WT * WN, 0, stream>>>(a, tiles_t, tiles_n);
}

template <int FMT>
void linear(const LinearArgs& a, hipStream_t stream) {
  if (a.T <= kFewRows) {
    launch_few<FMT>(a, stream);
    return;
  }
  // The tile whose rounds over the 256 CUs take the least, with the time of a round of each
  // kind as measured (8 bits, K 4096: 39 us of 256 x 256, 24 of 128 x 256, 17 of 128 x 128, 12
  // of 64 x 128); 64 x 64 where tiles of 64 x 128 leave half of the CUs without (it reads
  // more).  8 bits, tiles in that order: 16384 x 5120 x 2048 154, 183, 176, 197, 260 us; 4096
  // rows 50, 43, 43, 48, 63; 1024 rows 24, 15, 16, 15, 19; 2048 x 2048 x 4096 40, 25, 20, 20,
  // 26; 256 x 5120 x 2048 23, 14, 10, 7.8, 8.9; 64 rows 21, 13, 9.5, 6.6, 5.9.
  const auto tiles = [&](int bt, int bn) { return ((a.T + bt - 1) / bt) * ((a.N + bn - 1) / bn); };
  const auto rounds = [&](int bt, int bn) { return (tiles(bt, bn) + 255) / 256; };
  const int64_t cost[5] = {100 * rounds(256, 256), 62 * rounds(128, 256), 43 * rounds(128, 128), 30 * rounds(64, 128),
                           tiles(64, 128) < 128 ? 27 : INT64_MAX};
  switch (std::min_element(cost, cost + 5) - cost) {
    case 0:
      // (8-bit rows: a wave reads 64 of them and 128 outputs, not 128 and 64, a fifth less of
      // LDS: 171 us, so 167)
      if constexpr (FMT == MOE_FMT_MXFP8) launch_gemm<FMT, 4, 2, 2, 4>(a, stream);
      else launch_gemm<FMT, 2, 4, 4, 2>(a, stream);
      break;
    case 1: launch_gemm<FMT, 2, 4, 2, 2>(a, stream); break;
    case 2: launch_gemm<FMT, 2, 2, 2, 2>(a, stream); break;
    case 3: launch_gemm<FMT, 1, 4, 2, 1>(a, stream); break;
    default: launch_gemm<FMT, 2, 2, 1, 1>(a, stream);
  }
}

// One thread: 16 bytes of codes, or a row's scales of a step.
__global__ __launch_bounds__(256) void k_mx_pack(const uint8_t* codes, const uint8_t* scales, int N, int K,
                                                 int64_t chunks, int64_t words, uint8_t* packed, size_t at_scales) {
  const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
  const int steps = K / kMxStep;
  if (i < chunks) {
    const int64_t unit = i >> 6, n = unit / steps * kMxTile + (i & 15);
    const int64_t at = unit % steps * 64 + ((i >> 4) & 3) * 16;
    *reinterpret_cast<uint4*>(packed + i * 16) =
        n < N ? *reinterpret_cast<const uint4*>(codes + n * (K / 2) + at) : make_uint4(0, 0, 0, 0);
  } else if (i < chunks + words) {
    const int64_t k = i - chunks, unit = k >> 4, n = unit / steps * kMxTile + (k & 15);
    *reinterpret_cast<uint32_t*>(packed + at_scales + k * 4) =
        n < N ? *reinterpret_cast<const uint32_t*>(scales + n * (K / kMxBlock) + unit % steps * 4) : 0u;
  }
}

}  // namespace

hipError_t launch_mx_pack(int N, int K, const uint8_t* codes, const uint8_t* scales, void* packed,
                          hipStream_t stream) {
  const MxLayout l = mx_layout(N, K);
  const int64_t chunks = l.tiles * l.steps * 64, words = l.tiles * l.steps * 16;
  k_mx_pack<<<(unsigned)((chunks + words + 255) / 256), 256, 0, stream>>>(codes, scales, N, K, chunks, words,
                                                                          (uint8_t*)packed, l.scales);
  return hipGetLastError();
}

// Few rows whose codes a workgroup's waves hold: each workgroup makes them again (16 x 5120 x
// 2048, 8 bits: 6.8 us, where a launch of its own takes 2.3 beside the product's 5.4; 5 x
// 100003 x 2048, 512 workgroups, 25.5 against 24.2 for the two launches).
bool mx_linear_takes_rows(int64_t N, int64_t K, int64_t T) {
  const MxLayout l = mx_layout(N, K);
  const Few f = few_of((int)l.steps, (int)std::min(l.tiles, (int64_t)INT32_MAX));
  return T <= kFewRows && f.ks == 2 && f.passes == 1;
}

hipError_t launch_mx_linear(const moe_mx_matrix* w, int fmt, const uint16_t* x, int64_t x_stride,
                            const uint8_t* codes, const uint8_t* scales, int64_t T, void* y,
                            int64_t y_stride, int y_dtype, hipStream_t stream) {
  const MxLayout l = mx_layout(w->N, w->K);
  const uint8_t* p = (const uint8_t*)w->packed;
  const LinearArgs a{p, p + l.scales, w->bias, x, codes, scales, y, x_stride, y_stride, T,
                     w->N, w->K, (int)l.steps, (int)l.tiles, y_dtype == MOE_DTYPE_F32};
  if (fmt == MOE_FMT_MXFP4) linear<MOE_FMT_MXFP4>(a, stream);
  else linear<MOE_FMT_MXFP8>(a, stream);
  return hipGetLastError();
}

}  // namespace moe
