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
//
// Bound by the matrix units at the clock they hold under load: 8192 rows behind
// 8192 keys (32 heads of 128) 1350 to 1450 us over runs and cards, 1.14 to 1.22 PFLOP/s
// of visible pairs, where a large bf16 library product reaches 1.17.  16384 rows of
// nine prompts of 630 to 3150 rows: 323 to 347 us (359 as single launches under a
// profiler), 0.9 to 0.95; there every tile's start, the part of its last keys that is
// masked, and the output weigh more.  333 rows take 12 us: six tiles of keys one
// after the other, 1.1 us each, on a card that is mostly empty.  8192 rows at heads
// of 64, 128 and 256: 280, 478 and 1030 us (0.98, 1.15 and 1.07 PFLOP/s).
#include "attn_tile.h"

namespace moe {

namespace {

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

// One head's key or value rows of a sequence, as tiles of 64 rows that go
// straight from global memory into LDS: lane i of a load fills the 16 bytes at
// slot i and reads the chunk that belongs there.  Buffer loads: the lanes'
// offsets are the same for every tile, rows past the last one read as zero, and
// reads of other tiles need not wait for them.
template <int D, int WAVES>
struct Tiles {
  static constexpr int CPR = D / 8;                     // chunks of a row
  static constexpr int LOADS = kBN * CPR / 64 / WAVES;  // loads of a wave
  const uint16_t* base;
  int64_t stride, len;
  uint32_t off[LOADS];

  __device__ __forceinline__ Tiles(const uint16_t* p, int64_t st, int64_t n, int wave, int lane)
      : base(p), stride(st), len(n) {
#pragma unroll
    for (int i = 0; i < LOADS; ++i) {
      const int slot = (i * WAVES + wave) * 64 + lane;
      const int row = slot / CPR, chunk = swz<D>(row, slot % CPR);
      off[i] = (uint32_t)((row * stride + chunk * 8) * 2);
    }
  }
  __device__ __forceinline__ void load(uint8_t* lds, int it, int wave) const {
#if defined(__HIP_DEVICE_COMPILE__)  // (the host pass does not know the builtins)
    const int64_t t0 = (int64_t)it * kBN;
    const int64_t left = min(len - t0, (int64_t)kBN);
    const auto rsrc = __builtin_amdgcn_make_buffer_rsrc(
        const_cast<uint16_t*>(base + t0 * stride), 0, (int)(((left - 1) * stride + D) * 2), 0x00020000);
#pragma unroll
    for (int i = 0; i < LOADS; ++i)
      __builtin_amdgcn_raw_ptr_buffer_load_lds(
          rsrc, (__attribute__((address_space(3))) void*)(lds + (i * WAVES + wave) * 1024), 16,
          off[i], 0, 0, 0);
#endif
  }
};

// One wave's 32 query rows of one head; a lane column is a row.
template <int D>
struct Rows : TileRows<D> {
  static constexpr int KS = D / 16, NJ = D / 32;
  using TileRows<D>::qf;
  using TileRows<D>::o;
  using TileRows<D>::h;
  uint32_t ka[KS], va[NJ][2];  // this lane's places in a K and a V tile

  __device__ __forceinline__ void places(int lane) {
    const int n = lane & 31;
    h = lane >> 5;
#pragma unroll
    for (int s = 0; s < KS; ++s) ka[s] = n * (2 * D) + swz<D>(n, 2 * s + h) * 16;
#pragma unroll
    for (int j = 0; j < NJ; ++j)
#pragma unroll
      for (int q = 0; q < 2; ++q) {
        const int row = 8 * q + 4 * h + ((lane & 15) >> 2);
        const int col = 32 * j + ((lane >> 4) & 1) * 16 + 4 * (lane & 3);
        va[j][q] = row * (2 * D) + swz<D>(row, col >> 3) * 16 + (col & 4) * 2;
      }
  }
  // Key fragment: 16 elements (step s) of 32 keys (half t).  The permutation
  // of chunks repeats every 16 rows, so half t is a constant away.
  __device__ __forceinline__ v4u key(const uint8_t* kt, int t, int s) const {
    return *reinterpret_cast<const v4u*>(kt + ka[s] + t * (64 * D));
  }
  // Value fragment of 16 keys (step s) and 32 elements (block j), transposed
  // out of LDS: keys 4h.. and 8 + 4h.., as the score accumulators hold them.
  __device__ __forceinline__ v4u value(const uint8_t* vt, int s, int j) const {
    v4u f;
#pragma unroll
    for (int q = 0; q < 2; ++q) {
      const uint8_t* ad = vt + va[j][q] + s * (32 * D);
      const v4s r = __builtin_amdgcn_ds_read_tr16_b64_v4i16((__attribute__((address_space(3))) v4s*)(ad));
      const uint2 w = __builtin_bit_cast(uint2, r);
      f[2 * q] = w.x;
      f[2 * q + 1] = w.y;
    }
    return f;
  }
  __device__ __forceinline__ void scores(const uint8_t* kt, v16f (&x)[2]) const {
#pragma unroll
    for (int t = 0; t < 2; ++t) {
#pragma unroll
      for (int i = 0; i < 16; ++i) x[t][i] = 0.0f;
#pragma unroll
      for (int s = 0; s < KS; ++s) x[t] = mma(key(kt, t, s), qf[s], x[t]);
    }
  }
  template <bool NEXT>
  __device__ __forceinline__ void step(const uint8_t* kt, const uint8_t* vt, float c,
                                       v16f (&x)[2], v16f (&y)[2]) {
    this->template stream<NEXT>([&](int t, int s) { return key(kt, t, s); },
                                [&](int s, int j) { return value(vt, s, j); }, c, x, y, [](auto) {});
  }
};

// The tile once more with a running maximum, and with infinities and NaN kept
// from rows that do not see them: for data that the fast pass cannot hold.
template <int D, int WAVES>
__device__ __forceinline__ void careful_pass(Rows<D>& w, uint8_t* kt, uint8_t* vt,
                                             const Tiles<D, WAVES>& K, const Tiles<D, WAVES>& V,
                                             float c, int n_tiles, int64_t lo_wave, int wave,
                                             int lane) {
  constexpr int TILE = kBN * D * 2, NJ = D / 32;
  w.clear();
#pragma unroll 1
  for (int it = 0; it < n_tiles; ++it) {
    __syncthreads();
    K.load(kt, it, wave);
    V.load(vt, it, wave);
    wait_loads<0>();
    __syncthreads();
    const int64_t t0 = (int64_t)it * kBN;
    v16f x[2];
    v4u p[4];
    w.scores(kt, x);
    w.mask(x, t0);
    const float mx = w.top(x, c);
    if (__any(mx > w.m + kGrow)) {
      const float mn = fmaxf(w.m, mx), al = __builtin_amdgcn_exp2f(w.m - mn);
#pragma unroll
      for (int j = 0; j < NJ; ++j)
#pragma unroll
        for (int i = 0; i < 16; ++i) w.o[j][i] *= al;
      w.l *= al;
      w.m = mn;
    }
#pragma unroll
    for (int v = 0; v < 32; ++v) w.weight(x, c, p, v);
    bool any = false;
    if (t0 + kBN - 1 > lo_wave) {  // some row does not see all of the tile
#pragma unroll 1
      for (int i = lane; i < TILE / 16; i += 64) {
        const v4u f = reinterpret_cast<const v4u*>(vt)[i];
#pragma unroll
        for (int k = 0; k < 4; ++k)
          any |= (f[k] & 0x7f80u) == 0x7f80u || (f[k] & 0x7f800000u) == 0x7f800000u;
      }
    }
    const bool wild = __any(any);
#pragma unroll
    for (int s = 0; s < 4; ++s)
#pragma unroll
      for (int j = 0; j < NJ; ++j) {
        const v4u f = w.value(vt, s, j);
        if (!wild) {
          w.o[j] = mma(f, p[s], w.o[j]);
          continue;
        }
        // A zero weight would not silence them: one key at a time, added only
        // to the rows that see it.
#pragma unroll 1
        for (int tk = 0; tk < 16; ++tk) {
          const int at = 2 * (tk >> 3) + ((tk & 3) >> 1);
          const uint32_t keep = w.h == ((tk >> 2) & 1) ? 0xffffu << (16 * (tk & 1)) : 0u;
          const bool seen = t0 + 16 * s + tk <= w.limit;
          v4u one;
#pragma unroll
          for (int i = 0; i < 4; ++i) one[i] = i == at ? f[i] & keep : 0u;
          v16f z;
#pragma unroll
          for (int i = 0; i < 16; ++i) z[i] = 0.0f;
          z = mma(one, p[s], z);
#pragma unroll
          for (int i = 0; i < 16; ++i) w.o[j][i] += seen ? z[i] : 0.0f;
        }
      }
  }
}

// The weights are bf16, whose exponent range is that of fp32, so a row's
// maximum is taken from its first tile of keys only: later weights may exceed 1
// by any factor the range holds, without loss.  Where they leave it (a sum over
// kFar, or not finite: then also for infinities and NaN in the data) the
// workgroup goes over its tile again with a running maximum.
//
// Scores of the next tile are computed while the present one's go through the
// exponential: the two share nothing, so matrix and vector instructions fill
// one another's gaps within a wave.  Not so for the tiles that a row sees in part:
// there the code would be twice as long and need more registers than there are
// (nine prompts 337 us, so 393).
constexpr float kFar = 18446744073709551616.0f;  // 2^64

template <int D, int WAVES>
__global__ __launch_bounds__(64 * WAVES, D <= 128 ? 2 : 1) void k_attn_prompt(PromptArgs a) {
  constexpr int KS = D / 16, NJ = D / 32, BM = 32 * WAVES, TILE = kBN * D * 2;
  __shared__ __align__(16) uint8_t k_even[TILE], k_odd[TILE], v_even[TILE], v_odd[TILE];
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int lane = lane_id(), n = lane & 31, h = lane >> 5;

  // Workgroups go to the 8 dies in turn: each die takes its own heads, so that a
  // key/value head's tiles are shared in one die's cache.  Row tiles of all
  // sequences, the last ones (the most keys) first.
  int head, slot;
  if (a.n_q % 8 == 0) {
    const int per = a.n_q / 8, id = (int)(blockIdx.x >> 3);
    head = (int)(blockIdx.x & 7) * per + id % per;
    slot = id / per;
  } else {
    head = (int)(blockIdx.x % a.n_q);
    slot = (int)(blockIdx.x / a.n_q);
  }
  // Row tiles of sequence i, over the 64 lanes; up to 64 sequences are found
  // with one round of loads.
  int q0 = 0, q1 = 0, s0 = 0, s1 = 0, sum = 0, first = 0, before = 0, total = 0;
  const auto round = [&](int i0) {  // sum: tiles of sequences i0 .. i0 + lane
    const int i = min(i0 + lane, a.n_seq - 1);
    q0 = a.q_start[i]; q1 = a.q_start[i + 1];
    s0 = a.kv_start[i]; s1 = a.kv_start[i + 1];
    loaded(q0, q1, s0, s1);
    // (rows before 0 and from T on are left out; a row's position counts from the
    // sequence's end)
    q0 = max(q0, 0);
    const int64_t n = min((int64_t)q1, a.T) - q0;
    sum = wave_incl_scan(i0 + lane < a.n_seq && n > 0 ? (int)((n + BM - 1) / BM) : 0);
  };
  for (int i0 = 0; i0 < a.n_seq; i0 += 64) {
    round(i0);
    total += __builtin_amdgcn_readlane(sum, 63);
  }
  const int want = total - 1 - slot;
  if (want < 0) return;
  if (a.n_seq > 64) {
    for (; first < a.n_seq; first += 64) {
      round(first);
      const int all = __builtin_amdgcn_readlane(sum, 63);
      if (before + all > want) break;
      before += all;
    }
    if (first >= a.n_seq) return;  // (no sequence has it: starts that do not ascend)
  }
  const int at = __ffsll((unsigned long long)__ballot(before + sum > want)) - 1;
  const int64_t r0 = __builtin_amdgcn_readlane(q0, at), rows = __builtin_amdgcn_readlane(q1, at) - r0;
  const int64_t k0 = __builtin_amdgcn_readlane(s0, at), len = __builtin_amdgcn_readlane(s1, at) - k0;
  if (at > 0) before += __builtin_amdgcn_readlane(sum, at - 1);
  const int64_t tile = want - before;

  const int64_t i_wg = tile * BM;
  const bool keys = k0 >= 0 && k0 + len <= a.Tk;  // else nothing is read and the rows are NaN
  const int64_t hi = keys ? len - rows + min(i_wg + BM, rows) - 1 : -1;  // last key of the tile's rows
  const int64_t lo = len - rows + i_wg;                                  // key that all of them see
  // last key that some row of the wave sees
  const int64_t hi_wave = min(hi, len - rows + i_wg + (wave + 1) * 32 - 1);
  const int n_tiles = hi < 0 ? 0 : (int)(hi / kBN) + 1;
  const int n_full = lo < kBN - 1 ? 0 : (int)min((lo + 1) / kBN, (int64_t)n_tiles);

  Rows<D> w;
  const int64_t i_row = i_wg + wave * 32 + n, last_row = min(rows, a.T - r0) - 1;
  const bool live = i_row <= last_row;
  w.limit = live && keys ? len - rows + i_row : -1;
  // (a lane without a row takes the tile's last one: another tile's may be
  // overwritten meanwhile, where the output takes the queries' place)
  const uint16_t* qp = a.q + (r0 + min(i_row, last_row)) * a.q_stride + (int64_t)head * D + 8 * h;
#pragma unroll
  for (int s = 0; s < KS; ++s) w.qf[s] = *reinterpret_cast<const v4u*>(qp + 16 * s);
  w.places(lane);
  w.clear();
  const Tiles<D, WAVES> K(a.k + k0 * a.k_stride + (int64_t)(head / a.G) * D, a.k_stride, len, wave, lane);
  const Tiles<D, WAVES> V(a.v + k0 * a.v_stride + (int64_t)(head / a.G) * D, a.v_stride, len, wave, lane);

  if (n_tiles > 0) {
    constexpr int N = Tiles<D, WAVES>::LOADS;
    K.load(k_even, 0, wave);
    V.load(v_even, 0, wave);
    if (n_tiles > 1) {
      K.load(k_odd, 1, wave);
      wait_loads<2 * N>();
    } else {
      wait_loads<N>();
    }
    __syncthreads();
    v16f x[2];
    w.scores(k_even, x);
    if (n_full == 0) w.mask(x, 0);
    w.m = fmaxf(w.top(x, a.c), kNone);

    // x holds tile it's scores; K of it + 1 (in k1) and V of it (in v0) are on
    // their way, K of it + 2 goes to k0, V of it + 1 to v1.  The buffers are
    // variables of their own and named statically, so that no read waits for
    // a load into another one.
    const auto arrive = [&](int it, uint8_t* k0, uint8_t* v1) {
      wait_loads<0>();  // this wave's parts of the tiles
      __syncthreads();
      if (it + 2 < n_tiles) K.load(k0, it + 2, wave);
      if (it + 1 < n_tiles) V.load(v1, it + 1, wave);
    };
    const auto step = [&](int it, uint8_t* k0, uint8_t* k1, uint8_t* v0, uint8_t* v1) {
      arrive(it, k0, v1);
      v16f y[2];
      w.template step<true>(k1, v0, a.c, x, y);
      x[0] = y[0];
      x[1] = y[1];
    };
    // Tiles that not every row sees: a wave leaves out those none of its rows
    // does, and the scores of the one after its last.
    const int last = __builtin_amdgcn_readfirstlane(hi_wave < 0 ? -1 : (int)(hi_wave / kBN));
    const auto edge_step = [&](int it, uint8_t* k0, uint8_t* k1, uint8_t* v0, uint8_t* v1) {
      arrive(it, k0, v1);
      if (it > last) return;
      v16f y[2];
      if (it < last) {
        w.scores(k1, y);
        w.mask(y, (int64_t)(it + 1) * kBN);
      }
      w.template step<false>(k1, v0, a.c, x, y);
      x[0] = y[0];
      x[1] = y[1];
    };
    int it = 0;
#pragma unroll 1
    for (; it + 2 < n_full; it += 2) {
      step(it, k_even, k_odd, v_even, v_odd);
      step(it + 1, k_odd, k_even, v_odd, v_even);
    }
#pragma unroll 1
    for (; it < n_tiles; it += 2) {
      edge_step(it, k_even, k_odd, v_even, v_odd);
      if (it + 1 < n_tiles) edge_step(it + 1, k_odd, k_even, v_odd, v_even);
    }
  }
  w.finish();
  float bad = w.l <= kFar ? 0.0f : 1.0f;
#pragma unroll
  for (int j = 0; j < NJ; ++j)
#pragma unroll
    for (int i = 0; i < 16; ++i) bad = fmaf(w.o[j][i], 0.0f, bad);  // NaN if one is not finite
  if (__syncthreads_or(live && bad != 0.0f)) {
    careful_pass<D, WAVES>(w, k_even, v_even, K, V, a.c, n_tiles, lo + wave * 32, wave, lane);
    w.finish();
  }
  if (!live) return;
  const float inv = !keys ? __uint_as_float(0x7fc00000u) : w.limit < 0 ? 0.0f : 1.0f / w.l;
  // A lane holds 4 of every 8 elements, its partner in the other half of the wave
  // the other 4: one swap of two pieces gives each 8 in a row, for one store.
  uint16_t* d = a.out + (r0 + i_row) * a.out_stride + (int64_t)head * D + 8 * h;
#pragma unroll
  for (int j = 0; j < NJ; ++j)
#pragma unroll
    for (int i = 0; i < 16; i += 8) {
      const v16f& o = w.o[j];
      const auto lo = __builtin_amdgcn_permlane32_swap(bf16_pair(o[i] * inv, o[i + 1] * inv),
                                                       bf16_pair(o[i + 4] * inv, o[i + 5] * inv), false, false);
      const auto hi = __builtin_amdgcn_permlane32_swap(bf16_pair(o[i + 2] * inv, o[i + 3] * inv),
                                                       bf16_pair(o[i + 6] * inv, o[i + 7] * inv), false, false);
      *reinterpret_cast<uint4*>(d + 32 * j + 2 * i) = make_uint4(lo[0], hi[0], lo[1], hi[1]);
    }
}

template <int D, int WAVES>
hipError_t launch(const PromptArgs& a, hipStream_t stream) {
  const int64_t tiles = a.T / (32 * WAVES) + a.n_seq;  // at most: one part tile a sequence
  k_attn_prompt<D, WAVES><<<(unsigned)(tiles * a.n_q), 64 * WAVES, 0, stream>>>(a);
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
  // 128 rows a workgroup, two workgroups a CU: the best or within 4 % of it up to
  // 2048 rows (one MI355X, 32 heads of 128: 333 rows 12.3 us, 64 rows a workgroup
  // 11.7, 256 rows 15; 2048 rows 50, 54 and 59).  For long sequences 256 rows, which
  // read every key half as often: 4096 rows 136 us against 150, 8192 rows behind
  // 8192 keys 1360 against 1435.
  switch (D) {
    case 64: return launch<64, 4>(a, stream);
    case 128: return T / n_seq >= 4096 ? launch<128, 8>(a, stream) : launch<128, 4>(a, stream);
    default: return launch<256, 4>(a, stream);
  }
}

}  // namespace moe
