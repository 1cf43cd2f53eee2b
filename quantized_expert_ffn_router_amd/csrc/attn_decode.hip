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
//
// Measured on one MI355X, both launches, 32 query and 4 key/value heads of 128, inputs
// that no cache holds: 8 slots of 16 K tokens in bf16 49 us (5.5 TB/s, above a large
// copy's 5.15), in Q8_0 31 us (4.6 TB/s), in NVFP4 24 (3.2) and one slot of 262144
// tokens 33 us (4.6 TB/s); there decoding keeps the vector units busy beside the
// loads.  Heads of 64 and of 256, those 8 slots: 28, 19, 17 and 94, 59, 40 us.
#include <type_traits>

#include <algorithm>

#include "attn_common.h"

namespace moe {

namespace {

typedef _Float16 v2h __attribute__((ext_vector_type(2)));
typedef _Float16 v8h __attribute__((ext_vector_type(8)));
typedef __bf16 v8b __attribute__((ext_vector_type(8)));
typedef short v4s __attribute__((ext_vector_type(4)));
typedef uint32_t v2u __attribute__((ext_vector_type(2)));
typedef float v4f __attribute__((ext_vector_type(4)));
typedef uint32_t v4u __attribute__((ext_vector_type(4)));

constexpr int kWaves = 4;
constexpr int kStreamed = 2;         // cache policy of loads that are read once
constexpr float kNone = -3.0e38f;   // running maximum before any token
constexpr float kGrow = 8.0f;       // log2 headroom before the accumulators are rescaled

// Weights are relative to the running maximum less this (log2).  With fp16 weights
// (to 65504) the largest is 2^7 to 2^15, so that one vanishes only below 2^-32 of
// the largest, not 2^-25: 380 tokens of weight 2^-26 behind one of weight 1 and
// value 0 lose a quarter of their sum without, those that share its wave.  bf16
// weights have fp32's exponents.
template <int FMT>
constexpr float kRaise = FMT == MOE_FMT_BF16 ? 0.0f : 7.0f;

struct DecodeArgs {
  const uint8_t* pool;
  const uint16_t* q;
  uint16_t* out;
  float* part_o;   // [T * n_q][S][D]
  float2* part_ml; // [T * n_q][S]
  int* part_n;     // [T * n_q]: splits (1: the output is there already)
  int64_t q_stride, out_stride, T;
  SeqView s;
  int n_q, n_kv, G, S, room, likely;
  float scale_log2, v_ts;
};

// How a step's work is cut: into items of one tile of `size` query rows and
// `chunk` 32-token units of a sequence, the same chunk for all, so that
// workgroups are even however different the sequences' lengths are.  Every wave
// works it out from the lengths.
struct Item {
  int b, r0, rows, len;  // sequence (-1: there are not so many items), its first row, rows, length
  int inside;            // rows inside 0..T
  int tile, kvh, sp, splits, chunk;
};

// Units to go over at most: those of the page table and one more, which stands for
// all tokens past its end (none is there: rows that see it are NaN).
__device__ __forceinline__ int units_of_table(const SeqView& s) {
  return (int)min(((int64_t)s.max_pages << s.log2P) / 32 + 1, (int64_t)1 << 27);
}

// This lane's sequence: its rows from row 0 on (row t is token len - end + t
// wherever its first row lies).
struct LaneSeq {
  int start, end, len;
  int tiles, units;
  __device__ __forceinline__ LaneSeq(const SeqView& s, int i0, int64_t T, int G, int size) {
    const int i = min(i0 + lane_id(), s.n_seq - 1);
    start = max(s.row_start[i], 0);
    end = s.row_start[i + 1];
    len = s.kv_len[i];
    const int64_t n = i0 + lane_id() < s.n_seq ? min((int64_t)end, T) - start : 0;
    tiles = n > 0 ? (int)((uint32_t)((int)n * G + size - 1) / (uint32_t)size) : 0;
    units = n > 0 && len > 0 ? min((len - 1) / 32 + 1, units_of_table(s)) : 0;
  }
};

// The item of workgroup id.  S 1: sequences are not split.  chunk: a multiple of the
// waves, as small as keeps the items within `room` more than the tiles (what the grid
// holds), and kWhole units or more unless the 256 CUs need shorter ones (8 slots of
// 1000 to 60000 tokens: 33 us; as many chunks of each sequence as of any other, 37).
constexpr int kWhole = 4 * kWaves;
__device__ __forceinline__ Item find_item(const SeqView& s, int64_t T, int G, int size, int n_kv,
                                          int room, int S, int id) {
  Item r;
  r.b = -1;
  r.chunk = INT32_MAX;
  const LaneSeq first(s, 0, T, G, size);
  if (S > 1) {
    float work = 0.0f;
    int most = 0;
    for (int i0 = 0; i0 < s.n_seq; i0 += 64) {
      const LaneSeq q = i0 ? LaneSeq(s, i0, T, G, size) : first;
      work += (float)q.tiles * (float)q.units;
      most = max(most, q.units);
    }
    work = wave_sum(work);
    most = wave_max(most);
    // (a sequence has less than 2^27 units: held to 2^30, it stays an int)
    int chunk = (int)fminf(ceilf(work / (float)room), 0x1p30f);
    if (chunk < kWhole) chunk = max(chunk, min((int)ceilf(work * n_kv / 256.0f), kWhole));
    chunk = (max(chunk, (most + S - 1) / S) + kWaves - 1) / kWaves * kWaves;
    r.chunk = max(__builtin_amdgcn_readfirstlane(chunk), kWaves);
  }
  int before = 0;
  for (int i0 = 0; i0 < s.n_seq; i0 += 64) {
    const LaneSeq q = i0 ? LaneSeq(s, i0, T, G, size) : first;
    // (a row without tokens is answered too)
    const int splits = S > 1 && q.units ? (int)((uint32_t)(q.units - 1) / (uint32_t)r.chunk) + 1 : 1;
    const int sum = wave_incl_scan(q.tiles * splits * n_kv);
    const uint64_t past = __ballot(i0 + lane_id() < s.n_seq && before + sum > id);
    if (!past) {
      before += __builtin_amdgcn_readlane(sum, 63);
      continue;
    }
    const int l = __ffsll((unsigned long long)past) - 1;
    if (l > 0) before += __builtin_amdgcn_readlane(sum, l - 1);
    r.b = i0 + l;
    r.r0 = __builtin_amdgcn_readlane(q.start, l);
    const int64_t rows = (int64_t)__builtin_amdgcn_readlane(q.end, l) - r.r0;
    r.rows = (int)min(rows, (int64_t)INT32_MAX);
    r.len = __builtin_amdgcn_readlane(q.len, l);
    r.inside = (int)min(rows, T - r.r0);
    r.splits = __builtin_amdgcn_readlane(splits, l);
    const int at = (int)((uint32_t)(id - before) / (uint32_t)r.splits);
    r.sp = id - before - at * r.splits;
    r.tile = (int)((uint32_t)at / (uint32_t)n_kv);
    r.kvh = at - r.tile * n_kv;
    break;
  }
  return r;
}

// What one tile of `size` query rows (row r = i * G + g: packed row i, head g of
// the group) of a sequence sees.
struct TilePlan {
  int64_t hi;  // last token that any row of the tile sees (-1: none)
  int64_t lo;  // last token that all of them see
  int units;   // 32-token units up to hi, but units_of_table
};
__device__ __forceinline__ TilePlan tile_plan(const SeqView& s, const Item& it, int G, int size) {
  TilePlan p;
  const int last = min((int)((uint32_t)(it.tile * size + size - 1) / (uint32_t)G), it.inside - 1);
  p.hi = max((int64_t)it.len - it.rows + last, (int64_t)-1);
  p.lo = (int64_t)it.len - it.rows + (int)((uint32_t)(it.tile * size) / (uint32_t)G);
  p.units = min((int)((p.hi + 32) >> 5), units_of_table(s));
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

// The cache bytes of one lane for a unit of 32 tokens (two tiles of 16): of one
// token's key per tile, D/4 elements, and of four tokens' values, D/16 elements
// each.  A lane's bytes come in chunks of one load (16 bytes; 8 for 64 elements
// of 4 bits), spread so that a load of the wave covers whole pieces of 64 bytes
// and more: chunk i of group g of a key starts at byte 64 i + 16 g of its row,
// chunk i of lane n of a value quad at byte 256 i + 16 n.  Which elements those
// are does not matter to the products, as long as the query row is cut the same
// way and the output is put back.
template <int FMT, int D>
struct Unit {
  static constexpr int W = FMT == MOE_FMT_NVFP4 ? D / 32 : FMT == MOE_FMT_Q8_0 ? D / 16 : D / 8;
  static constexpr int CW = W < 4 ? W : 4;   // words of a chunk
  static constexpr int NC = W / CW;          // chunks of a lane and tile
  static constexpr int EK = D / 4 / NC;      // key elements of a chunk
  // value elements of a chunk (NVFP4: all of a lane's, for one or two tokens)
  static constexpr int JC = FMT == MOE_FMT_NVFP4 ? D / 16 : D / 16 / NC;
  static constexpr int NS = FMT == MOE_FMT_BF16 ? 1 : FMT == MOE_FMT_Q8_0 ? NC : 1;
  uint32_t k[2][W], v[2][W];
  uint16_t ks[2][NC];      // scales of a key chunk: one or two E4M3 bytes, or an fp16
  uint32_t vs[2][NS][2];   // of the 4 tokens: E4M3 bytes in [0], or 4 fp16 for each chunk

  // First key element of step s (8 elements) of group g.
  __device__ __forceinline__ static int key_dim(int s, int g) {
    return (s * 8 / EK) * (4 * EK) + g * EK + s * 8 % EK;
  }
  // Element of value fragment j in row m of its product.
  __device__ __forceinline__ static int value_dim(int m, int j) {
    return (j / JC) * (16 * JC) + m * JC + j % JC;
  }

  // Byte offsets of a lane inside the sections of a 16-token tile.
  struct Lane {
    uint32_t k, v, ks, vs;
    __device__ __forceinline__ Lane(int n, int g, int P) {
      k = n * (16 * W) + g * (4 * CW);
      v = FMT == MOE_FMT_NVFP4 ? (g * 16 + n) * (4 * W) : g * (64 * W) + n * 16;
      ks = FMT == MOE_FMT_NVFP4 ? n * (D / 16) + g * (EK / 16) : 2 * (n * (D / 32) + g / 2);
      vs = FMT == MOE_FMT_NVFP4 ? (n * D / 256) * P + 4 * g : 2 * (n / 8 * P + 4 * g);
    }
  };

  // blk: the (page, head) block; o: the unit's first token within the page.
  // Both are the same for the whole wave: a descriptor of the block and scalar
  // offsets of the sections, so that a lane's own offsets never change.  Keys and
  // values take 16 W bytes a token; they are not kept in the caches (read once).
  // bytes: readable bytes of the block; with 0 the loads come back at once, as
  // zeros.
  template <typename R>
  __device__ __forceinline__ static void words(R rsrc, uint32_t* d, uint32_t lane, uint32_t base) {
#if defined(__HIP_DEVICE_COMPILE__)  // (the host pass does not know the builtins)
    if constexpr (CW == 2) {
      const auto x = __builtin_amdgcn_raw_buffer_load_b64(rsrc, lane, base, kStreamed);
      d[0] = x[0]; d[1] = x[1];
    } else {
      const auto x = __builtin_amdgcn_raw_buffer_load_b128(rsrc, lane, base, kStreamed);
      d[0] = x[0]; d[1] = x[1]; d[2] = x[2]; d[3] = x[3];
    }
#endif
  }
  __device__ __forceinline__ void load_keys(const uint8_t* blk, const KvLayout lay, int bytes, int o, const Lane& at) {
#if defined(__HIP_DEVICE_COMPILE__)
    const auto rsrc = __builtin_amdgcn_make_buffer_rsrc(const_cast<uint8_t*>(blk), 0, bytes, 0x00020000);
#pragma unroll
    for (int t = 0; t < 2; ++t) {
      const uint32_t tok = o + 16 * t;
#pragma unroll
      for (int i = 0; i < NC; ++i) {
        words(rsrc, k[t] + i * CW, at.k + 64 * i, tok * (16 * W));
        if constexpr (FMT == MOE_FMT_NVFP4) {
          const uint32_t s = lay.ks + tok * (D / 16);
          if constexpr (EK == 16) ks[t][i] = (uint8_t)__builtin_amdgcn_raw_buffer_load_b8(rsrc, at.ks + 8 * i, s, 0);
          else ks[t][i] = (uint16_t)__builtin_amdgcn_raw_buffer_load_b16(rsrc, at.ks + 8 * i, s, 0);
        } else if constexpr (FMT == MOE_FMT_Q8_0) {
          ks[t][i] = (uint16_t)__builtin_amdgcn_raw_buffer_load_b16(rsrc, at.ks + 4 * i, lay.ks + 2 * tok * (D / 32), 0);
        }
      }
    }
#endif
  }
  __device__ __forceinline__ void load_values(const uint8_t* blk, const KvLayout lay, int bytes, int P, int o, const Lane& at) {
#if defined(__HIP_DEVICE_COMPILE__)
    const auto rsrc = __builtin_amdgcn_make_buffer_rsrc(const_cast<uint8_t*>(blk), 0, bytes, 0x00020000);
#pragma unroll
    for (int t = 0; t < 2; ++t) {
      const uint32_t tok = o + 16 * t;
#pragma unroll
      for (int i = 0; i < NC; ++i)
        words(rsrc, v[t] + i * CW, at.v + (FMT == MOE_FMT_NVFP4 ? 16 : 256) * i, lay.vq + tok * (16 * W));
      if constexpr (FMT == MOE_FMT_NVFP4) {
        vs[t][0][0] = __builtin_amdgcn_raw_buffer_load_b32(rsrc, at.vs, lay.vs + tok, 0);
      } else if constexpr (FMT == MOE_FMT_Q8_0) {
#pragma unroll
        for (int i = 0; i < NC; ++i) {
          const auto x = __builtin_amdgcn_raw_buffer_load_b64(rsrc, at.vs, lay.vs + 2 * (tok + 2 * i * P), 0);
          vs[t][i][0] = x[0]; vs[t][i][1] = x[1];
        }
      }
    }
#endif
  }

  // A key scale as a word.  Widened where it is used: beside its load, where the
  // compiler would put that, it would wait for a prefetch in the midst of a unit
  // (8 slots at 8 K tokens 17.2 us, with that 17.9).
  __device__ __forceinline__ uint32_t key_scale(int t, int i) const {
    uint16_t b = ks[t][i];
#if defined(__HIP_DEVICE_COMPILE__)
    asm("" : "+v"(b));
#endif
    return b;
  }

  // Key fragment s (8 elements of the lane's) of tile t, as 4 words.
  __device__ __forceinline__ v4u key(int t, int s) const {
    v4u r;
    const int i = s * 8 / EK;
    if constexpr (FMT == MOE_FMT_NVFP4) {
      const v2h sp = fp8_pair(key_scale(t, i), 0);
      const v2h sc = (s * 8 % EK) / 16 ? v2h{sp.y, sp.y} : v2h{sp.x, sp.x};
#pragma unroll
      for (int q = 0; q < 4; ++q) r[q] = bits(fp4_pair(k[t][s], q) * sc);
    } else if constexpr (FMT == MOE_FMT_Q8_0) {
      const v2h sp = halves(key_scale(t, i));
      const v2h sc = {sp.x, sp.x};
#pragma unroll
      for (int q = 0; q < 4; ++q) r[q] = bits(i8_pair(k[t][2 * s + (q >> 1)] ^ 0x80808080u, q & 1) * sc);
    } else {
#pragma unroll
      for (int q = 0; q < 4; ++q) r[q] = k[t][4 * s + q];
    }
    return r;
  }

  // Value fragment j of the block formats: tokens 4g.. of tile 0, then of tile 1
  // (the order of the score accumulators).
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
          r[2 * t + h] = bits(fp4_pair(w, (j & 7) >> 1) * fp8_pair(vs[t][0][0], h));
        } else if constexpr (FMT == MOE_FMT_Q8_0) {
          r[2 * t + h] = bits(i8_pair(v[t][j] ^ 0x80808080u, h) * halves(vs[t][j / JC][h]));
        }
      }
    }
    return r;
  }

  // Zeroes the values of this lane's tokens from the `left`-th of the unit on,
  // whatever they hold.
  __device__ __forceinline__ void cut(int left, int g) {
#pragma unroll
    for (int t = 0; t < 2; ++t) {
      const int n = min(max(left - 16 * t - 4 * g, 0), 4);
      const uint32_t m0 = n >= 2 ? ~0u : n == 1 ? 0xffffu : 0u;
      const uint32_t m1 = n >= 4 ? ~0u : n == 3 ? 0xffffu : 0u;
      if constexpr (FMT == MOE_FMT_NVFP4) {
        vs[t][0][0] = n >= 4 ? vs[t][0][0] : vs[t][0][0] & ((1u << (8 * n)) - 1u);
      } else if constexpr (FMT == MOE_FMT_Q8_0) {
#pragma unroll
        for (int i = 0; i < NC; ++i) { vs[t][i][0] &= m0; vs[t][i][1] &= m1; }
      } else {
#pragma unroll
        for (int j = 0; j < D / 16; ++j) { v[t][2 * j] &= m0; v[t][2 * j + 1] &= m1; }
      }
    }
  }

  // Keeps what is decoded from the value bytes from being computed ahead of a
  // rare loop, where it would take registers all along.
  __device__ __forceinline__ void pin() {
#if defined(__HIP_DEVICE_COMPILE__)
#pragma unroll
    for (int t = 0; t < 2; ++t)
#pragma unroll
      for (int i = 0; i < W; ++i) asm("" : "+v"(v[t][i]));
#endif
  }

  // Whether any of this lane's values is infinite or NaN (in the block
  // formats a NaN scale says so; an infinite fp16 scale counts too).
  __device__ __forceinline__ bool wild() const {
    bool any = false;
#pragma unroll
    for (int t = 0; t < 2; ++t) {
      if constexpr (FMT == MOE_FMT_NVFP4) {
#pragma unroll
        for (int i = 0; i < 4; ++i) any |= ((vs[t][0][0] >> (8 * i)) & 0x7fu) == 0x7fu;
      } else if constexpr (FMT == MOE_FMT_Q8_0) {
#pragma unroll
        for (int c = 0; c < NC; ++c)
#pragma unroll
          for (int i = 0; i < 2; ++i)
            any |= (vs[t][c][i] & 0x7c00u) == 0x7c00u || (vs[t][c][i] & 0x7c000000u) == 0x7c000000u;
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

// o + value fragment j times the weights p.  16-bit values come as the operands of
// two products of one tile of 16 tokens each, as they were loaded: put together
// for one product of both, they were copied where they arrive, which waits for
// every prefetch (8 slots of 16 K tokens 50 us, with that 74).
template <int FMT, int D>
__device__ __forceinline__ v4f weighted(const Unit<FMT, D>& c, int j, v4u p, v4f o) {
  if constexpr (FMT == MOE_FMT_BF16) {
#pragma unroll
    for (int t = 0; t < 2; ++t)
      o = __builtin_amdgcn_mfma_f32_16x16x16bf16_1k(
          __builtin_bit_cast(v4s, v2u{c.v[t][2 * j], c.v[t][2 * j + 1]}),
          __builtin_bit_cast(v4s, v2u{p[2 * t], p[2 * t + 1]}), o, 0, 0, 0);
    return o;
  } else {
    return mma<FMT>(c.value(j), p, o);
  }
}

// Two softmax weights as a pair of the product's operand type, rounded to
// nearest even (half a step, 2^-11 or 2^-8: the types that meet the matrix units),
// and their sum added to l: of the rounded weights, so that rounding does not shift
// the mean.
template <int FMT>
__device__ __forceinline__ uint32_t weight_pair(float a, float b, float* l) {
  if constexpr (FMT == MOE_FMT_BF16) {
    typedef __bf16 v2b __attribute__((ext_vector_type(2)));
    const v2b r = {(__bf16)a, (__bf16)b}, one = {(__bf16)1.0f, (__bf16)1.0f};
    *l = __builtin_amdgcn_fdot2_f32_bf16(r, one, *l, false);
    return __builtin_bit_cast(uint32_t, r);
  } else {
    const v2h r = {(_Float16)a, (_Float16)b}, one = {(_Float16)1.0f, (_Float16)1.0f};
    *l = __builtin_amdgcn_fdot2(r, one, *l, false);
    return bits(r);
  }
}

// What a wave carries for one tile of NT * 16 query rows (a lane column is one
// row of each 16): running maximum (less kRaise), sum, and the weighted values.
template <int FMT, int D, int NT>
struct Carry {
  static constexpr int KS = D / 32, NJ = D / 16;
  v4u qf[NT][KS];
  v4f o[NT][NJ];
  float m[NT], l[NT], qs[NT];
  int64_t limit[NT];  // last token the lane's row sees

  __device__ __forceinline__ void scores(const Unit<FMT, D>& c, v4f (&x)[NT][2]) const {
#pragma unroll
    for (int t = 0; t < 2; ++t) {
#pragma unroll
      for (int s = 0; s < KS; ++s) {
        const v4u k = c.key(t, s);
#pragma unroll
        for (int r = 0; r < NT; ++r)
          x[r][t] = mma<FMT>(k, qf[r][s], s ? x[r][t] : v4f{0.f, 0.f, 0.f, 0.f});
        __builtin_amdgcn_sched_barrier(0);  // one fragment decoded at a time
      }
    }
  }
  __device__ __forceinline__ void weights(v4f (&x)[NT][2], v4u (&p)[NT]) {
#pragma unroll
    for (int r = 0; r < NT; ++r) {
      float mx = fmaxf(fmaxf(x[r][0][0], x[r][0][1]), fmaxf(x[r][0][2], x[r][0][3]));
      mx = fmaxf(mx, fmaxf(fmaxf(x[r][1][0], x[r][1][1]), fmaxf(x[r][1][2], x[r][1][3])));
      mx = groups_max(mx) * qs[r];
      if (__any(mx > m[r] + (kRaise<FMT> + kGrow))) {
        const float mn = fmaxf(m[r], mx - kRaise<FMT>), al = __builtin_amdgcn_exp2f(m[r] - mn);
#pragma unroll
        for (int j = 0; j < NJ; ++j)
#pragma unroll
          for (int i = 0; i < 4; ++i) o[r][j][i] *= al;
        l[r] *= al;
        m[r] = mn;
      }
#pragma unroll
      for (int t = 0; t < 2; ++t) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          x[r][t][i] = __builtin_amdgcn_exp2f(fmaf(x[r][t][i], qs[r], -m[r]));
        }
        p[r][2 * t] = weight_pair<FMT>(x[r][t][0], x[r][t][1], &l[r]);
        p[r][2 * t + 1] = weight_pair<FMT>(x[r][t][2], x[r][t][3], &l[r]);
      }
    }
  }
  __device__ __forceinline__ void gather(const Unit<FMT, D>& c, const v4u (&p)[NT]) {
#pragma unroll
    for (int j = 0; j < NJ; ++j) {
#pragma unroll
      for (int r = 0; r < NT; ++r) o[r][j] = weighted(c, j, p[r], o[r][j]);
      __builtin_amdgcn_sched_barrier(0);
    }
  }

  __device__ __forceinline__ void mask(v4f (&x)[NT][2], int64_t t0, int g) const {
#pragma unroll
    for (int r = 0; r < NT; ++r) {
      const int seen = (int)min(max(limit[r] - t0, (int64_t)-1), (int64_t)32) - 4 * g;
#pragma unroll
      for (int t = 0; t < 2; ++t)
#pragma unroll
        for (int i = 0; i < 4; ++i)
          if (16 * t + i > seen) x[r][t][i] = -__builtin_inff();
    }
  }

  // One unit of 32 tokens from t0 on.  edge: not every row sees all of it;
  // left: its tokens that some row sees.  The unit's bytes make room for the next
  // one's as they are used: next_keys and next_values start those loads.
  // Returns whether the values are left to wild_values.
  template <typename FK, typename FV>
  __device__ __forceinline__ bool unit(Unit<FMT, D>& c, bool edge, int64_t t0, int left, int g,
                                       FK next_keys, FV next_values) {
    v4f x[NT][2];
    v4u p[NT];
    bool wild = false;
    scores(c, x);
    next_keys();
    __builtin_amdgcn_sched_barrier(0);
    if (edge) mask(x, t0, g);
    weights(x, p);
    if (edge) {
      c.cut(left, g);
      wild = __any(c.wild());
      if (wild) c.cut(0, g);
    }
    gather(c, p);
    next_values();
    __builtin_amdgcn_sched_barrier(0);
    return wild;
  }

  // The weighted values of a unit with infinities or NaN among them that some row
  // may not see, for rows t, added to out (this lane's row of D sums in LDS).  A
  // zero weight would not silence them: the rows by what they see, each with the
  // values behind its last token cut off.
  __device__ __forceinline__ void wild_values(Unit<FMT, D>& c, int t, int64_t t0, int left, int g,
                                              float* out) const {
    v4f x[NT][2];
    v4u p;
    scores(c, x);
    mask(x, t0, g);
    c.cut(left, g);
    if (!__any(c.wild())) return;
    float none = 0.0f;
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
      for (int i = 0; i < 4; i += 2) {
        const float e0 = __builtin_amdgcn_exp2f(fmaf(x[t][h][i], qs[t], -m[t]));
        const float e1 = __builtin_amdgcn_exp2f(fmaf(x[t][h][i + 1], qs[t], -m[t]));
        p[2 * h + i / 2] = weight_pair<FMT>(e0, e1, &none);
      }
#pragma unroll 1
    for (int k = 0; k < 32; ++k) {
      const bool mine = min(limit[t] - t0, (int64_t)31) == k;
      if (!__any(mine)) continue;
      Unit<FMT, D> seen = c;
      seen.pin();
      seen.cut(k + 1, g);
#pragma unroll
      for (int j = 0; j < NJ; ++j) {
        const v4f add = weighted(seen, j, p, v4f{0.f, 0.f, 0.f, 0.f});
#pragma unroll
        for (int i = 0; i < 4; ++i)
          if (mine) out[Unit<FMT, D>::value_dim(4 * g + i, j)] += add[i];
        __builtin_amdgcn_sched_barrier(0);
      }
    }
  }
};

template <int N>
__device__ __forceinline__ void store_row(uint16_t* d, const float (&v)[N]) {
  uint32_t w[N / 2];
#pragma unroll
  for (int j = 0; j < N / 2; ++j) w[j] = bf16_pair(v[2 * j], v[2 * j + 1]);
  if constexpr (N == 4) *reinterpret_cast<uint2*>(d) = make_uint2(w[0], w[1]);
  if constexpr (N >= 8) *reinterpret_cast<uint4*>(d) = make_uint4(w[0], w[1], w[2], w[3]);
  if constexpr (N == 16) *reinterpret_cast<uint4*>(d + 8) = make_uint4(w[4], w[5], w[6], w[7]);
}

// Waves per SIMD that the register use allows: the accumulators (NT * D / 4), the
// query fragments (half of that) and a unit's bytes.
constexpr int kDecodeOcc(int fmt, int D, int NT) {
  const int regs = NT * D / 4 * 3 / 2 + D * (fmt == MOE_FMT_NVFP4 ? 4 : fmt == MOE_FMT_Q8_0 ? 8 : 16) / 32;
  return regs <= 64 ? 4 : regs <= 80 ? 3 : regs <= 160 ? 2 : 1;
}

// One workgroup: a tile of NT * 16 query rows of one key/value head, and one
// split of the sequence's units, which its waves take in turn, the next unit's
// bytes on their way while one is worked on.
template <int FMT, int D, int NT>
__global__ __launch_bounds__(64 * kWaves, kDecodeOcc(FMT, D, NT)) void k_attn_decode(DecodeArgs a) {
  constexpr int KS = D / 32, NJ = D / 16, LD = D + 4;
  constexpr int E = 16 * D / (64 * kWaves);  // elements of a thread in the join
  __shared__ __align__(16) float o_s[kWaves][16][LD];
  __shared__ float m_s[kWaves][16], l_s[kWaves][16];
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int lane = lane_id(), n = lane & 15, g = lane >> 4;
  const Item it = find_item(a.s, a.T, a.G, 16 * NT, a.n_kv, a.room, a.S, (int)blockIdx.x);
  if (it.b < 0) return;
  const int b = it.b, r0 = it.r0, rows = it.rows, len = it.len, inside = it.inside, tile = it.tile;
  const int kvh = it.kvh, sp = it.sp;
  const int P = 1 << a.s.log2P;
  const KvLayout lay = kv_layout(FMT, D, P);
  const size_t page_bytes = (size_t)a.n_kv * lay.head;
  const uint8_t* heads = a.pool + (size_t)kvh * lay.head;
  const typename Unit<FMT, D>::Lane at(n, g, P);
  const TilePlan plan = tile_plan(a.s, it, a.G, 16 * NT);
  const int u_begin = sp > 0 ? sp * it.chunk : 0;
  const int u_end = min((int64_t)plan.units, (int64_t)u_begin + it.chunk);
  if (sp > 0 && u_begin >= u_end) {  // (split 0 also answers rows that see nothing)
    const int rr = tile * (16 * NT) + threadIdx.x, i = (int)((uint32_t)rr / (uint32_t)a.G);
    if (threadIdx.x < 16 * NT && rr < inside * a.G)
      a.part_ml[((int64_t)(r0 + i) * a.n_q + kvh * a.G + rr - i * a.G) * a.S + sp] = make_float2(kNone, 0.0f);
    return;
  }

  Unit<FMT, D> c;
  // Entries of the page table, by scalar loads (a wave's units are its own); a
  // unit past the table's end has none.
  const int* const row = a.s.page_table + (int64_t)b * a.s.max_pages;
  const auto page_at = [&](int u) {
    const int i = (int)(((int64_t)u * 32) >> a.s.log2P);
    const int p = *(const int __attribute__((address_space(4)))*)(uintptr_t)(row + min(i, a.s.max_pages - 1));
    return i < a.s.max_pages ? p : -1;
  };
  const auto block = [&](int page) {  // page 0 stands in for one that is not there
    return heads + (size_t)((unsigned)page < (unsigned)a.s.n_pages ? page : 0) * page_bytes;
  };
  // this lane's query rows, their last visible tokens and their fragments; a lane
  // without a row takes the tile's last one (its answer goes nowhere, but it has a
  // say in when the maxima move: another tile's row may be overwritten meanwhile,
  // where the output takes the queries' place)
  Carry<FMT, D, NT> w;
  const int last = inside * a.G - 1;
#pragma unroll
  for (int t = 0; t < NT; ++t) {
    const int r = (tile * NT + t) * 16 + n, mine = min(r, last), i = (int)((uint32_t)mine / (uint32_t)a.G);
    w.limit[t] = r <= last ? (int64_t)len - rows + i : -1;
    const uint16_t* qp = a.q + (int64_t)(r0 + i) * a.q_stride + (size_t)(kvh * a.G + mine - i * a.G) * D;
    w.qs[t] = a.scale_log2;
#pragma unroll
    for (int s = 0; s < KS; ++s) w.qf[t][s] = *reinterpret_cast<const v4u*>(qp + Unit<FMT, D>::key_dim(s, g));
  }
  __builtin_amdgcn_sched_barrier(0);

  int u = u_begin + wave, page = 0, next = 0;
  if (u < u_end) {
    page = page_at(u);
    next = page_at(min(u + kWaves, u_end - 1));
    c.load_keys(block(page), lay, lay.head, (u * 32) & (P - 1), at);
    c.load_values(block(page), lay, lay.head, P, (u * 32) & (P - 1), at);
  }

#pragma unroll
  for (int t = 0; t < NT; ++t) {
    if constexpr (FMT != MOE_FMT_BF16) {
      // bf16 -> fp16, scaled by the power of two that puts the row's largest
      // magnitude into [2^14, 2^15): exact for values above 2^-29 of it
      uint32_t top = 0;
#pragma unroll
      for (int s = 0; s < KS; ++s)
#pragma unroll
        for (int i = 0; i < 4; ++i)
          top = max(top, max(w.qf[t][s][i] & 0x7fffu, (w.qf[t][s][i] >> 16) & 0x7fffu));
      top = max(top, (uint32_t)__shfl_xor((int)top, 16));
      top = max(top, (uint32_t)__shfl_xor((int)top, 32));
      const int e = min(max(141 - (int)(top >> 7), -113), 126);
      const float up = __uint_as_float((uint32_t)(127 + e) << 23);
      w.qs[t] *= __uint_as_float((uint32_t)(127 - e) << 23);
#pragma unroll
      for (int s = 0; s < KS; ++s)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const v2h p = {(_Float16)(__uint_as_float(w.qf[t][s][i] << 16) * up),
                         (_Float16)(__uint_as_float(w.qf[t][s][i] & 0xffff0000u) * up)};
          w.qf[t][s][i] = bits(p);
        }
    } else {
#if defined(__HIP_DEVICE_COMPILE__)
      // (waited for here, not in every unit)
#pragma unroll
      for (int s = 0; s < KS; ++s) asm("" : "+v"(w.qf[t][s]));
#endif
    }
#pragma unroll
    for (int j = 0; j < NJ; ++j) w.o[t][j] = v4f{0.f, 0.f, 0.f, 0.f};
    w.m[t] = kNone;
    w.l[t] = 0.0f;
  }

  // The loads of the next unit are not conditional (after a wave's last one they
  // read nothing): a load that may or may not be there would have to be waited
  // for with the others.
  bool wild = false;
#pragma unroll 1
  for (; u < u_end; u += kWaves) {
    const int64_t t0 = (int64_t)u * 32;
    const bool more = u + kWaves < u_end;
    const int o = ((u + kWaves) * 32) & (P - 1), bytes = more ? (int)lay.head : 0;
    const uint8_t* blk = block(next);
    if ((unsigned)page >= (unsigned)a.s.n_pages) {
      // nothing to read: rows that see a token of it have no answer
#pragma unroll
      for (int t = 0; t < NT; ++t)
        if (w.limit[t] >= t0) w.l[t] = __uint_as_float(0x7fc00000u);
    }
    page = next;
    next = page_at(min(u + 2 * kWaves, u_end - 1));
    wild |= w.unit(c, t0 + 31 > plan.lo, t0, (int)min(plan.hi + 1 - t0, (int64_t)32), g,
           [&] { c.load_keys(blk, lay, bytes, o, at); },
                   [&] { c.load_values(blk, lay, bytes, P, o, at); });
  }

  // join the waves' parts
#pragma unroll
  for (int t = 0; t < NT; ++t) {
    const float l = groups_sum(w.l[t]);
    __syncthreads();  // former parts have been read
    if (g == 0) { m_s[wave][n] = w.m[t]; l_s[wave][n] = l; }
    float* const part = o_s[wave][n];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      constexpr int JC = Unit<FMT, D>::JC;
#pragma unroll
      for (int j = 0; j < NJ; j += JC < 4 ? 2 : 4) {
        float* e = part + Unit<FMT, D>::value_dim(4 * g + i, j);
        if constexpr (JC < 4)
          *reinterpret_cast<float2*>(e) = make_float2(w.o[t][j][i], w.o[t][j + 1][i]);
        else
          *reinterpret_cast<float4*>(e) =
              make_float4(w.o[t][j][i], w.o[t][j + 1][i], w.o[t][j + 2][i], w.o[t][j + 3][i]);
      }
    }
    if (wild) {
      for (int v = u_begin + wave; v < u_end; v += kWaves) {
        const int64_t t0 = (int64_t)v * 32;
        const int pg = page_at(v);
        if (t0 + 31 <= plan.lo || (unsigned)pg >= (unsigned)a.s.n_pages) continue;
        c.load_keys(block(pg), lay, lay.head, (v * 32) & (P - 1), at);
        c.load_values(block(pg), lay, lay.head, P, (v * 32) & (P - 1), at);
        w.wild_values(c, t, t0, (int)min(plan.hi + 1 - t0, (int64_t)32), g, part);
      }
    }
    __syncthreads();
    const int qr = threadIdx.x / (D / E), d0 = (threadIdx.x % (D / E)) * E;
    float M = kNone, L = 0.0f, acc[E];
#pragma unroll
    for (int i = 0; i < kWaves; ++i) M = fmaxf(M, m_s[i][qr]);
#pragma unroll
    for (int j = 0; j < E; ++j) acc[j] = 0.0f;
#pragma unroll
    for (int i = 0; i < kWaves; ++i) {
      const float f = __builtin_amdgcn_exp2f(m_s[i][qr] - M);
      L += f * l_s[i][qr];
#pragma unroll
      for (int j = 0; j < E; ++j) acc[j] += f * o_s[i][qr][d0 + j];
    }
    const int rr = (tile * NT + t) * 16 + qr, i = (int)((uint32_t)rr / (uint32_t)a.G);
    const int64_t orow = r0 + i, h = kvh * a.G + rr - i * a.G;
    if (rr >= inside * a.G) continue;
    if (d0 == 0 && sp == 0 && a.S > 1) a.part_n[orow * a.n_q + h] = it.splits;
    if (it.splits == 1) {
      const float inv = (int64_t)len - rows + i < 0 ? 0.0f : 1.0f / L;
#pragma unroll
      for (int j = 0; j < E; ++j) acc[j] = acc[j] * inv * a.v_ts;
      store_row<E>(a.out + orow * a.out_stride + h * D + d0, acc);
    } else {
      const int64_t at = (orow * a.n_q + h) * a.S + sp;
      if (d0 == 0) a.part_ml[at] = make_float2(M, L);
      float* d = a.part_o + at * D + d0;
#pragma unroll
      for (int j = 0; j < E; j += 4)
        *reinterpret_cast<float4*>(d + j) = make_float4(acc[j], acc[j + 1], acc[j + 2], acc[j + 3]);
    }
  }
}

// Joins the splits of EL elements of one (row, head): weights exp2(m_s - M),
// added in a fixed order, so the result does not depend on scheduling.  EL / 4
// lanes hold the elements and 1024 / EL groups of them the splits, PER at a time
// each; the loads of as many as are likely start before their number is known.
constexpr int kMaxSplit = 256;

template <int D, int EL, int PER>
__global__ __launch_bounds__(256) void k_attn_join(DecodeArgs a) {
  constexpr int LW = EL / 4, NG = 256 / LW;
  __shared__ __align__(16) float4 acc_s[4][LW];
  __shared__ float l_s[4];
  const uint32_t id = blockIdx.x / (D / EL);
  const int x = (int)(blockIdx.x % (D / EL)) * LW + threadIdx.x % LW, grp = threadIdx.x / LW;
  const int t = (int)(id / (uint32_t)a.n_q), h = (int)(id % (uint32_t)a.n_q);
  const int lane = lane_id(), wave = threadIdx.x >> 6;
  const int64_t at = ((int64_t)t * a.n_q + h) * a.S;
  // (a row outside the sequences has no number there: whatever it reads is not used)
  int ns = a.part_n[(int64_t)t * a.n_q + h];
  float2 ml[PER];
  float4 v[PER];
  const auto load = [&](int i, int s) {
    ml[i] = a.part_ml[at + s];
    v[i] = *reinterpret_cast<const float4*>(a.part_o + (at + s) * D + 4 * x);
  };
#pragma unroll
  for (int i = 0; i < PER; ++i)
    if (grp + NG * i < a.likely) load(i, grp + NG * i);
  const RowSeq q = find_row(a.s, t, &ns);
  ns = __builtin_amdgcn_readfirstlane(min(ns, a.S));
  if (q.b < 0 || ns == 1) return;
  float M = kNone, L = 0.0f;
  float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
  for (int s0 = grp; s0 < ns; s0 += NG * PER) {
    float top = M;
#pragma unroll
    for (int i = 0; i < PER; ++i) {
      const int s = s0 + NG * i;
      if (s >= ns) ml[i] = make_float2(kNone, 0.0f);
      else if (s >= a.likely || s0 != grp) load(i, s);
      top = fmaxf(top, ml[i].x);
    }
    const float down = __builtin_amdgcn_exp2f(M - top);
    o.x *= down; o.y *= down; o.z *= down; o.w *= down;
    L *= down;
    M = top;
#pragma unroll
    for (int i = 0; i < PER; ++i) {
      if (ml[i].x == kNone && ml[i].y == 0.0f) continue;  // nothing there
      const float f = __builtin_amdgcn_exp2f(ml[i].x - M);
      o.x += f * v[i].x; o.y += f * v[i].y; o.z += f * v[i].z; o.w += f * v[i].w;
      L += f * ml[i].y;
    }
  }
  float all = M;
#pragma unroll
  for (int d = LW; d < 64; d <<= 1) all = fmaxf(all, __shfl_xor(all, d));
  if (lane == 0) l_s[wave] = all;
  __syncthreads();
#pragma unroll
  for (int i = 0; i < 4; ++i) all = fmaxf(all, l_s[i]);
  const float down = __builtin_amdgcn_exp2f(M - all);
  o.x *= down; o.y *= down; o.z *= down; o.w *= down;
  L *= down;
#pragma unroll
  for (int d = LW; d < 64; d <<= 1) {
    o.x += __shfl_xor(o.x, d); o.y += __shfl_xor(o.y, d);
    o.z += __shfl_xor(o.z, d); o.w += __shfl_xor(o.w, d);
    L += __shfl_xor(L, d);
  }
  __syncthreads();
  if (lane < LW) acc_s[wave][lane] = o;
  if (lane == 0) l_s[wave] = L;
  __syncthreads();
  if (threadIdx.x < LW) {
    o = acc_s[0][lane];
    L = l_s[0];
#pragma unroll
    for (int i = 1; i < 4; ++i) {
      const float4 w = acc_s[i][lane];
      o.x += w.x; o.y += w.y; o.z += w.z; o.w += w.w;
      L += l_s[i];
    }
    const float inv = (int64_t)q.len - q.rows + (t - q.r0) < 0 ? 0.0f : 1.0f / L, ts = a.v_ts;
    uint16_t* d = a.out + t * a.out_stride + (int64_t)h * D + 4 * x;
    *reinterpret_cast<uint2*>(d) = make_uint2(bf16_pair(o.x * inv * ts, o.y * inv * ts),
                                              bf16_pair(o.z * inv * ts, o.w * inv * ts));
  }
}

// Up to 32 likely splits a whole head in one workgroup (32 rows with 16 splits:
// 4.0 us, with 32 elements in each 9.4); more, 32 elements in each.
template <int D>
void launch_join(const DecodeArgs& a, hipStream_t stream) {
  const unsigned heads = (unsigned)(a.T * a.n_q);
  if (a.likely <= 32) k_attn_join<D, D, 32 * D / 1024><<<heads, 256, 0, stream>>>(a);
  else if (a.likely <= 64) k_attn_join<D, 32, 2><<<heads * (D / 32), 256, 0, stream>>>(a);
  else k_attn_join<D, 32, kMaxSplit / 32><<<heads * (D / 32), 256, 0, stream>>>(a);
}

// Launch shape: query rows of a tile, splits there is room for in the workspace
// (1: no split), and for each key/value head chunks and items (the grid).
struct Shape {
  int tile, S, room, likely;
  int64_t items;
};
// Measured on one MI355X with 32 query and 4 key/value heads of 128 (us, graph
// replay, NVFP4 unless said otherwise):
//   - 16 query rows to a tile, 32 when a sequence has more (the cache is read
//     once for them: 4 rows of 8 slots at 16 K tokens 29 against 34);
//   - up to 12 units (384 tokens) no split, so no joining launch: 300 tokens 7.2
//     against 8.8, but 700 tokens 9.2 against 8.8; up to 31 units where the
//     sequences alone are more than half of the workgroups aimed at (32 slots of
//     700 tokens 10.5 against 12.5; in bf16 65 slots of 2000 tokens 68 against 63
//     with a split), up to 255 where they are more than all (257 slots of 4000 and
//     of 8000 tokens 108 and 212 against 120 and 224, but 256 of 500 and one of 8000
//     66 against 36 with a split, one of 131072 807 against 85);
//   - chunks of at least 4 units for each wave (64 slots of 500 tokens 9.6, at
//     one unit 16.5; 8 slots at 8 K tokens 16.4 and 17.5), unless the CUs need
//     shorter ones (8 slots of 2000 tokens 10.8, for 192 workgroups 11.5);
//   - at most 4 workgroups a CU where the registers allow them (1000 to 60000
//     tokens 33, with 3 a CU 36, with 2 38; equal lengths do not tell them apart),
//     2 for the wider formats, which have enough bytes on their way with those
//     (Q8_0, 8 x 16 K: 32, with 3 35; bf16 49 and 53), and for 32 rows (29 and 31).
Shape shape_of(int fmt, int D, int n_kv, int n_q, int n_seq, int64_t T, int64_t max_len) {
  const int G = n_q / n_kv;
  const int64_t per_seq = (T + n_seq - 1) / n_seq;
  const int64_t units = (std::min(max_len, (int64_t)INT32_MAX) + 31) / 32;  // (lengths are 32-bit)
  Shape r;
  r.tile = per_seq * G > 16 && D <= 128 ? 32 : 16;
  const int64_t tiles = T * G / r.tile + n_seq;  // at most: one part tile a sequence
  const int64_t base = (int64_t)n_seq * n_kv * ((per_seq * G + r.tile - 1) / r.tile);
  const int target = 256 * (fmt == MOE_FMT_NVFP4 && r.tile == 16 && D <= 128 ? 4 : 2);
  r.likely = (int)std::min(std::max(units / kWhole, 192 / base), target / base);
  // a single sequence may take all chunks; 64 MB of partial sums, 8 chunks or none
  int64_t S = (64 << 20) / (T * n_q * D * 4);
  const bool fits = S >= 8 && T * n_q <= kSplitPairs;
  S = std::min({S, (int64_t)kMaxSplit, (units + kWaves - 1) / kWaves});
  const int whole = r.likely > 1 ? 3 * kWaves : base > target ? 255 : 31;
  r.S = !fits || units <= whole ? 1 : (int)S;
  const int64_t fine = std::max((int64_t)256 / n_kv, tiles * ((units + kWhole - 1) / kWhole));
  r.likely = std::min(r.likely, r.S);
  r.room = (int)std::max((int64_t)1, std::min({(int64_t)target / n_kv, fine, tiles * r.S}));
  r.items = tiles + (r.S > 1 ? r.room + 1 : 0);
  return r;
}

template <int FMT>
void launch_decode(const DecodeArgs& a, int D, int tile, unsigned grid, hipStream_t stream) {
  constexpr int N = 64 * kWaves;
  if (D == 64 && tile == 16) k_attn_decode<FMT, 64, 1><<<grid, N, 0, stream>>>(a);
  else if (D == 64) k_attn_decode<FMT, 64, 2><<<grid, N, 0, stream>>>(a);
  else if (D == 128 && tile == 16) k_attn_decode<FMT, 128, 1><<<grid, N, 0, stream>>>(a);
  else if (D == 128) k_attn_decode<FMT, 128, 2><<<grid, N, 0, stream>>>(a);
  else k_attn_decode<FMT, 256, 1><<<grid, N, 0, stream>>>(a);
}

}  // namespace

size_t attn_decode_ws_bytes(int fmt, int n_kv, int D, int n_q, int n_seq, int64_t T, int64_t max_len) {
  if (n_seq < 1 || T < 1) return 0;
  const Shape sp = shape_of(fmt, D, n_kv, n_q, n_seq, T, max_len);
  if (sp.S == 1) return 0;
  const size_t n = (size_t)T * n_q * sp.S;
  return align_up(n * D * sizeof(float)) + align_up(n * sizeof(float2)) +
         align_up((size_t)T * n_q * sizeof(int));
}

hipError_t launch_attn_decode(const moe_kv_cache* c, const moe_seq_batch* s, int n_q,
                              const uint16_t* q, int64_t q_stride, int64_t T, int64_t max_len,
                              float scale, uint16_t* out, int64_t out_stride, void* ws,
                              hipStream_t stream) {
  const Shape sp = shape_of(c->fmt, c->D, c->n_kv, n_q, s->n_seq, T, max_len);
  int l2 = 0;
  while ((1 << l2) < c->page_tokens) ++l2;
  const bool fp4 = c->fmt == MOE_FMT_NVFP4;
  const size_t n = (size_t)T * n_q * sp.S;
  char* const ml = (char*)ws + align_up(n * c->D * sizeof(float));
  DecodeArgs a{(const uint8_t*)c->pool, q, out, (float*)ws, (float2*)ml,
               (int*)(ml + align_up(n * sizeof(float2))), q_stride, out_stride, T,
               SeqView{s->row_start, s->kv_len, s->page_table, s->n_seq, s->max_pages, c->n_pages, l2},
               n_q, c->n_kv, n_q / c->n_kv, sp.S, sp.room, sp.likely,
               scale * 1.4426950408889634f * (fp4 ? c->k_scale : 1.0f), fp4 ? c->v_scale : 1.0f};
  const unsigned grid = (unsigned)(sp.items * c->n_kv);
  switch (c->fmt) {
    case MOE_FMT_NVFP4: launch_decode<MOE_FMT_NVFP4>(a, c->D, sp.tile, grid, stream); break;
    case MOE_FMT_Q8_0: launch_decode<MOE_FMT_Q8_0>(a, c->D, sp.tile, grid, stream); break;
    default: launch_decode<MOE_FMT_BF16>(a, c->D, sp.tile, grid, stream);
  }
  hipError_t e = hipGetLastError();
  if (e != hipSuccess || sp.S == 1) return e;
  switch (c->D) {
    case 64: launch_join<64>(a, stream); break;
    case 128: launch_join<128>(a, stream); break;
    default: launch_join<256>(a, stream);
  }
  return hipGetLastError();
}

}  // namespace moe
