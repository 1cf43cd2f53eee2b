// attn_chunk.hip -- attention of a chunk of new tokens over the paged cache.
//
// A prompt is worked on in chunks beside the other slots' decode steps, each chunk
// attending to what the cache holds of its sequence (aiopssre.com, "Concurrency divides
// context unless you pay for more cache").  The cache is read where it lies, without a
// 16-bit copy: a workgroup takes one key/value head and a tile of its group's query rows
// (the heads of a group together, so that a tile needs few tokens), decodes each 64
// tokens once into LDS as bf16 and goes over them with
//   scores^T (64 tokens x 32 rows of a wave) = K Q^T,  out^T (D x 32) += V^T P^T
// as 32x32x16 matrix instructions, the running maximum and sum of the softmax in
// registers.  Where the tiles are fewer than the CUs hold, sequences are split along the
// tokens and the parts joined, as in a decode step.
#include <algorithm>
#include <type_traits>

#include "attn_split.h"
#include "attn_tile.h"

namespace moe {

namespace {

typedef float v2f __attribute__((ext_vector_type(2)));

#if defined(__HIP_DEVICE_COMPILE__)  // (the host pass does not know the builtins)
typedef __amdgpu_buffer_rsrc_t Rsrc;
#else
typedef const void* Rsrc;
#endif

__device__ __forceinline__ v2f fp4_pair(uint32_t w, int k) {  // byte k: two E2M1 codes
  switch (k) {
    case 0: return __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w, 1.0f, 0);
    case 1: return __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w, 1.0f, 1);
    case 2: return __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w, 1.0f, 2);
    default: return __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w, 1.0f, 3);
  }
}
__device__ __forceinline__ float half_value(uint32_t w, int k) {  // fp16 in half k of a word
  return (float)__builtin_bit_cast(_Float16, (uint16_t)(w >> (16 * k)));
}
// int8 code k of a word whose sign bits are flipped (128 + q), times s, rounded once.
__device__ __forceinline__ float q8_value(uint32_t biased, int k, float s, float minus) {
  return fmaf((float)((biased >> (8 * k)) & 0xffu), s, minus);
}

// Place of 16-byte chunk `chunk` (2 elements of 4 tokens) of a quad's values in LDS:
// permuted within 16 chunks so that neither the 16 lanes of a write, whose chunks lie
// apart, nor those of a read meet in a bank.
template <int D>
__device__ __forceinline__ int vswz(int quad, int chunk) {
  if constexpr (D == 64) return chunk ^ (((chunk >> 4) & 1) | ((quad & 1) << 1));
  else return chunk ^ ((chunk >> 4) & 7);
}

// 64 tokens of one key/value head on their way from the cache into LDS, where keys are
// rows of D bf16 (as in the prompt kernel) and values quads [16][D][4].  Each half, 32
// tokens, lies within one page.
struct Half {
  const uint8_t* block;  // the (page, head) block
  int bytes;             // of it: 0 where there is none
  int o;                 // the half's first token within the page
  __device__ __forceinline__ Rsrc rsrc() const {
#if defined(__HIP_DEVICE_COMPILE__)
    return __builtin_amdgcn_make_buffer_rsrc(const_cast<uint8_t*>(block), 0, bytes, 0x00020000);
#else
    return nullptr;
#endif
  }
};
struct Halves {
  Half a, b;
  __device__ __forceinline__ Half of(int token) const {  // (token: the same for the whole wave)
    const bool second = token >= 32;
    return Half{second ? b.block : a.block, second ? b.bytes : a.bytes, second ? b.o : a.o};
  }
};
template <int FMT, int D, int W>
struct CacheTile {
  static constexpr bool FP4 = FMT == MOE_FMT_NVFP4, Q8 = FMT == MOE_FMT_Q8_0;
  // Keys: 16 bytes of a token a lane, PT of them a token; TL neighbouring lanes take
  // neighbouring tokens (so that 16 lanes' writes fall into different banks), a load of
  // the wave PB pieces of 64 / PB tokens.
  static constexpr int ROW = FP4 ? D / 2 : Q8 ? D : 2 * D;  // bytes of a token's codes
  static constexpr int PT = ROW / 16;
  static constexpr int TL = FP4 ? (D == 64 ? 8 : 16) : D == 64 ? 4 : 8;
  static constexpr int PB = PT < 64 / TL ? PT : 64 / TL;
  static constexpr int KI = (PT + W - 1) / W;  // loads of a wave (PT in all)
  // Values: UQ pieces of a quad, a piece of UW words of a lane
  static constexpr int UQ = FP4 ? (D == 64 ? 8 : 16) : D / 4;
  static constexpr int UW = FP4 && D == 256 ? 8 : 4;
  static constexpr int VL = UQ / 4, VI = (VL + W - 1) / W;
  uint32_t kq[KI][4], ks[KI], vq[VI][UW], vs[VI][2];

  __device__ __forceinline__ static uint32_t load(Rsrc r, uint32_t at, uint32_t base, int bytes) {
#if defined(__HIP_DEVICE_COMPILE__)
    if (bytes == 2) return (uint16_t)__builtin_amdgcn_raw_buffer_load_b16(r, at, base, 0);
    return __builtin_amdgcn_raw_buffer_load_b32(r, at, base, 0);
#else
    return 0;
#endif
  }
  __device__ __forceinline__ static void load_16(Rsrc r, uint32_t* d, uint32_t at, uint32_t base) {
#if defined(__HIP_DEVICE_COMPILE__)
    const auto x = __builtin_amdgcn_raw_buffer_load_b128(r, at, base, 0);
    d[0] = x[0]; d[1] = x[1]; d[2] = x[2]; d[3] = x[3];
#endif
  }
  // Of key load i: its first token, this lane's token behind it and piece.
  __device__ __forceinline__ static int key_block(int wi) { return wi / (PT / PB) * (64 / PB); }
  __device__ __forceinline__ static int key_token(int lane) { return lane % TL + TL * (lane / TL / PB); }
  __device__ __forceinline__ static int key_piece(int wi, int lane) { return wi % (PT / PB) * PB + lane / TL % PB; }

  __device__ __forceinline__ void fetch(const Halves& half, const KvLayout lay, int P, int wave, int lane) {
#pragma unroll
    for (int i = 0; i < KI; ++i) {
      const int wi = i * W + wave;
      if (PT % W != 0 && wi >= PT) break;
      const int tb = key_block(wi);
      const Half hf = half.of(tb);
      const Rsrc block = hf.rsrc();
      const int tok = hf.o + (tb & 31) + key_token(lane), piece = key_piece(wi, lane);
      load_16(block, kq[i], tok * ROW + piece * 16, 0);
      if constexpr (FP4) ks[i] = load(block, tok * (D / 16) + piece * 2, lay.ks, 2);
      else ks[i] = load(block, 2 * (tok * (D / 32) + piece / 2), lay.ks, 2);
    }
#pragma unroll
    for (int i = 0; i < VI; ++i) {
      const int wi = i * W + wave;
      if (VL % W != 0 && wi >= VL) break;
      const int first = wi * 64 / UQ;  // quad
      const Half hf = half.of(4 * first);
      const Rsrc block = hf.rsrc();
      const int quad = first + lane / UQ, piece = lane % UQ, tok = hf.o + (quad & 7) * 4;
      const uint32_t at = tok * ROW + piece * (UW * 4);
      load_16(block, vq[i], at, lay.vq);
      if constexpr (UW == 8) load_16(block, vq[i] + 4, at + 16, lay.vq);
      const int e = piece * (D / UQ);  // first element
      if constexpr (FP4) {
        vs[i][0] = load(block, e / 16 * P + tok, lay.vs, 4);
      } else {
        const uint32_t s = 2 * (e / 32 * P + tok);
        vs[i][0] = load(block, s, lay.vs, 4);
        vs[i][1] = load(block, s + 4, lay.vs, 4);
      }
    }
  }

  // left: the tile's tokens that some row sees; values from there on count as 0, whatever
  // the cache holds.
  __device__ __forceinline__ void put(uint8_t* kt, uint8_t* vt, int left, int wave, int lane) {
#pragma unroll
    for (int i = 0; i < KI; ++i) {
      const int wi = i * W + wave;
      if (PT % W != 0 && wi >= PT) break;
      const int row = key_block(wi) + key_token(lane), piece = key_piece(wi, lane);
      uint8_t* const d = kt + row * (2 * D);
      if constexpr (FP4) {
        const v2f s = __builtin_amdgcn_cvt_scalef32_pk_f32_fp8(ks[i], 1.0f, false);
#pragma unroll
        for (int w = 0; w < 4; ++w) {
          const float f = w < 2 ? s[0] : s[1];
          uint32_t c[4];
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            const v2f v = fp4_pair(kq[i][w], k);
            c[k] = bf16_pair(v[0] * f, v[1] * f);
          }
          *reinterpret_cast<uint4*>(d + swz<D>(row, piece * 4 + w) * 16) = make_uint4(c[0], c[1], c[2], c[3]);
        }
      } else {
        const float f = half_value(ks[i], 0), minus = -128.0f * f;
#pragma unroll
        for (int w = 0; w < 4; w += 2) {
          uint32_t c[4];
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            const uint32_t b = kq[i][w + (k >> 1)] ^ 0x80808080u;
            c[k] = bf16_pair(q8_value(b, 2 * (k & 1), f, minus), q8_value(b, 2 * (k & 1) + 1, f, minus));
          }
          *reinterpret_cast<uint4*>(d + swz<D>(row, piece * 2 + w / 2) * 16) = make_uint4(c[0], c[1], c[2], c[3]);
        }
      }
    }
#pragma unroll
    for (int i = 0; i < VI; ++i) {
      const int wi = i * W + wave;
      if (VL % W != 0 && wi >= VL) break;
      const int quad = wi * 64 / UQ + lane / UQ, piece = lane % UQ;
      uint8_t* const d = vt + quad * (8 * D);
      if (left < kBN) {
        const int n = min(max(left - 4 * quad, 0), 4);
        if constexpr (FP4) {
          vs[i][0] = n >= 4 ? vs[i][0] : vs[i][0] & ((1u << (8 * n)) - 1u);
        } else {
          vs[i][0] &= n >= 2 ? ~0u : n == 1 ? 0xffffu : 0u;
          vs[i][1] &= n >= 4 ? ~0u : n == 3 ? 0xffffu : 0u;
        }
      }
      float s[4];
      if constexpr (FP4) {
        const v2f a = __builtin_amdgcn_cvt_scalef32_pk_f32_fp8(vs[i][0], 1.0f, false);
        const v2f b = __builtin_amdgcn_cvt_scalef32_pk_f32_fp8(vs[i][0], 1.0f, true);
        s[0] = a[0]; s[1] = a[1]; s[2] = b[0]; s[3] = b[1];
        constexpr int NC = D == 256 ? 8 : 4;  // chunks of a piece
#pragma unroll
        for (int e = 0; e < NC; ++e) {
          v2f p[4];
#pragma unroll
          for (int t = 0; t < 4; ++t) {
            // byte e of token t: [4][4 bytes], [4][8 bytes], or twice [4][2 bytes]
            if constexpr (D == 128) p[t] = fp4_pair(vq[i][t], e);
            else if constexpr (D == 256) p[t] = fp4_pair(vq[i][2 * t + e / 4], e % 4);
            else p[t] = fp4_pair(vq[i][e / 2 * 2 + t / 2], 2 * (t & 1) + (e & 1));
          }
          *reinterpret_cast<uint4*>(d + vswz<D>(quad, piece * NC + e) * 16) =
              make_uint4(bf16_pair(p[0][0] * s[0], p[1][0] * s[1]), bf16_pair(p[2][0] * s[2], p[3][0] * s[3]),
                         bf16_pair(p[0][1] * s[0], p[1][1] * s[1]), bf16_pair(p[2][1] * s[2], p[3][1] * s[3]));
        }
      } else {
        float minus[4];
#pragma unroll
        for (int t = 0; t < 4; ++t) {
          s[t] = half_value(vs[i][t >> 1], t & 1);
          minus[t] = -128.0f * s[t];
        }
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          uint32_t c[4];
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            const uint32_t b = vq[i][2 * e + (k >> 1)] ^ 0x80808080u;
            const int t = 2 * (k & 1);
            c[k] = bf16_pair(q8_value(b, t, s[t], minus[t]), q8_value(b, t + 1, s[t + 1], minus[t + 1]));
          }
          *reinterpret_cast<uint4*>(d + vswz<D>(quad, piece * 2 + e) * 16) = make_uint4(c[0], c[1], c[2], c[3]);
        }
      }
    }
  }
};

// 16-bit caches need no decoding: straight from global memory into LDS, lane i of a load
// filling the 16 bytes at slot i with the chunk that belongs there.
template <int D, int W>
struct CacheTile<MOE_FMT_BF16, D, W> {
  static constexpr int CPR = D / 8;       // loads of 1 KB: keys, and as many of values
  static constexpr int N = CPR / W;
  __device__ __forceinline__ static void fetch(const Halves& half, const KvLayout lay, uint8_t* kt, uint8_t* vt,
                                               int wave, int lane) {
#if defined(__HIP_DEVICE_COMPILE__)
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const int wi = i * W + wave, slot = wi * 64 + lane;
      const int first = wi * 64 / CPR, row = slot / CPR;  // token
      const Half hk = half.of(first);
      __builtin_amdgcn_raw_ptr_buffer_load_lds(
          hk.rsrc(), (__attribute__((address_space(3))) void*)(kt + wi * 1024), 16,
          (hk.o + (row & 31)) * (2 * D) + swz<D>(row, slot % CPR) * 16, 0, 0, 0);
      constexpr int CPQ = D / 2;  // chunks of a quad
      const int q0 = wi * 64 / CPQ, quad = slot / CPQ;
      const Half hv = half.of(4 * q0);
      __builtin_amdgcn_raw_ptr_buffer_load_lds(
          hv.rsrc(), (__attribute__((address_space(3))) void*)(vt + wi * 1024), 16,
          (hv.o / 4 + (quad & 7)) * (8 * D) + vswz<D>(quad, slot % CPQ) * 16, lay.vq, 0, 0);
    }
#endif
  }
};

// The rows of a wave against tiles whose values lie as quads.
template <int D>
struct ChunkRows : TileRows<D> {
  static constexpr int KS = D / 16, NJ = D / 32;
  using TileRows<D>::qf;
  using TileRows<D>::o;
  using TileRows<D>::h;
  using TileRows<D>::m;
  using TileRows<D>::l;
  uint32_t ka[KS], va[NJ];  // this lane's places in a K and a V tile

  __device__ __forceinline__ void places(int lane) {
    const int n = lane & 31;
    h = lane >> 5;
#pragma unroll
    for (int s = 0; s < KS; ++s) ka[s] = n * (2 * D) + swz<D>(n, 2 * s + h) * 16;
#pragma unroll
    for (int j = 0; j < NJ; ++j) va[j] = h * (8 * D) + vswz<D>(h, 16 * j + (n >> 1)) * 16 + (n & 1) * 8;
  }
  // Key fragment: 16 elements (step s) of 32 keys (half t).
  __device__ __forceinline__ v4u key(const uint8_t* kt, int t, int s) const {
    return *reinterpret_cast<const v4u*>(kt + ka[s] + t * (64 * D));
  }
  // Value fragment of 16 keys (step s) and 32 elements (block j): keys 4h.. and 8 + 4h..,
  // as the score accumulators hold them.
  __device__ __forceinline__ v4u value(const uint8_t* vt, int s, int j) const {
    v4u f;
#pragma unroll
    for (int q = 0; q < 2; ++q) {
      const uint2 w = *reinterpret_cast<const uint2*>(vt + va[j] + (4 * s + 2 * q) * (8 * D));
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
  // A new maximum for the rows whose weights would leave 2^kGrow (the others' answers do
  // not depend on them, bit for bit).
  __device__ __forceinline__ void raise(const v16f (&x)[2], float c) {
    const float mx = this->top(x, c);
    if (__any(mx > m + kGrow)) {
      const float mn = mx > m + kGrow ? mx : m, al = __builtin_amdgcn_exp2f(m - mn);
#pragma unroll
      for (int j = 0; j < NJ; ++j)
#pragma unroll
        for (int i = 0; i < 16; ++i) o[j][i] *= al;
      l *= al;
      m = mn;
    }
  }
  // The weighted values of a tile with infinities or NaN among them that some row may not
  // see: a zero weight would not silence them, so one key at a time, added only to the
  // rows that see it.
  __device__ __forceinline__ void gather_seen(const uint8_t* vt, const v4u (&p)[4], int64_t t0) {
#pragma unroll
    for (int s = 0; s < 4; ++s)
#pragma unroll
      for (int j = 0; j < NJ; ++j) {
        const v4u f = value(vt, s, j);
#pragma unroll 1
        for (int tk = 0; tk < 16; ++tk) {
          const int at = 2 * (tk >> 3) + ((tk & 3) >> 1);
          const uint32_t keep = h == ((tk >> 2) & 1) ? 0xffffu << (16 * (tk & 1)) : 0u;
          const bool seen = t0 + 16 * s + tk <= this->limit;
          v4u one;
          v16f z;
#pragma unroll
          for (int i = 0; i < 4; ++i) one[i] = i == at ? f[i] & keep : 0u;
#pragma unroll
          for (int i = 0; i < 16; ++i) z[i] = 0.0f;
          z = mma(one, p[s], z);
#pragma unroll
          for (int i = 0; i < 16; ++i) o[j][i] += seen ? z[i] : 0.0f;
        }
      }
  }
};

// Whether a tile of values holds an infinity or a NaN.
template <int D>
__device__ __forceinline__ bool wild(const uint8_t* vt, int lane) {
  bool any = false;
#pragma unroll 4
  for (int i = lane; i < kBN * D / 8; i += 64) {
    const v4u f = reinterpret_cast<const v4u*>(vt)[i];
#pragma unroll
    for (int k = 0; k < 4; ++k) any |= (f[k] & 0x7f80u) == 0x7f80u || (f[k] & 0x7f800000u) == 0x7f800000u;
  }
  return __any(any);
}

template <int FMT, int D, int W>
__global__ __launch_bounds__(64 * W, D <= 128 ? 2 : 1) void k_attn_chunk(SplitArgs a) {
  constexpr int KS = D / 16, NJ = D / 32, SIZE = 32 * W, TILE = kBN * D * 2;
  __shared__ __align__(16) uint8_t k_even[TILE], k_odd[TILE], v_even[TILE], v_odd[TILE];
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int lane = lane_id(), n = lane & 31;
  Item it = find_item(a.s, a.T, a.G, SIZE, a.n_kv, a.room, a.S, (int)blockIdx.x);
  if (it.b < 0) return;
  // (a sequence's last rows, which see the most, first)
  it.tile = (int)((uint32_t)(it.inside * a.G + SIZE - 1) / (uint32_t)SIZE) - 1 - it.tile;
  const int r0 = it.r0, rows = it.rows, len = it.len, inside = it.inside, kvh = it.kvh, sp = it.sp;
  const int P = 1 << a.s.log2P;
  const KvLayout lay = kv_layout(FMT, D, P);
  const size_t page_bytes = (size_t)a.n_kv * lay.head;
  const uint8_t* heads = a.pool + (size_t)kvh * lay.head;
  const TilePlan plan = tile_plan(a.s, it, a.G, SIZE);
  const int u_begin = sp > 0 ? sp * it.chunk : 0;
  const int u_end = (int)min((int64_t)plan.units, (int64_t)u_begin + it.chunk);
  if (sp > 0 && u_begin >= u_end) {  // (split 0 also answers rows that see nothing)
    const int rr = it.tile * SIZE + threadIdx.x, i = (int)((uint32_t)rr / (uint32_t)a.G);
    if (threadIdx.x < SIZE && rr < inside * a.G)
      a.part_ml[((int64_t)(r0 + i) * a.n_q + kvh * a.G + rr - i * a.G) * a.S + sp] = make_float2(kNone, 0.0f);
    return;
  }

  // this lane's query row; a lane without one takes the tile's last (its answer goes
  // nowhere: another tile's row may be overwritten meanwhile, where the output takes the
  // queries' place)
  ChunkRows<D> w;
  const int slot = (it.tile * W + wave) * 32 + n, last_slot = inside * a.G - 1;
  const int mine = min(slot, last_slot), row = (int)((uint32_t)mine / (uint32_t)a.G);
  const int64_t at = (int64_t)(r0 + row);
  const int head = kvh * a.G + mine - row * a.G;
  w.limit = slot <= last_slot ? (int64_t)len - rows + row : -1;
  const uint16_t* qp = a.q + at * a.q_stride + (int64_t)head * D + 8 * (lane >> 5);
#pragma unroll
  for (int s = 0; s < KS; ++s) w.qf[s] = *reinterpret_cast<const v4u*>(qp + 16 * s);
  w.places(lane);
  w.clear();
  // last token that some row of the wave sees
  const int wave_row = (int)((uint32_t)min((it.tile * W + wave) * 32 + 31, last_slot) / (uint32_t)a.G);
  const int64_t hi_wave = (it.tile * W + wave) * 32 <= last_slot ? (int64_t)len - rows + wave_row : -1;

  // Pages of the two halves of tile t (units 2t, 2t + 1), by scalar loads; a unit past the
  // table's end has none, and one past the last token that is looked at is not looked for.
  const int* const table = a.s.page_table + (int64_t)it.b * a.s.max_pages;
  const auto page_at = [&](int u) {
    if (u >= u_end) return -1;
    const int i = (int)(((int64_t)u * 32) >> a.s.log2P);
    const int p = *(const int __attribute__((address_space(4)))*)(uintptr_t)(table + min(i, a.s.max_pages - 1));
    return i < a.s.max_pages && (unsigned)p < (unsigned)a.s.n_pages ? p : -1;
  };
  const auto half_of = [&](int u) {
    const int p = page_at(u);
    return Half{heads + (size_t)max(p, 0) * page_bytes, p < 0 ? 0 : (int)lay.head, (u * 32) & (P - 1)};
  };

  const int first = u_begin / 2, end = (u_end + 1) / 2;
  CacheTile<FMT, D, W> raw;
  const auto fetch = [&](int t, uint8_t* kt, uint8_t* vt) {
    const Halves hf{half_of(2 * t), half_of(2 * t + 1)};
    if constexpr (FMT == MOE_FMT_BF16) raw.fetch(hf, lay, kt, vt, wave, lane);
    else raw.fetch(hf, lay, P, wave, lane);
  };
  const auto left_of = [&](int t) { return (int)min(plan.hi + 1 - (int64_t)t * kBN, (int64_t)kBN); };
  // Tile t against this wave's rows.
  const auto work = [&](int t, const uint8_t* kt, const uint8_t* vt) {
    const int64_t t0 = (int64_t)t * kBN;
    if (t0 > hi_wave) return;
    const bool edge = t0 + kBN - 1 > plan.lo;
    v16f x[2];
    v4u p[4];
    w.scores(kt, x);
    if (edge) w.mask(x, t0);
    w.raise(x, a.scale_log2);
#pragma unroll
    for (int v = 0; v < 32; ++v) w.weight(x, a.scale_log2, p, v);
#pragma unroll
    for (int k = 0; k < 2; ++k)  // nothing to read: rows that see a token of it have no answer
      if (page_at(2 * t + k) < 0 && w.limit >= t0 + 32 * k && 2 * t + k < u_end) w.l = __uint_as_float(0x7fc00000u);
    if (edge && wild<D>(vt, lane)) {
      w.gather_seen(vt, p, t0);
      return;
    }
#pragma unroll
    for (int s = 0; s < 4; ++s)
#pragma unroll
      for (int j = 0; j < NJ; ++j) w.o[j] = mma(w.value(vt, s, j), p[s], w.o[j]);
  };
  // 16-bit values behind the last one that is seen, cleared in LDS.
  const auto clear_behind = [&](int t, uint8_t* vt) {
    const int left = left_of(t);
    if (left >= kBN) return;
    for (int i = threadIdx.x; i < kBN * D / 4; i += 64 * W) {  // 4 tokens of one element
      const int quad = i / D, seen = min(max(left - 4 * quad, 0), 4);
      uint2* d = reinterpret_cast<uint2*>(vt) + i;
      uint2 v = *d;
      v.x &= seen >= 2 ? ~0u : seen == 1 ? 0xffffu : 0u;
      v.y &= seen >= 4 ? ~0u : seen == 3 ? 0xffffu : 0u;
      *d = v;
    }
    __syncthreads();
  };
  if (first < end) {
    if constexpr (FMT == MOE_FMT_BF16) {
      fetch(first, k_even, v_even);
      const auto turn = [&](int t, uint8_t* kt, uint8_t* vt, uint8_t* kn, uint8_t* vn) {
        wait_loads<0>();
        __syncthreads();
        clear_behind(t, vt);
        if (t + 1 < end) fetch(t + 1, kn, vn);
        work(t, kt, vt);
      };
#pragma unroll 1
      for (int t = first; t < end; t += 2) {
        turn(t, k_even, v_even, k_odd, v_odd);
        if (t + 1 < end) turn(t + 1, k_odd, v_odd, k_even, v_even);
      }
    } else {
      fetch(first, nullptr, nullptr);
      raw.put(k_even, v_even, left_of(first), wave, lane);
      if (first + 1 < end) fetch(first + 1, nullptr, nullptr);
      const auto turn = [&](int t, uint8_t* kt, uint8_t* vt, uint8_t* kn, uint8_t* vn) {
        __syncthreads();
        if (t + 1 < end) {
          raw.put(kn, vn, left_of(t + 1), wave, lane);
          if (t + 2 < end) fetch(t + 2, nullptr, nullptr);
        }
        work(t, kt, vt);
      };
#pragma unroll 1
      for (int t = first; t < end; t += 2) {
        turn(t, k_even, v_even, k_odd, v_odd);
        if (t + 1 < end) turn(t + 1, k_odd, v_odd, k_even, v_even);
      }
    }
  }
  w.finish();
  if (slot > last_slot) return;
  if (n == slot - (it.tile * W + wave) * 32 && lane < 32 && sp == 0 && a.S > 1) a.part_n[at * a.n_q + head] = it.splits;
  if (it.splits == 1) {
    const float inv = w.limit < 0 ? 0.0f : 1.0f / w.l, ts = a.v_ts;
    // A lane holds 4 of every 8 elements, its partner in the other half of the wave the
    // other 4: one swap of two pieces gives each 8 in a row, for one store.
    uint16_t* d = a.out + at * a.out_stride + (int64_t)head * D + 8 * w.h;
#pragma unroll
    for (int j = 0; j < NJ; ++j)
#pragma unroll
      for (int i = 0; i < 16; i += 8) {
        float v[8];
#pragma unroll
        for (int k = 0; k < 8; ++k) v[k] = w.o[j][i + k] * inv * ts;
        const auto lo = __builtin_amdgcn_permlane32_swap(bf16_pair(v[0], v[1]), bf16_pair(v[4], v[5]), false, false);
        const auto hi = __builtin_amdgcn_permlane32_swap(bf16_pair(v[2], v[3]), bf16_pair(v[6], v[7]), false, false);
        *reinterpret_cast<uint4*>(d + 32 * j + 2 * i) = make_uint4(lo[0], hi[0], lo[1], hi[1]);
      }
  } else {
    const int64_t part = (at * a.n_q + head) * a.S + sp;
    if (lane < 32) a.part_ml[part] = make_float2(w.m, w.l);
    float* d = a.part_o + part * D + 4 * w.h;
#pragma unroll
    for (int j = 0; j < NJ; ++j)
#pragma unroll
      for (int i = 0; i < 16; i += 4)
        *reinterpret_cast<float4*>(d + 32 * j + 2 * i) =
            make_float4(w.o[j][i], w.o[j][i + 1], w.o[j][i + 2], w.o[j][i + 3]);
  }
}

// Launch shape: splits there is room for in the workspace (1: no split), and for each
// key/value head chunks and items (the grid).
struct Shape {
  int S, room, likely;
  int64_t items;
};
constexpr int kChunkWaves = 4;
Shape shape_of(int D, int n_kv, int n_q, int n_seq, int64_t T, int64_t max_len) {
  const int G = n_q / n_kv, size = 32 * kChunkWaves;
  const int64_t units = (std::min(max_len, (int64_t)INT32_MAX) + 31) / 32;  // (lengths are 32-bit)
  const int64_t per_seq = (T + n_seq - 1) / n_seq;
  const int64_t tiles = T * G / size + n_seq;  // at most: one part tile a sequence
  const int64_t base = (int64_t)n_seq * n_kv * ((per_seq * G + size - 1) / size);
  const int target = 512;
  Shape r;
  int64_t S = ((int64_t)256 << 20) / (T * n_q * D * 4);
  S = std::min({S, (int64_t)kMaxSplit, (units + kWaves - 1) / kWaves});
  r.S = T * n_q > kChunkPairs || S < 2 || (n_seq == 1 && base >= 2 * target) || units <= 31 ? 1 : (int)S;
  r.likely = (int)std::min({(int64_t)std::max(units / kWhole, (int64_t)1), std::max(target / base, (int64_t)1), (int64_t)r.S});
  r.room = (int)std::max((int64_t)1, std::min((int64_t)target / n_kv, tiles * r.S));
  r.items = tiles + (r.S > 1 ? r.room + 1 : 0);
  return r;
}

template <int FMT>
void launch_chunk(const SplitArgs& a, int D, unsigned grid, hipStream_t stream) {
  constexpr int W = kChunkWaves, N = 64 * W;
  if (D == 64) k_attn_chunk<FMT, 64, W><<<grid, N, 0, stream>>>(a);
  else if (D == 128) k_attn_chunk<FMT, 128, W><<<grid, N, 0, stream>>>(a);
  else k_attn_chunk<FMT, 256, W><<<grid, N, 0, stream>>>(a);
}

}  // namespace

size_t attn_chunk_ws_bytes(int n_kv, int D, int n_q, int n_seq, int64_t T, int64_t max_len) {
  if (n_seq < 1 || T < 1) return 0;
  const Shape sp = shape_of(D, n_kv, n_q, n_seq, T, max_len);
  if (sp.S == 1) return 0;
  const size_t n = (size_t)T * n_q * sp.S;
  return align_up(n * D * sizeof(float)) + align_up(n * sizeof(float2)) + align_up((size_t)T * n_q * sizeof(int));
}

hipError_t launch_attn_chunk(const moe_kv_cache* c, const moe_seq_batch* s, int n_q,
                             const uint16_t* q, int64_t q_stride, int64_t T, int64_t max_len,
                             float scale, uint16_t* out, int64_t out_stride, void* ws,
                             hipStream_t stream) {
  const Shape sp = shape_of(c->D, c->n_kv, n_q, s->n_seq, T, max_len);
  int l2 = 0;
  while ((1 << l2) < c->page_tokens) ++l2;
  const bool fp4 = c->fmt == MOE_FMT_NVFP4;
  const size_t n = (size_t)T * n_q * sp.S;
  char* const ml = (char*)ws + align_up(n * c->D * sizeof(float));
  const SplitArgs a{(const uint8_t*)c->pool, q, out, (float*)ws, (float2*)ml,
                    (int*)(ml + align_up(n * sizeof(float2))), q_stride, out_stride, T,
                    SeqView{s->row_start, s->kv_len, s->page_table, s->n_seq, s->max_pages, c->n_pages, l2},
                    n_q, c->n_kv, n_q / c->n_kv, sp.S, sp.room, sp.likely,
                    scale * 1.4426950408889634f * (fp4 ? c->k_scale : 1.0f), fp4 ? c->v_scale : 1.0f};
  const unsigned grid = (unsigned)(sp.items * c->n_kv);
  switch (c->fmt) {
    case MOE_FMT_NVFP4: launch_chunk<MOE_FMT_NVFP4>(a, c->D, grid, stream); break;
    case MOE_FMT_Q8_0: launch_chunk<MOE_FMT_Q8_0>(a, c->D, grid, stream); break;
    default: launch_chunk<MOE_FMT_BF16>(a, c->D, grid, stream);
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
