// attn_chunk.hip -- attention of a chunk of new tokens over the paged cache.
//
// A prompt is worked on in chunks beside the other slots' decode steps, each chunk
// attending to what the cache holds of its sequence (aiopssre.com, "Concurrency divides
// context unless you pay for more cache").  The cache is read where it lies, without a
// 16-bit copy: a workgroup takes one key/value head and a tile of its group's query rows
// (the heads of a group together, so that a tile needs few tokens), decodes each 64
// tokens once into LDS (codes as fp16, 16-bit caches as they are) and goes over them with
//   scores^T (64 tokens x 32 rows of a wave) = K Q^T,  out^T (D x 32) += V^T P^T
// as 32x32x16 matrix instructions, the running maximum and sum of the softmax in
// registers.  Where the tiles are fewer than the CUs hold, sequences are split along the
// tokens and the parts joined, as in a decode step.
//
// 32 query and 4 key/value heads of 128 over NVFP4: 4096 rows behind 12288 tokens 863 to 930
// us (1.03 to 1.11 PFLOP/s; a bf16 library product 1.2; over Q8_0 954, 16 bits 844), 64 rows
// behind 32768 tokens 55 to 63 us (the join of 33 MB of parts 7 of it; Q8_0 62, 16 bits 57);
// 512 rows of 8 slots, 505 of them one's, over Q8_0 with heads of 64 85 to 91 us.  Beside
// the other calls, 512 rows behind 8192: 99 us, k_attn_decode 118, read back and k_attn_prompt
// 133; 64 rows behind 8192 37, 29 and 126; 4096 behind 12288 897, - and 775.  In the first the matrix units are half of the time busy at the
// 2.1 GHz they hold, the vector units (exponentials, maxima, rounding, decoding) as long and
// LDS as well (256 KB of fragments a turn): 256 rows a workgroup is what the registers hold,
// and it halves the decoding and the reads of the cache against 128 (1222 us).  Reading the
// first fragments of a turn before the waves meet, in a ring of three key buffers, changed
// nothing.
#include <algorithm>
#include <type_traits>

#include "attn_split.h"
#include "attn_tile.h"

namespace moe {

namespace {

#if defined(__HIP_DEVICE_COMPILE__)  // (the host pass does not know the builtins)
typedef __amdgpu_buffer_rsrc_t Rsrc;
#else
typedef const void* Rsrc;
#endif

// Place of 16-byte chunk `chunk` (2 elements of 4 tokens) of a quad's values in LDS:
// permuted within 16 chunks so that neither the 16 lanes of a write, whose chunks lie
// apart, nor those of a read meet in a bank.
template <int D>
__device__ __forceinline__ int vswz(int quad, int chunk) {
  if constexpr (D == 64) return chunk ^ (((chunk >> 4) & 1) | ((quad & 1) << 1));
  else return chunk ^ ((chunk >> 4) & 7);
}

// Where the 32 tokens of a unit lie.
struct Unit32 {
  const uint8_t* block;  // the (page, head) block
  int bytes;             // of it: 0 where there is none
  int o;                 // the unit's first token within the page
  __device__ __forceinline__ Rsrc rsrc() const {
#if defined(__HIP_DEVICE_COMPILE__)
    return __builtin_amdgcn_make_buffer_rsrc(const_cast<uint8_t*>(block), 0, bytes, 0x00020000);
#else
    return nullptr;
#endif
  }
};
// Where the 64 tokens of a tile lie.
struct Place {
  Unit32 a, b;
  __device__ __forceinline__ Unit32 of(int token) const {  // (token: the same for the whole wave)
    const bool second = token >= 32;
    return Unit32{second ? b.block : a.block, second ? b.bytes : a.bytes, second ? b.o : a.o};
  }
};

// A tile's codes on their way from the cache into LDS, where keys are rows of D bf16 (as
// in the prompt kernel) and values quads [16][D][4]: as they were loaded, decoded piece by
// piece.  A piece is one 16-byte store of a lane, 8 elements of a key or 2 of four tokens'
// values; every lane has N of each, so that no piece is behind a branch (which would let
// the compiler move the softmax out of the matrix instructions' shadow).
template <int FMT, int D, int W>
struct Codes {
  static constexpr bool FP4 = FMT == MOE_FMT_NVFP4;
  static constexpr int ROW = FP4 ? D / 2 : D;  // bytes of a token's codes
  static constexpr int N = D / 8 / W, PIECES = 2 * N;
  static_assert(D % (8 * W) == 0, "waves share the pieces evenly");
  // Keys: a lane takes 8 N elements of one token, KW words, TL neighbouring lanes those of
  // neighbouring tokens, so that 16 lanes' stores fall into different banks.
  static constexpr int KW = FP4 ? N : 2 * N, PARTS = D / 8 / N, TL = D == 64 ? 1 : D == 128 ? 8 : 16;
  // Values: a lane takes 2 N elements of a quad; those of NVFP4 heads below 256 are half of
  // what it loads, VW words.
  static constexpr int QL = D / 2 / N, VW = FP4 ? (D == 64 ? 2 : D == 128 ? 4 : 8) : 2 * N;
  uint32_t kq[KW], ks, vq[VW], vs[2];

  template <int BYTES>
  __device__ __forceinline__ static uint32_t load(Rsrc r, uint32_t at, uint32_t base) {
#if defined(__HIP_DEVICE_COMPILE__)
    if constexpr (BYTES == 1) return (uint8_t)__builtin_amdgcn_raw_buffer_load_b8(r, at, base, 0);
    if constexpr (BYTES == 2) return (uint16_t)__builtin_amdgcn_raw_buffer_load_b16(r, at, base, 0);
    return __builtin_amdgcn_raw_buffer_load_b32(r, at, base, 0);
#else
    return 0;
#endif
  }
  template <int WORDS>
  __device__ __forceinline__ static void load_words(Rsrc r, uint32_t* d, uint32_t at, uint32_t base) {
#if defined(__HIP_DEVICE_COMPILE__)
    if constexpr (WORDS == 1) {
      d[0] = __builtin_amdgcn_raw_buffer_load_b32(r, at, base, 0);
    } else if constexpr (WORDS == 2) {
      const auto x = __builtin_amdgcn_raw_buffer_load_b64(r, at, base, 0);
      d[0] = x[0]; d[1] = x[1];
    } else {
#pragma unroll
      for (int i = 0; i < WORDS; i += 4) {
        const auto x = __builtin_amdgcn_raw_buffer_load_b128(r, at + 4 * i, base, 0);
        d[i] = x[0]; d[i + 1] = x[1]; d[i + 2] = x[2]; d[i + 3] = x[3];
      }
    }
#endif
  }
  // This lane's token (row of the tile) and part of it.
  __device__ __forceinline__ static int key_row(int wave, int lane) {
    return TL == 1 ? wave * (64 / PARTS) + lane / PARTS : wave * (64 / PARTS) + lane % TL + TL * (lane / (TL * PARTS));
  }
  __device__ __forceinline__ static int key_part(int lane) { return TL == 1 ? lane % PARTS : lane / TL % PARTS; }
  // This lane's quad and place in it.
  __device__ __forceinline__ static int quad_of(int wave, int lane) { return wave * (64 / QL) + lane / QL; }

  __device__ __forceinline__ void fetch_keys(const Place& from, const KvLayout lay, int wave, int lane) {
    const Unit32 u = from.of(wave * (64 / PARTS));
    const Rsrc block = u.rsrc();
    const int tok = u.o + (key_row(wave, lane) & 31), part = key_part(lane);
    load_words<KW>(block, kq, tok * ROW + part * (4 * KW), 0);
    if constexpr (FP4) {  // scales of 16 elements: of 8 N / 16 blocks, or the one that holds the lane's
      constexpr int B = N >= 8 ? 4 : 1;
      ks = load<B>(block, tok * (D / 16) + part * 8 * N / 16, lay.ks);
    } else {
      constexpr int B = N >= 8 ? 4 : 2;
      ks = load<B>(block, 2 * (tok * (D / 32) + part * 8 * N / 32), lay.ks);
    }
  }
  __device__ __forceinline__ void fetch_values(const Place& from, const KvLayout lay, int P, int wave, int lane) {
    const Unit32 u = from.of(4 * (wave * (64 / QL)));
    const Rsrc block = u.rsrc();
    const int tok = u.o + (quad_of(wave, lane) & 7) * 4, ql = lane % QL, e = ql * 2 * N;  // first element
    if constexpr (FP4) {
      // [16][4 tokens][D/32 bytes] of a quad
      constexpr int LANES = QL / 16;  // lanes of a group
      load_words<VW>(block, vq, tok * ROW + ql / LANES * (4 * VW), lay.vq);
      vs[0] = load<4>(block, e / 16 * P + tok, lay.vs);
    } else {
      load_words<VW>(block, vq, tok * ROW + ql * (4 * VW), lay.vq);
      const uint32_t s = 2 * (e / 32 * P + tok);
      vs[0] = load<4>(block, s, lay.vs);
      vs[1] = load<4>(block, s + 4, lay.vs);
    }
  }

  __device__ __forceinline__ void put_key(int n, uint8_t* kt, int wave, int lane) const {
    const int row = key_row(wave, lane);
    uint32_t c[4];
    if constexpr (FP4) {
      const v2h s = fp8_pair(ks, n / 4);  // (pieces 2b, 2b + 1 are block b)
      const v2h f = n / 2 & 1 ? v2h{s.y, s.y} : v2h{s.x, s.x};
#pragma unroll
      for (int k = 0; k < 4; ++k) c[k] = bits(fp4_pair(kq[n], k) * f);
    } else {
      const v2h s = halves(ks), f = n / 4 ? v2h{s.y, s.y} : v2h{s.x, s.x};
#pragma unroll
      for (int k = 0; k < 4; ++k) c[k] = bits(i8_pair(kq[2 * n + (k >> 1)] ^ 0x80808080u, k & 1) * f);
    }
    *reinterpret_cast<uint4*>(kt + row * (2 * D) + swz<D>(row, key_part(lane) * N + n) * 16) = make_uint4(c[0], c[1], c[2], c[3]);
  }
  // Whether a value of the lane's that counts may be infinite or NaN: its scale says so
  // (fp16 scales below 512 make 65504 at most).
  __device__ __forceinline__ bool wild() const {
    bool any = false;
    if constexpr (FP4) {
#pragma unroll
      for (int i = 0; i < 4; ++i) any |= ((vs[0] >> (8 * i)) & 0x7fu) == 0x7fu;
    } else {
#pragma unroll
      for (int i = 0; i < 2; ++i) any |= (vs[i] & 0x7fffu) >= 0x6000u || (vs[i] & 0x7fff0000u) >= 0x60000000u;
    }
    return any;
  }
  // What was loaded, moved to where the pieces look for it; left: the tile's tokens that
  // some row sees; values from there on count as 0, whatever the cache holds.
  __device__ __forceinline__ void arrange_values(int left, int wave, int lane) {
    if constexpr (FP4 && D < 256) {  // the lane's half of its group
      const int by = (lane & 1) * (D == 64 ? 8 : 16);
#pragma unroll
      for (int i = 0; i < VW; ++i) vq[i] >>= by;
    }
    if constexpr (FP4) {
      // element j of two neighbouring tokens in one byte: even elements from the low
      // nibbles, odd ones from the high ones
      constexpr uint32_t L = 0x0f0f0f0fu;
      if constexpr (D == 64) {  // (a word: one byte of a token, one byte of the next above 16 bits)
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const uint32_t a = vq[i], b = a >> 16, even = (a & 0xfu) | (b << 4 & 0xf0u), odd = (a >> 4 & 0xfu) | (b & 0xf0u);
          vq[i] = even | odd << 8;
        }
      } else {
        constexpr int Q = VW / 4;  // words of a token
#pragma unroll
        for (int i = 0; i < 2; ++i)
#pragma unroll
          for (int j = 0; j < Q; ++j) {
            const uint32_t a = vq[2 * i * Q + j], b = vq[(2 * i + 1) * Q + j];
            vq[2 * i * Q + j] = (a & L) | (b << 4 & ~L);
            vq[(2 * i + 1) * Q + j] = (a >> 4 & L) | (b & ~L);
          }
      }
    }
    if (left < kBN) {
      const int n = min(max(left - 4 * quad_of(wave, lane), 0), 4);
      if constexpr (FP4) {
        vs[0] = n >= 4 ? vs[0] : vs[0] & ((1u << (8 * n)) - 1u);
      } else {
        vs[0] &= n >= 2 ? ~0u : n == 1 ? 0xffffu : 0u;
        vs[1] &= n >= 4 ? ~0u : n == 3 ? 0xffffu : 0u;
      }
    }
  }
  __device__ __forceinline__ void put_value(int n, uint8_t* vt, int wave, int lane) const {
    const int quad = quad_of(wave, lane);
    uint32_t c[4];
    if constexpr (FP4) {
#pragma unroll
      for (int k = 0; k < 4; ++k) {  // elements 2n (k < 2), 2n + 1 of tokens 0, 1 or 2, 3
        constexpr int Q = VW / 4;
        const v2h e = D == 64 ? fp4_pair(vq[k & 1], k >> 1) : fp4_pair(vq[(2 * (k & 1) + (k >> 1)) * Q + n / 4], n % 4);
        c[k] = bits(e * fp8_pair(vs[0], k & 1));
      }
    } else {
#pragma unroll
      for (int k = 0; k < 4; ++k) c[k] = bits(i8_pair(vq[2 * n + (k >> 1)] ^ 0x80808080u, k & 1) * halves(vs[k & 1]));
    }
    *reinterpret_cast<uint4*>(vt + quad * (8 * D) + vswz<D>(quad, lane % QL * N + n) * 16) = make_uint4(c[0], c[1], c[2], c[3]);
  }
  // Piece p: the keys' first.
  __device__ __forceinline__ void put(int p, uint8_t* kt, uint8_t* vt, int wave, int lane) const {
    if (p < N) put_key(p, kt, wave, lane);
    else put_value(p - N, vt, wave, lane);
  }
};

// 16-bit caches need no decoding: straight from global memory into LDS, lane i of a load
// filling the 16 bytes at slot i with the chunk that belongs there.
template <int D, int W>
struct Codes<MOE_FMT_BF16, D, W> {
  static constexpr int CPR = D / 8;  // loads of 1 KB: of keys, and as many of values
  static constexpr int N = CPR / W, PIECES = 0;
  __device__ __forceinline__ void put(int, uint8_t*, uint8_t*, int, int) const {}
  static_assert(CPR % W == 0, "waves share the loads evenly");
  __device__ __forceinline__ static void load(Rsrc r, uint8_t* lds, uint32_t at, uint32_t base) {
#if defined(__HIP_DEVICE_COMPILE__)
    __builtin_amdgcn_raw_ptr_buffer_load_lds(r, (__attribute__((address_space(3))) void*)lds, 16, at, base, 0, 0);
#endif
  }
  __device__ __forceinline__ static void keys(const Place& from, uint8_t* kt, int wave, int lane) {
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const int wi = i * W + wave, slot = wi * 64 + lane, row = slot / CPR;
      const Unit32 u = from.of(wi * 64 / CPR);
      load(u.rsrc(), kt + wi * 1024, (u.o + (row & 31)) * (2 * D) + swz<D>(row, slot % CPR) * 16, 0);
    }
  }
  __device__ __forceinline__ static void values(const Place& from, const KvLayout lay, uint8_t* vt, int wave, int lane) {
    constexpr int CPQ = D / 2;  // chunks of a quad
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const int wi = i * W + wave, slot = wi * 64 + lane, quad = slot / CPQ;
      const Unit32 u = from.of(4 * (wi * 64 / CPQ));
      load(u.rsrc(), vt + wi * 1024, (u.o / 4 + (quad & 7)) * (8 * D) + vswz<D>(quad, slot % CPQ) * 16, lay.vq);
    }
  }
};

// The rows of a wave against tiles whose values lie as quads.  HALF: codes were decoded to
// fp16; the maximum is then held less kRaise (log2), so that weights are 2^15 at most and
// vanish only below 2^-32 of the largest.
template <int D, bool HALF>
struct ChunkRows : TileRows<D, HALF> {
  static constexpr float kRaise = HALF ? 7.0f : 0.0f;
  static constexpr int KS = D / 16, NJ = D / 32;
  using TileRows<D, HALF>::qf;
  using TileRows<D, HALF>::o;
  using TileRows<D, HALF>::h;
  using TileRows<D, HALF>::m;
  using TileRows<D, HALF>::l;
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
      for (int s = 0; s < KS; ++s) {
        x[t] = mma<HALF>(key(kt, t, s), qf[s], x[t]);
        if (s % 4 == 3) __builtin_amdgcn_sched_barrier(0);  // (few fragments at a time)
      }
    }
  }
  // bf16 -> fp16, scaled by the power of two that puts the row's largest magnitude into
  // [2^14, 2^15): exact for values above 2^-29 of it (of rows whose largest one is below
  // 2^-82, less, which no score shows).  Returns what undoes it.
  __device__ __forceinline__ float halve() {
    uint32_t top = 0;
#pragma unroll
    for (int s = 0; s < KS; ++s)
#pragma unroll
      for (int i = 0; i < 4; ++i) top = max(top, max(qf[s][i] & 0x7fffu, (qf[s][i] >> 16) & 0x7fffu));
    const auto both = __builtin_amdgcn_permlane32_swap(top, top, false, false);
    const int e = min(max(141 - (int)(max(both[0], both[1]) >> 7), -113), 96);
    const float up = __uint_as_float((uint32_t)(127 + e) << 23);
#pragma unroll
    for (int s = 0; s < KS; ++s)
#pragma unroll
      for (int i = 0; i < 4; ++i)
        qf[s][i] = bits(v2h{(_Float16)(__uint_as_float(qf[s][i] << 16) * up),
                            (_Float16)(__uint_as_float(qf[s][i] & 0xffff0000u) * up)});
    return __uint_as_float((uint32_t)(127 - e) << 23);
  }
  // A new maximum for the rows whose weights would leave 2^kGrow with the largest scaled
  // score mx (the others' answers do not depend on them, bit for bit).
  __device__ __forceinline__ void raise(float mx) {
    if (__any(mx > m + (kRaise + kGrow))) {
      const float mn = mx > m + (kRaise + kGrow) ? mx - kRaise : m, al = __builtin_amdgcn_exp2f(m - mn);
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
  // rows that see it.  (The weights are in the rows' sums already.)
  __device__ __forceinline__ void gather_seen(const uint8_t* kt, const uint8_t* vt, int64_t t0, float c) {
    v16f x[2];
    v4u p[4];
    scores(kt, x);
    this->mask(x, t0);
    const float sum = l;
#pragma unroll
    for (int v = 0; v < 32; ++v) this->weight(x, c, p, v);
    l = sum;
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
          z = mma<HALF>(one, p[s], z);
#pragma unroll
          for (int i = 0; i < 16; ++i) o[j][i] += seen ? z[i] : 0.0f;
        }
      }
  }
};

// Whether a tile of values in LDS holds an infinity or a NaN.
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

// Tile t's scores are computed while the weights of tile t - 1 go through the exponential
// and, in the shadow of the same matrix instructions, the codes of keys t + 2 and values
// t + 1 are decoded into the LDS buffers that were read before; those of two tiles further
// on are on their way meanwhile.
template <int FMT, int D, int W>
__global__ __launch_bounds__(64 * W, D <= 128 ? 2 : 1) void k_attn_chunk(SplitArgs a) {
  constexpr int KS = D / 16, NJ = D / 32, SIZE = 32 * W, TILE = kBN * D * 2;
  constexpr bool DECODED = FMT != MOE_FMT_BF16;
  __shared__ __align__(16) uint8_t k_even[TILE], k_odd[TILE], v_even[TILE], v_odd[TILE];
  __shared__ int wild_even[W], wild_odd[W];  // what each wave found among the values it decoded
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int lane = lane_id(), n = lane & 31;
  Item it = find_item<true>(a.s, a.T, a.G, SIZE, a.n_kv, a.room, a.S, (int)blockIdx.x, a.rounds);
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
  ChunkRows<D, DECODED> w;
  const int slot = (it.tile * W + wave) * 32 + n, last_slot = inside * a.G - 1;
  const int mine = min(slot, last_slot), row = (int)((uint32_t)mine / (uint32_t)a.G);
  const int64_t at = (int64_t)(r0 + row);
  const int head = kvh * a.G + mine - row * a.G;
  w.limit = slot <= last_slot ? (int64_t)len - rows + row : -1;
  const uint16_t* qp = a.q + at * a.q_stride + (int64_t)head * D + 8 * (lane >> 5);
#pragma unroll
  for (int s = 0; s < KS; ++s) w.qf[s] = *reinterpret_cast<const v4u*>(qp + 16 * s);
  // (above 0, where masked scores, -inf, would become NaN; scores that far down are 0)
  const float c_log2 = DECODED ? fmaxf(a.scale_log2 * w.halve(), 0x1p-126f) : a.scale_log2;
  w.places(lane);
  w.clear();
  // last token that some row of the wave sees
  const int wave_row = (int)((uint32_t)min((it.tile * W + wave) * 32 + 31, last_slot) / (uint32_t)a.G);
  const int64_t hi_wave = (it.tile * W + wave) * 32 <= last_slot ? (int64_t)len - rows + wave_row : -1;

  // Pages of 64 units at a time, one a lane: -1 where the table or the pool has none, and
  // from the last token that is looked at on.  Rows that see a token of a page that is not
  // there have no answer.
  const int* const table = a.s.page_table + (int64_t)it.b * a.s.max_pages;
  int batch = u_begin, pages;
  const auto next_pages = [&] {
    const int64_t u = (int64_t)batch + lane, i = (u * 32) >> a.s.log2P;
    pages = -1;
    if (u < u_end && i < a.s.max_pages) pages = table[i];
    if ((unsigned)pages >= (unsigned)a.s.n_pages) pages = -1;
  };
  next_pages();
  const auto unit = [&](int u) {
    if (u - batch >= 64) {
      batch += 64;
      next_pages();
    }
    const int p = __builtin_amdgcn_readlane(pages, u - batch);
    if (p < 0 && u < u_end && w.limit >= (int64_t)u * 32) w.l = __uint_as_float(0x7fc00000u);
    return Unit32{heads + (size_t)max(p, 0) * page_bytes, p < 0 ? 0 : (int)lay.head, (u * 32) & (P - 1)};
  };
  const auto place = [&](int t) { return Place{unit(2 * t), unit(2 * t + 1)}; };
  const int first = u_begin / 2, end = (u_end + 1) / 2;
  // tiles before this one are seen by all rows
  const int full = (int)min(max((plan.lo + 1) >> 6, (int64_t)0), (int64_t)end);
  const auto left_of = [&](int t) { return (int)min(plan.hi + 1 - (int64_t)t * kBN, (int64_t)kBN); };

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

  // Whether a tile of values holds an infinity or a NaN.
  const auto is_wild = [&](const uint8_t* vt, const int* found) {
    if constexpr (!DECODED) return wild<D>(vt, lane);
    int any = 0;
#pragma unroll
    for (int i = 0; i < W; ++i) any |= found[i];
    return any != 0;
  };
  bool some_wild = false;
  typedef Codes<FMT, D, W> C;
  const auto put_all = [&](const C& c, uint8_t* kt, uint8_t* vt) {
    each<0, C::PIECES>([&](auto p) { c.put(p(), kt, vt, wave, lane); });
  };
  if (first < end) {
    // What an even and what an odd turn decode, fetched two turns ahead; heads of 256 have
    // registers for one.
    constexpr bool TWO = D <= 128;
    C c_even, c_two;
    C& c_odd = TWO ? c_two : c_even;
    Place next;  // of the keys fetched last: the values' one turn later
    // In a tile that not every row sees, infinities and NaN are looked for.
    const auto look = [&](const C& c, int t, int* found) {
      if constexpr (DECODED) {
        if (t < full) return;
        const bool any = __any(c.wild());
        if (lane == 0) found[wave] = any;
      }
    };
    // keys of tile t, values of tile t - 1
    const auto fetch = [&](C& c, int t, uint8_t* kt, uint8_t* vt) {
      const Place before = next;
      next = place(t);
      if constexpr (DECODED) {
        c.fetch_keys(next, lay, wave, lane);
        c.fetch_values(before, lay, P, wave, lane);
      } else {
        c.keys(next, kt, wave, lane);
        c.values(before, lay, vt, wave, lane);
      }
    };
    // The first tile's keys and values, the second one's keys; what the first two turns
    // decode (16 bits: load).
    const Place p0 = place(first);
    next = place(first + 1);
    if constexpr (DECODED) {
      C c0;
      c0.fetch_keys(p0, lay, wave, lane);
      c0.fetch_values(p0, lay, P, wave, lane);
      c_odd.fetch_keys(next, lay, wave, lane);
      c0.arrange_values(left_of(first), wave, lane);
      look(c0, first, wild_even);
      put_all(c0, k_even, v_even);
      each<0, C::N>([&](auto p) { c_odd.put(p(), k_odd, v_odd, wave, lane); });
      fetch(c_even, first + 2, nullptr, nullptr);
      if constexpr (TWO) fetch(c_odd, first + 3, nullptr, nullptr);
    } else {
      C::keys(p0, k_even, wave, lane);
      C::values(p0, lay, v_even, wave, lane);
      C::keys(next, k_odd, wave, lane);
      wait_loads<0>();
    }
    __syncthreads();
    v16f x[2];
    w.scores(k_even, x);
    if (first >= full) w.mask(x, (int64_t)first * kBN);
    w.raise(w.top(x, c_log2));

    // Turn t: x holds tile t's scores, which the maxima cover, k1 the keys of t + 1, v0 the values of t; the keys
    // of t + 2 go to k0, the values of t + 1 to v1.
    const auto begin = [&](int t, C& c, uint8_t* k0, uint8_t* v0, uint8_t* v1, int* found) {
      if constexpr (!DECODED) wait_loads<0>();
      __syncthreads();  // what this turn reads is there, what it overwrites has been read
      if constexpr (DECODED) {
        c.arrange_values(left_of(t + 1), wave, lane);
        look(c, t + 1, found);
      } else {
        clear_behind(t, v0);
        fetch(c, t + 2, k0, v1);
      }
    };
    const auto finish = [&](int t, C& c, const v16f (&y)[2]) {
      x[0] = y[0];
      x[1] = y[1];
      if constexpr (DECODED) fetch(c, t + (TWO ? 4 : 3), nullptr, nullptr);
    };
    const auto step = [&](int t, C& c, uint8_t* k0, uint8_t* k1, uint8_t* v0, uint8_t* v1, int* f1) {
      begin(t, c, k0, v0, v1, f1);
      v16f y[2];
      float most = -__builtin_inff();
      w.template stream<true>([&](int h, int s) { return w.key(k1, h, s); }, [&](int s, int j) { return w.value(v0, s, j); },
                              c_log2, x, y, [&](auto I) {
        constexpr int N = 2 * KS + 4 * NJ, i = I();
        each<C::PIECES * i / N, C::PIECES * (i + 1) / N>([&](auto p) { c.put(p(), k0, v1, wave, lane); });
        // the next scores' maximum, beside the second product
        constexpr int F = 2 * KS + 1, L = N - F;
        if constexpr (i >= F)
#pragma unroll
          for (int v = 32 * (i - F) / L; v < 32 * (i - F + 1) / L; ++v) most = fmaxf(most, y[v >> 4][v & 15]);
      });
      w.raise(w.over_halves(most) * c_log2);
      finish(t, c, y);
    };
    // Tiles that not every row sees, and the last ones: a wave leaves out those none of its
    // rows does.
    const auto edge_step = [&](int t, C& c, uint8_t* k0, uint8_t* k1, uint8_t* v0, uint8_t* v1, int* f0, int* f1) {
      begin(t, c, k0, v0, v1, f1);
      const int64_t t0 = (int64_t)t * kBN;
      v16f y[2];
      put_all(c, k0, v1);
      if (t0 <= hi_wave) {
        uint32_t keep = ~0u;
        if (t >= full && is_wild(v0, f0)) {
          keep = 0u;  // (left for later)
          some_wild = true;
        }
        w.template stream<false>([&](int, int) { return v4u{0, 0, 0, 0}; },
                                 [&](int s, int j) { return w.value(v0, s, j) & keep; }, c_log2, x, y, [](auto) {});
      }
      if (t + 1 < end && t0 + kBN <= hi_wave) {
        w.scores(k1, y);
        if (t + 1 >= full) w.mask(y, t0 + kBN);
        w.raise(w.top(y, c_log2));
      }
      finish(t, c, y);
    };
    // (waves without a row, in tiles of few, only decode)
    const int all = hi_wave < 0 ? first : full;
    int t = first;
#pragma unroll 1
    for (; t + 2 < all; t += 2) {
      step(t, c_even, k_even, k_odd, v_even, v_odd, wild_odd);
      step(t + 1, c_odd, k_odd, k_even, v_odd, v_even, wild_even);
    }
#pragma unroll 1
    for (; t < end; t += 2) {
      edge_step(t, c_even, k_even, k_odd, v_even, v_odd, wild_even, wild_odd);
      if (t + 1 < end) edge_step(t + 1, c_odd, k_odd, k_even, v_odd, v_even, wild_odd, wild_even);
    }
  }
  // Tiles with infinities or NaN among values that some row may not see, once more.
  if (__syncthreads_or(some_wild)) {
    batch = 2 * max(first, full);
    next_pages();
#pragma unroll 1
    for (int t = max(first, full); t < end; ++t) {
      const Place from = place(t);
      __syncthreads();
      if constexpr (DECODED) {
        C c;
        c.fetch_keys(from, lay, wave, lane);
        c.fetch_values(from, lay, P, wave, lane);
        c.arrange_values(left_of(t), wave, lane);
        wild_even[wave] = __any(c.wild());
        put_all(c, k_even, v_even);
        __syncthreads();
      } else {
        C::keys(from, k_even, wave, lane);
        C::values(from, lay, v_even, wave, lane);
        wait_loads<0>();
        __syncthreads();
        clear_behind(t, v_even);
      }
      if ((int64_t)t * kBN <= hi_wave && is_wild(v_even, wild_even)) w.gather_seen(k_even, v_even, (int64_t)t * kBN, c_log2);
    }
  }
  w.finish();
  if (slot > last_slot) return;
  if (lane < 32 && sp == 0 && a.S > 1) a.part_n[at * a.n_q + head] = it.splits;
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
  int S, room, likely, rounds;
  int64_t items;
};
constexpr int chunk_waves(int D) { return D <= 128 ? 8 : 4; }
Shape shape_of(int D, int n_kv, int n_q, int n_seq, int64_t T, int64_t max_len) {
  const int G = n_q / n_kv, size = 32 * chunk_waves(D);
  const int64_t units = (std::min(max_len, (int64_t)INT32_MAX) + 31) / 32;  // (lengths are 32-bit)
  const int64_t per_seq = (T + n_seq - 1) / n_seq;
  const int64_t tiles = T * G / size + n_seq;  // at most: one part tile a sequence
  const int64_t base = (int64_t)n_seq * n_kv * ((per_seq * G + size - 1) / size);
  Shape r;
  int64_t S = ((int64_t)256 << 20) / (T * n_q * D * 4);
  S = std::min({S, (int64_t)kMaxSplit, (units + kWaves - 1) / kWaves});
  r.room = std::max(256 / n_kv, 1);
  // (of one sequence it is known whether fit_chunk will split it)
  const int64_t once = std::max((tiles * units + r.room - 1) / r.room, (int64_t)kWaves) + 2 * kStart;
  const bool whole = n_seq == 1 && tiles <= r.room && units + kStart <= once;
  r.S = T * n_q > kChunkPairs || S < 2 || (n_seq == 1 && base >= 512) || units <= 8 || whole ? 1 : (int)S;
  r.likely = (int)std::min({std::max(units / kWaves, (int64_t)1), std::max(256 / base, (int64_t)1), (int64_t)r.S});
  // Workgroups without an item take their place on a CU too, 5 to 7 us for a round of them: a
  // second one only where it may save more (900 rows beside 6 slots of one, behind 11000 to
  // 17000 tokens, 326 us, with it 281; 130 rows over five slots behind 5000 46, with it 52).
  r.rounds = tiles <= r.room && tiles * units < (int64_t)240 * r.room ? 1 : 2;
  r.items = r.S == 1 ? tiles : n_seq > 64 ? tiles + r.room + 1 : std::max(tiles, (int64_t)r.rounds * r.room);
  return r;
}

template <int FMT>
void launch_chunk(const SplitArgs& a, int D, unsigned grid, hipStream_t stream) {
  if (D == 64) k_attn_chunk<FMT, 64, chunk_waves(64)><<<grid, 64 * chunk_waves(64), 0, stream>>>(a);
  else if (D == 128) k_attn_chunk<FMT, 128, chunk_waves(128)><<<grid, 64 * chunk_waves(128), 0, stream>>>(a);
  else k_attn_chunk<FMT, 256, chunk_waves(256)><<<grid, 64 * chunk_waves(256), 0, stream>>>(a);
}

// A few splits are joined by a wave (512 mixed rows of 24 heads, 4 to 6 splits each: 90 us with
// both launches; a workgroup for each row and head, 97).
template <int D>
void join(const SplitArgs& a, hipStream_t stream) {
  if (a.likely > 16) launch_join<D>(a, stream);
  else k_attn_join_heads<D, D == 64 ? 4 : 8><<<(unsigned)((a.T * a.n_q + 3) / 4), 256, 0, stream>>>(a);
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
                    n_q, c->n_kv, n_q / c->n_kv, sp.S, sp.room, sp.likely, sp.rounds,
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
    case 64: join<64>(a, stream); break;
    case 128: join<128>(a, stream); break;
    default: join<256>(a, stream);
  }
  return hipGetLastError();
}

}  // namespace moe
