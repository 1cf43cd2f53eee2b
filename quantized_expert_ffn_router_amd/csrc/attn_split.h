// attn_split.h -- how the attention over the cache is cut into work items, and how the
// parts of a split sequence are joined.
#pragma once

#include "attn_common.h"

namespace moe {

namespace {

constexpr int kWaves = 4;           // units a chunk is a multiple of: a decode workgroup's waves

struct SplitArgs {
  const uint8_t* pool;
  const uint16_t* q;
  uint16_t* out;
  float* part_o;   // [T * n_q][S][D]
  float2* part_ml; // [T * n_q][S]
  int* part_n;     // [T * n_q]: splits (1: the output is there already)
  int64_t q_stride, out_stride, T;
  SeqView s;
  int n_q, n_kv, G, S, room, likely, rounds;
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
  bool light;  // a single tile, a quarter of it or less filled
  __device__ __forceinline__ LaneSeq(const SeqView& s, int i0, int64_t T, int G, int size) {
    const int i = min(i0 + lane_id(), s.n_seq - 1);
    start = max(s.row_start[i], 0);
    end = s.row_start[i + 1];
    len = s.kv_len[i];
    const int64_t n = i0 + lane_id() < s.n_seq ? min((int64_t)end, T) - start : 0;
    tiles = n > 0 ? (int)((uint32_t)((int)n * G + size - 1) / (uint32_t)size) : 0;
    light = n * G <= size / 4;
    units = n > 0 && len > 0 ? min((len - 1) / 32 + 1, units_of_table(s)) : 0;
  }
};

// The item of workgroup id.  S 1: sequences are not split.  chunk: a multiple of the
// waves, as small as keeps the items within `room` more than the tiles (what the grid
// holds), and kWhole units or more unless the 256 CUs need shorter ones (8 slots of
// 1000 to 60000 tokens: 33 us; as many chunks of each sequence as of any other, 37).
constexpr int kWhole = 4 * kWaves;

// The same for workgroups of which one fits a CU: as long as there are no more than 64
// sequences, the shortest chunks whose items fit the room (workgroups that run at once, of
// one key/value head) once, or up to `rounds` times, whichever is done first: a round
// lasts as long as its longest item, a chunk and what a workgroup needs before and behind
// it, about kStart units; joining costs as much again.
constexpr int kStart = 8;
// Units go faster where most waves only decode (8 slots of one row behind 16000 tokens 70 us,
// of 85 rows 116; over NVFP4 48 and 90): chunks of such sequences are half as long again, and
// those of a sequence as even as they come (512 mixed rows over Q8_0 119 -> 98 us; 1.75 times
// as long, and uneven, 103, and 513 rows beside 7 slots of one behind 8000 tokens 156, not 141).
__device__ __forceinline__ int chunk_of(int chunk, bool light) { return light ? (chunk + chunk / 2) & ~1 : chunk; }
__device__ __forceinline__ int fit_chunk(const LaneSeq& q, int most, int room, int rounds, int least) {
  const auto items = [&](int c) {
    return wave_sum((float)q.tiles * (float)(q.units ? (int)((uint32_t)(q.units - 1) / (uint32_t)chunk_of(c, q.light)) + 1 : 1));
  };
  const float work = wave_sum((float)q.tiles * (float)q.units * (q.light ? 2.0f / 3.0f : 1.0f));
  const int whole = max((most + 1) & ~1, 2);
  const float tiles = items(whole);
  int chunk = whole;
  float cost = ceilf(tiles / (float)room) * (float)(most + kStart);
  for (int k = 1; k <= rounds; ++k) {
    const float cap = (float)(k * room);
    if (tiles > cap) continue;
    int lo = max((int)fminf(work / cap, 0x1p30f) & ~1, max(least, kWaves)), hi = whole;  // (too many items below lo)
    while (hi - lo > max(lo / 16, 2)) {
      const int c = (lo + (hi - lo) / 2) & ~1;
      if (items(c) <= cap) hi = c;
      else lo = c;
    }
    if (lo < hi && items(lo) <= cap) hi = lo;
    const float needs = (float)k * (float)(hi + kStart) + (float)kStart;
    if (needs < cost) {
      cost = needs;
      chunk = hi;
    }
  }
  return chunk;
}

// FIT: see fit_chunk.
template <bool FIT = false>
__device__ __forceinline__ Item find_item(const SeqView& s, int64_t T, int G, int size, int n_kv,
                                          int room, int S, int id, int rounds = 1) {
  Item r;
  r.b = -1;
  r.chunk = INT32_MAX;
  const LaneSeq first(s, 0, T, G, size);
  const bool fit = FIT && S > 1 && s.n_seq <= 64;
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
    if (fit) {
      r.chunk = __builtin_amdgcn_readfirstlane(fit_chunk(first, most, room, rounds, ((most + S - 1) / S + 1) & ~1));
    } else {
      // (a sequence has less than 2^27 units: held to 2^30, it stays an int)
      int chunk = (int)fminf(ceilf(work / (float)room), 0x1p30f);
      if (chunk < kWhole) chunk = max(chunk, min((int)ceilf(work * n_kv / 256.0f), kWhole));
      chunk = (max(chunk, (most + S - 1) / S) + kWaves - 1) / kWaves * kWaves;
      r.chunk = max(__builtin_amdgcn_readfirstlane(chunk), kWaves);
    }
  }
  int before = 0;
  for (int i0 = 0; i0 < s.n_seq; i0 += 64) {
    const LaneSeq q = i0 ? LaneSeq(s, i0, T, G, size) : first;
    // (a row without tokens is answered too)
    const auto parts = [&](int chunk) {
      return S > 1 && q.units ? (int)((uint32_t)(q.units - 1) / (uint32_t)chunk) + 1 : 1;
    };
    int chunk = r.chunk, splits = parts(chunk);
    if (fit) {  // (as even as they come)
      splits = parts(chunk_of(chunk, q.light));
      chunk = max(((int)((uint32_t)(q.units + splits - 1) / (uint32_t)splits) + 1) & ~1, 2);
      splits = parts(chunk);
    }
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
    r.chunk = __builtin_amdgcn_readlane(chunk, l);
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

// Joins the splits of EL elements of one (row, head): weights exp2(m_s - M),
// added in a fixed order, so the result does not depend on scheduling.  EL / 4
// lanes hold the elements and 1024 / EL groups of them the splits, PER at a time
// each; the loads of as many as are likely start before their number is known.
constexpr int kMaxSplit = 256;

template <int D, int EL, int PER>
__global__ __launch_bounds__(256) void k_attn_join(SplitArgs a) {
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
void launch_join(const SplitArgs& a, hipStream_t stream) {
  const unsigned heads = (unsigned)(a.T * a.n_q);
  if (a.likely <= 32) k_attn_join<D, D, 32 * D / 1024><<<heads, 256, 0, stream>>>(a);
  else if (a.likely <= 64) k_attn_join<D, 32, 2><<<heads * (D / 32), 256, 0, stream>>>(a);
  else k_attn_join<D, 32, kMaxSplit / 32><<<heads * (D / 32), 256, 0, stream>>>(a);
}

// The same with a wave for a row and head, four of them a workgroup: D / 4 lanes hold the
// elements, 256 / D groups of them the splits, PER at a time.
template <int D, int PER>
__global__ __launch_bounds__(256) void k_attn_join_heads(SplitArgs a) {
  constexpr int LW = D / 4, NG = 64 / LW;
  const int lane = lane_id(), x = lane % LW, grp = lane / LW;
  const int64_t id = (int64_t)blockIdx.x * 4 + __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  if (id >= a.T * a.n_q) return;
  const int t = (int)((uint32_t)id / (uint32_t)a.n_q), h = (int)((uint32_t)id % (uint32_t)a.n_q);
  const int64_t at = id * a.S;
  int ns = a.part_n[id];
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
  const float down = __builtin_amdgcn_exp2f(M - all);
  o.x *= down; o.y *= down; o.z *= down; o.w *= down;
  L *= down;
#pragma unroll
  for (int d = LW; d < 64; d <<= 1) {
    o.x += __shfl_xor(o.x, d); o.y += __shfl_xor(o.y, d);
    o.z += __shfl_xor(o.z, d); o.w += __shfl_xor(o.w, d);
    L += __shfl_xor(L, d);
  }
  if (grp == 0) {
    const float inv = (int64_t)q.len - q.rows + (t - q.r0) < 0 ? 0.0f : 1.0f / L, ts = a.v_ts;
    uint16_t* d = a.out + t * a.out_stride + (int64_t)h * D + 4 * x;
    *reinterpret_cast<uint2*>(d) = make_uint2(bf16_pair(o.x * inv * ts, o.y * inv * ts),
                                              bf16_pair(o.z * inv * ts, o.w * inv * ts));
  }
}

}  // namespace

}  // namespace moe
