// Pieces shared by the attention kernels: which slots an item sees, the split of the work over
// the CTAs, and the asynchronous copies.
#pragma once

#include <type_traits>

#include "cache_device.cuh"
#include "specdec_device.cuh"

namespace specdec {

constexpr int kStep = 16;                 // slots of a step
constexpr int kUnit = 8;                  // steps of a unit of the work split
// What an item counts for in the split besides its units: its queries' way in, its last tile's and its
// rows' way out take about as long.  0, 3, 4 and 8 measured (16 bits, 32 query and 8 key heads of 128, us):
// B=64, 600 slots, one token 46.5, 40.6, 40.6, 42.3; B=32, 2000 slots, 24 tokens 58.4, 52.4, 52.2, 55.3;
// B=64, 4000 slots, 8 tokens 127, 122, 123, 129; 24 trees of 64 nodes, 12000 slots 217, 205, 200, 200; 4-bit
// pages, B=64, 4000 slots, 24 tokens 184, 171, 163, 151.  Fewer items than CTAs, 0 and 4: B=1, a prompt of
// 1024 tokens 47.2, 42.2; B=2, 64 nodes over 5000 slots 58.7, 48.4; B=16, one token, 4000 slots 43.5, 39.5;
// B=1, one token, 2400 slots (a unit for each CTA) 16.0, 17.0, 32000 slots 36.7, 37.3.
constexpr int kItemUnits = 4;
constexpr float kLn2 = 0.6931471805599453f;
// A row's weights are 2^(s - m), m its reference.  In fp16 they keep their 11 bits down to 2^-14 and vanish
// below 2^-25, so there the reference stays 7 below the largest score: the weights reach 2^7 (2^15 where the
// reference lags), what vanishes is below 2^-32 of the largest, and many small weights beside a large one
// count in the product with V as they do in the sum.  (Sums, products and lse follow the reference.)
template <typename M>
constexpr float kBelow = std::is_same<M, __half>::value ? 7.f : 0.f;

// 16 (or 8, 4) bytes to shared memory, zeros where `there` is false (src is not read then).
template <int N>
__device__ __forceinline__ void copy_async(uint32_t dst, const void* src, bool there) {
  const int n = there ? N : 0;
  if constexpr (N == 16)
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(n) : "memory");
  else
    asm volatile("cp.async.ca.shared.global [%0], [%1], %2, %3;" ::"r"(dst), "l"(src), "n"(N), "r"(n) : "memory");
}
__device__ __forceinline__ void copy_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void copy_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// A row's query: row / G as a product (exact for rows below 2^24 and G below 2^16).
__device__ __forceinline__ int query_of(const AttendParams& P, int row) {
  return static_cast<int>((static_cast<uint64_t>(row) * P.g_magic) >> 40);
}

// ---- the work split ---------------------------------------------------------------------

// The visible slots of an item as steps of 16: `sink_steps` from slot 0, then from step
// `first_step` on, up to slot `end`.
struct Range {
  int sink_steps, first_step, steps, end;
  int lo, sinks;  // no query of the item sees a slot in [sinks, lo)
  __device__ __forceinline__ int slot(int step) const {
    return (step < sink_steps ? step : step - sink_steps + first_step) * kStep;
  }
};
__device__ __forceinline__ Range item_range(const AttendParams& P, const SeqLen& S, int row0, int rows) {
  Range r{0, 0, 0, 0, 0, 0};
  const int i0 = query_of(P, row0), i1 = min(query_of(P, row0 + rows - 1), S.nq - 1);
  if (!S.ok || i0 > i1) return r;
  const bool tree = P.tree_mask != nullptr;
  r.end = tree ? S.len : S.first + i1 + 1;
  int lo = 0;
  if (P.window > 0) lo = max(0, (tree ? S.first : S.first + i0) - (P.window - 1));
  r.lo = lo;
  r.sinks = min(P.sinks, lo);
  r.sink_steps = (r.sinks + kStep - 1) / kStep;
  r.first_step = lo / kStep;
  if (r.sink_steps >= r.first_step) r.sink_steps = r.first_step = 0;
  r.steps = r.sink_steps + (r.end + kStep - 1) / kStep - r.first_step;
  return r;
}
// A node's depth; a tree of n nodes is at most n - 1 deep, which the tests of whole steps use.
__device__ __forceinline__ int node_depth(const AttendParams& P, int i) {
  return min(max(__ldg(P.depth + i), 0), P.n - 1);
}
// Whether query i of a sequence whose lengths fit sees any slot: tells a row whose visible scores are
// all -inf (its softmax has no value: NaN) from one that sees nothing (zeros).  Asked where a row's
// weights sum to 0.
__device__ __forceinline__ bool sees_some(const AttendParams& P, int first, int nq, int i) {
  if (i >= nq) return false;
  if (P.tree_mask == nullptr) return true;  // itself
  auto position = [&](int j) { return first + (P.depth ? node_depth(P, j) : j); };
  const int pos = position(i);
  auto near = [&](int p) { return P.window == 0 || pos - p < P.window || p < P.sinks; };
  if (first > 0 && (near(first - 1) || near(0))) return true;  // the last slot before the tree, or the first one
  for (int j = 0; j < nq; ++j)
    if (__ldg(P.tree_mask + static_cast<int64_t>(i) * P.n + j) != 0 && near(position(j))) return true;
  return false;
}
template <int MR>
__device__ __forceinline__ int tile_rows(const AttendParams& P, int rt) { return min(MR, P.n * P.G - rt * MR); }

// Units of one key head's row tiles of a sequence: at least one each, so that every row is
// written by somebody, and kItemUnits more.  Those come last, hold no work, and no cut falls
// among them: a border there counts as the item's end.
template <int MR>
__device__ __forceinline__ int item_units(const AttendParams& P, const SeqLen& S, int rt) {
  const Range r = item_range(P, S, rt * MR, tile_rows<MR>(P, rt));
  return max(1, (r.steps + kUnit - 1) / kUnit) + kItemUnits;
}
// The CTAs make P.tracks rows of as many, each with its share of the key heads: CTA c is number
// c / tracks of row c % tracks.  (One row, or one for each key head: the heads of a sequence are then read
// side by side.)  A CTA's range of its row's units and the item it starts in.  scan(): all threads of the CTA call it, with
// shared memory for one int64_t per warp and three more.
struct Share {
  int64_t u, end;         // units [u, end) of all
  int64_t quota, extra;   // every CTA has quota units, the first `extra` one more
  int64_t first;          // first unit of the key heads' items of (b, rt)
  int b, rt, track, id;
};
template <int MR, int THREADS>
__device__ __forceinline__ Share scan_units(const AttendParams& P, int64_t slots, int64_t* sh) {
  constexpr int WARPS = THREADS / 32;
  const int tid = threadIdx.x, warp = tid / 32, lane = tid % 32;
  const int heads = P.tracks == 1 ? P.pages.kv_heads : 1, ctas = gridDim.x / P.tracks;
  // row tile rt of sequence b is number b * row_tiles + rt; thread t takes a run of them
  const int64_t all = static_cast<int64_t>(P.B) * P.row_tiles, per = (all + THREADS - 1) / THREADS;
  const int64_t lo_tile = min(all, tid * per), hi_tile = min(all, lo_tile + per);
  int b0 = 0, rt0 = 0;
  if (lo_tile < hi_tile) {
    b0 = P.row_tiles == 1 ? static_cast<int>(lo_tile) : static_cast<int>(lo_tile / P.row_tiles);
    rt0 = static_cast<int>(lo_tile - static_cast<int64_t>(b0) * P.row_tiles);
  }
  // calls f(b, rt, units) for the run until it says stop
  auto each = [&](auto&& f) {
    int b = b0, rt = rt0;
    SeqLen S{};
    for (int64_t k = lo_tile; k < hi_tile; ++k) {
      if (k == lo_tile || rt == 0) S = seq_len(P.context_len, P.query_len, b, P.n, slots);
      if (!f(b, rt, item_units<MR>(P, S, rt))) return;
      if (++rt == P.row_tiles) {
        rt = 0;
        ++b;
      }
    }
  };
  int64_t mine = 0;
  each([&](int, int, int units) {
    mine += static_cast<int64_t>(units) * heads;
    return true;
  });
  int64_t incl = mine;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int64_t v = __shfl_up_sync(0xffffffffu, incl, o);
    if (lane >= o) incl += v;
  }
  if (lane == 31) sh[warp] = incl;
  __syncthreads();
  int64_t before = 0, total = 0;
#pragma unroll
  for (int w = 0; w < WARPS; ++w) {
    if (w < warp) before += sh[w];
    total += sh[w];
  }
  Share s;
  if (total >> 32 == 0) {
    s.quota = static_cast<uint32_t>(total) / ctas;
    s.extra = static_cast<uint32_t>(total) % ctas;
  } else {
    s.quota = total / ctas;
    s.extra = total % ctas;
  }
  s.id = blockIdx.x / P.tracks;
  s.track = blockIdx.x - s.id * P.tracks;
  const int64_t cta = s.id;
  s.u = cta * s.quota + min(cta, s.extra);
  s.end = s.id < ctas ? s.u + s.quota + (cta < s.extra ? 1 : 0) : s.u;
  int64_t lo = before + incl - mine;
  if (s.u < s.end && s.u >= lo && s.u < lo + mine)  // exactly one thread
    each([&](int b, int rt, int units) {
      const int64_t n = static_cast<int64_t>(units) * heads;
      if (s.u < lo + n) {
        const int64_t at = s.u - lo;
        const int left = units - static_cast<int>(at >> 32 == 0 ? static_cast<uint32_t>(at) % static_cast<uint32_t>(units) : at % units);
        sh[WARPS] = (static_cast<int64_t>(b) << 32) | rt;
        sh[WARPS + 1] = lo;
        sh[WARPS + 2] = s.u + (left <= kItemUnits ? left : 0);
        return false;
      }
      lo += n;
      return true;
    });
  __syncthreads();
  if (s.u < s.end) {
    s.b = static_cast<int>(sh[WARPS] >> 32);
    s.rt = static_cast<int>(sh[WARPS] & 0xffffffff);
    s.first = sh[WARPS + 1];
    s.u = sh[WARPS + 2];
  }
  return s;
}

// Walks the items of a CTA's range.
template <int MR>
struct Walk {
  const AttendParams& P;
  int64_t slots, u, end, item;
  int b, rt, h, h_lo, h_hi, units;  // h_lo .. h_hi - 1: the row's key heads
  SeqLen S;
  __device__ __forceinline__ Walk(const AttendParams& p, int64_t n, const Share& s)
      : P(p), slots(n), u(s.u), end(s.end), b(s.b), rt(s.rt) {
    S = seq_len(P.context_len, P.query_len, b, P.n, slots);
    units = item_units<MR>(P, S, rt);
    h_lo = s.track;
    h_hi = P.tracks == 1 ? P.pages.kv_heads : h_lo + 1;
    const int64_t at = u - s.first;
    const int k = at >> 32 == 0 ? static_cast<int>(static_cast<uint32_t>(at) / static_cast<uint32_t>(units)) : static_cast<int>(at / units);
    item = s.first + static_cast<int64_t>(k) * units;
    h = h_lo + k;
    if (h == h_hi) turn();
  }
  __device__ __forceinline__ void turn() {  // to the next row tile's items
    h = h_lo;
    if (++rt == P.row_tiles) {
      rt = 0;
      ++b;
      S = seq_len(P.context_len, P.query_len, b, P.n, slots);
    }
    units = item_units<MR>(P, S, rt);
  }
  __device__ __forceinline__ int64_t seg_end() const { return min(end, item + units); }
  __device__ __forceinline__ bool ends() const { return seg_end() >= item + units - kItemUnits; }  // the item, in this segment
  __device__ __forceinline__ bool next() {  // false: the range is done
    u = seg_end();
    if (u >= end) return false;
    item += units;
    if (++h == h_hi) turn();
    return true;
  }
  // The entry of the workspace's split table for a segment that begins an item and does not
  // end it: the item and the number of CTAs that hold parts of it.
  __device__ __forceinline__ int4 split(const Share& s) const {
    const int64_t last = item + units - kItemUnits - 1, wide = s.extra * (s.quota + 1);
    const int64_t owner = last < wide ? last / (s.quota + 1) : s.extra + (last - wide) / s.quota;
    return make_int4(b, rt, h, static_cast<int>(owner - s.id + 1));
  }
};

// The rows of a segment whose WARPS warps left (unnormalised output, running maximum and sum) in shared memory,
// [WARPS][MR][D] and behind them [WARPS][MR]: written out where the segment is a whole item, else left as a part.
template <typename T, int D, int MR, int WARPS>
__device__ __forceinline__ void join_warps(const AttendParams& P, const Walk<MR>& w, const SeqLen& S, int row0, int rows, const char* smem) {
  const Pages& pg = P.pages;
  const int b = w.b, h = w.h;
  const float* const s_o = reinterpret_cast<const float*>(smem);
  const float2* const s_ml = reinterpret_cast<const float2*>(smem + WARPS * MR * D * 4);
  const bool begins = w.u == w.item, ends = w.ends();
  const int part = begins ? 1 : 0;  // a CTA has at most one part that goes on and one that began before
  for (int f = threadIdx.x; f < MR * (D / 4); f += 32 * WARPS) {
    const int r = f / (D / 4), d = (f % (D / 4)) * 4;
    if (r >= rows) continue;
    float m = -kInf;
#pragma unroll
    for (int k = 0; k < WARPS; ++k) m = fmaxf(m, s_ml[k * MR + r].x);
    const float base = m == -kInf ? 0.f : m;
    float l = 0.f;
    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
    for (int k = 0; k < WARPS; ++k) {
      const float2 ml = s_ml[k * MR + r];
      const float a = ex2(ml.x - base);
      const float4 x = *reinterpret_cast<const float4*>(s_o + (static_cast<size_t>(k) * MR + r) * D + d);
      l += a * ml.y;
      acc.x += a * x.x; acc.y += a * x.y; acc.z += a * x.z; acc.w += a * x.w;
    }
    if (begins && ends) {
      const int i = query_of(P, row0 + r), head = h * P.G + row0 + r - i * P.G;
      const int64_t at = (static_cast<int64_t>(b) * P.n + i) * P.Hq + head;
      float inv = l == 0.f ? 0.f : pg.v_scale / l, lse = m * kLn2 + logf(l);
      if (l == 0.f || i >= S.nq) { lse = -kInf; inv = 0.f; }
      uint2 four = make_uint2(Half16<T>::pack(acc.x * inv, acc.y * inv), Half16<T>::pack(acc.z * inv, acc.w * inv));
      if (i >= S.nq) four = make_uint2(0u, 0u);
      if (!S.ok || (l == 0.f && sees_some(P, S.first, S.nq, i))) {
        four = make_uint2(0x7fff7fffu, 0x7fff7fffu);
        lse = __int_as_float(0x7fffffff);
      }
      *reinterpret_cast<uint2*>(static_cast<T*>(P.out) + at * D + d) = four;
      if (d == 0 && P.lse) P.lse[at] = lse;
    } else {
      const int64_t at = (static_cast<int64_t>(blockIdx.x) * 2 + part) * MR + r;
      *reinterpret_cast<float4*>(P.part_o + at * D + d) = acc;
      if (d == 0) P.part_ml[at] = make_float2(m, l);
    }
  }
}

// ---- the warp-level kernels' matrix instruction ---------------------------------------------

template <typename T>
__device__ __forceinline__ void mma(float (&d)[4], const uint4& a, uint32_t b0, uint32_t b1) {
  if constexpr (sizeof(T) == 2 && std::is_same<T, __nv_bfloat16>::value)
    asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                 : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3]) : "r"(a.x), "r"(a.y), "r"(a.z), "r"(a.w), "r"(b0), "r"(b1));
  else
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                 : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3]) : "r"(a.x), "r"(a.y), "r"(a.z), "r"(a.w), "r"(b0), "r"(b1));
}

}  // namespace specdec
