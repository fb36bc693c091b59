// Attention over pages on the tensor cores with accumulators in tensor memory.
//
// The formula, the items and the split of the work are those of attend.cu.  A tile is 128 query
// rows of one key head by 128 slots:
//   S = Q K^T  (tcgen05.mma, Q and K from shared memory)  -> 128 columns of tensor memory
//   P = 2^(c S - m)                                       -> back to tensor memory, 16 bits
//   O += P V   (tcgen05.mma, P from tensor memory)        -> D columns of tensor memory
// Two such streams ("slots" 0 and 1 of the CTA) take turns, so that one's exponentials run while
// the other's products do: with more than 128 rows per key head they are two row tiles that share
// every staged K and V tile; with fewer, both hold the same rows and take every other tile, and
// their results join at the end.
//
// A row's reference m moves only when a tile exceeds what it was set for by more than 2^8: the weights
// then stay below 2^8 (2^15 in fp16, whose reference is 7 lower, kBelow), where 16-bit rounding is relative,
// and the accumulator is rescaled once or twice per item instead of once per tile.  The sum l takes the
// unrounded weights, in fp32.  Two threads hold a row, 64 columns each: the chain scores -> weights -> products of a
// slot is what bounds a short tile, and this halves its longest link.
//
// Warps 0-15: rows (slot = warp / 8, columns = warp / 4 % 2, lanes = warp % 4).  Then the warps that
// bring K and V: of 16-bit pages, 4 that copy rows asynchronously, 16 bytes at a time; of 4-bit
// pages, 8 that turn copied codes into their fp16 values (exact: at most 6 significant bits).
// Either way the tiles are 128-byte-swizzled and gathered row by row, so pages may have any size
// and stride.  One warp issues the matrix instructions, one walks the items ahead of everybody, and
// two bring query rows and, of 4-bit pages, the codes and scales.  The roles meet at mbarriers; every
// wait is bounded.  Where one runs out, the walk publishes no further item, every role finishes the
// item it is in (without waiting) and leaves; the row warps, which also meet at thread barriers, agree
// at each item whether they go on.  The CTA reports it.
//
// Measured (32 query and 8 key heads of 128, key bytes against the copy rate, products against the
// matrix rate):
//  - 64 requests, 8 tokens, up to 8190 slots in 16 bits (32 rows to a key head): 219 us, 6.2 TB/s, 0.91 of
//    the measured copy rate; HBM bounds it.
//  - 24 trees of 64 nodes, up to 12000 slots (256 rows): 204 us, 3.7 TB/s and 0.92 PFLOP/s, 0.55 of the
//    measured copy and 0.48 of the matrix rate.  A pair of 128-by-128 tiles takes about 4200 clocks against 2050 of products: the chain scores,
//    weights, products of one slot is longer than the other slot's products, for the exponentials
//    (128 x 128 at 32 a clock and SM are 512 clocks) come with two reads of the scores and one store
//    of the weights through tensor memory.
//  - 16 requests, 8 tokens, up to 32003 slots in 4 bits: 164 us, 2.3 TB/s, DRAM traffic equal to the
//    cache's bytes.  A tile takes about 2400 clocks: its codes' conversion 790 at 64 lanes a clock, but
//    with the copies in and the stores of the values (shared memory is busy for about 1500) the converting
//    warps need 2000.
//  - 35 rows, a window of 1024 slots, 96 requests: 60 us, 3.5 TB/s: an item is 9 tiles, and its first,
//    partial tile, the way out of its rows and the next one's queries cost about 4 more.
#pragma once

#include "attend_common.cuh"

namespace specdec {

namespace tc {

constexpr int kRowWarps = 16;
constexpr int kTile = kUnit * kStep;  // 128 slots
constexpr int kBadRing = 16;          // tiles whose out-of-range slots are remembered
constexpr int kItems = 4;             // items the walk may be ahead
constexpr float kSlack = 8.f;         // log2 of how far a tile may exceed what the reference was set for

// What the roles need to know of an item, for the CTA's segment of it.
struct Item {
  int b, h, row0, rows;     // rows row0 .. row0 + rows - 1 of the key head
  int t_lo, tiles;          // this segment's tiles
  int begins, ends, last;   // of the item; last: the CTA's last item
  int nq, first, ok;
  int sink_steps, first_step, steps, end, lo, sinks;
  int whole_lo[2], whole_hi[2];  // tiles that every row of a slot sees whole
  int clean_lo, clean_hi;        // tiles that every row of the item sees whole: others' values are scanned
};

// Row tiles: 32 rows, each in the four quarters of tensor memory's lanes, or 128, or two of 128.
enum Rows { kQuad, kOne, kTwo };

template <int D, Rows ROWS, bool FOUR>
struct Shape {
  static constexpr bool TWO = ROWS == kTwo, QUAD = ROWS == kQuad;
  static constexpr int MR = QUAD ? 32 : TWO ? 256 : 128;
  static constexpr int kCopyWarps = FOUR ? 8 : 4;
  static constexpr int kThreads = 32 * (kRowWarps + kCopyWarps + 4);
  // Who is who among the warps from 16 on.  16-bit pages: 16 .. 19 copy.  4-bit pages: 16 .. 23 convert, two
  // on each of an SM's four schedulers (warp % 4); with at most 32 rows, where a tile's copies are the
  // longer way, they keep off the scheduler of the two warps that copy.  (B=16, 16000 slots, D=128, us for
  // 32, 64 and 256 rows: 103, 120 and 266 two on each, 99, 127 and 279 on three schedulers.)
  static constexpr bool THREE = FOUR && QUAD;
  static constexpr int kWalker = THREE ? 16 : FOUR ? 24 : 20, kMma = FOUR ? 27 : 23;
  static constexpr int kQuery0 = THREE ? 20 : FOUR ? 25 : 21, kQuery1 = THREE ? 24 : FOUR ? 26 : 22;
  __device__ static constexpr int copy_index(int warp) {
    const int k = warp - kRowWarps;
    if (THREE) return k % 4 == 0 || k > 10 || k < 0 ? -1 : k / 4 * 3 + k % 4 - 1;  // 17, 18, 19, 21, 22, 23, 25, 26
    return k >= 0 && k < kCopyWarps ? k : -1;
  }
  static constexpr int kTileBytes = kTile * D * 2;
  static constexpr int RK = D == 64 ? 4 : (TWO || FOUR ? 2 : 3), RV = D == 64 ? 4 : 2;  // K tiles and V tiles staged
  // 4-bit pages: a tile's codes and scales (of K, then of V), copied ahead of their conversion
  static constexpr int kRawCodes = kTile * (D / 2), kRawScales = kTile * (D / 16), kRawBytes = 2 * (kRawCodes + kRawScales);
  // where the 16-byte piece of a row of codes lies: turned by the row, so that 8 rows meet no bank conflict
  __device__ static constexpr int raw_piece(int row, int piece) { return piece ^ ((row >> (D == 128 ? 1 : 2)) & (D / 32 - 1)); }
  static constexpr int RAW = !FOUR ? 0 : D == 64 ? 3 : TWO ? 1 : QUAD ? 2 : 3;
  static constexpr int kOffK = (TWO ? 2 : 1) * kTileBytes;
  static constexpr int kOffV = kOffK + RK * kTileBytes;
  static constexpr int kOffMl = kOffV + RV * kTileBytes;      // [2][2][128] (m, l) of slots and halves
  static constexpr int kOffRaw = kOffMl + 4 * 128 * 8;
  static constexpr int kOffQScale = kOffRaw + RAW * kRawBytes;  // [2][MR] scales of query rows (4-bit pages)
  static constexpr int kOffSum = kOffQScale + (FOUR ? 2 * MR * 4 : 0);  // [4][4][32][8] accumulators on their way, [32] 1 / l
  static constexpr int kOffItem = kOffSum + (QUAD ? 4 * 4 * 32 * 8 * 4 + 32 * 4 : 0);
  static constexpr int kOffScan = kOffItem + kItems * sizeof(Item);
  static constexpr int kOffBad = (kOffScan + (kThreads / 32 + 3) * 8 + 15) / 16 * 16;
  static constexpr int kOffBar = kOffBad + kBadRing * 16;
  static constexpr int kBars = 2 * (RK + RV + RAW) + 2 + 2 + 2 + 2 + 2 * kItems + 1;
  static constexpr int kOffMisc = kOffBar + kBars * 8;
  static constexpr int kBytes = kOffMisc + 16;

  // Tensor memory's 512 columns: S of slots 0 and 1, then O.  With D = 64 there is room for the
  // weights beside the scores, and a slot's next scores need not wait for its products (AHEAD); with
  // D = 128 the weights of a slot take the place of its scores, each half's of its own.
  static constexpr bool AHEAD = D == 64;
  static constexpr int kHalfP = AHEAD ? 32 : 64;  // columns between the weights of a tile's halves
  __host__ __device__ static constexpr int o_column(int slot) { return 256 + slot * D; }
  __host__ __device__ static constexpr int p_column(int slot) { return AHEAD ? 384 + slot * 64 : slot * 128; }
};

// ---- tcgen05 -----------------------------------------------------------------------------

// Shared-memory matrix descriptors: 128-byte swizzle.  The low word holds the address and the
// leading stride, the high one the stride between groups of 8 rows (1024 bytes).
__device__ __forceinline__ constexpr uint32_t desc_low(uint32_t addr, uint32_t lead) { return (addr >> 4) | ((lead >> 4) << 16); }
constexpr uint32_t kDescHigh = (1024u >> 4) | (1u << 14) | (2u << 29);
// Instruction descriptor: fp32 accumulator, 16-bit operands, M = 128.
template <typename M>
__device__ __forceinline__ constexpr uint32_t instr_desc(int n, bool b_mn_major) {
  const uint32_t type = std::is_same<M, __nv_bfloat16>::value ? 1u : 0u;
  return (1u << 4) | (type << 7) | (type << 10) | (b_mn_major ? 1u << 16 : 0u) | (static_cast<uint32_t>(n >> 3) << 17) |
         ((128u >> 4) << 24);
}
__device__ __forceinline__ void mma_ss(uint32_t d, uint32_t a, uint32_t b, uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n.reg .pred p;\n.reg .b64 da, db;\nmov.b64 da, {%1, %5};\nmov.b64 db, {%2, %5};\nsetp.ne.u32 p, %4, 0;\n"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], da, db, %3, p;\n}" ::"r"(d), "r"(a), "r"(b), "r"(idesc), "r"(accumulate),
      "r"(kDescHigh)
      : "memory");
}
__device__ __forceinline__ void mma_ts(uint32_t d, uint32_t a, uint32_t b, uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n.reg .pred p;\n.reg .b64 db;\nmov.b64 db, {%2, %5};\nsetp.ne.u32 p, %4, 0;\n"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], db, %3, p;\n}" ::"r"(d), "r"(a), "r"(b), "r"(idesc), "r"(accumulate),
      "r"(kDescHigh)
      : "memory");
}
// The barrier is arrived at when every matrix instruction issued so far is complete.
__device__ __forceinline__ void mma_commit(uint64_t* bar) {
  asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(smem_addr(bar)) : "memory");
}
__device__ __forceinline__ void fence_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void fence_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }

// 16 columns of this warp's 32 lanes.  The values are there after tmem_load_wait, which takes
// them so that no use moves above it.
__device__ __forceinline__ void tmem_load(uint32_t addr, uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
        "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
      : "r"(addr)
      : "memory");
}
__device__ __forceinline__ void tmem_load_wait(uint32_t (&r)[16]) {
  asm volatile("tcgen05.wait::ld.sync.aligned;"
               : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]), "+r"(r[6]), "+r"(r[7]),
                 "+r"(r[8]), "+r"(r[9]), "+r"(r[10]), "+r"(r[11]), "+r"(r[12]), "+r"(r[13]), "+r"(r[14]), "+r"(r[15])::"memory");
}
__device__ __forceinline__ void tmem_store8(uint32_t addr, const uint32_t (&r)[8]) {
  asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"r"(addr), "r"(r[0]), "r"(r[1]),
               "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7])
               : "memory");
}
__device__ __forceinline__ void tmem_store16(uint32_t addr, const uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(addr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
      "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
      : "memory");
}
__device__ __forceinline__ void tmem_store_wait() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

// A bounded wait: gives up after kMaxWaitNs, and at once when the CTA has given up elsewhere.
__device__ __forceinline__ bool wait_for(uint64_t* bar, uint32_t parity, volatile int* gave_up) {
  if (mbar_try_wait(bar, parity)) return true;
  const uint64_t t0 = global_timer_ns();
  while (!mbar_try_wait(bar, parity)) {
    if (*gave_up) return false;
    if (global_timer_ns() - t0 > kMaxWaitNs) {
      *gave_up = 1;
      return false;
    }
  }
  return true;
}
// One lane of the warp (the same one every time).
__device__ __forceinline__ bool elect_one() {
  uint32_t yes;
  asm volatile("{\n.reg .pred p;\nelect.sync _|p, 0xffffffff;\nselp.u32 %0, 1, 0, p;\n}" : "=r"(yes)::"memory");
  return yes != 0;
}
// Whether all row threads say yes (the barrier of all of them).
__device__ __forceinline__ bool rows_all(bool mine) {
  uint32_t all;
  asm volatile("{\n.reg .pred p, q;\nsetp.ne.u32 q, %1, 0;\nbarrier.cta.red.and.pred p, 1, 512, q;\nselp.u32 %0, 1, 0, p;\n}"
               : "=r"(all) : "r"(mine ? 1u : 0u) : "memory");
  return all != 0;
}
// Whether either warp of a pair (64 threads) says yes.
__device__ __forceinline__ bool pair_any(int barrier, bool mine) {
  uint32_t any;
  asm volatile("{\n.reg .pred p, q;\nsetp.ne.u32 q, %2, 0;\nbarrier.cta.red.or.pred p, %1, 64, q;\nselp.u32 %0, 1, 0, p;\n}"
               : "=r"(any) : "r"(barrier), "r"(mine ? 1u : 0u) : "memory");
  return any != 0;
}

// Where the 16-byte piece `piece` of row `row` of a tile of 128 rows of D values lies: blocks
// of 64 values, rows of 128 bytes, pieces swizzled by the row.
__device__ __forceinline__ uint32_t tile_offset(int row, int piece) {
  return (piece >> 3) * (kTile * 128) + row * 128 + (((piece & 7) ^ (row & 7)) << 4);
}
__device__ __forceinline__ float max3(float a, float b, float c) {
  float y;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(y) : "f"(a), "f"(b), "f"(c));
  return y;
}
// Bits lo..hi-1 of a step's 16 slots, both clamped to 0..16.
__device__ __forceinline__ uint32_t bits16(int lo, int hi) {
  lo = min(max(lo, 0), kStep);
  hi = min(max(hi, 0), kStep);
  return hi > lo ? ((1u << hi) - 1u) & ~((1u << lo) - 1u) : 0u;
}
// Bits lo..hi-1 of 64 slots, both clamped to 0..64.
__device__ __forceinline__ uint64_t bits64(int lo, int hi) {
  const uint64_t below = hi >= 64 ? ~0ull : (1ull << max(hi, 0)) - 1;
  return lo >= 64 ? 0ull : below & (~0ull << max(lo, 0));
}

template <typename T, int D, Rows ROWS, bool FOUR>
__global__ void __launch_bounds__(Shape<D, ROWS, FOUR>::kThreads, 1) attend_tc_kernel(const AttendParams P) {
  using Sh = Shape<D, ROWS, FOUR>;
  using M = typename std::conditional<FOUR, __half, T>::type;  // the matrix instructions' type
  constexpr int MR = Sh::MR, RK = Sh::RK, RV = Sh::RV, KT = D / 16, THREADS = Sh::kThreads;
  constexpr bool AHEAD = Sh::AHEAD, TWO = Sh::TWO, QUAD = Sh::QUAD;
  extern __shared__ __align__(1024) char smem[];
  const Pages& pg = P.pages;
  const int tid = threadIdx.x, warp = tid / 32, lane = tid % 32;
  uint32_t* const s_bad = reinterpret_cast<uint32_t*>(smem + Sh::kOffBad);
  uint64_t* const k_full = reinterpret_cast<uint64_t*>(smem + Sh::kOffBar);
  uint64_t* const k_empty = k_full + RK;
  uint64_t* const v_full = k_empty + RK;
  uint64_t* const v_empty = v_full + RV;
  uint64_t* const s_full = v_empty + RV;  // [2]
  uint64_t* const p_full = s_full + 2;      // [2]
  uint64_t* const o_full = p_full + 2;      // [2]
  uint64_t* const q_full = o_full + 2;
  uint64_t* const q_empty = q_full + 1;
  uint64_t* const it_full = q_empty + 1;    // [kItems]
  uint64_t* const it_empty = it_full + kItems;
  uint64_t* const done = it_empty + kItems;
  uint64_t* const raw_full = done + 1;      // [RAW], 4-bit pages
  uint64_t* const raw_empty = raw_full + Sh::RAW;
  uint32_t* const s_tmem = reinterpret_cast<uint32_t*>(smem + Sh::kOffMisc);
  volatile int* const gave_up = reinterpret_cast<int*>(smem + Sh::kOffMisc) + 1;
  volatile int* const s_odd = reinterpret_cast<int*>(smem + Sh::kOffMisc) + 2;  // a masked value that is not finite
  Item* const items = reinterpret_cast<Item*>(smem + Sh::kOffItem);
  float* const s_qscale = reinterpret_cast<float*>(smem + Sh::kOffQScale);

  if (tid == 0) {
    // copied tiles: every copy lane's copies have landed, and a warp's part of s_bad is written
    for (int r = 0; r < RK; ++r) {
      mbar_init(k_full + r, FOUR ? Sh::kCopyWarps : kTile + Sh::kCopyWarps);
      mbar_init(k_empty + r, 1);
    }
    for (int r = 0; r < RV; ++r) {
      mbar_init(v_full + r, FOUR ? Sh::kCopyWarps : kTile);
      mbar_init(v_empty + r, 1);
    }
    for (int s = 0; s < 2; ++s) {
      mbar_init(s_full + s, 1);
      mbar_init(p_full + s, kRowWarps / 2);
      mbar_init(o_full + s, 1);
    }
    mbar_init(q_full, 64);
    mbar_init(q_empty, 1);
    for (int k = 0; k < kItems; ++k) {
      mbar_init(it_full + k, 1);
      mbar_init(it_empty + k, kRowWarps + Sh::kCopyWarps + 1 + 2);
    }
    mbar_init(done, 1);
    for (int r = 0; r < Sh::RAW; ++r) {
      mbar_init(raw_full + r, 64 + 2);  // every lane's copies, and the two parts of s_bad
      mbar_init(raw_empty + r, Sh::kCopyWarps);
    }
    mbar_fence_init();
    *gave_up = 0;
    *s_odd = 0;
  }
  // (the launch may overlap the end of the kernel before it: nothing above touches global memory)
  grid_dependency_wait();
  grid_launch_dependents();
  if (tid == 0) P.split[blockIdx.x] = make_int4(0, 0, 0, 0);
  const int64_t slots = static_cast<int64_t>(pg.max_pages) * pg.page_size;
  const Share share = scan_units<MR, THREADS>(P, slots, reinterpret_cast<int64_t*>(smem + Sh::kOffScan));
  if (share.u >= share.end) {  // nothing for this CTA
    if (tid == 0) P.gave_up[blockIdx.x] = 0;
    return;
  }
  if (warp == Sh::kMma) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], 512;" ::"r"(smem_addr(s_tmem)) : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  }
  fence_before();
  __syncthreads();
  fence_after();
  const uint32_t tmem = *s_tmem;  // columns: S of slots 0 and 1, then O of slots 0 and 1

  if (warp == Sh::kWalker) {
    // ---- the items, ahead of the others
    if (lane == 0) {
      Walk<MR> w(P, slots, share);
      for (int n = 0;; ++n) {
        if (!wait_for(it_empty + n % kItems, ((n / kItems) & 1) ^ 1, gave_up)) break;
        volatile Item& it = items[n % kItems];
        const int row0 = w.rt * MR, rows = tile_rows<MR>(P, w.rt);
        const Range R = item_range(P, w.S, row0, rows);
        const int t_lo = static_cast<int>(w.u - w.item);
        const int t_hi = min(static_cast<int>(w.seg_end() - w.item), (R.steps + kUnit - 1) / kUnit);
        const bool begins = w.u == w.item, ends = w.ends();
        it.b = w.b;
        it.h = w.h;
        it.row0 = row0;
        it.rows = rows;
        it.t_lo = t_lo;
        it.tiles = max(0, t_hi - t_lo);
        it.begins = begins;
        it.ends = ends;
        it.nq = w.S.nq;
        it.first = w.S.first;
        it.ok = w.S.ok;
        it.sink_steps = R.sink_steps;
        it.first_step = R.first_step;
        it.steps = R.steps;
        it.end = R.end;
        it.lo = R.lo;
        it.sinks = R.sinks;
        int clean_lo = 0, clean_hi = INT32_MAX;
        for (int slot = 0; slot < 2; ++slot) {
          // tile t (past the sinks) is slots 128 t - 16 off ...: it ends before `limit`, and its first slot
          // is inside the last row's window
          const int r_lo = row0 + (TWO ? slot * 128 : 0), r_hi = min(row0 + rows, r_lo + 128) - 1;
          const bool tree = P.tree_mask != nullptr;
          const int limit = min(R.end, tree ? w.S.first : w.S.first + query_of(P, min(r_lo, row0 + rows - 1)) + 1);
          const int last = tree ? w.S.first + P.n - 1 : w.S.first + min(query_of(P, max(r_hi, 0)), w.S.nq - 1);
          const int from = P.window > 0 ? max(0, last - (P.window - 1)) : 0;
          const int off = R.sink_steps - R.first_step;
          const int lo = max(R.sink_steps, (from + kStep - 1) / kStep + off);
          const int hi = limit / kStep + off;  // steps before hi end before the limit
          const int whole_lo = (lo + kUnit - 1) / kUnit, whole_hi = hi < 0 ? 0 : hi / kUnit;
          it.whole_lo[slot] = whole_lo;
          it.whole_hi[slot] = whole_hi;
          if (slot == 0 || (TWO && r_lo < row0 + rows)) {
            clean_lo = max(clean_lo, whole_lo);
            clean_hi = min(clean_hi, whole_hi);
          }
        }
        it.clean_lo = clean_lo;
        it.clean_hi = clean_hi;
        if (begins && !ends) P.split[blockIdx.x] = w.split(share);
        const bool more = w.next();
        it.last = more ? 0 : 1;
        mbar_arrive(it_full + n % kItems);
        if (!more) break;
      }
    }
    __syncwarp();
  } else if (Sh::copy_index(warp) >= 0) {
    // ---- K and V
    const int cw = Sh::copy_index(warp);
    int tile = 0;
    for (int n = 0;; ++n) {
      if (!__all_sync(0xffffffffu, wait_for(it_full + n % kItems, (n / kItems) & 1, gave_up))) break;
      const Item it = items[n % kItems];
      __syncwarp();
      if (lane == 0) mbar_arrive(it_empty + n % kItems);
      Range R;
      R.sink_steps = it.sink_steps;
      R.first_step = it.first_step;
      const int t_lo = it.t_lo, t_hi = it.t_lo + it.tiles;
      const int32_t* table = pg.table + static_cast<int64_t>(it.b) * pg.max_pages;
      const char* const k_head = pg.k + it.h * pg.head_stride;
      const char* const v_head = pg.v + it.h * pg.head_stride;
      if constexpr (!FOUR) {
        // lane l of warp c brings slot 32 c + l of a tile; its page is looked up a tile ahead
        int page = 0, in_page = -1;  // slot of the page (-1: no query of the item sees it)
        auto look_up = [&](int t) {
          const int s = R.slot(t * kUnit + cw * 2 + lane / kStep) + lane % kStep;
          in_page = -1;
          if (s < it.end && (s >= it.lo || s < it.sinks)) {
            const int logical = page_of(pg, s);
            page = __ldg(table + logical);
            in_page = s - logical * pg.page_size;
          }
        };
        look_up(t_lo);
        for (int t = t_lo; t < t_hi; ++t, ++tile) {
          const bool want = in_page >= 0;
          const bool bad = want && static_cast<unsigned>(page) >= static_cast<unsigned>(pg.num_pages);
          const int64_t off = want && !bad ? page * pg.page_stride + in_page * pg.slot_stride : 0;
          look_up(t + 1);
          const uint32_t present = __ballot_sync(0xffffffffu, want && !bad), bads = __ballot_sync(0xffffffffu, bad);
#pragma unroll
          for (int kv = 0; kv < 2; ++kv) {
            const int stage = tile % (kv ? RV : RK);
            const uint32_t parity = ((tile / (kv ? RV : RK)) & 1) ^ 1;  // the first round of a fresh barrier passes
            wait_for((kv ? v_empty : k_empty) + stage, parity, gave_up);
            __syncwarp();
            if (kv == 0 && lane == 0) {
              s_bad[(tile % kBadRing) * 4 + cw] = bads;
              mbar_arrive(k_full + stage);
            }
            const char* const head = kv ? v_head : k_head;
            const uint32_t dst = smem_addr(smem + (kv ? Sh::kOffV : Sh::kOffK) + stage * Sh::kTileBytes);
            constexpr int CH = D / 8, RPI = 32 / CH;  // 16-byte pieces of a row, rows at a time
#pragma unroll 8
            for (int j = 0; j < 32 / RPI; ++j) {
              const int row = j * RPI + lane / CH, piece = lane % CH;
              const int64_t o = __shfl_sync(0xffffffffu, off, row);
              copy_async<16>(dst + tile_offset(cw * 32 + row, piece), head + o + piece * 16, (present >> row) & 1u);
            }
            // the barrier hears of it when this lane's copies so far have landed
            asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(smem_addr((kv ? v_full : k_full) + stage)) : "memory");
          }
        }
      } else {
        // lane l converts half l / 16 of slot 16 c + l % 16: D/2 values, D/16 words of codes, D/32 scales
        constexpr int W = D / 16, RAW = Sh::RAW;
        const int half = lane / 16, row = cw * 16 + lane % 16;
        for (int t = t_lo; t < t_hi; ++t, ++tile) {
          const int rs = tile % RAW;
          wait_for(raw_full + rs, (tile / RAW) & 1, gave_up);
          __syncwarp();
          const char* const src = smem + Sh::kOffRaw + rs * Sh::kRawBytes;
          uint32_t word[2][W], scale[2];
#pragma unroll
          for (int kv = 0; kv < 2; ++kv) {
            const uint4* const cp = reinterpret_cast<const uint4*>(src + kv * Sh::kRawCodes + row * (D / 2));
#pragma unroll
            for (int y = 0; y < W / 4; ++y) {
              const uint4 c4 = cp[Sh::raw_piece(row, half * (W / 4) + y)];
              word[kv][4 * y] = c4.x;
              word[kv][4 * y + 1] = c4.y;
              word[kv][4 * y + 2] = c4.z;
              word[kv][4 * y + 3] = c4.w;
            }
            const char* const sp = src + 2 * Sh::kRawCodes + kv * Sh::kRawScales + row * (D / 16) + half * (D / 32);
            scale[kv] = D == 128 ? *reinterpret_cast<const uint32_t*>(sp) : *reinterpret_cast<const uint16_t*>(sp);
          }
          __syncwarp();
          if (lane == 0) mbar_arrive(raw_empty + rs);
#pragma unroll
          for (int kv = 0; kv < 2; ++kv) {
            const int st = tile % (kv ? RV : RK);
            wait_for((kv ? v_empty : k_empty) + st, ((tile / (kv ? RV : RK)) & 1) ^ 1, gave_up);
            __syncwarp();
            char* const dst = smem + (kv ? Sh::kOffV : Sh::kOffK) + st * Sh::kTileBytes;
#pragma unroll
            for (int y = 0; y < W; ++y) {
              uint32_t f0, f1, f2, f3;
              e2m1x8_to_f16(word[kv][y], f0, f1, f2, f3);
              const uint32_t s2 = e4m3x2_to_f16(__byte_perm(scale[kv], 0, 0x11 * (y / 2)));
              *reinterpret_cast<uint4*>(dst + tile_offset(row, half * W + y)) =
                  make_uint4(mul_f16x2(f0, s2), mul_f16x2(f1, s2), mul_f16x2(f2, s2), mul_f16x2(f3, s2));
            }
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) mbar_arrive((kv ? v_full : k_full) + st);
          }
        }
      }
      if (it.last) break;
    }
    copy_commit();
    copy_wait<0>();
  } else if (warp == Sh::kMma) {
    // ---- matrix instructions, from one elected thread.  The whole warp runs the loops, on values that
    // are the same in all lanes: the operands' descriptors then live in uniform registers, as the
    // instructions take them (from a thread's own registers each one cost about 80 clocks to issue).
    constexpr uint32_t id_s = instr_desc<M>(kTile, false), id_o = instr_desc<M>(D, true);
    const bool leader = elect_one();
    const uint32_t base = __shfl_sync(0xffffffffu, tmem, 0);
    int k_tile = 0, v_tile = 0;
    uint32_t p_phase = 0;  // bit s: slot s
    for (int n = 0;; ++n) {
      if (!__all_sync(0xffffffffu, wait_for(it_full + n % kItems, (n / kItems) & 1, gave_up))) break;
      const int tiles = __shfl_sync(0xffffffffu, items[n % kItems].tiles, 0);
      const int last = __shfl_sync(0xffffffffu, items[n % kItems].last, 0);
      if (leader) mbar_arrive(it_empty + n % kItems);
      const int jobs = TWO ? 2 * tiles : tiles;
      wait_for(q_full, n & 1, gave_up);
      __syncwarp();
      fence_proxy_async_smem();
      fence_after();
      auto issue_s = [&](int j) {
        const int slot = j & 1, stage = k_tile % RK;
        if (!TWO || slot == 0) {
          wait_for(k_full + stage, (k_tile / RK) & 1, gave_up);
          __syncwarp();
          fence_proxy_async_smem();  // the landed copies, before the matrix instructions read them
        }
        fence_after();
        const uint32_t a = desc_low(smem_addr(smem + (TWO ? slot * Sh::kTileBytes : 0)), 16);
        const uint32_t b = desc_low(smem_addr(smem + Sh::kOffK + stage * Sh::kTileBytes), 16);
        const uint32_t d = base + slot * 128;
        if (leader) {
#pragma unroll
          for (int k = 0; k < KT; ++k) {
            const uint32_t o = ((k >> 2) * (kTile * 128) + (k & 3) * 32) >> 4;
            mma_ss(d, a + o, b + o, id_s, k > 0 ? 1u : 0u);
          }
          mma_commit(s_full + slot);
          if (!TWO || slot == 1) mma_commit(k_empty + stage);
          if (j == jobs - 1) mma_commit(q_empty);
        }
        if (!TWO || slot == 1) ++k_tile;
        __syncwarp();
      };
      if (jobs == 0 && leader) mma_commit(q_empty);
      if (jobs > 0) issue_s(0);
      if (jobs > 1) issue_s(1);
      for (int j = 0; j < jobs; ++j) {
        const int slot = j & 1, stage = v_tile % RV;
        wait_for(p_full + slot, (p_phase >> slot) & 1, gave_up);
        __syncwarp();
        p_phase ^= 1u << slot;
        if (AHEAD && j + 2 < jobs) issue_s(j + 2);
        if (!TWO || slot == 0) {
          wait_for(v_full + stage, (v_tile / RV) & 1, gave_up);
          __syncwarp();
          fence_proxy_async_smem();
        }
        fence_after();
        const uint32_t b = desc_low(smem_addr(smem + Sh::kOffV + stage * Sh::kTileBytes), kTile * 128);
        const uint32_t p = base + Sh::p_column(slot), d = base + Sh::o_column(slot);
        if (leader) {
#pragma unroll
          for (int k = 0; k < kTile / 16; ++k)
            mma_ts(d, p + (k & 3) * 8 + (k >> 2) * Sh::kHalfP, b + k * (2048 >> 4), id_o, (j >= 2 || k > 0) ? 1u : 0u);
          if (!TWO || slot == 1) mma_commit(v_empty + stage);
          if (AHEAD || j + 2 >= jobs) mma_commit(o_full + slot);
        }
        if (!TWO || slot == 1) ++v_tile;
        __syncwarp();
        if (!AHEAD && j + 2 < jobs) issue_s(j + 2);
      }
      if (last) break;
    }
    if (leader) {
      mma_commit(done);
      if (!mbar_wait(done, 0)) *gave_up = 1;
    }
    __syncwarp();
  } else if (warp == Sh::kQuery0 || warp == Sh::kQuery1) {
    // ---- query rows, and the codes and scales of 4-bit pages
    const int t2 = (warp == Sh::kQuery0 ? 0 : 32) + lane;
    int raw_tile = 0;
    for (int n = 0;; ++n) {
      if (!__all_sync(0xffffffffu, wait_for(it_full + n % kItems, (n / kItems) & 1, gave_up))) break;
      const Item it = items[n % kItems];
      const int b = it.b, h = it.h, row0 = it.row0, rows = it.rows;
      const bool last = it.last != 0;
      __syncwarp();
      if (lane == 0) mbar_arrive(it_empty + n % kItems);
      // warp w of the two brings slots 64 w ... of a tile; lane l looks up slots l and 32 + l of them, a
      // tile ahead
      int raw_t = it.t_lo;
      Range R;
      R.sink_steps = it.sink_steps;
      R.first_step = it.first_step;
      const int32_t* const table = pg.table + static_cast<int64_t>(b) * pg.max_pages;
      int raw_page[2] = {0, 0}, raw_in[2] = {-1, -1};  // page, slot of the page (-1: no query of the item sees it)
      auto raw_lookup = [&](int t) {
#pragma unroll
        for (int x = 0; x < 2; ++x) {
          const int s = R.slot(t * kUnit + t2 / 32 * 4 + x * 2 + lane / kStep) + lane % kStep;
          raw_in[x] = -1;
          if (s < it.end && (s >= it.lo || s < it.sinks)) {
            const int logical = page_of(pg, s);
            raw_page[x] = __ldg(table + logical);
            raw_in[x] = s - logical * pg.page_size;
          }
        }
      };
      if constexpr (FOUR) raw_lookup(raw_t);
      auto copy_raw = [&](int until) {
        if constexpr (FOUR) {
          constexpr int RAW = Sh::RAW, CPR = D / 32;  // CPR: 16-byte pieces of a row of codes
          const char* const k_head = pg.k + h * pg.head_stride;
          const char* const v_head = pg.v + h * pg.head_stride;
          const char* const ks_head = pg.k_scales + h * pg.scale_head_stride;
          const char* const vs_head = pg.v_scales + h * pg.scale_head_stride;
          const int w2 = t2 / 32;
#pragma unroll 1
          for (; raw_t < until; ++raw_t, ++raw_tile) {
            int64_t off[2], soff[2];
            uint32_t present[2];
            const int rs = raw_tile % RAW;
#pragma unroll
            for (int x = 0; x < 2; ++x) {
              const int page = raw_page[x], in_page = raw_in[x];
              const bool bad = in_page >= 0 && static_cast<unsigned>(page) >= static_cast<unsigned>(pg.num_pages);
              const bool there = in_page >= 0 && !bad;
              const uint32_t bads = __ballot_sync(0xffffffffu, bad);
              present[x] = __ballot_sync(0xffffffffu, there);
              off[x] = there ? page * pg.page_stride + in_page * pg.slot_stride : 0;
              soff[x] = there ? page * pg.scale_page_stride + in_page * pg.scale_slot_stride : 0;
              if (lane == 0) s_bad[(raw_tile % kBadRing) * 4 + w2 * 2 + x] = bads;
            }
            raw_lookup(raw_t + 1);
            wait_for(raw_empty + rs, ((raw_tile / RAW) & 1) ^ 1, gave_up);
            __syncwarp();
            if (lane == 0) mbar_arrive(raw_full + rs);
            const uint32_t dst = smem_addr(smem + Sh::kOffRaw + rs * Sh::kRawBytes);
#pragma unroll
            for (int j = 0; j < 64 * CPR / 32; ++j) {
              const int f = j * 32 + lane, row = f / CPR;  // row of the warp's 64
              const int x = j * 32 / CPR / 32;
              const int64_t o = __shfl_sync(0xffffffffu, off[x], row % 32) + (f % CPR) * 16;
              const bool there = (present[x] >> (row % 32)) & 1u;
              const uint32_t to = dst + (w2 * 64 + row) * (D / 2) + Sh::raw_piece(row, f % CPR) * 16;
              copy_async<16>(to, k_head + o, there);
              copy_async<16>(to + Sh::kRawCodes, v_head + o, there);
            }
#pragma unroll
            for (int x = 0; x < 2; ++x) {
              const uint32_t sd = dst + 2 * Sh::kRawCodes + (w2 * 64 + x * 32 + lane) * (D / 16);
              const bool there = (present[x] >> lane) & 1u;
              copy_async<D / 16>(sd, ks_head + soff[x], there);
              copy_async<D / 16>(sd + Sh::kRawScales, vs_head + soff[x], there);
            }
            asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(smem_addr(raw_full + rs)) : "memory");
          }
        }
      };
      // the first tiles may come before the last item's queries are done with
      copy_raw(it.t_lo + min(it.tiles, Sh::RAW));
      wait_for(q_empty, (n & 1) ^ 1, gave_up);
      __syncwarp();
      const T* const q_item = static_cast<const T*>(P.q) + b * P.q_sb + h * P.G * P.q_sh;
      constexpr int CH = D / 8, AT = 64 / CH;  // lanes of a row, rows at a time
      const int piece = t2 % CH;
      auto source = [&](int r) {
        const int i = query_of(P, row0 + r);
        return reinterpret_cast<const uint4*>(q_item + i * P.q_st + (row0 + r - i * P.G) * P.q_sh) + piece;
      };
      auto target = [&](int r) { return smem + (TWO ? r / 128 * Sh::kTileBytes : 0) + tile_offset(r % 128, piece); };
      // (rows past the item's keep what was there: they only reach rows of S that nobody reads)
      if (!FOUR && P.scale_log2 >= 0.f) {  // as they are
        const int di = query_of(P, AT), dg = AT - di * P.G;
        const int64_t on = di * P.q_st + dg * P.q_sh, wrap = P.q_st - P.G * P.q_sh;
        const int i0 = query_of(P, row0 + t2 / CH);
        int g = row0 + t2 / CH - i0 * P.G;
        const T* from = q_item + i0 * P.q_st + g * P.q_sh + piece * 8;
#pragma unroll 8
        for (int r = t2 / CH; r < rows; r += AT) {
#pragma unroll
          for (int q = 0; q < (QUAD ? 4 : 1); ++q) copy_async<16>(smem_addr(target(r + 32 * q)), from, true);
          from += on;
          g += dg;
          if (g >= P.G) {
            g -= P.G;
            from += wrap;
          }
        }
        asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(smem_addr(q_full)) : "memory");
      } else {
        constexpr int AHEAD = 4;
        for (int r0 = t2 / CH; r0 - t2 / CH < rows; r0 += AHEAD * AT) {
          uint4 x[AHEAD];
#pragma unroll
          for (int k = 0; k < AHEAD; ++k)
            x[k] = r0 + k * AT < rows ? __ldg(source(r0 + k * AT)) : make_uint4(0, 0, 0, 0);
#pragma unroll
          for (int k = 0; k < AHEAD; ++k) {
            const int r = r0 + k * AT;
            uint32_t y[4] = {x[k].x, x[k].y, x[k].z, x[k].w};
            if constexpr (FOUR && !std::is_same<T, __half>::value) {
              // bf16 queries over 4-bit pages: q / 2^(exponent of the row's largest value) is within
              // (-2, 2), and fp16 then holds it to 2^-25 of that value
              float a = 0.f;
#pragma unroll
              for (int e = 0; e < 4; ++e) {
                const float2 f = Half16<T>::to_f32(y[e]);
                a = fmaxf(a, fmaxf(fabsf(f.x), fabsf(f.y)));
              }
#pragma unroll
              for (int o = CH / 2; o > 0; o >>= 1) a = fmaxf(a, __shfl_xor_sync(0xffffffffu, a, o));
              const int e8 = (__float_as_int(a) >> 23) & 0xff;
              const float up = (e8 == 0 || e8 == 0xff) ? 1.f : __int_as_float(e8 << 23);
              if (piece == 0 && r < rows) s_qscale[(n & 1) * MR + r] = up;
              const float down = 1.f / up;
#pragma unroll
              for (int e = 0; e < 4; ++e) {
                const float2 f = Half16<T>::to_f32(y[e]);
                y[e] = Half16<__half>::pack(f.x * down, f.y * down);
              }
            }
            if (P.scale_log2 < 0.f) {  // the scale's sign goes into the queries
#pragma unroll
              for (int e = 0; e < 4; ++e) y[e] ^= 0x80008000u;
            }
            if (r < rows) {
#pragma unroll
              for (int q = 0; q < (QUAD ? 4 : 1); ++q)
                *reinterpret_cast<uint4*>(target(r + 32 * q)) = make_uint4(y[0], y[1], y[2], y[3]);
            }
          }
        }
        fence_proxy_async_smem();
        mbar_arrive(q_full);
      }
      copy_raw(it.t_lo + it.tiles);
      if (last) break;
    }
    copy_commit();
    copy_wait<0>();
  } else {
    // ---- rows: threads 128 half + row of a slot hold columns 64 half ... of the slot's row.  With 32 rows
    // (QUAD) every row is in each quarter of the lanes; quarter q holds its slots 32 q ..., 16 for
    // each half, with weights of 0 for the others', and accumulates them apart, under a reference of
    // its own: all threads then have a part of every tile.
    const int slot = warp / 8, half = (warp / 4) % 2, quarter = warp % 4;
    const int spot = tid % 128, row = QUAD ? lane : spot;  // spot: the lane of tensor memory
    const uint32_t lanes = static_cast<uint32_t>((warp % 4) * 32) << 16;
    const uint32_t s_at = tmem + lanes + slot * 128 + (QUAD ? quarter * 32 + half * 16 : half * 64), o_at = tmem + lanes + Sh::o_column(slot);
    const uint32_t p_at = tmem + lanes + Sh::p_column(slot) + (QUAD ? half * 8 : half * Sh::kHalfP);
    const int pair = 2 + slot * 4 + warp % 4;  // named barrier of the two warps that share rows
    float2* const s_ml = reinterpret_cast<float2*>(smem + Sh::kOffMl);
    uint32_t s_phase = 0, o_phase = 0;
    int tile_base = 0;  // tiles of earlier items
    for (int n = 0;; ++n) {
      // (all row threads are also done with the last item's accumulators and (m, l) here)
      if (!rows_all(wait_for(it_full + n % kItems, (n / kItems) & 1, gave_up))) break;
      const volatile Item& it = items[n % kItems];
      const int row0 = it.row0 + (TWO ? slot * 128 : 0), rows = min(128, it.rows - (TWO ? slot * 128 : 0));  // may be <= 0
      const int tiles = it.tiles, t_lo = it.t_lo, first = it.first, end = it.end;
      const int whole_lo = it.whole_lo[slot], whole_hi = it.whole_hi[slot];
      const int me = query_of(P, row0 + row);  // this row's query
      const int my_pos = first + (P.depth && me < P.n ? node_depth(P, me) : me);
      const bool tree = P.tree_mask != nullptr;
      auto slot_at = [&](int step) { return (step < it.sink_steps ? step : step - it.sink_steps + it.first_step) * kStep; };
      // which of the 16 slots of a step this row sees
      auto sees16 = [&](int step) -> uint32_t {
        if (step >= it.steps) return 0u;
        const int s0 = slot_at(step);
        uint32_t near = P.window > 0 ? bits16(my_pos - (P.window - 1) - s0, kStep) | bits16(0, P.sinks - s0) : 0xffffu;
        if (!tree) return near & bits16(0, min(first + me, end - 1) + 1 - s0);
        uint32_t see = near & bits16(0, min(first, end) - s0);
        if (s0 + kStep > first && me < P.n) {
          const uint8_t* const mask = P.tree_mask + static_cast<int64_t>(me) * P.n;
          const uint32_t there = bits16(first - s0, end - s0);
          uint32_t node = 0;
#pragma unroll
          for (int e = 0; e < kStep; ++e)
            if ((there >> e) & 1u) node |= (__ldg(mask + (s0 + e - first)) != 0 ? 1u : 0u) << e;
          if (P.window > 0 && P.depth) {
            near = 0;
#pragma unroll 1
            for (int e = 0; e < kStep; ++e)
              if ((there >> e) & 1u) {
                const int pos = first + node_depth(P, s0 + e - first);
                near |= (my_pos - pos < P.window || pos < P.sinks ? 1u : 0u) << e;
              }
          }
          see |= near & node;
        }
        return see;
      };

      const bool active = QUAD || quarter * 32 < rows;  // a warp without rows leaves its lanes as they are
      // (never 0, not by underflow either, so that a masked score stays infinite; the sign is in the
      // staged queries)
      constexpr float kLeast = 1.4e-45f;
      float c = fmaxf(fabsf(P.scale_log2), kLeast);
      constexpr uint32_t hidden = 0xff800000u;  // -inf
      float m = -kInf, l = 0.f;
      int jobs = 0;
      for (int t = TWO ? 0 : slot; t < tiles; t += TWO ? 1 : 2, ++jobs) {
        const int tile = tile_base + t;
        bool partial = rows > 0 && (t_lo + t < whole_lo || t_lo + t >= whole_hi);  // some row may not see some slot
        wait_for(s_full + slot, s_phase, gave_up);
        s_phase ^= 1;
        __syncwarp();  // (lanes leave a wait apart; tensor-memory instructions want them together)
        fence_after();
        uint32_t r[2][16];
        float top = -kInf;
        const uint4 bads = *reinterpret_cast<const uint4*>(s_bad + (tile % kBadRing) * 4);
        if (FOUR && !std::is_same<T, __half>::value && jobs == 0)
          c = fmaxf(c * s_qscale[(n & 1) * MR + (TWO ? slot * 128 : 0) + row], kLeast);
        uint32_t seen[2] = {~0u, ~0u};
        bool poisoned = false;  // the row sees a slot on a page out of range
        partial = partial || (rows > 0 && (bads.x | bads.y | bads.z | bads.w) != 0);
        if (QUAD && partial) {
          seen[0] = sees16((t_lo + t) * kUnit + 2 * quarter + half);
          const uint32_t mine = quarter == 0 ? bads.x : quarter == 1 ? bads.y : quarter == 2 ? bads.z : bads.w;
          poisoned = (seen[0] & (mine >> (16 * half))) != 0;
          __syncwarp();
        } else if (partial && active) {
          const int step0 = (t_lo + t) * kUnit + half * (kUnit / 2), s0 = slot_at(step0);
          if ((step0 >= it.sink_steps || step0 + 4 <= it.sink_steps) && !(tree && s0 + 64 > first)) {
            // 64 slots in a row, and no tree node among them
            const uint64_t near = P.window > 0 ? bits64(my_pos - (P.window - 1) - s0, 64) | bits64(0, P.sinks - s0) : ~0ull;
            const uint64_t see = near & bits64(0, (tree ? min(first, end) : min(first + me, end - 1) + 1) - s0);
            seen[0] = static_cast<uint32_t>(see);
            seen[1] = static_cast<uint32_t>(see >> 32);
          } else {
#pragma unroll 1
            for (int x = 0; x < 4; ++x) {
              const uint32_t see = sees16(step0 + x) << (16 * (x & 1)), keep = 0xffff0000u >> (16 * (x & 1));
              if (x < 2) seen[0] = (seen[0] & keep) | see;
              else seen[1] = (seen[1] & keep) | see;
            }
          }
          poisoned = ((seen[0] & (half ? bads.z : bads.x)) | (seen[1] & (half ? bads.w : bads.y))) != 0;
          __syncwarp();
        }
        auto mask_scores = [&](int ch, uint32_t (&r)[16]) {
          if (partial) {
            const uint32_t see = seen[ch >> 1] >> (16 * (ch & 1));
#pragma unroll
            for (int e = 0; e < 16; ++e) r[e] = (see >> e) & 1u ? r[e] : hidden;
          }
        };
        if constexpr (QUAD) {
          tmem_load(s_at, r[0]);
          tmem_load_wait(r[0]);
          mask_scores(0, r[0]);
#pragma unroll
          for (int e = 0; e < 16; e += 2) top = max3(top, __uint_as_float(r[0][e]), __uint_as_float(r[0][e + 1]));
          top *= c;
        } else if (active) {
#pragma unroll
          for (int h2 = 0; h2 < 2; ++h2) {  // 32 columns at a time
            tmem_load(s_at + 32 * h2, r[0]);
            tmem_load(s_at + 32 * h2 + 16, r[1]);
#pragma unroll
            for (int x = 0; x < 2; ++x) {
              tmem_load_wait(r[x]);
              mask_scores(2 * h2 + x, r[x]);
#pragma unroll
              for (int e = 0; e < 16; e += 2) top = max3(top, __uint_as_float(r[x][e]), __uint_as_float(r[x][e + 1]));
            }
          }
          top *= c;
        }
        if (AHEAD && jobs > 0) {  // the last products have read their weights and added to the accumulator
          wait_for(o_full + slot, o_phase, gave_up);
          o_phase ^= 1;
          __syncwarp();
          fence_after();
        }
        if (active) {
          if (pair_any(pair, top - m > kSlack + kBelow<M>)) {  // (also where m is still -inf) the reference moves
            s_ml[(slot * 2 + half) * 128 + spot].x = top;
            asm volatile("bar.sync %0, 64;" ::"r"(pair) : "memory");
            top = fmaxf(m, fmaxf(top, s_ml[(slot * 2 + (half ^ 1)) * 128 + spot].x) - kBelow<M>);
            const float alpha = m == top ? 1.f : ex2(m - (top == -kInf ? 0.f : top));
            m = top;
            l *= alpha;
            if (jobs > 0 && __any_sync(0xffffffffu, alpha != 1.f)) {  // each half rescales half of the accumulator
#pragma unroll 1
              for (int d = half * (D / 2); d < (half + 1) * (D / 2); d += 16) {
                tmem_load(o_at + d, r[1]);
                tmem_load_wait(r[1]);
#pragma unroll
                for (int e = 0; e < 16; ++e) r[1][e] = __float_as_uint(__uint_as_float(r[1][e]) * alpha);
                tmem_store16(o_at + d, r[1]);
              }
            }
          }
          // the weights, 16 at a time; where they overwrite scores, this thread has read them: weights 16 ch ...
          // go to columns 8 ch ..., scores 16 ch ... are in columns 16 ch ...
          const float base = m == -kInf ? 0.f : m;
          // (two at a time: packed fp32 products and sums, rounded as the scalar ones)
          const unsigned long long c2 = f2pack(c, c), base2 = f2pack(-base, -base);
          unsigned long long sum2[2] = {0ull, 0ull};
          if constexpr (!QUAD) tmem_load(s_at, r[0]);
#pragma unroll
          for (int ch = 0; ch < (QUAD ? 1 : 4); ++ch) {
            if constexpr (!QUAD) {
              tmem_load_wait(r[ch & 1]);
              if (ch < 3) tmem_load(s_at + 16 * (ch + 1), r[(ch + 1) & 1]);
              mask_scores(ch, r[ch & 1]);
            }
            uint32_t p[8];
#pragma unroll
            for (int e = 0; e < 16; e += 2) {
              float x0, x1;
              f2unpack(f2fma(f2pack(__uint_as_float(r[ch & 1][e]), __uint_as_float(r[ch & 1][e + 1])), c2, base2), x0, x1);
              const float p0 = ex2(x0), p1 = ex2(x1);
              sum2[(e >> 1) & 1] = f2add(sum2[(e >> 1) & 1], f2pack(p0, p1));
              p[e / 2] = Half16<M>::pack(p0, p1);
            }
            if constexpr (QUAD) {  // (both halves have read their scores: the pair met above)
              const uint32_t none[8] = {0, 0, 0, 0, 0, 0, 0, 0};
#pragma unroll
              for (int q = 0; q < 4; ++q) {
                const uint32_t at = p_at + (q & 1) * 16 + (q >> 1) * Sh::kHalfP;
                if (q == quarter) tmem_store8(at, p);
                else tmem_store8(at, none);
              }
            } else {
              tmem_store8(p_at + 8 * ch, p);
            }
          }
          float s0, s1;
          f2unpack(f2add(sum2[0], sum2[1]), s0, s1);
          l += poisoned ? __int_as_float(0x7fffffff) : s0 + s1;
        }
        // 0 times a value that is not finite is not 0: where some row does not see a slot, such
        // values are taken out of the staged tile; the rows that see them get them at the end.  Two row
        // tiles share the staged tile: the first one's warps scan it where either is partial, for their
        // product comes before the second's.
        if (TWO ? slot == 0 && (partial || t_lo + t < it.clean_lo || t_lo + t >= it.clean_hi) : partial) {
          wait_for(v_full + tile % RV, (tile / RV) & 1, gave_up);
          char* const vt = smem + Sh::kOffV + (tile % RV) * Sh::kTileBytes;
          constexpr uint32_t em = std::is_same<M, __half>::value ? 0x7c00u : 0x7f80u;
          bool found = false;
#pragma unroll 4
          for (int f = (warp % 8) * 32 + lane; f < kTile * (D / 8); f += 256) {
            uint4* const at = reinterpret_cast<uint4*>(vt + f * 16);
            uint32_t x[4] = {at->x, at->y, at->z, at->w};
            const uint32_t top2 = __vmaxu2(__vmaxu2(x[0] & 0x7fff7fffu, x[1] & 0x7fff7fffu), __vmaxu2(x[2] & 0x7fff7fffu, x[3] & 0x7fff7fffu));
            const bool here = (top2 & 0xffffu) >= em || top2 >= em << 16;
            if (here) {
#pragma unroll
              for (int e = 0; e < 4; ++e) {
                if ((x[e] & em) == em) x[e] &= 0xffff0000u;
                if ((x[e] & (em << 16)) == em << 16) x[e] &= 0xffffu;
              }
              *at = make_uint4(x[0], x[1], x[2], x[3]);
              found = true;
            }
          }
          if (found) {
            *s_odd = 1;
            fence_proxy_async_smem();
          }
          __syncwarp();
        }
        if (active) tmem_store_wait();
        fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(p_full + slot);
      }

      // ---- the item's rows, or the part of them that this segment holds
      if (jobs > 0) {
        wait_for(o_full + slot, o_phase, gave_up);
        o_phase ^= 1;
        fence_after();
      }
      s_ml[(slot * 2 + half) * 128 + spot] = make_float2(m, l);
      fence_before();
      // the halves of a row meet, and where both slots hold the same rows, the slots too
      if constexpr (TWO)
        asm volatile("bar.sync %0, 64;" ::"r"(pair) : "memory");
      else
        asm volatile("bar.sync 1, 512;" ::: "memory");
      fence_after();
      const bool whole_item = it.begins && it.ends;
      const int64_t token = static_cast<int64_t>(it.b) * P.n;
      const int64_t part0 = (static_cast<int64_t>(blockIdx.x) * 2 + (it.begins ? 1 : 0)) * MR;
      // 16 values d ... of this row's products with values that are not finite (rare)
      auto add_odd = [&](int d, float (&acc)[16]) {
        const int32_t* table = pg.table + static_cast<int64_t>(it.b) * pg.max_pages;
#pragma unroll 1
        for (int step = t_lo * kUnit; step < (t_lo + tiles) * kUnit; ++step) {
          if (step / kUnit >= it.clean_lo && step / kUnit < it.clean_hi) continue;  // not scanned
          for (uint32_t see = sees16(step); see != 0; see &= see - 1) {
            const int s = slot_at(step) + __ffs(see) - 1;
            const int page = __ldg(table + page_of(pg, s)), in_page = s - page_of(pg, s) * pg.page_size;
            if (static_cast<unsigned>(page) >= static_cast<unsigned>(pg.num_pages)) continue;
            if constexpr (FOUR) {  // only a group's scale can be NaN
              const uint8_t sb = *reinterpret_cast<const uint8_t*>(pg.v_scales + page * pg.scale_page_stride + in_page * pg.scale_slot_stride +
                                                                   it.h * pg.scale_head_stride + d / kGroup4);
              if ((sb & 0x7f) == 0x7f) {
#pragma unroll
                for (int x = 0; x < 16; ++x) acc[x] = __int_as_float(0x7fffffff);
              }
            } else {
              const T* v = reinterpret_cast<const T*>(pg.v + page * pg.page_stride + in_page * pg.slot_stride + it.h * pg.head_stride) + d;
#pragma unroll
              for (int x = 0; x < 16; ++x) {
                const float f = static_cast<float>(v[x]);
                if (!(fabsf(f) < kInf)) acc[x] += f;
              }
            }
          }
        }
      };
      // a row's slots that had tiles (what the others' accumulators hold says nothing)
      const bool had0 = TWO ? jobs > 0 : tiles > 0, had1 = TWO ? jobs > 0 : tiles > 1;
      if constexpr (QUAD) {
        // eight sums of every row: join them over slots here, over quarters in shared memory
        float mm[2][4], top = -kInf;
#pragma unroll
        for (int x = 0; x < 8; ++x) {
          mm[x / 4][x % 4] = s_ml[x / 4 * 256 + x % 4 * 32 + lane].x;
          top = fmaxf(top, mm[x / 4][x % 4]);
        }
        const float base = top == -kInf ? 0.f : top;
        float* const s_sum = reinterpret_cast<float*>(smem + Sh::kOffSum);
        float* const s_inv = s_sum + 4 * 4 * 32 * 8;
        if (warp == 0) {
          float sum = 0.f;
#pragma unroll
          for (int x = 0; x < 8; ++x) {
            const float2* const at = s_ml + x / 4 * 256 + x % 4 * 32 + lane;
            sum += ex2(mm[x / 4][x % 4] - base) * (at[0].y + at[128].y);
          }
          const bool none = sum == 0.f || me >= it.nq;
          const bool undefined = !it.ok || (whole_item && sum == 0.f && sees_some(P, first, it.nq, me));
          s_inv[lane] = undefined ? __int_as_float(0x7fffffff) : none ? 0.f : pg.v_scale / sum;
          if (row < rows && me < P.n) {
            if (whole_item) {
              if (P.lse)
                P.lse[(token + me) * P.Hq + it.h * P.G + row0 + row - me * P.G] =
                    undefined ? __int_as_float(0x7fffffff) : none ? -kInf : top * kLn2 + logf(sum);
            } else {
              P.part_ml[part0 + row] = make_float2(top, sum);
            }
          }
        }
        const int group = slot * 2 + half;
        const float scale0 = had0 ? ex2(s_ml[quarter * 32 + lane].x - base) : 0.f, scale1 = had1 ? ex2(s_ml[256 + quarter * 32 + lane].x - base) : 0.f;
        // `per` of a thread's D / 4 values at a time go through shared memory, as many as there is room for
        // with this many rows; thread 128 g + t of group g then sums two of a row's.  (16-byte pieces turned
        // by the row: 8 lanes meet no bank conflict.)
        const int per = rows <= 8 && D == 128 ? 32 : rows <= 16 ? 16 : 8, turn = per / 4 - 1;
        const int sum_row = 2 * spot / per, sum_me = query_of(P, row0 + sum_row), sum_at = 2 * spot % per;
        const int sum_head = it.h * P.G + row0 + sum_row - sum_me * P.G;
        const bool writes = sum_row < rows && sum_me < P.n;
        const float* const from = s_sum + group * 256 + sum_row * per + ((sum_at / 4) ^ (sum_row & turn)) * 4 + sum_at % 4;
        float* const to = s_sum + (quarter * 4 + group) * 256 + lane * per;
#pragma unroll 1
        for (int d = 0; d < D / 4; d += 16) {
          float acc[16];
          uint32_t x[16];
          const uint32_t at = tmem + lanes + group * (D / 4) + d;
#pragma unroll
          for (int e = 0; e < 16; ++e) acc[e] = 0.f;
          if (had0) {
            tmem_load(at + Sh::o_column(0), x);
            tmem_load_wait(x);
#pragma unroll
            for (int e = 0; e < 16; ++e) acc[e] = __uint_as_float(x[e]) * scale0;
          }
          if (had1) {
            tmem_load(at + Sh::o_column(1), x);
            tmem_load_wait(x);
#pragma unroll
            for (int e = 0; e < 16; ++e) acc[e] = fmaf(__uint_as_float(x[e]), scale1, acc[e]);
          }
          if (__builtin_expect(*s_odd != 0, 0) && quarter == 0 && row < rows && me < P.n) add_odd(group * (D / 4) + d, acc);
#pragma unroll
          for (int u = 0; u < 2; ++u) {
            const int piece = (d + 8 * u) % per / 4;
            if (lane * per < 256) {
              *reinterpret_cast<float4*>(to + (piece ^ (lane & turn)) * 4) = make_float4(acc[8 * u], acc[8 * u + 1], acc[8 * u + 2], acc[8 * u + 3]);
              *reinterpret_cast<float4*>(to + ((piece + 1) ^ (lane & turn)) * 4) = make_float4(acc[8 * u + 4], acc[8 * u + 5], acc[8 * u + 6], acc[8 * u + 7]);
            }
            if ((d + 8 * u + 8) % per != 0) continue;
            asm volatile("bar.sync 1, 512;" ::: "memory");
            float2 v = make_float2(0.f, 0.f);
#pragma unroll
            for (int q = 0; q < 4; ++q) {
              const float2 y = *reinterpret_cast<const float2*>(from + q * (4 * 32 * 8));
              v.x += y.x;
              v.y += y.y;
            }
            const int column = group * (D / 4) + d + 8 * u + 8 - per + sum_at;
            if (writes) {
              if (whole_item) {
                const float inv = s_inv[sum_row];
                *reinterpret_cast<uint32_t*>(static_cast<T*>(P.out) + ((token + sum_me) * P.Hq + sum_head) * D + column) =
                    inv == 0.f ? 0u : Half16<T>::pack(v.x * inv, v.y * inv);
              } else {
                *reinterpret_cast<float2*>(P.part_o + (part0 + sum_row) * D + column) = v;
              }
            }
            asm volatile("bar.sync 1, 512;" ::: "memory");
          }
        }
      } else {
        l = s_ml[slot * 256 + row].y + s_ml[slot * 256 + 128 + row].y;
        float scale_own = 1.f, scale_other = 0.f;
        if constexpr (!TWO) {
          const int o = (slot ^ 1) * 256 + row;
          const float other = s_ml[o].x, other_l = s_ml[o].y + s_ml[o + 128].y;
          const float top = fmaxf(m, other), base = top == -kInf ? 0.f : top;
          scale_own = ex2(m - base);
          scale_other = ex2(other - base);
          l = l * scale_own + other_l * scale_other;
          m = top;
        }
        __syncwarp();
        const bool mine = row < rows && me < P.n;
        const int64_t at = (token + me) * P.Hq + it.h * P.G + row0 + row - me * P.G;
        const int64_t part = part0 + (TWO ? slot * 128 : 0) + row;
        const bool none = l == 0.f || me >= it.nq;
        const bool undefined = !it.ok || (mine && whole_item && l == 0.f && sees_some(P, first, it.nq, me));
        const float inv = none ? 0.f : pg.v_scale / l;
        constexpr int COLS = TWO ? D / 2 : D / 4;  // of this thread
        const int d_lo = TWO ? half * COLS : (slot * 2 + half) * COLS;
        if (active) {
#pragma unroll 1
          for (int d = d_lo; d < d_lo + COLS; d += 16) {
            float acc[16];
            uint32_t r[16];
            __syncwarp();
#pragma unroll
            for (int e = 0; e < 16; ++e) acc[e] = 0.f;
            if (jobs > 0) {
              tmem_load(o_at + d, r);
              tmem_load_wait(r);
#pragma unroll
              for (int e = 0; e < 16; ++e) acc[e] = __uint_as_float(r[e]) * scale_own;
            }
            if (!TWO && (slot == 0 ? had1 : had0)) {
              tmem_load(tmem + lanes + Sh::o_column(slot ^ 1) + d, r);
              tmem_load_wait(r);
#pragma unroll
              for (int e = 0; e < 16; ++e) acc[e] = fmaf(__uint_as_float(r[e]), scale_other, acc[e]);
            }
            if (__builtin_expect(*s_odd != 0, 0) && mine) add_odd(d, acc);
            if (!mine) continue;
            if (whole_item) {
              uint32_t out[8];
#pragma unroll
              for (int e = 0; e < 8; ++e) {
                out[e] = none ? 0u : Half16<T>::pack(acc[2 * e] * inv, acc[2 * e + 1] * inv);
                if (undefined) out[e] = 0x7fff7fffu;
              }
              uint4* dst = reinterpret_cast<uint4*>(static_cast<T*>(P.out) + at * D + d);
              dst[0] = make_uint4(out[0], out[1], out[2], out[3]);
              dst[1] = make_uint4(out[4], out[5], out[6], out[7]);
            } else {
              float4* dst = reinterpret_cast<float4*>(P.part_o + part * D + d);
#pragma unroll
              for (int e = 0; e < 4; ++e) dst[e] = make_float4(acc[4 * e], acc[4 * e + 1], acc[4 * e + 2], acc[4 * e + 3]);
            }
          }
          if (mine && d_lo == 0) {
            if (whole_item) {
              if (P.lse) P.lse[at] = undefined ? __int_as_float(0x7fffffff) : none ? -kInf : m * kLn2 + logf(l);
            } else {
              P.part_ml[part] = make_float2(m, l);
            }
          }
        }
      }
      tile_base += tiles;
      fence_before();
      const bool last = it.last != 0;
      __syncwarp();
      if (lane == 0) mbar_arrive(it_empty + n % kItems);
      if (last) break;
    }
  }

  fence_before();
  __syncthreads();
  fence_after();
  if (warp == Sh::kMma)
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, 512;" ::"r"(tmem) : "memory");
  if (tid == 0) P.gave_up[blockIdx.x] = *gave_up;
}

template <typename T, int D, Rows ROWS, bool FOUR>
cudaError_t launch_shape(const AttendParams& P, cudaStream_t stream) {
  using Sh = Shape<D, ROWS, FOUR>;
  auto kernel = attend_tc_kernel<T, D, ROWS, FOUR>;
  static_assert(Sh::kBytes <= 227 * 1024, "shared memory of a CTA");
  if (cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, Sh::kBytes); e != cudaSuccess)
    return e;
  return launch_kernel(kernel, dim3(P.ctas), dim3(Sh::kThreads), Sh::kBytes, stream, 1, P);
}

template <typename T, int D, bool FOUR>
cudaError_t launch_rows(const AttendParams& P, int mr, cudaStream_t stream) {
  return mr == 32    ? launch_shape<T, D, kQuad, FOUR>(P, stream)
         : mr == 128 ? launch_shape<T, D, kOne, FOUR>(P, stream)
                     : launch_shape<T, D, kTwo, FOUR>(P, stream);
}

template <typename T, bool FOUR>
cudaError_t launch_typed(const AttendParams& P, int mr, cudaStream_t stream) {
  return P.pages.head_dim == 64 ? launch_rows<T, 64, FOUR>(P, mr, stream) : launch_rows<T, 128, FOUR>(P, mr, stream);
}

}  // namespace tc

}  // namespace specdec
