// Attention over 16-bit pages on the tensor cores with accumulators in tensor memory.
//
// The formula, the items and the split of the work are those of attend.cu.  A tile is 128 query
// rows of one key head by 128 slots:
//   S = Q K^T  (tcgen05.mma, Q and K from shared memory)  -> 128 columns of tensor memory
//   P = 2^(c S - m), one row per thread                   -> back to tensor memory, 16 bits
//   O += P V   (tcgen05.mma, P from tensor memory)        -> D columns of tensor memory
// Two such streams ("slots" 0 and 1 of the CTA) take turns, so that one's exponentials run while
// the other's products do: with more than 128 rows per key head they are two row tiles that share
// every staged K and V tile; with fewer, both hold the same rows and take every other tile, and
// their results join at the end.
//
// A thread keeps its row's reference m and moves it only when a tile exceeds it by more than
// 2^8: the weights then stay below 256, where 16-bit rounding is relative and as good as below
// 1, and the accumulator is rescaled once or twice per item instead of once per tile.  The sum l
// takes the unrounded weights, in fp32.
//
// Warps 0-3 and 4-7: rows of slots 0 and 1.  Warps 8-11: copies of K and V rows from their
// pages, 16 bytes at a time, into 128-byte-swizzled tiles (pages of any size and stride: a
// tile's rows need not be neighbours).  Warp 12: one thread issues the matrix instructions.  The
// roles meet at mbarriers; every wait is bounded, and a CTA whose wait runs out stops waiting,
// finishes its (finite) loops and reports it.

#include "attend_common.cuh"

namespace specdec {

namespace {

constexpr int kRowWarps = 8, kCopyWarps = 4;
constexpr int kTcThreads = 32 * 16;    // the last four warps: one issues matrix instructions, three rest
constexpr int kTile = kUnit * kStep;  // 128 slots
constexpr int kBadRing = 8;           // tiles whose out-of-range slots are remembered
constexpr float kSlack = 8.f;         // log2 of how far a weight may exceed 1
static_assert(kTile == 128 && kCopyWarps * 32 == kTile, "one copy lane per slot");

// What the row warps keep of an item.
struct Item {
  int b, h, row0, rows, t_lo, tiles, begins, ends, nq, first, ok, sink_steps, first_step, steps, end, more;
};

template <int D, bool TWO>
struct TcShape {
  static constexpr int MR = TWO ? 256 : 128;
  static constexpr int kTileBytes = kTile * D * 2;
  static constexpr int RING = D == 64 ? 4 : (TWO ? 2 : 3);  // K tiles and V tiles staged
  static constexpr int kOffK = (TWO ? 2 : 1) * kTileBytes;
  static constexpr int kOffV = kOffK + RING * kTileBytes;
  static constexpr int kOffMl = kOffV + RING * kTileBytes;  // [2][128] (m, l) of the slots
  static constexpr int kOffItem = kOffMl + 2 * 128 * 8;
  static constexpr int kOffScan = kOffItem + 2 * sizeof(Item);
  static constexpr int kOffBad = kOffScan + (kTcThreads / 32 + 2) * 8;
  static constexpr int kOffBar = kOffBad + kBadRing * kCopyWarps * 4;
  static constexpr int kBars = 4 * RING + 2 + 2 + 2 + 1 + 1;
  static constexpr int kOffMisc = kOffBar + kBars * 8;
  static constexpr int kBytes = kOffMisc + 16;
};

// ---- tcgen05 -----------------------------------------------------------------------------

// Shared-memory matrix descriptor: 128-byte swizzle, strides in bytes.
__device__ __forceinline__ uint64_t smem_desc(uint32_t addr, uint32_t lead, uint32_t stride) {
  return static_cast<uint64_t>((addr >> 4) & 0x3fff) | (static_cast<uint64_t>((lead >> 4) & 0x3fff) << 16) |
         (static_cast<uint64_t>((stride >> 4) & 0x3fff) << 32) | (1ull << 46) | (2ull << 61);
}
// Instruction descriptor: fp32 accumulator, 16-bit operands, M = 128.
template <typename T>
__device__ __forceinline__ constexpr uint32_t instr_desc(int n, bool b_mn_major) {
  const uint32_t type = std::is_same<T, __nv_bfloat16>::value ? 1u : 0u;
  return (1u << 4) | (type << 7) | (type << 10) | (b_mn_major ? 1u << 16 : 0u) | (static_cast<uint32_t>(n >> 3) << 17) |
         ((128u >> 4) << 24);
}
__device__ __forceinline__ void mma_ss(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, bool accumulate) {
  asm volatile(
      "{\n.reg .pred p;\nsetp.ne.u32 p, %4, 0;\n"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n}" ::"r"(d), "l"(a), "l"(b), "r"(idesc),
      "r"(accumulate ? 1u : 0u)
      : "memory");
}
__device__ __forceinline__ void mma_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, bool accumulate) {
  asm volatile(
      "{\n.reg .pred p;\nsetp.ne.u32 p, %4, 0;\n"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n}" ::"r"(d), "r"(a), "l"(b), "r"(idesc),
      "r"(accumulate ? 1u : 0u)
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
__device__ __forceinline__ void wait_for(uint64_t* bar, uint32_t parity, volatile int* gave_up) {
  if (mbar_try_wait(bar, parity)) return;
  const uint64_t t0 = global_timer_ns();
  while (!mbar_try_wait(bar, parity)) {
    if (*gave_up) return;
    if (global_timer_ns() - t0 > kMaxWaitNs) {
      *gave_up = 1;
      return;
    }
  }
}
// Where the 16-byte piece `piece` of row `row` of a tile of 128 rows of D values lies: blocks
// of 64 values, rows of 128 bytes, pieces swizzled by the row.
template <int D>
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

template <typename T, int D, bool TWO>
__global__ void __launch_bounds__(kTcThreads, 1) attend_tc_kernel(const AttendParams P) {
  using Sh = TcShape<D, TWO>;
  constexpr int MR = Sh::MR, RING = Sh::RING, KT = D / 16;
  extern __shared__ __align__(1024) char smem[];
  const Pages& pg = P.pages;
  const int tid = threadIdx.x, warp = tid / 32, lane = tid % 32;
  const int64_t slots = static_cast<int64_t>(pg.max_pages) * pg.page_size;
  int64_t* const s_scan = reinterpret_cast<int64_t*>(smem + Sh::kOffScan);
  uint32_t* const s_bad = reinterpret_cast<uint32_t*>(smem + Sh::kOffBad);
  uint64_t* const k_full = reinterpret_cast<uint64_t*>(smem + Sh::kOffBar);
  uint64_t* const k_empty = k_full + RING;
  uint64_t* const v_full = k_empty + RING;
  uint64_t* const v_empty = v_full + RING;
  uint64_t* const s_full = v_empty + RING;  // [2]
  uint64_t* const p_full = s_full + 2;      // [2]
  uint64_t* const o_full = p_full + 2;      // [2]
  uint64_t* const q_full = o_full + 2;
  uint64_t* const done = q_full + 1;
  uint32_t* const s_tmem = reinterpret_cast<uint32_t*>(smem + Sh::kOffMisc);
  volatile int* const gave_up = reinterpret_cast<int*>(smem + Sh::kOffMisc) + 1;
  volatile int* const s_odd = reinterpret_cast<int*>(smem + Sh::kOffMisc) + 2;  // a masked value that is not finite

  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  if (tid == 0) {
    for (int r = 0; r < RING; ++r) {
      mbar_init(k_full + r, kTile + kCopyWarps);  // every copy lane's copies have landed; a warp's s_bad is written
      mbar_init(k_empty + r, 1);
      mbar_init(v_full + r, kTile);
      mbar_init(v_empty + r, 1);
    }
    for (int s = 0; s < 2; ++s) {
      mbar_init(s_full + s, 1);
      mbar_init(p_full + s, 4);
      mbar_init(o_full + s, 1);
    }
    mbar_init(q_full, kRowWarps);
    mbar_init(done, 1);
    mbar_fence_init();
    *gave_up = 0;
    *s_odd = 0;
    P.split[blockIdx.x] = make_int4(0, 0, 0, 0);
  }
  const Share share = scan_units<MR, kTcThreads>(P, slots, s_scan);
  if (share.u >= share.end) {  // nothing for this CTA
    if (tid == 0) P.gave_up[blockIdx.x] = 0;
    return;
  }
  if (warp == kRowWarps + kCopyWarps) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], 512;" ::"r"(smem_addr(s_tmem)) : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  }
  fence_before();
  __syncthreads();
  fence_after();
  const uint32_t tmem = *s_tmem;  // columns: S of slots 0 and 1, then O of slots 0 and 1
  Walk<MR> w(P, slots, share);

  if (warp >= kRowWarps && warp < kRowWarps + kCopyWarps) {
    // ---- copies: lane l of copy warp c brings slot 32 c + l of every tile
    const int cw = warp - kRowWarps;
    int tile = 0;
    do {
      const int rows = tile_rows<MR>(P, w.rt);
      const Range R = item_range(P, w.S, w.rt * MR, rows);
      const int t_lo = static_cast<int>(w.u - w.item), t_hi = min(static_cast<int>(w.seg_end() - w.item), (R.steps + kUnit - 1) / kUnit);
      const int32_t* table = pg.table + static_cast<int64_t>(w.b) * pg.max_pages;
      const char* const k_head = pg.k + w.h * pg.head_stride;
      const char* const v_head = pg.v + w.h * pg.head_stride;
      auto slot_of = [&](int t) { return R.slot(t * kUnit + cw * 2 + lane / kStep) + lane % kStep; };
      auto wanted = [&](int t, int s) {  // a slot that some query of the item sees
        return t * kUnit + cw * 2 + lane / kStep < R.steps && s < R.end && (s >= R.lo || s < R.sinks);
      };
      int page = 0;
      if (t_lo < t_hi) {
        const int s = slot_of(t_lo);
        if (wanted(t_lo, s)) page = __ldg(table + s / pg.page_size);
      }
      for (int t = t_lo; t < t_hi; ++t) {
        const int s = slot_of(t);
        const bool want = wanted(t, s);
        const bool bad = want && static_cast<unsigned>(page) >= static_cast<unsigned>(pg.num_pages);
        const int64_t off = want && !bad ? page * pg.page_stride + (s % pg.page_size) * pg.slot_stride : 0;
        if (t + 1 < t_hi) {
          const int s1 = slot_of(t + 1);
          page = wanted(t + 1, s1) ? __ldg(table + s1 / pg.page_size) : 0;
        }
        const uint32_t present = __ballot_sync(0xffffffffu, want && !bad), bads = __ballot_sync(0xffffffffu, bad);
        const int stage = tile % RING;
        const uint32_t parity = ((tile / RING) & 1) ^ 1;  // the first round of a fresh barrier passes
#pragma unroll
        for (int kv = 0; kv < 2; ++kv) {
          wait_for((kv ? v_empty : k_empty) + stage, parity, gave_up);
          __syncwarp();
          if (kv == 0 && lane == 0) {
            s_bad[(tile % kBadRing) * kCopyWarps + cw] = bads;
            mbar_arrive(k_full + stage);
          }
          const char* const head = kv ? v_head : k_head;
          const uint32_t dst = smem_addr(smem + (kv ? Sh::kOffV : Sh::kOffK) + stage * Sh::kTileBytes);
          constexpr int CH = D / 8, RPI = 32 / CH;  // 16-byte pieces of a row, rows at a time
#pragma unroll 8
          for (int j = 0; j < 32 / RPI; ++j) {
            const int row = j * RPI + lane / CH, piece = lane % CH;
            const int64_t o = __shfl_sync(0xffffffffu, off, row);
            copy_async<16>(dst + tile_offset<D>(cw * 32 + row, piece), head + o + piece * 16, (present >> row) & 1u);
          }
          // the barrier hears of it when this lane's copies so far have landed
          asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(smem_addr((kv ? v_full : k_full) + stage)) : "memory");
        }
        ++tile;
      }
    } while (w.next());
    copy_commit();
    copy_wait<0>();
  } else if (warp >= kRowWarps + kCopyWarps) {
    // ---- matrix instructions, from one thread
    if (warp == kRowWarps + kCopyWarps && lane == 0) {
      constexpr uint32_t id_s = instr_desc<T>(kTile, false), id_o = instr_desc<T>(D, true);
      int k_tile = 0, v_tile = 0, segment = 0;
      uint32_t p_phase[2] = {0, 0};
      do {
        const Range R = item_range(P, w.S, w.rt * MR, tile_rows<MR>(P, w.rt));
        const int tiles = min(static_cast<int>(w.seg_end() - w.item), (R.steps + kUnit - 1) / kUnit) - static_cast<int>(w.u - w.item);
        const int jobs = tiles <= 0 ? 0 : TWO ? 2 * tiles : tiles;
        wait_for(q_full, segment & 1, gave_up);
        ++segment;
        fence_after();
        auto issue_s = [&](int n) {
          const int slot = n & 1, tile = k_tile, stage = tile % RING;
          if (!TWO || slot == 0) {
            wait_for(k_full + stage, (tile / RING) & 1, gave_up);
            fence_proxy_async_smem();  // the landed copies, before the matrix instructions read them
          }
          fence_after();
          const uint32_t a = smem_addr(smem + (TWO ? slot * Sh::kTileBytes : 0));
          const uint32_t b = smem_addr(smem + Sh::kOffK + stage * Sh::kTileBytes);
#pragma unroll
          for (int k = 0; k < KT; ++k) {
            const uint32_t o = (k >> 2) * (kTile * 128) + (k & 3) * 32;
            mma_ss(tmem + slot * 128, smem_desc(a + o, 16, 1024), smem_desc(b + o, 16, 1024), id_s, k > 0);
          }
          if (!TWO || slot == 1) {
            mma_commit(k_empty + stage);
            ++k_tile;
          }
          mma_commit(s_full + slot);
        };
        if (jobs > 0) issue_s(0);
        if (jobs > 1) issue_s(1);
        for (int n = 0; n < jobs; ++n) {
          const int slot = n & 1, tile = v_tile, stage = tile % RING;
          if (!TWO || slot == 0) {
            wait_for(v_full + stage, (tile / RING) & 1, gave_up);
            fence_proxy_async_smem();
          }
          wait_for(p_full + slot, p_phase[slot], gave_up);
          p_phase[slot] ^= 1;
          fence_after();
          const uint32_t b = smem_addr(smem + Sh::kOffV + stage * Sh::kTileBytes);
#pragma unroll
          for (int k = 0; k < kTile / 16; ++k)
            mma_ts(tmem + 256 + slot * 128, tmem + slot * 128 + k * 8, smem_desc(b + k * 2048, kTile * 128, 1024), id_o,
                   n >= 2 || k > 0);
          if (!TWO || slot == 1) {
            mma_commit(v_empty + stage);
            ++v_tile;
          }
          if (n + 2 >= jobs) mma_commit(o_full + slot);
          if (n + 2 < jobs) issue_s(n + 2);
        }
      } while (w.next());
      mma_commit(done);
      wait_for(done, 0, gave_up);
    }
    __syncwarp();
  } else {
    // ---- rows: thread = row of the slot's tile.  What an item is stays in shared memory, so
    // that the registers are free for a row of scores.
    const int slot = warp / 4, row = tid % 128;
    const uint32_t lanes = static_cast<uint32_t>((warp % 4) * 32) << 16;
    const uint32_t s_at = tmem + lanes + slot * 128, o_at = tmem + lanes + 256 + slot * 128;
    float2* const s_ml = reinterpret_cast<float2*>(smem + Sh::kOffMl);
    volatile Item& it = *reinterpret_cast<volatile Item*>(smem + Sh::kOffItem + slot * sizeof(Item));
    uint32_t s_phase = 0, o_phase = 0;
    int tile_base = 0;  // tiles of earlier segments
    bool more = true;
    while (more) {
      asm volatile("bar.sync %0, 128;" ::"r"(2 + slot) : "memory");  // the last item is done with
      if (row == 0) {
        const int item_rows = tile_rows<MR>(P, w.rt), row0 = w.rt * MR + (TWO ? slot * 128 : 0);
        const Range R = item_range(P, w.S, w.rt * MR, item_rows);
        const int t_lo = static_cast<int>(w.u - w.item);
        it.b = w.b;
        it.h = w.h;
        it.row0 = row0;
        it.rows = min(128, item_rows - (TWO ? slot * 128 : 0));  // may be <= 0
        it.t_lo = t_lo;
        it.tiles = max(0, min(static_cast<int>(w.seg_end() - w.item), (R.steps + kUnit - 1) / kUnit) - t_lo);
        it.begins = w.u == w.item;
        it.ends = w.seg_end() == w.item + w.units;
        it.nq = w.S.nq;
        it.first = w.S.first;
        it.ok = w.S.ok;
        it.sink_steps = R.sink_steps;
        it.first_step = R.first_step;
        it.steps = R.steps;
        it.end = R.end;
        if (it.begins && !it.ends && slot == 0) P.split[blockIdx.x] = w.split(share);
        it.more = w.next();
      }
      asm volatile("bar.sync %0, 128;" ::"r"(2 + slot) : "memory");
      more = it.more;
      const int rows = it.rows, row0 = it.row0, tiles = it.tiles, t_lo = it.t_lo, first = it.first;
      Range R;
      R.sink_steps = it.sink_steps;
      R.first_step = it.first_step;
      R.steps = it.steps;
      R.end = it.end;
      const bool tree = P.tree_mask != nullptr;

      // the query rows, zeros past the tile's: slot by slot, or together where both hold the same
      {
        constexpr int LOADERS = TWO ? 128 : 256;
        char* const dst = smem + (TWO ? slot * Sh::kTileBytes : 0);
        const T* const q_item = static_cast<const T*>(P.q) + it.b * P.q_sb + it.h * P.G * P.q_sh;
#pragma unroll 4
        for (int f = TWO ? row : tid; f < 128 * (D / 8); f += LOADERS) {
          const int r = f / (D / 8), piece = f % (D / 8);
          uint4 x = make_uint4(0, 0, 0, 0);
          if (r < rows)
            x = __ldg(reinterpret_cast<const uint4*>(q_item + ((row0 + r) / P.G) * P.q_st + ((row0 + r) % P.G) * P.q_sh) + piece);
          if (P.scale_log2 < 0.f) x = make_uint4(x.x ^ 0x80008000u, x.y ^ 0x80008000u, x.z ^ 0x80008000u, x.w ^ 0x80008000u);
          *reinterpret_cast<uint4*>(dst + tile_offset<D>(r, piece)) = x;
        }
        fence_proxy_async_smem();
        fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(q_full);
      }

      const int me = (row0 + row) / P.G;  // this row's query
      const int my_pos = first + (P.depth && me < P.n ? node_depth(P, me) : me);
      // every row of this slot's tile sees the 16 slots of a step
      auto whole_step = [&](int step) {
        const int s0 = R.slot(step);
        bool ok = step < R.steps && s0 + kStep <= R.end && s0 + kStep <= (tree ? first : first + row0 / P.G + 1);
        if (P.window > 0)
          ok = ok && ((tree ? first + P.n - 1 : first + min((row0 + rows - 1) / P.G, it.nq - 1)) - s0 < P.window || s0 + kStep <= P.sinks);
        return ok;
      };
      // the same of a whole tile, from its first and last step (a few false answers at the sinks)
      auto whole_tile = [&](int step) {
        const int s0 = R.slot(step), last = R.slot(step + kUnit - 1);
        return step + kUnit <= R.steps && last + kStep <= R.end && last + kStep <= (tree ? first : first + row0 / P.G + 1) &&
               (P.window == 0 || (tree ? first + P.n - 1 : first + min((row0 + rows - 1) / P.G, it.nq - 1)) - s0 < P.window);
      };
      // which of the 16 slots of a step this row sees
      auto sees16 = [&](int step) -> uint32_t {
        if (step >= R.steps) return 0u;
        const int s0 = R.slot(step);
        uint32_t near = P.window > 0 ? bits16(my_pos - (P.window - 1) - s0, kStep) | bits16(0, P.sinks - s0) : 0xffffu;
        if (!tree) return near & bits16(0, min(first + me, R.end - 1) + 1 - s0);
        uint32_t see = near & bits16(0, min(first, R.end) - s0);
        if (s0 + kStep > first && me < P.n) {
          const uint8_t* const mask = P.tree_mask + static_cast<int64_t>(me) * P.n;
          const uint32_t there = bits16(first - s0, R.end - s0);
          uint32_t node = 0;
#pragma unroll
          for (int e = 0; e < kStep; ++e)
            if ((there >> e) & 1u) node |= (__ldg(mask + (s0 + e - first)) != 0 ? 1u : 0u) << e;
          if (P.window > 0 && P.depth) {
            near = 0;
#pragma unroll
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

      const bool active = (warp % 4) * 32 < rows;  // a warp without rows leaves its lanes as they are
      // the sign of the scale is in the staged queries; a scale of 0 becomes the smallest one, so
      // that a masked score stays infinite
      const float c = P.scale_log2 == 0.f ? 1.4e-45f : fabsf(P.scale_log2);
      constexpr uint32_t hidden = 0xff800000u;  // -inf
      float m = -kInf, l = 0.f;
      int jobs = 0;
      for (int t = TWO ? 0 : slot; t < tiles; t += TWO ? 1 : 2, ++jobs) {
        const int tile = tile_base + t;
        wait_for(s_full + slot, s_phase, gave_up);
        s_phase ^= 1;
        __syncwarp();  // (lanes leave a wait apart; tensor-memory instructions want them together)
        fence_after();
        const int step0 = (t_lo + t) * kUnit;
        uint32_t partial = 0;  // chunks of 32 slots that not every row sees whole
        uint32_t seen[4] = {~0u, ~0u, ~0u, ~0u};
        bool poisoned = false;  // the row sees a slot on a page out of range
        if (rows > 0) {
          const uint4 bads = *reinterpret_cast<const uint4*>(s_bad + (tile % kBadRing) * kCopyWarps);
          if ((bads.x | bads.y | bads.z | bads.w) != 0 || !whole_tile(step0)) {
            const uint32_t bad4[4] = {bads.x, bads.y, bads.z, bads.w};
#pragma unroll
            for (int ch = 0; ch < 4; ++ch) {
              if (bad4[ch] != 0 || !whole_step(step0 + 2 * ch) || !whole_step(step0 + 2 * ch + 1)) {
                partial |= 1u << ch;
                if (active) seen[ch] = sees16(step0 + 2 * ch) | (sees16(step0 + 2 * ch + 1) << 16);
                poisoned = poisoned || (seen[ch] & bad4[ch]) != 0;
              }
            }
          }
        }
        if (active) {
          __syncwarp();
          auto mask_scores = [&](int ch, uint32_t (&r)[16]) {  // 16 scores: half of a chunk
            if ((partial >> (ch >> 1)) & 1u) {
              const uint32_t see = seen[ch >> 1] >> (16 * (ch & 1));
#pragma unroll
              for (int e = 0; e < 16; ++e) r[e] = (see >> e) & 1u ? r[e] : hidden;
            }
          };
          uint32_t r[2][16];
          float top = -kInf;
          tmem_load(s_at, r[0]);
#pragma unroll
          for (int ch = 0; ch < 8; ++ch) {
            tmem_load_wait(r[ch & 1]);
            if (ch < 7) tmem_load(s_at + 16 * (ch + 1), r[(ch + 1) & 1]);
            mask_scores(ch, r[ch & 1]);
#pragma unroll
            for (int e = 0; e < 16; e += 2) top = max3(top, __uint_as_float(r[ch & 1][e]), __uint_as_float(r[ch & 1][e + 1]));
          }
          top *= c;
          if (__any_sync(0xffffffffu, top > m + kSlack)) {  // (also where m is still -inf)
            top = fmaxf(m, top);
            const float alpha = m == top ? 1.f : ex2(m - (top == -kInf ? 0.f : top));
            m = top;
            l *= alpha;
            if (jobs > 0 && __any_sync(0xffffffffu, alpha != 1.f)) {
#pragma unroll 1
              for (int d = 0; d < D; d += 16) {
                tmem_load(o_at + d, r[1]);
                tmem_load_wait(r[1]);
#pragma unroll
                for (int e = 0; e < 16; ++e) r[1][e] = __float_as_uint(__uint_as_float(r[1][e]) * alpha);
                tmem_store16(o_at + d, r[1]);
              }
            }
          }
          // the weights, 16 at a time; they overwrite scores that have been read: weights 16 ch ... are
          // columns 8 ch ..., scores 16 ch ... columns 16 ch ...
          const float base = m == -kInf ? 0.f : m;
          float sum[4] = {0.f, 0.f, 0.f, 0.f};
          tmem_load(s_at, r[0]);
#pragma unroll
          for (int ch = 0; ch < 8; ++ch) {
            tmem_load_wait(r[ch & 1]);
            if (ch < 7) tmem_load(s_at + 16 * (ch + 1), r[(ch + 1) & 1]);
            mask_scores(ch, r[ch & 1]);
            uint32_t p[8];
#pragma unroll
            for (int e = 0; e < 16; e += 2) {
              const float p0 = ex2(fmaf(__uint_as_float(r[ch & 1][e]), c, -base));
              const float p1 = ex2(fmaf(__uint_as_float(r[ch & 1][e + 1]), c, -base));
              sum[(e >> 1) & 1] += p0;
              sum[2 + ((e >> 1) & 1)] += p1;
              p[e / 2] = Half16<T>::pack(p0, p1);
            }
            tmem_store8(s_at + 8 * ch, p);
          }
          l += poisoned ? __int_as_float(0x7fffffff) : (sum[0] + sum[1]) + (sum[2] + sum[3]);
        }
        if (partial) {
          // 0 times a value that is not finite is not 0: where some row does not see a slot, such
          // values are taken out of the staged tile; the rows that see them get them at the end
          wait_for(v_full + tile % RING, (tile / RING) & 1, gave_up);
          char* const vt = smem + Sh::kOffV + (tile % RING) * Sh::kTileBytes;
          constexpr uint32_t em = std::is_same<T, __half>::value ? 0x7c00u : 0x7f80u;
          bool found = false;
#pragma unroll 1
          for (int ch = 0; ch < 4; ++ch) {
            if (!((partial >> ch) & 1u)) continue;
#pragma unroll 4
            for (int f = row; f < 32 * (D / 8); f += 128) {
              uint4* const at = reinterpret_cast<uint4*>(vt + tile_offset<D>(32 * ch + f / (D / 8), f % (D / 8)));
              uint32_t x[4] = {at->x, at->y, at->z, at->w};
              bool here = false;
#pragma unroll
              for (int e = 0; e < 4; ++e) here = here || (x[e] & em) == em || (x[e] & (em << 16)) == em << 16;
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
      const bool whole_item = it.begins && it.ends;
      const int other_jobs = TWO ? 0 : (slot == 0 ? tiles / 2 : (tiles + 1) / 2);
      float scale_own = 1.f, scale_other = 0.f;
      if (jobs > 0) {
        wait_for(o_full + slot, o_phase, gave_up);
        o_phase ^= 1;
        fence_after();
      }
      if (!TWO) {  // both slots hold the same rows: join them; each half of the warps writes half of D
        s_ml[slot * 128 + row] = make_float2(m, l);
        fence_before();
        asm volatile("bar.sync 1, 256;" ::: "memory");
        const float2 other = s_ml[(slot ^ 1) * 128 + row];
        const float top = fmaxf(m, other.x), base = top == -kInf ? 0.f : top;
        scale_own = ex2(m - base);
        scale_other = ex2(other.x - base);
        l = l * scale_own + other.y * scale_other;
        m = top;
      }
      fence_after();
      __syncwarp();
      const bool mine = row < rows && me < P.n;
      const int head = it.h * P.G + (row0 + row) % P.G;
      const int64_t at = (static_cast<int64_t>(it.b) * P.n + me) * P.Hq + head;
      const int64_t part = (static_cast<int64_t>(blockIdx.x) * 2 + (it.begins ? 1 : 0)) * MR + (TWO ? slot * 128 : 0) + row;
      const bool none = l == 0.f || me >= it.nq;
      const float inv = none ? 0.f : pg.v_scale / l;
      const bool odd = *s_odd != 0;
      if (active) {
        constexpr int COLS = TWO ? D : D / 2;
#pragma unroll 1
        for (int d0 = 0; d0 < COLS; d0 += 16) {
          const int d = (TWO ? 0 : slot * COLS) + d0;
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
          if (!TWO && other_jobs > 0) {
            tmem_load(o_at + (slot == 0 ? 128 : -128) + d, r);
            tmem_load_wait(r);
#pragma unroll
            for (int e = 0; e < 16; ++e) acc[e] = fmaf(__uint_as_float(r[e]), scale_other, acc[e]);
          }
          if (odd && mine) {  // rare: values that are not finite, for the rows that see them
            const int32_t* table = pg.table + static_cast<int64_t>(it.b) * pg.max_pages;
#pragma unroll 1
            for (int step = t_lo * kUnit; step < (t_lo + tiles) * kUnit; ++step) {
              if (whole_step(step & ~1) && whole_step(step | 1)) continue;
              for (uint32_t see = sees16(step); see != 0; see &= see - 1) {
                const int s = R.slot(step) + __ffs(see) - 1;
                const int page = __ldg(table + s / pg.page_size);
                if (static_cast<unsigned>(page) >= static_cast<unsigned>(pg.num_pages)) continue;
                const T* v = reinterpret_cast<const T*>(pg.v + page * pg.page_stride + (s % pg.page_size) * pg.slot_stride +
                                                        it.h * pg.head_stride) + d;
#pragma unroll
                for (int x = 0; x < 16; ++x) {
                  const float f = static_cast<float>(v[x]);
                  if (!(fabsf(f) < kInf)) acc[x] += f;
                }
              }
            }
          }
          if (!mine) continue;
          if (whole_item) {
            uint32_t out[8];
#pragma unroll
            for (int e = 0; e < 8; ++e) {
              out[e] = none ? 0u : Half16<T>::pack(acc[2 * e] * inv, acc[2 * e + 1] * inv);
              if (!it.ok) out[e] = 0x7fff7fffu;
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
        if (mine && (TWO || slot == 0)) {
          if (whole_item) {
            if (P.lse) P.lse[at] = !it.ok ? __int_as_float(0x7fffffff) : none ? -kInf : m * kLn2 + logf(l);
          } else {
            P.part_ml[part] = make_float2(m, l);
          }
        }
      }
      tile_base += tiles;
      fence_before();
    }
  }

  fence_before();
  __syncthreads();
  fence_after();
  if (warp == kRowWarps + kCopyWarps)
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, 512;" ::"r"(tmem) : "memory");
  if (tid == 0) P.gave_up[blockIdx.x] = *gave_up;
}

template <typename T, int D, bool TWO>
cudaError_t launch_tc_shape(const AttendParams& P, cudaStream_t stream) {
  auto kernel = attend_tc_kernel<T, D, TWO>;
  constexpr int bytes = TcShape<D, TWO>::kBytes;
  static_assert(bytes <= 227 * 1024, "shared memory of a CTA");
  if (cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes); e != cudaSuccess) return e;
  return launch_kernel(kernel, dim3(P.ctas), dim3(kTcThreads), bytes, stream, 0, P);
}

template <typename T>
cudaError_t launch_tc_typed(const AttendParams& P, int mr, cudaStream_t stream) {
  if (P.pages.head_dim == 64)
    return mr == 256 ? launch_tc_shape<T, 64, true>(P, stream) : launch_tc_shape<T, 64, false>(P, stream);
  return mr == 256 ? launch_tc_shape<T, 128, true>(P, stream) : launch_tc_shape<T, 128, false>(P, stream);
}

}  // namespace

int attend_tc_rows(int64_t rows) { return rows <= 128 ? 128 : 256; }

cudaError_t launch_attend_tc(const AttendParams& P, specdec_dtype dt, int mr, cudaStream_t stream) {
  return dt == SPECDEC_BF16 ? launch_tc_typed<__nv_bfloat16>(P, mr, stream) : launch_tc_typed<__half>(P, mr, stream);
}

}  // namespace specdec
