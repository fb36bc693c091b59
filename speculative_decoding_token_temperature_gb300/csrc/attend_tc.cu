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

template <int D, bool TWO>
struct TcShape {
  static constexpr int MR = TWO ? 256 : 128;
  static constexpr int kTileBytes = kTile * D * 2;
  static constexpr int RING = D == 64 ? 4 : (TWO ? 2 : 3);  // K tiles and V tiles staged
  static constexpr int kOffK = (TWO ? 2 : 1) * kTileBytes;
  static constexpr int kOffV = kOffK + RING * kTileBytes;
  static constexpr int kOffMl = kOffV + RING * kTileBytes;  // [2][128] (m, l) of the slots
  static constexpr int kOffScan = kOffMl + 2 * 128 * 8;
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

// 32 columns of this warp's 32 lanes; the wait is part of the load, so the values are there.
__device__ __forceinline__ void tmem_load(uint32_t addr, uint32_t (&r)[32]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
      "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];\n"
      "tcgen05.wait::ld.sync.aligned;"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
        "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16]),
        "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]),
        "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
      : "r"(addr)
      : "memory");
}
__device__ __forceinline__ void tmem_store(uint32_t addr, const uint32_t* r) {  // 32 columns
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,"
      "%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31,%32};" ::"r"(addr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
      "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]), "r"(r[16]), "r"(r[17]), "r"(r[18]),
      "r"(r[19]), "r"(r[20]), "r"(r[21]), "r"(r[22]), "r"(r[23]), "r"(r[24]), "r"(r[25]), "r"(r[26]), "r"(r[27]),
      "r"(r[28]), "r"(r[29]), "r"(r[30]), "r"(r[31])
      : "memory");
}
__device__ __forceinline__ void tmem_store_wait() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

// Registers move from the warps that copy and issue to those that hold rows: 2 * 176 + 88 + 72 =
// 4 * 128, what the CTA was launched with.
template <int N> __device__ __forceinline__ void more_registers() { asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N)); }
template <int N> __device__ __forceinline__ void fewer_registers() { asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N)); }

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
__device__ __forceinline__ bool test_for(uint64_t* bar, uint32_t parity) {
  uint32_t ok;
  asm volatile("{\n.reg .pred p;\nmbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\nselp.u32 %0, 1, 0, p;\n}"
               : "=r"(ok) : "r"(smem_addr(bar)), "r"(parity) : "memory");
  return ok != 0;
}

// Where the 16-byte piece `piece` of row `row` of a tile of 128 rows of D values lies: blocks
// of 64 values, rows of 128 bytes, pieces swizzled by the row.
template <int D>
__device__ __forceinline__ uint32_t tile_offset(int row, int piece) {
  return (piece >> 3) * (kTile * 128) + row * 128 + (((piece & 7) ^ (row & 7)) << 4);
}

// One query row of an item and what it sees.
struct Row {
  int i, pos, hi, lo;  // chain: slots <= hi that are >= lo or among the sinks
};

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
      mbar_init(k_full + r, kCopyWarps);
      mbar_init(k_empty + r, 1);
      mbar_init(v_full + r, kCopyWarps);
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
    fewer_registers<88>();
    // ---- copies: lane l of copy warp c brings slot 32 c + l of every tile
    const int cw = warp - kRowWarps;
    int issued = 0, arrived = 0;  // groups: K of tile 0, V of tile 0, K of tile 1, ...
    auto arrive_oldest = [&]() {
      switch (issued - arrived) {  // copies in flight after the oldest
        case 1: copy_wait<0>(); break;
        case 2: copy_wait<1>(); break;
        case 3: copy_wait<2>(); break;
        case 4: copy_wait<3>(); break;
        case 5: copy_wait<4>(); break;
        case 6: copy_wait<5>(); break;
        case 7: copy_wait<6>(); break;
        default: copy_wait<7>(); break;
      }
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(((arrived & 1) ? v_full : k_full) + (arrived >> 1) % RING);
      ++arrived;
    };
    static_assert(2 * RING <= 8, "arrive_oldest counts at most 8 groups in flight");
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
        const int tile = issued >> 1, stage = tile % RING;
        if (lane == 0) s_bad[(tile % kBadRing) * kCopyWarps + cw] = bads;
#pragma unroll
        for (int kv = 0; kv < 2; ++kv) {
          uint64_t* const empty = (kv ? v_empty : k_empty) + stage;
          const uint32_t parity = ((tile / RING) & 1) ^ 1;  // the first round of a fresh barrier passes
          while (!__all_sync(0xffffffffu, test_for(empty, parity))) {
            if (arrived < issued)
              arrive_oldest();
            else
              wait_for(empty, parity, gave_up);
            if (*gave_up) break;
          }
          __syncwarp();
          const char* const head = kv ? v_head : k_head;
          const uint32_t dst = smem_addr(smem + (kv ? Sh::kOffV : Sh::kOffK) + stage * Sh::kTileBytes);
          constexpr int CH = D / 8, RPI = 32 / CH;  // 16-byte pieces of a row, rows at a time
#pragma unroll 8
          for (int j = 0; j < 32 / RPI; ++j) {
            const int row = j * RPI + lane / CH, piece = lane % CH;
            const int64_t o = __shfl_sync(0xffffffffu, off, row);
            copy_async<16>(dst + tile_offset<D>(cw * 32 + row, piece), head + o + piece * 16, (present >> row) & 1u);
          }
          copy_commit();
          ++issued;
        }
      }
    } while (w.next());
    while (arrived < issued) arrive_oldest();
  } else if (warp >= kRowWarps + kCopyWarps) {
    fewer_registers<72>();
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
          if (!TWO || slot == 0) wait_for(k_full + stage, (tile / RING) & 1, gave_up);
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
          if (!TWO || slot == 0) wait_for(v_full + stage, (tile / RING) & 1, gave_up);
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
    more_registers<176>();
    // ---- rows: thread = row of the slot's tile
    const int slot = warp / 4, row = tid % 128;
    const uint32_t lanes = static_cast<uint32_t>((warp % 4) * 32) << 16;
    const uint32_t s_at = tmem + lanes + slot * 128, o_at = tmem + lanes + 256 + slot * 128;
    float2* const s_ml = reinterpret_cast<float2*>(smem + Sh::kOffMl);
    uint32_t s_phase = 0, o_phase = 0;
    int tile_base = 0;  // tiles of earlier segments
    do {
      const SeqLen S = w.S;
      const int row0 = w.rt * MR + (TWO ? slot * 128 : 0), item_rows = tile_rows<MR>(P, w.rt);
      const int rows = min(128, item_rows - (TWO ? slot * 128 : 0));  // may be <= 0
      const Range R = item_range(P, S, w.rt * MR, item_rows);
      const int t_lo = static_cast<int>(w.u - w.item);
      const int tiles = max(0, min(static_cast<int>(w.seg_end() - w.item), (R.steps + kUnit - 1) / kUnit) - t_lo);
      const bool tree = P.tree_mask != nullptr;

      // the query rows, zeros past the tile's: slot by slot, or together where both hold the same
      {
        constexpr int LOADERS = TWO ? 128 : 256;
        char* const dst = smem + (TWO ? slot * Sh::kTileBytes : 0);
        for (int f = TWO ? row : tid; f < 128 * (D / 8); f += LOADERS) {
          const int r = f / (D / 8), piece = f % (D / 8);
          uint4 x = make_uint4(0, 0, 0, 0);
          if (r < rows)
            x = *(reinterpret_cast<const uint4*>(static_cast<const T*>(P.q) + w.b * P.q_sb + ((row0 + r) / P.G) * P.q_st +
                                                 (w.h * P.G + (row0 + r) % P.G) * P.q_sh) + piece);
          *reinterpret_cast<uint4*>(dst + tile_offset<D>(r, piece)) = x;
        }
        fence_proxy_async_smem();
        fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(q_full);
      }

      Row me;
      me.i = (row0 + row) / P.G;
      me.pos = S.first + (P.depth && me.i < P.n ? node_depth(P, me.i) : me.i);
      me.hi = min(S.first + me.i, R.end - 1);
      me.lo = P.window > 0 ? max(0, me.pos - (P.window - 1)) : 0;
      const int i0 = row0 / P.G, i1 = min((row0 + rows - 1) / P.G, S.nq - 1);
      // every row of this slot's tile sees slots [s0, s0 + 16)
      auto whole_step = [&](int step) {
        const int s0 = R.slot(step);
        bool ok = step < R.steps && s0 + kStep <= R.end;
        if (tree) {
          ok = ok && s0 + kStep <= S.first;
          if (P.window > 0) ok = ok && (S.first + P.n - 1 - s0 < P.window || s0 + kStep <= P.sinks);
        } else {
          ok = ok && s0 + kStep - 1 <= S.first + i0;
          if (P.window > 0) ok = ok && (S.first + i1 - s0 < P.window || s0 + kStep <= P.sinks);
        }
        return ok;
      };
      // the same of a whole tile, from its first and last step (a few false answers at the sinks)
      auto whole_tile = [&](int step) {
        const int first = R.slot(step), last = R.slot(step + kUnit - 1);
        return step + kUnit <= R.steps && last + kStep <= R.end &&
               last + kStep <= (tree ? S.first : S.first + i0 + 1) &&
               (P.window == 0 || (tree ? S.first + P.n - 1 : S.first + i1) - first < P.window);
      };
      auto sees = [&](int s) {
        if (!tree) return s <= me.hi && (s >= me.lo || s < P.sinks);
        const int j = s - S.first;
        bool ok = s < R.end;
        int pos = s;
        if (j >= 0) {
          ok = ok && me.i < P.n && __ldg(P.tree_mask + static_cast<int64_t>(me.i) * P.n + min(j, P.n - 1)) != 0;
          if (P.depth) pos = S.first + node_depth(P, min(j, P.n - 1));
        }
        return ok && (P.window == 0 || me.pos - pos < P.window || pos < P.sinks);
      };

      const bool active = (warp % 4) * 32 < rows;  // a warp without rows leaves its lanes as they are
      const int scanners = min(128, (rows + 31) / 32 * 32);
      // (a scale of 0 becomes the smallest one, so that a masked score stays infinite)
      const float c = P.scale_log2 == 0.f ? 1.4e-45f : P.scale_log2;
      const uint32_t hidden = __float_as_uint(c > 0.f ? -kInf : kInf);
      float m = -kInf, l = 0.f;
      int jobs = 0;
      for (int t = TWO ? 0 : slot; t < tiles; t += TWO ? 1 : 2, ++jobs) {
        const int tile = tile_base + t;
        wait_for(s_full + slot, s_phase, gave_up);
        s_phase ^= 1;
        __syncwarp();  // (lanes leave a wait apart; tensor-memory instructions want them together)
        fence_after();
        if (active) {
          const int step0 = (t_lo + t) * kUnit;
          uint32_t partial = 0;  // chunks of 32 slots that not every row sees whole
          uint32_t seen[4] = {~0u, ~0u, ~0u, ~0u};
          bool poisoned = false;  // the row sees a slot on a page out of range
          const uint4 bads = *reinterpret_cast<const uint4*>(s_bad + (tile % kBadRing) * kCopyWarps);
          if ((bads.x | bads.y | bads.z | bads.w) != 0 || !whole_tile(step0)) {
            const uint32_t bad4[4] = {bads.x, bads.y, bads.z, bads.w};
#pragma unroll
            for (int ch = 0; ch < 4; ++ch) {
              if (bad4[ch] == 0 && whole_step(step0 + 2 * ch) && whole_step(step0 + 2 * ch + 1)) continue;
              partial |= 1u << ch;
              uint32_t see = 0;
#pragma unroll 1
              for (int e = 0; e < 32; ++e) {
                const int step = step0 + 2 * ch + e / kStep;
                if (step < R.steps && sees(R.slot(step) + e % kStep)) see |= 1u << e;
              }
              seen[ch] = see;
              poisoned = poisoned || (see & bad4[ch]) != 0;
            }
          }
          __syncwarp();
          auto load_scores = [&](int ch, uint32_t (&r)[32]) {
            tmem_load(s_at + 32 * ch, r);
            if ((partial >> ch) & 1u) {
#pragma unroll
              for (int e = 0; e < 32; ++e) r[e] = (seen[ch] >> e) & 1u ? r[e] : hidden;
            }
          };
          uint32_t p[64];
          float fresh = 0.f;
          bool moved = m == -kInf;
#pragma unroll 1
          for (int pass = 0;; ++pass) {
            if (__any_sync(0xffffffffu, moved)) {  // the reference moves to the row's maximum so far
              float top = m;
#pragma unroll
              for (int ch = 0; ch < 4; ++ch) {
                uint32_t r[32];
                load_scores(ch, r);
#pragma unroll
                for (int e = 0; e < 32; ++e) top = fmaxf(top, __uint_as_float(r[e]) * c);
              }
              const float alpha = m == top ? 1.f : ex2(m - (top == -kInf ? 0.f : top));
              m = top;
              l *= alpha;
              if (jobs > 0 && __any_sync(0xffffffffu, alpha != 1.f)) {
#pragma unroll 1
                for (int d = 0; d < D; d += 32) {
                  uint32_t r[32];
                  tmem_load(o_at + d, r);
#pragma unroll
                  for (int e = 0; e < 32; ++e) r[e] = __float_as_uint(__uint_as_float(r[e]) * alpha);
                  tmem_store(o_at + d, r);
                }
                tmem_store_wait();
              }
            }
            const float base = m == -kInf ? 0.f : m;
            float top = -kInf, sum[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int ch = 0; ch < 4; ++ch) {
              uint32_t r[32];
              load_scores(ch, r);
#pragma unroll
              for (int e = 0; e < 32; e += 2) {
                const float x0 = fmaf(__uint_as_float(r[e]), c, -base), x1 = fmaf(__uint_as_float(r[e + 1]), c, -base);
                top = fmaxf(top, fmaxf(x0, x1));
                const float p0 = ex2(x0), p1 = ex2(x1);
                sum[(e >> 1) & 1] += p0;
                sum[2 + ((e >> 1) & 1)] += p1;
                p[16 * ch + e / 2] = Half16<T>::pack(p0, p1);
              }
            }
            fresh = (sum[0] + sum[1]) + (sum[2] + sum[3]);
            moved = top > kSlack;
            // (after a move no score exceeds the reference: at most one more pass)
            if (pass == 1 || !__any_sync(0xffffffffu, moved)) break;
          }
          if (poisoned) fresh = __int_as_float(0x7fffffff);
          l += fresh;
          if (partial) {
            // 0 times a value that is not finite is not 0: where some row does not see a slot, such
            // values are taken out of the staged tile; the rows that see them get them at the end
            wait_for(v_full + tile % RING, (tile / RING) & 1, gave_up);
            char* const vt = smem + Sh::kOffV + (tile % RING) * Sh::kTileBytes;
            constexpr uint32_t em = std::is_same<T, __half>::value ? 0x7c00u : 0x7f80u;
            bool found = false;
            for (int f = row; f < kTile * (D / 8); f += scanners) {
              const int r = f / (D / 8);
              if (!((partial >> (r / 32)) & 1u)) continue;
              uint4* const at = reinterpret_cast<uint4*>(vt + tile_offset<D>(r, f % (D / 8)));
              uint32_t x[4] = {at->x, at->y, at->z, at->w};
              bool here = false;
#pragma unroll
              for (int e = 0; e < 4; ++e) {
                if ((x[e] & em) == em) { x[e] &= 0xffff0000u; here = true; }
                if (((x[e] >> 16) & em) == em) { x[e] &= 0xffffu; here = true; }
              }
              if (here) {
                *at = make_uint4(x[0], x[1], x[2], x[3]);
                found = true;
              }
            }
            if (found) {
              *s_odd = 1;
              fence_proxy_async_smem();
            }
          }
          __syncwarp();
          tmem_store(s_at, p);
          tmem_store(s_at + 32, p + 32);
          tmem_store_wait();
        }
        fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(p_full + slot);
      }

      // ---- the item's rows, or the part of them that this segment holds
      const bool begins = w.u == w.item, ends = w.seg_end() == w.item + w.units;
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
        l = slot == 0 ? l * scale_own + other.y * scale_other : other.y * scale_other + l * scale_own;
        m = top;
      }
      fence_after();
      const int i = me.i;
      const bool mine = row < rows && i < P.n;
      const int head = w.h * P.G + (row0 + row) % P.G;
      const int64_t at = (static_cast<int64_t>(w.b) * P.n + i) * P.Hq + head;
      const int64_t part = (static_cast<int64_t>(blockIdx.x) * 2 + (begins ? 1 : 0)) * MR + (TWO ? slot * 128 : 0) + row;
      const bool none = l == 0.f || i >= S.nq;
      const float inv = none ? 0.f : pg.v_scale / l;
      const bool odd = *s_odd != 0;
      if (active) {
        constexpr int COLS = TWO ? D : D / 2;
#pragma unroll 1
        for (int d0 = 0; d0 < COLS; d0 += 32) {
          const int d = (TWO ? 0 : slot * COLS) + d0;
          __syncwarp();
          float acc[32];
#pragma unroll
          for (int e = 0; e < 32; ++e) acc[e] = 0.f;
          if (jobs > 0) {
            uint32_t r[32];
            tmem_load(o_at + d, r);
#pragma unroll
            for (int e = 0; e < 32; ++e) acc[e] = __uint_as_float(r[e]) * scale_own;
          }
          if (!TWO && other_jobs > 0) {
            uint32_t r[32];
            tmem_load(o_at + (slot == 0 ? 128 : -128) + d, r);
#pragma unroll
            for (int e = 0; e < 32; ++e) acc[e] = fmaf(__uint_as_float(r[e]), scale_other, acc[e]);
          }
          if (odd && mine) {  // rare: values that are not finite, for the rows that see them
            const int32_t* table = pg.table + static_cast<int64_t>(w.b) * pg.max_pages;
#pragma unroll 1
            for (int ch = t_lo * 4; ch < (t_lo + tiles) * 4; ++ch) {
              if (whole_step(2 * ch) && whole_step(2 * ch + 1)) continue;
#pragma unroll 1
              for (int e = 0; e < 32; ++e) {
                const int step = 2 * ch + e / kStep, s = R.slot(step) + e % kStep;
                if (step >= R.steps || s >= R.end || !sees(s)) continue;
                const int page = __ldg(table + s / pg.page_size);
                if (static_cast<unsigned>(page) >= static_cast<unsigned>(pg.num_pages)) continue;
                const T* v = reinterpret_cast<const T*>(pg.v + page * pg.page_stride + (s % pg.page_size) * pg.slot_stride +
                                                        w.h * pg.head_stride) + d;
#pragma unroll
                for (int x = 0; x < 32; ++x) {
                  const float f = static_cast<float>(v[x]);
                  if (!(fabsf(f) < kInf)) acc[x] += f;
                }
              }
            }
          }
          if (!mine) continue;
          if (begins && ends) {
            uint32_t out[16];
#pragma unroll
            for (int e = 0; e < 16; ++e) {
              out[e] = none ? 0u : Half16<T>::pack(acc[2 * e] * inv, acc[2 * e + 1] * inv);
              if (!S.ok) out[e] = 0x7fff7fffu;
            }
            uint4* dst = reinterpret_cast<uint4*>(static_cast<T*>(P.out) + at * D + d);
#pragma unroll
            for (int e = 0; e < 4; ++e) dst[e] = make_uint4(out[4 * e], out[4 * e + 1], out[4 * e + 2], out[4 * e + 3]);
          } else {
            float4* dst = reinterpret_cast<float4*>(P.part_o + part * D + d);
#pragma unroll
            for (int e = 0; e < 8; ++e) dst[e] = make_float4(acc[4 * e], acc[4 * e + 1], acc[4 * e + 2], acc[4 * e + 3]);
          }
        }
        if (mine && (TWO || slot == 0)) {
          if (begins && ends) {
            if (P.lse) P.lse[at] = !S.ok ? __int_as_float(0x7fffffff) : none ? -kInf : m * kLn2 + logf(l);
          } else {
            P.part_ml[part] = make_float2(m, l);
          }
        }
      }
      if (begins && !ends && tid == 0) P.split[blockIdx.x] = w.split(share);
      tile_base += tiles;
      fence_before();
    } while (w.next());
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
