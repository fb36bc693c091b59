// Attention of a round's query tokens over a paged cache, in 16 or in 4 bits.
//
//   out_i = sum_j p_ij v_j,  p_ij = 2^(s_ij - m) / sum_j 2^(s_ij - m),  s_ij = c q_i.k_j
// over the slots j that query i sees, c = scale * log2(e).  One pass over the keys keeps a
// running maximum m, sum l and unnormalised output O per row (fp32) and rescales them when m
// grows; parts of a row computed apart join as O = sum 2^(m_a - m) O_a, l likewise.
//
// The n * G query rows that share a key head are one matrix (row r: query r / G, head r % G),
// so a cached key is read once for all of them: 4 D flop per row and slot against 4 D bytes.  Up to a
// hundred rows or so the cache's bytes bound the call, beyond that the exponentials and products.
//
// Work split: an item is (sequence, row tile, key head); its visible slots, the first `sinks`
// and the window, make steps of 16 and units of 8 steps.  Every CTA takes an equal, contiguous
// range of all units (an item counting for a few more, kItemUnits), whatever the sequences' lengths,
// found by a scan over the lengths on the device (the host never reads them).  An item cut by a range
// border leaves parts in the workspace, which a second kernel, started while the first one runs, joins in
// a fixed order: the result depends on the number of CTAs only.
//
// Two kernels do the first part.  The one here is for a few rows (kWarpRows): m16n8k16 matrix
// instructions, each of 8 warps with a stream of slots of its own (every 8th step of a segment) and all
// 16 rows of the tile, copied ahead with 16-byte asynchronous copies three stages deep; no barrier
// until the warps join their rows through shared memory, once per segment.  It comes up faster than
// the tensor-memory kernel (attend_tc.cuh), which takes all other calls, and reaches the same share of
// HBM bandwidth on 16-bit pages: B=32, 8 key heads, 8000 slots at most, one token of 32 heads of 64
// in 68 us, 4.8 TB/s, 0.71 of the measured copy rate.  Over 4-bit pages it is bound by the conversion of
// codes (a conversion and a product for every two values, at 64 lanes a clock and SM): the same in
// 66 us, 1.4 TB/s.

#include <algorithm>

#include "attend_common.cuh"
#include "specdec_internal.h"

namespace specdec {

namespace {

constexpr int kRows = 16;     // rows of a tile
// Calls with at most this many query rows to a key head take the kernel here, unless heads of 128 make at
// least an item for every CTA; others the tensor-memory kernel.  Measured on either side (B requests of
// n tokens, 32 query and 8 key heads, us here / there).  128 values: 4 rows, B=1, 900 slots 13.1 / 15.0;
// B=16, 4000 slots 38.8 / 43.8; B=64, 600 slots 40.1 / 36.2; B=32, 8000 slots 116 / 114; 32 rows 210 /
// 118.  4-bit pages: 4 rows, B=1, 900 slots 16.2 / 17.4; B=64, 600 slots 46.9 / 43.6; B=32, 8000 slots
// 99 / 95; 32 rows 191 / 97.  64 values: 4 rows, B=4, 4000 slots 15.0 / 16.4; B=32, 8000 slots 67.8 / 68.3;
// 4-bit pages 15.5 / 19.6 and 68.2 / 70.7; 16 rows, B=32, 8000 slots 68.8 / 68.4 and 72.3 / 70.6.
constexpr int kWarpRows = 8;

__device__ __forceinline__ void load_matrices(uint32_t addr, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr) : "memory");
}
__device__ __forceinline__ void load_matrices_t(uint32_t addr, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr) : "memory");
}
template <typename T>
__device__ __forceinline__ void mma(float (&d)[4], const uint4& a, uint32_t b0, uint32_t b1) {
  if constexpr (sizeof(T) == 2 && std::is_same<T, __nv_bfloat16>::value)
    asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                 : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3]) : "r"(a.x), "r"(a.y), "r"(a.z), "r"(a.w), "r"(b0), "r"(b1));
  else
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                 : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3]) : "r"(a.x), "r"(a.y), "r"(a.z), "r"(a.w), "r"(b0), "r"(b1));
}
// ---- one 16-bit or 4-bit step ------------------------------------------------------------

// Sixteen slots' keys or values as staged: rows of D 16-bit values padded by 16 bytes (so that the
// matrix loads meet no bank conflicts), or rows of codes followed by the rows' scales.
template <int D, bool FOUR>
struct Stage {
  static constexpr int WARPS = 8;
  static constexpr int SUB = FOUR ? 2 : 1;     // steps of 16 that a warp takes at a time
  static constexpr int STAGES = 3;
  static constexpr int kRowBytes = FOUR ? D / 2 : 2 * D;
  static constexpr int kPitch = FOUR ? kRowBytes : kRowBytes + 16;
  static constexpr int kScaleBytes = FOUR ? D / kGroup4 : 0;
  static constexpr int kSide = SUB * kStep * (kPitch + kScaleBytes);  // K or V of a stage
  static constexpr int kBytes = 2 * kSide;
  static constexpr int kStagesBytes = WARPS * STAGES * kBytes;
  static constexpr int kJoinBytes = WARPS * kRows * (D * 4 + 8);  // the warps' rows, joined once per segment
  static constexpr int kOffQ = kStagesBytes > kJoinBytes ? kStagesBytes : kJoinBytes;
  static constexpr int kOffScale = kOffQ + kRows * D * 2;
  static constexpr int kSmem = kOffScale + kRows * 4;
};

template <typename T, int D, bool FOUR>
__global__ void __launch_bounds__(32 * Stage<D, FOUR>::WARPS, 1) attend_kernel(const AttendParams P) {
  using St = Stage<D, FOUR>;
  using M = typename std::conditional<FOUR, __half, T>::type;  // the matrix instructions' type
  constexpr int MR = kRows, WARPS = St::WARPS, SUB = St::SUB, SLOTS = SUB * kStep, STAGES = St::STAGES, THREADS = 32 * WARPS;
  constexpr int KT = D / 16, NT = D / 8;
  extern __shared__ __align__(128) char smem[];
  __shared__ int64_t s_scan[WARPS + 3];
  const Pages& pg = P.pages;
  const int tid = threadIdx.x, warp = tid / 32, lane = tid % 32, g = lane / 4, c = lane % 4;
  const int64_t slots = static_cast<int64_t>(pg.max_pages) * pg.page_size;
  char* const stages = smem + warp * STAGES * St::kBytes;
  float* const s_rowscale = reinterpret_cast<float*>(smem + St::kOffScale);

  // (the launch may overlap the end of the kernel before it: nothing above touches global memory)
  grid_dependency_wait();
  grid_launch_dependents();
  const Share share = scan_units<MR, THREADS>(P, slots, s_scan);
  const int64_t cta = blockIdx.x;
  if (tid == 0) {
    P.split[cta] = make_int4(0, 0, 0, 0);
    P.gave_up[cta] = 0;
  }
  if (share.u >= share.end) return;
  Walk<MR> w(P, slots, share);

  while (true) {
    // ---- the segment [u, seg_end) of item (b, rt, h)
    const SeqLen S = w.S;
    const int b = w.b, h = w.h;
    const int row0 = w.rt * MR, rows = tile_rows<MR>(P, w.rt);
    const Range R = item_range(P, S, row0, rows);
    const int t_lo = static_cast<int>(w.u - w.item) * kUnit;
    const int t_hi = min(static_cast<int>(w.seg_end() - w.item) * kUnit, R.steps);
    const int32_t* table = pg.table + static_cast<int64_t>(b) * pg.max_pages;
    const char* const k_head = pg.k + h * pg.head_stride;
    const char* const v_head = pg.v + h * pg.head_stride;

    // this lane's slot of the steps from t on (SUB = 1: lanes 16..31 repeat 0..15), and its page
    auto slot_of = [&](int t) { return R.slot(t + (SUB == 1 ? 0 : lane / kStep)) + lane % kStep; };
    auto wanted = [&](int t, int s) {
      return t + (SUB == 1 ? 0 : lane / kStep) < t_hi && s < R.end && (s >= R.lo || s < R.sinks);
    };
    auto entry = [&](int t) {
      const int s = slot_of(t);
      return wanted(t, s) ? __ldg(table + page_of(pg, s)) : 0;
    };
    // copies the steps from t on; the slots on pages out of range come back
    auto prefetch = [&](int t, int stage, int page) -> uint32_t {
      uint32_t bads = 0;
      if (t < t_hi) {
        const int s = slot_of(t);
        const bool want = wanted(t, s);
        const bool bad = want && static_cast<unsigned>(page) >= static_cast<unsigned>(pg.num_pages);
        const bool there = want && !bad;
        const int in_page = s - page_of(pg, s) * pg.page_size;
        const int64_t off = there ? page * pg.page_stride + in_page * pg.slot_stride : 0;
        bads = __ballot_sync(0xffffffffu, bad);
        if (SUB == 1) bads &= 0xffffu;
        const uint32_t present = __ballot_sync(0xffffffffu, there);
        char* const base = stages + stage * St::kBytes;
        constexpr int CH = St::kRowBytes / 16;  // 16-byte pieces of a row
        constexpr int RPI = 32 / CH;            // rows a warp copies at a time
#pragma unroll
        for (int j = 0; j < SLOTS / RPI; ++j) {
          const int row = j * RPI + lane / CH, piece = lane % CH;
          const int64_t o = __shfl_sync(0xffffffffu, off, row) + piece * 16;
          const bool ok = (present >> row) & 1u;
          const uint32_t dst = smem_addr(base + row * St::kPitch + piece * 16);
          copy_async<16>(dst, k_head + o, ok);
          copy_async<16>(dst + St::kSide, v_head + o, ok);
        }
        if constexpr (FOUR) {
          const int64_t so = there ? page * pg.scale_page_stride + in_page * pg.scale_slot_stride + h * pg.scale_head_stride : 0;
          const uint32_t dst = smem_addr(base + SLOTS * St::kPitch + lane * St::kScaleBytes);
          copy_async<St::kScaleBytes>(dst, pg.k_scales + so, there);
          copy_async<St::kScaleBytes>(dst + St::kSide, pg.v_scales + so, there);
        }
      }
      copy_commit();
      return bads;
    };

    // ---- the query rows, as the matrix instruction's fragments: [k step][lane]
    __syncthreads();  // the last segment's rows are written: its shared memory is free
    int t_next = t_lo + warp * SUB;  // the next steps this warp copies
    int page_next = entry(t_next);
    uint32_t bad_ring[STAGES];
#pragma unroll
    for (int s = 0; s < STAGES - 1; ++s) {
      const int page = page_next;
      page_next = entry(t_next + WARPS * SUB);
      bad_ring[s] = prefetch(t_next, s, page);
      t_next += WARPS * SUB;
    }
    auto q_row = [&](int r) {
      const int i = query_of(P, row0 + r);
      return static_cast<const T*>(P.q) + b * P.q_sb + i * P.q_st + (h * P.G + row0 + r - i * P.G) * P.q_sh;
    };
    if constexpr (FOUR && !std::is_same<T, __half>::value) {  // a row's power-of-two scale
      for (int r = warp; r < MR; r += WARPS) {
        float a = 0.f;
        if (r < rows)
          for (int d = 2 * lane; d < D; d += 64) {
            const float2 f = Half16<T>::to_f32(__ldg(reinterpret_cast<const uint32_t*>(q_row(r) + d)));
            a = fmaxf(a, fmaxf(fabsf(f.x), fabsf(f.y)));
          }
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) a = fmaxf(a, __shfl_xor_sync(0xffffffffu, a, o));
        // 2^(exponent of the row's largest value): q / it is within (-2, 2), and fp16 then
        // holds a bf16 query to 2^-25 of the row's largest value
        const int e = (__float_as_int(a) >> 23) & 0xff;
        if (lane == 0) s_rowscale[r] = (e == 0 || e == 0xff) ? 1.f : __int_as_float(e << 23);
      }
      __syncthreads();
    }
    for (int f = tid; f < KT * 32; f += THREADS) {
      const int fg = f % 32 / 4, fc = f % 4, t = f / 32;
      uint32_t a[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int r = fg + (e & 1) * 8;  // a0, a2: row g; a1, a3: row g + 8
        // 4-bit pages: the k index runs over D in the order the codes are read in
        const int d = FOUR ? (D / 4) * fc + 4 * t + (e >> 1) * 2 : 16 * t + 2 * fc + (e >> 1) * 8;
        a[e] = r < rows ? __ldg(reinterpret_cast<const uint32_t*>(q_row(r) + d)) : 0u;
        if constexpr (FOUR && !std::is_same<T, __half>::value) {
          const float2 v = Half16<T>::to_f32(a[e]);
          const float inv = 1.f / s_rowscale[r];
          a[e] = Half16<__half>::pack(v.x * inv, v.y * inv);
        }
      }
      reinterpret_cast<uint4*>(smem + St::kOffQ)[f] = make_uint4(a[0], a[1], a[2], a[3]);
    }
    __syncthreads();
    const uint4* const s_q = reinterpret_cast<const uint4*>(smem + St::kOffQ) + lane;

    // this thread's rows: g and g + 8
    int q_i[2], q_pos[2];
    float sc[2], row_m[2], row_l[2];
    float o[NT][4];
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      q_i[e] = query_of(P, row0 + g + e * 8);
      q_pos[e] = S.first + (P.depth && q_i[e] < P.n ? node_depth(P, q_i[e]) : q_i[e]);
      sc[e] = P.scale_log2;
      if constexpr (FOUR && !std::is_same<T, __half>::value) sc[e] *= s_rowscale[g + e * 8];
      row_m[e] = -kInf;
      row_l[e] = 0.f;
    }
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int e = 0; e < 4; ++e) o[nt][e] = 0.f;
    uint4 qf[FOUR ? 1 : KT];  // (16-bit pages: the fragments stay in registers)
    if constexpr (!FOUR) {
#pragma unroll
      for (int t = 0; t < KT; ++t) qf[t] = s_q[t * 32];
    }
    const int i0 = query_of(P, row0), i1 = min(query_of(P, row0 + rows - 1), S.nq - 1);
    const bool tree = P.tree_mask != nullptr;
    auto sees = [&](int e, int s) {
      const int j = s - S.first;
      bool ok = s < R.end;
      int pos = s;
      if (tree) {
        if (j >= 0) {
          ok = ok && q_i[e] < P.n && __ldg(P.tree_mask + static_cast<int64_t>(q_i[e]) * P.n + min(j, P.n - 1)) != 0;
          if (P.depth) pos = S.first + node_depth(P, min(j, P.n - 1));
        }
      } else {
        ok = ok && j <= q_i[e];
      }
      if (P.window > 0) ok = ok && (q_pos[e] - pos < P.window || pos < P.sinks);
      return ok;
    };
    // every row sees the 16 slots of a step
    auto whole_step = [&](int t) {
      const int s0 = R.slot(t);
      bool ok = t < t_hi && s0 + kStep <= R.end && s0 + kStep <= (tree ? S.first : S.first + i0 + 1);
      if (P.window > 0) ok = ok && ((tree ? S.first + P.n - 1 : S.first + i1) - s0 < P.window || s0 + kStep <= P.sinks);
      return ok;
    };

    int stage = 0;
    for (int t = t_lo + warp * SUB; t < t_hi; t += WARPS * SUB) {
      copy_wait<STAGES - 2>();
      __syncwarp();
      const uint32_t bads = bad_ring[0];
      {
        const int page = page_next;
        page_next = entry(t_next + WARPS * SUB);
        const uint32_t next = prefetch(t_next, stage == 0 ? STAGES - 1 : stage - 1, page);
        t_next += WARPS * SUB;
#pragma unroll
        for (int k = 0; k + 2 < STAGES; ++k) bad_ring[k] = bad_ring[k + 1];
        bad_ring[STAGES - 2] = next;
      }
      char* const kb = stages + stage * St::kBytes;
      char* const vb = kb + St::kSide;
      stage = stage + 1 == STAGES ? 0 : stage + 1;

      // S = Q K^T: 16 rows by tiles of 8 slots
      float s_acc[2 * SUB][4];
#pragma unroll
      for (int n = 0; n < 2 * SUB; ++n)
#pragma unroll
        for (int e = 0; e < 4; ++e) s_acc[n][e] = 0.f;
      if constexpr (!FOUR) {
        const uint32_t addr = smem_addr(kb + ((lane & 7) + (lane >> 4) * 8) * St::kPitch + ((lane >> 3) & 1) * 16);
#pragma unroll
        for (int k = 0; k < KT; ++k) {
          uint32_t f[4];
          load_matrices(addr + k * 32, f);
          mma<M>(s_acc[0], qf[k], f[0], f[1]);
          mma<M>(s_acc[1], qf[k], f[2], f[3]);
        }
      } else {
        // lane (g, c) takes D/4 consecutive codes of keys g, g + 8, ...: D/32 words
        constexpr int W = D / 32;
#pragma unroll
        for (int x = 0; x < W; ++x) {  // a word is two k steps
          uint32_t f[2 * SUB][4];
#pragma unroll
          for (int n = 0; n < 2 * SUB; ++n) {
            const uint32_t w32 = *reinterpret_cast<const uint32_t*>(kb + (g + 8 * n) * St::kPitch + c * (D / 8) + 4 * x);
            const uint32_t sb = *reinterpret_cast<const uint8_t*>(kb + SLOTS * St::kPitch + (g + 8 * n) * St::kScaleBytes + c * (W / 2) + x / 2);
            const uint32_t s2 = e4m3x2_to_f16(0x101u * sb);
            e2m1x8_to_f16(w32, f[n][0], f[n][1], f[n][2], f[n][3]);
#pragma unroll
            for (int e = 0; e < 4; ++e) f[n][e] = mul_f16x2(f[n][e], s2);
          }
#pragma unroll
          for (int y = 0; y < 2; ++y) {
            const uint4 a = s_q[(2 * x + y) * 32];
#pragma unroll
            for (int n = 0; n < 2 * SUB; ++n) mma<M>(s_acc[n], a, f[n][2 * y], f[n][2 * y + 1]);
          }
        }
      }

      // scale and mask; a slot on a page out of range gives NaN to the rows that see it
      bool whole = bads == 0;
#pragma unroll
      for (int x = 0; x < SUB; ++x) whole = whole && whole_step(t + x);
      uint32_t seen = 0;  // bit 4 n + e: element e of key tile n is visible
#pragma unroll
      for (int n = 0; n < 2 * SUB; ++n)
#pragma unroll
        for (int e = 0; e < 4; ++e) s_acc[n][e] *= sc[e / 2];
      if (!whole) {
#pragma unroll
        for (int n = 0; n < 2 * SUB; ++n)
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const int key = 8 * n + 2 * c + (e & 1);
            const bool ok = t + key / kStep < t_hi && sees(e / 2, R.slot(t + key / kStep) + key % kStep);
            float v = s_acc[n][e];
            if ((bads >> key) & 1u) v = __int_as_float(0x7fffffff);
            s_acc[n][e] = ok ? v : -kInf;
            seen |= (ok ? 1u : 0u) << (4 * n + e);
          }
      }

      // the running maximum and sum
      float alpha[2];
      uint4 p[SUB];
      {
        float pe[2 * SUB][4];
#pragma unroll
        for (int x = 0; x < 2; ++x) {
          float m = -kInf;
#pragma unroll
          for (int n = 0; n < 2 * SUB; ++n) m = fmaxf(m, fmaxf(s_acc[n][2 * x], s_acc[n][2 * x + 1]));
          m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 1));
          m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 2));
          const float now = fmaxf(row_m[x], m - kBelow<M>);
          const float base = now == -kInf ? 0.f : now;
          alpha[x] = ex2(row_m[x] - base);
          row_m[x] = now;
          float sum = 0.f;
#pragma unroll
          for (int n = 0; n < 2 * SUB; ++n)
#pragma unroll
            for (int y = 0; y < 2; ++y) {
              pe[n][2 * x + y] = ex2(s_acc[n][2 * x + y] - base);
              sum += pe[n][2 * x + y];
            }
          row_l[x] = row_l[x] * alpha[x] + sum;  // this lane's keys; joined at the end
        }
        // P in the matrix type: a rounding of 2^-8 (bf16) or 2^-11 (fp16) of each weight, as large as
        // that of the output itself (fp16 below 2^-21 of the row's largest weight: 2^-32 of that
        // one); l keeps the unrounded weights
#pragma unroll
        for (int u = 0; u < SUB; ++u)
          p[u] = make_uint4(Half16<M>::pack(pe[2 * u][0], pe[2 * u][1]), Half16<M>::pack(pe[2 * u][2], pe[2 * u][3]),
                            Half16<M>::pack(pe[2 * u + 1][0], pe[2 * u + 1][1]), Half16<M>::pack(pe[2 * u + 1][2], pe[2 * u + 1][3]));
      }
      if (__any_sync(0xffffffffu, alpha[0] != 1.f || alpha[1] != 1.f)) {
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int e = 0; e < 4; ++e) o[nt][e] *= alpha[e / 2];
      }

      // A value that is not finite must not reach rows that do not see its slot (0 * inf):
      // steps that some row sees in part look for such values, take them out of the product
      // and add them to the rows that do see them.
      uint32_t odd = 0;
      if (!whole) {
        if constexpr (!FOUR) {
          for (int f = lane; f < SLOTS * (D / 8); f += 32) {
            const uint4 x = *reinterpret_cast<const uint4*>(vb + (f / (D / 8)) * St::kPitch + (f % (D / 8)) * 16);
            const uint32_t ww[4] = {x.x, x.y, x.z, x.w};
            constexpr uint32_t em = std::is_same<T, __half>::value ? 0x7c00u : 0x7f80u;
            bool b4 = false;
#pragma unroll
            for (int e = 0; e < 4; ++e) b4 = b4 || (ww[e] & em) == em || ((ww[e] >> 16) & em) == em;
            if (b4) odd |= 1u << (f / (D / 8));
          }
        } else {
          for (int f = lane; f < SLOTS * St::kScaleBytes; f += 32)
            if ((*reinterpret_cast<const uint8_t*>(vb + SLOTS * St::kPitch + f) & 0x7f) == 0x7f) odd |= 1u << (f / St::kScaleBytes);
        }
        odd = __reduce_or_sync(0xffffffffu, odd);
      }

      // O += P V
#pragma unroll
      for (int u = 0; u < SUB; ++u) {
        const uint32_t odd16 = odd >> (16 * u);
        const uint32_t keep0 = ((odd16 >> (2 * c)) & 1u ? 0u : 0xffffu) | ((odd16 >> (2 * c + 1)) & 1u ? 0u : 0xffff0000u);
        const uint32_t keep1 = ((odd16 >> (2 * c + 8)) & 1u ? 0u : 0xffffu) | ((odd16 >> (2 * c + 9)) & 1u ? 0u : 0xffff0000u);
        if constexpr (!FOUR) {
          const uint32_t addr = smem_addr(vb + ((lane & 7) + ((lane >> 3) & 1) * 8) * St::kPitch + (lane >> 4) * 16);
#pragma unroll
          for (int d = 0; d < NT / 2; ++d) {
            uint32_t f[4];
            load_matrices_t(addr + d * 32, f);
            if (odd) {
              f[0] &= keep0; f[1] &= keep1; f[2] &= keep0; f[3] &= keep1;
            }
            mma<M>(o[2 * d], p[u], f[0], f[1]);
            mma<M>(o[2 * d + 1], p[u], f[2], f[3]);
          }
        } else {
          // lane (g, c) takes values (D/8) g ... of keys 2c, 2c+1, 2c+8, 2c+9: column g of tile
          // nt stands for value (D/8) g + nt
          constexpr int W = D / 64;  // words of those codes
          uint32_t scale[4];
          const char* row[4];
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            const int key = 16 * u + 2 * c + (k & 1) + (k >> 1) * 8;
            row[k] = vb + key * St::kPitch + g * (D / 16);
            scale[k] = *reinterpret_cast<const uint8_t*>(vb + SLOTS * St::kPitch + key * St::kScaleBytes + g * St::kScaleBytes / 8);
          }
          uint32_t s01 = e4m3x2_to_f16(scale[0] | (scale[1] << 8)), s23 = e4m3x2_to_f16(scale[2] | (scale[3] << 8));
          if (odd) {
            s01 &= keep0;
            s23 &= keep1;
          }
#pragma unroll
          for (int x = 0; x < W; ++x) {
            uint32_t f[2][8];
#pragma unroll
            for (int k = 0; k < 2; ++k) {  // pair the two keys' nibbles in a byte, even values then odd ones
              const uint32_t a = reinterpret_cast<const uint32_t*>(row[2 * k])[x], bb = reinterpret_cast<const uint32_t*>(row[2 * k + 1])[x];
              const uint32_t even = (a & 0x0f0f0f0fu) | ((bb & 0x0f0f0f0fu) << 4);
              const uint32_t odds = ((a >> 4) & 0x0f0f0f0fu) | (bb & 0xf0f0f0f0u);
              e2m1x8_to_f16(even, f[k][0], f[k][2], f[k][4], f[k][6]);
              e2m1x8_to_f16(odds, f[k][1], f[k][3], f[k][5], f[k][7]);
#pragma unroll
              for (int e = 0; e < 8; ++e) f[k][e] = mul_f16x2(f[k][e], k == 0 ? s01 : s23);
            }
#pragma unroll
            for (int e = 0; e < 8; ++e) mma<M>(o[8 * x + e], p[u], f[0][e], f[1][e]);
          }
        }
      }
      if (odd) {  // rare: the products taken out above, for the rows that see the slot
#pragma unroll 1
        for (uint32_t left = odd; left; left &= left - 1) {
          const int key = __ffs(left) - 1, n = key / 8;
          const int src = (lane & ~3) | ((key & 7) >> 1);
#pragma unroll
          for (int x = 0; x < 2; ++x) {
            uint32_t mine = 0;
#pragma unroll
            for (int u = 0; u < SUB; ++u) {
              if (n == 2 * u) mine = x ? p[u].y : p[u].x;
              if (n == 2 * u + 1) mine = x ? p[u].w : p[u].z;
            }
            const uint32_t got = __shfl_sync(0xffffffffu, mine, src);
            const uint32_t vis = __shfl_sync(0xffffffffu, seen, src);
            const float2 two = Half16<M>::to_f32(got);
            const float pk = key & 1 ? two.y : two.x;
            if (!((vis >> (4 * n + 2 * x + (key & 1))) & 1u)) continue;
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
              for (int y = 0; y < 2; ++y) {
                float v;
                if constexpr (!FOUR) {
                  const int d = 8 * nt + 2 * c + y;
                  const uint32_t pair = *reinterpret_cast<const uint32_t*>(vb + key * St::kPitch + (d & ~1) * 2);
                  const float2 vv = Half16<T>::to_f32(pair);
                  v = d & 1 ? vv.y : vv.x;
                } else {
                  const int d = (D / 8) * (2 * c + y) + nt;
                  const uint32_t byte = *reinterpret_cast<const uint8_t*>(vb + key * St::kPitch + d / 2);
                  uint32_t f0, f1, f2, f3;
                  e2m1x8_to_f16(d & 1 ? byte >> 4 : byte, f0, f1, f2, f3);
                  const uint32_t sb = *reinterpret_cast<const uint8_t*>(vb + SLOTS * St::kPitch + key * St::kScaleBytes + d / kGroup4);
                  v = Half16<__half>::to_f32(mul_f16x2(f0, e4m3x2_to_f16(sb))).x;
                }
                o[nt][2 * x + y] += pk * v;
              }
          }
        }
      }
    }
    copy_wait<0>();

    // ---- join the warps' rows
    __syncthreads();
    float* const s_o = reinterpret_cast<float*>(smem);                            // [WARPS][MR][D]
    float2* const s_ml = reinterpret_cast<float2*>(smem + WARPS * MR * D * 4);    // [WARPS][MR]
#pragma unroll
    for (int x = 0; x < 2; ++x) {
      float l = row_l[x];
      l += __shfl_xor_sync(0xffffffffu, l, 1);
      l += __shfl_xor_sync(0xffffffffu, l, 2);
      const int r = g + 8 * x;
      if (c == 0) s_ml[warp * MR + r] = make_float2(row_m[x], l);
      float* dst = s_o + (static_cast<size_t>(warp) * MR + r) * D;
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        if constexpr (!FOUR) {
          *reinterpret_cast<float2*>(dst + 8 * nt + 2 * c) = make_float2(o[nt][2 * x], o[nt][2 * x + 1]);
        } else {
          dst[(D / 8) * (2 * c) + nt] = o[nt][2 * x];
          dst[(D / 8) * (2 * c + 1) + nt] = o[nt][2 * x + 1];
        }
      }
    }
    __syncthreads();
    const bool begins = w.u == w.item, ends = w.ends();
    const int part = begins ? 1 : 0;  // a CTA has at most one part that goes on and one that began before
    for (int f = tid; f < MR * (D / 4); f += THREADS) {
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
        const int64_t at = (cta * 2 + part) * MR + r;
        *reinterpret_cast<float4*>(P.part_o + at * D + d) = acc;
        if (d == 0) P.part_ml[at] = make_float2(m, l);
      }
    }
    if (begins && !ends && tid == 0) P.split[cta] = w.split(share);
    if (!w.next()) break;
  }
}

// Joins the parts of items that more than one CTA worked on, and reports the sequences'
// status.  grid (CTAs of the first kernel, parts of a tile's rows): block (c, y) takes the
// item whose first part CTA c left.
constexpr int kJoinWarps = 4;

template <typename T, int D>
__global__ void __launch_bounds__(32 * kJoinWarps) attend_join_kernel(const AttendParams P, int MR) {
  const Pages& pg = P.pages;
  const int64_t slots = static_cast<int64_t>(pg.max_pages) * pg.page_size;
  const int cta = blockIdx.x;
  grid_launch_dependents();
  if (blockIdx.y == 0 && P.out_status) {  // a bad length, or a page that a query sees out of range
    for (int b = cta; b < P.B; b += gridDim.x) {
      const SeqLen S = seq_len(P.context_len, P.query_len, b, P.n, slots);
      int bad = S.ok ? 0 : 1;
      if (S.ok && S.nq > 0 && S.len > 0) {
        const int32_t* table = pg.table + static_cast<int64_t>(b) * pg.max_pages;
        const int lo = P.window > 0 ? max(0, S.first - (P.window - 1)) : 0;
        const int sink_pages = (min(P.sinks, lo) + pg.page_size - 1) / pg.page_size;
        for (int p = threadIdx.x; p <= (S.len - 1) / pg.page_size; p += blockDim.x)
          if (p < sink_pages || p >= lo / pg.page_size)
            bad |= static_cast<unsigned>(__ldg(table + p)) >= static_cast<unsigned>(pg.num_pages);
      }
      bad = __syncthreads_or(bad);
      if (threadIdx.x == 0) P.out_status[b] = bad ? SPECDEC_STATUS_BAD_CACHE : 0;
    }
  }
  grid_dependency_wait();
  if (blockIdx.y == 0 && P.out_status) {  // a bounded wait gave up somewhere: nothing counts
    int late = 0;
    for (int k = threadIdx.x; k < gridDim.x; k += blockDim.x) late |= P.gave_up[k];
    if (__syncthreads_or(late))
      for (int b = cta + threadIdx.x * gridDim.x; b < P.B; b += gridDim.x * blockDim.x) P.out_status[b] |= SPECDEC_STATUS_TIMEOUT;
  }
  const int4 it = P.split[cta];
  const int parts = it.w;
  if (parts == 0) return;
  const int b = it.x, row0 = it.y * MR, h = it.z;
  const int rows = min(MR, P.n * P.G - row0), warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  const SeqLen S = seq_len(P.context_len, P.query_len, b, P.n, slots);
  for (int r = blockIdx.y * kJoinWarps + warp; r < rows; r += gridDim.y * kJoinWarps) {
    auto at = [&](int p) { return (static_cast<int64_t>(cta + p * P.tracks) * 2 + (p == 0 ? 1 : 0)) * MR + r; };
    float m = -kInf;
    for (int p = lane; p < parts; p += 32) m = fmaxf(m, P.part_ml[at(p)].x);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
    const float base = m == -kInf ? 0.f : m;
    constexpr int E = D / 32;  // values of a lane
    float acc[E] = {}, l = 0.f;
#pragma unroll 4
    for (int p = 0; p < parts; ++p) {
      const float2 ml = P.part_ml[at(p)];
      const float a = ex2(ml.x - base);
      l += a * ml.y;
      const float* src = P.part_o + at(p) * D + lane * E;
      if constexpr (E == 4) {
        const float4 x = *reinterpret_cast<const float4*>(src);
        acc[0] += a * x.x; acc[1] += a * x.y; acc[2] += a * x.z; acc[3] += a * x.w;
      } else {
        const float2 x = *reinterpret_cast<const float2*>(src);
        acc[0] += a * x.x; acc[1] += a * x.y;
      }
    }
    const int i = query_of(P, row0 + r), head = h * P.G + row0 + r - i * P.G;
    const int64_t o_at = (static_cast<int64_t>(b) * P.n + i) * P.Hq + head;
    const bool none = l == 0.f || i >= S.nq, undefined = l == 0.f && sees_some(P, S.first, S.nq, i);
    const float inv = none ? 0.f : pg.v_scale / l;
    uint32_t w[E / 2];
#pragma unroll
    for (int e = 0; e < E / 2; ++e) {
      w[e] = none ? 0u : Half16<T>::pack(acc[2 * e] * inv, acc[2 * e + 1] * inv);
      if (undefined) w[e] = 0x7fff7fffu;
    }
    uint32_t* dst = reinterpret_cast<uint32_t*>(static_cast<T*>(P.out) + o_at * D) + lane * (E / 2);
#pragma unroll
    for (int e = 0; e < E / 2; ++e) dst[e] = w[e];
    if (lane == 0 && P.lse) P.lse[o_at] = undefined ? __int_as_float(0x7fffffff) : none ? -kInf : m * kLn2 + logf(l);
  }
}

// ---- launches -----------------------------------------------------------------------------

template <typename T, int D, bool FOUR>
cudaError_t launch_shape(const AttendParams& P, cudaStream_t stream) {
  using St = Stage<D, FOUR>;
  auto kernel = attend_kernel<T, D, FOUR>;
  static_assert(St::kSmem <= 227 * 1024 - 1024, "shared memory of a CTA");
  if (cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, St::kSmem); e != cudaSuccess)
    return e;
  return launch_kernel(kernel, dim3(P.ctas), dim3(32 * St::WARPS), St::kSmem, stream, 1, P);
}

template <typename T>
cudaError_t launch_typed(const AttendParams& P, bool four, cudaStream_t stream) {
  if (P.pages.head_dim == 64) return four ? launch_shape<T, 64, true>(P, stream) : launch_shape<T, 64, false>(P, stream);
  return four ? launch_shape<T, 128, true>(P, stream) : launch_shape<T, 128, false>(P, stream);
}

int attend_sms() {
  int dev = 0, sms = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess)
    return 0;
  return sms;
}
size_t round256(size_t x) { return (x + 255) / 256 * 256; }

constexpr int kMaxCtas = 160;  // the workspace's size does not depend on the device

}  // namespace

size_t attend_workspace_bytes(int n, int G, int D) {
  // (any row tile that a rule or the test hook may choose for these rows)
  const int64_t rows = static_cast<int64_t>(n) * G;
  const size_t mr = rows <= 128 ? 128 : 256;
  return round256(kMaxCtas * sizeof(int4)) + round256(kMaxCtas * sizeof(int)) + round256(kMaxCtas * 2 * mr * sizeof(float2)) +
         round256(kMaxCtas * 2 * mr * static_cast<size_t>(D) * sizeof(float));
}

cudaError_t launch_attend(AttendParams P, specdec_dtype dt, specdec_dtype format, void* workspace, cudaStream_t stream) {
  const int64_t rows = static_cast<int64_t>(P.n) * P.G;
  const bool four = format == SPECDEC_KV4;
  const int hook = test_hook(SPECDEC_HOOK_ATTEND_KERNEL);
  P.ctas = attend_sms();
  if (P.ctas <= 0) return cudaErrorInvalidDevice;
  if (P.ctas > kMaxCtas) P.ctas = kMaxCtas;
  const bool items = P.pages.head_dim == 128 && static_cast<int64_t>(P.B) * P.pages.kv_heads >= P.ctas;
  const bool tc = hook == 0 ? rows > kWarpRows || items : hook == 2;
  const int mr = tc ? attend_tc_rows(rows) : kRows;
  P.row_tiles = static_cast<int>((rows + mr - 1) / mr);
  // A row of CTAs for each key head, unless that leaves more than a sixteenth of the GPU out: a slot's heads
  // lie side by side, and are then read at about the same time (4-bit decode of 64 requests of 16000
  // slots: 1857 MB of DRAM reads and 313 us in one row, 740 MB, the cache's bytes, and 304 us in eight; a prompt chunk 55, 52; 24 requests of 300 slots 26.1, 24.1).
  P.tracks = P.pages.kv_heads <= P.ctas && (P.ctas % P.pages.kv_heads) * 16 <= P.ctas ? P.pages.kv_heads : 1;
  char* ws = static_cast<char*>(workspace);
  P.split = reinterpret_cast<int4*>(ws);
  ws += round256(kMaxCtas * sizeof(int4));
  P.gave_up = reinterpret_cast<int*>(ws);
  ws += round256(kMaxCtas * sizeof(int));
  P.part_ml = reinterpret_cast<float2*>(ws);
  ws += round256(static_cast<size_t>(kMaxCtas) * 2 * mr * sizeof(float2));
  P.part_o = reinterpret_cast<float*>(ws);
  if (tc)
    if (cudaError_t e = four ? launch_attend_tc4(P, dt, mr, stream) : launch_attend_tc(P, dt, mr, stream); e != cudaSuccess)
      return e;
  if (!tc)
    if (cudaError_t e = dt == SPECDEC_BF16 ? launch_typed<__nv_bfloat16>(P, four, stream)
                                           : launch_typed<__half>(P, four, stream);
        e != cudaSuccess)
      return e;
  auto join = P.pages.head_dim == 64
                  ? (dt == SPECDEC_BF16 ? attend_join_kernel<__nv_bfloat16, 64> : attend_join_kernel<__half, 64>)
                  : (dt == SPECDEC_BF16 ? attend_join_kernel<__nv_bfloat16, 128> : attend_join_kernel<__half, 128>);
  // a warp a row, as far as 16 blocks to an item go
  const int64_t item_rows = rows < mr ? rows : mr;
  const int blocks = static_cast<int>(std::min<int64_t>((item_rows + kJoinWarps - 1) / kJoinWarps, 16));
  return launch_kernel(join, dim3(P.ctas, blocks), dim3(32 * kJoinWarps), 0, stream, 1, P, int{mr});
}

}  // namespace specdec
