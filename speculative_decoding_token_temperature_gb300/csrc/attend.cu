// Attention of a round's query tokens over a paged cache, in 16 or in 4 bits.
//
//   out_i = sum_j p_ij v_j,  p_ij = 2^(s_ij - m) / sum_j 2^(s_ij - m),  s_ij = c q_i.k_j
// over the slots j that query i sees, c = scale * log2(e).  One pass over the keys keeps a
// running maximum m, sum l and unnormalised output O per row (fp32) and rescales them when m
// grows; parts of a row computed apart join as O = sum 2^(m_a - m) O_a, l likewise.
//
// The n * G query rows that share a key head are one matrix (row r: query r / G, head r % G),
// so a cached key is read once for all of them.  Row tiles of 16, 32 or 64 rows go through
// m16n8k16 matrix instructions.  Below about 64 rows per key head the cache's bytes bound the
// call: 4 D flop per row and slot against 4 D bytes.
//
// Work split: an item is (sequence, row tile, key head); its visible slots, the first `sinks`
// and the window, make steps of 16 and units of 8 steps.  Every CTA takes an equal, contiguous
// range of all units, whatever the sequences' lengths, found by a scan over the lengths on the
// device (the host never reads them).  An item cut by a range border leaves parts in the
// workspace, which a second kernel, started while the first one runs, joins in a fixed order:
// the result depends on the number of CTAs only.
//
// In a CTA, 8 warps: WR of them share a stream of keys and split the tile's rows, and 8 / WR
// such groups take every (8 / WR)-th step of a segment.  Each group copies its own steps ahead
// with 16-byte asynchronous copies, several stages deep, with no CTA-wide barrier; the groups
// join their rows through shared memory once per segment.  Rows of the staged keys are padded
// by 16 bytes, so the matrix loads meet no bank conflicts.

#include "attend_common.cuh"
#include "specdec_internal.h"

namespace specdec {

namespace {

constexpr int kWarps = 8;
constexpr int kThreads = 32 * kWarps;

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
// Barrier of the warps that share a stream of keys (one warp: its own lanes).
template <int WR>
__device__ __forceinline__ void group_sync(int group) {
  if constexpr (WR == 1)
    __syncwarp();
  else
    asm volatile("bar.sync %0, %1;" ::"r"(1 + group), "n"(32 * WR) : "memory");
}

// ---- one 16-bit or 4-bit step ------------------------------------------------------------

template <int D, bool FOUR>
struct Stage {
  static constexpr int kRowBytes = FOUR ? D / 2 : 2 * D;
  static constexpr int kPitch = FOUR ? kRowBytes : kRowBytes + 16;
  static constexpr int kScaleBytes = FOUR ? D / kGroup4 : 0;
  static constexpr int kSide = kStep * (kPitch + kScaleBytes);  // K or V of a step
  static constexpr int kBytes = 2 * kSide;
};

template <int D, bool FOUR, int MT, int WR>
struct Shape {
  static constexpr int MR = 16 * MT * WR;
  static constexpr int GROUPS = kWarps / WR;
  static constexpr int STAGES = FOUR ? 6 : (WR == 1 ? 3 : 5);
  static constexpr int kStagesBytes = GROUPS * STAGES * Stage<D, FOUR>::kBytes;
  static constexpr int kJoinBytes = GROUPS * MR * (D * 4 + 8);  // the groups' rows, joined once per segment
  static constexpr int kQBytes = MR * D * 2;
  static constexpr int kOffQ = kStagesBytes > kJoinBytes ? kStagesBytes : kJoinBytes;
  static constexpr int kOffScale = kOffQ + kQBytes;
  static constexpr int kOffBad = kOffScale + MR * 4;
  static constexpr int kBytes = kOffBad + GROUPS * STAGES * 4;
};

template <typename T, int D, bool FOUR, int MT, int WR>
__global__ void __launch_bounds__(kThreads, 1) attend_kernel(const AttendParams P) {
  using Sh = Shape<D, FOUR, MT, WR>;
  using St = Stage<D, FOUR>;
  using M = typename std::conditional<FOUR, __half, T>::type;  // the matrix instructions' type
  constexpr int MR = Sh::MR, GROUPS = Sh::GROUPS, STAGES = Sh::STAGES, KT = D / 16, NT = D / 8;
  extern __shared__ __align__(128) char smem[];
  __shared__ int64_t s_scan[kWarps + 2];
  const Pages& pg = P.pages;
  const int tid = threadIdx.x, warp = tid / 32, lane = tid % 32, g = lane / 4, c = lane % 4;
  const int group = warp / WR, wr = warp % WR;
  const int64_t slots = static_cast<int64_t>(pg.max_pages) * pg.page_size;
  char* const stages = smem + group * STAGES * St::kBytes;
  float* const s_rowscale = reinterpret_cast<float*>(smem + Sh::kOffScale);
  uint32_t* const s_bad = reinterpret_cast<uint32_t*>(smem + Sh::kOffBad) + group * STAGES;

  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const Share share = scan_units<MR, kThreads>(P, slots, s_scan);
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
    const int b = w.b, rt = w.rt, h = w.h;
    const int64_t u = w.u, item = w.item, seg_end = w.seg_end();
    const int row0 = rt * MR, rows = tile_rows<MR>(P, rt);
    const Range R = item_range(P, S, row0, rows);
    const int t_lo = static_cast<int>(u - item) * kUnit;
    const int t_hi = min(static_cast<int>(seg_end - item) * kUnit, R.steps);
    const int32_t* table = pg.table + static_cast<int64_t>(b) * pg.max_pages;
    const char* const k_head = pg.k + h * pg.head_stride;
    const char* const v_head = pg.v + h * pg.head_stride;
    const char* const ks_head = pg.k_scales + h * pg.scale_head_stride;
    const char* const vs_head = pg.v_scales + h * pg.scale_head_stride;

    // the table entry of this lane's slot of step t (lanes 16..31 repeat 0..15)
    auto entry = [&](int t) {
      const int s = R.slot(t) + (lane & 15);
      return t < t_hi && s < R.end ? __ldg(table + page_of(pg, s)) : 0;
    };
    auto prefetch = [&](int t, int stage, int page) {
      if (t < t_hi) {
        const int s = R.slot(t) + (lane & 15);
        const bool bad = s < R.end && static_cast<unsigned>(page) >= static_cast<unsigned>(pg.num_pages);
        const bool there = s < R.end && !bad;
        const int in_page = s - page_of(pg, s) * pg.page_size;
        const int64_t off = there ? page * pg.page_stride + in_page * pg.slot_stride : 0;
        const uint32_t bads = __ballot_sync(0xffffffffu, bad) & 0xffffu;
        const uint32_t present = __ballot_sync(0xffffffffu, there);
        if (lane == 0 && wr == 0) s_bad[stage] = bads;
        char* base = stages + stage * St::kBytes;
        constexpr int CH = St::kRowBytes / 16;        // 16-byte pieces of a row
        constexpr int RPI = 32 / CH;                  // rows a warp copies at a time
#pragma unroll
        for (int j = 0; j < kStep / RPI; ++j) {
          if (WR > 1 && j % WR != wr) continue;
          const int row = j * RPI + lane / CH, piece = lane % CH;
          const int64_t o = __shfl_sync(0xffffffffu, off, row);
          const bool ok = (present >> row) & 1u;
          const uint32_t dst = smem_addr(base + row * St::kPitch + piece * 16);
          copy_async<16>(dst, k_head + o + piece * 16, ok);
          copy_async<16>(dst + St::kSide, v_head + o + piece * 16, ok);
        }
        if constexpr (FOUR) {
          if (wr == 0) {  // lanes 0..15 the keys' scales, 16..31 the values'
            const int64_t so = there ? page * pg.scale_page_stride + in_page * pg.scale_slot_stride : 0;
            const uint32_t dst = smem_addr(base + kStep * St::kPitch + (lane & 15) * St::kScaleBytes);
            copy_async<St::kScaleBytes>(lane < 16 ? dst : dst + St::kSide, (lane < 16 ? ks_head : vs_head) + so, there);
          }
        }
      }
      copy_commit();
    };

    // ---- the query rows, as the matrix instruction's fragments: [wr][mt][k step][lane]
    __syncthreads();  // the last segment's rows are written: its shared memory is free
    int t_next = t_lo + group;  // the next step this group copies
    int page_next = entry(t_next);
#pragma unroll
    for (int s = 0; s < STAGES - 1; ++s) {
      const int page = page_next;
      page_next = entry(t_next + GROUPS);
      prefetch(t_next, s, page);
      t_next += GROUPS;
    }
    for (int r = warp; r < MR; r += kWarps) {  // a row's power-of-two scale (4-bit caches)
      if constexpr (FOUR && !std::is_same<T, __half>::value) {
        float a = 0.f;
        if (r < rows) {
          const T* src = static_cast<const T*>(P.q) + b * P.q_sb + query_of(P, row0 + r) * P.q_st +
                         (h * P.G + (row0 + r) - query_of(P, row0 + r) * P.G) * P.q_sh;
          for (int d = 2 * lane; d < D; d += 64) {
            const float2 f = Half16<T>::to_f32(*reinterpret_cast<const uint32_t*>(src + d));
            a = fmaxf(a, fmaxf(fabsf(f.x), fabsf(f.y)));
          }
        }
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) a = fmaxf(a, __shfl_xor_sync(0xffffffffu, a, o));
        // 2^(exponent of the row's largest value): q / it is within (-2, 2), and fp16 then
        // holds a bf16 query to 2^-25 of the row's largest value
        const int e = (__float_as_int(a) >> 23) & 0xff;
        if (lane == 0) s_rowscale[r] = (e == 0 || e == 0xff) ? 1.f : __int_as_float(e << 23);
      } else {
        if (lane == 0) s_rowscale[r] = 1.f;
      }
    }
    if constexpr (FOUR) __syncthreads();
    for (int f = tid; f < WR * MT * KT * 32; f += kThreads) {
      const int fl = f % 32, fg = fl / 4, fc = fl % 4, t = (f / 32) % KT, m = f / (32 * KT);
      uint32_t a[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int r = 16 * m + fg + (e & 1) * 8;  // a0, a2: row g; a1, a3: row g + 8
        // 4-bit caches: the k index runs over D in the order the codes are read in
        const int d = FOUR ? (D / 4) * fc + 4 * t + (e >> 1) * 2 : 16 * t + 2 * fc + (e >> 1) * 8;
        uint32_t w = 0;
        if (r < rows) {
          const T* src = static_cast<const T*>(P.q) + b * P.q_sb + query_of(P, row0 + r) * P.q_st +
                         (h * P.G + (row0 + r) - query_of(P, row0 + r) * P.G) * P.q_sh;
          w = *reinterpret_cast<const uint32_t*>(src + d);
          if constexpr (FOUR && !std::is_same<T, __half>::value) {
            const float2 v = Half16<T>::to_f32(w);
            const float inv = 1.f / s_rowscale[r];
            w = Half16<__half>::pack(v.x * inv, v.y * inv);
          }
        }
        a[e] = w;
      }
      reinterpret_cast<uint4*>(smem + Sh::kOffQ)[f] = make_uint4(a[0], a[1], a[2], a[3]);
    }
    __syncthreads();
    const uint4* const s_q = reinterpret_cast<const uint4*>(smem + Sh::kOffQ) + wr * MT * KT * 32 + lane;

    // this thread's rows: 16 mt + g and 16 mt + g + 8 of its warp's part of the tile
    int q_i[2 * MT], q_pos[2 * MT];
    float sc[2 * MT], row_m[2 * MT], row_l[2 * MT];
    float o[MT][NT][4];
#pragma unroll
    for (int e = 0; e < 2 * MT; ++e) {
      const int r = 16 * (wr * MT + e / 2) + g + (e % 2) * 8;
      q_i[e] = query_of(P, row0 + r);
      q_pos[e] = S.first + (P.depth && q_i[e] < P.n ? node_depth(P, q_i[e]) : q_i[e]);
      sc[e] = P.scale_log2 * s_rowscale[r];
      row_m[e] = -kInf;
      row_l[e] = 0.f;
    }
#pragma unroll
    for (int mt = 0; mt < MT; ++mt)
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int e = 0; e < 4; ++e) o[mt][nt][e] = 0.f;
    uint4 qf[MT == 1 ? KT : 1];
    if constexpr (MT == 1) {
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

    int stage = 0;
    for (int t = t_lo + group; t < t_hi; t += GROUPS) {
      copy_wait<STAGES - 2>();
      group_sync<WR>(group);
      {
        const int page = page_next;
        page_next = entry(t_next + GROUPS);
        prefetch(t_next, stage == 0 ? STAGES - 1 : stage - 1, page);
        t_next += GROUPS;
      }
      char* const kb = stages + stage * St::kBytes;
      char* const vb = kb + St::kSide;
      const uint32_t bads = s_bad[stage];
      stage = stage + 1 == STAGES ? 0 : stage + 1;

      // S = Q K^T: 16 MT rows by two tiles of 8 keys
      float s_acc[MT][2][4];
#pragma unroll
      for (int mt = 0; mt < MT; ++mt)
#pragma unroll
        for (int n = 0; n < 2; ++n)
#pragma unroll
          for (int e = 0; e < 4; ++e) s_acc[mt][n][e] = 0.f;
      if constexpr (!FOUR) {
        const uint32_t addr = smem_addr(kb + ((lane & 7) + (lane >> 4) * 8) * St::kPitch + ((lane >> 3) & 1) * 16);
#pragma unroll
        for (int k = 0; k < KT; ++k) {
          uint32_t f[4];
          load_matrices(addr + k * 32, f);
#pragma unroll
          for (int mt = 0; mt < MT; ++mt) {
            const uint4 a = MT == 1 ? qf[MT == 1 ? k : 0] : s_q[(mt * KT + k) * 32];
            mma<M>(s_acc[mt][0], a, f[0], f[1]);
            mma<M>(s_acc[mt][1], a, f[2], f[3]);
          }
        }
      } else {
        // lane (g, c) takes D/4 consecutive codes of keys g and g + 8
        constexpr int W = D / 32;  // 32-bit words of those codes
        uint32_t w[2][W], scale2[2][W / 2];
#pragma unroll
        for (int n = 0; n < 2; ++n) {
          const char* row = kb + (g + 8 * n) * St::kPitch + c * (D / 8);
          if constexpr (W == 4) {
            const uint4 x = *reinterpret_cast<const uint4*>(row);
            w[n][0] = x.x; w[n][1] = x.y; w[n][2] = x.z; w[n][3] = x.w;
          } else {
            const uint2 x = *reinterpret_cast<const uint2*>(row);
            w[n][0] = x.x; w[n][1] = x.y;
          }
          const char* sr = kb + kStep * St::kPitch + (g + 8 * n) * St::kScaleBytes + c * (W / 2);
#pragma unroll
          for (int x = 0; x < W / 2; ++x) scale2[n][x] = e4m3x2_to_f16(0x101u * *reinterpret_cast<const uint8_t*>(sr + x));
        }
#pragma unroll
        for (int x = 0; x < W; ++x) {  // a word is two k steps
          uint32_t f[2][4];
#pragma unroll
          for (int n = 0; n < 2; ++n) {
            e2m1x8_to_f16(w[n][x], f[n][0], f[n][1], f[n][2], f[n][3]);
#pragma unroll
            for (int e = 0; e < 4; ++e) f[n][e] = mul_f16x2(f[n][e], scale2[n][x / 2]);
          }
#pragma unroll
          for (int y = 0; y < 2; ++y) {
            const int k = 2 * x + y;
#pragma unroll
            for (int mt = 0; mt < MT; ++mt) {
              const uint4 a = MT == 1 ? qf[MT == 1 ? k : 0] : s_q[(mt * KT + k) * 32];
              mma<M>(s_acc[mt][0], a, f[0][2 * y], f[0][2 * y + 1]);
              mma<M>(s_acc[mt][1], a, f[1][2 * y], f[1][2 * y + 1]);
            }
          }
        }
      }

      // scale and mask; a slot on a page out of range gives NaN to the rows that see it
      const int s0 = R.slot(t);
      bool whole = s0 + kStep <= R.end && bads == 0;
      if (tree) {
        whole = whole && s0 + kStep <= S.first;
        if (P.window > 0) whole = whole && (S.first + P.n - 1 - s0 < P.window || s0 + kStep <= P.sinks);
      } else {
        whole = whole && s0 + kStep - 1 <= S.first + i0;
        if (P.window > 0) whole = whole && (S.first + i1 - s0 < P.window || s0 + kStep <= P.sinks);
      }
      uint32_t seen[MT];  // bit 8 e + 2 n + x: element (row e of mt, key tile n, x) is visible
#pragma unroll
      for (int mt = 0; mt < MT; ++mt) {
        seen[mt] = 0;
#pragma unroll
        for (int n = 0; n < 2; ++n)
#pragma unroll
          for (int e = 0; e < 4; ++e) s_acc[mt][n][e] *= sc[2 * mt + e / 2];
      }
      if (!whole) {
#pragma unroll
        for (int mt = 0; mt < MT; ++mt)
#pragma unroll
          for (int n = 0; n < 2; ++n)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const int key = 8 * n + 2 * c + (e & 1);
              const bool ok = sees(2 * mt + e / 2, s0 + key);
              float v = s_acc[mt][n][e];
              if ((bads >> key) & 1u) v = __int_as_float(0x7fffffff);
              s_acc[mt][n][e] = ok ? v : -kInf;
              seen[mt] |= (ok ? 1u : 0u) << (8 * (e / 2) + 2 * n + (e & 1));
            }
      }

      // the running maximum and sum
      uint4 p[MT];
#pragma unroll
      for (int mt = 0; mt < MT; ++mt) {
        float pe[2][4];
#pragma unroll
        for (int x = 0; x < 2; ++x) {
          float m = fmaxf(fmaxf(s_acc[mt][0][2 * x], s_acc[mt][0][2 * x + 1]),
                          fmaxf(s_acc[mt][1][2 * x], s_acc[mt][1][2 * x + 1]));
          m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 1));
          m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 2));
          const float old = row_m[2 * mt + x], now = fmaxf(old, m);
          const float base = now == -kInf ? 0.f : now;
          const float alpha = ex2(old - base);
          row_m[2 * mt + x] = now;
          float sum = 0.f;
#pragma unroll
          for (int n = 0; n < 2; ++n)
#pragma unroll
            for (int y = 0; y < 2; ++y) {
              const float v = ex2(s_acc[mt][n][2 * x + y] - base);
              pe[n][2 * x + y] = v;
              sum += v;
            }
          row_l[2 * mt + x] = row_l[2 * mt + x] * alpha + sum;  // this lane's keys; joined at the end
          if (__any_sync(0xffffffffu, alpha != 1.f)) {
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
              o[mt][nt][2 * x] *= alpha;
              o[mt][nt][2 * x + 1] *= alpha;
            }
          }
        }
        // P in the matrix type: a rounding of 2^-9 (bf16) or 2^-12 (fp16) of each weight, as
        // large as that of the output itself; l keeps the unrounded weights
        p[mt] = make_uint4(Half16<M>::pack(pe[0][0], pe[0][1]), Half16<M>::pack(pe[0][2], pe[0][3]),
                           Half16<M>::pack(pe[1][0], pe[1][1]), Half16<M>::pack(pe[1][2], pe[1][3]));
      }

      // A value that is not finite must not reach rows that do not see its slot (0 * inf):
      // steps that some row sees in part look for such values, take them out of the product
      // and add them to the rows that do see them.
      uint32_t odd = 0;
      if (!whole) {
        if constexpr (!FOUR) {
          for (int f = lane; f < kStep * (D / 8); f += 32) {
            const uint4 x = *reinterpret_cast<const uint4*>(vb + (f / (D / 8)) * St::kPitch + (f % (D / 8)) * 16);
            const uint32_t ww[4] = {x.x, x.y, x.z, x.w};
            constexpr uint32_t em = std::is_same<T, __half>::value ? 0x7c00u : 0x7f80u;
            bool b4 = false;
#pragma unroll
            for (int e = 0; e < 4; ++e) b4 = b4 || (ww[e] & em) == em || ((ww[e] >> 16) & em) == em;
            if (b4) odd |= 1u << (f / (D / 8));
          }
        } else {
          for (int f = lane; f < kStep * St::kScaleBytes; f += 32)
            if ((*reinterpret_cast<const uint8_t*>(vb + kStep * St::kPitch + f) & 0x7f) == 0x7f) odd |= 1u << (f / St::kScaleBytes);
        }
        odd = __reduce_or_sync(0xffffffffu, odd);
      }
      const uint32_t keep0 = ((odd >> (2 * c)) & 1u ? 0u : 0xffffu) | ((odd >> (2 * c + 1)) & 1u ? 0u : 0xffff0000u);
      const uint32_t keep1 = ((odd >> (2 * c + 8)) & 1u ? 0u : 0xffffu) | ((odd >> (2 * c + 9)) & 1u ? 0u : 0xffff0000u);

      // O += P V
      if constexpr (!FOUR) {
        const uint32_t addr = smem_addr(vb + ((lane & 7) + ((lane >> 3) & 1) * 8) * St::kPitch + (lane >> 4) * 16);
#pragma unroll
        for (int d = 0; d < NT / 2; ++d) {
          uint32_t f[4];
          load_matrices_t(addr + d * 32, f);
          if (odd) {
            f[0] &= keep0; f[1] &= keep1; f[2] &= keep0; f[3] &= keep1;
          }
#pragma unroll
          for (int mt = 0; mt < MT; ++mt) {
            mma<M>(o[mt][2 * d], p[mt], f[0], f[1]);
            mma<M>(o[mt][2 * d + 1], p[mt], f[2], f[3]);
          }
        }
      } else {
        // lane (g, c) takes values (D/8) g ... of keys 2c, 2c+1, 2c+8, 2c+9: column g of tile
        // nt stands for value (D/8) g + nt
        constexpr int W = D / 64;  // words of those codes
        uint32_t w[4][W], scale[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const int key = 2 * c + (k & 1) + (k >> 1) * 8;
          const char* row = vb + key * St::kPitch + g * (D / 16);
#pragma unroll
          for (int x = 0; x < W; ++x) w[k][x] = reinterpret_cast<const uint32_t*>(row)[x];
          scale[k] = *reinterpret_cast<const uint8_t*>(vb + kStep * St::kPitch + key * St::kScaleBytes + g * St::kScaleBytes / 8);
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
            const uint32_t a = w[2 * k][x], bb = w[2 * k + 1][x];
            const uint32_t even = (a & 0x0f0f0f0fu) | ((bb & 0x0f0f0f0fu) << 4);
            const uint32_t odds = ((a >> 4) & 0x0f0f0f0fu) | (bb & 0xf0f0f0f0u);
            e2m1x8_to_f16(even, f[k][0], f[k][2], f[k][4], f[k][6]);
            e2m1x8_to_f16(odds, f[k][1], f[k][3], f[k][5], f[k][7]);
#pragma unroll
            for (int e = 0; e < 8; ++e) f[k][e] = mul_f16x2(f[k][e], k == 0 ? s01 : s23);
          }
#pragma unroll
          for (int e = 0; e < 8; ++e)
#pragma unroll
            for (int mt = 0; mt < MT; ++mt) mma<M>(o[mt][8 * x + e], p[mt], f[0][e], f[1][e]);
        }
      }
      if (odd) {  // rare: the products taken out above, for the rows that see the slot
#pragma unroll 1
        for (uint32_t left = odd; left; left &= left - 1) {
          const int key = __ffs(left) - 1;
          const int src = (lane & ~3) | ((key & 7) >> 1);
#pragma unroll
          for (int mt = 0; mt < MT; ++mt)
#pragma unroll
            for (int x = 0; x < 2; ++x) {
              const uint32_t pw = key < 8 ? (x ? p[mt].y : p[mt].x) : (x ? p[mt].w : p[mt].z);
              const uint32_t got = __shfl_sync(0xffffffffu, pw, src);
              const uint32_t vis = __shfl_sync(0xffffffffu, seen[mt], src);
              const float2 two = Half16<M>::to_f32(got);
              const float pk = key & 1 ? two.y : two.x;
              if (!((vis >> (8 * x + 2 * (key >> 3) + (key & 1))) & 1u)) continue;
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
                    const uint32_t sb = *reinterpret_cast<const uint8_t*>(vb + kStep * St::kPitch + key * St::kScaleBytes + d / kGroup4);
                    v = Half16<__half>::to_f32(mul_f16x2(f0, e4m3x2_to_f16(sb))).x;
                  }
                  o[mt][nt][2 * x + y] += pk * v;
                }
            }
        }
      }
    }
    copy_wait<0>();

    // ---- join the groups' rows
    __syncthreads();
    float* const s_o = reinterpret_cast<float*>(smem);                               // [GROUPS][MR][D]
    float2* const s_ml = reinterpret_cast<float2*>(smem + GROUPS * MR * D * 4);      // [GROUPS][MR]
#pragma unroll
    for (int mt = 0; mt < MT; ++mt)
#pragma unroll
      for (int x = 0; x < 2; ++x) {
        float l = row_l[2 * mt + x];
        l += __shfl_xor_sync(0xffffffffu, l, 1);
        l += __shfl_xor_sync(0xffffffffu, l, 2);
        const int r = 16 * (wr * MT + mt) + g + 8 * x;
        if (c == 0) s_ml[group * MR + r] = make_float2(row_m[2 * mt + x], l);
        float* dst = s_o + (static_cast<size_t>(group) * MR + r) * D;
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          if constexpr (!FOUR) {
            *reinterpret_cast<float2*>(dst + 8 * nt + 2 * c) = make_float2(o[mt][nt][2 * x], o[mt][nt][2 * x + 1]);
          } else {
            dst[(D / 8) * (2 * c) + nt] = o[mt][nt][2 * x];
            dst[(D / 8) * (2 * c + 1) + nt] = o[mt][nt][2 * x + 1];
          }
        }
      }
    __syncthreads();
    const bool begins = u == item, ends = seg_end == item + w.units;
    const int part = begins ? 1 : 0;  // a CTA has at most one part that goes on and one that began before
    for (int f = tid; f < MR * (D / 4); f += kThreads) {
      const int r = f / (D / 4), d = (f % (D / 4)) * 4;
      if (r >= rows) continue;
      float m = -kInf;
#pragma unroll
      for (int k = 0; k < GROUPS; ++k) m = fmaxf(m, s_ml[k * MR + r].x);
      const float base = m == -kInf ? 0.f : m;
      float l = 0.f;
      float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
      for (int k = 0; k < GROUPS; ++k) {
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
        if (!S.ok) {
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
  asm volatile("griddepcontrol.wait;" ::: "memory");
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
    auto at = [&](int p) { return (static_cast<int64_t>(cta + p) * 2 + (p == 0 ? 1 : 0)) * MR + r; };
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
    const bool none = l == 0.f || i >= S.nq;
    const float inv = none ? 0.f : pg.v_scale / l;
    uint32_t w[E / 2];
#pragma unroll
    for (int e = 0; e < E / 2; ++e) w[e] = none ? 0u : Half16<T>::pack(acc[2 * e] * inv, acc[2 * e + 1] * inv);
    uint32_t* dst = reinterpret_cast<uint32_t*>(static_cast<T*>(P.out) + o_at * D) + lane * (E / 2);
#pragma unroll
    for (int e = 0; e < E / 2; ++e) dst[e] = w[e];
    if (lane == 0 && P.lse) P.lse[o_at] = none ? -kInf : m * kLn2 + logf(l);
  }
}

// ---- launches -----------------------------------------------------------------------------

// Row tile: the smallest of 16, 32 and 64 that holds a key head's rows; more rows take
// several tiles of 64.
int row_tile(int64_t rows) { return rows <= 16 ? 16 : rows <= 32 ? 32 : 64; }

template <typename T, int D, bool FOUR, int MT, int WR>
cudaError_t launch_shape(const AttendParams& P, cudaStream_t stream) {
  using Sh = Shape<D, FOUR, MT, WR>;
  auto kernel = attend_kernel<T, D, FOUR, MT, WR>;
  if (cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, Sh::kBytes); e != cudaSuccess)
    return e;
  return launch_kernel(kernel, dim3(P.ctas), dim3(kThreads), Sh::kBytes, stream, 0, P);
}

template <typename T, int D, bool FOUR>
cudaError_t launch_rows(const AttendParams& P, int mr, cudaStream_t stream) {
  if (mr == 16) return launch_shape<T, D, FOUR, 1, 1>(P, stream);
  if (mr == 32) return launch_shape<T, D, FOUR, 2, 1>(P, stream);
  return launch_shape<T, D, FOUR, 2, 2>(P, stream);
}

template <typename T>
cudaError_t launch_typed(const AttendParams& P, int mr, bool four, cudaStream_t stream) {
  if (P.pages.head_dim == 64)
    return four ? launch_rows<T, 64, true>(P, mr, stream) : launch_rows<T, 64, false>(P, mr, stream);
  return four ? launch_rows<T, 128, true>(P, mr, stream) : launch_rows<T, 128, false>(P, mr, stream);
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
  const bool tc = hook == 0 ? rows > 16 : hook == 2;
  const int mr = tc ? attend_tc_rows(rows) : row_tile(rows);
  P.row_tiles = static_cast<int>((rows + mr - 1) / mr);
  P.ctas = attend_sms();
  if (P.ctas <= 0) return cudaErrorInvalidDevice;
  if (P.ctas > kMaxCtas) P.ctas = kMaxCtas;
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
    if (cudaError_t e = dt == SPECDEC_BF16 ? launch_typed<__nv_bfloat16>(P, mr, four, stream)
                                           : launch_typed<__half>(P, mr, four, stream);
        e != cudaSuccess)
      return e;
  auto join = P.pages.head_dim == 64
                  ? (dt == SPECDEC_BF16 ? attend_join_kernel<__nv_bfloat16, 64> : attend_join_kernel<__half, 64>)
                  : (dt == SPECDEC_BF16 ? attend_join_kernel<__nv_bfloat16, 128> : attend_join_kernel<__half, 128>);
  return launch_kernel(join, dim3(P.ctas, mr / (2 * kJoinWarps)), dim3(32 * kJoinWarps), 0, stream, 1, P, int{mr});
}

}  // namespace specdec
