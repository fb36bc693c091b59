// Attention over 8-bit pages for a few rows to a key head (up to 32), on warp-level matrix instructions.
//
// The formula, the items, the split of the work and the join are those of attend.cu.  Keys and values are
// E4M3 codes, and the slots of a step of 16 lie in one block, so they share a scale 2^e for keys and one for values:
//   s_ij = (c 2^e_k) (q_i . code_j),   O_i += p_ij (2^e_v code_j)
// Codes are exact in fp16, and so are values, 2^e_v code (e from -15 to 7), so the products are those of
// fp16 with fp32 sums; the keys' scale goes into the scores' factor.  Queries in bf16 are held in fp16 relative to a power of
// two of their row, to 2^-25 of its largest value.
//
// Codes go from the copied tile straight into the matrix instruction's registers: a key's row is read in the order that makes a
// word the four codes of a step of the k index, two keys' words are interleaved by bytes for the product with V.
// So shared memory carries the codes once in and once out, and a conversion serves all rows of the tile: 16 rows, or 32 whose
// second 16 use the same registers of codes.

#include "attend_common.cuh"
#include "specdec_internal.h"

namespace specdec {

namespace {

// SUB steps of 16 slots as a warp takes them; RT tiles of 16 rows.
template <int D, int RT>
struct Stage8 {
  static constexpr int WARPS = 8, SUB = RT, SLOTS = SUB * kStep, STAGES = 3, MR = 16 * RT;
  // Rows of codes, padded so that the reads below meet no bank conflicts.
  static constexpr int kPitchK = D == 128 ? D + 16 : D, kPitchV = D + 16;
  static constexpr int kOffV = SLOTS * kPitchK, kBytes = SLOTS * (kPitchK + kPitchV);
  static constexpr int kStagesBytes = WARPS * STAGES * kBytes;
  static constexpr int kJoinBytes = WARPS * MR * (D * 4 + 8);  // the warps' rows, joined once per segment
  static constexpr int kOffQ = kStagesBytes > kJoinBytes ? kStagesBytes : kJoinBytes;
  static constexpr int kOffScale = kOffQ + MR * D * 2;
  static constexpr int kSmem = kOffScale + MR * 4;
};

template <typename T, int D, int RT>
__global__ void __launch_bounds__(32 * Stage8<D, RT>::WARPS, 1) attend8_kernel(const AttendParams P) {
  using St = Stage8<D, RT>;
  constexpr int MR = St::MR, WARPS = St::WARPS, SUB = St::SUB, SLOTS = St::SLOTS, STAGES = St::STAGES, THREADS = 32 * WARPS;
  constexpr int KT = D / 16, NT = D / 8, N = 2 * SUB;  // k steps, tiles of 8 values, tiles of 8 slots
  constexpr bool BRAIN = !std::is_same<T, __half>::value;
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
    // Copies the steps from t on.  Comes back with the slots on pages out of range and this lane's step's scale
    // bytes (keys', then values').  A step's slots are not all wanted where the visible range begins or ends
    // inside it; those that are lie in one block.
    // (Nothing is made of the bytes before they are used: it would wait for them.)
    struct Copied {
      uint32_t bads, scale_k, scale_v;
    };
    auto prefetch = [&](int t, int stage, int page) -> Copied {
      Copied got{0, 0, 0};
      if (t < t_hi) {
        const int s = slot_of(t);
        const bool want = wanted(t, s);
        const bool bad = want && static_cast<unsigned>(page) >= static_cast<unsigned>(pg.num_pages);
        const bool there = want && !bad;
        const int in_page = s - page_of(pg, s) * pg.page_size;
        const int64_t off = there ? page * pg.page_stride + in_page * pg.slot_stride : 0;
        got.bads = __ballot_sync(0xffffffffu, bad);
        if (SUB == 1) got.bads &= 0xffffu;
        const uint32_t present = __ballot_sync(0xffffffffu, there);
        if (there) {
          const int64_t so = page * pg.scale_page_stride + block_of(pg, in_page) * pg.scale_slot_stride + h * pg.scale_head_stride;
          got.scale_k = __ldg(reinterpret_cast<const uint8_t*>(pg.k_scales) + so);
          got.scale_v = __ldg(reinterpret_cast<const uint8_t*>(pg.v_scales) + so);
        }
        char* const base = stages + stage * St::kBytes;
        constexpr int CH = D / 16;     // 16-byte pieces of a row
        constexpr int RPI = 32 / CH;   // rows a warp copies at a time
#pragma unroll
        for (int j = 0; j < SLOTS / RPI; ++j) {
          const int row = j * RPI + lane / CH, piece = lane % CH;
          const int64_t o = __shfl_sync(0xffffffffu, off, row) + piece * 16;
          const bool ok = (present >> row) & 1u;
          copy_async<16>(smem_addr(base + row * St::kPitchK + piece * 16), k_head + o, ok);
          copy_async<16>(smem_addr(base + St::kOffV + row * St::kPitchV + piece * 16), v_head + o, ok);
        }
      }
      copy_commit();
      return got;
    };

    // ---- the query rows, as the matrix instruction's fragments: [tile][k step][lane]
    __syncthreads();  // the last segment's rows are written: its shared memory is free
    int t_next = t_lo + warp * SUB;  // the next steps this warp copies
    int page_next = entry(t_next);
    Copied ring[STAGES - 1];
#pragma unroll
    for (int s = 0; s < STAGES - 1; ++s) {
      const int page = page_next;
      page_next = entry(t_next + WARPS * SUB);
      ring[s] = prefetch(t_next, s, page);
      t_next += WARPS * SUB;
    }
    auto q_row = [&](int r) {
      const int i = query_of(P, row0 + r);
      return static_cast<const T*>(P.q) + b * P.q_sb + i * P.q_st + (h * P.G + row0 + r - i * P.G) * P.q_sh;
    };
    if constexpr (BRAIN) {  // a row's power-of-two scale
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
    for (int f = tid; f < RT * KT * 32; f += THREADS) {
      const int fg = f % 32 / 4, fc = f % 4, t = f / 32 % KT, rt = f / (32 * KT);
      uint32_t a[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int r = 16 * rt + fg + (e & 1) * 8;  // a0, a2: row g; a1, a3: row g + 8
        const int d = (D / 4) * fc + 4 * t + (e >> 1) * 2;  // the k index runs over D in the order the codes are read in
        a[e] = r < rows ? __ldg(reinterpret_cast<const uint32_t*>(q_row(r) + d)) : 0u;
        if constexpr (BRAIN) {
          const float2 v = Half16<T>::to_f32(a[e]);
          const float inv = 1.f / s_rowscale[r];
          a[e] = Half16<__half>::pack(v.x * inv, v.y * inv);
        }
      }
      reinterpret_cast<uint4*>(smem + St::kOffQ)[f] = make_uint4(a[0], a[1], a[2], a[3]);
    }
    __syncthreads();
    const uint4* const s_q = reinterpret_cast<const uint4*>(smem + St::kOffQ) + lane;

    // this thread's rows: g and g + 8 of each tile
    int q_i[RT][2], q_pos[RT][2];
    float sc[RT][2], row_m[RT][2], row_l[RT][2];
    float o[RT][NT][4];
#pragma unroll
    for (int r = 0; r < RT; ++r)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        q_i[r][e] = query_of(P, row0 + 16 * r + g + e * 8);
        q_pos[r][e] = S.first + (P.depth && q_i[r][e] < P.n ? node_depth(P, q_i[r][e]) : q_i[r][e]);
        sc[r][e] = P.scale_log2;
        if constexpr (BRAIN) sc[r][e] *= s_rowscale[16 * r + g + e * 8];
        row_m[r][e] = -kInf;
        row_l[r][e] = 0.f;
      }
#pragma unroll
    for (int r = 0; r < RT; ++r)
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int e = 0; e < 4; ++e) o[r][nt][e] = 0.f;
    uint4 qf[RT == 1 ? KT : 1];  // (one tile: the fragments stay in registers)
    if constexpr (RT == 1) {
#pragma unroll
      for (int t = 0; t < KT; ++t) qf[t] = s_q[t * 32];
    }
    const int i0 = query_of(P, row0), i1 = min(query_of(P, row0 + rows - 1), S.nq - 1);
    const bool tree = P.tree_mask != nullptr;
    auto sees = [&](int r, int e, int s) {
      const int j = s - S.first;
      bool ok = s < R.end;
      int pos = s;
      if (tree) {
        if (j >= 0) {
          ok = ok && q_i[r][e] < P.n && __ldg(P.tree_mask + static_cast<int64_t>(q_i[r][e]) * P.n + min(j, P.n - 1)) != 0;
          if (P.depth) pos = S.first + node_depth(P, min(j, P.n - 1));
        }
      } else {
        ok = ok && j <= q_i[r][e];
      }
      if (P.window > 0) ok = ok && (q_pos[r][e] - pos < P.window || pos < P.sinks);
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
      const Copied now = ring[0];
      {
        const int page = page_next;
        page_next = entry(t_next + WARPS * SUB);
        const Copied next = prefetch(t_next, stage == 0 ? STAGES - 1 : stage - 1, page);
        t_next += WARPS * SUB;
#pragma unroll
        for (int k = 0; k + 2 < STAGES; ++k) ring[k] = ring[k + 1];
        ring[STAGES - 2] = next;
      }
      const uint32_t bads = now.bads;
      char* const kb = stages + stage * St::kBytes;
      char* const vb = kb + St::kOffV;
      stage = stage + 1 == STAGES ? 0 : stage + 1;
      // the scales of the steps: from the largest byte of their lanes (slots that are not wanted give 0)
      int ek[SUB], ev[SUB];
#pragma unroll
      for (int u = 0; u < SUB; ++u) {
        const bool mine = SUB == 1 || lane / kStep == u;
        ek[u] = scale_exponent(__reduce_max_sync(0xffffffffu, mine ? now.scale_k : 0u));
        ev[u] = scale_exponent(__reduce_max_sync(0xffffffffu, mine ? now.scale_v : 0u));
      }

      // S = Q K^T: lane (g, c) takes D/4 consecutive codes of keys g, g + 8, ...; a word is a k step
      float s_acc[RT][N][4];
#pragma unroll
      for (int r = 0; r < RT; ++r)
#pragma unroll
        for (int n = 0; n < N; ++n)
#pragma unroll
          for (int e = 0; e < 4; ++e) s_acc[r][n][e] = 0.f;
#pragma unroll
      for (int y = 0; y < D / 64; ++y) {
        uint4 word[N];
#pragma unroll
        for (int n = 0; n < N; ++n) word[n] = *reinterpret_cast<const uint4*>(kb + (g + 8 * n) * St::kPitchK + c * (D / 4) + 16 * y);
#pragma unroll
        for (int z = 0; z < 4; ++z) {
          uint4 a[RT];
#pragma unroll
          for (int r = 0; r < RT; ++r) a[r] = RT == 1 ? qf[4 * y + z] : s_q[(r * KT + 4 * y + z) * 32];
#pragma unroll
          for (int n = 0; n < N; ++n) {
            uint32_t b0, b1;
            e4m3x4_to_f16(z == 0 ? word[n].x : z == 1 ? word[n].y : z == 2 ? word[n].z : word[n].w, b0, b1);
#pragma unroll
            for (int r = 0; r < RT; ++r) mma<__half>(s_acc[r][n], a[r], b0, b1);
          }
        }
      }

      // scale and mask; a slot on a page out of range gives NaN to the rows that see it
      bool whole = bads == 0;
#pragma unroll
      for (int u = 0; u < SUB; ++u) whole = whole && whole_step(t + u);
      uint32_t seen[RT];  // bit 4 n + e: element e of key tile n is visible
#pragma unroll
      for (int r = 0; r < RT; ++r) {
        seen[r] = 0;
#pragma unroll
        for (int n = 0; n < N; ++n) {
          const float f = power_f32(ek[n / 2]);
#pragma unroll
          for (int e = 0; e < 4; ++e) s_acc[r][n][e] *= sc[r][e / 2] * f;
        }
        if (!whole) {
#pragma unroll
          for (int n = 0; n < N; ++n)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const int key = 8 * n + 2 * c + (e & 1);
              const bool ok = t + key / kStep < t_hi && sees(r, e / 2, R.slot(t + key / kStep) + key % kStep);
              float v = s_acc[r][n][e];
              if ((bads >> key) & 1u) v = __int_as_float(0x7fffffff);
              s_acc[r][n][e] = ok ? v : -kInf;
              seen[r] |= (ok ? 1u : 0u) << (4 * n + e);
            }
        }
      }

      // the running maximum and sum
      uint4 p[RT][SUB];
#pragma unroll
      for (int r = 0; r < RT; ++r) {
        float alpha[2];
#pragma unroll
        for (int x = 0; x < 2; ++x) {
          float m = -kInf;
#pragma unroll
          for (int n = 0; n < N; ++n) m = fmaxf(m, fmaxf(s_acc[r][n][2 * x], s_acc[r][n][2 * x + 1]));
          m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 1));
          m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 2));
          const float top = fmaxf(row_m[r][x], m - kBelow<__half>);
          const float base = top == -kInf ? 0.f : top;
          alpha[x] = ex2(row_m[r][x] - base);
          row_m[r][x] = top;
          float sum = 0.f;
#pragma unroll
          for (int n = 0; n < N; ++n)
#pragma unroll
            for (int y = 0; y < 2; ++y) {
              s_acc[r][n][2 * x + y] = ex2(s_acc[r][n][2 * x + y] - base);
              sum += s_acc[r][n][2 * x + y];
            }
          row_l[r][x] = row_l[r][x] * alpha[x] + sum;  // this lane's keys; joined at the end
        }
        // P in fp16: a rounding of 2^-11 of each weight (below 2^-21 of the row's largest weight, of 2^-32 of that
        // one); l keeps the unrounded weights
#pragma unroll
        for (int u = 0; u < SUB; ++u)
          p[r][u] = make_uint4(Half16<__half>::pack(s_acc[r][2 * u][0], s_acc[r][2 * u][1]), Half16<__half>::pack(s_acc[r][2 * u][2], s_acc[r][2 * u][3]),
                               Half16<__half>::pack(s_acc[r][2 * u + 1][0], s_acc[r][2 * u + 1][1]),
                               Half16<__half>::pack(s_acc[r][2 * u + 1][2], s_acc[r][2 * u + 1][3]));
        if (__any_sync(0xffffffffu, alpha[0] != 1.f || alpha[1] != 1.f)) {
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int e = 0; e < 4; ++e) o[r][nt][e] *= alpha[e / 2];
        }
      }

      // A value that is not finite (a code of NaN) must not reach rows that do not see its slot (0 * NaN):
      // steps that some row sees in part look for such codes, take them out of the product
      // and add them to the rows that do see them.
      uint32_t odd = 0;
      if (!whole) {
        for (int f = lane; f < SLOTS * (D / 16); f += 32) {
          const uint4 x = *reinterpret_cast<const uint4*>(vb + (f / (D / 16)) * St::kPitchV + (f % (D / 16)) * 16);
          const uint32_t any = __vcmpeq4(x.x & 0x7f7f7f7fu, 0x7f7f7f7fu) | __vcmpeq4(x.y & 0x7f7f7f7fu, 0x7f7f7f7fu) |
                               __vcmpeq4(x.z & 0x7f7f7f7fu, 0x7f7f7f7fu) | __vcmpeq4(x.w & 0x7f7f7f7fu, 0x7f7f7f7fu);
          if (any) odd |= 1u << (f / (D / 16));
        }
        odd = __reduce_or_sync(0xffffffffu, odd);
      }

      // O += P V: lane (g, c) takes values (D/8) g ... of keys 2c, 2c+1, 2c+8, 2c+9; column g of tile
      // nt stands for value (D/8) g + nt
#pragma unroll
      for (int u = 0; u < SUB; ++u) {
        constexpr int W = D / 32;  // words of those codes
        const uint32_t odd16 = odd >> (16 * u);
        const uint32_t keep0 = ((odd16 >> (2 * c)) & 1u ? 0u : 0xffffu) | ((odd16 >> (2 * c + 1)) & 1u ? 0u : 0xffff0000u);
        const uint32_t keep1 = ((odd16 >> (2 * c + 8)) & 1u ? 0u : 0xffffu) | ((odd16 >> (2 * c + 9)) & 1u ? 0u : 0xffff0000u);
        uint32_t word[4][W];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const char* const row = vb + (16 * u + 2 * c + (k & 1) + (k >> 1) * 8) * St::kPitchV + g * (D / 8);
          if constexpr (W == 4) {
            const uint4 x = *reinterpret_cast<const uint4*>(row);
            word[k][0] = x.x; word[k][1] = x.y; word[k][2] = x.z; word[k][3] = x.w;
          } else {
            const uint2 x = *reinterpret_cast<const uint2*>(row);
            word[k][0] = x.x; word[k][1] = x.y;
          }
        }
        const uint32_t s2 = power_f16x2(ev[u]);
#pragma unroll
        for (int x = 0; x < W; ++x) {
          uint32_t f[2][4];
#pragma unroll
          for (int k = 0; k < 2; ++k) {  // pair the two keys' bytes
            const uint32_t a = word[2 * k][x], bb = word[2 * k + 1][x];
            e4m3x4_to_f16(__byte_perm(a, bb, 0x5140), f[k][0], f[k][1]);
            e4m3x4_to_f16(__byte_perm(a, bb, 0x7362), f[k][2], f[k][3]);
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              f[k][e] = mul_f16x2(f[k][e], s2);
              if (odd) f[k][e] &= k == 0 ? keep0 : keep1;
            }
          }
#pragma unroll
          for (int e = 0; e < 4; ++e)
#pragma unroll
            for (int r = 0; r < RT; ++r) mma<__half>(o[r][4 * x + e], p[r][u], f[0][e], f[1][e]);
        }
      }
      if (odd) {  // rare: what was taken out above, for the rows that see the slot
#pragma unroll 1
        for (uint32_t left = odd; left; left &= left - 1) {
          const int key = __ffs(left) - 1, n = key / 8;
          const int src = (lane & ~3) | ((key & 7) >> 1);
#pragma unroll
          for (int r = 0; r < RT; ++r)
#pragma unroll
            for (int x = 0; x < 2; ++x) {
              uint32_t mine = 0;
#pragma unroll
              for (int u = 0; u < SUB; ++u) {
                if (n == 2 * u) mine = x ? p[r][u].y : p[r][u].x;
                if (n == 2 * u + 1) mine = x ? p[r][u].w : p[r][u].z;
              }
              const uint32_t got = __shfl_sync(0xffffffffu, mine, src);
              const uint32_t vis = __shfl_sync(0xffffffffu, seen[r], src);
              const float2 two = Half16<__half>::to_f32(got);
              const float pk = key & 1 ? two.y : two.x;
              if (!((vis >> (4 * n + 2 * x + (key & 1))) & 1u)) continue;
#pragma unroll
              for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int y = 0; y < 2; ++y) {
                  const int d = (D / 8) * (2 * c + y) + nt;
                  const uint32_t byte = *reinterpret_cast<const uint8_t*>(vb + key * St::kPitchV + d);
                  int e = ev[0];
#pragma unroll
                  for (int u = 1; u < SUB; ++u)
                    if (key / kStep == u) e = ev[u];
                  o[r][nt][2 * x + y] += pk * Half16<__half>::to_f32(mul_f16x2(e4m3x2_to_f16(byte), power_f16x2(e))).x;
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
    for (int r = 0; r < RT; ++r)
#pragma unroll
      for (int x = 0; x < 2; ++x) {
        float l = row_l[r][x];
        l += __shfl_xor_sync(0xffffffffu, l, 1);
        l += __shfl_xor_sync(0xffffffffu, l, 2);
        const int row = 16 * r + g + 8 * x;
        if (c == 0) s_ml[warp * MR + row] = make_float2(row_m[r][x], l);
        float* const dst = s_o + (static_cast<size_t>(warp) * MR + row) * D;
#pragma unroll
        for (int y = 0; y < 2; ++y)
#pragma unroll
          for (int nt = 0; nt < NT; nt += 4)
            *reinterpret_cast<float4*>(dst + (D / 8) * (2 * c + y) + nt) =
                make_float4(o[r][nt][2 * x + y], o[r][nt + 1][2 * x + y], o[r][nt + 2][2 * x + y], o[r][nt + 3][2 * x + y]);
      }
    __syncthreads();
    join_warps<T, D, MR, WARPS>(P, w, S, row0, rows, smem);
    if (w.u == w.item && !w.ends() && tid == 0) P.split[cta] = w.split(share);
    if (!w.next()) break;
  }
}

template <typename T, int D, int RT>
cudaError_t launch_shape(const AttendParams& P, cudaStream_t stream) {
  using St = Stage8<D, RT>;
  auto kernel = attend8_kernel<T, D, RT>;
  static_assert(St::kSmem <= 227 * 1024 - 1024, "shared memory of a CTA");
  if (cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, St::kSmem); e != cudaSuccess)
    return e;
  return launch_kernel(kernel, dim3(P.ctas), dim3(32 * St::WARPS), St::kSmem, stream, 1, P);
}

template <typename T>
cudaError_t launch_typed(const AttendParams& P, int mr, cudaStream_t stream) {
  if (P.pages.head_dim == 64) return mr == 16 ? launch_shape<T, 64, 1>(P, stream) : launch_shape<T, 64, 2>(P, stream);
  return mr == 16 ? launch_shape<T, 128, 1>(P, stream) : launch_shape<T, 128, 2>(P, stream);
}

}  // namespace

int attend8_rows(int64_t rows) { return rows <= 16 ? 16 : 32; }

cudaError_t launch_attend8(const AttendParams& P, specdec_dtype dt, int mr, cudaStream_t stream) {
  return dt == SPECDEC_BF16 ? launch_typed<__nv_bfloat16>(P, mr, stream) : launch_typed<__half>(P, mr, stream);
}

}  // namespace specdec
