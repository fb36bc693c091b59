// Attention over 8-bit pages for a few rows to a key head (up to 16), on warp-level matrix instructions.
//
// The formula, the items, the split of the work and the join are those of attend.cu.  Keys and values are
// E4M3 codes, and the slots of a step of 16 lie in one block, so they share a scale 2^e for keys and one for values:
//   s_ij = (c 2^e_k) (q_i . code_j),   O_i += p_ij (2^e_v code_j)
// Codes are exact in fp16, and so are values, 2^e_v code (e from -15 to 7), so the products are those of
// fp16 with fp32 sums; the keys' scale goes into the scores' factor.  Queries in bf16 are held in fp16 relative to a power of
// two of their row, to 2^-25 of its largest value.
//
// The products are transposed: S^T = K Q^T and O^T = V^T P^T with 16 slots (16 values) by 8 query rows to an instruction, so that 8 rows
// cost half of what 16 do.  Codes go from the copied tile straight into the instruction's registers: a key's row is read in the order
// that makes a word the four codes of a step of the k index, two slots' words are interleaved by bytes for the product with V;
// the weights are turned by the matrix transposition of registers.  So shared memory carries the codes once in and once
// out, and a conversion serves all rows of the tile: 8 or 16.
//
// A row's reference m moves only when a score exceeds what it was set for by more than 2^8 (as in attend_tc.cuh; the
// weights stay below 2^15): most steps then need no maximum across lanes and no rescaling.
//
// One token of 96 requests over up to 16001 slots (8 rows to a key head): 310 us, 6.3 TB/s, 0.93 of the measured copy rate: HBM
// bounds it.  64 requests of 2 tokens over up to 8190 slots (8 rows) 127 us, 0.79; of 4 tokens (16 rows) 175 us, 0.57: two row
// tiles leave registers for two warps to a scheduler only.
//
// A step's 16 rows are a box of the pages' tensor (values, slots, heads, pages), which one TMA instruction brings, swizzled so that
// the reads meet no bank conflicts; a warp looks up 32 steps at a time, a lane each.  (16-byte asynchronous copies by all
// lanes, with a lookup for every step: 288 us for 64 requests of 8 tokens over up to 8190 slots, 485 us for one token of 96
// requests over up to 16001; over half of the instructions were the copies'.)

#include "attend_common.cuh"
#include "boxes.cuh"
#include "specdec_internal.h"

namespace specdec {

namespace {

// (Warps, steps, stages for 8 rows, us for the 96 requests above: 12, 2, 2: 312; 16, 1, 3: 332; 12, 1, 4: 340; 8, 2, 3: 359.  For 16
// rows, 64 requests: 8, 2, 3: 175; 8, 1, 5: 185; 12, 1, 4: 202; 10, 1, 5: 223.)
// RT tiles of 8 rows.  Warps, each with a stream of slots of its own; SUB steps of 16 slots as a warp takes them; stages.
template <int D, int RT>
struct Stage8 {
  static constexpr int WARPS = RT == 1 ? 12 : 8, SUB = 2, STAGES = RT == 1 ? 2 : 3, MR = 8 * RT;
  static constexpr int kBox = kStep * D, kBytes = 2 * SUB * kBox;  // keys, then values
  static constexpr int kStagesBytes = WARPS * STAGES * kBytes;
  static constexpr int kJoinBytes = WARPS * MR * (D * 4 + 8);  // the warps' rows, joined once per segment
  static constexpr int kOffQ = kStagesBytes > kJoinBytes ? kStagesBytes : kJoinBytes;
  static constexpr int kOffScale = kOffQ + MR * D * 2;
  static constexpr int kOffBar = kOffScale + MR * 4;
  static constexpr int kSmem = kOffBar + WARPS * STAGES * 8;
  // Where the 16-byte piece `piece` of row `row` of a box lies: rows of D bytes, swizzled as the copies do.
  __device__ static constexpr int at(int row, int piece) {
    return row * D + ((D == 128 ? piece ^ (row & 7) : piece ^ (row >> 1 & 3)) << 4);
  }
};
constexpr float kSlack = 8.f;  // log2 of how far a score may exceed what the reference was set for

// An 8 x 8 matrix of 16-bit values, a register of two from each lane, transposed.
__device__ __forceinline__ uint32_t transpose8x8(uint32_t x) {
  uint32_t y;
  asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
}

template <typename T, int D, int RT>
__global__ void __launch_bounds__(32 * Stage8<D, RT>::WARPS, 1) attend8_kernel(const AttendParams P, const __grid_constant__ Maps maps) {
  using St = Stage8<D, RT>;
  constexpr int MR = St::MR, WARPS = St::WARPS, SUB = St::SUB, STAGES = St::STAGES, THREADS = 32 * WARPS;
  constexpr int KT = D / 16, MT = D / 16;  // k steps of the scores, tiles of 16 values
  constexpr bool BRAIN = !std::is_same<T, __half>::value;
  extern __shared__ __align__(1024) char smem[];
  __shared__ int64_t s_scan[WARPS + 3];
  const Pages& pg = P.pages;
  const int tid = threadIdx.x, warp = tid / 32, lane = tid % 32, g = lane / 4, c = lane % 4;
  const int64_t slots = static_cast<int64_t>(pg.max_pages) * pg.page_size;
  char* const stages = smem + warp * STAGES * St::kBytes;
  float* const s_rowscale = reinterpret_cast<float*>(smem + St::kOffScale);
  uint64_t* const full = reinterpret_cast<uint64_t*>(smem + St::kOffBar) + warp * STAGES;  // a stage's copies have landed
  if (lane == 0) {
    for (int s = 0; s < STAGES; ++s) mbar_init(full + s, 1);
    mbar_fence_init();
  }
  int issued = 0, taken = 0;  // stages filled and read by this warp so far
  bool late = false;          // a bounded wait ran out

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

    // The warp's round n takes the steps first_step(n) ..; a look is 32 steps, a lane each.  (Every step has a slot that some
    // query sees, and its 16 slots are on one page and in one block.)
    auto first_step = [&](int n) { return t_lo + (n * WARPS + warp) * SUB; };
    const int rounds = first_step(0) >= t_hi ? 0 : (t_hi - first_step(0) - 1) / (WARPS * SUB) + 1;
    constexpr int LOOK = 32 / SUB;  // rounds of a look
    auto look_up = [&](int look) {
      Look l;
      const int t = first_step(look * LOOK + lane / SUB) + lane % SUB;
      l.find(pg, table, R.slot(t), t < t_hi);
      return l;
    };
    Look now{}, next{};
    // copies round n's steps (now is the look of the round that is taken, n the same or the next one)
    auto issue = [&](int n, bool ahead) {
      int page[SUB], in_page[SUB];
#pragma unroll
      for (int u = 0; u < SUB; ++u) {
        page[u] = __shfl_sync(0xffffffffu, ahead ? next.page : now.page, n % LOOK * SUB + u);
        in_page[u] = __shfl_sync(0xffffffffu, ahead ? next.in_page : now.in_page, n % LOOK * SUB + u);
      }
      if (lane == 0) {
        const int stage = issued % STAGES;
        const uint32_t dst = smem_addr(stages + stage * St::kBytes);
        uint32_t boxes = 0;
#pragma unroll
        for (int u = 0; u < SUB; ++u) boxes += static_cast<unsigned>(page[u]) < static_cast<unsigned>(pg.num_pages) ? 2 : 0;
        fence_proxy_async_smem();  // (the warp's reads of the stage, which its barrier ordered before this)
        mbar_expect_tx(full + stage, boxes * St::kBox);
#pragma unroll
        for (int u = 0; u < SUB; ++u)
          if (static_cast<unsigned>(page[u]) < static_cast<unsigned>(pg.num_pages)) {
            copy_box(dst + u * St::kBox, &maps.k, in_page[u], maps.heads ? h : 0, maps.pages ? page[u] : 0, full + stage);
            copy_box(dst + (SUB + u) * St::kBox, &maps.v, in_page[u], maps.heads ? h : 0, maps.pages ? page[u] : 0, full + stage);
          }
      }
      ++issued;
    };
    fence_proxy_async_smem();  // (the warps' rows that were written where boxes land now)
    __syncthreads();           // the last segment's rows are written: its shared memory is free
    if (!late) {
      now = look_up(0);
      next = look_up(1);
#pragma unroll
      for (int n = 0; n < STAGES - 1; ++n)
        if (n < rounds) issue(n, false);
      now.find_scales(pg, h);
    }

    // ---- the query rows, as the matrix instruction's fragments: [tile][k step][lane].  Rows that are no token's are zeros, whatever
    // a padded batch's queries hold: they take part in the vote on references, which may change another row's rounding.
    const int there = static_cast<int>(min(static_cast<int64_t>(rows), max(static_cast<int64_t>(S.nq) * P.G - row0, int64_t{0})));
    auto q_row = [&](int r) {
      const int i = query_of(P, row0 + r);
      return static_cast<const T*>(P.q) + b * P.q_sb + i * P.q_st + (h * P.G + row0 + r - i * P.G) * P.q_sh;
    };
    if constexpr (BRAIN) {  // a row's power-of-two scale
      for (int r = warp; r < MR; r += WARPS) {
        float a = 0.f;
        if (r < there)
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
      const int r = f / (32 * KT) * 8 + f % 32 / 4, t = f / 32 % KT;
      uint2 q = make_uint2(0u, 0u);  // the k index runs over D in the order the codes are read in
      if (r < there) q = __ldg(reinterpret_cast<const uint2*>(q_row(r) + (D / 4) * (f % 4) + 4 * t));
      if constexpr (BRAIN) {
        const float2 lo = Half16<T>::to_f32(q.x), hi = Half16<T>::to_f32(q.y);
        const float inv = 1.f / s_rowscale[r];
        q = make_uint2(Half16<__half>::pack(lo.x * inv, lo.y * inv), Half16<__half>::pack(hi.x * inv, hi.y * inv));
      }
      reinterpret_cast<uint2*>(smem + St::kOffQ)[f] = q;
    }
    __syncthreads();
    const uint2* const s_q = reinterpret_cast<const uint2*>(smem + St::kOffQ) + lane;

    // this thread's rows: 2 c and 2 c + 1 of each tile
    int q_i[RT][2], q_pos[RT][2];
    float sc[RT][2], row_m[RT][2], row_l[RT][2];
    float o[RT][MT][4];  // values (D/8) g + 2 m (of both rows) and the next one
#pragma unroll
    for (int r = 0; r < RT; ++r)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        q_i[r][e] = query_of(P, row0 + 8 * r + 2 * c + e);
        q_pos[r][e] = S.first + (P.depth && q_i[r][e] < P.n ? node_depth(P, q_i[r][e]) : q_i[r][e]);
        sc[r][e] = P.scale_log2;
        if constexpr (BRAIN) sc[r][e] *= s_rowscale[8 * r + 2 * c + e];
        row_m[r][e] = -kInf;
        row_l[r][e] = 0.f;
      }
#pragma unroll
    for (int r = 0; r < RT; ++r)
#pragma unroll
      for (int m = 0; m < MT; ++m)
#pragma unroll
        for (int e = 0; e < 4; ++e) o[r][m][e] = 0.f;
    uint2 qf[RT * KT];
#pragma unroll
    for (int t = 0; t < RT * KT; ++t) qf[t] = s_q[t * 32];
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

    for (int n = 0; n < rounds && !late; ++n) {
      const int t = first_step(n), stage = taken % STAGES;
      if (n > 0 && n % LOOK == 0) {
        now = next;
        next = look_up(n / LOOK + 1);
      }
      if (!__all_sync(0xffffffffu, mbar_wait(full + stage, (taken / STAGES) & 1))) {
        late = true;
        break;
      }
      ++taken;
      __syncwarp();  // every lane has read the round before, whose stage is filled again (votes and shuffles order no memory)
      if (n + STAGES - 1 < rounds) issue(n + STAGES - 1, (n + STAGES - 1) / LOOK != n / LOOK);
      if (n % LOOK == LOOK / 2) next.find_scales(pg, h);
      char* const kb = stages + stage * St::kBytes;
      char* const vb = kb + SUB * St::kBox;
#pragma unroll
      for (int u = 0; u < SUB; ++u) {
        // the step's scales, and whether its page is out of range
        const int lane_of = n % LOOK * SUB + u;
        const int ek = scale_exponent(__shfl_sync(0xffffffffu, now.scale_k, lane_of)), ev = scale_exponent(__shfl_sync(0xffffffffu, now.scale_v, lane_of));
        const bool bad = __shfl_sync(0xffffffffu, now.page, lane_of) >= pg.num_pages;
        const char* const ks = kb + u * St::kBox;
        const char* const vs = vb + u * St::kBox;

        // S^T = K Q^T: lane (g, c) takes D/4 consecutive codes of keys g and g + 8; a word is a k step
        float s[RT][4];  // slots g (of both rows) and g + 8
#pragma unroll
        for (int r = 0; r < RT; ++r)
#pragma unroll
          for (int e = 0; e < 4; ++e) s[r][e] = 0.f;
#pragma unroll
        for (int y = 0; y < D / 64; ++y) {
          const uint4 lo = *reinterpret_cast<const uint4*>(ks + St::at(g, c * (D / 64) + y)), hi = *reinterpret_cast<const uint4*>(ks + St::at(g + 8, c * (D / 64) + y));
          const uint32_t wl[4] = {lo.x, lo.y, lo.z, lo.w}, wh[4] = {hi.x, hi.y, hi.z, hi.w};
#pragma unroll
          for (int z = 0; z < 4; ++z) {
            uint4 a;
            e4m3x4_to_f16(wl[z], a.x, a.z);
            e4m3x4_to_f16(wh[z], a.y, a.w);
#pragma unroll
            for (int r = 0; r < RT; ++r) {
              const uint2 q = qf[r * KT + 4 * y + z];
              mma<__half>(s[r], a, q.x, q.y);
            }
          }
        }

        // scale and mask; a slot on a page out of range gives NaN to the rows that see it
        const bool whole = !bad && whole_step(t + u);
        const float factor = power_f32(ek);
        uint32_t seen = ~0u;  // bit 4 r + e
        bool moves = false;
#pragma unroll
        for (int r = 0; r < RT; ++r)
#pragma unroll
          for (int e = 0; e < 4; ++e) s[r][e] *= sc[r][e % 2] * factor;
        if (!whole) {
          seen = 0;
#pragma unroll
          for (int r = 0; r < RT; ++r)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const bool ok = t + u < t_hi && sees(r, e % 2, R.slot(t + u) + g + e / 2 * 8);
              s[r][e] = !ok ? -kInf : bad ? __int_as_float(0x7fffffff) : s[r][e];
              seen |= (ok ? 1u : 0u) << (4 * r + e);
            }
        }
#pragma unroll
        for (int r = 0; r < RT; ++r)
#pragma unroll
          for (int e = 0; e < 2; ++e) moves = moves || fmaxf(s[r][e], s[r][2 + e]) - row_m[r][e] > kSlack + kBelow<__half>;
        if (__any_sync(0xffffffffu, moves)) {  // (also where m is still -inf)
#pragma unroll
          for (int r = 0; r < RT; ++r)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              float top = fmaxf(s[r][e], s[r][2 + e]);
#pragma unroll
              for (int x = 4; x < 32; x <<= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, x));
              top = fmaxf(row_m[r][e], top - kBelow<__half>);
              const float alpha = row_m[r][e] == top ? 1.f : ex2(row_m[r][e] - top);
              row_m[r][e] = top;
              row_l[r][e] *= alpha;
#pragma unroll
              for (int m = 0; m < MT; ++m) {
                o[r][m][e] *= alpha;
                o[r][m][2 + e] *= alpha;
              }
            }
        }

        // the weights.  P in fp16: a rounding of 2^-11 of each (below 2^-21 of the row's largest, of 2^-32 of
        // that one); l keeps the unrounded ones
        uint32_t w2[RT][2];  // slot g, then g + 8, of both rows
        uint2 pf[RT];
#pragma unroll
        for (int r = 0; r < RT; ++r) {
          float pe[4];
#pragma unroll
          for (int e = 0; e < 4; ++e) pe[e] = ex2(s[r][e] - (row_m[r][e % 2] == -kInf ? 0.f : row_m[r][e % 2]));
          row_l[r][0] += pe[0] + pe[2];  // this lane's slots; joined at the end
          row_l[r][1] += pe[1] + pe[3];
          w2[r][0] = Half16<__half>::pack(pe[0], pe[1]);
          w2[r][1] = Half16<__half>::pack(pe[2], pe[3]);
          pf[r] = make_uint2(transpose8x8(w2[r][0]), transpose8x8(w2[r][1]));
        }

        // A value that is not finite (a code of NaN) must not reach rows that do not see its slot (0 * NaN):
        // steps that some row sees in part look for such codes, take them out of the product
        // and add them to the rows that do see them.
        uint32_t odd = 0;
        if (!whole) {
          for (int f = lane; f < kStep * (D / 16); f += 32) {  // (rows of a box are whole, whatever the order of their pieces)
            const uint4 x = *reinterpret_cast<const uint4*>(vs + f * 16);
            const uint32_t any = __vcmpeq4(x.x & 0x7f7f7f7fu, 0x7f7f7f7fu) | __vcmpeq4(x.y & 0x7f7f7f7fu, 0x7f7f7f7fu) |
                                 __vcmpeq4(x.z & 0x7f7f7f7fu, 0x7f7f7f7fu) | __vcmpeq4(x.w & 0x7f7f7f7fu, 0x7f7f7f7fu);
            if (any) odd |= 1u << (f / (D / 16));
          }
          odd = __reduce_or_sync(0xffffffffu, odd);
        }
        const uint32_t keep0 = ((odd >> (2 * c)) & 1u ? 0u : 0xffffu) | ((odd >> (2 * c + 1)) & 1u ? 0u : 0xffff0000u);
        const uint32_t keep1 = ((odd >> (2 * c + 8)) & 1u ? 0u : 0xffffu) | ((odd >> (2 * c + 9)) & 1u ? 0u : 0xffff0000u);

        // O^T += V^T P^T: lane (g, c) takes values (D/8) g ... of slots 2c, 2c+1, 2c+8, 2c+9
        constexpr int W = D / 32;  // words of those codes
        uint32_t word[4][W];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const int row = 2 * c + (k & 1) + (k >> 1) * 8;
          const char* const from = vs + (D == 128 ? St::at(row, g) : St::at(row, g / 2) + g % 2 * 8);
          if constexpr (W == 4) {
            const uint4 x = *reinterpret_cast<const uint4*>(from);
            word[k][0] = x.x; word[k][1] = x.y; word[k][2] = x.z; word[k][3] = x.w;
          } else {
            const uint2 x = *reinterpret_cast<const uint2*>(from);
            word[k][0] = x.x; word[k][1] = x.y;
          }
        }
        const uint32_t s2 = power_f16x2(ev);
#pragma unroll
        for (int x = 0; x < W; ++x) {
          uint32_t f[2][4];
#pragma unroll
          for (int k = 0; k < 2; ++k) {  // pair the two slots' bytes
            const uint32_t a = word[2 * k][x], bb = word[2 * k + 1][x];
            e4m3x4_to_f16(__byte_perm(a, bb, 0x5140), f[k][0], f[k][1]);
            e4m3x4_to_f16(__byte_perm(a, bb, 0x7362), f[k][2], f[k][3]);
#pragma unroll
            for (int e = 0; e < 4; ++e) f[k][e] = mul_f16x2(f[k][e], s2);
          }
          if (odd) {
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              f[0][e] &= keep0;
              f[1][e] &= keep1;
            }
          }
#pragma unroll
          for (int y = 0; y < 2; ++y)
#pragma unroll
            for (int r = 0; r < RT; ++r)
              mma<__half>(o[r][2 * x + y], make_uint4(f[0][2 * y], f[0][2 * y + 1], f[1][2 * y], f[1][2 * y + 1]), pf[r].x, pf[r].y);
        }
        if (odd) {  // rare: what was taken out above, for the rows that see the slot
#pragma unroll 1
          for (uint32_t left = odd; left; left &= left - 1) {
            const int key = __ffs(left) - 1, src = (key & 7) * 4 + c;
            const uint32_t vis = __shfl_sync(0xffffffffu, seen, src);
#pragma unroll
            for (int r = 0; r < RT; ++r) {
              const uint32_t got = __shfl_sync(0xffffffffu, key < 8 ? w2[r][0] : w2[r][1], src);
              const float2 p = Half16<__half>::to_f32(got);
#pragma unroll
              for (int y = 0; y < 2; ++y) {
                if (!((vis >> (4 * r + key / 8 * 2 + y)) & 1u)) continue;
                const float py = y ? p.y : p.x;
#pragma unroll
                for (int d = 0; d < 2 * MT; ++d) {
                  const int at = (D / 8) * g + d;
                  const uint32_t byte = *reinterpret_cast<const uint8_t*>(vs + St::at(key, at / 16) + at % 16);
                  o[r][d / 2][d % 2 * 2 + y] += py * Half16<__half>::to_f32(mul_f16x2(e4m3x2_to_f16(byte), s2)).x;
                }
              }
            }
          }
        }
      }
    }

    // ---- join the warps' rows
    __syncthreads();
    float* const s_o = reinterpret_cast<float*>(smem);                            // [WARPS][MR][D]
    float2* const s_ml = reinterpret_cast<float2*>(smem + WARPS * MR * D * 4);    // [WARPS][MR]
#pragma unroll
    for (int r = 0; r < RT; ++r)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        float l = row_l[r][e];
#pragma unroll
        for (int x = 4; x < 32; x <<= 1) l += __shfl_xor_sync(0xffffffffu, l, x);
        const int row = 8 * r + 2 * c + e;
        if (g == 0) s_ml[warp * MR + row] = make_float2(row_m[r][e], l);
        float* const dst = s_o + (static_cast<size_t>(warp) * MR + row) * D + (D / 8) * g;
#pragma unroll
        for (int m = 0; m < MT; m += 2)
          *reinterpret_cast<float4*>(dst + 2 * m) = make_float4(o[r][m][e], o[r][m][2 + e], o[r][m + 1][e], o[r][m + 1][2 + e]);
      }
    __syncthreads();
    join_warps<T, D, MR, WARPS>(P, w, S, row0, rows, smem);
    if (w.u == w.item && !w.ends() && tid == 0) P.split[cta] = w.split(share);
    if (!w.next()) break;
  }
  if (late) {  // nothing of the call counts; what is still on its way lands first
    for (; taken < issued; ++taken) mbar_wait(full + taken % STAGES, (taken / STAGES) & 1);
    if (lane == 0) P.gave_up[cta] = 1;
  }
}

template <typename T, int D, int RT>
cudaError_t launch_shape(const AttendParams& P, cudaStream_t stream) {
  using St = Stage8<D, RT>;
  auto kernel = attend8_kernel<T, D, RT>;
  static_assert(St::kSmem <= 227 * 1024 - 1024, "shared memory of a CTA");
  if (cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, St::kSmem); e != cudaSuccess)
    return e;
  Maps maps;
  if (cudaError_t e = encode_maps(P.pages, true, true, &maps); e != cudaSuccess) return e;
  return launch_kernel(kernel, dim3(P.ctas), dim3(32 * St::WARPS), St::kSmem, stream, 1, P, maps);
}

template <typename T, int D>
cudaError_t launch_rows(const AttendParams& P, int mr, cudaStream_t stream) {
  return mr == 8 ? launch_shape<T, D, 1>(P, stream) : launch_shape<T, D, 2>(P, stream);
}
template <typename T>
cudaError_t launch_typed(const AttendParams& P, int mr, cudaStream_t stream) {
  return P.pages.head_dim == 64 ? launch_rows<T, 64>(P, mr, stream) : launch_rows<T, 128>(P, mr, stream);
}

}  // namespace

int attend8_rows(int64_t rows) { return rows <= 8 ? 8 : 16; }

cudaError_t launch_attend8(const AttendParams& P, specdec_dtype dt, int mr, cudaStream_t stream) {
  return dt == SPECDEC_BF16 ? launch_typed<__nv_bfloat16>(P, mr, stream) : launch_typed<__half>(P, mr, stream);
}

}  // namespace specdec
