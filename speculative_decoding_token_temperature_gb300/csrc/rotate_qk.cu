// Norms of queries and keys for each head and the position rotation, in one pass, with the
// keys and values written to their cache pages.
//
// For a head's vector x of D values: y = x w / sqrt(mean(x^2) + eps) (no weight: y = x); the
// first `rot` values are rotated in pairs (j, j + rot/2), or (2j, 2j+1) interleaved, by the
// angle pos * f_j.  A frequency comes as a 64-bit count of 2^-64 turns for a position, so
// pos * f_j modulo a turn is one integer multiplication, exact at every position; its top 32
// bits become a float of at most half a turn in magnitude (error 2^-25 turns), which sincospi
// takes.  Statistics and rotation are in fp32; each value is rounded once, at the store.
//
// D/8 lanes hold a head's row, 8 values each: two pieces of 4 whose values pair up, so that the
// rotation needs no exchange, and a lane's 4 pairs are the same for every head, so that its sines,
// cosines and weights stay in registers.  A warp's rows are a token's heads; 1 to 8 warps share a
// token, the more the fewer tokens there are: a few tokens are bound by latency and want the rows
// side by side, prompts by instructions and want the angles computed once.  8193 tokens of 28 query and
// 4 key heads of 128 in bf16 (151 MB read and written) take 32.3 us, 4.7 TB/s: 52 % of the issue slots,
// 41 % of HBM (most of what is written stays in L2).

#include "cache_device.cuh"
#include "specdec_device.cuh"

namespace specdec {

namespace {

constexpr int kRotateThreads = 256;
constexpr int kRotateWarps = kRotateThreads / 32;
constexpr int kRowsAhead = 2;  // rows a lane group loads before it works on the first

template <typename T, int D, bool INTERLEAVED>
__global__ void __launch_bounds__(kRotateThreads, 4) rotate_qk_kernel(const RotateParams P, int warps_per_token) {
  constexpr int LPH = D / 8;     // lanes of a head
  constexpr int RPW = 32 / LPH;  // rows a warp takes at a time
  const int b = blockIdx.y, warp = threadIdx.x / 32, lane = threadIdx.x % 32, l = lane % LPH;
  const int i = blockIdx.x * (kRotateWarps / warps_per_token) + warp / warps_per_token;
  const Pages& pg = P.pages;
  const bool paged = P.k_out == nullptr;
  // this lane's two pieces of 4 values: the halves of 4 pairs, or values that are not rotated
  const int pairs = P.rot / 8;  // lanes with rotated values (interleaved: the same count)
  const bool turned = l < pairs;
  const int pa = INTERLEAVED ? 2 * l : turned ? l : 2 * l, pb = INTERLEAVED ? 2 * l + 1 : turned ? l + pairs : 2 * l + 1;
  const int group = lane / LPH, r_first = (warp % warps_per_token) * RPW + group, r_step = warps_per_token * RPW;
  // the first query rows, before anything else is known
  const T* q_row = static_cast<const T*>(P.q) + b * P.q_sb + i * P.q_st + r_first * P.q_sh;
  uint2 ra[kRowsAhead] = {}, rb[kRowsAhead] = {};
  if (i < P.n) {
#pragma unroll
    for (int u = 0; u < kRowsAhead; ++u)
      if (r_first + u * r_step < P.Hq) {
        const uint2* const src = reinterpret_cast<const uint2*>(q_row + u * r_step * P.q_sh);
        ra[u] = __ldg(src + pa);
        rb[u] = __ldg(src + pb);
      }
  }

  const SeqLen S = seq_len(P.context_len, P.query_len, b, P.n,
                           paged ? static_cast<int64_t>(pg.max_pages) * pg.page_size : INT32_MAX);
  const int32_t* table = pg.table + static_cast<int64_t>(b) * pg.max_pages;
  // a sequence with a bad length or page is left alone as a whole: every CTA looks at all of
  // its new tokens' pages
  bool bad = !S.ok;
  if (S.ok && paged && S.nq > 0) {
    const int p0 = page_of(pg, S.first), p1 = page_of(pg, S.len - 1);
    for (int p = p0 + threadIdx.x; p <= p1; p += kRotateThreads)
      bad = bad || static_cast<unsigned>(__ldg(table + p)) >= static_cast<unsigned>(pg.num_pages);
  }
  bad = __syncthreads_or(bad);
  if (blockIdx.x == 0 && threadIdx.x == 0 && P.out_status) P.out_status[b] = bad ? SPECDEC_STATUS_BAD_CACHE : 0;
  if (i >= P.n) return;
  const bool live = !bad && i < S.nq;

  float cs[4], sn[4];
  if (turned) {
    const int64_t pos = static_cast<int64_t>(S.first) + (P.depth ? __ldg(P.depth + i) : i);
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const uint64_t turn = static_cast<uint64_t>(pos) * __ldg(P.turns + 4 * l + e);
      sincospif(static_cast<float>(static_cast<int32_t>(turn >> 32)) * 0x1p-31f, &sn[e], &cs[e]);
    }
  } else {
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      cs[e] = 1.f;
      sn[e] = 0.f;
    }
  }
  int64_t page_off = 0;
  if (paged && live) {
    const int at = S.first + i, page = page_of(pg, at);
    page_off = static_cast<int64_t>(__ldg(table + page)) * pg.page_stride + static_cast<int64_t>(at - page * pg.page_size) * pg.slot_stride;
  }
  const int64_t token = static_cast<int64_t>(b) * P.n + i;
  // a new token that does not exist gives zeros, a sequence in error NaN
  const uint32_t fill = bad ? 0x7fff7fffu : 0u;

  // rows r_first, r_first + r_step, ... of `count` (the lane groups of a warp meet at the
  // exchanges, so they share the loop); src and dst are row r_first's.  `ahead`: the first rows are loaded.
  auto rotate_rows = [&](const T* src, int64_t src_stride, char* dst, int64_t dst_stride, int count, const void* weight, bool ahead) {
    unsigned long long w[4] = {};
    if (weight) {
      const uint2 w0 = __ldg(static_cast<const uint2*>(weight) + pa), w1 = __ldg(static_cast<const uint2*>(weight) + pb);
      const uint32_t ww[4] = {w0.x, w0.y, w1.x, w1.y};
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const float2 f = Half16<T>::to_f32(ww[e]);
        w[e] = f2pack(f.x, f.y);
      }
    }
    auto load = [&](int r, int u) {
      if (r < count) {
        const uint2* const at = reinterpret_cast<const uint2*>(src + u * r_step * src_stride);
        ra[u] = __ldg(at + pa);
        rb[u] = __ldg(at + pb);
      }
    };
    if (!ahead) {
#pragma unroll
      for (int u = 0; u < kRowsAhead; ++u) load(r_first + u * r_step, u);
    }
    for (int r0 = r_first; r0 - group < count; r0 += kRowsAhead * r_step) {
      src += kRowsAhead * r_step * src_stride;
#pragma unroll
      for (int u = 0; u < kRowsAhead; ++u) {
        const int r = r0 + u * r_step;
        const uint32_t in[4] = {ra[u].x, ra[u].y, rb[u].x, rb[u].y};
        load(r + kRowsAhead * r_step, u);
        unsigned long long x[4], ss2 = 0ull;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const float2 f = Half16<T>::to_f32(in[e]);
          x[e] = f2pack(f.x, f.y);
          ss2 = f2fma(x[e], x[e], ss2);
        }
        if (weight) {
          float s0, s1;
          f2unpack(ss2, s0, s1);
          float ss = s0 + s1;
#pragma unroll
          for (int o = LPH / 2; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
          const float inv = rsqrtf(ss * (1.f / D) + P.eps);
          const unsigned long long inv2 = f2pack(inv, inv);
#pragma unroll
          for (int e = 0; e < 4; ++e) x[e] = f2mul(f2mul(x[e], inv2), w[e]);
        }
        unsigned long long y[4];
        if constexpr (INTERLEAVED) {  // pairs (x0, x1), (x2, x3), ... are the halves of x[0], x[1], ...
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            float x0, x1;
            f2unpack(x[e], x0, x1);
            y[e] = f2pack(x0 * cs[e] - x1 * sn[e], x1 * cs[e] + x0 * sn[e]);
          }
        } else {  // pairs (x0, x4), (x1, x5), ...: x[0] with x[2], x[1] with x[3]
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const unsigned long long c2 = f2pack(cs[2 * e], cs[2 * e + 1]), s2 = f2pack(sn[2 * e], sn[2 * e + 1]);
            const unsigned long long m2 = f2pack(-sn[2 * e], -sn[2 * e + 1]);
            y[e] = f2fma(x[e + 2], m2, f2mul(x[e], c2));
            y[e + 2] = f2fma(x[e], s2, f2mul(x[e + 2], c2));
          }
          if (!turned) {  // (0 times an infinity is not 0)
#pragma unroll
            for (int e = 0; e < 4; ++e) y[e] = x[e];
          }
        }
        uint32_t out[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          float y0, y1;
          f2unpack(y[e], y0, y1);
          out[e] = live ? Half16<T>::pack(y0, y1) : fill;
        }
        if (r < count) {
          uint2* const at = reinterpret_cast<uint2*>(dst + u * r_step * dst_stride);
          at[pa] = make_uint2(out[0], out[1]);
          at[pb] = make_uint2(out[2], out[3]);
        }
      }
      dst += kRowsAhead * r_step * dst_stride;
    }
  };
  rotate_rows(q_row, P.q_sh, reinterpret_cast<char*>(static_cast<T*>(P.q_out) + (token * P.Hq + r_first) * D), D * sizeof(T), P.Hq,
              P.q_weight, true);
  const T* const k_row = static_cast<const T*>(P.k) + b * P.k_sb + i * P.k_st + r_first * P.k_sh;
  if (!paged) {
    rotate_rows(k_row, P.k_sh, reinterpret_cast<char*>(static_cast<T*>(P.k_out) + (token * P.Hkv + r_first) * D), D * sizeof(T), P.Hkv,
                P.k_weight, false);
    return;
  }
  if (!live) return;
  rotate_rows(k_row, P.k_sh, pg.k + page_off + r_first * pg.head_stride, pg.head_stride, P.Hkv, P.k_weight, false);
  for (int r = r_first; r < P.Hkv; r += r_step)  // values go as they are
    reinterpret_cast<uint4*>(pg.v + page_off + r * pg.head_stride)[l] =
        __ldg(reinterpret_cast<const uint4*>(static_cast<const T*>(P.v) + b * P.v_sb + i * P.v_st + r * P.v_sh) + l);
}

template <typename T, int D>
cudaError_t launch_typed(const RotateParams& P, cudaStream_t stream) {
  // warps that share a token: enough warps to fill the GPU (152 SMs of 48 warps and more)
  const int64_t tokens = static_cast<int64_t>(P.B) * P.n;
  // (8193 tokens of 36 heads: 36 us with one warp a token, 45.6 with two, 51.8 with four; a few hundred
  // tokens are latency, and one warp would go through all the heads by itself)
  const int wpt = tokens < 1024 ? 8 : tokens < 2048 ? 4 : tokens < 4096 ? 2 : 1;
  const int per_cta = kRotateWarps / wpt;
  const dim3 grid(static_cast<unsigned>((P.n + per_cta - 1) / per_cta), static_cast<unsigned>(P.B));
  const dim3 block(kRotateThreads);
  return P.interleaved ? launch_kernel(rotate_qk_kernel<T, D, true>, grid, block, 0, stream, 0, P, int{wpt})
                       : launch_kernel(rotate_qk_kernel<T, D, false>, grid, block, 0, stream, 0, P, int{wpt});
}

}  // namespace

cudaError_t launch_rotate_qk(const RotateParams& P, specdec_dtype dt, cudaStream_t stream) {
  if (P.D == 64) return dt == SPECDEC_BF16 ? launch_typed<__nv_bfloat16, 64>(P, stream) : launch_typed<__half, 64>(P, stream);
  return dt == SPECDEC_BF16 ? launch_typed<__nv_bfloat16, 128>(P, stream) : launch_typed<__half, 128>(P, stream);
}

}  // namespace specdec
