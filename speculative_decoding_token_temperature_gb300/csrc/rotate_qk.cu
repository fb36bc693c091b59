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
// side by side, prompts by instructions and want the angles computed once.

#include "cache_device.cuh"
#include "specdec_device.cuh"

namespace specdec {

namespace {

constexpr int kRotateThreads = 256;
constexpr int kRotateWarps = kRotateThreads / 32;
constexpr int kRowsAhead = 4;  // rows a lane group loads before it works on the first

template <typename T, int D, bool INTERLEAVED>
__global__ void __launch_bounds__(kRotateThreads) rotate_qk_kernel(const RotateParams P, int warps_per_token) {
  constexpr int LPH = D / 8;     // lanes of a head
  constexpr int RPW = 32 / LPH;  // rows a warp takes at a time
  const int b = blockIdx.y, warp = threadIdx.x / 32, lane = threadIdx.x % 32, l = lane % LPH;
  const int i = blockIdx.x * (kRotateWarps / warps_per_token) + warp / warps_per_token;
  if (i >= P.n) return;
  const Pages& pg = P.pages;
  const bool paged = P.k_out == nullptr;
  const int rotated = P.Hq + P.Hkv, heads = rotated + (paged ? P.Hkv : 0);
  const int r_first = (warp % warps_per_token) * RPW + lane / LPH, r_step = warps_per_token * RPW;

  // this lane's two pieces of 4 values: the halves of 4 pairs, or values that are not rotated
  const int pairs = P.rot / 8;  // lanes with rotated values (interleaved: the same count)
  const bool turned = l < pairs;
  const int pa = INTERLEAVED ? 2 * l : turned ? l : 2 * l, pb = INTERLEAVED ? 2 * l + 1 : turned ? l + pairs : 2 * l + 1;
  auto row_of = [&](int r) -> const T* {
    if (r < P.Hq) return static_cast<const T*>(P.q) + b * P.q_sb + i * P.q_st + r * P.q_sh;
    if (r < rotated) return static_cast<const T*>(P.k) + b * P.k_sb + i * P.k_st + (r - P.Hq) * P.k_sh;
    return static_cast<const T*>(P.v) + b * P.v_sb + i * P.v_st + (r - rotated) * P.v_sh;
  };
  uint2 ra[kRowsAhead], rb[kRowsAhead];
  auto load = [&](int r0) {
#pragma unroll
    for (int u = 0; u < kRowsAhead; ++u) {
      const int r = r0 + u * r_step;
      if (r < heads) {
        const uint2* const src = reinterpret_cast<const uint2*>(row_of(r));
        ra[u] = __ldg(src + pa);
        rb[u] = __ldg(src + pb);
      } else {
        ra[u] = rb[u] = make_uint2(0u, 0u);
      }
    }
  };
  load(r_first);

  const SeqLen S = seq_len(P.context_len, P.query_len, b, P.n,
                           paged ? static_cast<int64_t>(pg.max_pages) * pg.page_size : INT32_MAX);
  const int32_t* table = pg.table + static_cast<int64_t>(b) * pg.max_pages;
  // a sequence with a bad length or page is left alone as a whole: every warp looks at all of
  // its new tokens' pages
  bool bad = !S.ok;
  if (S.ok && paged && S.nq > 0) {
    const int p0 = page_of(pg, S.first), p1 = page_of(pg, S.len - 1);
    for (int p = p0 + lane; p <= p1; p += 32)
      bad = bad || static_cast<unsigned>(__ldg(table + p)) >= static_cast<unsigned>(pg.num_pages);
  }
  bad = __any_sync(0xffffffffu, bad);
  if (i == 0 && warp % warps_per_token == 0 && lane == 0 && P.out_status) P.out_status[b] = bad ? SPECDEC_STATUS_BAD_CACHE : 0;
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
  uint2 wq[2] = {}, wk[2] = {};
  if (P.q_weight) {
    wq[0] = __ldg(static_cast<const uint2*>(P.q_weight) + pa);
    wq[1] = __ldg(static_cast<const uint2*>(P.q_weight) + pb);
  }
  if (P.k_weight) {
    wk[0] = __ldg(static_cast<const uint2*>(P.k_weight) + pa);
    wk[1] = __ldg(static_cast<const uint2*>(P.k_weight) + pb);
  }
  int64_t page_off = 0;
  if (paged && live) {
    const int at = S.first + i, page = page_of(pg, at);
    page_off = static_cast<int64_t>(__ldg(table + page)) * pg.page_stride + static_cast<int64_t>(at - page * pg.page_size) * pg.slot_stride;
  }
  const int64_t token = static_cast<int64_t>(b) * P.n + i;

  // (lane groups of a warp share the loop, so that all lanes meet at the exchanges)
  for (int r0 = r_first; r0 - lane / LPH < heads; r0 += kRowsAhead * r_step) {
    uint2 xa[kRowsAhead], xb[kRowsAhead];
#pragma unroll
    for (int u = 0; u < kRowsAhead; ++u) {
      xa[u] = ra[u];
      xb[u] = rb[u];
    }
    load(r0 + kRowsAhead * r_step);
#pragma unroll
    for (int u = 0; u < kRowsAhead; ++u) {
      const int r = r0 + u * r_step;
      if (r - lane / LPH >= heads) break;  // the whole warp
      const bool is_q = r < P.Hq;
      float x[8];
      {
        const float2 a0 = Half16<T>::to_f32(xa[u].x), a1 = Half16<T>::to_f32(xa[u].y);
        const float2 b0 = Half16<T>::to_f32(xb[u].x), b1 = Half16<T>::to_f32(xb[u].y);
        x[0] = a0.x; x[1] = a0.y; x[2] = a1.x; x[3] = a1.y;
        x[4] = b0.x; x[5] = b0.y; x[6] = b1.x; x[7] = b1.y;
      }
      float ss = 0.f;
#pragma unroll
      for (int e = 0; e < 8; ++e) ss += x[e] * x[e];
#pragma unroll
      for (int o = LPH / 2; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
      if ((is_q ? P.q_weight : P.k_weight) != nullptr) {
        const float inv = rsqrtf(ss * (1.f / D) + P.eps);
        const uint2 w0 = is_q ? wq[0] : wk[0], w1 = is_q ? wq[1] : wk[1];
        const float2 f0 = Half16<T>::to_f32(w0.x), f1 = Half16<T>::to_f32(w0.y), f2 = Half16<T>::to_f32(w1.x), f3 = Half16<T>::to_f32(w1.y);
        const float wf[8] = {f0.x, f0.y, f1.x, f1.y, f2.x, f2.y, f3.x, f3.y};
#pragma unroll
        for (int e = 0; e < 8; ++e) x[e] = x[e] * inv * wf[e];
      }
      uint2 ya, yb;
      if constexpr (INTERLEAVED) {  // pairs (x0, x1), (x2, x3), ...
        float y[8];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          y[2 * e] = x[2 * e] * cs[e] - x[2 * e + 1] * sn[e];
          y[2 * e + 1] = x[2 * e + 1] * cs[e] + x[2 * e] * sn[e];
        }
        ya = make_uint2(Half16<T>::pack(y[0], y[1]), Half16<T>::pack(y[2], y[3]));
        yb = make_uint2(Half16<T>::pack(y[4], y[5]), Half16<T>::pack(y[6], y[7]));
      } else {  // pairs (x0, x4), (x1, x5), ...
        float y[8];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          y[e] = x[e] * cs[e] - x[e + 4] * sn[e];
          y[e + 4] = x[e + 4] * cs[e] + x[e] * sn[e];
        }
        if (!turned) {
#pragma unroll
          for (int e = 0; e < 8; ++e) y[e] = x[e];
        }
        ya = make_uint2(Half16<T>::pack(y[0], y[1]), Half16<T>::pack(y[2], y[3]));
        yb = make_uint2(Half16<T>::pack(y[4], y[5]), Half16<T>::pack(y[6], y[7]));
      }
      if (r >= heads) continue;
      if (r >= rotated) {  // values go as they are
        ya = xa[u];
        yb = xb[u];
      } else if (!live) {  // a new token that does not exist gives zeros, a sequence in error NaN
        const uint32_t f = bad ? 0x7fff7fffu : 0u;
        ya = yb = make_uint2(f, f);
      }
      uint2* dst;
      if (is_q) {
        dst = reinterpret_cast<uint2*>(static_cast<T*>(P.q_out) + (token * P.Hq + r) * D);
      } else if (!paged) {
        dst = reinterpret_cast<uint2*>(static_cast<T*>(P.k_out) + (token * P.Hkv + (r - P.Hq)) * D);
      } else {
        if (!live) continue;
        dst = reinterpret_cast<uint2*>((r < rotated ? pg.k : pg.v) + page_off + (r < rotated ? r - P.Hq : r - rotated) * pg.head_stride);
      }
      dst[pa] = ya;
      dst[pb] = yb;
    }
  }
}

template <typename T, int D>
cudaError_t launch_typed(const RotateParams& P, cudaStream_t stream) {
  // warps that share a token: enough warps to fill the GPU (152 SMs of 48 warps and more)
  const int64_t tokens = static_cast<int64_t>(P.B) * P.n;
  const int wpt = tokens < 1024 ? 8 : tokens < 2048 ? 4 : tokens < 16384 ? 2 : 1;
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
