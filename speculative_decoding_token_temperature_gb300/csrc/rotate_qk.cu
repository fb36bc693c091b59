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
// One CTA per token: its rot/2 angles are computed once, into shared memory, and used by all
// heads.  A head's row is D/8 lanes of 16 bytes; a lane's row loads are issued before the
// angles, so the two latencies overlap.  The kernel is bound by HBM on prompts and by the
// chain length -> page -> store for a few tokens.

#include "cache_device.cuh"
#include "specdec_device.cuh"

namespace specdec {

namespace {

constexpr int kRotateThreads = 256;
constexpr int kRowsAhead = 4;  // rows a lane group loads before it waits for the angles

template <typename T, int D>
__global__ void __launch_bounds__(kRotateThreads) rotate_qk_kernel(const RotateParams P) {
  constexpr int LPH = D / 8;  // lanes of a head
  constexpr int SLOTS = kRotateThreads / LPH;
  __shared__ float2 s_cs[D / 2];
  const int b = blockIdx.y, i = blockIdx.x;
  const int tid = threadIdx.x, slot = tid / LPH, l = tid % LPH;
  const Pages& pg = P.pages;
  const bool paged = P.k_out == nullptr;
  const int heads = P.Hq + P.Hkv + (paged ? P.Hkv : 0);

  auto src_row = [&](int r) -> const T* {
    if (r < P.Hq) return static_cast<const T*>(P.q) + b * P.q_sb + i * P.q_st + r * P.q_sh;
    if (r < P.Hq + P.Hkv) return static_cast<const T*>(P.k) + b * P.k_sb + i * P.k_st + (r - P.Hq) * P.k_sh;
    return static_cast<const T*>(P.v) + b * P.v_sb + i * P.v_st + (r - P.Hq - P.Hkv) * P.v_sh;
  };
  uint4 rows[kRowsAhead];
#pragma unroll
  for (int u = 0; u < kRowsAhead; ++u) {
    const int r = slot + u * SLOTS;
    if (r < heads) rows[u] = __ldg(reinterpret_cast<const uint4*>(src_row(r)) + l);
  }

  const SeqLen S = seq_len(P.context_len, P.query_len, b, P.n,
                           paged ? static_cast<int64_t>(pg.max_pages) * pg.page_size : INT32_MAX);
  const int32_t* table = pg.table + static_cast<int64_t>(b) * pg.max_pages;
  // a sequence with a bad length or page is left alone as a whole: every CTA looks at all of
  // its new tokens' pages
  int bad = S.ok ? 0 : 1;
  if (S.ok && paged && S.nq > 0) {
    const int p0 = S.first / pg.page_size, p1 = (S.len - 1) / pg.page_size;
    for (int p = p0 + tid; p <= p1; p += kRotateThreads)
      bad |= static_cast<unsigned>(__ldg(table + p)) >= static_cast<unsigned>(pg.num_pages);
  }
  if (tid < P.rot / 2) {
    const int64_t pos = static_cast<int64_t>(S.first) + (P.depth ? __ldg(P.depth + i) : i);
    const uint64_t turn = static_cast<uint64_t>(pos) * __ldg(P.turns + tid);
    const float half_turns = static_cast<float>(static_cast<int32_t>(turn >> 32)) * 0x1p-31f;
    float s, c;
    sincospif(half_turns, &s, &c);
    s_cs[tid] = make_float2(c, s);
  }
  bad = __syncthreads_or(bad);
  if (i == 0 && tid == 0 && P.out_status) P.out_status[b] = bad ? SPECDEC_STATUS_BAD_CACHE : 0;
  const bool live = !bad && i < S.nq;
  int64_t page_off = 0;
  if (paged && live) {
    const int at = S.first + i;
    page_off = static_cast<int64_t>(__ldg(table + at / pg.page_size)) * pg.page_stride +
               static_cast<int64_t>(at % pg.page_size) * pg.slot_stride;
  }
  const int half = P.rot / 16;  // lanes that hold the first half of the rotated values

  for (int r0 = slot; r0 - slot < heads; r0 += kRowsAhead * SLOTS) {
    if (r0 != slot) {
#pragma unroll
      for (int u = 0; u < kRowsAhead; ++u) {
        const int r = r0 + u * SLOTS;
        if (r < heads) rows[u] = __ldg(reinterpret_cast<const uint4*>(src_row(r)) + l);
      }
    }
#pragma unroll
    for (int u = 0; u < kRowsAhead; ++u) {
      const int r = r0 + u * SLOTS;  // lane groups of one warp may differ here: no early exit
      const bool is_q = r < P.Hq, is_v = r >= P.Hq + P.Hkv;
      const uint32_t in[4] = {rows[u].x, rows[u].y, rows[u].z, rows[u].w};
      float x[8];
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const float2 f = Half16<T>::to_f32(r < heads ? in[e] : 0u);
        x[2 * e] = f.x;
        x[2 * e + 1] = f.y;
      }
      const void* w = is_q ? P.q_weight : P.k_weight;
      float ss = 0.f;
#pragma unroll
      for (int e = 0; e < 8; ++e) ss += x[e] * x[e];
#pragma unroll
      for (int o = LPH / 2; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
      if (w != nullptr) {
        const float inv = rsqrtf(ss * (1.f / D) + P.eps);
        const uint4 wv = __ldg(static_cast<const uint4*>(w) + l);
        const uint32_t ww[4] = {wv.x, wv.y, wv.z, wv.w};
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const float2 f = Half16<T>::to_f32(ww[e]);
          x[2 * e] = x[2 * e] * inv * f.x;
          x[2 * e + 1] = x[2 * e + 1] * inv * f.y;
        }
      }
      float y[8];
      if (P.interleaved) {
#pragma unroll
        for (int e = 0; e < 8; e += 2) {
          const int j = (8 * l + e) / 2;
          const float2 cs = 2 * j < P.rot ? s_cs[j] : make_float2(1.f, 0.f);
          y[e] = x[e] * cs.x - x[e + 1] * cs.y;
          y[e + 1] = x[e + 1] * cs.x + x[e] * cs.y;
        }
      } else {
        const bool lo = l < half, turned = l < 2 * half;
        const int from = (tid & 31 & ~(LPH - 1)) + (lo ? l + half : turned ? l - half : l);
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const float other = __shfl_sync(0xffffffffu, x[e], from);
          const float2 cs = turned ? s_cs[(lo ? l : l - half) * 8 + e] : make_float2(1.f, 0.f);
          y[e] = lo ? x[e] * cs.x - other * cs.y : x[e] * cs.x + other * cs.y;
          if (!turned) y[e] = x[e];
        }
      }
      if (r >= heads) continue;
      uint4 out = rows[u];
      if (!is_v) {
        out.x = Half16<T>::pack(y[0], y[1]);
        out.y = Half16<T>::pack(y[2], y[3]);
        out.z = Half16<T>::pack(y[4], y[5]);
        out.w = Half16<T>::pack(y[6], y[7]);
        // a new token that does not exist gives zeros, a sequence in error NaN
        if (!live) {
          const uint32_t f = bad ? 0x7fff7fffu : 0u;
          out = make_uint4(f, f, f, f);
        }
      }
      const int64_t token = static_cast<int64_t>(b) * P.n + i;
      if (is_q) {
        reinterpret_cast<uint4*>(static_cast<T*>(P.q_out) + (token * P.Hq + r) * D)[l] = out;
      } else if (!paged) {
        reinterpret_cast<uint4*>(static_cast<T*>(P.k_out) + (token * P.Hkv + (r - P.Hq)) * D)[l] = out;
      } else if (live) {
        char* base = is_v ? pg.v : pg.k;
        const int h = is_v ? r - P.Hq - P.Hkv : r - P.Hq;
        reinterpret_cast<uint4*>(base + page_off + h * pg.head_stride)[l] = out;
      }
    }
  }
}

template <typename T>
cudaError_t launch_typed(const RotateParams& P, cudaStream_t stream) {
  const dim3 grid(static_cast<unsigned>(P.n), static_cast<unsigned>(P.B));
  const dim3 block(kRotateThreads);
  if (P.D == 64) return launch_kernel(rotate_qk_kernel<T, 64>, grid, block, 0, stream, 0, P);
  return launch_kernel(rotate_qk_kernel<T, 128>, grid, block, 0, stream, 0, P);
}

}  // namespace

cudaError_t launch_rotate_qk(const RotateParams& P, specdec_dtype dt, cudaStream_t stream) {
  return dt == SPECDEC_BF16 ? launch_typed<__nv_bfloat16>(P, stream) : launch_typed<__half>(P, stream);
}

}  // namespace specdec
