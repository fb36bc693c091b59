// Keys and values written to 4-bit cache pages, and read back.
//
// Along D, every 16 values share a scale.  With y = x / t (t a tensor-wide scale, applied as a
// product with 1/t rounded to fp32): s = E4M3(max|y| / 6), saturated at 448, and a value's
// code is the E2M1 number (0, 0.5, 1, 1.5, 2, 3, 4, 6 and signs) nearest to y / s, ties to the
// even code; s = 0 gives zeros.  The divisions are IEEE fp32, so codes and scales are defined
// bit for bit.  E2M1 has no NaN: a group with a value that is not finite stores the scale
// NaN, and reads back as NaN.  E2M1 x E4M3 has at most 6 significant bits, so a value before
// its tensor-wide scale is exact in 16 bits.
//
// One thread per group: 32 bytes in, 8 bytes of codes and a scale byte out; neighbouring
// threads take neighbouring groups, so a token's bytes are written whole.  Bound by HBM on
// prompts, by latency for a few tokens.

#include "cache_device.cuh"
#include "specdec_device.cuh"

namespace specdec {

namespace {

constexpr int kKv4Threads = 256;

// One group's 16 values as codes and a scale byte.
__device__ __forceinline__ uint2 quantise(const float (&x)[16], float inv_scale, uint8_t& scale) {
  float y[16], amax = 0.f;
  bool finite = true;
#pragma unroll
  for (int e = 0; e < 16; ++e) {
    y[e] = x[e] * inv_scale;
    finite = finite && fabsf(y[e]) < kInf;
    amax = fmaxf(amax, fabsf(y[e]));
  }
  if (!finite) {
    scale = 0x7f;
    return make_uint2(0u, 0u);
  }
  uint16_t s2;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(s2) : "f"(0.f), "f"(amax / 6.f));
  scale = static_cast<uint8_t>(s2 & 0xff);
  const float s = __half2float(__ushort_as_half(static_cast<unsigned short>(e4m3x2_to_f16(s2) & 0xffffu)));
  if (!(s > 0.f)) return make_uint2(0u, 0u);
  uint32_t w[2];
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    uint32_t word = 0;
#pragma unroll
    for (int p = 0; p < 4; ++p) {
      const float lo = y[8 * h + 2 * p] / s, hi = y[8 * h + 2 * p + 1] / s;
      uint32_t two;  // the first source goes to the high nibble
      asm("{\n.reg .b8 t;\ncvt.rn.satfinite.e2m1x2.f32 t, %1, %2;\ncvt.u32.u8 %0, t;\n}" : "=r"(two) : "f"(hi), "f"(lo));
      word |= (two & 0xffu) << (8 * p);
    }
    w[h] = word;
  }
  return make_uint2(w[0], w[1]);
}

// Whether sequence b's lengths and the pages of its slots [first, len) are in range; every
// thread of the CTA calls it, and gets the same answer.
__device__ __forceinline__ bool sequence_fits(const SeqLen& S, const Pages& pg, int b) {
  int bad = S.ok ? 0 : 1;
  if (S.ok && S.nq > 0) {
    const int32_t* table = pg.table + static_cast<int64_t>(b) * pg.max_pages;
    const int p0 = page_of(pg, S.first), p1 = page_of(pg, S.len - 1);
    for (int p = p0 + threadIdx.x; p <= p1; p += blockDim.x)
      bad |= static_cast<unsigned>(__ldg(table + p)) >= static_cast<unsigned>(pg.num_pages);
  }
  return !__syncthreads_or(bad);
}

// The group of a thread: token i, K or V, head h, group g of the head.
struct Group {
  int i, h, g;
  bool is_v;
};
__device__ __forceinline__ Group group_of(const Pages& pg) {
  const int shift = pg.head_dim == 128 ? 3 : 2;  // log2 of the groups of a head
  const unsigned at = blockIdx.x * kKv4Threads + threadIdx.x, per_token = 2u * pg.kv_heads << shift;
  Group r;
  r.i = static_cast<int>(at / per_token);
  unsigned k = at - r.i * per_token;
  r.is_v = k >= per_token / 2;
  if (r.is_v) k -= per_token / 2;
  r.h = static_cast<int>(k >> shift);
  r.g = static_cast<int>(k & ((1u << shift) - 1));
  return r;
}

// grid (chunks of a sequence's groups, B); the groups of a token: Hkv * D/16 of K, then of V
template <typename T>
__global__ void __launch_bounds__(kKv4Threads) append_kv4_kernel(const Kv4Params P) {
  const Pages& pg = P.pages;
  const int b = blockIdx.y;
  const Group at = group_of(pg);
  uint4 a = make_uint4(0, 0, 0, 0), c = a;
  if (at.i < P.n) {  // (before the lengths and pages are there)
    const T* src = static_cast<const T*>(at.is_v ? P.v : P.k) +
                   (at.is_v ? b * P.v_sb + at.i * P.v_st + at.h * P.v_sh : b * P.k_sb + at.i * P.k_st + at.h * P.k_sh) + at.g * kGroup4;
    a = __ldg(reinterpret_cast<const uint4*>(src));
    c = __ldg(reinterpret_cast<const uint4*>(src) + 1);
  }
  const SeqLen S = seq_len(P.context_len, P.query_len, b, P.n, static_cast<int64_t>(pg.max_pages) * pg.page_size);
  const bool fits = sequence_fits(S, pg, b);
  if (blockIdx.x == 0 && threadIdx.x == 0 && P.out_status) P.out_status[b] = fits ? 0 : SPECDEC_STATUS_BAD_CACHE;
  if (!fits || at.i >= S.nq) return;
  const int slot = S.first + at.i, logical = page_of(pg, slot);
  const int64_t page = __ldg(pg.table + static_cast<int64_t>(b) * pg.max_pages + logical);
  const int off = slot - logical * pg.page_size;
  const uint32_t in[8] = {a.x, a.y, a.z, a.w, c.x, c.y, c.z, c.w};
  float x[16];
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    const float2 f = Half16<T>::to_f32(in[e]);
    x[2 * e] = f.x;
    x[2 * e + 1] = f.y;
  }
  uint8_t scale;
  const uint2 codes = quantise(x, 1.f / (at.is_v ? pg.v_scale : pg.k_scale), scale);
  char* dst = (at.is_v ? pg.v : pg.k) + page * pg.page_stride + off * pg.slot_stride + at.h * pg.head_stride;
  char* sdst = (at.is_v ? pg.v_scales : pg.k_scales) + page * pg.scale_page_stride + off * pg.scale_slot_stride +
               at.h * pg.scale_head_stride;
  reinterpret_cast<uint2*>(dst)[at.g] = codes;
  reinterpret_cast<uint8_t*>(sdst)[at.g] = scale;
}

// The same groups read back: 8 bytes of codes and a scale in, 16 values out.
template <typename T>
__global__ void __launch_bounds__(kKv4Threads) read_kv4_kernel(const Kv4Params P) {
  const Pages& pg = P.pages;
  const int b = blockIdx.y;
  const SeqLen S = seq_len(P.context_len, P.query_len, b, P.n, static_cast<int64_t>(pg.max_pages) * pg.page_size);
  const bool fits = sequence_fits(S, pg, b);
  if (blockIdx.x == 0 && threadIdx.x == 0 && P.out_status) P.out_status[b] = fits ? 0 : SPECDEC_STATUS_BAD_CACHE;
  const Group at = group_of(pg);
  if (at.i >= P.n) return;
  uint32_t out[8];
  if (!fits || at.i >= S.nq) {  // NaN for a sequence in error, zeros for tokens it does not have
#pragma unroll
    for (int e = 0; e < 8; ++e) out[e] = fits ? 0u : 0x7fff7fffu;
  } else {
    const int slot = S.first + at.i, logical = page_of(pg, slot);
    const int64_t page = __ldg(pg.table + static_cast<int64_t>(b) * pg.max_pages + logical);
    const int off = slot - logical * pg.page_size;
    const char* src = (at.is_v ? pg.v : pg.k) + page * pg.page_stride + off * pg.slot_stride + at.h * pg.head_stride;
    const char* ssrc = (at.is_v ? pg.v_scales : pg.k_scales) + page * pg.scale_page_stride + off * pg.scale_slot_stride +
                       at.h * pg.scale_head_stride;
    const uint2 codes = reinterpret_cast<const uint2*>(src)[at.g];
    const uint32_t sb = reinterpret_cast<const uint8_t*>(ssrc)[at.g];
    const float s = __half2float(__ushort_as_half(static_cast<unsigned short>(e4m3x2_to_f16(sb) & 0xffffu)));
    const float t = at.is_v ? pg.v_scale : pg.k_scale;
    uint32_t f[8];
    e2m1x8_to_f16(codes.x, f[0], f[1], f[2], f[3]);
    e2m1x8_to_f16(codes.y, f[4], f[5], f[6], f[7]);
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const float2 v = Half16<__half>::to_f32(f[e]);
      out[e] = Half16<T>::pack(v.x * s * t, v.y * s * t);  // v * s is exact
    }
  }
  T* dst = static_cast<T*>(at.is_v ? P.v_out : P.k_out) +
           ((static_cast<int64_t>(b) * P.n + at.i) * pg.kv_heads + at.h) * pg.head_dim + at.g * kGroup4;
  reinterpret_cast<uint4*>(dst)[0] = make_uint4(out[0], out[1], out[2], out[3]);
  reinterpret_cast<uint4*>(dst)[1] = make_uint4(out[4], out[5], out[6], out[7]);
}

dim3 groups_grid(const Kv4Params& P) {
  const int64_t groups = static_cast<int64_t>(P.n) * 2 * P.pages.kv_heads * (P.pages.head_dim / kGroup4);
  return dim3(static_cast<unsigned>((groups + kKv4Threads - 1) / kKv4Threads), static_cast<unsigned>(P.B));
}

}  // namespace

cudaError_t launch_append_kv4(const Kv4Params& P, specdec_dtype dt, cudaStream_t stream) {
  const dim3 block(kKv4Threads);
  return dt == SPECDEC_BF16 ? launch_kernel(append_kv4_kernel<__nv_bfloat16>, groups_grid(P), block, 0, stream, 0, P)
                            : launch_kernel(append_kv4_kernel<__half>, groups_grid(P), block, 0, stream, 0, P);
}

cudaError_t launch_read_kv4(const Kv4Params& P, specdec_dtype dt, cudaStream_t stream) {
  const dim3 block(kKv4Threads);
  return dt == SPECDEC_BF16 ? launch_kernel(read_kv4_kernel<__nv_bfloat16>, groups_grid(P), block, 0, stream, 0, P)
                            : launch_kernel(read_kv4_kernel<__half>, groups_grid(P), block, 0, stream, 0, P);
}

}  // namespace specdec
