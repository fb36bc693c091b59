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
// A CTA takes some tokens of a sequence and up to 256 of a token's columns (16 values to write, 8 to
// read); a thread keeps its column for kSteps tokens, so that what is left to do for each is the work on
// its values: the tokens' places in the pages stand in shared memory, and a thread adds its column's.
// 8180 tokens of 8 key heads of 128 in fp16 are written in 14.7 us (42.9 MB, 2.9 TB/s) and read back in
// 12.5 us (43 %, then 54 % of the issue slots): bound by instructions, and by the ramp of so short a
// kernel.  One group a thread with its place worked out for each took 19.7 and 14.0 us; four tokens a
// thread against two 25.2 and 29.4 us for the pair, eight 25.3.  Few tokens are bound by latency: 512
// tokens take 6.5 us a call.  y / s is the IEEE quotient from one reciprocal per group: with r = RN(1/s) and
// q = RN(y r), RN(q + RN(y - q s) r) is the correct rounding of y / s (P. Markstein, "Computation of
// elementary functions on the IBM RISC System/6000 processor", 1990; s has 4 significant bits, and all
// significands of y and s agree): 3 operations for each value.

#include "cache_device.cuh"
#include "specdec_device.cuh"

namespace specdec {

namespace {

constexpr int kKv4Threads = 256;
constexpr int kSteps = 4;  // tokens of a thread

// y / s from r = RN(1/s)
__device__ __forceinline__ float quotient(float y, float s, float r) {
  const float q = y * r;
  return fmaf(fmaf(-q, s, y), r, q);
}

// One group's 16 values as codes and a scale byte.
template <typename T>
__device__ __forceinline__ uint2 quantise(const uint4& lo, const uint4& hi, float inv_scale, uint8_t& scale) {
  const uint32_t w[8] = {lo.x, lo.y, lo.z, lo.w, hi.x, hi.y, hi.z, hi.w};
  // The largest magnitude, as bits: NaN is above infinity, and infinity above the others.  The product
  // with inv_scale keeps the order, so its largest is that of the largest.
  uint32_t top = 0;
#pragma unroll
  for (int p = 0; p < 8; ++p) top = __vmaxu2(top, w[p] & 0x7fff7fffu);
  const float amax = Half16<T>::to_f32(__vmaxu2(top, top >> 16)).x * inv_scale;
  if (!(amax < kInf)) {
    scale = 0x7f;
    return make_uint2(0u, 0u);
  }
  uint16_t s2;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(s2) : "f"(0.f), "f"(quotient(amax, 6.f, 1.f / 6.f)));
  scale = static_cast<uint8_t>(s2 & 0xff);
  const float s = __half2float(__ushort_as_half(static_cast<unsigned short>(e4m3x2_to_f16(s2) & 0xffffu)));
  if (!(s > 0.f)) return make_uint2(0u, 0u);
  const float r = 1.f / s;
  uint32_t word[2] = {0, 0};
#pragma unroll
  for (int p = 0; p < 8; ++p) {
    const float2 x = Half16<T>::to_f32(w[p]);
    const float y0 = x.x * inv_scale, y1 = x.y * inv_scale;
    uint32_t two;  // the first source goes to the high nibble; the quotient's sum has made +0 of -0
    asm("{\n.reg .b8 t;\ncvt.rn.satfinite.e2m1x2.f32 t, %1, %2;\ncvt.u32.u8 %0, t;\n}"
        : "=r"(two) : "f"(copysignf(quotient(y1, s, r), y1)), "f"(copysignf(quotient(y0, s, r), y0)));
    word[p / 4] |= (two & 0xffu) << (8 * (p % 4));
  }
  return make_uint2(word[0], word[1]);
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

// A thread's column of PER values of a token (K's heads, then V's), and its tokens: i, i + rows, ...
template <int PER>
struct Column {
  int rows, i0, row, h, part;  // tokens at a time, the CTA's first one, the thread's of rows, its head, place in the head
  bool is_v, there;
  __device__ explicit Column(const Pages& pg) {
    const int shift = (PER == 16 ? 2 : 3) + (pg.head_dim == 128);  // log2 of the columns of a head
    const int columns = 2 * pg.kv_heads << shift, width = min(columns, kKv4Threads);
    const unsigned chunks = (columns + kKv4Threads - 1) / kKv4Threads, tokens = blockIdx.x / chunks;
    rows = kKv4Threads / width;
    i0 = tokens * rows * kSteps;
    row = threadIdx.x / width;
    int k = (blockIdx.x - tokens * chunks) * kKv4Threads + threadIdx.x - row * width;
    there = row < rows && k < columns;
    is_v = 2 * k >= columns;
    if (is_v) k -= columns / 2;
    h = k >> shift;
    part = k & ((1 << shift) - 1);
  }
};
// Where the CTA's tokens are: the offsets of their slots in the codes and in the scales.
struct Slots {
  longlong2 at[kSteps * kKv4Threads / (2 * 64 / kGroup4)];
  __device__ void find(const Pages& pg, const SeqLen& S, int b, int i0, int tokens) {
    for (int t = threadIdx.x; t < tokens && S.ok && i0 + t < S.nq; t += kKv4Threads) {
      const int slot = S.first + i0 + t, logical = page_of(pg, slot);
      const int64_t page = __ldg(pg.table + static_cast<int64_t>(b) * pg.max_pages + logical);
      const int off = slot - logical * pg.page_size;
      at[t] = make_longlong2(page * pg.page_stride + off * pg.slot_stride, page * pg.scale_page_stride + off * pg.scale_slot_stride);
    }
  }
};

// grid (chunks of a sequence's tokens x chunks of a token's columns, B)
template <typename T>
__global__ void __launch_bounds__(kKv4Threads) append_kv4_kernel(const Kv4Params P) {
  const Pages& pg = P.pages;
  const int b = blockIdx.y;
  __shared__ Slots slots;
  const Column<kGroup4> c(pg);
  const T* src = static_cast<const T*>(c.is_v ? P.v : P.k) + (c.is_v ? b * P.v_sb + c.h * P.v_sh : b * P.k_sb + c.h * P.k_sh) + c.part * kGroup4;
  const int64_t st = c.is_v ? P.v_st : P.k_st;
  uint4 in[kSteps][2];
#pragma unroll
  for (int u = 0; u < kSteps; ++u) {  // (before the lengths and pages are there)
    const int i = c.i0 + u * c.rows + c.row;
    if (c.there && i < P.n) {
      const uint4* const from = reinterpret_cast<const uint4*>(src + i * st);
      in[u][0] = __ldg(from);
      in[u][1] = __ldg(from + 1);
    }
  }
  const SeqLen S = seq_len(P.context_len, P.query_len, b, P.n, static_cast<int64_t>(pg.max_pages) * pg.page_size);
  slots.find(pg, S, b, c.i0, c.rows * kSteps);
  const bool fits = sequence_fits(S, pg, b);
  if (blockIdx.x == 0 && threadIdx.x == 0 && P.out_status) P.out_status[b] = fits ? 0 : SPECDEC_STATUS_BAD_CACHE;
  if (!fits || !c.there) return;
  char* const dst = (c.is_v ? pg.v : pg.k) + c.h * pg.head_stride + c.part * (kGroup4 / 2);
  char* const sdst = (c.is_v ? pg.v_scales : pg.k_scales) + c.h * pg.scale_head_stride + c.part;
  const float inv_scale = c.is_v ? P.v_inv : P.k_inv;
#pragma unroll
  for (int u = 0; u < kSteps; ++u) {
    const int t = u * c.rows + c.row;
    if (c.i0 + t >= S.nq) break;
    uint8_t scale;
    const uint2 codes = quantise<T>(in[u][0], in[u][1], inv_scale, scale);
    const longlong2 at = slots.at[t];
    *reinterpret_cast<uint2*>(dst + at.x) = codes;
    *reinterpret_cast<uint8_t*>(sdst + at.y) = scale;
  }
}

// Read back by columns of 8 values: 4 bytes of codes and a scale in, 16 bytes out.
template <typename T>
__global__ void __launch_bounds__(kKv4Threads) read_kv4_kernel(const Kv4Params P) {
  const Pages& pg = P.pages;
  const int b = blockIdx.y;
  __shared__ Slots slots;
  const Column<8> c(pg);
  const SeqLen S = seq_len(P.context_len, P.query_len, b, P.n, static_cast<int64_t>(pg.max_pages) * pg.page_size);
  slots.find(pg, S, b, c.i0, c.rows * kSteps);
  const bool fits = sequence_fits(S, pg, b);
  if (blockIdx.x == 0 && threadIdx.x == 0 && P.out_status) P.out_status[b] = fits ? 0 : SPECDEC_STATUS_BAD_CACHE;
  if (!c.there) return;
  const char* const src = (c.is_v ? pg.v : pg.k) + c.h * pg.head_stride + c.part * 4;
  const char* const ssrc = (c.is_v ? pg.v_scales : pg.k_scales) + c.h * pg.scale_head_stride + c.part / 2;
  uint32_t codes[kSteps], scales[kSteps];
#pragma unroll
  for (int u = 0; u < kSteps; ++u) {
    const int t = u * c.rows + c.row;
    if (fits && c.i0 + t < S.nq) {
      const longlong2 at = slots.at[t];
      codes[u] = *reinterpret_cast<const uint32_t*>(src + at.x);
      scales[u] = *reinterpret_cast<const uint8_t*>(ssrc + at.y);
    }
  }
  const float ts = c.is_v ? pg.v_scale : pg.k_scale;
  const int64_t token = static_cast<int64_t>(pg.kv_heads) * pg.head_dim;
  T* const dst = static_cast<T*>(c.is_v ? P.v_out : P.k_out) + b * (P.n * token) + c.h * pg.head_dim + c.part * 8;
#pragma unroll
  for (int u = 0; u < kSteps; ++u) {
    const int i = c.i0 + u * c.rows + c.row;
    if (i >= P.n) break;
    uint32_t out[4];
    if (!fits || i >= S.nq) {  // NaN for a sequence in error, zeros for tokens it does not have
#pragma unroll
      for (int e = 0; e < 4; ++e) out[e] = fits ? 0u : 0x7fff7fffu;
    } else {
      const uint32_t s2 = e4m3x2_to_f16(0x101u * scales[u]);
      uint32_t f[4];
      e2m1x8_to_f16(codes[u], f[0], f[1], f[2], f[3]);
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const float2 v = Half16<__half>::to_f32(mul_f16x2(f[e], s2));  // exact: at most 6 significant bits
        out[e] = Half16<T>::pack(v.x * ts, v.y * ts);
      }
    }
    *reinterpret_cast<uint4*>(dst + i * token) = make_uint4(out[0], out[1], out[2], out[3]);
  }
}

dim3 columns_grid(const Kv4Params& P, int per) {
  const int columns = 2 * P.pages.kv_heads * (P.pages.head_dim / per);
  const int tokens = kKv4Threads / (columns < kKv4Threads ? columns : kKv4Threads) * kSteps;
  return dim3(static_cast<unsigned>((P.n + tokens - 1) / tokens) * static_cast<unsigned>((columns + kKv4Threads - 1) / kKv4Threads),
              static_cast<unsigned>(P.B));
}

}  // namespace

cudaError_t launch_append_kv4(const Kv4Params& P, specdec_dtype dt, cudaStream_t stream) {
  const dim3 block(kKv4Threads);
  return dt == SPECDEC_BF16 ? launch_kernel(append_kv4_kernel<__nv_bfloat16>, columns_grid(P, kGroup4), block, 0, stream, 0, P)
                            : launch_kernel(append_kv4_kernel<__half>, columns_grid(P, kGroup4), block, 0, stream, 0, P);
}

cudaError_t launch_read_kv4(const Kv4Params& P, specdec_dtype dt, cudaStream_t stream) {
  const dim3 block(kKv4Threads);
  return dt == SPECDEC_BF16 ? launch_kernel(read_kv4_kernel<__nv_bfloat16>, columns_grid(P, 8), block, 0, stream, 0, P)
                            : launch_kernel(read_kv4_kernel<__half>, columns_grid(P, 8), block, 0, stream, 0, P);
}

}  // namespace specdec
