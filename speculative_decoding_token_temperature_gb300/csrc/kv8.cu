// Keys and values written to 8-bit cache pages, and read back.
//
// The slots of a block (scale_block slots of a page) share a scale 2^e for each head.  With y = x / t (t
// a tensor-wide scale, applied as a product with 1/t rounded to fp32): e is the smallest exponent in [-15, 7] with
// max|y| <= 448 * 2^e, and a value's code is the E4M3 number nearest to y / 2^e.  448 is 1.75 * 2^8, so e follows from
// the exponent of max|y| and one comparison of its significand, bit for bit.  Powers of two, because quotients by them are
// exact: a value is rounded once, and codes of a block whose scale grows later keep their significands (they are rounded
// again only where they become subnormal).  The range of e is what fp16 holds exactly: 448 * 2^7 is below 65504, and
// the smallest code, 2^-9, times 2^-15 is 2^-24.
//
// Calls one after another, 8 key heads of 128: 64 x 8 new tokens are written in 6.2 us (3.5 on the device, the rest is the host's)
// and 64 x 71 read back in 9.5 us: launches and a chain of dependent loads (lengths, pages, scales, codes).  4 x 2045 are written in 16.6 us
// (15.2 on the device; 50 MB, 3.3 TB/s) and 4 x 2060 read back in 13.8 us (50 MB, 3.7 TB/s), about twice what the copy rate would
// allow.  What holds these up is not measured; the write's CTAs go through that chain once each for four units of
// a few KB, and each of a read's store instructions fills half of the sectors that it touches.

#include "cache_device.cuh"
#include "specdec_device.cuh"

namespace specdec {

namespace {

constexpr int kThreads = 256;
constexpr int kPasses = 4;  // 16-byte pieces that a thread holds; more are read twice

// The largest finite magnitude of a piece as 16-bit bits, and whether some value is not finite.
template <typename T>
__device__ __forceinline__ uint32_t top_bits(const uint4& x, bool& odd) {
  constexpr uint32_t em = std::is_same<T, __half>::value ? 0x7c00u : 0x7f80u;
  const uint32_t w[4] = {x.x & 0x7fff7fffu, x.y & 0x7fff7fffu, x.z & 0x7fff7fffu, x.w & 0x7fff7fffu};
  const uint32_t m = __vmaxu2(__vmaxu2(w[0], w[1]), __vmaxu2(w[2], w[3]));
  uint32_t top = max(m & 0xffffu, m >> 16);
  odd = top >= em;
  if (odd) {
    top = 0;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const uint32_t lo = w[e] & 0xffffu, hi = w[e] >> 16;
      if (lo < em) top = max(top, lo);
      if (hi < em) top = max(top, hi);
    }
  }
  return top;
}

// The smallest e with a <= 448 * 2^e, clamped to the range (a >= 0; infinity, where a product with 1/t overflowed, gives the largest).
__device__ __forceinline__ int exponent_for(float a) {
  const int bits = __float_as_int(a);
  return min(max((bits >> 23) - 127 - 8 + ((bits & 0x7fffff) > 0x600000 ? 1 : 0), kLeastExponent), kMostExponent);
}

// Eight values as codes.  The product with the power of two is exact, so it goes into the factor, unless that could leave the normal
// range (inv_power 1 then says that it did not: the values are multiplied by it apart).
template <typename T>
__device__ __forceinline__ uint2 encode(const uint4& x, float inv_scale, float inv_power, bool odd) {
  const uint32_t w[4] = {x.x, x.y, x.z, x.w};
  uint32_t c[4];
#pragma unroll
  for (int p = 0; p < 4; ++p) {
    float2 f = Half16<T>::to_f32(w[p]);
    if (odd) {  // an infinity is NaN too
      if (!(fabsf(f.x) < kInf)) f.x = __int_as_float(0x7fffffff);
      if (!(fabsf(f.y) < kInf)) f.y = __int_as_float(0x7fffffff);
    }
    f.x *= inv_scale;
    f.y *= inv_scale;
    if (inv_power != 1.f) {
      f.x *= inv_power;
      f.y *= inv_power;
    }
    c[p] = to_e4m3x2(f.x, f.y);
  }
  return make_uint2(c[0] | (c[1] << 16), c[2] | (c[3] << 16));
}
// Eight codes for a scale 2^-shift times as large.
__device__ __forceinline__ uint2 encode_again(uint2 codes, float factor) {
  uint32_t w[2] = {codes.x, codes.y};
#pragma unroll
  for (int p = 0; p < 2; ++p) {
    uint32_t a, b;
    e4m3x4_to_f16(w[p], a, b);
    const float2 lo = Half16<__half>::to_f32(a), hi = Half16<__half>::to_f32(b);
    w[p] = to_e4m3x2(lo.x * factor, lo.y * factor) | (to_e4m3x2(hi.x * factor, hi.y * factor) << 16);
  }
  return make_uint2(w[0], w[1]);
}

// A unit is one block and one head of keys or values: UNIT threads, D / 8 to a slot.  grid (units of a sequence, B):
// the blocks that n new tokens may touch, times the columns (K's heads, then V's).
template <typename T, int D, int UNIT>
__global__ void __launch_bounds__(kThreads) append_kv8_kernel(const KvParams P) {
  const Pages& pg = P.pages;
  constexpr int PIECES = D / 8, ROWS = UNIT / PIECES, UNITS = kThreads / UNIT;  // slots at a time
  __shared__ uint32_t s_top[kThreads / 32];
  const int b = blockIdx.y, t = threadIdx.x % UNIT, piece = t % PIECES, columns = 2 * pg.kv_heads;
  const unsigned unit = blockIdx.x * UNITS + threadIdx.x / UNIT, block = unit / columns;
  const int column = static_cast<int>(unit - block * columns);
  const bool is_v = column >= pg.kv_heads;
  const int h = is_v ? column - pg.kv_heads : column;
  const SeqLen S = seq_len(P.context_len, P.query_len, b, P.n, static_cast<int64_t>(pg.max_pages) * pg.page_size);
  const int size = pg.scale_block;
  const int64_t from = (S.first / size + static_cast<int64_t>(block)) * size;  // the block's first slot
  const bool there = S.ok && S.nq > 0 && from < S.len;
  const int start = there ? static_cast<int>(from) : 0, lo = max(start, S.first);
  const int hi = there ? static_cast<int>(min(from + size, static_cast<int64_t>(S.len))) : 0;
  const T* const src = static_cast<const T*>(is_v ? P.v : P.k) + (is_v ? b * P.v_sb + h * P.v_sh : b * P.k_sb + h * P.k_sh) + piece * 8;
  const int64_t st = is_v ? P.v_st : P.k_st;
  auto load = [&](int slot) { return __ldg(reinterpret_cast<const uint4*>(src + (slot - S.first) * st)); };
  uint4 in[kPasses];
  bool odd[kPasses];
  if (there)
#pragma unroll
    for (int p = 0; p < kPasses; ++p) {
      const int slot = lo + t / PIECES + p * ROWS;
      in[p] = slot < hi ? load(slot) : make_uint4(0, 0, 0, 0);
    }
  // (the block's page and scale before the sequence's pages are known to fit: one wait less)
  const int logical = there ? page_of(pg, start) : 0, in_page = there ? start - logical * pg.page_size : 0;
  const int64_t page = there ? __ldg(pg.table + static_cast<int64_t>(b) * pg.max_pages + logical) : -1;
  uint8_t* const scale = reinterpret_cast<uint8_t*>(is_v ? pg.v_scales : pg.k_scales) + page * pg.scale_page_stride +
                         block_of(pg, in_page) * pg.scale_slot_stride + h * pg.scale_head_stride;
  int before = kLeastExponent;
  if (start < lo && page >= 0 && page < pg.num_pages) before = scale_exponent(*scale);
  const bool fits = sequence_fits(S, pg, b);
  if (blockIdx.x == 0 && threadIdx.x == 0 && P.out_status) P.out_status[b] = fits ? 0 : SPECDEC_STATUS_BAD_CACHE;
  if (!fits) return;
  const float inv_scale = is_v ? P.v_inv : P.k_inv;
  uint32_t top = 0;
  if (there) {
#pragma unroll
    for (int p = 0; p < kPasses; ++p) top = max(top, top_bits<T>(in[p], odd[p]));
    for (int slot = lo + t / PIECES + kPasses * ROWS; slot < hi; slot += ROWS) {
      bool any;
      top = max(top, top_bits<T>(load(slot), any));
    }
  }
  top = __reduce_max_sync(0xffffffffu, top);
  if constexpr (UNIT > 32) {
    if (threadIdx.x % 32 == 0) s_top[threadIdx.x / 32] = top;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < UNIT / 32; ++w) top = max(top, s_top[threadIdx.x / UNIT * (UNIT / 32) + w]);
  } else {
    __syncwarp();  // everybody has the scale of before
  }
  if (!there) return;
  // (the product with inv_scale keeps the order, so its largest is that of the largest)
  const int e = max(before, exponent_for(Half16<T>::to_f32(top).x * inv_scale));
  char* const dst = (is_v ? pg.v : pg.k) + page * pg.page_stride + in_page * pg.slot_stride + h * pg.head_stride + piece * 8;
  auto at = [&](int slot) { return reinterpret_cast<uint2*>(dst + (slot - start) * pg.slot_stride); };
  if (t == 0) *scale = static_cast<uint8_t>(e + 127);
  if (e > before)  // (of a block without earlier tokens there are none)
    for (int slot = start + t / PIECES; slot < lo; slot += ROWS) *at(slot) = encode_again(*at(slot), power_f32(before - e));
  const bool joint = inv_scale >= 0x1p-90f && inv_scale <= 0x1p90f;
  const float factor = joint ? inv_scale * power_f32(-e) : inv_scale, inv_power = joint ? 1.f : power_f32(-e);
#pragma unroll
  for (int p = 0; p < kPasses; ++p) {
    const int slot = lo + t / PIECES + p * ROWS;
    if (slot < hi) *at(slot) = encode<T>(in[p], factor, inv_power, odd[p]);
  }
  for (int slot = lo + t / PIECES + kPasses * ROWS; slot < hi; slot += ROWS) {
    const uint4 x = load(slot);
    *at(slot) = encode<T>(x, factor, inv_power, true);
  }
}

// Read back: a thread takes 16 codes of kReads tokens.  The places of a CTA's tokens stand in shared memory, and a thread adds
// its column's.  grid (chunks of a sequence's tokens x chunks of a token's columns, B)
constexpr int kReads = 4;

template <typename T, int D>
__global__ void __launch_bounds__(kThreads) read_kv8_kernel(const KvParams P) {
  const Pages& pg = P.pages;
  constexpr int PIECES = D / 16;
  __shared__ longlong2 s_at[kThreads / (2 * PIECES) * kReads];  // of a token's codes and scales
  const int b = blockIdx.y, columns = 2 * pg.kv_heads * PIECES, width = min(columns, kThreads), rows = kThreads / width;
  const unsigned chunks = (columns + kThreads - 1) / kThreads, part = blockIdx.x / chunks;
  const int i0 = static_cast<int>(part) * rows * kReads, row = threadIdx.x / width;
  int k = static_cast<int>(blockIdx.x - part * chunks) * kThreads + threadIdx.x - row * width;
  const bool mine = row < rows && k < columns, is_v = k >= columns / 2;
  if (is_v) k -= columns / 2;
  const int h = k / PIECES, piece = k % PIECES;
  const SeqLen S = seq_len(P.context_len, P.query_len, b, P.n, static_cast<int64_t>(pg.max_pages) * pg.page_size);
  for (int t = threadIdx.x; t < rows * kReads && S.ok && i0 + t < S.nq; t += kThreads) {
    const int slot = S.first + i0 + t, logical = page_of(pg, slot), in_page = slot - logical * pg.page_size;
    const int64_t page = __ldg(pg.table + static_cast<int64_t>(b) * pg.max_pages + logical);
    s_at[t] = make_longlong2(page * pg.page_stride + in_page * pg.slot_stride, page * pg.scale_page_stride + block_of(pg, in_page) * pg.scale_slot_stride);
  }
  const bool fits = sequence_fits(S, pg, b);
  if (blockIdx.x == 0 && threadIdx.x == 0 && P.out_status) P.out_status[b] = fits ? 0 : SPECDEC_STATUS_BAD_CACHE;
  if (!mine) return;
  const char* const src = (is_v ? pg.v : pg.k) + h * pg.head_stride + piece * 16;
  const uint8_t* const scales = reinterpret_cast<const uint8_t*>(is_v ? pg.v_scales : pg.k_scales) + h * pg.scale_head_stride;
  uint4 codes[kReads];
  uint32_t e[kReads];
#pragma unroll
  for (int u = 0; u < kReads; ++u) {
    const int t = u * rows + row;
    if (fits && i0 + t < S.nq) {
      const longlong2 at = s_at[t];
      codes[u] = *reinterpret_cast<const uint4*>(src + at.x);
      e[u] = scales[at.y];
    }
  }
  const float ts = is_v ? pg.v_scale : pg.k_scale;
  const int64_t token = static_cast<int64_t>(pg.kv_heads) * D;
  T* dst = static_cast<T*>(is_v ? P.v_out : P.k_out) + (static_cast<int64_t>(b) * P.n + i0 + row) * token + h * D + piece * 16;
#pragma unroll
  for (int u = 0; u < kReads; ++u, dst += rows * token) {
    const int i = i0 + u * rows + row;
    if (i >= P.n) break;
    uint32_t out[8];
    if (!fits || i >= S.nq) {  // NaN for a sequence in error, zeros for tokens it does not have
#pragma unroll
      for (int x = 0; x < 8; ++x) out[x] = fits ? 0u : 0x7fff7fffu;
    } else {
      const uint32_t s2 = power_f16x2(scale_exponent(e[u])), w[4] = {codes[u].x, codes[u].y, codes[u].z, codes[u].w};
#pragma unroll
      for (int x = 0; x < 4; ++x) {
        uint32_t f[2];
        e4m3x4_to_f16(w[x], f[0], f[1]);
#pragma unroll
        for (int y = 0; y < 2; ++y) {
          const float2 v = Half16<__half>::to_f32(mul_f16x2(f[y], s2));  // exact
          out[2 * x + y] = Half16<T>::pack(v.x * ts, v.y * ts);
        }
      }
    }
    reinterpret_cast<uint4*>(dst)[0] = make_uint4(out[0], out[1], out[2], out[3]);
    reinterpret_cast<uint4*>(dst)[1] = make_uint4(out[4], out[5], out[6], out[7]);
  }
}

template <typename T, int D>
cudaError_t append_shape(const KvParams& P, cudaStream_t stream) {
  const int size = P.pages.scale_block, rows = P.n < size ? P.n : size;
  const int64_t units = static_cast<int64_t>((static_cast<int64_t>(P.n) + size - 2) / size + 1) * 2 * P.pages.kv_heads;
  auto launch = [&](auto kernel, int unit) {
    const int64_t per = kThreads / unit;
    return launch_kernel(kernel, dim3(static_cast<unsigned>((units + per - 1) / per), static_cast<unsigned>(P.B)), dim3(kThreads), 0, stream, 0, P);
  };
  // A unit's pieces, and its threads: about four pieces a thread, for a CTA's way to its first byte (lengths, pages, scales) costs more
  // than its bytes.  Device time of 32, 64 and 256 threads, us (8 key heads; graphs of calls): 64 x 8 tokens, heads of 128 (128 pieces) 3.5,
  // 4.3, 8.9; 4 x 2045 tokens, heads of 64, a scale for 16 tokens (128) 7.8, 11.9, 33.6; the same with heads of 128 (256) 16.8, 15.2, 35.2;
  // 64 x 16 tokens (256) 5.4, 5.0, 9.5; a scale for 32 tokens (512) 17.9, 17.3, 20.6, of one request of 300 tokens 6.7, 4.4, 3.1; a scale
  // for 64 (1024) 27.2, 18.5, 13.6, for 256 (4096) 90.9, 48.9, 18.4.  (Between 256 and 1024 pieces long batches would like 64, short ones 256.)
  const int threads = rows * (D / 8);
  if (threads <= 128) return launch(append_kv8_kernel<T, D, 32>, 32);
  if (threads <= 256) return launch(append_kv8_kernel<T, D, 64>, 64);
  return launch(append_kv8_kernel<T, D, 256>, 256);
}
template <typename T, int D>
cudaError_t read_shape(const KvParams& P, cudaStream_t stream) {
  const int columns = 2 * P.pages.kv_heads * (D / 16), tokens = kThreads / (columns < kThreads ? columns : kThreads) * kReads;
  const unsigned grid = static_cast<unsigned>((P.n + tokens - 1) / tokens) * static_cast<unsigned>((columns + kThreads - 1) / kThreads);
  return launch_kernel(read_kv8_kernel<T, D>, dim3(grid, static_cast<unsigned>(P.B)), dim3(kThreads), 0, stream, 0, P);
}

}  // namespace

cudaError_t launch_append_kv8(const KvParams& P, specdec_dtype dt, cudaStream_t stream) {
  if (P.pages.head_dim == 64)
    return dt == SPECDEC_BF16 ? append_shape<__nv_bfloat16, 64>(P, stream) : append_shape<__half, 64>(P, stream);
  return dt == SPECDEC_BF16 ? append_shape<__nv_bfloat16, 128>(P, stream) : append_shape<__half, 128>(P, stream);
}

cudaError_t launch_read_kv8(const KvParams& P, specdec_dtype dt, cudaStream_t stream) {
  if (P.pages.head_dim == 64)
    return dt == SPECDEC_BF16 ? read_shape<__nv_bfloat16, 64>(P, stream) : read_shape<__half, 64>(P, stream);
  return dt == SPECDEC_BF16 ? read_shape<__nv_bfloat16, 128>(P, stream) : read_shape<__half, 128>(P, stream);
}

}  // namespace specdec
