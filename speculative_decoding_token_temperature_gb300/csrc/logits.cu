// What is done to the target's logits before they are verified, and the table of token counts it reads.
//
//   x = l;  if c > 0 or the token is in the prompt:  x = x > 0 ? x / r : x * r
//   y = x + (bias - (f c + p [c > 0])),  -inf where the row's mask has no bit
// for every token of every row, c the token's count among what the row follows: the sequence's own (`counts`) and the
// drafts before the row.  A token's bias and counts are the same for all rows of a sequence but for the few tokens that are
// drafts, so a thread keeps them for its columns in registers and runs over the rows; a column that is some
// draft's token takes a way of its own, which walks the row's drafts.

#include <algorithm>

#include "logits_ops.h"
#include "specdec_device.cuh"
#include "specdec_internal.h"

namespace specdec {

namespace {

constexpr int kThreads = 256;

template <typename T> struct Wide;  // 16 bytes of a row as fp32, and back
template <> struct Wide<float> {
  static __device__ __forceinline__ void unpack(const uint4& w, float (&x)[4]) {
    x[0] = __uint_as_float(w.x); x[1] = __uint_as_float(w.y); x[2] = __uint_as_float(w.z); x[3] = __uint_as_float(w.w);
  }
  static __device__ __forceinline__ uint4 pack(const float (&x)[4]) {
    return make_uint4(__float_as_uint(x[0]), __float_as_uint(x[1]), __float_as_uint(x[2]), __float_as_uint(x[3]));
  }
  static __device__ __forceinline__ float one(const float* p) { return *p; }
  static __device__ __forceinline__ void put(float* p, float x) { *p = x; }
};
__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {  // round to nearest even
  uint32_t w;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(w) : "f"(hi), "f"(lo));
  return w;
}
template <> struct Wide<uint16_t> {  // bf16
  static __device__ __forceinline__ void unpack(const uint4& w, float (&x)[8]) {
    x[0] = bf16_lo(w.x); x[1] = bf16_hi(w.x); x[2] = bf16_lo(w.y); x[3] = bf16_hi(w.y);
    x[4] = bf16_lo(w.z); x[5] = bf16_hi(w.z); x[6] = bf16_lo(w.w); x[7] = bf16_hi(w.w);
  }
  static __device__ __forceinline__ uint4 pack(const float (&x)[8]) {
    return make_uint4(pack_bf16(x[0], x[1]), pack_bf16(x[2], x[3]), pack_bf16(x[4], x[5]), pack_bf16(x[6], x[7]));
  }
  static __device__ __forceinline__ float one(const uint16_t* p) { return __uint_as_float(static_cast<uint32_t>(*p) << 16); }
  static __device__ __forceinline__ void put(uint16_t* p, float x) { *p = static_cast<uint16_t>(pack_bf16(x, 0.f)); }
};

struct Penalties {
  float repetition, presence, frequency;
  __device__ __forceinline__ float repeated(float x) const { return x > 0.f ? __fdiv_rn(x, repetition) : x * repetition; }
  // what is added for c occurrences
  __device__ __forceinline__ float added(int c, float bias) const { return c > 0 ? bias - fmaf(frequency, static_cast<float>(c), presence) : bias; }
};

// A CTA takes a chunk of the vocabulary and some rows of a sequence.  grid (chunks, groups of rows, B); VEC: 16 bytes of a row
// at a time, or one element where rows do not start on 16 bytes.
template <typename T, int VEC>
__global__ void __launch_bounds__(kThreads) process_kernel(const ProcessParams P) {
  constexpr int NV = VEC == 1 ? 4 : 1, CHUNK = kThreads * VEC * NV;
  __shared__ int s_bias[CHUNK];            // 1 + the entry of the bias list that counts for a token
  __shared__ uint32_t s_mark[CHUNK / 32];  // tokens of drafts
  extern __shared__ int s_draft[];         // [rows - 1] drafts, [rows - 1] their parents
  int* const s_parent = s_draft + P.rows - 1;
  const int b = blockIdx.z, lo = blockIdx.x * CHUNK, tid = threadIdx.x;
  int bad = 0, gamma = P.rows - 1;
  if (P.gammas) {
    gamma = __ldg(P.gammas + b);
    if (gamma < 0 || gamma >= P.rows) bad |= SPECDEC_STATUS_BAD_TOKEN;
  }
  const bool counted = bad == 0;
  Penalties pen;
  pen.repetition = P.repetition ? __ldg(P.repetition + b) : 1.f;
  pen.presence = P.presence ? __ldg(P.presence + b) : 0.f;
  pen.frequency = P.frequency ? __ldg(P.frequency + b) : 0.f;
  if (!(pen.repetition > 0.f && pen.repetition < kInf && fabsf(pen.presence) < kInf && fabsf(pen.frequency) < kInf))
    bad |= SPECDEC_STATUS_BAD_PENALTY;
  for (int k = tid; k < CHUNK; k += kThreads) s_bias[k] = 0;
  for (int k = tid; k < CHUNK / 32; k += kThreads) s_mark[k] = 0;
  __syncthreads();
  if (P.tokens && counted)
    for (int j = tid; j < gamma; j += kThreads) {
      const int t = __ldg(P.tokens + static_cast<int64_t>(b) * (P.rows - 1) + j);
      s_draft[j] = t;
      if (static_cast<unsigned>(t) >= static_cast<unsigned>(P.V)) bad |= SPECDEC_STATUS_BAD_TOKEN;
      else if (t >= lo && t - lo < CHUNK) atomicOr(&s_mark[(t - lo) / 32], 1u << ((t - lo) % 32));
      if (P.parents) {
        const int p = __ldg(P.parents + j);
        s_parent[j] = p;
        if (p < -1 || p >= j) bad |= SPECDEC_STATUS_BAD_TREE;
      }
    }
  for (int k = tid; k < P.num_bias; k += kThreads) {
    const int t = __ldg(P.bias_tokens + static_cast<int64_t>(b) * P.num_bias + k);
    if (t >= P.V) bad |= SPECDEC_STATUS_BAD_TOKEN;
    else if (t >= lo && t - lo < CHUNK) atomicMax(&s_bias[t - lo], k + 1);
  }
  // (__syncthreads_or gives a truth value: one for each bit)
  int status = 0;
#pragma unroll
  for (int bit : {SPECDEC_STATUS_BAD_TOKEN, SPECDEC_STATUS_BAD_TREE, SPECDEC_STATUS_BAD_PENALTY})
    if (__syncthreads_or(bad & bit)) status |= bit;
  if (blockIdx.x == 0 && blockIdx.y == 0 && tid == 0 && P.out_status) P.out_status[b] = status;

  // this thread's columns: VEC from col(v) on
  auto col = [&](int v) { return lo + (v * kThreads + tid) * VEC; };
  float add[NV][VEC];
  uint32_t seen[NV], mark[NV];  // bit e: column e is repeated, or some draft's token
#pragma unroll
  for (int v = 0; v < NV; ++v) {
    seen[v] = mark[v] = 0;
#pragma unroll
    for (int e = 0; e < VEC; ++e) {
      const int t = col(v) + e;
      add[v][e] = 0.f;
      if (t >= P.V) continue;
      const int c = P.counts ? __ldg(P.counts + static_cast<int64_t>(b) * P.V + t) : 0, k = s_bias[t - lo];
      add[v][e] = pen.added(c & 0x7fffffff, k ? __ldg(P.bias_values + static_cast<int64_t>(b) * P.num_bias + k - 1) : 0.f);
      seen[v] |= (c != 0 ? 1u : 0u) << e;
      mark[v] |= ((s_mark[(t - lo) / 32] >> ((t - lo) % 32)) & 1u) << e;
    }
  }
  // a column that is some draft's token
  auto marked = [&](float x, int t, int row) {
    int n = 0;
    for (int j = row - 1; j >= 0; j = P.parents ? s_parent[j] : j - 1) n += s_draft[j] == t;
    const int c = P.counts ? __ldg(P.counts + static_cast<int64_t>(b) * P.V + t) : 0, k = s_bias[t - lo];
    const float bias = k ? __ldg(P.bias_values + static_cast<int64_t>(b) * P.num_bias + k - 1) : 0.f;
    if (c != 0 || n > 0) x = pen.repeated(x);
    return x + pen.added((c & 0x7fffffff) + n, bias);
  };

  const int r0 = blockIdx.y * P.group, r1 = min(r0 + P.group, counted ? gamma + 1 : P.rows);
  for (int r = r0; r < r1; ++r) {
    const int64_t row = static_cast<int64_t>(b) * P.rows + r;
    const T* const src = static_cast<const T*>(P.logits) + row * P.V;
    T* const dst = static_cast<T*>(P.out) + row * P.V;
    const uint8_t* const mask = reinterpret_cast<const uint8_t*>(P.mask + (P.mask ? row * P.words : 0));
#pragma unroll
    for (int v = 0; v < NV; ++v) {
      const int t0 = col(v);
      if (t0 >= P.V) continue;
      uint32_t allowed = ~0u;
      if (P.mask) allowed = __ldg(mask + t0 / 8) >> (t0 % 8);
      float x[VEC];
      if constexpr (VEC == 1) x[0] = Wide<T>::one(src + t0);
      else Wide<T>::unpack(*reinterpret_cast<const uint4*>(src + t0), x);
#pragma unroll
      for (int e = 0; e < VEC; ++e) {
        if (status) x[e] = __int_as_float(0x7fffffff);
        else if (!((allowed >> e) & 1u)) x[e] = -kInf;
        else if ((mark[v] >> e) & 1u) x[e] = marked(x[e], t0 + e, r);
        else x[e] = ((seen[v] >> e) & 1u ? pen.repeated(x[e]) : x[e]) + add[v][e];
      }
      if constexpr (VEC == 1) Wide<T>::put(dst + t0, x[0]);
      else *reinterpret_cast<uint4*>(dst + t0) = Wide<T>::pack(x);
    }
  }
}

// ---- the table of counts --------------------------------------------------------------------

constexpr int kSign = static_cast<int>(0x80000000u);

__device__ __forceinline__ int tokens_of(const CountParams& P, int b) {
  return P.num_tokens ? min(max(__ldg(P.num_tokens + b), 0), P.n) : P.n;
}
// Whether the sequence has a token past the vocabulary (every thread of the CTA calls it).
__device__ __forceinline__ void report(const CountParams& P, int b, int n) {
  const int32_t* const tokens = P.tokens + b * P.token_stride;
  int bad = 0;
  for (int k = threadIdx.x; k < n; k += blockDim.x) bad |= __ldg(tokens + k) >= P.V;
  bad = __syncthreads_or(bad);
  if (threadIdx.x == 0) P.out_status[b] = bad ? SPECDEC_STATUS_BAD_TOKEN : 0;
}

// Tokens added one by one.  grid (tokens, B)
__global__ void __launch_bounds__(kThreads) count_kernel(const CountParams P) {
  const int b = blockIdx.y, n = tokens_of(P, b), k = blockIdx.x * kThreads + threadIdx.x;
  if (k < n) {
    const int t = __ldg(P.tokens + b * P.token_stride + k);
    int* const at = P.counts + static_cast<int64_t>(b) * P.V + t;
    if (static_cast<unsigned>(t) < static_cast<unsigned>(P.V)) {
      if (P.prompt) atomicOr(at, kSign);
      else atomicAdd(at, 1);
    }
  }
  if (blockIdx.x == 0 && P.out_status) report(P, b, n);
}

// A sequence's table from nothing: a CTA counts the tokens of its chunk of the vocabulary in shared memory and writes the
// chunk whole.  grid (chunks, B)
constexpr int kCountChunk = 8192;

__global__ void __launch_bounds__(kThreads) recount_kernel(const CountParams P) {
  __shared__ int s_count[kCountChunk];
  const int b = blockIdx.y, n = tokens_of(P, b), lo = blockIdx.x * kCountChunk;
  const int32_t* const tokens = P.tokens + b * P.token_stride;
  for (int k = threadIdx.x; k < kCountChunk; k += kThreads) s_count[k] = 0;
  __syncthreads();
  for (int k = threadIdx.x; k < n; k += kThreads) {
    const int t = __ldg(tokens + k);
    if (t < lo || t >= P.V || t - lo >= kCountChunk) continue;
    if (P.prompt) s_count[t - lo] = kSign;
    else atomicAdd(&s_count[t - lo], 1);
  }
  __syncthreads();
  int* const out = P.counts + static_cast<int64_t>(b) * P.V + lo;
  for (int k = threadIdx.x; k < kCountChunk && k < P.V - lo; k += kThreads) out[k] = s_count[k];
  if (blockIdx.x == 0 && P.out_status) report(P, b, n);
}

template <typename T, int VEC>
cudaError_t process_shape(ProcessParams P, cudaStream_t stream) {
  constexpr int CHUNK = kThreads * (VEC == 1 ? 4 : VEC);
  const int64_t chunks = (static_cast<int64_t>(P.V) + CHUNK - 1) / CHUNK;
  const int64_t want = 8 * device_sm_count(), have = chunks * P.B;  // CTAs: all SMs full once
  const int groups = static_cast<int>(std::min<int64_t>(P.rows, std::max<int64_t>(1, (want + have - 1) / have)));
  P.group = (P.rows + groups - 1) / groups;
  const size_t smem = P.tokens ? static_cast<size_t>(P.rows - 1) * 2 * sizeof(int) : 0;
  auto kernel = process_kernel<T, VEC>;
  if (cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kMaxProcessRows * 2 * static_cast<int>(sizeof(int))); e != cudaSuccess)
    return e;
  return launch_kernel(kernel, dim3(static_cast<unsigned>(chunks), static_cast<unsigned>((P.rows + P.group - 1) / P.group), static_cast<unsigned>(P.B)),
                       dim3(kThreads), smem, stream, 0, P);
}

}  // namespace

cudaError_t launch_process_logits(const ProcessParams& P, specdec_dtype dt, bool vec, cudaStream_t stream) {
  if (dt == SPECDEC_BF16) return vec ? process_shape<uint16_t, 8>(P, stream) : process_shape<uint16_t, 1>(P, stream);
  return vec ? process_shape<float, 4>(P, stream) : process_shape<float, 1>(P, stream);
}

cudaError_t launch_count_tokens(const CountParams& P, bool reset, cudaStream_t stream) {
  if (reset)
    return launch_kernel(recount_kernel, dim3(static_cast<unsigned>((static_cast<int64_t>(P.V) + kCountChunk - 1) / kCountChunk), static_cast<unsigned>(P.B)),
                         dim3(kThreads), 0, stream, 0, P);
  return launch_kernel(count_kernel, dim3(static_cast<unsigned>(std::max(1, (P.n + kThreads - 1) / kThreads)), static_cast<unsigned>(P.B)), dim3(kThreads), 0, stream, 0, P);
}

}  // namespace specdec
