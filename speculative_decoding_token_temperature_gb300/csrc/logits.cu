// What is done to the target's logits before they are verified, and the table of token counts it reads.
//
//   x = l;  if c > 0 or the token is in the prompt:  x = x > 0 ? x / r : x * r
//   y = x + (bias - (f c + p [c > 0])),  -inf where the row's mask has no bit
// for every token of every row, c the token's count among what the row follows: the sequence's own (`counts`) and the
// drafts before the row.
//
// Few tokens of a vocabulary have a count, a bias or are drafts; for all others y = l, or -inf.  So the call is a copy of the rows
// under their masks, bound by HBM, in which a few elements are changed on the way.  A CTA takes a chunk of the vocabulary and some
// rows of a sequence.  The rows come to shared memory by 16-byte asynchronous copies, kBatch at a time and two batches ahead, while
// the CTA lists its chunk's tokens that change; those are changed in shared memory, and the words go out.
//
// 256 x 8 rows of 128256 in bf16: 203 us, 0.86 of the measured copy rate; in place, where listed tokens alone are read and written, by single
// elements, 247 us against a floor of 69.  32 x 65 rows of 32001 under masks 107 us (floor 41), of 32000 83.  A draft's token is
// counted anew for each row, along the row's whole path: nothing at a round's tens of rows, but 1 x 1024 rows of different drafts take 0.2 ms (a
// chain) to 0.6 ms (a path of a tree), 8192 58 to 187 ms.

#include <algorithm>

#include "logits_ops.h"
#include "specdec_device.cuh"
#include "specdec_internal.h"

namespace specdec {

namespace {

constexpr int kThreads = 256;

template <typename T> struct Elem16;  // an element as fp32, and back
template <> struct Elem16<float> {
  static constexpr uint32_t kNone = 0xff800000u, kPair = 1;  // -inf in a word; elements of a word
  static __device__ __forceinline__ float part(const uint32_t (&w)[4], int e) { return __uint_as_float(w[e]); }
  static __device__ __forceinline__ float get(float x) { return x; }
  static __device__ __forceinline__ float put(float x) { return x; }
};
template <> struct Elem16<uint16_t> {  // bf16
  static constexpr uint32_t kNone = 0xff80ff80u, kPair = 2;
  static __device__ __forceinline__ uint16_t part(const uint32_t (&w)[4], int e) { return static_cast<uint16_t>(w[e / 2] >> (16 * (e % 2))); }
  static __device__ __forceinline__ float get(uint16_t x) { return __uint_as_float(static_cast<uint32_t>(x) << 16); }
  static __device__ __forceinline__ uint16_t put(float x) {  // round to nearest even
    uint16_t w;
    asm("cvt.rn.bf16.f32 %0, %1;" : "=h"(w) : "f"(x));
    return w;
  }
};

struct Penalties {
  float repetition, presence, frequency;
  // a token's value: the quotient or product, then the sum, each rounded to nearest (not contracted into one rounding, so that every
  // place where a value is computed gives the same bits)
  __device__ __forceinline__ float value(float x, bool repeated, float add) const {
    return __fadd_rn(!repeated ? x : x > 0.f ? __fdiv_rn(x, repetition) : __fmul_rn(x, repetition), add);
  }
  // what is added for c occurrences
  __device__ __forceinline__ float added(int c, float bias) const { return c > 0 ? bias - fmaf(frequency, static_cast<float>(c), presence) : bias; }
};

// Rows of a batch, and batches in flight.  256 x 8 rows of 128256 logits in bf16, 32 x 65 rows of 32001 under masks (us): 2, 2: 196,
// 110; 4, 2: 215, 117; 4, 1: 211, 107; 2, 3: 195, 112; 2, 4: 229, 125.  (Rows held in registers, and the tokens changed in them
// or in a pass of their own behind the copy: 217 to 275, 156 to 194.  All of these with products by a reciprocal; with quotients 2, 2: 203, 107.)
constexpr int kBatch = 2, kStages = 2;

__device__ __forceinline__ void copy_async16(void* dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(smem_addr(dst)), "l"(src) : "memory");
}
__device__ __forceinline__ void copy_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int LEFT>
__device__ __forceinline__ void copy_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(LEFT) : "memory");
}

// The columns of a CTA: 16 bytes of a row for each thread, one less where rows do not start on 16 bytes (and a chunk then
// touches a word more).
template <typename T, bool ALIGNED>
constexpr int kChunk = (ALIGNED ? kThreads : kThreads - 1) * (16 / static_cast<int>(sizeof(T)));

// ALIGNED: every row of logits and out starts on 16 bytes.  grid (chunks, groups of rows, B)
template <typename T, bool ALIGNED, bool MASKED>
__global__ void __launch_bounds__(kThreads) process_kernel(const ProcessParams P) {
  constexpr int N = 16 / sizeof(T), CHUNK = kChunk<T, ALIGNED>, WORDS = kThreads * N / 32;
  constexpr uint32_t kAll = (1u << N) - 1;
  using E = Elem16<T>;
  __shared__ __align__(16) T s_rows[kStages][kBatch][kThreads * N];
  __shared__ __align__(16) int s_value[kThreads * N];  // by column: 1 + the entry of the bias list that counts, then what is added
  __shared__ uint16_t s_list[kThreads * N];            // the columns that change
  __shared__ uint32_t s_some[WORDS], s_mark[WORDS];    // the same as bits; columns that are some draft's token
  __shared__ int s_sum[kThreads / 32], s_status;
  extern __shared__ int s_draft[];                     // [rows - 1] drafts, [rows - 1] their parents
  int* const s_parent = s_draft + P.rows - 1;
  const int b = blockIdx.z, lo = blockIdx.x * CHUNK, size = min(CHUNK, P.V - lo), tid = threadIdx.x, lane = tid % 32;
  const int64_t row0 = static_cast<int64_t>(b) * P.rows;
  const T* const logits = static_cast<const T*>(P.logits);

  int gamma = P.rows - 1;
  if (P.gammas) gamma = __ldg(P.gammas + b);
  const bool counted = gamma >= 0 && gamma < P.rows;
  const int r0 = blockIdx.y * P.group, r1 = min(r0 + P.group, counted ? gamma + 1 : P.rows);
  // the chunk's part of row r, and how many elements past a 16-byte border it starts
  auto from = [&](int r) { return logits + (row0 + r) * P.V + lo; };
  auto to = [&](int r) { return static_cast<T*>(P.out) + (row0 + r) * P.V + lo; };
  auto past = [&](const T* row) { return ALIGNED ? 0 : static_cast<int>(reinterpret_cast<uintptr_t>(row) / sizeof(T)) & (N - 1); };
  auto bit = [&](int r, int t) -> bool {
    return __ldg(reinterpret_cast<const uint8_t*>(P.mask + (row0 + r) * P.words) + (lo + t) / 8) >> ((lo + t) % 8) & 1u;
  };
  // This thread's word of a row is columns tid * N - past ..: the elements of it that are the chunk's, and those that the mask allows.
  auto mine = [&](int off) -> uint32_t {
    const int first = tid * N - off;
    if (ALIGNED) return first < size ? kAll : 0u;
    const uint32_t below = first >= 0 ? kAll : kAll & (kAll << -first), over = size - first >= N ? kAll : size > first ? (1u << (size - first)) - 1 : 0u;
    return below & over;
  };
  // (the first in the low byte, the second in the next)
  auto look = [&](int r) -> uint32_t {
    if (r >= r1) return 0u;
    const int off = past(from(r));
    const uint32_t there = mine(off);
    uint32_t some = there;
    if constexpr (MASKED) {
      if (some == 0) return 0u;
      const uint8_t* const m = reinterpret_cast<const uint8_t*>(P.mask + (row0 + r) * P.words);
      if constexpr (ALIGNED) {
        some &= __ldg(m + (lo + tid * N) / 8) >> ((lo + tid * N) % 8);
      } else {  // (a column below 0 belongs to another chunk or row: not looked at)
        const int first = lo + tid * N - off, last = min(first + N, P.V) - 1;
        uint32_t w = first >= 0 ? __ldg(m + first / 8) : 0u;
        if (last / 8 != (first < 0 ? -1 : first / 8)) w |= static_cast<uint32_t>(__ldg(m + last / 8)) << (first < 0 ? 0 : 8);
        some &= first >= 0 ? w >> (first % 8) : w << -first;
      }
    }
    return there | some << 8;
  };
  uint32_t looked[kStages][kBatch];  // of the batches in flight
  auto issue = [&](int r, int stage) {
#pragma unroll
    for (int k = 0; k < kBatch; ++k) {
      const uint32_t allowed = looked[stage][k] >> 8;
      if (allowed == 0) continue;
      const T* const row = from(r + k);
      const T* const at = row - past(row) + tid * N;
      T* const dst = s_rows[stage][k] + tid * N;
      if (ALIGNED || (at >= logits && at + N <= logits + static_cast<int64_t>(P.B) * P.rows * P.V)) {
        copy_async16(dst, at);
      } else {  // a word that reaches past the logits' ends
#pragma unroll
        for (int e = 0; e < N; ++e)
          if (allowed >> e & 1u) dst[e] = at[e];
      }
    }
    copy_commit();
  };
  // In place, and without masks, only the tokens that change are touched at all.
  const bool staged = MASKED || P.out != P.logits;
  if (staged) {  // (before the lists are there)
#pragma unroll
    for (int s = 0; s < kStages; ++s)
#pragma unroll
      for (int k = 0; k < kBatch; ++k) looked[s][k] = look(r0 + s * kBatch + k);
#pragma unroll
    for (int s = 0; s < kStages; ++s) issue(r0 + s * kBatch, s);
  }

  // ---- the tokens that change
  Penalties pen;
  pen.repetition = P.repetition ? __ldg(P.repetition + b) : 1.f;
  pen.presence = P.presence ? __ldg(P.presence + b) : 0.f;
  pen.frequency = P.frequency ? __ldg(P.frequency + b) : 0.f;
  const int32_t* const counts = P.counts ? P.counts + static_cast<int64_t>(b) * P.V + lo : nullptr;
  uint32_t some = 0;  // of the chunk's columns tid * N ...
  if (counts) {
    if (tid * N + N <= size && reinterpret_cast<uintptr_t>(counts) % 16 == 0) {
#pragma unroll
      for (int q = 0; q < N / 4; ++q) {
        const int4 c = __ldg(reinterpret_cast<const int4*>(counts + tid * N) + q);
        some |= ((c.x != 0 ? 1u : 0u) | (c.y != 0 ? 2u : 0u) | (c.z != 0 ? 4u : 0u) | (c.w != 0 ? 8u : 0u)) << (4 * q);
      }
    } else {
#pragma unroll
      for (int e = 0; e < N; ++e)
        if (tid * N + e < size && __ldg(counts + tid * N + e) != 0) some |= 1u << e;
    }
  }
  if (tid == 0) s_status = 0;
#pragma unroll
  for (int q = 0; q < N / 4; ++q) reinterpret_cast<int4*>(s_value)[tid + q * kThreads] = make_int4(0, 0, 0, 0);
  if (tid < WORDS) s_some[tid] = s_mark[tid] = 0;
  __syncthreads();
  if (some) atomicOr(&s_some[tid * N / 32], some << (tid * N % 32));
  int bad = counted ? 0 : SPECDEC_STATUS_BAD_TOKEN;
  if (!(pen.repetition > 0.f && pen.repetition < kInf && fabsf(pen.presence) < kInf && fabsf(pen.frequency) < kInf))
    bad |= SPECDEC_STATUS_BAD_PENALTY;
  if (P.tokens && counted)
    for (int j = tid; j < gamma; j += kThreads) {
      const int t = __ldg(P.tokens + static_cast<int64_t>(b) * (P.rows - 1) + j);
      s_draft[j] = t;
      if (static_cast<unsigned>(t) >= static_cast<unsigned>(P.V)) {
        bad |= SPECDEC_STATUS_BAD_TOKEN;
      } else if (t >= lo && t - lo < size) {
        atomicOr(&s_some[(t - lo) / 32], 1u << ((t - lo) % 32));
        atomicOr(&s_mark[(t - lo) / 32], 1u << ((t - lo) % 32));
      }
      if (P.parents) {
        const int p = __ldg(P.parents + j);
        s_parent[j] = p;
        if (p < -1 || p >= j) bad |= SPECDEC_STATUS_BAD_TREE;
      }
    }
  const float* const bias_values = P.bias_values + static_cast<int64_t>(b) * P.num_bias;
  for (int k = tid; k < P.num_bias; k += kThreads) {
    const int t = __ldg(P.bias_tokens + static_cast<int64_t>(b) * P.num_bias + k);
    if (t >= P.V) {
      bad |= SPECDEC_STATUS_BAD_TOKEN;
    } else if (t >= lo && t - lo < size) {
      atomicMax(&s_value[t - lo], k + 1);
      atomicOr(&s_some[(t - lo) / 32], 1u << ((t - lo) % 32));
    }
  }
  if (bad) atomicOr(&s_status, bad);
  __syncthreads();
  const int status = s_status;
  if (blockIdx.x == 0 && blockIdx.y == 0 && tid == 0 && P.out_status) P.out_status[b] = status;
  if (status) {  // nothing of the sequence counts
    copy_wait<0>();
    for (int r = r0; r < r1; ++r)
      for (int t = tid; t < size; t += kThreads) to(r)[t] = E::put(__int_as_float(0x7fffffff));
    return;
  }
  some = (s_some[tid * N / 32] >> (tid * N % 32)) & kAll;
  int at = __popc(some);
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int v = __shfl_up_sync(0xffffffffu, at, o);
    if (lane >= o) at += v;
  }
  if (lane == 31) s_sum[tid / 32] = at;
  __syncthreads();
  int listed = 0;
  at -= __popc(some);
#pragma unroll
  for (int w = 0; w < kThreads / 32; ++w) {
    if (w < tid / 32) at += s_sum[w];
    listed += s_sum[w];
  }
  // What is added to a column is the same in all rows, unless the token is some draft's.  An entry says whether the token was there
  // before (kScaled: x is divided, or multiplied), and whether it is a draft's (kOwn: counted anew for each row).
  constexpr int kScaled = 0x8000, kOwn = 0x4000;
  for (; some != 0; some &= some - 1, ++at) {
    const int t = tid * N + __ffs(some) - 1, c = counts ? __ldg(counts + t) : 0, k = s_value[t];
    const bool own = (s_mark[t / 32] >> (t % 32) & 1u) != 0;
    if (!own) s_value[t] = __float_as_int(pen.added(c & 0x7fffffff, k ? __ldg(bias_values + k - 1) : 0.f));
    s_list[at] = static_cast<uint16_t>(t | (c != 0 ? kScaled : 0) | (own ? kOwn : 0));
  }
  // Changes entry j of the list in `rows` rows from r on, x the place of its column 0 in each.
  auto change = [&](int j, int r, int rows, auto&& x) {
    const int entry = s_list[j], t = entry & 0x3fff;
    if (entry & kOwn) {
      const int c = counts ? __ldg(counts + t) : 0, k = s_value[t];
      const float bias = k ? __ldg(bias_values + k - 1) : 0.f;
      for (int i = 0; i < rows; ++i) {
        int n = 0;  // (ends, whatever the parents)
        for (int d = r + i - 1; d >= 0; d = P.parents ? min(s_parent[d], d - 1) : d - 1) n += s_draft[d] == lo + t;
        T* const e = x(i) + t;
        *e = E::put(pen.value(E::get(*e), c != 0 || n > 0, pen.added((c & 0x7fffffff) + n, bias)));
      }
    } else {
      const float add = __int_as_float(s_value[t]);
#pragma unroll
      for (int i = 0; i < kBatch; ++i)
        if (i < rows) {
          T* const e = x(i) + t;
          *e = E::put(pen.value(E::get(*e), (entry & kScaled) != 0, add));
        }
    }
  };
  if (!staged) {
    __syncthreads();
    for (int r = r0; r < r1; r += kBatch)
      for (int j = tid; j < listed; j += kThreads) change(j, r, min(kBatch, r1 - r), [&](int i) { return to(r + i); });
    return;
  }

  int stage = 0;
  for (int r = r0; r < r1; r += kBatch) {
    copy_wait<kStages - 1>();
    __syncthreads();  // everybody's copies, and the list
    for (int j = tid; j < listed; j += kThreads)
      change(j, r, min(kBatch, r1 - r), [&](int i) { return s_rows[stage][i] + past(from(r + i)); });
    __syncthreads();
#pragma unroll
    for (int k = 0; k < kBatch; ++k) {
      if (r + k >= r1) break;
      const T* const words = s_rows[stage][k];
      const int off = past(from(r + k));
      T* const dst = to(r + k);
      uint32_t bits = 0;
#pragma unroll
      for (int s = 0; s < kStages; ++s)
        if (s == stage) bits = looked[s][k];
      if (P.alike) {
        const uint32_t there = bits & kAll, keep = bits >> 8;
        if (there == 0) continue;
        const uint4 in = *reinterpret_cast<const uint4*>(words + tid * N);
        uint32_t w[4] = {in.x, in.y, in.z, in.w};
        if constexpr (MASKED) {
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            const uint32_t two = keep >> (q * E::kPair);
            const uint32_t m = E::kPair == 1 ? 0u - (two & 1u) : ((two & 1u) * 0xffffu) | ((two >> 1 & 1u) * 0xffff0000u);
            w[q] = (w[q] & m) | (E::kNone & ~m);
          }
        }
        T* const word = dst + tid * N - off;
        if (ALIGNED || there == kAll) {
          __stcs(reinterpret_cast<uint4*>(word), make_uint4(w[0], w[1], w[2], w[3]));
        } else {
#pragma unroll
          for (int e = 0; e < N; ++e)
            if (there >> e & 1u) word[e] = static_cast<T>(E::part(w, e));
        }
      } else {
        for (int t = tid; t < size; t += kThreads) dst[t] = !MASKED || bit(r + k, t) ? words[off + t] : E::put(-kInf);
      }
    }
    if (!P.alike) __syncthreads();  // (else a thread's words are its own)
#pragma unroll
    for (int s = 0; s < kStages; ++s)
      if (s == stage) {
#pragma unroll
        for (int k = 0; k < kBatch; ++k) looked[s][k] = look(r + kStages * kBatch + k);
        issue(r + kStages * kBatch, s);
      }
    stage = stage + 1 == kStages ? 0 : stage + 1;
  }
  copy_wait<0>();
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
// (64 prompts of 4095 tokens, V=128256, us: 12.5; 512 threads 12.4, 1024 16.3; chunks of 4096 13.7, of 16384 12.4.)
constexpr int kCountChunk = 8192, kCountThreads = 256;

__global__ void __launch_bounds__(kCountThreads) recount_kernel(const CountParams P) {
  __shared__ __align__(16) int s_count[kCountChunk];
  const int b = blockIdx.y, n = tokens_of(P, b), lo = blockIdx.x * kCountChunk, tid = threadIdx.x;
  const int32_t* const tokens = P.tokens + b * P.token_stride;
  // Whole words of four tokens, and what is before and behind them.  (The first words are on their way before the number of
  // tokens is there: P.n are.)
  constexpr int kFirst = 4;
  const int head = min(P.n, static_cast<int>((16 - reinterpret_cast<uintptr_t>(tokens) % 16) % 16 / 4)), words = (P.n - head) / 4, rest = head + 4 * words;
  int4 first[kFirst];
#pragma unroll
  for (int u = 0; u < kFirst; ++u) {
    const int k = tid + u * kCountThreads;
    first[u] = k < words ? __ldg(reinterpret_cast<const int4*>(tokens + head) + k) : make_int4(-1, -1, -1, -1);
  }
  const int single = tid < head ? tid : tid >= 32 && rest + tid - 32 < P.n ? rest + tid - 32 : -1;
  const int one = single >= 0 ? __ldg(tokens + single) : -1;
#pragma unroll
  for (int k = 0; k < kCountChunk / 4 / kCountThreads; ++k) reinterpret_cast<int4*>(s_count)[tid + k * kCountThreads] = make_int4(0, 0, 0, 0);
  __syncthreads();
  auto take = [&](int k, int t) {  // token number k
    if (k >= n || t < lo || t >= P.V || t - lo >= kCountChunk) return;
    if (P.prompt) s_count[t - lo] = kSign;
    else atomicAdd(&s_count[t - lo], 1);
  };
  auto take4 = [&](int k, const int4& t) {
    take(head + 4 * k, t.x);
    take(head + 4 * k + 1, t.y);
    take(head + 4 * k + 2, t.z);
    take(head + 4 * k + 3, t.w);
  };
  if (single >= 0) take(single, one);
#pragma unroll
  for (int u = 0; u < kFirst; ++u) take4(tid + u * kCountThreads, first[u]);
  for (int k = tid + kFirst * kCountThreads; k < words; k += kCountThreads) take4(k, __ldg(reinterpret_cast<const int4*>(tokens + head) + k));
  __syncthreads();
  int* const out = P.counts + static_cast<int64_t>(b) * P.V + lo;
  const int columns = min(kCountChunk, P.V - lo);
  if (reinterpret_cast<uintptr_t>(out) % 16 == 0 && columns % 4 == 0) {
    for (int k = tid; k < columns / 4; k += kCountThreads) reinterpret_cast<int4*>(out)[k] = reinterpret_cast<const int4*>(s_count)[k];
  } else {
    for (int k = tid; k < columns; k += kCountThreads) out[k] = s_count[k];
  }
  if (blockIdx.x == 0 && P.out_status) report(P, b, n);
}

template <typename T, bool ALIGNED, bool MASKED>
cudaError_t process_shape(ProcessParams P, cudaStream_t stream) {
  constexpr int CHUNK = kChunk<T, ALIGNED>;
  const int64_t chunks = (static_cast<int64_t>(P.V) + CHUNK - 1) / CHUNK;
  // Rows are split over CTAs until there are eight for an SM, four rows at least for each, as a chunk's list is made by every one.  (CTAs for an
  // SM, us: 32 x 65 rows of 32001 under masks 2: 146, 4: 121, 8: 107, 12: 104, 30: 107; 4 x 65 such rows 28.3, 21.4, 23.4, 23.5, 23.4; 256 x 8
  // and 16 x 8 rows of 128256 203 and 21.5 with any.  Rows at least: 2 x 8 rows of 128256 in fp32 2: 10.4, 4: 8.5, 8: 10.5; 1 x 8 in bf16 8.4,
  // 9.4, 12.5; 32 x 65 under masks 107 with any.)
  const int64_t want = 8 * device_sm_count(), have = chunks * P.B;
  const int groups = static_cast<int>(std::min<int64_t>(std::max(1, P.rows / 4), (want + have - 1) / have));
  P.group = (P.rows + groups - 1) / groups;
  const size_t smem = P.tokens ? static_cast<size_t>(P.rows - 1) * 2 * sizeof(int) : 0;
  auto kernel = process_kernel<T, ALIGNED, MASKED>;
  if (cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kMaxProcessRows * 2 * static_cast<int>(sizeof(int))); e != cudaSuccess)
    return e;
  return launch_kernel(kernel, dim3(static_cast<unsigned>(chunks), static_cast<unsigned>((P.rows + P.group - 1) / P.group), static_cast<unsigned>(P.B)),
                       dim3(kThreads), smem, stream, 0, P);
}

template <typename T>
cudaError_t process_typed(const ProcessParams& P, cudaStream_t stream) {
  const bool aligned = P.alike && reinterpret_cast<uintptr_t>(P.logits) % 16 == 0 && static_cast<int64_t>(P.V) * sizeof(T) % 16 == 0;
  if (aligned) return P.mask ? process_shape<T, true, true>(P, stream) : process_shape<T, true, false>(P, stream);
  return P.mask ? process_shape<T, false, true>(P, stream) : process_shape<T, false, false>(P, stream);
}

}  // namespace

cudaError_t launch_process_logits(const ProcessParams& P, specdec_dtype dt, cudaStream_t stream) {
  return dt == SPECDEC_BF16 ? process_typed<uint16_t>(P, stream) : process_typed<float>(P, stream);
}

cudaError_t launch_count_tokens(const CountParams& P, bool reset, cudaStream_t stream) {
  if (reset)
    return launch_kernel(recount_kernel, dim3(static_cast<unsigned>((static_cast<int64_t>(P.V) + kCountChunk - 1) / kCountChunk), static_cast<unsigned>(P.B)),
                         dim3(kCountThreads), 0, stream, 0, P);
  return launch_kernel(count_kernel, dim3(static_cast<unsigned>(std::max(1, (P.n + kThreads - 1) / kThreads)), static_cast<unsigned>(P.B)), dim3(kThreads), 0, stream, 0, P);
}

}  // namespace specdec
