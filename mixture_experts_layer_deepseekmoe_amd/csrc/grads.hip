// The global norm of many gradient tensors and clipping by it:
//
//   sumsq = sum over all elements g^2,  norm = sqrt(sumsq)
//   out = g min(1, max_norm / norm)     (sumsq not finite: out = g)
//
// Bound by HBM.  The tensors' pointers and sizes are launch arguments (112 to a
// launch); blocks take chunks of 4096 elements, whatever tensor they are of.
// Squares and their sums are in 64 bits (nothing overflows or is lost: the card's
// 64-bit rate is 30 times what HBM delivers), in a fixed order; an element is
// scaled in 64 bits and rounded to fp32 (from there to bf16).  Clipping goes through
// the chunks from the last to the first, so it begins with what the caches still
// hold, and does nothing in place where nothing is to be clipped.
//
// Measured, 571M fp32 elements: the sum 362 us (6.3 TB/s; chunks of 8192, more
// registers and fewer waves: 449), clipping into other tensors 727 us (6.3 TB/s; with
// 4096 blocks in turns 793, with 2048 and without the streaming hints 890).
#include "ends.hpp"

namespace moe {

namespace {

constexpr int THREADS = 256;

// 16 bytes at any element's address: four values of fp32, eight of bf16.
typedef float f32x4_any __attribute__((ext_vector_type(4), aligned(4)));
typedef uint32_t u32x4_any __attribute__((ext_vector_type(4), aligned(2)));
typedef uint32_t u32x2_any __attribute__((ext_vector_type(2), aligned(2)));

template <bool BF16>
struct Vec {
  static constexpr int N = BF16 ? 8 : 4, PER = GRAD_CHUNK / (THREADS * N);
  uint32_t w[4];

  // elements i .. of a tensor of n: zeros past its end.  LAST: with the streaming hint
  template <bool LAST>
  __device__ __forceinline__ void load(const void* p, long long i, long long n) {
    w[0] = w[1] = w[2] = w[3] = 0;
    if (i + N <= n) {
      const u32x4_any* q = reinterpret_cast<const u32x4_any*>(static_cast<const uint8_t*>(p) + i * (BF16 ? 2 : 4));
      u32x4_any v;
      if constexpr (LAST)
        v = __builtin_nontemporal_load(q);
      else
        v = *q;
#pragma unroll
      for (int e = 0; e < 4; ++e) w[e] = v[e];
    } else if (i < n) {
#pragma unroll
      for (int e = 0; e < N - 1; ++e) {
        if (i + e >= n) continue;
        if constexpr (BF16)
          w[e / 2] |= static_cast<uint32_t>(static_cast<const uint16_t*>(p)[i + e]) << 16 * (e % 2);
        else
          w[e] = static_cast<const uint32_t*>(p)[i + e];
      }
    }
  }
  __device__ __forceinline__ float value(int e) const {
    if constexpr (BF16) return __uint_as_float(e % 2 ? w[e / 2] & 0xffff0000u : w[e / 2] << 16);
    return __uint_as_float(w[e]);
  }
};

// Stores N values from element i on, as far as the tensor's n go.
template <int N>
__device__ __forceinline__ void store(void* o, long long i, long long n, bool bf16, const float (&v)[N]) {
  uint32_t h[N / 2];
#pragma unroll
  for (int e = 0; e < N / 2; ++e) h[e] = bf16x2(v[2 * e], v[2 * e + 1]);
  if (i + N <= n) {
    if (!bf16) {
      f32x4_any* q = reinterpret_cast<f32x4_any*>(static_cast<float*>(o) + i);
#pragma unroll
      for (int e = 0; e < N / 4; ++e)
        __builtin_nontemporal_store(f32x4_any{v[4 * e], v[4 * e + 1], v[4 * e + 2], v[4 * e + 3]}, q + e);
    } else if constexpr (N == 8) {
      *reinterpret_cast<u32x4_any*>(static_cast<uint16_t*>(o) + i) = u32x4_any{h[0], h[1], h[2], h[3]};
    } else {
      *reinterpret_cast<u32x2_any*>(static_cast<uint16_t*>(o) + i) = u32x2_any{h[0], h[1]};
    }
    return;
  }
#pragma unroll
  for (int e = 0; e < N - 1; ++e) {   // the tensor's last, in part
    if (i + e >= n) continue;
    if (bf16)
      static_cast<uint16_t*>(o)[i + e] = static_cast<uint16_t>(e % 2 ? h[e / 2] >> 16 : h[e / 2]);
    else
      static_cast<float*>(o)[i + e] = v[e];
  }
}

// The tensor that chunk c is of: the last whose chunks begin at or before c.
__device__ __forceinline__ int tensor_of(const GradArgs& a, uint32_t c) {
  int lo = 0, hi = a.n - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) / 2;
    if (a.first[mid] <= c) lo = mid; else hi = mid - 1;
  }
  return lo;
}

__device__ __forceinline__ double block_sum(double v, double* red) {
#pragma unroll
  for (int off = 32; off >= 1; off >>= 1) v += __shfl_xor(v, off);
  if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = v;
  __syncthreads();
  double s = 0.0;
  for (unsigned w = 0; w < blockDim.x / 64; ++w) s += red[w];
  return s;
}

template <bool BF16>
__device__ __forceinline__ double chunk_sumsq(const void* p, long long i0, long long n, double sum) {
  using V = Vec<BF16>;
  V r[V::PER];
#pragma unroll
  for (int j = 0; j < V::PER; ++j) r[j].template load<false>(p, i0 + V::N * (threadIdx.x + THREADS * j), n);
#pragma unroll
  for (int j = 0; j < V::PER; ++j)
#pragma unroll
    for (int e = 0; e < V::N; ++e) sum = fma(static_cast<double>(r[j].value(e)), static_cast<double>(r[j].value(e)), sum);
  return sum;
}

__global__ __launch_bounds__(THREADS) void grad_sumsq_kernel(GradArgs a, double* part) {
  __shared__ double red[THREADS / 64];
  double sum = 0.0;
  for (uint32_t c = blockIdx.x; c < a.first[a.n]; c += gridDim.x) {
    const int k = tensor_of(a, c);
    if (!MOE_CHECK(c >= a.first[k] && c < a.first[k + 1], 1001)) continue;
    const long long i0 = static_cast<long long>(c - a.first[k]) * GRAD_CHUNK;
    if (a.bf16[k] & 1)
      sum = chunk_sumsq<true>(a.data[k], i0, a.numel[k], sum);
    else
      sum = chunk_sumsq<false>(a.data[k], i0, a.numel[k], sum);
  }
  sum = block_sum(sum, red);
  if (threadIdx.x == 0) part[blockIdx.x] = sum;
}

__global__ __launch_bounds__(1024) void grad_finish_kernel(const double* part, long long n, double* sumsq) {
  __shared__ double red[16];
  double sum = 0.0;
  for (long long i = threadIdx.x; i < n; i += 1024) sum += part[i];
  sum = block_sum(sum, red);
  if (threadIdx.x == 0) *sumsq = sum;
}

template <bool BF16>
__device__ __forceinline__ void chunk_scale(const void* p, void* o, long long i0, long long n, bool out_bf16, double f) {
  using V = Vec<BF16>;
  V r[V::PER];
#pragma unroll
  for (int j = 0; j < V::PER; ++j) r[j].template load<true>(p, i0 + V::N * (threadIdx.x + THREADS * j), n);
#pragma unroll
  for (int j = 0; j < V::PER; ++j) {
    float v[V::N];
#pragma unroll
    for (int e = 0; e < V::N; ++e) v[e] = static_cast<float>(static_cast<double>(r[j].value(e)) * f);
    store<V::N>(o, i0 + V::N * (threadIdx.x + THREADS * j), n, out_bf16, v);
  }
}

__global__ __launch_bounds__(THREADS) void grad_clip_kernel(GradArgs a, const double* sumsq, double max_norm, float* norm) {
  const double s = sqrt(*sumsq);
  if (norm != nullptr && blockIdx.x == 0 && threadIdx.x == 0) *norm = static_cast<float>(s);
  const bool clip = s > max_norm && s < __builtin_inf();
  const double f = clip ? max_norm / s : 1.0;
  const uint32_t total = a.first[a.n];
  for (uint32_t d = blockIdx.x; d < total; d += gridDim.x) {
    const uint32_t c = total - 1 - d;
    const int k = tensor_of(a, c);
    if (!MOE_CHECK(c >= a.first[k] && c < a.first[k + 1], 1002)) continue;
    const void* p = a.data[k];
    if (!clip && p == a.out[k]) continue;
    const long long i0 = static_cast<long long>(c - a.first[k]) * GRAD_CHUNK;
    if (a.bf16[k] & 1)
      chunk_scale<true>(p, a.out[k], i0, a.numel[k], a.bf16[k] & 2, f);
    else
      chunk_scale<false>(p, a.out[k], i0, a.numel[k], a.bf16[k] & 2, f);
  }
}

}  // namespace

MOE_DEBUG_FILE(grads)

hipError_t launch_grad_sumsq(const GradArgs& a, double* part, hipStream_t s) {
  if (grad_blocks(a) > 0) hipLaunchKernelGGL(grad_sumsq_kernel, dim3(grad_blocks(a)), dim3(THREADS), 0, s, a, part);
  return hipGetLastError();
}

hipError_t launch_grad_finish(const double* part, long long n, double* sumsq, hipStream_t s) {
  hipLaunchKernelGGL(grad_finish_kernel, dim3(1), dim3(1024), 0, s, part, n, sumsq);
  return hipGetLastError();
}

hipError_t launch_grad_clip(const GradArgs& a, const double* sumsq, double max_norm, float* norm, hipStream_t s) {
  constexpr uint32_t MOST = 1 << 22;
  const uint32_t n = a.first[a.n], blocks = n < 1 ? 1 : n < MOST ? n : MOST;   // one writes the norm
  hipLaunchKernelGGL(grad_clip_kernel, dim3(blocks), dim3(THREADS), 0, s, a, sumsq, max_norm, norm);
  return hipGetLastError();
}

}  // namespace moe
