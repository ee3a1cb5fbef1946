// The global norm of many gradient tensors and clipping by it:
//
//   sumsq = sum over all elements g^2,  norm = sqrt(sumsq)
//   out = g min(1, max_norm / norm)     (sumsq not finite: out = g)
//
// Bound by HBM.  The tensors' pointers and sizes are launch arguments (112 to a
// launch); blocks take chunks of 8192 elements in turn, whatever tensor they are of.
// Squares and their sums are in 64 bits (nothing overflows or is lost: the card's
// 64-bit rate is 30 times what HBM delivers), in a fixed order; an element is
// scaled in 64 bits and rounded to fp32 (from there to bf16).  Clipping goes through the chunks from the
// last to the first, so it begins with what the caches still hold, and does nothing
// in place where nothing is to be clipped.
#include "ends.hpp"

namespace moe {

namespace {

constexpr int THREADS = 256, VEC = 8, PER = GRAD_CHUNK / (THREADS * VEC);

// The accesses of eight values at any element's address.
typedef float f32x4_any __attribute__((ext_vector_type(4), aligned(4)));
typedef uint32_t u32x4_any __attribute__((ext_vector_type(4), aligned(2)));

struct Raw {
  f32x4_any a, b;
};
__device__ __forceinline__ void load_vec(const void* p, long long i, bool bf16, Raw& r) {
  if (bf16) {
    r.a = __builtin_bit_cast(f32x4_any, *reinterpret_cast<const u32x4_any*>(static_cast<const uint16_t*>(p) + i));
  } else {
    const f32x4_any* q = reinterpret_cast<const f32x4_any*>(static_cast<const float*>(p) + i);
    r.a = q[0];
    r.b = q[1];
  }
}
__device__ __forceinline__ void values(const Raw& r, bool bf16, float (&v)[VEC]) {
#pragma unroll
  for (int e = 0; e < VEC; ++e) {
    if (bf16) {
      const uint32_t w = __float_as_uint(r.a[e / 2]);
      v[e] = __uint_as_float(e % 2 ? w & 0xffff0000u : w << 16);
    } else {
      v[e] = e < 4 ? r.a[e % 4] : r.b[e % 4];
    }
  }
}
__device__ __forceinline__ float load_one(const void* p, long long i, bool bf16) {
  return bf16 ? __uint_as_float(static_cast<uint32_t>(static_cast<const uint16_t*>(p)[i]) << 16)
              : static_cast<const float*>(p)[i];
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

__global__ __launch_bounds__(THREADS) void grad_sumsq_kernel(GradArgs a, double* part) {
  __shared__ double red[THREADS / 64];
  double sum = 0.0;
  for (uint32_t c = blockIdx.x; c < a.first[a.n]; c += gridDim.x) {
    const int k = tensor_of(a, c);
    if (!MOE_CHECK(c >= a.first[k] && c < a.first[k + 1], 1001)) continue;
    const bool bf16 = a.bf16[k] & 1;
    const long long i0 = static_cast<long long>(c - a.first[k]) * GRAD_CHUNK, n = a.numel[k];
    const void* p = a.data[k];
    if (i0 + GRAD_CHUNK <= n) {
      Raw r[PER];
#pragma unroll
      for (int j = 0; j < PER; ++j) load_vec(p, i0 + VEC * (threadIdx.x + THREADS * j), bf16, r[j]);
#pragma unroll
      for (int j = 0; j < PER; ++j) {
        float v[VEC];
        values(r[j], bf16, v);
#pragma unroll
        for (int e = 0; e < VEC; ++e) sum = fma(static_cast<double>(v[e]), static_cast<double>(v[e]), sum);
      }
    } else {
      for (long long i = i0 + threadIdx.x; i < n; i += THREADS) {
        const double v = load_one(p, i, bf16);
        sum = fma(v, v, sum);
      }
    }
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
    void* o = a.out[k];
    if (!clip && p == o) continue;
    const bool bf16 = a.bf16[k] & 1, obf16 = a.bf16[k] & 2;
    const long long i0 = static_cast<long long>(c - a.first[k]) * GRAD_CHUNK, n = a.numel[k];
    if (i0 + GRAD_CHUNK <= n) {
      Raw r[PER];
#pragma unroll
      for (int j = 0; j < PER; ++j) load_vec(p, i0 + VEC * (threadIdx.x + THREADS * j), bf16, r[j]);
#pragma unroll
      for (int j = 0; j < PER; ++j) {
        float v[VEC];
        values(r[j], bf16, v);
#pragma unroll
        for (int e = 0; e < VEC; ++e) v[e] = static_cast<float>(static_cast<double>(v[e]) * f);
        const long long i = i0 + VEC * (threadIdx.x + THREADS * j);
        if (obf16) {
          *reinterpret_cast<u32x4_any*>(static_cast<uint16_t*>(o) + i) =
              u32x4_any{bf16x2(v[0], v[1]), bf16x2(v[2], v[3]), bf16x2(v[4], v[5]), bf16x2(v[6], v[7])};
        } else {
          f32x4_any* q = reinterpret_cast<f32x4_any*>(static_cast<float*>(o) + i);
          q[0] = f32x4_any{v[0], v[1], v[2], v[3]};
          q[1] = f32x4_any{v[4], v[5], v[6], v[7]};
        }
      }
    } else {
      for (long long i = i0 + threadIdx.x; i < n; i += THREADS) {
        const float v = static_cast<float>(static_cast<double>(load_one(p, i, bf16)) * f);
        if (obf16)
          static_cast<uint16_t*>(o)[i] = static_cast<uint16_t>(bf16x2(v, 0.f));
        else
          static_cast<float*>(o)[i] = v;
      }
    }
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
  const int blocks = grad_blocks(a) > 0 ? grad_blocks(a) : 1;   // one writes the norm
  hipLaunchKernelGGL(grad_clip_kernel, dim3(blocks), dim3(THREADS), 0, s, a, sumsq, max_norm, norm);
  return hipGetLastError();
}

}  // namespace moe
