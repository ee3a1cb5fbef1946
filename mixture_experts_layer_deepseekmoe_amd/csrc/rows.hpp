// Rows of the residual stream in the registers of a block: loads and stores of
// eight columns a thread, sums over the block, 8-bit checkpoints.
#pragma once

#include "moe_common.hpp"

namespace moe {

// Eight consecutive values at element offset o of p (f32 or bf16).
struct Raw8 {
  uint4 a, b;
};
template <int FMT>
__device__ __forceinline__ Raw8 load8(const void* p, size_t o) {
  Raw8 r;
  if constexpr (FMT == FMT_F32) {
    const uint4* q = reinterpret_cast<const uint4*>(static_cast<const float*>(p) + o);
    r.a = q[0];
    r.b = q[1];
  } else {
    r.a = *reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(p) + o);
    r.b = make_uint4(0, 0, 0, 0);
  }
  return r;
}
template <int FMT>
__device__ __forceinline__ void values8(const Raw8& r, float (&v)[8]) {
  if constexpr (FMT == FMT_F32) {
    const uint32_t w[8] = {r.a.x, r.a.y, r.a.z, r.a.w, r.b.x, r.b.y, r.b.z, r.b.w};
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] = __uint_as_float(w[e]);
  } else {
    const uint32_t w[4] = {r.a.x, r.a.y, r.a.z, r.a.w};
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      v[2 * e] = __uint_as_float(w[e] << 16);
      v[2 * e + 1] = __uint_as_float(w[e] & 0xffff0000u);
    }
  }
}

__device__ __forceinline__ void load8f(const float* p, size_t o, float (&v)[8]) {
  values8<FMT_F32>(load8<FMT_F32>(p, o), v);
}

// Stores eight values (bf16: rounded to nearest even); v becomes what was stored.
template <int FMT>
__device__ __forceinline__ void store8(void* p, size_t o, float (&v)[8]) {
  if constexpr (FMT == FMT_F32) {
    float4* q = reinterpret_cast<float4*>(static_cast<float*>(p) + o);
    q[0] = make_float4(v[0], v[1], v[2], v[3]);
    q[1] = make_float4(v[4], v[5], v[6], v[7]);
  } else {
    Raw8 r;
    r.a = make_uint4(bf16x2(v[0], v[1]), bf16x2(v[2], v[3]), bf16x2(v[4], v[5]), bf16x2(v[6], v[7]));
    r.b = make_uint4(0, 0, 0, 0);
    *reinterpret_cast<uint4*>(static_cast<uint16_t*>(p) + o) = r.a;
    values8<FMT_BF16>(r, v);
  }
}

// Sum over the block's threads, the same in each of them: a butterfly in the
// wave, then the waves' sums in order.  `red` may be used again after the next
// barrier.
template <int TPB>
__device__ __forceinline__ float block_sum(float v, float (&red)[TPB / 64]) {
#pragma unroll
  for (int off = 32; off >= 1; off >>= 1) v += __shfl_xor(v, off);
  if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = v;
  __syncthreads();
  float s = 0.f;
#pragma unroll
  for (int w = 0; w < TPB / 64; ++w) s += red[w];
  return s;
}

__device__ __forceinline__ float rstd_of(float sumsq, int d, float eps) {
  return 1.0f / sqrtf(sumsq / static_cast<float>(d) + eps);
}

// The 1x128 tile that holds this thread's eight values (16 lanes to a tile):
// scale amax / 448, codes of v * (448 * (1 / amax)): the factor as 32-bit torch
// forms 448 / amax, rounded twice (the layer's own quantisers divide once: codes
// may differ by one there where v falls between two; either way scale * code is
// within the format's half step).  A tile below 2^-119, where
// that factor would overflow, counts as all zero: scale 1, zero codes.  amax is
// taken over the bits, where NaN stands above infinity and infinity above the
// rest (fmaxf would drop a NaN): such a tile has the scale NaN or infinity, and
// the code NaN wherever v * factor is NaN, so all of it is read as NaN.
__device__ __forceinline__ void save_tile(const float (&v)[8], uint8_t* codes, float* scales, size_t row, int d, int c) {
  uint32_t top = 0;
#pragma unroll
  for (int e = 0; e < 8; ++e) top = max(top, __float_as_uint(v[e]) & 0x7fffffffu);
#pragma unroll
  for (int off = 1; off <= 8; off <<= 1) top = max(top, __shfl_xor(top, off));
  const float m = __uint_as_float(top);
  const bool none = m < 0x1p-119f;
  const float inv = none ? 0.f : 448.f * (1.f / m);
  float t[8];
#pragma unroll
  for (int e = 0; e < 8; ++e) t[e] = v[e] * inv;
  uint32_t q[2] = {e4m3x4(t[0], t[1], t[2], t[3]), e4m3x4(t[4], t[5], t[6], t[7])};
  if (top >= 0x7f800000u) {   // e4m3x4 clamps, NaN too
#pragma unroll
    for (int e = 0; e < 8; ++e)
      if (t[e] != t[e]) q[e / 4] = (q[e / 4] & ~(0xffu << 8 * (e % 4))) | 0x7fu << 8 * (e % 4);
  }
  *reinterpret_cast<uint2*>(codes + row * d + c) = make_uint2(q[0], q[1]);
  if ((threadIdx.x & 15) == 0) scales[row * (d / 128) + c / 128] = none ? 1.f : m / 448.f;
}

// f.template operator()<NV, TPB>() with TPB threads x NV vectors of 8 columns
// for rows of d columns.  Few rows (up to 512, two to a CU) are spread over
// as many threads as they fill: a call's time is then its chain of loads.  The
// kernel's time with 1024 threads and with 256, block_out with the next norm / block_in, us:
//   7168 columns    16 rows 4.5, 6.0 / 3.0, 3.6     256 rows 5.7, 6.9 / 3.6, 3.9
//                  512 rows 8.5, 8.9 / 4.6, 4.5     768 rows 13.1, 12.0 / 6.2, 5.3
//   4096 columns   256 rows 4.6, 5.0 / 3.2, 3.3     512 rows 6.1, 6.0 / 4.0, 3.6
//                 1024 rows 10.6, 8.9 / 5.9, 4.4
template <class F>
hipError_t with_row_shape(int T, int d, F&& f) {
  if (d <= 2048) f.template operator()<1, 256>();
  else if (d <= 8192 && T <= 512) f.template operator()<1, 1024>();
  else if (d <= 4096) f.template operator()<2, 256>();
  else if (d <= 8192) f.template operator()<4, 256>();
  else f.template operator()<4, 1024>();
  return hipGetLastError();
}

template <class F>
hipError_t with_fmt(int fmt, F&& f) {   // f32 or bf16
  return fmt == FMT_F32 ? f.template operator()<FMT_F32>() : f.template operator()<FMT_BF16>();
}

}  // namespace moe
