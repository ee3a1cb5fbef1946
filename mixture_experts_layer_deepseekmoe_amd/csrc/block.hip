// The norms before and after a block, with its gate and residual scale:
//
//   block_in   n = x r w,  r = (mean_c x^2 + eps)^(-1/2)
//   block_out  z = y - skip,  x' = beta x + gate zh w,  zh = z r  (r = 1 and
//              w = 1 without a norm), then optionally the next block's norm of
//              x' as stored
//   backward   of v r w for the upstream g:  a = g w,  vh = v r,
//              dv = r (a - vh mean_c(a vh)),  dw = sum_t g vh
//              (block_in: g = dn - dn_sub, v = x; block_out: g = dout gate,
//              v = z, and dgate = w sum over the gate's rows of dout zh)
//
// With a checkpoint, v is also kept as E4M3 codes with one fp32 scale per
// 1x128 tile (read as the framework's other 1x128 tiles are), and the backward reads
// codes * scale instead of the rows: 1.03 bytes per value instead of 2 (x) or
// 6 (an fp32 y and a bf16 skip).  r stays that of the exact rows.
//
// All of it is bound by HBM: each value is loaded once into registers, where
// its row stays between the row's sum and its use, and each result is stored
// once.  (But for the backward above 8192 columns: its values, gate w and sums of
// 32 columns to a thread do not fit the 128 registers that 1024 threads leave it,
// and about 1 KB a thread goes through scratch for each row.  2048 rows of 8192
// columns: 46 us; of 8200: 303, of 16384: 408.)  Measured at 8192 x 7168 (a 1 GiB
// copy runs at 5.1 TB/s): block_in with a checkpoint 56 us (5.2 TB/s), block_out
// with one and the next norm 156 us (4.9 TB/s), their backward 214 us (4.7) and 110
// us (4.9).  A block takes whole rows, 8 consecutive columns to a thread (16-byte
// loads of bf16, 16 lanes to a 128-column tile).  Statistics and sums are fp32
// throughout, in a fixed order; outputs in bf16 are rounded once, at the store.
#include "around.hpp"
#include "rows.hpp"

namespace moe {

namespace {

__device__ __forceinline__ void decode8(const uint2 q, float s, float (&v)[8]) {
  const auto a = __builtin_amdgcn_cvt_pk_f32_fp8(q.x, false), b = __builtin_amdgcn_cvt_pk_f32_fp8(q.x, true);
  const auto c = __builtin_amdgcn_cvt_pk_f32_fp8(q.y, false), e = __builtin_amdgcn_cvt_pk_f32_fp8(q.y, true);
  v[0] = a[0] * s; v[1] = a[1] * s; v[2] = b[0] * s; v[3] = b[1] * s;
  v[4] = c[0] * s; v[5] = c[1] * s; v[6] = e[0] * s; v[7] = e[1] * s;
}

// ------------------------------------------------------------------ forward

template <int XF, int NF, int NV, int TPB>
__global__ __launch_bounds__(TPB) void block_in_kernel(BlockInArgs a) {
  __shared__ float red[TPB / 64];
  const size_t row = blockIdx.x;
  if (!MOE_CHECK(row < static_cast<size_t>(a.T) && a.d <= 8 * TPB * NV, 605)) return;
  float x[NV][8];
  Raw8 raw[NV];
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int c = 8 * (threadIdx.x + TPB * i);
    if (c < a.d) raw[i] = load8<XF>(a.x, row * a.d + c);
  }
  float ss = 0.f;
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int c = 8 * (threadIdx.x + TPB * i);
    if (c >= a.d) continue;
    values8<XF>(raw[i], x[i]);
#pragma unroll
    for (int e = 0; e < 8; ++e) ss = fmaf(x[i][e], x[i][e], ss);
  }
  const float r = rstd_of(block_sum<TPB>(ss, red), a.d, a.eps);
  if (a.rstd != nullptr && threadIdx.x == 0) a.rstd[row] = r;
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int c = 8 * (threadIdx.x + TPB * i);
    if (c >= a.d) continue;
    if (a.codes != nullptr) save_tile(x[i], a.codes, a.scales, row, a.d, c);
    float w[8];
    load8f(a.w, c, w);
#pragma unroll
    for (int e = 0; e < 8; ++e) w[e] *= x[i][e] * r;
    store8<NF>(a.n, row * a.d + c, w);
  }
}

template <int XF, int NF, int YF, int NV, int TPB>
__global__ __launch_bounds__(TPB) void block_out_kernel(BlockOutArgs a) {
  __shared__ float red[2][TPB / 64];
  const size_t row = blockIdx.x;
  Raw8 ry[NV], rs[NV], rx[NV];
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int c = 8 * (threadIdx.x + TPB * i);
    if (c >= a.d) continue;
    ry[i] = load8<YF>(a.y, row * a.d + c);
    if (a.skip != nullptr) rs[i] = load8<NF>(a.skip, row * a.d + c);
    rx[i] = load8<XF>(a.x, row * a.d + c);
  }
  float z[NV][8];
  float ss = 0.f;
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int c = 8 * (threadIdx.x + TPB * i);
    if (c >= a.d) continue;
    values8<YF>(ry[i], z[i]);
    if (a.skip != nullptr) {
      float s[8];
      values8<NF>(rs[i], s);
#pragma unroll
      for (int e = 0; e < 8; ++e) z[i][e] -= s[e];
    }
#pragma unroll
    for (int e = 0; e < 8; ++e) ss = fmaf(z[i][e], z[i][e], ss);
  }
  float r = 1.f;
  if (a.w != nullptr) {
    r = rstd_of(block_sum<TPB>(ss, red[0]), a.d, a.eps);
    if (a.rstd != nullptr && threadIdx.x == 0) a.rstd[row] = r;
  }
  const size_t grow = a.gate != nullptr && a.gate_rows > 0 ? row / a.gate_rows : 0;
  if (!MOE_CHECK(row < static_cast<size_t>(a.T) && (a.gate == nullptr || grow < static_cast<size_t>(a.gates)), 601)) return;
  ss = 0.f;
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int c = 8 * (threadIdx.x + TPB * i);
    if (c >= a.d) continue;
    if (a.codes != nullptr) save_tile(z[i], a.codes, a.scales, row, a.d, c);
    float x[8], t[8];
    if (a.w != nullptr) {
      load8f(a.w, c, t);
#pragma unroll
      for (int e = 0; e < 8; ++e) z[i][e] *= r * t[e];
    }
    if (a.gate != nullptr) {
      load8f(a.gate, grow * a.d + c, t);
#pragma unroll
      for (int e = 0; e < 8; ++e) z[i][e] *= t[e];
    }
    values8<XF>(rx[i], x);
#pragma unroll
    for (int e = 0; e < 8; ++e) z[i][e] = fmaf(a.res_scale, x[e], z[i][e]);
    store8<XF>(a.x_out, row * a.d + c, z[i]);   // z: x' as stored
#pragma unroll
    for (int e = 0; e < 8; ++e) ss = fmaf(z[i][e], z[i][e], ss);
  }
  if (a.w_next == nullptr) return;
  r = rstd_of(block_sum<TPB>(ss, red[1]), a.d, a.eps);
  if (a.rstd_next != nullptr && threadIdx.x == 0) a.rstd_next[row] = r;
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int c = 8 * (threadIdx.x + TPB * i);
    if (c >= a.d) continue;
    if (a.codes_next != nullptr) save_tile(z[i], a.codes_next, a.scales_next, row, a.d, c);
    float w[8];
    load8f(a.w_next, c, w);
#pragma unroll
    for (int e = 0; e < 8; ++e) w[e] *= z[i][e] * r;
    store8<NF>(a.n_next, row * a.d + c, w);
  }
}

// ------------------------------------------------------------------ backward

// Block b's rows.  Gate rows of at most a.rows rows (whole gates to a block):
// the block finishes their dgate itself and leaves sum g vh.  Longer ones are
// cut into runs of a.rows, none across a gate, and the block leaves sum dout vh
// of its run for the kernels below.
struct BwdRows {
  long long t0, t1;
};
__device__ __forceinline__ BwdRows bwd_rows(const BlockBwdArgs& a) {
  const long long L = a.gate_len, b = blockIdx.x;
  if (a.whole_gates) {
    const long long n = L * (a.rows / L);
    return {b * n, min(b * n + n, static_cast<long long>(a.T))};
  }
  const long long g = b / a.runs, j = b - g * a.runs;
  const long long t0 = g * L + j * a.rows;
  const long long t1 = min(min(t0 + a.rows, (g + 1) * L), static_cast<long long>(a.T));
  return {t0, t1};
}

// VF: the rows v: FMT_F32 / FMT_BF16 (less `skip`, of format SF, where given) or
// FMT_E4M3 codes.  gate w, the same for all rows of a gate, stays in registers.
template <int VF, int SF, int NV, int TPB>
__global__ __launch_bounds__(TPB) void block_bwd_kernel(BlockBwdArgs a) {
  __shared__ float red[2][TPB / 64];
  const BwdRows rows = bwd_rows(a);
  if (!MOE_CHECK(blockIdx.x < a.blocks && rows.t0 >= 0 && rows.t1 <= a.T, 602)) return;
  float acc[NV][8], gacc[NV][8], gw[NV][8];
#pragma unroll
  for (int i = 0; i < NV; ++i)
#pragma unroll
    for (int e = 0; e < 8; ++e) acc[i][e] = gacc[i][e] = 0.f;

  for (long long t = rows.t0; t < rows.t1; ++t) {
    const size_t row = static_cast<size_t>(t), ro = row * a.d;
    const size_t gro = a.gate != nullptr ? row / a.gate_len * a.d : 0;
    if (!MOE_CHECK(a.gate == nullptr || t / a.gate_len < a.gates, 603)) return;
    const bool first = t == rows.t0 || (a.whole_gates && t % a.gate_len == 0);   // of its gate, here
    const float r = a.w != nullptr ? a.rstd[row] : 1.f;
    Raw8 rg[NV], rs[NV], rv[NV], rk[NV], rr[NV];
    float sc[NV];
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int c = 8 * (threadIdx.x + TPB * i);
      if (c >= a.d) continue;
      rg[i] = load8<FMT_F32>(a.g, ro + c);
      if (a.g_sub != nullptr) rs[i] = load8<FMT_F32>(a.g_sub, ro + c);
      if (a.res != nullptr) rr[i] = load8<FMT_F32>(a.res, ro + c);
      if constexpr (VF == FMT_E4M3) {
        const uint2 q = *reinterpret_cast<const uint2*>(a.codes + ro + c);
        rv[i].a = make_uint4(q.x, q.y, 0, 0);
        sc[i] = a.scales[row * (a.d / 128) + c / 128];
      } else if (a.v != nullptr) {   // null: neither norm nor gate
        rv[i] = load8<VF>(a.v, ro + c);
        if (a.skip != nullptr) rk[i] = load8<SF>(a.skip, ro + c);
      }
    }
    float g[NV][8], v[NV][8], dot = 0.f;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int c = 8 * (threadIdx.x + TPB * i);
      if (c >= a.d) continue;
      float f[8];
      if (first) {
#pragma unroll
        for (int e = 0; e < 8; ++e) gw[i][e] = 1.f;
        if (a.w != nullptr) load8f(a.w, c, gw[i]);
        if (a.gate != nullptr) {
          load8f(a.gate, gro + c, f);
#pragma unroll
          for (int e = 0; e < 8; ++e) gw[i][e] *= f[e];
        }
      }
      values8<FMT_F32>(rg[i], g[i]);
      if (a.g_sub != nullptr) {
        values8<FMT_F32>(rs[i], f);
#pragma unroll
        for (int e = 0; e < 8; ++e) g[i][e] -= f[e];
      }
      if constexpr (VF == FMT_E4M3) {
        decode8(make_uint2(rv[i].a.x, rv[i].a.y), sc[i], v[i]);
      } else if (a.v != nullptr) {
        values8<VF>(rv[i], v[i]);
        if (a.skip != nullptr) {
          values8<SF>(rk[i], f);
#pragma unroll
          for (int e = 0; e < 8; ++e) v[i][e] -= f[e];
        }
      } else {
#pragma unroll
        for (int e = 0; e < 8; ++e) v[i][e] = 0.f;
      }
      // v: vh; gacc += g vh; g: a
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        v[i][e] *= r;
        gacc[i][e] = fmaf(g[i][e], v[i][e], gacc[i][e]);
        g[i][e] *= gw[i][e];
        dot = fmaf(g[i][e], v[i][e], dot);
      }
      // the row ends its gate (whole gates): gate gacc joins acc, w gacc is dgate
      if (a.whole_gates && (t + 1 == rows.t1 || (t + 1) % a.gate_len == 0)) {
        load8f(a.gate, gro + c, f);
#pragma unroll
        for (int e = 0; e < 8; ++e) acc[i][e] = fmaf(f[e], gacc[i][e], acc[i][e]);
        if (a.w != nullptr) {
          load8f(a.w, c, f);
#pragma unroll
          for (int e = 0; e < 8; ++e) gacc[i][e] *= f[e];
        }
        if (a.dgate != nullptr) store8<FMT_F32>(a.dgate, gro + c, gacc[i]);
#pragma unroll
        for (int e = 0; e < 8; ++e) gacc[i][e] = 0.f;
      }
    }
    const float mean = a.w != nullptr ? block_sum<TPB>(dot, red[t & 1]) / static_cast<float>(a.d) : 0.f;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int c = 8 * (threadIdx.x + TPB * i);
      if (c >= a.d) continue;
      if (a.w != nullptr) {
#pragma unroll
        for (int e = 0; e < 8; ++e) g[i][e] = r * (g[i][e] - v[i][e] * mean);
      }
      if (a.res != nullptr) {
        float s[8];
        values8<FMT_F32>(rr[i], s);
#pragma unroll
        for (int e = 0; e < 8; ++e) g[i][e] = fmaf(a.res_scale, s[e], g[i][e]);
      }
      store8<FMT_F32>(a.dv, ro + c, g[i]);
    }
  }
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int c = 8 * (threadIdx.x + TPB * i);
    if (c < a.d) store8<FMT_F32>(a.part, static_cast<size_t>(blockIdx.x) * a.d + c, a.whole_gates ? acc[i] : gacc[i]);
  }
}

// Column sums of the blocks' rows in a fixed order: 16 threads x 4 columns, 64 row
// lanes (row lane l takes rows l, l + 64, ...); a wave's four row lanes are joined
// by a butterfly, the 16 waves in order.  Block (x, y): columns 64 x .., gates y
// n_gates .. of n rows each; per gate g
//   s_g -> dgate[g] = w s_g,  and gate[g] s_g, summed over the block's gates into
//   out[y]  (dw, or with one gate to a block its summands)
struct ColSumArgs {
  const float* part;
  int n, d, n_gates;
  const float* w;      // nullable: ones
  const float* gate;   // nullable: ones
  float* dgate;        // nullable
  float* out;          // nullable
  long long rows, gates;   // rows of part and of gate from here on (the debug build's checks)
};
constexpr int CS_LANES = 64;
constexpr int CS_GATES = 8;   // up to so many gates are summed by one launch
__global__ __launch_bounds__(1024) void block_colsum_kernel(ColSumArgs a) {
  __shared__ float4 s[CS_GATES][16][16];
  const int tc = threadIdx.x & 15, l = threadIdx.x >> 4, w = threadIdx.x >> 6;
  const int c = 64 * blockIdx.x + 4 * tc;
  const size_t g0 = static_cast<size_t>(blockIdx.y) * a.n_gates;
  if (!MOE_CHECK(a.n_gates <= CS_GATES && (g0 + a.n_gates) * a.n <= static_cast<size_t>(a.rows) &&
                     ((a.gate == nullptr && a.dgate == nullptr) || g0 + a.n_gates <= static_cast<size_t>(a.gates)),
                 604))
    return;
  for (int k = 0; k < a.n_gates; ++k) {
    float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
    if (c < a.d) {
      const float* p = a.part + (g0 + k) * a.n * a.d + c;
#pragma unroll 4
      for (int r = l; r < a.n; r += CS_LANES) {
        const float4 x = *reinterpret_cast<const float4*>(p + static_cast<size_t>(r) * a.d);
        v.x += x.x; v.y += x.y; v.z += x.z; v.w += x.w;
      }
    }
#pragma unroll
    for (int off = 16; off <= 32; off <<= 1) {
      v.x += __shfl_xor(v.x, off);
      v.y += __shfl_xor(v.y, off);
      v.z += __shfl_xor(v.z, off);
      v.w += __shfl_xor(v.w, off);
    }
    if ((l & 3) == 0) s[k][w][tc] = v;
  }
  __syncthreads();
  // one column to a thread
  const int col = 64 * blockIdx.x + threadIdx.x;
  if (threadIdx.x >= 64 || col >= a.d) return;
  float dw = 0.f;
  for (int k = 0; k < a.n_gates; ++k) {
    const float* cs = reinterpret_cast<const float*>(&s[k][0][0]) + threadIdx.x;
    float sum = 0.f;
#pragma unroll
    for (int i = 0; i < 16; ++i) sum += cs[i * 64];
    const size_t o = (g0 + k) * a.d + col;
    if (a.dgate != nullptr) a.dgate[o] = a.w != nullptr ? a.w[col] * sum : sum;
    dw = fmaf(a.gate != nullptr ? a.gate[o] : 1.f, sum, dw);
  }
  if (a.out != nullptr) a.out[static_cast<size_t>(blockIdx.y) * a.d + col] = dw;
}

// with_row_shape (rows.hpp) for the backward, whose blocks take several rows in turn: 1024
// threads for up to 8192 columns (block_out forward + backward at 8192 x 7168: 271
// us, with 512 threads 281, with 256 threads x 4 vectors 356; taking 2 or 4 rows
// at once changed nothing).
template <class F>
hipError_t with_bwd_shape(int d, F&& f) {
  if (d <= 2048) f.template operator()<1, 256>();
  else if (d <= 4096) f.template operator()<1, 512>();
  else if (d <= 8192) f.template operator()<1, 1024>();
  else f.template operator()<4, 1024>();
  return hipGetLastError();
}

}  // namespace

MOE_DEBUG_FILE(block)

hipError_t launch_block_in(const BlockInArgs& a, hipStream_t s) {
  if (a.T == 0) return hipSuccess;
  return with_fmt(a.x_fmt, [&]<int XF>() {
    return with_fmt(a.n_fmt, [&]<int NF>() {
      return with_row_shape(a.T, a.d, [&]<int NV, int TPB>() {
        hipLaunchKernelGGL((block_in_kernel<XF, NF, NV, TPB>), dim3(a.T), dim3(TPB), 0, s, a);
      });
    });
  });
}

hipError_t launch_block_out(const BlockOutArgs& a, hipStream_t s) {
  if (a.T == 0) return hipSuccess;
  return with_fmt(a.x_fmt, [&]<int XF>() {
    return with_fmt(a.n_fmt, [&]<int NF>() {
      return with_fmt(a.y_fmt, [&]<int YF>() {
        return with_row_shape(a.T, a.d, [&]<int NV, int TPB>() {
          hipLaunchKernelGGL((block_out_kernel<XF, NF, YF, NV, TPB>), dim3(a.T), dim3(TPB), 0, s, a);
        });
      });
    });
  });
}

hipError_t launch_block_bwd(BlockBwdArgs a, hipStream_t s) {
  const BlockBwdPlan p = block_bwd_plan(a.T, a.gate_len, a.gates, a.gate != nullptr);
  a.whole_gates = p.whole_gates;
  a.runs = p.runs;
  a.rows = p.rows;
  a.blocks = p.blocks;
  if (p.blocks > 0) {
    const dim3 grid(static_cast<unsigned>(p.blocks));
    hipError_t e = with_bwd_shape(a.d, [&]<int NV, int TPB>() {
      if (a.codes != nullptr)
        hipLaunchKernelGGL((block_bwd_kernel<FMT_E4M3, FMT_F32, NV, TPB>), grid, dim3(TPB), 0, s, a);
      else if (a.v_fmt == FMT_F32 && a.skip_fmt == FMT_F32)
        hipLaunchKernelGGL((block_bwd_kernel<FMT_F32, FMT_F32, NV, TPB>), grid, dim3(TPB), 0, s, a);
      else if (a.v_fmt == FMT_F32)
        hipLaunchKernelGGL((block_bwd_kernel<FMT_F32, FMT_BF16, NV, TPB>), grid, dim3(TPB), 0, s, a);
      else if (a.skip_fmt == FMT_F32)
        hipLaunchKernelGGL((block_bwd_kernel<FMT_BF16, FMT_F32, NV, TPB>), grid, dim3(TPB), 0, s, a);
      else
        hipLaunchKernelGGL((block_bwd_kernel<FMT_BF16, FMT_BF16, NV, TPB>), grid, dim3(TPB), 0, s, a);
    });
    if (e != hipSuccess) return e;
  }
  const unsigned cb = static_cast<unsigned>(ceil_div(a.d, 64));
  if (p.whole_gates) {
    if (a.dw == nullptr) return hipSuccess;
    const ColSumArgs c{a.part, static_cast<int>(p.blocks), a.d, 1, nullptr, nullptr, nullptr, a.dw, p.blocks, 1};
    hipLaunchKernelGGL(block_colsum_kernel, dim3(cb, 1), dim3(1024), 0, s, c);
    return hipGetLastError();
  }
  if (a.dw == nullptr && a.dgate == nullptr) return hipSuccess;
  if (p.gates <= CS_GATES) {
    const ColSumArgs c{a.part, p.runs, a.d, static_cast<int>(p.gates), a.w, a.gate, a.dgate, a.dw, p.blocks, p.gates};
    hipLaunchKernelGGL(block_colsum_kernel, dim3(cb, 1), dim3(1024), 0, s, c);
    return hipGetLastError();
  }
  // many gates: a block each, then the sum of their shares of dw
  float* q = a.part + static_cast<size_t>(p.blocks) * a.d;
  const ColSumArgs c1{a.part, p.runs, a.d, 1, a.w, a.gate, a.dgate, a.dw == nullptr ? nullptr : q,
                      p.blocks, p.gates};
  // the grid's second dimension holds at most 65535 gates
  for (long long g0 = 0; g0 < p.gates; g0 += 32768) {
    ColSumArgs cg = c1;
    const long long n = p.gates - g0 < 32768 ? p.gates - g0 : 32768;
    const size_t go = static_cast<size_t>(g0) * a.d;
    cg.part += go * p.runs;
    cg.rows -= g0 * p.runs;
    cg.gates -= g0;
    if (cg.gate != nullptr) cg.gate += go;
    if (cg.dgate != nullptr) cg.dgate += go;
    if (cg.out != nullptr) cg.out += go;
    hipLaunchKernelGGL(block_colsum_kernel, dim3(cb, static_cast<unsigned>(n)), dim3(1024), 0, s, cg);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  if (a.dw != nullptr) {
    const ColSumArgs c2{q, static_cast<int>(p.gates), a.d, 1, nullptr, nullptr, nullptr, a.dw, p.gates, 1};
    hipLaunchKernelGGL(block_colsum_kernel, dim3(cb, 1), dim3(1024), 0, s, c2);
  }
  return hipGetLastError();
}

}  // namespace moe
