// The embedding and its gradient:
//
//   x_t = scale table[token_t]  (zeros for a token outside [0, V)), optionally
//         with the first block's norm of x_t as stored
//   dtable_v = scale sum_{t: token_t = v} dx_t
//
// Both are bound by HBM: the rows once, and of the gradient all V rows written
// (or, added to, the named rows alone).  For the gradient the rows are sorted by
// token (stable: rows of a token stay in order), so a wave finds the rows of a
// token side by side, sums them in registers, in fp32 and in a fixed order, and
// writes each row of the table once, zeros included: no atomics, no clearing pass.
#include "ends.hpp"
#include "gemm_core.hpp"
#include "rows.hpp"

namespace moe {

namespace {

template <int TF, int XF, int NF, int NV, int TPB>
__global__ __launch_bounds__(TPB) void embed_kernel(EmbedArgs a) {
  __shared__ float red[TPB / 64];
  const size_t row = blockIdx.x;
  if (!MOE_CHECK(row < static_cast<size_t>(a.T) && a.d <= 8 * TPB * NV, 901)) return;
  const int tok = a.tokens[row];
  const bool in = tok >= 0 && tok < a.V;
  const size_t at = static_cast<size_t>(in ? tok : 0) * a.d;
  float x[NV][8];
  Raw8 raw[NV];
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int c = 8 * (threadIdx.x + TPB * i);
    raw[i].a = raw[i].b = make_uint4(0, 0, 0, 0);
    if (in && c < a.d) raw[i] = load8<TF>(a.table, at + c);
  }
  float ss = 0.f;
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int c = 8 * (threadIdx.x + TPB * i);
    if (c >= a.d) continue;
    values8<TF>(raw[i], x[i]);
#pragma unroll
    for (int e = 0; e < 8; ++e) x[i][e] *= a.scale;
    store8<XF>(a.x, row * a.d + c, x[i]);   // x: as stored
#pragma unroll
    for (int e = 0; e < 8; ++e) ss = fmaf(x[i][e], x[i][e], ss);
  }
  if (a.w_next == nullptr) return;
  const float r = rstd_of(block_sum<TPB>(ss, red), a.d, a.eps);
  if (a.rstd != nullptr && threadIdx.x == 0) a.rstd[row] = r;
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int c = 8 * (threadIdx.x + TPB * i);
    if (c >= a.d) continue;
    if (a.codes != nullptr) save_tile(x[i], a.codes, a.scales, row, a.d, c);
    float w[8];
    load8f(a.w_next, c, w);
#pragma unroll
    for (int e = 0; e < 8; ++e) w[e] *= x[i][e] * r;
    store8<NF>(a.n, row * a.d + c, w);
  }
}

// ------------------------------------------------------------------ sorting

__device__ __forceinline__ int key_of(const EmbedBwdArgs& a, int t) {
  const int tok = a.tokens[t];
  return tok >= 0 && tok < a.V ? tok : a.V;
}

// A row's place is the number of rows before it: those of a lower token, and earlier
// ones of its own.  A block ranks 32 rows; its threads hold 8 keys each at a time.
constexpr int RANK_ROWS = 32, RANK_KEYS = 8, RANK_THREADS = 1024;
__global__ __launch_bounds__(RANK_THREADS) void embed_rank_kernel(EmbedBwdArgs a) {
  __shared__ int cnt[RANK_THREADS / 64][RANK_ROWS];
  const int w = wave_id(), lane = threadIdx.x & 63, t0 = blockIdx.x * RANK_ROWS;
  const int rows = min(RANK_ROWS, a.T - t0);
  const int mine = key_of(a, t0 + min(lane & (RANK_ROWS - 1), rows - 1));   // lane r: row t0 + r
  int n = 0;                                                              // lane r: rows before it
  for (int k0 = 0; k0 < a.T; k0 += RANK_KEYS * RANK_THREADS) {
    int key[RANK_KEYS];
#pragma unroll
    for (int j = 0; j < RANK_KEYS; ++j) {
      const int p = k0 + j * RANK_THREADS + static_cast<int>(threadIdx.x);
      key[j] = p < a.T ? key_of(a, p) : 0x7fffffff;
    }
    for (int r = 0; r < rows; ++r) {
      const int k = __builtin_amdgcn_readlane(mine, r), t = t0 + r;
      int c = 0;
#pragma unroll
      for (int j = 0; j < RANK_KEYS; ++j) {
        const int p = k0 + j * RANK_THREADS + static_cast<int>(threadIdx.x);
        c += __popcll(__ballot(key[j] < k + (p < t)));
      }
      if (lane == r) n += c;
    }
  }
  if (lane < RANK_ROWS) cnt[w][lane] = n;
  __syncthreads();
  if (static_cast<int>(threadIdx.x) >= rows) return;
  int at = 0;
#pragma unroll
  for (int k = 0; k < RANK_THREADS / 64; ++k) at += cnt[k][threadIdx.x];
  if (!MOE_CHECK(at >= 0 && at < a.T, 902)) return;
  a.ids[at] = mine;
  a.order[at] = t0 + threadIdx.x;
}

// Radix sort, 8 bits a pass, stable.  A block takes 4096 rows, each of its 4 waves a
// quarter of them, in order.
constexpr int RADIX_THREADS = 256, RADIX_WAVES = 4;
struct RadixArgs {
  EmbedBwdArgs e;
  const int32_t* ids;    // null: the first pass, straight from the tokens
  const int32_t* order;
  int32_t* ids_out;
  int32_t* order_out;
  int shift, blocks;
};

__global__ __launch_bounds__(RADIX_THREADS) void embed_hist_kernel(RadixArgs a) {
  __shared__ int h[256];
  h[threadIdx.x] = 0;
  __syncthreads();
  const int t0 = blockIdx.x * EMBED_RADIX_BLOCK, t1 = min(a.e.T, t0 + EMBED_RADIX_BLOCK);
  for (int t = t0 + threadIdx.x; t < t1; t += RADIX_THREADS)
    atomicAdd(&h[(a.ids != nullptr ? a.ids[t] : key_of(a.e, t)) >> a.shift & 255], 1);
  __syncthreads();
  if (!MOE_CHECK(static_cast<int>(blockIdx.x) < a.blocks, 903)) return;
  a.e.hist[threadIdx.x * a.blocks + blockIdx.x] = h[threadIdx.x];
}

// Exclusive sums over [256][blocks], by one block.
__global__ __launch_bounds__(1024) void embed_scan_kernel(RadixArgs a) {
  __shared__ int sums[16];
  const int n = 256 * a.blocks, lane = threadIdx.x & 63, w = wave_id();
  int before = 0;
  for (int i0 = 0; i0 < n; i0 += 4096) {
    const int i = i0 + 4 * threadIdx.x;   // n is a multiple of 4
    int4 v = make_int4(0, 0, 0, 0);
    if (i < n) v = *reinterpret_cast<const int4*>(a.e.hist + i);
    const int own = v.x + v.y + v.z + v.w;
    int run = own;
#pragma unroll
    for (int off = 1; off < 64; off <<= 1) {
      const int u = __shfl_up(run, off);
      if (lane >= off) run += u;
    }
    if (lane == 63) sums[w] = run;
    __syncthreads();
    int base = before;
    for (int k = 0; k < 16; ++k) {
      if (k < w) base += sums[k];
      before += sums[k];
    }
    run += base - own;
    if (i < n) *reinterpret_cast<int4*>(a.e.hist + i) = make_int4(run, run + v.x, run + v.x + v.y, run + v.x + v.y + v.z);
    __syncthreads();
  }
}

__global__ __launch_bounds__(RADIX_THREADS) void embed_scatter_kernel(RadixArgs a) {
  __shared__ int at[RADIX_WAVES][256];
  constexpr int PER = EMBED_RADIX_BLOCK / RADIX_WAVES;
  const int w = wave_id(), lane = threadIdx.x & 63;
  const int t0 = blockIdx.x * EMBED_RADIX_BLOCK + w * PER, t1 = min(a.e.T, t0 + PER);
  for (int k = 0; k < RADIX_WAVES; ++k) at[k][threadIdx.x] = 0;
  __syncthreads();
  for (int t = t0 + lane; t < t1; t += 64)
    atomicAdd(&at[w][(a.ids != nullptr ? a.ids[t] : key_of(a.e, t)) >> a.shift & 255], 1);
  __syncthreads();
  int sum = a.e.hist[threadIdx.x * a.blocks + blockIdx.x];
#pragma unroll
  for (int k = 0; k < RADIX_WAVES; ++k) {
    const int c = at[k][threadIdx.x];
    at[k][threadIdx.x] = sum;
    sum += c;
  }
  __syncthreads();
  for (int t = t0; t < t1; t += 64) {   // t0, t1: the wave's
    const bool live = t + lane < t1;
    const int id = !live ? 0 : a.ids != nullptr ? a.ids[t + lane] : key_of(a.e, t + lane);
    const int digit = id >> a.shift & 255;
    unsigned long long same = __ballot(live);
#pragma unroll
    for (int b = 0; b < 8; ++b) {
      const unsigned long long set = __ballot(digit >> b & 1);
      same &= digit >> b & 1 ? set : ~set;
    }
    const int before = __popcll(same & ((1ULL << lane) - 1));
    int base = 0;
    if (live) base = at[w][digit];
    __builtin_amdgcn_wave_barrier();
    if (live && before == 0) at[w][digit] = base + __popcll(same);
    __builtin_amdgcn_wave_barrier();
    if (!live || !MOE_CHECK(base + before >= 0 && base + before < a.e.T, 904)) continue;
    a.ids_out[base + before] = id;
    a.order_out[base + before] = a.order != nullptr ? a.order[t + lane] : t + lane;
  }
}

// ------------------------------------------------------------------ sums

constexpr int SLAB = 1024;   // columns of a wave: 4 times 4 to a lane
constexpr int SUM_THREADS = 256;

struct Slab {
  float4 v[SLAB / 256];
};
__device__ __forceinline__ void zero(Slab& s) {
#pragma unroll
  for (int i = 0; i < SLAB / 256; ++i) s.v[i] = make_float4(0.f, 0.f, 0.f, 0.f);
}
// Adds columns c0 .. of n rows of src, rows at[0], at[1], ... (null: 0, 1, ...), in
// order; N rows' loads go out together.
template <int N>
__device__ __forceinline__ void add_n(Slab& s, const float* src, const int32_t* at, int r0, int d, int c) {
  float4 v[N][SLAB / 256];
#pragma unroll
  for (int j = 0; j < N; ++j) {
    const size_t row = static_cast<size_t>(at != nullptr ? __builtin_amdgcn_readfirstlane(at[r0 + j]) : r0 + j);
    const float* p = src + row * d;
#pragma unroll
    for (int i = 0; i < SLAB / 256; ++i)
      if (c + 256 * i < d) v[j][i] = *reinterpret_cast<const float4*>(p + c + 256 * i);
  }
#pragma unroll
  for (int j = 0; j < N; ++j)
#pragma unroll
    for (int i = 0; i < SLAB / 256; ++i) {
      if (c + 256 * i >= d) continue;
      s.v[i].x += v[j][i].x;
      s.v[i].y += v[j][i].y;
      s.v[i].z += v[j][i].z;
      s.v[i].w += v[j][i].w;
    }
}
__device__ __forceinline__ void add_rows(Slab& s, const float* src, const int32_t* at, int n, int d, int c0) {
  const int c = c0 + 4 * (threadIdx.x & 63);
  int r = 0;
  for (; r + 4 <= n; r += 4) add_n<4>(s, src, at, r, d, c);
  for (; r < n; ++r) add_n<1>(s, src, at, r, d, c);
}

// The sums of chunks that hold one token throughout.
__global__ __launch_bounds__(SUM_THREADS) void embed_chunk_kernel(EmbedBwdArgs a) {
  const int chunk = blockIdx.x * (SUM_THREADS / 64) + wave_id(), c0 = blockIdx.y * SLAB;
  if (chunk >= a.T / EMBED_CHUNK) return;
  const int r0 = chunk * EMBED_CHUNK, id = a.ids[r0];
  if (id >= a.V || a.ids[r0 + EMBED_CHUNK - 1] != id) return;
  Slab s;
  zero(s);
  add_rows(s, a.dx, a.order + r0, EMBED_CHUNK, a.d, c0);
  const int c = c0 + 4 * (threadIdx.x & 63);
#pragma unroll
  for (int i = 0; i < SLAB / 256; ++i)
    if (c + 256 * i < a.d) *reinterpret_cast<float4*>(a.part + static_cast<size_t>(chunk) * a.d + c + 256 * i) = s.v[i];
}

// The first sorted row at or past `lo` whose token is at least v (a wave: 64 probes a
// step, so three steps for 2^18 rows).
__device__ __forceinline__ int lower_bound(const int32_t* ids, int lo, int hi, int v) {
  const int lane = threadIdx.x & 63;
  while (lo < hi) {   // the answer lies in [lo, hi]
    const int step = (hi - lo + 63) / 64;
    const long long p = lo + static_cast<long long>(lane) * step;
    const bool less = p < hi && ids[p] < v;
    const int c = __popcll(__ballot(less));   // the first c probes are less
    if (c == 0) return lo;
    const int next = lo + (c - 1) * step + 1;
    hi = min(static_cast<long long>(hi), lo + static_cast<long long>(c) * step);
    lo = next;
  }
  return lo;
}

// Writes row v of the gradient from sorted rows r0 .. r1 - 1 (none: zeros).
template <int GF>
__device__ __forceinline__ void write_row(const EmbedBwdArgs& a, int v, int r0, int r1, int c0) {
  Slab s;
  zero(s);
  if (r0 < r1) {
    // whole chunks have been summed: the rows before the first, the chunks, the rows behind the last
    const int k0 = (r0 + EMBED_CHUNK - 1) / EMBED_CHUNK, k1 = r1 / EMBED_CHUNK;
    if (k0 < k1) {
      add_rows(s, a.dx, a.order + r0, k0 * EMBED_CHUNK - r0, a.d, c0);
      add_rows(s, a.part + static_cast<size_t>(k0) * a.d, nullptr, k1 - k0, a.d, c0);
      add_rows(s, a.dx, a.order + k1 * EMBED_CHUNK, r1 - k1 * EMBED_CHUNK, a.d, c0);
    } else {
      add_rows(s, a.dx, a.order + r0, r1 - r0, a.d, c0);
    }
  }
  const int c = c0 + 4 * (threadIdx.x & 63);
#pragma unroll
  for (int i = 0; i < SLAB / 256; ++i) {
    if (c + 256 * i >= a.d) continue;
    const size_t off = static_cast<size_t>(v) * a.d + c + 256 * i;
    float4 x = s.v[i];
    x.x *= a.scale; x.y *= a.scale; x.z *= a.scale; x.w *= a.scale;
    if constexpr (GF == FMT_F32) {
      float4* p = reinterpret_cast<float4*>(static_cast<float*>(a.dtable) + off);
      if (a.accumulate) {
        const float4 o = *p;
        x.x += o.x; x.y += o.y; x.z += o.z; x.w += o.w;
      }
      *p = x;
    } else {
      uint2* p = reinterpret_cast<uint2*>(static_cast<uint16_t*>(a.dtable) + off);
      if (a.accumulate) {
        const uint2 o = *p;
        x.x += __uint_as_float(o.x << 16); x.y += __uint_as_float(o.x & 0xffff0000u);
        x.z += __uint_as_float(o.y << 16); x.w += __uint_as_float(o.y & 0xffff0000u);
      }
      *p = make_uint2(bf16x2(x.x, x.y), bf16x2(x.z, x.w));
    }
  }
}

// Every row of the table: a wave takes `rows` of them in turn, and the rows of each
// from the 64 sorted tokens it holds.
template <int GF>
__global__ __launch_bounds__(SUM_THREADS) void embed_grad_kernel(EmbedBwdArgs a, int rows) {
  const long long v0 = (static_cast<long long>(blockIdx.x) * (SUM_THREADS / 64) + wave_id()) * rows;
  const int v1 = static_cast<int>(min(static_cast<long long>(a.V), v0 + rows)), c0 = blockIdx.y * SLAB;
  const int lane = threadIdx.x & 63;
  if (v0 >= a.V || !MOE_CHECK(c0 < a.d, 905)) return;
  int r = lower_bound(a.ids, 0, a.T, static_cast<int>(v0));
  int base = r, id = r + lane < a.T ? a.ids[r + lane] : a.V;
  for (int v = static_cast<int>(v0); v < v1; ++v) {
    // r is the first row of a token >= v, and base <= r <= base + 64
    if (r == base + 64) {
      base = r;
      id = r + lane < a.T ? a.ids[r + lane] : a.V;
    }
    int r1 = r + __popcll(__ballot(id == v));
    if (r1 == base + 64) {   // it may go on behind the tokens held
      r1 = lower_bound(a.ids, r1, a.T, v + 1);
      if (r1 > base + 64) {
        write_row<GF>(a, v, r, r1, c0);
        r = base = r1;
        id = r + lane < a.T ? a.ids[r + lane] : a.V;
        continue;
      }
    }
    write_row<GF>(a, v, r, r1, c0);
    r = r1;
  }
}

// The named rows alone: the wave of a token's first sorted row takes them.
template <int GF>
__global__ __launch_bounds__(SUM_THREADS) void embed_grad_add_kernel(EmbedBwdArgs a) {
  const int r = blockIdx.x * (SUM_THREADS / 64) + wave_id();
  if (r >= a.T) return;
  const int v = __builtin_amdgcn_readfirstlane(a.ids[r]);
  if (v >= a.V || (r > 0 && __builtin_amdgcn_readfirstlane(a.ids[r - 1]) == v)) return;
  if (!MOE_CHECK(v >= 0, 906)) return;
  write_row<GF>(a, v, r, lower_bound(a.ids, r, a.T, v + 1), blockIdx.y * SLAB);
}

}  // namespace

MOE_DEBUG_FILE(embed)

hipError_t launch_embed(const EmbedArgs& a, hipStream_t s) {
  if (a.T == 0) return hipSuccess;
  return with_fmt(a.table_fmt, [&]<int TF>() {
    return with_fmt(a.x_fmt, [&]<int XF>() {
      return with_fmt(a.n_fmt, [&]<int NF>() {
        return with_row_shape(a.T, a.d, [&]<int NV, int TPB>() {   // as block_in: n is the same, bit for bit
          hipLaunchKernelGGL((embed_kernel<TF, XF, NF, NV, TPB>), dim3(a.T), dim3(TPB), 0, s, a);
        });
      });
    });
  });
}

hipError_t launch_embed_bwd(const EmbedBwdArgs& args, hipStream_t s) {
  EmbedBwdArgs a = args;
  if (a.T > EMBED_RANK_T) {
    RadixArgs r{};
    r.e = a;
    r.blocks = embed_radix_blocks(a.T);
    for (int p = 0; p < embed_radix_passes(a.V); ++p) {
      r.shift = 8 * p;
      r.ids = p == 0 ? nullptr : r.ids_out;
      r.order = p == 0 ? nullptr : r.order_out;
      r.ids_out = p % 2 == 0 ? a.ids : a.ids2;
      r.order_out = p % 2 == 0 ? a.order : a.order2;
      hipLaunchKernelGGL(embed_hist_kernel, dim3(r.blocks), dim3(RADIX_THREADS), 0, s, r);
      hipLaunchKernelGGL(embed_scan_kernel, dim3(1), dim3(1024), 0, s, r);
      hipLaunchKernelGGL(embed_scatter_kernel, dim3(r.blocks), dim3(RADIX_THREADS), 0, s, r);
    }
    a.ids = r.ids_out;
    a.order = r.order_out;
  } else if (a.T > 0) {
    hipLaunchKernelGGL(embed_rank_kernel, dim3(ceil_div(a.T, RANK_ROWS)), dim3(RANK_THREADS), 0, s, a);
  }
  constexpr int W = SUM_THREADS / 64;
  const int slabs = ceil_div(a.d, SLAB);
  if (a.T >= EMBED_CHUNK)
    hipLaunchKernelGGL(embed_chunk_kernel, dim3(ceil_div(a.T / EMBED_CHUNK, W), slabs), dim3(SUM_THREADS), 0, s, a);
  if (a.accumulate) {
    const dim3 grid(ceil_div(a.T, W), slabs);
    if (a.T == 0) return hipGetLastError();
    if (a.grad_fmt == FMT_F32)
      hipLaunchKernelGGL(embed_grad_add_kernel<FMT_F32>, grid, dim3(SUM_THREADS), 0, s, a);
    else
      hipLaunchKernelGGL(embed_grad_add_kernel<FMT_BF16>, grid, dim3(SUM_THREADS), 0, s, a);
    return hipGetLastError();
  }
  const int rows = 4;
  const dim3 grid(ceil_div(ceil_div(a.V, rows), W), slabs);
  if (a.grad_fmt == FMT_F32)
    hipLaunchKernelGGL(embed_grad_kernel<FMT_F32>, grid, dim3(SUM_THREADS), 0, s, a, rows);
  else
    hipLaunchKernelGGL(embed_grad_kernel<FMT_BF16>, grid, dim3(SUM_THREADS), 0, s, a, rows);
  return hipGetLastError();
}

}  // namespace moe
