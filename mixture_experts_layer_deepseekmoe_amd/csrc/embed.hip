// The embedding and its gradient:
//
//   x_t = scale table[token_t]  (zeros for a token outside [0, V)), optionally
//         with the first block's norm of x_t as stored
//   dtable_v = scale sum_{t: token_t = v} dx_t
//
// Both are bound by HBM: the rows once, and of the gradient all V rows written
// (or, added to, the named rows alone).  For the gradient the rows are sorted by
// token (stable: rows of a token stay in order), so a wave finds the rows of a
// token side by side and sums them in registers, in fp32 and in a fixed order: no
// atomics.  The table is cleared beside the sorting, which needs few of the CUs; the
// named rows are then written over.  (One pass that finds each row's run by a search
// and writes every row once took 417 us for 65536 x 7168 in fp32, where clearing takes
// 290 and the sums 80: its waves wait for their searches, loads and stores in turn.)
//
// Measured, us: 8192 rows of 7168 into 65536 in fp32, 466 with the forward: forward with
// the norm 54, clearing beside the sort 300 (6.3 TB/s), sums 26 + 5 + 82; 4096 rows of
// 2048 into 65536 in bf16, 84: 13, 40.5, 7, 21.  Added to a table, the backward alone 108
// of 414 and 25 of 60.
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

// Clears 128 KB of the table, by 1024 threads.
constexpr int CLEAR_THREADS = 1024;
constexpr long long CLEAR_BYTES = 128 << 10;
__host__ __device__ inline long long table_bytes(const EmbedBwdArgs& a) {
  return static_cast<long long>(a.V) * a.d * (a.grad_fmt == FMT_F32 ? 4 : 2);
}
__device__ __forceinline__ void clear_table(const EmbedBwdArgs& a, unsigned block) {
  const long long n = table_bytes(a);   // a multiple of 16
#pragma unroll
  for (int i = 0; i < CLEAR_BYTES / 16 / CLEAR_THREADS; ++i) {
    const long long at = block * CLEAR_BYTES + 16 * (threadIdx.x + CLEAR_THREADS * i);
    if (at < n) *reinterpret_cast<i32x4*>(static_cast<uint8_t*>(a.dtable) + at) = i32x4{0, 0, 0, 0};
  }
}
__global__ __launch_bounds__(CLEAR_THREADS) void embed_clear_kernel(EmbedBwdArgs a) {
  if (!MOE_CHECK(blockIdx.x * CLEAR_BYTES < table_bytes(a), 905)) return;
  clear_table(a, blockIdx.x);
}

// A row's place is the number of rows before it: those of a lower token, and earlier
// ones of its own, both in one comparison of (token, row) as a number of 32 bits where
// these suffice (U).  A block ranks 32 rows; its threads hold 8 keys each at a time.
constexpr int RANK_ROWS = 32, RANK_KEYS = 8, RANK_THREADS = 1024;
template <class U>
__global__ __launch_bounds__(RANK_THREADS) void embed_rank_kernel(EmbedBwdArgs a, int row_bits, int blocks) {
  __shared__ int cnt[RANK_THREADS / 64][RANK_ROWS];
  if (static_cast<int>(blockIdx.x) >= blocks) return clear_table(a, blockIdx.x - blocks);
  const int w = wave_id(), lane = threadIdx.x & 63, t0 = blockIdx.x * RANK_ROWS;
  const int rows = min(RANK_ROWS, a.T - t0);
  const int row = t0 + min(lane & (RANK_ROWS - 1), rows - 1);   // lane r: row t0 + r
  const int id = key_of(a, row);
  const U mine = static_cast<U>(id) << row_bits | static_cast<U>(row);
  int n = 0;                                                    // lane r: rows before it
  for (int k0 = 0; k0 < a.T; k0 += RANK_KEYS * RANK_THREADS) {
    U key[RANK_KEYS];
#pragma unroll
    for (int j = 0; j < RANK_KEYS; ++j) {
      const int p = k0 + j * RANK_THREADS + static_cast<int>(threadIdx.x);
      key[j] = p < a.T ? static_cast<U>(key_of(a, p)) << row_bits | static_cast<U>(p) : ~U{0};
    }
    const int held = min(RANK_KEYS, ceil_div(a.T - k0, RANK_THREADS));
    for (int r = 0; r < rows; ++r) {
      U k;
      if constexpr (sizeof(U) == 4)
        k = static_cast<U>(__builtin_amdgcn_readlane(mine, r));
      else
        k = static_cast<U>(static_cast<uint32_t>(__builtin_amdgcn_readlane(static_cast<int>(mine >> 32), r))) << 32 |
            static_cast<uint32_t>(__builtin_amdgcn_readlane(static_cast<int>(mine), r));
      int c = 0;
#pragma unroll
      for (int j = 0; j < RANK_KEYS; ++j)
        if (j < held) c += __popcll(__ballot(key[j] < k));
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
  a.ids[at] = id;
  a.order[at] = row;
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

constexpr int SUM_THREADS = 256, SUM_WAVES = SUM_THREADS / 64;

// A wave's number in a grid of one or (past 2^31 threads) two dimensions.
__device__ __forceinline__ int sum_wave() {
  return static_cast<int>((blockIdx.y * gridDim.x + blockIdx.x) * SUM_WAVES + wave_id());
}
inline dim3 sum_grid(long long waves) {
  constexpr long long WIDTH = 1 << 23;
  const long long blocks = (waves + SUM_WAVES - 1) / SUM_WAVES;
  if (blocks <= WIDTH) return dim3(static_cast<unsigned>(blocks));
  return dim3(WIDTH, static_cast<unsigned>((blocks + WIDTH - 1) / WIDTH));
}

// A wave's sums of 256 V columns, V times four to a lane: pairs of fours side by side
// for rows of bf16 (16 bytes a store).
template <int GF, int V>
struct Slab {
  float4 v[V];
  int c0, d;
  __device__ __forceinline__ Slab(int c0_, int d_) : c0(c0_), d(d_) {
#pragma unroll
    for (int i = 0; i < V; ++i) v[i] = make_float4(0.f, 0.f, 0.f, 0.f);
  }
  __device__ __forceinline__ int col(int i) const {
    const int lane = threadIdx.x & 63;
    return c0 + (GF == FMT_BF16 ? 8 * lane + 512 * (i / 2) + 4 * (i % 2) : 4 * lane + 256 * i);
  }
  __device__ __forceinline__ bool in(int i) const { return col(i) < d; }
  // Adds n rows of src, in order: rows 0, 1, ..., or those that lanes 0, 1, ... of `at`
  // name.  N rows' loads go out together.
  template <int N, bool AT>
  __device__ __forceinline__ void add(const float* src, int at, int n) {
#pragma unroll 1
    for (int r = 0; r < n; r += N) {
      float4 x[N][V];
#pragma unroll
      for (int j = 0; j < N; ++j) {
        if (r + j >= n) continue;
        const size_t row = static_cast<size_t>(AT ? __builtin_amdgcn_readlane(at, r + j) : r + j);
#pragma unroll
        for (int i = 0; i < V; ++i)
          if (in(i)) x[j][i] = *reinterpret_cast<const float4*>(src + row * d + col(i));
      }
#pragma unroll
      for (int j = 0; j < N; ++j) {
        if (r + j >= n) continue;
#pragma unroll
        for (int i = 0; i < V; ++i) {
          if (!in(i)) continue;
          v[i].x += x[j][i].x;
          v[i].y += x[j][i].y;
          v[i].z += x[j][i].z;
          v[i].w += x[j][i].w;
        }
      }
    }
  }
};

// The sums of chunks that hold one token throughout (LEVEL 2: of the chunks' chunks), 16
// rows at once.
template <int LEVEL>
__global__ __launch_bounds__(SUM_THREADS) void embed_chunk_kernel(EmbedBwdArgs a) {
  constexpr int C = LEVEL == 1 ? EMBED_CHUNK : EMBED_CHUNK2, N = LEVEL == 1 ? C : C / EMBED_CHUNK;
  const int slabs = ceil_div(a.d, 256), wave = sum_wave(), lane = threadIdx.x & 63;
  const int chunk = wave / slabs;   // waves side by side read a row's columns in order
  if (chunk >= a.T / C) return;
  const int r0 = chunk * C, id = a.ids[r0], last = a.ids[r0 + C - 1], at = LEVEL == 1 ? a.order[r0 + lane % C] : 0;
  if (id >= a.V || last != id || !MOE_CHECK(at >= 0 && at < a.T, 907)) return;
  Slab<FMT_F32, 1> s(wave % slabs * 256, a.d);
  if constexpr (LEVEL == 1)
    s.add<N, true>(a.dx, at, N);
  else
    s.add<N, false>(a.part + static_cast<size_t>(chunk) * N * a.d, 0, N);
  if (s.in(0))
    *reinterpret_cast<float4*>((LEVEL == 1 ? a.part : a.part2) + static_cast<size_t>(chunk) * a.d + s.col(0)) = s.v[0];
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

// Adds sorted rows r0 .. r1 - 1, all of one token, of which lanes hold the first 64 in
// `at`: whole chunks by their sums.  A long run is at most five stretches one after the
// other: rows, chunks, chunks' chunks, chunks, rows.
constexpr int SUM_ROWS = 4;   // in flight (8: 485 us instead of 474, 65536 x 7168)
template <class S>
__device__ __forceinline__ void add_run(S& s, const EmbedBwdArgs& a, int r0, int r1, int at) {
  if (r1 - r0 < EMBED_CHUNK) {
    s.template add<SUM_ROWS, true>(a.dx, at, r1 - r0);
    return;
  }
  auto up = [](int r, int c) { return (r + c - 1) / c * c; };
  const int lane = threadIdx.x & 63;
#pragma unroll 1
  for (int step = 0; step <= 4 && r0 < r1; ++step) {
    const int size = step == 2 ? EMBED_CHUNK2 : step % 4 != 0 ? EMBED_CHUNK : 1;
    if (size == EMBED_CHUNK2 && a.part2 == nullptr) continue;
    // to where the next stretch's chunks begin, or as far as this one's go
    const int to = step == 0 ? up(r0, EMBED_CHUNK) : step == 1 && a.part2 != nullptr ? up(r0, EMBED_CHUNK2) : r1;
    const int n = (min(to, r1) - r0) / size;
    if (size == 1) {   // fewer than a chunk
      if (step == 4) at = a.order[min(r0 + lane, a.T - 1)];
      s.template add<SUM_ROWS, true>(a.dx, at, n);
    } else {
      s.template add<SUM_ROWS, false>((size == EMBED_CHUNK ? a.part : a.part2) + static_cast<size_t>(r0 / size) * a.d, 0, n);
    }
    r0 += n * size;
  }
}

// The named rows of the gradient: the wave of a token's first sorted row sums them.
constexpr int SUM_COLS = 512;
template <int GF>
__global__ __launch_bounds__(SUM_THREADS) void embed_grad_kernel(EmbedBwdArgs a) {
  const int slabs = ceil_div(a.d, SUM_COLS), wave = sum_wave(), lane = threadIdx.x & 63;
  const int r = wave / slabs, held = min(r + lane, a.T - 1);
  if (r >= a.T) return;
  const int before = r > 0 ? a.ids[r - 1] : -1, at = a.order[held];
  int id = a.ids[held];
  if (r + lane >= a.T) id = a.V;
  const int v = __builtin_amdgcn_readfirstlane(id);
  if (v >= a.V || __builtin_amdgcn_readfirstlane(before) == v) return;
  if (!MOE_CHECK(v >= 0 && at >= 0 && at < a.T, 906)) return;
  int r1 = r + __popcll(__ballot(id == v));
  if (r1 == r + 64) r1 = lower_bound(a.ids, r1, a.T, v + 1);   // it may go on behind the rows held
  constexpr int V = SUM_COLS / 256;
  Slab<GF, V> s(wave % slabs * SUM_COLS, a.d);
  add_run(s, a, r, r1, at);
  const size_t off = static_cast<size_t>(v) * a.d;
  float x[V][4];
#pragma unroll
  for (int i = 0; i < V; ++i) {
    x[i][0] = s.v[i].x * a.scale;
    x[i][1] = s.v[i].y * a.scale;
    x[i][2] = s.v[i].z * a.scale;
    x[i][3] = s.v[i].w * a.scale;
  }
  if constexpr (GF == FMT_F32) {
#pragma unroll
    for (int i = 0; i < V; ++i) {
      if (!s.in(i)) continue;
      float4* p = reinterpret_cast<float4*>(static_cast<float*>(a.dtable) + off + s.col(i));
      if (a.accumulate) {
        const float4 o = *p;
        x[i][0] += o.x; x[i][1] += o.y; x[i][2] += o.z; x[i][3] += o.w;
      }
      *p = make_float4(x[i][0], x[i][1], x[i][2], x[i][3]);
    }
  } else {
#pragma unroll
    for (int i = 0; i < V; i += 2) {
      if (!s.in(i)) continue;   // d is a multiple of 8: both or none
      uint4* p = reinterpret_cast<uint4*>(static_cast<uint16_t*>(a.dtable) + off + s.col(i));
      if (a.accumulate) {
        const uint4 o = *p;
        const uint32_t w[4] = {o.x, o.y, o.z, o.w};
#pragma unroll
        for (int e = 0; e < 8; ++e) x[i + e / 4][e % 4] += __uint_as_float(e % 2 ? w[e / 2] & 0xffff0000u : w[e / 2] << 16);
      }
      *p = make_uint4(bf16x2(x[i][0], x[i][1]), bf16x2(x[i][2], x[i][3]), bf16x2(x[i + 1][0], x[i + 1][1]),
                      bf16x2(x[i + 1][2], x[i + 1][3]));
    }
  }
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
  const int clear = a.accumulate ? 0 : static_cast<int>((table_bytes(a) + CLEAR_BYTES - 1) / CLEAR_BYTES);
  if (a.T == 0 || a.T > EMBED_RANK_T) {
    if (clear > 0) hipLaunchKernelGGL(embed_clear_kernel, dim3(clear), dim3(CLEAR_THREADS), 0, s, a);
    if (a.T == 0) return hipGetLastError();
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
  } else {
    int row_bits = 0;
    while (a.T - 1 >> row_bits) ++row_bits;
    // (V, T - 1) is the largest, and all ones stand for no row
    const bool narrow = (static_cast<unsigned long long>(a.V) + 1) << row_bits <= 0xffffffffULL;
    const int blocks = ceil_div(a.T, RANK_ROWS);
    const dim3 grid(blocks + clear), block(RANK_THREADS);
    if (narrow)
      hipLaunchKernelGGL(embed_rank_kernel<uint32_t>, grid, block, 0, s, a, row_bits, blocks);
    else
      hipLaunchKernelGGL(embed_rank_kernel<uint64_t>, grid, block, 0, s, a, row_bits, blocks);
  }
  if (a.T < EMBED_PART2_T) a.part2 = nullptr;
  // rows times slabs: below 2^22 x 64 waves to a launch
  const dim3 block(SUM_THREADS);
  const int slabs = ceil_div(a.d, 256);
  if (a.T >= EMBED_CHUNK)
    hipLaunchKernelGGL(embed_chunk_kernel<1>, sum_grid(static_cast<long long>(a.T / EMBED_CHUNK) * slabs), block, 0, s, a);
  if (a.part2 != nullptr)
    hipLaunchKernelGGL(embed_chunk_kernel<2>, sum_grid(static_cast<long long>(a.T / EMBED_CHUNK2) * slabs), block, 0, s, a);
  const dim3 grid = sum_grid(static_cast<long long>(a.T) * ceil_div(a.d, SUM_COLS));
  if (a.grad_fmt == FMT_F32)
    hipLaunchKernelGGL(embed_grad_kernel<FMT_F32>, grid, block, 0, s, a);
  else
    hipLaunchKernelGGL(embed_grad_kernel<FMT_BF16>, grid, block, 0, s, a);
  return hipGetLastError();
}

}  // namespace moe
