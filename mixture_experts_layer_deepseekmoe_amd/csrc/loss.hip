// Cross entropy over a large vocabulary, without keeping the logits:
//
//   l_tv = h_t . w_v,  lse_t = log sum_v exp l_tv,  loss_t = lse_t - l_t,label
//   G_tv = (dloss_t + dlse_t) exp(l_tv - lse_t) - dloss_t [v = label_t]
//   dh = G w,  dw = G^T h
//
// forward   256 x 256 tiles of logits stay in the accumulators; a tile leaves
//           one (max, sum of exponentials) per row, which a second kernel
//           joins in tile order.
// backward  the vocabulary in pieces: the piece's logits are computed again
//           (bit for bit as in the forward), turned into G (bf16, a piece of
//           at most 512 MB) in the epilogue, and multiplied into dh (fp32, added
//           up over the pieces) and the piece's rows of dw.
//
// Only tokens with a label in [0, V) are rows of these products; the others
// (their hidden rows may hold anything) cost nothing, and their loss, lse and
// dh are zero.
//
// All three products are bound by the matrix cores.  Products are bf16 with
// fp32 accumulation; statistics and dh's sums are fp32; G is rounded to bf16
// once, as the operand of the two products that follow (a relative error of
// 2^-9 per element, as for the bf16 operands of the layer's backward).
#include "bwd_core.hpp"
#include "kernels.hpp"

namespace moe {

namespace {

constexpr int LT = LOSS_TILE;
constexpr int NXCDS = 8;

// Tile j of nm x nn, walked in groups of 8 m-tiles (m fastest): the 32 tiles
// an XCD's CUs hold at once share 8 row blocks and 4 column blocks in its L2.
// XCD x (blocks x, x + 8, ...) takes a contiguous eighth of the walk.
// Returns false where the block has no tile.
__device__ __forceinline__ bool loss_tile(int nm, int nn, int& m, int& n) {
  const long long total = static_cast<long long>(nm) * nn;
  const long long chunk = (total + NXCDS - 1) / NXCDS;
  const long long l = blockIdx.x / NXCDS, j = blockIdx.x % NXCDS * chunk + l;
  if (l >= chunk || j >= total) return false;
  constexpr int GM = 8;
  const int per = GM * nn, g = static_cast<int>(j / per), rem = static_cast<int>(j - static_cast<long long>(g) * per);
  const int gm = min(GM, nm - g * GM);
  m = g * GM + rem % gm;
  n = rem / gm;
  return true;
}
inline unsigned loss_grid(long long nm, long long nn) {
  return static_cast<unsigned>(NXCDS * ((nm * nn + NXCDS - 1) / NXCDS));
}

// m-tile m of `count` rows cut into nm = ceil(count / 256) nearly equal tiles
// (whole 16-row subtiles but for the last).
struct RowTile {
  int row0, rows;
};
__device__ __forceinline__ int row_tiles(int count) { return (count + LT - 1) / LT; }
__device__ __forceinline__ RowTile row_tile(int count, int nm, int m) {
  const int per = ((count + nm - 1) / nm + 15) / 16 * 16;   // at most 256
  const int r0 = m * per;
  return {r0, min(per, count - r0)};
}

// ------------------------------------------------------------------ rows

// The tokens with a label in [0, V), in order (one block; 1024 tokens at a
// time).  Forward: the others' loss and lse are zero.
__global__ __launch_bounds__(1024) void loss_rows_kernel(LossArgs a) {
  __shared__ int wsum[16];
  const int w = threadIdx.x >> 6, lane = threadIdx.x & 63;
  int base = 0;
  for (int t0 = 0; t0 < a.T; t0 += 1024) {
    const int t = t0 + threadIdx.x;
    const int lab = t < a.T ? a.labels[t] : -1;
    const bool ok = lab >= 0 && lab < a.V;
    const unsigned long long b = __ballot(ok);
    if (lane == 0) wsum[w] = __popcll(b);
    __syncthreads();
    int off = base, total = 0;
#pragma unroll
    for (int k = 0; k < 16; ++k) {
      if (k < w) off += wsum[k];
      total += wsum[k];
    }
    off += __popcll(b & ((1ULL << lane) - 1));
    if (t < a.T) {
      if (a.pos != nullptr) a.pos[t] = ok ? off : -1;
      if (ok) {
        a.rows[off] = t;
      } else if (a.loss != nullptr) {
        a.loss[t] = 0.f;
        a.lse[t] = 0.f;
      }
    }
    base += total;
    __syncthreads();
  }
  if (threadIdx.x == 0) a.count[0] = base;
}

// hc[r] = h[rows[r]]
__global__ __launch_bounds__(256) void loss_gather_kernel(LossArgs a) {
  const int r = blockIdx.x;
  if (r >= a.count[0]) return;
  const int t = a.rows[r];
  if (!MOE_CHECK(t >= 0 && t < a.T, 701)) return;
  const uint4* src = reinterpret_cast<const uint4*>(a.h + static_cast<size_t>(t) * a.d);
  uint4* dst = reinterpret_cast<uint4*>(a.hc + static_cast<size_t>(r) * a.d);
  for (int c = threadIdx.x; c < a.d / 8; c += 256) dst[c] = src[c];
}

// ------------------------------------------------------------------ logits

// The forward's grouped-GEMM pipeline: 8 MFMA waves (2 x 4) + 4 load waves, a
// ring of 5 stages of 32 K (all of the LDS).
using LP = Pipe<FMT_BF16, LT, LT, 5, 2, ACC_TIED, 8, 4>;
constexpr int LTHREADS = 768;
constexpr int LMI = LP::MI, LNJ = LP::NJ;

constexpr float NEG_INF = -__builtin_inff();

// Forward epilogue: per row of the tile (m, s) = (max, sum exp(l - m)) over its
// columns, and the label's logit where the label is one of them.
template <int NSUBC>
__device__ __forceinline__ void stats_epilogue(const LossArgs& a, const f32x4 (&acc)[LMI][LNJ], uint8_t* lds, int vt,
                                               RowTile rt, int ncol) {
  float2(*red)[LT] = reinterpret_cast<float2(*)[LT]>(lds);                 // [4][256]
  int* lab = reinterpret_cast<int*>(lds + 4 * LT * sizeof(float2));        // [256]
  const int w = wave_id(), lane = threadIdx.x & 63, lr = lane & 15, lg = lane >> 4, wm = w % 2, wn = w / 2;
  wait_vm_lgkm0<0>();
  block_barrier();   // every wave is done with the stage ring
  if (w >= LP::N_COMPUTE) {
    const int r = threadIdx.x - 64 * LP::N_COMPUTE;
    int l = -1;
    if (r < rt.rows) {
      const int t = a.rows[rt.row0 + r];
      if (MOE_CHECK(t >= 0 && t < a.T, 702)) l = a.labels[t] - vt * LT;
    }
    lab[r] = l;
  } else {
#pragma unroll
    for (int i = 0; i < NSUBC; ++i) {
      float m = NEG_INF;
#pragma unroll
      for (int j = 0; j < LNJ; ++j)
#pragma unroll
        for (int e = 0; e < 4; ++e)
          if (64 * wn + 16 * j + 4 * lg + e < ncol) m = fmaxf(m, acc[i][j][e]);
      m = fmaxf(m, __shfl_xor(m, 16));
      m = fmaxf(m, __shfl_xor(m, 32));
      const float mb = m == NEG_INF ? 0.f : m;   // no column, or all of them -inf: the sum is 0
      float s = 0.f;
#pragma unroll
      for (int j = 0; j < LNJ; ++j)
#pragma unroll
        for (int e = 0; e < 4; ++e)
          if (64 * wn + 16 * j + 4 * lg + e < ncol) s += __expf(acc[i][j][e] - mb);
      s += __shfl_xor(s, 16);
      s += __shfl_xor(s, 32);
      if (lg == 0) red[wn][16 * (2 * i + wm) + lr] = make_float2(m, s);
    }
  }
  wait_vm_lgkm0<0>();
  block_barrier();
  if (static_cast<int>(threadIdx.x) < rt.rows) {
    const int r = threadIdx.x;
    float m = red[0][r].x;
#pragma unroll
    for (int k = 1; k < 4; ++k) m = fmaxf(m, red[k][r].x);
    float s = 0.f;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const float2 p = red[k][r];
      s += p.x == NEG_INF ? p.y : p.y * __expf(p.x - m);
    }
    a.part[static_cast<size_t>(rt.row0 + r) * ceil_div(a.V, LT) + vt] = make_float2(m, s);
  }
  if (w >= LP::N_COMPUTE) return;
#pragma unroll
  for (int i = 0; i < NSUBC; ++i) {
    const int row = 16 * (2 * i + wm) + lr;
    if (row >= rt.rows) continue;
    const int l = lab[row];
    if (l < 0 || l >= ncol || l / 64 != wn || l / 4 % 4 != lg) continue;
#pragma unroll
    for (int j = 0; j < LNJ; ++j)
#pragma unroll
      for (int e = 0; e < 4; ++e)
        if (l % 64 / 16 == j && l % 4 == e) a.zlab[rt.row0 + row] = acc[i][j][e];
  }
}

// Backward epilogue: the tile of G, through LDS (whole lines per store).
template <int NSUBC>
__device__ __forceinline__ void grad_epilogue(const LossArgs& a, const f32x4 (&acc)[LMI][LNJ], uint8_t* lds, int vt,
                                              RowTile rt, int ncol) {
  constexpr int PITCH = LT * 2 + 16;   // padded rows: the 16 rows of a subtile hit different banks
  static_assert(LT * PITCH + LT * 16 <= 5 * LP::STAGE_BYTES, "tile and row data fit the stage ring");
  float4* rd = reinterpret_cast<float4*>(lds + LT * PITCH);   // lse, dloss + dlse, dloss, label's column (bits)
  const int w = wave_id(), lane = threadIdx.x & 63, lr = lane & 15, lg = lane >> 4, wm = w % 2, wn = w / 2;
  wait_vm_lgkm0<0>();
  block_barrier();   // every wave is done with the stage ring
  if (w >= LP::N_COMPUTE) {
    const int r = threadIdx.x - 64 * LP::N_COMPUTE;
    float4 v = make_float4(0.f, 0.f, 0.f, __int_as_float(-1));
    if (r < rt.rows) {
      const int t = a.rows[rt.row0 + r];
      if (MOE_CHECK(t >= 0 && t < a.T, 703)) {
        const float dl = a.dloss[t];
        v = make_float4(a.lse[t], a.dlse != nullptr ? dl + a.dlse[t] : dl, dl,
                        __int_as_float(a.labels[t] - a.v_first - vt * LT));
      }
    }
    rd[r] = v;
  }
  wait_vm_lgkm0<0>();
  block_barrier();
  if (w < LP::N_COMPUTE) {
#pragma unroll
    for (int i = 0; i < NSUBC; ++i) {
      const int row = 16 * (2 * i + wm) + lr;
      const float4 v = rd[row];
      const int l = __float_as_int(v.w);
#pragma unroll
      for (int j = 0; j < LNJ; ++j) {
        const int col = 64 * wn + 16 * j + 4 * lg;
        float g[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          g[e] = v.y * __expf(acc[i][j][e] - v.x);
          if (col + e == l) g[e] -= v.z;
          if (col + e >= ncol) g[e] = 0.f;
        }
        *reinterpret_cast<uint2*>(lds + row * PITCH + col * 2) = pack_bf16x4(g[0], g[1], g[2], g[3]);
      }
    }
  }
  wait_vm_lgkm0<0>();
  block_barrier();
  store_tile_from_lds<LT, PITCH, LTHREADS>(lds, rt.rows, LT, a.g + static_cast<size_t>(rt.row0) * a.ldg + vt * LT, a.ldg);
}

template <bool GRAD>
__global__ __launch_bounds__(LTHREADS, 1) void loss_logits_kernel(LossArgs a) {
  __shared__ __attribute__((aligned(1024))) uint8_t ring_lds[5 * LP::STAGE_BYTES];
  const int count = a.count[0];
  if (!MOE_CHECK(count >= 0 && count <= a.T, 704)) return;
  const int nm = row_tiles(count);
  int mt, vt;
  if (!loss_tile(nm, ceil_div(a.v_len, LT), mt, vt)) return;
  const RowTile rt = row_tile(count, nm, mt);
  const int v0 = a.v_first + vt * LT, ncol = min(LT, a.V - v0);
  const uint32_t ld = a.d * 2;

  auto make_pipe = [&]() {
    LP p;
    // rows past the tile's: an offset past the resource, so their loads
    // return zeros without touching memory
    if constexpr (GRAD) {
      p.init(make_rsrc(a.hc + static_cast<size_t>(rt.row0) * a.d, rt.rows * ld),
             [&](int r) { return static_cast<uint32_t>((r < rt.rows ? r : rt.rows) * ld); },
             make_rsrc(a.w + static_cast<size_t>(v0) * a.d, ncol * ld),
             [&](int r) { return static_cast<uint32_t>(r * ld); }, make_rsrc(a.w, 0), [](int) { return 0u; });
    } else {
      p.init(make_rsrc(a.h, a.T * ld),
             [&](int r) {
               const int t = r < rt.rows ? a.rows[rt.row0 + r] : a.T;
               return static_cast<uint32_t>((MOE_CHECK(t >= 0 && t <= a.T, 705) ? t : a.T) * ld);
             },
             make_rsrc(a.w + static_cast<size_t>(v0) * a.d, ncol * ld),
             [&](int r) { return static_cast<uint32_t>(r * ld); }, make_rsrc(a.w, 0), [](int) { return 0u; });
    }
    p.nks = a.d / 32;
    return p;
  };

  const Ring<5> ring = make_ring<5, LP::STAGE_BYTES>(ring_lds);
  const int w = wave_id(), wn = w / 2;
  const WRows<0> wr{16 * LNJ * wn};
  const int sub = (rt.rows + 15) / 16;
  // a wave row whose last subtile lies past the rows computes one fewer
  const bool short_row = w % 2 + 2 * ((sub + 1) / 2 - 1) >= sub;
  auto tile = [&]<int NSUB, int NSUBC>() {
    f32x4 acc[LMI][LNJ];
    zero_acc(acc);
    pipe_mainloop_ws<LP, NSUB, NSUBC>(make_pipe(), ring.s, a.d / 32, wr, acc);
    if constexpr (GRAD)
      grad_epilogue<NSUBC>(a, acc, ring_lds, vt, rt, ncol);
    else
      stats_epilogue<NSUBC>(a, acc, ring_lds, vt, rt, ncol);
  };
  dispatch_rows<LMI, 2>(rt.rows, [&]<int NSUB>() {
    if (short_row)
      tile.template operator()<NSUB, NSUB - 1>();
    else
      tile.template operator()<NSUB, NSUB>();
  });
}

// Joins a row's tiles, one wave per row: lane k takes tiles k, k + 64, ..., and
// a butterfly joins the lanes (max and rescaled sum: the same in either order).
__global__ __launch_bounds__(256) void loss_finish_kernel(LossArgs a) {
  const int count = a.count[0];
  const int r = blockIdx.x * 4 + wave_id(), lane = threadIdx.x & 63;
  if (r >= count) return;
  const int nv = ceil_div(a.V, LT);
  const float2* p = a.part + static_cast<size_t>(r) * nv;
  auto join = [](float2 p, float2 q) {
    const float m = fmaxf(p.x, q.x);
    const float sp = p.x == NEG_INF ? p.y : p.y * expf(p.x - m);
    const float sq = q.x == NEG_INF ? q.y : q.y * expf(q.x - m);
    return make_float2(m, sp + sq);
  };
  float2 v = make_float2(NEG_INF, 0.f);
#pragma unroll 4
  for (int t = lane; t < nv; t += 64) v = join(v, p[t]);
#pragma unroll
  for (int off = 32; off >= 1; off >>= 1) v = join(v, make_float2(__shfl_xor(v.x, off), __shfl_xor(v.y, off)));
  if (lane != 0) return;
  const float lse = v.x + logf(v.y);
  const int t = a.rows[r];
  if (!MOE_CHECK(t >= 0 && t < a.T, 706)) return;
  a.lse[t] = lse;
  a.loss[t] = lse - a.zlab[r];
}

// ------------------------------------------------------------------ dh = G w

// Split s of the piece: its columns k0 .. k0 + len - 1 (a multiple of 64 but
// for the last).
struct Run {
  int k0, len;
};
__device__ __forceinline__ Run split_run(int n, int splits, int s) {
  const int per = ((n + splits - 1) / splits + 63) / 64 * 64;
  return {s * per, max(0, min(per, n - s * per))};
}

__global__ __launch_bounds__(bt::THREADS, 1) void loss_dh_kernel(LossArgs a) {
  using namespace bt;
  __shared__ __attribute__((aligned(1024))) uint8_t ring[NSTG * STB];
  const int count = a.count[0];
  if (!MOE_CHECK(count >= 0 && count <= a.T, 707)) return;
  const int nm = row_tiles(count), nn = ceil_div(a.d, BT);
  int mt, ns;
  if (!loss_tile(nm, nn * a.splits, mt, ns)) return;
  const int s = ns / nn, n0 = (ns - s * nn) * BT;
  const RowTile rt = row_tile(count, nm, mt);
  const Run run = split_run(a.v_len, a.splits, s);
  const uint32_t ldg = a.ldg * 2, ldw = a.d * 2;
  const int nk = ceil_div(run.len, 32);
  f32x4 acc[MI][NJ];
  zero_acc(acc);
  if (wave_id() >= NMW) {
    // G's columns past V are zero, w's rows past V lie past the resource
    const Opnd oa = opnd_kc(make_rsrc(a.g + static_cast<size_t>(rt.row0) * a.ldg + run.k0, rt.rows * ldg - run.k0 * 2),
                            [&](int m) { return static_cast<uint32_t>((m < rt.rows ? m : rt.rows) * ldg); });
    const Opnd ob = opnd_ko(make_rsrc(a.w + static_cast<size_t>(a.v_first + run.k0) * a.d, run.len * ldw), ldw, n0);
    mainloop_pa(ring, oa, ob, nk, acc);
    return;
  }
  with_row_subtiles(rt.rows, [&]<int NS>() { mainloop_pa<NS>(ring, Opnd{}, Opnd{}, nk, acc); });
  const int w = wave_id(), lane = threadIdx.x & 63, wm = w % 2, wn = w / 2;
  const bool first = a.v_first == 0;
#pragma unroll
  for (int i = 0; i < MI; ++i) {
    const int row = 16 * (2 * i + wm) + (lane & 15);
    if (row >= rt.rows) continue;
    float* dst = a.acc + (static_cast<size_t>(s) * a.T + rt.row0 + row) * a.d;
#pragma unroll
    for (int j = 0; j < NJ; ++j) {
      const int col = n0 + 64 * wn + 16 * j + 4 * (lane >> 4);
      if (col >= a.d) continue;
      f32x4* p = reinterpret_cast<f32x4*>(dst + col);
      *p = first ? acc[i][j] : *p + acc[i][j];
    }
  }
}

// dh[t] = the sum of its row's splits, in order; zero for a token that is no row.
__global__ __launch_bounds__(256) void loss_dh_out_kernel(LossArgs a) {
  const size_t t = blockIdx.x;
  const int r = a.pos[t];
  if (!MOE_CHECK(r >= -1 && r < a.T, 708)) return;
  for (int c = 4 * threadIdx.x; c < a.d; c += 1024) {
    f32x4 v = {0.f, 0.f, 0.f, 0.f};
    if (r >= 0)
      for (int s = 0; s < a.splits; ++s)
        v += *reinterpret_cast<const f32x4*>(a.acc + (static_cast<size_t>(s) * a.T + r) * a.d + c);
    if (a.dh_fmt == FMT_F32)
      *reinterpret_cast<f32x4*>(static_cast<float*>(a.dh) + t * a.d + c) = v;
    else
      *reinterpret_cast<uint2*>(static_cast<uint16_t*>(a.dh) + t * a.d + c) = pack_bf16x4(v[0], v[1], v[2], v[3]);
  }
}

// ------------------------------------------------------------------ dw = G^T h

// Both operands K-outer (K: the rows): the load waves keep four stages of the
// ring of five ahead, two of them landed before each barrier.
__device__ __forceinline__ void mainloop_ko(uint8_t* ring, const bt::Opnd& a, const bt::Opnd& b, int nk,
                                            f32x4 (&acc)[bt::MI][bt::NJ]) {
  using namespace bt;
  const int w = wave_id();
  if (nk <= 0) return;
  if (w >= NMW) {
    for (int s = 0; s < 4 && s < nk; ++s) issue_stage(a, b, ring + s * STB, s);
    if (nk >= 4)
      wait_vm_lgkm0<2 * NLS>();   // stages 0 and 1
    else
      wait_vm_lgkm0<0>();
    for (int ks = 0; ks < nk; ++ks) {
      block_barrier();
      if (ks + 4 < nk) {
        issue_stage(a, b, ring + (ks + 4) % NSTG * STB, ks + 4);
        wait_vm_lgkm0<2 * NLS>();   // stage ks + 2
      } else {
        wait_vm_lgkm0<0>();
      }
    }
    return;
  }
  const int wm = w % 2, wn = w / 2;
  KoLane kl = ko_lane();
  i32x4 wf[NJ], xf;
  block_barrier();   // stages 0 and 1 have landed
#pragma unroll
  for (int j = 0; j < NJ; ++j) wf[j] = frag_ko(ring + OPB, 64 * wn + 16 * j, kl);
  xf = frag_ko(ring, 16 * wm, kl);
  acc_fence(acc);
  for (int ks = 0; ks < nk; ++ks) {
    asm volatile("" : "+v"(kl.base), "+v"(kl.y));
    const uint8_t* sa = ring + ks % NSTG * STB;
#pragma unroll
    for (int i = 0; i < MI; ++i) {
      i32x4 xn;
      if (i + 1 < MI) xn = frag_ko(sa, 16 * (2 * (i + 1) + wm), kl);
      __builtin_amdgcn_sched_barrier(0);
#pragma unroll
      for (int j = 0; j < NJ; ++j) mfma_bf16_tied(acc[i][j], wf[j], xf);
      __builtin_amdgcn_sched_barrier(0);
      if (i + 1 < MI) xf = xn;
    }
    if (ks + 1 < nk) {
      const uint8_t* na = ring + (ks + 1) % NSTG * STB;
#pragma unroll
      for (int j = 0; j < NJ; ++j) wf[j] = frag_ko(na + OPB, 64 * wn + 16 * j, kl);
      xf = frag_ko(na, 16 * wm, kl);
      block_barrier();
    }
  }
  acc_fence(acc);
}

__global__ __launch_bounds__(bt::THREADS, 1) void loss_dw_kernel(LossArgs a) {
  using namespace bt;
  __shared__ __attribute__((aligned(1024))) uint8_t ring[NSTG * STB];
  const int count = a.count[0];
  if (!MOE_CHECK(count >= 0 && count <= a.T, 709)) return;
  int vt, nt;
  if (!loss_tile(ceil_div(a.v_len, BT), ceil_div(a.d, BT), vt, nt)) return;
  const int n0 = nt * BT, v0 = a.v_first + vt * BT, vrows = min(BT, a.V - v0), ncols = min(BT, a.d - n0);
  const uint32_t ldg = a.ldg * 2, ldh = a.d * 2;
  const int nk = ceil_div(count, 32);
  f32x4 acc[MI][NJ];
  zero_acc(acc);
  if (wave_id() >= NMW) {
    const Opnd oa = opnd_ko(make_rsrc(a.g, count * ldg), ldg, vt * BT);
    const Opnd ob = opnd_ko(make_rsrc(a.hc, count * ldh), ldh, n0);
    mainloop_ko(ring, oa, ob, nk, acc);
  } else {
    mainloop_ko(ring, Opnd{}, Opnd{}, nk, acc);
  }
  const int w = wave_id(), lane = threadIdx.x & 63, lr = lane & 15, lg = lane >> 4, wm = w % 2, wn = w / 2;
  wait_vm_lgkm0<0>();
  block_barrier();   // every wave is done with the ring
  if (a.dw_fmt == FMT_BF16) {
    constexpr int PITCH = BT * 2 + 16;
    if (w < NMW) {
#pragma unroll
      for (int i = 0; i < MI; ++i)
#pragma unroll
        for (int j = 0; j < NJ; ++j)
          *reinterpret_cast<uint2*>(ring + (16 * (2 * i + wm) + lr) * PITCH + (64 * wn + 16 * j + 4 * lg) * 2) =
              pack4(acc[i][j]);
    }
    wait_vm_lgkm0<0>();
    block_barrier();
    store_tile_from_lds<BT, PITCH, THREADS>(ring, vrows, ncols,
                                            static_cast<uint16_t*>(a.dw) + static_cast<size_t>(v0) * a.d + n0, a.d);
    return;
  }
  // fp32: rows 0-127, then 128-255
  constexpr int PITCH = BT * 4 + 16;
  static_assert(128 * PITCH <= NSTG * STB, "half a tile fits the ring");
#pragma unroll
  for (int half = 0; half < 2; ++half) {
    if (half > 0) {
      wait_vm_lgkm0<0>();
      block_barrier();
    }
    if (w < NMW) {
#pragma unroll
      for (int i = 0; i < MI / 2; ++i)
#pragma unroll
        for (int j = 0; j < NJ; ++j)
          *reinterpret_cast<f32x4*>(ring + (16 * (2 * i + wm) + lr) * PITCH + (64 * wn + 16 * j + 4 * lg) * 4) =
              acc[i + half * MI / 2][j];
    }
    wait_vm_lgkm0<0>();
    block_barrier();
    float* dst = static_cast<float*>(a.dw) + static_cast<size_t>(v0 + 128 * half) * a.d + n0;
    for (int idx = threadIdx.x; idx < 128 * 64; idx += THREADS) {
      const int r = idx / 64, c = 4 * (idx % 64);
      if (128 * half + r < vrows && c < ncols)
        *reinterpret_cast<f32x4*>(dst + static_cast<size_t>(r) * a.d + c) =
            *reinterpret_cast<const f32x4*>(ring + r * PITCH + c * 4);
    }
  }
}

}  // namespace

MOE_DEBUG_FILE(loss)

int loss_splits(long long T, long long d, long long piece) {
  // the split count with the least of: rounds of 256 tiles at about 0.9 us per
  // 32-column step, and the splits' fp32 rows written and read at 4 TB/s
  const long long tiles = ((T + LT - 1) / LT) * ((d + LT - 1) / LT);
  int best = 1;
  double least = 0;
  for (int s = 1; s <= 64 && s * 256 <= piece; ++s) {
    const double rounds = static_cast<double>((tiles * s + 255) / 256);
    const double steps = static_cast<double>((piece + s - 1) / s + 31) / 32;
    const double us = rounds * steps * 0.9 + static_cast<double>(s) * T * d * 8 / 4e6;
    if (s == 1 || us < least) {
      best = s;
      least = us;
    }
  }
  return best;
}

hipError_t launch_loss_rows(const LossArgs& a, hipStream_t s) {
  hipLaunchKernelGGL(loss_rows_kernel, dim3(1), dim3(1024), 0, s, a);
  return hipGetLastError();
}

hipError_t launch_loss_forward(const LossArgs& a, hipStream_t s) {
  hipLaunchKernelGGL(loss_logits_kernel<false>, dim3(loss_grid(ceil_div(a.T, LT), ceil_div(a.v_len, LT))),
                     dim3(LTHREADS), 0, s, a);
  hipLaunchKernelGGL(loss_finish_kernel, dim3(ceil_div(a.T, 4)), dim3(256), 0, s, a);
  return hipGetLastError();
}

hipError_t launch_loss_gather(const LossArgs& a, hipStream_t s) {
  if (a.T > 0) hipLaunchKernelGGL(loss_gather_kernel, dim3(a.T), dim3(256), 0, s, a);
  return hipGetLastError();
}

// One piece: G, its part of dh, its rows of dw.
hipError_t launch_loss_piece(const LossArgs& a, hipStream_t s) {
  const long long nm = ceil_div(a.T, LT), nv = ceil_div(a.v_len, LT), nn = ceil_div(a.d, LT);
  if (a.T > 0) {
    hipLaunchKernelGGL(loss_logits_kernel<true>, dim3(loss_grid(nm, nv)), dim3(LTHREADS), 0, s, a);
    hipLaunchKernelGGL(loss_dh_kernel, dim3(loss_grid(nm, nn * a.splits)), dim3(bt::THREADS), 0, s, a);
  }
  hipLaunchKernelGGL(loss_dw_kernel, dim3(loss_grid(nv, nn)), dim3(bt::THREADS), 0, s, a);
  return hipGetLastError();
}

hipError_t launch_loss_dh(const LossArgs& a, hipStream_t s) {
  if (a.T > 0) hipLaunchKernelGGL(loss_dh_out_kernel, dim3(a.T), dim3(256), 0, s, a);
  return hipGetLastError();
}

}  // namespace moe
