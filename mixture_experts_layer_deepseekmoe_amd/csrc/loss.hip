// Cross entropy over a large vocabulary, without keeping the logits:
//
//   l_tv = h_t . w_v,  lse_t = log sum_v exp l_tv,  loss_t = lse_t - l_t,label
//   G_tv = (dloss_t + dlse_t) exp(l_tv - lse_t) - dloss_t [v = label_t]
//   dh = G w,  dw = G^T h
//
// forward   256 x 256 tiles of logits (64 entries for few tokens) stay in
//           the accumulators; a tile leaves one (max, sum of exponentials) per
//           row, which a second kernel joins.
// backward  the vocabulary in pieces: the piece's logits are computed again,
//           turned into G (bf16, a piece of at most 512 MB) in the epilogue, and
//           multiplied into dh (fp32, added up over the pieces) and the piece's
//           rows of dw.
//
// Only tokens with a label in [0, V) are rows of these products; the others
// (their hidden rows may hold anything) cost nothing, and their loss, lse and
// dh are zero.
//
// The large products are bound by the matrix cores at the clock the card's power
// holds (1.75-1.95 GHz; 76% of the cycles in the logits' kernel are MFMAs).
// 4096 tokens, a quarter ignored, d = 7168, V = 65536 (2.89 TFLOP each): logits 2.05
// ms (1.41 PFLOP/s; with the G epilogue 2.1), dh 2.25-2.4 ms (1.2-1.3), dw 2.5 (1.15).
// Library products of the same with 4096 rows: 1.23-1.26, 0.92-0.94, 0.92-1.06 on
// operands laid out as these are.  Few tokens are bound by reading w once.
//
// Products are bf16 with fp32 accumulation; statistics and dh's sums are fp32.  G
// is the operand of the two products that follow, in bf16.  For a gradient in fp32
// it is a pair of bf16 values, what the first rounds off in the second (2^-16 of
// an element is left): the product runs once for each, the second's sums added
// to the first's (4096 tokens, a quarter ignored, d = 7168, V = 65536, both gradients: 14.6
// ms against 8.85 in bf16; d = 2048, none ignored: 5.6 against 3.5).
// For a gradient in bf16, G is rounded to bf16 once (at most 2^-8 of an element), an
// error of the size of the output's own rounding.  The label's element outweighs
// the rest of its row, so its rounding is most of that error and, with few rows,
// does not average out:
//   dh   each row's rounding error at its label times the label's row of w is
//        added in fp32 where dh is written;
//   dw   up to 64 rows are summed with their rounding errors (LOSS_LO_ROWS); of
//        more, a tile's K-steps are followed by those of its labels (LabelSteps);
//   both G is held over the mantissa of the largest dloss: with the equal
//        weights of a mean the label's elements are p - 1, near a power of two,
//        and not all off by the one rounding of the weight.
// Against 64 bits, normwise: 2e-6 in fp32; 1.65e-3 in bf16, the outputs' own
// rounding (2.4e-3 without these, up to 2.9e-3 for few rows; 2.2e-3 of dw without its
// labels' steps).  They cost 4 us of 71 (207 rows, 10007 entries, d = 512) and 1% of the
// large products.  The labels' steps: a pair to a tile for 4096 tokens, a quarter
// ignored, 65536 entries, 0.3% (8.80 / 8.77 ms for d = 7168); 16 pairs beside a tile's
// own 64 for 4096 rows of 1000 entries, 199 / 149 us (d = 256).
#include "around.hpp"
#include "dense_core.hpp"

namespace moe {

namespace {

constexpr int LT = LOSS_TILE;
constexpr int NXCDS = 8;
constexpr float INF = __builtin_inff(), NEG_INF = -INF;

// The tiles of nm x nn that this block takes.  They are walked in groups of 8
// m-tiles (m fastest), so that the 32 tiles an XCD's CUs hold at once share 8
// row blocks and 4 column blocks in its L2; XCD x (blocks x, x + 8, ...) has a
// contiguous eighth of the walk, and its P blocks take every P-th tile of that.
struct TileWalk {
  int nm, nn;
  long long j0, n;   // the XCD's first tile and its number of them
  int l, P;
  __device__ __forceinline__ TileWalk(int nm_, int nn_) : nm(nm_), nn(nn_) {
    const long long total = static_cast<long long>(nm) * nn, chunk = (total + NXCDS - 1) / NXCDS;
    j0 = blockIdx.x % NXCDS * chunk;
    n = max(0LL, min(chunk, total - j0));
    l = blockIdx.x / NXCDS;
    P = gridDim.x / NXCDS;
  }
  __device__ __forceinline__ int count() const { return l < n ? static_cast<int>((n - l + P - 1) / P) : 0; }
  __device__ __forceinline__ void tile(int i, int& m, int& k) const {
    constexpr int GM = 8;
    const long long j = j0 + l + static_cast<long long>(i) * P;
    const int per = GM * nn, g = static_cast<int>(j / per), rem = static_cast<int>(j - static_cast<long long>(g) * per);
    const int gm = min(GM, nm - g * GM);
    m = g * GM + rem % gm;
    k = rem / gm;
  }
};
constexpr int NBLOCKS = 256;   // one per CU
inline unsigned loss_grid(long long nm, long long nn) {
  const long long per = (nm * nn + NXCDS - 1) / NXCDS;
  return static_cast<unsigned>(NXCDS * (per < NBLOCKS / NXCDS ? per : NBLOCKS / NXCDS));
}

// The rows in n nearly equal tiles of `per` rows (whole 16-row subtiles; the last
// takes what is left, at least one row): of at most 256 rows, and of down to 64
// while the tiles, with nn column tiles, still fit one round of the CUs (207
// rows, 10007 entries, d = 512, forward + backward: 90 -> 69 us; 256 rows over
// 50001 entries in two rounds of 128-row tiles: 197 -> 259 us).
struct RowTile {
  int row0, rows;
};
struct RowCut {
  int n, per, count;
  __device__ __forceinline__ RowCut(int count_, int nn) : count(count_) {
    const int least = (count + LT - 1) / LT, most = (count + 63) / 64;
    const int want = max(least, min(most, NBLOCKS / nn));
    per = want > 0 ? ((count + want - 1) / want + 15) / 16 * 16 : LT;
    n = (count + per - 1) / per;
  }
  __device__ __forceinline__ RowTile tile(int m) const { return {m * per, min(per, count - m * per)}; }
};
__device__ __forceinline__ int padded_rows(int count) { return (count + LT - 1) / LT * LT; }

// Cost of s splits of dh's sum for nm x nn tiles: rounds of 256 tiles at about
// 0.75 us per 32-column step, and the splits' fp32 tiles written and read at
// about 4 TB/s.  The least cost (the fewest splits of equal ones) is taken; the
// limits are those of loss_acc_rows.  A step's time is that of 256 rows, and taken for
// fewer as well: with 0.3 us instead, forward + backward of 256 x 8000 x 1024 takes 87
// us instead of 82, of 207 x 10007 x 512 75 instead of 71; with 1.5 us 82 and 72, of 128
// x 16000 x 2048 115 instead of 118.
__device__ __forceinline__ float split_cost(int s, int nm, int nn, int piece) {
  const int tiles = nm * nn;   // below 2^17
  if (s > 1 && (s * LT > piece || s * tiles > LOSS_SPLIT_TILES)) return 1e30f;
  const float rounds = static_cast<float>((tiles * s + NBLOCKS - 1) / NBLOCKS);
  return rounds * static_cast<float>(((piece + s - 1) / s + 31) / 32) * 0.75f + static_cast<float>(s) * tiles * 0.13f;
}

// dh's row tiles: fine ones would read w's piece again for every 64 rows, which
// pays only where a piece is short.  Forward + backward with fine and with 256-row
// tiles, us: 207 x 10007 x 512 71, 78; 256 x 8000 x 1024 82, 91; 256 x 16000 x 1024 90, 98;
// 256 x 16000 x 4096 240, 239; beyond: 256 x 20000 x 4096 271, 265; 256 x 32000 x 4096 397,
// 373; 512 x 24000 x 2048 260, 251 (but 256 x 32000 x 1024 119, 125; and within,
// 128 x 8000 x 7168 282, 274).
__device__ __forceinline__ RowCut dh_cut(int count, int d, int piece) {
  return RowCut(count, piece <= 16384 ? min(4 * ceil_div(d, LT), NBLOCKS) : NBLOCKS);
}

// Rows of dw's sum.
__device__ __forceinline__ int k_rows(int count) { return count <= LOSS_LO_ROWS ? 2 * count : count; }

// ------------------------------------------------------------------ rows

// The tokens with a label in [0, V), in order (one block; 1024 tokens at a
// time).  Forward: the others' loss and lse are zero.  Backward: also the splits
// of dh's sum, and the scale that G is held over: the mantissa, in [1, 2), of
// the largest finite |dloss| of a row (the range of G stays as it is).
__global__ __launch_bounds__(1024) void loss_rows_kernel(LossArgs a) {
  __shared__ int wsum[16];
  const int w = threadIdx.x >> 6, lane = threadIdx.x & 63;
  int base = 0, top = 0;   // top: bits of the largest |dloss|
  for (int t0 = 0; t0 < a.T; t0 += 1024) {
    const int t = t0 + threadIdx.x;
    const int lab = t < a.T ? a.labels[t] : -1;
    const int wt = a.acc != nullptr && t < a.T ? __float_as_int(a.dloss[t]) & 0x7fffffff : 0;
    const bool ok = lab >= 0 && lab < a.V;
    if (ok && wt < 0x7f800000) top = max(top, wt);
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
  if (a.acc == nullptr) return;
#pragma unroll
  for (int off = 32; off >= 1; off >>= 1) top = max(top, __shfl_xor(top, off));
  if (lane == 0) wsum[w] = top;
  __syncthreads();
  if (w > 0) return;
#pragma unroll
  for (int k = 1; k < 16; ++k) top = max(top, wsum[k]);
  // one lane per number of splits
  int best = lane + 1;
  static_assert(LOSS_SPLITS == 64, "one lane each");
  float cost = split_cost(best, dh_cut(base, a.d, a.ldg).n, ceil_div(a.d, LT), a.ldg);
#pragma unroll
  for (int off = 32; off >= 1; off >>= 1) {
    const float c = __shfl_xor(cost, off);
    const int o = __shfl_xor(best, off);
    if (c < cost || (c == cost && o < best)) {
      cost = c;
      best = o;
    }
  }
  if (lane == 0) {
    a.count[1] = best;
    a.count[2] = (top & 0x007fffff) | 0x3f800000;
  }
}

// The rows whose label lies in tile k of the vocabulary, in order (four waves, a
// quarter of the tokens each: the rows before them are counted, then listed).
__device__ __forceinline__ void list_labels(const LossArgs& a, int k) {
  __shared__ int before[4], inside[4];
  const int w = wave_id(), lane = threadIdx.x & 63;
  const int per = (a.T + 255) / 256 * 64, t0 = w * per, t1 = min(a.T, t0 + per);
  auto tile_of = [&](int t) {
    const int lab = t < t1 ? a.labels[t] : -1;
    return lab >= 0 && lab < a.V ? lab / LT : -1;
  };
  int b = 0, n = 0;
#pragma unroll 4
  for (int t = t0 + lane; t < t1; t += 64) {
    const int x = tile_of(t);
    b += x >= 0 && x < k;
    n += x == k;
  }
#pragma unroll
  for (int off = 32; off >= 1; off >>= 1) {
    b += __shfl_xor(b, off);
    n += __shfl_xor(n, off);
  }
  if (lane == 0) {
    before[w] = b;
    inside[w] = n;
  }
  __syncthreads();
  const int first = before[0] + before[1] + before[2] + before[3];
  if (threadIdx.x == 0) a.lab_first[k] = first;
  if (threadIdx.x == 0 && k == ceil_div(a.V, LT) - 1)
    a.lab_first[k + 1] = first + inside[0] + inside[1] + inside[2] + inside[3];
  int at = first;
  for (int i = 0; i < w; ++i) at += inside[i];
  for (int t = t0 + lane; t - lane < t1; t += 64) {
    const bool hit = tile_of(t) == k;
    const unsigned long long m = __ballot(hit);
    if (hit) {
      const int o = at + __popcll(m & ((1ULL << lane) - 1)), r = a.pos[t];
      if (MOE_CHECK(o < a.T && r >= 0 && r < a.T, 710))
        a.lab_list[o] = static_cast<uint32_t>(r) << 8 | static_cast<uint32_t>(a.labels[t] % LT);
    }
    at += __popcll(m);
  }
}

// hc[r] = h[rows[r]], and dw's rows of few tokens once more; the blocks after
// those list the labels by tile.
__global__ __launch_bounds__(256) void loss_gather_kernel(LossArgs a) {
  const int r = blockIdx.x, count = a.count[0], lists = loss_k_rows(a.T);
  if (r >= lists) {
    if (count > LOSS_LO_ROWS) list_labels(a, r - lists);
    return;
  }
  if (r >= k_rows(count)) return;
  const int t = a.rows[r < count ? r : r - count];
  if (!MOE_CHECK(t >= 0 && t < a.T, 701)) return;
  const uint4* src = reinterpret_cast<const uint4*>(a.h + static_cast<size_t>(t) * a.d);
  uint4* dst = reinterpret_cast<uint4*>(a.hc + static_cast<size_t>(r) * a.d);
  for (int c = threadIdx.x; c < a.d / 8; c += 256) dst[c] = src[c];
}

// ------------------------------------------------------------------ logits

using Acc = f32x4[dense::MI][dense::NJ];   // a wave's accumulators (dense_core.hpp)

// What the epilogues need of a tile's rows, in SPARE after the waves' staging:
// one entry per row, written by the load waves.
//   forward   the label's column in the tile (or outside it)
//   backward  lse, dloss + dlse, dloss, and the label's column (bits)
constexpr int ROW_DATA = dense::SPARE + dense::NMW * dense::STAGING;
static_assert(ROW_DATA + LT * 16 <= dense::RING_BYTES && 4 * LT * 8 <= dense::NMW * dense::STAGING,
              "the forward's (max, sum) and the row data fit the spare buffer");

// Forward epilogue: per row of the tile (m, s) = (max, sum exp(l - m)) over its
// columns, and the label's logit where the label is one of them.  One barrier.
template <int NSUB>
__device__ __forceinline__ void stats_epilogue(const LossArgs& a, const Acc& acc, uint8_t* ring, int vt, RowTile rt,
                                               int ncol) {
  float2(*red)[LT] = reinterpret_cast<float2(*)[LT]>(ring + dense::SPARE);   // [4][256]
  const int* lab = reinterpret_cast<const int*>(ring + ROW_DATA);            // [256]
  const int w = wave_id(), lane = dense::fresh_lane(), lr = lane & 15, lg = lane >> 4, wm = w % 2, wn = w / 2;
  auto stats = [&]<bool FULL>() {   // FULL: all 256 columns are there
#pragma unroll
    for (int i = 0; i < NSUB; ++i) {
      float m = NEG_INF;
#pragma unroll
      for (int j = 0; j < dense::NJ; ++j)
#pragma unroll
        for (int e = 0; e < 4; ++e)
          if (FULL || 64 * wn + 16 * j + 4 * lg + e < ncol) m = fmaxf(m, acc[i][j][e]);
      m = fmaxf(m, __shfl_xor(m, 16));
      m = fmaxf(m, __shfl_xor(m, 32));
      const float mb = m == NEG_INF ? 0.f : m;   // no column, or all of them -inf: the sum is 0
      float s = 0.f;
#pragma unroll
      for (int j = 0; j < dense::NJ; ++j)
#pragma unroll
        for (int e = 0; e < 4; ++e)
          if (FULL || 64 * wn + 16 * j + 4 * lg + e < ncol) s += __expf(acc[i][j][e] - mb);
      s += __shfl_xor(s, 16);
      s += __shfl_xor(s, 32);
      if (lg == 0) red[wn][16 * (2 * i + wm) + lr] = make_float2(m, s);
    }
  };
  if (ncol == LT)
    stats.template operator()<true>();
  else
    stats.template operator()<false>();
  dense::wait_lgkm0();
  block_barrier();   // red and the row data are written
  const int r = 64 * w + lane;
  if (r < rt.rows) {
    float m = red[0][r].x;
#pragma unroll
    for (int k = 1; k < 4; ++k) m = fmaxf(m, red[k][r].x);
    float s = 0.f;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const float2 p = red[k][r];
      s += p.x == NEG_INF ? p.y : p.y * __expf(p.x - m);
    }
    if (MOE_CHECK(rt.row0 + r < a.T && vt < a.tiles, 713))
      a.part[static_cast<size_t>(rt.row0 + r) * a.tiles + vt] = make_float2(m, s);
  }
#pragma unroll
  for (int i = 0; i < NSUB; ++i) {
    const int row = 16 * (2 * i + wm) + lr;
    if (row >= rt.rows) continue;
    const int c = lab[row];
    if (c < 0 || c >= ncol || c / 64 != wn || c / 4 % 4 != lg) continue;
#pragma unroll
    for (int j = 0; j < dense::NJ; ++j)
#pragma unroll
      for (int e = 0; e < 4; ++e)
        if (c % 64 / 16 == j && c % 4 == e) a.zlab[rt.row0 + row] = acc[i][j][e];
  }
}

// What rounding x to bf16 leaves, nothing of what is not finite.
__device__ __forceinline__ float rounding_error(float x) {
  const float e = x - __uint_as_float(bf16x2(x, 0.f) << 16);
  return fabsf(e) < INF ? e : 0.f;
}

// Backward epilogue: the tile of G, its rows' errors at the label, and with
// PAIRS, or of few rows (one tile of 64), the errors of all.  One barrier.
template <int NSUB, bool PAIRS>
__device__ __forceinline__ void grad_epilogue(const LossArgs& a, const Acc& acc, uint8_t* ring, int vt, RowTile rt,
                                              int ncol, int count) {
  const float4* rd = reinterpret_cast<const float4*>(ring + ROW_DATA);
  const int w = wave_id(), lane = dense::fresh_lane(), lr = lane & 15, lg = lane >> 4, wm = w % 2, wn = w / 2;
  block_barrier();   // the row data are written
  auto store = [&]<bool FULL>() {   // FULL: all 256 columns are there
    float4 d;
    float gl = 0.f;   // G at the label, on the lane that has it
    int l = 0;
    dense::store_bf16_tile<NSUB>(
        ring, 64,
        [&](int i, int j) {
          const int col = 64 * wn + 16 * j + 4 * lg;
          if (j == 0) {
            d = rd[16 * (2 * i + wm) + lr];
            l = __float_as_int(d.w);
          }
          float g[4];
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            g[e] = d.y * __expf(acc[i][j][e] - d.x);
            if (!FULL && col + e >= ncol) g[e] = 0.f;
          }
          const int row = 16 * (2 * i + wm) + lr;
          if ((l & ~3) == col) {   // the label is one of the four
#pragma unroll
            for (int e = 0; e < 4; ++e)
              if ((l & 3) == e) {
                g[e] -= d.z;
                gl = g[e];
              }
          }
          if (j == dense::NJ - 1 && l >> 6 == wn && (l >> 2 & 3) == lg)
            a.lab_lo[rt.row0 + row] = rounding_error(gl);
          if constexpr (PAIRS || NSUB == 2) {
            if ((PAIRS || count <= LOSS_LO_ROWS) && row < rt.rows &&
                MOE_CHECK(count + rt.row0 + row < a.g_rows && vt * LT + col + 4 <= a.ldg, 714))
              *reinterpret_cast<uint2*>(a.g + static_cast<size_t>(count + rt.row0 + row) * a.ldg + vt * LT + col) =
                  dense::pack4(rounding_error(g[0]), rounding_error(g[1]), rounding_error(g[2]), rounding_error(g[3]));
          }
          return dense::pack4(g[0], g[1], g[2], g[3]);
        },
        [&](int row) -> uint16_t* {
          return row < rt.rows && MOE_CHECK(rt.row0 + row < a.g_rows && (vt + 1) * LT <= a.ldg, 715) ? a.g + static_cast<size_t>(rt.row0 + row) * a.ldg + vt * LT + 64 * wn : nullptr;
        });
  };
  if (ncol == LT)
    store.template operator()<true>();
  else
    store.template operator()<false>();
}

template <bool GRAD, bool PAIRS>
__global__ __launch_bounds__(dense::THREADS, 1) void loss_logits_kernel(LossArgs a) {
  __shared__ __attribute__((aligned(1024))) uint8_t ring[dense::RING_BYTES];
  const int count = a.count[0];
  if (!MOE_CHECK(count >= 0 && count <= a.T, 704)) return;
  const int nk = a.d / 32;
  const RowCut cut(count, ceil_div(a.v_len, LT));
  const TileWalk walk(cut.n, ceil_div(a.v_len, LT));
  const int n = walk.count();
  const uint32_t ld = a.d * 2;
  if (wave_id() >= dense::NMW) {
    const int r = threadIdx.x - 64 * dense::NMW;   // the tile row whose data this thread fetches
    dense::Opnd oa, ob;
    float4 rd;
    RowTile rt;
    float inv = 1.f;
    if constexpr (GRAD) inv = 1.f / __int_as_float(a.count[2]);
    auto head = [&](int i) {
      int mt, vt;
      walk.tile(i, mt, vt);
      rt = cut.tile(mt);
      const int v0 = a.v_first + vt * LT;
      // rows past the tile's: an offset past the resource, so their loads
      // return zeros without touching memory
      if constexpr (GRAD) {
        oa = dense::opnd_kc(make_rsrc(a.hc + static_cast<size_t>(rt.row0) * a.d, rt.rows * ld),
                            [&](int m) { return static_cast<uint32_t>((m < rt.rows ? m : rt.rows) * ld); });
      } else {
        oa = dense::opnd_kc(make_rsrc(a.h, a.T * ld), [&](int m) {
          const int t = m < rt.rows ? a.rows[rt.row0 + m] : a.T;
          return static_cast<uint32_t>((MOE_CHECK(t >= 0 && t <= a.T, 705) ? t : a.T) * ld);
        });
      }
      ob = dense::opnd_kc(make_rsrc(a.w + static_cast<size_t>(v0) * a.d, min(LT, a.V - v0) * ld),
                          [&](int m) { return static_cast<uint32_t>(m * ld); });
      dense::with_rows(rt.rows, [&]<int NSUB>() { dense::load_head<NSUB / 2>(ring, oa, ob, nk); });
      rd = make_float4(0.f, 0.f, 0.f, __int_as_float(-1));
      if (r < rt.rows) {
        const int t = a.rows[rt.row0 + r];
        if (MOE_CHECK(t >= 0 && t < a.T, 702)) {
          rd.w = __int_as_float(a.labels[t] - v0);
          if constexpr (GRAD) {
            rd.x = a.lse[t];
            rd.z = a.dloss[t] * inv;
            rd.y = a.dlse != nullptr ? rd.z + a.dlse[t] * inv : rd.z;
          }
        }
      }
    };
    if (n > 0) head(0);
    for (int i = 0; i < n; ++i) {
      dense::with_rows(rt.rows, [&]<int NSUB>() { dense::load_body<NSUB / 2>(ring, oa, ob, nk); });
      block_barrier();   // the tile's stages are read
      if constexpr (GRAD)
        reinterpret_cast<float4*>(ring + ROW_DATA)[r] = rd;
      else
        reinterpret_cast<int*>(ring + ROW_DATA)[r] = __float_as_int(rd.w);
      dense::wait_lgkm0();
      if constexpr (GRAD) block_barrier();
      if (i + 1 < n) head(i + 1);
      if constexpr (!GRAD) block_barrier();
    }
    return;
  }
  for (int i = 0; i < n; ++i) {
    int mt, vt;
    walk.tile(i, mt, vt);
    const RowTile rt = cut.tile(mt);
    const int ncol = min(LT, a.V - a.v_first - vt * LT);
    dense::with_rows(rt.rows, [&]<int NSUB>() {
      Acc acc;
      dense::mfma_loop<dense::KC, dense::KC, NSUB>(ring, nk, acc);
      block_barrier();   // the tile's stages are read
      if constexpr (GRAD)
        grad_epilogue<NSUB, PAIRS>(a, acc, ring, vt, rt, ncol, count);
      else
        stats_epilogue<NSUB>(a, acc, ring, vt, rt, ncol);
    });
  }
}

// ------------------------------------------------------------------ logits of few tokens

// Up to 64 tokens (scoring, decoding): the time is that of reading w once.  A
// block takes 64 entries of the vocabulary; its 8 waves share K, pairs of
// K-steps (the 128-byte lines of 64 rows) in turn, straight from memory into
// MFMA fragments, and add their partial logits through LDS in order.  Of up to 16
// tokens four such blocks fit a CU, of up to 32 two, else one (LDS), with a pair of
// every wave in flight (8 KB); the tile pipeline has one block to a CU and at most 64
// KB of w in flight, but its blocks share the hidden rows among 256 entries.  (Two pairs
// in flight per wave cost a block its place on the CU: 20 tokens 66 -> 71 us.)
//
// GRAD: the piece's G by the same rule, with its rows' rounding errors below it
// (there are at most 64 rows).  Every column of the tile is written: G's past V
// are zero.
constexpr int SV = LOSS_STREAM_TILE, STHREADS = 512;

template <int NT, bool GRAD>
__global__ __launch_bounds__(STHREADS) void loss_stream_kernel(LossArgs a) {
  static_assert(16 * NT <= LOSS_LO_ROWS, "all rows have their rounding errors");
  __shared__ float red[8][16 * NT][SV + 4];
  __shared__ int rows[16 * NT], labs[16 * NT];
  __shared__ float3 rd[GRAD ? 16 * NT : 1];   // lse, (dloss + dlse) / scale, dloss / scale
  const int w = wave_id(), lane = threadIdx.x & 63, lr = lane & 15, lg = lane >> 4;
  // the rows, as loss_rows_kernel lists them (one lane a token)
  const int lab = lane < a.T ? a.labels[lane] : -1;
  const bool ok = lab >= 0 && lab < a.V;
  const unsigned long long valid = __ballot(ok);
  const int count = __popcll(valid), at = __popcll(valid & ((1ULL << lane) - 1));
  if (!MOE_CHECK(a.T <= 16 * NT && count <= a.T && (GRAD ? (blockIdx.x + 1) * SV <= a.ldg : blockIdx.x < a.tiles), 716))
    return;
  if (w == 0 && ok) {
    rows[at] = lane;
    labs[at] = lab;
    if constexpr (GRAD) {
      const float inv = 1.f / __int_as_float(a.count[2]), dl = a.dloss[lane] * inv;
      rd[at] = make_float3(a.lse[lane], a.dlse != nullptr ? dl + a.dlse[lane] * inv : dl, dl);
    }
  }
  if (!GRAD && blockIdx.x == 0 && w == 0) {
    if (ok)
      a.rows[at] = lane;
    else if (lane < a.T)
      a.loss[lane] = a.lse[lane] = 0.f;
    if (lane == 0) a.count[0] = count;
  }
  __syncthreads();
  if (count == 0) return;

  const int v0 = a.v_first + blockIdx.x * SV, nv = max(0, min(SV, a.V - v0));
  const uint32_t ld = a.d * 2;
  const rsrc_t rw = make_rsrc(a.w + static_cast<size_t>(v0) * a.d, nv * ld);   // entries past V: zeros
  const rsrc_t rh = make_rsrc(a.h, a.T * ld);
  uint32_t ow[4], oh[NT];
#pragma unroll
  for (int s = 0; s < 4; ++s) ow[s] = (16 * s + lr) * ld + 16 * lg;
#pragma unroll
  for (int t = 0; t < NT; ++t) oh[t] = (16 * t + lr < count ? rows[16 * t + lr] : a.T) * ld + 16 * lg;   // past: zeros
  f32x4 acc[NT][4];
#pragma unroll
  for (int t = 0; t < NT; ++t)
#pragma unroll
    for (int s = 0; s < 4; ++s) acc[t][s] = f32x4{0.f, 0.f, 0.f, 0.f};
  auto load = [](rsrc_t r, uint32_t off, uint32_t soff) {
    return __builtin_bit_cast(i32x4, __builtin_amdgcn_raw_buffer_load_b128(r, off, soff, 0));
  };
  const int np = a.d / 64;
#pragma unroll 2
  for (int p = w; p < np; p += 8) {
    i32x4 wf[2][4], hf[2][NT];
#pragma unroll
    for (int s = 0; s < 4; ++s)
#pragma unroll
      for (int k = 0; k < 2; ++k) wf[k][s] = load(rw, ow[s], 128 * p + 64 * k);
#pragma unroll
    for (int t = 0; t < NT; ++t)
#pragma unroll
      for (int k = 0; k < 2; ++k) hf[k][t] = load(rh, oh[t], 128 * p + 64 * k);
#pragma unroll
    for (int k = 0; k < 2; ++k)
#pragma unroll
      for (int t = 0; t < NT; ++t)
#pragma unroll
        for (int s = 0; s < 4; ++s) acc[t][s] = mfma_bf16(wf[k][s], hf[k][t], acc[t][s]);
  }
#pragma unroll
  for (int t = 0; t < NT; ++t)
#pragma unroll
    for (int s = 0; s < 4; ++s) *reinterpret_cast<f32x4*>(&red[w][16 * t + lr][16 * s + 4 * lg]) = acc[t][s];
  __syncthreads();
  // 16 lanes to a row, 4 columns each
  for (int r = threadIdx.x >> 4; r < count; r += STHREADS / 16) {
    const int c = 4 * (threadIdx.x & 15);
    f32x4 l = *reinterpret_cast<const f32x4*>(&red[0][r][c]);
#pragma unroll
    for (int k = 1; k < 8; ++k) l += *reinterpret_cast<const f32x4*>(&red[k][r][c]);
    if constexpr (GRAD) {
      const float3 q = rd[r];
      const int z = labs[r] - v0 - c;
      float g[4], lo[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        g[e] = c + e < nv ? q.y * __expf(l[e] - q.x) : 0.f;
        if (z == e) g[e] -= q.z;
        lo[e] = rounding_error(g[e]);
        if (z == e) a.lab_lo[r] = lo[e];
      }
      if (!MOE_CHECK(count + r < a.g_rows, 717)) continue;
      uint16_t* dst = a.g + static_cast<size_t>(r) * a.ldg + blockIdx.x * SV + c;
      *reinterpret_cast<uint2*>(dst) = dense::pack4(g[0], g[1], g[2], g[3]);
      *reinterpret_cast<uint2*>(dst + static_cast<size_t>(count) * a.ldg) = dense::pack4(lo[0], lo[1], lo[2], lo[3]);
      continue;
    }
    float m = NEG_INF;
#pragma unroll
    for (int e = 0; e < 4; ++e)
      if (c + e < nv) m = fmaxf(m, l[e]);
    m = wave_max_16(m);
    const float mb = m == NEG_INF ? 0.f : m;
    float s = 0.f;
#pragma unroll
    for (int e = 0; e < 4; ++e)
      if (c + e < nv) s += __expf(l[e] - mb);
#pragma unroll
    for (int off = 1; off < 16; off <<= 1) s += __shfl_xor(s, off);
    if (c == 0) a.part[static_cast<size_t>(r) * a.tiles + blockIdx.x] = make_float2(m, s);
    const int z = labs[r] - v0 - c;
#pragma unroll
    for (int e = 0; e < 4; ++e)
      if (z == e) a.zlab[r] = l[e];
  }
}

// Joins a row's tiles, WPR waves to a row: a thread takes every 64 WPR-th tile, a
// butterfly joins the lanes and the waves follow in order (max and rescaled
// sum: a butterfly's halves give the same).
template <int WPR>
__global__ __launch_bounds__(256) void loss_finish_kernel(LossArgs a) {
  __shared__ float2 s[4];
  const int count = a.count[0];
  const int w = wave_id(), lane = threadIdx.x & 63, r = blockIdx.x * (4 / WPR) + w / WPR;
  auto join = [](float2 p, float2 q) {
    const float m = fmaxf(p.x, q.x);
    const float sp = p.x == NEG_INF ? p.y : p.y * expf(p.x - m);
    const float sq = q.x == NEG_INF ? q.y : q.y * expf(q.x - m);
    return make_float2(m, sp + sq);
  };
  if (r < count) {
    const float2* p = a.part + static_cast<size_t>(r) * a.tiles;
    float2 v = make_float2(NEG_INF, 0.f);
#pragma unroll 4
    for (int t = 64 * (w % WPR) + lane; t < a.tiles; t += 64 * WPR) v = join(v, p[t]);
#pragma unroll
    for (int off = 32; off >= 1; off >>= 1) v = join(v, make_float2(__shfl_xor(v.x, off), __shfl_xor(v.y, off)));
    if (lane == 0) s[w] = v;
  }
  if constexpr (WPR > 1) __syncthreads();
  if (r >= count || lane != 0 || w % WPR != 0) return;
  float2 v = s[w];
#pragma unroll
  for (int k = 1; k < WPR; ++k) v = join(v, s[w + k]);
  const float lse = v.x + logf(v.y);
  const int t = a.rows[r];
  if (!MOE_CHECK(t >= 0 && t < a.T, 706)) return;
  a.lse[t] = lse;
  a.loss[t] = lse - a.zlab[r];
}

// ------------------------------------------------------------------ dh = G w

// Offset of the pairs' second values in G.
template <bool SECOND>
__device__ __forceinline__ size_t second_at(int count, int ldg) {
  return SECOND ? static_cast<size_t>(count) * ldg : 0;
}

// Split s of the piece: its columns k0 .. k0 + len - 1 (a multiple of 64 but
// for the last).
struct Run {
  int k0, len;
};
__device__ __forceinline__ Run split_run(int n, int splits, int s) {
  const int per = ((n + splits - 1) / splits + 63) / 64 * 64;
  return {s * per, max(0, min(per, n - s * per))};
}

// SECOND: of the pairs' second values, added to the sums of the first.
template <bool SECOND>
__global__ __launch_bounds__(dense::THREADS, 1) void loss_dh_kernel(LossArgs a) {
  __shared__ __attribute__((aligned(1024))) uint8_t ring[dense::RING_BYTES];
  const int count = a.count[0], splits = a.count[1];
  if (!MOE_CHECK(count >= 0 && count <= a.T && splits >= 1 && splits <= LOSS_SPLITS, 707)) return;
  const int nn = ceil_div(a.d, LT);
  const RowCut cut = dh_cut(count, a.d, a.ldg);
  const TileWalk walk(cut.n, nn * splits);
  const int n = walk.count();
  auto tile = [&](int i, RowTile& rt, Run& run, int& s, int& n0) {
    int mt, k;
    walk.tile(i, mt, k);
    s = k / nn;
    n0 = (k - s * nn) * LT;
    rt = cut.tile(mt);
    run = split_run(a.v_len, splits, s);
  };
  RowTile rt;
  Run run;
  int s, n0;
  if (wave_id() >= dense::NMW) {
    const uint32_t ldg = a.ldg * 2, ldw = a.d * 2;
    const uint16_t* g = a.g + second_at<SECOND>(count, a.ldg);
    dense::Opnd oa, ob;
    auto head = [&](int i) {
      tile(i, rt, run, s, n0);
      // G's columns past V are zero, w's rows past V lie past the resource
      oa = dense::opnd_kc(make_rsrc(g + static_cast<size_t>(rt.row0) * a.ldg + run.k0, rt.rows * ldg - run.k0 * 2),
                          [&](int m) { return static_cast<uint32_t>((m < rt.rows ? m : rt.rows) * ldg); });
      ob = dense::opnd_ko(make_rsrc(a.w + static_cast<size_t>(a.v_first + run.k0) * a.d, run.len * ldw), ldw, n0);
      dense::with_rows(rt.rows,
                       [&]<int NSUB>() { dense::load_head<NSUB / 2>(ring, oa, ob, ceil_div(run.len, 32)); });
    };
    if (n > 0) head(0);
    for (int i = 0; i < n; ++i) {
      dense::with_rows(rt.rows,
                       [&]<int NSUB>() { dense::load_body<NSUB / 2>(ring, oa, ob, ceil_div(run.len, 32)); });
      block_barrier();   // the tile's stages are read
      if (i + 1 < n) head(i + 1);
    }
    return;
  }
  const int w = wave_id(), wm = w % 2, wn = w / 2;
  const bool first = a.v_first == 0 && !SECOND;
  for (int t = 0; t < n; ++t) {
    tile(t, rt, run, s, n0);
    dense::with_rows(rt.rows, [&]<int NSUB>() {
      Acc acc;
      dense::mfma_loop<dense::KC, dense::KO, NSUB>(ring, ceil_div(run.len, 32), acc);
      block_barrier();   // the tile's stages are read
      const int lane = dense::fresh_lane();
#pragma unroll
      for (int i = 0; i < NSUB; ++i) {
        const int row = 16 * (2 * i + wm) + (lane & 15);
        if (row >= rt.rows) continue;
        if (!MOE_CHECK(static_cast<long long>(s) * padded_rows(count) + rt.row0 + row < a.acc_rows, 718)) continue;
        float* dst = a.acc + (static_cast<size_t>(s) * padded_rows(count) + rt.row0 + row) * a.d;
#pragma unroll
        for (int j = 0; j < dense::NJ; ++j) {
          const int col = n0 + 64 * wn + 16 * j + 4 * (lane >> 4);
          if (col >= a.d) continue;
          f32x4* p = reinterpret_cast<f32x4*>(dst + col);
          *p = first ? acc[i][j] : *p + acc[i][j];
        }
      }
    });
  }
}

// dh[t] = the sum of its row's splits, in order, and without pairs G's rounding
// error at the label; zero for a token that is no row.
__global__ __launch_bounds__(256) void loss_dh_out_kernel(LossArgs a) {
  const size_t t = blockIdx.x;
  const int r = a.pos[t], label = a.labels[t], rows = padded_rows(a.count[0]), splits = a.count[1];
  if (!MOE_CHECK(r >= -1 && r < a.T && splits <= LOSS_SPLITS &&
                     (r < 0 || (splits - 1LL) * rows + r < a.acc_rows), 708))
    return;
  const float scale = __int_as_float(a.count[2]), lo = r >= 0 && a.dh_fmt == FMT_BF16 ? a.lab_lo[r] : 0.f;
  const uint16_t* wl = a.w + static_cast<size_t>(r >= 0 ? label : 0) * a.d;
  for (int c = 4 * threadIdx.x; c < a.d; c += 1024) {
    f32x4 v = {0.f, 0.f, 0.f, 0.f};
    if (r >= 0) {
      const uint2 q = *reinterpret_cast<const uint2*>(wl + c);
#pragma unroll 8
      for (int s = 0; s < splits; ++s)
        v += *reinterpret_cast<const f32x4*>(a.acc + (static_cast<size_t>(s) * rows + r) * a.d + c);
      const f32x4 we = {__uint_as_float(q.x << 16), __uint_as_float(q.x & 0xffff0000u), __uint_as_float(q.y << 16),
                        __uint_as_float(q.y & 0xffff0000u)};
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const float x = lo * we[e];
        v[e] = scale * (fabsf(x) < INF ? v[e] + x : v[e]);   // an infinite w is in v already
      }
    }
    if (a.dh_fmt == FMT_F32)
      *reinterpret_cast<f32x4*>(static_cast<float*>(a.dh) + t * a.d + c) = v;
    else
      *reinterpret_cast<uint2*>(static_cast<uint16_t*>(a.dh) + t * a.d + c) = dense::pack4(v[0], v[1], v[2], v[3]);
  }
}

// ------------------------------------------------------------------ dw = G^T h

// The K-steps that follow a tile's own: what rounding took off G at its labels (in
// bf16), times those rows of h, 32 rows of the tile's list to a step.  The load
// waves write A's stage, zero but for each row's label, and gather B's from hc.
struct LabelSteps {
  int first, last;   // the tile's entries of the list
  __device__ __forceinline__ LabelSteps(const LossArgs& a, bool any, int tile, int count) {
    first = any ? a.lab_first[tile] : 0;
    last = any ? a.lab_first[tile + 1] : 0;
    if (!MOE_CHECK(first >= 0 && first <= last && last <= count, 711)) first = last;
  }
  __device__ __forceinline__ int pairs() const { return (last - first + 63) / 64; }

  // Load waves: this lane's entries of pair k, ahead of their use, and that pair
  // into the stages of steps s, s + 1 (hc's resource, columns from col0).
  static constexpr uint32_t NONE = ~0u;
  uint32_t e[2][dense::NLI];
  static __device__ __forceinline__ int k_row(int q) {   // as opnd_ko's
    return 2 * (wave_id() - dense::NMW + dense::NLW * q) + (threadIdx.x & 63) / 32;
  }
  __device__ __forceinline__ void fetch(const LossArgs& a, int k) {
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
      for (int q = 0; q < dense::NLI; ++q) {
        const int at = first + 64 * k + 32 * h + k_row(q);
        e[h][q] = at < last ? a.lab_list[at] : NONE;
      }
  }
  __device__ __forceinline__ void issue(const LossArgs& a, rsrc_t rh, uint8_t* ring, int s, int col0, int count) const {
    const int w = wave_id() - dense::NMW, lane = threadIdx.x & 63;
    auto chunk = [&](int q) __attribute__((always_inline)) { return (lane & 31) ^ dense::xko(k_row(q)); };
    auto ok = [&](uint32_t x) __attribute__((always_inline)) {
      return x != NONE && MOE_CHECK(static_cast<int>(x >> 8) < count, 712);
    };
    float lo[2][dense::NLI];
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
      for (int q = 0; q < dense::NLI; ++q) {
        const uint32_t x = e[h][q];
        lo[h][q] = ok(x) && (x & 255) >> 3 == static_cast<uint32_t>(chunk(q)) ? a.lab_lo[x >> 8] : 0.f;
      }
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
      for (int q = 0; q < dense::NLI; ++q) {
        const uint32_t c = e[h][q] & 255, v = bf16x2(lo[h][q], 0.f) << 16 * (c & 1), p = c >> 1 & 3;
        *reinterpret_cast<uint4*>(dense::stage(ring, s + h) + 1024 * (w + dense::NLW * q) + 16 * lane) =
            make_uint4(p == 0 ? v : 0, p == 1 ? v : 0, p == 2 ? v : 0, p == 3 ? v : 0);
      }
    dense::wait_lgkm0();   // written before a barrier says so
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
      for (int q = 0; q < dense::NLI; ++q) {
        const uint32_t x = e[h][q], r = ok(x) ? x >> 8 : static_cast<uint32_t>(count);   // past the resource: zeros
        dma16(rh, r * (a.d * 2u) + col0 * 2 + 16 * chunk(q), 0,
              dense::stage(ring, s + h) + dense::OPB + 1024 * (w + dense::NLW * q));
      }
  }
};
static_assert(dense::first_ops<4>() == dense::NLI, "as many DMA instructions as a pair's first half: load_body");

// SECOND: as for dh; fp32 only.
template <bool SECOND>
__global__ __launch_bounds__(dense::THREADS, 1) void loss_dw_kernel(LossArgs a) {
  using namespace dense;
  __shared__ __attribute__((aligned(1024))) uint8_t ring[dense::RING_BYTES];
  const int count = a.count[0];
  if (!MOE_CHECK(count >= 0 && count <= a.T, 709)) return;
  if (SECOND && count <= LOSS_LO_ROWS) return;   // the first product took both values
  const TileWalk walk(ceil_div(a.v_len, LT), ceil_div(a.d, LT));
  const int n = walk.count(), kr = SECOND ? count : k_rows(count), nk = ceil_div(kr, 32);
  const bool labels = !SECOND && a.dw_fmt == FMT_BF16 && count > LOSS_LO_ROWS;
  const int tile0 = a.v_first / LT, own = (nk + 1) / 2 * 2;   // the labels' steps start a pair (65 rows: the third)
  int vt, nt;
  if (wave_id() >= dense::NMW) {
    const uint32_t ldg = a.ldg * 2, ldh = a.d * 2;
    dense::Opnd oa, ob;
    auto head = [&](int i) {
      walk.tile(i, vt, nt);
      oa = dense::opnd_ko(make_rsrc(a.g + second_at<SECOND>(count, a.ldg), kr * ldg), ldg, vt * LT);
      ob = dense::opnd_ko(make_rsrc(a.hc, kr * ldh), ldh, nt * LT);
      dense::load_head<4>(ring, oa, ob, nk);
    };
    if (n > 0) head(0);
    for (int i = 0; i < n; ++i) {
      LabelSteps ls(a, labels, tile0 + vt, count);
      load_body<4>(
          ring, oa, ob, nk, ls.pairs(), [&](int k) __attribute__((always_inline)) { ls.fetch(a, k); },
          [&](int, int st) __attribute__((always_inline)) { ls.issue(a, ob.r, ring, st, nt * LT, count); });
      block_barrier();   // the tile's stages are read
      if (i + 1 < n) head(i + 1);
    }
    return;
  }
  const int w = wave_id(), wm = w % 2, wn = w / 2;
  const float scale = __int_as_float(a.count[2]);
  for (int i = 0; i < n; ++i) {
    walk.tile(i, vt, nt);
    const int v0 = a.v_first + vt * LT, vrows = min(LT, a.V - v0), n0 = nt * LT + 64 * wn, ncols = min(64, a.d - n0);
    const LabelSteps ls(a, labels, tile0 + vt, count);
    Acc acc;
    dense::mfma_loop<KO, KO, 8>(ring, own + 2 * ls.pairs(), acc);
    block_barrier();   // the tile's stages are read
    if (ncols <= 0) continue;
#pragma unroll
    for (int k = 0; k < MI; ++k)
#pragma unroll
      for (int j = 0; j < NJ; ++j) acc[k][j] *= scale;
    if (!SECOND && a.dw_fmt == FMT_BF16) {
      uint16_t* dst = static_cast<uint16_t*>(a.dw) + static_cast<size_t>(v0) * a.d + n0;
      dense::store_bf16_tile<8>(
          ring, ncols, [&](int k, int j) { return pack4(acc[k][j][0], acc[k][j][1], acc[k][j][2], acc[k][j][3]); },
          [&](int row) -> uint16_t* { return row < vrows ? dst + static_cast<size_t>(row) * a.d : nullptr; });
      continue;
    }
    // fp32: 16 rows x 64 columns at a time through the wave's staging, 256-byte rows
    float* dst = static_cast<float*>(a.dw) + static_cast<size_t>(v0) * a.d + n0;
    uint8_t* sg = ring + dense::SPARE + 4096 * w;
    const int lane = dense::fresh_lane(), lr = lane & 15, lg = lane >> 4;
#pragma unroll
    for (int k = 0; k < MI; ++k) {
#pragma unroll
      for (int j = 0; j < NJ; ++j)
        *reinterpret_cast<f32x4*>(sg + lr * 256 + (((4 * j + lg) ^ lr) << 4)) = acc[k][j];
      __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
      __builtin_amdgcn_wave_barrier();
      __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const int rr = 4 * q + (lane >> 4), c = lane & 15, row = 16 * (2 * k + wm) + rr;
        const f32x4 v = *reinterpret_cast<const f32x4*>(sg + rr * 256 + ((c ^ rr) << 4));
        if (row < vrows && 4 * c < ncols) {
          f32x4* p = reinterpret_cast<f32x4*>(dst + static_cast<size_t>(row) * a.d + 4 * c);
          *p = SECOND ? *p + v : v;
        }
      }
      __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
      __builtin_amdgcn_wave_barrier();
      __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
    }
  }
}

}  // namespace

MOE_DEBUG_FILE(loss)

hipError_t launch_loss_rows(const LossArgs& a, hipStream_t s) {
  hipLaunchKernelGGL(loss_rows_kernel, dim3(1), dim3(1024), 0, s, a);
  return hipGetLastError();
}

template <bool GRAD>
static void launch_stream(const LossArgs& a, int blocks, hipStream_t s) {
  if (a.T <= 16)
    hipLaunchKernelGGL((loss_stream_kernel<1, GRAD>), dim3(blocks), dim3(STHREADS), 0, s, a);
  else if (a.T <= 32)
    hipLaunchKernelGGL((loss_stream_kernel<2, GRAD>), dim3(blocks), dim3(STHREADS), 0, s, a);
  else if (a.T <= 48)
    hipLaunchKernelGGL((loss_stream_kernel<3, GRAD>), dim3(blocks), dim3(STHREADS), 0, s, a);
  else
    hipLaunchKernelGGL((loss_stream_kernel<4, GRAD>), dim3(blocks), dim3(STHREADS), 0, s, a);
}

hipError_t launch_loss_forward(const LossArgs& a, hipStream_t s) {
  if (loss_stream(a.T, a.d, a.V)) {
    launch_stream<false>(a, a.tiles, s);
    hipLaunchKernelGGL(loss_finish_kernel<4>, dim3(a.T), dim3(256), 0, s, a);
    return hipGetLastError();
  }
  const hipError_t e = launch_loss_rows(a, s);
  if (e != hipSuccess) return e;
  hipLaunchKernelGGL((loss_logits_kernel<false, false>), dim3(loss_grid(ceil_div(a.T, 64), a.tiles)),
                     dim3(dense::THREADS), 0, s, a);
  hipLaunchKernelGGL(loss_finish_kernel<1>, dim3(ceil_div(a.T, 4)), dim3(256), 0, s, a);
  return hipGetLastError();
}

hipError_t launch_loss_gather(const LossArgs& a, hipStream_t s) {
  const int lists = loss_labels(a.T, a.dw_fmt) ? ceil_div(a.V, LT) : 0;
  if (a.T > 0) hipLaunchKernelGGL(loss_gather_kernel, dim3(loss_k_rows(a.T) + lists), dim3(256), 0, s, a);
  return hipGetLastError();
}

// One piece: G, its part of dh, its rows of dw.
hipError_t launch_loss_piece(const LossArgs& a, hipStream_t s) {
  const long long nm = ceil_div(a.T, 64), nv = ceil_div(a.v_len, LT), nn = ceil_div(a.d, LT);
  const dim3 grid(loss_grid(nm, nv)), block(dense::THREADS);
  if (a.T > 0) {
    if (loss_stream(a.T, a.d, a.V))
      launch_stream<true>(a, static_cast<int>(nv) * (LT / SV), s);
    else if (loss_pairs(a.dh_fmt, a.dw_fmt))
      hipLaunchKernelGGL((loss_logits_kernel<true, true>), grid, block, 0, s, a);
    else
      hipLaunchKernelGGL((loss_logits_kernel<true, false>), grid, block, 0, s, a);
    const dim3 dh_grid(loss_grid(nm, nn * LOSS_SPLITS));
    hipLaunchKernelGGL(loss_dh_kernel<false>, dh_grid, block, 0, s, a);
    if (a.dh_fmt == FMT_F32) hipLaunchKernelGGL(loss_dh_kernel<true>, dh_grid, block, 0, s, a);
  }
  const dim3 dw_grid(loss_grid(nv, nn));
  hipLaunchKernelGGL(loss_dw_kernel<false>, dw_grid, block, 0, s, a);
  if (a.dw_fmt == FMT_F32 && a.T > LOSS_LO_ROWS) hipLaunchKernelGGL(loss_dw_kernel<true>, dw_grid, block, 0, s, a);
  return hipGetLastError();
}

hipError_t launch_loss_dh(const LossArgs& a, hipStream_t s) {
  if (a.T > 0) hipLaunchKernelGGL(loss_dh_out_kernel, dim3(a.T), dim3(256), 0, s, a);
  return hipGetLastError();
}

}  // namespace moe
