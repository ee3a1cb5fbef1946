// The layer's forward for a few tokens (1 to 64):
//
//   s = sigmoid(u E^T), the K largest of s + b, g = s / sum of the K selected s
//   h = SiLU(W_gate u) * (W_up u) for each selected and shared expert
//   y = u + sum_shared W_down h + sum_k g_k W_down h_k
//
// Each selected expert's matrices are read once and nothing else is large: the
// whole is bound by HBM.  The weights therefore go from global memory straight
// into the MFMAs' first operand (16 rows of weights, 16 bytes a lane), no LDS;
// the tokens are the second operand's 16 columns, read through the caches.  The
// waves of a block take 128-byte runs of K in turn and their sums meet in LDS.
//
//   few_route_kernel   partial logits, 16 experts and a slice of K to a block
//                      (8-bit weights: also u's 1x128 codes)
//   few_select_kernel  the experts of a token, by a wave.  Of up to 8 tokens every
//                      block of the next kernel selects them for itself instead (a
//                      launch and a trip through memory less)
//   few_gateup_kernel  (expert, 16 columns of I) units
//   few_quant_kernel   8-bit weights: h's 1x128 codes
//   few_down_kernel    16 columns of y to a block, over all experts in turn: the
//                      gated sum and the residual stay on chip, in a fixed order.  Where
//                      that leaves CUs idle, blocks share the experts' runs, and
//   few_sum_kernel     adds their sums
//
// Measured, us, with other inputs in every call (reading alone reaches 6.2 TB/s here): 1
// token, d = 7168 in bf16, 9 experts of 88 MB: 154 in all, gate and up 102 (5.2 TB/s),
// down 55 (4.8), the router 4.6; 4 tokens in 8 bits, 33 experts of 44 MB: 253, gate and
// up 162 (5.9), down 87 (5.6); 32 tokens, 164 experts: 2388, gate and up 1543 (6.2),
// down 801 (6.0).  1 token, d = 2048, 8 experts of 17 MB: 44 (40 where the last call's
// weights still lie in the caches), gate and up 26 (23 at best), down 15, the rest
// launches; of the 23, 8 are not loads (the selection, a block's sums, the last blocks).
//
// Sums are fp32.  With bf16 weights the operand h is a pair of bf16 values, what the
// first rounds off in the second; 2^-17 of it is left at most.  The experts' part of y
// is then 2.5e-6 from 64 bits, where fp32 values and products (fp32 weights) leave 3e-7
// and a single bf16 value would leave about 1e-3: the pair costs the MFMAs nothing, which
// wait for HBM, and fp32 products would take eight times as many.
#include "few.hpp"
#include "gemm_core.hpp"
#include "scores.hpp"

#include <type_traits>

namespace moe {

namespace {

constexpr int THREADS = 512, WAVES = 8;
// Two blocks to a CU, each taking units in turn: a third round of blocks would select
// again.  1 token, d = 7168: 159 us with 512, 160 with 256, 169 with 384, 164 with 1152;
// 32 tokens: 2430, 2445, 2724, 2520.
constexpr int GATEUP_BLOCKS = 512;

__device__ __forceinline__ i32x4 load16(rsrc_t r, uint32_t off, uint32_t soff) {
  return __builtin_bit_cast(i32x4, __builtin_amdgcn_raw_buffer_load_b128(r, off, soff, 0));
}
// Eight of a lane's 8-bit codes as bf16 values (exact).
__device__ __forceinline__ i32x4 codes_bf16(int lo, int hi) {
  typedef __bf16 pair __attribute__((ext_vector_type(2)));
  auto two = [](int c, auto upper) {
    const pair p = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(c, 1.0f, decltype(upper)::value);
    return __builtin_bit_cast(int, p);
  };
  constexpr std::false_type l{};
  constexpr std::true_type u{};
  return i32x4{two(lo, l), two(lo, u), two(hi, l), two(hi, u)};
}

// Codes of four values of a tile, times its factor, whose largest size has the bits `top`
// (over the bits, where NaN and infinity stand above the rest; fmaxf would drop a NaN).
// A tile that holds one gets the scale NaN or infinity, and the code NaN wherever value
// times factor is NaN (e4m3x4 alone makes -448 of it): what reads the tile is not finite.
__device__ __forceinline__ uint32_t codes_of(float a, float b, float c, float d, uint32_t top) {
  uint32_t q = e4m3x4(a, b, c, d);
  if (top >= 0x7f800000u) {
    const float t[4] = {a, b, c, d};
#pragma unroll
    for (int e = 0; e < 4; ++e)
      if (t[e] != t[e]) q = (q & ~(0xffu << 8 * e)) | 0x7fu << 8 * e;
  }
  return q;
}

// One 128-byte run of K: the products of 16 weight rows with 16 tokens.  A lane holds
// bytes 16 lg .. +15 of each half of the run, of its weight row and of its token alike.
// 8-bit codes go through the bf16 matrix instructions, which sum them as exactly as
// fp32 does (1e-8 of a run's product); the 8-bit ones keep 1.4e-5, and the matrix cores
// wait for HBM either way (4 tokens, d = 7168: 256 us with either).
template <int FMT>
__device__ __forceinline__ f32x4 run_product(const i32x4 (&w)[2], const i32x4 (&x)[2], f32x4 c) {
  if constexpr (FMT == FMT_BF16) {
    return mfma_bf16(w[1], x[1], mfma_bf16(w[0], x[0], c));
  } else if constexpr (FMT == FMT_F32) {
#pragma unroll
    for (int k = 0; k < 2; ++k)
#pragma unroll
      for (int e = 0; e < 4; ++e) c = mfma_f32(__int_as_float(w[k][e]), __int_as_float(x[k][e]), c);
    return c;
  } else {
#pragma unroll
    for (int k = 0; k < 2; ++k)
#pragma unroll
      for (int e = 0; e < 4; e += 2) c = mfma_bf16(codes_bf16(w[k][e], w[k][e + 1]), codes_bf16(x[k][e], x[k][e + 1]), c);
    return c;
  }
}

// ------------------------------------------------------------------ selection

// Largest value over the wave, in every lane.
template <int CTRL, int ROWS>
__device__ __forceinline__ uint32_t dpp_max(uint32_t v) {
  return max(v, static_cast<uint32_t>(__builtin_amdgcn_update_dpp(0, static_cast<int>(v), CTRL, ROWS, 0xf, false)));
}
__device__ __forceinline__ uint32_t wave_max_u32(uint32_t v) {
  v = dpp_max<0x111, 0xf>(v);   // row_shr 1, 2, 4, 8: lane 15 of each row has the row's
  v = dpp_max<0x112, 0xf>(v);
  v = dpp_max<0x114, 0xf>(v);
  v = dpp_max<0x118, 0xf>(v);
  v = dpp_max<0x142, 0xa>(v);   // row_bcast 15, 31: lane 63 has the wave's
  v = dpp_max<0x143, 0xc>(v);
  return __builtin_amdgcn_readlane(v, 63);
}

// Order-preserving bits of a key: above 0 for every value, NaN as -inf.
__device__ __forceinline__ uint32_t ordered(float v) {
  if (v != v) v = -INFINITY;
  const uint32_t u = __float_as_uint(v);
  return u ^ (static_cast<uint32_t>(static_cast<int32_t>(u) >> 31) | 0x80000000u);
}

// The top-K of one token by one wave, as the router's (descending s + b, exact ties
// to the lower expert, NaN below every number).  A lane holds experts lane + 64 q in
// descending order, so a round looks at the lanes' first ones alone (without, 2500
// cycles a round; 250 with).  `keys` is the wave's own LDS, for group-limited routing.
template <int NQ>
__device__ __forceinline__ void few_select(const FewArgs& a, int t, float* keys, int32_t* idx_out, float* gate_out) {
  const int lane = threadIdx.x & 63, N = a.n_routed;
  const size_t stride = static_cast<size_t>(a.T) * N;
  const float* src = a.logits + static_cast<size_t>(t) * N + lane;
  float s[NQ], b[NQ];
  uint32_t key[NQ];
  int id[NQ];
#pragma unroll
  for (int q = 0; q < NQ; ++q) {
    s[q] = 0.f;
    b[q] = lane + 64 * q < N ? a.bias[lane + 64 * q] : 0.f;
  }
  constexpr int NS = NQ <= 4 ? 16 : 8;   // slices whose loads go out together
  for (int k = 0; k < a.slices; k += NS) {
    float z[NS][NQ];
#pragma unroll
    for (int j = 0; j < NS; ++j)
#pragma unroll
      for (int q = 0; q < NQ; ++q) z[j][q] = k + j < a.slices && lane + 64 * q < N ? src[(k + j) * stride + 64 * q] : 0.f;
#pragma unroll
    for (int j = 0; j < NS; ++j)
#pragma unroll
      for (int q = 0; q < NQ; ++q) s[q] += z[j][q];
  }
#pragma unroll
  for (int q = 0; q < NQ; ++q) {
    key[q] = 0;
    id[q] = q;
    const int e = lane + 64 * q;
    if (e >= N) continue;
    s[q] = kept_score(s[q]);
    const float v = score_of(s[q]) + b[q];
    key[q] = ordered(v);
    if (a.topk_groups < a.n_groups) keys[e] = v != v ? -INFINITY : v;
  }
  if (a.topk_groups < a.n_groups) {
    // a group's score: the sum of its qg largest keys, largest first
    const int size = N / a.n_groups, qg = min((a.top_k + a.topk_groups - 1) / a.topk_groups, size);
    __builtin_amdgcn_wave_barrier();
    uint32_t score = 0;
    if (lane < a.n_groups) {
      const float* g = keys + lane * size;
      float sum = 0.f, pv = INFINITY;
      int pe = -1;
      for (int j = 0; j < qg; ++j) {
        float bv = -INFINITY;
        int be = 0x7fffffff;
        for (int m0 = 0; m0 < size; m0 += 8) {
          float x[8];
#pragma unroll
          for (int m = 0; m < 8; ++m) x[m] = g[min(m0 + m, size - 1)];
#pragma unroll
          for (int m = 0; m < 8; ++m) {   // after the last taken, and before what the pass has
            const bool take = (x[m] < pv || (x[m] == pv && m0 + m > pe)) && (x[m] > bv || be == 0x7fffffff) && m0 + m < size;
            bv = take ? x[m] : bv;
            be = take ? m0 + m : be;
          }
        }
        sum += bv;
        pv = bv;
        pe = be;
      }
      score = ordered(sum);
    }
    unsigned long long kept = 0;
    for (int j = 0; j < a.topk_groups; ++j) {
      const uint32_t m = wave_max_u32(score);
      const int g = __ffsll(__ballot(score == m)) - 1;
      kept |= 1ULL << g;
      if (lane == g) score = 0;
    }
#pragma unroll
    for (int q = 0; q < NQ; ++q) {
      const int e = lane + 64 * q;
      if (e < N && !((kept >> (e / size)) & 1ULL)) key[q] = 0;
    }
    __builtin_amdgcn_wave_barrier();
  }
  // neighbours change places where the later one is larger: equal keys keep their order
#pragma unroll
  for (int n = NQ - 1; n > 0; --n)
#pragma unroll
    for (int q = 0; q < n; ++q)
      if (key[q] < key[q + 1]) {
        const uint32_t k0 = key[q];
        const float s0 = s[q];
        const int i0 = id[q];
        key[q] = key[q + 1]; s[q] = s[q + 1]; id[q] = id[q + 1];
        key[q + 1] = k0; s[q + 1] = s0; id[q + 1] = i0;
      }
  int chosen = 0;
  float chosen_s = 0.f, sum = 0.f;
  for (int k = 0; k < a.top_k; ++k) {
    const uint32_t m = wave_max_u32(key[0]);
    unsigned long long same = __ballot(key[0] == m);
    int l = __ffsll(same) - 1, be = 64 * __builtin_amdgcn_readlane(id[0], l) + l;
    for (same &= same - 1; same != 0; same &= same - 1) {   // equal keys: the lowest expert
      const int l2 = __ffsll(same) - 1, e2 = 64 * __builtin_amdgcn_readlane(id[0], l2) + l2;
      if (e2 < be) { be = e2; l = l2; }
    }
    if (!MOE_CHECK(be >= 0 && be < N, 801)) be = 0;
    const float bs = __uint_as_float(__builtin_amdgcn_readlane(__float_as_uint(s[0]), l));
    sum += score_of(bs);
    if (lane == k) { chosen = be; chosen_s = bs; }
    if (lane == l) {
#pragma unroll
      for (int q = 0; q + 1 < NQ; ++q) { key[q] = key[q + 1]; s[q] = s[q + 1]; id[q] = id[q + 1]; }
      key[NQ - 1] = 0;
    }
  }
  const float gate = selected(chosen_s, sum, lane, a.top_k).gate;
  if (lane < a.top_k) {
    idx_out[lane] = chosen;
    gate_out[lane] = gate;
  }
}

// One wave per token.
template <int NQ>
__global__ __launch_bounds__(256) void few_select_kernel(FewArgs a) {
  __shared__ float keys[4][64 * NQ];
  const int w = wave_id(), t = blockIdx.x * 4 + w;
  if (t < a.T) few_select<NQ>(a, t, keys[w], a.idx + t * a.top_k, a.gate + t * a.top_k);
}

// The experts that have rows, in order, the shared ones last; each one's rows are
// its tokens in order.
struct Lists {
  unsigned long long mask[MAX_ROUTED + MAX_SHARED];   // tokens of entry i (first: of expert i)
  int32_t expert[MAX_ROUTED + MAX_SHARED];            // of entry i; N_r + s: shared
  int32_t row0[MAX_ROUTED + MAX_SHARED];              // first row of entry i
  int32_t at[MAX_ROUTED];                             // first row of expert e
  int32_t wave_n[WAVES], wave_rows[WAVES];
  int32_t n;
};

__device__ __forceinline__ void load_selection(const FewArgs& a, int32_t* idx) {
  for (int i = threadIdx.x; i < a.T * a.top_k; i += THREADS) {
    int e = a.idx[i];
    if (!MOE_CHECK(e >= 0 && e < a.n_routed, 806)) e = 0;
    idx[i] = e;
  }
}

// From idx [T][K] (LDS); `token` receives each routed row's token.
__device__ __forceinline__ void make_lists(const FewArgs& a, Lists& L, const int32_t* idx, int32_t* token) {
  const int tid = threadIdx.x, lane = tid & 63, w = wave_id(), TK = a.T * a.top_k;
  for (int e = tid; e < MAX_ROUTED; e += THREADS) L.mask[e] = 0;
  __syncthreads();
  for (int i = tid; i < TK; i += THREADS) atomicOr(&L.mask[idx[i]], 1ULL << (i / a.top_k));
  __syncthreads();
  static_assert(MAX_ROUTED <= THREADS, "a thread an expert");
  const unsigned long long mine = tid < a.n_routed ? L.mask[tid] : 0;
  const unsigned long long live = __ballot(mine != 0);
  const int rows = __popcll(mine);
  int before = rows;   // inclusive, then exclusive
#pragma unroll
  for (int off = 1; off < 64; off <<= 1) {
    const int v = __shfl_up(before, off);
    if (lane >= off) before += v;
  }
  if (lane == 63) {
    L.wave_n[w] = __popcll(live);
    L.wave_rows[w] = before;
  }
  before -= rows;
  __syncthreads();   // every mask is in a register now
  int n0 = 0, r0 = 0, n = 0;
#pragma unroll
  for (int k = 0; k < WAVES; ++k) {
    if (k < w) { n0 += L.wave_n[k]; r0 += L.wave_rows[k]; }
    n += L.wave_n[k];
  }
  if (tid < a.n_routed) {
    L.at[tid] = r0 + before;
    if (mine != 0) {
      const int i = n0 + __popcll(live & ((1ULL << lane) - 1));
      L.mask[i] = mine;
      L.expert[i] = tid;
      L.row0[i] = r0 + before;
      int row = r0 + before;
      for (unsigned long long m = mine; m != 0; m &= m - 1) token[row++] = __ffsll(m) - 1;
    }
  }
  if (tid < a.n_shared && a.T > 0) {
    L.mask[n + tid] = a.T < 64 ? (1ULL << a.T) - 1 : ~0ULL;
    L.expert[n + tid] = a.n_routed + tid;
    L.row0[n + tid] = TK + tid * a.T;
  }
  if (tid == 0) L.n = n + (a.T > 0 ? a.n_shared : 0);
  __syncthreads();
}

// ------------------------------------------------------------------ router

template <int FMT, int NT>
__global__ __launch_bounds__(THREADS) void few_route_kernel(FewArgs a, int blocks) {
  __shared__ f32x4 red[WAVES][NT][64];
  const int w = wave_id(), lane = threadIdx.x & 63, lr = lane & 15, lg = lane >> 4;
  if (static_cast<int>(blockIdx.x) >= blocks) {
    // 8-bit weights: u's 1x128 tiles, 16 lanes each, as moe_quantize_act_e4m3
    const int tiles = a.d / 128, i = (blockIdx.x - blocks) * (THREADS / 16) + (threadIdx.x >> 4);
    const bool live = i < a.T * tiles;
    uint4 raw = make_uint4(0, 0, 0, 0);
    const size_t off = static_cast<size_t>(i) * 128 + (lane & 15) * 8;
    if (live) raw = *reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(a.u) + off);
    const uint32_t words[4] = {raw.x, raw.y, raw.z, raw.w};
    float v[8];
    uint32_t top = 0;
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      v[e] = __uint_as_float(e % 2 ? words[e / 2] & 0xffff0000u : words[e / 2] << 16);
      top = max(top, __float_as_uint(v[e]) & 0x7fffffffu);
    }
#pragma unroll
    for (int o = 1; o <= 8; o <<= 1) top = max(top, __shfl_xor(top, o));
    const float m = __uint_as_float(top);
    const float inv = m == 0.f ? 0.f : 448.f / m;
    const uint32_t lo = codes_of(v[0] * inv, v[1] * inv, v[2] * inv, v[3] * inv, top);
    const uint32_t hi = codes_of(v[4] * inv, v[5] * inv, v[6] * inv, v[7] * inv, top);
    if (live) {
      *reinterpret_cast<uint2*>(a.uq + off) = make_uint2(lo, hi);
      if ((lane & 15) == 0) a.us[i] = m == 0.f ? 1.f : m / 448.f;
    }
    return;
  }
  if (blockIdx.x == 0 && threadIdx.x == 0) *a.taken = 0;   // for the next kernel
  const int tiles = (a.n_routed + 15) / 16, tile = blockIdx.x % tiles, slice = blockIdx.x / tiles;
  if (!MOE_CHECK(slice < a.slices, 802)) return;
  const uint32_t ld = a.d * (FMT == FMT_F32 ? 4 : 2);
  const int runs = ld / 128, per = (runs + a.slices - 1) / a.slices;
  const int p1 = min(runs, (slice + 1) * per);
  const rsrc_t re = make_rsrc(a.centroids, a.n_routed * ld), ru = make_rsrc(a.u, a.T * ld);   // past the end: zeros
  const uint32_t oe = (16 * tile + lr) * ld + 16 * lg;
  f32x4 acc[NT];
#pragma unroll
  for (int t = 0; t < NT; ++t) acc[t] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll 2
  for (int p = slice * per + w; p < p1; p += WAVES) {
    i32x4 e[2], x[NT][2];
#pragma unroll
    for (int k = 0; k < 2; ++k) e[k] = load16(re, oe, 128 * p + 64 * k);
#pragma unroll
    for (int t = 0; t < NT; ++t)
#pragma unroll
      for (int k = 0; k < 2; ++k) x[t][k] = load16(ru, (16 * t + lr) * ld + 16 * lg, 128 * p + 64 * k);
#pragma unroll
    for (int t = 0; t < NT; ++t) acc[t] = run_product<FMT>(e, x[t], acc[t]);
  }
#pragma unroll
  for (int t = 0; t < NT; ++t) red[w][t][lane] = acc[t];
  __syncthreads();
  if (w >= NT) return;
  f32x4 z = red[0][w][lane];
#pragma unroll
  for (int k = 1; k < WAVES; ++k) z += red[k][w][lane];
  // lane: token 16 w + lr, experts 16 tile + 4 lg .. +3
  const int t = 16 * w + lr;
  if (t >= a.T) return;
  float* dst = a.logits + (static_cast<size_t>(slice) * a.T + t) * a.n_routed;
#pragma unroll
  for (int r = 0; r < 4; ++r) {
    const int e = 16 * tile + 4 * lg + r;
    if (e < a.n_routed) dst[e] = z[r];
  }
}

// ------------------------------------------------------------------ gate, up, SwiGLU

// One unit's sums over this wave's runs: 16 gate rows and the 16 up rows beside them,
// with NT tiles of 16 tokens.
template <int FMT, int NT>
struct GateUp {
  rsrc_t rw, rx;
  uint32_t ow[2], ox[NT];
  const float *sg, *su, *sx[NT];   // e4m3: the scales of the unit's blocks, of the tokens' tiles
  f32x4 acc[2][NT];

  // NB runs from p on: all their loads go out before the first product
  template <int NB>
  __device__ __forceinline__ void runs(int p) {
    i32x4 a[NB][2][2], x[NB][NT][2];
    float g[NB], u[NB], st[NB][NT];
#pragma unroll
    for (int j = 0; j < NB; ++j) {
      if constexpr (FMT == FMT_E4M3) {
        g[j] = sg[p + j];
        u[j] = su[p + j];
#pragma unroll
        for (int t = 0; t < NT; ++t) st[j][t] = sx[t][p + j];
      }
#pragma unroll
      for (int s = 0; s < 2; ++s)
#pragma unroll
        for (int k = 0; k < 2; ++k) a[j][s][k] = load16(rw, ow[s], 128 * (p + j) + 64 * k);
#pragma unroll
      for (int t = 0; t < NT; ++t)
#pragma unroll
        for (int k = 0; k < 2; ++k) x[j][t][k] = load16(rx, ox[t], 128 * (p + j) + 64 * k);
    }
    __builtin_amdgcn_sched_barrier(0);
#pragma unroll
    for (int j = 0; j < NB; ++j) {
      if constexpr (FMT == FMT_E4M3) {
#pragma unroll
        for (int t = 0; t < NT; ++t) {
          const f32x4 zero = {0.f, 0.f, 0.f, 0.f};
          acc[0][t] += run_product<FMT>(a[j][0], x[j][t], zero) * (st[j][t] * g[j]);
          acc[1][t] += run_product<FMT>(a[j][1], x[j][t], zero) * (st[j][t] * u[j]);
        }
      } else {
#pragma unroll
        for (int t = 0; t < NT; ++t)
#pragma unroll
          for (int s = 0; s < 2; ++s) acc[s][t] = run_product<FMT>(a[j][s], x[j][t], acc[s][t]);
      }
    }
  }

  // Of n runs, an eighth each.  Four runs at a time, as far as the registers go, where a
  // wave has more than four; the kernels' time, us: 1 token, d = 7168 (14 runs), four
  // 158, two 162; d = 2048 (4 runs) 43.8, 41.9.  Two of 8-bit runs, which come with
  // scales: 4 tokens, d = 7168 265, four 300.
  __device__ __forceinline__ void all(int n) {
    constexpr int NB = FMT == FMT_E4M3 ? (NT == 4 ? 1 : 2) : 4 / NT;
    const int w = wave_id(), per = (n + WAVES - 1) / WAVES, p1 = min(n, (w + 1) * per);
    int p = w * per;
    if (NB <= 2 || per > NB)
#pragma unroll 1
      for (; p + NB <= p1; p += NB) runs<NB>(p);
    if constexpr (NB > 2)
#pragma unroll 1
      for (; p + 2 <= p1; p += 2) runs<2>(p);
    if constexpr (NB > 1)
      if (p < p1) runs<1>(p);
  }
};

// Two bf16 values whose sum is v to 2^-16: its rounding, and that of what it left
// (of v itself: not contracted with the product that v is, which only some builds do).
__device__ __forceinline__ void split4(const float (&v)[4], uint2& hi, uint2& lo) {
#pragma clang fp contract(off)
  hi = make_uint2(bf16x2(v[0], v[1]), bf16x2(v[2], v[3]));
  const uint32_t b[4] = {hi.x << 16, hi.x & 0xffff0000u, hi.y << 16, hi.y & 0xffff0000u};
  float r[4];
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    const float f = __uint_as_float(b[e]);
    r[e] = fabsf(f) < INFINITY ? v[e] - f : 0.f;   // infinities and NaN stay in the first
  }
  lo = make_uint2(bf16x2(r[0], r[1]), bf16x2(r[2], r[3]));
}

template <int FMT, int NT>
__device__ __forceinline__ void gateup_unit(const FewArgs& a, int e, int row0, int rows, const int32_t* token, int i0,
                                            f32x4 (*red)[2][64], int taken, int32_t* next) {
  constexpr int ES = FMT == FMT_F32 ? 4 : FMT == FMT_BF16 ? 2 : 1;
  const int w = wave_id(), lane = threadIdx.x & 63, lr = lane & 15, lg = lane >> 4;
  const bool shared = e >= a.n_routed;
  const int m = shared ? e - a.n_routed : e, TK = a.T * a.top_k;
  const uint32_t ld = a.d * ES;
  const uint8_t* base = static_cast<const uint8_t*>(shared ? a.ws_gate_up : a.w_gate_up) +
                        static_cast<size_t>(m) * 2 * a.inter * ld;
  GateUp<FMT, NT> q;
  q.rw = make_rsrc(base, 2u * a.inter * ld);
  q.rx = make_rsrc(FMT == FMT_E4M3 ? static_cast<const void*>(a.uq) : a.u, a.T * ld);
  q.ow[0] = (i0 + lr) * ld + 16 * lg;
  q.ow[1] = (a.inter + i0 + lr) * ld + 16 * lg;
  const int runs = a.d * ES / 128;
  if constexpr (FMT == FMT_E4M3) {
    q.sg = (shared ? a.ss_gate_up : a.s_gate_up) + (static_cast<size_t>(m) * 2 * a.inter + i0) / 128 * runs;
    q.su = q.sg + static_cast<size_t>(a.inter / 128) * runs;
  }
#pragma unroll
  for (int t = 0; t < NT; ++t) {
    const int r = 16 * t + lr;
    const int tok = r < rows ? (shared ? r : token[row0 + r]) : a.T;
    q.ox[t] = tok * ld + 16 * lg;   // past the last token: zeros
    if constexpr (FMT == FMT_E4M3) q.sx[t] = a.us + static_cast<size_t>(min(tok, a.T - 1)) * runs;
#pragma unroll
    for (int s = 0; s < 2; ++s) q.acc[s][t] = f32x4{0.f, 0.f, 0.f, 0.f};
  }
  q.all(runs);
  __syncthreads();   // the last unit's sums have been read
#pragma unroll
  for (int t = 0; t < NT; ++t)
#pragma unroll
    for (int s = 0; s < 2; ++s) red[w * NT + t][s][lane] = q.acc[s][t];
  if (next != nullptr && threadIdx.x == 0) *next = taken;   // the block's next unit
  __syncthreads();
  // wave t: row 16 t + lr, columns i0 + 4 lg .. +3
  if (w >= NT || 16 * w + lr >= rows) return;
  f32x4 g = red[w][0][lane], u = red[w][1][lane];
#pragma unroll
  for (int k = 1; k < WAVES; ++k) {
    g += red[k * NT + w][0][lane];
    u += red[k * NT + w][1][lane];
  }
  float h[4];
#pragma unroll
  for (int r = 0; r < 4; ++r) h[r] = g[r] / (1.0f + expf(-g[r])) * u[r];
  const int row = row0 + 16 * w + lr;
  if (!MOE_CHECK(row < TK + a.n_shared * a.T, 803)) return;
  const size_t off = static_cast<size_t>(row) * a.inter + i0 + 4 * lg;
  if constexpr (FMT == FMT_BF16) {
    uint2 hi, lo;
    split4(h, hi, lo);
    *reinterpret_cast<uint2*>(static_cast<uint16_t*>(a.h) + off) = hi;
    *reinterpret_cast<uint2*>(a.h_lo + off) = lo;
  } else {
    *reinterpret_cast<float4*>(static_cast<float*>(a.h) + off) = make_float4(h[0], h[1], h[2], h[3]);
  }
}

// NT: tiles of 16 tokens that an expert may have.  NQ: the block selects the experts
// itself, 64 NQ of them at most (0: few_select_kernel has).
template <int FMT, int NT, int NQ>
__global__ __launch_bounds__(THREADS, 4) void few_gateup_kernel(FewArgs a) {
  __shared__ Lists L;
  __shared__ int32_t token[16 * NT * MAX_TOPK];
  __shared__ float gate[NQ > 0 ? WAVES * MAX_TOPK : 1];
  __shared__ int32_t next[2];   // this unit's successor, and the last one's while waves still read it
  __shared__ union {
    struct {
      float keys[WAVES][64 * NQ + 1];
      // here, for two blocks' memory to fit a CU with NT = 4: 64 tokens, d = 2048, us, in
      // bf16 287 (one block), 278, in 8 bits 169, 163
      int32_t idx[16 * NT * MAX_TOPK];
    } select;
    f32x4 red[WAVES * NT][2][64];   // written after a barrier of its own
  } s;
  int32_t* const idx = s.select.idx;
  const int w = wave_id();
  if (!MOE_CHECK(a.T <= (NQ > 0 ? WAVES : 16 * NT), 804)) return;
  if constexpr (NQ > 0) {
    if (w < a.T) few_select<NQ>(a, w, s.select.keys[w], idx + w * a.top_k, gate + w * a.top_k);
  } else {
    load_selection(a, idx);
  }
  __syncthreads();
  make_lists(a, L, idx, token);
  if (blockIdx.x == 0) {
    const int TK = a.T * a.top_k;
    for (int i = threadIdx.x; i < TK; i += THREADS) {
      if constexpr (NQ > 0) {
        a.idx[i] = idx[i];
        a.gate[i] = gate[i];
      }
      if (a.perm_token != nullptr) a.perm_token[i] = token[i];
      if (a.pos != nullptr) {
        int row = L.at[idx[i]];
        while (token[row] != i / a.top_k) ++row;   // it is among its expert's rows
        a.pos[i] = row;
      }
    }
    for (int e = threadIdx.x; e < a.n_routed; e += THREADS) {
      if (a.counts != nullptr) a.counts[e] = (e + 1 < a.n_routed ? L.at[e + 1] : TK) - L.at[e];
      if (a.offsets != nullptr) a.offsets[e] = L.at[e];
    }
    if (a.offsets != nullptr && threadIdx.x == 0) a.offsets[a.n_routed] = TK;
  }
  // Above 16 tokens units differ: a shared expert's take longest.  Where rows are short (8
  // KB) they come first, and a block takes its next unit when it begins one.  In turn, that
  // way, us: d = 2048 in bf16 32 tokens 250, 241, 64 tokens 319, 299; d = 7168 in 8 bits 64
  // tokens 1728, 1675.  Longer rows are read faster in turn: d = 7168 in bf16 32 tokens
  // 2377, 2409, 64 tokens 3184, 3220.  Of equal units the counter's latency is all that is
  // left: 16 tokens, 8 bits, d = 2048 116, 124.
  constexpr int ES = FMT == FMT_F32 ? 4 : FMT == FMT_BF16 ? 2 : 1;
  const bool take = NT > 1 && a.d * ES <= 64 * 128;
  const int cols = a.inter / 16, units = L.n * cols;
  auto after = [&](int i, int turn) { return take ? __builtin_amdgcn_readfirstlane(next[turn]) : i + static_cast<int>(gridDim.x); };
  for (int i = blockIdx.x, turn = 0; i < units; i = after(i, turn), turn ^= 1) {
    const int k0 = i / cols, k = take ? L.n - 1 - k0 : k0, i0 = 16 * (i - k0 * cols);
    int taken = 0;
    if (take && threadIdx.x == 0) taken = gridDim.x + atomicAdd(a.taken, 1);
    const int e = __builtin_amdgcn_readfirstlane(L.expert[k]), row0 = __builtin_amdgcn_readfirstlane(L.row0[k]);
    const int rows = __builtin_amdgcn_readfirstlane(__popcll(L.mask[k]));
    if constexpr (NT >= 4) {
      if (rows > 32) {
        gateup_unit<FMT, 4>(a, e, row0, rows, token, i0, s.red, taken, take ? next + turn : nullptr);
        continue;
      }
    }
    if constexpr (NT >= 2) {
      if (rows > 16) {
        gateup_unit<FMT, 2>(a, e, row0, rows, token, i0, s.red, taken, take ? next + turn : nullptr);
        continue;
      }
    }
    gateup_unit<FMT, 1>(a, e, row0, rows, token, i0, s.red, taken, take ? next + turn : nullptr);
  }
}

// 8-bit weights: h's 1x128 tiles, 32 lanes each (4 columns a lane).
__global__ __launch_bounds__(256) void few_quant_kernel(FewArgs a) {
  const long long tiles = static_cast<long long>(a.T) * (a.top_k + a.n_shared) * (a.inter / 128);
  const long long i = static_cast<long long>(blockIdx.x) * 8 + (threadIdx.x >> 5);
  const int l = threadIdx.x & 31;
  if (i >= tiles) return;
  const size_t off = static_cast<size_t>(i) * 128 + 4 * l;
  const float4 v = *reinterpret_cast<const float4*>(static_cast<const float*>(a.h) + off);
  uint32_t top = max(max(__float_as_uint(v.x) & 0x7fffffffu, __float_as_uint(v.y) & 0x7fffffffu),
                     max(__float_as_uint(v.z) & 0x7fffffffu, __float_as_uint(v.w) & 0x7fffffffu));
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) top = max(top, __shfl_xor(top, o));
  const float m = __uint_as_float(top);
  const float inv = m == 0.f ? 0.f : 448.f / m;
  *reinterpret_cast<uint32_t*>(a.hq + off) = codes_of(v.x * inv, v.y * inv, v.z * inv, v.w * inv, top);
  if (l == 0) a.hs[i] = m == 0.f ? 1.f : m / 448.f;
}

// ------------------------------------------------------------------ down, gates, residual

// A wave's turns over the runs of all experts, one after the other.
struct Turn {
  int k, p;   // entry, run
  __device__ __forceinline__ void advance(int by, int runs, int n) {
    p += by;
    while (p >= runs && k < n) {
      p -= runs;
      ++k;
    }
  }
};

// y = u + sums, four columns at offset off.
__device__ __forceinline__ void store_y(const FewArgs& a, size_t off, const f32x4& y) {
  float v[4];
  if (a.x_fmt == FMT_F32) {
    const float4 u = *reinterpret_cast<const float4*>(static_cast<const float*>(a.u) + off);
    v[0] = u.x; v[1] = u.y; v[2] = u.z; v[3] = u.w;
  } else {
    const uint2 u = *reinterpret_cast<const uint2*>(static_cast<const uint16_t*>(a.u) + off);
    v[0] = __uint_as_float(u.x << 16); v[1] = __uint_as_float(u.x & 0xffff0000u);
    v[2] = __uint_as_float(u.y << 16); v[3] = __uint_as_float(u.y & 0xffff0000u);
  }
#pragma unroll
  for (int r = 0; r < 4; ++r) v[r] += y[r];
  if (a.out_fmt == FMT_F32)
    *reinterpret_cast<float4*>(static_cast<float*>(a.y) + off) = make_float4(v[0], v[1], v[2], v[3]);
  else
    *reinterpret_cast<uint2*>(static_cast<uint16_t*>(a.y) + off) = make_uint2(bf16x2(v[0], v[1]), bf16x2(v[2], v[3]));
}

template <int FMT, int NT>
__global__ __launch_bounds__(THREADS, 4) void few_down_kernel(FewArgs a) {
  constexpr int ES = FMT == FMT_F32 ? 4 : FMT == FMT_BF16 ? 2 : 1;
  constexpr int NB = NT == 4 ? 2 : 4;   // runs whose loads go out together
  // Rows of a tile: of bf16 pairs 8, whose columns 0 .. 7 are the first values and 8 ..
  // 15 the second, so that both take one load and one product.
  constexpr int TR = FMT == FMT_BF16 ? 8 : 16, TILES = 16 * NT / TR;
  __shared__ Lists L;
  __shared__ int32_t idx[16 * NT * MAX_TOPK], token[16 * NT * MAX_TOPK];
  __shared__ float gate[16 * NT * MAX_TOPK], gate_row[16 * NT * MAX_TOPK];
  __shared__ f32x4 sums[WAVES][16 * NT][5];   // by token, 16 columns (and a gap) each
  const int w = wave_id(), lane = threadIdx.x & 63, lr = lane & 15, lg = lane >> 4;
  const int TK = a.T * a.top_k, R = TK + a.n_shared * a.T, d0 = 16 * blockIdx.x;
  if (!MOE_CHECK(a.T <= 16 * NT && d0 + 16 <= a.d && gridDim.y == static_cast<unsigned>(a.splits), 805)) return;
  load_selection(a, idx);
  for (int i = threadIdx.x; i < TK; i += THREADS) gate[i] = a.gate[i];
  for (int i = lane; i < 16 * NT * 5; i += 64) (&sums[w][0][0])[i] = f32x4{0.f, 0.f, 0.f, 0.f};
  __syncthreads();
  make_lists(a, L, idx, token);
  for (int i = threadIdx.x; i < TK; i += THREADS) {
    int row = L.at[idx[i]];
    while (token[row] != i / a.top_k) ++row;   // it is among its expert's rows
    gate_row[row] = gate[i];
  }
  __syncthreads();

  const uint32_t ld = a.inter * ES;
  const int runs = ld / 128, n = L.n;
  const uint32_t planes = static_cast<uint32_t>(R) * ld, end = FMT == FMT_BF16 ? 2 * planes : planes;
  const rsrc_t rh = make_rsrc(FMT == FMT_E4M3 ? static_cast<const void*>(a.hq) : a.h, end);
  const uint32_t ow = lr * ld + 16 * lg;
  const int tr = lr % TR;                                        // this lane's row of a tile
  const uint32_t plane = lr >= TR ? planes : 0;                  // and which of its values
  auto row_at = [&](int row0, int rows, int t) {                 // past the last row: zeros
    const int r = TR * t + tr;
    return (r < rows ? static_cast<uint32_t>(row0 + r) * ld + plane : end) + 16 * lg;
  };
  f32x4 acc[TILES];
#pragma unroll
  for (int t = 0; t < TILES; ++t) acc[t] = f32x4{0.f, 0.f, 0.f, 0.f};
  // adds the products with entry k's rows to their tokens' sums: a row that an expert
  // does not have takes nothing from its weights, whatever they hold
  auto flush = [&](int k, int rows) {
    const int row0 = L.row0[k];
    const bool shared = L.expert[k] >= a.n_routed;
#pragma unroll
    for (int t = 0; t < TILES; ++t) {
      if (TR * t >= rows) continue;
      f32x4 v = acc[t];
      acc[t] = f32x4{0.f, 0.f, 0.f, 0.f};
      if constexpr (TR == 8) {
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          // the second values' column stands 8 lanes on; it says nothing where the first is not
          // finite (an infinite weight times a second value of 0 or of the other sign: NaN)
          const float lo = __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(v[e]), 0x128, 0xf, 0xf, false));
          v[e] = fabsf(v[e]) < INFINITY ? v[e] + lo : v[e];
        }
      }
      const int r = TR * t + lr;
      if (lr < TR && r < rows) {
        const float g = shared ? 1.f : gate_row[row0 + r];
        f32x4& s = sums[w][shared ? r : token[row0 + r]][lg];
#pragma unroll
        for (int e = 0; e < 4; ++e) s[e] = fmaf(g, v[e], s[e]);
      }
    }
  };
  int cur = -1, cur_rows = 0;
  // a share of the routed experts' runs, then of the shared ones', whose rows are all tokens
  const int split = blockIdx.y * WAVES + w, splits = gridDim.y * WAVES, routed = n - (a.T > 0 ? a.n_shared : 0);
  for (int phase = 0; phase < 2; ++phase) {
    const int k0 = phase == 0 ? 0 : routed, total = (phase == 0 ? routed : a.n_shared) * runs;
    const int per = (total + splits - 1) / splits;
    Turn turn{k0, 0};
    turn.advance(split * per, runs, n);
    for (int left = min(per, total - split * per); left > 0; left -= NB) {
      Turn at[NB];
      int e[NB], row0[NB], rows[NB];
      i32x4 wf[NB][2], x[NB][2];
      float sw[NB], sh[NB];   // e4m3: the block's scale, this lane's row's
#pragma unroll
      for (int j = 0; j < NB; ++j) {
        at[j] = turn;
        turn.advance(1, runs, n);
        if (at[j].k >= n) at[j].p = 0;       // past the end: some run of the last, unused
        const int k = min(at[j].k, n - 1);
        e[j] = L.expert[k];
        row0[j] = L.row0[k];
        rows[j] = __popcll(L.mask[k]);
      }
#pragma unroll
      for (int j = 0; j < NB; ++j) {
        e[j] = __builtin_amdgcn_readfirstlane(e[j]);
        row0[j] = __builtin_amdgcn_readfirstlane(row0[j]);
        rows[j] = __builtin_amdgcn_readfirstlane(rows[j]);
        const bool shared = e[j] >= a.n_routed;
        const size_t mat = shared ? e[j] - a.n_routed : e[j];
        const uint8_t* const base = static_cast<const uint8_t*>(shared ? a.ws_down : a.w_down) + (mat * a.d + d0) * ld;
        const rsrc_t rw = make_rsrc(base, 16 * ld);
        const uint32_t oh = row_at(row0[j], rows[j], 0);
        if constexpr (FMT == FMT_E4M3) {
          sw[j] = (shared ? a.ss_down : a.s_down)[(mat * a.d + d0) / 128 * runs + at[j].p];
          sh[j] = a.hs[static_cast<size_t>(row0[j] + min(lr, rows[j] - 1)) * runs + at[j].p];
        }
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          wf[j][h] = load16(rw, ow, 128 * at[j].p + 64 * h);
          x[j][h] = load16(rh, oh, 128 * at[j].p + 64 * h);
        }
      }
#pragma unroll
      for (int j = 0; j < NB; ++j) {
        if (j >= left) continue;
        if (at[j].k != cur) {
          if (cur >= 0) flush(cur, cur_rows);
          cur = at[j].k;
          cur_rows = rows[j];
        }
        auto product = [&](int t, const i32x4(&v)[2], float s) {
          if constexpr (FMT == FMT_E4M3)
            acc[t] += run_product<FMT>(wf[j], v, f32x4{0.f, 0.f, 0.f, 0.f}) * (s * sw[j]);
          else
            acc[t] = run_product<FMT>(wf[j], v, acc[t]);
        };
        product(0, x[j], sh[j]);
#pragma unroll
        for (int t0 = 1; t0 < TILES; t0 += 4) {   // more rows than a tile's: four tiles' loads together
          if (rows[j] <= TR * t0) continue;
          i32x4 v[4][2];
          float s[4];
#pragma unroll
          for (int i = 0; i < 4 && t0 + i < TILES; ++i) {
            const uint32_t oh = row_at(row0[j], rows[j], t0 + i);   // past the last row: zeros
            if constexpr (FMT == FMT_E4M3)
              s[i] = a.hs[static_cast<size_t>(row0[j] + min(TR * (t0 + i) + lr, rows[j] - 1)) * runs + at[j].p];
#pragma unroll
            for (int h = 0; h < 2; ++h) v[i][h] = load16(rh, oh, 128 * at[j].p + 64 * h);
          }
#pragma unroll
          for (int i = 0; i < 4 && t0 + i < TILES; ++i) product(t0 + i, v[i], s[i]);
        }
      }
    }
  }
  if (cur >= 0) flush(cur, cur_rows);
  __syncthreads();
  // 4 lanes to a token, 4 columns each
  const int t = threadIdx.x >> 2, g = threadIdx.x & 3;
  if (t >= a.T) return;
  f32x4 y = sums[0][t][g];
#pragma unroll
  for (int k = 1; k < WAVES; ++k) y += sums[k][t][g];
  const size_t off = static_cast<size_t>(t) * a.d + d0 + 4 * g;
  if (a.splits > 1)
    *reinterpret_cast<f32x4*>(a.part + static_cast<size_t>(blockIdx.y) * a.T * a.d + off) = y;
  else
    store_y(a, off, y);
}

// The splits' sums, in order, and the residual: four columns a thread.
__global__ __launch_bounds__(256) void few_sum_kernel(FewArgs a) {
  const size_t off = 4 * (static_cast<size_t>(blockIdx.x) * 256 + threadIdx.x), n = static_cast<size_t>(a.T) * a.d;
  if (off >= n) return;
  f32x4 y = *reinterpret_cast<const f32x4*>(a.part + off);
  for (int k = 1; k < a.splits; ++k) y += *reinterpret_cast<const f32x4*>(a.part + k * n + off);
  store_y(a, off, y);
}

template <class F>
void by_experts(int n, F&& f) {   // experts in multiples of 64 to a lane
  if (n <= 64)
    f(std::integral_constant<int, 1>{});
  else if (n <= 128)
    f(std::integral_constant<int, 2>{});
  else if (n <= 256)
    f(std::integral_constant<int, 4>{});
  else
    f(std::integral_constant<int, 8>{});
}

template <int NT>
struct Launch {
  static void route(const FewArgs& a, hipStream_t s) {
    const int blocks = (a.n_routed + 15) / 16 * a.slices;
    const int quant = a.w_fmt == FMT_E4M3 ? ceil_div(a.T * (a.d / 128), THREADS / 16) : 0;
    if (a.x_fmt == FMT_F32)
      hipLaunchKernelGGL((few_route_kernel<FMT_F32, NT>), dim3(blocks), dim3(THREADS), 0, s, a, blocks);
    else
      hipLaunchKernelGGL((few_route_kernel<FMT_BF16, NT>), dim3(blocks + quant), dim3(THREADS), 0, s, a, blocks);
  }
  template <int FMT>
  static void gateup(const FewArgs& a, hipStream_t s) {
    const int tk = a.T * a.top_k;
    const long long units = static_cast<long long>((tk < a.n_routed ? tk : a.n_routed) + a.n_shared) * (a.inter / 16);
    const dim3 grid(static_cast<unsigned>(units < 1 ? 1 : units < GATEUP_BLOCKS ? units : GATEUP_BLOCKS)), block(THREADS);
    if constexpr (NT == 1) {
      if (a.T <= WAVES) {
        by_experts(a.n_routed, [&](auto nq) {
          hipLaunchKernelGGL((few_gateup_kernel<FMT, NT, decltype(nq)::value>), grid, block, 0, s, a);
        });
        return;
      }
    }
    by_experts(a.n_routed, [&](auto nq) {
      hipLaunchKernelGGL(few_select_kernel<decltype(nq)::value>, dim3(ceil_div(a.T, 4)), dim3(256), 0, s, a);
    });
    hipLaunchKernelGGL((few_gateup_kernel<FMT, NT, 0>), grid, block, 0, s, a);
  }
  template <int FMT>
  static void down(const FewArgs& a, hipStream_t s) {
    hipLaunchKernelGGL((few_down_kernel<FMT, NT>), dim3(a.d / 16, a.splits), dim3(THREADS), 0, s, a);
    if (a.splits > 1)
      hipLaunchKernelGGL(few_sum_kernel, dim3(ceil_div(a.T * (a.d / 4), 256)), dim3(256), 0, s, a);
  }
};

template <class F>
hipError_t by_tokens(int T, F&& f) {
  if (T <= 16)
    f(Launch<1>{});
  else if (T <= 32)
    f(Launch<2>{});
  else
    f(Launch<4>{});
  return hipGetLastError();
}

}  // namespace

MOE_DEBUG_FILE(few)

hipError_t launch_few_route(const FewArgs& a, hipStream_t s) {
  return by_tokens(a.T, [&](auto l) { l.route(a, s); });
}

hipError_t launch_few_gateup(const FewArgs& a, hipStream_t s) {
  return by_tokens(a.T, [&](auto l) {
    if (a.w_fmt == FMT_F32)
      l.template gateup<FMT_F32>(a, s);
    else if (a.w_fmt == FMT_BF16)
      l.template gateup<FMT_BF16>(a, s);
    else
      l.template gateup<FMT_E4M3>(a, s);
  });
}

hipError_t launch_few_quant(const FewArgs& a, hipStream_t s) {
  const long long tiles = static_cast<long long>(a.T) * (a.top_k + a.n_shared) * (a.inter / 128);
  hipLaunchKernelGGL(few_quant_kernel, dim3(static_cast<unsigned>((tiles + 7) / 8)), dim3(256), 0, s, a);
  return hipGetLastError();
}

hipError_t launch_few_down(const FewArgs& a, hipStream_t s) {
  return by_tokens(a.T, [&](auto l) {
    if (a.w_fmt == FMT_F32)
      l.template down<FMT_F32>(a, s);
    else if (a.w_fmt == FMT_BF16)
      l.template down<FMT_BF16>(a, s);
    else
      l.template down<FMT_E4M3>(a, s);
  });
}

}  // namespace moe
