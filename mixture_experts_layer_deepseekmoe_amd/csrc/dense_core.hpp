// Tile pipeline of the loss's products: C[256 x 256] += A B over K in steps of
// 32, for large dense products whose operand tiles are shared in L2.
//
// 8 MFMA waves (2 x 4, 128 x 64 each: 8 x 4 subtiles of 16x16x32 bf16 MFMAs that
// accumulate in place) and 4 waves that only issue loads: a ring of 5 stages
// (A and B, 32 of K: 32 KB) filled by DMA in pairs of K-steps, the two 64-byte
// halves of a K-contiguous row's line back to back.  MFMA waves that issued the
// loads themselves (256 registers, fragments of two K-steps held, one or two
// barriers a pair) took 9 to 23% longer: they stall on the loads.
//
// With 3 waves to a SIMD a wave has 168 registers, too few for the B fragments
// of two K-steps.  Instead a step's last two subtiles run B-fragment by
// B-fragment, and each B register takes the next step's fragment as soon as its
// last MFMA is issued.
//
// Two barriers per pair q (K-steps 2q, 2q + 1):
//   A_q  after step 2q: its stage is free; the load waves refill the buffers of
//        stages 2q - 1 and 2q with pair q + 2;
//   B_q  two subtiles before the end of step 2q + 1: pair q + 1 has landed.
// A pair's loads take most of a step to issue (64 KB at 64 bytes a cycle), so
// half of them go out before B_q and half after it: all before it, B_q came
// late and the loop took 10% longer.
//
// The kernels are persistent: a block walks several tiles, and the load waves
// issue the next tile's first two pairs (buffers 0-3) while the MFMA waves
// finish the last one (through buffer 4: SPARE).
//
// Operands are K-contiguous (KC: rows of K) or K-outer (KO: rows along K, the M or N
// index contiguous): read through the LDS transpose read, which gives a lane four
// consecutive K values of its own column; two reads make an MFMA operand.
#pragma once

#include "gemm_core.hpp"

namespace moe {

namespace dense {

enum : int { KC = 0, KO = 1 };

constexpr int OPB = 16384;          // bytes of one operand in a stage (256 x 32 bf16)
constexpr int STB = 2 * OPB;        // stage bytes (A then B)
constexpr int MI = 8, NJ = 4;       // accumulator subtiles per MFMA wave
constexpr int NMW = 8;              // MFMA waves
constexpr int NLW = 4;              // load waves
constexpr int THREADS = 64 * (NMW + NLW);
constexpr int NST = 5;
constexpr int RING_BYTES = NST * STB;
constexpr int SPARE = 4 * STB;       // LDS offset of the buffer that no tile's first two pairs use
constexpr int NLI = 4;              // DMA instructions per operand, stage and load wave

// s_waitcnt vmcnt(N) alone; and lgkmcnt(0), which LDS writes before it in the
// program stay in front of (a wave's writes are done before a barrier after it)
template <int N>
__device__ __forceinline__ void wait_vm() {
  static_assert(N >= 0 && N < 64, "vmcnt range");
  __builtin_amdgcn_s_waitcnt((N & 15) | (7 << 4) | (15 << 8) | ((N >> 4) << 14));
}
__device__ __forceinline__ void wait_lgkm0() { asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory"); }

__device__ __forceinline__ uint2 pack4(float a, float b, float c, float d) {
  return make_uint2(bf16x2(a, b), bf16x2(c, d));
}

// K-outer stage rows are 512 bytes (256 bf16); the 16-byte chunk of a row is
// xor-ed with a function of the K-row.  One transpose read takes 32 bytes, an
// aligned pair of chunks, of each of 16 rows (8 g + j, g, j = 0..3): the xor
// moves whole pairs, so that the 8 rows of each half of the wave fall on the 8
// different pairs of the 256 bytes the LDS serves at once (no bank conflicts;
// moving single chunks there is about one per read, at the same time).
__device__ __forceinline__ int xko(int k) { return ((k & 3) << 1) | (((k >> 3) & 1) << 3); }

// One operand's loads (load waves only): a buffer resource over its valid bytes
// (reads past it return zeros), per-lane byte offsets of the lane's NLI 16-byte
// pieces at K-step 0, and the bytes one K-step advances.
struct Opnd {
  rsrc_t r;
  uint32_t off[NLI];
  uint32_t kstride;
};

// K-contiguous: tile row m at byte row_off(m) of the resource.
template <class F>
__device__ __forceinline__ Opnd opnd_kc(rsrc_t r, F row_off) {
  Opnd o;
  o.r = r;
  const int w = wave_id() - NMW, lane = threadIdx.x & 63;
#pragma unroll
  for (int q = 0; q < NLI; ++q) {
    const int row = 16 * (w + NLW * q) + lane / 4;
    o.off[q] = row_off(row) + (((lane & 3) ^ swz<64>(row)) << 4);
  }
  o.kstride = 64;
  return o;
}

// K-outer: K-row k at byte k * ld, the tile's columns from col0.
__device__ __forceinline__ Opnd opnd_ko(rsrc_t r, uint32_t ld, int col0) {
  Opnd o;
  o.r = r;
  const int w = wave_id() - NMW, lane = threadIdx.x & 63;
#pragma unroll
  for (int q = 0; q < NLI; ++q) {
    const int k = 2 * (w + NLW * q) + lane / 32;
    o.off[q] = k * ld + col0 * 2 + (((lane & 31) ^ xko(k)) << 4);
  }
  o.kstride = 32 * ld;
  return o;
}

__device__ __forceinline__ uint8_t* stage(uint8_t* ring, int s) { return ring + (s % NST) * STB; }

// The pair of K-steps s, s + 1: its first (HALF 0) or second half.  Of A only
// the first NA groups of 64 rows are loaded (KC, for a tile of at most 64 NA
// rows).  A tile of up to 64 rows is bound by memory, not by the loads' issue:
// all of a pair is its first half.
template <int NA>
constexpr int first_ops() {
  return NA == 1 ? NA + NLI : (NA + NLI) / 2;
}
template <int HALF, int NA>
__device__ __forceinline__ void issue_half(const Opnd& a, const Opnd& b, uint8_t* ring, int s) {
  const int w = wave_id() - NMW;
  uint8_t* s0 = stage(ring, s) + 1024 * w;
  uint8_t* s1 = stage(ring, s + 1) + 1024 * w;
#pragma unroll
  for (int k = HALF == 0 ? 0 : first_ops<NA>(); k < (HALF == 0 ? first_ops<NA>() : NA + NLI); ++k) {
    // B's groups between A's
    const bool is_a = NA == NLI ? k % 2 == 0 : k < NA;
    const int q = NA == NLI ? k / 2 : (is_a ? k : k - NA);
    const Opnd& o = is_a ? a : b;
    const int at = (is_a ? 0 : OPB) + 1024 * NLW * q;
    dma16(o.r, o.off[q], s * o.kstride, s0 + at);
    dma16(o.r, o.off[q], (s + 1) * o.kstride, s1 + at);
  }
}
template <int NA>
__device__ __forceinline__ void issue_pair(const Opnd& a, const Opnd& b, uint8_t* ring, int s) {
  issue_half<0, NA>(a, b, ring, s);
  issue_half<1, NA>(a, b, ring, s);
}

// Fragment reads.  A wave's A subtile i is rows (KO: columns) 16 (2 i + wm) ..
// + 15 of the tile, its B subtile j 64 wn + 16 j .. + 15; LDS byte addresses are
// a lane constant plus the stage's plus a constant per subtile -- added for
// 64-byte rows (KC), xor-ed into the lane constant for K-rows (KO: chunk 2 (2 i
// + wm) or 8 wn + 2 j, whose bits that depend on the subtile are xor-ed with the
// row's swizzle: bits 6-7 (A) or 5-6 (B) of the address, and + 256 for i >= 4).
// The lane, as a value the compiler takes for new: what is derived from it is
// computed where it is used (an epilogue's addresses, hoisted out of a block's
// loop over tiles, would be spilled across the K loop).
__device__ __forceinline__ int fresh_lane() {
  int l = threadIdx.x;
  asm volatile("" : "+v"(l));
  return l & 63;
}

typedef __attribute__((address_space(3))) i32x4 lds_i32x4;
typedef int i32x2 __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x4 __attribute__((ext_vector_type(4)));
typedef __attribute__((address_space(3))) bf16x4 lds_bf16x4;
struct Lane {
  uint32_t a, b;
};
template <int KA, int KB>
__device__ __forceinline__ Lane make_lane(int wm, int wn) {
  const int lane = fresh_lane(), lr = lane & 15, lg = lane >> 4;
  const uint32_t kc = lr * 64 + ((lg ^ swz<64>(lr)) << 4);
  // KO: lane 16 g + c reads K-rows 8 g + c / 4 and + 4, columns 4 (c % 4) .. + 3 of a subtile
  const int k0 = 8 * lg + (lr >> 2), kbase = k0 * 512 + 8 * (lr & 1), ky = ((lr & 3) >> 1) ^ xko(k0);
  Lane l;
  l.a = KA == KC ? kc + 1024 * wm : kbase + (((2 * wm) ^ ky) << 4);
  l.b = OPB + (KB == KC ? kc + 4096 * wn : kbase + (((8 * (wn & 1)) ^ ky) << 4) + 256 * (wn >> 1));
  return l;
}
template <int KIND>
__device__ __forceinline__ i32x4 frag_at(uint32_t addr) {
  if constexpr (KIND == KC) {
    return *reinterpret_cast<const lds_i32x4*>(addr);
  } else {
    const bf16x4 lo = __builtin_amdgcn_ds_read_tr16_b64_v4bf16(reinterpret_cast<lds_bf16x4*>(addr));
    const bf16x4 hi = __builtin_amdgcn_ds_read_tr16_b64_v4bf16(reinterpret_cast<lds_bf16x4*>(addr + 4 * 512));
    const i32x2 a = __builtin_bit_cast(i32x2, lo), b = __builtin_bit_cast(i32x2, hi);
    return i32x4{a.x, a.y, b.x, b.y};
  }
}
template <int KA>
__device__ __forceinline__ i32x4 frag_a(uint32_t st, int i, const Lane& l) {
  return frag_at<KA>(KA == KC ? l.a + st + 2048 * i : (l.a ^ (64 * (i & 3))) + st + 256 * (i >> 2));
}
template <int KB>
__device__ __forceinline__ i32x4 frag_b(uint32_t st, int j, const Lane& l) {
  return frag_at<KB>(KB == KC ? l.b + st + 1024 * j : (l.b ^ (32 * j)) + st);
}

// One K-step from stage st.  On entry bf holds its B fragments and xc its first
// A fragment, on exit those of the next stage nx.  A fragments are read one
// subtile ahead.  WAIT: a barrier before the first read of nx.
template <int KA, int KB, int NSUB, bool WAIT>
__device__ __forceinline__ void step(uint32_t st, uint32_t nx, const Lane& l, i32x4 (&bf)[NJ], i32x4& xc,
                                     f32x4 (&acc)[MI][NJ]) {
  constexpr int P = NSUB - 2, Q = NSUB - 1;
  i32x4 xq;
  if constexpr (NSUB == 2) xq = frag_a<KA>(st, Q, l);
#pragma unroll
  for (int i = 0; i < P; ++i) {
    const i32x4 xn = frag_a<KA>(st, i + 1, l);
    if (i == P - 1) xq = frag_a<KA>(st, Q, l);
    __builtin_amdgcn_sched_barrier(0);
#pragma unroll
    for (int j = 0; j < NJ; ++j) mfma_bf16_tied(acc[i][j], bf[j], xc);
    __builtin_amdgcn_sched_barrier(0);
    xc = xn;
  }
  if constexpr (WAIT) block_barrier();
#pragma unroll
  for (int j = 0; j < 2; ++j) {
    mfma_bf16_tied(acc[P][j], bf[j], xc);
    mfma_bf16_tied(acc[Q][j], bf[j], xq);
    __builtin_amdgcn_sched_barrier(0);
    bf[j] = frag_b<KB>(nx, j, l);
    __builtin_amdgcn_sched_barrier(0);
  }
  mfma_bf16_tied(acc[P][2], bf[2], xc);
  mfma_bf16_tied(acc[P][3], bf[3], xc);
  __builtin_amdgcn_sched_barrier(0);
  xc = frag_a<KA>(nx, 0, l);
  __builtin_amdgcn_sched_barrier(0);
#pragma unroll
  for (int j = 2; j < 4; ++j) {
    mfma_bf16_tied(acc[Q][j], bf[j], xq);
    __builtin_amdgcn_sched_barrier(0);
    bf[j] = frag_b<KB>(nx, j, l);
    __builtin_amdgcn_sched_barrier(0);
  }
}

// The load waves' half of a tile: load_head issues its first two pairs (the
// buffers 0-3 are free), load_body the rest, in step with mfma_loop.
template <int NA>
__device__ __forceinline__ void load_head(uint8_t* ring, const Opnd& a, const Opnd& b, int nk) {
  if (nk > 0) issue_pair<NA>(a, b, ring, 0);
  if (nk > 2) issue_pair<NA>(a, b, ring, 2);
}
//
// `more` further pairs may follow those of nk, in steps as the rest (at least two
// pairs are the tile's own then): fetch(k) starts what pair k needs, issue(k, s)
// then issues it into the stages of steps s, s + 1, with as many DMA instructions
// as a pair's first half has.
template <int NA, class F, class I>
__device__ __forceinline__ void load_body(uint8_t* ring, const Opnd& a, const Opnd& b, int nk, int more, F&& fetch,
                                          I&& issue) {
  constexpr int H0 = 2 * first_ops<NA>(), N = 2 * (NA + NLI);
  const int own = (nk + 1) / 2, np = own + more;
  if (np <= 0) return;
  if (np > 1)
    wait_vm<N>();   // pair 0
  else
    wait_vm<0>();
  block_barrier();
  int q = 0;
  for (; q + 2 < own; ++q) {
    block_barrier();   // A_q
    issue_half<0, NA>(a, b, ring, 2 * (q + 2));
    wait_vm<H0>();     // pair q + 1
    block_barrier();   // B_q
    issue_half<1, NA>(a, b, ring, 2 * (q + 2));
  }
  if (more > 0) fetch(0);
  for (; q < np; ++q) {
    block_barrier();   // A_q
    if (q + 2 < np) {
      issue(q + 2 - own, 2 * (q + 2));
      wait_vm<H0>();   // pair q + 1
    } else {
      wait_vm<0>();    // pair q + 1 (if any) is the newest
    }
    block_barrier();   // B_q
    if (q + 3 < np) fetch(q + 3 - own);
  }
}
template <int NA>
__device__ __forceinline__ void load_body(uint8_t* ring, const Opnd& a, const Opnd& b, int nk) {
  load_body<NA>(ring, a, b, nk, 0, [](int) {}, [](int, int) {});
}

// f.template operator()<NSUB>() with NSUB the number of 32-row steps (2, 4, 6 or
// 8) to compute for a tile of `rows` rows; its loads take NA = NSUB / 2.
template <class F>
__device__ __forceinline__ void with_rows(int rows, F&& f) {
  if (rows > 192)
    f.template operator()<8>();
  else if (rows > 128)
    f.template operator()<6>();
  else if (rows > 64)
    f.template operator()<4>();
  else
    f.template operator()<2>();
}

// acc[i][j][r] = C[16 (2 i + wm) + lane % 16][64 wn + 16 j + 4 (lane / 16) + r]
// over nk K-steps, for the tile's first 32 NSUB rows (NSUB 2, 4, 6 or 8), wm =
// wave % 2, wn = wave / 2; on the MFMA waves.  A K-step nk may be loaded and
// multiplied (nk odd): one operand's bytes there read as zeros, the other's
// are finite.
template <int KA, int KB, int NSUB>
__device__ __forceinline__ void mfma_loop(const uint8_t* ring, int nk, f32x4 (&acc)[MI][NJ]) {
  static_assert(NSUB >= 2 && NSUB <= MI && NSUB % 2 == 0, "row subtiles");
  const int np = (nk + 1) / 2;
  zero_acc(acc);
  if (np <= 0) return;
  const int w = wave_id();
  Lane l = make_lane<KA, KB>(w % 2, w / 2);
  const uint32_t base = lds_addr(ring);
  auto st = [&](int s) { return base + static_cast<uint32_t>(s % NST) * STB; };
  i32x4 bf[NJ], xc;
  block_barrier();   // pair 0
#pragma unroll
  for (int j = 0; j < NJ; ++j) bf[j] = frag_b<KB>(base, j, l);
  xc = frag_a<KA>(base, 0, l);
  acc_fence(acc);
  for (int q = 0; q < np; ++q) {
    asm volatile("" : "+v"(l.a), "+v"(l.b));
    step<KA, KB, NSUB, false>(st(2 * q), st(2 * q + 1), l, bf, xc, acc);
    block_barrier();   // A_q
    step<KA, KB, NSUB, true>(st(2 * q + 1), st(2 * q + 2), l, bf, xc, acc);   // B_q
  }
  acc_fence(acc);
}

constexpr int STAGING = 2048;        // bytes a wave's store_bf16_tile uses, from SPARE on

// Stores a wave's 128 x 64 outputs as bf16 rows, 16 x 64 at a time through its
// 2 KB of SPARE (chunks xor-ed with the row; the wave's LDS operations run in
// order), so that a store instruction writes 8 whole 128-byte lines.  conv(i, j,
// r..) gives the four packed values of acc[i][j]; row_of(row) the destination of
// tile row `row` at the wave's first column, or null; ncols: valid columns of
// the wave's 64 (a multiple of 8).
template <int NSUB, class C, class R>
__device__ __forceinline__ void store_bf16_tile(uint8_t* ring, int ncols, C conv, R row_of) {
  const int w = wave_id(), lane = fresh_lane(), lr = lane & 15, lg = lane >> 4, wm = w % 2;
  uint8_t* const sg = ring + SPARE + STAGING * w;
#pragma unroll
  for (int i = 0; i < NSUB; ++i) {
#pragma unroll
    for (int j = 0; j < NJ; ++j)
      *reinterpret_cast<uint2*>(sg + lr * 128 + (((2 * j + (lg >> 1)) ^ (lr & 7)) << 4) + 8 * (lg & 1)) = conv(i, j);
    __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
    __builtin_amdgcn_wave_barrier();
    __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int r = 8 * h + (lane >> 3), c = lane & 7;
      const uint4 v = *reinterpret_cast<const uint4*>(sg + r * 128 + ((c ^ (r & 7)) << 4));
      uint16_t* dst = row_of(16 * (2 * i + wm) + r);
      if (dst != nullptr && 8 * c < ncols) *reinterpret_cast<uint4*>(dst + 8 * c) = v;
    }
    __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
    __builtin_amdgcn_wave_barrier();
    __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
  }
}

}  // namespace dense

}  // namespace moe
