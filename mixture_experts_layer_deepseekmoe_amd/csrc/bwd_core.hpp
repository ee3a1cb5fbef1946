// Tile pipeline of the backward GEMMs: 256 x 256 outputs, 8 MFMA waves (2 x 4,
// 128 x 64 each, bf16 16x16x32 MFMAs accumulating in place) and 4 load waves
// that move 32-K stages into a ring of LDS buffers by DMA.  An operand is
// stored either K-contiguous (rows of K) or K-outer (rows along K, its M or N
// index contiguous).  K-outer fragments come from LDS transpose reads
// (ds_read_b64_tr_b16): lane 16 g + c of a read points at K-row 8 g + c / 4,
// columns 4 (c % 4) .. + 3, and receives the four K-rows 8 g .. 8 g + 3 of
// column 4 (c / 4)' ... -- i.e. each lane gets four consecutive K values of
// its own column; two reads give the eight a 16x16x32 MFMA operand holds.
#pragma once

#include "gemm_core.hpp"

namespace moe {

namespace bt {

constexpr int BT = 256;                 // tile rows and columns
constexpr int NSTG = 5;                 // stage buffers (5 x 32 KB: all of the LDS)
constexpr int NMW = 8;                  // MFMA waves
constexpr int NLW = 4;                  // load waves
constexpr int THREADS = 64 * (NMW + NLW);
constexpr int OPB = 16384;              // bytes of one operand in a stage (256 x 32 bf16)
constexpr int STB = 2 * OPB;            // stage bytes (A then B)
constexpr int NLI = 4;                  // DMA instructions per operand per stage and load wave
constexpr int NLS = 2 * NLI;            // ... for both operands
constexpr int MI = 8, NJ = 4;           // accumulator subtiles per MFMA wave

enum : int { KC = 0, KO = 1 };

typedef int i32x2 __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x4 __attribute__((ext_vector_type(4)));
typedef __attribute__((address_space(3))) bf16x4 lds_bf16x4;

// K-outer stage rows are 512 bytes (256 bf16); the 16-byte chunk of a row is
// xor-ed with a function of the K-row that gives the 16 rows one transpose
// read touches (8 g + j, g, j = 0..3) 16 different chunk positions.
__device__ __forceinline__ int xko(int k) { return (k & 3) | (((k >> 3) & 3) << 2); }

__device__ __forceinline__ i32x4 frag_kc(const uint8_t* op, int r0) {
  const int lane = threadIdx.x & 63;
  const int r = r0 + (lane & 15);
  return *reinterpret_cast<const i32x4*>(op + r * 64 + (((lane >> 4) ^ swz<64>(r)) << 4));
}

// The lane's constants for K-outer fragment reads.  Lane 16 g + c reads
// K-rows k0 = 8 g + c / 4 and k0 + 4, columns c0 + 4 (c % 4) .. + 3 of a
// 16-column subtile at c0 (a multiple of 16): byte (col % 8) * 2 = 8 (c % 2)
// of chunk col / 8 = c0 / 8 + (c % 4) / 2, stored at chunk position
// (col / 8) ^ xko(k0) (xko(k0 + 4) = xko(k0)); c0 / 8 is even, so that is
// (c0 / 8) ^ y with y = (c % 4) / 2 ^ xko(k0).
struct KoLane {
  int base;   // k0 * 512 + 8 (c % 2)
  int y;
};
__device__ __forceinline__ KoLane ko_lane() {
  const int lane = threadIdx.x & 63;
  const int g = lane >> 4, c = lane & 15;
  const int k0 = 8 * g + (c >> 2);
  return {k0 * 512 + 8 * (c & 1), ((c & 3) >> 1) ^ xko(k0)};
}

__device__ __forceinline__ i32x4 frag_ko(const uint8_t* op, int c0, KoLane kl) {
  const uint8_t* p0 = op + kl.base + ((((c0 >> 3) ^ kl.y)) << 4);
  const bf16x4 lo = __builtin_amdgcn_ds_read_tr16_b64_v4bf16((lds_bf16x4*)(const_cast<uint8_t*>(p0)));
  const bf16x4 hi = __builtin_amdgcn_ds_read_tr16_b64_v4bf16((lds_bf16x4*)(const_cast<uint8_t*>(p0 + 4 * 512)));
  const i32x2 a = __builtin_bit_cast(i32x2, lo), b = __builtin_bit_cast(i32x2, hi);
  return i32x4{a.x, a.y, b.x, b.y};
}

// One operand's loads: a buffer resource over its valid bytes (reads past it
// return zeros), per-lane byte offsets of the lane's NLI 16-byte pieces at
// K-step 0, and the bytes one K-step advances.
struct Opnd {
  rsrc_t r;
  uint32_t off[NLI];
  uint32_t kstride;
};

// K-contiguous operand: tile row m at byte row_off(m) of the resource, its
// 32-K steps 64 bytes apart.
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

// K-outer operand: K-row k at byte k * ld, the tile's columns from col0; a
// K-step is 32 rows.
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

__device__ __forceinline__ void issue_stage(const Opnd& a, const Opnd& b, uint8_t* st, int ks) {
  const int w = wave_id() - NMW;
#pragma unroll
  for (int q = 0; q < NLI; ++q) {
    dma16(a.r, a.off[q], ks * a.kstride, st + 1024 * (w + NLW * q));
    dma16(b.r, b.off[q], ks * b.kstride, st + OPB + 1024 * (w + NLW * q));
  }
}

// acc[i][j][r] = C[16 (2 i + wm) + lane % 16][64 wn + 16 j + 4 (lane / 16) + r]
// summed over K-steps 0 .. nk-1 (A: the M side, B: the N side).  Returns on
// every wave; one barrier per K-step keeps the roles in step:
//   before barrier ks  stages ks and ks+1 have landed (the load waves waited
//                      for them);
//   after barrier ks   nobody reads stage ks-1 any more, and the load waves
//                      refill its buffers.
// So the MFMA waves read the next stage's first fragments (its weight side
// and first activation subtile) at the end of a stage, and within a stage
// read each activation fragment one subtile ahead of its MFMAs: no LDS read
// latency stands between a barrier and the first MFMA.
//
// The Dgrad K loop (A K-contiguous, B K-outer) with the A loads paired: a
// K-contiguous row moves 64 bytes per K-step, half a 128-byte line, and two
// halves requested a K-step apart cost an L2 request each, while requested
// back to back they merge into one (B's K-rows are whole lines already).  So
// A is loaded two K-steps at a time into a ring of 3 pair buffers (32 KB),
// B one K-step at a time into a ring of 4 (16 KB): 160 KB in all.  After
// barrier ks the load waves refill B's buffer of stage ks - 1 with
// stage ks + 3 and, for even ks, A's buffer of the pair (ks - 2, ks - 1) with
// the pair (ks + 4, ks + 5).  Loads complete in order, so the wait for stage
// ks + 2 allows exactly the loads issued after it: this step's B and, for an
// even ks (or the step before, for an odd one), the next A pair.
constexpr int PA_A = 0, PA_B = 3 * 2 * OPB;   // A pair buffers, then B buffers
static_assert(PA_B + 4 * OPB <= NSTG * STB, "paired ring fits the stage ring");

__device__ __forceinline__ void issue_a_pair(const Opnd& a, uint8_t* ring, int p, int nk) {
  const int w = wave_id() - NMW;
  uint8_t* st = ring + PA_A + (p % 3) * 2 * OPB;
  const int k0 = 2 * p, k1 = min(2 * p + 1, nk - 1);   // past the end: a clamped load nobody reads
#pragma unroll
  for (int q = 0; q < NLI; ++q) {
    dma16(a.r, a.off[q], k0 * a.kstride, st + 1024 * (w + NLW * q));
    dma16(a.r, a.off[q], k1 * a.kstride, st + OPB + 1024 * (w + NLW * q));
  }
}

__device__ __forceinline__ void issue_b(const Opnd& b, uint8_t* ring, int s) {
  const int w = wave_id() - NMW;
#pragma unroll
  for (int q = 0; q < NLI; ++q) dma16(b.r, b.off[q], s * b.kstride, ring + PA_B + (s % 4) * OPB + 1024 * (w + NLW * q));
}

__device__ __forceinline__ const uint8_t* pa_a(uint8_t* ring, int s) {
  return ring + PA_A + ((s / 2) % 3) * 2 * OPB + (s % 2) * OPB;
}
__device__ __forceinline__ const uint8_t* pa_b(uint8_t* ring, int s) { return ring + PA_B + (s % 4) * OPB; }

template <int NSUB = MI>
__device__ __forceinline__ void mainloop_pa(uint8_t* ring, const Opnd& a, const Opnd& b, int nk,
                                            f32x4 (&acc)[MI][NJ]) {
  static_assert(NSUB >= 1 && NSUB <= MI, "row subtiles");
  const int w = wave_id();
  if (nk <= 0) return;
  if (w >= NMW) {
    // A pair 0, B 0, B 1, A pair 1, B 2: stages 0 and 1 first
    issue_a_pair(a, ring, 0, nk);
    issue_b(b, ring, 0);
    if (nk > 1) issue_b(b, ring, 1);
    if (nk > 2) {
      issue_a_pair(a, ring, 1, nk);
      issue_b(b, ring, 2);
      wait_vm_lgkm0<3 * NLI>();   // A pair 1 and B 2 may be in flight
    } else {
      wait_vm_lgkm0<0>();
    }
    for (int ks = 0; ks < nk; ++ks) {
      block_barrier();
      const bool ib = ks + 3 < nk;
      if (ib) issue_b(b, ring, ks + 3);
      if ((ks & 1) == 0) {
        const bool ia = ks + 4 < nk;
        if (ia) issue_a_pair(a, ring, ks / 2 + 2, nk);
        if (ia)
          wait_vm_lgkm0<3 * NLI>();   // stage ks + 2; this step's B and A pair in flight
        else if (ib)
          wait_vm_lgkm0<NLI>();       // this step's B in flight
        else
          wait_vm_lgkm0<0>();
      } else {
        if (ib)
          wait_vm_lgkm0<3 * NLI>();   // the previous step's A pair and this step's B in flight
        else
          wait_vm_lgkm0<0>();
      }
    }
    return;
  }
  const int wm = w % 2, wn = w / 2;
  KoLane kl = ko_lane();
  i32x4 wf[NJ], xf;
  block_barrier();   // stages 0 and 1 have landed
  {
#pragma unroll
    for (int j = 0; j < NJ; ++j) wf[j] = frag_ko(pa_b(ring, 0), 64 * wn + 16 * j, kl);
    xf = frag_kc(pa_a(ring, 0), 16 * wm);
  }
  acc_fence(acc);
  for (int ks = 0; ks < nk; ++ks) {
    asm volatile("" : "+v"(kl.base), "+v"(kl.y));
    const uint8_t* sa = pa_a(ring, ks);
#pragma unroll
    for (int i = 0; i < NSUB; ++i) {
      i32x4 xn;
      if (i + 1 < NSUB) xn = frag_kc(sa, 16 * (2 * (i + 1) + wm));
      __builtin_amdgcn_sched_barrier(0);
#pragma unroll
      for (int j = 0; j < NJ; ++j) mfma_bf16_tied(acc[i][j], wf[j], xf);
      __builtin_amdgcn_sched_barrier(0);
      if (i + 1 < NSUB) xf = xn;
    }
    if (ks + 1 < nk) {
      const uint8_t* nb = pa_b(ring, ks + 1);
#pragma unroll
      for (int j = 0; j < NJ; ++j) wf[j] = frag_ko(nb, 64 * wn + 16 * j, kl);
      xf = frag_kc(pa_a(ring, ks + 1), 16 * wm);
      block_barrier();
    }
  }
  acc_fence(acc);
}

// f.template operator()<NSUB>() with NSUB = the row subtiles wave row 0
// computes for a tile of `rows` rows (two wave rows of 16-row subtiles).
template <int N = 1, class F>
__device__ __forceinline__ void with_row_subtiles(int rows, F&& f) {
  if constexpr (N >= MI)
    f.template operator()<MI>();
  else if (rows <= 32 * N)
    f.template operator()<N>();
  else
    with_row_subtiles<N + 1>(rows, f);
}

__device__ __forceinline__ uint2 pack4(const f32x4& v) { return make_uint2(bf16x2(v[0], v[1]), bf16x2(v[2], v[3])); }

__device__ __forceinline__ void unpack4(uint2 p, float (&v)[4]) {
  v[0] = bf16_to_f32(static_cast<uint16_t>(p.x & 0xffffu));
  v[1] = bf16_to_f32(static_cast<uint16_t>(p.x >> 16));
  v[2] = bf16_to_f32(static_cast<uint16_t>(p.y & 0xffffu));
  v[3] = bf16_to_f32(static_cast<uint16_t>(p.y >> 16));
}

}  // namespace bt

}  // namespace moe
