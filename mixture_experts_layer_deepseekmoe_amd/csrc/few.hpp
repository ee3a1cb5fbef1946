// Internal launcher interface of the layer's forward for a few tokens (few.hip).
#pragma once

#include "kernels.hpp"

namespace moe {

constexpr int FEW_TOKENS = 64;   // a token per bit of an expert's 64-bit mask

struct FewArgs {
  const void* u;            // [T][d] x_fmt
  const void* centroids;    // [N_r][d] x_fmt
  const float* bias;        // [N_r]
  const void* w_gate_up;    // [N_r][2I][d] w_fmt
  const void* w_down;       // [N_r][d][I]
  const void* ws_gate_up;   // [N_s][2I][d]
  const void* ws_down;      // [N_s][d][I]
  const float* s_gate_up;   // e4m3: the block scales
  const float* s_down;
  const float* ss_gate_up;
  const float* ss_down;
  int T, d, n_routed, n_shared, inter, top_k, n_groups, topk_groups;
  int x_fmt, w_fmt, out_fmt;
  int slices;               // few_slices(...)
  float* logits;            // [slices][T][N_r] partial logits
  int32_t* idx;             // [T][K]
  float* gate;              // [T][K]
  // the rest of the routing, each null where not wanted
  int32_t* counts;          // [N_r]
  int32_t* offsets;         // [N_r + 1]
  int32_t* perm_token;      // [T*K]
  int32_t* pos;             // [T][K]
  // SwiGLU outputs by grouped row (expert-major, tokens ascending; then the shared experts'): fp32 values, or
  // their bf16 roundings (h) and what those left (h_lo)
  void* h;                  // [R][I] f32 (f32 and e4m3 weights) or bf16, and right behind it
  uint16_t* h_lo;           // [R][I] bf16
  uint8_t* hq;              // e4m3: [R][I] codes and [R][I/128] scales
  float* hs;
  uint8_t* uq;              // e4m3: [T][d] codes and [T][d/128] scales
  float* us;
  int splits;               // few_splits(...)
  int32_t* taken;           // gate/up units taken beyond the first round
  float* part;              // [splits][T][d] (more than one split)
  void* y;                  // [T][d] out_fmt
};

// 128-byte runs of a row of `cols` elements.
inline int few_runs(int cols, int fmt) { return cols * (fmt == FMT_F32 ? 4 : fmt == FMT_BF16 ? 2 : 1) / 128; }

// The router's K slices: a block takes 16 experts and a slice of K, a run of 128
// bytes a wave at a time, so one run for each of its 8 waves at least.  They go by the
// row alone: a token's logits, and with them its experts and gates, are then the same,
// bit for bit, in every batch (scores may be level to fp32's rounding).  At most 16, us:
// d = 7168 in bf16 1 token 153.6, 8 tokens 897, 64 tokens 3191; at most 8: 154.0, 898,
// 3192; one slice of 64 tokens (16 blocks) takes 29 more.
inline int few_slices(int d, int x_fmt) {
  const int most = (few_runs(d, x_fmt) + 7) / 8;
  return most < 16 ? most : 16;
}

// Blocks that share 16 columns of y, each a part of the experts' runs, where the
// columns alone leave CUs idle (two blocks to a CU are asked for) and each block has a
// number of runs left: with 64 at least, without splits and with 32, us, d = 2048 in
// bf16 (the one width at which the number was measured): 1 token 40.1, 42.9, 44.5; 8 tokens 138, 163, 136; 32 tokens 242, 296, 237; 64
// tokens 304, 422, 305.  More than one block but less than two to a CU: four splits even
// the CUs' shares out, once there is work for them; one split and four, us: d = 7168
// (448 blocks) in bf16 1 token (288 runs) 153, 164, 2 tokens (544) 292, 289, 32 tokens
// 2389, 2357, 64 tokens 3358, 3198, in 8 bits 2 tokens (272 runs) 171, 179, 64 tokens
// 1734, 1667; d = 5120 (320 blocks) in bf16 2 tokens (336 runs) 151, 147, 64 tokens 818,
// 692: the border lies between 288 and 336 runs, in 8 bits between 272 and 64 tokens'.  From 512 blocks on it does not pay: 768, 2 tokens 194, 236.
constexpr int FEW_SPLITS = 16, FEW_SPLIT_RUNS = 64, FEW_EVEN_RUNS = 320;
inline int few_splits(int T, int d, int n_routed, int n_shared, int inter, int top_k, int w_fmt) {
  const int blocks = d / 16, tk = T * top_k;
  const long long runs = static_cast<long long>((tk < n_routed ? tk : n_routed) + n_shared) * few_runs(inter, w_fmt);
  if (blocks > 256 && blocks < 512) return runs >= FEW_EVEN_RUNS ? 4 : 1;
  int s = 512 / blocks;
  if (s > FEW_SPLITS) s = FEW_SPLITS;
  while (s > 1 && runs < static_cast<long long>(s) * FEW_SPLIT_RUNS) --s;
  return s > 1 ? s : 1;
}

hipError_t launch_few_route(const FewArgs& a, hipStream_t s);
hipError_t launch_few_gateup(const FewArgs& a, hipStream_t s);
hipError_t launch_few_quant(const FewArgs& a, hipStream_t s);   // e4m3 only
hipError_t launch_few_down(const FewArgs& a, hipStream_t s);

#ifdef MOE_DEBUG
int debug_take_few();   // check ids 8xx
#endif

}  // namespace moe
