// Internal launcher interface of a model's two ends: the embedding with its
// gradient (embed.hip), the gradients' norm and clipping (grads.hip).
#pragma once

#include "kernels.hpp"

namespace moe {

// x = scale table[token], and the norm of x as stored.
struct EmbedArgs {
  const int32_t* tokens;  // [T]; outside [0, V): a row of zeros
  const void* table;      // [V][d] table_fmt
  const float* w_next;    // [d], or null: no norm
  int T, d, V, table_fmt, x_fmt, n_fmt;
  float scale, eps;
  void* x;                // [T][d]
  void* n;                // [T][d] (with w_next)
  float* rstd;            // the rest: null where not wanted
  uint8_t* codes;
  float* scales;
};

// A token of many rows is summed by many waves: the sums of 16 sorted rows that are all
// of one token are formed apart, and of batches of some size those of 256 from them.  Of n
// rows the longest sum of one wave is then 30 rows, 30 sums of 16 and n / 256 of 256; of
// smaller batches 30 rows and n / 16 sums of 16 (543 terms at most).
constexpr int EMBED_CHUNK = 16, EMBED_CHUNK2 = 256, EMBED_PART2_T = 8192;
constexpr int EMBED_RADIX_BLOCK = 4096;   // rows of a radix block
// Rows are ranked by comparing each with all others up to this many (one launch, T^2
// compares), by a radix sort beyond (three launches for every 8 bits of V).
constexpr int EMBED_RANK_T = 16384;

struct EmbedBwdArgs {
  const int32_t* tokens;  // [T]
  const float* dx;        // [T][d]
  int T, d, V, grad_fmt, accumulate;
  float scale;
  int32_t* ids;           // [T] sorted tokens (V: outside [0, V)), and
  int32_t* order;         // [T] the row of each
  int32_t* ids2;          // radix: the other copy of both
  int32_t* order2;
  int32_t* hist;          // radix: [256][blocks]
  float* part;            // [T / EMBED_CHUNK][d]
  float* part2;           // [T / EMBED_CHUNK2][d] (T at least EMBED_PART2_T)
  void* dtable;           // [V][d] grad_fmt
};
inline int embed_radix_blocks(int T) { return T > EMBED_RANK_T ? ceil_div(T, EMBED_RADIX_BLOCK) : 0; }
inline int embed_radix_passes(int V) {   // 8 bits of the keys 0 .. V each
  return V < (1 << 8) ? 1 : V < (1 << 16) ? 2 : V < (1 << 24) ? 3 : 4;
}

hipError_t launch_embed(const EmbedArgs& a, hipStream_t s);
hipError_t launch_embed_bwd(const EmbedBwdArgs& a, hipStream_t s);

// The gradients' tensors, as many as a launch's arguments hold.
constexpr int GRAD_TENSORS = 112;
constexpr int GRAD_CHUNK = 4096;    // elements of a block's turn
constexpr int GRAD_BLOCKS = 4096;   // blocks of a sum's launch: a partial sum each
struct GradArgs {
  const void* data[GRAD_TENSORS];
  void* out[GRAD_TENSORS];          // clipping only
  long long numel[GRAD_TENSORS];
  uint32_t first[GRAD_TENSORS + 1]; // chunks before tensor i (numbers below 2^32)
  uint8_t bf16[GRAD_TENSORS];       // bit 0: data, bit 1: out
  int n;
};

hipError_t launch_grad_sumsq(const GradArgs& a, double* part, hipStream_t s);
hipError_t launch_grad_finish(const double* part, long long n, double* sumsq, hipStream_t s);
hipError_t launch_grad_clip(const GradArgs& a, const double* sumsq, double max_norm, float* norm, hipStream_t s);
inline int grad_blocks(const GradArgs& a) {
  const uint32_t n = a.first[a.n];
  return static_cast<int>(n < static_cast<uint32_t>(GRAD_BLOCKS) ? n : GRAD_BLOCKS);
}

#ifdef MOE_DEBUG
int debug_take_embed();   // check ids 9xx
int debug_take_grads();   // 10xx
#endif

}  // namespace moe
