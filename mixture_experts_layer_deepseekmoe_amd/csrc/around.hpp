// Internal launcher interface of what stands around the layer: the norms before
// and after a block (block.hip) and the cross entropy over a vocabulary
// (loss.hip).  Every launcher enqueues on the given stream and returns the
// launch status.
#pragma once

#include "kernels.hpp"

namespace moe {

// The norm before a block (block.hip).  Null where not wanted: rstd, codes and
// scales (the checkpoint of x).
struct BlockInArgs {
  const void* x;          // [T][d] x_fmt
  const float* w;         // [d]
  int T, d, x_fmt, n_fmt;
  float eps;
  void* n;                // [T][d] n_fmt
  float* rstd;            // [T]
  uint8_t* codes;         // [T][d]
  float* scales;          // [T][d/128]
};

// The norm, gate and residual after a block, and the next block's norm.
struct BlockOutArgs {
  const void* x;          // [T][d] x_fmt
  const void* y;          // [T][d] y_fmt
  const void* skip;       // [T][d] n_fmt, or null: nothing to subtract
  const float* w;         // [d], or null: no norm
  const float* gate;      // [ceil(T / gate_rows)][d] (gate_rows 0: one row), or null: ones
  const float* w_next;    // [d], or null: no next norm
  int T, d, x_fmt, n_fmt, y_fmt, gate_rows;
  long long gates;        // rows of gate
  float eps, res_scale;
  void* x_out;            // [T][d] x_fmt
  void* n_next;           // [T][d] n_fmt (with w_next)
  float* rstd;            // the rest: null where not wanted
  uint8_t* codes;         // checkpoint of y - skip
  float* scales;
  float* rstd_next;
  uint8_t* codes_next;    // checkpoint of x_out
  float* scales_next;
};

// The backward of either: dv = d(v r w) for g, dw, dgate.
struct BlockBwdArgs {
  const float* g;         // [T][d] upstream
  const float* g_sub;     // [T][d] subtracted from g, or null
  const float* res;       // [T][d]: dv += res_scale * res, or null
  const void* v;          // [T][d] v_fmt rows, or null (codes; or neither norm nor gate)
  const void* skip;       // [T][d] skip_fmt subtracted from v, or null
  const uint8_t* codes;   // [T][d] checkpoint of v (read where v is null)
  const float* scales;    // [T][d/128]
  const float* w;         // [d], or null: no norm
  const float* gate;      // [gates][d], or null: ones
  const float* rstd;      // [T] (with w)
  int T, d, v_fmt, skip_fmt;
  long long gate_len;     // rows per gate (>= 1)
  long long gates;
  float res_scale;
  float* dv;              // [T][d]
  float* dw;              // [d], or null
  float* dgate;           // [gates][d], or null
  float* part;            // block_bwd_floats(...) of scratch
  // set by the launcher (block_bwd_plan)
  int whole_gates, runs, rows;
  long long blocks;
};

// A backward block takes `rows` rows and leaves one row of partial column sums
// (d floats, written and read again: 8 bytes a column beside the 9 to 20 of each of its
// rows).  Long batches take 16 rows to a block, where that is 3 to 6% of the rows'
// traffic; short ones trade it for parallelism, down to one row to a block (as much
// as 90%): 512 blocks, two to a CU.  Measured: 517 x 1992 with 16 rows to a block 27 us,
// with 2 rows 7; 8192 x 7168 with 8 rows to a block 3% slower than with 16.
struct BlockBwdPlan {
  int rows;
  int whole_gates;        // gates of at most `rows` rows, whole ones to a block
  int runs;               // else: blocks per gate
  long long gates, blocks;
};
inline BlockBwdPlan block_bwd_plan(long long T, long long gate_len, long long gates, bool has_gate) {
  BlockBwdPlan p{};
  p.gates = gates;
  p.rows = static_cast<int>(T <= 512 ? 1 : (T + 511) / 512);
  if (p.rows > 16) p.rows = 16;
  p.whole_gates = has_gate && T > 0 && gate_len <= p.rows;
  if (p.whole_gates) {
    const long long n = gate_len * (p.rows / gate_len);
    p.blocks = (T + n - 1) / n;
  } else {
    p.runs = static_cast<int>((gate_len + p.rows - 1) / p.rows);
    p.blocks = gates * p.runs;
  }
  return p;
}
inline long long block_bwd_floats(const BlockBwdPlan& p, int d) {
  return (p.blocks + (!p.whole_gates && p.gates != 1 ? p.gates : 0)) * d;
}

// Cross entropy over the vocabulary (loss.hip).  "Row" r is the r-th token with
// a label in [0, V); the other tokens take no part.
struct LossArgs {
  const uint16_t* h;      // [T][d] bf16 hidden rows
  const uint16_t* w;      // [V][d] bf16 vocabulary matrix
  const int32_t* labels;  // [T]
  int T, d, V;
  int32_t* rows;          // [T] token of each row
  int32_t* pos;           // [T] row of each token, or -1
  int32_t* count;         // [3] rows; backward: splits of dh's sum, the gradients' scale (fp32)
  // what the workspace holds, for the checks of the debug build
  long long g_rows, acc_rows;
  float* loss;            // [T] (forward)
  float* lse;             // [T] (backward: read)
  // forward
  float2* part;           // [T][tiles] each row's (max, sum exp(l - max)) by tile
  int tiles;              // loss_tiles(...)
  float* zlab;            // [T] the label's logit by row
  // backward
  const float* dloss;     // [T]
  const float* dlse;      // [T], or null
  uint16_t* hc;           // [loss_k_rows(T)][d] the rows' hidden rows, one after the other
  uint16_t* g;            // [g_rows = loss_g_rows(T, pairs)][ldg] a piece's G = dlogits / scale
  float* lab_lo;          // [T] by row: the rounding error of G at the label
  int32_t* lab_first;     // [tiles of V + 1] where loss_labels: a tile's first entry of
  uint32_t* lab_list;     // [T] rows by their label's tile: row << 8 | label % 256
  float* acc;             // [splits][row tiles of 256][d] dh by row (loss_acc_rows)
  int ldg;                // loss_piece
  int dh_fmt, dw_fmt;     // fp32: from pairs of bf16 values of G
  void* dh;               // [T][d]
  void* dw;               // [V][d]
  // the piece of the vocabulary: columns v_first .. v_first + v_len - 1
  int v_first, v_len;
};

constexpr int LOSS_TILE = 256;    // rows and columns of a tile
// The logits of few tokens (loss_stream_kernel, tiles of 64 entries) against the tile
// pipeline, by T, d, V (us, forward; stream / tiles):
//   up to 16 tokens   1, 2048, 32000: 26 / 36; 16, 512, 10007 with backward: 44 / 54;
//                     16, 4096, 65536: 101 / 130; 16, 2048, 131072: 101 / 131; the tiles
//                     win by 14% at most (16, 7168, 50001: 157 / 138; 16, 4096, 131072: 201 / 187)
//   up to 32          two blocks fit a CU: one round of them (32768 entries) wins at any d
//                     (32, 7168, 32000: 104 / 124; 20, 32768, 8192: 170 / 386); beyond it by
//                     the last round and the hidden rows that every block reads again: 32, 4096,
//                     65536: 115 / 131; 32, 2048, 131072: 115 / 132; 20, 2560, 100000: 117 / 122;
//                     but 28, 5120, 40000: 109 / 103; 32, 7168, 57000: 191 / 151; 32, 4096, 131072:
//                     221 / 187; 32, 4096, 50001: 109 / 105 and 32, 512, 500000: 142 / 130 are the
//                     worst within the rule, 32, 7168, 81920: 244 / 266 outside it
//   up to 64          one block to a CU, one round: 64, 1024, 16000: 18 / 23; 64, 7168, 2000: 57 / 79;
//                     64, 32768, 16000: 258 / 411; but 40, 2048, 24000: 37 / 39; 64, 4096, 32000: 79 / 73;
//                     37, 7168, 50001: 192 / 140
// The backward's logits go the same way (16, 2048, 32000 with backward: 135 / 144; 32, 7168,
// 50001: 718 / 635).  T counts the ignored tokens too: the host does not know the labels.
constexpr int LOSS_STREAM_TILE = 64;
inline bool loss_stream(int T, int d, int V) {
  if (T <= 16 || (T <= 64 && V <= 16384)) return true;
  return T <= 32 && (V <= 32768 || (d <= 4096 && static_cast<long long>(V) * d <= 1LL << 28));
}
inline int loss_tiles(int T, int d, int V) {
  return ceil_div(V, loss_stream(T, d, V) ? LOSS_STREAM_TILE : LOSS_TILE);
}

// A gradient in fp32 is summed from G held as pairs of bf16 values, what bf16
// rounds off of G below it (2^-16 of an element is left, where one bf16 value
// leaves 2^-8): one of its two products more.
inline bool loss_pairs(int dh_fmt, int dw_fmt) { return dh_fmt == FMT_F32 || dw_fmt == FMT_F32; }

// The backward's pieces of the vocabulary: as many whole tiles of columns as
// keep G within LOSS_G_BYTES (and a piece of w within 2^31 bytes).
constexpr long long LOSS_G_BYTES = 512LL << 20;
inline int loss_piece(long long T, long long d, long long V, bool pairs) {
  const long long vt = (V + LOSS_TILE - 1) / LOSS_TILE * LOSS_TILE, rows = pairs ? 2 * T : T;
  long long n = LOSS_G_BYTES / (2 * (rows > LOSS_TILE ? rows : LOSS_TILE)) / LOSS_TILE * LOSS_TILE;
  const long long nw = (1LL << 30) / d / LOSS_TILE * LOSS_TILE;
  if (n > nw) n = nw;
  if (n < LOSS_TILE) n = LOSS_TILE;
  return static_cast<int>(n < vt ? n : vt);
}

// dw = G^T h of up to 64 rows sums over 2 count rows in any case: count .. 2 count
// - 1 hold what rounding G to bf16 left, and the same hidden rows again.  The product
// is bound by writing dw; this costs it one or two K-steps.
constexpr int LOSS_LO_ROWS = 64;
constexpr int loss_k_rows(int T) {   // the most there can be
  return T < LOSS_LO_ROWS ? 2 * T : T < 2 * LOSS_LO_ROWS ? 2 * LOSS_LO_ROWS : T;
}
// Of more rows, a bf16 dw takes the rounding errors at the labels alone, tile by
// tile of the vocabulary, from a list of the rows by their label's tile.
inline bool loss_labels(int T, int dw_fmt) { return dw_fmt == FMT_BF16 && T > LOSS_LO_ROWS; }
constexpr long long loss_g_rows(long long T, bool pairs) {
  return pairs ? 2 * T : loss_k_rows(static_cast<int>(T));
}

// dh = G w sums over the whole piece: few rows make few tiles, so the piece is
// cut into up to 64 runs of columns, of a tile's width at least, with an fp32
// copy of dh each; their number is chosen on the device, where the rows are
// known, and keeps the copies' tiles within LOSS_SPLIT_TILES (512 MB).
constexpr int LOSS_SPLITS = 64, LOSS_SPLIT_TILES = 2048;
inline long long loss_acc_rows(long long T, long long d, long long piece) {   // rows of the copies together
  const long long nm = (T + LOSS_TILE - 1) / LOSS_TILE, nn = (d + LOSS_TILE - 1) / LOSS_TILE;
  const long long s = piece / LOSS_TILE < LOSS_SPLITS ? piece / LOSS_TILE : LOSS_SPLITS;
  long long tiles = nm * s < LOSS_SPLIT_TILES / nn ? nm * s : LOSS_SPLIT_TILES / nn;
  if (tiles < nm) tiles = nm;
  return tiles * LOSS_TILE;
}

hipError_t launch_loss_rows(const LossArgs& a, hipStream_t s);
hipError_t launch_loss_forward(const LossArgs& a, hipStream_t s);
hipError_t launch_loss_gather(const LossArgs& a, hipStream_t s);
hipError_t launch_loss_piece(const LossArgs& a, hipStream_t s);
hipError_t launch_loss_dh(const LossArgs& a, hipStream_t s);

hipError_t launch_block_in(const BlockInArgs& a, hipStream_t s);
hipError_t launch_block_out(const BlockOutArgs& a, hipStream_t s);
hipError_t launch_block_bwd(BlockBwdArgs a, hipStream_t s);

#ifdef MOE_DEBUG
// As the other files' (kernels.hpp).  Check ids: 6xx block norms, 7xx loss.
int debug_take_block();
int debug_take_loss();
#endif

}  // namespace moe
