// ns_sublayer.h - arguments, launch rules and launch interface of the
// mixture-of-experts sublayer's kernels: layer norm, routing, the experts'
// products, combine.
#pragma once

#include <hip/hip_runtime_api.h>
#include <stddef.h>
#include <stdint.h>

#include "../../include/ns_hip.h"
#include "ns_layout.h"

namespace ns {

// Whether an array is more than the L2s hold (8 of 4 MiB).  Outputs that are
// then leave them at once (store_whole): layer norm and gradient of 8192 x 7168
// bf16 111 us, 123 without; combine's gradient of 8192 x 8 rows of 2048 and its
// forward pass 175 and 189; the weight gradient of 128 x 1536 x 2048 from 65536
// rows 452 and 532, from 16384 rows 201 and 262, from 32 rows 138 and 136 (the
// same inputs again and again: what an output no longer displaces is then what
// the next call reads).
inline bool beyond_l2(long long bytes) { return bytes > (32ll << 20); }

// ------------------------------------------------------------ layer norm

struct LayerNormArgs {
  const void* x;  // [rows, cols], rows ldx elements apart
  const void *w, *b;  // [cols] or null
  void* y;        // [rows, cols] contiguous
  float *mean, *rstd;  // [rows] or null
  long long rows, ldx;
  int cols, param_dtype;
  float eps;
  bool stream;  // y is beyond_l2 (set at the launch, as below)
};
struct LayerNormGradArgs {
  const void *dy, *x;  // rows lddy / ldx elements apart
  const void* w;       // [cols] or null
  const float *mean, *rstd;
  void* dx;            // [rows, cols] contiguous, or null
  void *dw, *db;       // [cols] or null
  float* partials;     // [blocks][2][cols], null if neither dw nor db is wanted
  long long rows, lddy, ldx;
  int cols, param_dtype;
  bool stream;
};

// A row is held by tpr threads of vpt vectors of 8 elements (vpt 0: too long
// for the registers).  It goes by the row's length alone, so that a row's
// result does not hang on how many rows there are.  A wave holds up to 2048
// columns and needs no barrier for its sums; longer rows take a whole block,
// of as few waves as hold the row.  Forward / backward us, as here and as the
// next shape would have it (bf16):
//   8192 x 1024   64 x 2    7.8 / 17    256 x 1   14 / 23
//   8192 x 2048   64 x 4     14 / 26    256 x 1   16 / 27
//   8192 x 4096   256 x 2    25 / 41    64 x 8    30 / 56
//   8192 x 7168   256 x 4    38 / 79    1024 x 1  51 / 84
//   2048 x 12288  1024 x 2   24 / 40    1024 x 4  37 / 270, 1024 x 0  29 / 245
//   1024 x 32768  1024 x 4   33 / 196   1024 x 0  37 / 316
// 1024 x 4 spills 226 to 303 registers in the backward pass, and still beats
// reading rows again.  Rows of no whole vectors need more of them: 1024 x 4
// spills 154 to 166 forward too, 1024 x 2 22 to 31 backward:
//   2048 x 12287  1024 x 2   46 / 74    (fp32 47 / 100)
//   1024 x 32767  1024 x 4   96 / 426   (fp32 130 / 358)
struct NormShape {
  int tpr, vpt;
};
inline NormShape norm_shape(int cols) {
  const int nv = (cols + 7) / 8;
  return nv <= 64     ? NormShape{64, 1}
         : nv <= 128  ? NormShape{64, 2}
         : nv <= 256  ? NormShape{64, 4}
         : nv <= 512  ? NormShape{256, 2}
         : nv <= 1024 ? NormShape{256, 4}
         : nv <= 2048 ? NormShape{1024, 2}
         : nv <= 4096 ? NormShape{1024, 4}
                      : NormShape{1024, 0};
}
// columns of a row of partial sums: whole vectors
NS_HD constexpr int partials_ld(int cols) { return (cols + 7) / 8 * 8; }
// Blocks: enough to fill the card; in the backward pass as few as do, since
// each leaves partial sums.  8192 x 7168 backward with 256 / 512 / 1024 blocks:
// 85 / 79 / 89 us; 2048 x 16384, where one block fills a CU: 50 / 70 / 100 us.
constexpr int kNormForwardBlocks = 2048, kNormBackwardBlocks = 512, kNormLongBackwardBlocks = 256;
inline long long norm_blocks(long long rows, NormShape s, long long most) {
  const long long need = s.tpr == 64 ? (rows + 3) / 4 : rows;
  return need < most ? need : most;
}
// Blocks of the backward pass: each has 8 bytes of partial sums per column,
// so long rows get fewer (at most 256 MiB of partials).
inline int norm_backward_blocks(long long rows, int cols) {
  const NormShape s = norm_shape(cols);
  long long most = s.tpr == 1024 ? kNormLongBackwardBlocks : kNormBackwardBlocks;
  const long long fit = (1ll << 28) / (8ll * partials_ld(cols));
  if (most > fit) most = fit > 0 ? fit : 1;
  return (int)norm_blocks(rows, s, most);
}

hipError_t launch_layer_norm(int dtype, const LayerNormArgs& g, hipStream_t st);
// blocks: norm_backward_blocks (0 with no rows: dw and db become zero)
hipError_t launch_layer_norm_backward(int dtype, const LayerNormGradArgs& g, int blocks, hipStream_t st);

// --------------------------------------------------------------- routing

constexpr int kMaxExperts = 1024, kMaxTopK = 64, kMaxGroups = 64;
constexpr int kRouteLeastWaves = 8, kRouteWaves = 16;  // waves of a routing block, where it is not the only one
// Up to so many blocks each adds up the other blocks' counts itself, beyond
// them a scan does: that costs a launch, the other time that grows with the
// blocks.  16384 x 256 (256 blocks) 20.2 us without a scan, 22.3 with one;
// 8192 x 512 (512 blocks) 42 and 33 us.
constexpr int kRouteUnscannedBlocks = 256;
// of the one block that few tokens take: with more than 256 experts 8 waves, which leave a thread 256 registers
// (with more than 512, and a bias or groups, it needs 52 more: 8 x 1024 12 us, by logits 5 to 7)
constexpr int route_single_waves(int experts) { return experts > 256 ? kRouteWaves / 2 : kRouteWaves; }

struct RouteArgs {
  const void* logits;  // [tokens, experts], rows ld elements apart
  const float* bias;   // [experts] or null
  int* ids;            // [tokens, top_k]
  float* weights;      // [tokens, top_k]
  int *offsets, *rows, *slots;  // [experts + 1], [tokens * top_k], [tokens, top_k]; all null: no plan
  int* hist;           // workspace [blocks][hist_ld] counts, then [hist_ld] totals
  long long ld;
  int tokens, experts, top_k, groups, top_groups, group_best, score, renormalize, hist_ld;
  float scale;
  bool vec, vec_bias;  // logits, bias as whole vectors (set at the launch)
};
struct RouteGradArgs {
  const void* logits;
  const int* ids;
  const float* dweights;
  void* dlogits;       // [tokens, experts] contiguous
  long long ld;
  int tokens, experts, top_k, score, renormalize;
  float scale;
  bool vec, vec_out;
};
static_assert(route_single_waves(kMaxExperts) >= kRouteLeastWaves, "tokens for more than one block make more than one");
// A token takes a whole wave, or 16 lanes where the tokens fill the card and
// there are at most 256 experts: four tokens then share a wave's instructions,
// while a lane has four times the experts to go through.  512 x 256: 13.4 us
// with a wave each, 20.7 with 16 lanes; 4096 x 128: 13.2 and 15.3;
// 16384 x 128: 35 and 18.  A block has few waves as long as there are at most
// kRouteUnscannedBlocks blocks (8 waves and 16: 512 x 256 12.2 and 13.4 us,
// 8192 x 256 20.3 and 23.2).  As many tokens as one block has waves take one
// block and one launch (32 x 128 in two blocks 9.0 us, in one 12.5).
struct RouteShape {
  int tokens_per_wave, waves, blocks, hist_ld;
};
inline RouteShape route_shape(int tokens, int experts) {
  RouteShape r{1, route_single_waves(experts), 1, (experts + 3) / 4 * 4};
  if (tokens <= r.waves) {
    if (tokens > 0) r.waves = tokens;
    return r;
  }
  if (experts <= 256 && tokens > kRouteWaves * kRouteUnscannedBlocks) r.tokens_per_wave = 4;
  for (r.waves = kRouteLeastWaves;; r.waves *= 2) {
    const int tb = r.waves * r.tokens_per_wave;
    r.blocks = (int)(((long long)tokens + tb - 1) / tb);
    if (r.blocks <= kRouteUnscannedBlocks || r.waves == kRouteWaves) return r;
  }
}
inline size_t route_workspace(int tokens, int experts) {
  const RouteShape r = route_shape(tokens, experts);
  return r.blocks > 1 ? (size_t)(r.blocks + 1) * r.hist_ld * sizeof(int) : 0;
}
hipError_t launch_route(int dtype, const RouteArgs& g, hipStream_t st);
hipError_t launch_route_backward(int dtype, const RouteGradArgs& g, hipStream_t st);

// --------------------------------------------------- the experts' products

// Sorted rows: row i belongs to expert e for offsets[e] <= i < offsets[e + 1].
// Offsets are device data: they are clamped to [0, n_rows], and a row number
// outside [0, n_x) reads as a row of zeros.
enum ExpertsMode : int {
  EXP_PRODUCT = 0,     // out[i] = x[rows[i]] W_eᵀ
  EXP_INPUT_GRAD = 1,  // out[i] = dy[i] W_e
  EXP_WEIGHT_GRAD = 2  // out[e] = sum over e's rows of dy[i]ᵀ x[rows[i]]
};
struct ExpertsArgs {
  const void* x;       // [n_x, fan_in], rows ldx elements apart (product, weight gradient)
  const void* dy;      // [n_rows, fan_out] (gradients)
  const void* w;       // [experts, fan_out, fan_in] (product, input gradient)
  void* out;
  const int* offsets;  // [experts + 1]
  const int* rows;     // [n_rows], or null: row i of x
  long long ldx;
  int n_x, n_rows, experts, fan_out, fan_in;
  bool stream;
};
// What launch_experts runs, for ns_query_last_config: a format of the type's
// name, n_rows, experts, fan_out and fan_in.
const char* experts_config(int dtype, ExpertsMode mode, const ExpertsArgs& g);
hipError_t launch_experts(int dtype, ExpertsMode mode, const ExpertsArgs& g, hipStream_t st);

// ---------------------------------------------------------------- combine

struct CombineArgs {
  const void* y;         // [n_rows, cols]
  const int* slots;      // [tokens, top_k]: rows of y; one outside [0, n_rows) adds nothing
  const float* weights;  // [tokens, top_k], or null: 1
  void* out;             // [tokens, cols]
  int tokens, top_k, n_rows, cols;
  bool stream;
};
struct CombineGradArgs {
  const void *dout, *y;
  const int* slots;
  const float* weights;
  void* dy;         // [n_rows, cols], or null
  float* dweights;  // [tokens, top_k], or null
  int tokens, top_k, n_rows, cols;
  bool stream;
};
hipError_t launch_combine(int dtype, const CombineArgs& g, hipStream_t st);
hipError_t launch_combine_backward(int dtype, const CombineGradArgs& g, hipStream_t st);

}  // namespace ns
