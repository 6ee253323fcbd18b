// ns_scaled.h - arguments, launch rules and launch interface of RMS norm and of
// the operators on 8-bit values with scales: quantization, the experts' product.
#pragma once

#include <hip/hip_runtime_api.h>
#include <stddef.h>
#include <stdint.h>

#include "../../include/ns_hip.h"
#include "ns_layout.h"
#include "ns_sublayer.h"

namespace ns {

// Columns of a row, and rows of a weight, that share a scale; blocks of n.
constexpr int kScaleBlock = 128;
NS_HD constexpr long long scale_blocks(long long n) { return (n + kScaleBlock - 1) / kScaleBlock; }

// -------------------------------------------------------------- RMS norm

struct RmsNormArgs {
  const void *x, *residual;  // [rows, cols], rows ldx / ldr elements apart; residual null: none
  const void* w;             // [cols] or null
  void *total, *y;           // [rows, cols] contiguous; total with a residual, y or null
  uint8_t *q, *scales;       // [rows, cols], [rows, blocks], or both null
  float* rstd;               // [rows] or null
  long long rows, ldx, ldr;
  int cols, param_dtype;
  float eps;
  bool stream;  // the outputs are beyond_l2 (set at the launch, as below)
};
struct RmsNormGradArgs {
  const void *dy, *x, *dtotal;  // rows lddy / ldx / lddt elements apart; dtotal null: zeros
  const void* w;                // [cols] or null
  const float* rstd;
  void* dx;         // [rows, cols] contiguous, or null
  void* dw;         // [cols] or null
  float* partials;  // [blocks][partials_ld(cols)], null if dw is not wanted
  long long rows, lddy, ldx, lddt;
  int cols, param_dtype;
  bool stream;
};
// Rows are held as layer norm's, but for those of no whole vectors and 1025 to 2048
// columns: single columns are as many loads as there are columns to a thread, and
// 256 threads have 8 where 64 have 32.  Forward and backward, us, fp32, 256 x 1 and
// 64 x 4: 8192 x 2047 100 / 119, 8192 x 1531 85 / 100 (bf16 77 / 75); of 777 columns
// 65, 64 x 2 48.
inline NormShape rms_shape(int cols) {
  return cols % 8 != 0 && cols > 1024 && cols <= 2048 ? NormShape{256, 1} : norm_shape(cols);
}
inline int rms_backward_blocks(long long rows, int cols) {
  return (int)norm_blocks(rows, rms_shape(cols), norm_backward_blocks(1ll << 40, cols));  // as many at most
}
hipError_t launch_rms_norm(int dtype, const RmsNormArgs& g, hipStream_t st);
// blocks: rms_backward_blocks (0 with no rows: dw becomes zero)
hipError_t launch_rms_norm_backward(int dtype, const RmsNormGradArgs& g, int blocks, hipStream_t st);

// ---------------------------------------------------------- quantization

struct QuantizeArgs {
  const void* x;  // [rows, cols], rows ldx elements apart
  uint8_t *q, *scales;
  long long ldx;
  unsigned rows, cols, blocks;  // blocks: of a row
};
struct QuantizeWeightsArgs {
  const void* w;                  // [experts, fan_out, fan_in]
  uint8_t *q, *scales;            // the same, and [experts, blocks, blocks]
  uint8_t *qt, *scales_t;         // [experts, fan_in, fan_out] and its blocks, or null
  int experts, fan_out, fan_in;
};
struct DequantizeArgs {
  const uint8_t *q, *scales;
  void* x;
  unsigned rows, cols, blocks;    // all matrices' rows
  unsigned matrix_rows, matrix_blocks;  // of one matrix, and its blocks of rows (weights)
};
hipError_t launch_quantize(int dtype, const QuantizeArgs& g, hipStream_t st);
hipError_t launch_quantize_weights(int dtype, const QuantizeWeightsArgs& g, hipStream_t st);
// weights: a scale for each 128 x 128 block, not for each 128 columns of a row
hipError_t launch_dequantize(int dtype, bool weights, const DequantizeArgs& g, hipStream_t st);

// ---------------------------------------------------- the experts' product

// Sorted rows as in ExpertsArgs.
struct ScaledArgs {
  const uint8_t *x, *x_scales;  // [n_x, fan_in], [n_x, blocks]
  const uint8_t *w, *w_scales;  // [experts, fan_out, fan_in], [experts, blocks, blocks]
  void* out;
  const int* offsets;           // [experts + 1], or null: one expert has all rows
  const int* rows;              // [n_rows], or null: row i of x
  int n_x, n_rows, experts, fan_out, fan_in;
  bool stream;
  int most_row_tiles;  // of the tile that is launched, for offsets that ascend (set at the launch)
};
const char* experts_scaled_config(int dtype, const ScaledArgs& g);
hipError_t launch_experts_scaled(int dtype, const ScaledArgs& g, hipStream_t st);

}  // namespace ns
