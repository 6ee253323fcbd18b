// ns_scaled.cpp - host driver of RMS norm, quantization and the experts' products
// of 8-bit values: argument checks, workspace, launches.
#include "ns_scaled.h"

#include "ns_checks.h"

using namespace ns;

namespace {

int check_scaled_cols(int64_t n, const char* name) {
  if (int s = check_cols(n, name)) return s;
  if (n % 16 != 0) return fail(NS_ERR_ALIGNMENT, std::string(name) + " must be a multiple of 16 (16-byte rows)");
  return NS_OK;
}
int check_scales(const void* p, const char* name) {
  return p == nullptr ? fail(NS_ERR_INVALID_ARG, std::string(name) + " is NULL") : NS_OK;
}
int check_weights(int64_t experts, int64_t fan_out, int64_t fan_in) {
  if (experts < 1 || experts > kMaxExperts)
    return fail(NS_ERR_INVALID_ARG, "experts must be in [1, " + std::to_string(kMaxExperts) + "]");
  if (int s = check_scaled_cols(fan_out, "fan_out")) return s;
  if (int s = check_scaled_cols(fan_in, "fan_in")) return s;
  if (fan_out * fan_in >= (int64_t(1) << 29)) return fail(NS_ERR_INVALID_ARG, "an expert must hold fewer than 2^29 elements");
  return NS_OK;
}
// 8-bit x [n_x, fan_in], read through rows [n_rows] if given
int check_scaled_x(const void* x, const void* scales, int64_t n_x, const void* rows, int64_t n_rows) {
  if (int s = check_ptr(x, "x")) return s;
  if (int s = check_scales(scales, "x_scales")) return s;
  if (int s = check_opt4(rows, "rows")) return s;
  if (n_x < 1 || n_x >= kMaxRows) return fail(NS_ERR_INVALID_ARG, "n_x must be in [1, 2^31)");
  if (rows == nullptr && n_x < n_rows) return fail(NS_ERR_INVALID_ARG, "x has fewer rows than n_rows");
  if (rows != nullptr && n_rows >= (int64_t(1) << 29))
    return fail(NS_ERR_INVALID_ARG, "rows must hold fewer than 2^29 row numbers (2 GiB)");
  return NS_OK;
}
size_t block_count(int64_t experts, int64_t fan_out, int64_t fan_in) {
  return (size_t)(experts * scale_blocks(fan_out) * scale_blocks(fan_in));
}

}  // namespace

extern "C" {

int ns_rms_norm(const void* x, int64_t ldx, const void* residual, int64_t ldr, const void* weight, void* total, void* y,
                void* q, uint8_t* scales, float* rstd, int64_t rows, int64_t cols, int dtype, int param_dtype, float eps,
                void* stream) {
  return entry([&]() -> int {
    if (int s = check_dtype(dtype)) return s;
    if (int s = check_dtype(param_dtype)) return s;
    if (int s = check_rows(rows, "rows")) return s;
    if (int s = check_cols(cols, "cols")) return s;
    if (int s = check_ld(ldx, cols, "ldx")) return s;
    if (residual != nullptr)
      if (int s = check_ld(ldr, cols, "ldr")) return s;
    if (!(eps >= 0.0f)) return fail(NS_ERR_INVALID_ARG, "eps must be >= 0");
    if (int s = check_opt(weight, "weight")) return s;
    if (rows == 0) return NS_OK;
    if (int s = check_ptr(x, "x")) return s;
    if (int s = check_opt(residual, "residual")) return s;
    if (int s = check_opt(total, "total")) return s;
    if ((residual != nullptr) != (total != nullptr))
      return fail(NS_ERR_INVALID_ARG, "residual and total go together: both of them, or none");
    if (int s = check_opt(y, "y")) return s;
    if (int s = check_opt(q, "q")) return s;
    if ((q != nullptr) != (scales != nullptr))
      return fail(NS_ERR_INVALID_ARG, "q and scales go together: both of them, or none");
    if (y == nullptr && q == nullptr) return fail(NS_ERR_INVALID_ARG, "y and q are both NULL");
    if (q != nullptr)
      if (int s = check_scaled_cols(cols, "cols")) return s;
    if (int s = check_opt4(rstd, "rstd")) return s;
    const size_t es = elem_size(dtype), ps = elem_size(param_dtype), n = (size_t)rows * cols;
    const Span out[] = {{total, n * es, "total"}, {y, n * es, "y"}, {q, n, "q"},
                        {scales, (size_t)(rows * scale_blocks(cols)), "scales"}, {rstd, (size_t)rows * 4, "rstd"}};
    const Span in[] = {{x, span(rows, ldx, cols, es), "x"}, {residual, span(rows, ldr, cols, es), "residual"},
                       {weight, cols * ps, "weight"}};
    if (int s = check_apart(out, in)) return s;
    if (int s = check_arch()) return s;
    hipStream_t st = static_cast<hipStream_t>(stream);
    const RmsNormArgs g{x, residual, weight, total, y, static_cast<uint8_t*>(q), scales, rstd, rows, ldx, ldr, (int)cols,
                        param_dtype, eps};
    if (int s = check_hip(timed_launch(NS_KIND_RMS_NORM, st, [&] { return launch_rms_norm(dtype, g, st); }),
                          "rms norm launch"))
      return s;
    const NormShape shape = rms_shape((int)cols);
    set_config("rms norm: dtype=%s rows=%lld cols=%lld | %lld threads x %lld vectors of 8 per row, in 8 bits: %lld",
               type_name(dtype), rows, cols, shape.tpr, shape.vpt, q != nullptr);
    return NS_OK;
  });
}

int ns_rms_norm_backward(const void* dy, int64_t lddy, const void* x, int64_t ldx, const void* weight, const float* rstd,
                         const void* dtotal, int64_t lddt, void* dx, void* dweight, int64_t rows, int64_t cols, int dtype,
                         int param_dtype, void* stream) {
  return entry([&]() -> int {
    if (int s = check_dtype(dtype)) return s;
    if (int s = check_dtype(param_dtype)) return s;
    if (int s = check_rows(rows, "rows")) return s;
    if (int s = check_cols(cols, "cols")) return s;
    if (int s = check_ld(ldx, cols, "ldx")) return s;
    if (int s = check_ld(lddy, cols, "lddy")) return s;
    if (dtotal != nullptr)
      if (int s = check_ld(lddt, cols, "lddt")) return s;
    if (int s = check_opt(weight, "weight")) return s;
    if (int s = check_opt(dweight, "dweight")) return s;
    const size_t es = elem_size(dtype), ps = elem_size(param_dtype);
    if (rows > 0) {
      if (int s = check_ptr(dy, "dy")) return s;
      if (int s = check_ptr(x, "x")) return s;
      if (int s = check_ptr4(rstd, "rstd")) return s;
      if (int s = check_opt(dtotal, "dtotal")) return s;
      if (int s = check_opt(dx, "dx")) return s;
    }
    const Span out[] = {{dx, rows * cols * es, "dx"}, {dweight, cols * ps, "dweight"}};
    const Span in[] = {{dy, span(rows, lddy, cols, es), "dy"}, {x, span(rows, ldx, cols, es), "x"},
                       {dtotal, span(rows, lddt, cols, es), "dtotal"}, {weight, cols * ps, "weight"},
                       {rstd, (size_t)rows * 4, "rstd"}};
    if (int s = check_apart(out, in)) return s;
    if (dweight == nullptr && (rows == 0 || dx == nullptr)) return NS_OK;
    if (int s = check_arch()) return s;
    hipStream_t st = static_cast<hipStream_t>(stream);
    const int blocks = rms_backward_blocks(rows, (int)cols);
    const size_t bytes = dweight ? (size_t)blocks * partials_ld((int)cols) * sizeof(float) : 0;
    Workspace ws;  // held to the end of the call's launches
    if (bytes > 0) {
      if (int s = get_workspace(st, bytes, &ws)) return s;
      if (int s = poison(ws.ptr, bytes, st)) return s;
    }
    const RmsNormGradArgs g{dy, x, dtotal, weight, rstd, dx, dweight, reinterpret_cast<float*>(ws.ptr), rows, lddy, ldx,
                            lddt, (int)cols, param_dtype};
    if (int s = check_hip(timed_launch(NS_KIND_RMS_NORM, st,
                                       [&] { return launch_rms_norm_backward(dtype, g, blocks, st); }),
                          "rms norm backward launch"))
      return s;
    const NormShape shape = rms_shape((int)cols);
    set_config("rms norm backward: dtype=%s rows=%lld cols=%lld | %lld threads x %lld vectors of 8 per row, %lld blocks",
               type_name(dtype), rows, cols, shape.tpr, shape.vpt, blocks);
    return NS_OK;
  });
}

int ns_quantize(const void* x, int64_t ldx, void* q, uint8_t* scales, int64_t rows, int64_t cols, int dtype, void* stream) {
  return entry([&]() -> int {
    if (int s = check_dtype(dtype)) return s;
    if (int s = check_rows(rows, "rows")) return s;
    if (int s = check_scaled_cols(cols, "cols")) return s;
    if (int s = check_ld(ldx, cols, "ldx")) return s;
    if (rows * scale_blocks(cols) >= (int64_t(1) << 32)) return fail(NS_ERR_INVALID_ARG, "x must have fewer than 2^32 blocks");
    if (rows == 0) return NS_OK;
    if (int s = check_ptr(x, "x")) return s;
    if (int s = check_ptr(q, "q")) return s;
    if (int s = check_scales(scales, "scales")) return s;
    const Span out[] = {{q, (size_t)rows * cols, "q"}, {scales, (size_t)(rows * scale_blocks(cols)), "scales"}};
    const Span in[] = {{x, span(rows, ldx, cols, elem_size(dtype)), "x"}};
    if (int s = check_apart(out, in)) return s;
    if (int s = check_arch()) return s;
    hipStream_t st = static_cast<hipStream_t>(stream);
    const QuantizeArgs g{x, static_cast<uint8_t*>(q), scales, ldx, (unsigned)rows, (unsigned)cols, (unsigned)scale_blocks(cols)};
    if (int s = check_hip(timed_launch(NS_KIND_QUANTIZE, st, [&] { return launch_quantize(dtype, g, st); }),
                          "quantize launch"))
      return s;
    set_config("quantize: dtype=%s rows=%lld cols=%lld | a scale for each 128 columns", type_name(dtype), rows, cols);
    return NS_OK;
  });
}

int ns_quantize_weights(const void* w, void* q, uint8_t* scales, void* qt, uint8_t* scales_t, int64_t experts,
                        int64_t fan_out, int64_t fan_in, int dtype, void* stream) {
  return entry([&]() -> int {
    if (int s = check_dtype(dtype)) return s;
    if (int s = check_weights(experts, fan_out, fan_in)) return s;
    if (block_count(experts, fan_out, fan_in) >= size_t(1) << 24)  // 256 threads each
      return fail(NS_ERR_INVALID_ARG, "w must have fewer than 2^24 blocks");
    if (int s = check_ptr(w, "w")) return s;
    if (int s = check_ptr(q, "q")) return s;
    if (int s = check_scales(scales, "scales")) return s;
    if (int s = check_opt(qt, "qt")) return s;
    if ((qt != nullptr) != (scales_t != nullptr))
      return fail(NS_ERR_INVALID_ARG, "qt and scales_t go together: both of them, or none");
    const size_t n = (size_t)(experts * fan_out * fan_in), b = block_count(experts, fan_out, fan_in);
    const Span out[] = {{q, n, "q"}, {scales, b, "scales"}, {qt, n, "qt"}, {scales_t, b, "scales_t"}};
    const Span in[] = {{w, n * elem_size(dtype), "w"}};
    if (int s = check_apart(out, in)) return s;
    if (int s = check_arch()) return s;
    hipStream_t st = static_cast<hipStream_t>(stream);
    const QuantizeWeightsArgs g{w, static_cast<uint8_t*>(q), scales, static_cast<uint8_t*>(qt), scales_t, (int)experts,
                                (int)fan_out, (int)fan_in};
    if (int s = check_hip(timed_launch(NS_KIND_QUANTIZE, st, [&] { return launch_quantize_weights(dtype, g, st); }),
                          "quantize weights launch"))
      return s;
    set_config("quantize weights: dtype=%s experts=%lld fan_out=%lld fan_in=%lld | transposed too: %lld", type_name(dtype),
               experts, fan_out, fan_in, qt != nullptr);
    return NS_OK;
  });
}

int ns_dequantize(const void* q, const uint8_t* scales, void* x, int64_t matrices, int64_t rows, int64_t cols,
                  int block_rows, int dtype, void* stream) {
  return entry([&]() -> int {
    if (int s = check_dtype(dtype)) return s;
    if (block_rows != 1 && block_rows != kScaleBlock) return fail(NS_ERR_INVALID_ARG, "block_rows must be 1 or 128");
    if (matrices < 0 || matrices >= kMaxRows) return fail(NS_ERR_INVALID_ARG, "matrices must be in [0, 2^31)");
    if (int s = check_rows(rows, "rows")) return s;
    if (matrices * rows >= kMaxRows) return fail(NS_ERR_INVALID_ARG, "matrices * rows must be below 2^31");
    if (int s = check_scaled_cols(cols, "cols")) return s;
    if (matrices * rows == 0) return NS_OK;
    if (int s = check_ptr(q, "q")) return s;
    if (int s = check_scales(scales, "scales")) return s;
    if (int s = check_ptr(x, "x")) return s;
    const bool weights = block_rows == kScaleBlock;
    const int64_t n = matrices * rows, rb = weights ? scale_blocks(rows) : rows;
    const Span out[] = {{x, (size_t)(n * cols) * elem_size(dtype), "x"}};
    const Span in[] = {{q, (size_t)(n * cols), "q"}, {scales, (size_t)(matrices * rb * scale_blocks(cols)), "scales"}};
    if (int s = check_apart(out, in)) return s;
    if (int s = check_arch()) return s;
    hipStream_t st = static_cast<hipStream_t>(stream);
    const DequantizeArgs g{static_cast<const uint8_t*>(q), scales, x, (unsigned)n, (unsigned)cols,
                           (unsigned)scale_blocks(cols), (unsigned)rows, (unsigned)rb};
    if (int s = check_hip(timed_launch(NS_KIND_QUANTIZE, st, [&] { return launch_dequantize(dtype, weights, g, st); }),
                          "dequantize launch"))
      return s;
    set_config("dequantize: dtype=%s matrices=%lld rows=%lld cols=%lld | a scale for %lld x 128 values", type_name(dtype),
               matrices, rows, cols, block_rows);
    return NS_OK;
  });
}

int ns_experts_product_scaled(const void* x, const uint8_t* x_scales, int64_t n_x, const int32_t* rows, const void* w,
                              const uint8_t* w_scales, const int32_t* offsets, void* y, int64_t n_rows, int64_t experts,
                              int64_t fan_out, int64_t fan_in, int dtype, void* stream) {
  return entry([&]() -> int {
    if (int s = check_dtype(dtype)) return s;
    if (n_rows < 0 || n_rows > kMaxStepped) return fail(NS_ERR_INVALID_ARG, "n_rows must be in [0, 2^31 - 1024]");
    if (int s = check_weights(experts, fan_out, fan_in)) return s;
    if (offsets == nullptr && experts != 1) return fail(NS_ERR_INVALID_ARG, "offsets is NULL: only one expert can have all rows");
    if (n_rows == 0) return NS_OK;
    if (int s = check_scaled_x(x, x_scales, n_x, rows, n_rows)) return s;
    if (rows != nullptr && n_x * fan_in > kMaxRows - 16)
      return fail(NS_ERR_INVALID_ARG, "x read through rows must hold less than 2 GiB");
    if (int s = check_ptr(w, "w")) return s;
    if (int s = check_scales(w_scales, "w_scales")) return s;
    if (int s = check_opt4(offsets, "offsets")) return s;
    if (int s = check_ptr(y, "y")) return s;
    const Span out[] = {{y, n_rows * fan_out * elem_size(dtype), "y"}};
    const Span in[] = {{x, (size_t)(n_x * fan_in), "x"}, {x_scales, (size_t)(n_x * scale_blocks(fan_in)), "x_scales"},
                       {rows, (size_t)n_rows * 4, "rows"}, {w, (size_t)(experts * fan_out * fan_in), "w"},
                       {w_scales, block_count(experts, fan_out, fan_in), "w_scales"},
                       {offsets, (size_t)(experts + 1) * 4, "offsets"}};
    if (int s = check_apart(out, in)) return s;
    if (int s = check_arch()) return s;
    hipStream_t st = static_cast<hipStream_t>(stream);
    const ScaledArgs g{static_cast<const uint8_t*>(x), x_scales, static_cast<const uint8_t*>(w), w_scales, y, offsets, rows,
                       (int)n_x, (int)n_rows, (int)experts, (int)fan_out, (int)fan_in};
    if (int s = check_hip(timed_launch(NS_KIND_EXPERTS, st, [&] { return launch_experts_scaled(dtype, g, st); }),
                          "experts product of 8-bit values"))
      return s;
    set_config(experts_scaled_config(dtype, g), type_name(dtype), n_rows, experts, fan_out, fan_in);
    return NS_OK;
  });
}

int ns_experts_weight_grad_scaled(const void* dy, const void* x, const uint8_t* x_scales, int64_t n_x, const int32_t* rows,
                                  const int32_t* offsets, void* dw, int64_t n_rows, int64_t experts, int64_t fan_out,
                                  int64_t fan_in, int dtype, void* stream) {
  return entry([&]() -> int {
    if (int s = check_dtype(dtype)) return s;
    if (n_rows < 0 || n_rows > kMaxStepped) return fail(NS_ERR_INVALID_ARG, "n_rows must be in [0, 2^31 - 1024]");
    if (int s = check_weights(experts, fan_out, fan_in)) return s;
    const size_t es = elem_size(dtype);
    if (n_rows > 0) {
      if (int s = check_ptr(dy, "dy")) return s;
      if (int s = check_scaled_x(x, x_scales, n_x, rows, n_rows)) return s;
      if (rows != nullptr && n_x * fan_in * (int64_t)es > kMaxRows - 16)
        return fail(NS_ERR_INVALID_ARG, "x read through rows must hold less than 2 GiB in dtype");
    }
    if (int s = check_opt4(offsets, "offsets")) return s;
    if (offsets == nullptr && experts != 1) return fail(NS_ERR_INVALID_ARG, "offsets is NULL: only one expert can have all rows");
    if (int s = check_ptr(dw, "dw")) return s;
    const Span out[] = {{dw, experts * fan_out * fan_in * es, "dw"}};
    const Span in[] = {{dy, n_rows * fan_out * es, "dy"}, {x, n_rows ? (size_t)(n_x * fan_in) : 0, "x"},
                       {x_scales, n_rows ? (size_t)(n_x * scale_blocks(fan_in)) : 0, "x_scales"},
                       {rows, (size_t)n_rows * 4, "rows"}, {offsets, (size_t)(experts + 1) * 4, "offsets"}};
    if (int s = check_apart(out, in)) return s;
    if (int s = check_arch()) return s;
    hipStream_t st = static_cast<hipStream_t>(stream);
    // x is restored, then it is the other weight gradient: the k of its products are rows, each with a
    // scale of its own, which a matrix instruction on 8-bit rows could not apply (a conversion on the way
    // to the LDS could, 16 bytes of a row having one scale; it is not built).  bf16, 128 experts: 8192
    // rows of 2048, 65536 times named, take 12 of 512 us; 65536 sorted rows of 1536 49 of 544.  Rows that
    // no one names are restored too: which are is known on the device only.
    const int64_t used = n_rows == 0 ? 0 : rows != nullptr ? n_x : n_rows;
    const size_t bytes = (size_t)(used * fan_in) * es;
    Workspace ws;  // held to the end of the call's launches
    if (bytes > 0) {
      if (int s = get_workspace(st, bytes, &ws)) return s;
      if (int s = poison(ws.ptr, bytes, st)) return s;
      const DequantizeArgs d{static_cast<const uint8_t*>(x), x_scales, ws.ptr, (unsigned)used, (unsigned)fan_in,
                             (unsigned)scale_blocks(fan_in), (unsigned)used, (unsigned)used};
      if (int s = check_hip(timed_launch(NS_KIND_QUANTIZE, st, [&] { return launch_dequantize(dtype, false, d, st); }),
                            "dequantize launch"))
        return s;
    }
    const ExpertsArgs g{ws.ptr, dy, nullptr, dw, offsets, rows, fan_in, (int)(used > 0 ? used : 1), (int)n_rows, (int)experts,
                        (int)fan_out, (int)fan_in};
    if (int s = check_hip(timed_launch(NS_KIND_EXPERTS, st, [&] { return launch_experts(dtype, EXP_WEIGHT_GRAD, g, st); }),
                          "experts weight gradient"))
      return s;
    set_config(experts_config(dtype, EXP_WEIGHT_GRAD, g), type_name(dtype), g.n_rows, g.experts, g.fan_out, g.fan_in);
    return NS_OK;
  });
}

}  // extern "C"
