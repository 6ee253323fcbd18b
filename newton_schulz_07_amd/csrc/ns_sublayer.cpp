// ns_sublayer.cpp - host driver of the mixture-of-experts sublayer's entry
// points: argument checks, workspace, launches.
#include "ns_sublayer.h"

#include "ns_host.h"
#include "ns_kernels.h"
#include "ns_plan.h"

using namespace ns;

namespace {

constexpr int64_t kMaxDim = int64_t(1) << 20;     // columns of a row, and elements between rows
constexpr int64_t kMaxRows = int64_t(1) << 31;    // row counts stay below
// Choices of a routing and sorted rows of the experts: kernels step through
// them in 32-bit numbers, to the end of a block's or a tile's last step, which
// is up to 1024 past the last one.
constexpr int64_t kMaxStepped = kMaxRows - 1024;
constexpr int64_t kMaxTokens = int64_t(1) << 25;  // and routed tokens: a launch holds fewer than 2^32 threads, 64 to a token

int check_rows(int64_t n, const char* name) {
  if (n < 0 || n >= kMaxRows) return fail(NS_ERR_INVALID_ARG, std::string(name) + " must be in [0, 2^31)");
  return NS_OK;
}
int check_cols(int64_t n, const char* name) {
  if (n <= 0 || n > kMaxDim) return fail(NS_ERR_INVALID_ARG, std::string(name) + " must be in [1, 2^20]");
  return NS_OK;
}
int check_ld(int64_t ld, int64_t cols, const char* name) {
  if (ld < cols || ld > kMaxDim)
    return fail(NS_ERR_INVALID_ARG, std::string(name) + " must be at least the row's length and at most 2^20");
  return NS_OK;
}
// null is allowed; anything else is 16-byte aligned
int check_opt(const void* p, const char* name) { return p == nullptr ? NS_OK : check_ptr(p, name); }
// int32 and fp32 vectors need their own alignment only
int check_ptr4(const void* p, const char* name) {
  if (p == nullptr) return fail(NS_ERR_INVALID_ARG, std::string(name) + " is NULL");
  if (reinterpret_cast<uintptr_t>(p) % 4 != 0)
    return fail(NS_ERR_ALIGNMENT, std::string(name) + " is not 4-byte aligned");
  return NS_OK;
}
int check_opt4(const void* p, const char* name) { return p == nullptr ? NS_OK : check_ptr4(p, name); }

struct Span {
  const void* p;
  size_t bytes;
  const char* name;
};
// no output may share memory with an input or with another output
int check_apart(const Span* out, int n_out, const Span* in, int n_in) {
  for (int i = 0; i < n_out; ++i) {
    if (out[i].p == nullptr || out[i].bytes == 0) continue;
    for (int j = 0; j < n_in; ++j)
      if (in[j].p != nullptr && in[j].bytes != 0 && overlaps(out[i].p, out[i].bytes, in[j].p, in[j].bytes))
        return fail(NS_ERR_INVALID_ARG, std::string(out[i].name) + " overlaps " + in[j].name);
    for (int j = 0; j < i; ++j)
      if (out[j].p != nullptr && out[j].bytes != 0 && overlaps(out[i].p, out[i].bytes, out[j].p, out[j].bytes))
        return fail(NS_ERR_INVALID_ARG, std::string(out[i].name) + " overlaps " + out[j].name);
  }
  return NS_OK;
}
template <int NO, int NI>
int check_apart(const Span (&out)[NO], const Span (&in)[NI]) {
  return check_apart(out, NO, in, NI);
}
size_t span(int64_t rows, int64_t ld, int64_t cols, size_t es) { return rows > 0 ? ((rows - 1) * ld + cols) * es : 0; }

int poison(char* ws, size_t bytes, hipStream_t st) {
  if (!g_poison.load() || bytes == 0) return NS_OK;
  return check_hip(hipMemsetAsync(ws, 0xFF, bytes, st), "workspace poison fill");
}

const char* type_name(int dtype) { return dtype == NS_DTYPE_BF16 ? "bf16" : "fp32"; }

int check_route(int64_t tokens, int64_t experts, int64_t top_k, int64_t ld, int score, int dtype) {
  if (int s = check_dtype(dtype)) return s;
  if (tokens < 0 || tokens >= kMaxTokens) return fail(NS_ERR_INVALID_ARG, "tokens must be in [0, 2^25)");
  if (experts < 1 || experts > kMaxExperts)
    return fail(NS_ERR_INVALID_ARG, "experts must be in [1, " + std::to_string(kMaxExperts) + "]");
  if (top_k < 1 || top_k > kMaxTopK || top_k > experts)
    return fail(NS_ERR_INVALID_ARG, "top_k must be in [1, min(experts, " + std::to_string(kMaxTopK) + ")]");
  if (int s = check_ld(ld, experts, "ld")) return s;
  if (score != NS_SCORE_SOFTMAX && score != NS_SCORE_SIGMOID)
    return fail(NS_ERR_INVALID_ARG, "score must be NS_SCORE_SOFTMAX or NS_SCORE_SIGMOID");
  return NS_OK;
}

int check_experts(int64_t n_rows, int64_t experts, int64_t fan_out, int64_t fan_in, int dtype) {
  if (int s = check_dtype(dtype)) return s;
  if (n_rows < 0 || n_rows > kMaxStepped) return fail(NS_ERR_INVALID_ARG, "n_rows must be in [0, 2^31 - 1024]");
  if (experts < 1 || experts > kMaxExperts)
    return fail(NS_ERR_INVALID_ARG, "experts must be in [1, " + std::to_string(kMaxExperts) + "]");
  if (int s = check_cols(fan_out, "fan_out")) return s;
  if (int s = check_cols(fan_in, "fan_in")) return s;
  if (fan_out % 8 != 0 || fan_in % 8 != 0)
    return fail(NS_ERR_ALIGNMENT, "fan_out and fan_in must be multiples of 8 (16-byte rows), got " +
                                      std::to_string(fan_out) + " and " + std::to_string(fan_in));
  if (fan_out * fan_in >= (int64_t(1) << 29))
    return fail(NS_ERR_INVALID_ARG, "an expert must hold fewer than 2^29 elements (2 GiB of fp32)");
  return NS_OK;
}

// x [n_x, fan_in] with rows ldx apart, read through rows [n_rows] if given
int check_x(const void* x, int64_t ldx, int64_t n_x, const void* rows, int64_t n_rows, int64_t fan_in, int dtype) {
  if (int s = check_ptr(x, "x")) return s;
  if (int s = check_opt4(rows, "rows")) return s;
  if (int s = check_ld(ldx, fan_in, "ldx")) return s;
  if (ldx % 8 != 0) return fail(NS_ERR_ALIGNMENT, "ldx must be a multiple of 8 (16-byte rows)");
  if (n_x < 1 || n_x >= kMaxRows) return fail(NS_ERR_INVALID_ARG, "n_x must be in [1, 2^31)");
  if (rows == nullptr && n_x < n_rows) return fail(NS_ERR_INVALID_ARG, "x has fewer rows than n_rows");
  if (rows != nullptr && span(n_x, ldx, fan_in, elem_size(dtype)) > (size_t(1) << 31) - 16)
    return fail(NS_ERR_INVALID_ARG, "x read through rows must hold less than 2 GiB");
  if (rows != nullptr && n_rows >= (int64_t(1) << 29))
    return fail(NS_ERR_INVALID_ARG, "rows must hold fewer than 2^29 row numbers (2 GiB)");
  return NS_OK;
}

int run_experts(ExpertsMode mode, const char* what, const ExpertsArgs& g, int dtype, hipStream_t st) {
  const int s = check_hip(timed_launch(NS_KIND_EXPERTS, st, [&] { return launch_experts(dtype, mode, g, st); }), what);
  if (s) return s;
  set_config(experts_config(dtype, mode, g), type_name(dtype), g.n_rows, g.experts, g.fan_out, g.fan_in);
  return NS_OK;
}

}  // namespace

extern "C" {

int ns_layer_norm(const void* x, int64_t ldx, const void* weight, const void* bias, void* y, float* mean, float* rstd,
                  int64_t rows, int64_t cols, int dtype, int param_dtype, float eps, void* stream) {
  return entry([&]() -> int {
    if (int s = check_dtype(dtype)) return s;
    if (int s = check_dtype(param_dtype)) return s;
    if (int s = check_rows(rows, "rows")) return s;
    if (int s = check_cols(cols, "cols")) return s;
    if (int s = check_ld(ldx, cols, "ldx")) return s;
    if (!(eps >= 0.0f)) return fail(NS_ERR_INVALID_ARG, "eps must be >= 0");
    if (int s = check_opt(weight, "weight")) return s;
    if (int s = check_opt(bias, "bias")) return s;
    if (rows == 0) return NS_OK;
    if (int s = check_ptr(x, "x")) return s;
    if (int s = check_ptr(y, "y")) return s;
    if (int s = check_opt4(mean, "mean")) return s;
    if (int s = check_opt4(rstd, "rstd")) return s;
    const size_t es = elem_size(dtype), ps = elem_size(param_dtype);
    const Span out[] = {{y, rows * cols * es, "y"}, {mean, (size_t)rows * 4, "mean"}, {rstd, (size_t)rows * 4, "rstd"}};
    const Span in[] = {{x, span(rows, ldx, cols, es), "x"}, {weight, cols * ps, "weight"}, {bias, cols * ps, "bias"}};
    if (int s = check_apart(out, in)) return s;
    if (int s = check_arch()) return s;
    hipStream_t st = static_cast<hipStream_t>(stream);
    LayerNormArgs g{x, weight, bias, y, mean, rstd, rows, ldx, (int)cols, param_dtype, eps};
    if (int s = check_hip(timed_launch(NS_KIND_LAYER_NORM, st, [&] { return launch_layer_norm(dtype, g, st); }),
                          "layer norm launch"))
      return s;
    const NormShape n = norm_shape((int)cols);
    set_config("layer norm: dtype=%s rows=%lld cols=%lld | %lld threads x %lld vectors of 8 per row", type_name(dtype),
           rows, cols, n.tpr, n.vpt);
    return NS_OK;
  });
}

int ns_layer_norm_backward(const void* dy, int64_t lddy, const void* x, int64_t ldx, const void* weight,
                           const float* mean, const float* rstd, void* dx, void* dweight, void* dbias, int64_t rows,
                           int64_t cols, int dtype, int param_dtype, void* stream) {
  return entry([&]() -> int {
    if (int s = check_dtype(dtype)) return s;
    if (int s = check_dtype(param_dtype)) return s;
    if (int s = check_rows(rows, "rows")) return s;
    if (int s = check_cols(cols, "cols")) return s;
    if (int s = check_ld(ldx, cols, "ldx")) return s;
    if (int s = check_ld(lddy, cols, "lddy")) return s;
    if (int s = check_opt(weight, "weight")) return s;
    if (int s = check_opt(dweight, "dweight")) return s;
    if (int s = check_opt(dbias, "dbias")) return s;
    const size_t es = elem_size(dtype), ps = elem_size(param_dtype);
    if (rows > 0) {
      if (int s = check_ptr(dy, "dy")) return s;
      if (int s = check_ptr(x, "x")) return s;
      if (int s = check_ptr4(mean, "mean")) return s;
      if (int s = check_ptr4(rstd, "rstd")) return s;
      if (int s = check_opt(dx, "dx")) return s;
    }
    const Span out[] = {{dx, rows * cols * es, "dx"}, {dweight, cols * ps, "dweight"}, {dbias, cols * ps, "dbias"}};
    const Span in[] = {{dy, span(rows, lddy, cols, es), "dy"}, {x, span(rows, ldx, cols, es), "x"},
                       {weight, cols * ps, "weight"}, {mean, (size_t)rows * 4, "mean"}, {rstd, (size_t)rows * 4, "rstd"}};
    if (int s = check_apart(out, in)) return s;
    const bool params = dweight != nullptr || dbias != nullptr;
    if (!params && (rows == 0 || dx == nullptr)) return NS_OK;
    if (int s = check_arch()) return s;
    hipStream_t st = static_cast<hipStream_t>(stream);
    const int blocks = norm_backward_blocks(rows, (int)cols);
    const size_t bytes = params ? (size_t)blocks * 2 * partials_ld((int)cols) * sizeof(float) : 0;
    Workspace ws;  // held to the end of the call's launches
    if (bytes > 0) {
      if (int s = get_workspace(st, bytes, &ws)) return s;
      if (int s = poison(ws.ptr, bytes, st)) return s;
    }
    LayerNormGradArgs g{dy, x, weight, mean, rstd, dx, dweight, dbias, reinterpret_cast<float*>(ws.ptr),
                        rows, lddy, ldx, (int)cols, param_dtype};
    if (int s = check_hip(timed_launch(NS_KIND_LAYER_NORM, st,
                                       [&] { return launch_layer_norm_backward(dtype, g, blocks, st); }),
                          "layer norm backward launch"))
      return s;
    const NormShape n = norm_shape((int)cols);
    set_config("layer norm backward: dtype=%s rows=%lld cols=%lld | %lld threads x %lld vectors of 8 per row, %lld blocks",
           type_name(dtype), rows, cols, n.tpr, n.vpt, blocks);
    return NS_OK;
  });
}

int ns_route(const void* logits, int64_t ld, const float* bias, int32_t* ids, float* weights, int32_t* offsets,
             int32_t* rows, int32_t* slots, int64_t tokens, int64_t experts, int64_t top_k, int64_t groups,
             int64_t top_groups, int group_best, int score, int renormalize, float scale, int dtype, void* stream) {
  return entry([&]() -> int {
    if (int s = check_route(tokens, experts, top_k, ld, score, dtype)) return s;
    if (tokens * top_k > kMaxStepped)
      return fail(NS_ERR_INVALID_ARG, "tokens * top_k must be at most 2^31 - 1024");
    if (groups < 1 || groups > kMaxGroups || experts % groups != 0)
      return fail(NS_ERR_INVALID_ARG, "groups must be in [1, " + std::to_string(kMaxGroups) + "] and divide experts");
    if (top_groups < 1 || top_groups > groups)
      return fail(NS_ERR_INVALID_ARG, "top_groups must be in [1, groups]");
    if (top_groups * (experts / groups) < top_k)
      return fail(NS_ERR_INVALID_ARG, "the chosen groups hold fewer than top_k experts");
    if (group_best != 1 && group_best != 2) return fail(NS_ERR_INVALID_ARG, "group_best must be 1 or 2");
    const bool plan = offsets != nullptr;
    if (tokens > 0 && (plan != (rows != nullptr) || plan != (slots != nullptr)))
      return fail(NS_ERR_INVALID_ARG, "offsets, rows and slots go together: all of them, or none");
    if (int s = check_opt4(bias, "bias")) return s;
    if (int s = check_opt4(offsets, "offsets")) return s;
    if (int s = check_opt4(rows, "rows")) return s;
    if (int s = check_opt4(slots, "slots")) return s;
    const size_t es = elem_size(dtype), n = (size_t)tokens * top_k * 4;
    if (tokens > 0) {
      if (int s = check_ptr(logits, "logits")) return s;
      if (int s = check_ptr4(ids, "ids")) return s;
      if (int s = check_ptr4(weights, "weights")) return s;
    } else if (!plan) {
      return NS_OK;
    }
    const Span out[] = {{ids, n, "ids"}, {weights, n, "weights"}, {offsets, (size_t)(experts + 1) * 4, "offsets"},
                        {rows, n, "rows"}, {slots, n, "slots"}};
    const Span in[] = {{logits, span(tokens, ld, experts, es), "logits"}, {bias, (size_t)experts * 4, "bias"}};
    if (int s = check_apart(out, in)) return s;
    if (int s = check_arch()) return s;
    hipStream_t st = static_cast<hipStream_t>(stream);
    Workspace ws;  // held to the end of the call's launches
    const size_t bytes = route_workspace((int)tokens, (int)experts);
    if (plan && bytes > 0) {
      if (int s = get_workspace(st, bytes, &ws)) return s;
      if (int s = poison(ws.ptr, bytes, st)) return s;
    }
    RouteArgs g{logits, bias, ids, weights, offsets, rows, slots, reinterpret_cast<int*>(ws.ptr), ld, (int)tokens,
                (int)experts, (int)top_k, (int)groups, (int)top_groups, group_best, score, renormalize != 0,
                route_shape((int)tokens, (int)experts).hist_ld, scale};
    if (int s = check_hip(timed_launch(NS_KIND_ROUTE, st, [&] { return launch_route(dtype, g, st); }), "route launch"))
      return s;
    set_config("route: dtype=%s tokens=%lld experts=%lld top_k=%lld groups=%lld/%lld | keys in %lld bits, %lld blocks", type_name(dtype),
           g.tokens, g.experts, g.top_k, g.top_groups, g.groups, bias || groups > 1 ? 64 : 32, route_shape(g.tokens, g.experts).blocks);
    return NS_OK;
  });
}

int ns_route_backward(const void* logits, int64_t ld, const int32_t* ids, const float* dweights, void* dlogits,
                      int64_t tokens, int64_t experts, int64_t top_k, int score, int renormalize, float scale,
                      int dtype, void* stream) {
  return entry([&]() -> int {
    if (int s = check_route(tokens, experts, top_k, ld, score, dtype)) return s;
    if (tokens == 0) return NS_OK;
    if (int s = check_ptr(logits, "logits")) return s;
    if (int s = check_ptr4(ids, "ids")) return s;
    if (int s = check_ptr4(dweights, "dweights")) return s;
    if (int s = check_ptr(dlogits, "dlogits")) return s;
    const size_t es = elem_size(dtype), n = (size_t)tokens * top_k * 4;
    const Span out[] = {{dlogits, tokens * experts * es, "dlogits"}};
    const Span in[] = {{logits, span(tokens, ld, experts, es), "logits"}, {ids, n, "ids"}, {dweights, n, "dweights"}};
    if (int s = check_apart(out, in)) return s;
    if (int s = check_arch()) return s;
    hipStream_t st = static_cast<hipStream_t>(stream);
    RouteGradArgs g{logits, ids, dweights, dlogits, ld, (int)tokens, (int)experts, (int)top_k, score,
                    renormalize != 0, scale};
    if (int s = check_hip(timed_launch(NS_KIND_ROUTE, st, [&] { return launch_route_backward(dtype, g, st); }),
                          "route backward launch"))
      return s;
    set_config("route backward: dtype=%s tokens=%lld experts=%lld top_k=%lld", type_name(dtype), g.tokens, g.experts, g.top_k);
    return NS_OK;
  });
}

int ns_experts_product(const void* x, int64_t ldx, int64_t n_x, const int32_t* rows, const void* w,
                       const int32_t* offsets, void* y, int64_t n_rows, int64_t experts, int64_t fan_out,
                       int64_t fan_in, int dtype, void* stream) {
  return entry([&]() -> int {
    if (int s = check_experts(n_rows, experts, fan_out, fan_in, dtype)) return s;
    if (n_rows == 0) return NS_OK;
    if (int s = check_x(x, ldx, n_x, rows, n_rows, fan_in, dtype)) return s;
    if (int s = check_ptr(w, "w")) return s;
    if (int s = check_ptr4(offsets, "offsets")) return s;
    if (int s = check_ptr(y, "y")) return s;
    const size_t es = elem_size(dtype);
    const Span out[] = {{y, n_rows * fan_out * es, "y"}};
    const Span in[] = {{x, span(n_x, ldx, fan_in, es), "x"}, {rows, (size_t)n_rows * 4, "rows"},
                       {w, experts * fan_out * fan_in * es, "w"}, {offsets, (size_t)(experts + 1) * 4, "offsets"}};
    if (int s = check_apart(out, in)) return s;
    if (int s = check_arch()) return s;
    const ExpertsArgs g{x, nullptr, w, y, offsets, rows, ldx, (int)n_x, (int)n_rows, (int)experts, (int)fan_out,
                        (int)fan_in};
    return run_experts(EXP_PRODUCT, "experts product", g, dtype, static_cast<hipStream_t>(stream));
  });
}

int ns_experts_input_grad(const void* dy, const void* w, const int32_t* offsets, void* dx, int64_t n_rows,
                          int64_t experts, int64_t fan_out, int64_t fan_in, int dtype, void* stream) {
  return entry([&]() -> int {
    if (int s = check_experts(n_rows, experts, fan_out, fan_in, dtype)) return s;
    if (n_rows == 0) return NS_OK;
    if (int s = check_ptr(dy, "dy")) return s;
    if (int s = check_ptr(w, "w")) return s;
    if (int s = check_ptr4(offsets, "offsets")) return s;
    if (int s = check_ptr(dx, "dx")) return s;
    const size_t es = elem_size(dtype);
    const Span out[] = {{dx, n_rows * fan_in * es, "dx"}};
    const Span in[] = {{dy, n_rows * fan_out * es, "dy"}, {w, experts * fan_out * fan_in * es, "w"},
                       {offsets, (size_t)(experts + 1) * 4, "offsets"}};
    if (int s = check_apart(out, in)) return s;
    if (int s = check_arch()) return s;
    const ExpertsArgs g{nullptr, dy, w, dx, offsets, nullptr, fan_in, (int)n_rows, (int)n_rows, (int)experts,
                        (int)fan_out, (int)fan_in};
    return run_experts(EXP_INPUT_GRAD, "experts input gradient", g, dtype, static_cast<hipStream_t>(stream));
  });
}

int ns_experts_weight_grad(const void* dy, const void* x, int64_t ldx, int64_t n_x, const int32_t* rows,
                           const int32_t* offsets, void* dw, int64_t n_rows, int64_t experts, int64_t fan_out,
                           int64_t fan_in, int dtype, void* stream) {
  return entry([&]() -> int {
    if (int s = check_experts(n_rows, experts, fan_out, fan_in, dtype)) return s;
    if (n_rows > 0) {
      if (int s = check_ptr(dy, "dy")) return s;
      if (int s = check_x(x, ldx, n_x, rows, n_rows, fan_in, dtype)) return s;
    }
    if (int s = check_ptr4(offsets, "offsets")) return s;
    if (int s = check_ptr(dw, "dw")) return s;
    const size_t es = elem_size(dtype);
    const Span out[] = {{dw, experts * fan_out * fan_in * es, "dw"}};
    const Span in[] = {{dy, n_rows * fan_out * es, "dy"}, {x, n_rows ? span(n_x, ldx, fan_in, es) : 0, "x"},
                       {rows, (size_t)n_rows * 4, "rows"}, {offsets, (size_t)(experts + 1) * 4, "offsets"}};
    if (int s = check_apart(out, in)) return s;
    if (int s = check_arch()) return s;
    const ExpertsArgs g{x, dy, nullptr, dw, offsets, rows, ldx, (int)n_x, (int)n_rows, (int)experts, (int)fan_out,
                        (int)fan_in};
    return run_experts(EXP_WEIGHT_GRAD, "experts weight gradient", g, dtype, static_cast<hipStream_t>(stream));
  });
}

int ns_experts_combine(const void* y, const int32_t* slots, const float* weights, void* out, int64_t tokens,
                       int64_t top_k, int64_t n_rows, int64_t cols, int dtype, void* stream) {
  return entry([&]() -> int {
    if (int s = check_dtype(dtype)) return s;
    if (int s = check_rows(tokens, "tokens")) return s;
    if (int s = check_rows(n_rows, "n_rows")) return s;
    if (top_k < 1 || tokens * top_k >= kMaxRows) return fail(NS_ERR_INVALID_ARG, "top_k must be >= 1 and tokens * top_k below 2^31");
    if (int s = check_cols(cols, "cols")) return s;
    if (cols % 8 != 0) return fail(NS_ERR_ALIGNMENT, "cols must be a multiple of 8 (16-byte rows)");
    if (tokens == 0) return NS_OK;
    if (n_rows > 0)
      if (int s = check_ptr(y, "y")) return s;
    if (int s = check_ptr4(slots, "slots")) return s;
    if (int s = check_opt4(weights, "weights")) return s;
    if (int s = check_ptr(out, "out")) return s;
    const size_t es = elem_size(dtype), n = (size_t)tokens * top_k * 4;
    const Span to[] = {{out, tokens * cols * es, "out"}};
    const Span in[] = {{n_rows ? y : nullptr, n_rows * cols * es, "y"}, {slots, n, "slots"}, {weights, n, "weights"}};
    if (int s = check_apart(to, in)) return s;
    if (int s = check_arch()) return s;
    hipStream_t st = static_cast<hipStream_t>(stream);
    const CombineArgs g{y, slots, weights, out, (int)tokens, (int)top_k, (int)n_rows, (int)cols};
    if (int s = check_hip(timed_launch(NS_KIND_COMBINE, st, [&] { return launch_combine(dtype, g, st); }),
                          "combine launch"))
      return s;
    set_config("experts combine: dtype=%s tokens=%lld top_k=%lld cols=%lld", type_name(dtype), g.tokens, g.top_k, g.cols);
    return NS_OK;
  });
}

int ns_experts_combine_backward(const void* dout, const void* y, const int32_t* slots, const float* weights, void* dy,
                                float* dweights, int64_t tokens, int64_t top_k, int64_t n_rows, int64_t cols,
                                int dtype, void* stream) {
  return entry([&]() -> int {
    if (int s = check_dtype(dtype)) return s;
    if (int s = check_rows(tokens, "tokens")) return s;
    if (int s = check_rows(n_rows, "n_rows")) return s;
    if (top_k < 1 || tokens * top_k >= kMaxRows) return fail(NS_ERR_INVALID_ARG, "top_k must be >= 1 and tokens * top_k below 2^31");
    if (int s = check_cols(cols, "cols")) return s;
    if (cols % 8 != 0) return fail(NS_ERR_ALIGNMENT, "cols must be a multiple of 8 (16-byte rows)");
    if (tokens == 0 || (dy == nullptr && dweights == nullptr)) return NS_OK;
    if (int s = check_ptr(dout, "dout")) return s;
    if (int s = check_ptr4(slots, "slots")) return s;
    if (int s = check_opt4(weights, "weights")) return s;
    if (int s = check_opt(dy, "dy")) return s;
    if (int s = check_opt4(dweights, "dweights")) return s;
    if (dweights != nullptr && n_rows > 0)
      if (int s = check_ptr(y, "y")) return s;
    const size_t es = elem_size(dtype), n = (size_t)tokens * top_k * 4;
    const Span to[] = {{dy, n_rows * cols * es, "dy"}, {dweights, n, "dweights"}};
    const Span in[] = {{dout, tokens * cols * es, "dout"}, {dweights && n_rows ? y : nullptr, n_rows * cols * es, "y"},
                       {slots, n, "slots"}, {weights, n, "weights"}};
    if (int s = check_apart(to, in)) return s;
    if (int s = check_arch()) return s;
    hipStream_t st = static_cast<hipStream_t>(stream);
    const CombineGradArgs g{dout, y, slots, weights, dy, dweights, (int)tokens, (int)top_k, (int)n_rows, (int)cols};
    if (int s = check_hip(timed_launch(NS_KIND_COMBINE, st, [&] { return launch_combine_backward(dtype, g, st); }),
                          "combine backward launch"))
      return s;
    set_config("experts combine backward: dtype=%s tokens=%lld top_k=%lld cols=%lld", type_name(dtype), g.tokens, g.top_k,
           g.cols);
    return NS_OK;
  });
}

}  // extern "C"
