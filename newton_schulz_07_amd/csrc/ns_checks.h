// ns_checks.h - argument checks that the sublayer's entry points share.
#pragma once

#include "ns_host.h"
#include "ns_kernels.h"
#include "ns_plan.h"

namespace ns {

constexpr int64_t kMaxDim = int64_t(1) << 20;     // columns of a row, and elements between rows
constexpr int64_t kMaxRows = int64_t(1) << 31;    // row counts stay below
// Choices of a routing and sorted rows of the experts: kernels step through
// them in 32-bit numbers, to the end of a block's or a tile's last step, which
// is up to 1024 past the last one.
constexpr int64_t kMaxStepped = kMaxRows - 1024;
constexpr int64_t kMaxTokens = int64_t(1) << 25;  // and routed tokens: a launch holds fewer than 2^32 threads, 64 to a token

inline int check_rows(int64_t n, const char* name) {
  if (n < 0 || n >= kMaxRows) return fail(NS_ERR_INVALID_ARG, std::string(name) + " must be in [0, 2^31)");
  return NS_OK;
}
inline int check_cols(int64_t n, const char* name) {
  if (n <= 0 || n > kMaxDim) return fail(NS_ERR_INVALID_ARG, std::string(name) + " must be in [1, 2^20]");
  return NS_OK;
}
inline int check_ld(int64_t ld, int64_t cols, const char* name) {
  if (ld < cols || ld > kMaxDim)
    return fail(NS_ERR_INVALID_ARG, std::string(name) + " must be at least the row's length and at most 2^20");
  return NS_OK;
}
// null is allowed; anything else is 16-byte aligned
inline int check_opt(const void* p, const char* name) { return p == nullptr ? NS_OK : check_ptr(p, name); }
// int32 and fp32 vectors need their own alignment only
inline int check_ptr4(const void* p, const char* name) {
  if (p == nullptr) return fail(NS_ERR_INVALID_ARG, std::string(name) + " is NULL");
  if (reinterpret_cast<uintptr_t>(p) % 4 != 0)
    return fail(NS_ERR_ALIGNMENT, std::string(name) + " is not 4-byte aligned");
  return NS_OK;
}
inline int check_opt4(const void* p, const char* name) { return p == nullptr ? NS_OK : check_ptr4(p, name); }

struct Span {
  const void* p;
  size_t bytes;
  const char* name;
};
// no output may share memory with an input or with another output
inline int check_apart(const Span* out, int n_out, const Span* in, int n_in) {
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
inline int check_apart(const Span (&out)[NO], const Span (&in)[NI]) {
  return check_apart(out, NO, in, NI);
}
inline size_t span(int64_t rows, int64_t ld, int64_t cols, size_t es) { return rows > 0 ? ((rows - 1) * ld + cols) * es : 0; }

inline int poison(char* ws, size_t bytes, hipStream_t st) {
  if (!g_poison.load() || bytes == 0) return NS_OK;
  return check_hip(hipMemsetAsync(ws, 0xFF, bytes, st), "workspace poison fill");
}

inline const char* type_name(int dtype) { return dtype == NS_DTYPE_BF16 ? "bf16" : "fp32"; }

}  // namespace ns
