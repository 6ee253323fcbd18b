// ns_rows.h - how the norms' kernels hold a row: its columns in the registers of
// one wave or of one block, the parameters of those columns, sums over the row.
#pragma once

#include "ns_device.h"
#include "ns_lanes.h"

namespace ns {

// A thread's 8 V columns of a row, as it holds them: V vectors of 8 columns,
// TPR vectors apart, where rows are whole vectors (kAligned: at 16-byte
// addresses; kVectors: at any), otherwise single columns, TPR apart (kSingles:
// a wave's access is still one run of columns).  Which columns a thread sums
// thus goes by the row's length alone, and the result's bits do not hang on
// how far rows are apart.  Elements past the row's end are zero, and are not
// stored.
enum { kAligned, kVectors, kSingles };
template <int TPR, int HOW> __device__ __forceinline__ int column(int t, int i, int e) {
  return HOW != kSingles ? 8 * (t + i * TPR) + e : t + TPR * (8 * i + e);
}
template <typename T, int TPR, int HOW>
__device__ __forceinline__ Raw8<T> load8(const T* row, int t, int i, int cols) {
  Raw8<T> r{};
  if (HOW == kAligned) {
    if (column<TPR, HOW>(t, i, 0) < cols) r = reinterpret_cast<const Raw8<T>*>(row)[t + i * TPR];
  } else if (HOW == kVectors) {
    if (column<TPR, HOW>(t, i, 0) < cols) __builtin_memcpy(&r, row + column<TPR, HOW>(t, i, 0), sizeof(r));
  } else {
    T x[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) x[e] = row[min(column<TPR, HOW>(t, i, e), cols - 1)];
#pragma unroll
    for (int e = 0; e < 8; ++e) x[e] = column<TPR, HOW>(t, i, e) < cols ? x[e] : (T)0.0f;
    __builtin_memcpy(&r, x, sizeof(r));
  }
  return r;
}
template <typename T, int TPR, int HOW, bool STREAM>
__device__ __forceinline__ void store8(T* row, int t, int i, int cols, const float* f) {
  const Raw8<T> r = pack8(f, T());
  if (HOW != kSingles) {  // (outputs are contiguous: whole vectors are aligned)
    if (column<TPR, HOW>(t, i, 0) < cols) store_whole<STREAM>(reinterpret_cast<Raw8<T>*>(row) + t + i * TPR, r);
  } else {
    T x[8];
    __builtin_memcpy(x, &r, sizeof(r));
#pragma unroll
    for (int e = 0; e < 8; ++e)
      if (column<TPR, HOW>(t, i, e) < cols) row[column<TPR, HOW>(t, i, e)] = x[e];
  }
}
// the parameters of those columns (fp32 or bf16 by pdt; null: `fill`)
template <int TPR, int V, int HOW>
__device__ __forceinline__ void params(const void* p, int pdt, int t, int i0, int cols, float fill, float (&f)[V][8]) {
  if (p == nullptr) {
#pragma unroll
    for (int i = 0; i < V; ++i)
#pragma unroll
      for (int e = 0; e < 8; ++e) f[i][e] = fill;
  } else if (pdt == 1) {
#pragma unroll
    for (int i = 0; i < V; ++i) unpack8(load8<bf16, TPR, HOW>(reinterpret_cast<const bf16*>(p), t, i0 + i, cols), f[i]);
  } else {
#pragma unroll
    for (int i = 0; i < V; ++i) unpack8(load8<float, TPR, HOW>(reinterpret_cast<const float*>(p), t, i0 + i, cols), f[i]);
  }
}

// Sum of (a, b) over the TPR threads of a row: one wave, or a whole block
// (WPR waves), every thread with the same result in the same order.
template <int WPR>
__device__ __forceinline__ float2 row_sum(float a, float b, float2* red) {
  a = lanes_sum<64>(a);
  b = lanes_sum<64>(b);
  if (WPR > 1) {
    if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = make_float2(a, b);
    __syncthreads();
    a = b = 0.0f;
#pragma unroll
    for (int w = 0; w < WPR; ++w) {
      a += red[w].x;
      b += red[w].y;
    }
  }
  return make_float2(a, b);
}

// The same of one number.
template <int WPR>
__device__ __forceinline__ float row_sum(float a, float* red) {
  a = lanes_sum<64>(a);
  if (WPR > 1) {
    if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = a;
    __syncthreads();
    a = 0.0f;
#pragma unroll
    for (int w = 0; w < WPR; ++w) a += red[w];
  }
  return a;
}

__device__ __forceinline__ void store_param(void* p, int pdt, int c, float v) {
  if (p == nullptr) return;
  if (pdt == 1) reinterpret_cast<bf16*>(p)[c] = (bf16)v;
  else reinterpret_cast<float*>(p)[c] = v;
}

}  // namespace ns
