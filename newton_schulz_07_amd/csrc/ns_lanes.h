// ns_lanes.h - values exchanged between the lanes of a wave without the LDS:
// rotations within a row of 16 lanes (DPP) and swaps of whole rows.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace ns {

template <int R> __device__ __forceinline__ int ror(int v) {  // lane l of a row: what lane (l + R) % 16 holds
  return __builtin_amdgcn_update_dpp(0, v, 0x120 + R, 0xf, 0xf, false);
}
template <int R> __device__ __forceinline__ float ror(float v) { return __int_as_float(ror<R>(__float_as_int(v))); }
template <int R> __device__ __forceinline__ double ror(double v) {
  return __hiloint2double(ror<R>(__double2hiint(v)), ror<R>(__double2loint(v)));
}

// op over a lane's value and that of the lane 16 (32) away
template <typename OP> __device__ __forceinline__ float with_row(float v, OP op) {
  const auto r = __builtin_amdgcn_permlane16_swap(__float_as_uint(v), __float_as_uint(v), false, false);
  return op(__uint_as_float(r[0]), __uint_as_float(r[1]));
}
template <typename OP> __device__ __forceinline__ float with_half(float v, OP op) {
  const auto r = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
  return op(__uint_as_float(r[0]), __uint_as_float(r[1]));
}
template <typename OP> __device__ __forceinline__ int with_row(int v, OP op) {
  const auto r = __builtin_amdgcn_permlane16_swap((unsigned)v, (unsigned)v, false, false);
  return op((int)r[0], (int)r[1]);
}
template <typename OP> __device__ __forceinline__ int with_half(int v, OP op) {
  const auto r = __builtin_amdgcn_permlane32_swap((unsigned)v, (unsigned)v, false, false);
  return op((int)r[0], (int)r[1]);
}
template <typename OP> __device__ __forceinline__ double with_row(double v, OP op) {
  return op(v, __shfl_xor(v, 16, 64));
}
template <typename OP> __device__ __forceinline__ double with_half(double v, OP op) {
  return op(v, __shfl_xor(v, 32, 64));
}

// op over the values of L lanes, 16 (a row) or 64, the same in all of them:
// op is commutative, and every step joins what two lanes hold alike.
template <int L, typename F, typename OP>
__device__ __forceinline__ F over_lanes(F v, OP op) {
  v = op(v, ror<8>(v));
  v = op(v, ror<4>(v));
  v = op(v, ror<2>(v));
  v = op(v, ror<1>(v));
  if (L == 64) {
    v = with_row(v, op);
    v = with_half(v, op);
  }
  return v;
}

__device__ __forceinline__ float larger(float a, float b) { return fmaxf(a, b); }  // the other one of a NaN
__device__ __forceinline__ double larger(double a, double b) { return fmax(a, b); }
__device__ __forceinline__ int larger(int a, int b) { return a > b ? a : b; }
template <int L, typename F> __device__ __forceinline__ F lanes_max(F v) {
  return over_lanes<L>(v, [](F a, F b) { return larger(a, b); });
}
template <int L> __device__ __forceinline__ int lanes_min(int v) {
  return over_lanes<L>(v, [](int a, int b) { return a < b ? a : b; });
}
template <int L, typename F> __device__ __forceinline__ F lanes_sum(F v) {
  return over_lanes<L>(v, [](F a, F b) { return a + b; });
}

}  // namespace ns
