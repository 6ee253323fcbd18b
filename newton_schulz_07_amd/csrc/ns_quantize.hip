// ns_quantize.hip - values as e4m3 with a power of two as the scale of each 128
// columns of a row (activations) or of each 128 x 128 block (weights), and back.
//
//   s = 2^k, the least k >= -126 with max |x| <= 448 s over the block's finite x
//   q = x / s to the nearest e4m3, ties to even (infinities and NaN: NaN)
//   x' = q s
//
// A power of two divides exactly, and it is what the matrix instructions take as
// a scale.  Every pass is bound by HBM: values are read once, and the largest of
// a block is found in the registers that hold it.
#include <algorithm>

#include "ns_eight.h"
#include "ns_scaled.h"

namespace ns {
namespace {

// A block of a row takes 16 lanes of 8 columns each; a thread has kAhead of them
// on their way (65536 x 1536 bf16 47 us, 6.4 TB/s; with four or eight on their way
// and the way back, 89 us becomes 91 and 93).
constexpr int kAhead = 2;
template <typename T, bool ALIGNED>
__global__ __launch_bounds__(256) void quantize_kernel(const QuantizeArgs g) {
  const int sub = threadIdx.x & 15, group = threadIdx.x >> 4;
  const unsigned long long all = (unsigned long long)g.rows * g.blocks;  // below 2^32
  for (unsigned long long b0 = (unsigned long long)blockIdx.x * (16 * kAhead); b0 < all;
       b0 += (unsigned long long)gridDim.x * (16 * kAhead)) {
    Raw8<T> r[kAhead];
    size_t at[kAhead];
    bool in[kAhead];
#pragma unroll
    for (int u = 0; u < kAhead; ++u) {
      const unsigned long long b = b0 + u * 16 + group;
      const unsigned at32 = (unsigned)(b < all ? b : all - 1), row = at32 / g.blocks;
      const unsigned col = (at32 - row * g.blocks) * kScaleBlock + 8 * sub, from = min(col, g.cols - 8);
      in[u] = b < all && col < g.cols;
      at[u] = (size_t)row * g.cols + col;
      const T* x = reinterpret_cast<const T*>(g.x) + (long long)row * g.ldx + from;  // (past the end: not used)
      if (ALIGNED) r[u] = *reinterpret_cast<const Raw8<T>*>(x);
      else __builtin_memcpy(&r[u], x, sizeof(r[u]));
    }
#pragma unroll
    for (int u = 0; u < kAhead; ++u) {
      float f[8], m = 0.0f;
      unpack8(r[u], f);
#pragma unroll
      for (int e = 0; e < 8; ++e) m = fmaxf(m, finite_magnitude(f[e]));
      const unsigned s = scale_byte(lanes_max<16>(in[u] ? m : 0.0f));
      if (!in[u]) continue;
      *reinterpret_cast<uint2*>(g.q + at[u]) = to_eight(f, inverse_scale(s));
      if (sub == 0) g.scales[b0 + u * 16 + group] = (uint8_t)s;
    }
  }
}

// 4 x 4 bytes: row i of the result is byte i of each of the four rows
__device__ __forceinline__ void transpose4(const unsigned (&a)[4], unsigned (&t)[4]) {
  const unsigned lo01 = __builtin_amdgcn_perm(a[1], a[0], 0x05010400), lo23 = __builtin_amdgcn_perm(a[3], a[2], 0x05010400);
  const unsigned hi01 = __builtin_amdgcn_perm(a[1], a[0], 0x07030602), hi23 = __builtin_amdgcn_perm(a[3], a[2], 0x07030602);
  t[0] = __builtin_amdgcn_perm(lo23, lo01, 0x05040100);
  t[1] = __builtin_amdgcn_perm(lo23, lo01, 0x07060302);
  t[2] = __builtin_amdgcn_perm(hi23, hi01, 0x05040100);
  t[3] = __builtin_amdgcn_perm(hi23, hi01, 0x07060302);
}

// A 128 x 128 block of a weight takes a workgroup: thread t has the 8 x 8 values
// at rows 8 (t / 16) and columns 8 (t % 16).  Its transpose goes through the LDS
// as [column][8 rows], the place of the rows exchanged by the column's group, so
// that neither side meets bank conflicts.  128 x 1536 x 2048 bf16 in both layouts:
// 285 us (5.7 TB/s of what has to be moved).
template <typename T, bool BOTH>
__global__ __launch_bounds__(256) void quantize_weights_kernel(const QuantizeWeightsArgs g) {
  __shared__ float most[4];
  __shared__ uint2 turned[BOTH ? kScaleBlock * 16 : 1];
  const int nb = (int)scale_blocks(g.fan_out), kb = (int)scale_blocks(g.fan_in);
  const int e = blockIdx.x / (nb * kb), in = blockIdx.x - e * (nb * kb), bi = in / kb, bj = in - bi * kb;
  const int rg = threadIdx.x >> 4, cg = threadIdx.x & 15, lane = threadIdx.x & 63;
  const int i0 = bi * kScaleBlock + 8 * rg, j0 = bj * kScaleBlock + 8 * cg;
  const size_t base = (size_t)e * g.fan_out * g.fan_in;
  const T* w = reinterpret_cast<const T*>(g.w) + base;
  Raw8<T> r[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    r[i] = Raw8<T>{};
    if (i0 + i < g.fan_out && j0 < g.fan_in)
      r[i] = *reinterpret_cast<const Raw8<T>*>(w + (size_t)(i0 + i) * g.fan_in + j0);
  }
  float m = 0.0f;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    float f[8];
    unpack8(r[i], f);
#pragma unroll
    for (int c = 0; c < 8; ++c) m = fmaxf(m, finite_magnitude(f[c]));
  }
  m = lanes_max<64>(m);
  if (lane == 0) most[threadIdx.x >> 6] = m;
  __syncthreads();
  const unsigned s = scale_byte(fmaxf(fmaxf(most[0], most[1]), fmaxf(most[2], most[3])));
  const float inverse = inverse_scale(s);
  uint2 q[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    float f[8];
    unpack8(r[i], f);
    q[i] = to_eight(f, inverse);
    if (i0 + i < g.fan_out && j0 < g.fan_in)
      *reinterpret_cast<uint2*>(g.q + base + (size_t)(i0 + i) * g.fan_in + j0) = q[i];
  }
  if (threadIdx.x == 0) {
    g.scales[blockIdx.x] = (uint8_t)s;
    if (BOTH) g.scales_t[(size_t)e * nb * kb + (size_t)bj * nb + bi] = (uint8_t)s;
  }
  if constexpr (BOTH) {
#pragma unroll
    for (int h = 0; h < 2; ++h) {  // columns 4 h .. 4 h + 3 of the thread's eight
      const unsigned a[4] = {h ? q[0].y : q[0].x, h ? q[1].y : q[1].x, h ? q[2].y : q[2].x, h ? q[3].y : q[3].x};
      const unsigned b[4] = {h ? q[4].y : q[4].x, h ? q[5].y : q[5].x, h ? q[6].y : q[6].x, h ? q[7].y : q[7].x};
      unsigned x[4], y[4];
      transpose4(a, x);
      transpose4(b, y);
#pragma unroll
      for (int c = 0; c < 4; ++c) turned[(8 * cg + 4 * h + c) * 16 + (rg ^ cg)] = make_uint2(x[c], y[c]);
    }
    __syncthreads();
    // 16 lanes to a column: its 128 rows are 128 bytes in a row of the transpose
#pragma unroll
    for (int u = 0; u < 8; ++u) {
      const int c = u * 16 + rg, j = bj * kScaleBlock + c, i = bi * kScaleBlock + 8 * cg;
      if (j < g.fan_in && i < g.fan_out)
        *reinterpret_cast<uint2*>(g.qt + base + (size_t)j * g.fan_out + i) = turned[c * 16 + (cg ^ (c >> 3))];
    }
  }
}

// A thread has pieces of 16 bytes of the result, 256 pieces apart, so that a wave's
// store is one run of 1 KB (with 16 columns to a thread, whose stores leave gaps for
// one another, 65536 x 1536 to bf16 took 70 us, now 43).  128 weights of 1536 x 2048
// quantized in both layouts and restored 685 us, with four pieces to a thread 701.
constexpr int kPieces = 2;
template <typename T, bool WEIGHTS, bool STREAM>
__global__ __launch_bounds__(256) void dequantize_kernel(const DequantizeArgs g) {
  constexpr unsigned COLS = Elem<T>::kChunk;  // of a piece
  const unsigned pieces = g.cols / COLS;
  const unsigned long long all = (unsigned long long)g.rows * pieces;
  for (unsigned long long p0 = (unsigned long long)blockIdx.x * (256 * kPieces) + threadIdx.x; p0 < all;
       p0 += (unsigned long long)gridDim.x * (256 * kPieces)) {
    uint2 v[kPieces];
    float s[kPieces];
#pragma unroll
    for (int u = 0; u < kPieces; ++u) {
      const unsigned long long p = p0 + u * 256 < all ? p0 + u * 256 : all - 1;
      const unsigned row = all >> 32 ? (unsigned)(p / pieces) : (unsigned)p / pieces;
      const unsigned kb = (unsigned)(p - (unsigned long long)row * pieces) / (kScaleBlock / COLS);
      size_t at = (size_t)row * g.blocks + kb;
      if (WEIGHTS) {
        const unsigned e = row / g.matrix_rows, i = row - e * g.matrix_rows;
        at = ((size_t)e * g.matrix_blocks + i / kScaleBlock) * g.blocks + kb;
      }
      if constexpr (COLS == 8) v[u] = reinterpret_cast<const uint2*>(g.q)[p];
      else v[u].x = reinterpret_cast<const unsigned*>(g.q)[p];
      s[u] = scale_exponent(g.scales[at]);
    }
#pragma unroll
    for (int u = 0; u < kPieces; ++u) {
      if (p0 + u * 256 >= all) break;
      uint4 out;
      if constexpr (COLS == 8) {
        const uint2 lo = from_eight4(v[u].x, s[u], T()), hi = from_eight4(v[u].y, s[u], T());
        out = make_uint4(lo.x, lo.y, hi.x, hi.y);
      } else {
        out = from_eight4(v[u].x, s[u], T());
      }
      store_whole<STREAM>(reinterpret_cast<uint4*>(g.x) + p0 + u * 256, out);
    }
  }
}

// Blocks of so many pieces each: a launch holds fewer than 2^32 threads, more than that go round.
unsigned some_blocks(unsigned long long pieces, unsigned per_block) {
  return (unsigned)std::min(1ull << 20, (pieces + per_block - 1) / per_block);
}

}  // namespace

hipError_t launch_quantize(int dtype, const QuantizeArgs& g, hipStream_t st) {
  const dim3 grid(some_blocks((unsigned long long)g.rows * g.blocks, 16 * kAhead)), block(256);
  const bool aligned = g.ldx % 8 == 0;
  if (dtype == 1)
    aligned ? dispatch(quantize_kernel<bf16, true>, grid, block, st, g) : dispatch(quantize_kernel<bf16, false>, grid, block, st, g);
  else
    aligned ? dispatch(quantize_kernel<float, true>, grid, block, st, g) : dispatch(quantize_kernel<float, false>, grid, block, st, g);
  return hipGetLastError();
}

hipError_t launch_quantize_weights(int dtype, const QuantizeWeightsArgs& g, hipStream_t st) {
  const dim3 grid((unsigned)(g.experts * scale_blocks(g.fan_out) * scale_blocks(g.fan_in))), block(256);
  const bool both = g.qt != nullptr;
  if (dtype == 1)
    both ? dispatch(quantize_weights_kernel<bf16, true>, grid, block, st, g)
         : dispatch(quantize_weights_kernel<bf16, false>, grid, block, st, g);
  else
    both ? dispatch(quantize_weights_kernel<float, true>, grid, block, st, g)
         : dispatch(quantize_weights_kernel<float, false>, grid, block, st, g);
  return hipGetLastError();
}

template <typename T, bool WEIGHTS>
static void launch_dequantize_of(const DequantizeArgs& g, hipStream_t st) {
  const dim3 grid(some_blocks((unsigned long long)g.rows * (g.cols / Elem<T>::kChunk), 256 * kPieces)), block(256);
  if (beyond_l2((long long)g.rows * g.cols * (long long)sizeof(T))) dispatch(dequantize_kernel<T, WEIGHTS, true>, grid, block, st, g);
  else dispatch(dequantize_kernel<T, WEIGHTS, false>, grid, block, st, g);
}
hipError_t launch_dequantize(int dtype, bool weights, const DequantizeArgs& g, hipStream_t st) {
  if (dtype == 1) weights ? launch_dequantize_of<bf16, true>(g, st) : launch_dequantize_of<bf16, false>(g, st);
  else weights ? launch_dequantize_of<float, true>(g, st) : launch_dequantize_of<float, false>(g, st);
  return hipGetLastError();
}

}  // namespace ns
