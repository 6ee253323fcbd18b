// ns_norm.hip - layer norm over the columns of [rows, cols], forward and
// backward.
//
//   y  = (x - mean) rstd w + b,   rstd = 1 / sqrt(var + eps)
//   dx = rstd (g - mean(g) - xh mean(g xh)),   g = dy w,  xh = (x - mean) rstd
//   dw = sum over rows of dy xh,   db = sum over rows of dy
//
// Both passes are bound by HBM: a row is read once, held in registers as it
// was stored, and every sum is taken in fp32 (the variance from the centred
// values, in a second pass over the registers).  Results are rounded to their
// type once.  8192 x 7168 bf16: forward 45 us (5.2 TB/s of what has to be
// moved), backward 67 us (5.2 TB/s) and 6 us for the parameters' sums; a large
// copy reaches 4.8 TB/s.  The backward pass of more than 16384 columns
// does not fit the registers (norm_shape).  A single row of 2048: 3.0 us, a launch's latency.
// 1003 x 1531 fp32 (rows of odd length): 6.6, 12.6 and 4.0 us, bound by the
// instructions of single-column accesses and by latency.
#include "ns_device.h"
#include "ns_lanes.h"
#include "ns_sublayer.h"

namespace ns {
namespace {

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

// A row takes TPR threads (a wave: four rows to a block; or the whole block)
// of VPT vectors each.  A block walks rows with the grid's stride, so w and b
// are read once per block and stay in registers.  Bound by HBM.
template <typename T, int TPR, int VPT, int HOW>
__global__ __launch_bounds__(TPR == 64 ? 256 : TPR) void layer_norm_kernel(const LayerNormArgs g) {
  constexpr int WPR = TPR / 64, RPB = TPR == 64 ? 4 : 1;
  __shared__ float2 red[2][WPR];
  const int t = threadIdx.x % TPR;
  const float n = (float)g.cols;
  float w[VPT][8], b[VPT][8];
  params<TPR, VPT, HOW>(g.w, g.param_dtype, t, 0, g.cols, 1.0f, w);
  params<TPR, VPT, HOW>(g.b, g.param_dtype, t, 0, g.cols, 0.0f, b);
  for (long long row = (long long)blockIdx.x * RPB + threadIdx.x / TPR; row < g.rows;
       row += (long long)gridDim.x * RPB) {
    const T* x = reinterpret_cast<const T*>(g.x) + row * g.ldx;
    Raw8<T> r[VPT];
#pragma unroll
    for (int i = 0; i < VPT; ++i) r[i] = load8<T, TPR, HOW>(x, t, i, g.cols);
    float s = 0.0f;
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      float f[8];
      unpack8(r[i], f);
#pragma unroll
      for (int e = 0; e < 8; ++e) s += f[e];
    }
    const float mean = row_sum<WPR>(s, 0.0f, red[0]).x / n;
    s = 0.0f;
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      float f[8];
      unpack8(r[i], f);
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const float d = column<TPR, HOW>(t, i, e) < g.cols ? f[e] - mean : 0.0f;
        s = fmaf(d, d, s);
      }
    }
    const float rstd = 1.0f / sqrtf(row_sum<WPR>(s, 0.0f, red[1]).x / n + g.eps);
    T* y = reinterpret_cast<T*>(g.y) + row * (long long)g.cols;
    streaming(g.stream, [&](auto stream) __attribute__((always_inline)) {
#pragma unroll
      for (int i = 0; i < VPT; ++i) {
        float f[8];
        unpack8(r[i], f);
#pragma unroll
        for (int e = 0; e < 8; ++e) f[e] = fmaf((f[e] - mean) * rstd, w[i][e], b[i][e]);
        store8<T, TPR, HOW, stream.value>(y, t, i, g.cols, f);
      }
    });
    if (t == 0) {
      if (g.mean) g.mean[row] = mean;
      if (g.rstd) g.rstd[row] = rstd;
    }
  }
}

// Rows too long for the registers (above 32768 columns): three passes over the
// row (the later ones find it in the L2, which bounds it).
template <typename T, int HOW>
__global__ __launch_bounds__(1024) void layer_norm_long_kernel(const LayerNormArgs g) {
  __shared__ float2 red[2][16];
  const int t = threadIdx.x, nv = (g.cols + 8191) / 8192;  // rounds of 1024 x 8 columns
  const float n = (float)g.cols;
  for (long long row = blockIdx.x; row < g.rows; row += gridDim.x) {
    const T* x = reinterpret_cast<const T*>(g.x) + row * g.ldx;
    T* y = reinterpret_cast<T*>(g.y) + row * (long long)g.cols;
    float s = 0.0f, f[8];
    for (int i = 0; i < nv; ++i) {
      unpack8(load8<T, 1024, HOW>(x, t, i, g.cols), f);
#pragma unroll
      for (int e = 0; e < 8; ++e) s += f[e];
    }
    const float mean = row_sum<16>(s, 0.0f, red[0]).x / n;
    s = 0.0f;
    for (int i = 0; i < nv; ++i) {
      unpack8(load8<T, 1024, HOW>(x, t, i, g.cols), f);
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const float d = column<1024, HOW>(t, i, e) < g.cols ? f[e] - mean : 0.0f;
        s = fmaf(d, d, s);
      }
    }
    const float rstd = 1.0f / sqrtf(row_sum<16>(s, 0.0f, red[1]).x / n + g.eps);
    for (int i = 0; i < nv; ++i) {
      float w[1][8], b[1][8];
      params<1024, 1, HOW>(g.w, g.param_dtype, t, i, g.cols, 1.0f, w);
      params<1024, 1, HOW>(g.b, g.param_dtype, t, i, g.cols, 0.0f, b);
      unpack8(load8<T, 1024, HOW>(x, t, i, g.cols), f);
#pragma unroll
      for (int e = 0; e < 8; ++e) f[e] = fmaf((f[e] - mean) * rstd, w[0][e], b[0][e]);
      streaming(g.stream, [&](auto stream) __attribute__((always_inline)) {
        store8<T, 1024, HOW, stream.value>(y, t, i, g.cols, f);
      });
    }
    if (t == 0) {
      if (g.mean) g.mean[row] = mean;
      if (g.rstd) g.rstd[row] = rstd;
    }
  }
}

__device__ __forceinline__ void store_param(void* p, int pdt, int c, float v) {
  if (p == nullptr) return;
  if (pdt == 1) reinterpret_cast<bf16*>(p)[c] = (bf16)v;
  else reinterpret_cast<float*>(p)[c] = v;
}

// The gradients.  Each block keeps its rows' sums for dw and db in registers
// and writes them to its own row of `partials` [blocks][2][cols], which
// layer_norm_params_kernel adds up in a fixed order: no atomics, the same
// bits from the same inputs.  Bound by HBM; the partial sums of 512 blocks of
// 7168 columns are 29 MB beside the 352 MB of the rows.
template <typename T, int TPR, int VPT, int HOW>
__global__ __launch_bounds__(TPR == 64 ? 256 : TPR) void layer_norm_backward_kernel(const LayerNormGradArgs g) {
  constexpr int WPR = TPR / 64, RPB = TPR == 64 ? 4 : 1;
  __shared__ float2 red[2][WPR];
  __shared__ float part[RPB > 1 ? RPB - 1 : 1][RPB > 1 ? TPR * VPT * 8 : 1];
  const int t = threadIdx.x % TPR, rl = threadIdx.x / TPR;
  const float inv_n = 1.0f / (float)g.cols;
  float w[VPT][8], aw[VPT][8], ab[VPT][8];
  params<TPR, VPT, HOW>(g.w, g.param_dtype, t, 0, g.cols, 1.0f, w);
#pragma unroll
  for (int i = 0; i < VPT; ++i)
#pragma unroll
    for (int e = 0; e < 8; ++e) aw[i][e] = ab[i][e] = 0.0f;
  int turn = 0;  // a row's sums must not land where slower waves still read the last row's
  for (long long row = (long long)blockIdx.x * RPB + rl; row < g.rows; row += (long long)gridDim.x * RPB) {
    const T* x = reinterpret_cast<const T*>(g.x) + row * g.ldx;
    const T* dy = reinterpret_cast<const T*>(g.dy) + row * g.lddy;
    Raw8<T> rx[VPT], rd[VPT];
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      rd[i] = load8<T, TPR, HOW>(dy, t, i, g.cols);
      rx[i] = load8<T, TPR, HOW>(x, t, i, g.cols);
    }
    const float mean = g.mean[row], rstd = g.rstd[row];
    float c1 = 0.0f, c2 = 0.0f;
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      float fx[8], fd[8];
      unpack8(rx[i], fx);
      unpack8(rd[i], fd);
#pragma unroll
      for (int e = 0; e < 8; ++e) {  // past the row's end dy is zero: nothing is added
        const float xh = (fx[e] - mean) * rstd, d = fd[e] * w[i][e];
        c1 += d;
        c2 = fmaf(d, xh, c2);
        aw[i][e] = fmaf(fd[e], xh, aw[i][e]);
        ab[i][e] += fd[e];
      }
    }
    const float2 c = row_sum<WPR>(c1, c2, red[turn]);
    turn ^= 1;
    c1 = c.x * inv_n;
    c2 = c.y * inv_n;
    if (g.dx) {
      T* dx = reinterpret_cast<T*>(g.dx) + row * (long long)g.cols;
      streaming(g.stream, [&](auto stream) __attribute__((always_inline)) {
#pragma unroll
        for (int i = 0; i < VPT; ++i) {
          float fx[8], fd[8];
          unpack8(rx[i], fx);
          unpack8(rd[i], fd);
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            const float xh = (fx[e] - mean) * rstd;
            fx[e] = rstd * (fmaf(fd[e], w[i][e], -c1) - xh * c2);
          }
          store8<T, TPR, HOW, stream.value>(dx, t, i, g.cols, fx);
        }
      });
    }
  }
  if (g.partials == nullptr) return;
  const int ld = partials_ld(g.cols);
  float* out = g.partials + (size_t)blockIdx.x * 2 * ld;
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    if (RPB > 1) {  // the other waves' sums, in order
      __syncthreads();
      if (rl > 0)
#pragma unroll
        for (int i = 0; i < VPT; ++i)
#pragma unroll
          for (int e = 0; e < 8; ++e) part[rl - 1][(i * 8 + e) * TPR + t] = h ? ab[i][e] : aw[i][e];
      __syncthreads();
      if (rl > 0) continue;
    }
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      float x[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        x[e] = h ? ab[i][e] : aw[i][e];
        if (RPB > 1)
#pragma unroll
          for (int r = 0; r < RPB - 1; ++r) x[e] += part[r][(i * 8 + e) * TPR + t];
      }
      store8<float, TPR, HOW, false>(out + (size_t)h * ld, t, i, g.cols, x);
    }
  }
}

// Rows too long for the registers: a block's columns of dw and db are added
// up in its row of `partials`, which it alone touches.
template <typename T, int HOW>
__global__ __launch_bounds__(1024) void layer_norm_backward_long_kernel(const LayerNormGradArgs g) {
  __shared__ float2 red[2][16];
  const int t = threadIdx.x, nv = (g.cols + 8191) / 8192;
  const float inv_n = 1.0f / (float)g.cols;
  const int ld = partials_ld(g.cols);
  float* out = g.partials ? g.partials + (size_t)blockIdx.x * 2 * ld : nullptr;
  int turn = 0;
  bool first = true;
  for (long long row = blockIdx.x; row < g.rows; row += gridDim.x) {
    const T* x = reinterpret_cast<const T*>(g.x) + row * g.ldx;
    const T* dy = reinterpret_cast<const T*>(g.dy) + row * g.lddy;
    const float mean = g.mean[row], rstd = g.rstd[row];
    float c1 = 0.0f, c2 = 0.0f, fx[8], fd[8], w[1][8];
    for (int i = 0; i < nv; ++i) {
      unpack8(load8<T, 1024, HOW>(x, t, i, g.cols), fx);
      unpack8(load8<T, 1024, HOW>(dy, t, i, g.cols), fd);
      params<1024, 1, HOW>(g.w, g.param_dtype, t, i, g.cols, 1.0f, w);
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const float xh = (fx[e] - mean) * rstd, d = fd[e] * w[0][e];
        c1 += d;
        c2 = fmaf(d, xh, c2);
        const int c = column<1024, HOW>(t, i, e);
        if (out != nullptr && c < g.cols) {
          out[c] = first ? fd[e] * xh : fmaf(fd[e], xh, out[c]);
          out[ld + c] = first ? fd[e] : out[ld + c] + fd[e];
        }
      }
    }
    first = false;
    const float2 c = row_sum<16>(c1, c2, red[turn]);
    turn ^= 1;
    if (g.dx == nullptr) continue;
    c1 = c.x * inv_n;
    c2 = c.y * inv_n;
    T* dx = reinterpret_cast<T*>(g.dx) + row * (long long)g.cols;
    for (int i = 0; i < nv; ++i) {
      unpack8(load8<T, 1024, HOW>(x, t, i, g.cols), fx);
      unpack8(load8<T, 1024, HOW>(dy, t, i, g.cols), fd);
      params<1024, 1, HOW>(g.w, g.param_dtype, t, i, g.cols, 1.0f, w);
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const float xh = (fx[e] - mean) * rstd;
        fx[e] = rstd * (fmaf(fd[e], w[0][e], -c1) - xh * c2);
      }
      streaming(g.stream, [&](auto stream) __attribute__((always_inline)) {
        store8<T, 1024, HOW, stream.value>(dx, t, i, g.cols, fx);
      });
    }
  }
}

// dw and db: the sum of `blocks` rows of partials, 64 columns to a block, 16
// interleaved runs of rows each, joined in order.  A run's rows are on their
// way eight at a time: latency bounds it (6 us for 29 MB, which are in the L2
// or the last-level cache).
constexpr int kParamRuns = 16, kParamAhead = 8;
__global__ __launch_bounds__(64 * kParamRuns) void layer_norm_params_kernel(const float* partials, int blocks, int cols,
                                                                            void* dw, void* db, int pdt) {
  __shared__ float sum[kParamRuns][64];
  const int lane = threadIdx.x & 63, run = threadIdx.x >> 6, c = blockIdx.x * 64 + lane, h = blockIdx.y;
  const int ld = partials_ld(cols);
  float s = 0.0f;
  if (c < cols)
    for (int p0 = run; p0 < blocks; p0 += kParamRuns * kParamAhead) {
      float x[kParamAhead];
#pragma unroll
      for (int u = 0; u < kParamAhead; ++u)
        x[u] = partials[((size_t)min(p0 + u * kParamRuns, blocks - 1) * 2 + h) * ld + c];
#pragma unroll
      for (int u = 0; u < kParamAhead; ++u) s += p0 + u * kParamRuns < blocks ? x[u] : 0.0f;
    }
  sum[run][lane] = s;
  __syncthreads();
  if (run == 0 && c < cols) {
#pragma unroll
    for (int r = 1; r < kParamRuns; ++r) s += sum[r][lane];
    store_param(h ? db : dw, pdt, c, s);
  }
}

template <typename T, int HOW>
void launch_forward(const LayerNormArgs& g, hipStream_t st) {
  const NormShape s = norm_shape(g.cols);
  const dim3 grid((unsigned)norm_blocks(g.rows, s, kNormForwardBlocks)), block(s.tpr == 64 ? 256 : s.tpr);
#define NS_LN(TPR, VPT) \
  if (s.tpr == TPR && s.vpt == VPT) return dispatch(layer_norm_kernel<T, TPR, VPT, HOW>, grid, block, st, g)
  NS_LN(64, 1);
  NS_LN(64, 2);
  NS_LN(64, 4);
  NS_LN(256, 2);
  NS_LN(256, 4);
  NS_LN(1024, 2);
  NS_LN(1024, 4);
#undef NS_LN
  dispatch(layer_norm_long_kernel<T, HOW>, grid, block, st, g);
}

template <typename T, int HOW>
void launch_backward(const LayerNormGradArgs& g, int blocks, hipStream_t st) {
  const NormShape s = norm_shape(g.cols);
  const dim3 grid((unsigned)blocks), block(s.tpr == 64 ? 256 : s.tpr);
#define NS_LN(TPR, VPT) \
  if (s.tpr == TPR && s.vpt == VPT) return dispatch(layer_norm_backward_kernel<T, TPR, VPT, HOW>, grid, block, st, g)
  NS_LN(64, 1);
  NS_LN(64, 2);
  NS_LN(64, 4);
  NS_LN(256, 2);
  NS_LN(256, 4);
  NS_LN(1024, 2);
  NS_LN(1024, 4);
#undef NS_LN
  dispatch(layer_norm_backward_long_kernel<T, HOW>, grid, block, st, g);
}

}  // namespace

hipError_t launch_layer_norm(int dtype, const LayerNormArgs& args, hipStream_t st) {
  LayerNormArgs g = args;
  g.stream = beyond_l2(g.rows * g.cols * (dtype == 1 ? 2 : 4));
  const int how = g.cols % 8 != 0 ? kSingles : g.ldx % 8 != 0 ? kVectors : kAligned;
  if (dtype == 1)
    how == kAligned ? launch_forward<bf16, kAligned>(g, st)
    : how == kVectors ? launch_forward<bf16, kVectors>(g, st) : launch_forward<bf16, kSingles>(g, st);
  else
    how == kAligned ? launch_forward<float, kAligned>(g, st)
    : how == kVectors ? launch_forward<float, kVectors>(g, st) : launch_forward<float, kSingles>(g, st);
  return hipGetLastError();
}

hipError_t launch_layer_norm_backward(int dtype, const LayerNormGradArgs& args, int blocks, hipStream_t st) {
  LayerNormGradArgs g = args;
  g.stream = beyond_l2(g.rows * g.cols * (dtype == 1 ? 2 : 4));
  if (blocks > 0) {
    const int how = g.cols % 8 != 0 ? kSingles : g.ldx % 8 != 0 || g.lddy % 8 != 0 ? kVectors : kAligned;
    if (dtype == 1)
      how == kAligned ? launch_backward<bf16, kAligned>(g, blocks, st)
      : how == kVectors ? launch_backward<bf16, kVectors>(g, blocks, st) : launch_backward<bf16, kSingles>(g, blocks, st);
    else
      how == kAligned ? launch_backward<float, kAligned>(g, blocks, st)
      : how == kVectors ? launch_backward<float, kVectors>(g, blocks, st) : launch_backward<float, kSingles>(g, blocks, st);
    if (hipError_t e = hipGetLastError()) return e;
  }
  if (g.dw == nullptr && g.db == nullptr) return hipSuccess;
  dispatch(layer_norm_params_kernel, dim3((unsigned)((g.cols + 63) / 64), 2), dim3(64 * kParamRuns), st,
           (const float*)g.partials, blocks, g.cols, g.dw, g.db, g.param_dtype);
  return hipGetLastError();
}

}  // namespace ns
