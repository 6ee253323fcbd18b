// ns_rms.hip - RMS norm over the columns of [rows, cols] with the residual's
// addition, its result also in 8 bits with scales, and its gradients.
//
//   t  = x + residual, rounded to its type     y = t rstd w,  rstd = 1 / sqrt(mean(t^2) + eps)
//   dx = dtotal + rstd (g - th mean(g th)),    g = dy w,  th = t rstd
//   dw = sum over rows of dy th
//
// y is taken from t as it is stored: the backward pass and whoever else reads t
// then see what was normalised.  dx is the gradient of x and of the residual.
// All of it is bound by HBM; rows are held as layer norm's are (ns_rows.h,
// rms_shape).  8192 x 7168 bf16: forward with a residual and y in 8 bits 77 us (5.3
// TB/s of what has to be moved), backward 87 (5.4) and 6 for the sums of dw; a large
// copy reaches 5.2 TB/s.  A row of 2048: 4.0 us, a launch's latency and a square root
// in 64 bits.  1003 x 1531 fp32 (rows of odd length): 7.4, 8.1 and 3.4 us, bound by
// latency and the instructions of single-column accesses.
#include "ns_eight.h"
#include "ns_rows.h"
#include "ns_scaled.h"

namespace ns {
namespace {

// 128 columns are 16 vectors of 8, which 16 neighbouring lanes hold: the largest
// magnitude comes from one row of lanes.
template <int TPR, bool STREAM>
__device__ __forceinline__ void store_eight(const RmsNormArgs& g, long long row, int t, int i, const float* f) {
  float m = 0.0f;
#pragma unroll
  for (int e = 0; e < 8; ++e) m = fmaxf(m, finite_magnitude(f[e]));
  const unsigned b = scale_byte(lanes_max<16>(m));
  const int v = t + i * TPR;
  if (8 * v >= g.cols) return;
  const uint2 q = to_eight(f, inverse_scale(b));
  uint2* to = reinterpret_cast<uint2*>(g.q + row * g.cols) + v;
  if constexpr (STREAM) {
    typedef unsigned u32x2 __attribute__((ext_vector_type(2)));
    __builtin_nontemporal_store(u32x2{q.x, q.y}, reinterpret_cast<u32x2*>(to));
  } else {
    *to = q;
  }
  if (v % 16 == 0) g.scales[row * scale_blocks(g.cols) + v / 16] = (uint8_t)b;
}

template <typename T, int TPR, int HOW>
__device__ __forceinline__ Raw8<T> load_sum(const T* x, const T* r, int t, int i, int cols) {
  Raw8<T> a = load8<T, TPR, HOW>(x, t, i, cols);
  if (r != nullptr) {
    float f[8], h[8];
    unpack8(a, f);
    unpack8(load8<T, TPR, HOW>(r, t, i, cols), h);
#pragma unroll
    for (int e = 0; e < 8; ++e) f[e] += h[e];
    a = pack8(f, T());
  }
  return a;
}

// The squares are added in 64 bits, which hold those of every finite value (in 32
// bits a value of 2^64 or more made rstd 0, one below 2^-75 added nothing), and
// joined in them: y goes on to 8 bits, where an error of the last places moves
// values across the borders of the rounding.
__device__ __forceinline__ double add_squares(const float (&f)[8], double s) {
#pragma unroll
  for (int e = 0; e < 8; ++e) s = fma((double)f[e], (double)f[e], s);
  return s;
}
// rstd of a row from its threads' sums of squares
template <int WPR>
__device__ __forceinline__ float rstd_of(double squares, const RmsNormArgs& g, double* red) {
  double s = lanes_sum<64>(squares);
  if (WPR > 1) {
    if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = s;
    __syncthreads();
    s = 0.0;
#pragma unroll
    for (int w = 0; w < WPR; ++w) s += red[w];
  }
  return (float)(1.0 / sqrt(s / g.cols + (double)g.eps));
}

// A row takes TPR threads of VPT vectors each, as in layer_norm_kernel.
// EIGHT: y in 8 bits is wanted (cols a multiple of 16, so never kSingles).
template <typename T, int TPR, int VPT, int HOW, bool EIGHT>
__global__ __launch_bounds__(TPR == 64 ? 256 : TPR) void rms_norm_kernel(const RmsNormArgs g) {
  constexpr int WPR = TPR / 64, RPB = TPR == 64 ? 4 : 1;
  __shared__ double red[2][WPR];
  const int t = threadIdx.x % TPR;
  float w[VPT][8];
  params<TPR, VPT, HOW>(g.w, g.param_dtype, t, 0, g.cols, 1.0f, w);
  int turn = 0;  // a row's sum must not land where slower waves still read the last row's
  for (long long row = (long long)blockIdx.x * RPB + threadIdx.x / TPR; row < g.rows;
       row += (long long)gridDim.x * RPB) {
    const T* x = reinterpret_cast<const T*>(g.x) + row * g.ldx;
    const T* res = g.residual ? reinterpret_cast<const T*>(g.residual) + row * g.ldr : nullptr;
    Raw8<T> r[VPT];
#pragma unroll
    for (int i = 0; i < VPT; ++i) r[i] = load_sum<T, TPR, HOW>(x, res, t, i, g.cols);
    double s = 0.0;
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      float f[8];
      unpack8(r[i], f);
      s = add_squares(f, s);
    }
    const float rstd = rstd_of<WPR>(s, g, red[turn]);
    turn ^= 1;
    streaming(g.stream, [&](auto stream) __attribute__((always_inline)) {
#pragma unroll
      for (int i = 0; i < VPT; ++i) {
        float f[8];
        unpack8(r[i], f);
        if (g.total) store8<T, TPR, HOW, stream.value>(reinterpret_cast<T*>(g.total) + row * (long long)g.cols, t, i, g.cols, f);
#pragma unroll
        for (int e = 0; e < 8; ++e) f[e] = f[e] * rstd * w[i][e];
        if (g.y) store8<T, TPR, HOW, stream.value>(reinterpret_cast<T*>(g.y) + row * (long long)g.cols, t, i, g.cols, f);
        if constexpr (EIGHT) store_eight<TPR, stream.value>(g, row, t, i, f);
      }
    });
    if (t == 0 && g.rstd) g.rstd[row] = rstd;
  }
}

// Rows too long for the registers (above 32768 columns): two passes over the
// row.
template <typename T, int HOW, bool EIGHT>
__global__ __launch_bounds__(1024) void rms_norm_long_kernel(const RmsNormArgs g) {
  __shared__ double red[2][16];
  const int t = threadIdx.x, nv = (g.cols + 8191) / 8192;  // rounds of 1024 x 8 columns
  int turn = 0;
  for (long long row = blockIdx.x; row < g.rows; row += gridDim.x) {
    const T* x = reinterpret_cast<const T*>(g.x) + row * g.ldx;
    const T* res = g.residual ? reinterpret_cast<const T*>(g.residual) + row * g.ldr : nullptr;
    double s = 0.0;
    float f[8];
    for (int i = 0; i < nv; ++i) {
      unpack8(load_sum<T, 1024, HOW>(x, res, t, i, g.cols), f);
      s = add_squares(f, s);
    }
    const float rstd = rstd_of<16>(s, g, red[turn]);
    turn ^= 1;
    for (int i = 0; i < nv; ++i) {
      float w[1][8];
      params<1024, 1, HOW>(g.w, g.param_dtype, t, i, g.cols, 1.0f, w);
      unpack8(load_sum<T, 1024, HOW>(x, res, t, i, g.cols), f);
      if (g.total) store8<T, 1024, HOW, false>(reinterpret_cast<T*>(g.total) + row * (long long)g.cols, t, i, g.cols, f);
#pragma unroll
      for (int e = 0; e < 8; ++e) f[e] = f[e] * rstd * w[0][e];
      if (g.y) store8<T, 1024, HOW, false>(reinterpret_cast<T*>(g.y) + row * (long long)g.cols, t, i, g.cols, f);
      if constexpr (EIGHT) store_eight<1024, false>(g, row, t, i, f);
    }
    if (t == 0 && g.rstd) g.rstd[row] = rstd;
  }
}

// The gradients.  Each block keeps its rows' sums for dw in registers and writes
// them to its own row of `partials`, which rms_norm_params_kernel adds up in a
// fixed order: no atomics, the same bits from the same inputs.
template <typename T, int TPR, int VPT, int HOW>
__global__ __launch_bounds__(TPR == 64 ? 256 : TPR) void rms_norm_backward_kernel(const RmsNormGradArgs g) {
  constexpr int WPR = TPR / 64, RPB = TPR == 64 ? 4 : 1;
  __shared__ float red[2][WPR];
  __shared__ float part[RPB > 1 ? RPB - 1 : 1][RPB > 1 ? TPR * VPT * 8 : 1];
  const int t = threadIdx.x % TPR, rl = threadIdx.x / TPR;
  const float inv_n = 1.0f / (float)g.cols;
  float w[VPT][8], aw[VPT][8];
  params<TPR, VPT, HOW>(g.w, g.param_dtype, t, 0, g.cols, 1.0f, w);
#pragma unroll
  for (int i = 0; i < VPT; ++i)
#pragma unroll
    for (int e = 0; e < 8; ++e) aw[i][e] = 0.0f;
  int turn = 0;
  for (long long row = (long long)blockIdx.x * RPB + rl; row < g.rows; row += (long long)gridDim.x * RPB) {
    const T* x = reinterpret_cast<const T*>(g.x) + row * g.ldx;
    const T* dy = reinterpret_cast<const T*>(g.dy) + row * g.lddy;
    const T* dt = g.dtotal && g.dx ? reinterpret_cast<const T*>(g.dtotal) + row * g.lddt : nullptr;
    Raw8<T> rx[VPT], rd[VPT], rt[VPT];
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      rd[i] = load8<T, TPR, HOW>(dy, t, i, g.cols);
      rx[i] = load8<T, TPR, HOW>(x, t, i, g.cols);
      rt[i] = Raw8<T>{};
      if (dt != nullptr) rt[i] = load8<T, TPR, HOW>(dt, t, i, g.cols);
    }
    const float rstd = g.rstd[row];
    float c = 0.0f;
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      float fx[8], fd[8];
      unpack8(rx[i], fx);
      unpack8(rd[i], fd);
#pragma unroll
      for (int e = 0; e < 8; ++e) {  // past the row's end both are zero: nothing is added
        const float th = fx[e] * rstd;
        c = fmaf(fd[e] * w[i][e], th, c);
        aw[i][e] = fmaf(fd[e], th, aw[i][e]);
      }
    }
    c = row_sum<WPR>(c, red[turn]) * inv_n;
    turn ^= 1;
    if (g.dx) {
      T* dx = reinterpret_cast<T*>(g.dx) + row * (long long)g.cols;
      streaming(g.stream, [&](auto stream) __attribute__((always_inline)) {
#pragma unroll
        for (int i = 0; i < VPT; ++i) {
          float fx[8], fd[8], ft[8];
          unpack8(rx[i], fx);
          unpack8(rd[i], fd);
          unpack8(rt[i], ft);
#pragma unroll
          for (int e = 0; e < 8; ++e) fx[e] = fmaf(rstd, fmaf(fd[e], w[i][e], -(fx[e] * rstd) * c), ft[e]);
          store8<T, TPR, HOW, stream.value>(dx, t, i, g.cols, fx);
        }
      });
    }
  }
  if (g.partials == nullptr) return;
  float* out = g.partials + (size_t)blockIdx.x * partials_ld(g.cols);
  if (RPB > 1) {  // the other waves' sums, in order
    if (rl > 0)
#pragma unroll
      for (int i = 0; i < VPT; ++i)
#pragma unroll
        for (int e = 0; e < 8; ++e) part[rl - 1][(i * 8 + e) * TPR + t] = aw[i][e];
    __syncthreads();
    if (rl > 0) return;
  }
#pragma unroll
  for (int i = 0; i < VPT; ++i) {
    if (RPB > 1)
#pragma unroll
      for (int e = 0; e < 8; ++e)
#pragma unroll
        for (int r = 0; r < RPB - 1; ++r) aw[i][e] += part[r][(i * 8 + e) * TPR + t];
    store8<float, TPR, HOW, false>(out, t, i, g.cols, aw[i]);
  }
}

// Rows too long for the registers: a block's columns of dw are added up in its
// row of `partials`, which it alone touches.
template <typename T, int HOW>
__global__ __launch_bounds__(1024) void rms_norm_backward_long_kernel(const RmsNormGradArgs g) {
  __shared__ float red[2][16];
  const int t = threadIdx.x, nv = (g.cols + 8191) / 8192;
  const float inv_n = 1.0f / (float)g.cols;
  float* out = g.partials ? g.partials + (size_t)blockIdx.x * partials_ld(g.cols) : nullptr;
  int turn = 0;
  bool first = true;
  for (long long row = blockIdx.x; row < g.rows; row += gridDim.x) {
    const T* x = reinterpret_cast<const T*>(g.x) + row * g.ldx;
    const T* dy = reinterpret_cast<const T*>(g.dy) + row * g.lddy;
    const T* dt = g.dtotal ? reinterpret_cast<const T*>(g.dtotal) + row * g.lddt : nullptr;
    const float rstd = g.rstd[row];
    float c = 0.0f, fx[8], fd[8], ft[8], w[1][8];
    for (int i = 0; i < nv; ++i) {
      unpack8(load8<T, 1024, HOW>(x, t, i, g.cols), fx);
      unpack8(load8<T, 1024, HOW>(dy, t, i, g.cols), fd);
      params<1024, 1, HOW>(g.w, g.param_dtype, t, i, g.cols, 1.0f, w);
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const float th = fx[e] * rstd;
        c = fmaf(fd[e] * w[0][e], th, c);
        const int at = column<1024, HOW>(t, i, e);
        if (out != nullptr && at < g.cols) out[at] = first ? fd[e] * th : fmaf(fd[e], th, out[at]);
      }
    }
    first = false;
    c = row_sum<16>(c, red[turn]) * inv_n;
    turn ^= 1;
    if (g.dx == nullptr) continue;
    T* dx = reinterpret_cast<T*>(g.dx) + row * (long long)g.cols;
    for (int i = 0; i < nv; ++i) {
      unpack8(load8<T, 1024, HOW>(x, t, i, g.cols), fx);
      unpack8(load8<T, 1024, HOW>(dy, t, i, g.cols), fd);
      Raw8<T> rt{};
      if (dt != nullptr) rt = load8<T, 1024, HOW>(dt, t, i, g.cols);
      unpack8(rt, ft);
      params<1024, 1, HOW>(g.w, g.param_dtype, t, i, g.cols, 1.0f, w);
#pragma unroll
      for (int e = 0; e < 8; ++e) fx[e] = fmaf(rstd, fmaf(fd[e], w[0][e], -(fx[e] * rstd) * c), ft[e]);
      store8<T, 1024, HOW, false>(dx, t, i, g.cols, fx);
    }
  }
}

// dw: the sum of `blocks` rows of partials, 16 columns to a block, 64 interleaved
// runs of rows each.  Rows and runs are joined as a tree, in a fixed order: a row
// of the first 512 passes 9 additions (1003 x 1531: dw off by 0.92e-7, root mean square,
// 1.6e-7 with the runs one after another).  A run's rows are on their way eight at a
// time, so that 512 rows are one round of loads: latency bounds it (512 rows of 1531
// columns 3.4 us; 16 runs of 64 columns 5.4).
constexpr int kRuns = 64, kRunAhead = 8;
template <int N> __device__ __forceinline__ float tree_sum(float (&x)[N]) {
#pragma unroll
  for (int h = N / 2; h > 0; h /= 2)
#pragma unroll
    for (int u = 0; u < h; ++u) x[u] += x[u + h];
  return x[0];
}
__global__ __launch_bounds__(16 * kRuns) void rms_norm_params_kernel(const float* partials, int blocks, int cols, void* dw,
                                                                      int pdt) {
  __shared__ float sum[kRuns / 4][16];  // of a wave's four runs
  const int col = threadIdx.x & 15, run = threadIdx.x >> 4, c = blockIdx.x * 16 + col, ld = partials_ld(cols);
  float s = 0.0f;
  if (c < cols)
    for (int p0 = run; p0 < blocks; p0 += kRuns * kRunAhead) {
      float x[kRunAhead];
#pragma unroll
      for (int u = 0; u < kRunAhead; ++u) x[u] = partials[(size_t)min(p0 + u * kRuns, blocks - 1) * ld + c];
#pragma unroll
      for (int u = 0; u < kRunAhead; ++u) x[u] = p0 + u * kRuns < blocks ? x[u] : 0.0f;
      s += tree_sum(x);
    }
  s += __shfl_xor(s, 16, 64);
  s += __shfl_xor(s, 32, 64);
  if (run % 4 == 0) sum[run / 4][col] = s;
  __syncthreads();
  if (run == 0 && c < cols) {
    float x[kRuns / 4];
#pragma unroll
    for (int r = 0; r < kRuns / 4; ++r) x[r] = sum[r][col];
    store_param(dw, pdt, c, tree_sum(x));
  }
}

template <typename T, int HOW, bool EIGHT>
void launch_forward(const RmsNormArgs& g, hipStream_t st) {
  const NormShape s = rms_shape(g.cols);
  const dim3 grid((unsigned)norm_blocks(g.rows, s, kNormForwardBlocks)), block(s.tpr == 64 ? 256 : s.tpr);
#define NS_RMS(TPR, VPT) \
  if (s.tpr == TPR && s.vpt == VPT) return dispatch(rms_norm_kernel<T, TPR, VPT, HOW, EIGHT>, grid, block, st, g)
  NS_RMS(64, 1);
  NS_RMS(64, 2);
  NS_RMS(64, 4);
  if constexpr (HOW == kSingles) NS_RMS(256, 1);
  NS_RMS(256, 2);
  NS_RMS(256, 4);
  NS_RMS(1024, 2);
  NS_RMS(1024, 4);
#undef NS_RMS
  dispatch(rms_norm_long_kernel<T, HOW, EIGHT>, grid, block, st, g);
}

template <typename T, int HOW>
void launch_backward(const RmsNormGradArgs& g, int blocks, hipStream_t st) {
  const NormShape s = rms_shape(g.cols);
  const dim3 grid((unsigned)blocks), block(s.tpr == 64 ? 256 : s.tpr);
#define NS_RMS(TPR, VPT) \
  if (s.tpr == TPR && s.vpt == VPT) return dispatch(rms_norm_backward_kernel<T, TPR, VPT, HOW>, grid, block, st, g)
  NS_RMS(64, 1);
  NS_RMS(64, 2);
  NS_RMS(64, 4);
  if constexpr (HOW == kSingles) NS_RMS(256, 1);
  NS_RMS(256, 2);
  NS_RMS(256, 4);
  NS_RMS(1024, 2);
  NS_RMS(1024, 4);
#undef NS_RMS
  dispatch(rms_norm_backward_long_kernel<T, HOW>, grid, block, st, g);
}

template <typename T>
void launch_forward_of(const RmsNormArgs& g, hipStream_t st) {
  const bool vectors = g.ldx % 8 != 0 || (g.residual && g.ldr % 8 != 0);
  if (g.q)
    vectors ? launch_forward<T, kVectors, true>(g, st) : launch_forward<T, kAligned, true>(g, st);
  else if (g.cols % 8 != 0)
    launch_forward<T, kSingles, false>(g, st);
  else
    vectors ? launch_forward<T, kVectors, false>(g, st) : launch_forward<T, kAligned, false>(g, st);
}
template <typename T>
void launch_backward_of(const RmsNormGradArgs& g, int blocks, hipStream_t st) {
  if (g.cols % 8 != 0)
    launch_backward<T, kSingles>(g, blocks, st);
  else if (g.ldx % 8 != 0 || g.lddy % 8 != 0 || (g.dtotal && g.lddt % 8 != 0))
    launch_backward<T, kVectors>(g, blocks, st);
  else
    launch_backward<T, kAligned>(g, blocks, st);
}

}  // namespace

hipError_t launch_rms_norm(int dtype, const RmsNormArgs& args, hipStream_t st) {
  RmsNormArgs g = args;
  const long long n = g.rows * g.cols, es = dtype == 1 ? 2 : 4;
  g.stream = beyond_l2((g.total ? n * es : 0) + (g.y ? n * es : 0) + (g.q ? n : 0));
  dtype == 1 ? launch_forward_of<bf16>(g, st) : launch_forward_of<float>(g, st);
  return hipGetLastError();
}

hipError_t launch_rms_norm_backward(int dtype, const RmsNormGradArgs& args, int blocks, hipStream_t st) {
  RmsNormGradArgs g = args;
  g.stream = beyond_l2(g.rows * g.cols * (dtype == 1 ? 2 : 4));
  if (blocks > 0) {
    dtype == 1 ? launch_backward_of<bf16>(g, blocks, st) : launch_backward_of<float>(g, blocks, st);
    if (hipError_t e = hipGetLastError()) return e;
  }
  if (g.dw == nullptr) return hipSuccess;
  dispatch(rms_norm_params_kernel, dim3((unsigned)((g.cols + 15) / 16)), dim3(16 * kRuns), st, (const float*)g.partials, blocks,
           g.cols, g.dw, g.param_dtype);
  return hipGetLastError();
}

}  // namespace ns
