// ns_experts_scaled.hip - the products of a stack of experts with the rows routed to
// them, both in 8 bits with scales.
//
//   y[i, j] = sum_k xs[r, k / 128] ws[e, j / 128, k / 128] xq[r, k] wq[e, j, k],   r = rows[i], i in expert e's rows
//
// Scales are powers of two.  A stage of the K loop is one block of 128 columns,
// so a row of x and a row of w each have one scale byte in it, and
// v_mfma_scale_f32_32x32x64_f8f6f4 applies both at no cost: one accumulator
// runs through all blocks.  That instruction adds eight neighbouring products
// at a time after cutting each off at 2^-13 of the largest one's power of two
// (and eights in full fp32).  Rows of normal values lose 1.5e-5 of the result
// by that, rows of widely spread values 7e-5, where a bf16 result is rounded by
// 1.7e-3 (root mean squares).  Results in fp32 are exact to fp32 sums: the values,
// times their scales, are bf16 values, which are converted on their way to
// v_mfma_f32_32x32x16_bf16 at half the rate (7e-8 to 2e-7 of the result).
#include <algorithm>

#include "ns_eight.h"
#include "ns_scaled.h"
#include "ns_tiles.h"

namespace ns {
namespace {

typedef int i32x8 __attribute__((ext_vector_type(8)));
__device__ __forceinline__ i32x8 join(uint4 a, uint4 b) {
  return i32x8{(int)a.x, (int)a.y, (int)a.z, (int)a.w, (int)b.x, (int)b.y, (int)b.z, (int)b.w};
}

// 1 byte per lane, as a dword at m0 + 4 * lane of the LDS.
__device__ __forceinline__ void dma1(unsigned lds_byte_addr, unsigned voff, i32x4 rsrc) {
  asm volatile("s_mov_b32 m0, %0\n\tbuffer_load_ubyte %1, %2, 0 offen lds"
               :
               : "s"(lds_byte_addr), "v"(voff), "s"(rsrc)
               : "memory", "m0");
}

// The ring of the other products (ns_experts.hip): stage kt in slot kt % ST, its
// loads ST - 1 stages ahead, the next step's fragments read while a step's
// products run.  A stage is 128 bytes of k (8 chunks of 16) of BM rows of x and
// BN of w, and one scale byte of each row, as dwords.  x's rows are gathered on
// the way.  T: the result's type, and with it the arithmetic.
template <typename T, int BM, int BN, int WM, int WN, int ST, int OCC, bool ONCE>
__global__ __launch_bounds__(WM* WN * 64, (OCC * WM * WN + 3) / 4) void experts_scaled_kernel(const ScaledArgs g) {
  constexpr bool EXACT = sizeof(T) == 4;
  constexpr int NW = WM * WN, CPR = 8, BK = 16 * CPR;
  static_assert(BK == kScaleBlock, "a stage has one scale");
  constexpr int WTM = BM / WM, WTN = BN / WN, SM = WTM / 32, SN = WTN / 32;
  constexpr int LP = BM * CPR, LQ = BN * CPR, STAGE = LP + LQ;
  constexpr int NP = LP / 64 / NW, NQ = LQ / 64 / NW, LD = NP + NQ + 1;  // a wave's loads of a stage, one of scales
  constexpr int SP = (BM + 63) / 64, SQ = (BN + 63) / 64;  // waves whose scale loads are x's, and w's
  static_assert(SP + SQ <= NW, "one load of scales to a wave");
  static_assert(WTM % 32 == 0 && WTN % 32 == 0, "wave tile must be whole 32x32 blocks");
  static_assert(LP % (64 * NW) == 0 && LQ % (64 * NW) == 0, "operands must split into whole wave loads");
  static_assert(ST >= 2 && ST <= 5 && LD * (ST - 2) < 64, "ring depth");
  constexpr int OPITCH = WTN / Elem<T>::kChunk + 1, OUT = NW * 32 * OPITCH;
  __shared__ uint4 lds[ST * STAGE > OUT ? ST * STAGE : OUT];  // the ring, then the output
  __shared__ unsigned scale_ring[ST * NW * 64];

  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int wm = wave / WN, wn = wave % WN;
  const int N = g.fan_out, K = g.fan_in, tiles_n = (N + BN - 1) / BN;
  const int kb = (int)scale_blocks(K), nb = (int)scale_blocks(N);

  // this workgroup's tile: each XCD takes a contiguous run of the live ones
  Tile tl{};
  const int xcd = blockIdx.x % 8, local = blockIdx.x / 8;
  int upto = 0, total;
  if (g.offsets != nullptr) total = count_tiles(g, BM, &upto) * tiles_n;
  else total = (g.n_rows + BM - 1) / BM * tiles_n;
  const int per = total / 8, rem = total % 8;
  if (local >= per + (xcd < rem ? 1 : 0)) return;
  const int lin = xcd * per + min(xcd, rem) + local;
  if (g.offsets != nullptr) {
    tl = find_tile(g, BM, upto, lin / tiles_n);
    if (tl.count <= 0) return;  // (only offsets that are no prefix sums lead here)
  } else {
    tl.tile = lin / tiles_n;
    tl.count = g.n_rows;
  }
  const int i0 = tl.tile * BM, j0 = (lin % tiles_n) * BN;

  // Byte offsets of a wave's loads at k = 0, kOutOfRange for rows past the end.
  const bool gather = g.rows != nullptr;
  const int first = gather ? 0 : tl.begin + i0;              // row of x at the descriptors' start
  const int x_rows = gather ? g.n_x : min(BM, tl.count - i0);  // and rows that they cover
  const i32x4 rP = uniform(make_rsrc(g.x + (size_t)first * K, (unsigned)x_rows * (unsigned)K));
  const i32x4 rQ = uniform(make_rsrc(g.w + (size_t)tl.expert * N * K, (unsigned)N * (unsigned)K));
  auto row_of = [&](int r) __attribute__((always_inline)) {  // of x from `first` on; -1: none
    if (i0 + r >= tl.count) return -1;
    if (!gather) return first + r < g.n_x ? r : -1;
    const int x = g.rows[tl.begin + i0 + r];
    return (unsigned)x < (unsigned)g.n_x ? x : -1;
  };
  unsigned off[NP + NQ];
#pragma unroll
  for (int t = 0; t < NP + NQ; ++t) {
    const int idx = t < NP ? wave * NP + t : LP / 64 + wave * NQ + t - NP;
    const DmaSrc d = dma_src(idx, lane, BM, BN, CPR, 16, false, false, 1);
    if (t < NP) {
      const int r = row_of(d.row);
      off[t] = r >= 0 ? (unsigned)r * (unsigned)K + (unsigned)d.kpos : kOutOfRange;
    } else {
      const int j = j0 + d.row;
      off[t] = j < N ? (unsigned)j * (unsigned)K + (unsigned)d.kpos : kOutOfRange;
    }
  }
  // The scales: wave s < SP has those of x's rows 64 s .., the next SQ those of w's.
  unsigned soff = kOutOfRange;
  if (wave < SP) {
    const int r = 64 * wave + lane < BM ? row_of(64 * wave + lane) : -1;
    if (r >= 0) soff = (unsigned)r * (unsigned)kb;
  } else if (wave < SP + SQ) {
    const int j = j0 + 64 * (wave - SP) + lane;
    if (64 * (wave - SP) + lane < BN && j < N) soff = (unsigned)(j / kScaleBlock) * (unsigned)kb;
  }
  const i32x4 rS = uniform(wave < SP ? make_rsrc(g.x_scales + (size_t)first * kb, (unsigned)x_rows * (unsigned)kb)
                                     : make_rsrc(g.w_scales + (size_t)tl.expert * nb * kb, (unsigned)(nb * kb)));

  auto issue = [&](int kt, int slot, auto whole) __attribute__((always_inline)) {
    constexpr bool WHOLE = decltype(whole)::value;
    const int k0 = kt * BK;
    const bool all = WHOLE || k0 + BK <= K;
#pragma unroll
    for (int t = 0; t < NP + NQ; ++t) {
      const int idx = t < NP ? wave * NP + t : LP / 64 + wave * NQ + t - NP;
      const unsigned at = all || k0 + dma_src(idx, lane, BM, BN, CPR, 16, false, false, 1).kpos < K ? off[t] + (unsigned)k0
                                                                                                    : kOutOfRange;
      const unsigned to = lds_addr(lds + slot * STAGE + idx * 64);
      if (t < NP) dma16(to, at, rP);
      else if constexpr (ONCE) dma16_once(to, at, rQ);
      else dma16(to, at, rQ);
    }
    dma1(lds_addr(reinterpret_cast<const uint4*>(scale_ring + (slot * NW + wave) * 64)), soff + (unsigned)kt, rS);
  };

  f32x16 acc[SM][SN];
#pragma unroll
  for (int a = 0; a < SM; ++a)
#pragma unroll
    for (int b = 0; b < SN; ++b)
#pragma unroll
      for (int r = 0; r < 16; ++r) acc[a][b][r] = 0.0f;

  // A step is 64 bytes of k: chunks 2 s and 2 s + 1 of each half of the wave, the
  // same k for both operands.
  constexpr int KS = CPR / 4;
  int kcp[CPR / 2], kcq[CPR / 2];
#pragma unroll
  for (int s = 0; s < CPR / 2; ++s) {
    kcp[s] = kc_lane_byte(wm * WTM, s, lane, CPR);
    kcq[s] = kc_lane_byte(wn * WTN, s, lane, CPR) + LP * 16;
  }
  const char* lb = reinterpret_cast<const char*>(lds);
  struct Chunks { uint4 v[2]; };
  auto load_step = [&](int slot, int s, Chunks (&pf)[SM], Chunks (&qf)[SN]) __attribute__((always_inline)) {
    const char* st = lb + slot * STAGE * 16;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
#pragma unroll
      for (int a = 0; a < SM; ++a)
        pf[a].v[h] = *reinterpret_cast<const uint4*>(st + kcp[(2 * s + h) ^ kc_sigma(a, CPR)] + a * 32 * CPR * 16);
#pragma unroll
      for (int b = 0; b < SN; ++b)
        qf[b].v[h] = *reinterpret_cast<const uint4*>(st + kcq[(2 * s + h) ^ kc_sigma(b, CPR)] + b * 32 * CPR * 16);
    }
  };
  auto load_scales = [&](int slot, unsigned (&sp)[SM], unsigned (&sq)[SN]) __attribute__((always_inline)) {
    const unsigned* st = scale_ring + slot * NW * 64 + (lane & 31);
#pragma unroll
    for (int a = 0; a < SM; ++a) sp[a] = st[wm * WTM + 32 * a];
#pragma unroll
    for (int b = 0; b < SN; ++b) sq[b] = st[SP * 64 + wn * WTN + 32 * b];
  };

  const int nk = (K + BK - 1) / BK;
  Chunks pf[2][SM], qf[2][SN];
  unsigned sp[2][SM], sq[2][SN];
  auto wait_stage = [&](int kt, auto steady) __attribute__((always_inline)) {
    const int later = nk - 1 - kt;  // stages that may be in flight after kt, at most ST - 2
    if (decltype(steady)::value || later >= ST - 2) wait_vm_lgkm0<LD * (ST - 2)>();
    else if (ST > 4 && later == 2) wait_vm_lgkm0<LD * 2>();
    else if (ST > 3 && later == 1) wait_vm_lgkm0<LD * 1>();
    else wait_vm_lgkm0<0>();
    ring_barrier();
  };
  auto products = [&](const Chunks (&p)[SM], const Chunks (&q)[SN], const unsigned (&s)[SM], const unsigned (&z)[SN])
                      __attribute__((always_inline)) {
    if constexpr (EXACT) {
#pragma unroll
      for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int c = 0; c < 2; ++c) {  // 8 values of each row
          uint4 x[SM], w[SN];
#pragma unroll
          for (int a = 0; a < SM; ++a) {
            const uint2 lo = from_eight4(u4get(p[a].v[h], 2 * c), scale_exponent(s[a]), bf16());
            const uint2 hi = from_eight4(u4get(p[a].v[h], 2 * c + 1), scale_exponent(s[a]), bf16());
            x[a] = make_uint4(lo.x, lo.y, hi.x, hi.y);
          }
#pragma unroll
          for (int b = 0; b < SN; ++b) {
            const uint2 lo = from_eight4(u4get(q[b].v[h], 2 * c), scale_exponent(z[b]), bf16());
            const uint2 hi = from_eight4(u4get(q[b].v[h], 2 * c + 1), scale_exponent(z[b]), bf16());
            w[b] = make_uint4(lo.x, lo.y, hi.x, hi.y);
          }
#pragma unroll
          for (int a = 0; a < SM; ++a)
#pragma unroll
            for (int b = 0; b < SN; ++b) mfma_chunk(acc[a][b], w[b], x[a], bf16());
        }
    } else {
#pragma unroll
      for (int a = 0; a < SM; ++a)
#pragma unroll
        for (int b = 0; b < SN; ++b)
          acc[a][b] = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(join(q[b].v[0], q[b].v[1]), join(p[a].v[0], p[a].v[1]),
                                                                      acc[a][b], 0, 0, 0, (int)z[b], 0, (int)s[a]);
    }
  };
  // u: kt modulo an even multiple of ST, so that slots and the scales' buffers are known while compiling
  auto stage = [&](int kt, int u, auto steady) __attribute__((always_inline)) {
    constexpr bool STEADY = decltype(steady)::value;
    if (STEADY || kt + ST - 1 < nk) issue(kt + ST - 1, (u + ST - 1) % ST, steady);
#pragma unroll
    for (int s = 0; s < KS; ++s) {
      if (s + 1 < KS) {
        load_step(u % ST, s + 1, pf[(s + 1) & 1], qf[(s + 1) & 1]);
      } else if (STEADY || kt + 1 < nk) {
        wait_stage(kt + 1, steady);
        load_step((u + 1) % ST, 0, pf[0], qf[0]);
        load_scales((u + 1) % ST, sp[(u + 1) & 1], sq[(u + 1) & 1]);
      }
      __builtin_amdgcn_sched_barrier(0);  // keeps these reads ahead of the products
      products(pf[s & 1], qf[s & 1], sp[u & 1], sq[u & 1]);
    }
  };
  static_assert(KS % 2 == 0, "fragment buffers alternate");
#pragma unroll
  for (int s = 0; s < ST - 1; ++s)
    if (s < nk) issue(s, s, std::false_type());
  wait_stage(0, std::false_type());
  load_step(0, 0, pf[0], qf[0]);
  load_scales(0, sp[0], sq[0]);
  constexpr int UN = ST % 2 == 0 ? ST : 2 * ST;
  int kt0 = 0;
  for (; kt0 + UN + ST - 1 < nk; kt0 += UN) {
#pragma unroll
    for (int u = 0; u < UN; ++u) stage(kt0 + u, u, std::true_type());
  }
#pragma unroll
  for (int u = 0; u < UN + ST - 1; ++u)
    if (kt0 + u < nk) stage(kt0 + u, u, std::false_type());
  __syncthreads();

  T* O = reinterpret_cast<T*>(g.out) + (size_t)tl.begin * N;
  uint4* const mine = lds + wave * 32 * OPITCH;
#pragma unroll
  for (int a = 0; a < SM; ++a) store_32_rows<T>(acc[a], mine, O, i0 + wm * WTM + a * 32, j0 + wn * WTN, tl.count, N, g.stream);
}

template <typename T, int BM, int BN, int WM, int WN, int ST, int OCC>
hipError_t launch_tiles(ScaledArgs g, hipStream_t st) {
  const long long tiles_n = (g.fan_out + BN - 1) / BN;
  // sum of ceil(c / BM) over at most min(experts, n_rows) non-empty experts
  const long long some = g.experts < g.n_rows ? g.experts : g.n_rows;
  long long grid = ((g.n_rows + some * (BM - 1)) / BM) * tiles_n;
  grid = (grid + 7) / 8 * 8;  // every XCD reaches its last live tile
  if (grid <= 0) return hipSuccess;
  if (grid > 0x7fffffffll) return hipErrorInvalidValue;
  const dim3 blocks((unsigned)grid), threads(WM * WN * 64);
  constexpr bool FEW = BM == 32;
  const bool once = FEW && beyond_l2((long long)g.experts * g.fan_out * g.fan_in);
  g.stream = beyond_l2((long long)g.n_rows * g.fan_out * (long long)sizeof(T));
  if (once) dispatch(experts_scaled_kernel<T, BM, BN, WM, WN, ST, OCC, FEW>, blocks, threads, st, g);
  else dispatch(experts_scaled_kernel<T, BM, BN, WM, WN, ST, OCC, false>, blocks, threads, st, g);
  return hipGetLastError();
}

#define NS_SCALED_WIDE 256, 256, 2, 4, 2, 1
#define NS_SCALED_SMALL 64, 64, 2, 2, 3, 3
#define NS_SCALED_FEW 32, 64, 1, 2, 4, 3
enum ScaledTile { TILE_WIDE, TILE_SMALL, TILE_FEW };

ScaledTile choose_tile(int dtype, const ScaledArgs& g) {
  const int rows = g.n_rows / g.experts;  // an expert's, on average
  if (rows <= 16) return TILE_FEW;
  if (dtype == 1 && rows >= 128) return TILE_WIDE;
  return TILE_SMALL;
}

template <typename T>
hipError_t launch_type(ScaledTile tile, const ScaledArgs& g, hipStream_t st) {
  switch (tile) {
    case TILE_WIDE:
      if constexpr (sizeof(T) == 2) return launch_tiles<T, NS_SCALED_WIDE>(g, st);
      break;
    case TILE_SMALL: return launch_tiles<T, NS_SCALED_SMALL>(g, st);
    case TILE_FEW: return launch_tiles<T, NS_SCALED_FEW>(g, st);
  }
  return hipErrorInvalidValue;
}

}  // namespace

hipError_t launch_experts_scaled(int dtype, const ScaledArgs& g, hipStream_t st) {
  const ScaledTile tile = choose_tile(dtype, g);
  return dtype == 1 ? launch_type<bf16>(tile, g, st) : launch_type<float>(tile, g, st);
}

const char* experts_scaled_config(int dtype, const ScaledArgs& g) {
#define NS_TEXT(TILE) "experts product of 8-bit values: result=%s rows=%lld experts=%lld fan_out=%lld fan_in=%lld | tile=" TILE
  switch (choose_tile(dtype, g)) {
    case TILE_WIDE: return NS_TEXT("256x256");
    case TILE_SMALL: return NS_TEXT("64x64");
    default: return NS_TEXT("32x64");
  }
#undef NS_TEXT
}

}  // namespace ns
