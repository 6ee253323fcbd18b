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

// 16 bytes per lane to a buffer; an offset out of range stores nothing.
__device__ __forceinline__ void store16(u32x4 v, unsigned voff, i32x4 rsrc) {
  const __amdgpu_buffer_rsrc_t r = __builtin_amdgcn_make_buffer_rsrc(
      reinterpret_cast<void*>((unsigned long long)(unsigned)rsrc[0] | (unsigned long long)(unsigned)rsrc[1] << 32), 0, rsrc[2], rsrc[3]);
  __builtin_amdgcn_raw_buffer_store_b128(v, r, (int)voff, 0, 0);
}

// The ring of the other products (ns_experts.hip): stage kt in slot kt % ST, its
// loads ST - 1 stages ahead, the next step's fragments read while a step's
// products run.  A stage is 128 bytes of k (8 chunks of 16) of BM rows of x and
// BN of w, and one scale byte of each row, as dwords.  x's rows are gathered on
// the way.  T: the result's type, and with it the arithmetic.
// KG groups of waves share a tile, each with a ring and every KG-th block of k; the
// first adds the others' sums to its own, in order.
template <typename T, int BM, int BN, int WM, int WN, int ST, int OCC, int KG, bool ONCE>
__global__ __launch_bounds__(WM* WN* KG * 64, (OCC * WM * WN * KG + 3) / 4) void experts_scaled_kernel(const ScaledArgs g) {
  constexpr bool EXACT = sizeof(T) == 4;
  constexpr int NW = WM * WN, CPR = 8, BK = 16 * CPR;
  static_assert(BK == kScaleBlock, "a stage has one scale");
  constexpr int WTM = BM / WM, WTN = BN / WN, SM = WTM / 32, SN = WTN / 32;
  constexpr int LP = BM * CPR, LQ = BN * CPR, STAGE = LP + LQ;
  constexpr int SP = (BM + 63) / 64, SQ = (BN + 63) / 64;  // loads of x's scales, and of w's: one to a wave, or both to one
  constexpr bool BOTH = NW == 1;
  static_assert(SP + SQ <= (BOTH ? 2 : NW), "loads of scales");
  constexpr int NP = LP / 64 / NW, NQ = LQ / 64 / NW, LD = NP + NQ + (BOTH ? 2 : 1);  // a wave's loads of a stage
  constexpr int SCALES = (BOTH ? 2 : NW) * 64;                                         // of a stage, each a dword
  static_assert(WTM % 32 == 0 && WTN % 32 == 0, "wave tile must be whole 32x32 blocks");
  static_assert(LP % (64 * NW) == 0 && LQ % (64 * NW) == 0, "operands must split into whole wave loads");
  static_assert(ST >= 2 && ST <= 5 && LD * (ST - 2) < 64, "ring depth");
  constexpr int OPITCH = WTN / Elem<T>::kChunk + 1, OUT = NW * 32 * OPITCH;
  constexpr int PART = SM * SN * 4 * 64;  // chunks of a wave's sums
  static_assert(KG == 1 || OUT + (KG - 1) * NW * PART <= KG * ST * STAGE, "the groups' sums fit the ring");
  __shared__ uint4 lds[KG * ST * STAGE > OUT ? KG * ST * STAGE : OUT];  // the rings, then the output
  __shared__ unsigned scale_ring[KG * ST * SCALES];

  const int lane = threadIdx.x & 63;
  const int wave_of_all = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int wave = wave_of_all % NW, group = wave_of_all / NW;
  const int wm = wave / WN, wn = wave % WN;
  uint4* const ring = lds + group * ST * STAGE;
  unsigned* const scales = scale_ring + group * ST * SCALES;
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
  int ti, tj;
  if (g.offsets != nullptr) {
    tl = find_tile(g, BM, upto, lin / tiles_n);
    if (tl.count <= 0) return;  // (only offsets that are no prefix sums lead here)
  } else {
    tl.tile = lin / tiles_n;
    tl.count = g.n_rows;
  }
  // neighbours within an expert share rows of x or of w: up to 8 of its row tiles at a time, column by column
  rect_decode(tl.tile * tiles_n + lin % tiles_n, (tl.count + BM - 1) / BM, tiles_n, ti, tj);
  const int i0 = ti * BM, j0 = tj * BN;

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
  // The scales: load s < SP has those of x's rows 64 s .., the next SQ those of w's.
  unsigned soff[BOTH ? 2 : 1];
  i32x4 rS[BOTH ? 2 : 1];
#pragma unroll
  for (int u = 0; u < (BOTH ? 2 : 1); ++u) {
    const int s = BOTH ? u : wave;
    soff[u] = kOutOfRange;
    if (s < SP) {
      const int r = 64 * s + lane < BM ? row_of(64 * s + lane) : -1;
      if (r >= 0) soff[u] = (unsigned)r * (unsigned)kb;
    } else if (s < SP + SQ) {
      const int j = j0 + 64 * (s - SP) + lane;
      if (64 * (s - SP) + lane < BN && j < N) soff[u] = (unsigned)(j / kScaleBlock) * (unsigned)kb;
    }
    rS[u] = uniform(s < SP ? make_rsrc(g.x_scales + (size_t)first * kb, (unsigned)x_rows * (unsigned)kb)
                           : make_rsrc(g.w_scales + (size_t)tl.expert * nb * kb, (unsigned)(nb * kb)));
  }

  auto issue = [&](int kt, int slot, auto whole) __attribute__((always_inline)) {
    constexpr bool WHOLE = decltype(whole)::value;
    const int block = kt * KG + group, k0 = block * BK;
    const bool all = WHOLE || k0 + BK <= K;
#pragma unroll
    for (int t = 0; t < NP + NQ; ++t) {
      const int idx = t < NP ? wave * NP + t : LP / 64 + wave * NQ + t - NP;
      const unsigned at = all || k0 + dma_src(idx, lane, BM, BN, CPR, 16, false, false, 1).kpos < K ? off[t] + (unsigned)k0
                                                                                                    : kOutOfRange;
      const unsigned to = lds_addr(ring + slot * STAGE + idx * 64);
      if (t < NP) dma16(to, at, rP);
      else if constexpr (ONCE) dma16_once(to, at, rQ);
      else dma16(to, at, rQ);
    }
#pragma unroll
    for (int u = 0; u < (BOTH ? 2 : 1); ++u) {  // (past the row's last block there is no scale of its own)
      const unsigned at = KG == 1 || WHOLE || block < kb ? soff[u] + (unsigned)block : kOutOfRange;
      dma1(lds_addr(reinterpret_cast<const uint4*>(scales + slot * SCALES + (BOTH ? u : wave) * 64)), at, rS[u]);
    }
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
  const char* lb = reinterpret_cast<const char*>(ring);
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
    const unsigned* st = scales + slot * SCALES + (lane & 31);
#pragma unroll
    for (int a = 0; a < SM; ++a) sp[a] = st[wm * WTM + 32 * a];
#pragma unroll
    for (int b = 0; b < SN; ++b) sq[b] = st[SP * 64 + wn * WTN + 32 * b];
  };

  const int nk = (kb + KG - 1) / KG;
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
  if constexpr (KG > 1) {
    float4* const part = reinterpret_cast<float4*>(lds + OUT) + wave * PART + lane;
    auto place = [&](int from, int a, int b, int rg) { return part + (from - 1) * NW * PART + ((a * SN + b) * 4 + rg) * 64; };
#pragma unroll
    for (int a = 0; a < SM; ++a)
#pragma unroll
      for (int b = 0; b < SN; ++b)
#pragma unroll
        for (int rg = 0; rg < 4; ++rg)
          if (group > 0) *place(group, a, b, rg) = __builtin_bit_cast(float4, acc_of(acc[a][b], rg));
    __syncthreads();
    if (group > 0) return;
#pragma unroll
    for (int from = 1; from < KG; ++from)
#pragma unroll
      for (int a = 0; a < SM; ++a)
#pragma unroll
        for (int b = 0; b < SN; ++b)
#pragma unroll
          for (int rg = 0; rg < 4; ++rg) {
            const float4 v = *place(from, a, b, rg);
            acc[a][b][4 * rg] += v.x;
            acc[a][b][4 * rg + 1] += v.y;
            acc[a][b][4 * rg + 2] += v.z;
            acc[a][b][4 * rg + 3] += v.w;
          }
  }

  T* O = reinterpret_cast<T*>(g.out) + (size_t)tl.begin * N;
  uint4* const mine = lds + wave * 32 * OPITCH;
#pragma unroll
  for (int a = 0; a < SM; ++a) store_32_rows<T>(acc[a], mine, O, i0 + wm * WTM + a * 32, j0 + wn * WTN, tl.count, N, g.stream);
}

// v, as a value that the compiler does not know: what is computed from it for each
// tile is not kept in registers from one tile to the next.
__device__ __forceinline__ int fresh(int v) {
  asm volatile("" : "+v"(v));
  return v;
}

// Large tiles: 256 x 256 by four waves, each alone on its SIMD with 128 x 128 of it,
// one workgroup to a CU, which goes through tile after tile.
//
// The LDS holds two stages of 128 bytes of k.  Between a stage's 32 products (two
// steps of 64 bytes, 16 blocks of 32 x 32 each, 64 cycles apiece) a wave issues
// everything else:
//   products 0 ..      the reads of the second step's fragments, two at a time
//   product FREE       barrier: every wave has read the slot out; over the next
//                      SPREAD products the loads of the stage two later go out
//   product NEED       wait for the next stage's loads, barrier; the reads of its
//                      first fragments follow
// so that a load has 25 products' time and more to come back, which is what
// bounds a stage: 2660 cycles at 4096 x 4096 x 14336 and 2870 in 128 experts of
// 1536 x 2048, of which the products are 2048 (2156 without the loads).  The first
// in us: two waves on each SIMD 267, one with a single border for both barriers 195
// to 211, loads over 12, 16, 20 products from 10 on 186, 179, 177; lines brought to
// the L2 ahead by loads of a byte 201.  (Half of each line a stage and four stages
// 238: every line passes the L1 twice.)
// The last two stages of a tile load the first two of the next one, whose place
// and row numbers are looked up four stages ahead.  With 512 rows to each of 128
// experts: a workgroup for each tile 256 us, this 225, where the output's stores
// pass the L2 (nt) 241: a wave's pieces of 64 bytes then go to memory by themselves.
// The stores are 7500 cycles of a tile's 53000.  Tiles of 256 rows are padded by a
// quarter there.
constexpr int kWide = 256, kWideFree = 9, kWideNeed = 24, kWideSpread = 22, kWideLeastStages = 4;
__global__ __launch_bounds__(256, 1) void experts_scaled_wide_kernel(const ScaledArgs g) {
  constexpr int BK = kScaleBlock, SM = 4, SN = 4, NM = SM * SN, NA = 2 * NM;
  constexpr int LP = kWide * 8, STAGE = 2 * LP;  // chunks of 16 bytes
  constexpr int NP = LP / 64 / 4, LD = 2 * NP + 2;  // a wave's loads of a stage: 8 of x, 8 of w, a scale of 64 rows of each
  constexpr int READS = 2 * (SM + SN);
  constexpr int OPITCH = 5, OUT = 32 * OPITCH;  // chunks to 32 columns of output in the LDS, and to 32 such rows
  static_assert(2 * kWideFree >= READS && 2 * (NA - kWideNeed) >= READS, "two reads to a product");
  static_assert(kWideFree + kWideSpread <= NA, "a stage's loads go out within one stage");
  __shared__ uint4 ring[2 * STAGE];
  __shared__ uint4 staging[4 * 2 * OUT];
  __shared__ unsigned scale_ring[2 * 512];
  __shared__ int offsets[kMaxExperts + 1];
  __shared__ int row_numbers[256];

  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int wm = wave >> 1, wn = wave & 1;
  const int N = g.fan_out, K = g.fan_in, tiles_n = (N + kWide - 1) / kWide, nk = (K + BK - 1) / BK;
  const int kb = (int)scale_blocks(K), nb = (int)scale_blocks(N);
  const bool gather = g.rows != nullptr;

  for (int e = threadIdx.x; e <= g.experts; e += 256)
    offsets[e] = g.offsets != nullptr ? min(max(g.offsets[e], 0), g.n_rows) : e * g.n_rows;
  __syncthreads();
  struct {
    const int* offsets;
    int experts, n_rows, most_row_tiles;
  } const ex{offsets, g.experts, g.n_rows, g.most_row_tiles};
  int upto;
  const int total = count_tiles(ex, kWide, &upto) * tiles_n;
  // each XCD takes a contiguous run of the tiles, its workgroups one after another
  const int xcd = blockIdx.x % 8, per = total / 8, rem = total % 8;
  const int first_tile = xcd * per + min(xcd, rem), tiles = per + (xcd < rem ? 1 : 0);
  int local = blockIdx.x / 8;
  if (local >= tiles) return;

  struct Place {
    int expert, begin, count, i0, j0;
  };
  auto locate = [&](int at) __attribute__((always_inline)) {
    const int lin = first_tile + at;
    const Tile t = find_tile(ex, kWide, upto, lin / tiles_n);
    int ti, tj;  // neighbours within an expert share rows of x or of w: up to 8 of its row tiles at a time, column by column
    rect_decode(t.tile * tiles_n + lin % tiles_n, (max(t.count, 1) + kWide - 1) / kWide, tiles_n, ti, tj);
    return Place{t.expert, t.begin, t.count, ti * kWide, tj * kWide};
  };
  // the numbers of the wave's own 64 rows of x
  auto load_row_numbers = [&](const Place& p) __attribute__((always_inline)) {
    const i32x4 r = uniform(make_rsrc(g.rows + p.begin + p.i0, (unsigned)max(p.count - p.i0, 0) * 4u));
    dma4(lds_addr(reinterpret_cast<const uint4*>(row_numbers + wave * 64)), (unsigned)(wave * 64 + lane) * 4u, r);
  };

  // Where a tile's loads come from: a load covers 8 rows, lane l 16 bytes of row l / 8
  // at the place that the ring's swizzle gives it; byte offsets at k = 0.
  unsigned off[2 * NP], soff[2];
  i32x4 rP, rQ, rSP, rSQ;
  const int turn = (lane & 7) ^ (lane >> 3);
  auto source = [&](const Place& p) __attribute__((always_inline)) {
    const int lane = fresh(threadIdx.x & 63);
    const int turn = (lane & 7) ^ (lane >> 3);
    const int first = gather ? 0 : p.begin + p.i0;  // row of x at the descriptor's start
    const int x_rows = gather ? g.n_x : max(min(min(kWide, p.count - p.i0), g.n_x - first), 0);
    rP = uniform(make_rsrc(g.x + (size_t)first * K, (unsigned)x_rows * (unsigned)K));
    rQ = uniform(make_rsrc(g.w + (size_t)p.expert * N * K, (unsigned)N * (unsigned)K));
    rSP = uniform(make_rsrc(g.x_scales + (size_t)first * kb, (unsigned)x_rows * (unsigned)kb));
    rSQ = uniform(make_rsrc(g.w_scales + (size_t)p.expert * nb * kb, (unsigned)(nb * kb)));
    auto row_of = [&](int r) __attribute__((always_inline)) {  // r: of the wave's 64
      const int x = gather ? row_numbers[wave * 64 + r] : wave * 64 + r;
      return p.i0 + wave * 64 + r < p.count && (unsigned)x < (unsigned)x_rows ? x : -1;
    };
#pragma unroll
    for (int t = 0; t < NP; ++t) {
      const int x = row_of(8 * t + (lane >> 3)), j = p.j0 + wave * 64 + 8 * t + (lane >> 3);
      const unsigned kpos = (unsigned)(turn ^ t) * 16u;
      off[t] = x >= 0 ? (unsigned)x * (unsigned)K + kpos : kOutOfRange;
      off[NP + t] = j < N ? (unsigned)j * (unsigned)K + kpos : kOutOfRange;
    }
    const int x = row_of(lane), j = p.j0 + wave * 64 + lane;
    soff[0] = x >= 0 ? (unsigned)x * (unsigned)kb : kOutOfRange;
    soff[1] = j < N ? (unsigned)(j / kScaleBlock) * (unsigned)kb : kOutOfRange;
  };
  const unsigned ring_at = lds_addr(ring), scales_at = lds_addr(reinterpret_cast<const uint4*>(scale_ring));
  // load t of stage kt of the tile that `source` describes
  auto issue = [&](int kt, int slot, int t, int turn16) __attribute__((always_inline)) {
    if (t < 2 * NP) {
      const bool in = (turn16 ^ (t % NP * 16)) < K - kt * BK;
      const unsigned at = in ? off[t] + (unsigned)(kt * BK) : kOutOfRange;
      const unsigned to = ring_at + (unsigned)(slot * STAGE + (t < NP ? 0 : LP) + (wave * NP + t % NP) * 64) * 16u;
      dma16(to, at, t < NP ? rP : rQ);
    } else {
      const int h = t - 2 * NP;
      dma1(scales_at + (unsigned)(slot * 512 + h * 256 + wave * 64) * 4u, soff[h] + (unsigned)kt, h ? rSQ : rSP);
    }
  };

  f32x16 acc[SM][SN];
#pragma unroll
  for (int a = 0; a < SM; ++a)
#pragma unroll
    for (int b = 0; b < SN; ++b)
#pragma unroll
      for (int r = 0; r < 16; ++r) acc[a][b][r] = 0.0f;

  // A step is 64 bytes of k: chunks 2 s and 2 s + 1 of each half of the wave, the
  // same k for both operands.  The addresses move with the slot that is read.
  int kcp[4], kcq[4];
#pragma unroll
  for (int s = 0; s < 4; ++s) {
    kcp[s] = kc_lane_byte(wm * 128, s, lane, 8);
    kcq[s] = kc_lane_byte(wn * 128, s, lane, 8) + LP * 16;
  }
  const char* lb = reinterpret_cast<const char*>(ring);
  struct Chunks { uint4 v[2]; };
  Chunks pf[2][SM], qf[2][SN];
  // read r of a step's fragments, in the order in which the products take them
  auto read = [&](int s, int r) __attribute__((always_inline)) {
    const int h = r & 1, o = r / 2, a = o == 0 ? 0 : o - SN, b = o - 1;
    if (o == 0 || o > SN)
      pf[s][a].v[h] = *reinterpret_cast<const uint4*>(lb + kcp[(2 * s + h) ^ kc_sigma(a, 8)] + a * 32 * 128);
    else
      qf[s][b].v[h] = *reinterpret_cast<const uint4*>(lb + kcq[(2 * s + h) ^ kc_sigma(b, 8)] + b * 32 * 128);
  };
  struct Scales {
    unsigned p[SM], q[SN];
  };
  Scales z, z_next;
  auto read_scales = [&](int slot, Scales& to) __attribute__((always_inline)) {
    const unsigned* st = scale_ring + slot * 512 + (lane & 31);
#pragma unroll
    for (int a = 0; a < SM; ++a) to.p[a] = st[wm * 128 + 32 * a];
#pragma unroll
    for (int b = 0; b < SN; ++b) to.q[b] = st[256 + wn * 128 + 32 * b];
  };
  auto due = [](int at) { return at < kWideSpread ? at * LD / kWideSpread : LD; };  // loads out when `at` products are, from FREE on

  Place here = locate(local);
  if (gather) {
    load_row_numbers(here);
    wait_vm_lgkm0<0>();
    asm volatile("" ::: "memory");
  }
  source(here);
#pragma unroll
  for (int s = 0; s < 2; ++s)
#pragma unroll
    for (int t = 0; t < LD; ++t) issue(s, s, t, 16 * turn);
  wait_vm_lgkm0<0>();
  ring_barrier();
  read_scales(0, z);
#pragma unroll
  for (int r = 0; r < READS; ++r) read(0, r);

  // A tile's output goes out block by block (32 x 32, number j = 4 a + b): at turn t
  // block t is rounded into one of the wave's two buffers, block t - 1 read from the
  // other as whole rows, block t - 2 stored.  Every store is issued, rows and columns
  // past the end out of range, so that the waits know how many are in flight.
  constexpr int STORES = 2 * NM;
  uint4* const mine = staging + wave * 2 * OUT;
  u32x4 v[2][2];
  auto turn_out = [&](int t, int lane, i32x4 rO, int j0) __attribute__((always_inline)) {
    if (t >= 2) {
      const int j = t - 2, col = j0 + wn * 128 + j % SN * 32 + (lane & 3) * 8;
      const int row = wm * 128 + j / SN * 32 + (lane >> 2);
      const unsigned at = col < N ? (unsigned)(row * N + col) * 2u : kOutOfRange;
#pragma unroll
      for (int c = 0; c < 2; ++c) store16(v[j & 1][c], at + (unsigned)(c * 16 * N) * 2u, rO);
    }
    if (t >= 1 && t <= NM)
#pragma unroll
      for (int c = 0; c < 2; ++c)
        v[(t - 1) & 1][c] = __builtin_bit_cast(u32x4, mine[((t - 1) & 1) * OUT + (16 * c + (lane >> 2)) * OPITCH + (lane & 3)]);
    if (t < NM) {
      f32x16 block = acc[t / SN][t % SN];
      asm volatile("" : "+a"(block));  // until here it stays where the products put it
#pragma unroll
      for (int rg = 0; rg < 4; rg += 2) {
        const uint2 x = pack4(acc_of(block, rg)), y = pack4(acc_of(block, rg + 1));
        const auto p = __builtin_amdgcn_permlane32_swap(x.x, y.x, false, false);
        const auto q = __builtin_amdgcn_permlane32_swap(x.y, y.y, false, false);
        mine[(t & 1) * OUT + acc_i(lane) * OPITCH + rg + (lane >> 5)] = make_uint4(p[0], q[0], p[1], q[1]);
      }
    }
  };

  // Stage kt, in `slot`, with the loads of stage `later` of its own tile or the next.
  // first: it is a tile's first, whose products start from zero.  The last tile's stores
  // may be in flight too, which are newer than the loads that NEED waits for (there are
  // none in the first tile, whose first two stages have been waited for).
  auto stage = [&](int slot, int later, auto first) __attribute__((always_inline)) {
    constexpr bool FIRST = decltype(first)::value;
    const int turn16 = fresh(16 * turn);
#pragma unroll
    for (int n = 0; n < NA; ++n) {
      const int s = n / NM, i = n % NM;
      if (n == kWideFree) {
        wait_vm_lgkm0<63>();
        ring_barrier();
      }
      if (n == kWideNeed) {
        wait_vm_lgkm0<(kWideNeed - kWideFree) * LD / kWideSpread + (FIRST ? STORES : 0)>();
        ring_barrier();
        read_scales(slot ^ 1, z_next);
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          kcp[c] ^= STAGE * 16;
          kcq[c] ^= STAGE * 16;
        }
      }
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        if (s == 0 && 2 * i + h < READS) read(1, 2 * i + h);
        if (n >= kWideNeed && 2 * (n - kWideNeed) + h < READS) read(0, 2 * (n - kWideNeed) + h);
      }
      if (n >= kWideFree)
#pragma unroll
        for (int t = due(n - kWideFree); t < due(n - kWideFree + 1); ++t) issue(later, slot, t, turn16);
      __builtin_amdgcn_sched_barrier(0);  // keeps the loads and reads where they are
      f32x16 sum = acc[i / SN][i % SN];
      if (FIRST && s == 0) sum = f32x16{};
      sum = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(join(qf[s][i % SN].v[0], qf[s][i % SN].v[1]),
                                                            join(pf[s][i / SN].v[0], pf[s][i / SN].v[1]), sum, 0, 0, 0,
                                                            (int)z.q[i % SN], 0, (int)z.p[i / SN]);
      acc[i / SN][i % SN] = sum;
    }
    z = z_next;
  };
  int slot = 0;  // of the stage that is computed
  for (;;) {
    const bool more = local + (int)gridDim.x / 8 < tiles;
    Place next = here;
    auto ahead = [&](int kt) __attribute__((always_inline)) {  // what stage kt does for the next tile
      if (kt == nk - 4 && more) {
        next = locate(local + (int)gridDim.x / 8);
        if (gather) load_row_numbers(next);  // (older than the loads that may be in flight at NEED)
      }
      if (kt == nk - 2) {
        if (more) source(next);
        else rP[2] = rQ[2] = rSP[2] = rSQ[2] = 0;  // nothing is left to load: all of it is out of range
      }
    };
    ahead(0);
    stage(slot, 2, std::true_type());
    slot ^= 1;
    for (int kt = 1; kt < nk; ++kt) {
      ahead(kt);
      stage(slot, kt + 2 < nk ? kt + 2 : kt + 2 - nk, std::false_type());
      slot ^= 1;
    }
    const int rows = max(min(kWide, here.count - here.i0), 0), out_lane = fresh(lane);
    const i32x4 rO = uniform(make_rsrc(reinterpret_cast<bf16*>(g.out) + (size_t)(here.begin + here.i0) * N, (unsigned)(rows * N) * 2u));
#pragma unroll
    for (int t = 0; t < NM + 2; ++t) turn_out(t, out_lane, rO, here.j0);
    if (!more) break;
    here = next;
    local += (int)gridDim.x / 8;
  }
  wait_vm_lgkm0<0>();  // (loads of nothing may still be on their way to the LDS)
}

// Row tiles of bm that n_rows rows can make: the sum of ceil(c / bm) over at most min(experts, n_rows) experts with rows.
long long most_row_tiles(const ScaledArgs& g, int bm) {
  return (g.n_rows + (long long)std::min(g.experts, g.n_rows) * (bm - 1)) / bm;
}

template <typename T, int BM, int BN, int WM, int WN, int ST, int OCC, int KG>
hipError_t launch_tiles(ScaledArgs g, hipStream_t st) {
  const long long tiles_n = (g.fan_out + BN - 1) / BN;
  const long long most = most_row_tiles(g, BM);
  g.most_row_tiles = (int)most;
  long long grid = most * tiles_n;
  grid = (grid + 7) / 8 * 8;  // every XCD reaches its last live tile
  if (grid <= 0) return hipSuccess;
  if (grid * (WM * WN * KG * 64) >= 1ll << 32) return hipErrorInvalidValue;  // a launch holds fewer threads
  const dim3 blocks((unsigned)grid), threads(WM * WN * KG * 64);
  constexpr bool FEW = BM == 32;
  const bool once = FEW && beyond_l2((long long)g.experts * g.fan_out * g.fan_in);
  g.stream = beyond_l2((long long)g.n_rows * g.fan_out * (long long)sizeof(T));
  if (once) dispatch(experts_scaled_kernel<T, BM, BN, WM, WN, ST, OCC, KG, FEW>, blocks, threads, st, g);
  else dispatch(experts_scaled_kernel<T, BM, BN, WM, WN, ST, OCC, KG, false>, blocks, threads, st, g);
  return hipGetLastError();
}

// Tiles of a launch: BM, BN, waves, stages, workgroups per CU, groups of waves.
#define NS_SCALED_TALL 128, 256, 2, 4, 3, 1, 1
#define NS_SCALED_LONG 128, 128, 2, 4, 4, 1, 1
#define NS_SCALED_SMALL 64, 64, 2, 2, 3, 3, 1
#define NS_SCALED_FEW 32, 64, 1, 2, 4, 3, 1
#define NS_SCALED_SPLIT 32, 32, 1, 1, 4, 1, 4
enum ScaledTile { TILE_WIDE, TILE_TALL, TILE_LONG, TILE_SMALL, TILE_FEW, TILE_SPLIT };

// The largest tile that makes about 160 workgroups (240 of the small ones, of which
// three share a CU): a large tile reads less for each product, a small one fills
// the CUs and pads less.  An expert's last tile is taken as half full.  us, bf16
// results, 1536 x 2048 if not said (N: estimated tiles):
//   wide / tall   8 experts of 1024 rows 28 (216) / 36, of 512 rows 25 (120) / 19 (216);
//                 128 experts of 128 rows 113 / 117, of 64 rows 107 / 99;
//                 2048 rows, 4096 x 4096 43 (136) / 34 (264)
//   tall / long   8 experts of 256 rows 17 (120) / 13 (240); 1024 rows, 4096 x
//                 4096 26 (136) / 21 (272)
//   long / small  2048 rows 11.5 (198) / 13.4, 1024 rows 10.7 (102) / 9.3; 8
//                 experts of 128 rows 11.7 (144) / 10.8 (288)
//   small / few   1024 rows 9.3 (396) / 10.1; 128 rows, 4096 x 4096 11.2 (160) /
//                 8.6; 128 experts of 16 rows 80 / 71
// That holds where an expert has rows for much of a tile.  With fewer every expert has one
// tile whatever its height, so that many experts make many tiles, and what a tall one does
// for no rows counts.  By rows of each expert (E of 1536 x 2048; K: 64 of 1280 x 512), us:
//   bf16   16: E = 128 wide 81, tall 80, small 80, few 71    64: 53, 48, 42, 38   K: 21, 17, 13, 13
//          20:              84       80        83      79        52  47  45  41      22  17  13  14
//          28:              87       87        90      96        53  49  46  45      22  18  14  18
//          32:              87       91        93     103        53  49  47  50      22  18  14  18
//          48:              90       96       103     131        55  51  54  65      22  19  16  23
//   fp32   20: E = 128 tall 94, small 91, few 90             64: 56, 46, 46       K: 22, 15, 17
//          32:             104        98     110                 58  52  55          22  16  21
//          47:             116       111     131                 60  59  71          23  19  26
//          64:             121       128     154                 63  66  80          24  21  30
//   long, small: 32 of 1536 x 2048, 20 rows 27 / 25 (fp32 35 / 26), 24 of them 23 / 17 (32 / 19);
//                one to a CU, 8 of 4096 x 14336 84 / 92
//   few, small, 17 to 20 rows: 64 of 1280 x 512 14 / 13, 512 of 256 x 512 28 / 22, 128 of
//                2048 x 768 48 / 52, 256 of 512 x 1024 33 / 35, 4 of 24576 x 4096 71 / 83
// So with up to kFewRows rows 32 x 64 is taken there (from kFewLeastBlocks blocks of k on),
// and otherwise 64 x 64 with fewer than kTallRows.
// For one matrix, whose tiles are known, fewer than 240 small ones are taken too where
// those of 32 x 64 are more than one to a CU: 4096 x 14336, 128 rows (256 of them) 30 / 30, 129 rows (320) 31 / 58,
// 200 rows 32 / 60; x 512, 200 rows 4.1 / 4.8; 2048 x 7168, 256 rows (256) 17 / 12, 300
// rows (320) 17 / 18.
// fp32 results go the same way, without the wide tile: tall / long 8 experts of 512
// rows 29 / 36, of 256 rows 26 / 19; long / small 2048 rows 18 / 19, 1024 rows 16 / 14.
//
// Where tiles of 32 x 32 leave no CU more than one, and so few workgroups would wait
// for their loads one after another, four groups of waves share k (split), each with
// three stages on their way.  32 x 64 / split, us, one matrix, in a graph if below 8:
//   1 row: 4096 x 14336 29 / 15 (58.7 MB: 11.3 at a large copy's rate), 16 rows of
//   4096 x 4096 8.1 / 6.2, 1536 x 2048 5.1 / 4.4, x 512 3.7 / 3.4, x 384 3.5 / 3.4, x 256
//   3.3 / 3.4, x 128 3.1 / 3.4; 64 rows of 4096 x 14336 32 / 21, 128 rows of 2048 x 7168
//   (256 tiles) 11.5 / 8.7; 4 of 16 experts of 2048 x 7168 (256) 17.5 / 11.8; with more
//   tiles 1 row of 14336 x 4096 (448) 12.2 / 13.8, 128 rows of 4096 x 14336 (512) 32 / 39,
//   32 experts of 1536 x 2048 16 / 27.  fp32 results: 4096 x 14336 35 / 17, 16 rows of
//   4096 x 4096 12.3 / 7.7, 1536 x 384 3.9 / 3.6, x 256 3.5 / 3.6.
// (Two groups, two workgroups to a CU: 17 in the first case and 4 % less at 1536 x 512;
// 32 x 64 by four groups 23; six or eight groups with fewer stages 16 and 22.)
constexpr int kCUs = 256, kSplitLeastBlocks = 4;
constexpr int kFewRows = 20, kFewLeastBlocks = 5, kTallRows[2] = {48, 32};  // (fp32 results, bf16)
ScaledTile choose_tile(int dtype, const ScaledArgs& g) {
  const int rows = g.n_rows / g.experts;  // an expert's, on average
  auto tiles = [&](int bm, int bn) {
    return ((long long)g.n_rows / bm + std::min(g.experts, g.n_rows) / 2.0) * ((g.fan_out + bn - 1) / bn);
  };
  if (rows > 16) {
    const bool many = g.experts > 1, few = many && rows <= kFewRows;
    if (tiles(128, 256) >= 160) {
      if (few && scale_blocks(g.fan_in) >= kFewLeastBlocks) return TILE_FEW;
      if (many && rows < kTallRows[dtype]) return TILE_SMALL;
      return dtype == 1 && scale_blocks(g.fan_in) >= kWideLeastStages && tiles(kWide, kWide) >= 160 ? TILE_WIDE : TILE_TALL;
    }
    if (tiles(128, 128) >= 160) return few && g.experts * ((g.fan_out + 127) / 128) > kCUs ? TILE_SMALL : TILE_LONG;
    const bool rounds = g.experts == 1 && most_row_tiles(g, 32) * ((g.fan_out + 63) / 64) > kCUs;
    if (tiles(64, 64) >= 240 || rounds) return TILE_SMALL;
  }
  if (most_row_tiles(g, 32) * ((g.fan_out + 31) / 32) <= kCUs && scale_blocks(g.fan_in) >= kSplitLeastBlocks) return TILE_SPLIT;
  return TILE_FEW;
}

hipError_t launch_wide(ScaledArgs g, hipStream_t st) {
  const long long most = most_row_tiles(g, kWide), tiles = most * ((g.fan_out + kWide - 1) / kWide);
  if (tiles > 0x7fffffffll) return hipErrorInvalidValue;
  g.most_row_tiles = (int)most;
  const unsigned grid = (unsigned)std::min((tiles + 7) / 8 * 8, (long long)kCUs);  // a workgroup to each CU
  dispatch(experts_scaled_wide_kernel, dim3(grid), dim3(256), st, g);
  return hipGetLastError();
}

template <typename T>
hipError_t launch_type(ScaledTile tile, const ScaledArgs& g, hipStream_t st) {
  switch (tile) {
    case TILE_WIDE: return sizeof(T) == 2 ? launch_wide(g, st) : hipErrorInvalidValue;
    case TILE_TALL: return launch_tiles<T, NS_SCALED_TALL>(g, st);
    case TILE_LONG: return launch_tiles<T, NS_SCALED_LONG>(g, st);
    case TILE_SMALL: return launch_tiles<T, NS_SCALED_SMALL>(g, st);
    case TILE_SPLIT: return launch_tiles<T, NS_SCALED_SPLIT>(g, st);
    default: return launch_tiles<T, NS_SCALED_FEW>(g, st);
  }
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
    case TILE_TALL: return NS_TEXT("128x256");
    case TILE_LONG: return NS_TEXT("128x128");
    case TILE_SMALL: return NS_TEXT("64x64");
    case TILE_SPLIT: return NS_TEXT("32x32, k by 4 groups of waves");
    default: return NS_TEXT("32x64");
  }
#undef NS_TEXT
}

}  // namespace ns
