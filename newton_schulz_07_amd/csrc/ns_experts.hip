// ns_experts.hip - the products of a stack of experts with the rows routed
// to them, their gradients, and the weighted sum of the results per token.
//
//   product          y[i]  = x[rows[i]] W_eᵀ              i in expert e's rows
//   input gradient   dx[i] = dy[i] W_e
//   weight gradient  dW_e  = sum_i dy[i]ᵀ x[rows[i]]
//
// One tiled MFMA kernel runs all three: acc(i, j) = sum_k P(i, k) Q(j, k)
// with each operand read as K-contiguous rows or in its natural layout
// (ns_layout.h), so neither x nor W is ever gathered or transposed in memory:
//   product          P = rows of x, gathered   Q = rows of W_e
//   input gradient   P = rows of dy            Q = columns of W_e (natural)
//   weight gradient  P = columns of dy (natural), Q = columns of x (natural,
//                    gathered): k runs over the expert's rows
// Sums are in fp32 and rounded once.
//
// bf16, 128 experts of 1536 x 2048, rows spread at random: us with 1 GiB read
// between calls (TFLOP/s over the rows that there are), and the same call again
// and again, which finds part of its inputs in the last-level cache but runs at
// a lower clock:
//                           product          input gradient   weight gradient
//   65536 rows              483 (853), 527   440 (938), 473   489 (843), 456
//     rows sorted already   471 (875), 499                    478 (862), 499
//     half of them to one   534 (772), 595   477 (864), 516   781 (528), 670
//   16384 rows              210, 217         192, 197         234, 198
//   32 rows                 29, 27           31, 27           134, 136
//   65536 rows, 16 experts  363 (1137), 363  385 (1070), 395  356 (1159), 353
// A large square library product reaches 1200 TFLOP/s here.  With 4096 rows to
// an expert the matrix cores are busy 55 to 59 % of the time, at the 1.8 to 1.9
// GHz of such loads, and 53 % with 512 rows, where the product's tiles of 256
// rows are padded by 28 % and the input gradient's of 128 rows by 12 % (their
// tiles run at 1090 and 1050 TFLOP/s: the padding is what is lost), and the
// weight gradient's 16 stages do not cover a tile's first loads and its stores.
// More stages in flight, or dead blocks skipped, change that by 2 % at most.
// The weight gradient gives an output tile to one workgroup for all of the
// expert's rows, so an expert that has most of them is a tail of few
// workgroups.  At 16384 rows the weights and the output are 0.9 GB, and HBM
// bounds all three; at 32 rows the chosen experts' weights (179 MB) and the
// weight gradient's 805 MB of output do.
// fp32 runs on the fp32 MFMA, a sixteenth of the rate: 999 rows of 7 experts of
// 520 x 264 take 10, 13 and 11 us; one wave's 32 x 32 block over 520 columns of
// k is 8 us of matrix instructions.
//
// The experts' row counts are known on the device only.  The grid holds the
// most tiles that n_rows rows can make; every workgroup adds up the experts'
// tiles (one prefix sum by each wave) and takes its own, or ends.
#include <algorithm>
#include <type_traits>

#include "ns_device.h"
#include "ns_lanes.h"
#include "ns_sublayer.h"

namespace ns {
namespace {

constexpr unsigned kOutOfRange = 0x80000000u;  // past every descriptor below

struct Tile {
  int expert, tile;  // tile: row tile within the expert
  int begin, count;  // the expert's sorted rows
};

// Row tiles of all experts, and the running count at the end of each lane's
// experts (lane l: experts l per .. l per + per - 1).
__device__ __forceinline__ void expert_rows(const int* offsets, int e, int experts, int n_rows, int* begin, int* count) {
  *begin = *count = 0;
  if ((unsigned)e >= (unsigned)experts) return;
  const int b = min(max(offsets[e], 0), n_rows), c = min(max(offsets[e + 1], 0), n_rows);
  *begin = b;
  *count = c > b ? c - b : 0;
}
__device__ __forceinline__ int count_tiles(const ExpertsArgs& g, int bm, int* upto) {
  const int lane = threadIdx.x & 63, per = (g.experts + 63) / 64;
  int n = 0;
  for (int i = 0; i < per; ++i) {
    int b, c;
    expert_rows(g.offsets, lane * per + i, g.experts, g.n_rows, &b, &c);
    n += (c + bm - 1) / bm;
  }
#pragma unroll
  for (int o = 1; o < 64; o <<= 1) {
    const int u = __shfl_up(n, o, 64);
    if (lane >= o) n += u;
  }
  *upto = n;
  return __builtin_amdgcn_readlane(n, 63);
}
__device__ __forceinline__ Tile find_tile(const ExpertsArgs& g, int bm, int upto, int q) {
  const int per = (g.experts + 63) / 64;
  const int l = __ffsll((unsigned long long)__ballot(upto > q)) - 1;
  int left = q - (l > 0 ? __builtin_amdgcn_readlane(upto, l - 1) : 0);
  Tile t{};
  for (int i = 0; i < per; ++i) {
    int b, c;
    expert_rows(g.offsets, l * per + i, g.experts, g.n_rows, &b, &c);
    const int n = (c + bm - 1) / bm;
    if (left < n) {
      t = Tile{l * per + i, left, b, c};
      break;
    }
    left -= n;
  }
  t.expert = __builtin_amdgcn_readfirstlane(t.expert);
  t.tile = __builtin_amdgcn_readfirstlane(t.tile);
  t.begin = __builtin_amdgcn_readfirstlane(t.begin);
  t.count = __builtin_amdgcn_readfirstlane(t.count);
  return t;
}

typedef float f32x4 __attribute__((ext_vector_type(4)));
__device__ __forceinline__ f32x4 acc_of(const f32x16& v, int rg) {  // 4 columns of a 32 x 32 block's row
  return f32x4{v[4 * rg], v[4 * rg + 1], v[4 * rg + 2], v[4 * rg + 3]};
}
// bf16 pairs of 4 columns, each pair by one conversion
typedef __bf16 bf16x4 __attribute__((ext_vector_type(4)));
__device__ __forceinline__ uint2 pack4(f32x4 v) {
  return __builtin_bit_cast(uint2, __builtin_convertvector(v, bf16x4));
}

// The descriptor, in scalar registers (it is the same in every lane).
__device__ __forceinline__ i32x4 uniform(i32x4 r) {
  i32x4 u = {__builtin_amdgcn_readfirstlane(r[0]), __builtin_amdgcn_readfirstlane(r[1]),
             __builtin_amdgcn_readfirstlane(r[2]), __builtin_amdgcn_readfirstlane(r[3])};
  return u;
}

// GATHER: the weight gradient's x is read through rows.  ONCE: the weights are
// more than the L2s hold and few rows read each (4 tokens 31 us, 38 without; with
// more than one row tile to an expert it loses: 512 tokens 234 and 162).
template <typename T, int BM, int BN, int WM, int WN, int CPR, int ST, int OCC, int MODE, bool GATHER, bool ONCE>
__global__ __launch_bounds__(WM* WN * 64, (OCC * WM * WN + 3) / 4) void experts_kernel(const ExpertsArgs g) {
  constexpr bool PNAT = MODE == EXP_WEIGHT_GRAD, QNAT = MODE != EXP_PRODUCT;
  constexpr int NW = WM * WN;
  constexpr int EPC = Elem<T>::kChunk, ES = (int)sizeof(T), BK = CPR * EPC;
  constexpr int WTM = BM / WM, WTN = BN / WN, SM = WTM / 32, SN = WTN / 32;
  constexpr int LP = BM * CPR, LQ = BN * CPR, STAGE = LP + LQ;
  constexpr int NP = LP / 64 / NW, NQ = LQ / 64 / NW, NIW = NP + NQ;  // a wave's loads of a stage
  constexpr int OCH = WTN / EPC, OPITCH = OCH + 1;  // chunks of a wave's output row, and of its place in the LDS
  constexpr int OUT = NW * 32 * OPITCH;             // 32 such rows for each wave
  constexpr bool WG = MODE == EXP_WEIGHT_GRAD;
  static_assert(WG || !GATHER, "the other modes decide while they run");
  constexpr int RCP = BM / EPC, RCQ = BN / EPC;
  static_assert(WTM % 32 == 0 && WTN % 32 == 0, "wave tile must be whole 32x32 blocks");
  static_assert(LP % (64 * NW) == 0 && LQ % (64 * NW) == 0, "operands must split into whole wave loads");
  static_assert(ST >= 2 && NIW * (ST - 2) < 64, "ring depth");
  __shared__ uint4 lds[ST * STAGE > OUT ? ST * STAGE : OUT];  // the ring, then the output
  __shared__ int row_ring[GATHER ? ST * NW * 64 : 1];  // see read_rows

  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int wm = wave / WN, wn = wave % WN;
  const int M = MODE == EXP_WEIGHT_GRAD ? g.fan_out : 0;  // output rows (else the expert's)
  const int N = MODE == EXP_PRODUCT ? g.fan_out : g.fan_in;
  const int tiles_n = (N + BN - 1) / BN;

  // this workgroup's tile
  Tile tl;
  int i0, j0;
  if (MODE == EXP_WEIGHT_GRAD) {
    // The grid is [experts][tiles].  Workgroups go to the XCDs in turn, so each
    // XCD has an eighth of the tiles of every expert (experts differ in their
    // rows and so in the time of their tiles); with a multiple of 8 tiles it is
    // a run of neighbours, which share their columns of x.
    const int tiles_m = (M + BM - 1) / BM, tiles = gridDim.x, w = blockIdx.x;
    const int q = tiles % 8 == 0 ? w % 8 * (tiles / 8) + w / 8 : w;
    tl.expert = blockIdx.y;
    int tj;
    rect_decode(q, tiles_m, tiles_n, tl.tile, tj);
    i0 = tl.tile * BM;
    j0 = tj * BN;
    expert_rows(g.offsets, tl.expert, g.experts, g.n_rows, &tl.begin, &tl.count);
    tl.begin = __builtin_amdgcn_readfirstlane(tl.begin);
    tl.count = __builtin_amdgcn_readfirstlane(tl.count);
  } else {
    int upto;
    const int total = count_tiles(g, BM, &upto) * tiles_n;
    // each XCD takes a contiguous run of the live tiles (xcd_remap)
    const int xcd = blockIdx.x % 8, local = blockIdx.x / 8, per = total / 8, rem = total % 8;
    if (local >= per + (xcd < rem ? 1 : 0)) return;
    const int lin = xcd * per + min(xcd, rem) + local;
    tl = find_tile(g, BM, upto, lin / tiles_n);
    if (tl.count <= 0) return;  // (only offsets that are no prefix sums lead here)
    i0 = tl.tile * BM;
    j0 = (lin % tiles_n) * BN;
  }
  const int K = MODE == EXP_PRODUCT ? g.fan_in : MODE == EXP_INPUT_GRAD ? g.fan_out : tl.count;
  const int m_end = MODE == EXP_WEIGHT_GRAD ? M : tl.count;

  // Sources of a wave's loads t of a stage: P for t < NP, then Q.
  const T* W = reinterpret_cast<const T*>(g.w) + (size_t)tl.expert * g.fan_out * g.fan_in;
  auto src = [&](int t) __attribute__((always_inline)) {
    return dma_src(t < NP ? wave * NP + t : LP / 64 + wave * NQ + t - NP, lane, BM, BN, CPR, EPC, PNAT, QNAT, ES);
  };
  auto lds_of = [&](int slot, int t) __attribute__((always_inline)) {
    return lds_addr(lds + slot * STAGE + (t < NP ? wave * NP + t : LP / 64 + wave * NQ + t - NP) * 64);
  };

  // Product and input gradient: byte offsets at k0 = 0, kOutOfRange for rows
  // and columns past the end, and one descriptor for each operand.
  unsigned off[WG ? 1 : NIW];
  const unsigned step_q = (unsigned)((QNAT ? BK * g.fan_in : BK) * ES);
  i32x4 rP{}, rQ{};
  if constexpr (!WG) {
    const long long ld = MODE == EXP_PRODUCT ? g.ldx : g.fan_out;
    const bool gather = MODE == EXP_PRODUCT && g.rows != nullptr;
    const size_t rows = gather ? (size_t)g.n_x : (size_t)min(BM, tl.count - i0);
    rP = uniform(make_rsrc(reinterpret_cast<const T*>(MODE == EXP_PRODUCT ? g.x : g.dy) + (gather ? 0 : (tl.begin + i0) * ld),
                           (unsigned)(((rows - 1) * ld + K) * ES)));
    rQ = uniform(make_rsrc(W, (unsigned)((size_t)g.fan_out * g.fan_in * ES)));
#pragma unroll
    for (int t = 0; t < NIW; ++t) {
      const DmaSrc d = src(t);
      if (t < NP) {
        int r = d.row;
        bool ok = i0 + r < tl.count;
        if (gather) {
          r = ok ? g.rows[tl.begin + i0 + r] : 0;
          ok = ok && (unsigned)r < (unsigned)g.n_x;
        } else if (MODE == EXP_PRODUCT) {
          ok = ok && tl.begin + i0 + r < g.n_x;
        }
        off[t] = ok ? (unsigned)(((size_t)r * ld + d.kpos) * ES) : kOutOfRange;
      } else {
        const int j = j0 + d.row;
        off[t] = j >= N ? kOutOfRange
                        : (unsigned)((QNAT ? (size_t)d.kpos * g.fan_in + j : (size_t)j * g.fan_in + d.kpos) * ES);
      }
    }
  }

  // Weight gradient: a load covers 64 / RC k rows of a stage, lane l the one
  // of number l / RC, at a column that repeats with the bits of the k row that
  // nat_swz sees: every NCP (NCQ) loads.  Columns past the end read the last
  // ones: what they add up to is never stored.  k rows past the end must be
  // zero: the descriptor ends there, or the gathered row's offset is out of
  // range.
  constexpr int RPP = 64 / RCP, RPQ = 64 / RCQ, KRQ = NQ * RPQ;
  const unsigned ldp = (unsigned)(g.fan_out * ES), ldq = (unsigned)(g.ldx * ES);
  constexpr int SEENP = ES == 4 ? 8 : RCP % 16 == 0 ? 4 : 16, SEENQ = ES == 4 ? 8 : RCQ % 16 == 0 ? 4 : 16;
  constexpr int NCP = SEENP > RPP ? SEENP / RPP : 1, NCQ = SEENQ > RPQ ? SEENQ / RPQ : 1;
  static_assert(!WG || (NP % NCP == 0 && NQ % NCQ == 0), "a wave's first k row starts a period");
  static_assert(!QNAT || (ES == 4 ? RCQ >= 16 : RCQ >= 8), "nat_swz stays within a row");
  static_assert(!PNAT || (ES == 4 ? RCP >= 16 : RCP >= 8), "nat_swz stays within a row");
  unsigned colp[WG ? NCP : 1], colq[WG ? NCQ : 1];
  if constexpr (WG) {
#pragma unroll
    for (int t = 0; t < NCP; ++t)
      colp[t] = (unsigned)(min(i0 + src(t).row, M - EPC) * ES) + (unsigned)(lane / RCP) * ldp;
#pragma unroll
    for (int t = 0; t < NCQ; ++t)
      colq[t] = (unsigned)(min(j0 + src(NP + t).row, N - EPC) * ES) + (GATHER ? 0u : (unsigned)(lane / RCQ) * ldq);
    if constexpr (GATHER) rQ = uniform(make_rsrc(g.x, (unsigned)(g.n_x - 1) * ldq + (unsigned)(g.fan_in * ES)));
  }
  // x's row numbers: a wave keeps those of its own loads in the LDS, the KRQ of
  // stage kt at row_ring[kt % ST][wave].  They go out ST - 1 stages before the
  // loads that they are for, as one more load of that stage (LD in all), and
  // have landed a stage before those are issued: the wave has waited for its
  // loads of stage kt - (ST - 1) by then.  take_rows reads them to registers
  // ahead of that stage's last products.  (Scalar loads would return out of
  // order with the fragment reads, each of which would wait for all of them.)
  constexpr int LD = NIW + (GATHER ? 1 : 0);
  static_assert(!WG || KRQ <= 64, "one load holds a wave's row numbers");
  const i32x4 rR = GATHER ? uniform(make_rsrc(g.rows + tl.begin, (unsigned)K * 4u)) : i32x4{};
  int row_of[GATHER ? NQ : 1];
  auto read_rows = [&](int kt, int slot) __attribute__((always_inline)) {
    if constexpr (GATHER)
      dma4(lds_addr(reinterpret_cast<const uint4*>(row_ring + (slot * NW + wave) * 64)),
           (unsigned)(kt * BK + wave * KRQ + lane) * 4u, rR);  // past the expert's rows: zeros (not used)
  };
  auto take_rows = [&](int slot) __attribute__((always_inline)) {
    if constexpr (GATHER)
#pragma unroll
      for (int u = 0; u < NQ; ++u) row_of[u] = row_ring[(slot * NW + wave) * 64 + u * RPQ + lane / RCQ];
  };

  typedef std::integral_constant<int, 1> OfP;
  typedef std::integral_constant<int, 2> OfQ;
  typedef std::integral_constant<int, 3> Both;
  // The loads of stage kt into a slot: P's, Q's or both.  whole: the stage has
  // BK elements of k (known while compiling); otherwise that is looked at.
  auto issue = [&](int kt, int slot, auto what, auto whole) __attribute__((always_inline)) {
    constexpr bool DOP = decltype(what)::value & 1, DOQ = decltype(what)::value & 2, WHOLE = decltype(whole)::value;
    const int k0 = kt * BK;
    if constexpr (WG) {
      const unsigned left = WHOLE ? (unsigned)BK : (unsigned)min(BK, K - k0);  // > 0
      const char* dy = reinterpret_cast<const char*>(g.dy) + (size_t)(unsigned)(tl.begin + k0) * ldp;
      const char* x = reinterpret_cast<const char*>(g.x) + (size_t)(unsigned)(tl.begin + k0) * ldq;
      const i32x4 p = uniform(make_rsrc(dy, left * ldp));
      const i32x4 q = GATHER ? rQ : uniform(make_rsrc(x, (left - 1) * ldq + (unsigned)(g.fan_in * ES)));
#pragma unroll
      for (int t = 0; t < NIW; ++t) {
        if (t < NP ? !DOP : !DOQ) continue;
        if (t < NP) {
          dma16(lds_of(slot, t), colp[t % NCP] + (unsigned)(wave * NP + t) * RPP * ldp, p);
          continue;
        }
        const int u = t - NP;
        unsigned o = (unsigned)(wave * NQ + u) * RPQ * ldq;
        if constexpr (GATHER) {
          const int r = row_of[u], kr = wave * KRQ + u * RPQ + lane / RCQ;
          const unsigned at = (unsigned)r * ldq;
          const bool in = (WHOLE | (k0 + kr < K)) & ((unsigned)r < (unsigned)g.n_x);
          o = in ? at : kOutOfRange;
        }
        dma16(lds_of(slot, t), o + colq[u % NCQ], q);
      }
      if (DOQ) read_rows(kt + ST - 1, (slot + ST - 1) % ST);
    } else {
      const bool all = WHOLE || k0 + BK <= K;
#pragma unroll
      for (int t = 0; t < NIW; ++t) {
        if (t < NP ? !DOP : !DOQ) continue;
        // (an offset out of range stays there: kt steps are below 2^31)
        const unsigned o = off[t] + (unsigned)kt * (t < NP ? (unsigned)(BK * ES) : step_q);
        const unsigned at = all || k0 + src(t).kpos < K ? o : kOutOfRange;
        if (t < NP) dma16(lds_of(slot, t), at, rP);
        else if constexpr (ONCE) dma16_once(lds_of(slot, t), at, rQ);
        else dma16(lds_of(slot, t), at, rQ);
      }
    }
  };

  f32x16 acc[SM][SN];
#pragma unroll
  for (int a = 0; a < SM; ++a)
#pragma unroll
    for (int b = 0; b < SN; ++b)
#pragma unroll
      for (int r = 0; r < 16; ++r) acc[a][b][r] = 0.0f;

  // fragment reads: a per-lane base plus a compile-time offset
  constexpr int KS = CPR / 2, NH = sizeof(T) == 2 ? 2 : 4, QOFF = LP * 16;
  constexpr int NSP = nat_step_bytes(RCP, ES), NSQ = nat_step_bytes(RCQ, ES);
  int kcp[PNAT ? 1 : KS], kcq[QNAT ? 1 : KS];
  int natp[PNAT ? SM : 1][NH], natq[QNAT ? SN : 1][NH];
  if constexpr (PNAT) {
#pragma unroll
    for (int a = 0; a < SM; ++a)
#pragma unroll
      for (int h = 0; h < NH; ++h) natp[a][h] = nat_lane_byte(wm * WTM + 32 * a, h, lane, RCP, T());
  } else {
#pragma unroll
    for (int s = 0; s < KS; ++s) kcp[s] = kc_lane_byte(wm * WTM, s, lane, CPR);
  }
  if constexpr (QNAT) {
#pragma unroll
    for (int b = 0; b < SN; ++b)
#pragma unroll
      for (int h = 0; h < NH; ++h) natq[b][h] = nat_lane_byte(wn * WTN + 32 * b, h, lane, RCQ, T()) + QOFF;
  } else {
#pragma unroll
    for (int s = 0; s < KS; ++s) kcq[s] = kc_lane_byte(wn * WTN, s, lane, CPR) + QOFF;
  }
  const char* lb = reinterpret_cast<const char*>(lds);
  auto load_step = [&](int slot, int s, uint4 (&pf)[SM], uint4 (&qf)[SN]) __attribute__((always_inline)) {
    const char* st = lb + slot * STAGE * 16;
#pragma unroll
    for (int a = 0; a < SM; ++a) {
      if constexpr (PNAT) pf[a] = nat_frag(st + s * NSP, natp[a], T());
      else pf[a] = *reinterpret_cast<const uint4*>(st + kcp[s ^ kc_sigma(a, CPR)] + a * 32 * CPR * 16);
    }
#pragma unroll
    for (int b = 0; b < SN; ++b) {
      if constexpr (QNAT) qf[b] = nat_frag(st + s * NSQ, natq[b], T());
      else qf[b] = *reinterpret_cast<const uint4*>(st + kcq[s ^ kc_sigma(b, CPR)] + b * 32 * CPR * 16);
    }
  };
  // Ring of ST stages: stage kt lives in slot kt % ST, and its loads go out
  // ST - 1 stages ahead.  The fragments of step s + 1 are read while the MFMAs
  // of step s run, across the stages' border too: before a stage's last MFMAs
  // a wave waits for its own loads of the next stage, and the barrier there
  // publishes every wave's and certifies that this stage's slot is read out.
  const int nk = (K + BK - 1) / BK;
  uint4 pf[2][SM], qf[2][SN];
  auto wait_stage = [&](int kt, auto steady) __attribute__((always_inline)) {
    const int later = nk - 1 - kt;  // stages that may be in flight after kt, at most ST - 2
    if (decltype(steady)::value || later >= ST - 2) wait_vm_lgkm0<LD * (ST - 2)>();
    else if (ST > 4 && later == 2) wait_vm_lgkm0<LD * 2>();
    else if (ST > 3 && later == 1) wait_vm_lgkm0<LD * 1>();
    else wait_vm_lgkm0<0>();
    ring_barrier();
  };
  static_assert(ST <= 5 && KS % 2 == 0, "tail waits; fragment buffers alternate");
  // steady: more than ST stages follow, so that nothing has to be looked at
  // (branches and waits between the products of a stage are time that the
  // other waves, stopped by the same barrier, cannot fill).
  auto stage = [&](int kt, int u, auto steady) __attribute__((always_inline)) {
    constexpr bool STEADY = decltype(steady)::value;
    if (STEADY || kt + ST - 1 < nk) issue(kt + ST - 1, (u + ST - 1) % ST, Both(), steady);
#pragma unroll
    for (int s = 0; s < KS; ++s) {
      if (s + 1 < KS) {
        load_step(u, s + 1, pf[(s + 1) & 1], qf[(s + 1) & 1]);
      } else if (STEADY || kt + 1 < nk) {
        wait_stage(kt + 1, steady);
        take_rows(u % ST);  // stage kt + ST's
        load_step((u + 1) % ST, 0, pf[0], qf[0]);
      }
      __builtin_amdgcn_sched_barrier(0);  // keeps these reads ahead of the MFMAs
#pragma unroll
      for (int a = 0; a < SM; ++a)
#pragma unroll
        for (int b = 0; b < SN; ++b) mfma_chunk(acc[a][b], qf[s & 1][b], pf[s & 1][a], T());
    }
  };
  if constexpr (GATHER) {
    if (nk > 0) {  // P's first loads do not wait for the row numbers
#pragma unroll
      for (int s = 0; s < ST - 1; ++s) read_rows(s, s);
#pragma unroll
      for (int s = 0; s < ST - 1; ++s)
        if (s < nk) issue(s, s, OfP(), std::false_type());
      if (nk >= ST - 1) wait_vm_lgkm0<NP * (ST - 1)>();
      else wait_vm_lgkm0<0>();
      asm volatile("" ::: "memory");
    }
#pragma unroll
    for (int s = 0; s < ST - 1; ++s)
      if (s < nk) {
        take_rows(s);
        issue(s, s, OfQ(), std::false_type());
      }
    static_assert(ST <= 3, "the first wait");
    if (nk > 1) wait_vm_lgkm0<(NQ + 1) * (ST - 2)>();  // Q's loads of stage 1
    else wait_vm_lgkm0<0>();
  } else {
#pragma unroll
    for (int s = 0; s < ST - 1; ++s)
      if (s < nk) issue(s, s, Both(), std::false_type());
  }
  if (nk > 0) {
    wait_stage(0, std::false_type());
    take_rows(ST - 1);
    load_step(0, 0, pf[0], qf[0]);
  }
  int kt0 = 0;
  for (; kt0 + 2 * ST - 1 < nk; kt0 += ST) {
#pragma unroll
    for (int u = 0; u < ST; ++u) stage(kt0 + u, u, std::true_type());
  }
#pragma unroll
  for (int u = 0; u < 2 * ST - 1; ++u)
    if (kt0 + u < nk) stage(kt0 + u, u % ST, std::false_type());
  wait_vm_lgkm0<0>();  // (row numbers that nothing asked for may still be on their way)
  __syncthreads();

  // 32 rows of a wave's output at a time, through its place in the LDS to whole
  // rows of 16-byte stores.  (bf16: two lanes' four columns make one lane's
  // eight, so the LDS is written 16 bytes at a time too.)
  T* O = reinterpret_cast<T*>(g.out) + (WG ? (size_t)tl.expert * g.fan_out * g.fan_in : (size_t)tl.begin * N);
  uint4* const mine = lds + wave * 32 * OPITCH;
#pragma unroll
  for (int a = 0; a < SM; ++a) {
#pragma unroll
    for (int b = 0; b < SN; ++b) {
      if constexpr (ES == 2) {
#pragma unroll
        for (int rg = 0; rg < 4; rg += 2) {
          const uint2 x = pack4(acc_of(acc[a][b], rg)), y = pack4(acc_of(acc[a][b], rg + 1));
          const auto p = __builtin_amdgcn_permlane32_swap(x.x, y.x, false, false);
          const auto q = __builtin_amdgcn_permlane32_swap(x.y, y.y, false, false);
          mine[acc_i(lane) * OPITCH + b * 4 + rg + (lane >> 5)] = make_uint4(p[0], q[0], p[1], q[1]);
        }
      } else {
#pragma unroll
        for (int rg = 0; rg < 4; ++rg)
          mine[acc_i(lane) * OPITCH + b * 8 + acc_j(rg, lane) / 4] =
              __builtin_bit_cast(uint4, acc_of(acc[a][b], rg));
      }
    }
    __builtin_amdgcn_wave_barrier();
    streaming(g.stream, [&](auto stream) __attribute__((always_inline)) {
#pragma unroll
      for (int c0 = 0; c0 < 32 * OCH; c0 += 64) {
        const int r = (c0 + lane) / OCH, c = (c0 + lane) % OCH;
        const int i = i0 + wm * WTM + a * 32 + r, j = j0 + wn * WTN + c * EPC;
        const uint4 v = mine[r * OPITCH + c];
        if (i < m_end && j < N) store_whole<stream.value>(reinterpret_cast<uint4*>(O + (size_t)i * N + j), v);
      }
    });
    __builtin_amdgcn_wave_barrier();
  }
}

template <typename T, int BM, int BN, int WM, int WN, int CPR, int ST, int OCC, int MODE>
hipError_t launch_tiles(ExpertsArgs g, hipStream_t st) {
  const int N = MODE == EXP_PRODUCT ? g.fan_out : g.fan_in;
  const long long tiles_n = (N + BN - 1) / BN;
  long long grid, experts = 1;
  if (MODE == EXP_WEIGHT_GRAD) {
    grid = (g.fan_out + BM - 1) / BM * tiles_n;
    experts = g.experts;
  } else {
    // sum of ceil(c / BM) over at most min(experts, n_rows) non-empty experts
    const long long some = g.experts < g.n_rows ? g.experts : g.n_rows;
    grid = ((g.n_rows + some * (BM - 1)) / BM) * tiles_n;
    grid = (grid + 7) / 8 * 8;  // every XCD reaches its last live tile
  }
  if (grid <= 0) return hipSuccess;
  if (grid > 0x7fffffffll) return hipErrorInvalidValue;
  const dim3 blocks((unsigned)grid, (unsigned)experts), threads(WM * WN * 64);
  constexpr bool WG = MODE == EXP_WEIGHT_GRAD, FEW = !WG && BM == 32;
  const long long weights = (long long)g.experts * g.fan_out * g.fan_in * (long long)sizeof(T);
  g.stream = beyond_l2(WG ? weights : (long long)g.n_rows * N * (long long)sizeof(T));
#define NS_EXPERTS(GATHER, ONCE) \
  dispatch(experts_kernel<T, BM, BN, WM, WN, CPR, ST, OCC, MODE, GATHER, ONCE>, blocks, threads, st, g)
  if (WG && g.rows != nullptr) NS_EXPERTS(WG, false);
  else if (FEW && beyond_l2(weights)) NS_EXPERTS(false, FEW);
  else NS_EXPERTS(false, false);
#undef NS_EXPERTS
  return hipGetLastError();
}

// Tiles of a launch: BM, BN, waves, 16-byte chunks of k, stages, workgroups
// per CU.  A large tile reads less for each product; a small one pads less and
// makes more workgroups.  The rules go by rows and tiles; they were found with
// experts of 1536 x 2048, and no other shape is measured.  us, bf16 if not said:
//   256 x 256 against 128 x 256
//     product          500 rows to each of 8 experts 49 / 37 (138 tiles at
//                      most), 750 rows 51 / 64 (186), 1000 rows 55 / 67;
//                      128 experts: 128 rows 263 / 238, 256 rows 344 / 347,
//                      512 rows 495 / 541; 64 experts, 250 rows 178 / 164
//     weight gradient  (both with plain stores) 4096 rows to each of 16
//                      experts 370 / 415, 512 of 128 533 / 538, 500 of 32 137 /
//                      132, 128 of 128 268 / 262; 1000 rows of 8 78 / 65 (384
//                      tiles)
//     input gradient   128 experts: 256 rows 315 / 296, 512 rows 502 / 487; 1000
//                      rows of 8 experts 76 / 64: never 256 x 256
//   128 x 256 against 64 x 64   400 rows of 8 experts 37 / 18, 2000 rows 42 / 52
//   32 x 64   product: one row 14, against 35 with 128 x 256; 16 rows to each
//             of 128 experts 147 / 157.  Input gradient: one row 12 / 29, 16 rows
//             each 150 / 136.  fp32, 16 rows each: 394, with 64 x 64 434, with
//             128 x 128 790; 2000 rows of 8 experts: 64 x 64 1085, 128 x 128 1321
#define NS_EXPERTS_WIDE 256, 256, 2, 4, 8, 2, 1
#define NS_EXPERTS_WIDE_GRAD 256, 256, 2, 4, 4, 3, 1
#define NS_EXPERTS_LONG 128, 256, 2, 4, 4, 3, 2
#define NS_EXPERTS_SMALL 64, 64, 2, 2, 8, 3, 3
#define NS_EXPERTS_FEW 32, 64, 1, 2, 8, 4, 3
enum ExpertsTile { TILE_WIDE, TILE_LONG, TILE_SMALL, TILE_FEW };

// The most tiles of bm x bn that a launch can have.
long long most_tiles(ExpertsMode mode, const ExpertsArgs& g, int bm, int bn) {
  if (mode == EXP_WEIGHT_GRAD)
    return (long long)g.experts * ((g.fan_out + bm - 1) / bm) * ((g.fan_in + bn - 1) / bn);
  const int n = mode == EXP_PRODUCT ? g.fan_out : g.fan_in;
  return ((long long)g.n_rows / bm + std::min(g.experts, g.n_rows)) * ((n + bn - 1) / bn);
}

ExpertsTile choose_tile(int dtype, ExpertsMode mode, const ExpertsArgs& g) {
  const int rows = g.n_rows / g.experts;  // an expert's, on average
  const bool few = mode != EXP_WEIGHT_GRAD && rows <= 16;
  if (dtype != 1) return few ? TILE_FEW : TILE_SMALL;
  if (mode == EXP_PRODUCT && rows >= 256 && most_tiles(mode, g, 256, 256) >= 160) return TILE_WIDE;
  if (mode == EXP_WEIGHT_GRAD && rows >= 1024 && most_tiles(mode, g, 256, 256) >= 768) return TILE_WIDE;
  if (mode == EXP_PRODUCT && few) return TILE_FEW;
  if (most_tiles(mode, g, 128, 256) >= 192) return TILE_LONG;
  return few ? TILE_FEW : TILE_SMALL;
}

template <typename T, ExpertsMode MODE>
hipError_t launch_type(const ExpertsArgs& g, hipStream_t st) {
  constexpr bool BF16 = std::is_same<T, bf16>::value;
  switch (choose_tile(BF16 ? 1 : 0, MODE, g)) {
    case TILE_WIDE:
      if constexpr (BF16 && MODE == EXP_PRODUCT) return launch_tiles<T, NS_EXPERTS_WIDE, MODE>(g, st);
      if constexpr (BF16 && MODE == EXP_WEIGHT_GRAD) return launch_tiles<T, NS_EXPERTS_WIDE_GRAD, MODE>(g, st);
      break;
    case TILE_LONG:
      if constexpr (BF16) return launch_tiles<T, NS_EXPERTS_LONG, MODE>(g, st);
      break;
    case TILE_FEW:
      if constexpr (MODE != EXP_WEIGHT_GRAD) return launch_tiles<T, NS_EXPERTS_FEW, MODE>(g, st);
      break;
    case TILE_SMALL: return launch_tiles<T, NS_EXPERTS_SMALL, MODE>(g, st);
  }
  return hipErrorInvalidValue;
}

template <ExpertsMode MODE>
hipError_t launch_mode(int dtype, const ExpertsArgs& g, hipStream_t st) {
  return dtype == 1 ? launch_type<bf16, MODE>(g, st) : launch_type<float, MODE>(g, st);
}

// ---------------------------------------------------------------- combine

// out[t] = sum_j weights[t, j] y[slots[t, j]], in fp32, rounded once: TPT
// threads to a token, each walking its columns 8 at a time; eight rows are on
// their way before the first is added.  Bound by HBM: 8192 tokens x 8 rows of
// 2048 bf16 take 57 us (5.3 TB/s; rows of 4 KB at random), 47 with part of y
// still in the last-level cache; 32 tokens 3.0 us.
constexpr int kCombineAhead = 8;
template <typename T, int TPT>
__global__ __launch_bounds__(256) void combine_kernel(const CombineArgs g) {
  const int vpr = g.cols / 8;
  const Raw8<T>* y = reinterpret_cast<const Raw8<T>*>(g.y);
  for (long long t = (long long)blockIdx.x * (256 / TPT) + threadIdx.x / TPT; t < g.tokens;
       t += (long long)gridDim.x * (256 / TPT)) {
    for (int v = blockIdx.y * TPT + threadIdx.x % TPT; v < vpr; v += gridDim.y * TPT) {
      float s[8] = {0, 0, 0, 0, 0, 0, 0, 0};
      for (int j0 = 0; j0 < g.top_k; j0 += kCombineAhead) {
        Raw8<T> r[kCombineAhead];
        float w[kCombineAhead];
        int slot[kCombineAhead];
#pragma unroll
        for (int u = 0; u < kCombineAhead; ++u) {
          const int j = min(j0 + u, g.top_k - 1);
          slot[u] = g.slots[t * g.top_k + j];
          w[u] = g.weights ? g.weights[t * g.top_k + j] : 1.0f;
          if (j0 + u >= g.top_k || (unsigned)slot[u] >= (unsigned)g.n_rows) slot[u] = -1;
        }
#pragma unroll
        for (int u = 0; u < kCombineAhead; ++u) {
          r[u] = Raw8<T>{};
          if (slot[u] >= 0) r[u] = y[(size_t)slot[u] * vpr + v];
          else w[u] = 0.0f;
        }
#pragma unroll
        for (int u = 0; u < kCombineAhead; ++u) {
          float f[8];
          unpack8(r[u], f);
#pragma unroll
          for (int e = 0; e < 8; ++e) s[e] = fmaf(w[u], f[e], s[e]);
        }
      }
      streaming(g.stream, [&](auto stream) __attribute__((always_inline)) {
        store_whole<stream.value>(reinterpret_cast<Raw8<T>*>(g.out) + (size_t)t * vpr + v, pack8(s, T()));
      });
    }
  }
}

// dy[slot] = weight dout[t],  dweights[t, j] = <dout[t], y[slot]> (fp32): a wave
// to a token, eight choices at a time, so that dout is read once for them.
// Bound by HBM: 111 to 129 us for the same (4.4 to 5.1 TB/s).  32 tokens take 8
// us (fp32 12): a wave walks its token's columns in turn, and there are no more
// waves.
template <typename T>
__global__ __launch_bounds__(256) void combine_backward_kernel(const CombineGradArgs g) {
  const int lane = threadIdx.x & 63, vpr = g.cols / 8;
  const Raw8<T>* y = reinterpret_cast<const Raw8<T>*>(g.y);
  Raw8<T>* dy = reinterpret_cast<Raw8<T>*>(g.dy);
  for (long long t = (long long)blockIdx.x * 4 + (threadIdx.x >> 6); t < g.tokens; t += (long long)gridDim.x * 4) {
    const Raw8<T>* dout = reinterpret_cast<const Raw8<T>*>(g.dout) + (size_t)t * vpr;
    for (int j0 = 0; j0 < g.top_k; j0 += kCombineAhead) {
      int slot[kCombineAhead];
      float w[kCombineAhead], dot[kCombineAhead];
#pragma unroll
      for (int u = 0; u < kCombineAhead; ++u) {
        const bool on = j0 + u < g.top_k;
        slot[u] = on ? g.slots[t * g.top_k + j0 + u] : -1;
        if ((unsigned)slot[u] >= (unsigned)g.n_rows) slot[u] = -1;
        w[u] = on && g.weights ? g.weights[t * g.top_k + j0 + u] : 1.0f;
        dot[u] = 0.0f;
      }
      for (int v = lane; v < vpr; v += 64) {
        float d[8];
        unpack8(dout[v], d);
        Raw8<T> r[kCombineAhead];
        if (g.dweights) {
#pragma unroll
          for (int u = 0; u < kCombineAhead; ++u) {
            r[u] = Raw8<T>{};
            if (slot[u] >= 0) r[u] = y[(size_t)slot[u] * vpr + v];
          }
        }
        if (dy) {
          streaming(g.stream, [&](auto stream) __attribute__((always_inline)) {
#pragma unroll
            for (int u = 0; u < kCombineAhead; ++u) {
              if (slot[u] < 0) continue;
              float f[8];
#pragma unroll
              for (int e = 0; e < 8; ++e) f[e] = w[u] * d[e];
              store_whole<stream.value>(dy + (size_t)slot[u] * vpr + v, pack8(f, T()));
            }
          });
        }
        if (g.dweights) {
#pragma unroll
          for (int u = 0; u < kCombineAhead; ++u) {
            float f[8];
            unpack8(r[u], f);
#pragma unroll
            for (int e = 0; e < 8; ++e) dot[u] = fmaf(f[e], d[e], dot[u]);
          }
        }
      }
      if (g.dweights) {
#pragma unroll
        for (int u = 0; u < kCombineAhead; ++u) {
          const float s = lanes_sum<64>(dot[u]);
          if (lane == 0 && j0 + u < g.top_k) g.dweights[t * g.top_k + j0 + u] = slot[u] >= 0 ? s : 0.0f;
        }
      }
    }
  }
}

}  // namespace

hipError_t launch_experts(int dtype, ExpertsMode mode, const ExpertsArgs& g, hipStream_t st) {
  switch (mode) {
    case EXP_PRODUCT: return launch_mode<EXP_PRODUCT>(dtype, g, st);
    case EXP_INPUT_GRAD: return launch_mode<EXP_INPUT_GRAD>(dtype, g, st);
    default: return launch_mode<EXP_WEIGHT_GRAD>(dtype, g, st);
  }
}

const char* experts_config(int dtype, ExpertsMode mode, const ExpertsArgs& g) {
#define NS_TEXT(NAME, TILE) NAME ": dtype=%s rows=%lld experts=%lld fan_out=%lld fan_in=%lld | tile=" TILE
#define NS_TILES(NAME)                                  \
  tile == TILE_WIDE    ? NS_TEXT(NAME, "256x256")       \
  : tile == TILE_SMALL ? NS_TEXT(NAME, "64x64")         \
  : tile == TILE_FEW   ? NS_TEXT(NAME, "32x64")         \
                       : NS_TEXT(NAME, "128x256")
  const ExpertsTile tile = choose_tile(dtype, mode, g);
  return mode == EXP_PRODUCT      ? (NS_TILES("experts product"))
         : mode == EXP_INPUT_GRAD ? (NS_TILES("experts input gradient"))
                                  : (NS_TILES("experts weight gradient"));
#undef NS_TILES
#undef NS_TEXT
}

// Blocks of so many tokens each: a launch holds fewer than 2^32 threads, more tokens than that go round.
static unsigned combine_blocks(long long tokens, int per_block) {
  return (unsigned)std::min(1ll << 20, (tokens + per_block - 1) / per_block);
}
template <int TPT>
static void launch_combine_of(int dtype, const CombineArgs& g, int pieces, hipStream_t st) {
  const dim3 grid(combine_blocks(g.tokens, 256 / TPT), (unsigned)pieces);
  if (dtype == 1) dispatch(combine_kernel<bf16, TPT>, grid, dim3(256), st, g);
  else dispatch(combine_kernel<float, TPT>, grid, dim3(256), st, g);
}
// As many threads to a token as its columns keep busy, at most a block: 4096
// tokens of 128 columns 3.2 us with 16, 4.3 with 64, 4.5 with 256; of 512
// columns 6.1 with 64, 6.4 with 256; 8192 of 2048 columns 45 with 256, 49 with
// 64; 4 tokens of 2048 columns 2.9 and 6.2.
hipError_t launch_combine(int dtype, const CombineArgs& args, hipStream_t st) {
  CombineArgs g = args;
  g.stream = beyond_l2((long long)g.tokens * g.cols * (dtype == 1 ? 2 : 4));
  const int vpr = g.cols / 8;
  if (vpr > 64) launch_combine_of<256>(dtype, g, (vpr + 255) / 256, st);
  else if (vpr > 16) launch_combine_of<64>(dtype, g, 1, st);
  else launch_combine_of<16>(dtype, g, 1, st);
  return hipGetLastError();
}

hipError_t launch_combine_backward(int dtype, const CombineGradArgs& args, hipStream_t st) {
  CombineGradArgs g = args;
  g.stream = beyond_l2((long long)g.n_rows * g.cols * (dtype == 1 ? 2 : 4));
  const dim3 grid(combine_blocks(g.tokens, 4));
  if (dtype == 1) dispatch(combine_backward_kernel<bf16>, grid, dim3(256), st, g);
  else dispatch(combine_backward_kernel<float>, grid, dim3(256), st, g);
  return hipGetLastError();
}

}  // namespace ns
