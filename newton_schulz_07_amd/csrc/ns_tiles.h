// ns_tiles.h - what the kernels of the experts' products share: a workgroup's
// tile among those of all experts, whose row counts are known on the device
// only, and a tile's way from the accumulators to memory.
#pragma once

#include "ns_device.h"
#include "ns_sublayer.h"

namespace ns {

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
// Offsets that ascend make at most g.most_row_tiles, which the launch has a grid for:
// times the column tiles that is below 2^31.  Where experts claim the same rows again
// and again the sum itself stops at 2^30, so that it never turns negative.
constexpr int kMostTiles = (1 << 30) - 1;
template <typename G> __device__ __forceinline__ int count_tiles(const G& g, int bm, int* upto) {
  const int lane = threadIdx.x & 63, per = (g.experts + 63) / 64;
  int n = 0;
  for (int i = 0; i < per; ++i) {
    int b, c;
    expert_rows(g.offsets, lane * per + i, g.experts, g.n_rows, &b, &c);
    n = min(n + (c + bm - 1) / bm, kMostTiles);
  }
#pragma unroll
  for (int o = 1; o < 64; o <<= 1) {
    const int u = __shfl_up(n, o, 64);
    if (lane >= o) n = min(n + u, kMostTiles);
  }
  *upto = n;
  return min(__builtin_amdgcn_readlane(n, 63), g.most_row_tiles);
}
template <typename G> __device__ __forceinline__ Tile find_tile(const G& g, int bm, int upto, int q) {
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


// 32 rows of a wave's output (SN blocks beside each other, from row i0 and column
// j0 of O [m_end, N] on), through the wave's own 32 x OPITCH chunks of LDS to whole
// rows of 16-byte stores.  (bf16: two lanes' four columns make one lane's eight,
// so the LDS is written 16 bytes at a time too.)
template <typename T, int SN>
__device__ __forceinline__ void store_32_rows(const f32x16 (&acc)[SN], uint4* mine, T* O, int i0, int j0, int m_end, int N,
                                              bool stream_out) {
  constexpr int EPC = Elem<T>::kChunk, OCH = 32 * SN / EPC, OPITCH = OCH + 1;
  const int lane = threadIdx.x & 63;
#pragma unroll
  for (int b = 0; b < SN; ++b) {
    if constexpr (sizeof(T) == 2) {
#pragma unroll
      for (int rg = 0; rg < 4; rg += 2) {
        const uint2 x = pack4(acc_of(acc[b], rg)), y = pack4(acc_of(acc[b], rg + 1));
        const auto p = __builtin_amdgcn_permlane32_swap(x.x, y.x, false, false);
        const auto q = __builtin_amdgcn_permlane32_swap(x.y, y.y, false, false);
        mine[acc_i(lane) * OPITCH + b * 4 + rg + (lane >> 5)] = make_uint4(p[0], q[0], p[1], q[1]);
      }
    } else {
#pragma unroll
      for (int rg = 0; rg < 4; ++rg)
        mine[acc_i(lane) * OPITCH + b * 8 + acc_j(rg, lane) / 4] = __builtin_bit_cast(uint4, acc_of(acc[b], rg));
    }
  }
  __builtin_amdgcn_wave_barrier();
  streaming(stream_out, [&](auto stream) __attribute__((always_inline)) {
#pragma unroll
    for (int c0 = 0; c0 < 32 * OCH; c0 += 64) {
      const int r = (c0 + lane) / OCH, c = (c0 + lane) % OCH;
      const int i = i0 + r, j = j0 + c * EPC;
      const uint4 v = mine[r * OPITCH + c];
      if (i < m_end && j < N) store_whole<stream.value>(reinterpret_cast<uint4*>(O + (size_t)i * N + j), v);
    }
  });
  __builtin_amdgcn_wave_barrier();
}

}  // namespace ns
