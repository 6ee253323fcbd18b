// ns_device.h - device helpers and the launch helper that every kernel file
// shares: element types, MFMA steps, LDS-direct loads and their waits,
// transposed fragment reads.
#pragma once

#include <type_traits>

#include <hip/hip_ext.h>
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "ns_layout.h"

namespace ns {

typedef __bf16 bf16;
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef float f32x16 __attribute__((ext_vector_type(16)));

template <typename T> struct Elem;
template <> struct Elem<bf16> { static constexpr int kChunk = 8; };
template <> struct Elem<float> { static constexpr int kChunk = 4; };

__device__ __forceinline__ uint4 zero4() { return make_uint4(0u, 0u, 0u, 0u); }

__device__ __forceinline__ uint4 ldg16(const void* p) { return *reinterpret_cast<const uint4*>(p); }

__device__ __forceinline__ uint32_t u4get(const uint4& v, int i) {
  return i == 0 ? v.x : i == 1 ? v.y : i == 2 ? v.z : v.w;
}

__device__ __forceinline__ float bf16_lo(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float bf16_hi(uint32_t w) { return __uint_as_float(w & 0xffff0000u); }
__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
  return (uint32_t)__builtin_bit_cast(uint16_t, (bf16)lo) |
         ((uint32_t)__builtin_bit_cast(uint16_t, (bf16)hi) << 16);
}

// 4 consecutive elements of type T <-> 4 floats
template <typename T> struct Quad;
template <> struct Quad<bf16> {
  typedef uint2 Raw;  // 8 bytes
  __device__ __forceinline__ static void unpack(Raw r, float* f) {
    f[0] = bf16_lo(r.x); f[1] = bf16_hi(r.x); f[2] = bf16_lo(r.y); f[3] = bf16_hi(r.y);
  }
  __device__ __forceinline__ static Raw pack(const float* f) {
    return make_uint2(pack_bf16(f[0], f[1]), pack_bf16(f[2], f[3]));
  }
};
template <> struct Quad<float> {
  typedef uint4 Raw;  // 16 bytes
  __device__ __forceinline__ static void unpack(Raw r, float* f) {
    f[0] = __uint_as_float(r.x); f[1] = __uint_as_float(r.y);
    f[2] = __uint_as_float(r.z); f[3] = __uint_as_float(r.w);
  }
  __device__ __forceinline__ static Raw pack(const float* f) {
    return make_uint4(__float_as_uint(f[0]), __float_as_uint(f[1]), __float_as_uint(f[2]), __float_as_uint(f[3]));
  }
};

// 8 consecutive elements as they are stored
template <typename T> struct Raw8;
template <> struct Raw8<bf16> { uint4 a; };
template <> struct Raw8<float> { uint4 a, b; };

__device__ __forceinline__ void unpack8(const Raw8<bf16>& r, float* f) {
  f[0] = bf16_lo(r.a.x); f[1] = bf16_hi(r.a.x); f[2] = bf16_lo(r.a.y); f[3] = bf16_hi(r.a.y);
  f[4] = bf16_lo(r.a.z); f[5] = bf16_hi(r.a.z); f[6] = bf16_lo(r.a.w); f[7] = bf16_hi(r.a.w);
}
__device__ __forceinline__ void unpack8(const Raw8<float>& r, float* f) {
  f[0] = __uint_as_float(r.a.x); f[1] = __uint_as_float(r.a.y);
  f[2] = __uint_as_float(r.a.z); f[3] = __uint_as_float(r.a.w);
  f[4] = __uint_as_float(r.b.x); f[5] = __uint_as_float(r.b.y);
  f[6] = __uint_as_float(r.b.z); f[7] = __uint_as_float(r.b.w);
}
__device__ __forceinline__ Raw8<bf16> pack8(const float* f, bf16) {
  return Raw8<bf16>{make_uint4(pack_bf16(f[0], f[1]), pack_bf16(f[2], f[3]), pack_bf16(f[4], f[5]),
                               pack_bf16(f[6], f[7]))};
}
__device__ __forceinline__ Raw8<float> pack8(const float* f, float) {
  return Raw8<float>{make_uint4(__float_as_uint(f[0]), __float_as_uint(f[1]), __float_as_uint(f[2]),
                                __float_as_uint(f[3])),
                     make_uint4(__float_as_uint(f[4]), __float_as_uint(f[5]), __float_as_uint(f[6]),
                                __float_as_uint(f[7]))};
}

// 16-byte chunks of operand values -> one MFMA step of a 32x32 block.
// bf16: the chunk is the 8-element k slice of v_mfma_f32_32x32x16_bf16.
// fp32: the chunk is 4 k values, one per v_mfma_f32_32x32x2_f32; both
// operands use the same k assignment, so the sum is the same product.
__device__ __forceinline__ void mfma_chunk(f32x16& acc, uint4 a, uint4 b, bf16) {
  acc = __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(bf16x8, a),
                                                __builtin_bit_cast(bf16x8, b), acc, 0, 0, 0);
}
__device__ __forceinline__ void mfma_chunk(f32x16& acc, uint4 a, uint4 b, float) {
  acc = __builtin_amdgcn_mfma_f32_32x32x2f32(__uint_as_float(a.x), __uint_as_float(b.x), acc, 0, 0, 0);
  acc = __builtin_amdgcn_mfma_f32_32x32x2f32(__uint_as_float(a.y), __uint_as_float(b.y), acc, 0, 0, 0);
  acc = __builtin_amdgcn_mfma_f32_32x32x2f32(__uint_as_float(a.z), __uint_as_float(b.z), acc, 0, 0, 0);
  acc = __builtin_amdgcn_mfma_f32_32x32x2f32(__uint_as_float(a.w), __uint_as_float(b.w), acc, 0, 0, 0);
}

// ------------------------------------------------------------- MFMA kernel

__device__ __forceinline__ float wave_sum(float v) {
#pragma unroll
  for (int o = 32; o >= 1; o >>= 1) v += __shfl_xor(v, o, 64);
  return v;
}

typedef int i32x4 __attribute__((ext_vector_type(4)));

// Buffer descriptor (gfx9 V#) over `bytes` bytes at `base`, stride 0: a load
// at an offset >= bytes returns zeros.
__device__ __forceinline__ i32x4 make_rsrc(const void* base, unsigned bytes) {
  const unsigned long long a = reinterpret_cast<unsigned long long>(base);
  i32x4 r = {(int)(a & 0xffffffffu), (int)((a >> 32) & 0xffffu), (int)bytes, 0x00020000};
  return r;
}

// 16 bytes per lane from buffer offset voff into LDS at m0 + 16 * lane
// (buffer_load_dwordx4 ... lds).  Issued through asm so that the compiler,
// which cannot tell ring slots apart, does not wait for these loads before
// every LDS read; the kernel waits for them explicitly (wait_vm_lgkm0).
__device__ __forceinline__ void dma16(unsigned lds_byte_addr, unsigned voff, i32x4 rsrc) {
  asm volatile("s_mov_b32 m0, %0\n\tbuffer_load_dwordx4 %1, %2, 0 offen lds"
               :
               : "s"(lds_byte_addr), "v"(voff), "s"(rsrc)
               : "memory", "m0");
}

// The same for data that no other workgroup reads: its lines make room in the
// L2 first.
__device__ __forceinline__ void dma16_once(unsigned lds_byte_addr, unsigned voff, i32x4 rsrc) {
  asm volatile("s_mov_b32 m0, %0\n\tbuffer_load_dwordx4 %1, %2, 0 offen nt lds"
               :
               : "s"(lds_byte_addr), "v"(voff), "s"(rsrc)
               : "memory", "m0");
}

// The same, 4 bytes per lane at m0 + 4 * lane.
__device__ __forceinline__ void dma4(unsigned lds_byte_addr, unsigned voff, i32x4 rsrc) {
  asm volatile("s_mov_b32 m0, %0\n\tbuffer_load_dword %1, %2, 0 offen lds"
               :
               : "s"(lds_byte_addr), "v"(voff), "s"(rsrc)
               : "memory", "m0");
}

// *p = v, in pieces of 16 bytes.  STREAM: as part of an output that the L2 could
// not keep anyway; its lines then leave at once, in place of what other
// workgroups still read there.
typedef unsigned u32x4 __attribute__((ext_vector_type(4)));
template <bool STREAM, typename V> __device__ __forceinline__ void store_whole(V* p, const V& v) {
  constexpr int N = sizeof(V) / 16;
  static_assert(sizeof(V) % 16 == 0, "whole 16-byte pieces");
  u32x4 w[N];
  __builtin_memcpy(w, &v, sizeof(V));
  u32x4* to = reinterpret_cast<u32x4*>(p);
#pragma unroll
  for (int i = 0; i < N; ++i) {
    if constexpr (STREAM) __builtin_nontemporal_store(w[i], to + i);
    else to[i] = w[i];
  }
}
// f(whether to stream) for a condition that is the same in every lane.  (Without
// the empty statements the compiler would make one plain store of both kinds.)
template <typename F> __device__ __forceinline__ void streaming(bool stream, F f) {
  if (stream) {
    asm volatile("");
    f(std::true_type());
    asm volatile("");
  } else {
    f(std::false_type());
  }
}

__device__ __forceinline__ unsigned lds_addr(const uint4* p) {
  return (unsigned)reinterpret_cast<unsigned long long>((__attribute__((address_space(3))) const uint4*)p);
}

// s_waitcnt with vmcnt(N), lgkmcnt(0), expcnt unchanged (gfx9 encoding:
// vmcnt[3:0] bits 3:0, expcnt bits 6:4, lgkmcnt bits 11:8, vmcnt[5:4] bits 15:14).
template <int N> __device__ __forceinline__ void wait_vm_lgkm0() {
  static_assert(N >= 0 && N < 64, "vmcnt range");
  __builtin_amdgcn_s_waitcnt((N & 15) | ((N >> 4) << 14) | (7 << 4));
}

// Workgroup barrier that also keeps the compiler from moving memory accesses
// across it; the caller's explicit waits make the LDS data visible.
__device__ __forceinline__ void ring_barrier() {
  asm volatile("" ::: "memory");
  __builtin_amdgcn_s_barrier();
  asm volatile("" ::: "memory");
}

typedef short v4i16 __attribute__((ext_vector_type(4)));

// One MFMA operand fragment (8 bf16 or 4 fp32 k values of one tile row, the
// same k assignment as a K-contiguous chunk) from a NAT tile in LDS: `step`
// addresses the step's k rows, off[] holds the lane's byte offsets of its
// reads (nat_lane_byte_bf16 / _f32).
__device__ __forceinline__ uint4 nat_frag(const char* step, const int* off, bf16) {
  uint32_t w[4];
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const short* src = reinterpret_cast<const short*>(step + off[h]);
    const v4i16 v = __builtin_amdgcn_ds_read_tr16_b64_v4i16((__attribute__((address_space(3))) v4i16*)src);
    w[2 * h] = (uint32_t)(uint16_t)v[0] | ((uint32_t)(uint16_t)v[1] << 16);
    w[2 * h + 1] = (uint32_t)(uint16_t)v[2] | ((uint32_t)(uint16_t)v[3] << 16);
  }
  return make_uint4(w[0], w[1], w[2], w[3]);
}
__device__ __forceinline__ uint4 nat_frag(const char* step, const int* off, float) {
  uint32_t w[4];
#pragma unroll
  for (int e = 0; e < 4; ++e) w[e] = *reinterpret_cast<const uint32_t*>(step + off[e]);
  return make_uint4(w[0], w[1], w[2], w[3]);
}
__device__ __forceinline__ int nat_lane_byte(int rb, int h, int lane, int rc, bf16) {
  return nat_lane_byte_bf16(rb, h, lane, rc);
}
__device__ __forceinline__ int nat_lane_byte(int rb, int h, int lane, int rc, float) {
  return nat_lane_byte_f32(rb, h, lane, rc);
}

// Timing events of the launches this thread makes next (set_launch_events).
// They ride in the dispatch itself (hipExtLaunchKernelGGL): the start event
// takes the first dispatch's start, the stop event every dispatch's end (the
// last one stands), and no marker packet goes between the kernels.
extern thread_local hipEvent_t t_ev_start, t_ev_stop;

template <typename K, typename... A>
static void dispatch_lds(K kernel, dim3 grid, dim3 block, size_t lds, hipStream_t st, A... args) {
  if (t_ev_start == nullptr && t_ev_stop == nullptr) {
    hipLaunchKernelGGL(kernel, grid, block, lds, st, args...);
    return;
  }
  hipExtLaunchKernelGGL(kernel, grid, block, lds, st, t_ev_start, t_ev_stop, 0, args...);
  t_ev_start = nullptr;  // a later launch of the same kind moves only the stop
}
template <typename K, typename... A>
static void dispatch(K kernel, dim3 grid, dim3 block, hipStream_t st, A... args) {
  dispatch_lds(kernel, grid, block, 0, st, args...);
}

}  // namespace ns
