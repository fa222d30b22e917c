// What attention's kernels share: keys from memory straight into LDS, where they lie there, and how a wave's
// fragments of them are read.  C: a configuration with D, kChunks and kRowBytes.
#pragma once

#include "dfs_device.h"
#include "mfma_big.h"

namespace dfs {

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef short s16x4 __attribute__((ext_vector_type(4)));
typedef float f32x2 __attribute__((ext_vector_type(2)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef float f32x16 __attribute__((ext_vector_type(16)));

constexpr float kLag = 8.0f;  // a maximum may lag this far (in powers of two) before sums are rescaled

// 16 bytes per lane from memory straight into LDS at lds_base + 16 lane; kOnce: nobody else
// reads them (64 sequences x 17 nodes, 8192 keys: 203 us against 221 without the hint).
template <bool kOnce>
__device__ __forceinline__ void dma16(const void* p, uint32_t lds_base) {
  if constexpr (kOnce)
    asm volatile("s_mov_b32 m0, %1\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %0, off nt"
                 :
                 : "v"(p), "s"(lds_base)
                 : "memory", "m0");
  else
    asm volatile("s_mov_b32 m0, %1\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %0, off"
                 :
                 : "v"(p), "s"(lds_base)
                 : "memory", "m0");
}

// The same from a scalar address and 32 bits a lane.  The compiler may move reads of LDS across it: barriers keep those
// of the stage that it overwrites apart.
__device__ __forceinline__ void dma16s(const void* p, uint32_t off, uint32_t lds_base) {
  asm volatile("s_mov_b32 m0, %2\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %0, %1"
               :
               : "v"(off), "s"(p), "s"(lds_base)
               : "m0");
}

// 4 bytes per lane, at lds_base + 4 lane.
__device__ __forceinline__ void dma4(const void* p, uint32_t lds_base) {
  asm volatile("s_mov_b32 m0, %1\n\ts_nop 0\n\tglobal_load_lds_dword %0, off" : : "v"(p), "s"(lds_base) : "memory", "m0");
}

__device__ __forceinline__ uint32_t lds_addr(const void* p) {
  return (uint32_t)reinterpret_cast<uintptr_t>((big::lds_ptr_t)p);
}

// Where chunk c of key `row` lies: K so that 16 rows' equal chunks, V so that four rows'
// equal 64-byte blocks fall on distinct banks.
template <class C>
__device__ __forceinline__ int k_slot(int c, int row) {
  return C::kChunks == 16 ? c ^ (row & 15) : c ^ ((row >> 1) & 7);
}
template <class C>
__device__ __forceinline__ int v_slot(int c, int row) {
  return C::kChunks == 16 ? c ^ ((row & 3) << 2) : c ^ (((row >> 1) & 1) << 2);
}

__device__ __forceinline__ float xor32(float x, int lane) {
  return __uint_as_float(xor_lanes(__float_as_uint(x), 32, lane));
}

typedef __attribute__((address_space(3))) char* lds_t;

// Where a lane's fragments of a tile lie, from the start of its K (or V) rows.  K: key
// `lane % 32`, chunk 2 x + half at k ^ 32 x.  V: keys 4 half + lane / 4 % 4 (+ 8, 16, ...),
// the 16 d of the lane's group of 16 in 64-byte block dt at v[dt].
template <class C>
struct Frag {
  uint32_t k, v[C::D / 32];
  __device__ __forceinline__ explicit Frag(int lane) {
    const int r = lane & 31, h = lane >> 5, q = (lane >> 2) & 3;
    k = r * C::kRowBytes + 16 * k_slot<C>(h, r);
#pragma unroll
    for (int dt = 0; dt < C::D / 32; ++dt)
      v[dt] = (4 * h + q) * C::kRowBytes + 16 * v_slot<C>(4 * dt + 2 * ((lane >> 4) & 1), q) + 8 * (lane & 3);
  }
};

}  // namespace dfs
