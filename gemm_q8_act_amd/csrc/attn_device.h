// attn_device.h -- device helpers shared by the cache and attention kernels: element
// types, matrix products by type, exchanges between lanes.
#pragma once

#include "nvq.h"
#include "nvq_device.h"

namespace nvq {

typedef __bf16 bf16x2_t __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x8_t __attribute__((ext_vector_type(8)));
typedef float floatx2 __attribute__((ext_vector_type(2)));

// The element type of a cache format's codes (Q8_0's operands are binary16).
template <int FMT>
struct CacheType {
  typedef _Float16 type;
};
template <>
struct CacheType<NVQ_KV_BF16> {
  typedef __bf16 type;
};

// Two floats rounded to nearest even into one dword of 16-bit elements (one instruction), and back.
template <typename T>
__device__ __forceinline__ uint32_t pack_pair(float a, float b) {
  typedef T t2 __attribute__((ext_vector_type(2)));
  return __builtin_bit_cast(uint32_t, __builtin_convertvector((floatx2{a, b}), t2));
}
template <typename T>
__device__ __forceinline__ void unpack_pair(uint32_t v, float (&x)[2]) {
  typedef T t2 __attribute__((ext_vector_type(2)));
  const t2 t = __builtin_bit_cast(t2, v);
  x[0] = (float)t[0], x[1] = (float)t[1];
}

// Two neighbouring elements of a row as floats; p is aligned to the pair.
__device__ __forceinline__ void load_pair(const float* p, float (&x)[2]) {
  const floatx2 t = *reinterpret_cast<const floatx2*>(p);
  x[0] = t[0], x[1] = t[1];
}
template <typename T>
__device__ __forceinline__ void load_pair(const T* p, float (&x)[2]) {
  unpack_pair<T>(*reinterpret_cast<const uint32_t*>(p), x);
}
__device__ __forceinline__ void store_pair(float* p, float a, float b) { *reinterpret_cast<floatx2*>(p) = floatx2{a, b}; }
template <typename T>
__device__ __forceinline__ void store_pair(T* p, float a, float b) {
  *reinterpret_cast<uint32_t*>(p) = pack_pair<T>(a, b);
}

__device__ __forceinline__ void store_1(void* p, int type, int64_t at, float x) {
  if (type == NVQ_TYPE_F32)
    reinterpret_cast<float*>(p)[at] = x;
  else if (type == NVQ_TYPE_F16)
    reinterpret_cast<_Float16*>(p)[at] = (_Float16)x;
  else
    reinterpret_cast<__bf16*>(p)[at] = (__bf16)x;
}
// N (even) consecutive elements from element `at` on; `at` is a multiple of N or of 8.
template <int N>
__device__ __forceinline__ void store_n(void* p, int type, int64_t at, const float (&x)[N]) {
  if (type == NVQ_TYPE_F32) {
    float* d = reinterpret_cast<float*>(p) + at;
#pragma unroll
    for (int i = 0; i < N; i += 2) *reinterpret_cast<floatx2*>(d + i) = floatx2{x[i], x[i + 1]};
  } else {
    uint32_t w[N / 2];
#pragma unroll
    for (int i = 0; i < N / 2; ++i)
      w[i] = type == NVQ_TYPE_F16 ? pack_pair<_Float16>(x[2 * i], x[2 * i + 1]) : pack_pair<__bf16>(x[2 * i], x[2 * i + 1]);
    uint32_t* d = reinterpret_cast<uint32_t*>(reinterpret_cast<uint16_t*>(p) + at);
    if constexpr (N % 8 == 0) {
#pragma unroll
      for (int i = 0; i < N / 8; ++i) reinterpret_cast<u32x4*>(d)[i] = u32x4{w[4 * i], w[4 * i + 1], w[4 * i + 2], w[4 * i + 3]};
    } else {
#pragma unroll
      for (int i = 0; i < N / 2; ++i) d[i] = w[i];
    }
  }
}

// An operand of four dwords, and the two matrix products of the 16-bit types.
struct Frag {
  uint32_t v[4];
};
template <typename T>
__device__ __forceinline__ floatx4 mfma16(const Frag& a, const Frag& b, floatx4 c) {
  const u32x4 x = {a.v[0], a.v[1], a.v[2], a.v[3]}, y = {b.v[0], b.v[1], b.v[2], b.v[3]};
  if constexpr (__is_same(T, _Float16))
    return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(half8_t, x), __builtin_bit_cast(half8_t, y), c, 0, 0, 0);
  else
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8_t, x), __builtin_bit_cast(bf16x8_t, y), c, 0, 0, 0);
}
template <typename T>
__device__ __forceinline__ floatx16 mfma32(const Frag& a, const Frag& b, floatx16 c) {
  const u32x4 x = {a.v[0], a.v[1], a.v[2], a.v[3]}, y = {b.v[0], b.v[1], b.v[2], b.v[3]};
  if constexpr (__is_same(T, _Float16))
    return __builtin_amdgcn_mfma_f32_32x32x16_f16(__builtin_bit_cast(half8_t, x), __builtin_bit_cast(half8_t, y), c, 0, 0, 0);
  else
    return __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(bf16x8_t, x), __builtin_bit_cast(bf16x8_t, y), c, 0, 0, 0);
}

// Sum over the lanes up to and with the own one, in registers: shifts within rows of 16 lanes, then
// the rows' sums passed on (all lanes take part).
__device__ __forceinline__ int wave_running_sum(int v) {
  v += __builtin_amdgcn_update_dpp(0, v, 0x111, 0xF, 0xF, false);  // row_shr:1, 2, 4, 8
  v += __builtin_amdgcn_update_dpp(0, v, 0x112, 0xF, 0xF, false);
  v += __builtin_amdgcn_update_dpp(0, v, 0x114, 0xF, 0xF, false);
  v += __builtin_amdgcn_update_dpp(0, v, 0x118, 0xF, 0xF, false);
  v += __builtin_amdgcn_update_dpp(0, v, 0x142, 0xA, 0xF, false);  // row_bcast:15 into rows 1 and 3
  v += __builtin_amdgcn_update_dpp(0, v, 0x143, 0xC, 0xF, false);  // row_bcast:31 into rows 2 and 3
  return v;
}

// LDS address of a shared array's element.
__device__ __forceinline__ uint32_t lds_address(const void* p) {
  return (uint32_t)(uintptr_t)(__attribute__((address_space(3))) const void*)p;
}
// 16 bytes a lane from base + offset straight into LDS, lane after lane from `lds` on, of what
// is read once (non-temporal); the second form from an address a lane.  In assembly because the compiler, which cannot tell one part of LDS from another, waits for
// every such load before any LDS read; here the waits are written out (wait_loads).
__device__ __forceinline__ void load_once_to_lds(const uint8_t* base, uint32_t offset, uint32_t lds) {
  asm volatile("s_mov_b32 m0, %2\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %0, %1 nt" ::"v"(offset), "s"(base), "s"(lds) : "memory", "m0");
}
__device__ __forceinline__ void load_once_to_lds_far(const uint8_t* p, uint32_t lds) {
  asm volatile("s_mov_b32 m0, %1\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %0, off nt" ::"v"(p), "s"(lds) : "memory", "m0");
}
// The first `bytes` bytes from p on as a buffer: loads past its end give zeros.
__device__ __forceinline__ u32x4 buffer_of(const void* p, uint32_t bytes) {
  const uint64_t at = (uint64_t)p;
  return u32x4{(uint32_t)at, (uint32_t)(at >> 32) & 0xFFFFu, bytes, 0x00020000u};
}
// 16 bytes a lane from the buffer at `offset` into LDS, as above.  Orders itself with waits and
// barriers only: it may move among the LDS reads of other slots.
__device__ __forceinline__ void buffer_to_lds(u32x4 buffer, uint32_t offset, uint32_t lds) {
  asm volatile("s_mov_b32 m0, %2\n\ts_nop 0\n\tbuffer_load_dwordx4 %0, %1, 0 offen lds" ::"v"(offset), "s"(buffer), "s"(lds) : "m0");
}
// Until at most N of the wavefront's loads are on their way (they come back in order).
template <int N>
__device__ __forceinline__ void wait_loads() {
  asm volatile("s_waitcnt vmcnt(%0)" ::"n"(N) : "memory");
}
// Until the LDS reads so far have their data: what they read may be loaded over.
__device__ __forceinline__ void wait_reads() { asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory"); }

// Four rows' 16-bit elements of one column: of each 16 lanes, lanes 4 r .. 4 r + 3 give 32
// contiguous bytes of row r (8 a lane), and lane c gets column c of the four rows.
__device__ __forceinline__ u32x2 read_transposed(const uint8_t* p) {
  typedef short short4_t __attribute__((ext_vector_type(4)));
  return __builtin_bit_cast(u32x2, __builtin_amdgcn_ds_read_tr16_b64_v4i16((__attribute__((address_space(3))) short4_t*)p));
}

// c + both elements of a 16-bit pair, in float32
template <typename T>
__device__ __forceinline__ float add_pair(uint32_t v, float c) {
  if constexpr (__is_same(T, _Float16))
    return __builtin_amdgcn_fdot2(__builtin_bit_cast(half2_t, v), half2_t{(_Float16)1.0f, (_Float16)1.0f}, c, false);
  else
    return __builtin_amdgcn_fdot2_f32_bf16(__builtin_bit_cast(bf16x2_t, v), bf16x2_t{(__bf16)1.0f, (__bf16)1.0f}, c, false);
}
// c + 0 times both: c, or NaN if one of them is not finite
template <typename T>
__device__ __forceinline__ float zero_of_pair(uint32_t v, float c) {
  if constexpr (__is_same(T, _Float16))
    return __builtin_amdgcn_fdot2(__builtin_bit_cast(half2_t, v), half2_t{(_Float16)0.0f, (_Float16)0.0f}, c, false);
  else
    return __builtin_amdgcn_fdot2_f32_bf16(__builtin_bit_cast(bf16x2_t, v), bf16x2_t{(__bf16)0.0f, (__bf16)0.0f}, c, false);
}

// 2^x (v_exp_f32: about one unit in the last place; results below the normal range are 0)
__device__ __forceinline__ float exp2_fast(float x) { return __builtin_amdgcn_exp2f(x); }

// Largest and sum over the lanes 32 apart, 16 apart: the instruction swaps halves of two
// registers.  (The results go into scalars first: a bit cast of a vector's element reads
// element 0.)
struct Halves {
  float a, b;
};
__device__ __forceinline__ Halves halves_32(float x) {
  const uint32_t u = __builtin_bit_cast(uint32_t, x);
  const auto r = __builtin_amdgcn_permlane32_swap(u, u, false, false);
  const uint32_t a = r[0], b = r[1];
  return {__builtin_bit_cast(float, a), __builtin_bit_cast(float, b)};
}
__device__ __forceinline__ Halves halves_16(float x) {
  const uint32_t u = __builtin_bit_cast(uint32_t, x);
  const auto r = __builtin_amdgcn_permlane16_swap(u, u, false, false);
  const uint32_t a = r[0], b = r[1];
  return {__builtin_bit_cast(float, a), __builtin_bit_cast(float, b)};
}
__device__ __forceinline__ float max_32(float x) {
  const Halves h = halves_32(x);
  return fmaxf(h.a, h.b);
}
__device__ __forceinline__ float sum_32(float x) {
  const Halves h = halves_32(x);
  return h.a + h.b;
}
__device__ __forceinline__ float max_16(float x) {
  const Halves h = halves_16(x);
  return fmaxf(h.a, h.b);
}
__device__ __forceinline__ float sum_16(float x) {
  const Halves h = halves_16(x);
  return h.a + h.b;
}

}  // namespace nvq
