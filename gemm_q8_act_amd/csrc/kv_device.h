// kv_device.h -- device helpers of the kernels that write and read the paged key-value cache:
// Q8_0 of a block held by 16 lanes, and a lane's part of a row in wide accesses.
#pragma once

#include "attn_device.h"

namespace nvq {

// Largest of the unsigned values of a row's 16 or 8 lanes, the same in all of them; magnitudes' bits order as their values do,
// infinity and NaN last
template <int STEP>
__device__ __forceinline__ uint32_t moved(uint32_t x) {
  return (uint32_t)__builtin_amdgcn_update_dpp(0, (int)x, STEP, 0xF, 0xF, true);
}
template <int LANES>
__device__ __forceinline__ uint32_t lanes_max(uint32_t v) {
  v = max(v, moved<0xB1>(v)), v = max(v, moved<0x4E>(v)), v = max(v, moved<0x141>(v));
  if constexpr (LANES == 16) v = max(v, moved<0x140>(v));
  return v;
}

// Q8_0 of a pair of a block whose largest magnitude's bits are `top`: its two codes, and the
// block's binary16 scale.  The definition's IEEE divisions (amax / 127, x / d, ties to even)
// come out bit for bit without their long instruction sequences, which bound the kernel:
//   d: amax * fl(1/127) and one fma correction give fl(amax / 127) for every finite float.
//   x / d: fma(x, rcp(d), 128) is within 4.2e-5 of 128 + fl(x / d) (one-ulp reciprocal, |x / d|
//     <= 127.00002), so unless it lies within 2^-14 of a rounding tie its nearest whole number
//     is the code + 128; nearer ones, and blocks whose reciprocal could leave the normal range,
//     divide.
// A block with an infinity or NaN takes a NaN scale: it reads back as NaN, never as numbers.
__device__ __forceinline__ uint16_t quant_pair(const float (&x)[2], uint32_t top, uint16_t& scale) {
  constexpr float kInv127 = 0x1.020408p-7f;  // fl(1 / 127)
  const float amax = __builtin_bit_cast(float, top), t = amax * kInv127;
  const float d = top < 0x7F800000u ? __builtin_fmaf(__builtin_fmaf(-t, 127.0f, amax), kInv127, t) : __builtin_nanf("");
  const float r = d > 0.0f ? __builtin_amdgcn_rcpf(d) : 0.0f;
  const float u0 = __builtin_fmaf(x[0], r, 128.0f), u1 = __builtin_fmaf(x[1], r, 128.0f);
  float k0 = __builtin_rintf(u0), k1 = __builtin_rintf(u1);
  if (fmaxf(fabsf(u0 - k0), fabsf(u1 - k1)) > 0.5f - 0x1.0p-14f || (d > 0.0f && d < 0x1.0p-100f)) {
    k0 = fminf(fmaxf(__builtin_rintf(x[0] / d), -127.0f), 127.0f) + 128.0f;
    k1 = fminf(fmaxf(__builtin_rintf(x[1] / d), -127.0f), 127.0f) + 128.0f;
  }
  const uint32_t codes = __builtin_amdgcn_cvt_pk_u8_f32(k1, 1u, __builtin_amdgcn_cvt_pk_u8_f32(k0, 0u, 0u));
  scale = __builtin_bit_cast(uint16_t, (_Float16)d);
  return (uint16_t)(codes ^ 0x8080u);
}

// N 16-bit pieces moved with the widest accesses that their common alignment allows (the
// address is a multiple of 2 N bytes from a 16-byte aligned base)
template <int N>
__device__ __forceinline__ void store_halves(void* p, const uint16_t (&v)[N]) {
  if constexpr (N % 8 == 0) {
#pragma unroll
    for (int i = 0; i < N / 8; ++i) {
      u32x4 w;
#pragma unroll
      for (int j = 0; j < 4; ++j) w[j] = v[8 * i + 2 * j] | ((uint32_t)v[8 * i + 2 * j + 1] << 16);
      reinterpret_cast<u32x4*>(p)[i] = w;
    }
  } else if constexpr (N % 4 == 0) {
#pragma unroll
    for (int i = 0; i < N / 4; ++i)
      reinterpret_cast<u32x2*>(p)[i] = u32x2{v[4 * i] | ((uint32_t)v[4 * i + 1] << 16), v[4 * i + 2] | ((uint32_t)v[4 * i + 3] << 16)};
  } else if constexpr (N % 2 == 0) {
#pragma unroll
    for (int i = 0; i < N / 2; ++i) reinterpret_cast<uint32_t*>(p)[i] = v[2 * i] | ((uint32_t)v[2 * i + 1] << 16);
  } else {
#pragma unroll
    for (int i = 0; i < N; ++i) reinterpret_cast<uint16_t*>(p)[i] = v[i];
  }
}
template <int N>
__device__ __forceinline__ void load_halves(const void* p, uint16_t (&v)[N]) {
  if constexpr (N % 8 == 0) {
#pragma unroll
    for (int i = 0; i < N / 8; ++i) {
      const u32x4 w = reinterpret_cast<const u32x4*>(p)[i];
#pragma unroll
      for (int j = 0; j < 4; ++j) v[8 * i + 2 * j] = (uint16_t)w[j], v[8 * i + 2 * j + 1] = (uint16_t)(w[j] >> 16);
    }
  } else if constexpr (N % 4 == 0) {
#pragma unroll
    for (int i = 0; i < N / 4; ++i) {
      const u32x2 w = reinterpret_cast<const u32x2*>(p)[i];
      v[4 * i] = (uint16_t)w[0], v[4 * i + 1] = (uint16_t)(w[0] >> 16), v[4 * i + 2] = (uint16_t)w[1], v[4 * i + 3] = (uint16_t)(w[1] >> 16);
    }
  } else if constexpr (N % 2 == 0) {
#pragma unroll
    for (int i = 0; i < N / 2; ++i) {
      const uint32_t w = reinterpret_cast<const uint32_t*>(p)[i];
      v[2 * i] = (uint16_t)w, v[2 * i + 1] = (uint16_t)(w >> 16);
    }
  } else {
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] = reinterpret_cast<const uint16_t*>(p)[i];
  }
}

}  // namespace nvq
