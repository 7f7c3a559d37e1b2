// kv_cache.hip -- the paged key-value cache on gfx950: rows written into it (quantised to
// Q8_0 on the way, or converted to a 16-bit type) and read back.
//
// A cache row is one token's D channels of one key or value head.  16 lanes own a row
// and lane n of them holds elements 32 b + 2 n and 32 b + 2 n + 1 of every 32-block b, so a
// block's largest magnitude is a reduction over one DPP row, the row's loads are 128 (64)
// contiguous bytes a block, and the lane's codes are the 2 D/32 consecutive bytes that
// the quantised row's element order gives it (nvq.h): one wide store.
//
// HBM-bound: D * (element bytes + 34/32) a row, each byte once; 16411 tokens of 8 key heads of
// 128, bfloat16 to Q8_0: written in 25.5 us (4.0 TB/s), read in 20 us (5.2 TB/s; a large copy
// 4.75).  Keys and values go in one launch: a decode step writes a few rows and is all launch (one
// token: 2.6 us written, 1.8 read).
#include "attn_device.h"
#include "nvq_launch.h"

namespace nvq {

namespace {

struct KvArgs {
  const void* rows[2];   // keys, values (write: read from; read: written to)
  int64_t stride_t[2], stride_h[2];
  uint8_t* codes[2];
  uint16_t* scales[2];
  const int64_t* slots;
  int n_rows;            // tokens * heads
  int64_t n_slots;       // pages * page size
  uint32_t heads;
  uint32_t page_shift;
};

// Largest of 16 lanes' unsigned values; magnitudes' bits order as their values do, infinity and NaN last
__device__ __forceinline__ uint32_t row16_umax(uint32_t v) {
  v = max(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0xB1, 0xF, 0xF, true));
  v = max(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x4E, 0xF, 0xF, true));
  v = max(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x141, 0xF, 0xF, true));
  v = max(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x140, 0xF, 0xF, true));
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
    *reinterpret_cast<u32x2*>(p) = u32x2{v[0] | ((uint32_t)v[1] << 16), v[2] | ((uint32_t)v[3] << 16)};
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
    const u32x2 w = *reinterpret_cast<const u32x2*>(p);
    v[0] = (uint16_t)w[0], v[1] = (uint16_t)(w[0] >> 16), v[2] = (uint16_t)w[1], v[3] = (uint16_t)(w[1] >> 16);
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

// Where row r = token * heads + head lives: its cache row's number, or -1 (a negative slot: no
// token) or -2 (a slot past the cache)
struct KvRow {
  int64_t t, h, cache;
};
__device__ __forceinline__ KvRow locate(const KvArgs& a, int r) {
  KvRow o;
  const uint32_t t = (uint32_t)r / a.heads;
  o.t = t, o.h = (uint32_t)r - t * a.heads;
  const int64_t s = a.slots[o.t];
  const int64_t pg = s >> a.page_shift, off = s & ((1ll << a.page_shift) - 1);
  o.cache = s < 0 ? -1 : s >= a.n_slots ? -2 : ((pg * a.heads + o.h) << a.page_shift) + off;
  return o;
}

template <typename T>
__device__ __forceinline__ const T* row_at(const KvArgs& a, const KvRow& row, int w) {
  return reinterpret_cast<const T*>(a.rows[w]) + row.t * a.stride_t[w] + row.h * a.stride_h[w] + 2 * (threadIdx.x & 15);
}

// T: the rows' type.  FMT: the cache's.  NB: 32-blocks of a row.  16 lanes take a token's key row
// and value row of one head; all loads go out before the slot is looked at (the rows are there
// whatever it says), so one round trip to memory covers both.
template <typename T, int FMT, int NB>
__global__ __launch_bounds__(256) void kv_write_kernel(KvArgs a) {
  const int r = (int)blockIdx.x * 16 + (int)(threadIdx.x >> 4);
  if (r >= a.n_rows) return;  // whole 16-lane rows leave together
  const int n = (int)(threadIdx.x & 15);
  const KvRow row = locate(a, r);
  float x[2][NB][2];
#pragma unroll
  for (int w = 0; w < 2; ++w)
#pragma unroll
    for (int b = 0; b < NB; ++b) load_pair(row_at<T>(a, row, w) + 32 * b, x[w][b]);
#pragma unroll
  for (int w = 0; w < 2; ++w) {
    if constexpr (FMT == NVQ_KV_Q8_0) {
      uint16_t code[NB], scale[NB];
#pragma unroll
      for (int b = 0; b < NB; ++b) {
        const uint32_t u0 = __builtin_bit_cast(uint32_t, x[w][b][0]) & 0x7FFFFFFFu;
        const uint32_t u1 = __builtin_bit_cast(uint32_t, x[w][b][1]) & 0x7FFFFFFFu;
        code[b] = quant_pair(x[w][b], row16_umax(max(u0, u1)), scale[b]);
      }
      if (row.cache >= 0) {
        store_halves<NB>(a.codes[w] + row.cache * (32 * NB) + 2 * NB * n, code);
        if (n == 0) store_halves<NB>(a.scales[w] + row.cache * NB, scale);
      }
    } else if (row.cache >= 0) {
      // one rounding, to nearest even, to the cache's type
      uint32_t* dst = reinterpret_cast<uint32_t*>(a.codes[w] + row.cache * (64 * NB)) + n;
#pragma unroll
      for (int b = 0; b < NB; ++b) dst[16 * b] = pack_pair<typename CacheType<FMT>::type>(x[w][b][0], x[w][b][1]);
    }
  }
}

template <typename T, int FMT, int NB>
__global__ __launch_bounds__(256) void kv_read_kernel(KvArgs a) {
  const int r = (int)blockIdx.x * 16 + (int)(threadIdx.x >> 4);
  if (r >= a.n_rows) return;
  const int n = (int)(threadIdx.x & 15);
  const KvRow row = locate(a, r);
  const int64_t at = max(row.cache, (int64_t)0);  // a slot that names no row: any row, unused
  float x[2][NB][2];
  if constexpr (FMT == NVQ_KV_Q8_0) {
    uint16_t code[2][NB], scale[2][NB];
#pragma unroll
    for (int w = 0; w < 2; ++w) {
      load_halves<NB>(a.codes[w] + at * (32 * NB) + 2 * NB * n, code[w]);
      load_halves<NB>(a.scales[w] + at * NB, scale[w]);
    }
#pragma unroll
    for (int w = 0; w < 2; ++w)
#pragma unroll
      for (int b = 0; b < NB; ++b) {
        const float d = f16_bits_to_f32(scale[w][b]);
        x[w][b][0] = (float)(int8_t)(code[w][b] & 0xFF) * d;  // 8 + 11 significant bits: exact
        x[w][b][1] = (float)(int8_t)(code[w][b] >> 8) * d;
      }
  } else {
    uint32_t pair[2][NB];
#pragma unroll
    for (int w = 0; w < 2; ++w)
#pragma unroll
      for (int b = 0; b < NB; ++b) pair[w][b] = reinterpret_cast<const uint32_t*>(a.codes[w] + at * (64 * NB))[16 * b + n];
#pragma unroll
    for (int w = 0; w < 2; ++w)
#pragma unroll
      for (int b = 0; b < NB; ++b) unpack_pair<typename CacheType<FMT>::type>(pair[w][b], x[w][b]);
  }
  const float none = row.cache == -1 ? 0.0f : __builtin_nanf("");
#pragma unroll
  for (int w = 0; w < 2; ++w) {
    T* dst = const_cast<T*>(row_at<T>(a, row, w));
#pragma unroll
    for (int b = 0; b < NB; ++b) store_pair(dst + 32 * b, row.cache < 0 ? none : x[w][b][0], row.cache < 0 ? none : x[w][b][1]);
  }
}

template <typename T, int FMT, int NB>
void launch_nb(const KvArgs& a, bool write, hipStream_t s) {
  const dim3 grid(((unsigned)a.n_rows + 15) / 16);
  if (write)
    hipLaunchKernelGGL((kv_write_kernel<T, FMT, NB>), grid, dim3(256), 0, s, a);
  else
    hipLaunchKernelGGL((kv_read_kernel<T, FMT, NB>), grid, dim3(256), 0, s, a);
}
template <typename T, int FMT>
void launch_fmt(const KvArgs& a, int nb, bool write, hipStream_t s) {
  switch (nb) {
    case 1: return launch_nb<T, FMT, 1>(a, write, s);
    case 2: return launch_nb<T, FMT, 2>(a, write, s);
    case 3: return launch_nb<T, FMT, 3>(a, write, s);
    case 4: return launch_nb<T, FMT, 4>(a, write, s);
    case 5: return launch_nb<T, FMT, 5>(a, write, s);
    case 6: return launch_nb<T, FMT, 6>(a, write, s);
    case 7: return launch_nb<T, FMT, 7>(a, write, s);
    default: return launch_nb<T, FMT, 8>(a, write, s);
  }
}
template <typename T>
void launch_type(const KvArgs& a, int fmt, int nb, bool write, hipStream_t s) {
  if (fmt == NVQ_KV_Q8_0) return launch_fmt<T, NVQ_KV_Q8_0>(a, nb, write, s);
  if (fmt == NVQ_KV_F16) return launch_fmt<T, NVQ_KV_F16>(a, nb, write, s);
  return launch_fmt<T, NVQ_KV_BF16>(a, nb, write, s);
}

}  // namespace

hipError_t launch_kv_copy(bool write, int fmt, int type, const void* k, const void* v, const int64_t strides[4],
                          const int64_t* slots, int64_t T, int64_t heads, int64_t D, const KvCache& c, hipStream_t stream) {
  KvArgs a;
  a.stride_t[0] = strides[0], a.stride_h[0] = strides[1], a.stride_t[1] = strides[2], a.stride_h[1] = strides[3];
  a.codes[0] = (uint8_t*)c.k, a.codes[1] = (uint8_t*)c.v;
  a.scales[0] = (uint16_t*)c.k_d, a.scales[1] = (uint16_t*)c.v_d;
  a.n_slots = c.n_pages << c.page_shift;
  a.heads = (uint32_t)heads;
  a.page_shift = (uint32_t)c.page_shift;
  const int nb = (int)(D / 32);
  // a launch takes fewer than 2^32 threads, 16 to a row: longer calls go in pieces
  const int64_t most = ((int64_t(1) << 28) - 16) / heads;
  for (int64_t t = 0; t < T; t += most) {
    a.n_rows = (int)((T - t < most ? T - t : most) * heads);
    for (int w = 0; w < 2; ++w)
      a.rows[w] = (const char*)(w ? v : k) + t * a.stride_t[w] * (type == NVQ_TYPE_F32 ? 4 : 2);
    a.slots = slots + t;
    if (type == NVQ_TYPE_F32)
      launch_type<float>(a, fmt, nb, write, stream);
    else if (type == NVQ_TYPE_F16)
      launch_type<_Float16>(a, fmt, nb, write, stream);
    else
      launch_type<__bf16>(a, fmt, nb, write, stream);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

}  // namespace nvq
