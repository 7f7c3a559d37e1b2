// kv_cache.hip -- the paged key-value cache on gfx950: rows written into it (quantised to
// Q8_0 on the way, or converted to a 16-bit type) and read back.
//
// A cache row is one token's D channels of one key or value head.  16 lanes own a row
// and lane n of them holds elements 32 b + 2 n and 32 b + 2 n + 1 of every 32-block b, so a
// block's largest magnitude is a reduction over one DPP row, the row's loads are 128 (64)
// contiguous bytes a block, and the lane's codes are the 2 D/32 consecutive bytes that
// the quantised row's element order gives it (nvq.h): one wide store.
//
// HBM-bound: D * (element bytes + 34/32) a row, each byte once.  Both tensors go in one
// launch (blockIdx.y: keys, values): a decode step writes a few rows and is all launch.
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
  int64_t n_rows;        // tokens * heads
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
__device__ __forceinline__ KvRow locate(const KvArgs& a, int64_t r) {
  KvRow o;
  // 32-bit division where the row number allows it
  if (a.n_rows <= 0xFFFFFFFFll) {
    const uint32_t t = (uint32_t)r / a.heads;
    o.t = t, o.h = (uint32_t)r - t * a.heads;
  } else {
    o.t = r / a.heads, o.h = r - o.t * a.heads;
  }
  const int64_t s = a.slots[o.t];
  const int64_t pg = s >> a.page_shift, off = s & ((1ll << a.page_shift) - 1);
  o.cache = s < 0 ? -1 : s >= a.n_slots ? -2 : ((pg * a.heads + o.h) << a.page_shift) + off;
  return o;
}

// T: the rows' type.  FMT: the cache's.  NB: 32-blocks of a row.
template <typename T, int FMT, int NB>
__global__ __launch_bounds__(256) void kv_write_kernel(KvArgs a) {
  const int64_t r = (int64_t)blockIdx.x * 16 + (threadIdx.x >> 4);
  if (r >= a.n_rows) return;  // whole 16-lane rows leave together
  const int n = (int)(threadIdx.x & 15), w = (int)blockIdx.y;
  const KvRow row = locate(a, r);
  if (row.cache < 0) return;
  const T* src = reinterpret_cast<const T*>(a.rows[w]) + row.t * a.stride_t[w] + row.h * a.stride_h[w] + 2 * n;
  float x[NB][2];
#pragma unroll
  for (int b = 0; b < NB; ++b) load_pair(src + 32 * b, x[b]);
  if constexpr (FMT == NVQ_KV_Q8_0) {
    uint16_t code[NB], scale[NB];
#pragma unroll
    for (int b = 0; b < NB; ++b) {
      const uint32_t u0 = __builtin_bit_cast(uint32_t, x[b][0]) & 0x7FFFFFFFu;
      const uint32_t u1 = __builtin_bit_cast(uint32_t, x[b][1]) & 0x7FFFFFFFu;
      // the activation quantiser's arithmetic: IEEE divisions, ties to even.  An infinite
      // or NaN element makes the scale infinite or NaN and the codes 0: the block reads
      // back as NaN, never as numbers.
      const float d = __builtin_bit_cast(float, row16_umax(max(u0, u1))) / 127.0f;
      int q0 = 0, q1 = 0;
      if (d > 0.0f && d < __builtin_inff()) {
        q0 = (int)fminf(fmaxf(__builtin_rintf(x[b][0] / d), -127.0f), 127.0f);
        q1 = (int)fminf(fmaxf(__builtin_rintf(x[b][1] / d), -127.0f), 127.0f);
      }
      code[b] = (uint16_t)((q0 & 0xFF) | ((q1 & 0xFF) << 8));
      scale[b] = __builtin_bit_cast(uint16_t, (_Float16)d);
    }
    store_halves<NB>(a.codes[w] + row.cache * (32 * NB) + 2 * NB * n, code);
    if (n == 0) store_halves<NB>(a.scales[w] + row.cache * NB, scale);
  } else {
    // one rounding, to nearest even, to the cache's type
    uint32_t* dst = reinterpret_cast<uint32_t*>(a.codes[w] + row.cache * (64 * NB)) + n;
#pragma unroll
    for (int b = 0; b < NB; ++b) dst[16 * b] = pack_pair<typename CacheType<FMT>::type>(x[b][0], x[b][1]);
  }
}

template <typename T, int FMT, int NB>
__global__ __launch_bounds__(256) void kv_read_kernel(KvArgs a) {
  const int64_t r = (int64_t)blockIdx.x * 16 + (threadIdx.x >> 4);
  if (r >= a.n_rows) return;
  const int n = (int)(threadIdx.x & 15), w = (int)blockIdx.y;
  const KvRow row = locate(a, r);
  T* dst = reinterpret_cast<T*>(const_cast<void*>(a.rows[w])) + row.t * a.stride_t[w] + row.h * a.stride_h[w] + 2 * n;
  float x[NB][2];
  if (row.cache < 0) {
    const float v = row.cache == -1 ? 0.0f : __builtin_nanf("");
#pragma unroll
    for (int b = 0; b < NB; ++b) x[b][0] = x[b][1] = v;
  } else if constexpr (FMT == NVQ_KV_Q8_0) {
    uint16_t code[NB], scale[NB];
    load_halves<NB>(a.codes[w] + row.cache * (32 * NB) + 2 * NB * n, code);
    load_halves<NB>(a.scales[w] + row.cache * NB, scale);
#pragma unroll
    for (int b = 0; b < NB; ++b) {
      const float d = f16_bits_to_f32(scale[b]);
      x[b][0] = (float)(int8_t)(code[b] & 0xFF) * d;  // 8 + 11 significant bits: exact
      x[b][1] = (float)(int8_t)(code[b] >> 8) * d;
    }
  } else {
    const uint32_t* src = reinterpret_cast<const uint32_t*>(a.codes[w] + row.cache * (64 * NB)) + n;
#pragma unroll
    for (int b = 0; b < NB; ++b) unpack_pair<typename CacheType<FMT>::type>(src[16 * b], x[b]);
  }
#pragma unroll
  for (int b = 0; b < NB; ++b) store_pair(dst + 32 * b, x[b][0], x[b][1]);
}

template <typename T, int FMT, int NB>
void launch_nb(const KvArgs& a, bool write, hipStream_t s) {
  const dim3 grid((unsigned)((a.n_rows + 15) / 16), 2);
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
  a.rows[0] = k, a.rows[1] = v;
  a.stride_t[0] = strides[0], a.stride_h[0] = strides[1], a.stride_t[1] = strides[2], a.stride_h[1] = strides[3];
  a.codes[0] = (uint8_t*)c.k, a.codes[1] = (uint8_t*)c.v;
  a.scales[0] = (uint16_t*)c.k_d, a.scales[1] = (uint16_t*)c.v_d;
  a.slots = slots;
  a.n_rows = T * heads;
  a.n_slots = c.n_pages << c.page_shift;
  a.heads = (uint32_t)heads;
  a.page_shift = (uint32_t)c.page_shift;
  const int nb = (int)(D / 32);
  if (type == NVQ_TYPE_F32)
    launch_type<float>(a, fmt, nb, write, stream);
  else if (type == NVQ_TYPE_F16)
    launch_type<_Float16>(a, fmt, nb, write, stream);
  else
    launch_type<__bf16>(a, fmt, nb, write, stream);
  return hipGetLastError();
}

}  // namespace nvq
