// rope.hip -- norms of query and key heads and the position rotation on gfx950, into rows or
// into the paged key-value cache:
//     y = x * rsqrt(mean(x^2) + eps) * w                      (optional)
//     (a, b) -> (a cos - b sin, b cos + a sin)                 for the pairs of the first R channels
// A pair is (c, c + R/2) or (2 c, 2 c + 1); its cosine and sine stand in the row of a table that the
// token's position (one, or one of up to four axes by the pair's section) names.
//
// 16 lanes own a row, and lane n of them holds elements 32 b + 2 n and 32 b + 2 n + 1 of every
// 32-block b, as in the cache's own kernels: a Q8_0 block's largest magnitude and the row's sum of
// squares are reductions over one DPP row.  A neighbour pair sits in one lane.
#include "kv_device.h"
#include "nvq_launch.h"

#include <type_traits>

namespace nvq {

namespace {

constexpr int kThreads = 256;

struct Args {
  RopeRows r;
  KvCache c;
  const int64_t* slots;
  int64_t n_slots;
  uint32_t per;     // rows of a token
  uint32_t groups;  // 16-lane groups of a token
  uint32_t total;   // of the launch
  int fmt;          // of the cache, -1: none
};

// Sum over 16 lanes, the same in all of them.
__device__ __forceinline__ float row16_sum(float v) {
  const auto moved = [](float x, auto step) {
    return __builtin_bit_cast(float, __builtin_amdgcn_update_dpp(0, __builtin_bit_cast(int, x), decltype(step)::value, 0xF, 0xF, true));
  };
  v += moved(v, std::integral_constant<int, 0xB1>{});
  v += moved(v, std::integral_constant<int, 0x4E>{});
  v += moved(v, std::integral_constant<int, 0x141>{});
  v += moved(v, std::integral_constant<int, 0x140>{});
  return v;
}

// Two neighbouring elements from element `at` of a row argument on.
__device__ __forceinline__ void load_any(const void* p, int type, int64_t at, float (&x)[2]) {
  if (type == NVQ_TYPE_F32)
    load_pair(reinterpret_cast<const float*>(p) + at, x);
  else if (type == NVQ_TYPE_F16)
    load_pair(reinterpret_cast<const _Float16*>(p) + at, x);
  else
    load_pair(reinterpret_cast<const __bf16*>(p) + at, x);
}
__device__ __forceinline__ void store_any(void* p, int type, int64_t at, float a, float b) {
  if (type == NVQ_TYPE_F32)
    store_pair(reinterpret_cast<float*>(p) + at, a, b);
  else if (type == NVQ_TYPE_F16)
    store_pair(reinterpret_cast<_Float16*>(p) + at, a, b);
  else
    store_pair(reinterpret_cast<__bf16*>(p) + at, a, b);
}

// Cosine and sine of pair c at the token's position; a position outside the table gives NaN.
__device__ __forceinline__ void angle_of(const RopeRows& r, const int (&at)[4], int c, float& cos, float& sin) {
  const int axis = (c >= r.ends[0]) + (c >= r.ends[1]) + (c >= r.ends[2]);
  const int p = axis == 0 ? at[0] : axis == 1 ? at[1] : axis == 2 ? at[2] : at[3];
  const bool in = (uint32_t)p < (uint32_t)r.n_pos;
  const float* row = r.table + (in ? (int64_t)p * r.rot : 0);
  cos = in ? row[c] : __builtin_nanf("");
  sin = in ? row[c + r.rot / 2] : __builtin_nanf("");
}

template <int NB>
__global__ __launch_bounds__(kThreads) void rope_kernel(Args a) {
  const uint32_t id = blockIdx.x * (kThreads / 16) + (threadIdx.x >> 4);
  if (id >= a.total) return;  // whole 16-lane rows leave together
  const int n = (int)(threadIdx.x & 15);
  const uint32_t t = id / a.per, h = id - t * a.per;
  const RopeRows& r = a.r;
  // queries, keys, values
  const int kind = h < r.heads[0] ? 0 : h < r.heads[0] + r.heads[1] ? 1 : 2;
  const uint32_t head = h - (kind > 0 ? r.heads[0] : 0) - (kind > 1 ? r.heads[1] : 0);
  const int64_t from = (int64_t)t * r.in_t[kind] + (int64_t)head * r.in_h[kind];
  float x[NB][2];
#pragma unroll
  for (int b = 0; b < NB; ++b) load_any(r.in[kind], r.type, from + 32 * b + 2 * n, x[b]);
  if (kind < 2) {
    float norm = 1.0f;
    const float* w = r.weight[kind];
    if (w) {
      float s = 0.0f;
#pragma unroll
      for (int b = 0; b < NB; ++b) s = __builtin_fmaf(x[b][0], x[b][0], __builtin_fmaf(x[b][1], x[b][1], s));
      norm = __builtin_amdgcn_rsqf(row16_sum(s) * (1.0f / (32 * NB)) + r.eps);
#pragma unroll
      for (int b = 0; b < NB; ++b) {
        float y[2];
        load_pair(w + 32 * b + 2 * n, y);
        x[b][0] = x[b][0] * norm * y[0], x[b][1] = x[b][1] * norm * y[1];
      }
    }
    int at[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) at[i] = i < r.axes ? r.positions[(int64_t)i * r.axis_stride + t] : -1;
    if (r.neighbours) {
#pragma unroll
      for (int b = 0; b < NB; ++b) {
        const int c = 16 * b + n;
        if (2 * c < r.rot) {
          float cos, sin;
          angle_of(r, at, c, cos, sin);
          const float u = x[b][0], v = x[b][1];
          x[b][0] = u * cos - v * sin, x[b][1] = v * cos + u * sin;
        }
      }
    } else {
      const int half = r.rot / 2;
#pragma unroll
      for (int b = 0; b < NB; ++b) {
        const int e = 32 * b + 2 * n;
        if (e < r.rot) {
          const bool low = e < half;
          const int c = low ? e : e - half, o = low ? e + half : e - half;
          float y[2];
          load_any(r.in[kind], r.type, from + o, y);
          if (w) y[0] = y[0] * norm * w[o], y[1] = y[1] * norm * w[o + 1];
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            float cos, sin;
            angle_of(r, at, c + i, cos, sin);
            x[b][i] = low ? x[b][i] * cos - y[i] * sin : x[b][i] * cos + y[i] * sin;
          }
        }
      }
    }
  }
  if (kind == 0 || a.fmt < 0) {
    const int64_t to = (int64_t)t * r.out_t[kind & 1] + (int64_t)head * r.out_h[kind & 1];
#pragma unroll
    for (int b = 0; b < NB; ++b) store_any(r.out[kind & 1], r.out_type, to + 32 * b + 2 * n, x[b][0], x[b][1]);
    return;
  }
  const int64_t slot = a.slots[t];
  const int64_t page = slot >> a.c.page_shift, off = slot & ((int64_t(1) << a.c.page_shift) - 1);
  const int64_t row = ((page * r.heads[1] + head) << a.c.page_shift) + off;
  const bool in = slot >= 0 && slot < a.n_slots;
  uint8_t* codes = reinterpret_cast<uint8_t*>(const_cast<void*>(kind == 1 ? a.c.k : a.c.v));
  if (a.fmt == NVQ_KV_Q8_0) {
    uint16_t code[NB], scale[NB];
#pragma unroll
    for (int b = 0; b < NB; ++b) {
      const uint32_t u0 = __builtin_bit_cast(uint32_t, x[b][0]) & 0x7FFFFFFFu;
      const uint32_t u1 = __builtin_bit_cast(uint32_t, x[b][1]) & 0x7FFFFFFFu;
      code[b] = quant_pair(x[b], row16_umax(max(u0, u1)), scale[b]);
    }
    if (in) {
      store_halves<NB>(codes + row * (32 * NB) + 2 * NB * n, code);
      if (n == 0) store_halves<NB>(reinterpret_cast<uint16_t*>(const_cast<void*>(kind == 1 ? a.c.k_d : a.c.v_d)) + row * NB, scale);
    }
  } else if (in) {
#pragma unroll
    for (int b = 0; b < NB; ++b) {
      if (a.fmt == NVQ_KV_F16)
        store_pair(reinterpret_cast<_Float16*>(codes) + row * (32 * NB) + 32 * b + 2 * n, x[b][0], x[b][1]);
      else
        store_pair(reinterpret_cast<__bf16*>(codes) + row * (32 * NB) + 32 * b + 2 * n, x[b][0], x[b][1]);
    }
  }
}

template <int NB>
void launch_nb(const Args& a, hipStream_t s) {
  constexpr uint32_t kGroups = kThreads / 16;
  hipLaunchKernelGGL((rope_kernel<NB>), dim3((a.total + kGroups - 1) / kGroups), dim3(kThreads), 0, s, a);
}

size_t bytes_of(int type) { return type == NVQ_TYPE_F32 ? 4 : 2; }

}  // namespace

hipError_t launch_rope(const RopeRows& rows, int64_t T, int64_t D, int fmt, const KvCache* c, const int64_t* slots, hipStream_t stream) {
  Args a;
  a.r = rows;
  a.fmt = fmt;
  a.c = c ? *c : KvCache{};
  a.n_slots = c ? c->n_pages << c->page_shift : 0;
  a.per = rows.heads[0] + rows.heads[1] + rows.heads[2];
  a.groups = a.per;
  // a launch takes fewer than 2^32 threads, 16 to a row: longer calls go in pieces
  const int64_t most = ((int64_t(1) << 28) - 16) / a.groups;
  for (int64_t t = 0; t < T; t += most) {
    a.total = (uint32_t)((T - t < most ? T - t : most) * a.groups);
    for (int w = 0; w < 3; ++w)
      if (rows.in[w]) a.r.in[w] = (const char*)rows.in[w] + t * rows.in_t[w] * (int64_t)bytes_of(rows.type);
    for (int w = 0; w < 2; ++w)
      if (rows.out[w]) a.r.out[w] = (char*)rows.out[w] + t * rows.out_t[w] * (int64_t)bytes_of(rows.out_type);
    a.r.positions = rows.positions + t;
    a.slots = slots ? slots + t : nullptr;
    switch (D / 32) {
      case 1: launch_nb<1>(a, stream); break;
      case 2: launch_nb<2>(a, stream); break;
      case 3: launch_nb<3>(a, stream); break;
      case 4: launch_nb<4>(a, stream); break;
      case 5: launch_nb<5>(a, stream); break;
      case 6: launch_nb<6>(a, stream); break;
      case 7: launch_nb<7>(a, stream); break;
      default: launch_nb<8>(a, stream); break;
    }
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

}  // namespace nvq
