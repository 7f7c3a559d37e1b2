// rope.hip -- norms of query and key heads and the position rotation on gfx950, into rows or
// into the paged key-value cache:
//     y = x * rsqrt(mean(x^2) + eps) * w                      (optional)
//     (a, b) -> (a cos - b sin, b cos + a sin)                 for the pairs of the first R channels
// A pair is (c, c + R/2) or (2 c, 2 c + 1); its cosine and sine stand in the row of a table that the
// token's position (one, or one of up to four axes by the pair's section) names.
//
// 8 lanes own a row, and lane n of them holds elements 32 b + 4 n .. + 3 of every 32-block b: a
// neighbour pair sits in one lane, halves that lie whole blocks apart too, a block's largest magnitude
// and the row's sum of squares are three exchanges between lanes, and the lane's Q8_0 codes are
// consecutive bytes of the row (nvq.h).  Halves that end elsewhere (D or R of an odd number of blocks) read
// their partners once more, with 16 lanes to a row.
//
// HBM-bound: every row is read and written once.  40/8 heads of 128, normed and turned: 2048 float32 tokens
// to bfloat16 14.5 us (5.3 TB/s; a large copy 4.75, part of this stays in the Infinity Cache), 16411
// bfloat16 tokens with three axes 90 us (4.6 TB/s); into a bfloat16 cache, half of the channels turned,
// 93 us (5.1 TB/s).  What got it there from 294 us: one look at the table for a lane's pairs in wide
// loads (four heads to a row's lanes, to share it, was slower: 120), and one kind of rows to a workgroup,
// so that what differs between queries, keys and values is uniform and all loads go out before any wait
// (107 -> 90 us).  A decode step is one launch: 2.6 us, 3 round trips to memory.
#include "kv_device.h"
#include "nvq_launch.h"

namespace nvq {

namespace {

constexpr int kThreads = 256;

struct Args {
  RopeRows r;
  KvCache c;
  const int64_t* slots;
  int64_t n_slots;
  int blocks[2];  // workgroups of queries, and of queries and keys
  int T;          // tokens of the launch
  int fmt;        // of the cache, -1: none
};

// Sum over a row's lanes (16 or 8), the same in all of them.
template <int STEP>
__device__ __forceinline__ float moved_f(float x) {
  return __builtin_bit_cast(float, moved<STEP>(__builtin_bit_cast(uint32_t, x)));
}
template <int LANES>
__device__ __forceinline__ float lanes_sum(float v) {
  v += moved_f<0xB1>(v), v += moved_f<0x4E>(v), v += moved_f<0x141>(v);
  if constexpr (LANES == 16) v += moved_f<0x140>(v);
  return v;
}

// E neighbouring elements of a row argument, in its own bits; as floats; and back.
template <typename T, int E>
struct Raw {
  static constexpr int WORDS = E * (int)sizeof(T) / 4;
  uint32_t v[WORDS];
};
template <typename T, int E>
__device__ __forceinline__ Raw<T, E> load_raw(const T* p) {
  Raw<T, E> r;
  if constexpr (r.WORDS == 1) {
    r.v[0] = *reinterpret_cast<const uint32_t*>(p);
  } else {
    const Words<r.WORDS> w = load_words<r.WORDS>(p);
#pragma unroll
    for (int i = 0; i < r.WORDS; ++i) r.v[i] = w.v[i];
  }
  return r;
}
template <typename T, int E>
__device__ __forceinline__ void to_floats(const Raw<T, E>& r, float (&x)[E]) {
#pragma unroll
  for (int i = 0; i < E; i += 2) {
    if constexpr (sizeof(T) == 4)
      x[i] = __builtin_bit_cast(float, r.v[i]), x[i + 1] = __builtin_bit_cast(float, r.v[i + 1]);
    else
      unpack_pair<T>(r.v[i / 2], reinterpret_cast<float(&)[2]>(x[i]));
  }
}
template <int E>
__device__ __forceinline__ void store_some(void* p, int type, int64_t at, const float (&x)[E]) {
  if (type == NVQ_TYPE_F32) {
    Words<E> w;
#pragma unroll
    for (int i = 0; i < E; ++i) w.v[i] = __builtin_bit_cast(uint32_t, x[i]);
    store_words<E>(reinterpret_cast<float*>(p) + at, w);
  } else {
    uint32_t w[E / 2];
#pragma unroll
    for (int i = 0; i < E / 2; ++i) w[i] = type == NVQ_TYPE_F16 ? pack_pair<_Float16>(x[2 * i], x[2 * i + 1]) : pack_pair<__bf16>(x[2 * i], x[2 * i + 1]);
    uint16_t* d = reinterpret_cast<uint16_t*>(p) + at;
    if constexpr (E == 4)
      *reinterpret_cast<u32x2*>(d) = u32x2{w[0], w[1]};
    else
      *reinterpret_cast<uint32_t*>(d) = w[0];
  }
}

// How a row's pairs lie: neighbours; halves that lie HB blocks apart in the same lane (R = 64 HB); other halves,
// whose partners are read from memory once more.
constexpr int kNeighbours = 0, kApart = -1;

// T: the rows' type.  NB: 32-blocks of a row.  PAIR: kNeighbours, kApart or HB.
template <typename T, int NB, int PAIR>
__global__ __launch_bounds__(kThreads) void rope_kernel(Args a) {
  constexpr int E = PAIR == kApart ? 2 : 4;  // elements of a block that a lane has (halves end at multiples of 2)
  constexpr int LANES = 32 / E;              // of a row
  const RopeRows& r = a.r;
  // a workgroup takes queries, keys or values
  const int kind = (int)blockIdx.x < a.blocks[0] ? 0 : (int)blockIdx.x < a.blocks[1] ? 1 : 2;
  const uint32_t first = kind == 0 ? 0u : (uint32_t)a.blocks[kind - 1];
  const uint32_t id = (blockIdx.x - first) * (kThreads / LANES) + threadIdx.x / LANES;
  const uint32_t heads = r.heads[kind], t = id / heads, head = id - t * heads;
  if (t >= (uint32_t)a.T) return;  // a row's lanes leave together
  const int n = (int)(threadIdx.x % LANES);
  const T* p = reinterpret_cast<const T*>(r.in[kind]) + (int64_t)t * r.in_t[kind] + (int64_t)head * r.in_h[kind];
  const int half = r.rot / 2;
  const float* weight = kind < 2 ? r.weight[kind] : nullptr;
  const auto element = [&](int b) __attribute__((always_inline)) { return 32 * b + E * n; };
  const auto partner = [&](int b) __attribute__((always_inline)) {
    const int e = element(b);
    return e >= r.rot ? e : e < half ? e + half : e - half;
  };

  // Everything that is read goes out before anything is used: rows, weights, then what the position says.
  Raw<T, E> raw[NB], raw_y[PAIR == kApart ? NB : 1];
#pragma unroll
  for (int b = 0; b < NB; ++b) raw[b] = load_raw<T, E>(p + element(b));
  constexpr int TURNS = PAIR > 0 ? PAIR : NB, EACH = PAIR == kNeighbours ? E / 2 : E;
  float cos[TURNS][EACH], sin[TURNS][EACH];
  Words<E> w[NB];
  float w_y[PAIR == kApart ? NB : 1][2];
  if (kind < 2) {
    int at[4];
    at[0] = r.positions[t];
#pragma unroll
    for (int i = 1; i < 4; ++i) at[i] = i < r.axes ? r.positions[(int64_t)i * r.axis_stride + t] : -1;
    if constexpr (PAIR == kApart) {
#pragma unroll
      for (int b = 0; b < NB; ++b) raw_y[b] = load_raw<T, E>(p + partner(b));
    }
    if (weight) {
#pragma unroll
      for (int b = 0; b < NB; ++b) w[b] = load_words<E>(weight + element(b));
      if constexpr (PAIR == kApart) {
#pragma unroll
        for (int b = 0; b < NB; ++b) load_pair(weight + partner(b), w_y[b]);
      }
    }
    const auto row_of = [&](int place, int c) __attribute__((always_inline)) { return r.table + ((uint32_t)place < (uint32_t)r.n_pos ? (int64_t)place * r.rot : 0) + c; };
    const auto angles = [&](const float* row, int b) __attribute__((always_inline)) {
#pragma unroll
      for (int i = 0; i < EACH; i += 2) {  // (half is even, and no more in general)
        load_pair(row + i, reinterpret_cast<float(&)[2]>(cos[b][i]));
        load_pair(row + half + i, reinterpret_cast<float(&)[2]>(sin[b][i]));
      }
    };
    // the first pair of block b that the lane turns
    const auto pair_of = [&](int b) __attribute__((always_inline)) {
      const int e = element(b);
      return PAIR == kNeighbours ? e / 2 : PAIR > 0 || e < half ? e : e - half;
    };
    if (r.axes == 1) {
#pragma unroll
      for (int b = 0; b < TURNS; ++b)
        if (PAIR > 0 || element(b) < r.rot) angles(row_of(at[0], pair_of(b)), b);
      if ((uint32_t)at[0] >= (uint32_t)r.n_pos) {
#pragma unroll
        for (int b = 0; b < TURNS; ++b)
#pragma unroll
          for (int i = 0; i < EACH; ++i) cos[b][i] = sin[b][i] = __builtin_nanf("");
      }
    } else {
      const auto place_of = [&](int c) __attribute__((always_inline)) {
        const int x = c < r.ends[0] ? at[0] : at[1], y = c < r.ends[2] ? at[2] : at[3];
        return c < r.ends[1] ? x : y;
      };
      const auto axis_of = [&](int c) __attribute__((always_inline)) { return (c >= r.ends[0]) + (c >= r.ends[1]) + (c >= r.ends[2]); };
#pragma unroll
      for (int b = 0; b < TURNS; ++b) {
        if (PAIR <= 0 && element(b) >= r.rot) continue;
        const int c = pair_of(b);
        if (axis_of(c) == axis_of(c + EACH - 1)) {  // pairs of one section, as all are unless a section ends inside
          const int place = place_of(c);
          angles(row_of(place, c), b);
          if ((uint32_t)place >= (uint32_t)r.n_pos) {
#pragma unroll
            for (int i = 0; i < EACH; ++i) cos[b][i] = sin[b][i] = __builtin_nanf("");
          }
        } else {
#pragma unroll
          for (int i = 0; i < EACH; ++i) {
            const int place = place_of(c + i);
            const float* row = row_of(place, c + i);
            const bool in = (uint32_t)place < (uint32_t)r.n_pos;
            const float co = row[0], si = row[half];
            cos[b][i] = in ? co : __builtin_nanf(""), sin[b][i] = in ? si : __builtin_nanf("");
          }
        }
      }
    }
  }
  const int64_t slot = kind > 0 && a.fmt >= 0 ? a.slots[t] : 0;

  float x[NB][E];
#pragma unroll
  for (int b = 0; b < NB; ++b) to_floats<T, E>(raw[b], x[b]);
  if (kind < 2) {
    float y[PAIR == kApart ? NB : 1][E];
    if constexpr (PAIR == kApart) {
#pragma unroll
      for (int b = 0; b < NB; ++b) to_floats<T, E>(raw_y[b], y[b]);
    }
    if (weight) {
      const auto mean_square = [&](float eps) __attribute__((always_inline)) {
        float s = 0.0f;
#pragma unroll
        for (int b = 0; b < NB; ++b)
#pragma unroll
          for (int i = 0; i < E; ++i) s = __builtin_fmaf(x[b][i], x[b][i], s);
        return lanes_sum<LANES>(s) * (1.0f / (32 * NB)) + eps;
      };
      float mean = mean_square(r.eps);
      if (mean < 0x1p-100f) {  // squares that float32 may not hold (a row's lanes agree): elements, below 2^-46, times 2^100, eps by its square
#pragma unroll
        for (int b = 0; b < NB; ++b)
#pragma unroll
          for (int i = 0; i < E; ++i) {
            x[b][i] *= 0x1p100f;
            if constexpr (PAIR == kApart) y[b][i] *= 0x1p100f;
          }
        mean = mean_square(r.eps * 0x1p100f * 0x1p100f);
      }
      const float norm = __builtin_amdgcn_rsqf(mean);
#pragma unroll
      for (int b = 0; b < NB; ++b)
#pragma unroll
        for (int i = 0; i < E; ++i) {
          x[b][i] = x[b][i] * norm * __builtin_bit_cast(float, w[b].v[i]);
          if constexpr (PAIR == kApart) y[b][i] = y[b][i] * norm * w_y[b][i];
        }
    }
    if constexpr (PAIR == kNeighbours) {
#pragma unroll
      for (int b = 0; b < NB; ++b)
        if (element(b) < r.rot) {
#pragma unroll
          for (int i = 0; i < E; i += 2) {
            const float u = x[b][i], v = x[b][i + 1];
            x[b][i] = u * cos[b][i / 2] - v * sin[b][i / 2], x[b][i + 1] = v * cos[b][i / 2] + u * sin[b][i / 2];
          }
        }
    } else if constexpr (PAIR == kApart) {
#pragma unroll
      for (int b = 0; b < NB; ++b) {
        const int e = element(b);
        if (e < r.rot) {
#pragma unroll
          for (int i = 0; i < E; ++i) x[b][i] = e < half ? x[b][i] * cos[b][i] - y[b][i] * sin[b][i] : x[b][i] * cos[b][i] + y[b][i] * sin[b][i];
        }
      }
    } else {
#pragma unroll
      for (int b = 0; b < PAIR; ++b)
#pragma unroll
        for (int i = 0; i < E; ++i) {
          const float u = x[b][i], v = x[b + PAIR][i];
          x[b][i] = u * cos[b][i] - v * sin[b][i], x[b + PAIR][i] = v * cos[b][i] + u * sin[b][i];
        }
    }
  }
  if (kind == 0 || a.fmt < 0) {
    const int64_t to = (int64_t)t * r.out_t[kind & 1] + (int64_t)head * r.out_h[kind & 1];
#pragma unroll
    for (int b = 0; b < NB; ++b) store_some<E>(r.out[kind & 1], r.out_type, to + element(b), x[b]);
    return;
  }
  const int64_t page = slot >> a.c.page_shift, off = slot & ((int64_t(1) << a.c.page_shift) - 1);
  const int64_t row = ((page * heads + head) << a.c.page_shift) + off;
  const bool in = slot >= 0 && slot < a.n_slots;
  uint8_t* codes = reinterpret_cast<uint8_t*>(const_cast<void*>(kind == 1 ? a.c.k : a.c.v));
  if (a.fmt == NVQ_KV_Q8_0) {
    uint16_t code[E / 2 * NB], scale[NB];
#pragma unroll
    for (int b = 0; b < NB; ++b) {
      uint32_t top = 0;
#pragma unroll
      for (int i = 0; i < E; ++i) top = max(top, __builtin_bit_cast(uint32_t, x[b][i]) & 0x7FFFFFFFu);
      top = lanes_max<LANES>(top);
#pragma unroll
      for (int i = 0; i < E / 2; ++i) {
        const float two[2] = {x[b][2 * i], x[b][2 * i + 1]};
        code[i * NB + b] = quant_pair(two, top, scale[b]);
      }
    }
    if (in) {
      store_halves<E / 2 * NB>(codes + row * (32 * NB) + E * NB * n, code);
      if (n == 0) store_halves<NB>(reinterpret_cast<uint16_t*>(const_cast<void*>(kind == 1 ? a.c.k_d : a.c.v_d)) + row * NB, scale);
    }
  } else if (in) {
#pragma unroll
    for (int b = 0; b < NB; ++b) store_some<E>(codes, a.fmt == NVQ_KV_F16 ? NVQ_TYPE_F16 : NVQ_TYPE_BF16, row * (32 * NB) + element(b), x[b]);
  }
}

template <typename T, int NB, int PAIR>
void launch_pair(Args& a, hipStream_t s) {
  constexpr int64_t kRows = PAIR == kApart ? kThreads / 16 : kThreads / 8;
  int64_t blocks = 0;
  for (int i = 0; i < 3; ++i) {
    blocks += ((int64_t)a.T * a.r.heads[i] + kRows - 1) / kRows;
    if (i < 2) a.blocks[i] = (int)blocks;
  }
  hipLaunchKernelGGL((rope_kernel<T, NB, PAIR>), dim3((unsigned)blocks), dim3(kThreads), 0, s, a);
}
template <typename T, int NB>
void launch_nb(Args& a, hipStream_t s) {
  if (a.r.neighbours) return launch_pair<T, NB, kNeighbours>(a, s);
  if constexpr (NB % 2 == 0) {
    if (a.r.rot == 32 * NB) return launch_pair<T, NB, NB / 2>(a, s);
  }
  if constexpr (NB % 4 == 0) {
    if (a.r.rot == 16 * NB) return launch_pair<T, NB, NB / 4>(a, s);
  }
  launch_pair<T, NB, kApart>(a, s);
}
template <typename T>
void launch_type(Args& a, int nb, hipStream_t s) {
  switch (nb) {
    case 1: return launch_nb<T, 1>(a, s);
    case 2: return launch_nb<T, 2>(a, s);
    case 3: return launch_nb<T, 3>(a, s);
    case 4: return launch_nb<T, 4>(a, s);
    case 5: return launch_nb<T, 5>(a, s);
    case 6: return launch_nb<T, 6>(a, s);
    case 7: return launch_nb<T, 7>(a, s);
    default: return launch_nb<T, 8>(a, s);
  }
}

size_t bytes_of(int type) { return type == NVQ_TYPE_F32 ? 4 : 2; }

}  // namespace

hipError_t launch_rope(const RopeRows& rows, int64_t T, int64_t D, int fmt, const KvCache* c, const int64_t* slots, hipStream_t stream) {
  Args a;
  a.r = rows;
  a.fmt = fmt;
  a.c = c ? *c : KvCache{};
  a.n_slots = c ? c->n_pages << c->page_shift : 0;
  // a launch takes fewer than 2^32 threads, 16 to a row at most, and up to a workgroup more for each kind: longer
  // calls go in pieces
  const int64_t most = ((int64_t(1) << 28) - 64) / (rows.heads[0] + rows.heads[1] + rows.heads[2]);
  for (int64_t t = 0; t < T; t += most) {
    a.T = (int)(T - t < most ? T - t : most);
    for (int w = 0; w < 3; ++w)
      if (rows.in[w]) a.r.in[w] = (const char*)rows.in[w] + t * rows.in_t[w] * (int64_t)bytes_of(rows.type);
    for (int w = 0; w < 2; ++w)
      if (rows.out[w]) a.r.out[w] = (char*)rows.out[w] + t * rows.out_t[w] * (int64_t)bytes_of(rows.out_type);
    a.r.positions = rows.positions + t;
    a.slots = slots ? slots + t : nullptr;
    if (rows.type == NVQ_TYPE_F32)
      launch_type<float>(a, (int)(D / 32), stream);
    else if (rows.type == NVQ_TYPE_F16)
      launch_type<_Float16>(a, (int)(D / 32), stream);
    else
      launch_type<__bf16>(a, (int)(D / 32), stream);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

}  // namespace nvq
