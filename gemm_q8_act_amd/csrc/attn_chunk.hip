// attn_chunk.hip -- causal attention of several new tokens per sequence over the paged key-value
// cache that holds them and everything before them, on gfx950:
//     out[i][h] = sum_j p_ij v_j / sum_j p_ij,  p_ij = exp(scale q[i][h] . k[j][h / G]),
// where query i of the m new ones among n keys stands at place p = i + n - m and sees keys j <= p,
// with a window those of j > p - window and the first `sinks` only.
//
// A row of the work is one query of one head; the G query heads of a key head read the same keys,
// so a workgroup takes 128 rows (query, head) of a key head, a wavefront 32 of them, and
// walks the keys in tiles of 64 with a running maximum and sum.  Both products are
// v_mfma_f32_32x32x16 with rows as columns:
//     S^T [keys][32 rows] = K Q^T,      O^T [D][32 rows] += V^T P^T
// Few rows behind many keys are split over workgroups by keys and joined in order by a second kernel.
//
// Q8_0.  Codes times scales, rounded to binary16's 11 bits, are the operands, with one power of two a
// tile taken out of the scales: scores take it back, the accumulator is held in units of the
// largest value power so far.  A row's channels keep the cache's order (interleaved over its
// blocks), which is as good as any for the contraction: queries and results are permuted instead.
#include "attn_tiles.h"
#include "nvq_launch.h"

namespace nvq {

namespace {

constexpr int kWaves = kTileWaves;
constexpr int kRows = 32 * kWaves;  // of a workgroup
constexpr int kMinPart = 2;         // tiles: the shortest part
constexpr int kTargetGroups = 512;

struct ChunkArgs {
  const uint16_t* q;
  uint16_t* out;
  int64_t q_t, q_h, o_t, o_h;  // token and head strides, elements
  KvCache c;
  const int32_t *table, *cu_q, *lengths;
  float* acc;   // [slot * key heads][slot_waves][D/32][4][64 lanes] float4
  float* stat;  // [slot * key heads][2][128]: maximum (base 2), sum
  float scale_log2;  // not negative; the sign is in flip
  uint32_t flip;     // sign bits of a query pair
  int table_stride;  // pages of a table row
  int B, Hq, Hkv, G, Tq;
  int window, sinks;
  int type;
  int target;      // parts wanted of a key head
  int slot_waves;  // wavefronts' rows that a part's slot holds
};

// Tiles that the 128 rows of one workgroup see of n keys, at most: with a window, those of the first keys, and of
// the windows of up to 128 queries.
__device__ __forceinline__ int tiles_seen(const ChunkArgs& a, int n) {
  const int all = (n + kKeys - 1) / kKeys;
  return min(all, (min(a.sinks, n) + kKeys - 1) / kKeys + (a.window + kRows - 1 + kKeys - 1) / kKeys + 1);
}

struct Seq {
  int q0, m, n;    // first query, number of them, and keys (0 if out of range, and bad is set)
  int tiles, most; // row tiles; key tiles of one of them, at most
  bool bad;
};
__device__ __forceinline__ Seq load_seq(const ChunkArgs& a, int i) {
  Seq s = {0, 0, 0, 0, 0, false};
  if (i < a.B) {
    int lo = a.cu_q[i], hi = a.cu_q[i + 1];
    const int n = a.lengths[i];
    lo = min(max(lo, 0), a.Tq), hi = min(max(hi, lo), a.Tq);
    s.q0 = lo, s.m = hi - lo;
    s.bad = n < 0 || n > (a.table_stride << a.c.page_shift);
    s.n = s.bad ? 0 : n;
    s.tiles = (int)(((uint32_t)s.m * (uint32_t)a.G + kRows - 1) / kRows);
    s.most = tiles_seen(a, s.n);
  }
  return s;
}

// How the work is cut: the key tiles of a row tile go in parts of `part_tiles`, of a length for the whole
// call that makes about `target` parts of a key head.
struct Work {
  Seq s;
  int b;            // sequence, -1: no such work
  int tile;         // row tile of it
  int part;         // part of the tile (main kernel)
  int parts;        // parts that its row tiles have at most
  int part_tiles;
  int slot;         // of the part, or of the row tile's first part; -1: the sequence is not split
};

// join: `want` counts the row tiles of split sequences, else all parts.  A sequence's last row tiles, which see
// the most keys, come first.
__device__ __forceinline__ Work find_work(const ChunkArgs& a, int want, bool join) {
  const int lane = (int)(threadIdx.x & 63);
  int total = 0;  // (below 2^31: host check)
  for (int i = lane; i - lane < a.B; i += 64) {
    const Seq s = load_seq(a, i);
    total += s.tiles * s.most;
  }
  total = __builtin_amdgcn_readlane(wave_running_sum(total), 63);
  Work w;
  w.part_tiles = max(kMinPart, (int)(((uint32_t)total + (uint32_t)a.target - 1) / (uint32_t)a.target));
  w.b = -1;
  int base = 0, slots = 0;
  for (int i0 = 0; i0 < a.B; i0 += 64) {
    const Seq s = load_seq(a, i0 + lane);
    const int parts = max(1, (s.most + w.part_tiles - 1) / w.part_tiles);
    const int taken = parts > 1 ? s.tiles * parts : 0;
    const int mine = join ? (parts > 1 ? s.tiles : 0) : s.tiles * parts;
    const int incl = wave_running_sum(mine), incl_slots = wave_running_sum(taken);
    const uint64_t hit = __ballot(base + incl > want);
    if (hit) {
      const int l = __builtin_ctzll(hit);
      const auto of = [&](int v) { return __builtin_amdgcn_readlane(v, l); };
      w.b = i0 + l;
      w.s = {of(s.q0), of(s.m), of(s.n), of(s.tiles), of(s.most), of((int)s.bad) != 0};
      w.parts = of(parts);
      const int at = want - (base + of(incl) - of(mine));
      const int turn = join ? at : at / w.parts;
      w.part = join ? 0 : at - turn * w.parts;
      w.tile = w.s.tiles - 1 - turn;
      w.slot = w.parts > 1 ? slots + of(incl_slots) - of(taken) + turn * w.parts + w.part : -1;
      return w;
    }
    base += __builtin_amdgcn_readlane(incl, 63);
    slots += __builtin_amdgcn_readlane(incl_slots, 63);
  }
  return w;
}

// A row tile: its rows and what they see.
struct Rows {
  int r0, count;  // first row, rows
  int first, last;  // places of its first and last query
  int end;        // keys below it are seen by some row
  int start, sink;  // keys from `start` on are in some row's window, those below `sink` are first ones
  int sink_tiles, skip;  // tiles with first ones; tiles between them and the windows
  int tiles;      // key tiles
};
__device__ __forceinline__ Rows rows_of(const ChunkArgs& a, const Work& w) {
  Rows r;
  const int rows = w.s.m * a.G, shift = w.s.n - w.s.m;
  r.r0 = w.tile * kRows;
  r.count = min(kRows, rows - r.r0);
  r.first = r.r0 / a.G + shift, r.last = (r.r0 + r.count - 1) / a.G + shift;
  r.end = min(max(r.last + 1, 0), w.s.n);
  r.start = max(r.first - a.window + 1, 0);
  r.sink = min(a.sinks, r.start);
  r.sink_tiles = (r.sink + kKeys - 1) / kKeys;
  r.skip = max(r.start / kKeys - r.sink_tiles, 0);
  r.tiles = max((r.end + kKeys - 1) / kKeys - r.skip, 0);
  return r;
}

template <int FMT, int NB>
struct Cached {
  static constexpr bool Q8 = FMT == NVQ_KV_Q8_0;
  static constexpr int ROW = Q8 ? 32 * NB : 64 * NB;  // bytes of a cache row
  static constexpr int WORDS = ROW / 16;              // dwords that a lane stages of it (4 lanes to a row)
  static constexpr int SCALES = Q8 ? NB : 1;
};

// The channel of place p of a row's order in the cache
template <bool Q8, int NB>
__device__ __forceinline__ int channel_of(int p) {
  if constexpr (!Q8) return p;
  const int pair = p >> 1;
  return 32 * (pair % NB) + 2 * (pair / NB) + (p & 1);
}

// N dwords of a buffer from a byte offset that is a multiple of 4 N up to 16
template <int N>
__device__ __forceinline__ void load_dwords(__amdgpu_buffer_rsrc_t r, uint32_t at, uint32_t* v) {
  if constexpr (N % 4 == 0) {
#pragma unroll
    for (int i = 0; i < N / 4; ++i) {
      const u32x4 t = __builtin_bit_cast(u32x4, __builtin_amdgcn_raw_buffer_load_b128(r, at + 16 * i, 0, 0));
#pragma unroll
      for (int j = 0; j < 4; ++j) v[4 * i + j] = t[j];
    }
  } else {
    static_assert(N % 2 == 0, "pairs of dwords");
#pragma unroll
    for (int i = 0; i < N / 2; ++i) {
      const u32x2 t = __builtin_bit_cast(u32x2, __builtin_amdgcn_raw_buffer_load_b64(r, at + 8 * i, 0, 0));
      v[2 * i] = t[0], v[2 * i + 1] = t[1];
    }
  }
}

// Which of a pair of 16-bit elements are not finite: their bits set
template <typename T>
__device__ __forceinline__ uint32_t not_finite(uint32_t w) {
  constexpr uint32_t e = __is_same(T, _Float16) ? 0x7C00u : 0x7F80u;
  return ((w & e) == e ? 0xFFFFu : 0u) | (((w >> 16) & e) == e ? 0xFFFF0000u : 0u);
}

// Largest of a wavefront's unsigned values
__device__ __forceinline__ uint32_t wave_umax(uint32_t v) {
#pragma unroll
  for (int step = 1; step < 64; step *= 2) v = max(v, (uint32_t)__shfl_xor((int)v, step));
  return v;
}

template <typename T, int FMT, int NB>
__global__ __launch_bounds__(64 * kWaves, NB <= 4 ? 2 : 1) void attn_chunk_kernel(ChunkArgs a) {
  typedef Stage<NB> S;
  typedef Cached<FMT, NB> C;
  __shared__ __align__(16) uint8_t s_keys[S::BYTES], s_values[S::BYTES];
  __shared__ uint32_t s_top[2][kWaves];   // largest key and value scale of each group of the tile
  __shared__ uint64_t s_broken[kWaves];   // lanes whose part of a value row is not finite
  __shared__ int s_bad;                   // a page number outside the cache
  const int tid = (int)threadIdx.x, lane = tid & 63, c = lane & 31, hi = lane >> 5;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int kvh = (int)blockIdx.x % a.Hkv;
  const Work w = find_work(a, (int)blockIdx.x / a.Hkv, false);
  if (w.b < 0) return;
  const Rows rt = rows_of(a, w);
  const int t_begin = w.part * w.part_tiles, t_end = min(rt.tiles, t_begin + w.part_tiles);
  const bool split = rt.tiles > w.part_tiles;
  if (w.part > 0 && t_begin >= rt.tiles) return;
  if (tid == 0) s_bad = 0;

  // the lane's row
  const int rows = w.s.m * a.G, r = rt.r0 + 32 * wave + c;
  const bool mine = 32 * wave < rt.count, live = r < rows;
  const int rr = min(r, rows - 1), qi = rr / a.G, head = kvh * a.G + rr - qi * a.G;
  const int place = qi + w.s.n - w.s.m;
  const int place_first = __builtin_amdgcn_readlane(place, 0), place_last = __builtin_amdgcn_readlane(place, 31);
  const auto seen = [&](int key) __attribute__((always_inline)) { return key <= place && (key > place - a.window || key < a.sinks); };

  // its query, 16 places of the row's order at a time
  Frag qf[2 * NB];
  float to_log2 = a.scale_log2;
  {
    const uint16_t* row = a.q + (int64_t)(w.s.q0 + qi) * a.q_t + (int64_t)head * a.q_h;
    float top = 0.0f;
#pragma unroll
    for (int ks = 0; ks < 2 * NB; ++ks)
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        qf[ks].v[j] = *reinterpret_cast<const uint32_t*>(row + channel_of<C::Q8, NB>(16 * ks + 8 * hi + 2 * j)) ^ a.flip;
        if constexpr (C::Q8) {
          float x[2];
          unpack_pair<__bf16>(qf[ks].v[j], x);
          top = fmaxf(top, fmaxf(fabsf(x[0]), fabsf(x[1])));
        }
      }
    if constexpr (C::Q8) {
      if (a.type == NVQ_TYPE_BF16) {
        // bfloat16 into binary16 operands: scaled to 2^7 .. 2^8, exact down to 2^-32 of the largest
        top = max_32(top);
        const int e = top > 0.0f && top < __builtin_inff() ? 8 - __builtin_amdgcn_frexp_expf(top) : 0;
#pragma unroll
        for (int ks = 0; ks < 2 * NB; ++ks)
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            float x[2];
            unpack_pair<__bf16>(qf[ks].v[j], x);
            qf[ks].v[j] = pack_pair<_Float16>(__builtin_amdgcn_ldexpf(x[0], e), __builtin_amdgcn_ldexpf(x[1], e));
          }
        to_log2 = __builtin_amdgcn_ldexpf(to_log2, -e);
      }
    }
  }

  // One 16-key group of a tile, from its page: the wavefront stages it, 4 lanes to a row.
  const auto* table = (const __attribute__((address_space(4))) int32_t*)(a.table + (int64_t)w.b * a.table_stride);
  const int page_mask = (1 << a.c.page_shift) - 1;
  const auto tile_key = [&](int t) __attribute__((always_inline)) { return (t < rt.sink_tiles ? t : t + rt.skip) * kKeys; };
  const int row_in = lane >> 2, seg = lane & 3;
  bool bad_page = false;
  uint32_t kw[C::WORDS], vw[C::WORDS];
  uint16_t kd[C::SCALES], vd[C::SCALES];
  const auto load = [&](int t) __attribute__((always_inline)) {
    const int key0 = tile_key(t) + 16 * wave;
    int count = min(max(rt.end - key0, 0), 16);
    if (key0 + 15 < rt.start && key0 >= rt.sink) count = 0;  // no row sees any of it
    const int page = count > 0 ? table[key0 >> a.c.page_shift] : 0;
    const bool out = (uint32_t)page >= (uint32_t)a.c.n_pages;
    bad_page |= out;
    if (out) count = 0;
    const int64_t row = (((int64_t)(out ? 0 : page) * a.Hkv + kvh) << a.c.page_shift) + (key0 & page_mask);
    const auto buffer = [&](const void* p, int bytes) __attribute__((always_inline)) {
      return __builtin_amdgcn_make_buffer_rsrc((void*)(reinterpret_cast<const uint8_t*>(p) + row * bytes), 0, count * bytes, 0x00020000);
    };
    const auto k = buffer(a.c.k, C::ROW), v = buffer(a.c.v, C::ROW);
    if constexpr (C::Q8) {
      load_dwords<C::WORDS>(k, row_in * C::ROW + seg * (C::ROW / 4), kw);
      load_dwords<C::WORDS>(v, row_in * C::ROW + seg * (C::ROW / 4), vw);
      const auto kds = buffer(a.c.k_d, 2 * NB), vds = buffer(a.c.v_d, 2 * NB);
#pragma unroll
      for (int b = 0; b < NB; ++b) {
        kd[b] = (uint16_t)__builtin_amdgcn_raw_buffer_load_b16(kds, 2 * (row_in * NB + b), 0, 0);
        vd[b] = (uint16_t)__builtin_amdgcn_raw_buffer_load_b16(vds, 2 * (row_in * NB + b), 0, 0);
      }
    } else {
#pragma unroll
      for (int i = 0; i < NB; ++i) {
        load_dwords<4>(k, row_in * C::ROW + 16 * (4 * i + seg), kw + 4 * i);
        load_dwords<4>(v, row_in * C::ROW + 16 * (4 * i + seg), vw + 4 * i);
      }
    }
  };
  // Q8_0: the exponents of the tile's largest scales, from all wavefronts
  const auto publish = [&]() __attribute__((always_inline)) {
    if constexpr (C::Q8) {
      const auto top = [&](const uint16_t (&d)[C::SCALES]) __attribute__((always_inline)) {
        uint32_t x = 0;
#pragma unroll
        for (int b = 0; b < NB; ++b) {
          const uint32_t u = d[b] & 0x7FFFu;
          x = max(x, u < 0x7C00u ? u : 0u);
        }
        return wave_umax(x);
      };
      const uint32_t k = top(kd), v = top(vd);
      if (lane == 0) s_top[0][wave] = k, s_top[1][wave] = v;
    }
  };
  const auto top_exponent = [&](int which) __attribute__((always_inline)) {  // frexp's, or a large negative for all zero
    uint32_t x = 0;
#pragma unroll
    for (int i = 0; i < kWaves; ++i) x = max(x, s_top[which][i]);
    return x ? __builtin_amdgcn_frexp_expf(f16_bits_to_f32((uint16_t)x)) : -1000;
  };
  // A lane's part of a row into the tile.
  const auto stage = [&](uint8_t* tile, const uint32_t (&raw)[C::WORDS], const uint16_t (&d)[C::SCALES], int e, bool keys) __attribute__((always_inline)) {
    const int row = 16 * wave + row_in;
    half2_t f[C::SCALES];
    if constexpr (C::Q8) {
#pragma unroll
      for (int b = 0; b < NB; ++b) {
        const _Float16 x = (_Float16)__builtin_amdgcn_ldexpf(f16_bits_to_f32(d[b]), -e);
        f[b] = half2_t{x, x};
      }
    }
#pragma unroll
    for (int i = 0; i < NB; ++i) {
      u32x4 x;
      const int piece = C::Q8 ? NB * seg + i : 4 * i + seg;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        if constexpr (C::Q8) {
          const int pair = 4 * i + j;
          const uint32_t u = perm(0x64646464u, raw[pair / 2] ^ 0x80808080u, pair & 1 ? 0x04030402u : 0x04010400u);
          x[j] = __builtin_bit_cast(uint32_t, (__builtin_bit_cast(half2_t, u) - half2_t{(_Float16)1152.0f, (_Float16)1152.0f}) * f[pair % NB]);
        } else {
          x[j] = raw[4 * i + j];
        }
      }
      *reinterpret_cast<u32x4*>(tile + row * S::ROW + 16 * (keys ? S::key_piece(row, piece) : S::value_piece(row, piece))) = x;
    }
  };

  floatx16 acc[NB];
#pragma unroll
  for (int d = 0; d < NB; ++d)
#pragma unroll
    for (int j = 0; j < 16; ++j) acc[d][j] = 0.0f;
  float m = -__builtin_inff(), l = 0.0f;
  constexpr int kUnset = -10000;
  int unit = kUnset;  // Q8_0: the accumulator is in units of 2^unit

  uint32_t key_offset[2 * NB], value_offset[NB];
#pragma unroll
  for (int ks = 0; ks < 2 * NB; ++ks) key_offset[ks] = (uint32_t)(c * S::ROW + 16 * S::key_piece(c, 2 * ks + hi));
  {
    const int jj = lane & 15, in = 4 * hi + (jj >> 2), half = (lane >> 4) & 1;
#pragma unroll
    for (int d = 0; d < NB; ++d) value_offset[d] = (uint32_t)(in * S::ROW + 16 * S::value_piece(in, 4 * d + 2 * half + ((jj & 3) >> 1)) + 8 * (jj & 1));
  }

  if (t_begin < t_end) load(t_begin);
  for (int t = t_begin; t < t_end; ++t) {
    const int key0 = tile_key(t);
    const bool partly = key0 + kKeys - 1 > rt.first || (key0 <= rt.last - a.window && key0 + kKeys - 1 >= a.sinks);  // some row does not see some key
    publish();
    __syncthreads();  // everyone is done with the last tile
    int ek = 0, ev = 0;
    if constexpr (C::Q8) {
      ek = top_exponent(0);
      ek = ek > -1000 ? ek - 5 : 0;
      const int x = top_exponent(1);
      if (x > -1000 && (unit == kUnset || x - unit > 9)) {
        if (unit != kUnset) {
          const float f = __builtin_amdgcn_ldexpf(1.0f, unit - (x - 5));
#pragma unroll
          for (int d = 0; d < NB; ++d) acc[d] *= f;
        }
        unit = x - 5;
      }
      ev = unit == kUnset ? 0 : unit;
    }
    if (partly) {
      // what is not finite in a value row must not meet a probability of 0 in rows that do not see it: it
      // stays out of the tile, and rows that see it get it below
      bool broken = false;
      if constexpr (C::Q8) {
#pragma unroll
        for (int b = 0; b < NB; ++b) broken |= (vd[b] & 0x7C00u) == 0x7C00u;
      } else {
#pragma unroll
        for (int i = 0; i < C::WORDS; ++i) broken |= not_finite<T>(vw[i]) != 0;
      }
      const uint64_t any = __ballot(broken);
      if (lane == 0) s_broken[wave] = any;
      if (any) {
        if constexpr (C::Q8) {
#pragma unroll
          for (int b = 0; b < NB; ++b) vd[b] = (vd[b] & 0x7C00u) == 0x7C00u ? 0 : vd[b];
        } else {
#pragma unroll
          for (int i = 0; i < C::WORDS; ++i) vw[i] &= ~not_finite<T>(vw[i]);
        }
      }
    }
    stage(s_keys, kw, kd, ek, true);
    stage(s_values, vw, vd, ev, false);
    if (t + 1 < t_end) load(t + 1);
    __syncthreads();
    if (!mine) continue;

    floatx16 s[2];
#pragma unroll
    for (int kb = 0; kb < 2; ++kb)
#pragma unroll
      for (int j = 0; j < 16; ++j) s[kb][j] = 0.0f;
#pragma unroll
    for (int ks = 0; ks < 2 * NB; ++ks)
#pragma unroll
      for (int kb = 0; kb < 2; ++kb) {
        const u32x4 x = *reinterpret_cast<const u32x4*>(s_keys + key_offset[ks] + 32 * kb * S::ROW);
        s[kb] = mfma32<T>(Frag{x[0], x[1], x[2], x[3]}, qf[ks], s[kb]);
      }
    // (not 0, which would make NaN of a masked score)
    const float factor = C::Q8 ? fmaxf(__builtin_amdgcn_ldexpf(to_log2, ek), 1e-37f) : to_log2;
    if (key0 + kKeys - 1 > place_first || (key0 <= place_last - a.window && key0 + kKeys - 1 >= a.sinks)) {
#pragma unroll
      for (int kb = 0; kb < 2; ++kb)
#pragma unroll
        for (int j = 0; j < 16; ++j)
          if (!seen(key0 + 32 * kb + 8 * (j >> 2) + 4 * hi + (j & 3))) s[kb][j] = -__builtin_inff();
    }
    float top = s[0][0];
#pragma unroll
    for (int kb = 0; kb < 2; ++kb)
#pragma unroll
      for (int j = 0; j < 16; ++j) top = fmaxf(top, s[kb][j]);
    top *= factor;
    if (__any(top > m + Range<T>::SLACK)) {
      const float m_new = fmaxf(m, max_32(top));
      const float f = m_new == -__builtin_inff() ? 1.0f : exp2_fast(m - m_new);
      l *= f;
#pragma unroll
      for (int d = 0; d < NB; ++d) acc[d] *= f;
      m = m_new;
    }
    const float base = score_base<T>(m);
    Frag pf[2][2];
#pragma unroll
    for (int kb = 0; kb < 2; ++kb)
#pragma unroll
      for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const float x = exp2_fast(__builtin_fmaf(s[kb][8 * h + 2 * j], factor, -base));
          const float y = exp2_fast(__builtin_fmaf(s[kb][8 * h + 2 * j + 1], factor, -base));
          pf[kb][h].v[j] = pack_pair<T>(x, y);
          l = add_pair<T>(pf[kb][h].v[j], l);
        }
#pragma unroll
    for (int kb = 0; kb < 2; ++kb)
#pragma unroll
      for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int d = 0; d < NB; ++d) {
          Frag f;
#pragma unroll
          for (int x = 0; x < 2; ++x) {
            const u32x2 y = read_transposed(s_values + value_offset[d] + (32 * kb + 16 * h + 8 * x) * S::ROW);
            f.v[2 * x] = y[0], f.v[2 * x + 1] = y[1];
          }
          acc[d] = mfma32<T>(f, pf[kb][h], acc[d]);
        }
    if (partly) {
      for (int g = 0; g < kWaves; ++g)
        for (uint64_t any = s_broken[g]; any;) {
          const int row4 = __builtin_ctzll(any) >> 2, key = key0 + 16 * g + row4;
          any &= ~(uint64_t(15) << (4 * row4));
          const int64_t row = (((int64_t)table[key >> a.c.page_shift] * a.Hkv + kvh) << a.c.page_shift) + (key & page_mask);
          if (!seen(key)) continue;
#pragma unroll
          for (int d = 0; d < NB; ++d)
#pragma unroll
            for (int j = 0; j < 16; ++j) {
              const int at = 32 * d + 8 * (j >> 2) + 4 * hi + (j & 3);
              if constexpr (C::Q8) {
                const uint16_t x = reinterpret_cast<const uint16_t*>(a.c.v_d)[row * NB + (at >> 1) % NB];
                if ((x & 0x7C00u) == 0x7C00u) acc[d][j] = __builtin_nanf("");
              } else {
                const uint16_t x = reinterpret_cast<const uint16_t*>(a.c.v)[row * (32 * NB) + at];
                if (not_finite<T>(x) & 0xFFFFu) acc[d][j] += (float)__builtin_bit_cast(T, x);
              }
            }
        }
    }
  }
  if (bad_page) s_bad = 1;
  __syncthreads();
  if (!mine) return;
  l = sum_32(l);
  if (s_bad || w.s.bad) l = __builtin_nanf("");
  if (C::Q8 && unit != kUnset) {
    const float f = __builtin_amdgcn_ldexpf(1.0f, unit);
#pragma unroll
    for (int d = 0; d < NB; ++d) acc[d] *= f;
  }
  if (split) {
    const int64_t slot = (int64_t)w.slot * a.Hkv + kvh;
    floatx4* dst = reinterpret_cast<floatx4*>(a.acc) + (slot * a.slot_waves + wave) * (NB * 4 * 64) + lane;
#pragma unroll
    for (int d = 0; d < NB; ++d)
#pragma unroll
      for (int j = 0; j < 4; ++j) dst[(4 * d + j) * 64] = floatx4{acc[d][4 * j], acc[d][4 * j + 1], acc[d][4 * j + 2], acc[d][4 * j + 3]};
    if (hi == 0) {
      a.stat[slot * (2 * kRows) + 32 * wave + c] = m;
      a.stat[slot * (2 * kRows) + kRows + 32 * wave + c] = l;
    }
    return;
  }
  if (!live) return;
  const float inv = l == 0.0f ? 0.0f : 1.0f / l;  // a query that sees no key gives zeros
  uint16_t* row = a.out + (int64_t)(w.s.q0 + qi) * a.o_t + (int64_t)head * a.o_h;
#pragma unroll
  for (int d = 0; d < NB; ++d)
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const float x = acc[d][2 * j] * inv, y = acc[d][2 * j + 1] * inv;
      const int at = channel_of<C::Q8, NB>(32 * d + 8 * (j >> 1) + 4 * hi + 2 * (j & 1));
      *reinterpret_cast<uint32_t*>(row + at) = a.type == NVQ_TYPE_F16 ? pack_pair<_Float16>(x, y) : pack_pair<__bf16>(x, y);
    }
}

// Joins the parts of one row tile of a key head in their order: a workgroup takes 32 channels of its rows.
template <int FMT, int NB>
__global__ __launch_bounds__(64 * kWaves) void attn_chunk_join_kernel(ChunkArgs a) {
  typedef Cached<FMT, NB> C;
  const int tid = (int)threadIdx.x, lane = tid & 63, c = lane & 31, hi = lane >> 5;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int kvh = (int)blockIdx.x % a.Hkv, d = (int)blockIdx.y;
  const Work w = find_work(a, (int)blockIdx.x / a.Hkv, true);
  if (w.b < 0) return;
  const Rows rt = rows_of(a, w);
  const int parts = (rt.tiles + w.part_tiles - 1) / w.part_tiles;
  if (parts <= 1 || 32 * wave >= rt.count) return;
  floatx4 acc[4];
#pragma unroll
  for (int j = 0; j < 4; ++j) acc[j] = floatx4{0.f, 0.f, 0.f, 0.f};
  float sum = 0.0f, top = -__builtin_inff();
  for (int i = 0; i < parts; ++i) {
    const int64_t slot = (int64_t)(w.slot + i) * a.Hkv + kvh;
    const floatx4* src = reinterpret_cast<const floatx4*>(a.acc) + (slot * a.slot_waves + wave) * (NB * 4 * 64) + 4 * d * 64 + lane;
    const float m = a.stat[slot * (2 * kRows) + 32 * wave + c], l = a.stat[slot * (2 * kRows) + kRows + 32 * wave + c];
    const float m_new = fmaxf(top, m);
    const float f = top == -__builtin_inff() ? 0.0f : exp2_fast(top - m_new), g = m == -__builtin_inff() ? 0.0f : exp2_fast(m - m_new);
    sum = sum * f + l * g;  // (a part that sees no key holds zeros; a NaN stays one)
#pragma unroll
    for (int j = 0; j < 4; ++j) acc[j] = acc[j] * f + src[j * 64] * g;
    top = m_new;
  }
  const int r = rt.r0 + 32 * wave + c;
  if (r >= w.s.m * a.G) return;
  const int qi = r / a.G, head = kvh * a.G + r - qi * a.G;
  const float inv = sum == 0.0f ? 0.0f : 1.0f / sum;
  uint16_t* row = a.out + (int64_t)(w.s.q0 + qi) * a.o_t + (int64_t)head * a.o_h;
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    const float x = acc[j >> 1][2 * (j & 1)] * inv, y = acc[j >> 1][2 * (j & 1) + 1] * inv;
    const int at = channel_of<C::Q8, NB>(32 * d + 8 * (j >> 1) + 4 * hi + 2 * (j & 1));
    *reinterpret_cast<uint32_t*>(row + at) = a.type == NVQ_TYPE_F16 ? pack_pair<_Float16>(x, y) : pack_pair<__bf16>(x, y);
  }
}

// What the host knows of the work's size.
struct Bound {
  int64_t tiles;   // row tiles of a key head
  int64_t keys;    // key tiles of one
  int64_t target;  // parts wanted
  int64_t parts;   // parts at most
  int64_t slots;   // of them of split row tiles
  int slot_waves;
};
Bound bound_of(int64_t B, int64_t Tq, int64_t Hq, int64_t Hkv, int64_t capacity, int64_t window, int64_t sinks) {
  Bound b;
  const int64_t G = Hq / Hkv;
  b.tiles = Tq * G / kRows + B;
  b.keys = (capacity + kKeys - 1) / kKeys;
  if (window) {
    const int64_t seen = (sinks + kKeys - 1) / kKeys + (window + kRows - 1 + kKeys - 1) / kKeys + 1;
    b.keys = seen < b.keys ? seen : b.keys;
  }
  b.target = kTargetGroups / Hkv < 1 ? 1 : kTargetGroups / Hkv;
  // a sequence of `tiles` row tiles that see up to `most` key tiles is cut into tiles * ceil(most / part), and part is at
  // least sum(tiles * most) / target
  const int64_t each = (b.keys + kMinPart - 1) / kMinPart, all = b.tiles * each;
  b.parts = all < b.target + b.tiles ? all : b.target + b.tiles;
  b.slots = each <= 1 ? 0 : all < 2 * b.target ? all : 2 * b.target;
  const int64_t rows = Tq * G < kRows ? Tq * G : kRows;
  b.slot_waves = (int)((rows + 31) / 32);
  return b;
}

template <typename T, int FMT, int NB>
hipError_t launch_nb(const ChunkArgs& a, const Bound& b, hipStream_t s) {
  hipLaunchKernelGGL((attn_chunk_kernel<T, FMT, NB>), dim3((unsigned)(b.parts * a.Hkv)), dim3(64 * kWaves), 0, s, a);
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess || b.slots == 0) return e;
  const int64_t tiles = b.slots / 2 < b.tiles ? b.slots / 2 : b.tiles;  // two parts at least to each
  hipLaunchKernelGGL((attn_chunk_join_kernel<FMT, NB>), dim3((unsigned)(tiles * a.Hkv), NB), dim3(64 * kWaves), 0, s, a);
  return hipGetLastError();
}
template <typename T, int FMT>
hipError_t launch_fmt(const ChunkArgs& a, int nb, const Bound& b, hipStream_t s) {
  switch (nb) {
    case 1: return launch_nb<T, FMT, 1>(a, b, s);
    case 2: return launch_nb<T, FMT, 2>(a, b, s);
    case 3: return launch_nb<T, FMT, 3>(a, b, s);
    case 4: return launch_nb<T, FMT, 4>(a, b, s);
    case 5: return launch_nb<T, FMT, 5>(a, b, s);
    case 6: return launch_nb<T, FMT, 6>(a, b, s);
    case 7: return launch_nb<T, FMT, 7>(a, b, s);
    default: return launch_nb<T, FMT, 8>(a, b, s);
  }
}

}  // namespace

size_t attn_chunk_workspace(int64_t B, int64_t Tq, int64_t Hq, int64_t Hkv, int64_t D, int64_t capacity, int64_t window, int64_t sinks) {
  const Bound b = bound_of(B, Tq, Hq, Hkv, capacity, window, sinks);
  return (size_t)(b.slots * Hkv) * ((size_t)b.slot_waves * 32 * D * 4 + 2 * kRows * 4);
}

bool attn_chunk_fits(int64_t B, int64_t Tq, int64_t Hq, int64_t Hkv, int64_t capacity) {
  const Bound b = bound_of(B, Tq, Hq, Hkv, capacity, 0, 0);
  return Tq * (Hq / Hkv) < (int64_t(1) << 31) - 2 * kRows && b.tiles < (int64_t(1) << 31) / b.keys && b.parts * Hkv * (64 * kWaves) < int64_t(1) << 32;
}

hipError_t launch_attn_chunk(int fmt, int type, const void* q, void* out, const int64_t strides[4], int64_t B, int64_t Tq, int64_t Hq,
                             int64_t Hkv, int64_t D, const KvCache& c, const int32_t* table, int64_t table_stride, const int32_t* cu_q,
                             const int32_t* lengths, int window, int sinks, float scale, void* workspace, hipStream_t stream) {
  const Bound b = bound_of(B, Tq, Hq, Hkv, table_stride << c.page_shift, window, sinks);
  ChunkArgs a;
  a.q = (const uint16_t*)q, a.out = (uint16_t*)out;
  a.q_t = strides[0], a.q_h = strides[1], a.o_t = strides[2], a.o_h = strides[3];
  a.c = c;
  a.table = table, a.cu_q = cu_q, a.lengths = lengths;
  a.acc = (float*)workspace;
  a.stat = a.acc + b.slots * Hkv * b.slot_waves * 32 * D;
  // a negative scale turns the queries round, so that the largest score is the largest product
  // (a scale of 0 becomes a number that still makes -infinity of a masked score)
  a.scale_log2 = __builtin_fabsf(scale) * 1.44269504088896340736f;
  if (a.scale_log2 == 0.0f) a.scale_log2 = 1e-37f;
  a.flip = __builtin_signbit(scale) ? 0x80008000u : 0u;
  a.table_stride = (int)table_stride;
  a.B = (int)B, a.Hq = (int)Hq, a.Hkv = (int)Hkv, a.G = (int)(Hq / Hkv), a.Tq = (int)Tq;
  a.window = window ? window : 1 << 30, a.sinks = window ? sinks : 0;
  a.type = type;
  a.target = (int)b.target;
  a.slot_waves = b.slot_waves;
  const int nb = (int)(D / 32);
  if (fmt == NVQ_KV_Q8_0) return launch_fmt<_Float16, NVQ_KV_Q8_0>(a, nb, b, stream);
  if (fmt == NVQ_KV_F16) return launch_fmt<_Float16, NVQ_KV_F16>(a, nb, b, stream);
  return launch_fmt<__bf16, NVQ_KV_BF16>(a, nb, b, stream);
}

}  // namespace nvq
