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
// Tiles are in LDS twice: while one is multiplied, the next is on its way (16-bit caches: straight from memory, with
// no register in between; Q8_0: through registers, converted between the score products), one barrier a tile.
// Probabilities and queries stay in registers.  Rows of a tile that no row of the work sees are not read and come as
// zeros; masks are looked at only in tiles that some row does not see whole.
//
// Work split: few rows behind many keys are split over workgroups by keys, in parts whose length is chosen on the
// device from the lengths, and joined in order by a second kernel (results do not depend on timing).
//
// Q8_0.  Codes times scales, rounded to binary16, are the operands, with one power of two a tile taken out of the
// scales: scores take the keys' back, the accumulator is held in units of the values', which changes where
// a tile's largest scale leaves it by 2^4 either way.  Scales far below the tile's largest lose bits by it, as it may be where
// every row sees both; a tile of which some row does not see all has no part in the loop if a scale does, and is computed in float32
// behind it, key by key (about 2 us a key for heads of 128: 16 queries whose last key's values are 2^24 times the others' 113 us
// for 17).  What that costs calls without such tiles: 16 tokens behind 484 keys 16.4 us for 15.7, 2048 queries behind 14336 keys 1 %, a
// batch that is not turned first up to 6 %.  A row's channels keep the cache's order (interleaved over its
// blocks), which is as good as any for the contraction: queries and results are permuted instead.
//
// Roundings to 16 bits: Q8_0's operands (11 bits; what is behind them has 8), probabilities (to the operands' type, as
// in the prompt's kernel; the sum that divides them is of the rounded ones), results.
//
// What bounds it.  Many queries: the matrix and the vector unit in turn.  2048 queries (40 heads of 128 on 8) behind
// 14336 keys in bfloat16 take 635 us, 1015 TFLOP/s; matrix
// instructions are issued 50 % of the time, vector ones 40 %, no LDS conflicts.  Over Q8_0 715 to 740 us.  Heads of 64 have half
// the products to the same softmax, and a wavefront's score products have no vector work beside them: 1024 queries, window of 4096, 59 us,
// 580 TFLOP/s (matrix 25 %, vector 42 %).  Few queries: memory.  32 single
// tokens behind 8000 keys each, bfloat16, 186 us (5.6 TB/s); over Q8_0 155 to 160 (3.6 TB/s: each tile is converted for 5 rows of 128).
// A mixed batch of 24 (bfloat16): 49 to 55 us in 504 parts of up to 18 tiles.  The smallest calls are
// latency: 16 tokens behind 484 keys 16 us in the two kernels.
#include "attn_tiles.h"
#include "nvq_launch.h"

namespace nvq {

namespace {

constexpr int kWaves = kTileWaves;
constexpr int kRows = 32 * kWaves;  // of a workgroup
// The shortest part, in tiles: 16 tokens behind 484 keys take 15 us with parts of one tile, 19 with parts of four
// (a tile's latency against one more part to join); longer calls the same.
constexpr int kMinPart = 1;
constexpr int kAhead = 4;  // products that the scores' operands are read ahead
// Parts for one round of workgroups over the chip, or for two where a workgroup's share of the call is more than
// kOneRound tiles, so that what the last one leaves idle weighs less.  40 heads of 128 on 8, bfloat16, one round and two: a
// prompt of 2048 tokens (40 tiles) 63 and 91 us, 32 tokens behind 8000 keys each (62) 190 and 198; 1024 queries of
// 16384 keys (160) 389 and 346, 2048 (320) 701 and 638.  Three: 636 and no gain elsewhere.
constexpr int kOneRound = 128, kRounds = 2;
// Q8_0 is turned into binary16 first from so many rows (query, head) a sequence on, on average, in so much workspace
// at most: a tile is then converted once for all row tiles, and read from there in twice the bytes.  One sequence, 5
// heads to a key head: 100 queries behind 32768 keys 112 us without and 142 with it, 205 behind 16000 122 and 122 (1025
// rows), 512 of 16384 259 and 226, 2048 929 and 747.  The average is the batch's: 2048 queries with 23 single tokens behind 4000
// keys each are not turned and take 218 us (92 and 100 in two calls), nor are 4096 beside 3 tokens behind 100000 keys, whose rows
// would pass kExpandBytes, 905 us (238 and 190).
constexpr int64_t kExpandRows = 8 * kRows, kExpandBytes = int64_t(1) << 30;
// Workgroups that a call is planned for at once, for nb 32-blocks a row: about what registers hold to a compute unit.
// Measured against one more: heads of 64, 1024 queries in a window 59 and 62 us; of 96, 512 queries of 4096 keys 51 and
// 59; of 32, three, four and five: 32 tokens behind 8000 Q8_0 keys each 75, 68 and 68 us, 8 x 16 of 2000 keys 16, 16 and 19.
constexpr int places(int nb) { return 256 * (nb <= 1 ? 4 : nb <= 2 ? 3 : nb <= 4 ? 2 : 1); }

constexpr int kWide = 0x100;  // in units

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
  int places;      // workgroups at once of a key head
  int slot_waves;  // wavefronts' rows that a part's slot holds
  int slots;       // that there are
  // Q8_0 turned into binary16 before (kExpanded): rows [sequence][key head][tile][64] in the cache's channel order, and of
  // each tile the powers of two that its keys (lowest byte) and values (upper half) were divided by
  uint16_t *keys, *values;
  int* units;      // (kWide besides where scales lost bits by it)
  int tiles;       // of a sequence there
};

// Tiles that the 128 rows of one workgroup see of n keys, at most: with a window, those of the first keys, and of
// the windows of up to 128 queries.
__device__ __forceinline__ int tiles_seen(const ChunkArgs& a, int n) {
  const int all = (n + kKeys - 1) / kKeys;
  return min(all, (min(a.sinks, n) + kKeys - 1) / kKeys + (a.window + kRows - 1 + kKeys - 1) / kKeys + 1);
}

// Scores (base 2) from whose maximum so large on a difference may round to 1 and more: a probability would pass the range that
// Range leaves it, and with larger ones every range, either way.  There differences come first, of scores rounded as the
// maximum was, and end where it may be passed.
constexpr float kFar = 0x1p22f;
__device__ __forceinline__ float m_finite(float m) { return m == -__builtin_inff() ? 0.0f : m; }

__device__ __forceinline__ float difference(float s, float factor, float m) {
#pragma clang fp contract(off)
  const float score = s * factor;
  return score - m;
}

// A value that all lanes share, in a scalar register (what a division leaves in a vector one would drag all that
// follows along)
__device__ __forceinline__ int uniform(int x) { return __builtin_amdgcn_readfirstlane(x); }

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

// How the work is cut: the key tiles of a row tile go in equal parts of `part_tiles`, at most of a length for the
// whole call that makes about as many parts as the chip has places for, or twice that.
struct Work {
  Seq s;
  int b;            // sequence, -1: no such work
  int tile;         // row tile of it
  int part;         // part of the tile (main kernel)
  int parts;        // parts that its row tiles have at most
  int part_tiles;   // key tiles of a part
  int slot;         // of the part, or of the row tile's first part; -1: the sequence is not split
};

// join: `want` counts the row tiles of split sequences, else all parts.  A sequence's last row tiles, which see
// the most keys, come first.
__device__ __forceinline__ Work find_work(const ChunkArgs& a, int want, bool join) {
  const int lane = (int)(threadIdx.x & 63);
  int total = 0, all = 0;  // key tiles of all row tiles (below 2^31: host check), and row tiles
  const Seq head = load_seq(a, lane);
  for (int i0 = 0; i0 < a.B; i0 += 64) {
    const Seq s = i0 ? load_seq(a, i0 + lane) : head;
    total += s.tiles * s.most, all += s.tiles;
  }
  total = __builtin_amdgcn_readlane(wave_running_sum(total), 63);
  Work w = {};
  all = __builtin_amdgcn_readlane(wave_running_sum(all), 63);
  // (a row tile's last part is a part of one: half of one is taken off for each)
  const int rounds = total / kOneRound > a.places ? kRounds : 1;
  const uint32_t whole = (uint32_t)max(rounds * a.places - all / 2, (a.places + 3) / 4);
  const int most = uniform(max(kMinPart, (int)(((uint32_t)total + whole - 1) / whole)));
  w.b = -1;
  int base = 0, slots = 0;
  for (int i0 = 0; i0 < a.B; i0 += 64) {
    const Seq s = i0 ? load_seq(a, i0 + lane) : head;
    const int parts = max(1, (s.most + most - 1) / most);
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
      w.part_tiles = max(1, uniform((w.s.most + w.parts - 1) / w.parts));  // parts of equal length
      const int at = want - (base + of(incl) - of(mine));
      const int turn = join ? at : uniform(at / w.parts);
      w.part = join ? 0 : at - turn * w.parts;
      w.tile = w.s.tiles - 1 - turn;
      w.slot = w.parts > 1 ? slots + of(incl_slots) - of(taken) + turn * w.parts + w.part : -1;
      // (only offsets that do not ascend make more of them than there is room for)
      if (w.slot + (join ? w.parts : 1) > a.slots) w.b = -1;
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
  r.first = uniform(r.r0 / a.G) + shift, r.last = uniform((r.r0 + r.count - 1) / a.G) + shift;
  r.end = min(max(r.last + 1, 0), w.s.n);
  r.start = max(r.first - a.window + 1, 0);
  r.sink = min(a.sinks, r.start);
  r.sink_tiles = (r.sink + kKeys - 1) / kKeys;
  r.skip = max(r.start / kKeys - r.sink_tiles, 0);
  r.tiles = max((r.end + kKeys - 1) / kKeys - r.skip, 0);
  return r;
}

// Tiles of a row tile that some row sees and some row does not see whole, at most: 128 rows' places lie within 128 keys, so
// up to 3 tiles hold the ends of what they see and 3 the beginnings of their windows, and one the last of the first keys
constexpr int kPartly = 8;

constexpr int kExpanded = 16;
template <int FMT, int NB>
struct Cached {
  static constexpr bool Q8 = FMT == NVQ_KV_Q8_0, EXPANDED = FMT == kExpanded;
  static constexpr bool MIXED = Q8 || EXPANDED;       // channels in the quantised order, tiles in units of a power of two
  static constexpr int ROW = Q8 ? 32 * NB : 64 * NB;  // bytes of a cache row
  static constexpr int WORDS = Q8 ? 2 * NB : 1;       // Q8_0: dwords that a lane takes of it (4 lanes to a row)
  static constexpr int SCALES = Q8 ? (NB + 1) / 2 : 1;  // its scales, two a dword
};

// The channel of place p of a row's order in the cache
template <bool Q8, int NB>
__device__ __forceinline__ int channel_of(int p) {
  if constexpr (!Q8) return p;
  const int pair = p >> 1;
  return 32 * (pair % NB) + 2 * (pair / NB) + (p & 1);
}

// N dwords, as a vector: an array that is copied about would be kept in memory
template <int N>
struct Dwords {
  typedef uint32_t type __attribute__((ext_vector_type(N)));
};
// N dwords of a buffer from a byte offset that is a multiple of 4 N up to 16
template <int N>
__device__ __forceinline__ typename Dwords<N>::type load_dwords(__amdgpu_buffer_rsrc_t r, uint32_t at) {
  typename Dwords<N>::type v;
  if constexpr (N % 4 == 0) {
#pragma unroll
    for (int i = 0; i < N / 4; ++i) {
      const u32x4 t = __builtin_bit_cast(u32x4, __builtin_amdgcn_raw_buffer_load_b128(r, at + 16 * i, 0, 0));
#pragma unroll
      for (int j = 0; j < 4; ++j) v[4 * i + j] = t[j];
    }
  } else if constexpr (N % 2 == 0) {
#pragma unroll
    for (int i = 0; i < N / 2; ++i) {
      const u32x2 t = __builtin_bit_cast(u32x2, __builtin_amdgcn_raw_buffer_load_b64(r, at + 8 * i, 0, 0));
      v[2 * i] = t[0], v[2 * i + 1] = t[1];
    }
  } else {
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] = __builtin_amdgcn_raw_buffer_load_b32(r, at + 4 * i, 0, 0);
  }
  return v;
}

// Which of a pair of 16-bit elements are not finite: their bits set
template <typename T>
__device__ __forceinline__ uint32_t not_finite(uint32_t w) {
  constexpr uint32_t e = __is_same(T, _Float16) ? 0x7C00u : 0x7F80u;
  return ((w & e) == e ? 0xFFFFu : 0u) | (((w >> 16) & e) == e ? 0xFFFF0000u : 0u);
}

typedef uint16_t u16x2_t __attribute__((ext_vector_type(2)));
__device__ __forceinline__ uint32_t max_halves(uint32_t a, uint32_t b) {
  return __builtin_bit_cast(uint32_t, __builtin_elementwise_max(__builtin_bit_cast(u16x2_t, a), __builtin_bit_cast(u16x2_t, b)));
}
__device__ __forceinline__ uint32_t finite_halves(uint32_t w) { return w & 0x7FFF7FFFu & ~not_finite<_Float16>(w); }

// Largest of a lane's scales, both halves; and over a wavefront whose quads hold the same, in the upper
// half of a and of b: the result's halves
template <int N>
__device__ __forceinline__ uint32_t largest_scale(typename Dwords<N>::type d) {
  uint32_t x = 0;
#pragma unroll
  for (int i = 0; i < N; ++i) x = max_halves(x, finite_halves(d[i]));
  return max_halves(x, x << 16);
}
__device__ __forceinline__ uint32_t wave_largest(uint32_t a, uint32_t b) {
  uint32_t x = perm(a, b, 0x07060302u);
  x = max_halves(x, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)x, 0x141, 0xF, 0xF, true));
  x = max_halves(x, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)x, 0x140, 0xF, 0xF, true));
  const auto p = __builtin_amdgcn_permlane16_swap(x, x, false, false);
  x = max_halves(p[0], p[1]);
  const auto q = __builtin_amdgcn_permlane32_swap(x, x, false, false);
  return max_halves(q[0], q[1]);
}

// A positive binary16 number's exponent as frexp gives it; kNone of 0
constexpr int kNone = -1000;
__device__ __forceinline__ int exponent_of(uint32_t bits) {
  return bits >= 0x400u ? (int)(bits >> 10) - 14 : bits ? 8 - __builtin_clz(bits) : kNone;
}
// The power of two that takes a scale of exponent e to the highest place where its largest code is a binary16 number, which leaves
// the most below it (and not past what scale_down has: a scale so small is exact there)
__device__ __forceinline__ int highest(int e) { return max(e - 9, -30); }
// Scales times 2^-e, in two steps that binary16 holds
template <int N>
__device__ __forceinline__ typename Dwords<N>::type scale_down(typename Dwords<N>::type d, int e) {
  const auto power = [](int x) { return __builtin_bit_cast(half2_t, (uint32_t)(15 - x) * 0x04000400u); };
  const half2_t f = power(e >> 1), g = power(e - (e >> 1));
#pragma unroll
  for (int i = 0; i < N; ++i) {
    const uint32_t x = d[i];  // (a bit cast of a vector's element reads element 0)
    d[i] = __builtin_bit_cast(uint32_t, __builtin_bit_cast(half2_t, x) * f * g);
  }
  return d;
}

// Whether scales x lost bits in it: some came out below the normal range (what was subnormal before is exact where it does not)
template <int N>
__device__ __forceinline__ bool lost_bits(typename Dwords<N>::type x, typename Dwords<N>::type scaled) {
  uint32_t lost = 0;
#pragma unroll
  for (int i = 0; i < N; ++i)
    lost |= (uint32_t)(((scaled[i] & 0x7C00u) == 0) & ((x[i] & 0x7FFFu) != 0)) | (uint32_t)(((scaled[i] & 0x7C000000u) == 0) & ((x[i] & 0x7FFF0000u) != 0));
  return lost != 0;
}

// The scales of row `row_in` of a group
template <int NB>
__device__ __forceinline__ typename Dwords<(NB + 1) / 2>::type load_row_scales(__amdgpu_buffer_rsrc_t r, int row_in) {
  if constexpr (NB % 2 == 0) {
    return load_dwords<NB / 2>(r, 2 * NB * row_in);
  } else {
    typename Dwords<(NB + 1) / 2>::type x;
#pragma unroll
    for (int i = 0; i < (NB + 1) / 2; ++i) {
      const uint32_t u = (uint16_t)__builtin_amdgcn_raw_buffer_load_b16(r, 2 * (NB * row_in + 2 * i), 0, 0);
      const uint32_t v = 2 * i + 1 < NB ? (uint16_t)__builtin_amdgcn_raw_buffer_load_b16(r, 2 * (NB * row_in + 2 * i + 1), 0, 0) : 0u;
      x[i] = u | v << 16;
    }
    return x;
  }
}
// Codes times scales, eight of them: piece i of a quarter of a row.  (1152 = 1024 + 128: the byte, its sign bit turned,
// is the end of a binary16 number's mantissa)
template <int NB>
__device__ __forceinline__ u32x4 to_halves(typename Dwords<2 * NB>::type codes, typename Dwords<(NB + 1) / 2>::type scales, int i) {
  u32x4 y;
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const int pair = 4 * i + j, b = pair % NB;
    const uint32_t two = scales[b / 2];
    const half2_t d = __builtin_bit_cast(half2_t, two), f = half2_t{d[b & 1], d[b & 1]};
    const uint32_t u = perm(0x64646464u, codes[pair / 2] ^ 0x80808080u, pair & 1 ? 0x04030402u : 0x04010400u);
    y[j] = __builtin_bit_cast(uint32_t, (__builtin_bit_cast(half2_t, u) - half2_t{(_Float16)1152.0f, (_Float16)1152.0f}) * f);
  }
  return y;
}

template <typename T, int FMT, int NB>
__global__ __launch_bounds__(64 * kWaves, NB <= 4 ? 2 : 1) void attn_chunk_kernel(ChunkArgs a) {
  typedef Stage<NB> S;
  typedef Cached<FMT, NB> C;
  __shared__ __align__(16) uint8_t s_keys[2 * S::BYTES], s_values[2 * S::BYTES];
  __shared__ __align__(16) uint32_t s_top[4][kWaves];  // Q8_0: the groups' largest scales, keys' in the upper half
  __shared__ int s_bad, s_broken;  // a page number outside the cache; a value that is not finite in a tile of which some row does not see all
  __shared__ int s_wide[kPartly];  // Q8_0: the part's partly seen tiles, in order: not 0 if left out at first
  const int tid = (int)threadIdx.x, lane = tid & 63, c = lane & 31, hi = lane >> 5;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int item = uniform((int)blockIdx.x / a.Hkv), kvh = (int)blockIdx.x - item * a.Hkv;
  const Work w = find_work(a, item, false);
  if (w.b < 0) return;
  const Rows rt = rows_of(a, w);
  const int t_begin = w.part * w.part_tiles, t_end = min(rt.tiles, t_begin + w.part_tiles);
  const bool split = rt.tiles > w.part_tiles;
  if (w.part > 0 && t_begin >= rt.tiles) return;
  if (tid == 0) s_bad = s_broken = 0;
  if (C::Q8 && tid < kPartly) s_wide[tid] = 0;

  // A lane's row; past the last row it again, which is not stored
  const bool mine = 32 * wave < rt.count;
  struct Row {
    int query, head, place;
    bool live;
  };
  const auto row_of = [&](int column) __attribute__((always_inline)) {
    const int rows = w.s.m * a.G, r = rt.r0 + 32 * wave + column, rr = min(r, rows - 1), query = rr / a.G;
    return Row{query, kvh * a.G + rr - query * a.G, query + w.s.n - w.s.m, r < rows};
  };
  const int place = row_of(c).place;
  const int place_first = __builtin_amdgcn_readlane(place, 0), place_last = __builtin_amdgcn_readlane(place, 31);
  const auto seen_by = [&](int place, int key) __attribute__((always_inline)) { return (key <= place) & ((key > place - a.window) | (key < a.sinks)); };

  // Its query, 16 places of the cache's channel order at a time, on the way before the keys' place is known
  Frag qf[2 * NB];
  {
    const Row at = row_of(c);
    const uint16_t* row = a.q + (int64_t)(w.s.q0 + at.query) * a.q_t + (int64_t)at.head * a.q_h;
#pragma unroll
    for (int ks = 0; ks < 2 * NB; ++ks) {
      if constexpr (C::MIXED) {
#pragma unroll
        for (int j = 0; j < 4; ++j) qf[ks].v[j] = *reinterpret_cast<const uint32_t*>(row + channel_of<true, NB>(16 * ks + 8 * hi + 2 * j));
      } else {
        const u32x4 x = *reinterpret_cast<const u32x4*>(row + 16 * ks + 8 * hi);
#pragma unroll
        for (int j = 0; j < 4; ++j) qf[ks].v[j] = x[j];
      }
    }
  }

  // The wavefront's 16-key group of each tile: where it is in the cache, and how many of its rows are read.
  const auto* table = (const __attribute__((address_space(4))) int32_t*)(a.table + (int64_t)w.b * a.table_stride);
  const int page_mask = (1 << a.c.page_shift) - 1;
  const auto tile_key = [&](int t) __attribute__((always_inline)) { return (t < rt.sink_tiles ? t : t + rt.skip) * kKeys; };
  bool bad_page = false;
  struct Group {
    int64_t row;
    int count;
  };
  const auto rows_seen = [&](int t) __attribute__((always_inline)) {
    const int key0 = tile_key(t) + 16 * wave;
    const bool none = t >= t_end || (key0 + 15 < rt.start && key0 >= rt.sink);  // no row sees any of it
    return none ? 0 : min(max(rt.end - key0, 0), 16);
  };
  const auto page_of = [&](int t) __attribute__((always_inline)) { return !C::EXPANDED && rows_seen(t) > 0 ? table[(tile_key(t) + 16 * wave) >> a.c.page_shift] : 0; };
  const int64_t first_tile = C::EXPANDED ? ((int64_t)w.b * a.Hkv + kvh) * a.tiles : 0;
  const auto group_of = [&](int t, int page) __attribute__((always_inline)) {
    const auto at = [&](int64_t row, int count) __attribute__((always_inline)) {
      return Group{(int64_t)(uint32_t)uniform((int)row) | (int64_t)uniform((int)(row >> 32)) << 32, uniform(count)};
    };
    if constexpr (C::EXPANDED) return at(first_tile * kKeys + (t < t_end ? tile_key(t) : 0) + 16 * wave, rows_seen(t));
    const bool out = (uint32_t)page >= (uint32_t)a.c.n_pages;
    bad_page |= out;
    const int64_t row = (((int64_t)(out ? 0 : page) * a.Hkv + kvh) << a.c.page_shift) + ((tile_key(t) + 16 * wave) & page_mask);
    return at(row, out ? 0 : rows_seen(t));
  };
  const auto partly = [&](int t) __attribute__((always_inline)) {  // some row does not see some key of the tile
    const int key0 = tile_key(t);
    return (key0 + kKeys - 1 > rt.first) | ((key0 <= rt.last - a.window) & (key0 + kKeys - 1 >= a.sinks));
  };

  // 16-bit caches: straight into LDS, 64 pieces of 16 bytes a load, in LDS order.  Rows that are not read come
  // as zeros: a group's buffer ends behind its last one.
  uint32_t key_from[C::Q8 ? 1 : NB], value_from[C::Q8 ? 1 : NB];
  const uint32_t keys_at = lds_address(s_keys) + (uint32_t)(wave * 16 * S::ROW), values_at = lds_address(s_values) + (uint32_t)(wave * 16 * S::ROW);
  if constexpr (!C::Q8) {
#pragma unroll
    for (int j = 0; j < NB; ++j) {
      const int id = 64 * j + lane, row = id / S::PIECES, pos = id % S::PIECES;
      key_from[j] = (uint32_t)(row * S::ROW + 16 * S::key_piece(row, pos));
      value_from[j] = (uint32_t)(row * S::ROW + 16 * S::value_piece(row, pos));
    }
  }
  const void* const all_keys = C::EXPANDED ? a.keys : a.c.k;
  const void* const all_values = C::EXPANDED ? a.values : a.c.v;
  const auto buffer16 = [&](const void* p, Group g) __attribute__((always_inline)) {
    return buffer_of(reinterpret_cast<const uint8_t*>(p) + g.row * C::ROW, (uint32_t)(g.count * C::ROW));
  };
  const auto async_rows = [&](const void* p, Group g, const uint32_t* from, uint32_t at) __attribute__((always_inline)) {
    const u32x4 buffer = buffer16(p, g);
#pragma unroll
    for (int j = 0; j < NB; ++j) buffer_to_lds(buffer, from[j], (uint32_t)uniform((int)(at + 1024 * j)));
  };

  // Q8_0: through registers, 4 lanes to a row, and converted into LDS a step later.
  typedef typename Dwords<C::WORDS>::type Codes;
  typedef typename Dwords<C::SCALES>::type Scales;
  const int row_in = lane >> 2, seg = lane & 3;
  const auto load_scales = [&](const void* p, Group g) __attribute__((always_inline)) {
    const auto rsrc = __builtin_amdgcn_make_buffer_rsrc((void*)(reinterpret_cast<const uint16_t*>(p) + g.row * NB), 0, g.count * (2 * NB), 0x00020000);
    return load_row_scales<NB>(rsrc, row_in);
  };
  const auto load_codes = [&](const void* p, Group g) __attribute__((always_inline)) {
    const auto rsrc = __builtin_amdgcn_make_buffer_rsrc((void*)(reinterpret_cast<const uint8_t*>(p) + g.row * C::ROW), 0, g.count * C::ROW, 0x00020000);
    return load_dwords<C::WORDS>(rsrc, row_in * C::ROW + seg * (C::ROW / 4));
  };
  // The largest scales of a key tile and a value tile, from all wavefronts: exponents one barrier later
  const auto publish = [&](int slot, Scales k, Scales v) __attribute__((always_inline)) {
    const uint32_t x = wave_largest(largest_scale<C::SCALES>(k), largest_scale<C::SCALES>(v));
    if (lane == 0) s_top[slot][wave] = x;
  };
  const auto published = [&](int slot) __attribute__((always_inline)) {
    const u32x4 x = *reinterpret_cast<const u32x4*>(s_top[slot]);
    return (uint32_t)__builtin_amdgcn_readfirstlane((int)max_halves(max_halves(x[0], x[1]), max_halves(x[2], x[3])));
  };
  // Rows between the first keys and the windows, in a group that is read: their scales become 0, so that they have no
  // part in the tile's largest
  const auto hide = [&](int t, Scales& k, Scales& v) __attribute__((always_inline)) {
    if (tile_key(t) < rt.start) {
      const int key = tile_key(t) + 16 * wave + row_in;
      const bool unseen = (key >= rt.sink) & (key < rt.start);
#pragma unroll
      for (int i = 0; i < C::SCALES; ++i) k[i] = unseen ? 0u : k[i], v[i] = unseen ? 0u : v[i];
    }
  };
  // Piece i of the lane's part of a row, with the scales times 2^-e, into a tile
  const auto convert = [&](uint8_t* tile, Codes codes, Scales scales, int i, bool keys) __attribute__((always_inline)) {
    if constexpr (C::Q8) {
      const int row = 16 * wave + row_in, piece = NB * seg + i;
      *reinterpret_cast<u32x4*>(tile + row * S::ROW + 16 * (keys ? S::key_piece(row, piece) : S::value_piece(row, piece))) = to_halves<NB>(codes, scales, i);
    }
  };

  floatx16 acc[NB];
#pragma unroll
  for (int d = 0; d < NB; ++d)
#pragma unroll
    for (int j = 0; j < 16; ++j) acc[d][j] = 0.0f;
  float m = -__builtin_inff(), l = 0.0f;
  bool far = false;  // some row's maximum passes kFar
  int unit = kNone;  // Q8_0: the accumulator is in units of 2^unit

  // What is not finite in a value row must not meet a probability of 0 in rows that do not see it: it stays out of
  // a tile that has keys that some row does not see, and rows that see it get it behind the last one.
  const auto keep_finite = [&](Scales d) __attribute__((always_inline)) {
    uint32_t found = 0;
#pragma unroll
    for (int i = 0; i < C::SCALES; ++i) found |= not_finite<_Float16>(d[i]);
    if (__any(found != 0)) {
      s_broken = 1;
#pragma unroll
      for (int i = 0; i < C::SCALES; ++i) d[i] &= ~not_finite<_Float16>(d[i]);
    }
    return d;
  };
  // Q8_0: a tile's scales times their powers of two.  Of a partly seen tile none may lose bits by it, to a row that others
  // see: the tile, the part's number `number` of them, is left out at first
  const auto scale_both = [&](bool part_seen, int number, Scales& k, int ek, Scales& v, int ev) __attribute__((always_inline)) {
    const Scales k_old = k;
    if (part_seen) v = keep_finite(v);
    const Scales v_old = v;
    k = scale_down<C::SCALES>(k_old, ek), v = scale_down<C::SCALES>(v_old, ev);
    if (part_seen) {
      if (__any(lost_bits<C::SCALES>(k_old, k) | lost_bits<C::SCALES>(v_old, v))) s_wide[number] = 1;
    }
  };
  int at = 0;                         // partly seen tiles so far
  bool here = partly(t_begin);        // this tile is one
  bool any_wide = false;              // one was left out
  // the same for a 16-bit tile that is in LDS: a wavefront its group's rows
  const auto check_values = [&](int slot) __attribute__((always_inline)) {
    uint8_t* p = s_values + slot * S::BYTES + wave * 16 * S::ROW + 16 * lane;
    float z = 0.0f;
#pragma unroll
    for (int j = 0; j < NB; ++j) {
      const u32x4 x = *reinterpret_cast<const u32x4*>(p + 1024 * j);
#pragma unroll
      for (int i = 0; i < 4; ++i) z = zero_of_pair<T>(x[i], z);
    }
    if (__any(z != z)) {
      s_broken = 1;
#pragma unroll
      for (int j = 0; j < NB; ++j) {
        u32x4 x = *reinterpret_cast<const u32x4*>(p + 1024 * j);
#pragma unroll
        for (int i = 0; i < 4; ++i) x[i] &= ~not_finite<T>(x[i]);
        *reinterpret_cast<u32x4*>(p + 1024 * j) = x;
      }
    }
  };
  const auto barrier = [&]() __attribute__((always_inline)) {
    wait_reads();
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
  };

  // The first tiles on their way.
  Group g0, g1;
  {
    const int p0 = page_of(t_begin), p1 = page_of(t_begin + 1);
    g0 = group_of(t_begin, p0), g1 = group_of(t_begin + 1, p1);
  }
  int next_page = page_of(t_begin + 2);
  Codes k0, v0, k_codes, v_codes;  // Q8_0: the first tile, and the one that the next step converts
  Scales k0_d, v0_d, k_scales, v_scales;
  if constexpr (C::Q8) {
    k0_d = load_scales(a.c.k_d, g0), v0_d = load_scales(a.c.v_d, g0), k_scales = load_scales(a.c.k_d, g1), v_scales = load_scales(a.c.v_d, g1);
    k0 = load_codes(a.c.k, g0), v0 = load_codes(a.c.v, g0), k_codes = load_codes(a.c.k, g1), v_codes = load_codes(a.c.v, g1);
  } else {
    async_rows(all_keys, g0, key_from, keys_at);
    async_rows(all_values, g0, value_from, values_at);
  }

  // bfloat16 queries into binary16 operands: scaled to 2^7 .. 2^8, exact down to 2^-32 of the largest
  float to_log2 = a.scale_log2;
  if constexpr (C::MIXED) {
    if (a.type == NVQ_TYPE_BF16) {
      float largest = 0.0f;
#pragma unroll
      for (int ks = 0; ks < 2 * NB; ++ks)
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          float x[2];
          unpack_pair<__bf16>(qf[ks].v[j], x);
          largest = fmaxf(largest, fmaxf(fabsf(x[0]), fabsf(x[1])));
        }
      largest = max_32(largest);
      const int e = largest > 0.0f && largest < __builtin_inff() ? 8 - __builtin_amdgcn_frexp_expf(largest) : 0;
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
#pragma unroll
  for (int ks = 0; ks < 2 * NB; ++ks)
#pragma unroll
    for (int j = 0; j < 4; ++j) qf[ks].v[j] ^= a.flip;

  uint32_t key_offset[2 * NB], value_offset[NB];
#pragma unroll
  for (int ks = 0; ks < 2 * NB; ++ks) key_offset[ks] = in_vgpr((uint32_t)(c * S::ROW + 16 * S::key_piece(c, 2 * ks + hi)));
  {
    const int jj = lane & 15, in = 4 * hi + (jj >> 2), half = (lane >> 4) & 1;
#pragma unroll
    for (int d = 0; d < NB; ++d)
      value_offset[d] = in_vgpr((uint32_t)(in * S::ROW + 16 * S::value_piece(in, 4 * d + 2 * half + ((jj & 3) >> 1)) + 8 * (jj & 1)));
  }

  // Tile t in a slot, seen with scores times `factor`, or (wide) not at all; between the first products, `turn` has its turns
  const auto step = [&](int t, int slot, float factor, bool wide, auto turn) __attribute__((always_inline)) {
    floatx16 s[2];
#pragma unroll
    for (int kb = 0; kb < 2; ++kb)
#pragma unroll
      for (int j = 0; j < 16; ++j) s[kb][j] = 0.0f;
#pragma unroll
    for (int ks = 0; ks < 2 * NB; ++ks)
#pragma unroll
      for (int kb = 0; kb < 2; ++kb) {
        const u32x4 x = *reinterpret_cast<const u32x4*>(s_keys + slot * S::BYTES + key_offset[ks] + 32 * kb * S::ROW);
        s[kb] = mfma32<T>(Frag{x[0], x[1], x[2], x[3]}, qf[ks], s[kb]);
        if (kb) turn(ks);
      }
    // Order asked of the compiler: the operands' reads stay kAhead products ahead (left alone, it reads each right before
    // its product: 650 us for 635 of 2048 bfloat16 queries behind 14336 keys; 2 ahead 635, 8 ahead 641)
    __builtin_amdgcn_sched_group_barrier(0x100, kAhead, 0);  // LDS reads
#pragma unroll
    for (int i = 0; i < 4 * NB; ++i) {
      __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);  // a matrix product
      if (i + kAhead < 4 * NB) __builtin_amdgcn_sched_group_barrier(0x100, 1, 0);
    }
    const int key0 = tile_key(t);
    if (wide || key0 + kKeys - 1 > place_first || (key0 <= place_last - a.window && key0 + kKeys - 1 >= a.sinks)) {
      const int from = wide ? -1 : place;
#pragma unroll
      for (int kb = 0; kb < 2; ++kb)
#pragma unroll
        for (int j = 0; j < 16; ++j)
          if (!seen_by(from, key0 + 32 * kb + 8 * (j >> 2) + 4 * hi + (j & 3))) s[kb][j] = -__builtin_inff();
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
      far = __any(fabsf(m_finite(m)) >= kFar);
    }
    float base = score_base<T>(m), times = factor;
    if (far) {
#pragma unroll
      for (int kb = 0; kb < 2; ++kb)
#pragma unroll
        for (int j = 0; j < 16; ++j) {
          const float x = difference(s[kb][j], factor, m_finite(m));
          s[kb][j] = x > Range<T>::SLACK ? Range<T>::SLACK : x;
        }
      base = -Range<T>::SHIFT, times = 1.0f;
    }
    Frag pf[2][2];
#pragma unroll
    for (int kb = 0; kb < 2; ++kb)
#pragma unroll
      for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const float x = exp2_fast(__builtin_fmaf(s[kb][8 * h + 2 * j], times, -base));
          const float y = exp2_fast(__builtin_fmaf(s[kb][8 * h + 2 * j + 1], times, -base));
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
            const u32x2 y = read_transposed(s_values + slot * S::BYTES + value_offset[d] + (32 * kb + 16 * h + 8 * x) * S::ROW);
            f.v[2 * x] = y[0], f.v[2 * x + 1] = y[1];
          }
          acc[d] = mfma32<T>(f, pf[kb][h], acc[d]);
        }
  };
  // Exponents for a tile with the largest scales x (keys' in the upper half): the keys', and the values', which is the
  // accumulator's unit from that tile on
  const auto key_unit = [&](uint32_t x) __attribute__((always_inline)) {
    const int e = exponent_of(x >> 16);
    return e == kNone ? 0 : highest(e);
  };
  const auto value_unit = [&](bool part_seen, uint32_t x) __attribute__((always_inline)) {
    const int e = exponent_of(x & 0xFFFFu);
    const int u = part_seen ? highest(e) : unit != kNone && e - unit <= 9 && e - unit >= 2 ? unit : e - 5;
    return e == kNone ? unit : u;
  };
  // base 2, of a score with the keys in units of 2^e (not 0, which would make NaN of a masked score)
  const auto factor_of = [&](int e) __attribute__((always_inline)) { return fmaxf(__builtin_amdgcn_ldexpf(to_log2, e), 1e-37f); };

  const auto use_unit = [&](int u) __attribute__((always_inline)) {
    if (u != unit) {
      if (unit != kNone) {
        const float f = __builtin_amdgcn_ldexpf(1.0f, unit - u);
#pragma unroll
        for (int d = 0; d < NB; ++d) acc[d] *= f;
      }
      unit = u;
    }
  };
  const auto* units = (const __attribute__((address_space(4))) int*)(C::EXPANDED ? a.units + first_tile : nullptr);
  const auto unit_of = [&](int t) __attribute__((always_inline)) { return C::EXPANDED && t < t_end ? units[tile_key(t) / kKeys] : 0; };
  int next_unit = unit_of(t_begin);

  if (t_begin < t_end) {
    float factor = 0.0f;
    if constexpr (C::Q8) {
      hide(t_begin, k0_d, v0_d);
      hide(t_begin + 1, k_scales, v_scales);
      publish(2, k0_d, v0_d);
      publish(1, k_scales, v_scales);
      barrier();
      const uint32_t x = published(2);
      const int e = key_unit(x);
      unit = value_unit(here, x);
      scale_both(here, 0, k0_d, e, v0_d, unit == kNone ? 0 : unit);
#pragma unroll
      for (int i = 0; i < NB; ++i) convert(s_keys, k0, k0_d, i, true);
#pragma unroll
      for (int i = 0; i < NB; ++i) convert(s_values, v0, v0_d, i, false);
      factor = factor_of(e);
    } else {
      wait_loads<0>();
    }
    barrier();
    // Step t.  16-bit: tile t + 1 goes on its way.  Q8_0: tile t + 1, in registers, is converted between the first products,
    // and the loads of tile t + 2 begin, scales first: their largest are known to everyone one barrier later.
    const auto pass = [&](int t, int slot) __attribute__((always_inline)) {
      const Group g2 = group_of(t + 2, next_page);
      next_page = page_of(t + 3);
      uint8_t* const keys = s_keys + (slot ^ 1) * S::BYTES;
      uint8_t* const values = s_values + (slot ^ 1) * S::BYTES;
      if constexpr (C::Q8) {
        Scales k_next = load_scales(a.c.k_d, g2), v_next = load_scales(a.c.v_d, g2);
        const bool wide = here && uniform(s_wide[at]) != 0;
        at += here, any_wide |= wide, here = partly(t + 1);
        const uint32_t x = published(slot ^ 1);
        const int e = key_unit(x), u = value_unit(here, x);
        scale_both(here, at, k_scales, e, v_scales, u == kNone ? 0 : u);
        const auto turn = [&](int j) __attribute__((always_inline)) {
          if (j < NB)
            convert(keys, k_codes, k_scales, j, true);
          else
            convert(values, v_codes, v_scales, j - NB, false);
        };
        if (mine) {
          step(t, slot, factor, wide, turn);
        } else {
#pragma unroll
          for (int j = 0; j < 2 * NB; ++j) turn(j);
        }
        use_unit(u);
        factor = factor_of(e);
        k_codes = load_codes(a.c.k, g2), v_codes = load_codes(a.c.v, g2);
        hide(t + 2, k_next, v_next);
        publish(slot, k_next, v_next);
        k_scales = k_next, v_scales = v_next;
      } else {
        if (partly(t)) {
          check_values(slot);
          barrier();
        }
        const u32x4 kb = buffer16(all_keys, g1), vb = buffer16(all_values, g1);
        const auto turn = [&](int j) __attribute__((always_inline)) {
          if (j < NB)
            buffer_to_lds(kb, key_from[j], (uint32_t)uniform((int)(keys_at + (slot ^ 1) * S::BYTES + 1024 * j)));
          else
            buffer_to_lds(vb, value_from[j - NB], (uint32_t)uniform((int)(values_at + (slot ^ 1) * S::BYTES + 1024 * (j - NB))));
        };
        float f = a.scale_log2;
        bool wide = false;
        if constexpr (C::EXPANDED) {
          f = factor_of((int8_t)next_unit);
          wide = (next_unit & kWide) && partly(t);
          any_wide |= wide;
          use_unit(next_unit >> 16);
          next_unit = unit_of(t + 1);
        }
        if (mine) {
          step(t, slot, f, wide, turn);
        } else {
#pragma unroll
          for (int j = 0; j < 2 * NB; ++j) turn(j);
        }
        wait_loads<0>();
      }
      g1 = g2;
      barrier();
    };
    for (int t = t_begin, slot = 0; t < t_end; ++t, slot ^= 1) pass(t, slot);
  }
  if (bad_page) s_bad = 1;
  __syncthreads();
  if (!mine) return;
  l = sum_32(l);
  const Row row = row_of(in_vgpr((uint32_t)lane) & 31);
  // From here on arguments are read again, from an address that the compiler does not know: it would keep them all along, and the
  // loop's scalars go to lanes of vector registers (with 28 of them no operand of the value products was read ahead: 2048 queries
  // behind 14336 Q8_0 keys 798 us for 724)
  auto* late = (const __attribute__((address_space(4))) ChunkArgs*)__builtin_amdgcn_kernarg_segment_ptr();
  asm volatile("" : "+s"(late));
  const auto* pages = (const __attribute__((address_space(4))) int32_t*)(late->table + (int64_t)w.b * late->table_stride);
  if (C::MIXED && unit != kNone) {
    const float f = __builtin_amdgcn_ldexpf(1.0f, unit);
#pragma unroll
    for (int d = 0; d < NB; ++d) acc[d] *= f;
  }
  // Tiles that were left out, with codes and scales out of the cache, in float32: lanes have rows as before, and half of their channels.
  // Rare, so it is kept from costing the loop registers: the accumulator waits where the tiles were.
  if constexpr (C::MIXED) {
    if (any_wide) {
      floatx4* const mem = reinterpret_cast<floatx4*>((wave & 2 ? s_values : s_keys) + (wave & 1) * S::BYTES) + lane;
#pragma unroll
      for (int d = 0; d < NB; ++d)
#pragma unroll
        for (int i = 0; i < 4; ++i) mem[(4 * d + i) * 64] = floatx4{acc[d][4 * i], acc[d][4 * i + 1], acc[d][4 * i + 2], acc[d][4 * i + 3]};
      // words 2 x + hi of a row are the lane's, of keys and values alike: pairs 4 x + 2 hi and + 1 in the cache's order
      uint32_t q[8 * NB];
      {
        const uint16_t* query = late->q + (int64_t)(w.s.q0 + row.query) * late->q_t + (int64_t)row.head * late->q_h;
#pragma unroll
        for (int x = 0; x < 8 * NB; ++x) q[x] = *reinterpret_cast<const uint32_t*>(query + channel_of<true, NB>(4 * (2 * (x >> 1) + hi) + 2 * (x & 1)));
      }
      const float signed_scale = late->flip ? -late->scale_log2 : late->scale_log2;
      for (int t = t_begin, number = 0; t < t_end; ++t) {
        if (!partly(t)) continue;
        const bool left_out = C::Q8 ? uniform(s_wide[number]) != 0 : (unit_of(t) & kWide) != 0;
        ++number;
        if (!left_out) continue;
        const int key_end = min(tile_key(t) + kKeys, rt.end);
#pragma unroll 1
        for (int key = tile_key(t); key < key_end; ++key) {
          const bool visible = (key <= row.place) & ((key > row.place - late->window) | (key < late->sinks));
          if (!__any(visible)) continue;
          const int page = pages[key >> late->c.page_shift];
          const bool out = (uint32_t)page >= (uint32_t)late->c.n_pages;
          const int64_t from = (((int64_t)(out ? 0 : page) * late->Hkv + kvh) << late->c.page_shift) + (key & ((1 << late->c.page_shift) - 1));
          uint32_t codes[2][4 * NB];
          float scales[2][NB];  // of pairs x, x + NB, .. of the lane's
#pragma unroll
          for (int v = 0; v < 2; ++v) {
            const uint32_t* words = reinterpret_cast<const uint32_t*>(reinterpret_cast<const uint8_t*>(v ? late->c.v : late->c.k) + from * (32 * NB)) + hi;
            const uint16_t* d = reinterpret_cast<const uint16_t*>(v ? late->c.v_d : late->c.k_d) + from * NB;
#pragma unroll
            for (int x = 0; x < 4 * NB; ++x) codes[v][x] = words[2 * x];
#pragma unroll
            for (int x = 0; x < NB; ++x) scales[v][x] = f16_bits_to_f32(d[(x + 2 * hi) % NB]);
          }
#pragma unroll
          for (int x = 0; x < NB; ++x) scales[1][x] = visible ? scales[1][x] : 0.0f;
          const auto element = [&](int v, int x, int y) __attribute__((always_inline)) {  // element y of the lane's word x
            return scales[v][(4 * x + (y >> 1)) % NB] * (float)(int)(int8_t)(codes[v][x] >> (8 * y));
          };
          float s = 0.0f;
#pragma unroll
          for (int x = 0; x < 8 * NB; ++x) {
            float two[2];
            if (late->type == NVQ_TYPE_F16)
              unpack_pair<_Float16>(q[x], two);
            else
              unpack_pair<__bf16>(q[x], two);
#pragma unroll
            for (int y = 0; y < 2; ++y) s = __builtin_fmaf(element(0, x >> 1, 2 * (x & 1) + y), two[y] * signed_scale, s);
          }
          s = out ? __builtin_nanf("") : sum_32(s);
          if (!visible) s = -__builtin_inff();
          const float m_new = s > m + Range<T>::SLACK ? s : m, f = m_new == m ? 1.0f : exp2_fast(m - m_new);
          m = m_new;
          const float p = exp2_fast(s - m_finite(m) + Range<T>::SHIFT);
          l = l * f + p;
#pragma unroll
          for (int i = 0; i < 4 * NB; ++i) {
            floatx4 x = mem[i * 64] * f;
#pragma unroll
            for (int y = 0; y < 4; ++y) x[y] = __builtin_fmaf(p, element(1, i, y), x[y]);
            mem[i * 64] = x;
          }
        }
      }
#pragma unroll
      for (int d = 0; d < NB; ++d)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const floatx4 x = mem[(4 * d + i) * 64];
#pragma unroll
          for (int j = 0; j < 4; ++j) acc[d][4 * i + j] = x[j];
        }
    }
  }
  if (s_broken) {
    for (int t = t_begin; t < t_end; ++t)
      for (int j = partly(t) ? 0 : kKeys; j < kKeys; ++j) {
        const int key = tile_key(t) + j;
        if (!(key <= row.place && (key > row.place - late->window || key < late->sinks))) continue;
        const int page = C::EXPANDED ? 0 : pages[key >> late->c.page_shift];
        if ((uint32_t)page >= (uint32_t)late->c.n_pages) continue;
        const int64_t from = C::EXPANDED ? first_tile * kKeys + key : (((int64_t)page * late->Hkv + kvh) << late->c.page_shift) + (key & ((1 << late->c.page_shift) - 1));
#pragma unroll
        for (int d = 0; d < NB; ++d)
#pragma unroll
          for (int i = 0; i < 16; ++i) {
            const int at = 32 * d + 8 * (i >> 2) + 4 * hi + (i & 3);
            if constexpr (C::Q8) {
              const uint16_t x = reinterpret_cast<const uint16_t*>(late->c.v_d)[from * NB + (at >> 1) % NB];
              if ((x & 0x7C00u) == 0x7C00u) acc[d][i] = __builtin_nanf("");
            } else {
              const uint16_t x = reinterpret_cast<const uint16_t*>(C::EXPANDED ? late->values : late->c.v)[from * (32 * NB) + at];
              if (not_finite<T>(x) & 0xFFFFu) acc[d][i] += (float)__builtin_bit_cast(T, x);
            }
          }
      }
  }
  if (s_bad || w.s.bad) l = __builtin_nanf("");
  if (split) {
    const int64_t slot = (int64_t)w.slot * late->Hkv + kvh;
    floatx4* dst = reinterpret_cast<floatx4*>(late->acc) + (slot * late->slot_waves + wave) * (NB * 4 * 64) + lane;
#pragma unroll
    for (int d = 0; d < NB; ++d)
#pragma unroll
      for (int j = 0; j < 4; ++j) dst[(4 * d + j) * 64] = floatx4{acc[d][4 * j], acc[d][4 * j + 1], acc[d][4 * j + 2], acc[d][4 * j + 3]};
    if (hi == 0) {
      late->stat[slot * (2 * kRows) + 32 * wave + c] = m;
      late->stat[slot * (2 * kRows) + kRows + 32 * wave + c] = l;
    }
    return;
  }
  if (!row.live) return;
  const float inv = l == 0.0f ? 0.0f : 1.0f / l;  // a query that sees no key gives zeros
  uint16_t* out = late->out + (int64_t)(w.s.q0 + row.query) * late->o_t + (int64_t)row.head * late->o_h;
#pragma unroll
  for (int d = 0; d < NB; ++d)
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const float x = acc[d][2 * j] * inv, y = acc[d][2 * j + 1] * inv;
      const int at = channel_of<C::MIXED, NB>(32 * d + 8 * (j >> 1) + 4 * hi + 2 * (j & 1));
      *reinterpret_cast<uint32_t*>(out + at) = late->type == NVQ_TYPE_F16 ? pack_pair<_Float16>(x, y) : pack_pair<__bf16>(x, y);
    }
}

// Q8_0 into binary16, tile blockIdx.x of key head and sequence blockIdx.y, where a sequence has so many row tiles
// that converting each tile once and reading twice the bytes costs less than converting it in every one of
// them.  Bound by memory: 16384 keys of 8 key heads of 128, 36 MB read and 67 written, 31 us.  A page number outside
// the cache makes NaN of its keys.
template <int NB>
__global__ __launch_bounds__(64 * kWaves) void attn_chunk_expand_kernel(ChunkArgs a) {
  typedef Cached<NVQ_KV_Q8_0, NB> C;
  __shared__ uint32_t s_top[kWaves];
  __shared__ int s_lost;
  const int lane = (int)threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6);
  const int b = uniform((int)blockIdx.y / a.Hkv), kvh = (int)blockIdx.y - b * a.Hkv;
  const Seq s = load_seq(a, b);
  const int n = uniform(s.n), m = uniform(s.m);
  const int start = max(n - m - a.window + 1, 0);  // of the first query's window
  const auto wanted = [&](int key, int count) { return m > 0 && key < n && (key + count > start || key < a.sinks); };
  const int tile0 = (int)blockIdx.x * kKeys, key0 = tile0 + 16 * wave;
  if (!wanted(tile0, kKeys)) return;
  int page = 0, count = 0;
  if (wanted(key0, 16)) {
    page = uniform(a.table[(int64_t)b * a.table_stride + (key0 >> a.c.page_shift)]);
    count = min(n - key0, 16);
  }
  const bool out = (uint32_t)page >= (uint32_t)a.c.n_pages;
  const int64_t from = (((int64_t)(out ? 0 : page) * a.Hkv + kvh) << a.c.page_shift) + (key0 & ((1 << a.c.page_shift) - 1));
  const int rows = out ? 0 : count, row_in = lane >> 2, seg = lane & 3;
  const auto buffer = [&](const void* p, int bytes) __attribute__((always_inline)) {
    return __builtin_amdgcn_make_buffer_rsrc((void*)(reinterpret_cast<const uint8_t*>(p) + from * bytes), 0, rows * bytes, 0x00020000);
  };
  typename Dwords<C::WORDS>::type codes[2];
  typename Dwords<C::SCALES>::type d[2];
#pragma unroll
  for (int x = 0; x < 2; ++x) {
    codes[x] = load_dwords<C::WORDS>(buffer(x ? a.c.v : a.c.k, C::ROW), row_in * C::ROW + seg * (C::ROW / 4));
    d[x] = load_row_scales<NB>(buffer(x ? a.c.v_d : a.c.k_d, 2 * NB), row_in);
  }
  if (!wanted(key0 + row_in, 1)) {  // between the first keys and the first query's window: no part in the tile's largest
#pragma unroll
    for (int i = 0; i < C::SCALES; ++i) d[0][i] = d[1][i] = 0;
  }
  const uint32_t mine = wave_largest(largest_scale<C::SCALES>(d[0]), largest_scale<C::SCALES>(d[1]));
  if (lane == 0) s_top[wave] = mine;
  if (threadIdx.x == 0) s_lost = 0;
  __syncthreads();
  const uint32_t top = (uint32_t)uniform((int)max_halves(max_halves(s_top[0], s_top[1]), max_halves(s_top[2], s_top[3])));
  // values: their largest scale in 2^1 .. 2^9, so that most tiles have one power, or where that loses bits, as the keys, as high as it goes
  const int ek = exponent_of(top >> 16), ev = exponent_of(top & 0xFFFFu);
  int e[2] = {ek == kNone ? 0 : highest(ek), ev == kNone ? 0 : max(((ev - 2) >> 3) << 3, -24)};
  if (ev != kNone && __syncthreads_or(lost_bits<C::SCALES>(d[1], scale_down<C::SCALES>(d[1], e[1])))) e[1] = highest(ev);
  const int64_t tile = (int64_t)blockIdx.y * a.tiles + blockIdx.x;
#pragma unroll
  for (int x = 0; x < 2; ++x) {
    const auto scales = scale_down<C::SCALES>(d[x], e[x]);
    if (__any(lost_bits<C::SCALES>(d[x], scales))) s_lost = 1;
    u32x4* const dst = reinterpret_cast<u32x4*>((x ? a.values : a.keys) + (tile * kKeys + 16 * wave + row_in) * (32 * NB)) + NB * seg;
#pragma unroll
    for (int i = 0; i < NB; ++i) {
      const u32x4 y = to_halves<NB>(codes[x], scales, i);
      dst[i] = x == 0 && out ? u32x4{~0u, ~0u, ~0u, ~0u} : y;
    }
  }
  __syncthreads();
  if (threadIdx.x == 0) a.units[tile] = (e[0] & 0xFF) | (s_lost ? kWide : 0) | (int)((uint32_t)e[1] << 16);
}

// Joins the parts of one row tile of a key head in their order: a workgroup takes 32 channels of its rows, so that a
// short call's few row tiles are on many compute units.  Latency: about 4 us of a small call.
template <int FMT, int NB>
__global__ __launch_bounds__(64 * kWaves) void attn_chunk_join_kernel(ChunkArgs a) {
  typedef Cached<FMT, NB> C;
  const int tid = (int)threadIdx.x, lane = tid & 63, c = lane & 31, hi = lane >> 5;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int item = uniform((int)blockIdx.x / a.Hkv), kvh = (int)blockIdx.x - item * a.Hkv, d = (int)blockIdx.y;
  const Work w = find_work(a, item, true);
  if (w.b < 0) return;
  const Rows rt = rows_of(a, w);
  const int parts = uniform((rt.tiles + w.part_tiles - 1) / w.part_tiles);
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
    const int at = channel_of<C::MIXED, NB>(32 * d + 8 * (j >> 1) + 4 * hi + 2 * (j & 1));
    *reinterpret_cast<uint32_t*>(row + at) = a.type == NVQ_TYPE_F16 ? pack_pair<_Float16>(x, y) : pack_pair<__bf16>(x, y);
  }
}

// What the host knows of the work's size.
struct Bound {
  int64_t tiles;   // row tiles of a key head
  int64_t keys;    // key tiles of one
  int64_t places;  // workgroups at once
  int64_t target;  // parts wanted, at most
  int64_t parts;   // parts at most
  int64_t slots;   // of them of split row tiles
  int slot_waves;
  int64_t expanded;  // Q8_0: key tiles of a sequence, turned into binary16 first; 0: not
};
Bound bound_of(int fmt, int64_t B, int64_t Tq, int64_t Hq, int64_t Hkv, int64_t D, int64_t capacity, int64_t window, int64_t sinks) {
  Bound b;
  const int64_t G = Hq / Hkv;
  b.tiles = Tq * G / kRows + B;
  b.keys = (capacity + kKeys - 1) / kKeys;
  if (window) {
    const int64_t seen = (sinks + kKeys - 1) / kKeys + (window + kRows - 1 + kKeys - 1) / kKeys + 1;
    b.keys = seen < b.keys ? seen : b.keys;
  }
  const int64_t at_once = places((int)(D / 32)) / Hkv;
  b.places = at_once < 1 ? 1 : at_once;
  b.target = kRounds * b.places;
  // a sequence of `tiles` row tiles that see up to `most` key tiles is cut into tiles * ceil(most / part), and part is at
  // least sum(tiles * most) / target
  const int64_t each = (b.keys + kMinPart - 1) / kMinPart, all = b.tiles * each;
  b.parts = all < b.target + b.tiles ? all : b.target + b.tiles;
  b.slots = each <= 1 ? 0 : all < 2 * b.target ? all : 2 * b.target;
  const int64_t rows = Tq * G < kRows ? Tq * G : kRows;
  b.slot_waves = (int)((rows + 31) / 32);
  const int64_t tiles = (capacity + kKeys - 1) / kKeys;
  const bool expand = fmt == NVQ_KV_Q8_0 && Tq * G >= B * kExpandRows && tiles <= kExpandBytes / (B * Hkv) / (kKeys * D * 4) && B * Hkv < 65536;
  b.expanded = expand ? tiles : 0;
  return b;
}

size_t partial_bytes(const Bound& b, int64_t Hkv, int64_t D) { return (size_t)(b.slots * Hkv) * ((size_t)b.slot_waves * 32 * D * 4 + 2 * kRows * 4); }

template <typename T, int FMT, int NB>
hipError_t launch_nb(const ChunkArgs& a, const Bound& b, hipStream_t s) {
  if constexpr (FMT == kExpanded) {
    hipLaunchKernelGGL((attn_chunk_expand_kernel<NB>), dim3((unsigned)b.expanded, (unsigned)(a.B * a.Hkv)), dim3(64 * kWaves), 0, s, a);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
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

size_t attn_chunk_workspace(int fmt, int64_t B, int64_t Tq, int64_t Hq, int64_t Hkv, int64_t D, int64_t capacity, int64_t window, int64_t sinks) {
  const Bound b = bound_of(fmt, B, Tq, Hq, Hkv, D, capacity, window, sinks);
  return partial_bytes(b, Hkv, D) + (size_t)(B * Hkv * b.expanded) * (size_t)(kKeys * D * 4 + 16);
}

bool attn_chunk_fits(int64_t B, int64_t Tq, int64_t Hq, int64_t Hkv, int64_t D, int64_t capacity) {
  const Bound b = bound_of(NVQ_KV_F16, B, Tq, Hq, Hkv, D, capacity, 0, 0);
  return Tq * (Hq / Hkv) < (int64_t(1) << 31) - 2 * kRows && b.tiles < (int64_t(1) << 31) / b.keys && b.parts * Hkv * (64 * kWaves) < int64_t(1) << 32;
}

hipError_t launch_attn_chunk(int fmt, int type, const void* q, void* out, const int64_t strides[4], int64_t B, int64_t Tq, int64_t Hq,
                             int64_t Hkv, int64_t D, const KvCache& c, const int32_t* table, int64_t table_stride, const int32_t* cu_q,
                             const int32_t* lengths, int window, int sinks, float scale, void* workspace, hipStream_t stream) {
  const Bound b = bound_of(fmt, B, Tq, Hq, Hkv, D, table_stride << c.page_shift, window, sinks);
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
  a.places = (int)b.places;
  a.slot_waves = b.slot_waves;
  a.slots = (int)b.slots;
  a.tiles = (int)b.expanded;
  a.keys = (uint16_t*)((uint8_t*)workspace + partial_bytes(b, Hkv, D));
  a.values = a.keys + B * Hkv * b.expanded * kKeys * D;
  a.units = (int*)(a.values + B * Hkv * b.expanded * kKeys * D);
  const int nb = (int)(D / 32);
  if (b.expanded) return launch_fmt<_Float16, kExpanded>(a, nb, b, stream);
  if (fmt == NVQ_KV_Q8_0) return launch_fmt<_Float16, NVQ_KV_Q8_0>(a, nb, b, stream);
  if (fmt == NVQ_KV_F16) return launch_fmt<_Float16, NVQ_KV_F16>(a, nb, b, stream);
  return launch_fmt<__bf16, NVQ_KV_BF16>(a, nb, b, stream);
}

}  // namespace nvq
