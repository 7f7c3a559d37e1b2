// attn_decode.hip -- attention of one new token per sequence over a paged key-value
// cache, on gfx950: out[b][h] = sum_j p_j v_j / sum_j p_j,  p_j = exp(scale q[b][h] . k_j).
//
// One pass over the cache with a running maximum and sum.  A workgroup takes one chunk of
// one sequence's keys and one key head; its four wavefronts take 32-key tiles in turn, each
// with statistics and an accumulator of its own, joined in LDS at the end.  All query heads
// of the key head (16 at a time) are the 16 columns of the matrix products:
//     S^T [32 keys][16 heads] = K [keys][D] q^T      (v_mfma_f32_16x16x32, keys are rows)
//     O^T [D][16 heads]      += V^T [D][keys] P^T
// A lane's scores are the keys 4 g + i (g = lane / 16) of two 16-key groups, and exactly
// those eight keys are the lane's part of the second product's contraction, whose order is
// free: the probabilities never leave their registers.
//
// Types.  Scores and results are as exact as float32 arithmetic makes them: the float
// operands (q and P) go in as the sum of two binary16 terms (22 bits; a query's channels are held to
// 2^-32 of its largest at least, a P too small for them goes another way) or three bfloat16
// terms (24 bits), accumulated in float32.  Q8_0 codes are whole numbers, exact in either type:
// a block's 32 channels are one instruction's contraction over the keys' codes, whose scale
// multiplies the block's sum in float32; the value scale goes into P.
//
// Loads.  A wavefront's tiles come straight into LDS (no registers wait for them), two tiles
// deep, with waits of its own counting; rows arrive in 1 KB loads whatever order the lanes read
// them in.  Non-temporal, since nothing reads a row again (64 sequences, bfloat16: 205 -> 187 us).
//
// What bounds it: memory.  64 ragged sequences of up to 8192 (8 key heads of 128, bfloat16, 1.09 GB):
// 190 us, 5.7 TB/s of the 7.1 that a plain read reaches.  Q8_0 halves the bytes and adds the
// conversions: 131071 keys (285 MB) 57 us, 5.0 TB/s, about 390 vector instructions a 32-key tile.
// Short calls are latency: 500 keys take 10 us in the two kernels, of which 3 join.
//
// Work split: the keys of all sequences are cut into chunks of one length, chosen on the
// device from the lengths so that about `target` workgroups share the chip; a second kernel
// joins the chunks of a sequence in their order (results do not depend on timing).
#include "attn_device.h"
#include "nvq_launch.h"

namespace nvq {

namespace {

constexpr int kTile = 32;          // keys of one wavefront's step
// The shortest chunk is one tile to a wavefront: 500 keys of 8 key heads in chunks of 128 take
// 10.2 us, in chunks of 256 11.6 (a tile's latency, 1.8 us, against the wait for one more part).
constexpr int kMinChunk = 128;  // keys
// Two workgroups to each of 256 compute units.  LDS holds that many at once, or more, over Q8_0 up
// to 128 channels and in 16 bits up to 64; from 160 channels in Q8_0 and 96 in 16 bits it holds one,
// and the second half waits.  Q8_0, 128 channels: 131071 keys 59 us, with 256 the same, with 1024 63 (8 ragged
// sequences of up to 4096: 17.6, 18.1 and 23).  No one number is best where one workgroup fits: binary16, 8 x 4096
// keys, 4 heads of 256: 44 us, with 256 34; bfloat16, 64 ragged sequences of 128 channels: 190 at either, with
// 1024 186.
constexpr int kTargetGroups = 512;
constexpr int kJoinWaves = 8;
// A score may pass the running maximum by 2^kSlack before everything is rescaled.
constexpr float kSlack = 8.0f;
// Over a bfloat16 cache P and its sum are taken times this, so that P is at most 1: values reach to the
// top of float32, and times 2^kSlack they would pass it where the result does not.
constexpr float kTopScale = 0x1p-8f;
// Over a binary16 cache P (at most 2^kSlack) goes in times kHalfScale, as two binary16 terms: the
// largest stays inside binary16, and 2^-20 of any P from kHalfLeast on is held.  Smaller ones lose
// bits and vanish below 2^-32, and behind a heavy key whose values are 0 what they add is the
// whole result; so a tile that has one goes in as bfloat16 terms, of P and of the values, which hold
// float32's range (5 products for 2).  64 x <= 8192 keys, 8 key heads of 128: 190 us with few such tiles
// (scores of width 1), 205 with most (width 3 and more); 16 x <= 2000, 16 of 64: 20.9 and 23.9.
constexpr float kHalfScale = 128.0f, kHalfLeast = 0x1p-12f;

struct DecodeArgs {
  const void* q;
  int64_t q_stride_b, q_stride_h;
  KvCache c;
  const int32_t* table;
  const int32_t* lengths;
  void* out;
  float* acc;   // [chunk * key heads * head tiles][2 D/32][64 lanes] float4
  float* stat;  // [chunk * key heads * head tiles][2][16]: maximum (base 2), sum
  float scale_log2;
  int type, B, Hq, Hkv, G, HT;
  int table_stride;  // pages of a table row
  int target;        // chunks wanted
};

// How the keys are cut: the chunk's length and, for chunk c, its sequence.
struct Plan {
  int b;       // sequence, -1: no such chunk
  int len;     // its keys (0 if the length is out of range, and bad is set)
  int first;   // its first chunk
  int count;   // its chunks, at least 1
  int chunk;   // keys of a chunk
  bool bad;
};

// want_b: find sequence `want`, else find the sequence of chunk `want`.  The whole wavefront
// calls it; the answer is uniform.  Capacities are below 2^30 keys in all (host check).
__device__ __forceinline__ Plan make_plan(const DecodeArgs& a, int want, bool want_b) {
  const int lane = (int)(threadIdx.x & 63);
  const int cap = a.table_stride << a.c.page_shift;
  int total = 0;
  for (int i = lane; i < a.B; i += 64) {
    const int n = a.lengths[i];
    total += n < 0 || n > cap ? 0 : n;
  }
  total = __builtin_amdgcn_readlane(wave_running_sum(total), 63);
  Plan p;
  // chunk >= total / target, so there are at most target + B chunks (chunk_bound); a multiple of
  // a step of four wavefronts
  const uint32_t unit = kTile * 4;
  // (every sequence's last chunk is a part of one: half of one is taken off for each)
  const uint32_t whole = (uint32_t)max(a.target - a.B / 2, (a.target + 3) / 4);
  const uint32_t even = ((uint32_t)total + whole - 1) / whole;
  p.chunk = max(kMinChunk, (int)((even + unit - 1) / unit * unit));
  int base = 0;
  p.b = -1;
  for (int i0 = 0; i0 < a.B; i0 += 64) {
    const int i = i0 + lane;
    const int raw = i < a.B ? a.lengths[i] : 0;
    const bool bad = raw < 0 || raw > cap;
    const int n = bad ? 0 : raw;
    const int chunks = i < a.B ? max(1, (int)(((uint32_t)n + (uint32_t)p.chunk - 1) / (uint32_t)p.chunk)) : 0;
    const int incl = wave_running_sum(chunks);
    const uint64_t hit = __ballot(want_b ? i == want : base + incl > want);
    if (hit) {
      const int l = __builtin_ctzll(hit);
      p.b = i0 + l;
      p.len = __builtin_amdgcn_readlane(n, l);
      p.count = __builtin_amdgcn_readlane(chunks, l);
      p.first = base + __builtin_amdgcn_readlane(incl, l) - p.count;
      p.bad = __builtin_amdgcn_readlane((int)bad, l) != 0;
      return p;
    }
    base += __builtin_amdgcn_readlane(incl, 63);
  }
  return p;
}

// N dwords of LDS from an address that is a multiple of 4 N bytes (up to 16) away from a
// 16-byte aligned one
template <int N>
__device__ __forceinline__ void read_dwords(const uint8_t* p, uint32_t* v) {
  if constexpr (N % 4 == 0) {
#pragma unroll
    for (int i = 0; i < N / 4; ++i) {
      const u32x4 t = reinterpret_cast<const u32x4*>(p)[i];
#pragma unroll
      for (int j = 0; j < 4; ++j) v[4 * i + j] = t[j];
    }
  } else if constexpr (N % 2 == 0) {
#pragma unroll
    for (int i = 0; i < N / 2; ++i) {
      const u32x2 t = reinterpret_cast<const u32x2*>(p)[i];
      v[2 * i] = t[0], v[2 * i + 1] = t[1];
    }
  } else {
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] = reinterpret_cast<const uint32_t*>(p)[i];
  }
}

template <int FMT, int NB>
struct Shape {
  static constexpr bool Q8 = FMT == NVQ_KV_Q8_0;
  static constexpr int ROW = Q8 ? 32 * NB : 64 * NB;  // bytes of a cache row
  static constexpr int KW = Q8 ? 2 * NB : 4 * NB;     // dwords of a lane's key row part
  static constexpr int VW = Q8 ? (NB + 1) / 2 : NB;   // dwords of a lane's part of one value row
  static constexpr int DW = Q8 ? 2 * NB : 1;          // dwords of four rows' scales
  static constexpr int TERMS = FMT == NVQ_KV_BF16 ? 3 : 2;  // of a query
  // P over Q8_0 goes in as bfloat16 terms: with the value scale in it, it needs float32's range
  typedef typename CacheType<Q8 ? NVQ_KV_BF16 : FMT>::type P;
  static constexpr int P_TERMS = Q8 || FMT == NVQ_KV_BF16 ? 3 : 2;
  static constexpr int TILES = 2 * NB;                // 16-channel tiles of the result
  // LDS of a tile: two 16-key groups of keys, the same of values, then both groups' key
  // scales and value scales
  static constexpr int GROUP = 16 * ROW, SCALES = Q8 ? 32 * NB : 0;
  static constexpr int SLOT = 4 * GROUP + 4 * SCALES;
  // Two tiles' room a wavefront.  Rows wider than 256 bytes leave room for two wavefronts.
  static constexpr int WAVES = 2 * 4 * SLOT <= 144 * 1024 ? 4 : 2;
  // Wavefronts of a SIMD that the registers are cut for: two (also where LDS leaves room for one), so that
  // the accumulator stays in ordinary registers (with one it moves to the other half and back in
  // every step), where it all fits.
  static constexpr int EU_WAVES = NB <= (Q8 ? 4 : 5) ? 2 : 1;
  // 16-byte pieces of a key row, and which row bits they are exchanged by in LDS, so that the
  // lanes of one piece of different rows fall on different banks (64 of 4 bytes)
  static constexpr int PIECES = ROW / 16;
  static constexpr bool SWIZZLE = (PIECES & (PIECES - 1)) == 0 && PIECES >= 4;
  static constexpr int SWIZZLE_SHIFT = PIECES >= 16 ? 0 : PIECES == 8 ? 1 : 2;
  // load instructions (1 KB each, or what is left) of a group; of a tile's keys with all scales
  static constexpr int LOADS = (GROUP + 1023) / 1024;
  static constexpr int K_LOADS = 2 * LOADS + (Q8 ? 1 : 0), V_LOADS = 2 * LOADS;
  static __device__ __forceinline__ int piece(int row, int i) { return SWIZZLE ? i ^ ((row >> SWIZZLE_SHIFT) & (PIECES - 1)) : i; }
};

// Where the lane's 16 bytes of load i of a group of key rows come from: LDS takes the pieces in
// order, so the exchange is made on this side.
template <int FMT, int NB>
__device__ __forceinline__ uint32_t swizzled_offset(int lane, int i) {
  typedef Shape<FMT, NB> S;
  const int at = 64 * i + lane, row = at / S::PIECES;
  return (uint32_t)(row * S::ROW + 16 * S::piece(row, at % S::PIECES));
}
__device__ __forceinline__ float half_of(const uint32_t* w, int i) {
  return f16_bits_to_f32((uint16_t)(i & 1 ? w[i >> 1] >> 16 : w[i >> 1]));
}

// Signed byte i of a and of b as a bfloat16 pair (whole numbers up to 127: exact, so the upper
// halves of their floats are it).
__device__ __forceinline__ uint32_t codes_to_bf16(uint32_t a, uint32_t b, int i) {
  const float x = (float)(int)(int8_t)(a >> (8 * i)), y = (float)(int)(int8_t)(b >> (8 * i));
  return perm(__builtin_bit_cast(uint32_t, y), __builtin_bit_cast(uint32_t, x), 0x07060302u);
}

// A binary16 pair as two bfloat16 pairs whose sum it is: the upper 8 of its 11 bits, and the rest.
__device__ __forceinline__ void halves_to_bf16(uint32_t v, uint32_t& top, uint32_t& rest) {
  float x[2];
  unpack_pair<_Float16>(v, x);
  const uint32_t a = __builtin_bit_cast(uint32_t, x[0]), b = __builtin_bit_cast(uint32_t, x[1]);
  top = perm(b, a, 0x07060302u);
  rest = perm(__builtin_bit_cast(uint32_t, x[1] - __builtin_bit_cast(float, b & 0xFFFF0000u)),
              __builtin_bit_cast(uint32_t, x[0] - __builtin_bit_cast(float, a & 0xFFFF0000u)), 0x07060302u);
}

// Eight floats as the sum of TERMS 16-bit operands, each the rounding of what the ones before
// leave (an exact difference).
template <typename T, int TERMS>
__device__ __forceinline__ void split_terms(const float (&x)[8], Frag (&f)[TERMS]) {
  float r[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) r[i] = x[i];
#pragma unroll
  for (int t = 0; t < TERMS; ++t) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      f[t].v[i] = pack_pair<T>(r[2 * i], r[2 * i + 1]);
      if (t + 1 < TERMS) {
        float h[2];
        unpack_pair<T>(f[t].v[i], h);
        r[2 * i] -= h[0], r[2 * i + 1] -= h[1];
      }
    }
  }
}

// The lane's 8 channels of each 32-block of a query row, from element `at` on.
template <int NB>
__device__ __forceinline__ void load_queries(const DecodeArgs& a, int64_t at, u32x4 (&raw)[NB][2]) {
  if (a.type == NVQ_TYPE_F32) {
    const float* p = reinterpret_cast<const float*>(a.q) + at;
#pragma unroll
    for (int bl = 0; bl < NB; ++bl)
#pragma unroll
      for (int i = 0; i < 2; ++i) raw[bl][i] = *reinterpret_cast<const u32x4*>(p + 32 * bl + 4 * i);
  } else {
    const uint16_t* p = reinterpret_cast<const uint16_t*>(a.q) + at;
#pragma unroll
    for (int bl = 0; bl < NB; ++bl) raw[bl][0] = *reinterpret_cast<const u32x4*>(p + 32 * bl), raw[bl][1] = u32x4{0, 0, 0, 0};
  }
}

// Their operands; over binary16 operands scaled to 2^7 .. 2^8 by a power of two, whose inverse is
// returned.
template <int FMT, int NB>
__device__ __forceinline__ float split_queries(int type, const u32x4 (&raw)[NB][2], Frag (&qf)[NB][Shape<FMT, NB>::TERMS]) {
  typedef Shape<FMT, NB> S;
  float x[NB][8];
#pragma unroll
  for (int bl = 0; bl < NB; ++bl)
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      float t[2];
      if (type == NVQ_TYPE_F32) {
        const uint32_t u = raw[bl][i >> 1][2 * (i & 1)], v = raw[bl][i >> 1][2 * (i & 1) + 1];
        t[0] = __builtin_bit_cast(float, u), t[1] = __builtin_bit_cast(float, v);
      } else if (type == NVQ_TYPE_F16) {
        unpack_pair<_Float16>(raw[bl][0][i], t);
      } else {
        unpack_pair<__bf16>(raw[bl][0][i], t);
      }
      x[bl][2 * i] = t[0], x[bl][2 * i + 1] = t[1];
    }
  float back = 1.0f;
  if constexpr (FMT != NVQ_KV_BF16) {
    float top = 0.0f;
#pragma unroll
    for (int bl = 0; bl < NB; ++bl)
#pragma unroll
      for (int i = 0; i < 8; ++i) top = fmaxf(top, fabsf(x[bl][i]));
    top = max_32(max_16(top));
    const int e = top > 0.0f && top < __builtin_inff() ? 8 - __builtin_amdgcn_frexp_expf(top) : 0;
#pragma unroll
    for (int bl = 0; bl < NB; ++bl)
#pragma unroll
      for (int i = 0; i < 8; ++i) x[bl][i] = __builtin_amdgcn_ldexpf(x[bl][i], e);
    back = __builtin_amdgcn_ldexpf(1.0f, -e);
  }
#pragma unroll
  for (int bl = 0; bl < NB; ++bl) split_terms<typename CacheType<FMT>::type, S::TERMS>(x[bl], qf[bl]);
  return back;
}

// Q (Q8_0): columns to a head.  With few query heads to a key head most of the 16 columns would
// be idle while every lane multiplies its probabilities by all blocks' value scales and splits
// them; so a head takes Q columns, and column q of them carries P times the scales of blocks q,
// q + Q, .. only.  All columns go through the products; of a block's channels, the column that
// carries its scale is the result.
template <int FMT, int NB, int Q>
__global__ __launch_bounds__((64 * Shape<FMT, NB>::WAVES), (Shape<FMT, NB>::EU_WAVES)) void attn_decode_kernel(DecodeArgs a) {
  typedef Shape<FMT, NB> S;
  constexpr int SETS = (NB + Q - 1) / Q;  // blocks of a column
  constexpr int kWaves = S::WAVES;
  typedef typename CacheType<FMT>::type T;
  const int lane = (int)(threadIdx.x & 63), n = lane & 15, g = lane >> 4;
  const int wave = __builtin_amdgcn_readfirstlane((int)(threadIdx.x >> 6));
  const int per = a.Hkv * a.HT;
  const int c = (int)blockIdx.x / per, hh = (int)blockIdx.x - c * per;
  const int kvh = hh / a.HT, h0 = (hh - kvh * a.HT) * 16;
  const Plan plan = make_plan(a, c, false);
  if (plan.b < 0) return;
  const int b = plan.b;
  const int k0 = (c - plan.first) * plan.chunk, k1 = min(plan.len, k0 + plan.chunk);

  // The query heads' rows on their way, in the keys' operand order: block bl, slot (g, s) is
  // channel 32 bl + 8 g + s.  Columns past the last head read it again.
  const int head = h0 + n / Q, group = n % Q;
  const bool live = head < a.G;
  u32x4 q_raw[NB][2];
  load_queries<NB>(a, b * a.q_stride_b + (int64_t)(kvh * a.G + min(head, a.G - 1)) * a.q_stride_h + 8 * g, q_raw);

  floatx4 acc[S::TILES];
#pragma unroll
  for (int t = 0; t < S::TILES; ++t) acc[t] = floatx4{0.f, 0.f, 0.f, 0.f};
  float m = -__builtin_inff(), l = 0.0f;
  bool bad_page = false;

  // The wavefront's tiles are s0, s0 + kWaves, ..; tile number t of them sits in slot t % 2.
  constexpr int kJoin = (kWaves - 1) * S::TILES * 64 * 16;
  __shared__ __align__(16) uint8_t s_ring[kWaves * 2 * S::SLOT > kJoin ? kWaves * 2 * S::SLOT : kJoin];
  uint8_t* const ring = s_ring + wave * (2 * S::SLOT);
  const uint32_t ring_at = __builtin_amdgcn_readfirstlane(lds_address(ring));
  const auto* table = (const __attribute__((address_space(4))) int32_t*)(a.table + (int64_t)b * a.table_stride);
  const int steps = (k1 - k0 + kTile - 1) / kTile;
  const int mine = steps > wave ? (steps - wave + kWaves - 1) / kWaves : 0;
  const int page_mask = (1 << a.c.page_shift) - 1;
  // a group past the end is the last group again (its scores are masked)
  const auto key_of = [&](int t, int u) __attribute__((always_inline)) { return min(k0 + (wave + t * kWaves) * kTile + 16 * u, (k1 - 1) & ~15); };
  const auto page_of = [&](int t, int u) __attribute__((always_inline)) { return mine > 0 ? table[key_of(t, u) >> a.c.page_shift] : 0; };
  // the cache rows of both groups of the tile that is loaded next (plain variables: an array
  // here would be kept in memory)
  int page_a = 0, page_b = 0;
  int64_t row_a = 0, row_b = 0;
  const auto row_in = [&](int page, int key) __attribute__((always_inline)) {
    const bool out = (uint32_t)page >= (uint32_t)a.c.n_pages;
    bad_page |= out;
    return (((int64_t)(out ? 0 : page) * a.Hkv + kvh) << a.c.page_shift) + (key & page_mask);
  };
  const auto look_up = [&](int t) __attribute__((always_inline)) { page_a = page_of(t, 0), page_b = page_of(t, 1); };
  const auto find_rows = [&](int t) __attribute__((always_inline)) { row_a = row_in(page_a, key_of(t, 0)), row_b = row_in(page_b, key_of(t, 1)); };
  const auto load_rows = [&](const void* codes, uint32_t at, bool keys) __attribute__((always_inline)) {
#pragma unroll
    for (int u = 0; u < 2; ++u)
#pragma unroll
      for (int i = 0; i < S::LOADS; ++i) {
        const uint32_t offset = S::SWIZZLE && keys ? swizzled_offset<FMT, NB>(lane, i) : (uint32_t)(16 * lane + 1024 * i);
        if (1024 * (i + 1) <= S::GROUP || 16 * lane + 1024 * i < S::GROUP)
          load_once_to_lds(reinterpret_cast<const uint8_t*>(codes) + (u ? row_b : row_a) * S::ROW, offset, at + u * S::GROUP + 1024 * i);
      }
  };
  const auto load_keys = [&](uint32_t at) __attribute__((always_inline)) {
    load_rows(a.c.k, at, true);
    if constexpr (S::Q8) {
      // lanes: 2 NB pieces each of the key scales of group 0, group 1, the value scales' 0, 1
      const int which = lane / (2 * NB), i = lane % (2 * NB);
      const uint8_t* kd = reinterpret_cast<const uint8_t*>(a.c.k_d);
      const int64_t row = (which & 1) ? row_b : row_a;
      const uint8_t* p = (which & 2 ? reinterpret_cast<const uint8_t*>(a.c.v_d) : kd) + row * (2 * NB) + 16 * i;
      if (lane < 8 * NB) load_once_to_lds_far(p, at + 4 * S::GROUP);
    }
  };
  const auto load_values = [&](uint32_t at) __attribute__((always_inline)) { load_rows(a.c.v, at + 2 * S::GROUP, false); };

  if (mine > 0) {
    look_up(0);
    find_rows(0);
    load_keys(ring_at);
    load_values(ring_at);
    if (mine > 1) look_up(1);
  }
  // (the first use of the queries waits for all loads so far: the first tile is among them,
  // the second one follows)
  Frag qf[NB][S::TERMS];
  const float to_log2 = a.scale_log2 * split_queries<FMT, NB>(a.type, q_raw, qf);
  if (mine > 1) {
    find_rows(1);
    load_keys(ring_at + S::SLOT);
    load_values(ring_at + S::SLOT);
    if (mine > 2) look_up(2);
  }

  for (int t = 0; t < mine; ++t) {
    const int key0 = k0 + (wave + t * kWaves) * kTile;
    const uint8_t* slot = ring + (t & 1) * S::SLOT;
    const uint32_t slot_at = ring_at + (t & 1) * S::SLOT;
    // outstanding behind this tile's keys: its values and the next tile
    if (t + 1 < mine)
      wait_loads<S::V_LOADS + S::K_LOADS + S::V_LOADS>();
    else
      wait_loads<S::V_LOADS>();
    uint32_t kw[2][S::KW], kd[2][S::DW];
    uint16_t vd[S::Q8 ? SETS : 1][8];  // the value scales that the column carries
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      const uint8_t* p = slot + u * S::GROUP + n * S::ROW;
      if constexpr (S::Q8 && S::SWIZZLE) {
#pragma unroll
        for (int i = 0; i < NB / 2; ++i) read_dwords<4>(p + 16 * S::piece(n, NB / 2 * g + i), kw[u] + 4 * i);
      } else if constexpr (S::Q8) {
        read_dwords<S::KW>(p + 8 * NB * g, kw[u]);
      } else {
#pragma unroll
        for (int bl = 0; bl < NB; ++bl) read_dwords<4>(p + 16 * S::piece(n, 4 * bl + g), kw[u] + 4 * bl);
      }
      if constexpr (S::Q8) {
        // both tensors' scales come and go with the keys: they are read before the next keys are
        // sent for
        read_dwords<S::DW>(slot + 4 * S::GROUP + u * S::SCALES + 8 * NB * g, kd[u]);
        const uint16_t* d = reinterpret_cast<const uint16_t*>(slot + 4 * S::GROUP + (2 + u) * S::SCALES) + 4 * g * NB;
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
          for (int set = 0; set < SETS; ++set) vd[set][4 * u + i] = d[i * NB + min(set * Q + group, NB - 1)];
      }
    }
    const bool more = t + 2 < mine;
    if (more) {
      find_rows(t + 2);
      wait_reads();
      load_keys(slot_at);
      if (t + 3 < mine) look_up(t + 3);
    }
    float sc[8];
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      floatx4 sum = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int bl = 0; bl < NB; ++bl) {
        Frag f;
        if constexpr (S::Q8) {
#pragma unroll
          for (int j = 0; j < 4; ++j) {  // the pair of channels 32 bl + 8 g + 2 j, + 1
            const int at = 2 * NB * j + 2 * bl;
            const uint32_t w = perm(0x64646464u, kw[u][at / 4] ^ 0x80808080u, at & 2 ? 0x04030402u : 0x04010400u);
            f.v[j] = __builtin_bit_cast(uint32_t, __builtin_bit_cast(half2_t, w) - half2_t{(_Float16)1152.0f, (_Float16)1152.0f});
          }
          floatx4 part = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
          for (int e = 0; e < S::TERMS; ++e) part = mfma16<T>(f, qf[bl][e], part);
#pragma unroll
          for (int i = 0; i < 4; ++i) sum[i] = __builtin_fmaf(half_of(kd[u], i * NB + bl), part[i], sum[i]);
        } else {
#pragma unroll
          for (int j = 0; j < 4; ++j) f.v[j] = kw[u][4 * bl + j];
#pragma unroll
          for (int e = 0; e < S::TERMS; ++e) sum = mfma16<T>(f, qf[bl][e], sum);
        }
      }
#pragma unroll
      for (int i = 0; i < 4; ++i) sc[4 * u + i] = sum[i] * to_log2;
    }

    if (more)
      wait_loads<S::K_LOADS + S::V_LOADS + S::K_LOADS>();
    else if (t + 1 < mine)
      wait_loads<S::K_LOADS + S::V_LOADS>();
    else
      wait_loads<0>();
    uint32_t vw[2][4][S::VW];
#pragma unroll
    for (int u = 0; u < 2; ++u)
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const uint8_t* p = slot + (2 + u) * S::GROUP + (4 * g + i) * S::ROW;
        if constexpr (!S::Q8) {
          read_dwords<S::VW>(p + 4 * NB * n, vw[u][i]);
        } else if constexpr (NB % 2 == 0) {
          read_dwords<S::VW>(p + 2 * NB * n, vw[u][i]);
        } else {
          const uint16_t* h = reinterpret_cast<const uint16_t*>(p + 2 * NB * n);
#pragma unroll
          for (int bl = 0; bl < NB; bl += 2) vw[u][i][bl / 2] = h[bl] | (bl + 1 < NB ? (uint32_t)h[bl + 1] << 16 : 0u);
        }
      }
    if (more) {
      wait_reads();
      load_values(slot_at);
    }

    if (key0 + kTile > k1) {
      // keys past the end: no probability, and nothing of what their rows hold (never written,
      // perhaps NaN) may reach the products
#pragma unroll
      for (int u = 0; u < 2; ++u)
#pragma unroll
        for (int i = 0; i < 4; ++i)
          if (key0 + 16 * u + 4 * g + i >= k1) {
            sc[4 * u + i] = -__builtin_inff();
            if constexpr (S::Q8) {
#pragma unroll
              for (int set = 0; set < SETS; ++set) vd[set][4 * u + i] = 0;
            } else {
#pragma unroll
              for (int w = 0; w < S::VW; ++w) vw[u][i][w] = 0;
            }
          }
    }
    float top = sc[0];
#pragma unroll
    for (int i = 1; i < 8; ++i) top = fmaxf(top, sc[i]);
    if (__any(top > m + kSlack)) {
      const float m_new = fmaxf(m, max_32(max_16(top)));
      const float f = m_new == -__builtin_inff() ? 1.0f : exp2_fast(m - m_new);
      l *= f;
#pragma unroll
      for (int i = 0; i < S::TILES; ++i) acc[i] *= f;
      m = m_new;
    }
    const float m_safe = m == -__builtin_inff() ? 0.0f : m;
    float p[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      p[i] = exp2_fast(sc[i] - m_safe);
      if constexpr (FMT == NVQ_KV_BF16) p[i] *= kTopScale;
      l += p[i];
    }
    if constexpr (S::Q8) {
#pragma unroll
      for (int set = 0; set < SETS; ++set) {
        float x[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) x[i] = __builtin_fmaf(f16_bits_to_f32(vd[set][i]), p[i], 0.0f);
        Frag pf[S::P_TERMS];
        split_terms<typename S::P, S::P_TERMS>(x, pf);
#pragma unroll
        for (int at = 2 * Q * set; at < 2 * min(Q * set + Q, NB); ++at) {  // channels 32 (at / 2) + 2 n + at % 2
          Frag f;
#pragma unroll
          for (int j = 0; j < 4; ++j)  // keys 2 j, 2 j + 1 of the lane's eight
            f.v[j] = codes_to_bf16(vw[j >> 1][2 * (j & 1)][at >> 2], vw[j >> 1][2 * (j & 1) + 1][at >> 2], at & 3);
#pragma unroll
          for (int k = 0; k < S::P_TERMS; ++k) acc[at] = mfma16<typename S::P>(f, pf[k], acc[at]);
        }
      }
    } else {
      const auto values = [&](int i) __attribute__((always_inline)) {  // channels 2 NB n + i
        Frag f;
#pragma unroll
        for (int j = 0; j < 4; ++j)
          f.v[j] = perm(vw[j >> 1][2 * (j & 1) + 1][i >> 1], vw[j >> 1][2 * (j & 1)][i >> 1], i & 1 ? 0x07060302u : 0x05040100u);
        return f;
      };
      bool small = false;
      if constexpr (FMT == NVQ_KV_F16) {
        uint32_t least = ~0u;  // of the P that are not 0: its bits, less 1
#pragma unroll
        for (int i = 0; i < 8; ++i) least = min(least, __builtin_bit_cast(uint32_t, p[i]) - 1u);
        small = __any(least < __builtin_bit_cast(uint32_t, kHalfLeast) - 1u);
#pragma unroll
        for (int i = 0; i < 8; ++i) p[i] *= kHalfScale;
      }
      if (!small) {
        Frag pf[S::P_TERMS];
        split_terms<typename S::P, S::P_TERMS>(p, pf);
#pragma unroll
        for (int i = 0; i < S::TILES; ++i) {
          const Frag f = values(i);
#pragma unroll
          for (int k = 0; k < S::P_TERMS; ++k) acc[i] = mfma16<typename S::P>(f, pf[k], acc[i]);
        }
      } else {
        Frag pf[3];
        split_terms<__bf16, 3>(p, pf);
#pragma unroll
        for (int i = 0; i < S::TILES; ++i) {
          Frag f = values(i), rest;
#pragma unroll
          for (int j = 0; j < 4; ++j) halves_to_bf16(f.v[j], f.v[j], rest.v[j]);
#pragma unroll
          for (int k = 0; k < 3; ++k) acc[i] = mfma16<__bf16>(f, pf[k], acc[i]);
#pragma unroll
          for (int k = 0; k < 2; ++k) acc[i] = mfma16<__bf16>(rest, pf[k], acc[i]);  // (the third: below 2^-25 of it all)
        }
      }
    }
  }

  // Join the wavefronts.
  __shared__ float s_m[kWaves][16], s_l[kWaves][16];
  floatx4* const s_acc = reinterpret_cast<floatx4*>(s_ring);  // [kWaves - 1][TILES][64]; the tiles have been read
  l = sum_32(sum_16(l));
  if (bad_page || plan.bad) l = __builtin_nanf("");
  if (g == 0) s_m[wave][n] = m, s_l[wave][n] = l;
  __syncthreads();
  float all = s_m[0][n];
#pragma unroll
  for (int w = 1; w < kWaves; ++w) all = fmaxf(all, s_m[w][n]);
  const auto weight = [&](float x) { return x == -__builtin_inff() ? 0.0f : exp2_fast(x - all); };
  const float wt = FMT == NVQ_KV_F16 ? weight(m) / kHalfScale : weight(m);
#pragma unroll
  for (int t = 0; t < S::TILES; ++t) acc[t] *= wt;
  if (wave != 0) {
#pragma unroll
    for (int t = 0; t < S::TILES; ++t) s_acc[((wave - 1) * S::TILES + t) * 64 + lane] = acc[t];
  }
  __syncthreads();
  if (wave != 0) return;
  float sum = 0.0f;
#pragma unroll
  for (int w = 0; w < kWaves; ++w) sum += weight(s_m[w][n]) * s_l[w][n];
#pragma unroll
  for (int w = 0; w < kWaves - 1; ++w)
#pragma unroll
    for (int t = 0; t < S::TILES; ++t) acc[t] += s_acc[(w * S::TILES + t) * 64 + lane];

  if (plan.count > 1) {
    floatx4* dst = reinterpret_cast<floatx4*>(a.acc) + (int64_t)blockIdx.x * (S::TILES * 64) + lane;
#pragma unroll
    for (int t = 0; t < S::TILES; ++t) dst[t * 64] = acc[t];
    if (g == 0) {
      a.stat[(int64_t)blockIdx.x * 32 + n] = all;
      a.stat[(int64_t)blockIdx.x * 32 + 16 + n] = sum;
    }
    return;
  }
  if (!live) return;
  // no key, or none with a probability: zeros
  const float inv = sum == 0.0f ? 0.0f : 1.0f / sum;
  const int64_t at = ((int64_t)b * a.Hq + kvh * a.G + head) * (32 * NB);
  if constexpr (S::Q8) {
#pragma unroll
    for (int bl = 0; bl < NB; ++bl) {
      if (group != bl % Q) continue;
      float x[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) x[i] = acc[2 * bl + (i & 1)][i >> 1] * inv;
      store_n<8>(a.out, a.type, at + 32 * bl + 8 * g, x);
    }
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      float x[2 * NB];
#pragma unroll
      for (int t = 0; t < S::TILES; ++t) x[t] = acc[t][i] * inv;
      store_n<2 * NB>(a.out, a.type, at + 2 * NB * (4 * g + i), x);
    }
  }
}

// Joins the chunks of sequence blockIdx.x / (Hkv HT) in their order.  Of a workgroup's eight
// wavefronts, APART take 16-channel tiles of their own and the others share those tiles'
// chunks: all eight apart where there are sequences enough to fill the chip (64 sequences of
// about 4 chunks, 128 channels: 5 us; sharing 15), none where a few sequences have many chunks.
template <int FMT, int NB, int Q, int APART>
__global__ __launch_bounds__(64 * kJoinWaves) void attn_decode_join_kernel(DecodeArgs a) {
  typedef Shape<FMT, NB> S;
  constexpr int kWaves = kJoinWaves / APART;
  const int lane = (int)(threadIdx.x & 63), n = lane & 15, g = lane >> 4;
  const int wave_id = __builtin_amdgcn_readfirstlane((int)(threadIdx.x >> 6));
  const int own_tile = wave_id % APART, wave = wave_id / APART;
  const int per = a.Hkv * a.HT;
  const int b = (int)blockIdx.x / per, hh = (int)blockIdx.x - b * per;
  const bool in = (int)blockIdx.y * APART + own_tile < S::TILES;
  const int tile = min((int)blockIdx.y * APART + own_tile, S::TILES - 1);
  const Plan plan = make_plan(a, b, true);
  if (plan.count <= 1) return;
  // per is the distance of a sequence's chunks; a wavefront takes chunks wave, wave + kWaves, ..,
  // four at a time with all their loads in flight, with a running maximum of its own
  const float* stat = a.stat + ((int64_t)plan.first * per + hh) * 32 + n;
  const floatx4* src = reinterpret_cast<const floatx4*>(a.acc) + ((int64_t)plan.first * per + hh) * (S::TILES * 64) + tile * 64 + lane;
  floatx4 acc = {0.f, 0.f, 0.f, 0.f};
  float sum = 0.0f, top = -__builtin_inff();
  constexpr int kBatch = 4;
  for (int c0 = wave; c0 < plan.count; c0 += kBatch * kWaves) {
    floatx4 part[kBatch];
    float m[kBatch], l[kBatch];
#pragma unroll
    for (int j = 0; j < kBatch; ++j) {
      const int64_t c = (int64_t)min(c0 + j * kWaves, plan.count - 1) * per;
      part[j] = src[c * (S::TILES * 64)];
      m[j] = stat[c * 32], l[j] = stat[c * 32 + 16];
    }
    float m_new = top;
#pragma unroll
    for (int j = 0; j < kBatch; ++j) {
      if (c0 + j * kWaves >= plan.count) m[j] = -__builtin_inff(), l[j] = 0.0f, part[j] = floatx4{0.f, 0.f, 0.f, 0.f};
      m_new = fmaxf(m_new, m[j]);
    }
    const float f = m_new == -__builtin_inff() ? 1.0f : exp2_fast(top - m_new);
    acc *= f, sum *= f;
#pragma unroll
    for (int j = 0; j < kBatch; ++j) {
      const float w = m[j] == -__builtin_inff() ? 0.0f : exp2_fast(m[j] - m_new);
      acc += part[j] * w, sum += l[j] * w;
    }
    top = m_new;
  }
  if constexpr (kWaves > 1) {
    __shared__ float s_top[kWaves][16], s_sum[kWaves - 1][64];
    __shared__ floatx4 s_acc[kWaves - 1][64];
    static_assert(APART == 1, "one tile to a workgroup whose wavefronts share it");
    if (g == 0) s_top[wave][n] = top;
    __syncthreads();
    float all = s_top[0][n];
#pragma unroll
    for (int w = 1; w < kWaves; ++w) all = fmaxf(all, s_top[w][n]);
    const float own = top == -__builtin_inff() ? 0.0f : exp2_fast(top - all);
    acc *= own, sum *= own;
    if (wave != 0) s_acc[wave - 1][lane] = acc, s_sum[wave - 1][lane] = sum;
    __syncthreads();
    if (wave != 0) return;
#pragma unroll
    for (int w = 0; w < kWaves - 1; ++w) acc += s_acc[w][lane], sum += s_sum[w][lane];
  }
  if (!in) return;
  const int kvh = hh / a.HT, head = (hh - kvh * a.HT) * 16 + n / Q;
  if (head >= a.G || n % Q != (tile >> 1) % Q) return;
  const float inv = sum == 0.0f ? 0.0f : 1.0f / sum;
  const int64_t at = ((int64_t)b * a.Hq + kvh * a.G + head) * (32 * NB);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int ch = S::Q8 ? 32 * (tile >> 1) + 8 * g + 2 * i + (tile & 1) : 2 * NB * (4 * g + i) + tile;
    store_1(a.out, a.type, at + ch, acc[i] * inv);
  }
}

int head_tiles(int64_t G) { return (int)((G + 15) / 16); }

// Chunks wanted, and the most there can be.
int64_t chunk_target(int64_t Hkv, int64_t G) {
  const int64_t t = kTargetGroups / (Hkv * head_tiles(G));
  return t < 1 ? 1 : t;
}
int64_t chunk_bound(int64_t B, int64_t Hkv, int64_t G, int64_t capacity) {
  const int64_t most = B * ((capacity + kMinChunk - 1) / kMinChunk);
  const int64_t t = chunk_target(Hkv, G) + B;
  return most < t ? most : t;
}

template <int FMT, int NB, int Q>
hipError_t launch_q(const DecodeArgs& a, int64_t blocks, bool join, hipStream_t s) {
  hipLaunchKernelGGL((attn_decode_kernel<FMT, NB, Q>), dim3((unsigned)blocks), dim3(64 * Shape<FMT, NB>::WAVES), 0, s, a);
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess || !join) return e;
  const unsigned rows = (unsigned)(a.B * a.Hkv * a.HT);
  if (rows >= 256)
    hipLaunchKernelGGL((attn_decode_join_kernel<FMT, NB, Q, kJoinWaves>), dim3(rows, (2 * NB + kJoinWaves - 1) / kJoinWaves), dim3(64 * kJoinWaves), 0, s, a);
  else
    hipLaunchKernelGGL((attn_decode_join_kernel<FMT, NB, Q, 1>), dim3(rows, 2 * NB), dim3(64 * kJoinWaves), 0, s, a);
  return hipGetLastError();
}
template <int FMT, int NB>
hipError_t launch_nb(const DecodeArgs& a, int64_t blocks, bool join, hipStream_t s) {
  if constexpr (FMT == NVQ_KV_Q8_0) {
    if constexpr (NB >= 4) {
      if (a.G <= 4) return launch_q<FMT, NB, 4>(a, blocks, join, s);
    }
    if constexpr (NB >= 3) {
      if (a.G <= 5) return launch_q<FMT, NB, 3>(a, blocks, join, s);
    }
    if constexpr (NB >= 2) {
      if (a.G <= 8) return launch_q<FMT, NB, 2>(a, blocks, join, s);
    }
  }
  return launch_q<FMT, NB, 1>(a, blocks, join, s);
}
template <int FMT>
hipError_t launch_fmt(const DecodeArgs& a, int nb, int64_t blocks, bool join, hipStream_t s) {
  switch (nb) {
    case 1: return launch_nb<FMT, 1>(a, blocks, join, s);
    case 2: return launch_nb<FMT, 2>(a, blocks, join, s);
    case 3: return launch_nb<FMT, 3>(a, blocks, join, s);
    case 4: return launch_nb<FMT, 4>(a, blocks, join, s);
    case 5: return launch_nb<FMT, 5>(a, blocks, join, s);
    case 6: return launch_nb<FMT, 6>(a, blocks, join, s);
    case 7: return launch_nb<FMT, 7>(a, blocks, join, s);
    default: return launch_nb<FMT, 8>(a, blocks, join, s);
  }
}

}  // namespace

size_t attn_decode_workspace(int64_t B, int64_t Hq, int64_t Hkv, int64_t D, int64_t capacity) {
  if (capacity <= kMinChunk) return 0;  // one chunk to a sequence: nothing to join
  const int64_t G = Hq / Hkv;
  const int64_t groups = chunk_bound(B, Hkv, G, capacity) * Hkv * head_tiles(G);
  return (size_t)groups * ((size_t)(D / 16) * 64 * 16 + 2 * 16 * 4);
}

bool attn_decode_fits(int64_t B, int64_t Hq, int64_t Hkv, int64_t capacity) {
  constexpr int64_t most = int64_t(1) << 32;
  const int64_t per = Hkv * head_tiles(Hq / Hkv);
  return chunk_bound(B, Hkv, Hq / Hkv, capacity) * per * 256 < most && (capacity <= kMinChunk || B * per * (64 * kJoinWaves) < most);
}

hipError_t launch_attn_decode(int fmt, int type, const void* q, int64_t q_stride_b, int64_t q_stride_h, int64_t B,
                              int64_t Hq, int64_t Hkv, int64_t D, const KvCache& c, const int32_t* table,
                              int64_t table_stride, const int32_t* lengths, float scale, void* out, void* workspace,
                              hipStream_t stream) {
  DecodeArgs a;
  a.q = q, a.q_stride_b = q_stride_b, a.q_stride_h = q_stride_h;
  a.c = c;
  a.table = table, a.lengths = lengths, a.out = out;
  a.scale_log2 = scale * 1.44269504088896340736f;  // log2(e): powers of two from here on
  a.type = type, a.B = (int)B, a.Hq = (int)Hq, a.Hkv = (int)Hkv, a.G = (int)(Hq / Hkv), a.HT = head_tiles(Hq / Hkv);
  a.table_stride = (int)table_stride;
  a.target = (int)chunk_target(Hkv, a.G);
  const int64_t capacity = table_stride << c.page_shift;
  const int64_t groups = chunk_bound(B, Hkv, a.G, capacity) * Hkv * a.HT;
  a.acc = (float*)workspace;
  a.stat = a.acc + groups * (D / 16) * 64 * 4;
  const bool join = capacity > kMinChunk;
  const int nb = (int)(D / 32);
  if (fmt == NVQ_KV_Q8_0) return launch_fmt<NVQ_KV_Q8_0>(a, nb, groups, join, stream);
  if (fmt == NVQ_KV_F16) return launch_fmt<NVQ_KV_F16>(a, nb, groups, join, stream);
  return launch_fmt<NVQ_KV_BF16>(a, nb, groups, join, stream);
}

}  // namespace nvq
