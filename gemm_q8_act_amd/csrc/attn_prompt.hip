// attn_prompt.hip -- causal attention of whole packed prompts on gfx950, grouped heads:
//     out[i][h] = sum_j p_ij v_j / sum_j p_ij,  p_ij = exp(scale q[i][h] . k[j][h / G]),
// where query i of a sequence with m queries and n keys sees keys j <= i + n - m.
//
// A workgroup takes 128 queries of one head, a wavefront 32 of them, and walks the keys
// in tiles with a running maximum and sum.  Both products are v_mfma_f32_32x32x16 with
// queries as columns:
//     S^T [keys][32 queries] = K Q^T,      O^T [D][32 queries] += V^T P^T
// A lane's scores are keys 8 j + 4 (lane / 32) + i of its query, and exactly those are its
// part of the second product's contraction, whose order is free: the probabilities go from
// the softmax into the product without leaving their registers.  V^T's operands are read from
// the row-major tile by the transposing LDS read (ds_read_b64_tr_b16).
//
// Probabilities enter the second product rounded once to the operands' type, as the sum that divides it
// takes them; scores, statistics and accumulators are float32.  That rounding is as large as the
// result's own and makes errors 1.1 to 1.4 times those of a float32 form.  Two terms would double the
// second product, half of the work.
//
// What bounds it: issue.  A wavefront's 64-key step is 8 D/32 products of 32 cycles, each beside
// one exponential and about 4 other vector instructions (128 channels): 8192 tokens of
// 40 heads of 128 over 8 key heads take 610 to 640 us by the card, up to 1120 TFLOP/s, the matrix cores busy
// 59 % of it.
// So a step's vector work (the softmax of tile t) stands beside products that do not depend on it
// (the scores of tile t + 1), two wavefronts share a SIMD, and tiles come straight into LDS, which is
// read for one product at a time.  32 queries a wavefront, since 64 do not fit the registers
// (1980 us); all of a wavefront's keys by itself, since two wavefronts to 32 queries, every
// other tile each, take 685 us (2048 tokens: 67 against 54; 256 tokens: 12.5 against 10.5).
// Short prompts are latency: 256 tokens 10.5 us, of which 3 are start-up and 4 steps of 1.3.
#include "attn_device.h"
#include "nvq_launch.h"

namespace nvq {

namespace {

// Every query tile of every head; a multiple of the chip's parts (find_place).
int64_t prompt_groups(int64_t B, int64_t Tq, int64_t Hq) { return ((Tq / 128 + B) * Hq + 7) / 8 * 8; }

constexpr int kWaves = 4;
constexpr int kQueries = 32 * kWaves;
constexpr int kKeys = 64;  // of a tile
// A score may pass the running maximum by 2^SLACK before everything is rescaled; probabilities are
// taken times 2^SHIFT.  In bfloat16 they are at most 1 with it: values reach to the top of float32, and
// times 2^SLACK they would pass it where the result does not.  In binary16 together 2^15, all that the type has room for: it keeps its 11
// bits of a probability down to 2^-25 of the largest (17 nats) and holds them down to 2^-36.  (With 2^8
// and 2^0, keys 16 nats below a heavy one whose values are 0 were off by 9 times the half unit.  The smaller slack
// costs nothing at scores of width 1 and 1.6 % at width 3: 8192 tokens 675 and 696 us.)
template <typename T>
struct Range {
  static constexpr float SLACK = 8.0f, SHIFT = -8.0f;
};
template <>
struct Range<_Float16> {
  static constexpr float SLACK = 4.0f, SHIFT = 11.0f;
};
// What is taken from a score (base 2) with the running maximum m
template <typename T>
__device__ __forceinline__ float score_base(float m) {
  return (m == -__builtin_inff() ? 0.0f : m) - Range<T>::SHIFT;
}

struct PromptArgs {
  const uint16_t *q, *k, *v;
  uint16_t* out;
  int64_t q_t, q_h, k_t, k_h, v_t, v_h, o_t, o_h;  // token and head strides, elements
  const int32_t *cu_q, *cu_k;
  int B, Hq, Hkv, G;
  int Tq, Tk;
  float scale_log2;  // not negative; the sign is in flip
  uint32_t flip;     // sign bits of a query pair
  int causal;
};

// Which head and which query tile (of all sequences) a workgroup takes.  Workgroups go round the
// chip's 8 dies, each with an L2 of its own, so the query heads of a key head stay on one die
// (or, with fewer than 8 key heads, on as few as there are): its keys and values are read into
// one L2.  Tiles in rising order on every die; find_span counts them from the long ones.
struct Place {
  int head, tile;
};
__device__ __forceinline__ Place find_place(const PromptArgs& a) {
  const int x = (int)blockIdx.x % 8, r = (int)blockIdx.x / 8;
  int kvh, g, tile;
  if (a.Hkv % 8 == 0) {
    const int heads = a.G * (a.Hkv / 8), i = r % heads;
    tile = r / heads, kvh = x + 8 * (i / a.G), g = i % a.G;
  } else if (8 % a.Hkv == 0) {
    const int i = r * (8 / a.Hkv) + x / a.Hkv;
    tile = i / a.G, kvh = x % a.Hkv, g = i % a.G;
  } else {
    tile = (int)blockIdx.x / a.Hq;
    return {(int)blockIdx.x % a.Hq, tile};
  }
  return {kvh * a.G + g, tile};
}

struct Span {
  int q0, m, k0, n;  // the sequence's first query and number of them, and keys
  int tile;          // its query tile
};

// The sequence and its tile that tile number `want` falls in (last tiles, with the most keys,
// first).  Row numbers out of order or past the tensors are brought into range.
__device__ __forceinline__ bool find_span(const PromptArgs& a, int want, Span& s) {
  const int lane = (int)(threadIdx.x & 63);
  int base = 0;
  for (int i0 = 0; i0 < a.B; i0 += 64) {
    const int i = i0 + lane;
    int lo = 0, hi = 0, key_lo = 0, key_hi = 0;
    if (i < a.B) {  // (both tensors' offsets in one round trip to memory)
      lo = a.cu_q[i], hi = a.cu_q[i + 1], key_lo = a.cu_k[i], key_hi = a.cu_k[i + 1];
      lo = min(max(lo, 0), a.Tq), hi = min(max(hi, lo), a.Tq);
      key_lo = min(max(key_lo, 0), a.Tk), key_hi = min(max(key_hi, key_lo), a.Tk);
    }
    const int tiles = (hi - lo + kQueries - 1) / kQueries;
    const int incl = wave_running_sum(tiles);
    const uint64_t hit = __ballot(base + incl > want);
    if (hit) {
      const int l = __builtin_ctzll(hit);
      s.q0 = __builtin_amdgcn_readlane(lo, l);
      s.m = __builtin_amdgcn_readlane(hi, l) - s.q0;
      s.tile = base + __builtin_amdgcn_readlane(incl, l) - 1 - want;
      s.k0 = __builtin_amdgcn_readlane(key_lo, l);
      s.n = __builtin_amdgcn_readlane(key_hi, l) - s.k0;
      return true;
    }
    base += __builtin_amdgcn_readlane(incl, 63);
  }
  return false;
}

// A staged tile of 64 key (or value) rows: where its 16-byte pieces sit.  The rows follow one
// another; within a row the pieces are exchanged by row bits, so that the lanes of one LDS
// read, which take one piece of different rows (keys), or 32 bytes of each of four rows
// (values, transposed), fall on different banks (64 of 4 bytes).
template <int NB>
struct Stage {
  static constexpr int ROW = 64 * NB, PIECES = 4 * NB, BYTES = kKeys * ROW;
  static constexpr int LOADS = BYTES / 1024 / kWaves;  // 1 KB loads of a wavefront
  // (an exchange stays inside aligned groups of 16, 8 or 4 pieces, so it fits any row)
  static __device__ __forceinline__ int key_piece(int row, int i) {
    return PIECES % 16 == 0 ? i ^ (row & 15) : PIECES % 8 == 0 ? i ^ ((row >> 1) & 7) : i ^ ((row >> 2) & 3);
  }
  static __device__ __forceinline__ int value_piece(int row, int i) {
    return PIECES % 16 == 0 ? i ^ ((row & 3) << 2) : PIECES % 8 == 0 ? i ^ ((row & 2) << 1) : i;
  }
};

// Query `row_q` of a head by itself, out of memory and on the vector unit, for its keys 0 .. limit:
// lanes take keys for the scores, pairs of channels for the result.  `base`: what is taken from the
// scores (score_base).  Its tiles reached to row `last` of the values: nothing is done if no
// channel has a value that is not finite behind `limit`, or if a NaN among the last 64 rows up to it
// makes the same NaN of the channel (as where a channel is NaN in every row).  A query costs all its keys
// in one wavefront, so a call the square of its length.  40/8 heads of 128, 2048 tokens: 0.44 ms with NaN in every
// value, 4.5 with one such row, 10 with an infinite channel, and at 8192 tokens 115.
template <typename T, int NB>
__device__ __forceinline__ void one_query(const PromptArgs& a, const Span& sp, int head, int kvh, int row_q, int limit, int last, float base) {
  const int lane = (int)(threadIdx.x & 63);
  constexpr int SETS = (NB + 3) / 4;  // pairs 64 x + lane
  const auto value_pair = [&](int j, int x, float (&y)[2]) __attribute__((always_inline)) {
    unpack_pair<T>(*reinterpret_cast<const uint32_t*>(a.v + (int64_t)(sp.k0 + j) * a.v_t + (int64_t)kvh * a.v_h + 2 * (64 * x + lane)), y);
  };
  bool lost = false;
#pragma unroll
  for (int x = 0; x < SETS; ++x)
    if (64 * x + lane < 16 * NB) {
      float unseen[2] = {0.0f, 0.0f}, seen[2] = {0.0f, 0.0f}, y[2];
#pragma unroll 4
      for (int j = limit + 1 < 0 ? 0 : limit + 1; j <= last; ++j) {
        value_pair(j, x, y);
        unseen[0] = __builtin_fmaf(y[0], 0.0f, unseen[0]), unseen[1] = __builtin_fmaf(y[1], 0.0f, unseen[1]);
      }
#pragma unroll 4
      for (int j = limit < 63 ? 0 : limit - 63; j <= limit; ++j) {
        value_pair(j, x, y);
        seen[0] = y[0] != y[0] ? y[0] : seen[0], seen[1] = y[1] != y[1] ? y[1] : seen[1];
      }
#pragma unroll
      for (int e = 0; e < 2; ++e) lost |= unseen[e] != unseen[e] && seen[e] == seen[e];
    }
  if (!__any(lost)) return;
  const uint16_t* q = a.q + (int64_t)row_q * a.q_t + (int64_t)head * a.q_h;
  float acc[SETS][2] = {}, l = 0.0f;
  for (int j0 = 0; j0 <= limit; j0 += 64) {
    float p = 0.0f;
    if (j0 + lane <= limit) {
      const uint16_t* k = a.k + (int64_t)(sp.k0 + j0 + lane) * a.k_t + (int64_t)kvh * a.k_h;
      float s = 0.0f;
      for (int ch = 0; ch < 32 * NB; ch += 8) {
        const u32x4 u = *reinterpret_cast<const u32x4*>(q + ch), w = *reinterpret_cast<const u32x4*>(k + ch);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          float x[2], y[2];
          unpack_pair<T>(u[e] ^ a.flip, x);
          unpack_pair<T>(w[e], y);
          s = __builtin_fmaf(x[0], y[0], s), s = __builtin_fmaf(x[1], y[1], s);
        }
      }
      float t[2];  // (rounded to the operand type as everywhere)
      unpack_pair<T>(pack_pair<T>(exp2_fast(__builtin_fmaf(s, a.scale_log2, -base)), 0.0f), t);
      p = t[0];
    }
    const int some = min(64, limit - j0 + 1);
#pragma unroll 4
    for (int jj = 0; jj < some; ++jj) {
      const float pj = __builtin_bit_cast(float, __builtin_amdgcn_readlane(__builtin_bit_cast(int, p), jj));
      l += pj;
#pragma unroll
      for (int x = 0; x < SETS; ++x)
        if (64 * x + lane < 16 * NB) {
          float y[2];
          value_pair(j0 + jj, x, y);
          acc[x][0] = __builtin_fmaf(pj, y[0], acc[x][0]), acc[x][1] = __builtin_fmaf(pj, y[1], acc[x][1]);
        }
    }
  }
  const float inv = l == 0.0f ? 0.0f : 1.0f / l;
  uint16_t* out = a.out + (int64_t)row_q * a.o_t + (int64_t)head * a.o_h;
#pragma unroll
  for (int x = 0; x < SETS; ++x)
    if (64 * x + lane < 16 * NB) *reinterpret_cast<uint32_t*>(out + 2 * (64 * x + lane)) = pack_pair<T>(acc[x][0] * inv, acc[x][1] * inv);
}

template <typename T, int NB>
__global__ __launch_bounds__(64 * kWaves, NB <= 4 ? 2 : 1) void attn_prompt_kernel(PromptArgs a) {
  typedef Stage<NB> S;
  __shared__ __align__(16) uint8_t s_keys[2 * S::BYTES], s_values[2 * S::BYTES];
  const int tid = (int)threadIdx.x, lane = tid & 63, c = lane & 31, hi = lane >> 5;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const Place place = find_place(a);
  Span sp;
  if (!find_span(a, place.tile, sp)) return;
  const int head = place.head, kvh = head / a.G;
  const int i0 = sp.tile * kQueries, iw = i0 + 32 * wave, i = iw + c;  // the block's and the wavefront's first query, the lane's
  const int shift = sp.n - sp.m;
  const int limit = a.causal ? min(i + shift, sp.n - 1) : sp.n - 1;  // the last key it sees; below 0: none
  // keys that the block's and the wavefront's last query see, in tiles
  const int end = a.causal ? min(sp.n, min(i0 + kQueries, sp.m) + shift) : sp.n;
  const int end_w = iw >= sp.m ? 0 : a.causal ? min(sp.n, min(iw + 32, sp.m) + shift) : sp.n;
  const int tiles = end > 0 ? (end + kKeys - 1) / kKeys : 0, mine = end_w > 0 ? (end_w + kKeys - 1) / kKeys : 0;
  // from here on a tile has keys that some of the wavefront's queries do not see
  const int whole = (a.causal ? min(sp.n, max(iw + shift + 1, 0)) : sp.n) / kKeys;

  // Tiles on their way into LDS: load j of the wavefront takes 64 pieces, one a lane, in LDS
  // order.  A tile's descriptor ends behind the sequence's last row: what a load asks for past
  // it comes as zeros (and nothing is read), the same for whole tiles past the end.
  uint32_t key_from[S::LOADS], value_from[S::LOADS];
#pragma unroll
  for (int j = 0; j < S::LOADS; ++j) {
    const int id = (wave * S::LOADS + j) * 64 + lane, row = id / S::PIECES, pos = id % S::PIECES;
    key_from[j] = (uint32_t)row * (uint32_t)(2 * a.k_t) + 16 * S::key_piece(row, pos);
    value_from[j] = (uint32_t)row * (uint32_t)(2 * a.v_t) + 16 * S::value_piece(row, pos);
  }
  const uint32_t keys_at = lds_address(s_keys) + (uint32_t)(wave * S::LOADS * 1024);
  const uint32_t values_at = lds_address(s_values) + (uint32_t)(wave * S::LOADS * 1024);
  const auto tile_of = [&](const uint16_t* p, int64_t stride_t, int64_t stride_h, int t) __attribute__((always_inline)) {
    const int rows = min(sp.n - t * kKeys, kKeys);
    return buffer_of(p + ((int64_t)sp.k0 + (int64_t)t * kKeys) * stride_t + (int64_t)kvh * stride_h,
                     rows > 0 ? (uint32_t)(rows - 1) * (uint32_t)(2 * stride_t) + S::ROW : 0u);
  };

  const auto load_values = [&](int t, int slot) __attribute__((always_inline)) {
    const u32x4 values = tile_of(a.v, a.v_t, a.v_h, t);
#pragma unroll
    for (int j = 0; j < S::LOADS; ++j) buffer_to_lds(values, value_from[j], values_at + slot * S::BYTES + 1024 * j);
  };
  const auto load_keys = [&](int t, int slot) __attribute__((always_inline)) {
    const u32x4 keys = tile_of(a.k, a.k_t, a.k_h, t);
#pragma unroll
    for (int j = 0; j < S::LOADS; ++j) buffer_to_lds(keys, key_from[j], keys_at + slot * S::BYTES + 1024 * j);
  };
  // (in the order in which they are needed: the queries come back behind the first tile)
  if (tiles > 0) {
    load_keys(0, 0);
    load_values(0, 0);
    load_keys(1, 1);
  }
  Frag qf[2 * NB];
  {
    const uint16_t* row = a.q + (int64_t)(sp.q0 + min(i, sp.m - 1)) * a.q_t + (int64_t)head * a.q_h;
#pragma unroll
    for (int ks = 0; ks < 2 * NB; ++ks) {
      const u32x4 w = *reinterpret_cast<const u32x4*>(row + 16 * ks + 8 * hi);
#pragma unroll
      for (int j = 0; j < 4; ++j) qf[ks].v[j] = w[j] ^ a.flip;
    }
  }

  floatx16 acc[NB];
#pragma unroll
  for (int t = 0; t < NB; ++t)
#pragma unroll
    for (int j = 0; j < 16; ++j) acc[t][j] = 0.0f;
  float m = -__builtin_inff(), l = 0.0f, top = -__builtin_inff();

  uint32_t key_offset[2 * NB], value_offset[NB];
#pragma unroll
  for (int ks = 0; ks < 2 * NB; ++ks) key_offset[ks] = in_vgpr((uint32_t)(c * S::ROW + 16 * S::key_piece(c, 2 * ks + hi)));
  {
    const int jj = lane & 15, row_in = 4 * hi + (jj >> 2), half = (lane >> 4) & 1;
#pragma unroll
    for (int d = 0; d < NB; ++d)
      value_offset[d] = in_vgpr((uint32_t)(row_in * S::ROW + 16 * S::value_piece(row_in, 4 * d + 2 * half + ((jj & 3) >> 1)) + 8 * (jj & 1)));
  }
  // S^T of the tile in a slot; between the products, the loads of the values and keys that
  // come next, one to two products, so that none waits for the others' issue
  const auto scores = [&](int slot, floatx16 (&s)[2], auto load) __attribute__((always_inline)) {
    const uint8_t* tile = s_keys + slot * S::BYTES;
#pragma unroll
    for (int kb = 0; kb < 2; ++kb)
#pragma unroll
      for (int j = 0; j < 16; ++j) s[kb][j] = 0.0f;
#pragma unroll
    for (int ks = 0; ks < 2 * NB; ++ks)
#pragma unroll
      for (int kb = 0; kb < 2; ++kb) {
        const u32x4 w = *reinterpret_cast<const u32x4*>(tile + key_offset[ks] + 32 * kb * S::ROW);
        s[kb] = mfma32<T>(Frag{w[0], w[1], w[2], w[3]}, qf[ks], s[kb]);
        if (kb) load(ks);
      }
  };
  // Tile t: no score for keys that the query does not see; then its largest (the lane's part)
  const auto largest = [&](floatx16 (&s)[2]) __attribute__((always_inline)) {
    float x = s[0][0];
#pragma unroll
    for (int kb = 0; kb < 2; ++kb)
#pragma unroll
      for (int j = 0; j < 16; ++j) x = fmaxf(x, s[kb][j]);
    top = x * a.scale_log2;
  };
  const auto finish_scores = [&](int t, floatx16 (&s)[2]) __attribute__((always_inline)) {
    if (t >= whole) {
#pragma unroll
      for (int kb = 0; kb < 2; ++kb)
#pragma unroll
        for (int j = 0; j < 16; ++j)
          if (t * kKeys + 32 * kb + 8 * (j >> 2) + 4 * hi + (j & 3) > limit) s[kb][j] = -__builtin_inff();
      largest(s);
    }
  };
  // Tile t in `slot`: its probabilities and their product with the values, and the next tile's
  // scores, which depend on neither
  const auto step = [&](int t, int slot, floatx16 (&s)[2], floatx16 (&next)[2]) __attribute__((always_inline)) {
    if (__any(top > m + Range<T>::SLACK)) {
      const float m_new = fmaxf(m, max_32(top));
      const float f = m_new == -__builtin_inff() ? 1.0f : exp2_fast(m - m_new);
      l *= f;
#pragma unroll
      for (int d = 0; d < NB; ++d) acc[d] *= f;
      m = m_new;
    }
    const u32x4 values = tile_of(a.v, a.v_t, a.v_h, t + 1), keys = tile_of(a.k, a.k_t, a.k_h, t + 2);
    scores(slot ^ 1, next, [&](int j) __attribute__((always_inline)) {
      if (j < S::LOADS)
        buffer_to_lds(values, value_from[j], values_at + (slot ^ 1) * S::BYTES + 1024 * j);
      else
        buffer_to_lds(keys, key_from[j - S::LOADS], keys_at + slot * S::BYTES + 1024 * (j - S::LOADS));
    });
    const float base = score_base<T>(m);
    Frag pf[2][2];
#pragma unroll
    for (int kb = 0; kb < 2; ++kb)
#pragma unroll
      for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const float x = exp2_fast(__builtin_fmaf(s[kb][8 * h + 2 * j], a.scale_log2, -base));
          const float y = exp2_fast(__builtin_fmaf(s[kb][8 * h + 2 * j + 1], a.scale_log2, -base));
          pf[kb][h].v[j] = pack_pair<T>(x, y);
          l = add_pair<T>(pf[kb][h].v[j], l);
        }
    const uint8_t* tile = s_values + slot * S::BYTES;
#pragma unroll
    for (int kb = 0; kb < 2; ++kb)
#pragma unroll
      for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int d = 0; d < NB; ++d) {
          Frag f;
#pragma unroll
          for (int r = 0; r < 2; ++r) {
            const u32x2 x = read_transposed(tile + value_offset[d] + (32 * kb + 16 * h + 8 * r) * S::ROW);
            f.v[2 * r] = x[0], f.v[2 * r + 1] = x[1];
          }
          acc[d] = mfma32<T>(f, pf[kb][h], acc[d]);
        }
    largest(next);
    finish_scores(t + 1, next);
  };

  // Before tile t's step: its values and the next tile's keys are there, and everyone is done
  // with the slots that the step's loads go to.  Wavefronts with no query that sees the tile
  // only load their share.
  const auto turn = [&]() __attribute__((always_inline)) {
    wait_loads<0>();
    wait_reads();
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
  };
  floatx16 sa[2], sb[2];
  if (tiles > 0) {
    turn();
    if (mine > 0) {
      scores(0, sa, [](int) __attribute__((always_inline)) {});
      largest(sa);
      finish_scores(0, sa);
    }
    const auto pass = [&](int t, int slot, floatx16 (&s)[2], floatx16 (&next)[2]) __attribute__((always_inline)) {
      turn();
      if (t < mine) {
        step(t, slot, s, next);
      } else {
        load_values(t + 1, slot ^ 1);
        load_keys(t + 2, slot);
      }
    };
    for (int t = 0;;) {
      pass(t, 0, sa, sb);
      if (++t >= tiles) break;
      pass(t, 1, sb, sa);
      if (++t >= tiles) break;
    }
    wait_loads<0>();  // (zeros for tiles past the end): LDS is another workgroup's next
  }

  l = sum_32(l);
  const float inv = l == 0.0f ? 0.0f : 1.0f / l;  // a query that sees no key gives zeros
  // A value that is not finite, in a row that a query does not see but whose tile it takes part
  // in, has made 0 times it, NaN, of the query's sum.  So a query with numbers for its
  // probabilities and none for its result is done again by itself.  (The test behind the stores, in
  // four chains, is hidden: 256 tokens 10.5 us with and without it; in front of them 10.9.)
  float z[4] = {0.0f, 0.0f, 0.0f, 0.0f};  // 0, or NaN if any result is not finite
  uint16_t* row = a.out + (int64_t)(sp.q0 + min(i, sp.m - 1)) * a.o_t + (int64_t)head * a.o_h;
#pragma unroll
  for (int t = 0; t < NB; ++t)
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const u32x2 w = {pack_pair<T>(acc[t][4 * j] * inv, acc[t][4 * j + 1] * inv), pack_pair<T>(acc[t][4 * j + 2] * inv, acc[t][4 * j + 3] * inv)};
      if (i < sp.m) *reinterpret_cast<u32x2*>(row + 32 * t + 8 * j + 4 * hi) = w;
      z[j] = zero_of_pair<T>(w[1], zero_of_pair<T>(w[0], z[j]));
    }
  const float none = (z[0] + z[1]) + (z[2] + z[3]);
  const uint64_t broken = __ballot(a.causal && i < sp.m && l == l && none != none);
  uint32_t again = (uint32_t)broken | (uint32_t)(broken >> 32);
  if (__builtin_expect(again == 0, 1)) return;
  wait_loads<0>();  // (for the stores: the rows are written over)
  for (; again; again &= again - 1) {
    const int x = __builtin_ctz(again);
    const float m_x = __builtin_bit_cast(float, __builtin_amdgcn_readlane(__builtin_bit_cast(int, m), x));
    one_query<T, NB>(a, sp, head, kvh, sp.q0 + iw + x, min(iw + x + shift, sp.n - 1), min(sp.n, mine * kKeys) - 1, score_base<T>(m_x));
  }
}

template <typename T, int NB>
hipError_t launch_nb(const PromptArgs& a, hipStream_t s) {
  hipLaunchKernelGGL((attn_prompt_kernel<T, NB>), dim3((unsigned)prompt_groups(a.B, a.Tq, a.Hq)), dim3(64 * kWaves), 0, s, a);
  return hipGetLastError();
}
template <typename T>
hipError_t launch_type(const PromptArgs& a, int nb, hipStream_t s) {
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

}  // namespace

bool attn_prompt_fits(int64_t B, int64_t Tq, int64_t Hq) { return prompt_groups(B, Tq, Hq) * (64 * kWaves) < int64_t(1) << 32; }

hipError_t launch_attn_prompt(int type, const void* q, const void* k, const void* v, void* out, const int64_t strides[8],
                              const int32_t* cu_q, const int32_t* cu_k, int64_t B, int64_t Tq, int64_t Tk, int64_t Hq,
                              int64_t Hkv, int64_t D, float scale, int causal, hipStream_t stream) {
  PromptArgs a;
  a.q = (const uint16_t*)q, a.k = (const uint16_t*)k, a.v = (const uint16_t*)v, a.out = (uint16_t*)out;
  a.q_t = strides[0], a.q_h = strides[1], a.k_t = strides[2], a.k_h = strides[3];
  a.v_t = strides[4], a.v_h = strides[5], a.o_t = strides[6], a.o_h = strides[7];
  // the token stride of a single row, which has no meaning, tells the kernel where rows end
  if (Tk <= 1) a.k_t = a.v_t = D;
  a.cu_q = cu_q, a.cu_k = cu_k;
  a.B = (int)B, a.Hq = (int)Hq, a.Hkv = (int)Hkv, a.G = (int)(Hq / Hkv), a.Tq = (int)Tq, a.Tk = (int)Tk;
  // a negative scale turns the queries round, so that the largest score is the largest product
  // (a scale of 0 becomes a number that still makes -infinity of a masked score)
  a.scale_log2 = __builtin_fabsf(scale) * 1.44269504088896340736f;
  if (a.scale_log2 == 0.0f) a.scale_log2 = 1e-37f;
  a.flip = __builtin_signbit(scale) ? 0x80008000u : 0u;
  a.causal = causal;

  if (type == NVQ_TYPE_F16) return launch_type<_Float16>(a, (int)(D / 32), stream);
  return launch_type<__bf16>(a, (int)(D / 32), stream);
}

}  // namespace nvq
