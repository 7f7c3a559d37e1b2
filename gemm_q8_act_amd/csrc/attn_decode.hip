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
// operands (q and P) go in as the sum of two binary16 terms (22 bits) or three bfloat16 terms
// (24 bits), accumulated in float32.  Q8_0 codes are whole numbers, exact in either type:
// a block's 32 channels are one instruction's contraction over the keys' codes, whose scale
// multiplies the block's sum in float32; the value scale goes into P.
//
// Work split: the keys of all sequences are cut into chunks of one length, chosen on the
// device from the lengths so that about `target` workgroups share the chip; a second kernel
// joins the chunks of a sequence in their order (results do not depend on timing).
#include "attn_device.h"
#include "nvq_launch.h"

namespace nvq {

namespace {

constexpr int kWaves = 4;
constexpr int kTile = 32;          // keys of one wavefront's step
constexpr int kMinChunk = 256;     // keys
constexpr int kTargetGroups = 1024;
// A score may pass the running maximum by 2^kSlack before everything is rescaled.
constexpr float kSlack = 8.0f;
// Over a binary16 cache P (at most 2^kSlack) goes in times this: both its terms stay inside
// binary16, and one that is 2^-22 of the largest still has 11 bits.
constexpr float kHalfScale = 128.0f;

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

__device__ __forceinline__ int wave_sum(int v) {
#pragma unroll
  for (int o = 32; o; o >>= 1) v += __shfl_xor(v, o, 64);
  return v;
}

// want_b: find sequence `want`, else find the sequence of chunk `want`.  The whole wavefront
// calls it; the answer is uniform.  Capacities are below 2^31 keys in all (host check).
__device__ __forceinline__ Plan make_plan(const DecodeArgs& a, int want, bool want_b) {
  const int lane = (int)(threadIdx.x & 63);
  const int cap = a.table_stride << a.c.page_shift;
  int total = 0;
  for (int i = lane; i < a.B; i += 64) {
    const int n = a.lengths[i];
    total += n < 0 || n > cap ? 0 : n;
  }
  total = wave_sum(total);
  Plan p;
  // chunk >= total / target, so there are at most target + B chunks; a multiple of a step
  // of all four wavefronts
  const uint32_t unit = kTile * kWaves;
  const uint32_t even = ((uint32_t)total + (uint32_t)a.target - 1) / (uint32_t)a.target;
  p.chunk = max(kMinChunk, (int)((even + unit - 1) / unit * unit));
  int base = 0;
  p.b = -1;
  for (int i0 = 0; i0 < a.B; i0 += 64) {
    const int i = i0 + lane;
    const int raw = i < a.B ? a.lengths[i] : 0;
    const bool bad = raw < 0 || raw > cap;
    const int n = bad ? 0 : raw;
    const int chunks = i < a.B ? max(1, (int)(((uint32_t)n + (uint32_t)p.chunk - 1) / (uint32_t)p.chunk)) : 0;
    int incl = chunks;
#pragma unroll
    for (int o = 1; o < 64; o <<= 1) {
      const int t = __shfl_up(incl, o, 64);
      incl += lane >= o ? t : 0;
    }
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

// N dwords from an address that is a multiple of 4 N bytes (up to 16) away from a 16-byte
// aligned one
template <int N>
__device__ __forceinline__ void load_dwords(const uint8_t* p, uint32_t* v) {
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
};

// One wavefront's 32 keys: group u holds keys base_u .. base_u + 15, all in one page.
template <int FMT, int NB>
struct Tile {
  typedef Shape<FMT, NB> S;
  uint32_t k[2][S::KW];
  uint32_t v[2][4][S::VW];
  uint32_t kd[2][S::DW], vd[2][S::DW];
};

template <int FMT, int NB>
__device__ __forceinline__ void load_group(const DecodeArgs& a, int64_t row0, int u, Tile<FMT, NB>& t) {
  typedef Shape<FMT, NB> S;
  const int lane = (int)(threadIdx.x & 63), n = lane & 15, g = lane >> 4;
  const uint8_t* k = reinterpret_cast<const uint8_t*>(a.c.k) + row0 * S::ROW;
  const uint8_t* v = reinterpret_cast<const uint8_t*>(a.c.v) + row0 * S::ROW;
  if constexpr (S::Q8) {
    load_dwords<S::KW>(k + (uint32_t)(n * S::ROW + 8 * NB * g), t.k[u]);
  } else {
#pragma unroll
    for (int b = 0; b < NB; ++b) load_dwords<4>(k + (uint32_t)(n * S::ROW + 64 * b + 16 * g), t.k[u] + 4 * b);
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if constexpr (S::Q8) {
      const uint8_t* p = v + (uint32_t)((4 * g + i) * S::ROW + 2 * NB * n);
      if constexpr (NB % 2 == 0) {
        load_dwords<S::VW>(p, t.v[u][i]);
      } else {
        const uint16_t* h = reinterpret_cast<const uint16_t*>(p);
#pragma unroll
        for (int b = 0; b < NB; b += 2) t.v[u][i][b / 2] = h[b] | (b + 1 < NB ? (uint32_t)h[b + 1] << 16 : 0u);
      }
    } else {
      load_dwords<S::VW>(v + (uint32_t)((4 * g + i) * S::ROW + 4 * NB * n), t.v[u][i]);
    }
  }
  if constexpr (S::Q8) {
    load_dwords<S::DW>(reinterpret_cast<const uint8_t*>(a.c.k_d) + row0 * (2 * NB) + (uint32_t)(8 * NB * g), t.kd[u]);
    load_dwords<S::DW>(reinterpret_cast<const uint8_t*>(a.c.v_d) + row0 * (2 * NB) + (uint32_t)(8 * NB * g), t.vd[u]);
  }
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

template <int FMT, int NB>
__global__ __launch_bounds__(64 * kWaves, NB <= 3 ? 2 : 1) void attn_decode_kernel(DecodeArgs a) {
  typedef Shape<FMT, NB> S;
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

  // The query heads' rows, scaled to 2^7 .. 2^8 by a power of two (binary16 terms), in the
  // keys' operand order: block bl, slot (g, s) is channel 32 bl + 8 g + s.
  const bool live = h0 + n < a.G;
  Frag qf[NB][S::TERMS];
  float to_log2 = a.scale_log2;
  {
    float x[NB][8];
    float top = 0.0f;
#pragma unroll
    for (int bl = 0; bl < NB; ++bl) {
      if (live)
        load_8(a.q, a.type, b * a.q_stride_b + (int64_t)(kvh * a.G + h0 + n) * a.q_stride_h + 32 * bl + 8 * g, x[bl]);
      else
        for (int i = 0; i < 8; ++i) x[bl][i] = 0.0f;
#pragma unroll
      for (int i = 0; i < 8; ++i) top = fmaxf(top, fabsf(x[bl][i]));
    }
    if constexpr (FMT != NVQ_KV_BF16) {
      top = max_32(max_16(top));
      const int e = top > 0.0f && top < __builtin_inff() ? 8 - __builtin_amdgcn_frexp_expf(top) : 0;
#pragma unroll
      for (int bl = 0; bl < NB; ++bl)
#pragma unroll
        for (int i = 0; i < 8; ++i) x[bl][i] = __builtin_amdgcn_ldexpf(x[bl][i], e);
      to_log2 = __builtin_amdgcn_ldexpf(to_log2, -e);
    }
#pragma unroll
    for (int bl = 0; bl < NB; ++bl) split_terms<T, S::TERMS>(x[bl], qf[bl]);
  }

  floatx4 acc[S::TILES];
#pragma unroll
  for (int t = 0; t < S::TILES; ++t) acc[t] = floatx4{0.f, 0.f, 0.f, 0.f};
  float m = -__builtin_inff(), l = 0.0f;
  bool bad_page = false;

  const int32_t* table = a.table + (int64_t)b * a.table_stride;
  const int steps = (k1 - k0 + kTile - 1) / kTile;
  const int page_mask = (1 << a.c.page_shift) - 1;
  const auto load_tile = [&](int s, Tile<FMT, NB>& t) {
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      // a group past the end reads the last group again (its scores are masked)
      const int key = min(k0 + s * kTile + 16 * u, (k1 - 1) & ~15);
      int pg = table[key >> a.c.page_shift];
      const bool out = (uint32_t)pg >= (uint32_t)a.c.n_pages;
      bad_page |= out;
      pg = out ? 0 : pg;
      load_group<FMT, NB>(a, (((int64_t)pg * a.Hkv + kvh) << a.c.page_shift) + (key & page_mask), u, t);
    }
  };

  const auto step = [&](int s, Tile<FMT, NB>& t) {
    const int key0 = k0 + s * kTile;
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
            const uint32_t w = perm(0x64646464u, t.k[u][at / 4] ^ 0x80808080u, at & 2 ? 0x04030402u : 0x04010400u);
            f.v[j] = __builtin_bit_cast(uint32_t, __builtin_bit_cast(half2_t, w) - half2_t{(_Float16)1152.0f, (_Float16)1152.0f});
          }
          floatx4 part = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
          for (int e = 0; e < S::TERMS; ++e) part = mfma16<T>(f, qf[bl][e], part);
#pragma unroll
          for (int i = 0; i < 4; ++i) sum[i] = __builtin_fmaf(half_of(t.kd[u], i * NB + bl), part[i], sum[i]);
        } else {
#pragma unroll
          for (int j = 0; j < 4; ++j) f.v[j] = t.k[u][4 * bl + j];
#pragma unroll
          for (int e = 0; e < S::TERMS; ++e) sum = mfma16<T>(f, qf[bl][e], sum);
        }
      }
#pragma unroll
      for (int i = 0; i < 4; ++i) sc[4 * u + i] = sum[i] * to_log2;
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
              for (int bl = 0; bl < NB; ++bl) {
                const int at = i * NB + bl;
                t.vd[u][at >> 1] &= at & 1 ? 0x0000FFFFu : 0xFFFF0000u;
              }
            } else {
#pragma unroll
              for (int w = 0; w < S::VW; ++w) t.v[u][i][w] = 0;
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
      l += p[i];
    }
    if constexpr (FMT == NVQ_KV_F16) {
#pragma unroll
      for (int i = 0; i < 8; ++i) p[i] *= kHalfScale;
    }
    if constexpr (S::Q8) {
#pragma unroll
      for (int bl = 0; bl < NB; ++bl) {
        float x[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) x[i] = p[i] * half_of(t.vd[i >> 2], (i & 3) * NB + bl);
        Frag pf[S::P_TERMS];
        split_terms<typename S::P, S::P_TERMS>(x, pf);
#pragma unroll
        for (int e = 0; e < 2; ++e) {  // channels 32 bl + 2 n + e
          Frag f;
          const int at = 2 * bl + e;
#pragma unroll
          for (int j = 0; j < 4; ++j)  // keys 2 j, 2 j + 1 of the lane's eight
            f.v[j] = codes_to_bf16(t.v[j >> 1][2 * (j & 1)][at >> 2], t.v[j >> 1][2 * (j & 1) + 1][at >> 2], at & 3);
#pragma unroll
          for (int k = 0; k < S::P_TERMS; ++k) acc[2 * bl + e] = mfma16<typename S::P>(f, pf[k], acc[2 * bl + e]);
        }
      }
    } else {
      Frag pf[S::P_TERMS];
      split_terms<typename S::P, S::P_TERMS>(p, pf);
#pragma unroll
      for (int i = 0; i < S::TILES; ++i) {  // channels 2 NB n + i
        Frag f;
#pragma unroll
        for (int j = 0; j < 4; ++j)
          f.v[j] = perm(t.v[j >> 1][2 * (j & 1) + 1][i >> 1], t.v[j >> 1][2 * (j & 1)][i >> 1], i & 1 ? 0x07060302u : 0x05040100u);
#pragma unroll
        for (int k = 0; k < S::P_TERMS; ++k) acc[i] = mfma16<typename S::P>(f, pf[k], acc[i]);
      }
    }
  };

  // one tile in flight while the one before is computed
  Tile<FMT, NB> ta, tb;
  int s = wave;
  if (s < steps) {
    load_tile(s, ta);
    while (true) {
      if (s + kWaves < steps) load_tile(s + kWaves, tb);
      step(s, ta);
      s += kWaves;
      if (s >= steps) break;
      if (s + kWaves < steps) load_tile(s + kWaves, ta);
      step(s, tb);
      s += kWaves;
      if (s >= steps) break;
    }
  }

  // Join the wavefronts.
  __shared__ float s_m[kWaves][16], s_l[kWaves][16];
  __shared__ floatx4 s_acc[kWaves - 1][S::TILES][64];
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
    for (int t = 0; t < S::TILES; ++t) s_acc[wave - 1][t][lane] = acc[t];
  }
  __syncthreads();
  if (wave != 0) return;
  float sum = 0.0f;
#pragma unroll
  for (int w = 0; w < kWaves; ++w) sum += weight(s_m[w][n]) * s_l[w][n];
#pragma unroll
  for (int w = 0; w < kWaves - 1; ++w)
#pragma unroll
    for (int t = 0; t < S::TILES; ++t) acc[t] += s_acc[w][t][lane];

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
  const int64_t at = ((int64_t)b * a.Hq + kvh * a.G + h0 + n) * (32 * NB);
  if constexpr (S::Q8) {
#pragma unroll
    for (int bl = 0; bl < NB; ++bl) {
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

// Joins the chunks of sequence blockIdx.x / (Hkv HT) in their order: blockIdx.y is one
// 16-channel tile, a wavefront takes every fourth chunk.
template <int FMT, int NB>
__global__ __launch_bounds__(64 * kWaves) void attn_decode_join_kernel(DecodeArgs a) {
  typedef Shape<FMT, NB> S;
  const int lane = (int)(threadIdx.x & 63), n = lane & 15, g = lane >> 4;
  const int wave = __builtin_amdgcn_readfirstlane((int)(threadIdx.x >> 6));
  const int per = a.Hkv * a.HT;
  const int b = (int)blockIdx.x / per, hh = (int)blockIdx.x - b * per, tile = (int)blockIdx.y;
  const Plan plan = make_plan(a, b, true);
  if (plan.count <= 1) return;
  const float* stat = a.stat + ((int64_t)plan.first * per + hh) * 32 + n;
  const int64_t stat_step = (int64_t)per * 32;
  float all = -__builtin_inff();
  for (int c = g; c < plan.count; c += 4) all = fmaxf(all, stat[c * stat_step]);
  all = max_32(max_16(all));
  const floatx4* src = reinterpret_cast<const floatx4*>(a.acc) + ((int64_t)plan.first * per + hh) * (S::TILES * 64) + tile * 64 + lane;
  const int64_t step = (int64_t)per * (S::TILES * 64);
  floatx4 acc = {0.f, 0.f, 0.f, 0.f};
  float sum = 0.0f;
#pragma unroll 8
  for (int c = wave; c < plan.count; c += kWaves) {
    const float m = stat[c * stat_step];
    const float w = m == -__builtin_inff() ? 0.0f : exp2_fast(m - all);
    acc += src[c * step] * w;
    sum += stat[c * stat_step + 16] * w;
  }
  __shared__ floatx4 s_acc[kWaves - 1][64];
  __shared__ float s_sum[kWaves - 1][64];
  if (wave != 0) s_acc[wave - 1][lane] = acc, s_sum[wave - 1][lane] = sum;
  __syncthreads();
  if (wave != 0) return;
#pragma unroll
  for (int w = 0; w < kWaves - 1; ++w) acc += s_acc[w][lane], sum += s_sum[w][lane];
  const int kvh = hh / a.HT, h0 = (hh - kvh * a.HT) * 16;
  if (h0 + n >= a.G) return;
  const float inv = sum == 0.0f ? 0.0f : 1.0f / sum;
  const int64_t at = ((int64_t)b * a.Hq + kvh * a.G + h0 + n) * (32 * NB);
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

template <int FMT, int NB>
hipError_t launch_nb(const DecodeArgs& a, int64_t blocks, bool join, hipStream_t s) {
  hipLaunchKernelGGL((attn_decode_kernel<FMT, NB>), dim3((unsigned)blocks), dim3(64 * kWaves), 0, s, a);
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess || !join) return e;
  hipLaunchKernelGGL((attn_decode_join_kernel<FMT, NB>), dim3((unsigned)(a.B * a.Hkv * a.HT), 2 * NB), dim3(64 * kWaves), 0, s, a);
  return hipGetLastError();
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

int64_t attn_decode_groups(int64_t B, int64_t Hq, int64_t Hkv, int64_t capacity) {
  const int64_t G = Hq / Hkv;
  return chunk_bound(B, Hkv, G, capacity) * Hkv * head_tiles(G);
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
  const int64_t groups = attn_decode_groups(B, Hq, Hkv, capacity);
  a.acc = (float*)workspace;
  a.stat = a.acc + groups * (D / 16) * 64 * 4;
  const bool join = capacity > kMinChunk;
  const int nb = (int)(D / 32);
  if (fmt == NVQ_KV_Q8_0) return launch_fmt<NVQ_KV_Q8_0>(a, nb, groups, join, stream);
  if (fmt == NVQ_KV_F16) return launch_fmt<NVQ_KV_F16>(a, nb, groups, join, stream);
  return launch_fmt<NVQ_KV_BF16>(a, nb, groups, join, stream);
}

}  // namespace nvq
