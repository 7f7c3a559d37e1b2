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
#include "attn_device.h"
#include "nvq_launch.h"

namespace nvq {

namespace {

constexpr int kWaves = 4;
constexpr int kQueries = 32 * kWaves;
constexpr float kSlack = 8.0f;

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
    int lo = 0, hi = 0;
    if (i < a.B) {
      lo = min(max(a.cu_q[i], 0), a.Tq);
      hi = min(max(a.cu_q[i + 1], lo), a.Tq);
    }
    const int tiles = (hi - lo + kQueries - 1) / kQueries;
    int incl = tiles;
#pragma unroll
    for (int o = 1; o < 64; o <<= 1) {
      const int t = __shfl_up(incl, o, 64);
      incl += lane >= o ? t : 0;
    }
    const uint64_t hit = __ballot(base + incl > want);
    if (hit) {
      const int l = __builtin_ctzll(hit);
      s.q0 = __builtin_amdgcn_readlane(lo, l);
      s.m = __builtin_amdgcn_readlane(hi, l) - s.q0;
      s.tile = base + __builtin_amdgcn_readlane(incl, l) - 1 - want;
      s.k0 = min(max(a.cu_k[i0 + l], 0), a.Tk);
      s.n = min(max(a.cu_k[i0 + l + 1], s.k0), a.Tk) - s.k0;
      return true;
    }
    base += __builtin_amdgcn_readlane(incl, 63);
  }
  return false;
}

template <typename T, int NB>
__global__ __launch_bounds__(64 * kWaves) void attn_prompt_kernel(PromptArgs a) {
  constexpr int D = 32 * NB, TK = NB <= 4 ? 64 : 32, KB = TK / 32;
  constexpr int ROW = D + 8;  // halves of a staged row
  __shared__ uint16_t s_k[TK * ROW], s_v[TK * ROW];
  const int tid = (int)threadIdx.x, lane = tid & 63, c = lane & 31, hi = lane >> 5;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int head = (int)blockIdx.x % a.Hq, kvh = head / a.G;
  Span sp;
  if (!find_span(a, (int)blockIdx.x / a.Hq, sp)) return;
  const int i0 = sp.tile * kQueries, iw = i0 + 32 * wave, i = iw + c;  // this lane's query
  const int shift = sp.n - sp.m;
  const int limit = a.causal ? min(i + shift, sp.n - 1) : sp.n - 1;  // the last key it sees, -1 or less: none
  const int end = a.causal ? min(sp.n, min(i0 + kQueries, sp.m) + shift) : sp.n;

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
  float m = -__builtin_inff(), l = 0.0f;
  const uint16_t* kb = a.k + (int64_t)sp.k0 * a.k_t + (int64_t)kvh * a.k_h;
  const uint16_t* vb = a.v + (int64_t)sp.k0 * a.v_t + (int64_t)kvh * a.v_h;

  for (int kt = 0; kt < end; kt += TK) {
    __syncthreads();
#pragma unroll
    for (int u = 0; u < (TK * 4 * NB + 255) / 256; ++u) {
      const int id = u * 256 + tid, r = id / (4 * NB), ch = id % (4 * NB);
      if (TK * 4 * NB % 256 != 0 && id >= TK * 4 * NB) break;
      const int key = min(kt + r, sp.n - 1);
      *reinterpret_cast<u32x4*>(s_k + r * ROW + 8 * ch) = *reinterpret_cast<const u32x4*>(kb + (int64_t)key * a.k_t + 8 * ch);
      *reinterpret_cast<u32x4*>(s_v + r * ROW + 8 * ch) = *reinterpret_cast<const u32x4*>(vb + (int64_t)key * a.v_t + 8 * ch);
    }
    __syncthreads();
    floatx16 s[KB];
#pragma unroll
    for (int b = 0; b < KB; ++b) {
#pragma unroll
      for (int j = 0; j < 16; ++j) s[b][j] = 0.0f;
#pragma unroll
      for (int ks = 0; ks < 2 * NB; ++ks) {
        const u32x4 w = *reinterpret_cast<const u32x4*>(s_k + (32 * b + c) * ROW + 16 * ks + 8 * hi);
        s[b] = mfma32<T>(Frag{w[0], w[1], w[2], w[3]}, qf[ks], s[b]);
      }
    }
    if (kt + TK - 1 > (a.causal ? iw + shift : sp.n - 1) || kt + TK > sp.n) {
#pragma unroll
      for (int b = 0; b < KB; ++b)
#pragma unroll
        for (int j = 0; j < 16; ++j)
          if (kt + 32 * b + 8 * (j >> 2) + 4 * hi + (j & 3) > limit) s[b][j] = -__builtin_inff();
    }
    float top = s[0][0];
#pragma unroll
    for (int b = 0; b < KB; ++b)
#pragma unroll
      for (int j = 0; j < 16; ++j) top = fmaxf(top, s[b][j]);
    top *= a.scale_log2;
    if (__any(top > m + kSlack)) {
      const float m_new = fmaxf(m, max_32(top));
      const float f = m_new == -__builtin_inff() ? 1.0f : exp2_fast(m - m_new);
      l *= f;
#pragma unroll
      for (int t = 0; t < NB; ++t) acc[t] *= f;
      m = m_new;
    }
    const float m_safe = m == -__builtin_inff() ? 0.0f : m;
#pragma unroll
    for (int b = 0; b < KB; ++b) {
#pragma unroll
      for (int j = 0; j < 16; ++j) {
        s[b][j] = exp2_fast(__builtin_fmaf(s[b][j], a.scale_log2, -m_safe));
        l += s[b][j];
      }
#pragma unroll
      for (int t = 0; t < 2; ++t) {
        Frag pf;
#pragma unroll
        for (int j = 0; j < 4; ++j) pf.v[j] = pack_pair<T>(s[b][8 * t + 2 * j], s[b][8 * t + 2 * j + 1]);
#pragma unroll
        for (int dt = 0; dt < NB; ++dt) {
          Frag vf;
#pragma unroll
          for (int r = 0; r < 2; ++r) {
            const int jj = lane & 15, gg = lane >> 4;
            typedef short s4 __attribute__((ext_vector_type(4)));
            const uint16_t* p = s_v + (32 * b + 16 * t + 8 * r + 4 * hi + (jj >> 2)) * ROW + 32 * dt + 16 * (gg & 1) + 4 * (jj & 3);
            const s4 w = __builtin_amdgcn_ds_read_tr16_b64_v4i16((__attribute__((address_space(3))) s4*)p);
            const u32x2 x = __builtin_bit_cast(u32x2, w);
            vf.v[2 * r] = x[0], vf.v[2 * r + 1] = x[1];
          }
          acc[dt] = mfma32<T>(vf, pf, acc[dt]);
        }
      }
    }
  }
  l = sum_32(l);
  if (i >= sp.m) return;
  const float inv = l == 0.0f ? 0.0f : 1.0f / l;  // a query that sees no key gives zeros
  uint16_t* row = a.out + (int64_t)(sp.q0 + i) * a.o_t + (int64_t)head * a.o_h;
#pragma unroll
  for (int t = 0; t < NB; ++t)
#pragma unroll
    for (int j = 0; j < 4; ++j)
      *reinterpret_cast<u32x2*>(row + 32 * t + 8 * j + 4 * hi) =
          u32x2{pack_pair<T>(acc[t][4 * j] * inv, acc[t][4 * j + 1] * inv), pack_pair<T>(acc[t][4 * j + 2] * inv, acc[t][4 * j + 3] * inv)};
}

template <typename T>
hipError_t launch_type(const PromptArgs& a, int nb, int64_t blocks, hipStream_t s) {
  const dim3 grid((unsigned)blocks), block(64 * kWaves);
  switch (nb) {
    case 1: hipLaunchKernelGGL((attn_prompt_kernel<T, 1>), grid, block, 0, s, a); break;
    case 2: hipLaunchKernelGGL((attn_prompt_kernel<T, 2>), grid, block, 0, s, a); break;
    case 3: hipLaunchKernelGGL((attn_prompt_kernel<T, 3>), grid, block, 0, s, a); break;
    case 4: hipLaunchKernelGGL((attn_prompt_kernel<T, 4>), grid, block, 0, s, a); break;
    case 5: hipLaunchKernelGGL((attn_prompt_kernel<T, 5>), grid, block, 0, s, a); break;
    case 6: hipLaunchKernelGGL((attn_prompt_kernel<T, 6>), grid, block, 0, s, a); break;
    case 7: hipLaunchKernelGGL((attn_prompt_kernel<T, 7>), grid, block, 0, s, a); break;
    default: hipLaunchKernelGGL((attn_prompt_kernel<T, 8>), grid, block, 0, s, a); break;
  }
  return hipGetLastError();
}

}  // namespace

int64_t attn_prompt_groups(int64_t B, int64_t Tq, int64_t Hq) { return (Tq / kQueries + B) * Hq; }

hipError_t launch_attn_prompt(int type, const void* q, const void* k, const void* v, void* out, const int64_t strides[8],
                              const int32_t* cu_q, const int32_t* cu_k, int64_t B, int64_t Tq, int64_t Tk, int64_t Hq,
                              int64_t Hkv, int64_t D, float scale, int causal, hipStream_t stream) {
  PromptArgs a;
  a.q = (const uint16_t*)q, a.k = (const uint16_t*)k, a.v = (const uint16_t*)v, a.out = (uint16_t*)out;
  a.q_t = strides[0], a.q_h = strides[1], a.k_t = strides[2], a.k_h = strides[3];
  a.v_t = strides[4], a.v_h = strides[5], a.o_t = strides[6], a.o_h = strides[7];
  a.cu_q = cu_q, a.cu_k = cu_k;
  a.B = (int)B, a.Hq = (int)Hq, a.Hkv = (int)Hkv, a.G = (int)(Hq / Hkv), a.Tq = (int)Tq, a.Tk = (int)Tk;
  // a negative scale turns the queries round, so that the largest score is the largest product
  // (a scale of 0 becomes a number that still makes -infinity of a masked score)
  a.scale_log2 = __builtin_fabsf(scale) * 1.44269504088896340736f;
  if (a.scale_log2 == 0.0f) a.scale_log2 = 1e-37f;
  a.flip = __builtin_signbit(scale) ? 0x80008000u : 0u;
  a.causal = causal;

  const int64_t blocks = attn_prompt_groups(B, Tq, Hq);
  if (type == NVQ_TYPE_F16) return launch_type<_Float16>(a, (int)(D / 32), blocks, stream);
  return launch_type<__bf16>(a, (int)(D / 32), blocks, stream);
}

}  // namespace nvq
