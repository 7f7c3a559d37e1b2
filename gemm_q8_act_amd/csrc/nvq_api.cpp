// nvq_api.cpp -- the C ABI of libnvq (declared in include/nvq.h).
//
// Every entry validates its arguments on the host first (pointers, shapes,
// alignment) and returns a negative status before touching the HIP runtime, so a
// rejected call enqueues nothing and leaves outputs untouched.  Only then is the
// current device's architecture checked (gfx950 only; there is no other code
// path) and the kernel enqueued on the caller's stream.
#include "nvq.h"
#include "nvq_probe.h"

#include <hip/hip_runtime.h>

#include <atomic>
#include <cmath>
#include <cstdarg>
#include <cstdio>
#include <cstring>

#include "nvq_launch.h"

namespace {

thread_local char g_err[512] = "";

nvq_status fail(nvq_status s, const char* fmt, ...) {
  va_list ap;
  va_start(ap, fmt);
  vsnprintf(g_err, sizeof(g_err), fmt, ap);
  va_end(ap);
  return s;
}

bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

// Shapes are bounded so that every byte offset fits comfortably in int64 and every
// grid dimension in 32 bits.
constexpr int64_t kMaxDim = int64_t(1) << 31;
constexpr int64_t kMaxElems = int64_t(1) << 40;
// Largest M of the tiled entries (grid dimension y counts 16-token tiles).
constexpr int64_t kMaxM = int64_t(1) << 20;

nvq_status check_dims(int64_t M, int64_t N, int64_t K, int64_t kmul, int64_t mmin, int64_t mmax) {
  if (K < kmul || K % kmul != 0) return fail(NVQ_ERR_SHAPE, "K=%lld must be a positive multiple of %lld", (long long)K, (long long)kmul);
  if (K >= kMaxDim) return fail(NVQ_ERR_SHAPE, "K=%lld too large", (long long)K);
  if (N < 1 || N >= kMaxDim) return fail(NVQ_ERR_SHAPE, "N=%lld out of range", (long long)N);
  if (M < mmin || M > mmax) return fail(NVQ_ERR_SHAPE, "M=%lld outside [%lld, %lld] for this entry", (long long)M, (long long)mmin, (long long)mmax);
  if (M > kMaxElems / K || N > kMaxElems / K || M > kMaxElems / N)
    return fail(NVQ_ERR_SHAPE, "M*K, N*K or M*N too large");
  return NVQ_OK;
}

// Per-device result of the architecture check: 0 unknown, 1 gfx950, -1 other.
// Written once per device; the only state the library keeps.
std::atomic<int> g_arch_ok[64];

nvq_status check_device() {
  int dev = 0;
  hipError_t e = hipGetDevice(&dev);
  if (e != hipSuccess) return fail(NVQ_ERR_HIP, "hipGetDevice: %s", hipGetErrorString(e));
  if (dev < 0 || dev >= 64) return fail(NVQ_ERR_DEVICE, "device index %d unsupported", dev);
  int st = g_arch_ok[dev].load(std::memory_order_relaxed);
  if (st == 0) {
    hipDeviceProp_t prop;
    e = hipGetDeviceProperties(&prop, dev);
    if (e != hipSuccess) return fail(NVQ_ERR_HIP, "hipGetDeviceProperties: %s", hipGetErrorString(e));
    st = (std::strncmp(prop.gcnArchName, "gfx950", 6) == 0) ? 1 : -1;
    g_arch_ok[dev].store(st, std::memory_order_relaxed);
  }
  if (st != 1) return fail(NVQ_ERR_DEVICE, "device %d is not gfx950", dev);
  return NVQ_OK;
}

nvq_status launched(hipError_t e, const char* what) {
  if (e != hipSuccess) return fail(NVQ_ERR_HIP, "%s launch: %s", what, hipGetErrorString(e));
  g_err[0] = '\0';
  return NVQ_OK;
}

#define NVQ_TRY(x)                  \
  do {                              \
    nvq_status s_ = (x);            \
    if (s_ != NVQ_OK) return s_;    \
  } while (0)

}  // namespace

extern "C" {

const char* nvq_status_str(nvq_status s) {
  switch (s) {
    case NVQ_OK: return "NVQ_OK";
    case NVQ_ERR_NULL: return "NVQ_ERR_NULL";
    case NVQ_ERR_SHAPE: return "NVQ_ERR_SHAPE";
    case NVQ_ERR_RANGE: return "NVQ_ERR_RANGE";
    case NVQ_ERR_ALIGN: return "NVQ_ERR_ALIGN";
    case NVQ_ERR_DEVICE: return "NVQ_ERR_DEVICE";
    case NVQ_ERR_HIP: return "NVQ_ERR_HIP";
    case NVQ_ERR_WORKSPACE: return "NVQ_ERR_WORKSPACE";
    default: return "NVQ_ERR_UNKNOWN";
  }
}

const char* nvq_last_error(void) { return g_err; }

size_t nvq_nvfp4_weight_bytes(int64_t N, int64_t K) {
  if (N < 1 || K < 64 || K % 64 != 0 || N >= kMaxDim || K >= kMaxDim || N > kMaxElems / K) return 0;
  const int64_t np = (N + 15) / 16 * 16, kp = (K + 127) / 128 * 128;
  return (size_t)(np * kp / 2 + np * kp / 16);
}

size_t nvq_q4_1_weight_bytes(int64_t N, int64_t K) {
  if (N < 1 || K < 32 || K % 32 != 0 || N >= kMaxDim || K >= kMaxDim || N > kMaxElems / K) return 0;
  return (size_t)(N * K / 2 + N * K / 8);
}

size_t nvq_q4_k_weight_bytes(int64_t N, int64_t K) {
  if (N < 1 || K < 256 || K % 256 != 0 || N >= kMaxDim || K >= kMaxDim || N > kMaxElems / K) return 0;
  return (size_t)(N * K / 2 + N * (K / 256) * 16);
}

size_t nvq_q5_k_weight_bytes(int64_t N, int64_t K) {
  if (N < 1 || K < 256 || K % 256 != 0 || N >= kMaxDim || K >= kMaxDim || N > kMaxElems / K) return 0;
  return (size_t)(N * (K / 256) * 176);
}

size_t nvq_q6_k_weight_bytes(int64_t N, int64_t K) {
  if (N < 1 || K < 256 || K % 256 != 0 || N >= kMaxDim || K >= kMaxDim || N > kMaxElems / K) return 0;
  return (size_t)(N * (K / 256) * 210);
}

size_t nvq_iq4_xs_weight_bytes(int64_t N, int64_t K) {
  if (N < 1 || K < 256 || K % 256 != 0 || N >= kMaxDim || K >= kMaxDim || N > kMaxElems / K) return 0;
  return (size_t)(N * K / 2 + N * (K / 256) * 8);
}

size_t nvq_gemm_workspace_bytes(int fmt, int64_t M, int64_t N, int64_t K) {
  // fp32 partial tiles of the K-split work items that fill the last round over the
  // compute units (the two-term and integer-MFMA GEMM kernels).
  if (M < 1 || N < 1 || K < 64 || K % 64 != 0) return 0;
  if (fmt == NVQ_FMT_NVFP4) return nvq::gemm_nvfp4_workspace(M, N, K);
  if (fmt == NVQ_FMT_Q4_1) return nvq::gemm_q4_1_workspace(M, N, K);
  if ((fmt == NVQ_FMT_Q4_K || fmt == NVQ_FMT_IQ4_XS || fmt == NVQ_FMT_Q5_K || fmt == NVQ_FMT_Q6_K) && K % 256 == 0)
    return nvq::gemm_q4_k_workspace(M, N, K, fmt == NVQ_FMT_Q6_K);
  return 0;
}

nvq_status nvq_pack_nvfp4(const uint8_t* codes, const uint8_t* ue4m3, int64_t N, int64_t K,
                          void* dst_host) {
  if (!codes || !ue4m3 || !dst_host) return fail(NVQ_ERR_NULL, "nvq_pack_nvfp4: NULL pointer");
  if (nvq_nvfp4_weight_bytes(N, K) == 0) return fail(NVQ_ERR_SHAPE, "nvq_pack_nvfp4: N=%lld K=%lld (K %% 64 == 0 required)", (long long)N, (long long)K);
  for (int64_t i = 0; i < N * K; ++i)
    if (codes[i] > 15) return fail(NVQ_ERR_RANGE, "nvq_pack_nvfp4: code > 15 at weight %lld", (long long)i);
  for (int64_t i = 0; i < N * K / 16; ++i)
    if ((ue4m3[i] & 0x80) || ue4m3[i] == 0x7F) return fail(NVQ_ERR_RANGE, "nvq_pack_nvfp4: invalid UE4M3 byte 0x%02x at scale %lld", ue4m3[i], (long long)i);
  // Tile-interleaved layout: 16-row x 128-k tile-chunks; codes of lane l = 16*g + n
  // (row n, k = 32g .. 32g+31 of the chunk) at 16*l, scales (subblocks 2g, 2g+1)
  // at 2*l of the chunk's 128-byte scale block.  Padding rows / k are zero.
  uint8_t* dst = static_cast<uint8_t*>(dst_host);
  const int64_t ntiles = (N + 15) / 16, nch = (K + 127) / 128, ns = K / 16;
  uint8_t* sc = dst + ntiles * nch * 1024;
  for (int64_t t = 0; t < ntiles; ++t)
    for (int64_t c = 0; c < nch; ++c) {
      uint8_t* blk = dst + (t * nch + c) * 1024;
      uint8_t* sblk = sc + (t * nch + c) * 128;
      for (int l = 0; l < 64; ++l) {
        const int64_t row = t * 16 + (l & 15);
        const int64_t k0 = c * 128 + 32 * (l >> 4);
        const bool live = row < N && k0 < K;
        const uint8_t* cr = codes + row * K + k0;
        for (int b = 0; b < 16; ++b)
          blk[16 * l + b] = live ? (uint8_t)(cr[2 * b] | (cr[2 * b + 1] << 4)) : 0;
        for (int j = 0; j < 2; ++j) {
          const int64_t s = k0 / 16 + j;
          sblk[2 * l + j] = (live && s < ns) ? ue4m3[row * ns + s] : 0;
        }
      }
    }
  g_err[0] = '\0';
  return NVQ_OK;
}

}  // extern "C"

namespace {

// The packers check every input before writing any byte of dst.
nvq_status check_max(const uint8_t* v, int64_t n, unsigned maxv, const char* who, const char* what) {
  for (int64_t i = 0; i < n; ++i)
    if (v[i] > maxv) return fail(NVQ_ERR_RANGE, "%s: %s > %u at index %lld", who, what, maxv, (long long)i);
  return NVQ_OK;
}

// codes (their low four bits) two per byte: code 2i in bits 0..3, 2i+1 in bits 4..7
void pack_nibbles(const uint8_t* q, int64_t n, uint8_t* dst) {
  for (int64_t i = 0; i < n / 2; ++i) dst[i] = (uint8_t)((q[2 * i] & 15) | ((q[2 * i + 1] & 15) << 4));
}

// 16-byte K-quant header per 256 weights: d, dmin, then sc_0..7, mn_0..7 as 6-bit
// fields of a little-endian 96-bit number
void pack_kq_headers(const uint8_t* sc, const uint8_t* mn, const uint16_t* d, const uint16_t* dmin, int64_t nsb,
                     uint8_t* dst) {
  for (int64_t i = 0; i < nsb; ++i) {
    uint8_t h[16] = {};
    std::memcpy(h, &d[i], 2);
    std::memcpy(h + 2, &dmin[i], 2);
    for (int f = 0; f < 16; ++f) {
      const uint8_t v = f < 8 ? sc[8 * i + f] : mn[8 * i + f - 8];
      for (int bit = 0; bit < 6; ++bit)
        if ((v >> bit) & 1) h[4 + (6 * f + bit) / 8] |= (uint8_t)(1u << ((6 * f + bit) % 8));
    }
    std::memcpy(dst + 16 * i, h, 16);
  }
}

// bit `bit` of 32 codes as one word: even codes k = 2e at bit e, odd codes k = 2e + 1 at
// bit 16 + e (the arrangement the kernels' even / odd code planes read)
uint32_t pack_code_bits(const uint8_t* q32, int bit) {
  uint32_t w = 0;
  for (int e = 0; e < 16; ++e) {
    w |= (uint32_t)((q32[2 * e] >> bit) & 1) << e;
    w |= (uint32_t)((q32[2 * e + 1] >> bit) & 1) << (16 + e);
  }
  return w;
}

}  // namespace

extern "C" {

nvq_status nvq_pack_q4_1(const uint8_t* q, const uint16_t* d_f16, const uint16_t* m_f16,
                         int64_t N, int64_t K, void* dst_host) {
  if (!q || !d_f16 || !m_f16 || !dst_host) return fail(NVQ_ERR_NULL, "nvq_pack_q4_1: NULL pointer");
  if (nvq_q4_1_weight_bytes(N, K) == 0) return fail(NVQ_ERR_SHAPE, "nvq_pack_q4_1: N=%lld K=%lld (K %% 32 == 0 required)", (long long)N, (long long)K);
  NVQ_TRY(check_max(q, N * K, 15, "nvq_pack_q4_1", "code"));
  uint8_t* dst = static_cast<uint8_t*>(dst_host);
  const int64_t nc = N * K / 2;
  pack_nibbles(q, N * K, dst);
  const int64_t nb = N * K / 32;
  for (int64_t i = 0; i < nb; ++i) {
    const uint32_t pair = (uint32_t)d_f16[i] | ((uint32_t)m_f16[i] << 16);
    std::memcpy(dst + nc + 4 * i, &pair, 4);
  }
  g_err[0] = '\0';
  return NVQ_OK;
}

nvq_status nvq_pack_q4_k(const uint8_t* q, const uint8_t* sc, const uint8_t* mn, const uint16_t* d_f16,
                         const uint16_t* dmin_f16, int64_t N, int64_t K, void* dst_host) {
  if (!q || !sc || !mn || !d_f16 || !dmin_f16 || !dst_host) return fail(NVQ_ERR_NULL, "nvq_pack_q4_k: NULL pointer");
  if (nvq_q4_k_weight_bytes(N, K) == 0) return fail(NVQ_ERR_SHAPE, "nvq_pack_q4_k: N=%lld K=%lld (K %% 256 == 0 required)", (long long)N, (long long)K);
  NVQ_TRY(check_max(q, N * K, 15, "nvq_pack_q4_k", "code"));
  NVQ_TRY(check_max(sc, N * K / 32, 63, "nvq_pack_q4_k", "scale"));
  NVQ_TRY(check_max(mn, N * K / 32, 63, "nvq_pack_q4_k", "min"));
  uint8_t* dst = static_cast<uint8_t*>(dst_host);
  pack_nibbles(q, N * K, dst);
  pack_kq_headers(sc, mn, d_f16, dmin_f16, N * K / 256, dst + N * K / 2);
  g_err[0] = '\0';
  return NVQ_OK;
}

nvq_status nvq_pack_q5_k(const uint8_t* q, const uint8_t* sc, const uint8_t* mn, const uint16_t* d_f16,
                         const uint16_t* dmin_f16, int64_t N, int64_t K, void* dst_host) {
  if (!q || !sc || !mn || !d_f16 || !dmin_f16 || !dst_host) return fail(NVQ_ERR_NULL, "nvq_pack_q5_k: NULL pointer");
  if (nvq_q5_k_weight_bytes(N, K) == 0) return fail(NVQ_ERR_SHAPE, "nvq_pack_q5_k: N=%lld K=%lld (K %% 256 == 0 required)", (long long)N, (long long)K);
  NVQ_TRY(check_max(q, N * K, 31, "nvq_pack_q5_k", "code"));
  NVQ_TRY(check_max(sc, N * K / 32, 63, "nvq_pack_q5_k", "scale"));
  NVQ_TRY(check_max(mn, N * K / 32, 63, "nvq_pack_q5_k", "min"));
  uint8_t* dst = static_cast<uint8_t*>(dst_host);
  pack_nibbles(q, N * K, dst);
  pack_kq_headers(sc, mn, d_f16, dmin_f16, N * K / 256, dst + N * K / 2);
  uint8_t* hb = dst + N * K / 2 + N * K / 16;
  for (int64_t b = 0; b < N * K / 32; ++b) {
    const uint32_t w4 = pack_code_bits(q + 32 * b, 4);
    std::memcpy(hb + 4 * b, &w4, 4);
  }
  g_err[0] = '\0';
  return NVQ_OK;
}

nvq_status nvq_pack_q6_k(const uint8_t* q, const int8_t* sc, const uint16_t* d_f16, int64_t N, int64_t K,
                         void* dst_host) {
  if (!q || !sc || !d_f16 || !dst_host) return fail(NVQ_ERR_NULL, "nvq_pack_q6_k: NULL pointer");
  if (nvq_q6_k_weight_bytes(N, K) == 0) return fail(NVQ_ERR_SHAPE, "nvq_pack_q6_k: N=%lld K=%lld (K %% 256 == 0 required)", (long long)N, (long long)K);
  NVQ_TRY(check_max(q, N * K, 63, "nvq_pack_q6_k", "code"));
  uint8_t* dst = static_cast<uint8_t*>(dst_host);
  pack_nibbles(q, N * K, dst);
  std::memcpy(dst + N * K / 2, sc, (size_t)(N * K / 16));
  uint8_t* hb = dst + N * K / 2 + N * K / 16;
  for (int64_t b = 0; b < N * K / 32; ++b) {
    const uint32_t w[2] = {pack_code_bits(q + 32 * b, 4), pack_code_bits(q + 32 * b, 5)};
    std::memcpy(hb + 8 * b, w, 8);
  }
  std::memcpy(dst + N * K / 2 + N * K / 16 + N * K / 4, d_f16, (size_t)(N * K / 256) * 2);
  g_err[0] = '\0';
  return NVQ_OK;
}

nvq_status nvq_pack_iq4_xs(const uint8_t* q, const uint8_t* ls, const uint16_t* d_f16, int64_t N, int64_t K,
                           void* dst_host) {
  if (!q || !ls || !d_f16 || !dst_host) return fail(NVQ_ERR_NULL, "nvq_pack_iq4_xs: NULL pointer");
  if (nvq_iq4_xs_weight_bytes(N, K) == 0) return fail(NVQ_ERR_SHAPE, "nvq_pack_iq4_xs: N=%lld K=%lld (K %% 256 == 0 required)", (long long)N, (long long)K);
  NVQ_TRY(check_max(q, N * K, 15, "nvq_pack_iq4_xs", "code"));
  NVQ_TRY(check_max(ls, N * K / 32, 63, "nvq_pack_iq4_xs", "scale"));
  uint8_t* dst = static_cast<uint8_t*>(dst_host);
  const int64_t nc = N * K / 2;
  pack_nibbles(q, N * K, dst);
  // one 8-byte header per (row, 256 weights): d, then ls_0..7 as 6-bit fields of a
  // little-endian 48-bit number
  const int64_t nsb = N * K / 256;
  for (int64_t i = 0; i < nsb; ++i) {
    uint64_t f = 0;
    for (int j = 0; j < 8; ++j) f |= (uint64_t)ls[8 * i + j] << (6 * j);
    uint8_t h[8];
    std::memcpy(h, &d_f16[i], 2);
    for (int b = 0; b < 6; ++b) h[2 + b] = (uint8_t)(f >> (8 * b));
    std::memcpy(dst + nc + 8 * i, h, 8);
  }
  g_err[0] = '\0';
  return NVQ_OK;
}

nvq_status nvq_quantize_act_q8_0(const float* x, int64_t M, int64_t K, int8_t* q,
                                 uint16_t* d_f16, int16_t* bsum16, void* stream) {
  if (!x || !q || !d_f16) return fail(NVQ_ERR_NULL, "nvq_quantize_act_q8_0: NULL pointer");
  if (K < 32 || K % 32 != 0 || K >= kMaxDim) return fail(NVQ_ERR_SHAPE, "nvq_quantize_act_q8_0: K=%lld must be a positive multiple of 32", (long long)K);
  if (M < 1 || M > kMaxElems / K) return fail(NVQ_ERR_SHAPE, "nvq_quantize_act_q8_0: M=%lld out of range", (long long)M);
  if (!aligned(x, 16) || !aligned(q, 16) || !aligned(d_f16, 2) || (bsum16 && !aligned(bsum16, 2)))
    return fail(NVQ_ERR_ALIGN, "nvq_quantize_act_q8_0: x and q must be 16-byte aligned, d_f16/bsum16 2-byte");
  NVQ_TRY(check_device());
  return launched(nvq::launch_act_quant(x, M, K, q, d_f16, bsum16, (hipStream_t)stream), "act_quant");
}

static nvq_status check_common(const void* w, const int8_t* q, const uint16_t* d_f16, const void* y, const char* who) {
  if (!w || !q || !d_f16 || !y) return fail(NVQ_ERR_NULL, "%s: NULL pointer", who);
  if (!aligned(w, 16) || !aligned(q, 16) || !aligned(y, 16) || !aligned(d_f16, 2))
    return fail(NVQ_ERR_ALIGN, "%s: w, q and y must be 16-byte aligned, d_f16 2-byte", who);
  return NVQ_OK;
}

// The decode GEMV kernels keep the whole activation table of a row in LDS.
static bool gemv_fits_lds(int64_t K) { return nvq::gemv_lds_bytes(K) <= 160 * 1024 - 1024; }

nvq_status nvq_gemv_nvfp4(const void* w, float w_scale, const int8_t* q, const uint16_t* d_f16,
                          int64_t M, int64_t N, int64_t K, float* y, void* stream) {
  NVQ_TRY(check_common(w, q, d_f16, y, "nvq_gemv_nvfp4"));
  NVQ_TRY(check_dims(M, N, K, 64, 1, NVQ_GEMV_MAX_M));
  if (M > 1 && M * K >= (int64_t(1) << 32))  // the batched kernel indexes activations in 32 bits
    return fail(NVQ_ERR_SHAPE, "nvq_gemv_nvfp4: M*K=%lld too large for the batched kernel (< 2^32)", (long long)(M * K));
  NVQ_TRY(check_device());
  const uint8_t* wb = static_cast<const uint8_t*>(w);
  if (M == 1 && gemv_fits_lds(K))
    return launched(nvq::launch_gemv_nvfp4_m1(wb, w_scale, q, d_f16, N, K, y, nullptr, 0, (hipStream_t)stream), "gemv_nvfp4");
  if (M > 1)
    return launched(nvq::launch_gemv_nvfp4_batch_f16(wb, w_scale, q, d_f16, M, N, K, y, nullptr, (hipStream_t)stream), "gemv_nvfp4 (batched)");
  return launched(nvq::launch_gemm_nvfp4(wb, w_scale, q, d_f16, M, N, K, y, nullptr, nullptr, (hipStream_t)stream), "gemv_nvfp4 (tiled)");
}

nvq_status nvq_gemv_nvfp4_fused(const void* w, float w_scale, const float* x, int64_t N, int64_t K, float* y,
                                int8_t* q_out, uint16_t* d_out, void* stream) {
  if (!w || !x || !y) return fail(NVQ_ERR_NULL, "nvq_gemv_nvfp4_fused: NULL pointer");
  if ((q_out == nullptr) != (d_out == nullptr))
    return fail(NVQ_ERR_NULL, "nvq_gemv_nvfp4_fused: q_out and d_out are given together or not at all");
  if (!aligned(w, 16) || !aligned(x, 16) || !aligned(y, 16) || (q_out && !aligned(q_out, 16)) ||
      (d_out && !aligned(d_out, 2)))
    return fail(NVQ_ERR_ALIGN, "nvq_gemv_nvfp4_fused: w, x, y and q_out must be 16-byte aligned, d_out 2-byte");
  NVQ_TRY(check_dims(1, N, K, 64, 1, 1));
  if (!gemv_fits_lds(K)) return fail(NVQ_ERR_SHAPE, "nvq_gemv_nvfp4_fused: K=%lld too large for the LDS activation table", (long long)K);
  NVQ_TRY(check_device());
  return launched(nvq::launch_gemv_nvfp4_fused(static_cast<const uint8_t*>(w), w_scale, x, N, K, y, q_out, d_out,
                                               (hipStream_t)stream), "gemv_nvfp4_fused");
}

nvq_status nvq_gemv_nvfp4_routed(const void* w, const float* w_scales, const int32_t* ids, int64_t n_experts,
                                 int64_t n_active, const int8_t* q, const uint16_t* d_f16, int64_t M, int64_t N,
                                 int64_t K, float* y, void* stream) {
  NVQ_TRY(check_common(w, q, d_f16, y, "nvq_gemv_nvfp4_routed"));
  if (!w_scales || !ids) return fail(NVQ_ERR_NULL, "nvq_gemv_nvfp4_routed: NULL pointer");
  if (!aligned(w_scales, 4) || !aligned(ids, 4))
    return fail(NVQ_ERR_ALIGN, "nvq_gemv_nvfp4_routed: w_scales and ids must be 4-byte aligned");
  if (n_experts < 1 || n_experts >= kMaxDim || n_active < 1 || n_active > 65535)
    return fail(NVQ_ERR_SHAPE, "nvq_gemv_nvfp4_routed: n_experts=%lld n_active=%lld out of range", (long long)n_experts,
                (long long)n_active);
  NVQ_TRY(check_dims(M, N, K, 64, 1, 65535 / n_active));
  if (!gemv_fits_lds(K)) return fail(NVQ_ERR_SHAPE, "nvq_gemv_nvfp4_routed: K=%lld too large for the LDS activation table", (long long)K);
  if ((int64_t)nvq_nvfp4_weight_bytes(N, K) > (int64_t)INT64_MAX / n_experts)
    return fail(NVQ_ERR_SHAPE, "nvq_gemv_nvfp4_routed: expert table too large");
  NVQ_TRY(check_device());
  return launched(nvq::launch_gemv_nvfp4_routed(static_cast<const uint8_t*>(w), w_scales, ids, n_experts, n_active, M, q,
                                                d_f16, N, K, y, (hipStream_t)stream),
                  "gemv_nvfp4_routed");
}

nvq_status nvq_gemv_nvfp4_dot4(const void* w, float w_scale, const int8_t* q, const uint16_t* d_f16,
                               int64_t M, int64_t N, int64_t K, float* y, void* stream) {
  NVQ_TRY(check_common(w, q, d_f16, y, "nvq_gemv_nvfp4_dot4"));
  NVQ_TRY(check_dims(M, N, K, 64, 1, NVQ_GEMV_MAX_M));
  if (!gemv_fits_lds(K)) return fail(NVQ_ERR_SHAPE, "nvq_gemv_nvfp4_dot4: K=%lld too large for the LDS activation table", (long long)K);
  NVQ_TRY(check_device());
  const uint8_t* wb = static_cast<const uint8_t*>(w);
  for (int64_t m = 0; m < M; ++m) {
    hipError_t e = nvq::launch_gemv_nvfp4_m1(wb, w_scale, q + m * K, d_f16 + m * (K / 32), N, K, y + m * N,
                                             nullptr, 1, (hipStream_t)stream);
    if (e != hipSuccess) return fail(NVQ_ERR_HIP, "gemv_nvfp4_dot4 launch: %s", hipGetErrorString(e));
  }
  g_err[0] = '\0';
  return NVQ_OK;
}

static nvq_status check_gemm_nvfp4(const void* w, const int8_t* q, const uint16_t* d_f16, const void* y, int64_t M,
                                    int64_t N, int64_t K, const char* who) {
  NVQ_TRY(check_common(w, q, d_f16, y, who));
  NVQ_TRY(check_dims(M, N, K, 64, 16, kMaxM));
  if ((M + 255) / 256 > (int64_t)1 << 31 || (N + 255) / 256 > (((int64_t)1 << 31) - 1) / ((M + 255) / 256))
    return fail(NVQ_ERR_SHAPE, "%s: M=%lld x N=%lld has too many 256 x 256 tiles for one launch", who, (long long)M, (long long)N);
  return NVQ_OK;
}

nvq_status nvq_gemm_nvfp4(const void* w, float w_scale, const int8_t* q, const uint16_t* d_f16,
                          int64_t M, int64_t N, int64_t K, float* y, void* workspace,
                          size_t ws_bytes, void* stream) {
  NVQ_TRY(check_gemm_nvfp4(w, q, d_f16, y, M, N, K, "nvq_gemm_nvfp4"));
  const size_t need = nvq_gemm_workspace_bytes(NVQ_FMT_NVFP4, M, N, K);
  if (ws_bytes < need || (need && !workspace)) return fail(NVQ_ERR_WORKSPACE, "nvq_gemm_nvfp4: workspace of %zu bytes required", need);
  if (need && !aligned(workspace, 16)) return fail(NVQ_ERR_ALIGN, "nvq_gemm_nvfp4: workspace must be 16-byte aligned");
  NVQ_TRY(check_device());
  return launched(nvq::launch_gemm_nvfp4(static_cast<const uint8_t*>(w), w_scale, q, d_f16, M, N, K, y, nullptr,
                                         static_cast<float*>(workspace), (hipStream_t)stream), "gemm_nvfp4");
}

nvq_status nvq_gemm_nvfp4_noalloc(const void* w, float w_scale, const int8_t* q, const uint16_t* d_f16,
                                  int64_t M, int64_t N, int64_t K, float* y, void* stream) {
  NVQ_TRY(check_gemm_nvfp4(w, q, d_f16, y, M, N, K, "nvq_gemm_nvfp4_noalloc"));
  const size_t need = nvq_gemm_workspace_bytes(NVQ_FMT_NVFP4, M, N, K);
  if (need > nvq::gemm_nvfp4_noalloc_scratch_bytes() || need > NVQ_NOALLOC_SCRATCH_BYTES)
    return fail(NVQ_ERR_WORKSPACE, "nvq_gemm_nvfp4_noalloc: shape needs %zu bytes of scratch, more than the static %zu",
                need, (size_t)NVQ_NOALLOC_SCRATCH_BYTES);
  NVQ_TRY(check_device());
  return launched(nvq::launch_gemm_nvfp4_noalloc(static_cast<const uint8_t*>(w), w_scale, q, d_f16, M, N, K, y,
                                                 (hipStream_t)stream), "gemm_nvfp4_noalloc");
}

nvq_status nvq_gemv_q4_1(const void* w, const int8_t* q, const uint16_t* d_f16,
                         const int16_t* bsum16, int64_t M, int64_t N, int64_t K, float* y,
                         void* stream) {
  NVQ_TRY(check_common(w, q, d_f16, y, "nvq_gemv_q4_1"));
  if (!bsum16) return fail(NVQ_ERR_NULL, "nvq_gemv_q4_1: bsum16 is required");
  if (!aligned(bsum16, 2)) return fail(NVQ_ERR_ALIGN, "nvq_gemv_q4_1: bsum16 must be 2-byte aligned");
  NVQ_TRY(check_dims(M, N, K, 32, 1, NVQ_GEMV_MAX_M));
  NVQ_TRY(check_device());
  return launched(nvq::launch_gemv_q4_1(static_cast<const uint8_t*>(w), q, d_f16, bsum16, M, N, K, y, nullptr,
                                        (hipStream_t)stream), "gemv_q4_1");
}

nvq_status nvq_gemm_q4_1(const void* w, const int8_t* q, const uint16_t* d_f16,
                         const int16_t* bsum16, int64_t M, int64_t N, int64_t K, float* y,
                         void* workspace, size_t ws_bytes, void* stream) {
  NVQ_TRY(check_common(w, q, d_f16, y, "nvq_gemm_q4_1"));
  if (!bsum16) return fail(NVQ_ERR_NULL, "nvq_gemm_q4_1: bsum16 is required");
  if (!aligned(bsum16, 2)) return fail(NVQ_ERR_ALIGN, "nvq_gemm_q4_1: bsum16 must be 2-byte aligned");
  NVQ_TRY(check_dims(M, N, K, 32, 16, kMaxM));
  const size_t need = nvq_gemm_workspace_bytes(NVQ_FMT_Q4_1, M, N, K);
  if (ws_bytes < need || (need && !workspace)) return fail(NVQ_ERR_WORKSPACE, "nvq_gemm_q4_1: workspace of %zu bytes required", need);
  if (need && !aligned(workspace, 16)) return fail(NVQ_ERR_ALIGN, "nvq_gemm_q4_1: workspace must be 16-byte aligned");
  NVQ_TRY(check_device());
  return launched(nvq::launch_gemm_q4_1(static_cast<const uint8_t*>(w), q, d_f16, bsum16, M, N, K, y, nullptr,
                                        static_cast<float*>(workspace), (hipStream_t)stream), "gemm_q4_1");
}

nvq_status nvq_gemv_q4_k(const void* w, const int8_t* q, const uint16_t* d_f16,
                         const int16_t* bsum16, int64_t M, int64_t N, int64_t K, float* y,
                         void* stream) {
  NVQ_TRY(check_common(w, q, d_f16, y, "nvq_gemv_q4_k"));
  if (!bsum16) return fail(NVQ_ERR_NULL, "nvq_gemv_q4_k: bsum16 is required");
  if (!aligned(bsum16, 2)) return fail(NVQ_ERR_ALIGN, "nvq_gemv_q4_k: bsum16 must be 2-byte aligned");
  NVQ_TRY(check_dims(M, N, K, 256, 1, NVQ_GEMV_MAX_M));
  NVQ_TRY(check_device());
  return launched(nvq::launch_gemv_q4_k(static_cast<const uint8_t*>(w), q, d_f16, bsum16, M, N, K, y, nullptr,
                                        (hipStream_t)stream), "gemv_q4_k");
}

nvq_status nvq_gemm_q4_k(const void* w, const int8_t* q, const uint16_t* d_f16,
                         const int16_t* bsum16, int64_t M, int64_t N, int64_t K, float* y,
                         void* workspace, size_t ws_bytes, void* stream) {
  NVQ_TRY(check_common(w, q, d_f16, y, "nvq_gemm_q4_k"));
  if (!bsum16) return fail(NVQ_ERR_NULL, "nvq_gemm_q4_k: bsum16 is required");
  if (!aligned(bsum16, 2)) return fail(NVQ_ERR_ALIGN, "nvq_gemm_q4_k: bsum16 must be 2-byte aligned");
  NVQ_TRY(check_dims(M, N, K, 256, 16, kMaxM));
  const size_t need = nvq_gemm_workspace_bytes(NVQ_FMT_Q4_K, M, N, K);
  if (ws_bytes < need || (need && !workspace)) return fail(NVQ_ERR_WORKSPACE, "nvq_gemm_q4_k: workspace of %zu bytes required", need);
  if (need && !aligned(workspace, 16)) return fail(NVQ_ERR_ALIGN, "nvq_gemm_q4_k: workspace must be 16-byte aligned");
  NVQ_TRY(check_device());
  return launched(nvq::launch_gemm_q4_k(static_cast<const uint8_t*>(w), q, d_f16, bsum16, M, N, K, y, nullptr,
                                        static_cast<float*>(workspace), (hipStream_t)stream), "gemm_q4_k");
}

nvq_status nvq_gemv_q5_k(const void* w, const int8_t* q, const uint16_t* d_f16,
                         const int16_t* bsum16, int64_t M, int64_t N, int64_t K, float* y,
                         void* stream) {
  NVQ_TRY(check_common(w, q, d_f16, y, "nvq_gemv_q5_k"));
  if (!bsum16) return fail(NVQ_ERR_NULL, "nvq_gemv_q5_k: bsum16 is required");
  if (!aligned(bsum16, 2)) return fail(NVQ_ERR_ALIGN, "nvq_gemv_q5_k: bsum16 must be 2-byte aligned");
  NVQ_TRY(check_dims(M, N, K, 256, 1, NVQ_GEMV_MAX_M));
  NVQ_TRY(check_device());
  return launched(nvq::launch_gemv_q5_k(static_cast<const uint8_t*>(w), q, d_f16, bsum16, M, N, K, y, nullptr,
                                        (hipStream_t)stream), "gemv_q5_k");
}

nvq_status nvq_gemm_q5_k(const void* w, const int8_t* q, const uint16_t* d_f16,
                         const int16_t* bsum16, int64_t M, int64_t N, int64_t K, float* y,
                         void* workspace, size_t ws_bytes, void* stream) {
  NVQ_TRY(check_common(w, q, d_f16, y, "nvq_gemm_q5_k"));
  if (!bsum16) return fail(NVQ_ERR_NULL, "nvq_gemm_q5_k: bsum16 is required");
  if (!aligned(bsum16, 2)) return fail(NVQ_ERR_ALIGN, "nvq_gemm_q5_k: bsum16 must be 2-byte aligned");
  NVQ_TRY(check_dims(M, N, K, 256, 16, kMaxM));
  const size_t need = nvq_gemm_workspace_bytes(NVQ_FMT_Q5_K, M, N, K);
  if (ws_bytes < need || (need && !workspace)) return fail(NVQ_ERR_WORKSPACE, "nvq_gemm_q5_k: workspace of %zu bytes required", need);
  if (need && !aligned(workspace, 16)) return fail(NVQ_ERR_ALIGN, "nvq_gemm_q5_k: workspace must be 16-byte aligned");
  NVQ_TRY(check_device());
  return launched(nvq::launch_gemm_q5_k(static_cast<const uint8_t*>(w), q, d_f16, bsum16, M, N, K, y, nullptr,
                                        static_cast<float*>(workspace), (hipStream_t)stream), "gemm_q5_k");
}

nvq_status nvq_gemv_q6_k(const void* w, const int8_t* q, const uint16_t* d_f16, int64_t M, int64_t N, int64_t K,
                         float* y, void* stream) {
  NVQ_TRY(check_common(w, q, d_f16, y, "nvq_gemv_q6_k"));
  NVQ_TRY(check_dims(M, N, K, 256, 1, NVQ_GEMV_MAX_M));
  NVQ_TRY(check_device());
  return launched(nvq::launch_gemv_q6_k(static_cast<const uint8_t*>(w), q, d_f16, M, N, K, y, nullptr,
                                        (hipStream_t)stream), "gemv_q6_k");
}

nvq_status nvq_gemm_q6_k(const void* w, const int8_t* q, const uint16_t* d_f16, int64_t M, int64_t N, int64_t K,
                         float* y, void* workspace, size_t ws_bytes, void* stream) {
  NVQ_TRY(check_common(w, q, d_f16, y, "nvq_gemm_q6_k"));
  NVQ_TRY(check_dims(M, N, K, 256, 16, kMaxM));
  const size_t need = nvq_gemm_workspace_bytes(NVQ_FMT_Q6_K, M, N, K);
  if (ws_bytes < need || (need && !workspace)) return fail(NVQ_ERR_WORKSPACE, "nvq_gemm_q6_k: workspace of %zu bytes required", need);
  if (need && !aligned(workspace, 16)) return fail(NVQ_ERR_ALIGN, "nvq_gemm_q6_k: workspace must be 16-byte aligned");
  NVQ_TRY(check_device());
  return launched(nvq::launch_gemm_q6_k(static_cast<const uint8_t*>(w), q, d_f16, M, N, K, y, nullptr,
                                        static_cast<float*>(workspace), (hipStream_t)stream), "gemm_q6_k");
}

nvq_status nvq_gemv_iq4_xs(const void* w, const int8_t* table, const int8_t* q, const uint16_t* d_f16, int64_t M,
                           int64_t N, int64_t K, float* y, void* stream) {
  NVQ_TRY(check_common(w, q, d_f16, y, "nvq_gemv_iq4_xs"));
  if (!table) return fail(NVQ_ERR_NULL, "nvq_gemv_iq4_xs: table is required");
  NVQ_TRY(check_dims(M, N, K, 256, 1, NVQ_GEMV_MAX_M));
  NVQ_TRY(check_device());
  return launched(nvq::launch_gemv_iq4_xs(static_cast<const uint8_t*>(w), table, q, d_f16, M, N, K, y, nullptr,
                                          (hipStream_t)stream), "gemv_iq4_xs");
}

nvq_status nvq_gemm_iq4_xs(const void* w, const int8_t* table, const int8_t* q, const uint16_t* d_f16, int64_t M,
                           int64_t N, int64_t K, float* y, void* workspace, size_t ws_bytes, void* stream) {
  NVQ_TRY(check_common(w, q, d_f16, y, "nvq_gemm_iq4_xs"));
  if (!table) return fail(NVQ_ERR_NULL, "nvq_gemm_iq4_xs: table is required");
  NVQ_TRY(check_dims(M, N, K, 256, 16, kMaxM));
  const size_t need = nvq_gemm_workspace_bytes(NVQ_FMT_IQ4_XS, M, N, K);
  if (ws_bytes < need || (need && !workspace)) return fail(NVQ_ERR_WORKSPACE, "nvq_gemm_iq4_xs: workspace of %zu bytes required", need);
  if (need && !aligned(workspace, 16)) return fail(NVQ_ERR_ALIGN, "nvq_gemm_iq4_xs: workspace must be 16-byte aligned");
  NVQ_TRY(check_device());
  return launched(nvq::launch_gemm_iq4_xs(static_cast<const uint8_t*>(w), table, q, d_f16, M, N, K, y, nullptr,
                                          static_cast<float*>(workspace), (hipStream_t)stream), "gemm_iq4_xs");
}

nvq_status nvq_debug_isums_iq4_xs(const int8_t* table, int path, const void* w, const int8_t* q, int64_t M,
                                  int64_t N, int64_t K, int32_t* isums, void* stream) {
  if (path != NVQ_PATH_GEMV && path != NVQ_PATH_GEMM) return fail(NVQ_ERR_RANGE, "nvq_debug_isums_iq4_xs: path=%d", path);
  if (!table || !w || !q || !isums) return fail(NVQ_ERR_NULL, "nvq_debug_isums_iq4_xs: NULL pointer");
  if (!aligned(w, 16) || !aligned(q, 16) || !aligned(isums, 4)) return fail(NVQ_ERR_ALIGN, "nvq_debug_isums_iq4_xs: w and q must be 16-byte aligned, isums 4-byte");
  NVQ_TRY(check_dims(M, N, K, 256, 1, kMaxM));
  if (M > kMaxElems / (N * (K / 16))) return fail(NVQ_ERR_SHAPE, "nvq_debug_isums_iq4_xs: output too large");
  NVQ_TRY(check_device());
  const uint8_t* wb = static_cast<const uint8_t*>(w);
  hipStream_t st = (hipStream_t)stream;
  if (path == NVQ_PATH_GEMM)
    return launched(nvq::launch_gemm_iq4_xs(wb, table, q, nullptr, M, N, K, nullptr, isums, nullptr, st), "debug gemm_iq4_xs");
  return launched(nvq::launch_gemv_iq4_xs(wb, table, q, nullptr, M, N, K, nullptr, isums, st), "debug gemv_iq4_xs");
}

nvq_status nvq_debug_isums(int fmt, int path, const void* w, const int8_t* q, int64_t M,
                           int64_t N, int64_t K, int32_t* isums, void* stream) {
  if (fmt != NVQ_FMT_NVFP4 && fmt != NVQ_FMT_Q4_1 && fmt != NVQ_FMT_Q4_K && fmt != NVQ_FMT_Q5_K && fmt != NVQ_FMT_Q6_K)
    return fail(NVQ_ERR_RANGE, "nvq_debug_isums: fmt=%d (IQ4_XS sums need its value table: nvq_debug_isums_iq4_xs)", fmt);
  const bool kq = fmt == NVQ_FMT_Q4_K || fmt == NVQ_FMT_Q5_K || fmt == NVQ_FMT_Q6_K;
  if (path != NVQ_PATH_GEMV && path != NVQ_PATH_GEMM && !(path == NVQ_PATH_GEMV_DOT4 && fmt == NVQ_FMT_NVFP4))
    return fail(NVQ_ERR_RANGE, "nvq_debug_isums: path=%d", path);
  if (!w || !q || !isums) return fail(NVQ_ERR_NULL, "nvq_debug_isums: NULL pointer");
  if (!aligned(w, 16) || !aligned(q, 16) || !aligned(isums, 4)) return fail(NVQ_ERR_ALIGN, "nvq_debug_isums: w and q must be 16-byte aligned, isums 4-byte");
  NVQ_TRY(check_dims(M, N, K, fmt == NVQ_FMT_NVFP4 ? 64 : (kq ? 256 : 32), 1, kMaxM));
  if (M > kMaxElems / (N * (K / 16))) return fail(NVQ_ERR_SHAPE, "nvq_debug_isums: output too large");
  if (fmt == NVQ_FMT_NVFP4 && path == NVQ_PATH_GEMV && M > 1 && (M < 16 ? M : 16) * K >= (int64_t(1) << 32))
    return fail(NVQ_ERR_SHAPE, "nvq_debug_isums: K=%lld too large for the batched kernel (16 * K < 2^32)", (long long)K);
  if (path == NVQ_PATH_GEMV_DOT4 && !gemv_fits_lds(K))
    return fail(NVQ_ERR_SHAPE, "nvq_debug_isums: K=%lld too large for the v_dot4 decode kernel", (long long)K);
  NVQ_TRY(check_device());
  const uint8_t* wb = static_cast<const uint8_t*>(w);
  hipStream_t st = (hipStream_t)stream;
  // The sums come from the kernel the product entry would run for this shape: the GEMM
  // dispatch (tiled at M = 1, batched up to 16, two-term above) or the GEMV dispatch
  // (the M = 1 decode kernel, or the tiled one for rows past its LDS table; the
  // batched kernel for M >= 2, 16 tokens per launch).
  if (path == NVQ_PATH_GEMM) {
    if (fmt == NVQ_FMT_NVFP4) return launched(nvq::launch_gemm_nvfp4(wb, 1.0f, q, nullptr, M, N, K, nullptr, isums, nullptr, st), "debug gemm_nvfp4");
    if (fmt == NVQ_FMT_Q4_K) return launched(nvq::launch_gemm_q4_k(wb, q, nullptr, nullptr, M, N, K, nullptr, isums, nullptr, st), "debug gemm_q4_k");
    if (fmt == NVQ_FMT_Q5_K) return launched(nvq::launch_gemm_q5_k(wb, q, nullptr, nullptr, M, N, K, nullptr, isums, nullptr, st), "debug gemm_q5_k");
    if (fmt == NVQ_FMT_Q6_K) return launched(nvq::launch_gemm_q6_k(wb, q, nullptr, M, N, K, nullptr, isums, nullptr, st), "debug gemm_q6_k");
    return launched(nvq::launch_gemm_q4_1(wb, q, nullptr, nullptr, M, N, K, nullptr, isums, nullptr, st), "debug gemm_q4_1");
  }
  if (fmt == NVQ_FMT_Q4_1) return launched(nvq::launch_gemv_q4_1(wb, q, nullptr, nullptr, M, N, K, nullptr, isums, st), "debug gemv_q4_1");
  if (fmt == NVQ_FMT_Q4_K) return launched(nvq::launch_gemv_q4_k(wb, q, nullptr, nullptr, M, N, K, nullptr, isums, st), "debug gemv_q4_k");
  if (fmt == NVQ_FMT_Q5_K) return launched(nvq::launch_gemv_q5_k(wb, q, nullptr, nullptr, M, N, K, nullptr, isums, st), "debug gemv_q5_k");
  if (fmt == NVQ_FMT_Q6_K) return launched(nvq::launch_gemv_q6_k(wb, q, nullptr, M, N, K, nullptr, isums, st), "debug gemv_q6_k");
  if (path == NVQ_PATH_GEMV) {
    if (M > 1) return launched(nvq::launch_gemv_nvfp4_batch_f16(wb, 1.0f, q, nullptr, M, N, K, nullptr, isums, st), "debug gemv_nvfp4 (batched)");
    if (!gemv_fits_lds(K)) return launched(nvq::launch_gemm_nvfp4(wb, 1.0f, q, nullptr, M, N, K, nullptr, isums, nullptr, st), "debug gemv_nvfp4 (tiled)");
  }
  const int64_t per_m = N * (K / 16);
  for (int64_t m = 0; m < M; ++m) {
    hipError_t e = nvq::launch_gemv_nvfp4_m1(wb, 1.0f, q + m * K, nullptr, N, K, nullptr, isums + m * per_m,
                                             path == NVQ_PATH_GEMV_DOT4 ? 1 : 0, st);
    if (e != hipSuccess) return fail(NVQ_ERR_HIP, "debug gemv launch: %s", hipGetErrorString(e));
  }
  g_err[0] = '\0';
  return NVQ_OK;
}

// ---- paged key-value cache and attention ----

namespace {

size_t type_bytes(int type) { return type == NVQ_TYPE_F32 ? 4 : 2; }

// A row argument [T][H][D]: every row starts at a multiple of 16 bytes.  The stride of a
// dimension of one has no meaning.
nvq_status check_rows(const char* who, const char* name, const void* p, int type, int64_t T, int64_t H, int64_t stride_t,
                      int64_t stride_h) {
  if (T <= 1) stride_t = 0;
  if (H <= 1) stride_h = 0;
  if (stride_t < 0 || stride_h < 0 || stride_t >= kMaxElems || stride_h >= kMaxElems)
    return fail(NVQ_ERR_SHAPE, "%s: strides of %s out of range", who, name);
  if (!aligned(p, 16) || stride_t * (int64_t)type_bytes(type) % 16 != 0 || stride_h * (int64_t)type_bytes(type) % 16 != 0)
    return fail(NVQ_ERR_ALIGN, "%s: every row of %s must start at a multiple of 16 bytes", who, name);
  return NVQ_OK;
}

// Rows that are written must not lie on one another.
nvq_status check_apart(const char* who, const char* name, int64_t T, int64_t H, int64_t D, int64_t stride_t, int64_t stride_h) {
  const bool heads_inside = H == 1 || (stride_h >= D && (T == 1 || stride_t >= (H - 1) * stride_h + D));
  const bool tokens_inside = T == 1 || (stride_t >= D && (H == 1 || stride_h >= (T - 1) * stride_t + D));
  if (!heads_inside && !tokens_inside) return fail(NVQ_ERR_SHAPE, "%s: rows of %s overlap", who, name);
  return NVQ_OK;
}

nvq_status check_head(const char* who, int64_t Hkv, int64_t D) {
  if (D < 32 || D > 256 || D % 32 != 0) return fail(NVQ_ERR_SHAPE, "%s: D=%lld must be a multiple of 32 in 32 .. 256", who, (long long)D);
  if (Hkv < 1 || Hkv > 65536) return fail(NVQ_ERR_SHAPE, "%s: Hkv=%lld outside [1, 65536]", who, (long long)Hkv);
  return NVQ_OK;
}

bool page_ok(int64_t page) { return page >= 16 && page <= 65536 && (page & (page - 1)) == 0; }

nvq_status check_cache(const char* who, int fmt, const void* k, const void* v, const void* k_d, const void* v_d, int64_t Hkv,
                       int64_t D, int64_t n_pages, int64_t page, nvq::KvCache& c) {
  if (fmt != NVQ_KV_Q8_0 && fmt != NVQ_KV_F16 && fmt != NVQ_KV_BF16) return fail(NVQ_ERR_RANGE, "%s: fmt=%d is not NVQ_KV_*", who, fmt);
  NVQ_TRY(check_head(who, Hkv, D));
  if (!k || !v || (fmt == NVQ_KV_Q8_0 && (!k_d || !v_d))) return fail(NVQ_ERR_NULL, "%s: NULL cache pointer", who);
  if (fmt != NVQ_KV_Q8_0 && (k_d || v_d)) return fail(NVQ_ERR_RANGE, "%s: a 16-bit cache has no scales", who);
  if (!page_ok(page)) return fail(NVQ_ERR_SHAPE, "%s: page=%lld must be a power of two in 16 .. 65536", who, (long long)page);
  if (n_pages < 1 || n_pages >= kMaxDim || n_pages * page > kMaxElems / Hkv)
    return fail(NVQ_ERR_SHAPE, "%s: n_pages=%lld out of range", who, (long long)n_pages);
  if (!aligned(k, 16) || !aligned(v, 16) || !aligned(k_d, 16) || !aligned(v_d, 16))
    return fail(NVQ_ERR_ALIGN, "%s: cache pointers must be 16-byte aligned", who);
  c = {k, v, k_d, v_d, n_pages, __builtin_ctzll((unsigned long long)page)};
  return NVQ_OK;
}

nvq_status kv_copy(bool write, const char* who, int fmt, int type, const void* k, int64_t k_st, int64_t k_sh, const void* v,
                   int64_t v_st, int64_t v_sh, const int64_t* slots, int64_t T, int64_t Hkv, int64_t D, const void* k_cache,
                   const void* v_cache, const void* k_d, const void* v_d, int64_t n_pages, int64_t page, void* stream) {
  if (type < NVQ_TYPE_F32 || type > NVQ_TYPE_BF16) return fail(NVQ_ERR_RANGE, "%s: type=%d is not NVQ_TYPE_*", who, type);
  nvq::KvCache c;
  NVQ_TRY(check_cache(who, fmt, k_cache, v_cache, k_d, v_d, Hkv, D, n_pages, page, c));
  if (T < 0 || T > ((int64_t(1) << 31) - 16) / Hkv) return fail(NVQ_ERR_SHAPE, "%s: T=%lld out of range", who, (long long)T);
  if (T == 0) return NVQ_OK;
  if (!k || !v || !slots) return fail(NVQ_ERR_NULL, "%s: NULL pointer", who);
  NVQ_TRY(check_rows(who, "k", k, type, T, Hkv, k_st, k_sh));
  NVQ_TRY(check_rows(who, "v", v, type, T, Hkv, v_st, v_sh));
  if (!write) {
    NVQ_TRY(check_apart(who, "k", T, Hkv, D, k_st, k_sh));
    NVQ_TRY(check_apart(who, "v", T, Hkv, D, v_st, v_sh));
  }
  if (!aligned(slots, 8)) return fail(NVQ_ERR_ALIGN, "%s: slots must be 8-byte aligned", who);
  NVQ_TRY(check_device());
  const int64_t strides[4] = {k_st, k_sh, v_st, v_sh};
  return launched(nvq::launch_kv_copy(write, fmt, type, k, v, strides, slots, T, Hkv, D, c, (hipStream_t)stream), who);
}

}  // namespace

nvq_status nvq_kv_write(int fmt, int type, const void* k, int64_t k_stride_t, int64_t k_stride_h, const void* v,
                        int64_t v_stride_t, int64_t v_stride_h, const int64_t* slots, int64_t T, int64_t Hkv, int64_t D,
                        void* k_cache, void* v_cache, uint16_t* k_d, uint16_t* v_d, int64_t n_pages, int64_t page,
                        void* stream) {
  return kv_copy(true, "nvq_kv_write", fmt, type, k, k_stride_t, k_stride_h, v, v_stride_t, v_stride_h, slots, T, Hkv, D,
                 k_cache, v_cache, k_d, v_d, n_pages, page, stream);
}

nvq_status nvq_kv_read(int fmt, int type, void* k, int64_t k_stride_t, int64_t k_stride_h, void* v, int64_t v_stride_t,
                       int64_t v_stride_h, const int64_t* slots, int64_t T, int64_t Hkv, int64_t D, const void* k_cache,
                       const void* v_cache, const uint16_t* k_d, const uint16_t* v_d, int64_t n_pages, int64_t page,
                       void* stream) {
  return kv_copy(false, "nvq_kv_read", fmt, type, k, k_stride_t, k_stride_h, v, v_stride_t, v_stride_h, slots, T, Hkv, D,
                 k_cache, v_cache, k_d, v_d, n_pages, page, stream);
}

nvq_status nvq_rope_table(const double* inv_freq, int64_t P, int64_t R, float* table) {
  const char* who = "nvq_rope_table";
  if (!inv_freq || !table) return fail(NVQ_ERR_NULL, "%s: NULL pointer", who);
  if (R < 4 || R > 256 || R % 4 != 0) return fail(NVQ_ERR_SHAPE, "%s: R=%lld must be a multiple of 4 in 4 .. 256", who, (long long)R);
  if (P < 1 || P >= kMaxDim) return fail(NVQ_ERR_SHAPE, "%s: P=%lld out of range", who, (long long)P);
  for (int64_t p = 0; p < P; ++p)
    for (int64_t c = 0; c < R / 2; ++c) {
      const double angle = (double)p * inv_freq[c];
      table[p * R + c] = (float)std::cos(angle), table[p * R + R / 2 + c] = (float)std::sin(angle);
    }
  g_err[0] = '\0';
  return NVQ_OK;
}

namespace {

// What the two rotating entries have in common.  Rows are left out by having no heads.
nvq_status check_rope(const char* who, nvq::RopeRows& r, int64_t T, int64_t Hq, int64_t Hkv, int64_t D, const int64_t in_st[3][2],
                      const int64_t out_st[2][2], const float* q_weight, const float* k_weight, float eps, const float* table, int64_t P,
                      int64_t R, int pairs, const int32_t* positions, int axes, const int32_t* sections) {
  if (r.type < NVQ_TYPE_F32 || r.type > NVQ_TYPE_BF16) return fail(NVQ_ERR_RANGE, "%s: type=%d is not NVQ_TYPE_*", who, r.type);
  if (r.out_type < NVQ_TYPE_F32 || r.out_type > NVQ_TYPE_BF16) return fail(NVQ_ERR_RANGE, "%s: out_type=%d is not NVQ_TYPE_*", who, r.out_type);
  if (pairs != NVQ_ROPE_HALVES && pairs != NVQ_ROPE_NEIGHBOURS) return fail(NVQ_ERR_RANGE, "%s: pairs=%d is not NVQ_ROPE_*", who, pairs);
  if (!(eps >= 0.0f) || eps > 3e38f) return fail(NVQ_ERR_RANGE, "%s: eps must be a number and not negative", who);
  if (R < 4 || R > D || R % 4 != 0) return fail(NVQ_ERR_SHAPE, "%s: R=%lld must be a multiple of 4 in 4 .. D", who, (long long)R);
  if (P < 1 || P >= kMaxDim) return fail(NVQ_ERR_SHAPE, "%s: P=%lld out of range", who, (long long)P);
  if (axes < 1 || axes > 4) return fail(NVQ_ERR_RANGE, "%s: axes=%d outside 1 .. 4", who, axes);
  if (axes == 1 && sections) return fail(NVQ_ERR_RANGE, "%s: one axis has no sections", who);
  if (axes > 1 && !sections) return fail(NVQ_ERR_NULL, "%s: several axes need sections", who);
  int64_t end = 0;
  for (int i = 0; i < 3; ++i) r.ends[i] = (int)(R / 2);
  for (int i = 0; axes > 1 && i < axes; ++i) {
    if (sections[i] < 0 || sections[i] > R / 2) return fail(NVQ_ERR_RANGE, "%s: sections[%d]=%d out of range", who, i, (int)sections[i]);
    end += sections[i];
    if (i < 3) r.ends[i] = (int)end;
  }
  if (axes > 1 && end != R / 2) return fail(NVQ_ERR_RANGE, "%s: the sections must have R/2=%lld pairs in all", who, (long long)(R / 2));
  if (T > 0) {
    if (!table || !positions) return fail(NVQ_ERR_NULL, "%s: NULL pointer", who);
    if (!aligned(table, 16) || !aligned(positions, 4) || !aligned(q_weight, 16) || !aligned(k_weight, 16))
      return fail(NVQ_ERR_ALIGN, "%s: table and weights must be 16-byte aligned, positions 4-byte", who);
    static const char* const names[] = {"q", "k", "v"};
    const int64_t H[3] = {Hq, Hkv, Hkv};
    for (int i = 0; i < 3; ++i)
      if (r.heads[i]) NVQ_TRY(check_rows(who, names[i], r.in[i], r.type, T, H[i], in_st[i][0], in_st[i][1]));
    for (int i = 0; i < 2; ++i)
      if (r.out[i]) {
        NVQ_TRY(check_rows(who, i ? "k_out" : "q_out", r.out[i], r.out_type, T, H[i], out_st[i][0], out_st[i][1]));
        NVQ_TRY(check_apart(who, i ? "k_out" : "q_out", T, H[i], D, out_st[i][0], out_st[i][1]));
      }
  }
  for (int i = 0; i < 3; ++i) r.in_t[i] = in_st[i][0], r.in_h[i] = in_st[i][1];
  for (int i = 0; i < 2; ++i) r.out_t[i] = out_st[i][0], r.out_h[i] = out_st[i][1];
  r.weight[0] = q_weight, r.weight[1] = k_weight;
  r.eps = eps, r.table = table, r.n_pos = (int)P, r.rot = (int)R, r.neighbours = pairs == NVQ_ROPE_NEIGHBOURS;
  r.positions = positions, r.axes = axes, r.axis_stride = T;
  return NVQ_OK;
}

}  // namespace

nvq_status nvq_qk_norm_rope(int type, int out_type, const void* q, int64_t q_stride_t, int64_t q_stride_h, const void* k,
                            int64_t k_stride_t, int64_t k_stride_h, int64_t T, int64_t Hq, int64_t Hkv, int64_t D,
                            const float* q_weight, const float* k_weight, float eps, const float* table, int64_t P, int64_t R,
                            int pairs, const int32_t* positions, int axes, const int32_t* sections, void* q_out,
                            int64_t qo_stride_t, int64_t qo_stride_h, void* k_out, int64_t ko_stride_t, int64_t ko_stride_h,
                            void* stream) {
  const char* who = "nvq_qk_norm_rope";
  NVQ_TRY(check_head(who, Hkv, D));
  if (Hq < 1 || Hq > 65536) return fail(NVQ_ERR_SHAPE, "%s: Hq=%lld outside [1, 65536]", who, (long long)Hq);
  if (T < 0 || T >= kMaxDim / (Hq + Hkv)) return fail(NVQ_ERR_SHAPE, "%s: T=%lld out of range", who, (long long)T);
  if (T > 0 && (!q != !q_out || !k != !k_out || (!q && !k)))
    return fail(NVQ_ERR_NULL, "%s: q with q_out, k with k_out, or both", who);
  nvq::RopeRows r = {};
  r.type = type, r.out_type = out_type;
  r.in[0] = q, r.in[1] = k, r.out[0] = q_out, r.out[1] = k_out;
  r.heads[0] = q ? (uint32_t)Hq : 0, r.heads[1] = k ? (uint32_t)Hkv : 0;
  const int64_t in_st[3][2] = {{q_stride_t, q_stride_h}, {k_stride_t, k_stride_h}, {0, 0}};
  const int64_t out_st[2][2] = {{qo_stride_t, qo_stride_h}, {ko_stride_t, ko_stride_h}};
  NVQ_TRY(check_rope(who, r, T, Hq, Hkv, D, in_st, out_st, q_weight, k_weight, eps, table, P, R, pairs, positions, axes, sections));
  if (T == 0) return NVQ_OK;
  NVQ_TRY(check_device());
  return launched(nvq::launch_rope(r, T, D, -1, nullptr, nullptr, (hipStream_t)stream), who);
}

nvq_status nvq_rope_kv_write(int fmt, int type, int out_type, const void* q, int64_t q_stride_t, int64_t q_stride_h,
                             const void* k, int64_t k_stride_t, int64_t k_stride_h, const void* v, int64_t v_stride_t,
                             int64_t v_stride_h, int64_t T, int64_t Hq, int64_t Hkv, int64_t D, const float* q_weight,
                             const float* k_weight, float eps, const float* table, int64_t P, int64_t R, int pairs,
                             const int32_t* positions, int axes, const int32_t* sections, const int64_t* slots, void* q_out,
                             int64_t qo_stride_t, int64_t qo_stride_h, void* k_cache, void* v_cache, uint16_t* k_d,
                             uint16_t* v_d, int64_t n_pages, int64_t page, void* stream) {
  const char* who = "nvq_rope_kv_write";
  nvq::KvCache c;
  NVQ_TRY(check_cache(who, fmt, k_cache, v_cache, k_d, v_d, Hkv, D, n_pages, page, c));
  if (Hq < 1 || Hq > 65536) return fail(NVQ_ERR_SHAPE, "%s: Hq=%lld outside [1, 65536]", who, (long long)Hq);
  if (T < 0 || T >= kMaxDim / (Hq + 2 * Hkv)) return fail(NVQ_ERR_SHAPE, "%s: T=%lld out of range", who, (long long)T);
  if (T > 0 && (!k || !v || !slots || !q != !q_out)) return fail(NVQ_ERR_NULL, "%s: NULL pointer (k, v and slots; q with q_out)", who);
  nvq::RopeRows r = {};
  r.type = type, r.out_type = out_type;
  r.in[0] = q, r.in[1] = k, r.in[2] = v, r.out[0] = q_out;
  r.heads[0] = q ? (uint32_t)Hq : 0, r.heads[1] = r.heads[2] = (uint32_t)Hkv;
  const int64_t in_st[3][2] = {{q_stride_t, q_stride_h}, {k_stride_t, k_stride_h}, {v_stride_t, v_stride_h}};
  const int64_t out_st[2][2] = {{qo_stride_t, qo_stride_h}, {0, 0}};
  NVQ_TRY(check_rope(who, r, T, Hq, Hkv, D, in_st, out_st, q_weight, k_weight, eps, table, P, R, pairs, positions, axes, sections));
  if (T > 0 && !aligned(slots, 8)) return fail(NVQ_ERR_ALIGN, "%s: slots must be 8-byte aligned", who);
  if (T == 0) return NVQ_OK;
  NVQ_TRY(check_device());
  return launched(nvq::launch_rope(r, T, D, fmt, &c, slots, (hipStream_t)stream), who);
}

// One new token per sequence: the capacity in keys of all sequences stays below 2^30, so that
// key numbers and rounded chunk lengths fit an int.
static bool decode_shape_ok(int64_t B, int64_t Hq, int64_t Hkv, int64_t D, int64_t max_pages, int64_t page) {
  return B >= 1 && B < kMaxDim && Hkv >= 1 && Hkv <= 65536 && Hq >= Hkv && Hq <= 65536 && Hq % Hkv == 0 && D >= 32 && D <= 256 &&
         D % 32 == 0 && page_ok(page) && max_pages >= 1 && max_pages < kMaxDim / 2 / page && B * (max_pages * page) < kMaxDim / 2 &&
         nvq::attn_decode_fits(B, Hq, Hkv, max_pages * page);
}

size_t nvq_attn_decode_workspace_bytes(int64_t B, int64_t Hq, int64_t Hkv, int64_t D, int64_t max_pages, int64_t page) {
  if (!decode_shape_ok(B, Hq, Hkv, D, max_pages, page)) return 0;
  return nvq::attn_decode_workspace(B, Hq, Hkv, D, max_pages * page);
}

static nvq_status attn_decode(const char* who, int fmt, int type, const void* q, int64_t q_stride_b, int64_t q_stride_h, int64_t B,
                              int64_t Hq, int64_t Hkv, int64_t D, const void* k_cache, const void* v_cache, const uint16_t* k_d,
                              const uint16_t* v_d, int64_t n_pages, int64_t page, const int32_t* table, int64_t max_pages,
                              const int32_t* lengths, float scale, int64_t window, int64_t sinks, void* out, void* workspace,
                              size_t ws_bytes, void* stream) {
  if (type < NVQ_TYPE_F32 || type > NVQ_TYPE_BF16) return fail(NVQ_ERR_RANGE, "%s: type=%d is not NVQ_TYPE_*", who, type);
  nvq::KvCache c;
  NVQ_TRY(check_cache(who, fmt, k_cache, v_cache, k_d, v_d, Hkv, D, n_pages, page, c));
  if (window < 0 || sinks < 0) return fail(NVQ_ERR_RANGE, "%s: window=%lld and sinks=%lld must not be negative", who, (long long)window, (long long)sinks);
  if (B == 0) return NVQ_OK;
  if (!decode_shape_ok(B, Hq, Hkv, D, max_pages, page))
    return fail(NVQ_ERR_SHAPE, "%s: B=%lld, Hq=%lld, Hkv=%lld, max_pages=%lld, page=%lld out of range (Hq a multiple of Hkv, B * max_pages * page < 2^30, B * Hkv * ceil(Hq / Hkv / 16) < 2^23)",
                who, (long long)B, (long long)Hq, (long long)Hkv, (long long)max_pages, (long long)page);
  if (!q || !table || !lengths || !out) return fail(NVQ_ERR_NULL, "%s: NULL pointer", who);
  NVQ_TRY(check_rows(who, "q", q, type, B, Hq, q_stride_b, q_stride_h));
  if (!aligned(out, 16) || !aligned(table, 4) || !aligned(lengths, 4))
    return fail(NVQ_ERR_ALIGN, "%s: out must be 16-byte aligned, table and lengths 4-byte", who);
  // (no sequence has more keys than the tables' pages hold; a window of them all, or first keys that are all, is none)
  const int64_t keys = max_pages * page;
  if (window >= keys || sinks >= keys) window = 0;
  const size_t need = nvq::attn_decode_workspace(B, Hq, Hkv, D, window ? nvq::attn_window_capacity(keys, window, sinks) : keys);
  if (need > 0 && (!workspace || ws_bytes < need)) return fail(NVQ_ERR_WORKSPACE, "%s: workspace of %zu bytes required, got %zu", who, need, workspace ? ws_bytes : (size_t)0);
  if (need > 0 && !aligned(workspace, 16)) return fail(NVQ_ERR_ALIGN, "%s: workspace must be 16-byte aligned", who);
  NVQ_TRY(check_device());
  if (window)
    return launched(nvq::launch_attn_decode_window(fmt, type, q, q_stride_b, q_stride_h, B, Hq, Hkv, D, c, table, max_pages, lengths, scale,
                                                   (int)window, (int)sinks, out, workspace, (hipStream_t)stream), who);
  return launched(nvq::launch_attn_decode(fmt, type, q, q_stride_b, q_stride_h, B, Hq, Hkv, D, c, table, max_pages, lengths, scale, out,
                                          workspace, (hipStream_t)stream), who);
}

nvq_status nvq_attn_decode(int fmt, int type, const void* q, int64_t q_stride_b, int64_t q_stride_h, int64_t B, int64_t Hq,
                           int64_t Hkv, int64_t D, const void* k_cache, const void* v_cache, const uint16_t* k_d,
                           const uint16_t* v_d, int64_t n_pages, int64_t page, const int32_t* table, int64_t max_pages,
                           const int32_t* lengths, float scale, void* out, void* workspace, size_t ws_bytes, void* stream) {
  return attn_decode("nvq_attn_decode", fmt, type, q, q_stride_b, q_stride_h, B, Hq, Hkv, D, k_cache, v_cache, k_d, v_d, n_pages, page, table,
                     max_pages, lengths, scale, 0, 0, out, workspace, ws_bytes, stream);
}

nvq_status nvq_attn_decode_window(int fmt, int type, const void* q, int64_t q_stride_b, int64_t q_stride_h, int64_t B, int64_t Hq,
                                  int64_t Hkv, int64_t D, const void* k_cache, const void* v_cache, const uint16_t* k_d,
                                  const uint16_t* v_d, int64_t n_pages, int64_t page, const int32_t* table, int64_t max_pages,
                                  const int32_t* lengths, float scale, int64_t window, int64_t sinks, void* out, void* workspace,
                                  size_t ws_bytes, void* stream) {
  return attn_decode("nvq_attn_decode_window", fmt, type, q, q_stride_b, q_stride_h, B, Hq, Hkv, D, k_cache, v_cache, k_d, v_d, n_pages, page,
                     table, max_pages, lengths, scale, window, sinks, out, workspace, ws_bytes, stream);
}

nvq_status nvq_attn_prompt(int type, const void* q, const void* k, const void* v, void* out, const int64_t* strides,
                           const int32_t* cu_q, const int32_t* cu_k, int64_t B, int64_t Tq, int64_t Tk, int64_t Hq,
                           int64_t Hkv, int64_t D, float scale, int causal, void* stream) {
  const char* who = "nvq_attn_prompt";
  if (type != NVQ_TYPE_F16 && type != NVQ_TYPE_BF16) return fail(NVQ_ERR_RANGE, "%s: type=%d must be NVQ_TYPE_F16 or NVQ_TYPE_BF16", who, type);
  NVQ_TRY(check_head(who, Hkv, D));
  if (Hq < Hkv || Hq > 65536 || Hq % Hkv != 0) return fail(NVQ_ERR_SHAPE, "%s: Hq=%lld must be a multiple of Hkv=%lld", who, (long long)Hq, (long long)Hkv);
  constexpr int64_t most = int64_t(1) << 30;
  if (B < 0 || B >= most || Tq < 0 || Tq >= most || Tk < 0 || Tk >= most)
    return fail(NVQ_ERR_SHAPE, "%s: B=%lld, Tq=%lld, Tk=%lld out of range", who, (long long)B, (long long)Tq, (long long)Tk);
  if (B == 0 || Tq == 0) return NVQ_OK;
  if (!q || !out || !strides || !cu_q || !cu_k || (Tk > 0 && (!k || !v))) return fail(NVQ_ERR_NULL, "%s: NULL pointer", who);
  NVQ_TRY(check_rows(who, "q", q, type, Tq, Hq, strides[0], strides[1]));
  NVQ_TRY(check_rows(who, "k", k, type, Tk, Hkv, strides[2], strides[3]));
  NVQ_TRY(check_rows(who, "v", v, type, Tk, Hkv, strides[4], strides[5]));
  NVQ_TRY(check_rows(who, "out", out, type, Tq, Hq, strides[6], strides[7]));
  NVQ_TRY(check_apart(who, "out", Tq, Hq, D, strides[6], strides[7]));
  // a tile's 64 rows are addressed by 32-bit offsets
  if (Tk > 1 && (strides[2] >= (int64_t(1) << 24) || strides[4] >= (int64_t(1) << 24)))
    return fail(NVQ_ERR_SHAPE, "%s: token strides of k and v must be below 2^24 elements", who);
  if (!nvq::attn_prompt_fits(B, Tq, Hq))
    return fail(NVQ_ERR_SHAPE, "%s: B=%lld, Tq=%lld: too many query tiles ((Tq / 128 + B) * Hq < 2^24)", who, (long long)B, (long long)Tq);
  if (!aligned(cu_q, 4) || !aligned(cu_k, 4)) return fail(NVQ_ERR_ALIGN, "%s: cu_q and cu_k must be 4-byte aligned", who);
  NVQ_TRY(check_device());
  return launched(nvq::launch_attn_prompt(type, q, k, v, out, strides, cu_q, cu_k, B, Tq, Tk, Hq, Hkv, D, scale, causal ? 1 : 0,
                                          (hipStream_t)stream), who);
}

static bool chunk_shape_ok(int64_t B, int64_t Tq, int64_t Hq, int64_t Hkv, int64_t D, int64_t max_pages, int64_t page) {
  constexpr int64_t most = int64_t(1) << 30;
  return B >= 1 && B < most && Tq >= 1 && Tq < most && Hkv >= 1 && Hkv <= 65536 && Hq >= Hkv && Hq <= 65536 && Hq % Hkv == 0 && D >= 32 && D <= 256 &&
         D % 32 == 0 && page_ok(page) && max_pages >= 1 && max_pages < most / page && nvq::attn_chunk_fits(B, Tq, Hq, Hkv, D, max_pages * page);
}

// A window of all keys that the tables' pages can hold, or first keys that are all of them, is none.
static int64_t chunk_window(int64_t keys, int64_t window, int64_t sinks) { return window >= keys || sinks >= keys ? 0 : window; }

size_t nvq_attn_chunk_workspace_bytes(int fmt, int64_t B, int64_t Tq, int64_t Hq, int64_t Hkv, int64_t D, int64_t max_pages, int64_t page,
                                      int64_t window, int64_t sinks) {
  if (!chunk_shape_ok(B, Tq, Hq, Hkv, D, max_pages, page) || window < 0 || sinks < 0 || fmt < NVQ_KV_Q8_0 || fmt > NVQ_KV_BF16) return 0;
  return nvq::attn_chunk_workspace(fmt, B, Tq, Hq, Hkv, D, max_pages * page, chunk_window(max_pages * page, window, sinks), sinks);
}

nvq_status nvq_attn_chunk(int fmt, int type, const void* q, const int64_t* strides, int64_t B, int64_t Tq, int64_t Hq, int64_t Hkv,
                          int64_t D, const void* k_cache, const void* v_cache, const uint16_t* k_d, const uint16_t* v_d,
                          int64_t n_pages, int64_t page, const int32_t* table, int64_t max_pages, const int32_t* cu_q,
                          const int32_t* lengths, float scale, int64_t window, int64_t sinks, void* out, void* workspace,
                          size_t ws_bytes, void* stream) {
  const char* who = "nvq_attn_chunk";
  if (type != NVQ_TYPE_F16 && type != NVQ_TYPE_BF16) return fail(NVQ_ERR_RANGE, "%s: type=%d must be NVQ_TYPE_F16 or NVQ_TYPE_BF16", who, type);
  nvq::KvCache c;
  NVQ_TRY(check_cache(who, fmt, k_cache, v_cache, k_d, v_d, Hkv, D, n_pages, page, c));
  if (fmt != NVQ_KV_Q8_0 && (fmt == NVQ_KV_F16) != (type == NVQ_TYPE_F16))
    return fail(NVQ_ERR_RANGE, "%s: queries over a 16-bit cache must be of its type", who);
  if (window < 0 || sinks < 0) return fail(NVQ_ERR_RANGE, "%s: window=%lld and sinks=%lld must not be negative", who, (long long)window, (long long)sinks);
  if (B < 0 || Tq < 0) return fail(NVQ_ERR_SHAPE, "%s: B=%lld, Tq=%lld out of range", who, (long long)B, (long long)Tq);
  if (B == 0 || Tq == 0) return NVQ_OK;
  if (!chunk_shape_ok(B, Tq, Hq, Hkv, D, max_pages, page))
    return fail(NVQ_ERR_SHAPE, "%s: B=%lld, Tq=%lld, Hq=%lld, Hkv=%lld, max_pages=%lld, page=%lld out of range (Hq a multiple of Hkv, max_pages * page < 2^30, "
                "(Tq * Hq / Hkv / 128 + B) * ceil(max_pages * page / 64) < 2^31, (Tq * Hq / Hkv / 128 + B) * Hkv < 2^24 - 512)",
                who, (long long)B, (long long)Tq, (long long)Hq, (long long)Hkv, (long long)max_pages, (long long)page);
  if (!q || !strides || !table || !cu_q || !lengths || !out) return fail(NVQ_ERR_NULL, "%s: NULL pointer", who);
  NVQ_TRY(check_rows(who, "q", q, type, Tq, Hq, strides[0], strides[1]));
  NVQ_TRY(check_rows(who, "out", out, type, Tq, Hq, strides[2], strides[3]));
  NVQ_TRY(check_apart(who, "out", Tq, Hq, D, strides[2], strides[3]));
  if (!aligned(table, 4) || !aligned(cu_q, 4) || !aligned(lengths, 4)) return fail(NVQ_ERR_ALIGN, "%s: table, cu_q and lengths must be 4-byte aligned", who);
  const int64_t keys = max_pages * page;
  window = chunk_window(keys, window, sinks);
  const size_t need = nvq::attn_chunk_workspace(fmt, B, Tq, Hq, Hkv, D, keys, window, sinks);
  if (need > 0 && (!workspace || ws_bytes < need)) return fail(NVQ_ERR_WORKSPACE, "%s: workspace of %zu bytes required, got %zu", who, need, workspace ? ws_bytes : (size_t)0);
  if (need > 0 && !aligned(workspace, 16)) return fail(NVQ_ERR_ALIGN, "%s: workspace must be 16-byte aligned", who);
  NVQ_TRY(check_device());
  return launched(nvq::launch_attn_chunk(fmt, type, q, out, strides, B, Tq, Hq, Hkv, D, c, table, max_pages, cu_q, lengths, (int)window,
                                         window ? (int)sinks : 0, scale, workspace, (hipStream_t)stream), who);
}

// ---- measurement probes (include/nvq_probe.h) ----

nvq_status nvq_probe_read(const void* src, size_t bytes, int blocks, uint32_t* sink, void* stream) {
  if (!src || !sink) return fail(NVQ_ERR_NULL, "nvq_probe_read: NULL pointer");
  if (!aligned(src, 16) || !aligned(sink, 4))
    return fail(NVQ_ERR_ALIGN, "nvq_probe_read: src must be 16-byte aligned, sink 4-byte");
  if (bytes == 0 || bytes % 16 != 0 || bytes >= (size_t(1) << 46))
    return fail(NVQ_ERR_SHAPE, "nvq_probe_read: bytes=%zu must be a positive multiple of 16", bytes);
  if (blocks < 1 || blocks > 65536) return fail(NVQ_ERR_SHAPE, "nvq_probe_read: blocks=%d outside [1, 65536]", blocks);
  NVQ_TRY(check_device());
  return launched(nvq::launch_probe_read(src, (int64_t)(bytes / 16), blocks, sink, (hipStream_t)stream), "probe_read");
}

nvq_status nvq_probe_gemv_loads(const void* w, int64_t N, int64_t K, int splits, int waves, int batch,
                                uint32_t* sink, void* stream) {
  if (!w || !sink) return fail(NVQ_ERR_NULL, "nvq_probe_gemv_loads: NULL pointer");
  if (!aligned(w, 16) || !aligned(sink, 4))
    return fail(NVQ_ERR_ALIGN, "nvq_probe_gemv_loads: w must be 16-byte aligned, sink 4-byte");
  NVQ_TRY(check_dims(1, N, K, 64, 1, 1));
  const int64_t nch = (K + 127) / 128;
  if (splits < 1 || splits > 8 || splits > nch)
    return fail(NVQ_ERR_RANGE, "nvq_probe_gemv_loads: splits=%d outside [1, min(8, %lld)]", splits, (long long)nch);
  if ((waves != 4 && waves != 8 && waves != 16) || (batch != 3 && batch != 5))
    return fail(NVQ_ERR_RANGE, "nvq_probe_gemv_loads: waves=%d, batch=%d not in {4, 8, 16} x {3, 5}", waves, batch);
  if (((N + 15) / 16) * splits >= (int64_t(1) << 31))
    return fail(NVQ_ERR_SHAPE, "nvq_probe_gemv_loads: grid too large");
  NVQ_TRY(check_device());
  return launched(nvq::launch_probe_gemv_loads(static_cast<const uint8_t*>(w), N, K, splits, waves, batch, sink,
                                               (hipStream_t)stream), "probe_gemv_loads");
}

nvq_status nvq_probe_mfma(int blocks, int64_t iters, int random_operands, float* out, void* stream) {
  if (!out) return fail(NVQ_ERR_NULL, "nvq_probe_mfma: NULL pointer");
  if (!aligned(out, 4)) return fail(NVQ_ERR_ALIGN, "nvq_probe_mfma: out must be 4-byte aligned");
  if (blocks < 1 || blocks > 65536) return fail(NVQ_ERR_SHAPE, "nvq_probe_mfma: blocks=%d outside [1, 65536]", blocks);
  if (iters < 1 || iters > (int64_t(1) << 31)) return fail(NVQ_ERR_SHAPE, "nvq_probe_mfma: iters=%lld outside [1, 2^31]", (long long)iters);
  NVQ_TRY(check_device());
  return launched(nvq::launch_probe_mfma(blocks, iters, random_operands, out, (hipStream_t)stream), "probe_mfma");
}

}  // extern "C"
