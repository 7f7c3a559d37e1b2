// attn_decode.hip -- attention of one new token per sequence over all of its keys; the kernels are
// in attn_decode.h.
#include "attn_decode.h"

namespace nvq {

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
  return launch_with<false>(fmt, type, q, q_stride_b, q_stride_h, B, Hq, Hkv, D, c, table, table_stride, lengths, scale, 0, 0,
                            table_stride << c.page_shift, out, workspace, stream);
}

}  // namespace nvq
