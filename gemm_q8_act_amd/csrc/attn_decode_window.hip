// attn_decode_window.hip -- attention of one new token per sequence over a sliding window of its keys and
// the first ones; the kernels are in attn_decode.h.
#include "attn_decode.h"

namespace nvq {

int64_t attn_window_capacity(int64_t capacity, int64_t window, int64_t sinks) {
  // both parts' groups of 16 reach at most 15 keys further
  const int64_t most = window + sinks + 30;
  return capacity < most ? capacity : most;
}

hipError_t launch_attn_decode_window(int fmt, int type, const void* q, int64_t q_stride_b, int64_t q_stride_h, int64_t B,
                                     int64_t Hq, int64_t Hkv, int64_t D, const KvCache& c, const int32_t* table,
                                     int64_t table_stride, const int32_t* lengths, float scale, int window, int sinks, void* out,
                                     void* workspace, hipStream_t stream) {
  return launch_with<true>(fmt, type, q, q_stride_b, q_stride_h, B, Hq, Hkv, D, c, table, table_stride, lengths, scale, window, sinks,
                           attn_window_capacity(table_stride << c.page_shift, window, sinks), out, workspace, stream);
}

}  // namespace nvq
