// Attention over the 8-bit KV cache: kernels for head dimension 64.
#include "kv8_attn.cuh"
#include "kv8_tile.cuh"

namespace bltdec {
cudaError_t kv8_attend_d64(int fmt, const Kv8View& c, const Kv8AttnArgs& a, int max_keys, int sm_count, cudaStream_t st) {
  return fmt == BLT_KV8_INT8 ? kv8_attend_dh<64, 0>(c, a, max_keys, sm_count, st) : kv8_attend_dh<64, 1>(c, a, max_keys, sm_count, st);
}
}  // namespace bltdec
