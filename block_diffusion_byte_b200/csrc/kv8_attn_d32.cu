// Attention over the 8-bit KV cache: kernels for head dimension 32.
#include "kv8_attn.cuh"
#include "kv8_tile.cuh"

namespace bltdec {
cudaError_t kv8_attend_d32(int fmt, const Kv8View& c, const Kv8AttnArgs& a, int max_keys, int sm_count, cudaStream_t st) {
  return fmt == BLT_KV8_INT8 ? kv8_attend_dh<32, 0>(c, a, max_keys, sm_count, st) : kv8_attend_dh<32, 1>(c, a, max_keys, sm_count, st);
}
}  // namespace bltdec
