// Attention of one new token per sequence over a paged key-value cache (see
// decode.cuh).
#include "decode.cuh"

namespace eba {

cudaError_t launch_decode(const DecodeArgs& a, int ctas, bool join, cudaStream_t stream) {
  return launch_decode_any<false>(a, ctas, join, stream);
}

}  // namespace eba
