// Attention of one new token per sequence over the last keys of a paged key-value cache and its first
// ones (see
// decode.cuh).
#include "decode.cuh"

namespace eba {

cudaError_t launch_decode_window(const DecodeArgs& a, int ctas, bool join, cudaStream_t stream) {
  return launch_decode_any<true>(a, ctas, join, stream);
}

}  // namespace eba
