// Launch of the attention of one new token per sequence over the last keys of a paged cache
// and its first ones (decode.cuh with WINDOW): the list holds only the tiles with a visible
// key, so a call reads what it uses, in whole tiles. 64 sequences of up to 50021 keys that see
// 4096 and 4 sinks, 8 heads of 128 for 32: 173 us, 6.2 TB/s, 93 % of a copy; one sequence that
// sees 1024: 10 us on the GPU.
#include "decode.cuh"

namespace eba {

cudaError_t launch_decode_window(const DecodeArgs& a, int ctas, bool join, cudaStream_t stream) {
  return launch_decode_any<true>(a, ctas, join, stream);
}

}  // namespace eba
