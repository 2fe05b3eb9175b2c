// Launch of the forward kernel within a sliding window (see fwd.cuh, WindowTiles): tiles
// without a visible pair are left out, the others computed whole, as tensor cores want them.
// What is computed beyond the visible pairs is half a tile at each end of a tile's window, and
// what bounds it is what bounds the dense kernel, at items of fewer rounds: 12544 tokens, 1568
// keys each, 16 heads on 4 of 128: 179 us, 850 TFLOP/s of visible pairs (dense: 1277);
// 2 x 6273 tokens, 784 keys to both sides, 16 heads of 64: 145 us, 523 TFLOP/s. Both lists
// are 5.2 to 5.3 rounds of the SMs and take six, and a query tile computes a whole key tile for
// the sinks, be it one.
#include "fwd.cuh"

namespace eba {

cudaError_t launch_fwd_window(const CUtensorMap& tq, const CUtensorMap& tk, const CUtensorMap& tv,
                              const FwdArgs& a, const WindowTiles& wt, int d, cudaStream_t stream) {
  const long long items = static_cast<long long>(a.n_pairs) * a.B * a.H;
  return d == 64 ? launch_fwd_t<64, false>(tq, tk, tv, a, wt, items, stream)
                 : launch_fwd_t<128, false>(tq, tk, tv, a, wt, items, stream);
}

}  // namespace eba
