// Launch of the backward kernels within a sliding window (see bwd.cuh, WindowTiles): as the
// dense ones without the tiles that hold no visible pair, and with the first tokens' key
// tiles, which all later queries see, cut in pieces. 12544 tokens, 1568 keys each, 16 heads on
// 4 of 128: 577 us, 661 TFLOP/s of visible pairs (dense: 917; 388 whole items and 28 pieces on
// 152 SMs take three rounds of 2.4); 2 x 6273 tokens, 784 keys to both sides, 16 heads of 64:
// 357 us, 529 TFLOP/s.
#include "bwd.cuh"

namespace eba {

cudaError_t launch_bwd_window(const CUtensorMap& tq, const CUtensorMap& tk, const CUtensorMap& tv,
                              const CUtensorMap& tdo, const CUtensorMap& tdqa, const BwdArgs& a,
                              const WindowTiles& wt, int d, cudaStream_t stream) {
  const long long items =
      (a.n_ktiles - wt.blind_tiles + static_cast<long long>(wt.cut_tiles) * (wt.pieces - 1)) * a.B * a.H_kv;
  const double tpi = static_cast<double>(a.group) * wt.run_tiles;
  if (a.group > 1)
    return d == 64 ? launch_bwd_k<64, WindowTiles, true>(tq, tk, tv, tdo, tdqa, a, wt, items, tpi, stream)
                   : launch_bwd_k<128, WindowTiles, true>(tq, tk, tv, tdo, tdqa, a, wt, items, tpi, stream);
  return d == 64 ? launch_bwd_k<64, WindowTiles>(tq, tk, tv, tdo, tdqa, a, wt, items, tpi, stream)
                 : launch_bwd_k<128, WindowTiles>(tq, tk, tv, tdo, tdqa, a, wt, items, tpi, stream);
}

}  // namespace eba
