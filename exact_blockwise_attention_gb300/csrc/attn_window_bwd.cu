// Launch of the backward kernels within a sliding window (see bwd.cuh, WindowTiles).
#include "bwd.cuh"

namespace eba {

cudaError_t launch_bwd_window(const CUtensorMap& tq, const CUtensorMap& tk, const CUtensorMap& tv,
                              const CUtensorMap& tdo, const CUtensorMap& tdqa, const BwdArgs& a,
                              const WindowTiles& wt, int d, cudaStream_t stream) {
  const long long items =
      (a.n_ktiles + static_cast<long long>(wt.cut_tiles) * (wt.pieces - 1)) * a.B * a.H_kv;
  const double tpi = static_cast<double>(a.group) * wt.run_tiles;
  if (a.group > 1)
    return d == 64 ? launch_bwd_k<64, WindowTiles, true>(tq, tk, tv, tdo, tdqa, a, wt, items, tpi, stream)
                   : launch_bwd_k<128, WindowTiles, true>(tq, tk, tv, tdo, tdqa, a, wt, items, tpi, stream);
  return d == 64 ? launch_bwd_k<64, WindowTiles>(tq, tk, tv, tdo, tdqa, a, wt, items, tpi, stream)
                 : launch_bwd_k<128, WindowTiles>(tq, tk, tv, tdo, tdqa, a, wt, items, tpi, stream);
}

}  // namespace eba
