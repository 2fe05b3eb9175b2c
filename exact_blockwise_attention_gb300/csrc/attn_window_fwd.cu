// Launch of the forward kernel within a sliding window (see fwd.cuh, WindowTiles).
#include "fwd.cuh"

namespace eba {

cudaError_t launch_fwd_window(const CUtensorMap& tq, const CUtensorMap& tk, const CUtensorMap& tv,
                              const FwdArgs& a, const WindowTiles& wt, int d, cudaStream_t stream) {
  const long long items = static_cast<long long>(a.n_pairs) * a.B * a.H;
  return d == 64 ? launch_fwd_t<64, false>(tq, tk, tv, a, wt, items, stream)
                 : launch_fwd_t<128, false>(tq, tk, tv, a, wt, items, stream);
}

}  // namespace eba
