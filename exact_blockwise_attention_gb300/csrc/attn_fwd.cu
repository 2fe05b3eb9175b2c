// Launches of the forward kernel over dense heads, KV chunks, packed sequences, short
// sequences and e4m3 operands (see fwd.cuh).
#include "fwd.cuh"

namespace eba {

cudaError_t launch_fwd(const CUtensorMap& tq, const CUtensorMap& tk, const CUtensorMap& tv,
                       const FwdArgs& a, int d, bool partial, cudaStream_t stream) {
  const long long items = static_cast<long long>(a.n_pairs) * a.B * a.H * a.n_chunks;
  const NoVarlen nv{};
  if (d == 64) return partial ? launch_fwd_t<64, true>(tq, tk, tv, a, nv, items, stream)
                              : launch_fwd_t<64, false>(tq, tk, tv, a, nv, items, stream);
  return partial ? launch_fwd_t<128, true>(tq, tk, tv, a, nv, items, stream)
                 : launch_fwd_t<128, false>(tq, tk, tv, a, nv, items, stream);
}

cudaError_t launch_fwd_fp8(const CUtensorMap& tq, const CUtensorMap& tk, const CUtensorMap& tvt,
                           const FwdArgs& a, cudaStream_t stream) {
  const long long items = static_cast<long long>(a.n_pairs) * a.B * a.H;
  return launch_fwd_t<128, false, NoVarlen, true>(tq, tk, tvt, a, NoVarlen{}, items, stream);
}

cudaError_t launch_fwd_packed(const CUtensorMap& tq, const CUtensorMap& tk, const CUtensorMap& tv,
                              const FwdArgs& a, const PackedTiles& pt, int d, cudaStream_t stream) {
  const long long tiles = (static_cast<long long>(pt.n_seqs) + pt.pack - 1) / pt.pack;
  const long long items = (tiles + 1) / 2;  // two tiles per item
  return d == 64 ? launch_fwd_t<64, false>(tq, tk, tv, a, pt, items, stream)
                 : launch_fwd_t<128, false>(tq, tk, tv, a, pt, items, stream);
}

cudaError_t launch_fwd_varlen(const CUtensorMap& tq, const CUtensorMap& tk, const CUtensorMap& tv,
                              const FwdArgs& a, const VarlenTable& vt, int d, cudaStream_t stream) {
  const long long items = static_cast<long long>(vt.total) * a.H;
  return d == 64 ? launch_fwd_t<64, false>(tq, tk, tv, a, vt, items, stream)
                 : launch_fwd_t<128, false>(tq, tk, tv, a, vt, items, stream);
}

}  // namespace eba
