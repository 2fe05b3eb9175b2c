// Launches of the backward kernels over dense and grouped-query heads, packed sequences
// and short sequences (see bwd.cuh).
#include "bwd.cuh"

namespace eba {

cudaError_t launch_bwd(const CUtensorMap& tq, const CUtensorMap& tk, const CUtensorMap& tv,
                       const CUtensorMap& tdo, const CUtensorMap& tdqa, const BwdArgs& a, int d,
                       cudaStream_t stream) {
  const long long items = static_cast<long long>(a.n_ktiles) * a.B * a.H_kv;
  const double tpi = static_cast<double>(a.group) * a.n_qtiles;
  const NoVarlen nv{};
  if (a.group > 1)
    return d == 64 ? launch_bwd_k<64, NoVarlen, true>(tq, tk, tv, tdo, tdqa, a, nv, items, tpi, stream)
                   : launch_bwd_k<128, NoVarlen, true>(tq, tk, tv, tdo, tdqa, a, nv, items, tpi, stream);
  return d == 64 ? launch_bwd_k<64, NoVarlen>(tq, tk, tv, tdo, tdqa, a, nv, items, tpi, stream)
                 : launch_bwd_k<128, NoVarlen>(tq, tk, tv, tdo, tdqa, a, nv, items, tpi, stream);
}

cudaError_t launch_bwd_varlen(const CUtensorMap& tq, const CUtensorMap& tk, const CUtensorMap& tv,
                              const CUtensorMap& tdo, const CUtensorMap& tdqa, const BwdArgs& a,
                              const VarlenTable& vt, int d, cudaStream_t stream) {
  const long long items = static_cast<long long>(vt.total) * a.H_kv;
  // query tiles per item, averaged over the items (a sequence's key tiles
  // each walk its query tiles, for every head of the group)
  double tiles = 0.0;
  for (int s = 0; s < vt.n_seqs; ++s)
    tiles += static_cast<double>(vt.cu_items[s + 1] - vt.cu_items[s]) * (vt.cu_qt[s + 1] - vt.cu_qt[s]);
  const double tpi = vt.total > 0 ? a.group * tiles / vt.total : 0.0;
  if (a.group > 1)
    return d == 64 ? launch_bwd_k<64, VarlenTable, true>(tq, tk, tv, tdo, tdqa, a, vt, items, tpi, stream)
                   : launch_bwd_k<128, VarlenTable, true>(tq, tk, tv, tdo, tdqa, a, vt, items, tpi, stream);
  return d == 64 ? launch_bwd_k<64, VarlenTable>(tq, tk, tv, tdo, tdqa, a, vt, items, tpi, stream)
                 : launch_bwd_k<128, VarlenTable>(tq, tk, tv, tdo, tdqa, a, vt, items, tpi, stream);
}

cudaError_t launch_bwd_packed(const CUtensorMap& tq, const CUtensorMap& tk, const CUtensorMap& tv,
                              const CUtensorMap& tdo, const CUtensorMap& tdqa, const BwdArgs& a,
                              const PackedTiles& pt, int d, cudaStream_t stream) {
  const long long items = (static_cast<long long>(pt.n_seqs) + pt.pack - 1) / pt.pack;
  return d == 64 ? launch_bwd_k<64, PackedTiles>(tq, tk, tv, tdo, tdqa, a, pt, items, 1.0, stream)
                 : launch_bwd_k<128, PackedTiles>(tq, tk, tv, tdo, tdqa, a, pt, items, 1.0, stream);
}

}  // namespace eba
