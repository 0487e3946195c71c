// Instances of the few-row chunk kernel with 4-bit keys (see chunk_few.cuh), and the dispatch.
#include "chunk_few.cuh"

namespace kvq {
namespace few {

LaunchFn find_4(const Dims& d, int rows) {
  KVQ_CHUNK_FEW_4(KVQ_CHUNK_FEW_ENTRY)
  return nullptr;
}

}  // namespace few

namespace {
few::LaunchFn find(const Dims& d, int T) {
  const int rows = d.n_rep * T;
  if (d.var || d.dv != few::kDV) return nullptr;
  if (d.sr) return few::find_side(d, rows);
  if (rows > 24) return nullptr;
  few::LaunchFn fn = few::find_4(d, rows);
  return fn ? fn : few::find_28(d, rows);
}
}  // namespace

bool chunk_few_supported(const Dims& d, int T) { return find(d, T) != nullptr; }

cudaError_t launch_chunk_few(const Dims& d, const CacheBufs& c, const ChunkArgs& a, cudaStream_t s) {
  few::LaunchFn fn = find(d, a.T);
  return fn ? fn(d, c, a, s) : cudaErrorNotSupported;
}

}  // namespace kvq
