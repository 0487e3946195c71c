// Instances of the few-row chunk kernel with 4-bit keys (see chunk_few.cuh), and the dispatch.
#include "chunk_few.cuh"

namespace kvq {
namespace few {

LaunchFn find_4(const Dims& d, int rows) {
  KVQ_CHUNK_FEW_4(KVQ_CHUNK_FEW_ENTRY)
  return nullptr;
}

}  // namespace few

bool chunk_few_supported(const Dims& d, int T) {
  if (d.var || d.sr || d.dv != few::kDV || d.n_rep * T > 16) return false;
  return few::find_4(d, d.n_rep * T) || few::find_28(d, d.n_rep * T);
}

cudaError_t launch_chunk_few(const Dims& d, const CacheBufs& c, const ChunkArgs& a, cudaStream_t s) {
  few::LaunchFn fn = few::find_4(d, d.n_rep * a.T);
  if (!fn) fn = few::find_28(d, d.n_rep * a.T);
  return fn ? fn(d, c, a, s) : cudaErrorNotSupported;
}

}  // namespace kvq
