// Instances of the few-row chunk kernel with a side code (see chunk_few.cuh).
#include "chunk_few.cuh"

namespace kvq {
namespace few {

LaunchFn find_side(const Dims& d, int rows) {
  KVQ_CHUNK_FEW_SIDE(KVQ_CHUNK_FEW_ENTRY)
  return nullptr;
}

}  // namespace few

}  // namespace kvq
