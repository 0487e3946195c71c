// Instances of the few-row chunk kernel with 2- and 8-bit keys (see chunk_few.cuh).
#include "chunk_few.cuh"

namespace kvq {
namespace few {

LaunchFn find_28(const Dims& d, int rows) {
  KVQ_CHUNK_FEW_28(KVQ_CHUNK_FEW_ENTRY)
  return nullptr;
}

}  // namespace few

}  // namespace kvq
