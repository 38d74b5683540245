// paged_decode_d64.cu -- the paged decode at head dim 64, one new token.
#include "paged_decode.cuh"

namespace gqa {

cudaError_t launch_paged_decode_64(PagedParams& p, const PagedPool& pool, cudaStream_t stream) {
  return launch_paged_rows<64, false>(p, pool, stream);
}

}  // namespace gqa
