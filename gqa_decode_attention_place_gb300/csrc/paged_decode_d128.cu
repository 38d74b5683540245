// paged_decode_d128.cu -- the paged decode at head dim 128, one new token.
#include "paged_decode.cuh"

namespace gqa {

cudaError_t launch_paged_decode_128(PagedParams& p, const PagedPool& pool, cudaStream_t stream) {
  return launch_paged_rows<128, false>(p, pool, stream);
}

}  // namespace gqa
