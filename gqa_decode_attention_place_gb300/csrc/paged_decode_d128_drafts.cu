// paged_decode_d128_drafts.cu -- the paged decode at head dim 128, several new tokens.
#include "paged_decode.cuh"

namespace gqa {

cudaError_t launch_paged_decode_128_drafts(PagedParams& p, const PagedPool& pool,
                                           cudaStream_t stream) {
  return launch_paged_rows<128, true>(p, pool, stream);
}

}  // namespace gqa
