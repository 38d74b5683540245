// paged_decode_d64_drafts.cu -- the paged decode at head dim 64, several new tokens.
#include "paged_decode.cuh"

namespace gqa {

cudaError_t launch_paged_decode_64_drafts(PagedParams& p, const PagedPool& pool,
                                          cudaStream_t stream) {
  return launch_paged_rows<64, true>(p, pool, stream);
}

}  // namespace gqa
