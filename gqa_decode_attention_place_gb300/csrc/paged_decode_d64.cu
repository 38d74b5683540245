// paged_decode_d64.cu -- the paged decode at head dim 64.
#include "paged_decode.cuh"

namespace gqa {

cudaError_t launch_paged_decode_64(PagedParams& p, const CUtensorMap& mk, const CUtensorMap& mv,
                                   cudaStream_t stream) {
  return launch_paged_rows<64>(p, mk, mv, stream);
}

}  // namespace gqa
