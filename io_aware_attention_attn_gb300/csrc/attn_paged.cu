// attn_paged.cu -- instantiations of the paged attention for one new token a request.
#include "attn_paged_kernel.cuh"

namespace attn {

cudaError_t launch_fwd_paged(const PagedParams& p, int d, bool e4m3, int max_tiles,
                             cudaStream_t stream) {
  const int ctas = max_tiles < kPagedMaxCtas ? max_tiles : kPagedMaxCtas;
  if (d == 64)
    return e4m3 ? launch_rows<64, true, false>(p, ctas, stream) : launch_rows<64, false, false>(p, ctas, stream);
  return e4m3 ? launch_rows<128, true, false>(p, ctas, stream) : launch_rows<128, false, false>(p, ctas, stream);
}

}  // namespace attn
