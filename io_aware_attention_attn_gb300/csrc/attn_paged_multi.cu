// attn_paged_multi.cu -- instantiations of the paged attention for the few new tokens of requests.
#include "attn_paged_kernel.cuh"

namespace attn {

cudaError_t launch_fwd_paged_multi(const PagedParams& p, int d, bool e4m3, int max_tiles,
                                   cudaStream_t stream) {
  const int ctas = max_tiles < kPagedMaxCtas ? max_tiles : kPagedMaxCtas;
  if (d == 64)
    return e4m3 ? launch_rows<64, true, true>(p, ctas, stream) : launch_rows<64, false, true>(p, ctas, stream);
  return e4m3 ? launch_rows<128, true, true>(p, ctas, stream) : launch_rows<128, false, true>(p, ctas, stream);
}

}  // namespace attn
