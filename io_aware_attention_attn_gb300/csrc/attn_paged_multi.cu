// attn_paged_multi.cu -- instantiations of the paged attention for the few new tokens of requests, or the few requests
// behind a prefix, and the merge of the latter's two results.
#include "attn_paged_kernel.cuh"

namespace attn {
namespace {

// The block merge of two rows over different keys: weights by their log-sum-exp.  Four columns a thread.
template <int D>
__global__ void __launch_bounds__(256) pair_merge_kernel(const __grid_constant__ PagedParams p, int groups) {
  pdl_wait();
  const int64_t all = static_cast<int64_t>(p.T) * p.H;
  const int64_t rows = static_cast<int64_t>(min(max(p.cu[groups], 0), p.T)) * p.H;
  const int64_t i = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x, at = i / (D / 4);
  const int c4 = static_cast<int>(i % (D / 4));
  if (at >= rows) return;
  const float x = p.pair_lse[at], y = p.pair_lse[all + at], top = fmaxf(x, y);
  const float4 a = *reinterpret_cast<const float4*>(p.pair_o + at * D + 4 * c4);
  const float4 b = *reinterpret_cast<const float4*>(p.pair_o + (all + at) * D + 4 * c4);
  const float wa = x == -INFINITY ? 0.f : ex2_approx((x - top) * 1.4426950408889634f);
  const float wb = y == -INFINITY ? 0.f : ex2_approx((y - top) * 1.4426950408889634f);
  const float sum = wa + wb;
  const bool some = sum > 0.f || sum != sum;
  const float inv = some ? 1.f / sum : 0.f;
  const int64_t token = at / p.H, head = at - token * p.H, to = head * p.o_head + token * p.o_token;
  *reinterpret_cast<uint2*>(p.o + to + 4 * c4) =
      make_uint2(pack_bf16x2((a.x * wa + b.x * wb) * inv, (a.y * wa + b.y * wb) * inv),
                 pack_bf16x2((a.z * wa + b.z * wb) * inv, (a.w * wa + b.w * wb) * inv));
  if (c4 == 0) p.lse[to / D] = some ? top + log2f(sum) * 0.69314718055994530942f : -INFINITY;
}

}  // namespace

cudaError_t launch_fwd_paged_multi(const PagedParams& p, int d, bool e4m3, int max_tiles,
                                   cudaStream_t stream) {
  if (d == 64)
    return e4m3 ? launch_rows<64, true, true>(p, max_tiles, stream) : launch_rows<64, false, true>(p, max_tiles, stream);
  return e4m3 ? launch_rows<128, true, true>(p, max_tiles, stream) : launch_rows<128, false, true>(p, max_tiles, stream);
}

cudaError_t launch_pair_merge(const PagedParams& p, int groups, int d, cudaStream_t stream) {
  const int64_t threads = static_cast<int64_t>(p.T) * p.H * (d / 4);  // T H is below 2^31
  const dim3 grid(static_cast<unsigned>((threads + 255) / 256));
  return d == 64 ? launch_dependent(pair_merge_kernel<64>, grid, 256, 0, stream, p, groups)
                 : launch_dependent(pair_merge_kernel<128>, grid, 256, 0, stream, p, groups);
}

}  // namespace attn
