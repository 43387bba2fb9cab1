// attn_kv_slots.cu -- pages, slots and positions of the new tokens of a batch of requests.
//
// need_s = ceil((len_s + new_s) / P) - ceil(len_s / P) pages are taken from the free list, request
// by request, so request s's first new page sits at *free_head + sum_{r<s} need_r.  Every CTA
// builds that prefix sum over all requests in shared memory (a few loads a thread), then places its
// own 256 tokens: a search for the token's request in the prefix sums of the new tokens, the page
// from the block table (an old page) or straight from the free list (a new one).  So no CTA waits for
// another, one launch is enough, and the only entries of the table that are read are old ones while
// the only ones written are new ones (by the token that is first in its page).
// What bounds it: latency.  It moves 12 bytes a token and 20 a request.
#include "attn_gen.cuh"
#include "attn_gen.h"
#include "sm103_ptx.cuh"

#include <atomic>
#include <climits>

namespace attn {
namespace {

__global__ void __launch_bounds__(kSlotThreads) kv_slots_kernel(SlotsParams p) {
  extern __shared__ int s_mem[];
  int* s_cu = s_mem;               // [B + 1] first new token of each request, clamped into [0, T]
  int* s_first = s_mem + p.B + 1;  // [B] pages needed by earlier requests
  __shared__ int s_warp[kSlotThreads / 32];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  bool bad = false;
  pdl_wait();
  for (int s = tid; s <= p.B; s += kSlotThreads) {
    const int c = p.cu_new[s];
    s_cu[s] = min(max(c, 0), p.T);
    bad |= c != s_cu[s] || (s == 0 && c != 0) || (s == p.B && c != p.T);
  }
  __syncthreads();
  auto pages = [&](long long tokens) {
    return static_cast<int>(min((tokens + p.page_size - 1) / p.page_size,
                                static_cast<long long>(p.max_pages)));
  };
  auto added = [&](int s) { return max(s_cu[s + 1] - s_cu[s], 0); };
  for (int s = tid; s < p.B; s += kSlotThreads) {
    bad |= s_cu[s + 1] < s_cu[s];
    const int old = max(p.seq_lens[s], 0);
    const long long total = static_cast<long long>(old) + added(s);
    s_first[s] = pages(total) - pages(old);
    if (blockIdx.x == 0)
      p.seq_lens_out[s] = static_cast<int>(min(total, static_cast<long long>(INT_MAX)));
  }
  if (blockIdx.x == 0 && bad) atomicCAS(p.status, 0, kStatusBadSeqlens);
  __syncthreads();
  // exclusive prefix sum of s_first: each thread a run of consecutive requests
  const int per = (p.B + kSlotThreads - 1) / kSlotThreads;
  const int lo = min(tid * per, p.B), hi = min(lo + per, p.B);
  int sum = 0;
  for (int s = lo; s < hi; ++s) sum += s_first[s];
  int scan = sum;
  #pragma unroll
  for (int off = 1; off < 32; off <<= 1) {
    const int up = __shfl_up_sync(0xffffffffu, scan, off);
    if (lane >= off) scan += up;
  }
  if (lane == 31) s_warp[warp] = scan;
  __syncthreads();
  int before = scan - sum, all = 0;
  #pragma unroll
  for (int w = 0; w < kSlotThreads / 32; ++w) {
    if (w < warp) before += s_warp[w];
    all += s_warp[w];
  }
  for (int s = lo; s < hi; ++s) {
    const int need = s_first[s];
    s_first[s] = before;
    before += need;
  }
  const int head = *p.free_head;
  if (blockIdx.x == 0 && tid == 0) *p.free_head_out = head + all;
  __syncthreads();
  for (long long t = static_cast<long long>(blockIdx.x) * kSlotThreads + tid; t < p.T;
       t += static_cast<long long>(gridDim.x) * kSlotThreads) {
    int a = 0, b = p.B;  // the last request whose first new token is not after t
    while (b - a > 1) {
      const int m = (a + b) >> 1;
      if (s_cu[m] <= t) a = m; else b = m;
    }
    int64_t slot = -1;
    int pos = 0;
    if (t >= s_cu[a] && t < s_cu[a + 1]) {
      const int old = max(p.seq_lens[a], 0);
      const long long at = old + (t - s_cu[a]);
      pos = static_cast<int>(min(at, static_cast<long long>(INT_MAX)));
      const long long j = at / p.page_size;
      if (j < p.max_pages) {
        int* entry = p.block_table + static_cast<size_t>(a) * p.max_pages + j;
        const int fresh = static_cast<int>(j) - pages(old);
        int page;
        if (fresh < 0) {
          page = *entry;
        } else {
          const long long f = static_cast<long long>(head) + s_first[a] + fresh;
          page = f >= 0 && f < p.n_free ? p.free_pages[f] : -1;
          if (at % p.page_size == 0) *entry = page;
        }
        if (page >= 0) slot = static_cast<int64_t>(page) * p.page_size + at % p.page_size;
      }
      if (slot < 0) atomicCAS(p.status, 0, kStatusNoPage);
    }
    p.slots[t] = slot;
    p.positions[t] = pos;
  }
}

}  // namespace

cudaError_t launch_kv_slots(const SlotsParams& p, cudaStream_t stream) {
  const int smem = (2 * p.B + 1) * 4;
  static std::atomic<uint64_t> attr_done{0};
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  const uint64_t bit = 1ull << (dev & 63);
  if (!(attr_done.load(std::memory_order_acquire) & bit)) {
    e = cudaFuncSetAttribute(kv_slots_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             (2 * kMaxSlotSeqs + 1) * 4);
    if (e != cudaSuccess) return e;
    attr_done.fetch_or(bit, std::memory_order_acq_rel);
  }
  const long long want = (static_cast<long long>(p.T) + kSlotThreads - 1) / kSlotThreads;
  const int ctas = static_cast<int>(want < 1 ? 1 : want > 608 ? 608 : want);
  return launch_dependent(kv_slots_kernel, dim3(static_cast<unsigned>(ctas)), kSlotThreads, smem, stream, p);
}

}  // namespace attn
