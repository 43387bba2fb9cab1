// attn_chunk.cu -- the join of the parts that attn_chunk_kernel leaves, its instantiations and launcher.
#include <atomic>

#include "attn_chunk_kernel.cuh"

namespace attn {
namespace {

// Merge of units' parts: M = max m_j, weights 2^(m_j - M).  A unit is merged that one share ends and an earlier one began;
// every block looks the shares' records through for those, and the units' pieces -- 32 rows and 8 columns, a warp each;
// parts lie column by column, so its loads are contiguous -- go round the blocks.  Of units of many parts a warp takes every
// second, fourth or eighth, joined through shared memory.  What bounds it is the latency of the few loads in a row (blocks
// of their own for each share, most of which end no unit: 15 us for 8 units of 10 parts, 30 for 150 of 2).
constexpr int kJoinWarps = 8, kAtOnce = 4, kJoinBlocks = 4 * 152;

template <int D>
__global__ void __launch_bounds__(kJoinWarps * 32) chunk_join_kernel(const __grid_constant__ ChunkParams p) {
  __shared__ float s_o[kJoinWarps][8][32];
  __shared__ float2 s_ml[kJoinWarps][32];
  __shared__ int s_ends[kChunkMaxShares];  // shares that end a unit of several
  __shared__ int s_count;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  if (threadIdx.x == 0) s_count = 0;
  const bool idle = p.few_rows > 0 && chunk::all_few(p);
  pdl_wait();  // by every block, so that the work after this one waits for the parts' kernel too
  if (idle) return;
  const int total = p.head[0], n_shares = p.head[1], most = p.clusters * p.max_rounds;
  if (warp == 0) {  // in order, by one warp
    int n = 0;
    for (int x0 = 0; x0 < most; x0 += 32 * 10) {  // (all records, so that they need not wait for the count)
      int tiles[10];
      #pragma unroll
      for (int k = 0; k < 10; ++k) {
        const int x = x0 + 32 * k + lane;
        tiles[k] = x < most ? p.desc[x].tiles : -1;
      }
      #pragma unroll
      for (int k = 0; k < 10; ++k) {
        const bool ends = tiles[k] >= 0 && x0 + 32 * k + lane < n_shares;
        const uint32_t has = __ballot_sync(0xffffffffu, ends);
        if (ends) s_ends[n + __popc(has & ((1u << lane) - 1u))] = x0 + 32 * k + lane;
        n += __popc(has);
      }
    }
    if (lane == 0) s_count = n;
  }
  __syncthreads();
  const int units = s_count;
  if (units == 0) return;
  const Shares shares(static_cast<uint32_t>(total), static_cast<uint32_t>(n_shares));
  // warps of a piece, by the parts of a unit on average
  const int mean = n_shares / units + 1;
  const int share = mean <= kAtOnce ? 1 : mean <= 2 * kAtOnce ? 2 : mean <= 4 * kAtOnce ? 4 : 8;
  const int side = kJoinWarps / share, sub = warp % share;
  const int groups = (p.part_rows + 31) / 32;             // of 32 rows
  const int per = (groups * (D / 8) + side - 1) / side;   // blocks of a unit
  for (int it = blockIdx.x; it < units * per; it += gridDim.x) {
    const int x = s_ends[it / per];
    const ChunkDesc d = p.desc[x];
    const int i0 = shares.owner(static_cast<uint32_t>(d.unit0)), n = x - i0 + 1;
    // the beginning share's second part, if it holds tiles of the unit before
    const int second = second_part(shares.start(i0), d.unit0, p.shape.cost);
    const int z = d.u / p.n_rg, head0 = (d.u - z * p.n_rg) * p.rg_rows;
    const int task = (it % per) * side + warp / share, c8 = task % (D / 8);
    const int at = (task / (D / 8)) * 32 + lane, row = at & (kChunkRows - 1);
    const int tok_in = row / p.rg_rows, head = row - tok_in * p.rg_rows;
    const int tok = (at >> 7) * p.cta_tokens + tok_in;
    const bool valid = at < p.part_rows && tok_in < p.cta_tokens && tok < d.n_tok && head0 + head < p.group;
    const int64_t tq = d.tok + tok, hq = z * p.group + head0 + head;
    // the same row over other keys, on its way while the parts are
    float other = -INFINITY;
    float4 ta = make_float4(0.f, 0.f, 0.f, 0.f), tb = ta;
    if (p.tail_o && sub == 0 && valid) {
      other = p.tail_lse[tq * p.H + hq];
      const float4* src = reinterpret_cast<const float4*>(p.tail_o + (tq * p.H + hq) * D + 8 * c8);
      ta = src[0];
      tb = src[1];
    }
    float acc[8], m = -INFINITY, l = 0.f;
    #pragma unroll
    for (int c = 0; c < 8; ++c) acc[c] = 0.f;
    if (valid) {
      for (int j0 = sub; j0 < n; j0 += kAtOnce * share) {
        float2 ml[kAtOnce];
        float4 a[kAtOnce], b[kAtOnce];
        #pragma unroll
        for (int k = 0; k < kAtOnce; ++k) {
          const int j = j0 + k * share;
          ml[k] = make_float2(-INFINITY, 0.f);
          a[k] = b[k] = make_float4(0.f, 0.f, 0.f, 0.f);
          if (j < n) {
            const int64_t slot = 2 * (i0 + j) + (j == 0 ? second : 0);
            ml[k] = *reinterpret_cast<const float2*>(p.part_ml + (slot * p.part_rows + at) * 2);
            const float4* src = reinterpret_cast<const float4*>(p.part_o + slot * p.part_rows * D) + at;
            a[k] = src[(2 * c8) * p.part_rows];
            b[k] = src[(2 * c8 + 1) * p.part_rows];
          }
        }
        float top = m;
        #pragma unroll
        for (int k = 0; k < kAtOnce; ++k) top = fmaxf(top, ml[k].x);
        // a maximum of -inf: nothing, or NaN, which stays
        const float keep = m == -INFINITY ? 1.f : ex2_approx(m - top);
        l *= keep;
        #pragma unroll
        for (int c = 0; c < 8; ++c) acc[c] *= keep;
        #pragma unroll
        for (int k = 0; k < kAtOnce; ++k) {
          const float wt = ml[k].x == -INFINITY ? 1.f : ex2_approx(ml[k].x - top);
          const float v[8] = {a[k].x, a[k].y, a[k].z, a[k].w, b[k].x, b[k].y, b[k].z, b[k].w};
          l = fmaf(wt, ml[k].y, l);
          #pragma unroll
          for (int c = 0; c < 8; ++c) acc[c] = fmaf(wt, v[c], acc[c]);
        }
        m = top;
      }
    }
    if (share > 1) {  // the same for the whole block
      #pragma unroll
      for (int c = 0; c < 8; ++c) s_o[warp][c][lane] = acc[c];
      s_ml[warp][lane] = make_float2(m, l);
      __syncthreads();
      if (sub == 0) {
        float top = -INFINITY;
        for (int k = 0; k < share; ++k) top = fmaxf(top, s_ml[warp + k][lane].x);
        m = top;
        l = 0.f;
        #pragma unroll
        for (int c = 0; c < 8; ++c) acc[c] = 0.f;
        for (int k = 0; k < share; ++k) {
          const float2 ml = s_ml[warp + k][lane];
          const float wt = ml.x == -INFINITY ? 1.f : ex2_approx(ml.x - top);
          l = fmaf(wt, ml.y, l);
          #pragma unroll
          for (int c = 0; c < 8; ++c) acc[c] = fmaf(wt, s_o[warp + k][c][lane], acc[c]);
        }
      }
      __syncthreads();
    }
    if (sub != 0 || !valid) continue;
    float wt = l > 0.f || l != l ? 1.f / l : 0.f;
    float lse = l > 0.f || l != l ? (m + log2f(l)) * 0.69314718055994530942f : -INFINITY;
    #pragma unroll
    for (int c = 0; c < 8; ++c) acc[c] *= wt;
    if (p.tail_o) {
      const float top = fmaxf(lse, other);
      const float wa = lse == -INFINITY ? 0.f : ex2_approx((lse - top) * 1.4426950408889634f);
      const float wb = other == -INFINITY ? 0.f : ex2_approx((other - top) * 1.4426950408889634f);
      const float sum = wa + wb, inv = sum > 0.f || sum != sum ? 1.f / sum : 0.f;
      const float v[8] = {ta.x, ta.y, ta.z, ta.w, tb.x, tb.y, tb.z, tb.w};
      #pragma unroll
      for (int c = 0; c < 8; ++c) acc[c] = (acc[c] * wa + v[c] * wb) * inv;
      lse = sum > 0.f || sum != sum ? top + log2f(sum) * 0.69314718055994530942f : -INFINITY;
    }
    const int64_t to = hq * p.o_head + tq * p.o_token;
    *reinterpret_cast<uint4*>(p.o + to + 8 * c8) =
        make_uint4(pack_bf16x2(acc[0], acc[1]), pack_bf16x2(acc[2], acc[3]), pack_bf16x2(acc[4], acc[5]),
                   pack_bf16x2(acc[6], acc[7]));
    if (c8 == 0) p.lse[to / D] = lse;
  }
}

template <int D, bool E4M3>
cudaError_t launch(const ChunkParams& p, cudaStream_t stream) {
  using L = ChunkLayout<D, E4M3>;
  auto* kernel = attn_chunk_kernel<D, E4M3>;
  static std::atomic<int> fit[64] = {};  // clusters that fit at once, per device (0: not known yet)
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  int clusters = fit[dev & 63].load(std::memory_order_acquire);
  if (clusters == 0) {
    e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, L::kDyn);
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(2 * kChunkClusters);
    cfg.blockDim = dim3(L::kThreads);
    cfg.dynamicSmemBytes = L::kDyn;
    int n = 0;
    if (cudaOccupancyMaxActiveClusters(&n, kernel, &cfg) != cudaSuccess || n <= 0) {
      (void)cudaGetLastError();
      n = kChunkClusters;
    }
    clusters = n < kChunkClusters ? n : kChunkClusters;
    fit[dev & 63].store(clusters, std::memory_order_release);
  }
  ChunkParams q = p;
  if (q.clusters > clusters) q.clusters = clusters;
  e = launch_dependent(kernel, dim3(2 * static_cast<unsigned>(q.clusters)), L::kThreads, L::kDyn, stream, q);
  if (e != cudaSuccess) return e;
  return launch_dependent(chunk_join_kernel<D>, dim3(kJoinBlocks), kJoinWarps * 32, 0, stream, q);
}

}  // namespace

cudaError_t launch_chunk(const ChunkParams& p, int d, bool e4m3, cudaStream_t stream) {
  if (d == 64) return e4m3 ? launch<64, true>(p, stream) : launch<64, false>(p, stream);
  return e4m3 ? launch<128, true>(p, stream) : launch<128, false>(p, stream);
}

}  // namespace attn
