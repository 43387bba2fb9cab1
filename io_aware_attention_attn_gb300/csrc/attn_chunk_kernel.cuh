// attn_chunk_kernel.cuh -- attention of several query rows a K/V head over a paged cache, head dim 64 or 128,
// bf16 or E4M3 pages: new tokens of a request behind its older rows, or the requests that share a prefix.
//
// For a unit -- a request's K/V head (or group of its query heads) and a run of its new tokens --
// the rows of the products are (token, query head), so that the query heads that share a K/V head share its
// tiles in one product:  S = scale Q K^T,  O = softmax(S) V  over the request's pages, causal from the end
// (token i of n sees keys 0 .. L - n + i) or over all of them.
//
// Products and tensor memory are those of the whole-sequence forward (attn_fwd_2sm_kernel.cuh): a
// cluster of two CTAs takes 256 rows, M = 256 products of cta_group::2, each CTA half of every K and V tile, three
// score buffers beside O (P over S's place), the softmax with a reference maximum that is moved only when a tile's sum
// passes kSumLimit.  What differs:
//   - Roles: a producer and two issuers, eight softmax warps (32 rows and 64 of a tile's 128 keys each: two warps share a
//     row, its reference and its sum, and meet when one of them needs the reference moved), four that store a unit's
//     O while the next one's tiles run, and over E4M3 pages four that turn V.  Registers go to the softmax (setmaxnreg).
//     With one softmax warp a row, which stored O too, 2048 tokens behind 14336 took 375 us, now 310 (events).
//   - The producer walks the units and tells the others what comes next through a ring in shared memory.
//   - K and V come page by page: a tile is up to 8 + 8 boxes a CTA (one each from pages of 64 rows up), a
//     lane each; a part of a tile past the request's rows is asked for outside the map, which gives
//     zeros without reading.
//   - Work is cut by places, not units (attn_chunk_split.h): a cluster takes equal shares of the line of all
//     key tiles, so few long rows and many short ones both fill the GPU.  A unit inside one share is finished here; the
//     parts of one that spans several go to the workspace, fp32, and chunk_join_kernel merges them.
//   - A tile of 256 x 128 takes the pair about 0.75 us (bf16) where its products alone would take 0.5: the chain scores ->
//     softmax -> P V over three buffers bounds it.  E4M3: 1.1 us, for the instructions of softmax and conversion, which
//     together pass what a sub-partition keeps of them: code written out more often ran slower throughout.
//   - E4M3 pages.  Scores: K's codes go to the product as they are (kind::f8f6f4); a query row becomes two
//     E4M3 pieces, x = hi + lo, after scaling by a power of two (8 significant bits, as bf16 has; what
//     is smaller than 2^-9 of a row's largest element loses bits, 2^-17 of that element at most), for the
//     time of one bf16 product.  A key's K scale multiplies its scores, which are below 2^24 before (d 2^8 448): scales of up to
//     2^100 keep them finite before the row's factor does.  Values: four warps turn V's codes into bf16
//     (exact), and a key's V scale multiplies its P before that is rounded to bf16, whose range holds any product
//     of a P below 2^16 and a scale below 2^100.
//
// P is rounded to bf16 (2^-8 of itself at most) for the product, as in the other forwards; sums of P are of the unrounded ones, in
// fp32, and so are partial results.
#pragma once

#include <cmath>

#include "attn_chunk.h"
#include "attn_gen.cuh"
#include "attn_gen.h"
#include "attn_params.h"
#include "sm103_ptx.cuh"

namespace attn {
namespace chunk {

constexpr int kStartsBarrier = 5;  // (1 to 4: the two warps of a row)
enum : int { kRoleProducer = 9, kRoleIssuer = 10, kRoleSoftmax = 11, kRoleConvert = 12, kRoleStore = 13 };

__device__ __forceinline__ float u2f(uint32_t x) { return __uint_as_float(x); }
__device__ __forceinline__ uint32_t f2u(float x) { return __float_as_uint(x); }

// A bounded wait as mbar_wait_warp, in few instructions: it is written out some forty times, and what the warps of a
// sub-partition run in turn should fit its instruction cache.  What gave up is kept in the CTA's abort word, which
// goes to the status word at the kernel's end.
__device__ __forceinline__ bool wait_warp(uint32_t bar, uint32_t parity, volatile int* abort, int role, int site) {
  if (__all_sync(0xffffffffu, mbar_try_wait(bar, parity))) return true;
  const unsigned long long t0 = global_timer_ns();
  bool stop;
  do {
    if (__all_sync(0xffffffffu, mbar_try_wait(bar, parity))) return true;
    stop = global_timer_ns() - t0 > kWaitLimitNs;
    if (stop && *abort == 0) *abort = kStatusTimeout | (role << 8) | (site << 16);
    stop = *abort != 0;
  } while (!__any_sync(0xffffffffu, stop));
  return false;
}

// The registers of a warp's threads from here on (all four warps of a group together).
// Issue + 2 softmax + store (+ convert): no more than the block was launched with, 4 x 128 (E4M3: 5 x 96).
template <bool E4M3>
struct ChunkRegs {
  static constexpr int kIssue = E4M3 ? 64 : 80, kSoftmax = E4M3 ? 152 : 160, kStore = E4M3 ? 64 : 112, kConvert = 48;
  static_assert(kIssue + 2 * kSoftmax + kStore + (E4M3 ? kConvert : 0) == (E4M3 ? 5 * 96 : 4 * 128), "registers");
};
template <int N>
__device__ __forceinline__ void regs_release() {
  asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N));
}
template <int N>
__device__ __forceinline__ void regs_take() {
  asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N));
}

// 4-D load whose completion is counted on a barrier that may sit in the peer CTA.
__device__ __forceinline__ void tma_load_4d_pair(uint32_t dst, const void* tmap, uint32_t bar_cluster, int x,
                                                 int y, int z, int w, uint64_t policy) {
  asm volatile(
      "cp.async.bulk.tensor.4d.cta_group::2.shared::cluster.global.tile"
      ".mbarrier::complete_tx::bytes.L2::cache_hint [%0], [%1, {%3, %4, %5, %6}], [%2], %7;" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(tmap)), "r"(bar_cluster), "r"(x), "r"(y), "r"(z), "r"(w), "l"(policy)
      : "memory");
}
__device__ __forceinline__ void mma_f8_ss_pair(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc,
                                               uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::2.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
      "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate)
      : "memory");
}
// K-major operand of 64-byte rows, 64-byte swizzle (4): groups of 8 rows 512 bytes apart.
__device__ __forceinline__ uint64_t sdesc_sw64(uint32_t saddr) {
  return static_cast<uint64_t>((saddr >> 4) & 0x3FFFu) | (static_cast<uint64_t>(512 >> 4) << 32) | (1ull << 46) |
         (4ull << 61);
}

// First token and rows of request s, clamped into the tensors (no new tokens where they are another kernel's).
__device__ __forceinline__ int cu_at(const ChunkParams& p, int s) { return min(max(p.cu[s], 0), p.T); }
__device__ __forceinline__ ChunkReq req_at(const ChunkParams& p, int s, int& tok0) {
  tok0 = cu_at(p, s);
  const int n = max(cu_at(p, s + 1) - tok0, 0);
  return ChunkReq{n * p.group > p.few_rows ? n : 0, min(max(p.seq_lens[s], 0), p.max_pages << p.page_shift)};
}

// Whether every request is the kernel's for few rows, which was launched before this one; a block's threads together, and
// before its wait: that kernel's join lets the next launch start when all before the join is done, so that this
// look at cu is over when the join is, and a call without longer requests ends some 4 us sooner (32 requests of 4 tokens over
// 4096 keys, E4M3: 85 -> 81 us; without the second kernel at all it would be 74).
__device__ __forceinline__ bool all_few(const ChunkParams& p) {
  bool any = false;
  for (int s = threadIdx.x; s < p.B; s += static_cast<int>(blockDim.x))
    any |= max(cu_at(p, s + 1) - cu_at(p, s), 0) * p.group > p.few_rows;
  return !__syncthreads_or(any);
}

// Where a role is: the share's round, and the unit and key tile within the share.
struct Walk {
  int s, u, t, j, left;   // request, K/V head x row group, row tile, key tile, places of the share to come
  ChunkReq r;
  int tok0, nt, n;        // the request's first token and row tiles; the unit's key tiles
};

__device__ __forceinline__ void enter(const ChunkParams& p, Walk& w) {
  w.nt = row_tiles(w.r, p.shape);
  w.n = key_tiles(w.r, p.shape, w.t);
}
__device__ __forceinline__ void next_unit(const ChunkParams& p, Walk& w) {
  w.j = 0;
  if (++w.t >= w.nt) {
    w.t = 0;
    if (++w.u >= p.H_kv * p.n_rg) {
      w.u = 0;
      w.r.n = 0;
      w.r.L = 0;
      #pragma unroll 1
      while (w.r.n == 0 && ++w.s < p.B) w.r = req_at(p, w.s, w.tok0);  // (no new tokens: no units)
      w.nt = row_tiles(w.r, p.shape);
    }
  }
  w.n = key_tiles(w.r, p.shape, w.t);
}
__device__ __forceinline__ Walk walk_from(const ChunkParams& p, const ChunkStart& st) {
  Walk w{st.s, st.u, st.t, st.j, st.left, {st.n, st.L}, st.tok0, 0, 0};
  enter(p, w);
  return w;
}
// Behind tiles [j, end) of the unit: the places they took, and on to the next unit.
__device__ __forceinline__ void advance(const ChunkParams& p, Walk& w, int end) {
  w.left -= places_done(w.j, end, w.n, p.shape.cost);
  if (w.left > 0) next_unit(p, w);
}

// Places of all units, by a block of T threads, and s_pre[i]: those of the requests before i's share of
// ceil(B / T); `wide`: rows of requests with several row tiles.  Where cu falls the requests' tokens are more than T, and their
// places may not fit 32 bits: there are none.  Ends with the block in step.
template <int T>
__device__ uint32_t block_places(const ChunkParams& p, int* s_pre, int* s_warp, float& wide) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, per = p.H_kv * p.n_rg;
  const int share = (p.B + T - 1) / T, lo = min(tid * share, p.B), hi = min(lo + share, p.B);
  int sum = 0;
  float rows = 0.f;
  bool bad = false, falls = false;
  #pragma unroll 1
  for (int s = lo; s < hi; ++s) {
    int tok0;
    const ChunkReq r = req_at(p, s, tok0);
    sum += unit_row_places(r, p.shape);
    if (row_tiles(r, p.shape) > 1) rows += static_cast<float>(r.L);
    const int x = p.cu[s], y = p.cu[s + 1];
    falls |= y < x;
    bad |= y < x || (s == 0 && x != 0) || y > p.T;
  }
  if (bad && blockIdx.x == 0) atomicCAS(p.status, 0, kStatusBadSeqlens);
  int scan = sum;
  #pragma unroll
  for (int off = 1; off < 32; off <<= 1) {
    const int up = __shfl_up_sync(0xffffffffu, scan, off);
    if (lane >= off) scan += up;
  }
  #pragma unroll
  for (int off = 16; off > 0; off >>= 1) rows += __shfl_xor_sync(0xffffffffu, rows, off);
  if (lane == 31) {
    s_warp[2 * warp] = scan;
    s_warp[2 * warp + 1] = __float_as_int(rows);
  }
  falls = __syncthreads_or(falls);
  int before = scan - sum, total = 0;
  wide = 0.f;
  #pragma unroll
  for (int i = 0; i < T / 32; ++i) {
    if (i < warp) before += s_warp[2 * i];
    total += s_warp[2 * i];
    wide += __int_as_float(s_warp[2 * i + 1]);
  }
  s_pre[tid] = before * per;
  __syncthreads();
  return falls ? 0u : static_cast<uint32_t>(total) * per;
}

// The unit at place `at` (a warp's lanes together; w.j past its tiles means in the places after them), if it is of one of the 32
// requests from s0 on, before which there are `before` places: lane i has request s0 + i, its places over all heads and
// `scan`, their sum up to there.  Returns the unit's first place, or -1.
__device__ int find_among(const ChunkParams& p, int at, int before, int s0, const ChunkReq& r, int tok0, int places,
                          int scan, Walk& w) {
  const int lane = threadIdx.x & 31;
  const uint32_t past = __ballot_sync(0xffffffffu, before + scan > at);
  if (!past) return -1;
  const int src = __ffs(past) - 1;
  before += __shfl_sync(0xffffffffu, scan - places, src);
  w.s = s0 + src;
  w.r.n = __shfl_sync(0xffffffffu, r.n, src);
  w.r.L = __shfl_sync(0xffffffffu, r.L, src);
  w.tok0 = __shfl_sync(0xffffffffu, tok0, src);
  const int row = __shfl_sync(0xffffffffu, places, src) / (p.H_kv * p.n_rg);
  w.nt = row_tiles(w.r, p.shape);
  w.u = (at - before) / row;
  const int in = at - before - w.u * row;
  int lo = 0, len = w.nt;  // the row tile is among lo .. lo + len - 1
  #pragma unroll 1
  while (len > 1) {
    const int step = (len + 31) >> 5, t = lo + step * lane;
    const bool le = step * lane < len && places_before(w.r, p.shape, t) <= in;
    const int c = __popc(__ballot_sync(0xffffffffu, le)) - 1;
    const int end = lo + len;
    lo += step * c;
    len = min(step, end - lo);
  }
  w.t = lo;
  w.j = in - places_before(w.r, p.shape, lo);
  w.n = key_tiles(w.r, p.shape, lo);
  return at - w.j;
}
__device__ __forceinline__ int scan_lanes(int x) {
  #pragma unroll
  for (int off = 1; off < 32; off <<= 1) {
    const int up = __shfl_up_sync(0xffffffffu, x, off);
    if ((threadIdx.x & 31) >= off) x += up;
  }
  return x;
}
// The same among all requests, from the sums of block_places.
template <int T>
__device__ int find(const ChunkParams& p, const int* s_pre, int at, Walk& w) {
  const int lane = threadIdx.x & 31, per = p.H_kv * p.n_rg;
  int k = 0;
  #pragma unroll
  for (int i = 0; i < T; i += 32) k += __popc(__ballot_sync(0xffffffffu, s_pre[i + lane] <= at));
  --k;
  int before = s_pre[k];
  #pragma unroll 1
  for (int s0 = k * ((p.B + T - 1) / T); s0 < p.B; s0 += 32) {
    const int s = s0 + lane;
    int tok0 = 0;
    ChunkReq r{0, 0};
    if (s < p.B) r = req_at(p, s, tok0);
    const int places = s < p.B ? unit_row_places(r, p.shape) * per : 0;
    const int scan = scan_lanes(places);
    const int unit0 = find_among(p, at, before, s0, r, tok0, places, scan, w);
    if (unit0 >= 0) return unit0;
    before += __shfl_sync(0xffffffffu, scan, 31);
  }
  w = Walk{p.B, 0, 0, 0, 0, {0, 0}, 0, 0, 1};  // (not reached: at is below the number of places)
  return at;
}

// Two E4M3 codes, in bytes 1 and 3 of y, to bf16, exactly but for NaN: exponent and fraction moved to bf16's places
// are the value times 2^-120 (a code below the normal range becomes a bf16 below its own), and a product with 2^120
// puts that right.  (The conversion instructions share a pipe of 16 a clock with exp2, which the softmax fills.)
__device__ __forceinline__ uint32_t codes_to_bf16x2(uint32_t y) {
  const uint32_t x = ((y >> 4) & 0x07f007f0u) | (y & 0x80008000u);
  uint32_t r;
  asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(x), "r"(0x7b807b80u));
  return r;
}
// Bits 7 of the bytes that hold a code of NaN.
__device__ __forceinline__ uint32_t nan_codes(uint32_t v) { return ((v & 0x7f7f7f7fu) + 0x01010101u) & 0x80808080u; }
// value of the E4M3 code nearest to x, two at a time
__device__ __forceinline__ void e4m3x2_values(uint16_t codes, float& lo, float& hi) {
  const uint32_t h = e4m3x2_to_f16x2(codes);
  asm("{\n\t.reg .b16 a, b;\n\tmov.b32 {a, b}, %2;\n\tcvt.f32.f16 %0, a;\n\tcvt.f32.f16 %1, b;\n\t}"
      : "=f"(lo), "=f"(hi)
      : "r"(h));
}

}  // namespace chunk

template <int D, bool E4M3>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__((ChunkLayout<D, E4M3>::kThreads), 1)
    attn_chunk_kernel(const __grid_constant__ ChunkParams p) {
  using namespace chunk;
  using L = ChunkLayout<D, E4M3>;
  constexpr int SK = L::SK, SV = L::SV, NB = kChunkSBufs, T = L::kThreads;
  // as in the whole-sequence forward: at head dim 64 rank 0 holds V's columns, rank 1's V stages stay zero
  constexpr bool kVBoth = D == 128;
  constexpr uint32_t kColO = 128u * NB;
  constexpr uint16_t kBoth = 0x3;
  constexpr int kSIssuerWarp = 2, kSoftmaxWarp = 4, kStoreWarp = 12, kConvertWarp = 16;

  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw_s = smem_u32(smem_raw);
  const uint32_t sbase = (raw_s + 1023u) & ~1023u;
  uint8_t* smem = smem_raw + (sbase - raw_s);
  uint32_t* misc = reinterpret_cast<uint32_t*>(smem + L::kMisc);
  ChunkStart* starts = reinterpret_cast<ChunkStart*>(smem + L::kStart);
  volatile int* wc = reinterpret_cast<volatile int*>(misc + 1);  // set where a wait gave up
  auto bar = [&](int i) -> uint32_t { return sbase + L::kBar + 8u * static_cast<uint32_t>(i); };
  const uint32_t rank = cluster_ctarank();
  const bool leader = rank == 0;
  const uint32_t lbar0 = mapa_shared(sbase + L::kBar, 0);
  auto lbar = [&](int i) -> uint32_t { return lbar0 + 8u * static_cast<uint32_t>(i); };
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int G = static_cast<int>(gridDim.x) >> 1, c0 = static_cast<int>(blockIdx.x) >> 1;

  if (p.few_rows > 0 && all_few(p)) {
    pdl_launch_dependents();
    pdl_wait();  // the work after this one waits for the kernel before it too
    return;
  }
  if (threadIdx.x == 0) {
    for (int b = 0; b < 2; ++b) {
      mbar_init(bar(L::bQF + b), E4M3 ? 2 * 4 : 1);
      mbar_init(bar(L::bQE + b), 1);
      mbar_init(bar(L::bDR + b), 1);
    }
    for (int s = 0; s < SK; ++s) {
      mbar_init(bar(L::bKF + s), 1);
      mbar_init(bar(L::bKE + s), 1);
    }
    for (int s = 0; s < SV; ++s) {
      mbar_init(bar(L::bVF + s), E4M3 ? (kVBoth ? 2 * 4 : 4) : 1);
      mbar_init(bar(L::bVE + s), 1);
    }
    for (int b = 0; b < NB; ++b) {
      mbar_init(bar(L::bSF + b), 1);
      mbar_init(bar(L::bPF + b), 2 * 8);  // one arrival a softmax warp of both CTAs
      mbar_init(bar(L::bPV + b), 1);
    }
    for (int i = 0; i < kChunkUnits; ++i) mbar_init(bar(L::bUF + i), 1);
    mbar_init(bar(L::bOD), 1);
    mbar_init(bar(L::bOE), 2 * 4);
    for (int i = 0; i < kChunkStats; ++i) mbar_init(bar(L::bEL + i), 8);
    mbar_init(bar(L::bLF), 1);
    mbar_init(bar(L::bLE), 4);
    for (int s = 0; s < kChunkRawV; ++s) {
      mbar_init(bar(L::bRF + s), 1);
      mbar_init(bar(L::bRE + s), 4);
    }
    for (int s = 0; s < kChunkScales; ++s) {
      mbar_init(bar(L::bCF + s), 32);
      mbar_init(bar(L::bCE + s), 8);
    }
    fence_barrier_init();
    misc[1] = 0;
    tma_prefetch_desc(&p.tm_q);
    tma_prefetch_desc(&p.tm_k);
    tma_prefetch_desc(&p.tm_v);
  }
  if (!kVBoth && rank == 1) {
    for (int i = threadIdx.x; i < SV * L::kVBytes / 16; i += blockDim.x)
      st_shared_v4(sbase + L::kV + i * 16, 0u, 0u, 0u, 0u);
    fence_proxy_async_smem();
  }
  if (warp == 1) {
    tmem_alloc_pair(sbase + L::kMisc, 512);
    tmem_relinquish_pair();
  }
  tc_fence_before();
  cluster_sync_all();  // barriers initialised and tensor memory allocated in both CTAs
  tc_fence_after();
  const uint32_t tmem = misc[0];
  pdl_wait();
  pdl_launch_dependents();
  // The shares of this cluster, one a round, and for the join the unit that each begins inside: by a warp each, from the
  // lengths in its lanes where that is enough (2.7 us less for the block's sums and barriers to the first copy), else from
  // sums of the whole block.  The other warps wait for the producer, warp 0, to tell them what comes.
  int rounds = 0;
  Walk w0{};  // the first share's beginning
  {
    const bool few = p.B <= 32;
    int* s_pre = reinterpret_cast<int*>(smem + L::kOut);
    float wide = 0.f;
    uint32_t total = 0;
    ChunkReq mine{0, 0};
    int tok0 = 0, places = 0, scan = 0;
    if (!few) {
      total = block_places<T>(p, s_pre, s_pre + T, wide);
    } else if (warp < kChunkRounds) {
      bool bad = false, falls = false;
      if (lane < p.B) {
        mine = req_at(p, lane, tok0);
        const int x = p.cu[lane], y = p.cu[lane + 1];
        falls = y < x;
        bad = y < x || (lane == 0 && x != 0) || y > p.T;
        places = unit_row_places(mine, p.shape) * (p.H_kv * p.n_rg);
        if (row_tiles(mine, p.shape) > 1) wide = static_cast<float>(mine.L);
      }
      if (bad && blockIdx.x == 0) atomicCAS(p.status, 0, kStatusBadSeqlens);
      scan = scan_lanes(places);
      total = static_cast<uint32_t>(__shfl_sync(0xffffffffu, scan, 31));
      if (__any_sync(0xffffffffu, falls)) total = 0;  // (as block_places)
      #pragma unroll
      for (int off = 16; off > 0; off >>= 1) wide += __shfl_xor_sync(0xffffffffu, wide, off);
    }
    if (warp < p.max_rounds) {
      const int most = chunk_rounds(total, G, wide * static_cast<float>(p.H_kv * D * (E4M3 ? 2 : 4)), p.max_rounds);
      const int n_shares = total == 0 ? 0 : chunk_shares(total, G, most);
      rounds = (n_shares + G - 1) / G;
      if (blockIdx.x == 0 && threadIdx.x == 0) {
        p.head[0] = static_cast<int>(total);
        p.head[1] = n_shares;
      }
      const int share = warp * G + c0;
      Walk w{};
      if (share < n_shares) {
        const Shares shares(total, static_cast<uint32_t>(n_shares));
        const int at = shares.start(share), next = shares.start(share + 1);
        int left = next - at;
        const int unit0 = few ? find_among(p, at, 0, 0, mine, tok0, places, scan, w) : find<T>(p, s_pre, at, w);
        ChunkDesc d{0, -1, 0, 0, 0, 0};
        // inside a unit of an earlier share, whose last tile is in this one
        if (w.j > 0 && w.j < w.n && unit0 + w.n <= next)
          d = ChunkDesc{unit0, w.n, w.u, w.tok0 + w.t * p.shape.tokens, min(w.r.n - w.t * p.shape.tokens, p.shape.tokens), 0};
        if (leader && lane == 0) p.desc[share] = d;
        if (w.j >= w.n) {  // begins behind a unit's last tile
          left -= unit0 + w.n + p.shape.cost - at;
          if (left > 0) next_unit(p, w);
        }
        w.left = left;
      }
      if (warp == 0) w0 = w;
      else if (lane == 0) starts[warp] = ChunkStart{w.s, w.u, w.t, w.j, w.left, w.r.n, w.tok0, w.r.L};
    }
    if (!few) __syncthreads();  // O goes out through where s_pre is, which the searching warps have read
  }
  const ChunkUnit* units = reinterpret_cast<const ChunkUnit*>(smem + L::kUnits);
  // The uq-th unit (or part): false when there is none, or a wait gave up.
  auto unit_at = [&](int uq, ChunkUnit& w, bool& ok, int role) {
    const int i = uq % kChunkUnits;
    ok = wait_warp(bar(L::bUF + i), static_cast<uint32_t>(uq / kChunkUnits) & 1u, wc, role, 15);
    if (!ok) return false;
    w = units[i];
    return w.j >= 0;
  };

  // Registers of the warps that issue, store and convert go to those of the softmax (with the same for all the
  // E4M3 kernel spilled and took 2.1 us a tile).
  // Counters kept by every role: uq = units (or parts) done so far, g = key tiles done so far.
  if (warp < kSoftmaxWarp) {
    regs_release<ChunkRegs<E4M3>::kIssue>();
    if (warp > 0 && warp < kChunkRounds && rounds > 1)
      asm volatile("bar.arrive %0, %1;" ::"r"(kStartsBarrier), "r"(kChunkRounds * 32) : "memory");
    if (warp == 0) {
      // ===================================================================== producer
      const uint64_t keep = l2_policy_evict_last(), once = l2_policy_evict_first();
      const int box = 31 - __clz(p.box_rows);
      const int page_rows = 1 << p.page_shift;
      const int pages_tile = max(kChunkTile >> p.page_shift, 1);
      // this lane's box of K and of V: its rows within the tile and, for K, its block of columns
      constexpr int kKBlks = E4M3 ? 1 : D / 64;
      const int k_part = lane / kKBlks, k_blk = lane % kKBlks;
      const bool k_on = (k_part << box) < 64, v_on = (lane << box) < kChunkTile;
      const int k_row = 64 * static_cast<int>(rank) + (k_part << box), v_row = lane << box;
      bool ok = true;
      int g = 0, uq = 0;
      int entries = 0, entry_base = 0, entry_s = -1;  // this lane's entry of the 32 looked up last
      for (int r = 0; ok && r < rounds; ++r) {
        if (r == 1) named_barrier_sync(kStartsBarrier, kChunkRounds * 32);  // the later rounds' starts are there
        Walk w = r == 0 ? w0 : walk_from(p, starts[r]);
        bool first = true;  // of the share's units: its part, if it is one, has the share's first place in the workspace
        while (ok && w.left > 0) {
          const int j_end = min(w.n, w.j + w.left);
          const int z = p.n_rg == 1 ? w.u : w.u / p.n_rg;
          const uint64_t policy = w.nt > 1 || p.n_rg > 1 ? keep : once;
          const int tok_t = w.t * p.shape.tokens;
          {  // query rows of this CTA
            const int qb = uq & 1;
            const uint32_t dst = E4M3 ? sbase + L::kLand : sbase + L::kQ + qb * L::kQBytes;
            const int bytes = p.rg_rows * p.cta_tokens * 128 * (D / 64);
            if (E4M3) {
              if (uq >= 1) ok = wait_warp(bar(L::bLE), static_cast<uint32_t>(uq - 1) & 1u, wc, kRoleProducer, 1);
            } else {
              if (uq >= 2)
                ok = wait_warp(bar(L::bQE + qb), static_cast<uint32_t>((uq - 2) >> 1) & 1u, wc, kRoleProducer, 2);
            }
            if (!ok) break;
            if (lane == 0) {
              // (those who read entry uq - kChunkUnits are through with it: nobody is that many units behind)
              *reinterpret_cast<ChunkUnit*>(smem + L::kUnits + (uq % kChunkUnits) * sizeof(ChunkUnit)) =
                  ChunkUnit{w.j, j_end, w.n, w.r.L, z, (w.u - z * p.n_rg) * p.rg_rows, w.tok0 + tok_t,
                            min(w.r.n - tok_t, p.shape.tokens), w.r.L - w.r.n + tok_t, 2 * (r * G + c0) + (first ? 0 : 1)};
              mbar_arrive(bar(L::bUF + uq % kChunkUnits));
              if (E4M3) mbar_arrive_expect_tx(bar(L::bLF), bytes);
              else if (leader) mbar_arrive_expect_tx(bar(L::bQF + qb), 2 * bytes);
              const int head = z * p.group + (w.u - z * p.n_rg) * p.rg_rows;
              const int tok = w.tok0 + tok_t + static_cast<int>(rank) * p.cta_tokens;
              #pragma unroll
              for (int c = 0; c < D / 64; ++c) {
                if (E4M3)
                  tma_load_3d_hint(dst + c * 16384, &p.tm_q, bar(L::bLF), c * 64, head, tok, once);
                else
                  tma_load_3d_pair(dst + c * 16384, &p.tm_q, lbar(L::bQF + qb), c * 64, head, tok, once);
              }
            }
            __syncwarp();
          }
          for (int j = w.j; j < j_end; ++j, ++g) {
            const int key0 = j * kChunkTile;
            const int page0 = key0 >> p.page_shift;
            if (entry_s != w.s || page0 < entry_base || page0 + pages_tile > entry_base + 32) {
              entry_s = w.s;
              entry_base = page0;
              const int e = page0 + lane, have = (w.r.L + page_rows - 1) >> p.page_shift;
              entries = -1;  // a page of zeros
              if (e < have) {
                entries = p.table[static_cast<size_t>(w.s) * p.max_pages + e];
                if (static_cast<unsigned>(entries) >= static_cast<unsigned>(p.num_pages)) {
                  atomicCAS(p.status, 0, kStatusBadPage);
                  entries = -1;
                }
              }
            }
            const int k_pg = __shfl_sync(0xffffffffu, entries, (((key0 + k_row) >> p.page_shift) - entry_base) & 31);
            const int v_pg = __shfl_sync(0xffffffffu, entries, (((key0 + v_row) >> p.page_shift) - entry_base) & 31);
            const int sk = g % SK;
            if (g >= SK && !(ok = wait_warp(bar(L::bKE + sk), (static_cast<uint32_t>(g / SK) & 1u) ^ 1u, wc,
                                                 kRoleProducer, 3)))
              break;
            if (leader && lane == 0) mbar_arrive_expect_tx(bar(L::bKF + sk), 2 * L::kKBytes);
            __syncwarp();
            if (k_on)
              tma_load_4d_pair(sbase + L::kK + sk * L::kKBytes + k_blk * 8192 +
                                   (k_part << box) * (E4M3 ? D : 128),
                               &p.tm_k, lbar(L::bKF + sk), k_blk * 64, (key0 + k_row) & (page_rows - 1), z,
                               k_pg >= 0 ? k_pg : p.num_pages, policy);
            if (E4M3) {
              // scales of keys 4 lane .. 4 lane + 3; past the request's rows: zeros
              const int sc = g % kChunkScales;
              if (g >= kChunkScales &&
                  !(ok = wait_warp(bar(L::bCE + sc), (static_cast<uint32_t>(g / kChunkScales) & 1u) ^ 1u, wc,
                                        kRoleProducer, 4)))
                break;
              const int key = key0 + 4 * lane;
              const int pg = __shfl_sync(0xffffffffu, entries, ((key >> p.page_shift) - entry_base) & 31);
              const uint32_t dst = sbase + L::kScale + sc * 1024 + lane * 16;
              const int64_t at = ((static_cast<int64_t>(pg) * p.H_kv + z) << p.page_shift) + (key & (page_rows - 1));
              const int live = pg >= 0 ? w.r.L - key : 0;
              if (live >= 4) {
                copy16(dst, p.ks + at);
                copy16(dst + 512, p.vs + at);
                copy_arrive(bar(L::bCF + sc));
              } else {
                float x[8];
                #pragma unroll
                for (int i = 0; i < 4; ++i) {
                  x[i] = i < live ? p.ks[at + i] : 0.f;
                  x[4 + i] = i < live ? p.vs[at + i] : 0.f;
                }
                st_shared_v4(dst, f2u(x[0]), f2u(x[1]), f2u(x[2]), f2u(x[3]));
                st_shared_v4(dst + 512, f2u(x[4]), f2u(x[5]), f2u(x[6]), f2u(x[7]));
                mbar_arrive(bar(L::bCF + sc));
              }
              __syncwarp();
            }
            if (!kVBoth && !leader) continue;
            if (E4M3) {
              const int sv = g % kChunkRawV;
              if (g >= kChunkRawV &&
                  !(ok = wait_warp(bar(L::bRE + sv), (static_cast<uint32_t>(g / kChunkRawV) & 1u) ^ 1u, wc,
                                        kRoleProducer, 5)))
                break;
              if (lane == 0) mbar_arrive_expect_tx(bar(L::bRF + sv), 8192);
              __syncwarp();
              if (v_on)
                tma_load_4d_hint(sbase + L::kVRaw + sv * 8192 + v_row * 64, &p.tm_v, bar(L::bRF + sv),
                                 64 * static_cast<int>(rank), (key0 + v_row) & (page_rows - 1), z,
                                 v_pg >= 0 ? v_pg : p.num_pages, policy);
            } else {
              const int sv = g % SV;
              if (g >= SV && !(ok = wait_warp(bar(L::bVE + sv), (static_cast<uint32_t>(g / SV) & 1u) ^ 1u, wc,
                                                   kRoleProducer, 6)))
                break;
              if (leader && lane == 0) mbar_arrive_expect_tx(bar(L::bVF + sv), (kVBoth ? 2 : 1) * L::kVBytes);
              __syncwarp();
              if (v_on)
                tma_load_4d_pair(sbase + L::kV + sv * L::kVBytes + v_row * 128, &p.tm_v, lbar(L::bVF + sv),
                                 64 * static_cast<int>(rank), (key0 + v_row) & (page_rows - 1), z,
                                 v_pg >= 0 ? v_pg : p.num_pages, policy);
            }
          }
          ++uq;
          first = false;
          if (ok) advance(p, w, j_end);
        }
      }
      if (ok && lane == 0) {
        *reinterpret_cast<int*>(smem + L::kUnits + (uq % kChunkUnits) * sizeof(ChunkUnit)) = -1;
        mbar_arrive(bar(L::bUF + uq % kChunkUnits));
      }
      if (!ok) {  // copies in flight land within microseconds: before the cluster exits
        if (E4M3) copy_wait<0>();
        const unsigned long long t0 = global_timer_ns();
        while (global_timer_ns() - t0 < 100000ull) {
        }
      }
    } else if (warp == 1 || warp == kSIssuerWarp) {
      // ========================================= MMA issuers (rank 0): P V on warp 1, S on another
      if (leader) {
        bool ok = true;
        int g = 0, uq = 0;
        if (warp == kSIssuerWarp) {
          constexpr uint32_t kIdS = E4M3 ? idesc_e4m3_f32(2 * kChunkRows, kChunkTile)
                                         : idesc_bf16_f32(2 * kChunkRows, kChunkTile, false, false);
          for (ChunkUnit w; unit_at(uq, w, ok, kRoleIssuer);) {
            const int j_end = w.j_end;
            const int qb = uq & 1;
            if (!(ok = wait_warp(bar(L::bQF + qb), static_cast<uint32_t>(uq >> 1) & 1u, wc, kRoleIssuer, 1)))
              break;
            const uint32_t q_at = sbase + L::kQ + qb * L::kQBytes;
            for (int j = w.j; j < j_end; ++j, ++g) {
              if (!(ok = wait_warp(bar(L::bKF + g % SK), static_cast<uint32_t>(g / SK) & 1u, wc, kRoleIssuer, 3)))
                break;
              if (g >= NB && !(ok = wait_warp(bar(L::bPV + g % NB), static_cast<uint32_t>((g - NB) / NB) & 1u,
                                                   wc, kRoleIssuer, 2)))
                break;
              tc_fence_after();
              if (lane == 0) {
                const uint32_t k_at = sbase + L::kK + (g % SK) * L::kKBytes;
                const uint32_t d = tmem + 128u * static_cast<uint32_t>(g % NB);
                if constexpr (E4M3) {
                  // (hi + lo) K^T: both pieces on one accumulator
                  const uint64_t a = D == 128 ? sdesc_sw128(q_at, 16, 1024) : sdesc_sw64(q_at);
                  const uint64_t b = D == 128 ? sdesc_sw128(k_at, 16, 1024) : sdesc_sw64(k_at);
                  #pragma unroll
                  for (int piece = 0; piece < 2; ++piece)
                    #pragma unroll
                    for (int k = 0; k < D / 32; ++k)
                      mma_f8_ss_pair(d, a + ((piece * kChunkRows * D + k * 32) >> 4), b + ((k * 32) >> 4), kIdS,
                                     piece + k > 0 ? 1u : 0u);
                } else {
                  const uint64_t a = sdesc_sw128(q_at, 16, 1024), b = sdesc_sw128(k_at, 16, 1024);
                  #pragma unroll
                  for (int k = 0; k < D / 16; ++k)
                    mma_bf16_ss_pair(d, a + (((k >> 2) * 16384 + (k & 3) * 32) >> 4),
                                     b + (((k >> 2) * 8192 + (k & 3) * 32) >> 4), kIdS, k > 0 ? 1u : 0u);
                }
                mma_commit_pair(bar(L::bSF + g % NB), kBoth);
                mma_commit_pair(bar(L::bKE + g % SK), kBoth);
                if (j == j_end - 1) mma_commit_pair(bar(L::bQE + qb), kBoth);
              }
              __syncwarp();
            }
            if (!ok) break;
            ++uq;
          }
          if (!ok) {  // unwinding: wait for every MMA this thread issued
            if (lane == 0) mma_commit_pair(bar(L::bDR), 0x1);
            __syncwarp();
            mbar_wait_drain(bar(L::bDR), 0);
          }
        } else {
          constexpr uint32_t kIdO = idesc_bf16_f32(2 * kChunkRows, k2smPVN, false, true);  // P, V MN
          const uint64_t desc_v = sdesc_sw128(sbase + L::kV, 16384, 1024);
          for (ChunkUnit w; unit_at(uq, w, ok, kRoleIssuer);) {
            const int j_end = w.j_end;
            for (int j = w.j; j < j_end; ++j, ++g) {
              const int b = g % NB, sv = g % SV;
              if (!(ok = wait_warp(bar(L::bVF + sv), static_cast<uint32_t>(g / SV) & 1u, wc, kRoleIssuer, 4)))
                break;
                // the first product of a unit overwrites O: the previous unit's epilogue has read it
              if (j == w.j && uq > 0 &&
                  !(ok = wait_warp(bar(L::bOE), static_cast<uint32_t>(uq - 1) & 1u, wc, kRoleIssuer, 6)))
                break;
              if constexpr (!E4M3) {
                // rows of the last page past the request's end may hold anything: zeroed in both CTAs' halves,
                // so that P = 0 there meets no value that is not finite
                const int valid = w.L - j * kChunkTile;
                if (valid < kChunkTile) {
                  const uint32_t vbase = sbase + L::kV + sv * L::kVBytes;
                  const uint32_t vpeer = mapa_shared(vbase, 1);
                  for (int i = max(valid, 0) * 8 + lane; i < kChunkTile * 8; i += 32) {
                    st_shared_v4(vbase + i * 16, 0u, 0u, 0u, 0u);
                    if (kVBoth) st_shared_cluster_v4(vpeer + i * 16, 0u, 0u, 0u, 0u);
                  }
                  fence_proxy_async_cluster();
                }
                __syncwarp();
              }
              if (!(ok = wait_warp(bar(L::bPF + b), static_cast<uint32_t>(g / NB) & 1u, wc, kRoleIssuer, 5)))
                break;
              tc_fence_after();
              if (lane == 0) {
                const uint64_t bv = desc_v + static_cast<uint64_t>(sv * (L::kVBytes >> 4));
                const uint32_t a = tmem + 128u * static_cast<uint32_t>(b);
                #pragma unroll
                for (int k = 0; k < kChunkTile / 16; ++k)  // P of keys 64 on begins at column 64
                  mma_bf16_ts_pair(tmem + kColO, a + k * 8 + (k >> 2) * 32, bv + static_cast<uint64_t>(k * (2048 >> 4)),
                                   kIdO, (j > w.j || k > 0) ? 1u : 0u);
                mma_commit_pair(bar(L::bPV + b), kBoth);
                mma_commit_pair(bar(L::bVE + sv), kBoth);
                if (j == j_end - 1) mma_commit_pair(bar(L::bOD), kBoth);
              }
              __syncwarp();
            }
            if (!ok) break;
            ++uq;
          }
          if (!ok) {
            if (lane == 0) mma_commit_pair(bar(L::bDR + 1), 0x1);
            __syncwarp();
            mbar_wait_drain(bar(L::bDR + 1), 0);
          }
        }
      }
    }
  } else if (warp < kStoreWarp) {
    // ===================================================================== softmax
    regs_take<ChunkRegs<E4M3>::kSoftmax>();
    const int half = (warp - kSoftmaxWarp) >> 2;  // keys 64 half .. + 63 of a tile; of O, half of the columns
    const int quarter = warp & 3;       // tensor-memory lanes this warp may access: 32 quarter .. + 31
    const int row = quarter * 32 + lane;
    const uint32_t t_lane = tmem + (static_cast<uint32_t>(quarter * 32) << 16);
    const uint32_t o_col = t_lane + kColO + (D / 2) * half;
    // this row's token (within the unit) and query head (within the row group)
    const int my_tok = row / p.rg_rows, my_head = row - my_tok * p.rg_rows;
    const int unit_tok = static_cast<int>(rank) * p.cta_tokens + my_tok;
    // A value of this row with the warp that has the row's other keys (both together).
    float* mine = reinterpret_cast<float*>(smem + L::kPair) + (quarter * 2 + half) * 32 + lane;
    const float* theirs = reinterpret_cast<const float*>(smem + L::kPair) + (quarter * 2 + (half ^ 1)) * 32 + lane;
    auto exchange = [&](float x) {
      *mine = x;
      named_barrier_sync(1 + quarter, 64);
      const float y = *theirs;
      named_barrier_sync(1 + quarter, 64);
      return y;
    };
    // The two meet at barriers that have no limit, so neither leaves the other there: one whose wait gave up says so (a value
    // of 2) where they meet next, and both stop.  What that is for this warp: nothing, the other knows (0); as in a first
    // tile, which is the next unit's, or the other's leave (1); as in a later tile (2).
    int meet = 1;
    bool ok = true;
    int g = 0, uq = 0;
    for (ChunkUnit w; unit_at(uq, w, ok, kRoleSoftmax);) {
      const int j_end = w.j_end;
      const bool valid = my_tok < p.cta_tokens && unit_tok < w.n_tok && w.head0 + my_head < p.group;
      const bool any = __any_sync(0xffffffffu, valid);   // a warp without rows only keeps step
      // keys that this row sees, and the fewest that a row of this warp sees (what the lanes without a row compute, of
      // whatever lies in their rows of the products, is not used)
      const int sees = !valid ? 0 : p.shape.causal ? min(w.L, w.pos0 + unit_tok + 1) : w.L;
      const int least = __reduce_min_sync(0xffffffffu, valid ? sees : 0x7fffffff);
      float sl2 = p.scale_log2;
      float m2 = -INFINITY;                // reference maximum of the scaled scores (log2 units)
      float le[4] = {0.f, 0.f, 0.f, 0.f};  // sums of 2^(t - m)
      for (int j = w.j; j < j_end; ++j, ++g) {
        const int b = g % NB;
        if (!(ok = wait_warp(bar(L::bSF + b), static_cast<uint32_t>(g / NB) & 1u, wc, kRoleSoftmax, 1))) {
          meet = any && j > w.j ? 2 : 1;
          break;
        }
        const float* sc = reinterpret_cast<const float*>(smem + L::kScale + (g % kChunkScales) * 1024) + 64 * half;
        if (E4M3) {
          // (the factors of the rows were written before the product that this wait is for could be issued)
          if (j == w.j)
            sl2 = p.scale_log2 * reinterpret_cast<const float*>(smem + L::kRow)[(uq % kChunkRowDepth) * 128 + row];
          if (!(ok = wait_warp(bar(L::bCF + g % kChunkScales), static_cast<uint32_t>(g / kChunkScales) & 1u, wc,
                               kRoleSoftmax, 2))) {
            meet = any && j > w.j ? 2 : 1;
            break;
          }
        }
        tc_fence_after();
        if (any) {
          const uint32_t s_col = t_lane + 128u * static_cast<uint32_t>(b) + 64u * half;
          float s[64];
          {
            uint32_t u[2][32];
            #pragma unroll
            for (int h = 0; h < 2; ++h) tmem_ld32(s_col + 32 * h, u[h]);
            #pragma unroll
            for (int h = 0; h < 2; ++h) {
              float4 k4[8];  // K scales of 32 keys, on their way while the scores are
              if (E4M3) {
                #pragma unroll
                for (int i = 0; i < 8; ++i) k4[i] = *reinterpret_cast<const float4*>(sc + 32 * h + 4 * i);
              }
              tmem_wait_ld_regs(u[h]);
              #pragma unroll
              for (int i = 0; i < 32; ++i) s[32 * h + i] = u2f(u[h][i]);
              if (E4M3) {
                #pragma unroll
                for (int i = 0; i < 8; ++i) {
                  float* x = s + 32 * h + 4 * i;
                  fmul2(x[0], x[1], x[0], x[1], k4[i].x, k4[i].y);
                  fmul2(x[2], x[3], x[2], x[3], k4[i].z, k4[i].w);
                }
              }
            }
          }
          const int key0 = j * kChunkTile + 64 * half;
          if (key0 + 64 > least) {
            const int lim = sees - key0;
            #pragma unroll
            for (int cc = 0; cc < 64; ++cc) s[cc] = (cc < lim) ? s[cc] : -INFINITY;
          }
          // P = 2^(t - m) over the first 32 of the half's columns; ts = its row sums.  Pass 0 takes the current
          // reference, the same for both halves of a row; the row maximum is taken (pass 1) only on the first tile
          // or when a row's sum in one of the halves exceeds kSumLimit.
          float ts[4];
          bool moved = false;
          float alpha = 1.f;
          bool need = j == w.j;
          #pragma unroll 1
          for (int pass = (j == w.j) ? 1 : 0; pass < 2; ++pass) {
            float m_use = m2;
            if (pass == 1) {
              float mx[8];
              #pragma unroll
              for (int k = 0; k < 8; ++k) mx[k] = s[k];
              #pragma unroll
              for (int cc = 8; cc + 16 <= 64; cc += 16)
                #pragma unroll
                for (int k = 0; k < 8; ++k) mx[k] = fmax3(mx[k], s[cc + k], s[cc + 8 + k]);
              #pragma unroll
              for (int k = 0; k < 8; ++k) mx[k] = fmaxf(mx[k], s[64 - 8 + k]);
              const float mt = fmax3(fmax3(mx[0], mx[1], mx[2]), fmax3(mx[3], mx[4], mx[5]),
                                     fmaxf(mx[6], mx[7])) * sl2;
              const float both = fmaxf(mt, exchange(mt));
              const float other = exchange(need ? 1.f : 0.f);
              if (other == 2.f) {
                ok = false;
                break;
              }
              need |= other != 0.f;
              const float m_new = need ? fmaxf(both, m2) : m2;
              moved = (m_new != m2);
              m_use = (m_new == -INFINITY) ? 0.f : m_new;
              alpha = moved ? ex2_approx(m2 - m_use) : 1.f;
              m2 = m_new;
              if (moved) {
                #pragma unroll
                for (int k = 0; k < 4; ++k) le[k] *= alpha;
              }
              tmem_wait_st();  // pass 0's stores land before these overwrite them
            }
            const float neg_m = -m_use;
            #pragma unroll
            for (int k = 0; k < 4; ++k) ts[k] = 0.f;
            #pragma unroll
            for (int h = 0; h < 2; ++h) {
              uint32_t pk[16];
              float4 v4[8];  // V scales of 32 keys
              if (E4M3) {
                #pragma unroll
                for (int i = 0; i < 8; ++i) v4[i] = *reinterpret_cast<const float4*>(sc + 128 + 32 * h + 4 * i);
              }
              #pragma unroll
              for (int i = 0; i < 16; ++i) {
                const int cc = 32 * h + 2 * i;
                float x0, x1;
                ffma2(x0, x1, s[cc], s[cc + 1], sl2, sl2, neg_m, neg_m);
                float p0 = ex2_approx(x0), p1 = ex2_approx(x1);
                fadd2(ts[2 * (i & 1)], ts[2 * (i & 1) + 1], p0, p1);
                if (E4M3) {
                  if (i & 1) fmul2(p0, p1, p0, p1, v4[i / 2].z, v4[i / 2].w);
                  else fmul2(p0, p1, p0, p1, v4[i / 2].x, v4[i / 2].y);
                }
                pk[i] = pack_bf16x2(p0, p1);
              }
              tmem_st16(s_col + 16 * h, pk);
            }
            if (pass == 0) {
              need = sees > 0 && !(((ts[0] + ts[1]) + (ts[2] + ts[3])) <= kSumLimit);  // also inf, NaN
              if (!named_barrier_or(1 + quarter, 64, need)) break;
            }
          }
          if (!ok) {
            meet = 0;
            break;
          }
          #pragma unroll
          for (int k = 0; k < 4; ++k) le[k] += ts[k];
          // O holds P V up to the tile before once that product completes; bring it to the new reference
          if (j > w.j && __any_sync(0xffffffffu, moved)) {
            if (!(ok = wait_warp(bar(L::bPV + (g - 1) % NB), static_cast<uint32_t>((g - 1) / NB) & 1u, wc,
                                 kRoleSoftmax, 3))) {
              meet = j + 1 < j_end ? 2 : 1;
              break;
            }
            tc_fence_after();
            #pragma unroll 1
            for (int cc = 0; cc < D / 64; ++cc) {  // its half of the columns
              uint32_t o[32];
              tmem_ld32(o_col + cc * 32, o);
              tmem_wait_ld_regs(o);
              #pragma unroll
              for (int i = 0; i < 32; ++i) o[i] = f2u(u2f(o[i]) * alpha);
              tmem_st32(o_col + cc * 32, o);
            }
          }
          tmem_wait_st();
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) {
          if (E4M3) mbar_arrive(bar(L::bCE + g % kChunkScales));
          mbar_arrive_cluster(lbar(L::bPF + b));
        }
      }
      if (!ok) break;
      // the row's maximum and sums for the warps that store O
      float* stats = reinterpret_cast<float*>(smem + L::kStats) + (uq % kChunkStats) * 384;
      const float l = (le[0] + le[1]) + (le[2] + le[3]);
      stats[half * 128 + row] = sees > 0 ? l : 0.f;
      if (half == 0) stats[256 + row] = sees > 0 ? m2 : -INFINITY;
      __syncwarp();
      if (lane == 0) mbar_arrive(bar(L::bEL + uq % kChunkStats));
      ++uq;
    }
    if (meet == 2) named_barrier_or(1 + quarter, 64, true);
    #pragma unroll 1
    for (int i = 0; meet > 0 && i < 2; ++i) exchange(2.f);
  } else if (warp < kConvertWarp) {
    // ===================================================================== O out
    // Warps of their own, so that the softmax goes on with the next unit while a unit's last product runs and its
    // rows are stored (with the softmax's warps doing it, a unit cost 2.6 us beside its tiles).
    regs_release<ChunkRegs<E4M3>::kStore>();
    const int quarter = warp & 3, row = quarter * 32 + lane;
    const uint32_t o_col = tmem + (static_cast<uint32_t>(quarter * 32) << 16) + kColO;
    const int my_tok = row / p.rg_rows, my_head = row - my_tok * p.rg_rows;
    const int unit_tok = static_cast<int>(rank) * p.cta_tokens + my_tok;
    const uint32_t area = L::kOut + static_cast<uint32_t>(quarter) * 2048u;  // 32 rows of 32 columns on their way out
    bool ok = true;
    int uq = 0;
    for (ChunkUnit w; unit_at(uq, w, ok, kRoleStore);) {
      const bool valid = my_tok < p.cta_tokens && unit_tok < w.n_tok && w.head0 + my_head < p.group;
      const bool any = __any_sync(0xffffffffu, valid);
      const int sees = !valid ? 0 : p.shape.causal ? min(w.L, w.pos0 + unit_tok + 1) : w.L;
      if (!(ok = wait_warp(bar(L::bEL + uq % kChunkStats), static_cast<uint32_t>(uq / kChunkStats) & 1u, wc, kRoleStore, 1)))
        break;
      const float* stats = reinterpret_cast<const float*>(smem + L::kStats) + (uq % kChunkStats) * 384;
      const float l = stats[row] + stats[128 + row], m2 = stats[256 + row];
      const bool part = w.j > 0 || w.j_end < w.n;
      const int tok = w.tok + unit_tok, head = w.z * p.group + w.head0 + my_head;
      const int64_t at = valid ? head * p.o_head + tok * p.o_token : -1;  // this row's elements
      const int64_t row_at = static_cast<int64_t>(tok) * p.H + head;
      float wt = 1.f, wo = 0.f;  // weights of this row's O and of the same row over other keys
      if (!part) {
        wt = l > 0.f || l != l ? 1.f / l : 0.f;  // a row that sees nothing: zeros
        float lse = l > 0.f || l != l ? (m2 + log2f(l)) * 0.69314718055994530942f : -INFINITY;
        if (p.tail_o && valid) {  // the block merge of the two
          const float tail = p.tail_lse[row_at], most = fmaxf(lse, tail);
          const float a = lse == -INFINITY ? 0.f : ex2_approx((lse - most) * 1.4426950408889634f);
          const float b = tail == -INFINITY ? 0.f : ex2_approx((tail - most) * 1.4426950408889634f);
          const float sum = a + b, inv = sum > 0.f || sum != sum ? 1.f / sum : 0.f;
          wt *= a * inv;
          wo = b * inv;
          lse = sum > 0.f || sum != sum ? most + log2f(sum) * 0.69314718055994530942f : -INFINITY;
        }
        if (valid) p.lse[at / D] = lse;
      } else if (valid) {
        *reinterpret_cast<float2*>(p.part_ml + (static_cast<int64_t>(w.slot) * p.part_rows + rank * kChunkRows + row) * 2) =
            make_float2(m2, l);
      }
      if (!(ok = wait_warp(bar(L::bOD), static_cast<uint32_t>(uq) & 1u, wc, kRoleStore, 2))) break;
      tc_fence_after();
      if (any) {
        #pragma unroll 1
        for (int c = 0; c < D / 32; ++c) {
          uint32_t u[32];
          tmem_ld32(o_col + c * 32, u);
          tmem_wait_ld_regs(u);
          if (c == D / 32 - 1) {  // all of O is read: the next unit's first product may overwrite it
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive_cluster(lbar(L::bOE));
          }
          float o[32];
          #pragma unroll
          for (int i = 0; i < 32; ++i) o[i] = sees <= 0 ? 0.f : u2f(u[i]) * wt;
          if (part) {
            if (valid) {
              // four columns of all rows together: a warp's stores are contiguous
              float4* dst = reinterpret_cast<float4*>(p.part_o + static_cast<int64_t>(w.slot) * p.part_rows * D) +
                            c * 8 * p.part_rows + rank * kChunkRows + row;
              #pragma unroll
              for (int i = 0; i < 8; ++i)
                dst[i * p.part_rows] = make_float4(o[4 * i], o[4 * i + 1], o[4 * i + 2], o[4 * i + 3]);
            }
            continue;
          }
          if (p.tail_o && valid) {
            const float4* src = reinterpret_cast<const float4*>(p.tail_o + row_at * D + c * 32);
            #pragma unroll
            for (int i = 0; i < 8; ++i) {
              const float4 x = src[i];
              o[4 * i] = fmaf(x.x, wo, o[4 * i]);
              o[4 * i + 1] = fmaf(x.y, wo, o[4 * i + 1]);
              o[4 * i + 2] = fmaf(x.z, wo, o[4 * i + 2]);
              o[4 * i + 3] = fmaf(x.w, wo, o[4 * i + 3]);
            }
          }
          // bf16 rows through this warp's area, 16-byte chunks XOR-ed by the row; then a row by four lanes
          #pragma unroll
          for (int i = 0; i < 4; ++i)
            st_shared_v4(sbase + area + lane * 64 + ((i ^ ((lane >> 1) & 3)) << 4), pack_bf16x2(o[8 * i], o[8 * i + 1]),
                         pack_bf16x2(o[8 * i + 2], o[8 * i + 3]), pack_bf16x2(o[8 * i + 4], o[8 * i + 5]),
                         pack_bf16x2(o[8 * i + 6], o[8 * i + 7]));
          __syncwarp();
          #pragma unroll
          for (int r0 = 0; r0 < 32; r0 += 8) {
            const int rr = r0 + (lane >> 2), q = lane & 3;
            const int64_t to = __shfl_sync(0xffffffffu, at, rr);
            if (to >= 0)
              *reinterpret_cast<uint4*>(p.o + to + c * 32 + q * 8) = *reinterpret_cast<const uint4*>(
                  smem + area + rr * 64 + ((q ^ ((rr >> 1) & 3)) << 4));
          }
          __syncwarp();
        }
      } else {
        tc_fence_before();
        if (lane == 0) mbar_arrive_cluster(lbar(L::bOE));
      }
      ++uq;
    }
  } else if constexpr (E4M3) {
    // ===================================================================== converters
    regs_release<ChunkRegs<E4M3>::kConvert>();
    const int tid = (warp - kConvertWarp) * 32 + lane;  // 128 threads
    bool ok = true;
    int g = 0, uq = 0;
    for (ChunkUnit w; unit_at(uq, w, ok, kRoleConvert);) {
      const int j_end = w.j_end;
      {
        // query row tid: scaled by a power of two to a largest element of 2^7 .. 2^8, then hi = its E4M3
        // rounding and lo = that of what is left
        const int qb = uq & 1;
        if (!(ok = wait_warp(bar(L::bLF), static_cast<uint32_t>(uq) & 1u, wc, kRoleConvert, 1))) break;
        if (uq >= 2 && !(ok = wait_warp(bar(L::bQE + qb), static_cast<uint32_t>((uq - 2) >> 1) & 1u, wc,
                                             kRoleConvert, 2)))
          break;
        const uint8_t* land = smem + L::kLand;
        auto chunk_at = [&](int c) {  // 8 elements
          return *reinterpret_cast<const uint4*>(land + (c >> 3) * 16384 + tid * 128 + (((c & 7) ^ (tid & 7)) << 4));
        };
        float amax = 0.f;
        bool bad = false;
        #pragma unroll 1
        for (int c = 0; c < D / 8; ++c) {
          const uint4 x = chunk_at(c);
          const uint32_t v[4] = {x.x, x.y, x.z, x.w};
          #pragma unroll
          for (int i = 0; i < 4; ++i) {
            const float a = fabsf(bf16lo_to_f32(v[i])), b = fabsf(bf16hi_to_f32(v[i]));
            amax = fmax3(amax, a, b);
            bad |= !(a < INFINITY) || !(b < INFINITY);
          }
        }
        // the exponent field of the largest, kept where both factors are normal
        const int e = min(max(static_cast<int>(__float_as_uint(amax) >> 23), 16), 254) - 7;
        const float down = __uint_as_float(static_cast<uint32_t>(254 - e) << 23);  // 2^(127 - e)
        const float up = __uint_as_float(static_cast<uint32_t>(e) << 23);          // 2^(e - 127)
        // (a row with an infinity or a NaN has no attention: its scores become NaN)
        reinterpret_cast<float*>(smem + L::kRow)[(uq % kChunkRowDepth) * 128 + tid] = bad ? NAN : up;
        const uint32_t q_at = sbase + L::kQ + qb * L::kQBytes;
        #pragma unroll 1
        for (int c = 0; c < D / 16; ++c) {
          uint32_t hi[4], lo[4];
          #pragma unroll
          for (int half = 0; half < 2; ++half) {
            const uint4 x = chunk_at(2 * c + half);
            const uint32_t v[4] = {x.x, x.y, x.z, x.w};
            uint16_t h16[4], l16[4];
            #pragma unroll
            for (int i = 0; i < 4; ++i) {
              const float a = bf16lo_to_f32(v[i]) * down, b = bf16hi_to_f32(v[i]) * down;
              h16[i] = pack_e4m3x2(a, b);
              float va, vb;
              e4m3x2_values(h16[i], va, vb);
              l16[i] = pack_e4m3x2(a - va, b - vb);
            }
            hi[2 * half] = h16[0] | static_cast<uint32_t>(h16[1]) << 16;
            hi[2 * half + 1] = h16[2] | static_cast<uint32_t>(h16[3]) << 16;
            lo[2 * half] = l16[0] | static_cast<uint32_t>(l16[1]) << 16;
            lo[2 * half + 1] = l16[2] | static_cast<uint32_t>(l16[3]) << 16;
          }
          const uint32_t dst = q_at + tid * D + ((D == 128 ? c ^ (tid & 7) : c ^ ((tid >> 1) & 3)) << 4);
          st_shared_v4(dst, hi[0], hi[1], hi[2], hi[3]);
          st_shared_v4(dst + kChunkRows * D, lo[0], lo[1], lo[2], lo[3]);
        }
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) {
          mbar_arrive_cluster(lbar(L::bQF + qb));
          mbar_arrive(bar(L::bLE));
        }
      }
      for (int j = w.j; j < j_end; ++j, ++g) {
        if (!kVBoth && !leader) continue;
        const int sr = g % kChunkRawV, sv = g % SV;
        if (!(ok = wait_warp(bar(L::bRF + sr), static_cast<uint32_t>(g / kChunkRawV) & 1u, wc, kRoleConvert, 3)))
          break;
        if (g >= SV && !(ok = wait_warp(bar(L::bVE + sv), (static_cast<uint32_t>(g / SV) & 1u) ^ 1u, wc,
                                             kRoleConvert, 4)))
          break;
        const int valid = w.L - j * kChunkTile;  // rows past the request's end may hold anything: zeros
        #pragma unroll 1
        for (int i = 0; i < 4; ++i) {
          const int key = (tid >> 2) + 32 * i, c = tid & 3;
          const uint4 x = *reinterpret_cast<const uint4*>(smem + L::kVRaw + sr * 8192 + key * 64 + c * 16);
          const uint32_t v[4] = {x.x, x.y, x.z, x.w};
          uint32_t y[8];
          #pragma unroll
          for (int k = 0; k < 4; ++k) {
            y[2 * k] = codes_to_bf16x2(__byte_perm(v[k], 0, 0x1404));
            y[2 * k + 1] = codes_to_bf16x2(__byte_perm(v[k], 0, 0x3424));
          }
          if (nan_codes(v[0]) | nan_codes(v[1]) | nan_codes(v[2]) | nan_codes(v[3])) {
            #pragma unroll
            for (int k = 0; k < 4; ++k) {
              const uint32_t bad = nan_codes(v[k]);
              y[2 * k] |= ((bad & 0x80u) ? 0x7fc0u : 0u) | ((bad & 0x8000u) ? 0x7fc00000u : 0u);
              y[2 * k + 1] |= ((bad & 0x800000u) ? 0x7fc0u : 0u) | ((bad & 0x80000000u) ? 0x7fc00000u : 0u);
            }
          }
          if (key >= valid) {
            #pragma unroll
            for (int k = 0; k < 8; ++k) y[k] = 0u;
          }
          const uint32_t dst = sbase + L::kV + sv * L::kVBytes + key * 128;
          st_shared_v4(dst + (((2 * c) ^ (key & 7)) << 4), y[0], y[1], y[2], y[3]);
          st_shared_v4(dst + (((2 * c + 1) ^ (key & 7)) << 4), y[4], y[5], y[6], y[7]);
        }
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) {
          mbar_arrive_cluster(lbar(L::bVF + sv));
          mbar_arrive(bar(L::bRE + sr));
        }
      }
      if (!ok) break;
      ++uq;
    }
  }
  tc_fence_before();
  cluster_sync_all();  // no MMA, copy or remote arrival of either CTA is still in flight
  if (threadIdx.x == 0 && misc[1] != 0) atomicCAS(p.status, 0, static_cast<int>(misc[1]));
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc_pair(tmem, 512);
  }
}

}  // namespace attn
