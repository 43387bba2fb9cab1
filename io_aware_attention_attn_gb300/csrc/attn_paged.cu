// attn_paged.cu -- attention of one new token per request over a paged key-value cache.
//
// For each (request s, K/V head, group of up to 32 of its query rows) -- a unit -- with K, V the
// request's rows:  S = scale Q K^T,  O = softmax(S) V,  read once in tiles of 64 keys.
//
// What bounds it: reading K and V (64 requests of 16384 tokens, 32 query and 8 K/V heads, d = 128: 4.3 GB
// in 593-602 us, 7.2 TB/s; 48 requests of up to 16384 from E4M3 pages of 16 rows: 130 us, 6.4 TB/s).  A key
// costs 4 d bytes (bf16) and 4 d operations a query row, so at up to 32 rows the tensor work is far
// below what the copy takes and the kernel is built around the copies: a producer warp fills a ring of
// tiles by TMA (one box per page part), four consumer warps each take 16 of a tile's 64 keys and never
// wait for one another inside a unit.
//
// Products: with few query rows the keys go on the 16-row side of the warp product,
// S^T[keys x rows] = K Q^T and O^T[d x rows] += V^T P^T, rows in groups of 8 -- half the products and
// half the registers of the other orientation at up to 8 rows.  (A tcgen05 product has 64 or 128
// rows at least, its result sits in tensor memory, and each tile would pay a
// commit, a load and two hand-offs between warps; a warp product leaves everything in registers.)
// P^T needs the score tile transposed between the products: two movmatrix per 8 rows.
//
// Softmax: each warp keeps a reference maximum m of its own keys per row (log2 units) that, over a bf16
// cache, trails the true one by at most 8, so P <= 256; the maximum is looked for across lanes only when some
// score passes m + 8.  Row sums stay per lane, in fp32 and of the unrounded P, until a unit ends.  P is
// rounded to V's type for the product, as in the whole-sequence forward: its errors average out like
// the rounding of O itself and are as large (2.2e-3 of O's norm against 1.7e-3 of a correctly rounded
// O); two bf16 pieces of P would remove them for twice the products (64 requests of 16384 0.3 % slower,
// short ones 2 %, 32 rows a K/V head 16 to 19 %).
//
// E4M3 cache: codes become f16 on the way from shared memory to the product (exact; the 8-bit products of
// a warp, with q in two pieces, would take K's codes as they are but were slower: 144 us for 131);
// q becomes f16 after a power-of-two scaling of its row (exact down to 2^-22 of the row's largest
// element); a key's K scale multiplies its scores, its V scale v its P, which is then rounded to f16 (2^-11
// of the value).  So that f16 holds P v whatever the scales are, the reference m follows P v: it is set to
// the largest score + log2 |v| of a row, less 6, and moved when P |v| passes 2^15, so an operand falls
// below f16's normal range only 2^20 under the row's largest.  A key whose weight is nothing cannot set
// it, nor one whose codes are all zero (its scale may be anything; looked for only where m would move: all
// rows zero, with scale 1, 32 requests of 8192 take 149 us instead of 82).  P by itself is then anything fp32 holds, 2^124 at most (it is 2^115 where m is set because V's scales are below
// 2^-109, or nothing but zeros meets the largest scores), and its row sums are kept 2^-16 smaller.
//
// Work split: the tiles of all units in order (request, head, row group), each unit with a few more for
// what its end costs, are cut into equal shares, one a CTA.  A unit inside one share is finished by
// its CTA; the parts of a unit that spans several go to the workspace, at most two a CTA, and
// paged_join_kernel merges them.  It works out for itself which CTAs hold a unit's parts, from the
// lengths, while it waits for them.
#include "attn_gen.cuh"
#include "attn_gen.h"
#include "attn_paged_split.h"
#include "sm103_ptx.cuh"

#include <atomic>
#include <cmath>

namespace attn {
namespace {

constexpr int kSlices = 4;                       // key slices of 16 in a tile, a warp each
enum : int { kRoleProducer = 7, kRoleConsumer = 8 };

// The reference maximum of a row over an E4M3 cache, in log2 units (see above).
constexpr float kNoRef = 3.402823466e+38f;        // -m of a row without one: P of any score is infinite
constexpr float kPvSet = 6.f, kPSet = 115.f;      // P |v| and P at most where m is set
constexpr float kTrailE4m3 = 9.f;                 // and how far past that m is moved
constexpr float kSumLog2 = 16.f;                  // row sums are of 2^-16 P

// NT: groups of 8 query rows a warp holds; RW: row slices, each with four warps of its own.
template <int D, bool E4M3, int NT, int RW>
struct PagedCfg {
  static constexpr int kWarps = kSlices * RW;                     // consumers; one producer more
  static constexpr int kThreads = (kWarps + 1) * 32;
  // CTAs an SM holds: as many as registers allow, by the five warps of a CTA on four sub-partitions.
  // The smaller a tile, the less time a warp's chain of dependent steps has for it (e4m3, d = 128, ragged
  // requests on 16-row pages: 159 us with two CTAs, 135 with three; bf16 is at the HBM rate with two as well, 588 us
  // for the 4.3 GB above against 597 with three, but short requests are bound by that chain too: 256
  // of 64 tokens 19.2 us with two, 16.9 with three).
  static constexpr int kCtas = RW == 2 ? 1 : D == 64 ? (NT == 1 ? 4 : NT == 2 ? 3 : 2)
                                                     : NT == 2 ? 2 : 3;
  static constexpr int kRowBytes = D * (E4M3 ? 1 : 2);
  static constexpr int kBlk = kRowBytes < 128 ? kRowBytes : 128;  // bytes of a row in one box
  static constexpr int kBlks = kRowBytes / kBlk;                  // boxes side by side
  static constexpr int kSide = kPagedTile * kRowBytes;            // K or V of a tile
  static constexpr int kStage = 2 * kSide;
  static constexpr int kMergeLd = D + 4;                          // spreads rows over the banks
  // row groups merged at once: all, but where that would cost the ring one of its three tiles
  static constexpr int kMergeNt = kCtas == 2 && kStage == 32768 ? 1 : NT;
  static constexpr int kMergeBytes = kMergeNt * 2 * 8 * kMergeLd * 4;  // of one row slice
  static constexpr int kStatBytes = 2 * kMergeNt * kSlices * 8 * 2 * 4;  // likewise, of two merges
  // tiles in the ring: what shared memory holds beside the rest (each CTA's 1 KB of the system's and
  // 1 KB for alignment), 8 at most
  static constexpr int kScaleBytes = E4M3 ? 2 * kPagedTile * 4 : 0;
  static constexpr int kFit = (233472 / kCtas - 2048 - RW * (kMergeBytes + kStatBytes) - 32) /
                              (kStage + kScaleBytes + 16);
  static constexpr int kStages = kFit < 8 ? kFit : 8;
  static constexpr int kScales = kStages * kStage;                // [stage][2][64] fp32
  static constexpr int kMerge = kScales + kStages * kScaleBytes;
  static constexpr int kStat = kMerge + RW * kMergeBytes;
  static constexpr int kBar = kStat + RW * kStatBytes;
  static constexpr int kMisc = kBar + 2 * kStages * 8;
  static constexpr int kBytes = kMisc + 32;
  static constexpr int kDyn = kBytes + 1024;
  static_assert(kStages >= 2 && kCtas * (kDyn + 1024) <= 233472, "paged ring exceeds shared memory");
};

// The unit and tile a CTA is at.
struct Walk {
  int s, h, rg, t, n, len;  // request, K/V head, row group, tile, tiles of the request, its length
  int ahead;                // the next request's length, asked for when this one began
};

__device__ __forceinline__ int req_len(const PagedParams& p, int s) {
  const int most = p.max_pages << p.page_shift;
  return min(max(p.seq_lens[s], 0), most);
}
// A request of length 0 has one empty tile, so that its O and lse are written.
__device__ __forceinline__ int req_tiles(int len) {
  return max((len + kPagedTile - 1) / kPagedTile, 1);
}
__device__ __forceinline__ void next_unit(const PagedParams& p, Walk& w) {
  w.t = 0;
  if (++w.rg < p.n_rg) return;
  w.rg = 0;
  if (++w.h < p.H_kv) return;
  w.h = 0;
  ++w.s;
  w.len = w.ahead;
  w.n = req_tiles(w.len);
  w.ahead = w.s + 1 < p.B ? req_len(p, w.s + 1) : 0;
}
// Places in the order of all units: a unit takes its tiles and `p.unit_cost` places more.
__device__ __forceinline__ int req_places(const PagedParams& p, int s) {
  return s < p.B ? req_tiles(req_len(p, s)) + p.unit_cost : 0;
}
// Places of all requests, by one warp.
__device__ __forceinline__ int all_places(const PagedParams& p) {
  int n = 0;
  for (int s0 = threadIdx.x & 31; s0 < p.B; s0 += 256) {
    #pragma unroll
    for (int k = 0; k < 8; ++k) n += req_places(p, s0 + 32 * k);
  }
  return __reduce_add_sync(0xffffffffu, n) * (p.H_kv * p.n_rg);
}
// Places of all requests, by a block of T threads for which one look each is not enough, and s_pre[i]:
// those of the requests before i's share of ceil(B / T).  Ends with the block in step.
template <int T>
__device__ int block_places(const PagedParams& p, int* s_pre, int* s_warp) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int share = (p.B + T - 1) / T, lo = min(tid * share, p.B), hi = min(lo + share, p.B);
  int sum = 0;
  #pragma unroll 8
  for (int s = lo; s < hi; ++s) sum += req_places(p, s);
  int scan = sum;
  #pragma unroll
  for (int off = 1; off < 32; off <<= 1) {
    const int up = __shfl_up_sync(0xffffffffu, scan, off);
    if (lane >= off) scan += up;
  }
  if (lane == 31) s_warp[warp] = scan;
  __syncthreads();
  int before = scan - sum, total = 0;
  #pragma unroll
  for (int i = 0; i < T / 32; ++i) {
    if (i < warp) before += s_warp[i];
    total += s_warp[i];
  }
  s_pre[tid] = before * (p.H_kv * p.n_rg);
  __syncthreads();
  return total * (p.H_kv * p.n_rg);
}
// The share of block_places that holds place `at`.
template <int T>
__device__ int share_of(const int* s_pre, int at) {
  int n = 0;
  #pragma unroll
  for (int i = 0; i < T; i += 32)
    n += __popc(__ballot_sync(0xffffffffu, s_pre[i + (threadIdx.x & 31)] <= at));
  return n - 1;
}
// Walk at place `at` (a warp's lanes together; w.t past the tiles: in the places after them), looked for
// from request `from` on, before which there are `before` places; returns the first place of its unit.
__device__ int find(const PagedParams& p, int at, Walk& w, int from = 0, int before = 0) {
  const int lane = threadIdx.x & 31, per = p.H_kv * p.n_rg;
  for (int s0 = from; s0 < p.B; s0 += 32) {
    const int s = s0 + lane;
    const int len = s < p.B ? req_len(p, s) : 0;
    const int n = s < p.B ? req_tiles(len) + p.unit_cost : 0;
    int scan = n * per;
    #pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
      const int up = __shfl_up_sync(0xffffffffu, scan, off);
      if (lane >= off) scan += up;
    }
    const uint32_t past = __ballot_sync(0xffffffffu, before + scan > at);
    if (past) {
      const int k = __ffs(past) - 1;
      before += __shfl_sync(0xffffffffu, scan - n * per, k);
      const int places = __shfl_sync(0xffffffffu, n, k);
      w.s = s0 + k;
      w.n = places - p.unit_cost;
      w.len = __shfl_sync(0xffffffffu, len, k);
      const UnitAt u = unit_at(static_cast<uint32_t>(at - before), static_cast<uint32_t>(places), p.n_rg);
      w.t = u.t;
      w.h = u.h;
      w.rg = u.rg;
      const int after = __shfl_sync(0xffffffffu, len, (k + 1) & 31);
      w.ahead = k < 31 ? after : w.s + 1 < p.B ? req_len(p, w.s + 1) : 0;
      return at - w.t;
    }
    before += __shfl_sync(0xffffffffu, scan, 31);
  }
  w = Walk{p.B, 0, 0, 0, 1, 0, 0};
  return at;
}

// This lane's share of the B operand of K Q^T (query row g of each group of 8, the elements that its
// positions along d stand for), and the factors of scores (log2 units) of rows 2 q4, 2 q4 + 1.  (Plain
// loads, as everywhere here: the read-only path is for what no kernel writes while this one lives, and
// this one may be set up while the kernel that writes q still runs.)
template <int D, bool E4M3, int NT>
__device__ __forceinline__ void load_q(const PagedParams& p, const Walk& w, int row_slice,
                                       uint32_t (&qf)[NT][D / 16][2], float (&mul)[NT][2]) {
  const int lane = threadIdx.x & 31, g = lane >> 2, q4 = lane & 3;
  const int row0 = w.rg * p.rg_rows, rows = min(p.rg_rows, p.group - row0);
  const __nv_bfloat16* q =
      p.q + (static_cast<int64_t>(w.s) * p.H + static_cast<int64_t>(w.h) * p.group + row0) * D;
  #pragma unroll
  for (int nt = 0; nt < NT; ++nt) {
    const int r = (row_slice * NT + nt) * 8 + g;
    #pragma unroll
    for (int k = 0; k < D / 16; ++k) {
      qf[nt][k][0] = qf[nt][k][1] = 0u;
      if (r < rows) {
        const __nv_bfloat16* src = q + r * D + 16 * k;
        if (E4M3) {  // codes 4 q4 .. 4 q4 + 3 of a key arrive in one register
          const uint2 v = *reinterpret_cast<const uint2*>(src + 4 * q4);
          qf[nt][k][0] = v.x;
          qf[nt][k][1] = v.y;
        } else {
          qf[nt][k][0] = *reinterpret_cast<const uint32_t*>(src + 2 * q4);
          qf[nt][k][1] = *reinterpret_cast<const uint32_t*>(src + 2 * q4 + 8);
        }
      }
    }
    if (E4M3) {
      float amax = 0.f;
      #pragma unroll
      for (int k = 0; k < D / 16; ++k)
        #pragma unroll
        for (int j = 0; j < 2; ++j)
          amax = fmax3(amax, fabsf(bf16lo_to_f32(qf[nt][k][j])), fabsf(bf16hi_to_f32(qf[nt][k][j])));
      amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 1));
      amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 2));
      // largest element to 2^8 .. 2^9: its exponent field, kept where both factors are normal
      const int e = min(max(static_cast<int>(__float_as_uint(amax) >> 23), 16), 254) - 8;
      const float down = __uint_as_float(static_cast<uint32_t>(254 - e) << 23);  // 2^(127 - e)
      const float up = __uint_as_float(static_cast<uint32_t>(e) << 23);          // 2^(e - 127)
      #pragma unroll
      for (int k = 0; k < D / 16; ++k)
        #pragma unroll
        for (int j = 0; j < 2; ++j)
          qf[nt][k][j] = pack_f16x2(bf16lo_to_f32(qf[nt][k][j]) * down,
                                    bf16hi_to_f32(qf[nt][k][j]) * down);
      mul[nt][0] = p.scale_log2 * __shfl_sync(0xffffffffu, up, (2 * q4) * 4);
      mul[nt][1] = p.scale_log2 * __shfl_sync(0xffffffffu, up, (2 * q4 + 1) * 4);
    } else {
      mul[nt][0] = mul[nt][1] = p.scale_log2;
    }
  }
}

// The largest value of a row's eight lanes (keys), scores of keys past the request's end, rows of O^T scaled.
__device__ __forceinline__ float max_of_keys(float v) {
  #pragma unroll
  for (int off = 4; off < 32; off <<= 1) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, off));
  return v;
}
// x 2^d.  Row sums over an E4M3 cache may be large where 2^d by itself is below fp32's range: references
// of two warps' rows are as far apart as log2 |v| of what they saw, and 2^-115 for keys without values.
__device__ __forceinline__ float times_exp2(float x, float d) {
  const float a = fmaxf(d, -120.f);
  return x * ex2_approx(a) * ex2_approx(d - a);
}
template <int NT>
__device__ __forceinline__ void mask_tail(float (&s)[NT][4], int live, bool in0, bool in1) {
  if (live >= 16) return;
  #pragma unroll
  for (int nt = 0; nt < NT; ++nt) {
    s[nt][0] = in0 ? s[nt][0] : -INFINITY;
    s[nt][1] = in0 ? s[nt][1] : -INFINITY;
    s[nt][2] = in1 ? s[nt][2] : -INFINITY;
    s[nt][3] = in1 ? s[nt][3] : -INFINITY;
  }
}
template <int STEPS>
__device__ __forceinline__ void scale_rows(float (&acc)[STEPS][4], const float (&c)[2]) {
  #pragma unroll
  for (int k = 0; k < STEPS; ++k) {
    acc[k][0] *= c[0];
    acc[k][1] *= c[1];
    acc[k][2] *= c[0];
    acc[k][3] *= c[1];
  }
}

template <int D, bool E4M3, int NT, int RW>
__global__ void __launch_bounds__((kSlices * RW + 1) * 32, PagedCfg<D, E4M3, NT, RW>::kCtas)
paged_kernel(const __grid_constant__ PagedParams p) {
  using L = PagedCfg<D, E4M3, NT, RW>;
  extern __shared__ uint8_t smem_raw[];
  const uint32_t base = (smem_u32(smem_raw) + 1023u) & ~1023u;
  uint8_t* sm = smem_raw + (base - smem_u32(smem_raw));
  int* misc = reinterpret_cast<int*>(sm + L::kMisc);  // [0] abort
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  auto full = [&](int st) { return base + L::kBar + st * 8; };
  auto empty = [&](int st) { return base + L::kBar + (L::kStages + st) * 8; };
  if (tid == 0) {
    misc[0] = 0;
    for (int i = 0; i < L::kStages; ++i) {
      mbar_init(full(i), E4M3 ? 33 : 1);  // E4M3: each producer lane's scale copies too
      mbar_init(empty(i), L::kWarps);
    }
    fence_barrier_init();
    tma_prefetch_desc(&p.tm_k);
    tma_prefetch_desc(&p.tm_v);
  }
  pdl_wait();
  // places of all units (fewer than 2^31: the host's check): each warp for itself where eight loads a
  // lane are enough (2000 requests of 16 tokens: 87 us then, each warp for itself 108)
  const bool few = p.B <= 256;
  int* s_pre = reinterpret_cast<int*>(sm + L::kMerge);
  const int total = few ? all_places(p) : block_places<L::kThreads>(p, s_pre, s_pre + L::kThreads);
  if (few) __syncthreads();
  pdl_launch_dependents();
  const int cta = static_cast<int>(blockIdx.x), G = min(p.ctas, total);
  if (cta >= G) return;
  const Shares shares(static_cast<uint32_t>(total), static_cast<uint32_t>(G));
  const int place0 = shares.start(cta);
  Walk w;
  int unit0;
  if (few) {
    unit0 = find(p, place0, w);
  } else {
    const int k = share_of<L::kThreads>(s_pre, place0);
    unit0 = find(p, place0, w, k * ((p.B + L::kThreads - 1) / L::kThreads), s_pre[k]);
    __syncthreads();  // what follows may write where s_pre is
  }
  int left = shares.start(cta + 1) - place0;  // places of this CTA still to come
  if (w.t >= w.n) {  // it starts behind a unit's last tile
    left -= unit0 + w.n + p.unit_cost - place0;
    if (left <= 0) return;
    next_unit(p, w);
  }
  const WaitCtx ctx{misc, p.status};

  if (warp == L::kWarps) {
    // ------------------------------------------------------------------------------ producer
    const uint64_t policy = l2_policy_evict_first();
    const int wide_shift = 31 - __clz(p.box_rows);
    const int pages_tile = max(kPagedTile >> p.page_shift, 1);
    int entries = 0, entry_base = -1, entry_s = -1;  // lane's entry of the 32 looked up last
    bool ok = true;
    int it = 0, st = 0;
    uint32_t phase = 1;  // of the empty barrier waited for, from the second round on
    for (; left > 0; ++it) {
      const int rows = min(kPagedTile, w.len - w.t * kPagedTile);
      // A last tile of 32 rows or fewer comes in boxes of 16: a box is read whole, and one more costs the
      // SM ~43 ns, the time of 2 KB (2000 requests of 16 tokens on 64-row pages, 8 K/V heads,
      // d = 128: 67 us instead of 87).
      const bool narrow = rows <= 32 && p.box_rows > 16;
      const int box_shift = narrow ? 4 : wide_shift, box_rows = 1 << box_shift;
      const int parts = rows > 0 ? (rows + box_rows - 1) >> box_shift : 0;
      const int page0 = (w.t * kPagedTile) >> p.page_shift;
      if (parts > 0 && (entry_s != w.s || page0 < entry_base || page0 + pages_tile > entry_base + 32)) {
        entry_s = w.s;
        entry_base = page0;
        const int e = page0 + lane;
        const int have = (w.len + (1 << p.page_shift) - 1) >> p.page_shift;
        entries = e < have ? p.table[static_cast<size_t>(w.s) * p.max_pages + e] : 0;
        if (e < have && static_cast<unsigned>(entries) >= static_cast<unsigned>(p.num_pages)) {
          atomicCAS(p.status, 0, kStatusBadPage);
          entries = -1;
        }
      }
      if (it >= L::kStages)
        ok = mbar_wait_warp(empty(st), phase, ctx, kRoleProducer, 1);
      if (!ok) break;
      const uint32_t stage = base + st * L::kStage;
      if (E4M3) {  // lane: the scales of rows 4 r4 .. 4 r4 + 3 of K or V; zeros of a page that is none
        const int side = lane >> 4, row = (lane & 15) * 4;
        const int at = ((w.t * kPagedTile + row) >> p.page_shift) - entry_base;
        const int pg = __shfl_sync(0xffffffffu, entries, at & 31);
        if ((row >> box_shift) < parts) {
          const uint32_t dst = base + L::kScales + ((st * 2 + side) * kPagedTile + row) * 4;
          if (pg >= 0)
            copy16(dst, (side ? p.vs : p.ks) + (((static_cast<int64_t>(pg) * p.H_kv + w.h) << p.page_shift) +
                                                ((w.t * kPagedTile + row) & ((1 << p.page_shift) - 1))));
          else
            st_shared_v4(dst, 0u, 0u, 0u, 0u);
        }
        copy_arrive(full(st));
        __syncwarp();
      }
      if (lane == 0)
        mbar_arrive_expect_tx(full(st), static_cast<uint32_t>(parts) * box_rows * 2 * L::kRowBytes);
      __syncwarp();
      {  // lane -> (part, block, K or V); every lane takes part in the look-up of its page
        constexpr int kPerPart = 2 * L::kBlks;
        const int q = lane / kPerPart, o = lane % kPerPart;
        const int side = o / L::kBlks, blk = o % L::kBlks;
        const int row0 = w.t * kPagedTile + q * box_rows;
        const int at = (row0 >> p.page_shift) - entry_base;
        const int pg = __shfl_sync(0xffffffffu, entries, at & 31);
        if (q < parts)
          tma_load_4d_hint(stage + side * L::kSide + blk * (kPagedTile * L::kBlk) +
                               q * box_rows * L::kBlk,
                           narrow ? (side ? &p.tm_v16 : &p.tm_k16) : side ? &p.tm_v : &p.tm_k,
                           full(st), blk * (L::kBlk / (E4M3 ? 1 : 2)),
                           row0 & ((1 << p.page_shift) - 1), w.h, pg >= 0 ? pg : p.num_pages,
                           policy);
      }
      if (++st == L::kStages) {
        st = 0;
        phase ^= 1;
      }
      --left;
      if (++w.t == w.n) {
        left -= p.unit_cost;
        if (left > 0) next_unit(p, w);
      }
    }
    if (!ok) {  // copies in flight land before the CTA's shared memory goes
      if (E4M3) copy_wait<0>();
      for (int k = it > L::kStages ? it - L::kStages : 0; k < it; ++k)
        mbar_wait_drain(full(k % L::kStages), static_cast<uint32_t>((k / L::kStages) & 1));
    }
    return;
  }

  // -------------------------------------------------------------------------------- consumers
  const int g = lane >> 2, q4 = lane & 3;
  const int slice = warp % kSlices, row_slice = RW == 1 ? 0 : warp / kSlices;
  constexpr int kSteps = D / 16;      // k16 steps of S, m16 tiles of O^T
  bool dead = false;                  // a wait gave up: go through the motions, compute nothing
  int st = 0, merges = 0;
  uint32_t phase = 0;
  bool first = true;                  // the CTA's first unit
  float* merge = reinterpret_cast<float*>(sm + L::kMerge + row_slice * L::kMergeBytes);
  float* stat = reinterpret_cast<float*>(sm + L::kStat + row_slice * L::kStatBytes);
  uint32_t qf[NT][kSteps][2];
  float mul[NT][2];
  load_q<D, E4M3, NT>(p, w, row_slice, qf, mul);
  while (left > 0) {
    const int t_begin = w.t, t_end = min(w.n, w.t + left);
    // per row: nm = -m; over bf16, above: the score past which m is moved (-inf while there is no m)
    float acc[NT][kSteps][4], nm[NT][2], above[NT][2], l[NT][2];
    #pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      nm[nt][0] = nm[nt][1] = E4M3 ? kNoRef : 0.f;
      above[nt][0] = above[nt][1] = -INFINITY;
      l[nt][0] = l[nt][1] = 0.f;
      #pragma unroll
      for (int k = 0; k < kSteps; ++k)
        #pragma unroll
        for (int j = 0; j < 4; ++j) acc[nt][k][j] = 0.f;
    }
    auto no_ref = [&](int nt, int j) { return E4M3 ? nm[nt][j] == kNoRef : above[nt][j] == -INFINITY; };

    for (int t = t_begin; t < t_end; ++t) {
      if (!dead && !mbar_wait_warp(full(st), phase, ctx, kRoleConsumer, 2)) dead = true;
      const int live = w.len - t * kPagedTile - slice * 16;  // of this warp's 16 keys
      if (!dead && live > 0) {
        const uint32_t kst = base + st * L::kStage, vst = kst + L::kSide;
        // lane (g, q4): s[0], s[1] = key g, rows 2 q4, 2 q4 + 1;  s[2], s[3] = key g + 8
        const bool in0 = g < live, in1 = g + 8 < live;
        uint32_t pf[NT][2];
        if constexpr (!E4M3) {
          float s[NT][4];
          #pragma unroll
          for (int nt = 0; nt < NT; ++nt) s[nt][0] = s[nt][1] = s[nt][2] = s[nt][3] = 0.f;
          const int key = slice * 16 + (lane & 15);
          #pragma unroll
          for (int k = 0; k < kSteps; ++k) {
            const int chunk = (k & 3) * 2 + (lane >> 4);
            uint32_t a[4];
            ldsm4(kst + (k >> 2) * (kPagedTile * 128) + key * 128 + ((chunk ^ (key & 7)) << 4), a);
            #pragma unroll
            for (int nt = 0; nt < NT; ++nt)
              mma16816<false>(s[nt], a[0], a[1], a[2], a[3], qf[nt][k][0], qf[nt][k][1]);
          }
          mask_tail<NT>(s, live, in0, in1);
          bool grow = false;
          #pragma unroll
          for (int nt = 0; nt < NT; ++nt)
            grow |= fmaxf(s[nt][0], s[nt][2]) > above[nt][0] || fmaxf(s[nt][1], s[nt][3]) > above[nt][1];
          if (__any_sync(0xffffffffu, grow)) {
            #pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
              float c[2];
              #pragma unroll
              for (int j = 0; j < 2; ++j) {
                const float top = max_of_keys(fmaxf(s[nt][j], s[nt][j + 2]));
                const float m = top * p.scale_log2;
                const bool none = no_ref(nt, j);  // no m yet: acc and l are 0 (or NaN)
                c[j] = 1.f;
                if (top != -INFINITY && (none || m > -nm[nt][j])) {
                  c[j] = none ? 1.f : ex2_approx(-nm[nt][j] - m);
                  nm[nt][j] = -m;
                  above[nt][j] = top + p.trail;
                }
                l[nt][j] *= c[j];
              }
              scale_rows<kSteps>(acc[nt], c);
            }
          }
          #pragma unroll
          for (int nt = 0; nt < NT; ++nt) {
            const float p0 = ex2_approx(fmaf(s[nt][0], p.scale_log2, nm[nt][0]));
            const float p1 = ex2_approx(fmaf(s[nt][1], p.scale_log2, nm[nt][1]));
            const float p2 = ex2_approx(fmaf(s[nt][2], p.scale_log2, nm[nt][0]));
            const float p3 = ex2_approx(fmaf(s[nt][3], p.scale_log2, nm[nt][1]));
            l[nt][0] += p0 + p2;
            l[nt][1] += p1 + p3;
            pf[nt][0] = transpose8x8(pack_bf16x2(p0, p1));
            pf[nt][1] = transpose8x8(pack_bf16x2(p2, p3));
          }
        } else {
          const float* sc =
              reinterpret_cast<const float*>(sm + L::kScales) + st * 2 * kPagedTile + slice * 16;
          const float sk0 = sc[g], sk1 = sc[g + 8];
          float sv0 = in0 ? sc[kPagedTile + g] : 0.f, sv1 = in1 ? sc[kPagedTile + g + 8] : 0.f;
          float sum[NT][2];  // of a lane's P
          // A key whose codes are all zero (of either sign) weighs nothing: its scale is taken as 0.  Lane i
          // looks at key i % 16, at sixteen codes, and at the others only where those of some key are zero.
          auto drop_zeros = [&] {
            const uint8_t* codes = sm + (vst - base) + (slice * 16 + (lane & 15)) * L::kBlk;
            auto some = [&](int c) {
              const uint4 x = *reinterpret_cast<const uint4*>(codes + 16 * c);
              return ((x.x | x.y | x.z | x.w) & 0x7f7f7f7fu) != 0u;
            };
            uint32_t keys = __ballot_sync(0xffffffffu, some(0));
            if (keys == 0xffffffffu) return;
            bool any = false;
            #pragma unroll
            for (int c = 1; c < L::kRowBytes / 16; ++c) any |= some(c);
            keys |= __ballot_sync(0xffffffffu, any);
            if (!(keys >> g & 1u) && fabsf(sv0) < INFINITY) sv0 = 0.f;
            if (!(keys >> (g + 8) & 1u) && fabsf(sv1) < INFINITY) sv1 = 0.f;
          };
          // Twice where m has to move: the scores are formed again (they are rarely needed
          // twice, and cost no registers then).
          for (bool move = t == t_begin;; move = true) {
            float e[NT][4];
            #pragma unroll
            for (int nt = 0; nt < NT; ++nt) e[nt][0] = e[nt][1] = e[nt][2] = e[nt][3] = 0.f;
            const int key = slice * 16 + (lane & 15);
            #pragma unroll
            for (int k = 0; k < kSteps; k += 2) {
              const int chunk = k + (lane >> 4);
              const int sw = L::kBlk == 128 ? chunk ^ (key & 7) : chunk ^ ((key >> 1) & 3);
              uint32_t a[4];
              ldsm4(kst + key * L::kBlk + (sw << 4), a);
              #pragma unroll
              for (int j = 0; j < 2; ++j) {
                const uint32_t lo0 = e4m3x2_to_f16x2(a[2 * j]), hi0 = e4m3x2_to_f16x2(a[2 * j] >> 16);
                const uint32_t lo1 = e4m3x2_to_f16x2(a[2 * j + 1]),
                               hi1 = e4m3x2_to_f16x2(a[2 * j + 1] >> 16);
                #pragma unroll
                for (int nt = 0; nt < NT; ++nt)
                  mma16816<true>(e[nt], lo0, lo1, hi0, hi1, qf[nt][k + j][0], qf[nt][k + j][1]);
              }
            }
            #pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
              e[nt][0] *= mul[nt][0] * sk0;
              e[nt][1] *= mul[nt][1] * sk0;
              e[nt][2] *= mul[nt][0] * sk1;
              e[nt][3] *= mul[nt][1] * sk1;
            }
            mask_tail<NT>(e, live, in0, in1);
            if (move) {
              if (t == t_begin) drop_zeros();
              // (a scale that is infinite or NaN makes O what it is without a reference's help)
              const float lv0 = fabsf(sv0) < INFINITY ? __log2f(fabsf(sv0)) - kPvSet : -INFINITY;
              const float lv1 = fabsf(sv1) < INFINITY ? __log2f(fabsf(sv1)) - kPvSet : -INFINITY;
              #pragma unroll
              for (int nt = 0; nt < NT; ++nt) {
                float c[2];
                #pragma unroll
                for (int j = 0; j < 2; ++j) {
                  const float m = floorf(max_of_keys(
                      fmax3(fmaxf(e[nt][j], e[nt][j + 2]) - kPSet, e[nt][j] + lv0, e[nt][j + 2] + lv1)));
                  const bool none = no_ref(nt, j);  // no m yet: acc and l are 0 (or NaN)
                  c[j] = 1.f;
                  if (m != -INFINITY && (none || m + nm[nt][j] >= kTrailE4m3)) {
                    if (!none) {
                      c[j] = ex2_approx(-nm[nt][j] - m);
                      l[nt][j] = times_exp2(l[nt][j], -nm[nt][j] - m);
                    }
                    nm[nt][j] = -m;
                  }
                }
                scale_rows<kSteps>(acc[nt], c);
              }
            }
            float most = 0.f, most0 = 0.f, most1 = 0.f;
            #pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
              const float p0 = ex2_approx(e[nt][0] + nm[nt][0]), p1 = ex2_approx(e[nt][1] + nm[nt][1]);
              const float p2 = ex2_approx(e[nt][2] + nm[nt][0]), p3 = ex2_approx(e[nt][3] + nm[nt][1]);
              const float o0 = p0 * sv0, o1 = p1 * sv0, o2 = p2 * sv1, o3 = p3 * sv1;
              most0 = fmax3(most0, fabsf(o0), fabsf(o1));
              most1 = fmax3(most1, fabsf(o2), fabsf(o3));
              sum[nt][0] = p0 + p2;
              sum[nt][1] = p1 + p3;
              most = fmax3(most, sum[nt][0], sum[nt][1]);
              pf[nt][0] = pack_f16x2(o0, o1);
              pf[nt][1] = pack_f16x2(o2, o3);
            }
            auto over = [&] {
              return __any_sync(0xffffffffu, most > 0x1p124f || fmaxf(most0, most1) > 0x1p15f);
            };
            if (move || !over()) break;
            drop_zeros();
            if (sv0 == 0.f) most0 = 0.f;
            if (sv1 == 0.f) most1 = 0.f;
            if (!over()) {  // it was they
              #pragma unroll
              for (int nt = 0; nt < NT; ++nt) {
                pf[nt][0] = sv0 == 0.f ? 0u : pf[nt][0];
                pf[nt][1] = sv1 == 0.f ? 0u : pf[nt][1];
              }
              break;
            }
          }
          #pragma unroll
          for (int nt = 0; nt < NT; ++nt) {
            l[nt][0] = fmaf(sum[nt][0], 0x1p-16f, l[nt][0]);
            l[nt][1] = fmaf(sum[nt][1], 0x1p-16f, l[nt][1]);
            pf[nt][0] = transpose8x8(pf[nt][0]);
            pf[nt][1] = transpose8x8(pf[nt][1]);
          }
        }
        // V rows past the request's end may hold anything: taken as zero
        const bool tail = live < 16;
        const uint32_t keep0 = (2 * q4 < live ? 0xffffu : 0u) | (2 * q4 + 1 < live ? 0xffff0000u : 0u);
        const uint32_t keep1 = (2 * q4 + 8 < live ? 0xffffu : 0u) | (2 * q4 + 9 < live ? 0xffff0000u : 0u);
        if (!E4M3) {
          const int key = slice * 16 + ((lane >> 4) << 3) + (lane & 7);
          #pragma unroll
          for (int k = 0; k < kSteps; ++k) {
            const int chunk = (k & 3) * 2 + ((lane >> 3) & 1);
            uint32_t a[4];
            ldsm4_t(vst + (k >> 2) * (kPagedTile * 128) + key * 128 + ((chunk ^ (key & 7)) << 4), a);
            if (tail) {
              a[0] &= keep0;
              a[1] &= keep0;
              a[2] &= keep1;
              a[3] &= keep1;
            }
            #pragma unroll
            for (int nt = 0; nt < NT; ++nt)
              mma16816<false>(acc[nt][k], a[0], a[1], a[2], a[3], pf[nt][0], pf[nt][1]);
          }
        } else {
          const int key = slice * 16 + (lane & 15);
          #pragma unroll
          for (int k = 0; k < kSteps; k += 2) {
            const int chunk = k + (lane >> 4);
            const int sw = L::kBlk == 128 ? chunk ^ (key & 7) : chunk ^ ((key >> 1) & 3);
            uint32_t a[4];
            ldsm4_t(vst + key * L::kBlk + (sw << 4), a);
            // a register: key pair x columns 2g, 2g + 1; split into the column's key pairs
            #pragma unroll
            for (int j = 0; j < 2; ++j) {
              const uint32_t x0 = __byte_perm(a[2 * j], 0, 0x3120);
              const uint32_t x1 = __byte_perm(a[2 * j + 1], 0, 0x3120);
              uint32_t v0 = e4m3x2_to_f16x2(x0), v1 = e4m3x2_to_f16x2(x0 >> 16);
              uint32_t v2 = e4m3x2_to_f16x2(x1), v3 = e4m3x2_to_f16x2(x1 >> 16);
              if (tail) {
                v0 &= keep0;
                v1 &= keep0;
                v2 &= keep1;
                v3 &= keep1;
              }
              #pragma unroll
              for (int nt = 0; nt < NT; ++nt)
                mma16816<true>(acc[nt][k + j], v0, v1, v2, v3, pf[nt][0], pf[nt][1]);
            }
          }
        }
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(empty(st));
      if (++st == L::kStages) {
        st = 0;
        phase ^= 1;
      }
    }
    left -= places_done(t_begin, t_end, w.n, p.unit_cost);

    // ---- end of the unit (or of this CTA's part of it): the four warps' results become one, while
    // the next unit's query rows are on their way
    const bool whole = t_begin == 0 && t_end == w.n;
    const int len = w.len;
    const int part = 2 * cta + (first ? 0 : 1);
    first = false;
    const int row0 = w.rg * p.rg_rows, rows = min(p.rg_rows, p.group - row0);
    const int64_t out0 = static_cast<int64_t>(w.s) * p.H + static_cast<int64_t>(w.h) * p.group + row0;
    if (left > 0) {
      next_unit(p, w);
      load_q<D, E4M3, NT>(p, w, row_slice, qf, mul);
    }
    // what the row sums are relative to
    auto sum_ref = [&](int nt, int j) { return E4M3 ? kSumLog2 - nm[nt][j] : -nm[nt][j]; };
    // element (row, column) of this lane's j-th accumulator of tile k
    auto cell = [&](int k, int j) {
      const int row = 2 * q4 + (j & 1);
      const int col = E4M3 ? 16 * k + 2 * g + (j >> 1) : 16 * k + g + 8 * (j >> 1);
      return row * L::kMergeLd + col;
    };
    #pragma unroll
    for (int n0 = 0; n0 < NT; n0 += L::kMergeNt) {
      float* st2 = stat + (merges & 1) * (L::kMergeNt * kSlices * 16);
      ++merges;
      #pragma unroll
      for (int i = 0; i < L::kMergeNt; ++i) {
        const int nt = n0 + i;
        #pragma unroll
        for (int j = 0; j < 2; ++j) {
          #pragma unroll
          for (int off = 4; off < 32; off <<= 1)
            l[nt][j] += __shfl_xor_sync(0xffffffffu, l[nt][j], off);
          if (g == 0)
            *reinterpret_cast<float2*>(st2 + ((i * kSlices + slice) * 8 + 2 * q4 + j) * 2) = make_float2(
                no_ref(nt, j) ? -INFINITY : sum_ref(nt, j), l[nt][j]);
        }
      }
      named_barrier_sync(1 + row_slice, kSlices * 32);
      #pragma unroll
      for (int i = 0; i < L::kMergeNt; ++i) {
        const int nt = n0 + i;
        #pragma unroll
        for (int j = 0; j < 2; ++j) {
          float top = -INFINITY;
          #pragma unroll
          for (int x = 0; x < kSlices; ++x)
            top = fmaxf(top, st2[((i * kSlices + x) * 8 + 2 * q4 + j) * 2]);
          // no m: no finite score, so acc and l are 0 (or NaN, which stays)
          const float c = (no_ref(nt, j) ? 1.f : ex2_approx(sum_ref(nt, j) - top)) *
                          (E4M3 ? 0x1p-16f : 1.f);
          #pragma unroll
          for (int k = 0; k < kSteps; ++k) {
            acc[nt][k][j] *= c;
            acc[nt][k][j + 2] *= c;
          }
        }
        // slices 0 and 2 share a buffer, 1 and 3 the other: each writes the half of the columns
        // that its partner then adds its own to
        float* half = merge + (2 * i + (slice & 1)) * 8 * L::kMergeLd;
        if (slice >= 2) {
          #pragma unroll
          for (int k = 0; k < kSteps / 2; ++k)
            #pragma unroll
            for (int j = 0; j < 4; ++j) half[cell(k, j)] = acc[nt][k][j];
        } else {
          #pragma unroll
          for (int k = kSteps / 2; k < kSteps; ++k)
            #pragma unroll
            for (int j = 0; j < 4; ++j) half[cell(k, j)] = acc[nt][k][j];
        }
      }
      named_barrier_sync(1 + row_slice, kSlices * 32);
      #pragma unroll
      for (int i = 0; i < L::kMergeNt; ++i) {
        const int nt = n0 + i;
        float* half = merge + (2 * i + (slice & 1)) * 8 * L::kMergeLd;
        if (slice < 2) {
          #pragma unroll
          for (int k = 0; k < kSteps / 2; ++k)
            #pragma unroll
            for (int j = 0; j < 4; ++j) half[cell(k, j)] += acc[nt][k][j];
        } else {
          #pragma unroll
          for (int k = kSteps / 2; k < kSteps; ++k)
            #pragma unroll
            for (int j = 0; j < 4; ++j) half[cell(k, j)] += acc[nt][k][j];
        }
      }
      named_barrier_sync(1 + row_slice, kSlices * 32);
      const int base_row = (row_slice * NT + n0) * 8;
      const int cells = min(L::kMergeNt * 8, rows - base_row) * (D / 4);
      for (int e = slice * 32 + lane; e < cells; e += kSlices * 32) {
        const int r = e / (D / 4), c4 = e % (D / 4), i = r / 8, row = base_row + r;
        float top = -INFINITY, sum = 0.f;
        float2 ml[kSlices];
        #pragma unroll
        for (int x = 0; x < kSlices; ++x) {
          ml[x] = *reinterpret_cast<const float2*>(st2 + ((i * kSlices + x) * 8 + (r & 7)) * 2);
          top = fmaxf(top, ml[x].x);
        }
        #pragma unroll
        for (int x = 0; x < kSlices; ++x) {
          if (E4M3) sum += ml[x].x == -INFINITY ? ml[x].y : times_exp2(ml[x].y, ml[x].x - top);
          else sum += (ml[x].x == -INFINITY ? 1.f : ex2_approx(ml[x].x - top)) * ml[x].y;
        }
        const float* at0 = merge + (2 * i * 8 + (r & 7)) * L::kMergeLd + 4 * c4;
        const float4 a = *reinterpret_cast<const float4*>(at0);
        const float4 b = *reinterpret_cast<const float4*>(at0 + 8 * L::kMergeLd);
        float4 v = make_float4(a.x + b.x, a.y + b.y, a.z + b.z, a.w + b.w);
        if (whole) {
          const float inv = len > 0 ? 1.f / sum : 0.f;
          const int64_t at = out0 + row;
          *reinterpret_cast<uint2*>(p.o + at * D + 4 * c4) =
              make_uint2(pack_bf16x2(v.x * inv, v.y * inv), pack_bf16x2(v.z * inv, v.w * inv));
          if (c4 == 0)
            p.lse[at] = sum > 0.f || sum != sum ? (top + log2f(sum)) * 0.69314718055994530942f
                                                : -INFINITY;
        } else {
          const int64_t at = static_cast<int64_t>(part) * p.rg_rows + row;
          const uint32_t exponent = __float_as_uint(sum) >> 23;
          if (E4M3 && exponent - 1u < 253u) {  // relative to a power of two near the sum, as the join expects
            const float f = __uint_as_float((254u - exponent) << 23);
            v = make_float4(v.x * f, v.y * f, v.z * f, v.w * f);
            sum *= f;
            top += static_cast<float>(static_cast<int>(exponent) - 127);
          }
          *reinterpret_cast<float4*>(p.part_o + at * D + 4 * c4) = v;
          if (c4 == 0)
            *reinterpret_cast<float2*>(p.part_ml + at * 2) = make_float2(top, sum);
        }
      }
    }
  }
}

// Merge of one unit's parts: of the CTA that holds its first tile, then the first part of each that
// follows, to the one that holds its last.  Block x is for unit x, or, when there are more units than
// CTAs, for the unit that CTA x ends and an earlier one began.  M = max m_j, weights 2^(m_j - M).
// A row's parts are shared out to 1, 2, 4 or 8 of the block's warps, by how many there are, and joined
// through shared memory; a lane holds d/32 columns.  Latency bounds it, so who holds what is worked out
// before the wait, many rows go side by side (32 rows of 2 or 3 parts each, four rows one after another
// in a block, took 8 us), and the blocks are few and light enough to be there when the parts are.
constexpr int kJoinWarps = 8, kAtOnce = 4;
__host__ __device__ constexpr int join_share(int parts) {  // warps of a row
  return parts <= kAtOnce ? 1 : parts <= 2 * kAtOnce ? 2 : parts <= 4 * kAtOnce ? 4 : 8;
}

template <int D>
__global__ void __launch_bounds__(kJoinWarps * 32, 4) paged_join_kernel(const __grid_constant__ PagedParams p) {
  constexpr int kPer = D / 32;
  __shared__ __align__(16) float s_o[kJoinWarps][D];
  __shared__ float2 s_ml[kJoinWarps];
  static_assert(kJoinWarps * D >= kJoinWarps * 32 + kJoinWarps, "s_o holds block_places' sums");
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  // (the lengths were complete before the first kernel began, and it let this one start only then)
  constexpr int kThreads = kJoinWarps * 32;
  int* s_pre = reinterpret_cast<int*>(s_o);
  const bool few = p.B <= 256;
  const int total = few ? all_places(p) : block_places<kThreads>(p, s_pre, s_pre + kThreads);
  const int G = min(p.ctas, total), x = static_cast<int>(blockIdx.x);
  const Shares shares(static_cast<uint32_t>(total), static_cast<uint32_t>(G));
  int unit, unit0, tiles;  // its number, first place and tiles
  bool mine = true;
  if (p.by_unit) {
    const int per = p.H_kv * p.n_rg, s = x / per;
    int before = 0;
    for (int r = lane; r < s; r += 32) before += req_places(p, r);
    const int places = req_places(p, s);
    unit = x;
    unit0 = __reduce_add_sync(0xffffffffu, before) * per + (x - s * per) * places;
    tiles = places - p.unit_cost;
  } else {
    Walk w;
    mine = x < G;
    const int place = mine ? shares.start(x) : 0, k = few ? 0 : share_of<kThreads>(s_pre, place);
    unit0 = few ? find(p, place, w)
                : find(p, place, w, k * ((p.B + kThreads - 1) / kThreads), s_pre[k]);
    unit = (w.s * p.H_kv + w.h) * p.n_rg + w.rg;
    tiles = w.n;
    mine = mine && w.t > 0 && w.t < w.n && shares.owner(unit0 + tiles - 1) == x;
  }
  const int i0 = shares.owner(unit0), n = shares.owner(unit0 + tiles - 1) - i0 + 1;
  // the beginning CTA's second part, if it holds tiles of the unit before
  const int second = second_part(shares.start(i0), unit0, p.unit_cost);
  __syncthreads();  // s_pre has been read
  pdl_wait();  // by every block, so that the work after this one waits for the parts' kernel too
  if (!mine || n == 1) return;
  const int rg = unit % p.n_rg, sh = unit / p.n_rg;
  const int row0 = rg * p.rg_rows, rows = min(p.rg_rows, p.group - row0);
  const int share = join_share(n);
  const int side = kJoinWarps / share, sub = warp % share;
  for (int r0 = blockIdx.y * side; r0 < rows; r0 += gridDim.y * side) {
    const int row = r0 + warp / share;
    float acc[kPer], m = -INFINITY, l = 0.f;
    #pragma unroll
    for (int c = 0; c < kPer; ++c) acc[c] = 0.f;
    if (row < rows) {
      // so many parts at a time, against the largest maximum so far
      for (int j0 = sub; j0 < n; j0 += kAtOnce * share) {
        float2 ml[kAtOnce];
        float x[kAtOnce][kPer];
        #pragma unroll
        for (int u = 0; u < kAtOnce; ++u) {
          const int j = j0 + u * share;
          ml[u] = make_float2(-INFINITY, 0.f);
          #pragma unroll
          for (int c = 0; c < kPer; ++c) x[u][c] = 0.f;
          if (j < n) {
            const int64_t at =
                static_cast<int64_t>(2 * (i0 + j) + (j == 0 ? second : 0)) * p.rg_rows + row;
            ml[u] = *reinterpret_cast<const float2*>(p.part_ml + at * 2);
            const float* src = p.part_o + at * D + lane * kPer;
            if constexpr (kPer == 4)
              *reinterpret_cast<float4*>(x[u]) = *reinterpret_cast<const float4*>(src);
            else
              *reinterpret_cast<float2*>(x[u]) = *reinterpret_cast<const float2*>(src);
          }
        }
        float top = m;
        #pragma unroll
        for (int u = 0; u < kAtOnce; ++u) top = fmaxf(top, ml[u].x);
        // a maximum of -inf: nothing, or NaN, which stays
        const float keep = m == -INFINITY ? 1.f : ex2_approx(m - top);
        l *= keep;
        #pragma unroll
        for (int c = 0; c < kPer; ++c) acc[c] *= keep;
        #pragma unroll
        for (int u = 0; u < kAtOnce; ++u) {
          const float wt = ml[u].x == -INFINITY ? 1.f : ex2_approx(ml[u].x - top);
          l = fmaf(wt, ml[u].y, l);
          #pragma unroll
          for (int c = 0; c < kPer; ++c) acc[c] = fmaf(wt, x[u][c], acc[c]);
        }
        m = top;
      }
    }
    if (share > 1) {  // the same for the whole block
      #pragma unroll
      for (int c = 0; c < kPer; ++c) s_o[warp][lane * kPer + c] = acc[c];
      if (lane == 0) s_ml[warp] = make_float2(m, l);
      __syncthreads();
      if (sub == 0) {
        float top = -INFINITY;
        for (int u = 0; u < share; ++u) top = fmaxf(top, s_ml[warp + u].x);
        m = top;
        l = 0.f;
        #pragma unroll
        for (int c = 0; c < kPer; ++c) acc[c] = 0.f;
        for (int u = 0; u < share; ++u) {
          const float2 ml = s_ml[warp + u];
          const float wt = ml.x == -INFINITY ? 1.f : ex2_approx(ml.x - top);
          l = fmaf(wt, ml.y, l);
          #pragma unroll
          for (int c = 0; c < kPer; ++c) acc[c] = fmaf(wt, s_o[warp + u][lane * kPer + c], acc[c]);
        }
      }
      __syncthreads();
    }
    if (sub == 0 && row < rows) {
      const int64_t out = static_cast<int64_t>(sh / p.H_kv) * p.H +
                          static_cast<int64_t>(sh % p.H_kv) * p.group + row0 + row;
      const float inv = 1.f / l;
      __nv_bfloat16* dst = p.o + out * D + lane * kPer;
      if constexpr (kPer == 4)
        *reinterpret_cast<uint2*>(dst) = make_uint2(pack_bf16x2(acc[0] * inv, acc[1] * inv),
                                                    pack_bf16x2(acc[2] * inv, acc[3] * inv));
      else
        *reinterpret_cast<uint32_t*>(dst) = pack_bf16x2(acc[0] * inv, acc[1] * inv);
      if (lane == 0)
        p.lse[out] = l > 0.f || l != l ? (m + log2f(l)) * 0.69314718055994530942f : -INFINITY;
    }
  }
}

template <int D, bool E4M3, int NT, int RW>
cudaError_t launch(const PagedParams& p, int ctas, cudaStream_t stream) {
  using L = PagedCfg<D, E4M3, NT, RW>;
  auto* kernel = paged_kernel<D, E4M3, NT, RW>;
  static std::atomic<uint64_t> attr_done{0};
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  const uint64_t bit = 1ull << (dev & 63);
  if (!(attr_done.load(std::memory_order_acquire) & bit)) {
    e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, L::kDyn);
    if (e != cudaSuccess) return e;
    attr_done.fetch_or(bit, std::memory_order_acq_rel);
  }
  const int most = L::kCtas * 152;
  static_assert(L::kCtas * 152 <= kPagedMaxCtas, "the workspace holds the parts of fewer CTAs");
  if (ctas > most) ctas = most;
  // one join a unit where there are no more units than CTAs, else one a CTA
  const long long units = static_cast<long long>(p.B) * p.H_kv * p.n_rg;
  PagedParams q = p;
  q.ctas = ctas;
  q.unit_cost = NT * RW == 4 ? kPagedMaxCost : 1;
  q.by_unit = units <= ctas;
  const int joins = q.by_unit ? static_cast<int>(units) : ctas;
  // blocks of a join: as many as its rows keep busy at the mean number of parts
  const int blocks = (p.rg_rows * join_share(ctas / joins + 2) + kJoinWarps - 1) / kJoinWarps;
  e = launch_dependent(kernel, dim3(static_cast<unsigned>(ctas)), L::kThreads, L::kDyn, stream, q);
  if (e != cudaSuccess) return e;
  return launch_dependent(paged_join_kernel<D>,
                          dim3(static_cast<unsigned>(joins), static_cast<unsigned>(blocks)),
                          kJoinWarps * 32, 0, stream, q);
}

template <int D, bool E4M3>
cudaError_t launch_rows(const PagedParams& p, int ctas, cudaStream_t stream) {
  if (p.rg_rows <= 8) return launch<D, E4M3, 1, 1>(p, ctas, stream);
  if (p.rg_rows <= 16) return launch<D, E4M3, 2, 1>(p, ctas, stream);
  // Up to 32 rows: two slices of warps, so that the accumulators fit, each reading the tile.  For codes
  // that converts them twice, so at d = 64, where four groups of rows fit one warp, they take that
  // though it spills 300 bytes (32 requests of 8192, 8 K/V heads: 107 us against 140); for bf16 the two are
  // near (98 against 103 us) and the slices' fewer CTAs leave fewer parts to join (37 ragged requests: 17 us
  // against 20).
  if constexpr (D == 64 && E4M3) return launch<D, E4M3, 4, 1>(p, ctas, stream);
  else return launch<D, E4M3, 2, 2>(p, ctas, stream);
}

}  // namespace

cudaError_t launch_fwd_paged(const PagedParams& p, int d, bool e4m3, int max_tiles,
                             cudaStream_t stream) {
  const int ctas = max_tiles < kPagedMaxCtas ? max_tiles : kPagedMaxCtas;
  if (d == 64) return e4m3 ? launch_rows<64, true>(p, ctas, stream) : launch_rows<64, false>(p, ctas, stream);
  return e4m3 ? launch_rows<128, true>(p, ctas, stream) : launch_rows<128, false>(p, ctas, stream);
}

}  // namespace attn
