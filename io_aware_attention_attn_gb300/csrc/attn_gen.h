// attn_gen.h -- launch parameters of the generation path: slots of new tokens, the step before
// attention (norm, rotation, layout, cache write) and its backward, and attention over a paged cache.
#pragma once

#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "attn_gb300.h"

namespace attn {

// kinds of the status word that this path adds (low byte)
enum : int { kStatusNoPage = 4, kStatusBadPage = 5 };

enum : int { kCacheNone = 0, kCacheBf16 = 1, kCacheE4m3 = 2 };  // cache types a kernel is built for

// ------------------------------------------------------------------------------ slots, positions
constexpr int kSlotThreads = 256;
constexpr int kMaxSlotSeqs = 16384;  // two int32 arrays of B in shared memory: 128 KB

struct SlotsParams {
  const int* seq_lens;
  const int* cu_new;
  int* block_table;
  const int* free_pages;
  const int* free_head;
  int64_t* slots;
  int* positions;
  int* seq_lens_out;
  int* free_head_out;
  int* status;
  int B, T, max_pages, n_free, page_size;
};
cudaError_t launch_kv_slots(const SlotsParams& p, cudaStream_t stream);

// --------------------------------------------------------------- norm, rotation, layout, cache
struct RopeParams {
  const __nv_bfloat16* qkv;   // [tokens][ld]
  int64_t ld;
  const __nv_bfloat16* wq;    // norm weights [d] or null
  const __nv_bfloat16* wk;
  float eps;
  const double* inv_freq;     // [rot / 2]
  int rot;
  float rope_scale;
  const int* positions;       // [tokens]
  __nv_bfloat16* q;           // [B][H][N][d] or null
  __nv_bfloat16* k;           // [B][H_kv][N][d] or null
  __nv_bfloat16* v;
  uint8_t* kc;                // cache (forward only)
  uint8_t* vc;
  float* ks;
  float* vs;
  int64_t page_stride;        // elements
  int num_pages, page_shift;
  const int64_t* slots;
  int* status;
  const __nv_bfloat16* dq;    // backward: gradients in
  const __nv_bfloat16* dk;
  const __nv_bfloat16* dv;
  __nv_bfloat16* dqkv;        // [tokens][ld_out]
  int64_t ld_out;
  float* dwq;
  float* dwk;
  float* partial;             // [CTAs][2][d] sums of one CTA's rows
  int N, H, H_kv, tokens;
  int parts;                  // warps that share a token
};
constexpr int kRopeThreads = 256;
constexpr int kRopeBwdCtas = 304;  // at most: 2 on each of 152 SMs
cudaError_t launch_qkv_rope(RopeParams& p, int d, bool interleaved, int cache_kind,
                            cudaStream_t stream);
cudaError_t launch_qkv_rope_bwd(RopeParams& p, int d, bool interleaved, cudaStream_t stream);

// -------------------------------------------------------------------- attention over a paged cache
constexpr int kPagedTile = 64;         // keys of a tile
constexpr int kPagedMaxCtas = 608;     // 4 on each of 152 SMs
constexpr int kPagedMaxCost = 2;       // places that a unit takes beside its tiles, at most
// The same with several rows a request, whose ends take longer (4 requests of 8 tokens over 3000 keys, E4M3: 25 us, with 2
// 29; 100 of 1 to 8 over up to 2000 78 and 89), and behind shared prefixes, where most units are the few own rows of one
// request (64 groups of 4 behind 4000, E4M3: 139 us with 4, 129 with 2; 30 groups of 8 behind 500 60 and 54).
constexpr int kFewCost = 4, kSharedCost = 2;
constexpr float kPagedTrail = 8.f;     // how far a score may pass the reference maximum, in log2 units
constexpr int kPagedMaxRows = 32;      // query rows (heads of one K/V head) of a unit

// What the join of several rows a request knows of a CTA (tiles -1: of no unit): the unit's first place and tiles, its K/V
// head, first row, rows, its request's first token, and whether that is from own_first on.
struct PagedDesc {
  int unit0, tiles, h, row0, rows, tok0, own;
};

struct PagedParams {
  CUtensorMap tm_k;     // 4-D {d, page_size, H_kv, pages}, box {128 bytes of d, box_rows, 1, 1}
  CUtensorMap tm_v;
  CUtensorMap tm_k16;   // the same with boxes of 16 rows
  CUtensorMap tm_v16;
  const __nv_bfloat16* q;
  __nv_bfloat16* o;
  float* o32;           // where the rows go instead of o, unrounded (null: to o)
  float* lse;
  const int* table;
  const int* seq_lens;
  const float* ks;
  const float* vs;
  float* part_o;        // [2 * CTAs][rows][d] unnormalised partial outputs
  float* part_ml;       // [2 * CTAs][rows][2] reference maximum (log2 units), row sum
  int* status;
  int B, H, H_kv, group, n_rg, rg_rows;  // row groups of a K/V head and the rows of one
  int max_pages, num_pages, page_shift, box_rows;
  int ctas;             // of the parts' kernel
  int unit_cost;        // places that a unit takes beside its tiles
  bool by_unit;         // one join a unit, else one a CTA
  // several rows a request and K/V head (launch_fwd_paged_multi)
  const int* cu;        // [B + 1] first token of each request
  int T, causal, most_rows;  // (requests of more rows have no units)
  int64_t q_head, q_token, o_head, o_token;  // elements from one query head, one token to the next
  bool one_cta;         // a unit a CTA, nothing to join (one request of few tiles)
  int long_units;       // how many units of the longest request all units are together, by the shape of the tables
  PagedDesc* desc;      // [CTAs]
  int* head;            // [0] places in all, [1] CTAs with a share
  // Requests that share a prefix: requests from own_first on are the tokens again, one each, over rows of their own;
  // results go unrounded to pair_o [2][T][H][d] and pair_lse [2][T][H], prefixes first (null: to o and lse).
  int own_first, own_max_pages;
  const int* own_table;
  const int* own_lens;
  float* pair_o;
  float* pair_lse;
  float scale_log2;     // scale * log2(e)
  float trail;          // the same before the scale (bf16 cache)
};
struct PagedLayout {
  size_t o_off, ml_off, total;
};
inline int paged_row_groups(int group) {
  return (group + kPagedMaxRows - 1) / kPagedMaxRows;
}
inline PagedLayout paged_layout_rows(size_t rows, int d) {
  auto up = [](size_t x) { return (x + 255) / 256 * 256; };
  PagedLayout L{};
  L.ml_off = up(2 * kPagedMaxCtas * rows * d * 4);
  L.total = L.ml_off + up(2 * kPagedMaxCtas * rows * 2 * 4);
  return L;
}
inline PagedLayout paged_layout(int group, int d) {
  const size_t n_rg = paged_row_groups(group);
  return paged_layout_rows((group + n_rg - 1) / n_rg, d);
}
// With several rows a request: the records of the join behind them.
struct FewLayout : PagedLayout {
  size_t desc_off, head_off;
};
inline FewLayout few_layout(size_t rows, int d) {
  FewLayout L{};
  static_cast<PagedLayout&>(L) = paged_layout_rows(rows, d);
  L.desc_off = L.total;
  L.head_off = (L.desc_off + kPagedMaxCtas * sizeof(PagedDesc) + 255) / 256 * 256;
  L.total = L.head_off + 256;
  return L;
}
cudaError_t launch_fwd_paged(const PagedParams& p, int d, bool e4m3, int max_tiles,
                             cudaStream_t stream);

// The same of units of up to p.rg_rows (8, 16 or 32) rows of a request's tokens; `max_tiles`: places of all units, at most.
cudaError_t launch_fwd_paged_multi(const PagedParams& p, int d, bool e4m3, int max_tiles,
                                   cudaStream_t stream);

// o and lse of tokens 0 .. min(cu[groups], T) - 1 from the two halves of pair_o and pair_lse.
cudaError_t launch_pair_merge(const PagedParams& p, int groups, int d, cudaStream_t stream);

// The sizes that attn_fwd_paged takes, and its launch on checked arguments (attn_gen_abi.cu); with o32 the rows
// go there in fp32 instead of to o.
bool paged_sizes_fit(int B, int H, int H_kv, int max_pages, int page_size);
int run_fwd_paged(const void* q, const attn_kv_cache& cache, const int32_t* block_table,
                  const int32_t* seq_lens, void* o, float* o32, float* lse, int B, int H, int H_kv,
                  int d, int max_pages, float scale, void* workspace, cudaStream_t stream);

// The maps of the cache and what else a launch of either kind takes alike (attn_gen_abi.cu); returns a status.
int fill_paged(PagedParams& p, const attn_kv_cache& cache, int H_kv, int d, float scale);

// Encode the 4-D map of a paged cache's K or V (attn_abi.cu).  Returns a CUresult.
int encode_cache_map(CUtensorMap* map, const void* base, bool e4m3, uint64_t d, uint64_t page_size,
                     uint64_t heads, uint64_t pages, uint64_t page_stride, uint32_t box_rows);

}  // namespace attn
