// attn_gen.h -- launch parameters of the generation path: slots of new tokens, the step before
// attention (norm, rotation, layout, cache write) and its backward, and attention over a paged cache.
#pragma once

#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cstdint>

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
constexpr float kPagedTrail = 8.f;     // how far a score may pass the reference maximum, in log2 units
constexpr int kPagedMaxRows = 32;      // query rows (heads of one K/V head) of a unit

struct PagedParams {
  CUtensorMap tm_k;     // 4-D {d, page_size, H_kv, pages}, box {128 bytes of d, box_rows, 1, 1}
  CUtensorMap tm_v;
  CUtensorMap tm_k16;   // the same with boxes of 16 rows
  CUtensorMap tm_v16;
  const __nv_bfloat16* q;
  __nv_bfloat16* o;
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
  float scale_log2;     // scale * log2(e)
  float trail;          // the same before the scale (bf16 cache)
};
struct PagedLayout {
  size_t o_off, ml_off, total;
};
inline int paged_row_groups(int group) {
  return (group + kPagedMaxRows - 1) / kPagedMaxRows;
}
inline PagedLayout paged_layout(int group, int d) {
  const size_t n_rg = paged_row_groups(group);
  const size_t rows = (group + n_rg - 1) / n_rg;
  auto up = [](size_t x) { return (x + 255) / 256 * 256; };
  PagedLayout L{};
  L.ml_off = up(2 * kPagedMaxCtas * rows * d * 4);
  L.total = L.ml_off + up(2 * kPagedMaxCtas * rows * 2 * 4);
  return L;
}
cudaError_t launch_fwd_paged(const PagedParams& p, int d, bool e4m3, int max_tiles,
                             cudaStream_t stream);

// Encode the 4-D map of a paged cache's K or V (attn_abi.cu).  Returns a CUresult.
int encode_cache_map(CUtensorMap* map, const void* base, bool e4m3, uint64_t d, uint64_t page_size,
                     uint64_t heads, uint64_t pages, uint64_t page_stride, uint32_t box_rows);

}  // namespace attn
