// attn_gen_abi.cu -- entry points of the generation path: argument validation and launch of the
// kernels for slots, the step before attention, its backward, and attention over a paged cache.
#include <climits>
#include <cmath>

#include "attn_cache_host.h"
#include "attn_gb300.h"
#include "attn_gen.h"
#include "attn_host.h"

namespace attn {
namespace {

// Checks that attn_qkv_rope and its backward share; fills the common fields.
int rope_common(RopeParams& p, const void* qkv, int64_t ld, const void* wq, const void* wk,
                float eps, const double* inv_freq, int rot, float rope_scale,
                const int32_t* positions, int B, int N, int H, int H_kv, int d) {
  if (d != 64 && d != 128) return ATTN_ERR_HEAD_DIM;
  if (rot < 0 || rot > d || rot % 16 != 0) return ATTN_ERR_SHAPE;
  if (H_kv <= 0 || H % H_kv != 0) return ATTN_ERR_SHAPE;
  const int64_t width = (static_cast<int64_t>(H) + 2 * static_cast<int64_t>(H_kv)) * d;
  if (width > INT_MAX || ld < width || ld % 8 != 0) return ATTN_ERR_SHAPE;
  const int64_t tokens = static_cast<int64_t>(B) * N;
  if (tokens > INT_MAX - 1024 || ld > LLONG_MAX / 4 / tokens) return ATTN_ERR_SHAPE;
  if (!qkv || (rot > 0 && (!inv_freq || !positions))) return ATTN_ERR_NULL;
  if (!aligned(qkv, 16) || !aligned(wq, 16) || !aligned(wk, 16) || !aligned(inv_freq, 8) ||
      !aligned(positions, 4))
    return ATTN_ERR_ALIGN;
  if (!(eps >= 0.f) || !std::isfinite(eps) || !std::isfinite(rope_scale)) return ATTN_ERR_SCALE;
  p.qkv = static_cast<const __nv_bfloat16*>(qkv);
  p.ld = ld;
  p.wq = static_cast<const __nv_bfloat16*>(wq);
  p.wk = static_cast<const __nv_bfloat16*>(wk);
  p.eps = eps;
  p.inv_freq = inv_freq;
  p.rot = rot;
  p.rope_scale = rope_scale;
  p.positions = positions;
  p.N = N;
  p.H = H;
  p.H_kv = H_kv;
  p.tokens = static_cast<int>(tokens);
  return ATTN_OK;
}

}  // namespace

// The kernel numbers tiles, and the places a unit takes beside them, in 32 bits.
bool paged_sizes_fit(int B, int H, int H_kv, int max_pages, int page_size) {
  const int64_t most = static_cast<int64_t>(max_pages) * page_size;
  if (most > INT_MAX - kPagedTile) return false;
  const int64_t units = static_cast<int64_t>(B) * H_kv * paged_row_groups(H / H_kv);
  const int64_t tiles = most > 0 ? (most + kPagedTile - 1) / kPagedTile : 1;
  return static_cast<int64_t>(B) * H <= INT_MAX && units <= INT_MAX / (tiles + kPagedMaxCost);
}

int fill_paged(PagedParams& p, const attn_kv_cache& cache, int H_kv, int d, float scale) {
  const bool e4m3 = cache.dtype == ATTN_CACHE_E4M3;
  p.box_rows = cache.page_size < kPagedTile ? cache.page_size : kPagedTile;
  auto encode = [&](CUtensorMap* map, const void* base, uint32_t rows) {
    return encode_cache_map(map, base, e4m3, d, cache.page_size, H_kv, cache.num_pages,
                            cache.page_stride, rows) == CUDA_SUCCESS;
  };
  if (!encode(&p.tm_k, cache.k, p.box_rows) || !encode(&p.tm_v, cache.v, p.box_rows) ||
      !encode(&p.tm_k16, cache.k, 16) || !encode(&p.tm_v16, cache.v, 16))
    return ATTN_ERR_LAUNCH;
  p.ks = cache.k_scale;
  p.vs = cache.v_scale;
  p.H_kv = H_kv;
  p.num_pages = cache.num_pages;
  p.page_shift = log2_of(cache.page_size);
  p.scale_log2 = scale * 1.4426950408889634f;
  p.trail = kPagedTrail / p.scale_log2;
  p.status = status_word();
  return p.status ? ATTN_OK : ATTN_ERR_LAUNCH;
}

int run_fwd_paged(const void* q, const attn_kv_cache& cache, const int32_t* block_table,
                  const int32_t* seq_lens, void* o, float* o32, float* lse, int B, int H, int H_kv,
                  int d, int max_pages, float scale, void* workspace, cudaStream_t stream) {
  PagedParams p{};
  const int rc = fill_paged(p, cache, H_kv, d, scale);
  if (rc != ATTN_OK) return rc;
  const int group = H / H_kv;
  const PagedLayout L = paged_layout(group, d);
  p.q = static_cast<const __nv_bfloat16*>(q);
  p.o = static_cast<__nv_bfloat16*>(o);
  p.o32 = o32;
  p.lse = lse;
  p.table = block_table;
  p.seq_lens = seq_lens;
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  p.part_o = reinterpret_cast<float*>(ws + L.o_off);
  p.part_ml = reinterpret_cast<float*>(ws + L.ml_off);
  p.B = B;
  p.H = H;
  p.group = group;
  p.n_rg = paged_row_groups(group);
  p.rg_rows = (group + p.n_rg - 1) / p.n_rg;
  p.max_pages = max_pages;
  const int64_t most = static_cast<int64_t>(max_pages) * cache.page_size;
  const int64_t tiles = most > 0 ? (most + kPagedTile - 1) / kPagedTile : 1;
  const int64_t units = static_cast<int64_t>(B) * H_kv * p.n_rg;
  return launch_fwd_paged(p, d, cache.dtype == ATTN_CACHE_E4M3, static_cast<int>(units * tiles),
                          stream) == cudaSuccess
             ? ATTN_OK
             : ATTN_ERR_LAUNCH;
}

}  // namespace attn

using namespace attn;

extern "C" int attn_kv_slots(const int32_t* seq_lens, const int32_t* cu_new, int32_t* block_table,
                             const int32_t* free_pages, const int32_t* free_head, int64_t* slots,
                             int32_t* positions, int32_t* seq_lens_out, int32_t* free_head_out,
                             int B, int T, int max_pages, int n_free, int page_size,
                             void* stream) {
  if (B < 0 || T < 0 || max_pages < 0 || n_free < 0 || B > kMaxSlotSeqs || page_size < 1 ||
      page_size > 65536)
    return ATTN_ERR_SHAPE;
  if (B == 0) return T > 0 ? ATTN_ERR_SHAPE : ATTN_OK;  // tokens but no requests
  if (!seq_lens || !cu_new || !free_head || !seq_lens_out || !free_head_out ||
      (max_pages > 0 && !block_table) || (n_free > 0 && !free_pages) ||
      (T > 0 && (!slots || !positions)))
    return ATTN_ERR_NULL;
  if (!aligned(seq_lens, 4) || !aligned(cu_new, 4) || !aligned(block_table, 4) ||
      !aligned(free_pages, 4) || !aligned(free_head, 4) || !aligned(slots, 8) ||
      !aligned(positions, 4) || !aligned(seq_lens_out, 4) || !aligned(free_head_out, 4))
    return ATTN_ERR_ALIGN;
  if (seq_lens_out == seq_lens || free_head_out == free_head) return ATTN_ERR_UNSUPPORTED;
  const int rc = check_device();
  if (rc != 0) return rc;
  SlotsParams p{seq_lens, cu_new, block_table, free_pages, free_head, slots, positions,
                seq_lens_out, free_head_out, status_word(), B, T, max_pages, n_free, page_size};
  if (!p.status) return ATTN_ERR_LAUNCH;
  return launch_kv_slots(p, static_cast<cudaStream_t>(stream)) == cudaSuccess ? ATTN_OK
                                                                             : ATTN_ERR_LAUNCH;
}

extern "C" int attn_qkv_rope(const void* qkv, int64_t ld, const void* wq, const void* wk, float eps,
                             const double* inv_freq, int rot, int interleaved, float rope_scale,
                             const int32_t* positions, void* q, void* k, void* v,
                             const attn_kv_cache* cache, const int64_t* slots, int B, int N, int H,
                             int H_kv, int d, void* stream) {
  if (B < 0 || N < 0 || H < 0 || H_kv < 0) return ATTN_ERR_SHAPE;
  if (B == 0 || N == 0 || H == 0) return ATTN_OK;
  RopeParams p{};
  int rc = rope_common(p, qkv, ld, wq, wk, eps, inv_freq, rot, rope_scale, positions, B, N, H, H_kv,
                       d);
  if (rc != ATTN_OK) return rc;
  if ((k == nullptr) != (v == nullptr) || (cache && !slots)) return ATTN_ERR_NULL;
  if (!aligned(q, 16) || !aligned(k, 16) || !aligned(v, 16) || !aligned(slots, 8))
    return ATTN_ERR_ALIGN;
  int kind = kCacheNone;
  if (cache) {
    if ((rc = check_cache(*cache, H_kv, d)) != ATTN_OK) return rc;
    kind = cache->dtype == ATTN_CACHE_E4M3 ? kCacheE4m3 : kCacheBf16;
    p.kc = static_cast<uint8_t*>(cache->k);
    p.vc = static_cast<uint8_t*>(cache->v);
    p.ks = cache->k_scale;
    p.vs = cache->v_scale;
    p.page_stride = cache->page_stride;
    p.num_pages = cache->num_pages;
    p.page_shift = log2_of(cache->page_size);
    p.slots = slots;
  }
  if (!q && !k && !cache) return ATTN_OK;
  if ((rc = check_device()) != 0) return rc;
  p.q = static_cast<__nv_bfloat16*>(q);
  p.k = static_cast<__nv_bfloat16*>(k);
  p.v = static_cast<__nv_bfloat16*>(v);
  p.status = status_word();
  if (!p.status) return ATTN_ERR_LAUNCH;
  return launch_qkv_rope(p, d, interleaved != 0, kind, static_cast<cudaStream_t>(stream)) ==
                 cudaSuccess
             ? ATTN_OK
             : ATTN_ERR_LAUNCH;
}

extern "C" size_t attn_qkv_rope_bwd_workspace_bytes(int B, int N, int H, int H_kv, int d) {
  if (B <= 0 || N <= 0 || H <= 0 || H_kv <= 0 || (d != 64 && d != 128)) return 0;
  return static_cast<size_t>(kRopeBwdCtas) * 2 * d * 4;
}

extern "C" int attn_qkv_rope_bwd(const void* dq, const void* dk, const void* dv, const void* qkv,
                                 int64_t ld, const void* wq, const void* wk, float eps,
                                 const double* inv_freq, int rot, int interleaved,
                                 float rope_scale, const int32_t* positions, void* dqkv,
                                 int64_t ld_out, float* dwq, float* dwk, int B, int N, int H,
                                 int H_kv, int d, void* workspace, size_t workspace_bytes,
                                 void* stream) {
  if (B < 0 || N < 0 || H < 0 || H_kv < 0) return ATTN_ERR_SHAPE;
  if (B == 0 || N == 0 || H == 0) return ATTN_OK;
  RopeParams p{};
  int rc = rope_common(p, qkv, ld, wq, wk, eps, inv_freq, rot, rope_scale, positions, B, N, H, H_kv,
                       d);
  if (rc != ATTN_OK) return rc;
  const int64_t width = (static_cast<int64_t>(H) + 2 * H_kv) * d;
  if (ld_out < width || ld_out % 8 != 0 || ld_out > LLONG_MAX / 4 / p.tokens) return ATTN_ERR_SHAPE;
  if (!dq || !dk || !dv || !dqkv || (wq && !dwq) || (wk && !dwk)) return ATTN_ERR_NULL;
  if (!aligned(dq, 16) || !aligned(dk, 16) || !aligned(dv, 16) || !aligned(dqkv, 16) ||
      !aligned(dwq, 4) || !aligned(dwk, 4))
    return ATTN_ERR_ALIGN;
  if (wq || wk) {
    if (!workspace || !aligned(workspace, 256) ||
        workspace_bytes < attn_qkv_rope_bwd_workspace_bytes(B, N, H, H_kv, d))
      return ATTN_ERR_WORKSPACE;
    p.partial = static_cast<float*>(workspace);
  }
  if ((rc = check_device()) != 0) return rc;
  p.dq = static_cast<const __nv_bfloat16*>(dq);
  p.dk = static_cast<const __nv_bfloat16*>(dk);
  p.dv = static_cast<const __nv_bfloat16*>(dv);
  p.dqkv = static_cast<__nv_bfloat16*>(dqkv);
  p.ld_out = ld_out;
  p.dwq = wq ? dwq : nullptr;
  p.dwk = wk ? dwk : nullptr;
  return launch_qkv_rope_bwd(p, d, interleaved != 0, static_cast<cudaStream_t>(stream)) ==
                 cudaSuccess
             ? ATTN_OK
             : ATTN_ERR_LAUNCH;
}

extern "C" size_t attn_fwd_paged_workspace_bytes(int B, int H, int H_kv, int d) {
  if (B <= 0 || H <= 0 || H_kv <= 0 || H % H_kv != 0 || (d != 64 && d != 128)) return 0;
  return paged_layout(H / H_kv, d).total;
}

extern "C" int attn_fwd_paged(const void* q, const attn_kv_cache* cache, const int32_t* block_table,
                              const int32_t* seq_lens, void* o, float* lse, int B, int H, int H_kv,
                              int d, int max_pages, float scale, void* workspace,
                              size_t workspace_bytes, void* stream) {
  if (B < 0 || H < 0 || H_kv < 0 || max_pages < 0) return ATTN_ERR_SHAPE;
  if (B == 0 || H == 0) return ATTN_OK;
  if (d != 64 && d != 128) return ATTN_ERR_HEAD_DIM;
  if (H_kv == 0 || H % H_kv != 0) return ATTN_ERR_SHAPE;
  if (!q || !cache || !seq_lens || !o || !lse || (max_pages > 0 && !block_table))
    return ATTN_ERR_NULL;
  if (!aligned(q, 16) || !aligned(o, 16) || !aligned(lse, 4) || !aligned(block_table, 4) ||
      !aligned(seq_lens, 4))
    return ATTN_ERR_ALIGN;
  int rc = check_cache(*cache, H_kv, d);
  if (rc != ATTN_OK) return rc;
  if (!(scale > 0.f) || !std::isfinite(scale)) return ATTN_ERR_SCALE;
  const int group = H / H_kv;
  if (!paged_sizes_fit(B, H, H_kv, max_pages, cache->page_size)) return ATTN_ERR_SHAPE;
  if (!workspace || !aligned(workspace, 256) || workspace_bytes < paged_layout(group, d).total)
    return ATTN_ERR_WORKSPACE;
  if ((rc = check_device()) != 0) return rc;
  return run_fwd_paged(q, *cache, block_table, seq_lens, o, nullptr, lse, B, H, H_kv, d, max_pages,
                       scale, workspace, static_cast<cudaStream_t>(stream));
}
