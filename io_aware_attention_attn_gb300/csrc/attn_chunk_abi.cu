// attn_chunk_abi.cu -- entry points of work over a paged cache beyond one new token a request: argument
// validation and launch of attention of several new tokens, of requests behind a shared prefix, and of the
// kernels that write rows into a cache and read them back.
#include <climits>
#include <cmath>

#include "attn_cache_host.h"
#include "attn_chunk.h"
#include "attn_gb300.h"
#include "attn_gen.h"
#include "attn_host.h"

namespace attn {
namespace {

// Places that a unit takes beside its key tiles: loading the query rows, the first tile's maximum, O out (16 prompts of
// 128 to 4096 tokens, 16 heads: 385 us with 1, 373 with 2).
constexpr int kChunkCost = 2;

// Which of the two kernels takes a request goes by its rows (new tokens times the query heads of a K/V head): up to
// kFewRows the one of warp products, whose time is that of reading K and V, above the one of 256-row products.
// Measured through the public call, 32 requests over 4096 keys, 32 query and 8 K/V heads, d = 128, bf16 / E4M3 pages, us: 4 rows
// 89 / 54, 16 rows 91 / 65, 32 rows 96 / 86 by the first (with the second's empty launch); 80 rows by the second 109 / 142, as
// any up to 256 (by events, 115 / 154, with 99 / 63 for 4 rows by the first).
// Over E4M3 the first takes up to 64, in two units: 33 to 64 rows of 32 requests 150 to 153 us and 149, of 8 requests over 2000
// keys 34 and 41 (bf16: 171 and 108, 32 and 33).
constexpr int kFewRows = 32, kFewRowsE4m3 = 64;
int few_most(const attn_kv_cache& c) { return c.dtype == ATTN_CACHE_E4M3 ? kFewRowsE4m3 : kFewRows; }
constexpr int kOneCtaTiles = 8;  // tiles that a CTA goes through sooner than a second launch joins its parts
enum Kernels { kFew = 1, kMany = 2 };
// Rows of one unit of the first, by how many there can be; a call's units, by the mean of its requests.
int few_group(int64_t rows) { return rows <= 8 ? 8 : rows <= 16 ? 16 : 32; }
int few_rows_of(int64_t rows, int B) { return few_group((rows + B - 1) / B); }
// What the host knows: the tokens in all.  Where they may lie either way both kernels are launched, each taking its own
// requests; requests with more than twice kFewRows rows on average leave the first out (a kernel that finds nothing to do, and its
// join, take 3 to 7 us, and the second kernel is right for any request).
int kernels_for(int64_t rows, int B, int few) {
  if (rows <= few) return kFew;
  return B > 1 && rows <= 2ll * kFewRows * B ? kFew | kMany : kMany;
}
size_t chunk_workspace(int T, int group, int d, const ChunkSizes& z) {
  const size_t few = few_layout(few_group(static_cast<int64_t>(T) * group), d).total;
  return few > z.total ? few : z.total;
}

constexpr int kMostRequests = INT_MAX - 1024;  // the kernels step over them by blocks

// The kernel numbers places in 32 bits and rows and tokens with some room to spare.
bool chunk_sizes_fit(int B, int T, int H, int H_kv, int max_pages, int page_size, const ChunkSizes& z) {
  if (B > kMostRequests || static_cast<int64_t>(T) * H > INT_MAX) return false;
  const int64_t most = static_cast<int64_t>(max_pages) * page_size;
  if (most > INT_MAX - 1024 || T > INT_MAX - 1024 || static_cast<int64_t>(H_kv) * z.n_rg > INT_MAX) return false;
  const int64_t tiles = (most + kChunkTile - 1) / kChunkTile + 1;
  const int64_t rows = static_cast<int64_t>(T) / (2 * z.cta_tokens) + (B < T ? B : T);  // row tiles, at most
  return rows <= INT_MAX / (tiles + kChunkCost) / (static_cast<int64_t>(H_kv) * z.n_rg);
}
// Whether the kernel for few rows can number the places of `rows` rows a K/V head, too: its units are of fewer rows and its
// tiles of fewer keys.
bool few_sizes_fit(int B, int T, int64_t rows, int H_kv, int max_pages, int page_size) {
  const int64_t most = static_cast<int64_t>(max_pages) * page_size, tiles = (most + kPagedTile - 1) / kPagedTile + 1;
  const int64_t units = rows / few_rows_of(rows, B) + (B < T ? B : T);
  return units <= INT_MAX / (tiles + kFewCost) / H_kv;
}

struct QueryLayout {
  int64_t head, token;  // elements from one query head, one token to the next
};

// Launches on checked arguments: of the kernel for few rows,
// (own: the tokens are requests that share a prefix and have rows of their own as well)
struct OwnRows {
  const int32_t* table;
  const int32_t* lens;
  int max_pages;
  float* pair_o;
  float* pair_lse;
};
int run_few(const void* q, const attn_kv_cache& c, const int32_t* table, const int32_t* seq_lens, const int32_t* cu,
            void* o, float* lse, const OwnRows* own, int B, int T, int H, int H_kv, int d, int max_pages, int causal,
            float scale, QueryLayout at, int most_rows, uint8_t* ws, cudaStream_t stream) {
  PagedParams p{};
  const int rc = fill_paged(p, c, H_kv, d, scale);
  if (rc != ATTN_OK) return rc;
  p.group = H / H_kv;
  const int64_t rows = static_cast<int64_t>(T) * p.group;
  p.n_rg = 1;
  p.rg_rows = few_rows_of(rows, B);
  const FewLayout L = few_layout(p.rg_rows, d);
  p.q = static_cast<const __nv_bfloat16*>(q);
  p.o = static_cast<__nv_bfloat16*>(o);
  p.lse = lse;
  p.table = table;
  p.seq_lens = seq_lens;
  p.part_o = reinterpret_cast<float*>(ws + L.o_off);
  p.part_ml = reinterpret_cast<float*>(ws + L.ml_off);
  p.desc = reinterpret_cast<PagedDesc*>(ws + L.desc_off);
  p.head = reinterpret_cast<int*>(ws + L.head_off);
  p.B = B;
  p.H = H;
  p.max_pages = max_pages;
  p.cu = cu;
  p.T = T;
  p.causal = causal;
  p.most_rows = most_rows;
  p.q_head = p.o_head = at.head;
  p.q_token = p.o_token = at.token;
  p.own_first = INT_MAX;
  int64_t most = static_cast<int64_t>(max_pages) * c.page_size;
  int64_t units = (rows / p.rg_rows + (B < T ? B : T)) * H_kv;
  if (own) {
    p.B = B + T;
    p.own_first = B;
    p.own_table = own->table;
    p.own_lens = own->lens;
    p.own_max_pages = own->max_pages;
    p.pair_o = own->pair_o;
    p.pair_lse = own->pair_lse;
    units += static_cast<int64_t>(T) * H_kv;
    if (own->max_pages > max_pages) most = static_cast<int64_t>(own->max_pages) * c.page_size;
  }
  const int64_t tiles = most > 0 ? (most + kPagedTile - 1) / kPagedTile : 1;
  int64_t like = static_cast<int64_t>(B) * H_kv;
  if (own) {  // the own rows' units, by their places
    const int64_t own_tiles = static_cast<int64_t>(own->max_pages) * c.page_size / kPagedTile + 1;
    const int64_t prefix_tiles = static_cast<int64_t>(max_pages) * c.page_size / kPagedTile + 1;
    like += static_cast<int64_t>(T) * H_kv * (own_tiles + kSharedCost) / (prefix_tiles + kSharedCost);
  }
  p.long_units = like < INT_MAX ? static_cast<int>(like) : INT_MAX;
  // One request over a few tiles: a CTA goes through all of a unit's in less time than a second launch takes to join
  // its parts (5 tokens behind 295, 16 query and 4 K/V heads, d = 64: 7.8 us, with the join 13.4).
  p.one_cta = p.B == 1 && tiles <= kOneCtaTiles && units <= kPagedMaxCtas / 4;
  const int64_t places = p.one_cta ? units : units * tiles;
  if (launch_fwd_paged_multi(p, d, c.dtype == ATTN_CACHE_E4M3,
                             places < INT_MAX ? static_cast<int>(places) : INT_MAX, stream) != cudaSuccess)
    return ATTN_ERR_LAUNCH;
  return !own || launch_pair_merge(p, B, d, stream) == cudaSuccess ? ATTN_OK : ATTN_ERR_LAUNCH;
}

// of the one for many,
int run_many(const void* q, const attn_kv_cache& c, const int32_t* table, const int32_t* seq_lens, const int32_t* cu,
              void* o, float* lse, const float* tail_o, const float* tail_lse, int B, int T, int H, int H_kv, int d,
             int max_pages, int causal, float scale, QueryLayout at, int few_rows, const ChunkSizes& z, uint8_t* ws,
             cudaStream_t stream) {
  const bool e4m3 = c.dtype == ATTN_CACHE_E4M3;
  ChunkParams p{};
  p.box_rows = c.page_size < 64 ? c.page_size : 64;
  if (encode_query_map(&p.tm_q, q, d, H, T, at.head * 2, at.token * 2, z.rg_rows, z.cta_tokens) != CUDA_SUCCESS ||
      encode_page_map(&p.tm_k, c.k, e4m3, d, c.page_size, H_kv, c.num_pages, c.page_stride, e4m3 ? d : 64, p.box_rows,
                      false) != CUDA_SUCCESS ||
      encode_page_map(&p.tm_v, c.v, e4m3, d, c.page_size, H_kv, c.num_pages, c.page_stride, 64, p.box_rows, e4m3) !=
          CUDA_SUCCESS)
    return ATTN_ERR_LAUNCH;
  p.cu = cu;
  p.seq_lens = seq_lens;
  p.table = table;
  p.ks = c.k_scale;
  p.vs = c.v_scale;
  p.o = static_cast<__nv_bfloat16*>(o);
  p.lse = lse;
  p.o_head = at.head;
  p.o_token = at.token;
  p.tail_o = tail_o;
  p.tail_lse = tail_lse;
  p.part_o = reinterpret_cast<float*>(ws + z.o_off);
  p.part_ml = reinterpret_cast<float*>(ws + z.ml_off);
  p.desc = reinterpret_cast<ChunkDesc*>(ws + z.desc_off);
  p.head = reinterpret_cast<int*>(ws + z.head_off);
  p.status = status_word();
  if (!p.status) return ATTN_ERR_LAUNCH;
  p.B = B;
  p.T = T;
  p.H = H;
  p.H_kv = H_kv;
  p.group = H / H_kv;
  p.n_rg = z.n_rg;
  p.rg_rows = z.rg_rows;
  p.cta_tokens = z.cta_tokens;
  p.max_pages = max_pages;
  p.num_pages = c.num_pages;
  p.page_shift = log2_of(c.page_size);
  p.part_rows = z.part_rows;
  p.max_rounds = z.rounds;
  p.few_rows = few_rows;
  p.shape = ChunkShape{2 * z.cta_tokens, causal, kChunkCost};
  p.scale_log2 = scale * 1.4426950408889634f;
  // clusters: no more than the largest number of shares that the table's shape allows
  const int64_t most = static_cast<int64_t>(max_pages) * c.page_size;
  const int64_t tiles = (most + kChunkTile - 1) / kChunkTile + 1;
  const int64_t units = (static_cast<int64_t>(T) / (2 * z.cta_tokens) + (B < T ? B : T)) * H_kv * z.n_rg;
  const int64_t shares = units * (tiles + kChunkCost) / kChunkMinShare + 1;
  p.clusters = shares < kChunkClusters ? static_cast<int>(shares) : kChunkClusters;
  return launch_chunk(p, d, e4m3, stream) == cudaSuccess ? ATTN_OK : ATTN_ERR_LAUNCH;
}

// Whether the first takes requests that share prefixes: they are about as many in each group, so one kernel takes them
// all, by their mean, and the first takes each request's own rows in the same launch (12 groups of 4 behind up to 4096
// rows, E4M3: 31 us with launches of their own for those).
bool few_behind_prefix(int groups, int B, int H, int H_kv, int max_prefix_pages, int max_pages, const attn_kv_cache& c) {
  const int64_t rows = static_cast<int64_t>(B) * (H / H_kv);
  if (rows > static_cast<int64_t>(few_most(c)) * groups) return false;
  const int64_t most = static_cast<int64_t>(max_prefix_pages > max_pages ? max_prefix_pages : max_pages) * c.page_size;
  const int64_t units = rows / 8 + (groups < B ? groups : B) + static_cast<int64_t>(B) * (H / H_kv / 8 + 1);
  return units <= INT_MAX / ((most + kPagedTile - 1) / kPagedTile + 1 + kFewCost) / H_kv;  // places in 32 bits
}

size_t up256(size_t x) { return (x + 255) / 256 * 256; }

struct SharedLayout {
  size_t tail_o, tail_lse, chunk, total;  // the paged attention's workspace comes first
};
SharedLayout shared_layout(int B, int H, int group, int d, const ChunkSizes& z) {
  SharedLayout s{};
  s.tail_o = paged_layout(group, d).total;
  s.tail_lse = s.tail_o + up256(2ull * B * H * d * 4);  // (two halves where one launch takes prefixes and own rows)
  s.chunk = s.tail_lse + up256(2ull * B * H * 4);
  s.total = s.chunk + chunk_workspace(B, group, d, z);
  return s;
}

}  // namespace
}  // namespace attn

using namespace attn;

extern "C" size_t attn_fwd_paged_varlen_workspace_bytes(int T, int H, int H_kv, int d) {
  if (T <= 0 || H <= 0 || H_kv <= 0 || H % H_kv != 0 || (d != 64 && d != 128)) return 0;
  return chunk_workspace(T, H / H_kv, d, chunk_sizes(H / H_kv, T, d));
}

extern "C" int attn_fwd_paged_varlen(const void* q, const attn_kv_cache* cache, const int32_t* block_table,
                                     const int32_t* seq_lens, const int32_t* cu_new, void* o, float* lse, int B, int T,
                                     int H, int H_kv, int d, int max_pages, int causal, float scale, void* workspace,
                                     size_t workspace_bytes, void* stream) {
  if (B < 0 || T < 0 || H < 0 || H_kv < 0 || max_pages < 0 || (B == 0 && T > 0)) return ATTN_ERR_SHAPE;
  if (B == 0 || T == 0 || H == 0) return ATTN_OK;
  if (d != 64 && d != 128) return ATTN_ERR_HEAD_DIM;
  if (H_kv == 0 || H % H_kv != 0) return ATTN_ERR_SHAPE;
  if (!q || !cache || !seq_lens || !cu_new || !o || !lse || (max_pages > 0 && !block_table)) return ATTN_ERR_NULL;
  if (!aligned(q, 16) || !aligned(o, 16) || !aligned(lse, 4) || !aligned(block_table, 4) || !aligned(seq_lens, 4) ||
      !aligned(cu_new, 4))
    return ATTN_ERR_ALIGN;
  int rc = check_cache(*cache, H_kv, d);
  if (rc != ATTN_OK) return rc;
  if (!(scale > 0.f) || !std::isfinite(scale)) return ATTN_ERR_SCALE;
  const ChunkSizes z = chunk_sizes(H / H_kv, T, d);
  if (!chunk_sizes_fit(B, T, H, H_kv, max_pages, cache->page_size, z)) return ATTN_ERR_SHAPE;
  if (!workspace || !aligned(workspace, 256) || workspace_bytes < chunk_workspace(T, H / H_kv, d, z))
    return ATTN_ERR_WORKSPACE;
  if ((rc = check_device()) != 0) return rc;
  const QueryLayout at{static_cast<int64_t>(T) * d, d};
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  const int64_t rows = static_cast<int64_t>(T) * (H / H_kv);
  const int few_rows = few_most(*cache);
  // (where only the kernel for many rows can number the places, it takes all requests)
  const int which = few_sizes_fit(B, T, rows, H_kv, max_pages, cache->page_size) ? kernels_for(rows, B, few_rows) : kMany;
  // of both, one after the other on one workspace
  if (which & kFew)
    rc = run_few(q, *cache, block_table, seq_lens, cu_new, o, lse, nullptr, B, T, H, H_kv, d, max_pages, causal != 0, scale,
                 at, which & kMany ? few_rows : INT_MAX, ws, static_cast<cudaStream_t>(stream));
  if (rc == ATTN_OK && (which & kMany))
    rc = run_many(q, *cache, block_table, seq_lens, cu_new, o, lse, nullptr, nullptr, B, T, H, H_kv, d, max_pages,
                  causal != 0, scale, at, which & kFew ? few_rows : 0, z, ws, static_cast<cudaStream_t>(stream));
  return rc;
}

extern "C" size_t attn_fwd_paged_shared_workspace_bytes(int B, int H, int H_kv, int d) {
  if (B <= 0 || H <= 0 || H_kv <= 0 || H % H_kv != 0 || (d != 64 && d != 128)) return 0;
  return shared_layout(B, H, H / H_kv, d, chunk_sizes(H / H_kv, B, d)).total;
}

extern "C" int attn_fwd_paged_shared(const void* q, const attn_kv_cache* cache, const int32_t* prefix_table,
                                     const int32_t* prefix_lens, const int32_t* cu_groups, const int32_t* block_table,
                                     const int32_t* seq_lens, void* o, float* lse, int groups, int B, int H, int H_kv,
                                     int d, int max_prefix_pages, int max_pages, float scale, void* workspace,
                                     size_t workspace_bytes, void* stream) {
  if (groups < 0 || B < 0 || H < 0 || H_kv < 0 || max_prefix_pages < 0 || max_pages < 0 || (groups == 0 && B > 0))
    return ATTN_ERR_SHAPE;
  if (groups == 0 || B == 0 || H == 0) return ATTN_OK;
  if (d != 64 && d != 128) return ATTN_ERR_HEAD_DIM;
  if (H_kv == 0 || H % H_kv != 0) return ATTN_ERR_SHAPE;
  if (!q || !cache || !prefix_lens || !cu_groups || !seq_lens || !o || !lse || (max_prefix_pages > 0 && !prefix_table) ||
      (max_pages > 0 && !block_table))
    return ATTN_ERR_NULL;
  if (!aligned(q, 16) || !aligned(o, 16) || !aligned(lse, 4) || !aligned(prefix_table, 4) || !aligned(prefix_lens, 4) ||
      !aligned(cu_groups, 4) || !aligned(block_table, 4) || !aligned(seq_lens, 4))
    return ATTN_ERR_ALIGN;
  int rc = check_cache(*cache, H_kv, d);
  if (rc != ATTN_OK) return rc;
  if (!(scale > 0.f) || !std::isfinite(scale)) return ATTN_ERR_SCALE;
  const ChunkSizes z = chunk_sizes(H / H_kv, B, d);
  if (groups > kMostRequests - B || !paged_sizes_fit(B, H, H_kv, max_pages, cache->page_size) ||
      !chunk_sizes_fit(groups, B, H, H_kv, max_prefix_pages, cache->page_size, z))
    return ATTN_ERR_SHAPE;
  const SharedLayout s = shared_layout(B, H, H / H_kv, d, z);
  if (!workspace || !aligned(workspace, 256) || workspace_bytes < s.total) return ATTN_ERR_WORKSPACE;
  if ((rc = check_device()) != 0) return rc;
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  float* tail_o = reinterpret_cast<float*>(ws + s.tail_o);
  float* tail_lse = reinterpret_cast<float*>(ws + s.tail_lse);
  const QueryLayout at{d, static_cast<int64_t>(H) * d};
  if (few_behind_prefix(groups, B, H, H_kv, max_prefix_pages, max_pages, *cache)) {
    const OwnRows own{block_table, seq_lens, max_pages, tail_o, tail_lse};
    return run_few(q, *cache, prefix_table, prefix_lens, cu_groups, o, lse, &own, groups, B, H, H_kv, d, max_prefix_pages, 0,
                   scale, at, INT_MAX, ws + s.chunk, static_cast<cudaStream_t>(stream));
  }
  // each request's own rows first, in fp32; the prefix's results are merged with them where they are finished
  rc = run_fwd_paged(q, *cache, block_table, seq_lens, nullptr, tail_o, tail_lse, B, H, H_kv, d, max_pages, scale, ws,
                     static_cast<cudaStream_t>(stream));
  if (rc != ATTN_OK) return rc;
  return run_many(q, *cache, prefix_table, prefix_lens, cu_groups, o, lse, tail_o, tail_lse, groups, B, H, H_kv, d,
                  max_prefix_pages, 0, scale, at, 0, z, ws + s.chunk, static_cast<cudaStream_t>(stream));
}

namespace {

// What writing and reading take alike.
void cache_fields(KvRowsParams& p, const attn_kv_cache& c, int H_kv) {
  p.kc = static_cast<uint8_t*>(c.k);
  p.vc = static_cast<uint8_t*>(c.v);
  p.ks = c.k_scale;
  p.vs = c.v_scale;
  p.page_stride = c.page_stride;
  p.num_pages = c.num_pages;
  p.page_shift = log2_of(c.page_size);
  p.H_kv = H_kv;
}

// Whether strides (elements) keep rows on 16 bytes and their offsets within 64 bits.
bool strides_ok(const int64_t* s, int B, int H, int N) {
  const int64_t n[3] = {B, H, N};
  int64_t left = 1ll << 62;
  for (int i = 0; i < 3; ++i) {
    if (n[i] <= 1) continue;
    if (s[i] < 0 || s[i] % 8 != 0 || s[i] > left / n[i]) return false;
    left -= s[i] * n[i];
  }
  return true;
}

}  // namespace

extern "C" int attn_kv_write(const void* k, const int64_t* k_strides, const void* v, const int64_t* v_strides,
                             const attn_kv_cache* cache, const int64_t* slots, int B, int N, int H_kv, int d,
                             void* stream) {
  if (B < 0 || N < 0 || H_kv < 0) return ATTN_ERR_SHAPE;
  if (B == 0 || N == 0 || H_kv == 0) return ATTN_OK;
  if (d != 64 && d != 128) return ATTN_ERR_HEAD_DIM;
  if (!k || !k_strides || !v || !v_strides || !cache || !slots) return ATTN_ERR_NULL;
  if (static_cast<int64_t>(B) * N > INT_MAX - 1024 || !strides_ok(k_strides, B, H_kv, N) ||
      !strides_ok(v_strides, B, H_kv, N))
    return ATTN_ERR_SHAPE;
  if (!aligned(k, 16) || !aligned(v, 16) || !aligned(slots, 8)) return ATTN_ERR_ALIGN;
  int rc = check_cache(*cache, H_kv, d);
  if (rc != ATTN_OK) return rc;
  if ((rc = check_device()) != 0) return rc;
  KvRowsParams p{};
  cache_fields(p, *cache, H_kv);
  p.k = static_cast<const __nv_bfloat16*>(k);
  p.v = static_cast<const __nv_bfloat16*>(v);
  p.k_batch = k_strides[0];
  p.k_head = k_strides[1];
  p.k_token = k_strides[2];
  p.v_batch = v_strides[0];
  p.v_head = v_strides[1];
  p.v_token = v_strides[2];
  p.slots = slots;
  p.B = B;
  p.N = N;
  p.status = status_word();
  if (!p.status) return ATTN_ERR_LAUNCH;
  return launch_kv_write(p, d, cache->dtype == ATTN_CACHE_E4M3, static_cast<cudaStream_t>(stream)) == cudaSuccess
             ? ATTN_OK
             : ATTN_ERR_LAUNCH;
}

extern "C" int attn_kv_read(const attn_kv_cache* cache, const int32_t* block_table, const int32_t* cu_rows,
                            const int32_t* first, void* k, void* v, int B, int T, int H_kv, int d, int max_pages,
                            void* stream) {
  if (B < 0 || T < 0 || H_kv < 0 || max_pages < 0 || (B == 0 && T > 0)) return ATTN_ERR_SHAPE;
  if (B == 0 || T == 0 || H_kv == 0) return ATTN_OK;
  if (d != 64 && d != 128) return ATTN_ERR_HEAD_DIM;
  if (!cache || !cu_rows || !k || !v || (max_pages > 0 && !block_table)) return ATTN_ERR_NULL;
  if (T > INT_MAX - 1024 || B > kMostRequests) return ATTN_ERR_SHAPE;
  if (!aligned(k, 16) || !aligned(v, 16) || !aligned(block_table, 4) || !aligned(cu_rows, 4) || !aligned(first, 4))
    return ATTN_ERR_ALIGN;
  int rc = check_cache(*cache, H_kv, d);
  if (rc != ATTN_OK) return rc;
  if ((rc = check_device()) != 0) return rc;
  KvRowsParams p{};
  cache_fields(p, *cache, H_kv);
  p.ko = static_cast<__nv_bfloat16*>(k);
  p.vo = static_cast<__nv_bfloat16*>(v);
  p.table = block_table;
  p.cu = cu_rows;
  p.first = first;
  p.max_pages = max_pages;
  p.B = B;
  p.T = T;
  p.status = status_word();
  if (!p.status) return ATTN_ERR_LAUNCH;
  return launch_kv_read(p, d, cache->dtype == ATTN_CACHE_E4M3, static_cast<cudaStream_t>(stream)) == cudaSuccess
             ? ATTN_OK
             : ATTN_ERR_LAUNCH;
}
