// attn_chunk.h -- launch parameters and shared-memory layout of attention of several query rows a K/V head
// over a paged cache (new tokens of a request; requests that share a prefix), and of the kernels that write rows
// into a cache and read them back.
#pragma once

#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "attn_chunk_split.h"

namespace attn {

constexpr int kChunkRows = 128;      // query rows of a CTA; a unit has two CTAs' worth
constexpr int kChunkClusters = 76;   // CTA pairs at once, at most
constexpr int kChunkMaxShares = kChunkClusters * kChunkRounds;
constexpr int kChunkStagesK = 4, kChunkStagesV = 4, kChunkSBufs = 3;
constexpr int kChunkRawV = 3, kChunkStagesV8 = 3, kChunkScales = 4, kChunkRowDepth = 8;  // E4M3

// Where a share begins: request, unit of it (K/V head, row group), row tile, key tile, places of the share,
// and the request's new tokens, first token and rows.
struct ChunkStart {
  int s, u, t, j, left, n, tok0, L;
};
// What the producer tells the other warps of the unit, or the share's part of it, that comes next.
struct ChunkUnit {
  int j, j_end, n, L;    // its key tiles (j -1: nothing comes), those of the whole unit, rows of the request
  int z, head0;          // K/V head, first query head within its group
  int tok, n_tok, pos0;  // first token, tokens, rows of the request before the first
  int slot;              // of the workspace, if it is a part
};
// As many of them: the producer is at most three units ahead of the issue of the scores (E4M3), which is at most three
// tiles, so three units, ahead of the softmax.
constexpr int kChunkUnits = 8;
// Units whose statistics are kept: the softmax is at most three tiles ahead of a unit whose O is not stored.
constexpr int kChunkStats = 4;
// What the join knows of a share: the unit it begins inside (tiles -1: none that it ends).
struct ChunkDesc {
  int unit0, tiles;         // the unit's first place, its key tiles
  int u, tok, n_tok, pad;   // its K/V head and row group, first token, tokens
};

struct ChunkParams {
  CUtensorMap tm_q;      // {d, H, tokens}, box {64, rows of a row group, tokens of a CTA}
  CUtensorMap tm_k;      // cache: {d, page_size, H_kv, pages}, box_rows rows of 128 bytes (64 for codes of d = 64)
  CUtensorMap tm_v;      // boxes of 64 columns
  const int* cu;         // [B + 1] first token of each request
  const int* seq_lens;   // [B] rows in the cache
  const int* table;      // [B][max_pages]
  const float* ks;
  const float* vs;
  __nv_bfloat16* o;
  float* lse;
  int64_t o_head, o_token;      // elements from one head, one token to the next; lse: the same over d
  const float* tail_o;   // fp32 rows [tokens][H][d] to merge with (null: none), and their log-sum-exp [tokens][H]
  const float* tail_lse;
  float* part_o;         // [2 * shares][d / 4][part_rows][4] unnormalised partial outputs
  float* part_ml;        // [2 * shares][part_rows][2] reference maximum (log2 units), row sum
  ChunkDesc* desc;       // [shares]
  int* head;             // [0] places in all, [1] shares
  int* status;
  int B, T, H, H_kv, group, n_rg, rg_rows;
  int cta_tokens;        // tokens of a CTA's rows
  int max_pages, num_pages, page_shift, box_rows;
  int part_rows, clusters, max_rounds;
  int few_rows;          // requests of so many rows a K/V head or fewer have no units here
  ChunkShape shape;
  float scale_log2;
};

struct ChunkSizes {
  int n_rg, rg_rows, cta_tokens, part_rows, rounds;
  size_t o_off, ml_off, desc_off, head_off, total;
};
inline ChunkSizes chunk_sizes(int group, int T, int d) {
  ChunkSizes z{};
  z.n_rg = (group + kChunkRows - 1) / kChunkRows;
  z.rg_rows = (group + z.n_rg - 1) / z.n_rg;
  z.cta_tokens = kChunkRows / z.rg_rows;
  // a unit's rows in the workspace: the second CTA's only where some unit can have them
  z.part_rows = T <= z.cta_tokens ? T * z.rg_rows : 2 * kChunkRows;
  // one row tile a request at most: nothing is read twice
  z.rounds = T <= 2 * z.cta_tokens ? 1 : kChunkRounds;
  auto up = [](size_t x) { return (x + 255) / 256 * 256; };
  const size_t parts = 2ull * kChunkClusters * z.rounds;
  z.ml_off = up(parts * z.part_rows * d * 4);
  z.desc_off = z.ml_off + up(parts * z.part_rows * 8);
  z.head_off = z.desc_off + up(sizeof(ChunkDesc) * kChunkClusters * z.rounds);
  z.total = z.head_off + 256;
  return z;
}

template <int D, bool E4M3>
struct ChunkLayout {
  static constexpr int kWarps = E4M3 ? 20 : 16;  // three issue, one idles, eight softmax, four store; E4M3: four convert
  static constexpr int kThreads = kWarps * 32;
  static constexpr int SK = kChunkStagesK;
  static constexpr int SV = E4M3 ? kChunkStagesV8 : kChunkStagesV;
  static constexpr int kQRaw = kChunkRows * D * 2;                     // a CTA's query rows
  static constexpr int kQBytes = kChunkRows * D * 2;                   // E4M3: two pieces of D bytes a row
  static constexpr int kKBytes = 64 * D * (E4M3 ? 1 : 2);              // 64 keys of a tile
  static constexpr int kVBytes = kChunkTile * 64 * 2;                  // 64 value columns of a tile
  static constexpr int kLand = 0;                                      // E4M3: where query rows arrive
  static constexpr int kQ = E4M3 ? kQRaw : 0;                          // [2]
  static constexpr int kK = kQ + 2 * kQBytes;
  static constexpr int kV = kK + SK * kKBytes;
  static constexpr int kOut = kV + SV * kVBytes;                       // [4 warps][32 rows x 64 bytes]
  static constexpr int kStats = kOut + 4 * 2048;                       // [4][sums of two halves, maximum][128]
  static constexpr int kVRaw = kStats + kChunkStats * 1536;                        // E4M3: codes of 64 value columns
  static constexpr int kScale = kVRaw + (E4M3 ? kChunkRawV * 8192 : 0);   // [stage][K, V][128] fp32
  static constexpr int kRow = kScale + (E4M3 ? kChunkScales * 1024 : 0);  // [8][128] factors of query rows
  static constexpr int kPair = kRow + (E4M3 ? kChunkRowDepth * 512 : 0);  // [8 warps][32] for the other warp of a row
  static constexpr int kStart = kPair + 1024;
  static constexpr int kUnits = kStart + kChunkRounds * 32;
  static constexpr int kBar = kUnits + kChunkUnits * static_cast<int>(sizeof(ChunkUnit));
  enum {
    bQF = 0,             // query rows ready in both CTAs (leader)          [2]
    bQE = bQF + 2,       // query buffer free (both)                        [2]
    bKF = bQE + 2,       // K stage full (leader)                           [SK]
    bKE = bKF + SK,      // K stage free (both)                             [SK]
    bVF = bKE + SK,      // V stage full (leader)                           [SV]
    bVE = bVF + SV,      // V stage free (both)                             [SV]
    bSF = bVE + SV,      // scores in buffer b (both)                       [3]
    bPF = bSF + kChunkSBufs,   // probabilities in buffer b (leader)        [3]
    bPV = bPF + kChunkSBufs,   // P V from buffer b done (both)             [3]
    bOD = bPV + kChunkSBufs,   // a unit's last P V done (both)
    bOE = bOD + 1,             // O read by the epilogue (leader)
    bDR = bOE + 1,             // drain after an abort, one an issuer       [2]
    bLF = bDR + 2,             // E4M3: query rows arrived (own CTA)
    bLE = bLF + 1,             //       and have been converted
    bRF = bLE + 1,             // V codes arrived (own CTA)                 [3]
    bRE = bRF + kChunkRawV,    //   and have been converted
    bCF = bRE + kChunkRawV,    // scales arrived (own CTA)                  [4]
    bCE = bCF + kChunkScales,  //   and have been read
    bUF = bCE + kChunkScales,  // a unit is told (own CTA)                  [8]
    bEL = bUF + kChunkUnits,   // a unit's statistics are there (own CTA)   [4]
    kNumBars = bEL + kChunkStats
  };
  static constexpr int kMisc = kBar + kNumBars * 8;  // [0] tensor memory [1] abort [2] rounds [3] shares
  static constexpr int kBytes = kMisc + 32;
  static constexpr int kDyn = kBytes + 1024;
  static_assert(kK % 1024 == 0 && kV % 1024 == 0 && kOut % 1024 == 0, "swizzled areas sit on 1024 bytes");
  static_assert(kDyn <= 232448, "more than an SM's shared memory");
};

cudaError_t launch_chunk(const ChunkParams& p, int d, bool e4m3, cudaStream_t stream);

// 3-D map of query rows {d, heads, tokens} with the given strides in bytes, box {64, heads, tokens}; 4-D map
// of a cache with boxes of `cols` elements (128 or 64 bytes, swizzled as wide; `flat`: not swizzled).
int encode_query_map(CUtensorMap* map, const void* base, uint64_t d, uint64_t heads, uint64_t tokens,
                     uint64_t head_bytes, uint64_t token_bytes, uint32_t box_heads, uint32_t box_tokens);
int encode_page_map(CUtensorMap* map, const void* base, bool e4m3, uint64_t d, uint64_t page_size,
                    uint64_t heads, uint64_t pages, uint64_t page_stride, uint32_t cols, uint32_t box_rows,
                    bool flat);

// ------------------------------------------------------------- rows into a cache and back
struct KvRowsParams {
  const __nv_bfloat16* k;       // write: rows in
  const __nv_bfloat16* v;
  int64_t k_batch, k_head, k_token, v_batch, v_head, v_token;  // elements
  __nv_bfloat16* ko;            // read: rows out [H_kv][T][d]
  __nv_bfloat16* vo;
  uint8_t* kc;
  uint8_t* vc;
  float* ks;
  float* vs;
  int64_t page_stride;          // elements
  int num_pages, page_shift, max_pages;
  const int64_t* slots;         // write
  const int* cu;                // read
  const int* first;
  const int* table;
  int* status;
  int B, N, T, H_kv;
};
cudaError_t launch_kv_write(const KvRowsParams& p, int d, bool e4m3, cudaStream_t stream);
cudaError_t launch_kv_read(const KvRowsParams& p, int d, bool e4m3, cudaStream_t stream);

}  // namespace attn
