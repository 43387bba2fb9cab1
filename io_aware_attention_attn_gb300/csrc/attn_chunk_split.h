// attn_chunk_split.h -- how the attention of several new tokens over pages is shared out, in numbers alone:
// what the kernels and a program on the host take alike.
//
// A unit is a K/V head (or a group of its query heads) and `tokens` consecutive new tokens of a request:
// row tile t.  It takes one place for each tile of kChunkTile keys that its last token sees, one at least, and
// `cost` places more for what its end costs.  All units, in order (request, head, row tile), lie on one line
// of places, which is cut into equal shares (Shares in attn_paged_split.h).
#pragma once

#include "attn_paged_split.h"

namespace attn {

constexpr int kChunkTile = 128;  // keys of a tile

// What a request brings: new tokens n and rows L in the cache (the new ones among them).
struct ChunkReq {
  int n, L;
};
struct ChunkShape {
  int tokens;   // of a row tile
  int causal;
  int cost;
};

// sum of floor((a i + b) / m) over i < n, as lattice points below a line: whole parts out, then the axes
// swapped, as in Euclid's algorithm.  The result and a n + b are below 2^32 (a row of units has fewer than 2^31 places, and
// so, where each row tile sees `tokens` keys more than the one before, fewer than 2^20 that see any).
ATTN_HD uint32_t floor_sum(uint32_t n, uint32_t m, uint32_t a, uint32_t b) {
  uint32_t sum = 0;
#ifdef __CUDACC__
  #pragma unroll 1
#endif
  while (n > 0) {
    if (a >= m) {
      const uint32_t q = a / m;
      sum += static_cast<uint32_t>(static_cast<uint64_t>(n) * (n - 1) / 2) * q;
      a -= q * m;
    }
    if (b >= m) {
      const uint32_t q = b / m;
      sum += n * q;
      b -= q * m;
    }
    const uint32_t y = a * n + b;
    n = y / m;
    b = y - n * m;
    const uint32_t t = m;
    m = a;
    a = t;
  }
  return sum;
}

ATTN_HD int row_tiles(const ChunkReq& r, const ChunkShape& c) { return (r.n + c.tokens - 1) / c.tokens; }
// Keys that the last token of row tile t sees (none: zero or less).
ATTN_HD int keys_seen(const ChunkReq& r, const ChunkShape& c, int t) {
  if (!c.causal) return r.L;
  const int seen = r.L - r.n + (t + 1) * c.tokens;
  return seen < r.L ? seen : r.L;
}
ATTN_HD int key_tiles(const ChunkReq& r, const ChunkShape& c, int t) {
  const int seen = keys_seen(r, c, t);
  return seen > kChunkTile ? (seen + kChunkTile - 1) / kChunkTile : 1;
}
// Places of the row tiles before t of a unit row (t up to row_tiles).
ATTN_HD int places_before(const ChunkReq& r, const ChunkShape& c, int t) {
  if (t <= 0) return 0;
  if (!c.causal) return t * (key_tiles(r, c, 0) + c.cost);
  const int last = row_tiles(r, c) - 1;      // the one that ends with the request's last token
  const int x = t <= last ? t : last;        // of the others, token (t + 1) tokens - 1 sees a + (t + 1) tokens keys
  const int a = r.L - r.n;
  int none = a < 0 ? -a / c.tokens : 0;      // row tiles that see nothing: one tile each
  if (none > x) none = x;
  const int tiles = none + static_cast<int>(floor_sum(static_cast<uint32_t>(x - none), kChunkTile,
                                                      static_cast<uint32_t>(c.tokens),
                                                      static_cast<uint32_t>(a + (none + 1) * c.tokens + kChunkTile - 1)));
  return tiles + x * c.cost + (t > last ? key_tiles(r, c, last) + c.cost : 0);
}
ATTN_HD int unit_row_places(const ChunkReq& r, const ChunkShape& c) {
  return places_before(r, c, row_tiles(r, c));
}

// Rounds: the shares are taken in so many rounds, one a cluster in each, so that the clusters are near one another on
// the line and read the same K and V from L2 while they last: `wide_bytes`, what requests with several row tiles keep in the
// cache over all heads, shared out to rounds of up to 96 MB, where a share stays long beside the parts that its ends
// leave.  (4096 tokens behind 12288, 32 K/V heads, 268 MB: 620 us in one round, 600 in two; 16 prompts of 181 to 3879
// tokens, 16 heads, 277 MB: 356 in one, 373 in two, whose shares are 107 tiles long.)
constexpr int kChunkRounds = 4;
constexpr int kChunkMinShare = 4;   // places of a share, at least
ATTN_HD int chunk_rounds(uint32_t total, int clusters, float wide_bytes, int most) {
  int r = 1;
  while (r < most && wide_bytes > r * 100663296.f && total / (2u * r * clusters) >= 256u) r *= 2;
  return r;
}
ATTN_HD int chunk_shares(uint32_t total, int clusters, int rounds) {
  const uint32_t fit = total / kChunkMinShare, all = static_cast<uint32_t>(clusters) * rounds;
  return static_cast<int>(fit < 1 ? 1 : fit < all ? fit : all);
}

}  // namespace attn
