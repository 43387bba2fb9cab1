// attn_paged_split.h -- how the paged attention's work is shared out, in numbers alone: what the kernels
// and a program on the host take alike.
//
// The tiles of all units (request, K/V head, row group), in order, lie on one line of places, `cost` places
// after each unit's tiles for what its end takes.  The line is cut into equal shares, one a CTA.
#pragma once

#include <cstdint>

#ifdef __CUDACC__
#define ATTN_HD __host__ __device__ __forceinline__
#else
#define ATTN_HD inline
#endif

namespace attn {

// CTA i's share of `total` places among G: starts at i * (total / G) plus one for each earlier CTA of
// the first total % G, which take one place more.
struct Shares {
  uint32_t q, r;
  ATTN_HD Shares(uint32_t total, uint32_t G) : q(total / G), r(total - q * G) {}
  ATTN_HD int start(uint32_t i) const { return static_cast<int>(i * q + (i < r ? i : r)); }
  ATTN_HD int owner(uint32_t place) const {
    const uint32_t big = r * (q + 1);
    return static_cast<int>(place < big ? place / (q + 1) : r + (place - big) / q);
  }
};

// What lies at a place `in` places after its request's first, each unit of which has `places` (its tiles
// and the cost): t past the tiles is in the places after them.
struct UnitAt {
  int h, rg, t;
};
ATTN_HD UnitAt unit_at(uint32_t in, uint32_t places, int n_rg) {
  const uint32_t u = in / places;
  UnitAt a;
  a.t = static_cast<int>(in - u * places);
  a.h = static_cast<int>(n_rg == 1 ? u : u / n_rg);
  a.rg = static_cast<int>(u) - a.h * n_rg;
  return a;
}

// Places that a CTA is through with when it has done tiles [begin, end) of a unit of n.
ATTN_HD int places_done(int begin, int end, int n, int cost) {
  return end - begin + (end == n ? cost : 0);
}

// Whether the CTA whose share starts at `start` and holds the first tile of the unit at `unit0` holds tiles
// of the unit before as well: its part of this one is then its second.
ATTN_HD int second_part(int start, int unit0, int cost) { return start < unit0 - cost ? 1 : 0; }

}  // namespace attn
