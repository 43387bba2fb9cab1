// attn_kv_rows.cu -- rows of K and V into a paged cache at given slots, and the rows of requests back out of it.
//
// Both are one pass: a token's place in the cache is found once a block and token (its slot; or its request, by
// halves, and that request's page), then D/8 lanes take a row, 16 bytes of bf16 each, four tokens' K and V at a
// time, so a thread has up to eight loads of 16 bytes in flight.  HBM bounds them.
// An E4M3 row: scale = amax / 448 (1 where that is below fp32's normal range), code = E4M3
// round-to-nearest-even of the fp32 quotient x / scale, as the step before attention stores it.
#include <type_traits>

#include "attn_chunk.h"
#include "attn_gen.cuh"
#include "attn_gen.h"
#include "sm103_ptx.cuh"

namespace attn {
namespace {

constexpr int kThreads = 256, kDeep = 4;  // (writing E4M3 rows takes its eight rows of a lane together)

__device__ __forceinline__ uint32_t max_bf16x2(uint32_t a, uint32_t b) {  // (a NaN gives way to a number)
  uint32_t r;
  asm("max.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}

// The largest magnitude in each of eight rows, of which this lane (one of D/8 that hold a row together) has x[0..7]: the
// lanes hand each other half of the rows in each step, so lane i is left with row i % 8 alone (8 steps across lanes
// instead of 32).
template <int D>
__device__ __forceinline__ float amax_of_rows(const uint4 (&x)[8], int i) {
  uint32_t m[8];
  #pragma unroll
  for (int r = 0; r < 8; ++r)
    m[r] = max_bf16x2(max_bf16x2(x[r].x & 0x7fff7fffu, x[r].y & 0x7fff7fffu),
                      max_bf16x2(x[r].z & 0x7fff7fffu, x[r].w & 0x7fff7fffu));
  #pragma unroll
  for (int bit = 4; bit > 0; bit >>= 1) {  // rows with this bit of their number go to the lanes that have it
    const bool up = i & bit;
    #pragma unroll
    for (int r = 0; r < bit; ++r) {
      const uint32_t keep = up ? m[r + bit] : m[r], give = up ? m[r] : m[r + bit];
      m[r] = max_bf16x2(keep, __shfl_xor_sync(0xffffffffu, give, bit));
    }
  }
  if (D == 128) m[0] = max_bf16x2(m[0], __shfl_xor_sync(0xffffffffu, m[0], 8));
  return fmaxf(bf16lo_to_f32(m[0]), bf16hi_to_f32(m[0]));
}

// 8 bf16 values -> 8 codes of x / sc rounded to nearest fp32, from rc = RN(1 / sc) and one remainder correction
// (Markstein's method, as in the quantizer of attn_fp8.cu, whose check covers every bf16 x and scale that a bf16 row can
// have), two at a time; the sign of a value that rounds to zero is x's.
__device__ __forceinline__ uint2 quantize(const uint4& x, float sc, float rc) {
  const uint32_t v[4] = {x.x, x.y, x.z, x.w};
  const bool fast = sc >= 0x1p-100f && sc <= 0x1p100f;
  uint32_t c[4];
  #pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float a = bf16lo_to_f32(v[i]), b = bf16hi_to_f32(v[i]);
    float q0, q1, r0, r1;
    fmul2(q0, q1, a, b, rc, rc);
    ffma2(r0, r1, -sc, -sc, q0, q1, a, b);
    ffma2(q0, q1, r0, r1, rc, rc, q0, q1);
    c[i] = pack_e4m3x2(q0, q1);
  }
  if (!fast) {
    #pragma unroll
    for (int i = 0; i < 4; ++i)
      c[i] = pack_e4m3x2(__fdiv_rn(bf16lo_to_f32(v[i]), sc), __fdiv_rn(bf16hi_to_f32(v[i]), sc));
  }
  uint32_t out[2];
  #pragma unroll
  for (int i = 0; i < 2; ++i)
    out[i] = ((c[2 * i] | c[2 * i + 1] << 16) & 0x7f7f7f7fu) | (__byte_perm(v[2 * i], v[2 * i + 1], 0x7531) & 0x80808080u);
  return make_uint2(out[0], out[1]);
}

// x y, of 28 significant bits here, as the fp32 number that rounds to bf16 as it does: of the two around it the odd one (no
// middle of two bf16 numbers is odd), itself where it is one.
__device__ __forceinline__ float mul_odd(float x, float y) {
  const float lo = __fmul_rd(x, y), hi = __fmul_ru(x, y);
  return (__float_as_uint(lo) & 1u) ? lo : hi;
}

// 8 codes x scale -> 8 bf16 values
__device__ __forceinline__ uint4 dequantize(const uint2& codes, float sc) {
  uint32_t out[4];
  #pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint32_t h = e4m3x2_to_f16x2((i < 2 ? codes.x : codes.y) >> (16 * (i & 1)));
    float lo, hi;
    asm("{\n\t.reg .b16 a, b;\n\tmov.b32 {a, b}, %2;\n\tcvt.f32.f16 %0, a;\n\tcvt.f32.f16 %1, b;\n\t}"
        : "=f"(lo), "=f"(hi)
        : "r"(h));
    out[i] = pack_bf16x2(mul_odd(lo, sc), mul_odd(hi, sc));
  }
  return make_uint4(out[0], out[1], out[2], out[3]);
}

// A token's page and row of it; page -1: none, -2: not this call's to touch.
struct Place {
  int page, row;
};

template <int D, bool E4M3>
__global__ void __launch_bounds__(kThreads, 4) kv_write_kernel(const __grid_constant__ KvRowsParams p) {
  constexpr int kLanes = D / 8, kGroups = kThreads / kLanes, kTokens = kGroups * kDeep;
  __shared__ Place s_place[kTokens];
  pdl_wait();
  const int64_t tokens = static_cast<int64_t>(p.B) * p.N, t0 = static_cast<int64_t>(blockIdx.x) * kTokens;
  const int64_t most = static_cast<int64_t>(p.num_pages) << p.page_shift;
  for (int i = threadIdx.x; i < kTokens; i += kThreads) {
    Place at{-1, 0};
    if (t0 + i < tokens) {
      const int64_t slot = p.slots[t0 + i];
      if (slot >= most) atomicCAS(p.status, 0, kStatusBadPage);
      if (slot >= 0 && slot < most)
        at = Place{static_cast<int>(slot >> p.page_shift), static_cast<int>(slot & ((1 << p.page_shift) - 1))};
    }
    s_place[i] = at;
  }
  __syncthreads();
  const int group = threadIdx.x / kLanes, c = threadIdx.x % kLanes, lane = threadIdx.x & 31;
  for (int h = blockIdx.y; h < p.H_kv; h += gridDim.y) {
    uint4 x[2 * kDeep];  // K rows of the four tokens, then V rows
    Place at[kDeep];
    #pragma unroll
    for (int u = 0; u < kDeep; ++u) {
      const int i = group + u * kGroups;
      at[u] = s_place[i];
      x[u] = x[kDeep + u] = make_uint4(0, 0, 0, 0);
      if (at[u].page >= 0) {
        const int64_t t = t0 + i, b = p.N == 1 ? t : p.B == 1 ? 0 : t / p.N, n = t - b * p.N;
        x[u] = *reinterpret_cast<const uint4*>(p.k + b * p.k_batch + h * p.k_head + n * p.k_token + 8 * c);
        x[kDeep + u] = *reinterpret_cast<const uint4*>(p.v + b * p.v_batch + h * p.v_head + n * p.v_token + 8 * c);
      }
    }
    float sc = 1.f, rc = 1.f;
    if constexpr (E4M3) {  // of row c % 8
      const float amax = amax_of_rows<D>(x, c);
      sc = __fdiv_rn(amax, 448.f);
      if (!(sc >= 0x1p-126f)) sc = 1.f;
      rc = __frcp_rn(sc);
      const Place mine = s_place[group + (c & 3) * kGroups];
      if (c < 8 && mine.page >= 0)
        (c < kDeep ? p.ks : p.vs)[((static_cast<int64_t>(mine.page) * p.H_kv + h) << p.page_shift) + mine.row] = sc;
    }
    #pragma unroll
    for (int side = 0; side < 2; ++side) {
      uint8_t* cache = side ? p.vc : p.kc;
      #pragma unroll
      for (int u = 0; u < kDeep; ++u) {
        const int64_t to = at[u].page * p.page_stride + ((static_cast<int64_t>(h) << p.page_shift) + at[u].row) * D + 8 * c;
        if constexpr (E4M3) {
          const int from = (lane & ~(kLanes - 1)) + side * kDeep + u;  // the lane that has this row's scale
          const uint2 codes = quantize(x[side * kDeep + u], __shfl_sync(0xffffffffu, sc, from),
                                       __shfl_sync(0xffffffffu, rc, from));
          if (at[u].page >= 0) *reinterpret_cast<uint2*>(cache + to) = codes;
        } else {
          if (at[u].page >= 0) *reinterpret_cast<uint4*>(cache + 2 * to) = x[side * kDeep + u];
        }
      }
    }
  }
}

template <int D, bool E4M3>
__global__ void __launch_bounds__(kThreads) kv_read_kernel(const __grid_constant__ KvRowsParams p) {
  constexpr int kLanes = D / 8, kGroups = kThreads / kLanes, kTokens = kGroups * kDeep;
  __shared__ Place s_place[kTokens];
  pdl_wait();
  auto cu = [&](int s) { return min(max(p.cu[s], 0), p.T); };
  const int64_t t0 = static_cast<int64_t>(blockIdx.x) * kTokens;
  for (int i = threadIdx.x; i < kTokens; i += kThreads) {
    Place at{-2, 0};
    const int64_t t = t0 + i;
    if (t < p.T) {
      int a = 0, b = p.B;  // the request whose rows hold t, if one does
      while (b - a > 1) {
        const int m = a + ((b - a) >> 1);
        if (cu(m) <= t) a = m;
        else b = m;
      }
      if (cu(a) <= t && t < cu(a + 1)) {
        const int64_t row = (p.first ? p.first[a] : 0) + (t - cu(a));
        const int64_t j = row >> p.page_shift;
        at = Place{-1, static_cast<int>(row & ((1 << p.page_shift) - 1))};
        if (row >= 0 && j < p.max_pages) {
          const int e = p.table[static_cast<int64_t>(a) * p.max_pages + j];
          if (static_cast<unsigned>(e) < static_cast<unsigned>(p.num_pages)) at.page = e;
        }
        if (at.page < 0) atomicCAS(p.status, 0, kStatusBadPage);
      }
    }
    s_place[i] = at;
  }
  if (blockIdx.x == 0 && blockIdx.y == 0) {
    for (int s = threadIdx.x; s < p.B; s += kThreads)
      if (p.cu[s + 1] < p.cu[s] || (s == 0 && p.cu[0] != 0) || p.cu[s + 1] > p.T)
        atomicCAS(p.status, 0, kStatusBadSeqlens);
  }
  __syncthreads();
  const int group = threadIdx.x / kLanes, c = threadIdx.x % kLanes;
  for (int h = blockIdx.y; h < p.H_kv; h += gridDim.y) {
    using Chunk = typename std::conditional<E4M3, uint2, uint4>::type;
    Chunk x[2][kDeep];
    float sc[2][kDeep];
    Place at[kDeep];
    #pragma unroll
    for (int u = 0; u < kDeep; ++u) {
      at[u] = s_place[group + u * kGroups];
      const int64_t in = (static_cast<int64_t>(h) << p.page_shift) + at[u].row;
      #pragma unroll
      for (int side = 0; side < 2; ++side) {
        x[side][u] = Chunk{};
        sc[side][u] = 0.f;
        if (at[u].page >= 0) {
          const int64_t from = at[u].page * p.page_stride + in * D + 8 * c;
          x[side][u] = *reinterpret_cast<const Chunk*>((side ? p.vc : p.kc) + from * (E4M3 ? 1 : 2));
          if (E4M3) sc[side][u] = (side ? p.vs : p.ks)[((static_cast<int64_t>(at[u].page) * p.H_kv) << p.page_shift) + in];
        }
      }
    }
    #pragma unroll
    for (int u = 0; u < kDeep; ++u) {
      if (at[u].page < -1) continue;
      const int64_t to = (static_cast<int64_t>(h) * p.T + t0 + group + u * kGroups) * D + 8 * c;
      #pragma unroll
      for (int side = 0; side < 2; ++side) {
        uint4 y;
        if constexpr (E4M3) y = dequantize(x[side][u], sc[side][u]);
        else y = x[side][u];
        *reinterpret_cast<uint4*>((side ? p.vo : p.ko) + to) = y;
      }
    }
  }
}

// Blocks along heads: enough for several rounds of the GPU's blocks, else a block takes several heads for each look at its
// tokens' places.
dim3 grid_of(int64_t tokens, int H_kv, int d) {
  const int64_t per = kThreads / (d / 8) * kDeep, x = (tokens + per - 1) / per;
  const int64_t want = (32 * 152 + x - 1) / x;
  int64_t y = want < H_kv ? want : H_kv;
  if (y > 65535) y = 65535;
  return dim3(static_cast<unsigned>(x), static_cast<unsigned>(y));
}

}  // namespace

cudaError_t launch_kv_write(const KvRowsParams& p, int d, bool e4m3, cudaStream_t stream) {
  const dim3 grid = grid_of(static_cast<int64_t>(p.B) * p.N, p.H_kv, d);
  auto* kernel = d == 64 ? (e4m3 ? kv_write_kernel<64, true> : kv_write_kernel<64, false>)
                         : (e4m3 ? kv_write_kernel<128, true> : kv_write_kernel<128, false>);
  return launch_dependent(kernel, grid, kThreads, 0, stream, p);
}

cudaError_t launch_kv_read(const KvRowsParams& p, int d, bool e4m3, cudaStream_t stream) {
  const dim3 grid = grid_of(p.T, p.H_kv, d);
  auto* kernel = d == 64 ? (e4m3 ? kv_read_kernel<64, true> : kv_read_kernel<64, false>)
                         : (e4m3 ? kv_read_kernel<128, true> : kv_read_kernel<128, false>);
  return launch_dependent(kernel, grid, kThreads, 0, stream, p);
}

}  // namespace attn
