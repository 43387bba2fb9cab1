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

constexpr int kThreads = 256, kDeep = 4;

// x / sc rounded to nearest fp32 from rc = RN(1 / sc) and one remainder correction (Markstein's method, as in the
// quantizer of attn_fp8.cu, whose check covers every bf16 x and scale that a bf16 row can have).
__device__ __forceinline__ float quotient(float x, float sc, float rc) {
  const float q0 = __fmul_rn(x, rc);
  return copysignf(__fmaf_rn(__fmaf_rn(-sc, q0, x), rc, q0), x);
}

// 8 bf16 values -> 8 codes, with the D/8 lanes that hold the row; returns the row's scale.
template <int D>
__device__ __forceinline__ float quantize(const uint4& x, uint2& codes) {
  const uint32_t v[4] = {x.x, x.y, x.z, x.w};
  float f[8], amax = 0.f;
  #pragma unroll
  for (int i = 0; i < 4; ++i) {
    f[2 * i] = bf16lo_to_f32(v[i]);
    f[2 * i + 1] = bf16hi_to_f32(v[i]);
    amax = fmax3(amax, fabsf(f[2 * i]), fabsf(f[2 * i + 1]));
  }
  #pragma unroll
  for (int off = D / 16; off > 0; off >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, off));
  float sc = __fdiv_rn(amax, 448.f);
  if (!(sc >= 0x1p-126f)) sc = 1.f;
  uint16_t c[4];
  if (sc >= 0x1p-100f && sc <= 0x1p100f) {
    const float rc = __frcp_rn(sc);
    #pragma unroll
    for (int i = 0; i < 4; ++i) c[i] = pack_e4m3x2(quotient(f[2 * i], sc, rc), quotient(f[2 * i + 1], sc, rc));
  } else {
    #pragma unroll
    for (int i = 0; i < 4; ++i) c[i] = pack_e4m3x2(__fdiv_rn(f[2 * i], sc), __fdiv_rn(f[2 * i + 1], sc));
  }
  codes = make_uint2(c[0] | static_cast<uint32_t>(c[1]) << 16, c[2] | static_cast<uint32_t>(c[3]) << 16);
  return sc;
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
    out[i] = pack_bf16x2(lo * sc, hi * sc);
  }
  return make_uint4(out[0], out[1], out[2], out[3]);
}

// A token's page and row of it; page -1: none, -2: not this call's to touch.
struct Place {
  int page, row;
};

template <int D, bool E4M3>
__global__ void __launch_bounds__(kThreads) kv_write_kernel(const __grid_constant__ KvRowsParams p) {
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
  const int group = threadIdx.x / kLanes, c = threadIdx.x % kLanes;
  for (int h = blockIdx.y; h < p.H_kv; h += gridDim.y) {
    uint4 x[2][kDeep];
    Place at[kDeep];
    #pragma unroll
    for (int u = 0; u < kDeep; ++u) {
      const int i = group + u * kGroups;
      at[u] = s_place[i];
      x[0][u] = x[1][u] = make_uint4(0, 0, 0, 0);
      if (at[u].page >= 0) {
        const int64_t t = t0 + i, b = p.N == 1 ? t : p.B == 1 ? 0 : t / p.N, n = t - b * p.N;
        x[0][u] = *reinterpret_cast<const uint4*>(p.k + b * p.k_batch + h * p.k_head + n * p.k_token + 8 * c);
        x[1][u] = *reinterpret_cast<const uint4*>(p.v + b * p.v_batch + h * p.v_head + n * p.v_token + 8 * c);
      }
    }
    #pragma unroll
    for (int u = 0; u < kDeep; ++u) {
      const int64_t in = (static_cast<int64_t>(h) << p.page_shift) + at[u].row;
      #pragma unroll
      for (int side = 0; side < 2; ++side) {
        uint8_t* cache = side ? p.vc : p.kc;
        const int64_t to = at[u].page * p.page_stride + in * D + 8 * c;
        if constexpr (E4M3) {
          uint2 codes;
          const float sc = quantize<D>(x[side][u], codes);
          if (at[u].page >= 0) {
            *reinterpret_cast<uint2*>(cache + to) = codes;
            if (c == 0)
              (side ? p.vs : p.ks)[((static_cast<int64_t>(at[u].page) * p.H_kv) << p.page_shift) + in] = sc;
          }
        } else {
          if (at[u].page >= 0) *reinterpret_cast<uint4*>(cache + 2 * to) = x[side][u];
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
        const int m = (a + b) >> 1;
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

// Blocks along heads: enough to fill the GPU where tokens alone are too few, else a block takes several heads
// for each look at its tokens' places.
dim3 grid_of(int64_t tokens, int H_kv, int d) {
  const int64_t per = kThreads / (d / 8) * kDeep, x = (tokens + per - 1) / per;
  const int64_t want = (8 * 152 + x - 1) / x;
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
