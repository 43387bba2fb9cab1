// attn_qkv_rope.cu -- the step before attention and its backward: RMS norm of each query and key
// head, rotation by position, token-major rows to head-major tensors, rows into a paged cache.
//
// What bounds it: memory, one read and one write of every row; then, below it, instructions, so the
// arithmetic is packed and nothing is computed twice.
//
// A head's row of d elements is held by d/16 lanes with 16 elements each, as two 16-byte chunks
// chosen so that every pair (a, b) of the rotation lies in one lane: chunks l and l + rot/16 when
// element i turns with i + rot/2, any two when 2i turns with 2i + 1.  The mean of squares is then
// the only value that crosses lanes.  A warp-wide load covers 4 rows (d = 128) or 8 (d = 64).
//
// A warp takes a token (or, when there are few tokens, a share of a token's rows) and works alone: it
// puts the token's coefficients into its own shared memory, 64 pairs of them at d = 128, two a lane,
// and streams the token's heads through them, loads a batch ahead.  In the forward the norm's
// weight is folded in: with r the inverse root mean square,
//   (y_a, y_b) = r (x_a, x_b) * (w_a c, w_b c) + r (x_b, x_a) * (-w_b s, w_a s),
// three packed operations a pair.
//
// Angles: t = position * inv_freq modulo one turn, in 64-bit fixed point (a turn is 2^64), so the
// product wraps exactly and a position of 2^20 costs no accuracy; the top 32 bits go to sincospi.
// The frequency is brought to fixed point by an integer product, not in float64, which this GPU
// computes at 1/64 of its fp32 rate.
#include "attn_gen.h"
#include "sm103_ptx.cuh"

#include <cmath>

namespace attn {
namespace {

constexpr int kWarps = kRopeThreads / 32;

// inv_freq (radians a position) in turns a position, modulo 1, times 2^64.
__device__ __forceinline__ uint64_t turn_step(double f) {
  const uint64_t bits = static_cast<uint64_t>(__double_as_longlong(f));
  const int e = static_cast<int>((bits >> 52) & 0x7FF) - 1023;  // |f| = m * 2^(e - 63)
  const uint64_t m = ((bits << 11) & 0x7FFFFFFFFFFFFFFFull) | 0x8000000000000000ull;
  const uint64_t p = __umul64hi(m, 0xA2F9836E4E44152Aull);      // round(2^66 / (2 pi))
  const int sh = e - 1;                                         // |f| / (2 pi) = p * 2^(e - 65)
  uint64_t step = sh >= 64 || sh <= -64 ? 0 : sh >= 0 ? p << sh : p >> -sh;
  return bits >> 63 ? 0 - step : step;
}
// cos and sin (times scale) of pair `f` of a token.
__device__ __forceinline__ void angle(const RopeParams& p, int position, int f, float& c, float& s) {
  const uint64_t phase =
      static_cast<uint64_t>(static_cast<int64_t>(position)) * turn_step(__ldg(p.inv_freq + f));
  sincospif(static_cast<float>(static_cast<int>(phase >> 32)) * 0x1p-31f, &s, &c);  // 2^31: half a turn
  c *= p.rope_scale;
  s *= p.rope_scale;
}

// A lane's 16 elements as 8 pairs.  Half layout: pair i is element i of chunk a and of chunk b.
// Interleaved: pairs 0..3 are chunk a's neighbours, 4..7 chunk b's.
template <int D, bool INTER>
struct Lane {
  static constexpr int kLanes = D / 16;
  int a, b;        // chunks
  bool ta, tb;     // whether a chunk's pairs turn
  __device__ __forceinline__ Lane(int l, int rot) {
    if (INTER) {
      a = l;
      b = l + kLanes;
      ta = 8 * a < rot;
      tb = 8 * b < rot;
    } else {
      const int half = rot >> 4;
      a = l < half ? l : 2 * half + 2 * (l - half);
      b = l < half ? l + half : a + 1;
      ta = tb = l < half;
    }
  }
  // elements and frequency of pair i
  __device__ __forceinline__ int first(int i) const {
    return INTER ? (i < 4 ? 8 * a + 2 * i : 8 * b + 2 * (i - 4)) : 8 * a + i;
  }
  __device__ __forceinline__ int second(int i) const { return INTER ? first(i) + 1 : 8 * b + i; }
  __device__ __forceinline__ int freq(int i) const { return INTER ? first(i) >> 1 : 8 * a + i; }
  __device__ __forceinline__ bool turns(int i) const { return i < 4 ? ta : tb; }
  // 16 bf16 values to pairs and back
  static __device__ __forceinline__ void unpack(const uint4& va, const uint4& vb, float (&x)[8][2]) {
    const uint32_t wa[4] = {va.x, va.y, va.z, va.w}, wb[4] = {vb.x, vb.y, vb.z, vb.w};
    #pragma unroll
    for (int i = 0; i < 4; ++i) {
      if (INTER) {
        x[i][0] = bf16lo_to_f32(wa[i]);
        x[i][1] = bf16hi_to_f32(wa[i]);
        x[4 + i][0] = bf16lo_to_f32(wb[i]);
        x[4 + i][1] = bf16hi_to_f32(wb[i]);
      } else {
        x[2 * i][0] = bf16lo_to_f32(wa[i]);
        x[2 * i + 1][0] = bf16hi_to_f32(wa[i]);
        x[2 * i][1] = bf16lo_to_f32(wb[i]);
        x[2 * i + 1][1] = bf16hi_to_f32(wb[i]);
      }
    }
  }
  static __device__ __forceinline__ void pack(const float (&x)[8][2], uint4& va, uint4& vb) {
    uint32_t wa[4], wb[4];
    #pragma unroll
    for (int i = 0; i < 4; ++i) {
      if (INTER) {
        wa[i] = pack_bf16x2(x[i][0], x[i][1]);
        wb[i] = pack_bf16x2(x[4 + i][0], x[4 + i][1]);
      } else {
        wa[i] = pack_bf16x2(x[2 * i][0], x[2 * i + 1][0]);
        wb[i] = pack_bf16x2(x[2 * i][1], x[2 * i + 1][1]);
      }
    }
    va = make_uint4(wa[0], wa[1], wa[2], wa[3]);
    vb = make_uint4(wb[0], wb[1], wb[2], wb[3]);
  }
};

template <int D>
__device__ __forceinline__ float row_sum(float v) {
  #pragma unroll
  for (int off = D / 32; off > 0; off >>= 1) v += __shfl_xor_sync(0xffffffffu, v, off);
  return v;
}

// A row's E4M3 codes and scale into the cache.
template <int D, bool INTER>
__device__ __forceinline__ void store_codes(const float (&x)[8][2], uint8_t* row, float* scale, int ca,
                                            int cb, bool write, bool first_lane) {
  float amax = 0.f;
  #pragma unroll
  for (int i = 0; i < 8; ++i) amax = fmax3(amax, fabsf(x[i][0]), fabsf(x[i][1]));
  #pragma unroll
  for (int off = D / 32; off > 0; off >>= 1)
    amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, off));
  float sc = __fdiv_rn(amax, 448.f);
  if (!(sc >= 0x1p-126f)) sc = 1.f;
  if (!write) return;
  uint32_t wa[2], wb[2];
  auto codes = [&](float a, float b, float c, float e) {
    return static_cast<uint32_t>(pack_e4m3x2(__fdiv_rn(a, sc), __fdiv_rn(b, sc))) |
           static_cast<uint32_t>(pack_e4m3x2(__fdiv_rn(c, sc), __fdiv_rn(e, sc))) << 16;
  };
  #pragma unroll
  for (int i = 0; i < 2; ++i) {
    if (INTER) {
      wa[i] = codes(x[2 * i][0], x[2 * i][1], x[2 * i + 1][0], x[2 * i + 1][1]);
      wb[i] = codes(x[4 + 2 * i][0], x[4 + 2 * i][1], x[5 + 2 * i][0], x[5 + 2 * i][1]);
    } else {
      wa[i] = codes(x[4 * i][0], x[4 * i + 1][0], x[4 * i + 2][0], x[4 * i + 3][0]);
      wb[i] = codes(x[4 * i][1], x[4 * i + 1][1], x[4 * i + 2][1], x[4 * i + 3][1]);
    }
  }
  *reinterpret_cast<uint2*>(row + 8 * ca) = make_uint2(wa[0], wa[1]);
  *reinterpret_cast<uint2*>(row + 8 * cb) = make_uint2(wb[0], wb[1]);
  if (first_lane) *scale = sc;
}

// The rows a warp-wide load covers: group gi of a token, 0 .. nq - 1 query heads, then key, then
// value heads.
template <int RW>
struct Groups {
  int nq, nk, all;
  __device__ __forceinline__ Groups(int H, int H_kv)
      : nq((H + RW - 1) / RW), nk((H_kv + RW - 1) / RW), all(nq + 2 * nk) {}
  // 0 query, 1 key, 2 value; `h`: this lane's head of that kind
  __device__ __forceinline__ int kind(int gi, int sub, int& h) const {
    const int k = gi < nq ? 0 : gi < nq + nk ? 1 : 2;
    h = (gi - (k == 0 ? 0 : k == 1 ? nq : nq + nk)) * RW + sub;
    return k;
  }
};

constexpr int kBatch = 4;  // groups a warp loads before it uses the first

template <int D, bool INTER, int CACHE>
__global__ void __launch_bounds__(kRopeThreads) qkv_rope_kernel(RopeParams p) {
  using L = Lane<D, INTER>;
  constexpr int kLanes = D / 16, kRw = 32 / kLanes;
  __shared__ float4 s_coef[kWarps][2][D / 2];  // [query, key][pair i of lane l at i * kLanes + l]
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int l = lane % kLanes, sub = lane / kLanes;
  const int t = blockIdx.x * (kWarps / p.parts) + warp / p.parts;
  if (t >= p.tokens) return;
  const int part = warp % p.parts;
  const L ln(l, p.rot);
  const Groups<kRw> gr(p.H, p.H_kv);
  const int b = t / p.N, n = t - b * p.N;
  const uint4* row = reinterpret_cast<const uint4*>(p.qkv + static_cast<int64_t>(t) * p.ld);
  uint4 xa[kBatch], xb[kBatch];
  auto load = [&](int g0) {
    #pragma unroll
    for (int u = 0; u < kBatch; ++u) {
      int h;
      const int kind = gr.kind(g0 + u * p.parts, sub, h);
      xa[u] = xb[u] = make_uint4(0u, 0u, 0u, 0u);
      if (g0 + u * p.parts < gr.all && h < (kind ? p.H_kv : p.H)) {
        const int hh = h + (kind == 0 ? 0 : kind == 1 ? p.H : p.H + p.H_kv);
        xa[u] = __ldcs(row + hh * (D / 8) + ln.a);
        xb[u] = __ldcs(row + hh * (D / 8) + ln.b);
      }
    }
  };
  load(part);
  {
    const int position = p.rot ? p.positions[t] : 0;
    #pragma unroll
    for (int j = lane; j < D / 2; j += 32) {
      const int i = j / kLanes, lj = j % kLanes;
      const L o(lj, p.rot);
      float c = 1.f, s = 0.f;
      if (o.turns(i)) angle(p, position, o.freq(i), c, s);
      #pragma unroll
      for (int k = 0; k < 2; ++k) {
        const __nv_bfloat16* w = k ? p.wk : p.wq;
        const float wa = w ? __bfloat162float(w[o.first(i)]) : 1.f;
        const float wb = w ? __bfloat162float(w[o.second(i)]) : 1.f;
        s_coef[warp][k][j] = make_float4(wa * c, wb * c, -(wb * s), wa * s);
      }
    }
    __syncwarp();
  }
  const int64_t step = static_cast<int64_t>(p.N) * D;
  const int64_t tq = (static_cast<int64_t>(b) * p.H * p.N + n) * D;
  const int64_t tk = (static_cast<int64_t>(b) * p.H_kv * p.N + n) * D;
  int64_t slot = -1, page = 0;
  if (CACHE != kCacheNone) {
    slot = p.slots[t];
    page = slot >> p.page_shift;
    if (slot >= 0 && page >= p.num_pages) {
      if (lane == 0) atomicCAS(p.status, 0, kStatusBadPage);
      slot = -1;
    }
  }
  for (int g0 = part; g0 < gr.all; g0 += kBatch * p.parts) {
    if (g0 != part) load(g0);
    #pragma unroll
    for (int u = 0; u < kBatch; ++u) {
      if (g0 + u * p.parts >= gr.all) break;
      int h;
      const int kind = gr.kind(g0 + u * p.parts, sub, h);
      const bool live = h < (kind ? p.H_kv : p.H);
      uint4 oa = xa[u], ob = xb[u];
      float x[8][2];
      if (kind < 2) {
        L::unpack(xa[u], xb[u], x);
        if (kind ? p.wk != nullptr : p.wq != nullptr) {
          float s0 = 0.f, s1 = 0.f;
          #pragma unroll
          for (int i = 0; i < 8; ++i)
            ffma2(s0, s1, x[i][0], x[i][1], x[i][0], x[i][1], s0, s1);
          const float r = rsqrtf(row_sum<D>(s0 + s1) * (1.f / D) + p.eps);
          #pragma unroll
          for (int i = 0; i < 8; ++i) fmul2(x[i][0], x[i][1], x[i][0], x[i][1], r, r);
        }
        const float4* co = s_coef[warp][kind] + l;
        #pragma unroll
        for (int i = 0; i < 8; ++i) {
          const float4 c = co[i * kLanes];
          float y0, y1;
          fmul2(y0, y1, x[i][0], x[i][1], c.x, c.y);
          if (ln.turns(i)) ffma2(y0, y1, x[i][1], x[i][0], c.z, c.w, y0, y1);
          x[i][0] = y0;
          x[i][1] = y1;
        }
        L::pack(x, oa, ob);
      } else if (CACHE == kCacheE4m3) {
        L::unpack(xa[u], xb[u], x);
      }
      __nv_bfloat16* out = kind == 0 ? p.q : kind == 1 ? p.k : p.v;
      if (live && out) {
        uint4* dst = reinterpret_cast<uint4*>(out + (kind ? tk : tq) + h * step);
        dst[ln.a] = oa;
        dst[ln.b] = ob;
      }
      if (CACHE != kCacheNone && kind > 0) {
        const bool write = live && slot >= 0;
        const int64_t at_row =
            (static_cast<int64_t>(h) << p.page_shift) + (slot & ((1 << p.page_shift) - 1));
        const int64_t at = page * p.page_stride + at_row * D;
        uint8_t* base = kind == 2 ? p.vc : p.kc;
        if (CACHE == kCacheBf16) {
          if (write) {
            uint4* dst = reinterpret_cast<uint4*>(base + 2 * at);
            dst[ln.a] = oa;
            dst[ln.b] = ob;
          }
        } else {
          float* scales = kind == 2 ? p.vs : p.ks;
          store_codes<D, INTER>(x, base + (write ? at : 0),
                                scales + (write ? ((page * p.H_kv) << p.page_shift) + at_row : 0),
                                ln.a, ln.b, write, l == 0);
        }
      }
    }
  }
}

// Gradients of the rows, and each CTA's share of the weights' gradients.  With t = x r, g the
// gradient turned back and u = g w:  dx = r (u - t mean(u t)),  dw += g t.
constexpr int kBatchBwd = 2;

template <int D, bool INTER>
__global__ void __launch_bounds__(kRopeThreads, 2) qkv_rope_bwd_kernel(RopeParams p) {
  using L = Lane<D, INTER>;
  constexpr int kLanes = D / 16, kRw = 32 / kLanes;
  __shared__ __align__(16) float s_dw[kWarps][D];     // the weights' sums, at the end
  __shared__ float2 s_cs[kWarps][D / 2];              // cos, sin of pair i of lane l
  __shared__ float2 s_w[2][D / 2];                    // the weights, likewise
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int l = lane % kLanes, sub = lane / kLanes;
  const L ln(l, p.rot);
  const Groups<kRw> gr(p.H, p.H_kv);
  for (int j = threadIdx.x; j < D; j += kRopeThreads) {
    const int k = j / (D / 2), jj = j % (D / 2);
    const L o(jj % kLanes, p.rot);
    const __nv_bfloat16* w = k ? p.wk : p.wq;
    s_w[k][jj] = w ? make_float2(__bfloat162float(w[o.first(jj / kLanes)]),
                                 __bfloat162float(w[o.second(jj / kLanes)]))
                   : make_float2(1.f, 1.f);
  }
  __syncthreads();
  float dw[2][8][2];
  #pragma unroll
  for (int k = 0; k < 2; ++k)
    #pragma unroll
    for (int i = 0; i < 8; ++i) dw[k][i][0] = dw[k][i][1] = 0.f;
  const int64_t step = static_cast<int64_t>(p.N) * D;
  const int64_t tasks = static_cast<int64_t>(p.tokens) * p.parts;
  for (int64_t task = static_cast<int64_t>(blockIdx.x) * kWarps + warp; task < tasks;
       task += static_cast<int64_t>(gridDim.x) * kWarps) {
    const int t = static_cast<int>(task / p.parts), part = static_cast<int>(task - static_cast<int64_t>(t) * p.parts);
    const int b = t / p.N, n = t - b * p.N;
    const uint4* row = reinterpret_cast<const uint4*>(p.qkv + static_cast<int64_t>(t) * p.ld);
    uint4* out = reinterpret_cast<uint4*>(p.dqkv + static_cast<int64_t>(t) * p.ld_out);
    const int64_t tq = (static_cast<int64_t>(b) * p.H * p.N + n) * D;
    const int64_t tk = (static_cast<int64_t>(b) * p.H_kv * p.N + n) * D;
    uint4 ga[kBatchBwd], gb[kBatchBwd], xa[kBatchBwd], xb[kBatchBwd];
    auto load = [&](int g0) {
      #pragma unroll
      for (int u = 0; u < kBatchBwd; ++u) {
        int h;
        const int kind = gr.kind(g0 + u * p.parts, sub, h);
        ga[u] = gb[u] = xa[u] = xb[u] = make_uint4(0u, 0u, 0u, 0u);
        if (g0 + u * p.parts < gr.all && h < (kind ? p.H_kv : p.H)) {
          const __nv_bfloat16* dy = kind == 0 ? p.dq : kind == 1 ? p.dk : p.dv;
          const uint4* src = reinterpret_cast<const uint4*>(dy + (kind ? tk : tq) + h * step);
          ga[u] = __ldcs(src + ln.a);
          gb[u] = __ldcs(src + ln.b);
          if (kind == 0 ? p.wq != nullptr : kind == 1 && p.wk != nullptr) {
            const int hh = h + (kind ? p.H : 0);
            xa[u] = __ldcs(row + hh * (D / 8) + ln.a);
            xb[u] = __ldcs(row + hh * (D / 8) + ln.b);
          }
        }
      }
    };
    load(part);
    __syncwarp();
    const int position = p.rot ? p.positions[t] : 0;
    #pragma unroll
    for (int j = lane; j < D / 2; j += 32) {
      const L o(j % kLanes, p.rot);
      float c = 1.f, s = 0.f;
      if (o.turns(j / kLanes)) angle(p, position, o.freq(j / kLanes), c, s);
      s_cs[warp][j] = make_float2(c, s);
    }
    __syncwarp();
    for (int g0 = part; g0 < gr.all; g0 += kBatchBwd * p.parts) {
      if (g0 != part) load(g0);
      #pragma unroll
      for (int u = 0; u < kBatchBwd; ++u) {
        if (g0 + u * p.parts >= gr.all) break;
        int h;
        const int kind = gr.kind(g0 + u * p.parts, sub, h);
        const bool live = h < (kind ? p.H_kv : p.H);
        uint4 oa = ga[u], ob = gb[u];
        if (kind < 2) {
          float g[8][2];
          L::unpack(ga[u], gb[u], g);
          #pragma unroll
          for (int i = 0; i < 8; ++i) {
            if (!ln.turns(i)) continue;
            const float2 cs = s_cs[warp][i * kLanes + l];
            float y0, y1;
            fmul2(y0, y1, g[i][1], g[i][0], cs.y, -cs.y);
            ffma2(g[i][0], g[i][1], g[i][0], g[i][1], cs.x, cs.x, y0, y1);
          }
          if (kind ? p.wk != nullptr : p.wq != nullptr) {
            float x[8][2];
            L::unpack(xa[u], xb[u], x);
            float s0 = 0.f, s1 = 0.f, d0 = 0.f, d1 = 0.f;
            #pragma unroll
            for (int i = 0; i < 8; ++i)
              ffma2(s0, s1, x[i][0], x[i][1], x[i][0], x[i][1], s0, s1);
            const float r = rsqrtf(row_sum<D>(s0 + s1) * (1.f / D) + p.eps);
            auto weigh = [&](float (&acc)[8][2]) {
              #pragma unroll
              for (int i = 0; i < 8; ++i) {
                const float2 w = s_w[kind][i * kLanes + l];
                fmul2(x[i][0], x[i][1], x[i][0], x[i][1], r, r);
                ffma2(acc[i][0], acc[i][1], g[i][0], g[i][1], x[i][0], x[i][1], acc[i][0], acc[i][1]);
                fmul2(g[i][0], g[i][1], g[i][0], g[i][1], w.x, w.y);
                ffma2(d0, d1, g[i][0], g[i][1], x[i][0], x[i][1], d0, d1);
              }
            };
            if (kind) weigh(dw[1]); else weigh(dw[0]);
            const float mean = row_sum<D>(d0 + d1) * (-1.f / D);
            #pragma unroll
            for (int i = 0; i < 8; ++i) {
              ffma2(g[i][0], g[i][1], x[i][0], x[i][1], mean, mean, g[i][0], g[i][1]);
              fmul2(g[i][0], g[i][1], g[i][0], g[i][1], r, r);
            }
          }
          L::pack(g, oa, ob);
        }
        if (live) {
          const int hh = h + (kind == 0 ? 0 : kind == 1 ? p.H : p.H + p.H_kv);
          out[hh * (D / 8) + ln.a] = oa;
          out[hh * (D / 8) + ln.b] = ob;
        }
      }
    }
  }
  if (!p.partial) return;
  // the CTA's sums: over the rows of a warp's groups by shuffles, over the warps in order
  #pragma unroll
  for (int k = 0; k < 2; ++k) {
    #pragma unroll
    for (int i = 0; i < 8; ++i)
      #pragma unroll
      for (int j = 0; j < 2; ++j)
        #pragma unroll
        for (int off = 16; off >= kLanes; off >>= 1)
          dw[k][i][j] += __shfl_xor_sync(0xffffffffu, dw[k][i][j], off);
    __syncthreads();
    if (sub == 0) {
      #pragma unroll
      for (int i = 0; i < 8; ++i) {
        s_dw[warp][ln.first(i)] = dw[k][i][0];
        s_dw[warp][ln.second(i)] = dw[k][i][1];
      }
    }
    __syncthreads();
    if (threadIdx.x < D) {
      float v = 0.f;
      #pragma unroll
      for (int wi = 0; wi < kWarps; ++wi) v += s_dw[wi][threadIdx.x];
      p.partial[(static_cast<size_t>(blockIdx.x) * 2 + k) * D + threadIdx.x] = v;
    }
  }
}

// dwq (block 0) and dwk (block 1): the CTAs' shares, runs of CTAs summed side by side, then joined
// in order.
__global__ void __launch_bounds__(1024) rope_dw_kernel(const float* __restrict__ partial, int ctas,
                                                       int d, float* dwq, float* dwk) {
  __shared__ float s_sum[1024];
  float* out = blockIdx.x ? dwk : dwq;
  if (!out) return;
  const int runs = 1024 / d, c = threadIdx.x % d, run = threadIdx.x / d;
  float v = 0.f;
  #pragma unroll 8
  for (int i = run; i < ctas; i += runs)
    v += partial[(static_cast<size_t>(i) * 2 + blockIdx.x) * d + c];
  s_sum[threadIdx.x] = v;
  __syncthreads();
  if (run == 0) {
    for (int i = 1; i < runs; ++i) v += s_sum[i * d + c];
    out[c] = v;
  }
}

template <int D, bool INTER>
cudaError_t launch_fwd(const RopeParams& p, int kind, int ctas, cudaStream_t st) {
  if (kind == kCacheNone) qkv_rope_kernel<D, INTER, kCacheNone><<<ctas, kRopeThreads, 0, st>>>(p);
  else if (kind == kCacheBf16) qkv_rope_kernel<D, INTER, kCacheBf16><<<ctas, kRopeThreads, 0, st>>>(p);
  else qkv_rope_kernel<D, INTER, kCacheE4m3><<<ctas, kRopeThreads, 0, st>>>(p);
  return cudaGetLastError();
}

// Warps of one token: one while the tokens alone fill the GPU (two CTAs of 8 warps on each of 152
// SMs); else more, so that each has fewer rows one after another.
int parts_of(int tokens) {
  int parts = 1;
  while (parts < kWarps && static_cast<int64_t>(tokens) * parts < 2 * kWarps * 152) parts *= 2;
  return parts;
}

}  // namespace

cudaError_t launch_qkv_rope(RopeParams& p, int d, bool interleaved, int kind, cudaStream_t st) {
  p.parts = parts_of(p.tokens);
  const int tok_cta = kWarps / p.parts;
  const int ctas = (p.tokens + tok_cta - 1) / tok_cta;
  if (d == 64)
    return interleaved ? launch_fwd<64, true>(p, kind, ctas, st)
                       : launch_fwd<64, false>(p, kind, ctas, st);
  return interleaved ? launch_fwd<128, true>(p, kind, ctas, st)
                     : launch_fwd<128, false>(p, kind, ctas, st);
}

cudaError_t launch_qkv_rope_bwd(RopeParams& p, int d, bool interleaved, cudaStream_t st) {
  p.parts = parts_of(p.tokens);
  const int64_t want = (static_cast<int64_t>(p.tokens) * p.parts + kWarps - 1) / kWarps;
  const int ctas = static_cast<int>(want < kRopeBwdCtas ? want : kRopeBwdCtas);
  if (d == 64) {
    if (interleaved) qkv_rope_bwd_kernel<64, true><<<ctas, kRopeThreads, 0, st>>>(p);
    else qkv_rope_bwd_kernel<64, false><<<ctas, kRopeThreads, 0, st>>>(p);
  } else {
    if (interleaved) qkv_rope_bwd_kernel<128, true><<<ctas, kRopeThreads, 0, st>>>(p);
    else qkv_rope_bwd_kernel<128, false><<<ctas, kRopeThreads, 0, st>>>(p);
  }
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess || !p.partial) return e;
  rope_dw_kernel<<<2, 1024, 0, st>>>(p.partial, ctas, d, p.dwq, p.dwk);
  return cudaGetLastError();
}

}  // namespace attn
