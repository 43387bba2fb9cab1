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
// A warp takes a token, or two and more share a token's rows; they put the token's coefficients into
// shared memory, 64 pairs of them at d = 128, and each streams its heads through them, loads a batch
// ahead, without another wait for the others.  In the forward the norm's
// weight is folded in: with r the inverse root mean square,
//   (y_a, y_b) = r (x_a, x_b) * (w_a c, w_b c) + r (x_b, x_a) * (-w_b s, w_a s),
// three packed operations on two values each.  (33333 rows of 16 query and 16 K/V heads, d = 128: 126 us, 96 % of
// the copy rate; into a bf16 cache too 167 us, 97 %; into E4M3 codes, two CTAs an SM and a division an element, 182 us, 78 %.)
//
// Angles: t = position * inv_freq modulo one turn, in 64-bit fixed point (a turn is 2^64), so the
// product wraps exactly and a position of 2^20 costs no accuracy; the top 32 bits go to sincospi.
// The frequency is brought to fixed point by an integer product, not in float64, which this GPU
// computes at 1/64 of its fp32 rate.
#include "attn_gen.cuh"
#include "attn_gen.h"
#include "sm103_ptx.cuh"

#include <atomic>
#include <cmath>
#include <type_traits>

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
// cos and sin (times scale) of a position's angle.
__device__ __forceinline__ void angle(const RopeParams& p, int position, uint64_t step, float& c,
                                      float& s) {
  const uint64_t phase = static_cast<uint64_t>(static_cast<int64_t>(position)) * step;
  sincospif(static_cast<float>(static_cast<int>(phase >> 32)) * 0x1p-31f, &s, &c);  // 2^31: half a turn
  c *= p.rope_scale;
  s *= p.rope_scale;
}

// A lane's 16 elements as 8 pairs (a_i, b_i).  Half layout: element i of chunk a and of chunk b.
// Interleaved: pairs 0..3 are chunk a's neighbours, 4..7 chunk b's.  The a's and the b's are two
// arrays, so that packed operations run along i in both layouts.
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
  static __device__ __forceinline__ void unpack(const uint4& va, const uint4& vb, float (&xa)[8],
                                                float (&xb)[8]) {
    const uint32_t wa[4] = {va.x, va.y, va.z, va.w}, wb[4] = {vb.x, vb.y, vb.z, vb.w};
    #pragma unroll
    for (int i = 0; i < 4; ++i) {
      if (INTER) {
        xa[i] = bf16lo_to_f32(wa[i]);
        xb[i] = bf16hi_to_f32(wa[i]);
        xa[4 + i] = bf16lo_to_f32(wb[i]);
        xb[4 + i] = bf16hi_to_f32(wb[i]);
      } else {
        xa[2 * i] = bf16lo_to_f32(wa[i]);
        xa[2 * i + 1] = bf16hi_to_f32(wa[i]);
        xb[2 * i] = bf16lo_to_f32(wb[i]);
        xb[2 * i + 1] = bf16hi_to_f32(wb[i]);
      }
    }
  }
  static __device__ __forceinline__ void pack(const float (&xa)[8], const float (&xb)[8], uint4& va,
                                              uint4& vb) {
    uint32_t wa[4], wb[4];
    #pragma unroll
    for (int i = 0; i < 4; ++i) {
      if (INTER) {
        wa[i] = pack_bf16x2(xa[i], xb[i]);
        wb[i] = pack_bf16x2(xa[4 + i], xb[4 + i]);
      } else {
        wa[i] = pack_bf16x2(xa[2 * i], xa[2 * i + 1]);
        wb[i] = pack_bf16x2(xb[2 * i], xb[2 * i + 1]);
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
__device__ __forceinline__ float sum_squares(const float (&xa)[8], const float (&xb)[8]) {
  float s0 = 0.f, s1 = 0.f;
  #pragma unroll
  for (int i = 0; i < 8; i += 2) {
    ffma2(s0, s1, xa[i], xa[i + 1], xa[i], xa[i + 1], s0, s1);
    ffma2(s0, s1, xb[i], xb[i + 1], xb[i], xb[i + 1], s0, s1);
  }
  return s0 + s1;
}

// A row's E4M3 codes and scale into the cache.
template <int D, bool INTER>
__device__ __forceinline__ void store_codes(const float (&xa)[8], const float (&xb)[8], uint8_t* row,
                                            float* scale, int ca, int cb, bool write,
                                            bool first_lane) {
  float amax = 0.f;
  #pragma unroll
  for (int i = 0; i < 8; ++i) amax = fmax3(amax, fabsf(xa[i]), fabsf(xb[i]));
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
      wa[i] = codes(xa[2 * i], xb[2 * i], xa[2 * i + 1], xb[2 * i + 1]);
      wb[i] = codes(xa[4 + 2 * i], xb[4 + 2 * i], xa[5 + 2 * i], xb[5 + 2 * i]);
    } else {
      wa[i] = codes(xa[4 * i], xa[4 * i + 1], xa[4 * i + 2], xa[4 * i + 3]);
      wb[i] = codes(xb[4 * i], xb[4 * i + 1], xb[4 * i + 2], xb[4 * i + 3]);
    }
  }
  *reinterpret_cast<uint2*>(row + 8 * ca) = make_uint2(wa[0], wa[1]);
  *reinterpret_cast<uint2*>(row + 8 * cb) = make_uint2(wb[0], wb[1]);
  if (first_lane) *scale = sc;
}

// A warp-wide load covers kRw consecutive heads of the row (group g: heads g kRw ..), query, key and
// value heads alike; a group may hold heads of two kinds.  Two groups are computed while the next
// two are on their way.
constexpr int kBatch = 2;

template <int D, bool INTER, int CACHE>
__global__ void __launch_bounds__(kRopeThreads, CACHE == kCacheE4m3 ? 2 : 3) qkv_rope_kernel(RopeParams p) {
  using L = Lane<D, INTER>;
  constexpr int kLanes = D / 16, kRw = 32 / kLanes;
  // per warp and kind (query, key): of pairs 2m, 2m + 1 of lane l, at m * kLanes + l,
  // (w_a c, w_a c, w_b c, w_b c) and (-w_b s, -w_b s, w_a s, w_a s)
  __shared__ float4 s_coef[kWarps][2][2][D / 4];  // by the first warp of those that share a token
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int l = lane % kLanes, sub = lane / kLanes;
  const int task = blockIdx.x * kWarps + warp, t = task / p.parts, part = task - t * p.parts;
  const int team = min(p.parts, kWarps), leader = warp / team * team;  // this token's warps in the CTA
  pdl_wait();
  if (t >= p.tokens) return;  // a whole team: parts is a power of two
  const L ln(l, p.rot);
  const int heads = p.H + 2 * p.H_kv, groups = (heads + kRw - 1) / kRw;
  const int b = t / p.N, n = t - b * p.N;
  const uint4* row = reinterpret_cast<const uint4*>(p.qkv + static_cast<int64_t>(t) * p.ld);
  const uint4 *row_a = row + ln.a, *row_b = row + ln.b;
  uint4 na[kBatch], nb[kBatch];
  auto load = [&](int g0) {
    #pragma unroll
    for (int u = 0; u < kBatch; ++u) {
      const int hh = (g0 + u * p.parts) * kRw + sub;
      na[u] = nb[u] = make_uint4(0u, 0u, 0u, 0u);
      if (hh < heads) {
        na[u] = __ldcs(row_a + hh * (D / 8));
        nb[u] = __ldcs(row_b + hh * (D / 8));
      }
    }
  };
  load(part);
  {
    const int position = p.rot ? p.positions[t] : 0;
    for (int j = (warp - leader) * 32 + lane; j < D / 2; j += 32 * team) {
      const int i = j / kLanes;
      const L o(j % kLanes, p.rot);
      float c = 1.f, s = 0.f;
      if (o.turns(i)) angle(p, position, turn_step(p.inv_freq[o.freq(i)]), c, s);
      #pragma unroll
      for (int k = 0; k < 2; ++k) {
        const __nv_bfloat16* w = k ? p.wk : p.wq;
        const float wa = w ? __bfloat162float(w[o.first(i)]) : 1.f;
        const float wb = w ? __bfloat162float(w[o.second(i)]) : 1.f;
        const int at = (i >> 1) * kLanes + j % kLanes;
        float* cc = reinterpret_cast<float*>(&s_coef[leader][k][0][at]) + (i & 1);
        float* cs = reinterpret_cast<float*>(&s_coef[leader][k][1][at]) + (i & 1);
        cc[0] = wa * c;
        cc[2] = wb * c;
        cs[0] = -(wb * s);
        cs[2] = wa * s;
      }
    }
    if (team == 1) __syncwarp();
    else named_barrier_sync(1 + leader / team, team * 32);
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
  for (int g0 = part; g0 < groups; g0 += kBatch * p.parts) {
    uint4 oa[kBatch], ob[kBatch];
    #pragma unroll
    for (int u = 0; u < kBatch; ++u) {
      oa[u] = na[u];
      ob[u] = nb[u];
    }
    if (g0 + kBatch * p.parts < groups) load(g0 + kBatch * p.parts);
    #pragma unroll
    for (int u = 0; u < kBatch; ++u) {
      const int g = g0 + u * p.parts;
      if (g >= groups) break;
      const int hh = g * kRw + sub;
      const bool live = hh < heads;
      // KIND: query heads, key heads, value heads, or heads of two kinds in one group
      auto rows = [&](auto kind) {
        constexpr int KIND = decltype(kind)::value;
        const bool is_q = KIND == 0 || (KIND == 3 && hh < p.H);
        const bool is_v = KIND == 2 || (KIND == 3 && hh >= p.H + p.H_kv);
        float xa[8], xb[8];
        if (KIND != 2 || CACHE == kCacheE4m3) L::unpack(oa[u], ob[u], xa, xb);
        if constexpr (KIND != 2) {
          const bool normed = is_q ? p.wq != nullptr : !is_v && p.wk != nullptr;
          if (KIND == 3 ? p.wq != nullptr || p.wk != nullptr : normed) {
            float r = rsqrtf(row_sum<D>(sum_squares(xa, xb)) * (1.f / D) + p.eps);
            if (KIND == 3) r = normed ? r : 1.f;
            #pragma unroll
            for (int i = 0; i < 8; i += 2) {
              fmul2(xa[i], xa[i + 1], xa[i], xa[i + 1], r, r);
              fmul2(xb[i], xb[i + 1], xb[i], xb[i + 1], r, r);
            }
          }
          const float4* cc = &s_coef[leader][is_q ? 0 : 1][0][l];
          auto turn = [&](int i, bool turns) {
            const float4 c = cc[(i >> 1) * kLanes];
            float ya0, ya1, yb0, yb1;
            fmul2(ya0, ya1, xa[i], xa[i + 1], c.x, c.y);
            fmul2(yb0, yb1, xb[i], xb[i + 1], c.z, c.w);
            if (turns) {
              const float4 s = cc[D / 4 + (i >> 1) * kLanes];
              ffma2(ya0, ya1, xb[i], xb[i + 1], s.x, s.y, ya0, ya1);
              ffma2(yb0, yb1, xa[i], xa[i + 1], s.z, s.w, yb0, yb1);
            }
            xa[i] = ya0;
            xa[i + 1] = ya1;
            xb[i] = yb0;
            xb[i + 1] = yb1;
          };
          if (!is_v) {
            if (p.rot == D) {
              #pragma unroll
              for (int i = 0; i < 8; i += 2) turn(i, true);
            } else {
              #pragma unroll
              for (int i = 0; i < 8; i += 2) turn(i, ln.turns(i));
            }
            L::pack(xa, xb, oa[u], ob[u]);
          }
        }
        const int h = hh - (is_q ? 0 : is_v ? p.H + p.H_kv : p.H);
        __nv_bfloat16* out = is_q ? p.q : is_v ? p.v : p.k;
        if (live && out) {
          uint4* dst = reinterpret_cast<uint4*>(out + (is_q ? tq : tk) + h * step);
          dst[ln.a] = oa[u];
          dst[ln.b] = ob[u];
        }
        if constexpr (CACHE != kCacheNone && KIND != 0) {
          const bool write = live && !is_q && slot >= 0;
          const int64_t at_row =
              (static_cast<int64_t>(h) << p.page_shift) + (slot & ((1 << p.page_shift) - 1));
          const int64_t at = page * p.page_stride + at_row * D;
          uint8_t* base = is_v ? p.vc : p.kc;
          if constexpr (CACHE == kCacheBf16) {
            if (write) {
              uint4* dst = reinterpret_cast<uint4*>(base + 2 * at);
              dst[ln.a] = oa[u];
              dst[ln.b] = ob[u];
            }
          } else {
            float* scales = is_v ? p.vs : p.ks;
            store_codes<D, INTER>(xa, xb, base + (write ? at : 0),
                                  scales + (write ? ((page * p.H_kv) << p.page_shift) + at_row : 0),
                                  ln.a, ln.b, write, l == 0);
          }
        }
      };
      const int h0 = g * kRw, h1 = h0 + kRw;
      if (h1 <= p.H) rows(std::integral_constant<int, 0>());
      else if (h0 >= p.H && h1 <= p.H + p.H_kv) rows(std::integral_constant<int, 1>());
      else if (h0 >= p.H + p.H_kv) rows(std::integral_constant<int, 2>());
      else rows(std::integral_constant<int, 3>());
    }
  }
}

// Gradients of the rows, and each CTA's share of the weights' gradients.  With h = r g, g the gradient
// turned back, and u = h w:  dx = u - x r^2 mean(u x),  dw += h x.
// A warp walks (token, share of its groups) tasks.  Its rows come through a ring in shared memory, each
// lane copying and reading its own chunks, so that kDepth - 1 groups are in flight without holding
// registers, across tokens too (B = 2, N = 4096, H = 32, H_kv = 8, d = 128: two groups in registers, per
// token, took 69 us, this 54, and with the paths below for heads of one kind 48).
constexpr int kDepth = 4;

template <int D, bool INTER>
__global__ void __launch_bounds__(kRopeThreads, 2) qkv_rope_bwd_kernel(RopeParams p) {
  using L = Lane<D, INTER>;
  constexpr int kLanes = D / 16, kRw = 32 / kLanes, kPairs = D / 64;  // pairs a lane has angles of
  extern __shared__ uint4 s_ring[];                   // [warp][kDepth][dy a, dy b, x a, x b][lane]
  __shared__ __align__(16) float s_dw[kWarps][D];     // the weights' sums, at the end
  // of pairs 2m, 2m + 1 of lane l, at m * kLanes + l: (c, c, s, s), per warp
  __shared__ float4 s_cs[kWarps][D / 4];
  __shared__ float2 s_ns[kWarps][D / 4];              // (-s, -s), likewise
  __shared__ float4 s_w[2][D / 4];                    // (w_a, w_a, w_b, w_b), likewise
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int l = lane % kLanes, sub = lane / kLanes;
  const L ln(l, p.rot);
  pdl_wait();
  pdl_launch_dependents();
  const int heads = p.H + 2 * p.H_kv, groups = (heads + kRw - 1) / kRw;
  const int64_t step = static_cast<int64_t>(p.N) * D;
  const int tasks = p.tokens * p.parts, stride = gridDim.x * kWarps;
  uint4* ring = s_ring + warp * (kDepth * 4 * 32) + lane;
  const uint32_t ring32 = smem_u32(ring);
  // what is copied next: group i_g of task i_task; past the last task: empty commits
  int i_task = blockIdx.x * kWarps + warp, i_g = i_task % p.parts, i_slot = 0;
  const uint4 *i_row = nullptr, *i_q = nullptr, *i_k = nullptr, *i_v = nullptr;
  auto aim = [&] {
    if (i_task >= tasks) return;
    const int t = i_task / p.parts, b = t / p.N, n = t - b * p.N;
    const int64_t tk = (static_cast<int64_t>(b) * p.H_kv * p.N + n) * D;
    i_row = reinterpret_cast<const uint4*>(p.qkv + static_cast<int64_t>(t) * p.ld);
    i_q = reinterpret_cast<const uint4*>(p.dq + (static_cast<int64_t>(b) * p.H * p.N + n) * D);
    i_k = reinterpret_cast<const uint4*>(p.dk + tk);
    i_v = reinterpret_cast<const uint4*>(p.dv + tk);
  };
  auto issue = [&] {
    if (i_task < tasks) {
      const int hh = i_g * kRw + sub;
      const uint32_t dst = ring32 + i_slot * (4 * 32 * 16);
      auto copy = [&](const uint4* src, bool normed) {
        copy16(dst, src + ln.a);
        copy16(dst + 32 * 16, src + ln.b);
        if (normed) {
          copy16(dst + 64 * 16, i_row + hh * (D / 8) + ln.a);
          copy16(dst + 96 * 16, i_row + hh * (D / 8) + ln.b);
        }
      };
      if (i_g * kRw + kRw <= p.H) {
        copy(i_q + hh * (step / 8), p.wq != nullptr);
      } else if (hh < heads) {
        const bool is_q = hh < p.H, is_v = hh >= p.H + p.H_kv;
        const int h = hh - (is_q ? 0 : is_v ? p.H + p.H_kv : p.H);
        copy((is_q ? i_q : is_v ? i_v : i_k) + h * (step / 8),
             is_q ? p.wq != nullptr : !is_v && p.wk != nullptr);
      }
      i_slot = i_slot + 1 == kDepth ? 0 : i_slot + 1;
      if ((i_g += p.parts) >= groups) {
        i_task += stride;
        i_g = i_task % p.parts;
        aim();
      }
    }
    copy_commit();
  };
  aim();
  #pragma unroll
  for (int i = 0; i < kDepth - 1; ++i) issue();

  for (int j = threadIdx.x; j < D; j += kRopeThreads) {
    const int k = j / (D / 2), jj = j % (D / 2), i = jj / kLanes;
    const L o(jj % kLanes, p.rot);
    const __nv_bfloat16* w = k ? p.wk : p.wq;
    float* f = reinterpret_cast<float*>(&s_w[k][(i >> 1) * kLanes + jj % kLanes]) + (i & 1);
    f[0] = w ? __bfloat162float(w[o.first(i)]) : 1.f;
    f[2] = w ? __bfloat162float(w[o.second(i)]) : 1.f;
  }
  uint64_t turn[kPairs];
  #pragma unroll
  for (int k = 0; k < kPairs; ++k) {
    const int j = lane + 32 * k;
    const L o(j % kLanes, p.rot);
    turn[k] = o.turns(j / kLanes) ? turn_step(p.inv_freq[o.freq(j / kLanes)]) : 0;
  }
  __syncthreads();
  float dqa[8], dqb[8], dka[8], dkb[8];
  #pragma unroll
  for (int i = 0; i < 8; ++i) dqa[i] = dqb[i] = dka[i] = dkb[i] = 0.f;
  int slot = 0;
  const int first = blockIdx.x * kWarps + warp;
  int next_pos = p.rot && first < tasks ? p.positions[first / p.parts] : 0;
  for (int task = first; task < tasks; task += stride) {
    const int t = task / p.parts, part = task - t * p.parts;
    uint4* out = reinterpret_cast<uint4*>(p.dqkv + static_cast<int64_t>(t) * p.ld_out);
    const int position = next_pos;
    if (p.rot && task + stride < tasks) next_pos = p.positions[(task + stride) / p.parts];
    __syncwarp();
    #pragma unroll
    for (int k = 0; k < kPairs; ++k) {
      const int j = lane + 32 * k, i = j / kLanes;
      float c, s;
      angle(p, position, turn[k], c, s);
      float* f = reinterpret_cast<float*>(&s_cs[warp][(i >> 1) * kLanes + j % kLanes]) + (i & 1);
      f[0] = c;
      f[2] = s;
      reinterpret_cast<float*>(&s_ns[warp][(i >> 1) * kLanes + j % kLanes])[i & 1] = -s;
    }
    __syncwarp();
    for (int g = part; g < groups; g += p.parts) {
      issue();
      copy_wait<kDepth - 1>();
      const uint4* in = ring + slot * (4 * 32);
      slot = slot + 1 == kDepth ? 0 : slot + 1;
      const int hh = g * kRw + sub;
      uint4 oa = in[0], ob = in[32];
      // KIND: query heads, key heads, or heads of two kinds in one group
      auto rows = [&](auto kind) {
        constexpr int KIND = decltype(kind)::value;
        const bool is_q = KIND == 0 || (KIND == 2 && hh < p.H);
        const bool is_v = KIND == 2 && hh >= p.H + p.H_kv;
        float fa[8], fb[8];
        L::unpack(oa, ob, fa, fb);
        auto back_turn = [&](int i) {
          const float4 c = s_cs[warp][(i >> 1) * kLanes + l];
          const float2 ns = s_ns[warp][(i >> 1) * kLanes + l];
          float ta0, ta1, tb0, tb1;
          fmul2(ta0, ta1, fb[i], fb[i + 1], c.z, c.w);
          fmul2(tb0, tb1, fa[i], fa[i + 1], ns.x, ns.y);
          ffma2(fa[i], fa[i + 1], fa[i], fa[i + 1], c.x, c.y, ta0, ta1);
          ffma2(fb[i], fb[i + 1], fb[i], fb[i + 1], c.x, c.y, tb0, tb1);
        };
        if (ln.ta && !is_v) {
          #pragma unroll
          for (int i = 0; i < (INTER ? 4 : 8); i += 2) back_turn(i);
        }
        if (INTER && ln.tb && !is_v) {
          #pragma unroll
          for (int i = 4; i < 8; i += 2) back_turn(i);
        }
        const bool normed = is_q ? p.wq != nullptr : !is_v && p.wk != nullptr;
        if (KIND == 2 ? p.wq != nullptr || p.wk != nullptr : normed) {
          float xa[8], xb[8];
          uint4 va = make_uint4(0u, 0u, 0u, 0u), vb = va;
          if (normed) {
            va = in[64];
            vb = in[96];
          }
          L::unpack(va, vb, xa, xb);
          float r = rsqrtf(row_sum<D>(sum_squares(xa, xb)) * (1.f / D) + p.eps);
          r = normed ? r : 1.f;
          #pragma unroll
          for (int i = 0; i < 8; i += 2) {
            fmul2(fa[i], fa[i + 1], fa[i], fa[i + 1], r, r);
            fmul2(fb[i], fb[i + 1], fb[i], fb[i + 1], r, r);
          }
          if constexpr (KIND < 2) {
            float(&da)[8] = KIND == 0 ? dqa : dka;
            float(&db)[8] = KIND == 0 ? dqb : dkb;
            #pragma unroll
            for (int i = 0; i < 8; i += 2) {
              ffma2(da[i], da[i + 1], fa[i], fa[i + 1], xa[i], xa[i + 1], da[i], da[i + 1]);
              ffma2(db[i], db[i + 1], fb[i], fb[i + 1], xb[i], xb[i + 1], db[i], db[i + 1]);
            }
          } else {
            #pragma unroll
            for (int i = 0; i < 8; ++i) {
              if (is_q) {
                dqa[i] = fmaf(fa[i], xa[i], dqa[i]);
                dqb[i] = fmaf(fb[i], xb[i], dqb[i]);
              } else if (!is_v) {
                dka[i] = fmaf(fa[i], xa[i], dka[i]);
                dkb[i] = fmaf(fb[i], xb[i], dkb[i]);
              }
            }
          }
          float d0 = 0.f, d1 = 0.f;
          if (KIND < 2 || normed) {
            const float4* wt = &s_w[is_q ? 0 : 1][l];
            #pragma unroll
            for (int i = 0; i < 8; i += 2) {
              const float4 w = wt[(i >> 1) * kLanes];
              fmul2(fa[i], fa[i + 1], fa[i], fa[i + 1], w.x, w.y);
              fmul2(fb[i], fb[i + 1], fb[i], fb[i + 1], w.z, w.w);
              ffma2(d0, d1, fa[i], fa[i + 1], xa[i], xa[i + 1], d0, d1);
              ffma2(d0, d1, fb[i], fb[i + 1], xb[i], xb[i + 1], d0, d1);
            }
          }
          const float back = row_sum<D>(d0 + d1) * (-1.f / D) * (r * r);
          if (KIND < 2 || normed) {
            #pragma unroll
            for (int i = 0; i < 8; i += 2) {
              ffma2(fa[i], fa[i + 1], xa[i], xa[i + 1], back, back, fa[i], fa[i + 1]);
              ffma2(fb[i], fb[i + 1], xb[i], xb[i + 1], back, back, fb[i], fb[i + 1]);
            }
          }
        }
        if (!is_v) L::pack(fa, fb, oa, ob);
      };
      const int h0 = g * kRw;
      if (h0 + kRw <= p.H) rows(std::integral_constant<int, 0>());
      else if (h0 >= p.H && h0 + kRw <= p.H + p.H_kv) rows(std::integral_constant<int, 1>());
      else if (h0 < p.H + p.H_kv) rows(std::integral_constant<int, 2>());
      if (hh < heads) {
        out[hh * (D / 8) + ln.a] = oa;
        out[hh * (D / 8) + ln.b] = ob;
      }
    }
  }
  if (!p.partial) return;
  // the CTA's sums: over the rows of a warp's groups by shuffles, over the warps in order
  #pragma unroll
  for (int k = 0; k < 2; ++k) {
    float* va = k ? dka : dqa;
    float* vb = k ? dkb : dqb;
    #pragma unroll
    for (int i = 0; i < 8; ++i)
      #pragma unroll
      for (int off = 16; off >= kLanes; off >>= 1) {
        va[i] += __shfl_xor_sync(0xffffffffu, va[i], off);
        vb[i] += __shfl_xor_sync(0xffffffffu, vb[i], off);
      }
    __syncthreads();
    if (sub == 0) {
      #pragma unroll
      for (int i = 0; i < 8; ++i) {
        s_dw[warp][ln.first(i)] = va[i];
        s_dw[warp][ln.second(i)] = vb[i];
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

// dwq (block 0) and dwk (block 1): the CTAs' shares, in runs of every 32nd or 64th CTA summed side by
// side (four columns a thread, ten loads in flight at most), then joined in order.
template <int D>
__global__ void __launch_bounds__(1024) rope_dw_kernel(const float* partial, int ctas, float* dwq,
                                                       float* dwk) {
  constexpr int kRuns = 1024 / (D / 4), kLoads = (kRopeBwdCtas + kRuns - 1) / kRuns;
  __shared__ float4 s_sum[kRuns][D / 4];
  float* out = blockIdx.x ? dwk : dwq;
  const int c4 = threadIdx.x % (D / 4), run = threadIdx.x / (D / 4);
  pdl_wait();
  if (!out) return;
  float4 x[kLoads];
  #pragma unroll
  for (int k = 0; k < kLoads; ++k) {
    const int i = run + k * kRuns;
    x[k] = i < ctas ? reinterpret_cast<const float4*>(partial)[(static_cast<size_t>(i) * 2 + blockIdx.x) * (D / 4) + c4]
                    : make_float4(0.f, 0.f, 0.f, 0.f);
  }
  float4 v = x[0];
  #pragma unroll
  for (int k = 1; k < kLoads; ++k) {
    v.x += x[k].x;
    v.y += x[k].y;
    v.z += x[k].z;
    v.w += x[k].w;
  }
  s_sum[run][c4] = v;
  __syncthreads();
  if (threadIdx.x < D) {
    const float* column = reinterpret_cast<const float*>(s_sum) + threadIdx.x;
    float sum = 0.f;
    #pragma unroll 16
    for (int i = 0; i < kRuns; ++i) sum += column[i * D];
    out[threadIdx.x] = sum;
  }
}

template <int D, bool INTER>
cudaError_t launch_fwd(const RopeParams& p, int kind, int ctas, cudaStream_t st) {
  const dim3 grid(static_cast<unsigned>(ctas));
  if (kind == kCacheNone)
    return launch_dependent(qkv_rope_kernel<D, INTER, kCacheNone>, grid, kRopeThreads, 0, st, p);
  if (kind == kCacheBf16)
    return launch_dependent(qkv_rope_kernel<D, INTER, kCacheBf16>, grid, kRopeThreads, 0, st, p);
  return launch_dependent(qkv_rope_kernel<D, INTER, kCacheE4m3>, grid, kRopeThreads, 0, st, p);
}

// Warps that share a token: the count up to 32 (a power of two where they work as a team) that minimises
// rounds of `resident` warps times a warp's work in groups of rows, its own share and `fixed` for the
// token's angles (the smaller on ties).  Many tokens: few, so that the angles are not computed again;
// few tokens: as many as have rows.
int parts_of(int tokens, int groups, int resident, int fixed, bool team) {
  int best = 1;
  int64_t best_cost = -1;
  for (int parts = 1; parts <= 32 && parts < 2 * groups; parts += team ? parts : 1) {
    const int64_t rounds = (static_cast<int64_t>(tokens) * parts + resident - 1) / resident;
    const int64_t cost = rounds * ((groups + parts - 1) / parts + fixed);
    if (best_cost < 0 || cost < best_cost) {
      best_cost = cost;
      best = parts;
    }
  }
  return best;
}
int groups_of(const RopeParams& p, int d) {
  const int rows = 32 / (d / 16);
  return (p.H + 2 * p.H_kv + rows - 1) / rows;
}

}  // namespace

cudaError_t launch_qkv_rope(RopeParams& p, int d, bool interleaved, int kind, cudaStream_t st) {
  // three CTAs an SM (two where E4M3 codes are written, for which the count was not measured apart); the
  // angles and coefficients of a token take about as long as two groups
  p.parts = parts_of(p.tokens, groups_of(p, d), 3 * 152 * kWarps, 2, true);
  const int ctas = static_cast<int>((static_cast<int64_t>(p.tokens) * p.parts + kWarps - 1) / kWarps);
  if (d == 64)
    return interleaved ? launch_fwd<64, true>(p, kind, ctas, st)
                       : launch_fwd<64, false>(p, kind, ctas, st);
  return interleaved ? launch_fwd<128, true>(p, kind, ctas, st)
                     : launch_fwd<128, false>(p, kind, ctas, st);
}

namespace {

template <int D, bool INTER>
cudaError_t launch_bwd(const RopeParams& p, int ctas, cudaStream_t st) {
  constexpr int kSmem = kWarps * kDepth * 4 * 32 * 16;
  auto* kernel = qkv_rope_bwd_kernel<D, INTER>;
  static std::atomic<uint64_t> attr_done{0};
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  const uint64_t bit = 1ull << (dev & 63);
  if (!(attr_done.load(std::memory_order_acquire) & bit)) {
    e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem);
    if (e != cudaSuccess) return e;
    attr_done.fetch_or(bit, std::memory_order_acq_rel);
  }
  e = launch_dependent(kernel, dim3(static_cast<unsigned>(ctas)), kRopeThreads, kSmem, st, p);
  if (e != cudaSuccess || !p.partial) return e;
  // the sums of the CTAs' shares: set up while the rows' kernel still runs
  return launch_dependent(rope_dw_kernel<D>, dim3(2), 1024, 0, st,
                          static_cast<const float*>(p.partial), ctas, p.dwq, p.dwk);
}

}  // namespace

cudaError_t launch_qkv_rope_bwd(RopeParams& p, int d, bool interleaved, cudaStream_t st) {
  // the angles of a token take about as long as one group
  p.parts = parts_of(p.tokens, groups_of(p, d), kRopeBwdCtas * kWarps, 1, false);
  const int64_t want = (static_cast<int64_t>(p.tokens) * p.parts + kWarps - 1) / kWarps;
  const int ctas = static_cast<int>(want < kRopeBwdCtas ? want : kRopeBwdCtas);
  if (d == 64) return interleaved ? launch_bwd<64, true>(p, ctas, st) : launch_bwd<64, false>(p, ctas, st);
  return interleaved ? launch_bwd<128, true>(p, ctas, st) : launch_bwd<128, false>(p, ctas, st);
}

}  // namespace attn
