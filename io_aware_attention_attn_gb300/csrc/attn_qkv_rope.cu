// attn_qkv_rope.cu -- the step before attention and its backward: RMS norm of each query and key
// head, rotation by position, token-major rows to head-major tensors, rows into a paged cache.
//
// A head's row of d elements is held by d/16 lanes with 16 elements each, as two 16-byte chunks
// chosen so that every pair (a, b) of the rotation lies in one lane: chunks l and l + rot/16 when
// element i turns with i + rot/2, any two when 2i turns with 2i + 1.  The mean of squares is then
// the only value that crosses lanes.  A CTA takes a few tokens and all (or, when there are few
// tokens, some) of their heads; cos and sin are computed once per token and pair into shared
// memory and shared by the heads.
//
// Angles: t = position * inv_freq modulo one turn, in 64-bit fixed point (a turn is 2^64), so the
// product wraps exactly and a position of 2^20 costs no accuracy; the top 32 bits go to sincospi.
// A float64 frequency leaves position * 2^-53 relative error at most.
//
// What bounds it: memory, one read and one write of every row.
#include "attn_gen.h"
#include "sm103_ptx.cuh"

#include <cmath>

namespace attn {
namespace {

constexpr int kBatch = 4;  // rows a thread loads before it uses the first

// cos and sin (times rope_scale) of the CTA's tokens, [token][rot/2] each.
__device__ __forceinline__ void fill_angles(const RopeParams& p, int t0, int nt, float* s_cos,
                                            float* s_sin) {
  const int nf = p.rot >> 1;
  for (int i = threadIdx.x; i < nt * nf; i += kRopeThreads) {
    const int tok = i / nf, f = i - tok * nf;
    double turns = p.inv_freq[f] * 0.15915494309189533577;  // 1 / (2 pi)
    turns -= rint(turns);
    const uint64_t step = static_cast<uint64_t>(__double2ll_rn(turns * 18446744073709551616.0));
    const uint64_t phase =
        static_cast<uint64_t>(static_cast<int64_t>(p.positions[t0 + tok])) * step;
    const int half_turns = static_cast<int>(phase >> 32);  // 2^31 is half a turn
    float s, c;
    sincospif(static_cast<float>(half_turns) * 0x1p-31f, &s, &c);
    s_cos[i] = c * p.rope_scale;
    s_sin[i] = s * p.rope_scale;
  }
}

// The two 16-byte chunks of a lane, and the first pair of each that turns (-1: none).
template <int D, bool INTER>
struct Chunks {
  int a, b, fa, fb;
  __device__ __forceinline__ Chunks(int l, int rot) {
    constexpr int kLanes = D / 16;
    if (INTER) {
      a = l;
      b = l + kLanes;
      fa = 8 * a < rot ? 4 * a : -1;
      fb = 8 * b < rot ? 4 * b : -1;
    } else {
      const int half = rot >> 4;
      a = l < half ? l : 2 * half + 2 * (l - half);
      b = l < half ? l + half : a + 1;
      fa = fb = l < half ? 8 * l : -1;
    }
  }
};

__device__ __forceinline__ void unpack8(const uint4& w, float* f) {
  f[0] = bf16lo_to_f32(w.x); f[1] = bf16hi_to_f32(w.x);
  f[2] = bf16lo_to_f32(w.y); f[3] = bf16hi_to_f32(w.y);
  f[4] = bf16lo_to_f32(w.z); f[5] = bf16hi_to_f32(w.z);
  f[6] = bf16lo_to_f32(w.w); f[7] = bf16hi_to_f32(w.w);
}
__device__ __forceinline__ uint4 pack8(const float* f) {
  return make_uint4(pack_bf16x2(f[0], f[1]), pack_bf16x2(f[2], f[3]), pack_bf16x2(f[4], f[5]),
                    pack_bf16x2(f[6], f[7]));
}

// Turns a lane's 16 elements by its token's angles (SIGN = -1: back).
template <int D, bool INTER, int SIGN>
__device__ __forceinline__ void turn(float* f, const Chunks<D, INTER>& ch, const float* cs,
                                     const float* sn) {
  if (INTER) {
    #pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int f0 = h ? ch.fb : ch.fa;
      if (f0 < 0) continue;
      const float4 c4 = *reinterpret_cast<const float4*>(cs + f0);
      const float4 s4 = *reinterpret_cast<const float4*>(sn + f0);
      const float c[4] = {c4.x, c4.y, c4.z, c4.w};
      const float s[4] = {s4.x, s4.y, s4.z, s4.w};
      #pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float x = f[8 * h + 2 * i], y = f[8 * h + 2 * i + 1];
        f[8 * h + 2 * i] = x * c[i] - SIGN * y * s[i];
        f[8 * h + 2 * i + 1] = y * c[i] + SIGN * x * s[i];
      }
    }
  } else if (ch.fa >= 0) {
    #pragma unroll
    for (int h = 0; h < 2; ++h) {
      const float4 c4 = *reinterpret_cast<const float4*>(cs + ch.fa + 4 * h);
      const float4 s4 = *reinterpret_cast<const float4*>(sn + ch.fa + 4 * h);
      const float c[4] = {c4.x, c4.y, c4.z, c4.w};
      const float s[4] = {s4.x, s4.y, s4.z, s4.w};
      #pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float x = f[4 * h + i], y = f[8 + 4 * h + i];
        f[4 * h + i] = x * c[i] - SIGN * y * s[i];
        f[8 + 4 * h + i] = y * c[i] + SIGN * x * s[i];
      }
    }
  }
}

template <int D>
__device__ __forceinline__ float row_sum(float v) {
  #pragma unroll
  for (int off = D / 32; off > 0; off >>= 1) v += __shfl_xor_sync(0xffffffffu, v, off);
  return v;
}

// A row's E4M3 codes and scale into the cache.
template <int D>
__device__ __forceinline__ void store_codes(const float* f, uint8_t* row, float* scale, int ca,
                                            int cb, bool write, bool first_lane) {
  float amax = 0.f;
  #pragma unroll
  for (int i = 0; i < 16; ++i) amax = fmaxf(amax, fabsf(f[i]));
  #pragma unroll
  for (int off = D / 32; off > 0; off >>= 1)
    amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, off));
  float sc = __fdiv_rn(amax, 448.f);
  if (!(sc >= 0x1p-126f)) sc = 1.f;
  if (!write) return;
  uint32_t w[4];
  #pragma unroll
  for (int i = 0; i < 4; ++i)
    w[i] = static_cast<uint32_t>(pack_e4m3x2(__fdiv_rn(f[4 * i], sc), __fdiv_rn(f[4 * i + 1], sc))) |
           static_cast<uint32_t>(pack_e4m3x2(__fdiv_rn(f[4 * i + 2], sc),
                                             __fdiv_rn(f[4 * i + 3], sc))) << 16;
  *reinterpret_cast<uint2*>(row + 8 * ca) = make_uint2(w[0], w[1]);
  *reinterpret_cast<uint2*>(row + 8 * cb) = make_uint2(w[2], w[3]);
  if (first_lane) *scale = sc;
}

template <int D, bool INTER, int CACHE>
__global__ void __launch_bounds__(kRopeThreads) qkv_rope_kernel(RopeParams p) {
  extern __shared__ __align__(16) float s_angles[];
  constexpr int kLanes = D / 16, kRows = kRopeThreads / kLanes;
  const int l = threadIdx.x % kLanes, grp = threadIdx.x / kLanes;
  const Chunks<D, INTER> ch(l, p.rot);
  const int heads = p.H + 2 * p.H_kv;
  const int t0 = blockIdx.x * p.tok_cta, nt = min(p.tok_cta, p.tokens - t0);
  const int h0 = blockIdx.y * p.head_cta, nh = min(p.head_cta, heads - h0);
  const int rows = nt * nh, nf = p.rot >> 1;
  float* s_cos = s_angles;
  float* s_sin = s_angles + p.tok_cta * nf;
  uint4 xa[kBatch], xb[kBatch];
  auto load = [&](int base) {
    #pragma unroll
    for (int u = 0; u < kBatch; ++u) {
      const int r = base + u * kRows + grp;
      if (r < rows) {
        const int tok = r / nh;
        const uint4* src = reinterpret_cast<const uint4*>(
            p.qkv + static_cast<int64_t>(t0 + tok) * p.ld + (h0 + r - tok * nh) * D);
        xa[u] = __ldcs(src + ch.a);
        xb[u] = __ldcs(src + ch.b);
      } else {
        xa[u] = xb[u] = make_uint4(0u, 0u, 0u, 0u);
      }
    }
  };
  load(0);
  fill_angles(p, t0, nt, s_cos, s_sin);
  __syncthreads();
  for (int base = 0; base < rows; base += kBatch * kRows) {
    if (base > 0) load(base);
    #pragma unroll
    for (int u = 0; u < kBatch; ++u) {
      if (base + u * kRows >= rows) break;  // the same for all threads
      const int r = base + u * kRows + grp;
      const bool live = r < rows;
      const int tok = live ? r / nh : 0;
      const int hh = live ? h0 + r - tok * nh : 0;
      const bool is_q = hh < p.H, is_v = hh >= p.H + p.H_kv;
      const int h = is_q ? hh : is_v ? hh - p.H - p.H_kv : hh - p.H;
      float f[16];
      unpack8(xa[u], f);
      unpack8(xb[u], f + 8);
      const __nv_bfloat16* w = is_q ? p.wq : is_v ? nullptr : p.wk;
      float ss = 0.f;
      #pragma unroll
      for (int i = 0; i < 16; ++i) ss = fmaf(f[i], f[i], ss);
      ss = row_sum<D>(ss);
      if (w) {
        const float rn = rsqrtf(ss * (1.f / D) + p.eps);
        float wf[16];
        unpack8(__ldg(reinterpret_cast<const uint4*>(w) + ch.a), wf);
        unpack8(__ldg(reinterpret_cast<const uint4*>(w) + ch.b), wf + 8);
        #pragma unroll
        for (int i = 0; i < 16; ++i) f[i] = f[i] * rn * wf[i];
      }
      if (!is_v) turn<D, INTER, 1>(f, ch, s_cos + tok * nf, s_sin + tok * nf);
      const int t = t0 + tok;
      const uint4 oa = pack8(f), ob = pack8(f + 8);
      __nv_bfloat16* out = is_q ? p.q : is_v ? p.v : p.k;
      if (live && out) {
        const int b = t / p.N, n = t - b * p.N;
        uint4* dst = reinterpret_cast<uint4*>(
            out + ((static_cast<int64_t>(b) * (is_q ? p.H : p.H_kv) + h) * p.N + n) * D);
        dst[ch.a] = oa;
        dst[ch.b] = ob;
      }
      if (CACHE != kCacheNone) {
        const int64_t slot = live && !is_q ? p.slots[t] : -1;
        const int64_t page = slot >> p.page_shift;
        const bool write = slot >= 0 && page < p.num_pages;
        if (slot >= 0 && !write) atomicCAS(p.status, 0, kStatusBadPage);
        const int64_t row =
            (static_cast<int64_t>(h) << p.page_shift) + (slot & ((1 << p.page_shift) - 1));
        uint8_t* base8 = is_v ? p.vc : p.kc;
        const int64_t at = page * p.page_stride + row * D;
        if (CACHE == kCacheBf16) {
          if (write) {
            uint4* dst = reinterpret_cast<uint4*>(base8 + 2 * at);
            dst[ch.a] = oa;
            dst[ch.b] = ob;
          }
        } else {
          store_codes<D>(f, base8 + (write ? at : 0),
                         (is_v ? p.vs : p.ks) +
                             (write ? ((page * p.H_kv) << p.page_shift) + row : 0),
                         ch.a, ch.b, write, l == 0);
        }
      }
    }
  }
}

// Gradients of the rows, and each CTA's share of the weights' gradients.
template <int D, bool INTER>
__global__ void __launch_bounds__(kRopeThreads) qkv_rope_bwd_kernel(RopeParams p) {
  extern __shared__ __align__(16) float s_angles[];
  constexpr int kLanes = D / 16, kRows = kRopeThreads / kLanes, kWarps = kRopeThreads / 32;
  __shared__ __align__(16) float s_dw[kWarps][D];
  const int l = threadIdx.x % kLanes, grp = threadIdx.x / kLanes;
  const Chunks<D, INTER> ch(l, p.rot);
  const int heads = p.H + 2 * p.H_kv, nf = p.rot >> 1;
  float* s_cos = s_angles;
  float* s_sin = s_angles + p.tok_cta * nf;
  float dwq[16], dwk[16];
  #pragma unroll
  for (int i = 0; i < 16; ++i) dwq[i] = dwk[i] = 0.f;
  const int groups = (p.tokens + p.tok_cta - 1) / p.tok_cta;
  for (int g = blockIdx.x; g < groups; g += gridDim.x) {
    const int t0 = g * p.tok_cta, nt = min(p.tok_cta, p.tokens - t0);
    const int rows = nt * heads;
    __syncthreads();
    fill_angles(p, t0, nt, s_cos, s_sin);
    __syncthreads();
    for (int base = 0; base < rows; base += kRows) {
      const int r = base + grp;
      const bool live = r < rows;
      const int tok = live ? r / heads : 0;
      const int hh = live ? r - tok * heads : 0;
      const bool is_q = hh < p.H, is_v = hh >= p.H + p.H_kv;
      const int h = is_q ? hh : is_v ? hh - p.H - p.H_kv : hh - p.H;
      const int t = t0 + tok, b = t / p.N, n = t - b * p.N;
      const __nv_bfloat16* w = is_q ? p.wq : is_v ? nullptr : p.wk;
      const __nv_bfloat16* dy = is_q ? p.dq : is_v ? p.dv : p.dk;
      float gr[16], x[16];
      #pragma unroll
      for (int i = 0; i < 16; ++i) gr[i] = x[i] = 0.f;
      if (live) {
        const uint4* src = reinterpret_cast<const uint4*>(
            dy + ((static_cast<int64_t>(b) * (is_q ? p.H : p.H_kv) + h) * p.N + n) * D);
        unpack8(__ldcs(src + ch.a), gr);
        unpack8(__ldcs(src + ch.b), gr + 8);
        if (w) {
          const uint4* xs = reinterpret_cast<const uint4*>(p.qkv + static_cast<int64_t>(t) * p.ld +
                                                           hh * D);
          unpack8(__ldcs(xs + ch.a), x);
          unpack8(__ldcs(xs + ch.b), x + 8);
        }
      }
      if (!is_v) turn<D, INTER, -1>(gr, ch, s_cos + tok * nf, s_sin + tok * nf);
      float wf[16], ss = 0.f, dot = 0.f;
      if (w) {
        unpack8(__ldg(reinterpret_cast<const uint4*>(w) + ch.a), wf);
        unpack8(__ldg(reinterpret_cast<const uint4*>(w) + ch.b), wf + 8);
        #pragma unroll
        for (int i = 0; i < 16; ++i) {
          ss = fmaf(x[i], x[i], ss);
          dot = fmaf(gr[i] * wf[i], x[i], dot);
        }
      }
      ss = row_sum<D>(ss);
      dot = row_sum<D>(dot);
      if (w) {
        const float rn = rsqrtf(ss * (1.f / D) + p.eps);
        const float back = rn * rn * dot * (1.f / D);
        #pragma unroll
        for (int i = 0; i < 16; ++i) {
          const float gx = gr[i] * x[i] * rn;
          if (is_q) dwq[i] += gx; else dwk[i] += gx;
          gr[i] = rn * (gr[i] * wf[i] - x[i] * back);
        }
      }
      if (live) {
        uint4* dst =
            reinterpret_cast<uint4*>(p.dqkv + static_cast<int64_t>(t) * p.ld_out + hh * D);
        dst[ch.a] = pack8(gr);
        dst[ch.b] = pack8(gr + 8);
      }
    }
  }
  if (!p.partial) return;
  // the CTA's sums: over the warp's row groups by shuffles, over the warps in order
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  #pragma unroll
  for (int which = 0; which < 2; ++which) {
    float* acc = which ? dwk : dwq;
    #pragma unroll
    for (int i = 0; i < 16; ++i)
      #pragma unroll
      for (int off = 16; off >= kLanes; off >>= 1)
        acc[i] += __shfl_xor_sync(0xffffffffu, acc[i], off);
    __syncthreads();
    if (lane < kLanes) {
      #pragma unroll
      for (int i = 0; i < 8; ++i) {
        s_dw[warp][8 * ch.a + i] = acc[i];
        s_dw[warp][8 * ch.b + i] = acc[8 + i];
      }
    }
    __syncthreads();
    if (threadIdx.x < D) {
      float v = 0.f;
      #pragma unroll
      for (int wi = 0; wi < kWarps; ++wi) v += s_dw[wi][threadIdx.x];
      p.partial[(static_cast<size_t>(blockIdx.x) * 2 + which) * D + threadIdx.x] = v;
    }
  }
}

// dwq (block 0) and dwk (block 1): the CTAs' shares, 8 runs of CTAs summed side by side, then joined
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
cudaError_t launch_fwd(const RopeParams& p, int kind, dim3 grid, int smem, cudaStream_t st) {
  if (kind == kCacheNone) qkv_rope_kernel<D, INTER, kCacheNone><<<grid, kRopeThreads, smem, st>>>(p);
  else if (kind == kCacheBf16)
    qkv_rope_kernel<D, INTER, kCacheBf16><<<grid, kRopeThreads, smem, st>>>(p);
  else qkv_rope_kernel<D, INTER, kCacheE4m3><<<grid, kRopeThreads, smem, st>>>(p);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_qkv_rope(RopeParams& p, int d, bool interleaved, int kind, cudaStream_t st) {
  const int heads = p.H + 2 * p.H_kv, rows_cta = kRopeThreads / (d / 16);
  // Enough tokens for four CTAs of four tokens on every SM: four tokens a CTA share the angles'
  // work and a CTA's rows of one head are neighbours.  Fewer: one row a thread, for latency.
  const bool many = p.tokens >= 4 * 4 * 152;
  p.tok_cta = many ? 4 : 1;
  p.head_cta = many ? heads : rows_cta;
  const dim3 grid((p.tokens + p.tok_cta - 1) / p.tok_cta, (heads + p.head_cta - 1) / p.head_cta);
  const int smem = p.tok_cta * p.rot * 4;
  if (d == 64)
    return interleaved ? launch_fwd<64, true>(p, kind, grid, smem, st)
                       : launch_fwd<64, false>(p, kind, grid, smem, st);
  return interleaved ? launch_fwd<128, true>(p, kind, grid, smem, st)
                     : launch_fwd<128, false>(p, kind, grid, smem, st);
}

cudaError_t launch_qkv_rope_bwd(RopeParams& p, int d, bool interleaved, cudaStream_t st) {
  p.tok_cta = 4;
  const int groups = (p.tokens + p.tok_cta - 1) / p.tok_cta;
  const int ctas = groups < kRopeBwdMaxCtas ? groups : kRopeBwdMaxCtas;
  const int smem = p.tok_cta * p.rot * 4;
  if (d == 64) {
    if (interleaved) qkv_rope_bwd_kernel<64, true><<<ctas, kRopeThreads, smem, st>>>(p);
    else qkv_rope_bwd_kernel<64, false><<<ctas, kRopeThreads, smem, st>>>(p);
  } else {
    if (interleaved) qkv_rope_bwd_kernel<128, true><<<ctas, kRopeThreads, smem, st>>>(p);
    else qkv_rope_bwd_kernel<128, false><<<ctas, kRopeThreads, smem, st>>>(p);
  }
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess || !p.partial) return e;
  rope_dw_kernel<<<2, 1024, 0, st>>>(p.partial, ctas, d, p.dwq, p.dwk);
  return cudaGetLastError();
}

}  // namespace attn
