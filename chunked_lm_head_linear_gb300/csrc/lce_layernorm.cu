// Layer norm in front of the LM head, forward and backward:
//
//   mu_i = mean_k x_ik,   r_i = 1 / sqrt(mean_k (x_ik - mu_i)^2 + eps)
//   xh   = (x - mu) r,    H = bf16(xh w + b)
//   g    = dH w,          dx = r (g - mean_k g - xh mean_k (g xh))
//   dw_k = sum_i dH_ik xh_ik,   db_k = sum_i dH_ik
//
// x is bf16 or fp32, w and b are fp32 or bf16 (or absent: ones and zeros), H
// and dH bf16. Everything between is fp32, one rounding a result. The variance
// is the mean of squared distances from the mean, taken in a second pass over
// the row: it does not cancel where the mean is large.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "lce_internal.h"
#include "sm100_ptx.cuh"

namespace lce {

namespace {

constexpr int kLnThreads = 256;
constexpr int kLnWarps = kLnThreads / 32;

// Eight neighbouring elements of a row, as they are held in registers.
template <bool F32>
struct Group;
template <>
struct Group<false> {
  uint4 v;
  static constexpr int kBytes = 16;
  __device__ __forceinline__ void load(const void* p, long long i) { v = static_cast<const uint4*>(p)[i]; }
  __device__ __forceinline__ void clear() { v = make_uint4(0u, 0u, 0u, 0u); }
  __device__ __forceinline__ void get(float (&f)[8]) const {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      f[2 * q] = __uint_as_float(w[q] << 16);
      f[2 * q + 1] = __uint_as_float(w[q] & 0xffff0000u);
    }
  }
};
template <>
struct Group<true> {
  float4 a, b;
  static constexpr int kBytes = 32;
  __device__ __forceinline__ void load(const void* p, long long i) {
    a = static_cast<const float4*>(p)[2 * i];
    b = static_cast<const float4*>(p)[2 * i + 1];
  }
  __device__ __forceinline__ void clear() { a = b = make_float4(0.f, 0.f, 0.f, 0.f); }
  __device__ __forceinline__ void get(float (&f)[8]) const {
    f[0] = a.x; f[1] = a.y; f[2] = a.z; f[3] = a.w;
    f[4] = b.x; f[5] = b.y; f[6] = b.z; f[7] = b.w;
  }
};

__device__ __forceinline__ void store8(void* p, long long i, const float (&f)[8], bool f32) {
  if (f32) {
    static_cast<float4*>(p)[2 * i] = make_float4(f[0], f[1], f[2], f[3]);
    static_cast<float4*>(p)[2 * i + 1] = make_float4(f[4], f[5], f[6], f[7]);
  } else {
    static_cast<uint4*>(p)[i] = make_uint4(pack_bf16x2(f[0], f[1]), pack_bf16x2(f[2], f[3]), pack_bf16x2(f[4], f[5]),
                                           pack_bf16x2(f[6], f[7]));
  }
}

// Eight weights (or biases) of column group i; `none` where there are none.
__device__ __forceinline__ void param8(const void* w, int bf16, int i, float none, float (&f)[8]) {
  if (w == nullptr) {
#pragma unroll
    for (int k = 0; k < 8; ++k) f[k] = none;
  } else if (bf16) {
    Group<false> g;
    g.v = __ldg(static_cast<const uint4*>(w) + i);
    g.get(f);
  } else {
    const float4 a = __ldg(static_cast<const float4*>(w) + 2 * i), b = __ldg(static_cast<const float4*>(w) + 2 * i + 1);
    f[0] = a.x; f[1] = a.y; f[2] = a.z; f[3] = a.w;
    f[4] = b.x; f[5] = b.y; f[6] = b.z; f[7] = b.w;
  }
}

__device__ __forceinline__ float warp_total(float v) {
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) v += __shfl_xor_sync(0xffffffffu, v, off);
  return v;
}

// Persistent warps, R rows at a time; lane l owns the column groups l, l + 32,
// ... of a row, of which the first G stay in registers through the three passes
// (sum, squares, result) and the rest, of rows longer than 256 G, is read again.
template <bool F32, int G, int R>
__global__ void __launch_bounds__(kLnThreads) k_layernorm_fwd(const LayerNormArgs p) {
  grid_dep_wait();
  grid_dep_launch();
  const int lane = threadIdx.x & 31, groups = p.d / 8;
  const long long warps = static_cast<long long>(gridDim.x) * kLnWarps;
  const float d = static_cast<float>(p.d);
  for (long long i0 = (static_cast<long long>(blockIdx.x) * kLnWarps + (threadIdx.x >> 5)) * R; i0 < p.N; i0 += warps * R) {
    Group<F32> v[R][G];
    float sum[R], sq[R];
#pragma unroll
    for (int q = 0; q < R; ++q) {
#pragma unroll
      for (int j = 0; j < G; ++j) {
        const int gI = lane + 32 * j;
        if (i0 + q < p.N && gI < groups)
          v[q][j].load(p.x, (i0 + q) * groups + gI);
        else
          v[q][j].clear();
      }
    }
#pragma unroll
    for (int q = 0; q < R; ++q) {
      sum[q] = sq[q] = 0.f;
      float f[8];
#pragma unroll
      for (int j = 0; j < G; ++j) {
        v[q][j].get(f);
#pragma unroll
        for (int k = 0; k < 8; ++k) sum[q] += f[k];
      }
      if (R == 1)
        for (int gI = lane + 32 * G; gI < groups; gI += 32) {
          Group<F32> t;
          t.load(p.x, i0 * groups + gI);
          t.get(f);
#pragma unroll
          for (int k = 0; k < 8; ++k) sum[q] += f[k];
        }
    }
#pragma unroll
    for (int q = 0; q < R; ++q) sum[q] = warp_total(sum[q]) / d;  // the mean from here on
#pragma unroll
    for (int q = 0; q < R; ++q) {
      float f[8];
#pragma unroll
      for (int j = 0; j < G; ++j) {
        v[q][j].get(f);
        if (lane + 32 * j < groups) {
#pragma unroll
          for (int k = 0; k < 8; ++k) sq[q] = fmaf(f[k] - sum[q], f[k] - sum[q], sq[q]);
        }
      }
      if (R == 1)
        for (int gI = lane + 32 * G; gI < groups; gI += 32) {
          Group<F32> t;
          t.load(p.x, i0 * groups + gI);
          t.get(f);
#pragma unroll
          for (int k = 0; k < 8; ++k) sq[q] = fmaf(f[k] - sum[q], f[k] - sum[q], sq[q]);
        }
    }
#pragma unroll
    for (int q = 0; q < R; ++q) {
      sq[q] = 1.f / sqrtf(warp_total(sq[q]) / d + p.eps);  // 1 / deviation from here on
      if (lane == 0 && i0 + q < p.N) {
        if (p.mean != nullptr) p.mean[i0 + q] = sum[q];
        if (p.rstd != nullptr) p.rstd[i0 + q] = sq[q];
      }
    }
    auto result = [&](const Group<F32>& x, int gI, int q, const float (&w)[8], const float (&b)[8]) {
      float f[8];
      x.get(f);
#pragma unroll
      for (int k = 0; k < 8; ++k) f[k] = fmaf((f[k] - sum[q]) * sq[q], w[k], b[k]);
      store8(p.H, (i0 + q) * groups + gI, f, false);
    };
#pragma unroll
    for (int j = 0; j < G; ++j) {
      const int gI = lane + 32 * j;
      if (gI < groups) {
        float w[8], b[8];
        param8(p.w, p.w_bf16, gI, 1.f, w);
        param8(p.b, p.w_bf16, gI, 0.f, b);
#pragma unroll
        for (int q = 0; q < R; ++q)
          if (i0 + q < p.N) result(v[q][j], gI, q, w, b);
      }
    }
    if (R == 1)
      for (int gI = lane + 32 * G; gI < groups; gI += 32) {
        float w[8], b[8];
        param8(p.w, p.w_bf16, gI, 1.f, w);
        param8(p.b, p.w_bf16, gI, 0.f, b);
        Group<F32> t;
        t.load(p.x, i0 * groups + gI);
        result(t, gI, 0, w, b);
      }
  }
}

// dx, one warp per row, in two passes over it.
template <bool F32>
__global__ void __launch_bounds__(kLnThreads) k_layernorm_dx(const LayerNormArgs p) {
  grid_dep_wait();
  grid_dep_launch();
  const int lane = threadIdx.x & 31, groups = p.d / 8;
  const long long warps = static_cast<long long>(gridDim.x) * kLnWarps;
  const float inv_d = 1.f / static_cast<float>(p.d);
  for (long long i = static_cast<long long>(blockIdx.x) * kLnWarps + (threadIdx.x >> 5); i < p.N; i += warps) {
    const float mu = p.mean[i], r = p.rstd[i];
    float sg = 0.f, sx = 0.f;
    for (int gI = lane; gI < groups; gI += 32) {
      Group<F32> x;
      Group<false> h;
      float f[8], g[8], w[8];
      x.load(p.x, i * groups + gI);
      h.load(p.dH, i * groups + gI);
      param8(p.w, p.w_bf16, gI, 1.f, w);
      x.get(f);
      h.get(g);
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        g[k] *= w[k];
        sg += g[k];
        sx = fmaf(g[k], (f[k] - mu) * r, sx);
      }
    }
    sg = warp_total(sg) * inv_d;
    sx = warp_total(sx) * inv_d;
    for (int gI = lane; gI < groups; gI += 32) {
      Group<F32> x;
      Group<false> h;
      float f[8], g[8], w[8];
      x.load(p.x, i * groups + gI);
      h.load(p.dH, i * groups + gI);
      param8(p.w, p.w_bf16, gI, 1.f, w);
      x.get(f);
      h.get(g);
#pragma unroll
      for (int k = 0; k < 8; ++k) f[k] = r * (g[k] * w[k] - sg - (f[k] - mu) * r * sx);
      store8(p.dx, i * groups + gI, f, F32);
    }
  }
}

// Partial sums of dw and db: block (c, s) owns 256 columns and every gridDim.y-th
// group of 8 rows from the s-th on; warp q of it takes the rows q of its groups.
template <bool F32>
__global__ void __launch_bounds__(kLnThreads) k_layernorm_dw(const LayerNormArgs p) {
  grid_dep_wait();
  grid_dep_launch();
  __shared__ float red[kLnWarps][32][17];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, groups = p.d / 8;
  const int gI = blockIdx.x * 32 + lane;
  float aw[8] = {}, ab[8] = {};
  if (gI < groups)
    for (long long i = static_cast<long long>(blockIdx.y) * kLnWarps + warp; i < p.N; i += static_cast<long long>(gridDim.y) * kLnWarps) {
      const float mu = p.mean[i], r = p.rstd[i];
      Group<F32> x;
      Group<false> h;
      float f[8], g[8];
      x.load(p.x, i * groups + gI);
      h.load(p.dH, i * groups + gI);
      x.get(f);
      h.get(g);
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        aw[k] = fmaf(g[k], (f[k] - mu) * r, aw[k]);
        ab[k] += g[k];
      }
    }
#pragma unroll
  for (int k = 0; k < 8; ++k) {
    red[warp][lane][k] = aw[k];
    red[warp][lane][8 + k] = ab[k];
  }
  __syncthreads();
  // thread t: the two sums of column t of the block
  const int c = threadIdx.x, col = blockIdx.x * 256 + c;
  if (col >= p.d) return;
  float tw = 0.f, tb = 0.f;
  for (int q = 0; q < kLnWarps; ++q) {
    tw += red[q][c / 8][c % 8];
    tb += red[q][c / 8][8 + c % 8];
  }
  const long long parts = gridDim.y, at = static_cast<long long>(blockIdx.y) * p.d + col;
  p.part[at] = tw;
  p.part[parts * p.d + at] = tb;
}

// dw and db from their partial sums, in a fixed order: a block covers 32
// columns of one of them, warp s sums the parts s, s + 8, ... in order.
__global__ void __launch_bounds__(kLnThreads) k_layernorm_sum(const LayerNormArgs p, int parts) {
  grid_dep_wait();
  grid_dep_launch();
  __shared__ float red[kLnWarps][33];
  float* out = blockIdx.y == 0 ? p.dw : p.db;
  if (out == nullptr) return;
  const int lane = threadIdx.x & 31, s = threadIdx.x >> 5, k = blockIdx.x * 32 + lane;
  const float* part = p.part + static_cast<long long>(blockIdx.y) * parts * p.d;
  float t = 0.f;
  if (k < p.d)
    for (int b = s; b < parts; b += kLnWarps) t += part[static_cast<long long>(b) * p.d + k];
  red[s][lane] = t;
  __syncthreads();
  if (s == 0 && k < p.d) {
    for (int q = 1; q < kLnWarps; ++q) t += red[q][lane];
    out[k] = t;
  }
}

template <bool F32, int G, int R>
cudaError_t fwd(const LayerNormArgs& p, int num_sms, cudaStream_t s) {
  const long long need = (p.N + kLnWarps * R - 1) / (kLnWarps * R), most = 8LL * num_sms;
  return launch_k(k_layernorm_fwd<F32, G, R>, static_cast<unsigned>(need < most ? need : most), kLnThreads, 0, s, p);
}

template <bool F32>
cudaError_t fwd_rows(const LayerNormArgs& p, int num_sms, cudaStream_t s) {
  if (p.d <= 256) return fwd<F32, 1, 4>(p, num_sms, s);
  if (p.d <= 512) return fwd<F32, 2, 2>(p, num_sms, s);
  if (p.d <= 1024) return fwd<F32, 4, 1>(p, num_sms, s);
  if (p.d <= 2048) return fwd<F32, 8, 1>(p, num_sms, s);
  return fwd<F32, 16, 1>(p, num_sms, s);
}

template <bool F32>
cudaError_t bwd(const LayerNormArgs& p, int num_sms, cudaStream_t s) {
  if (p.dx != nullptr && p.N > 0) {
    const long long need = (p.N + kLnWarps - 1) / kLnWarps, most = 8LL * num_sms;
    const cudaError_t e =
        launch_k(k_layernorm_dx<F32>, static_cast<unsigned>(need < most ? need : most), kLnThreads, 0, s, p);
    if (e != cudaSuccess) return e;
  }
  if (p.dw == nullptr && p.db == nullptr) return cudaSuccess;
  const int parts = layernorm_parts(p.N, p.d);
  const cudaError_t e = launch_k(k_layernorm_dw<F32>, dim3((p.d + 255) / 256, parts), kLnThreads, 0, s, p);
  if (e != cudaSuccess) return e;
  return launch_k(k_layernorm_sum, dim3((p.d + 31) / 32, 2), kLnThreads, 0, s, p, parts);
}

}  // namespace

int layernorm_parts(long long N, long long d) {
  const long long rows = (N + kLnWarps - 1) / kLnWarps, most = 512 / ((d + 255) / 256) + 1;
  const long long parts = rows < most ? rows : most;
  return static_cast<int>(parts > 0 ? parts : 1);
}

cudaError_t launch_layernorm_fwd(const LayerNormArgs& p, int num_sms, cudaStream_t s) {
  if (p.N <= 0) return cudaSuccess;
  return p.x_f32 ? fwd_rows<true>(p, num_sms, s) : fwd_rows<false>(p, num_sms, s);
}

cudaError_t launch_layernorm_bwd(const LayerNormArgs& p, int num_sms, cudaStream_t s) {
  return p.x_f32 ? bwd<true>(p, num_sms, s) : bwd<false>(p, num_sms, s);
}

}  // namespace lce
