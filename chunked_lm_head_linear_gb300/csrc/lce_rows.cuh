// What the row kernels of the token operators and of the losses on
// log-probabilities share: a row's partial sums and their merge, the row of the
// gradient tile, sums over a block.
#pragma once

#include <math.h>

#include "lce_internal.h"
#include "sm100_ptx.cuh"

namespace lce {
namespace {

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;
constexpr float kFloor = -1.0e30f;   // stands in for -inf where it is multiplied by a zero probability
constexpr float kMasked = -1.0e30f;  // the logit of a column past the vocabulary: no probability, and finite over T

// ----------------------------------------------------------------------------
// A row's four numbers and their merge
// ----------------------------------------------------------------------------
// Merged under the row's maximum M, found first: a half tile below it moves its
// c into s, s' = f (s + c) and t' = f (t + (s + c) (m - M)/T), f = exp((m - M)/T).
struct RowSum {
  float s, t, c;
};

__device__ __forceinline__ void add_partial(RowSum& a, const float4& q, float M, float inv_t) {
  if (q.x == M) {
    a.s += q.y;
    a.t += q.z;
    a.c += q.w;
  } else {
    const float d = (q.x - M) * inv_t, f = ex2_approx(d * kLog2e), all = q.y + q.w;
    a.s = fmaf(all, f, a.s);
    a.t = fmaf(fmaf(all, fmaxf(d, kFloor), q.z), f, a.t);
  }
}
__device__ __forceinline__ RowSum warp_add(RowSum a) {
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) {
    a.s += __shfl_xor_sync(0xffffffffu, a.s, off);
    a.t += __shfl_xor_sync(0xffffffffu, a.t, off);
    a.c += __shfl_xor_sync(0xffffffffu, a.c, off);
  }
  return a;
}

__device__ __forceinline__ float warp_max(float v) {
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, off));
  return v;
}

constexpr int kGroups = 8;  // groups of 32 running sums a row is merged through

__device__ __forceinline__ RowSum add_groups(const RowSum* g) {
  RowSum a = g[0];
#pragma unroll
  for (int i = 1; i < kGroups; ++i) {
    a.s += g[i].s;
    a.t += g[i].t;
    a.c += g[i].c;
  }
  return a;
}

// log of the sum of exp((z - M)/T): log(c + s).
__device__ __forceinline__ float log_sum(const RowSum& a) { return logf(a.c) + log1pf(a.s / a.c); }

// ----------------------------------------------------------------------------
// The gradient tile
// ----------------------------------------------------------------------------
// A row of the gradient tile: entries p (c0 + c1 log p) with c0 = -a - e entropy
// and c1 = -e, and + a at the label (a = g_logp / T where the label is given,
// e = g_entropy / T), all over the row's scale. A row without upstream gradient
// is zero whatever its logits are: masked tokens may hold anything.
//
// The scale is the label's entry: usually by far the row's largest, it is 1 in
// the tile and not rounded, and dH, multiplied by the scale in fp32 behind its
// GEMM, is left with the rounding of its result. dW's operand is bf16(scale H):
// one rounding in place of the label entry's, but of every element on its own
// and so averaged over the row (errors against fp64, in units of one bf16
// rounding, 250 rows: dH 1.3-1.6 -> 1.0, bf16 dW 1.3-1.5 -> 1.2-1.3).
// An entry costs a sum, two fma, an exponential and a product: x = (z - m) k - L log2 e, p = 2^x,
// g = p (c0 + c1 x), with the row's maximum m and L = log sum exp((z - m)/T): x errs by its own
// rounding only, and log p + entropy keeps its relative precision in confident rows. Without them
// m = 0 and L = lse, whose rounding at the size of z / T is an error of all of the row's p alike
// (2^-23 |z / T|): the calls that have only lse take it for temperatures where that is small.
struct GradRow {
  float m = 0.f, k = 0.f, shift = 0.f;  // x = (z - m) k + shift
  float c0 = 0.f, c1 = 0.f;    // (-a - e entropy, -e ln 2) over the scale
  int y = -1;                  // the label, -1 where it is not given
  uint32_t keep = 0;           // 0: no upstream gradient, all bits: some
};

struct Upstream {
  float a, e;  // g_logp (0 where the label is not given) and g_entropy, over T
  int y;
};

__device__ __forceinline__ Upstream upstream(int r, const int64_t* labels, long long ignore_index, int V,
                                             const float* g_logp, const float* g_entropy, float inv_t) {
  const long long y = labels[r];
  Upstream u;
  u.y = y != ignore_index && y >= 0 && y < V ? static_cast<int>(y) : -1;
  u.a = u.y >= 0 ? g_logp[r] * inv_t : 0.f;
  u.e = g_entropy != nullptr ? g_entropy[r] * inv_t : 0.f;
  return u;
}

// The label's entry a (1 - p) - p e (log p + entropy), from its log-probability.
__device__ __forceinline__ float label_entry(const Upstream& u, float logp, const float* entropy, int r) {
  if (u.y < 0) return 0.f;
  float g = -expm1f(logp) * u.a;
  if (u.e != 0.f) g -= expf(logp) * u.e * (logp + entropy[r]);
  return g;
}

// The row's scale: that entry, or 1 where it is too small, or not a number, to divide by.
__device__ __forceinline__ float row_scale(const Upstream& u, float entry) {
  const float size = fabsf(entry);
  return size >= 1.0e-30f && size <= 1.0e30f && size >= 1.0e-12f * (fabsf(u.a) + fabsf(u.e)) ? entry : 1.f;
}

__device__ __forceinline__ GradRow grad_row(const Upstream& u, float scale, const float2* stats, const float* lse,
                                            const float* entropy, int r, float inv_t) {
  GradRow g;
  const float2 st = stats != nullptr ? stats[r] : make_float2(0.f, lse[r]);
  const float inv = 1.f / scale, e = u.e * inv;
  g.y = u.y;
  g.k = inv_t * kLog2e;
  g.m = st.x;
  g.shift = -st.y * kLog2e;
  g.c0 = -u.a * inv;
  if (u.e != 0.f) g.c0 -= e * entropy[r];
  g.c1 = -e * kLn2;
  g.keep = u.a == 0.f && u.e == 0.f ? 0u : ~0u;
  return g;
}

// Two entries, in bf16.
__device__ __forceinline__ uint32_t grad_pair(float z0, float z1, const GradRow& r) {
  const uint64_t x = fma_pair(add_pair(pair_f32(z0, z1), pair_f32(-r.m, -r.m)), pair_f32(r.k, r.k),
                              pair_f32(r.shift, r.shift));
  float x0, x1, g0, g1;
  unpair_f32(x, x0, x1);
  const uint64_t p = pair_f32(ex2_approx(x0), ex2_approx(x1));
  unpair_f32(mul_pair(p, fma_pair(x, pair_f32(r.c1, r.c1), pair_f32(r.c0, r.c0))), g0, g1);
  return pack_bf16x2(g0, g1) & r.keep;
}
// Ht = bf16(scale H), a row of dW's second operand; zeros without a share in the gradient: 0 x NaN is not 0.
__device__ __forceinline__ void scale_row(const uint4* hr, uint4* tr, int groups, float scale, bool share, int tid,
                                          int threads) {
  for (int i = tid; i < groups; i += threads) {
    const uint4 h = share ? hr[i] : make_uint4(0u, 0u, 0u, 0u);
    const uint32_t w[4] = {h.x, h.y, h.z, h.w};
    uint32_t o[4];
#pragma unroll
    for (int q = 0; q < 4; ++q)
      o[q] = pack_bf16x2(__uint_as_float(w[q] << 16) * scale, __uint_as_float(w[q] & 0xffff0000u) * scale);
    tr[i] = make_uint4(o[0], o[1], o[2], o[3]);
  }
}

// A row of the gradient tile from its stored logits: 4 bytes read and 2 written a logit. A row without
// upstream gradient is written without reading its logits. label: the label's entry, written by the
// thread that holds its eight columns.
__device__ __forceinline__ void write_grad_row(const GradRow& row, float label, const float* z, __nv_bfloat16* g, int V,
                                               int tid, int threads) {
  for (int c = tid * 8; c < V; c += threads * 8) {
    // columns past V (up to 7) lie inside the row's padding: never read by the GEMMs
    uint32_t o[4] = {0u, 0u, 0u, 0u};
    if (row.keep != 0) {
      const float4 x = __ldcs(reinterpret_cast<const float4*>(z + c));
      const float4 w = __ldcs(reinterpret_cast<const float4*>(z + c + 4));
      o[0] = grad_pair(x.x, x.y, row);
      o[1] = grad_pair(x.z, x.w, row);
      o[2] = grad_pair(w.x, w.y, row);
      o[3] = grad_pair(w.z, w.w, row);
    }
    *reinterpret_cast<uint4*>(g + c) = make_uint4(o[0], o[1], o[2], o[3]);
    const int yo = row.y - c;
    if (row.y >= 0 && row.keep != 0 && yo >= 0 && yo < 8) g[row.y] = __float2bfloat16_rn(label);
  }
}

// ----------------------------------------------------------------------------
// A block of kRowThreads threads per row
// ----------------------------------------------------------------------------
constexpr int kRowThreads = 32 * kGroups;

__device__ __forceinline__ float block_sum(float v, float* red) {
  for (int off = 16; off > 0; off >>= 1) v += __shfl_xor_sync(0xffffffffu, v, off);
  __syncthreads();
  if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = v;
  __syncthreads();
  float s = 0.f;
  for (int i = 0; i < kRowThreads / 32; ++i) s += red[i];
  return s;
}
__device__ __forceinline__ float block_max(float v, float* red) {
  for (int off = 16; off > 0; off >>= 1) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, off));
  __syncthreads();
  if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = v;
  __syncthreads();
  float s = red[0];
  for (int i = 1; i < kRowThreads / 32; ++i) s = fmaxf(s, red[i]);
  return s;
}

}  // namespace
}  // namespace lce
