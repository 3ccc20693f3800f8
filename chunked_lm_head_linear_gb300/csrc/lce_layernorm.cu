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
constexpr int kSumWarps = 32;
constexpr int kSms = 152;        // the one-pass backward runs one or two persistent blocks a SM
constexpr int kLnFusedD = 8192;  // longest row whose backward is one pass
constexpr int kLnCluster = 16;    // blocks of a backward that is one cluster

// Eight neighbouring elements of a row, as they are held in registers.
template <bool F32>
struct Group;
template <>
struct Group<false> {
  uint4 v;
  __device__ __forceinline__ void load(const void* p, long long i) { v = static_cast<const uint4*>(p)[i]; }
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
  __device__ __forceinline__ void load(const void* p, long long i) {
    a = static_cast<const float4*>(p)[2 * i];
    b = static_cast<const float4*>(p)[2 * i + 1];
  }
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

// ----------------------------------------------------------------------------
// Rows through shared memory. A block holds teams of T threads; a team takes R
// rows at a time and its thread t owns their column groups t, t + T, ... (at most
// K). Every warp copies its own threads' groups ahead of their use into its own
// part of a ring of D turns (cp.async, 16 bytes a lane, neighbouring lanes
// neighbouring pieces) and reads only those back: the copies need no barrier
// beyond the warp, and what is on its way from HBM does not take registers.
// ----------------------------------------------------------------------------
__device__ __forceinline__ void copy16(uint4* dst, const void* src, long long i, bool on) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;"
               :
               : "r"(smem_u32(dst)), "l"(static_cast<const uint4*>(src) + i), "r"(on ? 16 : 0)
               : "memory");
}
__device__ __forceinline__ void copies_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void copies_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

template <bool F32, int T, int K, int R, int PER>
struct Ring {
  static constexpr int kBlock = T < 256 ? 256 : T;
  static constexpr int kSlots = R * K * PER;  // 16-byte slots of a thread and turn
  static constexpr int bytes(int D) { return D * kSlots * kBlock * 16; }
};

// The eight elements of this thread's group in a slot of 32 (bf16) or 64 (fp32) pieces of its warp.
template <bool F32>
__device__ __forceinline__ void slot_get(const uint4* warp_slot, int lane, float (&f)[8]) {
  if constexpr (F32) {
    const float4 a = reinterpret_cast<const float4*>(warp_slot)[2 * lane], b = reinterpret_cast<const float4*>(warp_slot)[2 * lane + 1];
    f[0] = a.x; f[1] = a.y; f[2] = a.z; f[3] = a.w;
    f[4] = b.x; f[5] = b.y; f[6] = b.z; f[7] = b.w;
  } else {
    Group<false> g;
    g.v = warp_slot[lane];
    g.get(f);
  }
}

// The copies of that slot: group g0 + lane of a row whose groups begin at `row`, groups at or behind `groups` (or all,
// for a row that does not exist) as zeros.
template <bool F32>
__device__ __forceinline__ void slot_copy(uint4* warp_slot, int lane, const void* src, long long row, int g0, int groups,
                                          bool on) {
  constexpr int PER = F32 ? 2 : 1;
#pragma unroll
  for (int e = 0; e < PER; ++e) {
    const int piece = e * 32 + lane;
    const bool in = on && g0 + piece / PER < groups;
    copy16(warp_slot + piece, src, in ? (row + g0) * PER + piece : 0, in);
  }
}

// Sums of R values over a team of W warps, in order; buf is not used again before a barrier.
template <int W, int R>
__device__ __forceinline__ void team_total(float (&v)[R], float (*buf)[R], int warp, int lane) {
#pragma unroll
  for (int q = 0; q < R; ++q) v[q] = warp_total(v[q]);
  if (W > 1) {
    if (lane == 0) {
#pragma unroll
      for (int q = 0; q < R; ++q) buf[warp][q] = v[q];
    }
    __syncthreads();
#pragma unroll
    for (int q = 0; q < R; ++q) {
      v[q] = buf[0][q];
#pragma unroll
      for (int i = 1; i < W; ++i) v[q] += buf[i][q];
    }
  }
}

template <bool F32, int T, int K, int R, int D, int B>
__global__ void __launch_bounds__(T < 256 ? 256 : T, B) k_layernorm_fwd(const LayerNormArgs p) {
  grid_dep_wait();
  grid_dep_launch();
  constexpr int PER = F32 ? 2 : 1;
  using Rg = Ring<F32, T, K, R, PER>;
  constexpr int BL = Rg::kBlock, S = BL / T, W = T / 32;
  constexpr bool kHold = T <= 256;  // weights and biases in registers
  extern __shared__ uint4 ring[];
  __shared__ float red[2][S][W][R];
  const int tid = threadIdx.x, team = tid / T, t = tid % T, lane = tid & 31, warp = t >> 5;
  const int groups = p.d / 8;
  const float d = static_cast<float>(p.d), inv_d = 1.f / d;
  float w[K][8], b[K][8];
#pragma unroll
  for (int j = 0; j < K; ++j) {
    if (kHold && t + T * j < groups) {
      param8(p.w, p.w_bf16, t + T * j, 1.f, w[j]);
      param8(p.b, p.w_bf16, t + T * j, 0.f, b[j]);
    }
  }
  const long long first = (static_cast<long long>(blockIdx.x) * S + team) * R, step = static_cast<long long>(gridDim.x) * S * R;
  // this warp's 32 PER pieces of slot (q, j)
  auto slot = [&](int turn, int q, int j) {
    return ring + ((turn * R + q) * K + j) * PER * BL + (tid >> 5) * 32 * PER;
  };
  auto fetch = [&](long long i, int turn) {
#pragma unroll
    for (int q = 0; q < R; ++q) {
#pragma unroll
      for (int j = 0; j < K; ++j)
        slot_copy<F32>(slot(turn, q, j), lane, p.x, (i + q) * groups, warp * 32 + T * j, groups, i + q < p.N);
    }
    copies_commit();
  };
#pragma unroll
  for (int n = 0; n < D - 1; ++n) fetch(first + n * step, n);
  int turn = 0;
  // the loop's length is the block's, so that its teams meet at the barriers
  for (long long i0 = static_cast<long long>(blockIdx.x) * S * R, i = first; i0 < p.N; i0 += step, i += step) {
    fetch(i + (D - 1) * step, turn == 0 ? D - 1 : turn - 1);
    copies_wait<D - 1>();
    __syncwarp();
    float x[R][K][8], mean[R], rstd[R];
#pragma unroll
    for (int q = 0; q < R; ++q) {
      mean[q] = 0.f;
#pragma unroll
      for (int j = 0; j < K; ++j) {
        slot_get<F32>(slot(turn, q, j), lane, x[q][j]);
#pragma unroll
        for (int k = 0; k < 8; ++k) mean[q] += x[q][j][k];
      }
    }
    __syncwarp();  // read by all of the warp before the next turn's copies
    team_total<W, R>(mean, red[0][team], warp, lane);
#pragma unroll
    for (int q = 0; q < R; ++q) {
      const float s = mean[q] * inv_d;
      mean[q] = fmaf(fmaf(-s, d, mean[q]), inv_d, s);  // sum / d without the rounding of 1 / d: exact for flat rows
      rstd[q] = 0.f;
#pragma unroll
      for (int j = 0; j < K; ++j) {
        if (t + T * j < groups) {
#pragma unroll
          for (int k = 0; k < 8; ++k) {
            x[q][j][k] -= mean[q];
            rstd[q] = fmaf(x[q][j][k], x[q][j][k], rstd[q]);
          }
        }
      }
    }
    team_total<W, R>(rstd, red[1][team], warp, lane);
#pragma unroll
    for (int q = 0; q < R; ++q) {
      rstd[q] = rsqrtf(fmaf(rstd[q], inv_d, p.eps));
      if (t == 0 && i + q < p.N) {
        if (p.mean != nullptr) p.mean[i + q] = mean[q];
        if (p.rstd != nullptr) p.rstd[i + q] = rstd[q];
      }
#pragma unroll
      for (int j = 0; j < K; ++j) {
        const int gI = t + T * j;
        if (i + q < p.N && gI < groups) {
          if (!kHold) {
            param8(p.w, p.w_bf16, gI, 1.f, w[j]);
            param8(p.b, p.w_bf16, gI, 0.f, b[j]);
          }
          float f[8];
#pragma unroll
          for (int k = 0; k < 8; ++k) f[k] = fmaf(x[q][j][k] * rstd[q], w[j][k], b[j][k]);
          store8(p.H, (i + q) * groups + gI, f, false);
        }
      }
    }
    turn = turn == D - 1 ? 0 : turn + 1;
  }
  copies_wait<0>();
}

// dx, dw and db in one pass over x and dH (d up to 2048 K): the two sums of a row
// are one exchange in its team, x and dH stay in registers between them and dx,
// and dw and db grow in registers over all of the block's rows. At the end the
// teams' shares are added in order and the block writes one partial row of each.
// ONE: the launch is one cluster, whose blocks add their shares through each
// other's shared memory, in order; there is nothing left for another launch.
// Bound by HBM: x and dH read once, dx written once, 65536 rows of bf16 in 19 us
// (d = 256), 37, 68, 134, 246 (4096) with the sum of the partial rows, 32768 of
// fp32 in 107 (2048), 201 (4096); at the copy rate 15, 30, 59, 119, 237 and 99, 198.
// (dx and dw in two kernels, each reading both, took 596 us at 65536 x 4096.)
template <bool F32, int T, int K, int R, int D, int B, bool ONE>
__global__ void __launch_bounds__(kLnThreads, B) k_layernorm_bwd(const LayerNormArgs p) {
  grid_dep_wait();
  grid_dep_launch();
  constexpr int PX = F32 ? 2 : 1, PER = PX + 1;
  constexpr int S = kLnThreads / T, W = T / 32;
  extern __shared__ uint4 ring[];
  __shared__ float red[2][S][W][2 * R];
  __shared__ float share[S][T][17];
  const int tid = threadIdx.x, team = tid / T, t = tid % T, lane = tid & 31, warp = t >> 5;
  const int groups = p.d / 8;
  const float inv_d = 1.f / static_cast<float>(p.d);
  float aw[K][8], ab[K][8], w[K][8];
#pragma unroll
  for (int j = 0; j < K; ++j) {
#pragma unroll
    for (int k = 0; k < 8; ++k) aw[j][k] = ab[j][k] = w[j][k] = 0.f;
    if (t + T * j < groups) param8(p.w, p.w_bf16, t + T * j, 1.f, w[j]);
  }
  const long long first = (static_cast<long long>(blockIdx.x) * S + team) * R, step = static_cast<long long>(gridDim.x) * S * R;
  // this warp's pieces of slot (q, j): 32 PX of x, then 32 of dH
  auto slot = [&](int turn, int q, int j) {
    return ring + ((turn * R + q) * K + j) * PER * kLnThreads + (tid >> 5) * 32 * PER;
  };
  auto fetch = [&](long long i, int turn) {
#pragma unroll
    for (int q = 0; q < R; ++q) {
#pragma unroll
      for (int j = 0; j < K; ++j) {
        uint4* s = slot(turn, q, j);
        slot_copy<F32>(s, lane, p.x, (i + q) * groups, warp * 32 + T * j, groups, i + q < p.N);
        slot_copy<false>(s + 32 * PX, lane, p.dH, (i + q) * groups, warp * 32 + T * j, groups, i + q < p.N);
      }
    }
    copies_commit();
  };
  float mu_next[R], r_next[R];
  auto statistics = [&](long long i) {
#pragma unroll
    for (int q = 0; q < R; ++q) {
      mu_next[q] = i + q < p.N ? p.mean[i + q] : 0.f;
      r_next[q] = i + q < p.N ? p.rstd[i + q] : 0.f;
    }
  };
#pragma unroll
  for (int n = 0; n < D - 1; ++n) fetch(first + n * step, n);
  statistics(first);
  int turn = 0, half = 0;
  for (long long i0 = static_cast<long long>(blockIdx.x) * S * R, i = first; i0 < p.N; i0 += step, i += step, half ^= 1) {
    fetch(i + (D - 1) * step, turn == 0 ? D - 1 : turn - 1);
    copies_wait<D - 1>();
    __syncwarp();
    float xh[R][K][8], g[R][K][8], r[R], sums[2 * R];  // (x - mean) rstd, dH w
#pragma unroll
    for (int q = 0; q < R; ++q) {
      const float mu = mu_next[q];
      r[q] = r_next[q];
      sums[2 * q] = sums[2 * q + 1] = 0.f;
#pragma unroll
      for (int j = 0; j < K; ++j) {
        slot_get<F32>(slot(turn, q, j), lane, xh[q][j]);
        slot_get<false>(slot(turn, q, j) + 32 * PX, lane, g[q][j]);
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          const float h = g[q][j][k];
          xh[q][j][k] = (xh[q][j][k] - mu) * r[q];
          g[q][j][k] = h * w[j][k];
          sums[2 * q] += g[q][j][k];
          sums[2 * q + 1] = fmaf(g[q][j][k], xh[q][j][k], sums[2 * q + 1]);
          aw[j][k] = fmaf(h, xh[q][j][k], aw[j][k]);
          ab[j][k] += h;
        }
      }
    }
    statistics(i + step);
    __syncwarp();  // read by all of the warp before the next turn's copies
    turn = turn == D - 1 ? 0 : turn + 1;
    if (p.dx == nullptr) continue;
    team_total<W, 2 * R>(sums, red[half][team], warp, lane);  // two buffers: one barrier a turn is enough
#pragma unroll
    for (int q = 0; q < R; ++q) {
      const float c0 = sums[2 * q] * inv_d * r[q], c1 = sums[2 * q + 1] * inv_d * r[q];
#pragma unroll
      for (int j = 0; j < K; ++j) {
        const int gI = t + T * j;
        if (i + q < p.N && gI < groups) {
          float f[8];
#pragma unroll
          for (int k = 0; k < 8; ++k) f[k] = fmaf(-xh[q][j][k], c1, fmaf(g[q][j][k], r[q], -c0));
          store8(p.dx, (i + q) * groups + gI, f, F32);
        }
      }
    }
  }
  copies_wait<0>();
  if (p.dw == nullptr && p.db == nullptr) return;
  if (ONE) __syncthreads();  // the ring is free
  float* mine = reinterpret_cast<float*>(ring);  // ONE: this block's dw and db
#pragma unroll
  for (int j = 0; j < K; ++j) {
    if (S > 1) {
      if (j > 0) __syncthreads();
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        share[team][t][k] = aw[j][k];
        share[team][t][8 + k] = ab[j][k];
      }
      __syncthreads();
      if (team == 0) {
#pragma unroll
        for (int k = 0; k < 8; ++k)
          for (int s = 1; s < S; ++s) {
            aw[j][k] += share[s][t][k];
            ab[j][k] += share[s][t][8 + k];
          }
      }
    }
    const int gI = t + T * j;
    if (team == 0 && gI < groups) {
      const long long at = ONE ? gI : static_cast<long long>(blockIdx.x) * groups + gI;
      store8(ONE ? mine : p.part, at, aw[j], true);
      store8(ONE ? mine : p.part, (ONE ? groups : static_cast<long long>(gridDim.x) * groups) + at, ab[j], true);
    }
  }
  if (ONE) {
    cluster_sync_all();
    const int per = (2 * p.d + kLnCluster - 1) / kLnCluster, c0 = static_cast<int>(cluster_ctarank()) * per;
    const uint32_t base = smem_u32(mine);
    for (int c = c0 + tid; c < c0 + per && c < 2 * p.d; c += kLnThreads) {
      float v[kLnCluster];
#pragma unroll
      for (int r = 0; r < kLnCluster; ++r) v[r] = ld_shared_cluster(mapa_shared(base + 4 * c, r));
#pragma unroll
      for (int r = 1; r < kLnCluster; ++r) v[0] += v[r];
      float* out = c < p.d ? p.dw : p.db;
      if (out != nullptr) out[c < p.d ? c : c - p.d] = v[0];
    }
    cluster_sync_all();  // no block leaves while its memory is read
  }
}

// dx alone, one warp per row, in two passes over it (rows of more than kLnFusedD).
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

// Partial sums of dw and db alone (d above kLnFusedD): block (c, s) owns 256 columns and every gridDim.y-th
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
// columns of one of them, warp s sums the parts s, s + 32, ... in order.
__global__ void __launch_bounds__(32 * kSumWarps) k_layernorm_sum(const LayerNormArgs p, int parts) {
  grid_dep_wait();
  grid_dep_launch();
  __shared__ float red[kSumWarps][33];
  float* out = blockIdx.y == 0 ? p.dw : p.db;
  if (out == nullptr) return;
  const int lane = threadIdx.x & 31, s = threadIdx.x >> 5, k = blockIdx.x * 32 + lane;
  const float* part = p.part + static_cast<long long>(blockIdx.y) * parts * p.d;
  float t = 0.f;
  if (k < p.d)
#pragma unroll 4
    for (int b = s; b < parts; b += kSumWarps) t += part[static_cast<long long>(b) * p.d + k];
  red[s][lane] = t;
  __syncthreads();
  if (s == 0 && k < p.d) {
    for (int q = 1; q < kSumWarps; ++q) t += red[q][lane];
    out[k] = t;
  }
}

template <typename Kern>
cudaError_t launch_ring(Kern kern, int blocks, int threads, int bytes, const LayerNormArgs& p, cudaStream_t s) {
  const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
  if (e != cudaSuccess) return e;
  return launch_k(kern, static_cast<unsigned>(blocks), threads, bytes, s, p);
}

template <bool F32, int T, int K, int R, int D, int B>
cudaError_t fwd(const LayerNormArgs& p, int num_sms, cudaStream_t s) {
  using Rg = Ring<F32, T, K, R, F32 ? 2 : 1>;
  constexpr int rows = Rg::kBlock / T * R;
  const long long need = (p.N + rows - 1) / rows, most = static_cast<long long>(B) * num_sms;
  return launch_ring(k_layernorm_fwd<F32, T, K, R, D, B>, static_cast<int>(need < most ? need : most), Rg::kBlock,
                     Rg::bytes(D), p, s);
}

// Teams of a warp (no barrier) up to rows of 1024, then as few threads as keep a row in registers; rows a turn, turns and
// blocks a SM as measured (65536 rows bf16, 32768 fp32, us; the copy rate would take 10, 20, 40, 79, 158 and 59, 119):
// 256: 11. 512: warps 22, teams of 64 25. 1024: 43, 45. 2048: teams of 128 in two blocks a SM 84, of 256 in three 92; fp32
// 61, 67. 4096: two blocks a SM 164, three 191, four 197; fp32 four 121, three 138.
template <bool F32>
cudaError_t fwd_rows(const LayerNormArgs& p, int num_sms, cudaStream_t s) {
  if (p.d <= 256) return fwd<F32, 32, 1, 2, 4, 3>(p, num_sms, s);
  if (p.d <= 512) return fwd<F32, 32, 2, 1, 4, 2>(p, num_sms, s);
  if (p.d <= 1024) return fwd<F32, 32, 4, 1, F32 ? 3 : 4, 1>(p, num_sms, s);
  if (p.d <= 2048) return fwd<F32, F32 ? 256 : 128, F32 ? 1 : 2, F32 ? 4 : 1, F32 ? 2 : 4, 2>(p, num_sms, s);
  if (p.d <= 4096) return fwd<F32, 256, 2, 1, F32 ? 3 : 4, F32 ? 4 : 2>(p, num_sms, s);
  if (p.d <= 8192) return fwd<F32, 256, 4, 1, 3, 2>(p, num_sms, s);
  if (p.d <= 16384) return fwd<F32, 512, 4, 1, 3, 1>(p, num_sms, s);
  return fwd<F32, 1024, 4, 1, F32 ? 1 : 2, 1>(p, num_sms, s);
}

// Elements of x up to which the backward is one cluster of sixteen blocks: one launch, which is what small calls wait for
// (1531 x 264: 20 us a call, 25 with a second launch that adds the blocks' partial rows; on the device alone 9.0 and 5.5).
// A row of fewer than 256 elements takes a team's turn as one of 256 does, and counts as one (60001 x 8 on the device: 114 us
// as one cluster, 16 with many blocks; 4000 x 128 10.0 and 5.5).
constexpr long long kLnOneLaunch = 1 << 19;

bool one_launch(long long N, long long d) { return d <= kLnFusedD && N * (d > 256 ? d : 256) <= kLnOneLaunch; }

// The pass as a launch of one cluster, where dw or db is wanted and such a cluster fits the SMs there are (not on a small
// partition of them): *done. cudaSuccess without *done: it does not.
template <bool F32, int T, int K, int R, int D, int B>
cudaError_t bwd_cluster(const LayerNormArgs& p, int bytes, bool* done, cudaStream_t s) {
  auto kern = k_layernorm_bwd<F32, T, K, R, D, B, true>;
  const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
  if (e != cudaSuccess) return e;
  const cudaError_t wide = cudaFuncSetAttribute(kern, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);  // above 8 blocks
  if (wide != cudaSuccess) return wide;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = kLnCluster;
  attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(kLnCluster);
  cfg.blockDim = dim3(kLnThreads);
  cfg.dynamicSmemBytes = bytes;
  cfg.stream = s;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  int fit = 0;
  if (cudaOccupancyMaxActiveClusters(&fit, kern, &cfg) != cudaSuccess || fit < 1) {
    (void)cudaGetLastError();
    return cudaSuccess;
  }
  *done = true;
  return cudaLaunchKernelEx(&cfg, kern, p);
}

// *done: dw and db are written, else the blocks' partial rows are.
template <bool F32, int T, int K, int R, int D, int B = 2>
cudaError_t bwd_pass(const LayerNormArgs& p, int parts, bool* done, cudaStream_t s) {
  constexpr int bytes = Ring<F32, T, K, R, F32 ? 3 : 2>::bytes(D);
  static_assert(bytes >= 2 * 4 * 8 * T * K, "a block's dw and db fit the ring");
  if ((p.dw != nullptr || p.db != nullptr) && !p.no_cluster && one_launch(p.N, p.d)) {
    const cudaError_t e = bwd_cluster<F32, T, K, R, D, B>(p, bytes, done, s);
    if (e != cudaSuccess || *done) return e;
  }
  return launch_ring(k_layernorm_bwd<F32, T, K, R, D, B, false>, parts, kLnThreads, bytes, p, s);
}

// Rows that a block of the one-pass backward takes at a time.
int bwd_rows(long long d) {
  return d <= 256 ? 8 * 2 : d <= 512 ? 8 : d <= 1024 ? 4 : d <= 2048 ? 2 : 1;
}

template <bool F32>
cudaError_t bwd(const LayerNormArgs& p, int num_sms, cudaStream_t s) {
  const bool sums = p.dw != nullptr || p.db != nullptr;
  const int parts = layernorm_parts(p.N, p.d);
  cudaError_t e = cudaSuccess;
  bool done = !sums;
  if (p.d <= 256)
    e = bwd_pass<F32, 32, 1, 2, F32 ? 3 : 4>(p, parts, &done, s);
  else if (p.d <= 512)
    e = bwd_pass<F32, 32, 2, 1, F32 ? 3 : 4>(p, parts, &done, s);
  else if (p.d <= 1024)
    e = bwd_pass<F32, 64, 2, 1, F32 ? 3 : 4>(p, parts, &done, s);
  else if (p.d <= 2048)
    e = bwd_pass<F32, 256, 1, 2, 4>(p, parts, &done, s);
  else if (p.d <= 4096)
    e = bwd_pass<F32, 256, 2, 1, 4>(p, parts, &done, s);
  else if (p.d <= kLnFusedD)
    e = bwd_pass<F32, 256, 4, 1, 4, 1>(p, parts, &done, s);
  else {
    if (p.dx != nullptr && p.N > 0) {
      const long long need = (p.N + kLnWarps - 1) / kLnWarps, most = 8LL * num_sms;
      e = launch_k(k_layernorm_dx<F32>, static_cast<unsigned>(need < most ? need : most), kLnThreads, 0, s, p);
    }
    if (e == cudaSuccess && sums) e = launch_k(k_layernorm_dw<F32>, dim3((p.d + 255) / 256, parts), kLnThreads, 0, s, p);
  }
  if (e != cudaSuccess || done) return e;
  return launch_k(k_layernorm_sum, dim3((p.d + 31) / 32, 2), 32 * kSumWarps, 0, s, p, parts);
}

}  // namespace

// Blocks of the backward, each with a partial row of dw and db.
int layernorm_parts(long long N, long long d) {
  const long long rows = d <= kLnFusedD ? bwd_rows(d) : kLnWarps;
  const long long need = (N + rows - 1) / rows, most = d <= 4096 ? 2 * kSms : d <= kLnFusedD ? kSms : 512 / ((d + 255) / 256) + 1;
  const long long parts = need < most ? need : most;
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
