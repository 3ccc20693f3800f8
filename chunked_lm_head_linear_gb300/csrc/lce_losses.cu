// Losses on the log-probabilities of given tokens, with their gradients: the
// clipped policy loss with a KL term and the loss of paired sequences' log
// ratios. Both are, per row, a factor a_i = dloss/dlogp_i; the gradient of the
// logits is then
//   G_v = a_i ([v = y_i] - p_v) / T,   dH = G W,   dW = G^T H
// and everything but a_i is the token operators': the logits GEMM with its
// partial sums, the gradient tile over the row's scale (lce_rows.cuh) and the
// backward GEMMs. A policy row knows its factor as soon as its log-probability
// is known; a pair's factor needs all rows of its two sequences.
//
// Two ways to the gradient tile. Small calls keep the fp32 logits and write the
// tile in a pass over them. Large ones never store logits: the label's logit z_y
// is a product of two rows, known before the GEMM, so that its epilogue can write
// E_v = exp((z_v - z_y)/T) in bf16 at once. With R the sum of E over v != y
//   logp = -log1p(R),  p_v = E_v / (1 + R),  G_v = -(a / T) / (1 + R) (E_v, at y: -R)
// so E with -R in the label's place is the tile, the factor the row's scale, and
// neither p_y near 1 (R keeps its relative precision) nor a far label loses
// anything as long as the sums are finite. That z_y is a sum of its own, which
// errs otherwise than the tensor core's sums of the row: by 2e-5 at d = 2048, 1e-4
// at 7168, and all of E with it. The GEMM meets the label's column too; with its
// value z_y' and f = exp((z_y - z_y')/T) the row's sum is f R, and the
// log-probabilities are those of the other operators. Where a sum is not finite (a
// label more than 60 nats below its row's maximum, at T = 1, or a logit that is not
// finite), a guard turns on two launches that otherwise return at once: exact
// statistics, and the exact gradient tile. A factor so small that a / (T (1 + R))
// leaves fp32 is lost.
//
// The kernels here are short beside the GEMMs (1024 rows of d = 2048 and V =
// 151936: label logits 7.3 us, rows 9.0, of 1130): one block a row, bound by the
// latency of its few dependent reads; over kept logits by HBM (6 bytes a logit).
#include "lce_rows.cuh"

namespace lce {
namespace {

// ----------------------------------------------------------------------------
// The parts of a row kernel
// ----------------------------------------------------------------------------
struct RowStats {
  float M, logs;  // max z, log sum exp((z - M)/T)
};

// A row's partial sums merged in a fixed order by the block.
__device__ __forceinline__ RowStats merge_row(const LossRowArgs& p, int r, float* red, RowSum* sums) {
  const float4* pr = p.partials + static_cast<long long>(r) * p.nparts;
  const int tid = threadIdx.x, tiles = (p.V + 127) / 128;
  float M = -INFINITY;
  for (int t = tid; t < tiles; t += kRowThreads) M = fmaxf(M, pr[t].x);
  M = block_max(M, red);
  RowSum acc{0.f, 0.f, 0.f};
  for (int t = tid; t < tiles; t += kRowThreads) add_partial(acc, pr[t], M, p.inv_t);
  acc = warp_add(acc);
  if ((tid & 31) == 0) sums[tid >> 5] = acc;
  __syncthreads();
  return RowStats{M, log_sum(add_groups(sums))};
}

// Sum of a row of the exp tile without its label, in a fixed order.
__device__ __forceinline__ float exp_rest(const LossRowArgs& p, int r, float* red) {
  const float* pr = p.sums + static_cast<long long>(r) * p.nparts;
  float s = 0.f;
  for (int t = threadIdx.x; t < p.nparts; t += kRowThreads) s += pr[t];
  return block_sum(s, red);
}

// What the entries of row r, which has a label, and their sum are multiplied by to be against the GEMM's own z_y.
__device__ __forceinline__ float exp_shift(const LossRowArgs& p, int r) { return expf((p.ref[r] - p.ztgt[r]) * p.inv_t); }

// The row's scale, the label's entry of the exp tile and the row of dW's second operand. The entry is
// rounded to bf16; the scale makes up for that, as the label's is as a rule the row's largest share.
__device__ __forceinline__ void exp_gradient(const LossRowArgs& p, int r, int y, float a, float rest, float shift) {
  const int tid = threadIdx.x;
  const __nv_bfloat16 label = __float2bfloat16_rn(rest);
  const float held = __bfloat162float(label);
  float scale = -a * p.inv_t * shift / fmaf(rest, shift, 1.f);
  if (held >= 1.0e-30f) scale *= rest / held;
  if (tid == 0) {
    p.rowscale[r] = scale;
    if (y >= 0 && in_bounds(y, p.ldg, &p.st->flags)) p.G[static_cast<long long>(r) * p.ldg + y] = __hneg(label);
  }
  if (p.Ht != nullptr) {
    const int groups = p.d / 8;
    const long long at = static_cast<long long>(r) * groups;
    scale_row(p.H + at, p.Ht + at, groups, scale, a != 0.f, tid, kRowThreads);
  }
}

// The label of row r, -1 where none is given.
__device__ __forceinline__ int given_label(const int64_t* y, long long r, long long ignore_index, int V) {
  const long long v = y[r];
  return v != ignore_index && v >= 0 && v < V ? static_cast<int>(v) : -1;
}

// The row's scale, its row of dW's second operand and of the gradient tile (TILE), for the factor a.
template <bool TILE>
__device__ __forceinline__ void row_gradient(const LossRowArgs& p, int r, int y, float a, float logp, const RowStats& s) {
  const int tid = threadIdx.x;
  const Upstream u{a * p.inv_t, 0.f, y};
  const float entry = label_entry(u, logp, nullptr, r), scale = row_scale(u, entry);
  const float label = scale == 1.f ? entry : 1.f;
  if (tid == 0) {
    p.rowscale[r] = scale;
    p.label[r] = label;
    if (p.a != nullptr) p.a[r] = a;
  }
  if (p.Ht != nullptr) {
    const int groups = p.d / 8;
    const long long at = static_cast<long long>(r) * groups;
    scale_row(p.H + at, p.Ht + at, groups, scale, u.a != 0.f, tid, kRowThreads);
  }
  if (!TILE) return;
  GradRow g;
  g.m = s.M;
  g.k = p.inv_t * kLog2e;
  g.shift = -s.logs * kLog2e;
  g.c0 = -u.a * (1.f / scale);
  g.y = y;
  g.keep = u.a == 0.f ? 0u : ~0u;
  write_grad_row(g, label, p.Z + static_cast<long long>(r) * p.ldz, p.G + static_cast<long long>(r) * p.ldg, p.V, tid,
                 kRowThreads);
}

// Sum of n numbers in fp64, in an order that depends on n alone.
template <typename X>
__device__ __forceinline__ double block_total(const X* x, long long n, double* red) {
  const int tid = threadIdx.x;
  double sum = 0.0;
  for (long long i = tid; i < n; i += kRowThreads) sum += static_cast<double>(__ldcg(x + i));
  red[tid] = sum;
  __syncthreads();
  for (int w = kRowThreads / 2; w > 0; w >>= 1) {
    if (tid < w) red[tid] += red[tid + w];
    __syncthreads();
  }
  return red[0];
}

// True in the block that finishes last of `total`, which then sees what the others wrote.
__device__ __forceinline__ bool last_block(DevStatus* st, int total) {
  __shared__ int s_last;
  if (threadIdx.x == 0) {
    __threadfence();
    s_last = atomicAdd(&st->rows_done, 1) == total - 1;
  }
  __syncthreads();
  if (s_last) __threadfence();
  return s_last != 0;
}

// ----------------------------------------------------------------------------
// Policy loss
// ----------------------------------------------------------------------------
// With l = logp, r = exp(l - old) (1 without old) and s = min(r A, clip(r) A),
// for A < 0 not below dual A:
//   row = w (kl_coef KL - s),   a = w (kl_coef dKL/dl - [the unclipped side] r A)
//   KL of u = l - ref: k1 = u, k2 = u^2 / 2, k3 = exp(-u) - 1 + u
// A weight of zero leaves nothing, whatever the row holds; an advantage of zero
// has no share even of an infinite ratio. r and u are fp32, as logp is; the
// row's loss is formed from them in fp64, as the rows' losses cancel in their sum.
struct PolicyRow {
  float w, A, ratio, side, u, e;  // side: what A is multiplied by; e = exp(-u) - 1
  float a;
};

__device__ __forceinline__ PolicyRow policy_row(const PolicyArgs& p, int r, float logp) {
  PolicyRow x{p.weights != nullptr ? p.weights[r] : 1.f, 0.f, 1.f, 0.f, 0.f, 0.f, 0.f};
  if (x.w == 0.f) return x;
  x.A = p.advantages[r];
  if (x.A != 0.f) {
    if (p.old_logp != nullptr) x.ratio = expf(logp - p.old_logp[r]);
    const float clipped = fminf(fmaxf(x.ratio, 1.f - p.clip_low), 1.f + p.clip_high);
    x.side = clipped * x.A < x.ratio * x.A ? clipped : x.ratio;
    x.a = clipped * x.A < x.ratio * x.A ? 0.f : -x.ratio * x.A;
    if (x.A < 0.f && p.dual_clip > 0.f && x.side > p.dual_clip) {
      x.side = p.dual_clip;
      x.a = 0.f;
    }
  }
  if (p.ref_logp != nullptr) {
    x.u = logp - p.ref_logp[r];
    x.e = expm1f(-x.u);  // exp(-u) - 1 without what the difference loses near 0
    x.a = fmaf(p.kl_coef, p.kl == 1 ? 1.f : p.kl == 2 ? x.u : -x.e, x.a);
  }
  x.a *= x.w;
  return x;
}

__device__ __forceinline__ double policy_loss(const PolicyArgs& p, const PolicyRow& x) {
  if (x.w == 0.f) return 0.0;
  const double u = x.u, kl = p.kl == 1 ? u : p.kl == 2 ? 0.5 * u * u : static_cast<double>(x.e) + u;
  double row = x.A != 0.f ? -static_cast<double>(x.side) * static_cast<double>(x.A) : 0.0;
  if (p.ref_logp != nullptr) row += static_cast<double>(p.kl_coef) * kl;
  return row * static_cast<double>(x.w);
}

// One block per row of the chunk. EXP: from the exp tile, or, where its guard is set, from the partial sums.
template <bool GRAD, bool TILE, bool EXP>
__global__ void __launch_bounds__(kRowThreads, 8) k_policy_row(const PolicyArgs p) {
  grid_dep_wait();
  grid_dep_launch();
  __shared__ float red[kRowThreads / 32];
  __shared__ RowSum s_sum[kGroups];
  __shared__ double s_total[kRowThreads];
  const int r = blockIdx.x, tid = threadIdx.x;
  const LossRowArgs& q = p.row;
  const int y = given_label(q.y, r, q.ignore_index, q.V);
  float logp = 0.f, a = 0.f, rest = 0.f, shift = 1.f;
  double row = 0.0;  // thread 0's
  RowStats s{0.f, 0.f};
  const bool by_exp = EXP && *q.guard == 0;
  if (y >= 0) {
    if (by_exp) {
      rest = exp_rest(q, r, red);
      shift = exp_shift(q, r);
      logp = -log1pf(rest * shift);
    } else {
      s = merge_row(q, r, red, s_sum);
      const float z = q.Z != nullptr ? q.Z[static_cast<long long>(r) * q.ldz + y] : q.ztgt[r];
      logp = (z - s.M) * q.inv_t - s.logs;
    }
    const PolicyRow x = policy_row(p, r, logp);
    a = x.a;
    if (tid == 0) row = policy_loss(p, x);
  }
  if (tid == 0) {
    q.logp[r] = logp;
    p.row_loss[r] = static_cast<float>(row);
    p.row64[r] = row;
    if (GRAD && q.stats != nullptr) q.stats[r] = make_float2(s.M, s.logs);
    if (p.loss != nullptr) {
      if (y >= 0) atomicAdd(reinterpret_cast<unsigned long long*>(&q.st->n_counted), 1ull);
      if (y < 0 && q.y[r] != q.ignore_index) atomicOr(&q.st->flags, kFlagLabelRange);
    }
  }
  if (GRAD) {
    if (by_exp)
      exp_gradient(q, r, y, a, rest, shift);
    else
      row_gradient<TILE>(q, r, y, a, logp, s);
  }
  if (p.loss == nullptr) return;
  if (!last_block(q.st, static_cast<int>(p.N))) return;
  const double sum = block_total(p.all_rows, p.N, s_total);
  if (tid == 0) {
    const long long counted = __ldcg(&q.st->n_counted), n = p.n_override >= 0 ? p.n_override : counted;
    const double weight = p.mean ? (n > 0 ? 1.0 / static_cast<double>(n) : 0.0) : 1.0;
    q.st->n_valid = n;
    q.st->gscale = static_cast<float>((p.grad_loss != nullptr ? static_cast<double>(*p.grad_loss) : 1.0) * weight);
    *p.loss = static_cast<float>(sum * weight);
  }
}

// The rows' losses of a call of several chunks, summed.
__global__ void __launch_bounds__(kRowThreads) k_policy_total(const double* __restrict__ rows, long long N,
                                                              const DevStatus* st, float* __restrict__ loss) {
  grid_dep_wait();
  grid_dep_launch();
  __shared__ double red[kRowThreads];
  const double sum = block_total(rows, N, red);
  if (threadIdx.x == 0) *loss = static_cast<float>(sum * st->lscale);
}

// ----------------------------------------------------------------------------
// Preference loss
// ----------------------------------------------------------------------------
__device__ __forceinline__ long long bound_at(const void* cu, int cu32, long long i) {
  return cu32 ? static_cast<long long>(static_cast<const int32_t*>(cu)[i]) : static_cast<const int64_t*>(cu)[i];
}

__device__ __forceinline__ double softplus(double x) { return fmax(x, 0.0) + log1p(exp(-fabs(x))); }
__device__ __forceinline__ double sigmoid(double x) {
  const double e = exp(-fabs(x));
  return (x >= 0 ? 1.0 : e) / (1.0 + e);
}

// One block per pair p: sequences 2 p (chosen) and 2 p + 1 (rejected). With S
// their log-probabilities (sums in fp64, or means, over the given tokens),
// delta = (S_c - S_r) - (ref_c - ref_r) and x = beta delta - margin
//   sigmoid  -(1 - e) log sig(x) - e log sig(-x),   hinge  max(0, 1 - x)
//   ipo      (delta - 1 / (2 beta))^2
// Bounds that fall or leave [0, N] set the status bit; the pair then has no part in loss and gradient.
__device__ __forceinline__ void pair_scales(const PairArgs& p) {
  p.st->gscale = static_cast<float>((p.grad_loss != nullptr ? static_cast<double>(*p.grad_loss) : 1.0) * p.weight);
}

// Rows [c[h], c[h + 1]) of pair's two sequences; false, and no rows, where the bounds fall or leave [0, N].
__device__ __forceinline__ bool pair_bounds(const PairArgs& p, long long pair, long long (&c)[3]) {
  for (int i = 0; i < 3; ++i) c[i] = bound_at(p.cu, p.cu32, 2 * pair + i);
  if (c[0] >= 0 && c[0] <= c[1] && c[1] <= c[2] && c[2] <= p.N) return true;
  c[0] = c[1] = c[2] = 0;
  return false;
}

// This thread's share of a sequence's sum and count: rows from + first, + first + step, ...
__device__ __forceinline__ void sequence_share(const PairArgs& p, long long from, long long to, int first, int step,
                                               double& sum, int& cnt) {
  sum = 0.0;
  cnt = 0;
#pragma unroll 4
  for (long long r = from + first; r < to; r += step)
    if (given_label(p.y, r, p.ignore_index, p.V) >= 0) {
      sum += static_cast<double>(__ldcg(p.logp + r));
      ++cnt;
    }
}

// A pair's results from its sequences' sums and counts (one thread).
__device__ __forceinline__ void pair_result(const PairArgs& p, long long pair, bool ok, const double* sum, const int* cnt) {
  if (!ok) atomicOr(&p.st->flags, kFlagLabelRange);
  double per[2], S[2];
  for (int h = 0; h < 2; ++h) {
    per[h] = p.average ? (cnt[h] > 0 ? 1.0 / cnt[h] : 0.0) : 1.0;
    S[h] = sum[h] * per[h];
    p.seq_logp[2 * pair + h] = static_cast<float>(S[h]);
  }
  double delta = S[0] - S[1];
  if (p.ref != nullptr) delta -= static_cast<double>(p.ref[2 * pair]) - static_cast<double>(p.ref[2 * pair + 1]);
  const double beta = p.beta, x = beta * delta - p.margin, e = p.smoothing;
  double loss, slope;
  if (p.kind == 0) {
    loss = (1.0 - e) * softplus(-x) + (e > 0.0 ? e * softplus(x) : 0.0);
    slope = beta * (e * sigmoid(x) - (1.0 - e) * sigmoid(-x));
  } else if (p.kind == 1) {
    loss = x < 1.0 ? 1.0 - x : x != x ? x : 0.0;
    slope = x < 1.0 ? -beta : x != x ? x : 0.0;
  } else {
    const double far = delta - 0.5 / beta;
    loss = far * far;
    slope = 2.0 * far;
  }
  if (!ok) loss = slope = 0.0;
  p.pair_loss[pair] = static_cast<float>(loss);
  p.coef[2 * pair] = static_cast<float>(slope * per[0]);
  p.coef[2 * pair + 1] = static_cast<float>(-slope * per[1]);
}

__global__ void __launch_bounds__(kRowThreads) k_pairs(const PairArgs p) {
  grid_dep_wait();
  grid_dep_launch();
  __shared__ double s_red[kRowThreads];
  __shared__ double s_sum[2];
  __shared__ int s_cnt[2];
  const int tid = threadIdx.x;
  if (blockIdx.x == 0 && tid == 0) pair_scales(p);
  if (p.P == 0) {
    if (tid == 0) *p.loss = 0.f;
    return;
  }
  if (tid < 2) s_cnt[tid] = 0;
  long long c[3];
  const bool ok = pair_bounds(p, blockIdx.x, c);
  for (int h = 0; h < 2; ++h) {
    double sum;
    int cnt;
    sequence_share(p, c[h], c[h + 1], tid, kRowThreads, sum, cnt);
    __syncthreads();
    s_red[tid] = sum;
    cnt = __reduce_add_sync(0xffffffffu, cnt);
    if ((tid & 31) == 0) atomicAdd(&s_cnt[h], cnt);
    __syncthreads();
    for (int w = kRowThreads / 2; w > 0; w >>= 1) {
      if (tid < w) s_red[tid] += s_red[tid + w];
      __syncthreads();
    }
    if (tid == 0) s_sum[h] = s_red[0];
  }
  if (tid == 0) pair_result(p, blockIdx.x, ok, s_sum, s_cnt);
  if (!last_block(p.st, static_cast<int>(p.P))) return;
  const double sum = block_total(p.pair_loss, p.P, s_red);
  if (tid == 0) *p.loss = static_cast<float>(sum * p.weight);
}

// The rows' log-probabilities with what the gradient needs of them again, one block a row: from the exp tile's sums
// (EXP, unless its guard is set) or the partial sums. PAIRS: the block that finishes last goes through the few pairs (at
// most kPairsHere), a warp a sequence.
template <bool EXP, bool PAIRS>
__global__ void __launch_bounds__(kRowThreads) k_logp_rows(const LossRowArgs p, const PairArgs q) {
  grid_dep_wait();
  grid_dep_launch();
  __shared__ float red[kRowThreads / 32];
  __shared__ RowSum s_rows[kGroups];
  __shared__ double s_red[kRowThreads], s_sum[2 * kPairsHere];
  __shared__ int s_cnt[2 * kPairsHere];
  const int r = blockIdx.x, tid = threadIdx.x;
  const int y = given_label(p.y, r, p.ignore_index, p.V);
  float logp = 0.f, rest = 0.f;
  RowStats s{0.f, 0.f};
  if (y >= 0) {
    if (EXP && *p.guard == 0) {
      rest = exp_rest(p, r, red);
      logp = -log1pf(rest * exp_shift(p, r));
    } else {
      s = merge_row(p, r, red, s_rows);
      const float z = p.Z != nullptr ? p.Z[static_cast<long long>(r) * p.ldz + y] : p.ztgt[r];
      logp = (z - s.M) * p.inv_t - s.logs;
    }
  }
  if (tid == 0) {
    p.logp[r] = logp;
    p.stats[r] = make_float2(s.M, s.logs);
    if (EXP) p.rest[r] = rest;
    if (y < 0 && p.y[r] != p.ignore_index) atomicOr(&p.st->flags, kFlagLabelRange);
  }
  if (!PAIRS) return;
  if (!last_block(p.st, static_cast<int>(q.N))) return;
  if (tid == 0) pair_scales(q);
  const int warp = tid >> 5;
  if (warp < 2 * q.P) {
    long long c[3];
    pair_bounds(q, warp / 2, c);
    double sum;
    int cnt;
    sequence_share(q, c[warp & 1], c[(warp & 1) + 1], tid & 31, 32, sum, cnt);
    for (int off = 16; off > 0; off >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, off);
    cnt = __reduce_add_sync(0xffffffffu, cnt);
    if ((tid & 31) == 0) {
      s_sum[warp] = sum;
      s_cnt[warp] = cnt;
    }
  }
  __syncthreads();
  if (tid < q.P) {
    long long c[3];
    const bool ok = pair_bounds(q, tid, c);
    pair_result(q, tid, ok, s_sum + 2 * tid, s_cnt + 2 * tid);
    __threadfence();
  }
  __syncthreads();
  const double sum = block_total(q.pair_loss, q.P, s_red);
  if (tid == 0) *q.loss = static_cast<float>(sum * q.weight);
}

// The sequence that holds row r: the last whose first row is not behind r. -1 before the first, >= S behind the last.
__device__ __forceinline__ long long sequence_of(const void* cu, int cu32, long long S, long long r) {
  long long lo = 0, hi = S + 1;  // bounds [0, lo) are <= r, [hi, S] are > r
  while (lo < hi) {
    const long long mid = (lo + hi) >> 1;
    if (bound_at(cu, cu32, mid) <= r)
      lo = mid + 1;
    else
      hi = mid;
  }
  return lo - 1;
}

// One block per row of the chunk, once the pairs' factors are known.
template <bool TILE, bool EXP>
__global__ void __launch_bounds__(kRowThreads, 8) k_preference_row(const PreferenceArgs p) {
  grid_dep_wait();
  grid_dep_launch();
  const int r = blockIdx.x;
  const LossRowArgs& q = p.row;
  const int y = given_label(q.y, r, q.ignore_index, q.V);
  float a = 0.f;
  if (y >= 0 && p.P > 0) {  // (without pairs there may be no bounds)
    const long long s = sequence_of(p.cu, p.cu32, 2 * p.P, p.c0 + r);
    if (s >= 0 && s < 2 * p.P) a = p.coef[s];
  }
  if (EXP && *q.guard == 0) {
    exp_gradient(q, r, y, a, q.rest[r], y >= 0 ? exp_shift(q, r) : 1.f);
    return;
  }
  const float2 st = q.stats[r];
  row_gradient<TILE>(q, r, y, a, q.logp[r], RowStats{st.x, st.y});
}

// One warp per row: H_i . W_{y_i} in fp32. The call's first launch: its first block clears the status block, the
// guards and the dH part counters (clear.st null: an earlier launch did).
__global__ void __launch_bounds__(256) k_label_logits(const uint4* __restrict__ H, const uint4* __restrict__ W,
                                                      const int64_t* __restrict__ y, long long N, int groups, int V,
                                                      long long ignore_index, float* __restrict__ z, const LossClear clear) {
  grid_dep_wait();
  grid_dep_launch();
  if (clear.st != nullptr && blockIdx.x == 0) {
    for (int i = threadIdx.x; i < clear.nguards; i += blockDim.x) clear.guards[i] = 0;
    for (int i = threadIdx.x; i < clear.ncnt; i += blockDim.x) clear.cnt[i] = 0;
    if (threadIdx.x == 0) *clear.st = DevStatus{};
  }
  const long long r = (blockIdx.x * static_cast<long long>(blockDim.x) + threadIdx.x) >> 5;
  const int lane = threadIdx.x & 31;
  if (r >= N) return;
  const int v = given_label(y, r, ignore_index, V);
  float s = 0.f;
  if (v >= 0) {
    const uint4 *h = H + r * groups, *w = W + static_cast<long long>(v) * groups;
#pragma unroll 4
    for (int i = lane; i < groups; i += 32) {
      const uint4 a = h[i], b = w[i];
      const uint32_t x[4] = {a.x, a.y, a.z, a.w}, u[4] = {b.x, b.y, b.z, b.w};
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        s = fmaf(__uint_as_float(x[q] << 16), __uint_as_float(u[q] << 16), s);
        s = fmaf(__uint_as_float(x[q] & 0xffff0000u), __uint_as_float(u[q] & 0xffff0000u), s);
      }
    }
  }
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) s += __shfl_xor_sync(0xffffffffu, s, off);
  if (lane == 0) z[r] = s;
}

}  // namespace

cudaError_t launch_label_logits(const void* H, const void* W, const int64_t* y, long long N, int d, int V,
                                long long ignore_index, float* z, const LossClear& clear, cudaStream_t s) {
  if (N <= 0) return cudaSuccess;
  return launch_k(k_label_logits, static_cast<unsigned>((N + 7) / 8), 256, 0, s, static_cast<const uint4*>(H),
                  static_cast<const uint4*>(W), y, N, d / 8, V, ignore_index, z, clear);
}

cudaError_t launch_policy_row(const PolicyArgs& p, int rows, cudaStream_t s) {
  if (rows <= 0) return cudaSuccess;
  if (p.row.rowscale == nullptr) return launch_k(k_policy_row<false, false, false>, rows, kRowThreads, 0, s, p);
  return p.row.sums != nullptr ? launch_k(k_policy_row<true, false, true>, rows, kRowThreads, 0, s, p)
                               : launch_k(k_policy_row<true, true, false>, rows, kRowThreads, 0, s, p);
}

cudaError_t launch_policy_total(const double* rows, long long N, const DevStatus* st, float* loss, cudaStream_t s) {
  return launch_k(k_policy_total, 1, kRowThreads, 0, s, rows, N, st, loss);
}

cudaError_t launch_pairs(const PairArgs& p, cudaStream_t s) {
  return launch_k(k_pairs, static_cast<unsigned>(p.P > 0 ? p.P : 1), kRowThreads, 0, s, p);
}

cudaError_t launch_logp_rows(const LossRowArgs& p, const PairArgs& q, bool with_pairs, int rows, cudaStream_t s) {
  if (rows <= 0) return cudaSuccess;
  if (p.sums != nullptr)
    return with_pairs ? launch_k(k_logp_rows<true, true>, rows, kRowThreads, 0, s, p, q)
                      : launch_k(k_logp_rows<true, false>, rows, kRowThreads, 0, s, p, q);
  return with_pairs ? launch_k(k_logp_rows<false, true>, rows, kRowThreads, 0, s, p, q)
                    : launch_k(k_logp_rows<false, false>, rows, kRowThreads, 0, s, p, q);
}

cudaError_t launch_preference_row(const PreferenceArgs& p, int rows, cudaStream_t s) {
  if (rows <= 0) return cudaSuccess;
  if (p.row.sums != nullptr) return launch_k(k_preference_row<false, true>, rows, kRowThreads, 0, s, p);
  return p.row.Z != nullptr ? launch_k(k_preference_row<true, false>, rows, kRowThreads, 0, s, p)
                            : launch_k(k_preference_row<false, false>, rows, kRowThreads, 0, s, p);
}

}  // namespace lce
