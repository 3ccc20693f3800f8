// Token operators of the LM head beside its cross-entropy: log-probabilities
// of given tokens with entropy and top alternatives, their gradient, and the
// distillation loss against a teacher's top logits. They share the pair GEMM
// of lce_gemm.cuh (z = H W^T, never a whole [N, V] in memory) and the backward
// GEMMs of lce_kernels.cu; what differs is the tile epilogue and the per-row
// kernels behind it.
//
// Per row i, with z' = z / T:
//   lse = log sum_v exp z'_v, logp = z'_y - lse, entropy = lse - sum_v p_v z'_v
// The GEMM's epilogue keeps, per (row, 128 vocabulary columns), four numbers
//   m = max z, with c = 1 (merged: how many half tiles reach the row's maximum),
//   s = sum exp((z - m)/T) over the others,  t = sum exp((z - m)/T) (z - m)/T
// from which, merged over the row, log-sum-exp = m/T + log c + log1p(s/c) and
// entropy = log c + log1p(s/c) - t/(c + s): one exponential per logit for both,
// no difference of two large numbers, and because the terms of the maxima, 1
// exactly, are counted apart, a log-probability near 0 (a confident model's token) keeps
// its relative precision instead of the 2^-24 of a sum near 1.
#include <math.h>

#include "lce_gemm.cuh"
#include "lce_internal.h"
#include "lce_rows.cuh"

namespace lce {
namespace {

// A tile's running maximum and the sums over the logits other than it (m = kMasked: nothing yet).
struct Mst {
  float m, s, t;
};

// 32 logits added to them; v is overwritten. A pass of maxima and minima leaves the maximum of all,
// the old one included, apart from the 32 that lose against it, so that no comparison is needed to
// leave it out of the sums; they run in strands, two logits an instruction, because a warp has its
// issue slots to itself and waits for its own chains.
__device__ __forceinline__ void add_columns(Mst& a, float (&v)[32], float inv_t) {
  const float k = inv_t * kLog2e;
  float x[4] = {v[0], v[1], v[2], v[3]};
#pragma unroll
  for (int c = 4; c < 32; c += 4) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float hi = max_nan(x[i], v[c + i]);
      v[c + i] = min_nan(x[i], v[c + i]);
      x[i] = hi;
    }
  }
  float m = a.m;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float hi = max_nan(m, x[i]);
    v[i] = min_nan(m, x[i]);
    m = hi;
  }
  if (m != a.m) {
    const float d = a.m - m, f = ex2_approx(d * k);
    a.t = f * fmaf(a.s, fmaxf(d * inv_t, kFloor), a.t);
    a.s *= f;
    a.m = m;
  }
  // The maximum is subtracted before the product with k, as in the merges behind: exponents
  // err by their own rounding only, whatever the size of z / T. (One fma, z k - fl(m k), with what m k
  // loses made good behind the sums, saves 1% at d = 256 and overflows at |m| / T above 3e9.)
  const uint64_t m2 = pair_f32(-m, -m), k2 = pair_f32(k, k);
  uint64_t s[2] = {0, 0}, t[2] = {0, 0};
#pragma unroll
  for (int c = 0; c < 32; c += 4) {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const uint64_t y = mul_pair(add_pair(pair_f32(v[c + 2 * i], v[c + 2 * i + 1]), m2), k2);
      float y0, y1;
      unpair_f32(y, y0, y1);
      const uint64_t e = pair_f32(ex2_approx(y0), ex2_approx(y1));
      s[i] = add_pair(s[i], e);
      t[i] = fma_pair(e, y, t[i]);
    }
  }
  float s0, s1, t0, t1;
  unpair_f32(add_pair(s[0], s[1]), s0, s1);
  unpair_f32(add_pair(t[0], t[1]), t0, t1);
  a.s += s0 + s1;
  a.t = fmaf(t0 + t1, kLn2, a.t);
}

// ----------------------------------------------------------------------------
// Tile epilogue: an epilogue warp owns 32 rows x 128 columns, one thread a row.
//   TOK_STATS    the four numbers of each (row, half tile) and the label's logit
//   TOK_STATS_Z  the four numbers, and the fp32 logits themselves into the chunk's
//                buffer (top alternatives and distillation read them again:
//                4 bytes a logit, written behind a main loop of d/16 MMAs)
//   TOK_GRAD     the gradient tile of (logp, entropy) in bf16, from the saved
//                statistics and entropy, over the row's scale (see GradRow):
//                  G_v = ([v = y] a - p_v (a + e (z'_v - lse + entropy))) / T
//                rounded to bf16 once (the operand type of the two GEMMs that
//                follow), everything before it in fp32.
//   TOK_EXP      E_v = exp((z_v - z_y)/T) in bf16 against the label's logit, known
//                before the GEMM, and the sums of E without the label's column: with
//                R their sum logp = -log1p(R) and p_v = E_v / (1 + R), so that the
//                tile is the gradient's up to a factor per row and nothing needs the
//                logits again. The label's logit as this GEMM has it goes out too, for
//                the row kernels to refer R to. A sum that is too large, or NaN, or the
//                two logits of a label far apart, set the guard.
// ----------------------------------------------------------------------------
__device__ __forceinline__ void clear_status(DevStatus* st, int* cnt, int ncnt, int thread, int threads) {
  for (int i = thread; i < ncnt; i += threads) cnt[i] = 0;
  if (thread == 0) {
    st->flags = 0;
    st->rows_done = 0;
    st->n_valid = 0;
    st->n_counted = 0;
    st->gscale = 0.f;
    st->lscale = 0.0;
  }
}

// The first launch of a call clears the status word (or block) from its first block's epilogue warps,
// before anything can have been reported: a wait that gives up does so after two seconds, a bad label
// is reported by a later kernel. (The checked build, whose blocks may report an index at once, clears
// it by a launch.)
__device__ __forceinline__ void reset_status(const TokParams& p) {
  if (blockIdx.x != 0) return;
  const int thread = static_cast<int>(threadIdx.x) - 32 * EPI_WARP0;
  if (p.clear_st != nullptr)
    clear_status(p.clear_st, p.cnt, p.ncnt, thread, 32 * EPI_WARPS);
  else if (p.reset && thread == 0)
    *p.flags = 0;
}

template <int MODE>
struct TokEpi {
  using Params = TokParams;
  struct State {
    long long y;  // TOK_EXP: the row's label and its logit
    float z;
  };

  // 32 columns c0.. of the half tile: their logits stored, the row's four numbers brought up to date.
  // The maximum and the sums run in four strands each: a warp has its sub-partition's issue slots to
  // itself, and what bounds it is the latency of its chains.
  static __device__ __forceinline__ void stats_group(const Params& p, const EpiCtx& ctx, float (&v)[32], int c0,
                                                     int col0, int row, int vlim, bool rows_in, int ycol, Mst& a,
                                                     float& zt, bool& have_t) {
    if (MODE == TOK_STATS_Z && rows_in) {
      stage_acquire(ctx);
#pragma unroll
      for (int q = 0; q < 8; ++q)
        *reinterpret_cast<float4*>(ctx.stage + stage_off(ctx.lane, q)) =
            make_float4(v[4 * q], v[4 * q + 1], v[4 * q + 2], v[4 * q + 3]);
      stage_release(ctx, col0 + c0, row, false);
    }
    if (vlim < c0 + 32) {
#pragma unroll
      for (int c = 0; c < 32; ++c)
        if (c0 + c >= vlim) v[c] = kMasked;
    }
    if (MODE == TOK_STATS) {
      const int yo = ycol - c0;
      if (yo >= 0 && yo < 32) {
#pragma unroll
        for (int c = 0; c < 32; ++c)
          if (c == yo) {
            zt = v[c];
            have_t = true;
          }
      }
    }
    add_columns(a, v, p.inv_t);
  }

  static __device__ __forceinline__ void stats_tile(const Params& p, const EpiCtx& ctx, int m0, int col0,
                                                    uint32_t taddr) {
    const int r = m0 + ctx.row0 + ctx.lane;
    const bool live = r < p.rows;
    const int vlim = p.V - col0;  // columns >= vlim are past the vocabulary (warp-uniform)
    const int part = col0 / EPI_COLS;
    Mst acc{kMasked, 0.f, 0.f};
    float zt = 0.f;
    bool have_t = false;
    int ycol = -1;
    if (MODE == TOK_STATS && live) {
      const long long yc = static_cast<long long>(p.y[r]) - col0;
      if (yc >= 0 && yc < EPI_COLS && p.y[r] != p.ignore_index) ycol = static_cast<int>(yc);
    }
    const bool rows_in = m0 + ctx.row0 < p.rows;  // a store box never starts past the rows
    const int row = m0 + ctx.row0;
    if (vlim > 0) {
      // two groups of 32 columns in flight (a group past the vocabulary holds zeros and is not used)
      float va[32], vb[32];
      tmem_ld_issue_x32(taddr, va);
#pragma unroll 1
      for (int c0 = 0; c0 < EPI_COLS; c0 += 64) {
        tmem_ld_wait(va);
        tmem_ld_issue_x32(taddr + c0 + 32, vb);
        stats_group(p, ctx, va, c0, col0, row, vlim, rows_in, ycol, acc, zt, have_t);
        tmem_ld_wait(vb);
        if (c0 + 64 < EPI_COLS) tmem_ld_issue_x32(taddr + c0 + 64, va);
        if (c0 + 32 < vlim) stats_group(p, ctx, vb, c0 + 32, col0, row, vlim, rows_in, ycol, acc, zt, have_t);
        if (c0 + 64 >= vlim) break;
      }
      tmem_ld_wait(va);  // a load that a break left under way
    }
    if (!live || !in_bounds(part, p.nparts, p.flags)) return;
    p.partials[static_cast<long long>(r) * p.nparts + part] =
        vlim > 0 ? make_float4(acc.m, acc.s, acc.t, 1.f) : make_float4(-INFINITY, 0.f, 0.f, 0.f);
    if (MODE == TOK_STATS && have_t) p.ztgt[r] = zt;
  }

  // 32 columns c0.. of the exp tile in bf16; their sum is added to s. zt: the label's logit, if it is among them.
  static __device__ __forceinline__ void exp_group(float (&v)[32], int c0, int vlim, int ycol, float z, float k,
                                                   uint32_t keep, uint64_t (&s)[2], uint32_t (&pk)[16], float& zt) {
    if (vlim < c0 + 32) {
#pragma unroll
      for (int c = 0; c < 32; ++c)
        if (c0 + c >= vlim) v[c] = kMasked;
    }
    const int yo = ycol - c0;
    if (yo >= 0 && yo < 32) {  // the label's own column has no part in the sum; its entry is written later
#pragma unroll
      for (int c = 0; c < 32; ++c)
        if (c == yo) {
          zt = v[c];
          v[c] = kMasked;
        }
    }
    const uint64_t z2 = pair_f32(-z, -z), k2 = pair_f32(k, k);
#pragma unroll
    for (int c = 0; c < 32; c += 2) {
      float x0, x1;
      unpair_f32(mul_pair(add_pair(pair_f32(v[c], v[c + 1]), z2), k2), x0, x1);
      const float e0 = ex2_approx(x0), e1 = ex2_approx(x1);
      s[(c / 2) & 1] = add_pair(s[(c / 2) & 1], pair_f32(e0, e1));
      pk[c / 2] = pack_bf16x2(e0, e1) & keep;
    }
  }

  static __device__ __forceinline__ void exp_tile(const Params& p, const State& st, const EpiCtx& ctx, int m0, int col0,
                                                  uint32_t taddr) {
    const int r = m0 + ctx.row0 + ctx.lane;
    const int vlim = p.V - col0, part = col0 / EPI_COLS;
    if (m0 + ctx.row0 >= p.rows) return;  // no row of this warp
    const bool live = r < p.rows;
    const long long y = st.y;
    const bool given = live && y != p.ignore_index && y >= 0 && y < p.V;
    const long long yc = y - col0;
    const int ycol = given && yc >= 0 && yc < EPI_COLS ? static_cast<int>(yc) : -1;
    const float z = given ? st.z : 0.f, k = p.inv_t * kLog2e;
    float sum = 0.f, zt = z;
    if (vlim > 0) {
      const uint32_t keep = given ? ~0u : 0u;  // rows without a token are zero whatever they hold
      uint64_t s[2] = {0, 0};
      float va[32], vb[32];
      tmem_ld_issue_x32(taddr, va);
#pragma unroll 1
      for (int c0 = 0; c0 < EPI_COLS; c0 += 64) {  // two groups of 32 columns in flight, a staged tile of 64
        if (c0 >= vlim) break;
        uint32_t pa[16], pb[16];
        tmem_ld_wait(va);
        tmem_ld_issue_x32(taddr + c0 + 32, vb);
        exp_group(va, c0, vlim, ycol, z, k, keep, s, pa, zt);
        tmem_ld_wait(vb);
        if (c0 + 64 < EPI_COLS) tmem_ld_issue_x32(taddr + c0 + 64, va);
        exp_group(vb, c0 + 32, vlim, ycol, z, k, keep, s, pb, zt);
        stage_acquire(ctx);  // the store before this one is read while the exponentials are computed
        stage_bf16(ctx, pa, pb);
        stage_release(ctx, col0 + c0, m0 + ctx.row0, false);
      }
      tmem_ld_wait(va);  // a load that a break left under way
      float s0, s1;
      unpair_f32(add_pair(s[0], s[1]), s0, s1);
      sum = s0 + s1 + (z - z);  // NaN, and so the guard, where the label's logit is not finite
    }
    if (!live || !in_bounds(part, p.nparts, p.flags)) return;
    p.sums[static_cast<long long>(r) * p.nparts + part] = sum;
    if (ycol >= 0) p.ztgt[r] = zt;
    if (given && !(sum <= kExpGuard && fabsf(z - zt) * p.inv_t <= kExpShift)) *p.guard = 1;
  }

  static __device__ __forceinline__ void grad_tile(const Params& p, const EpiCtx& ctx, int m0, int col0,
                                                   uint32_t taddr) {
    const int r = m0 + ctx.row0 + ctx.lane;
    const int vlim = p.V - col0;
    if (m0 + ctx.row0 >= p.rows || vlim <= 0) return;  // nothing of this half tile is stored
    GradRow g;
    float label = 0.f;
    if (r < p.rows) {
      g = grad_row(upstream(r, p.y, p.ignore_index, p.V, p.g_logp, p.g_entropy, p.inv_t), p.rowscale[r], p.stats,
                   p.lse, p.entropy, r, p.inv_t);
      label = p.label[r];
    }
    const int ycol = g.y - col0;  // a column of this half tile, or outside [0, 128)
#pragma unroll 1
    for (int u = 0; u < EPI_COLS / 64; ++u) {
      if (u * 64 >= vlim) break;
      stage_acquire(ctx);
#pragma unroll 1
      for (int hh = 0; hh < 2; ++hh) {
        const int c0 = u * 64 + hh * 32;
        float v[32];
        tmem_ld_32x32b_x32(taddr + c0, v);
        uint32_t pk[16];
#pragma unroll
        for (int c = 0; c < 32; c += 2) pk[c / 2] = grad_pair(v[c], v[c + 1], g);
#pragma unroll
        for (int q = 0; q < 4; ++q)
          *reinterpret_cast<uint4*>(ctx.stage + stage_off(ctx.lane, hh * 4 + q)) =
              make_uint4(pk[4 * q], pk[4 * q + 1], pk[4 * q + 2], pk[4 * q + 3]);
      }
      const int yo = ycol - u * 64;  // the label's entry, by the thread that holds its row
      if (g.y >= 0 && g.keep != 0 && yo >= 0 && yo < 64)
        *reinterpret_cast<__nv_bfloat16*>(ctx.stage + stage_off(ctx.lane, yo / 8) + (yo % 8) * 2) =
            __float2bfloat16_rn(label);
      stage_release(ctx, col0 + u * 64, m0 + ctx.row0, false);
    }
  }
};

// The logits of a chunk with one of these epilogues; tiles walk M first, so
// the pairs running at once share W tiles.
template <int MODE>
struct TokProb {
  struct Params {
    CUtensorMap a, b, c;
    int m_tiles, n_tiles, k_blocks;
    TokParams ep;
  };
  using State = typename TokEpi<MODE>::State;
  static __device__ __forceinline__ bool skip(const Params& p) { return p.ep.only_if != nullptr && *p.ep.only_if == 0; }
  static __device__ __forceinline__ bool no_loads(const Params& p) { return p.ep.no_loads != 0; }
  static __device__ __forceinline__ int* flags(const Params& p) { return p.ep.flags; }
  using Plan = RoundRobin;
  static __device__ __forceinline__ Plan plan(const Params& p, int c, int P) {
    return round_robin(p.m_tiles * p.n_tiles, c, P);
  }
  static __device__ __forceinline__ int num_jobs(const Plan& s) { return s.jobs; }
  static __device__ __forceinline__ TileJob job(const Params& p, const Plan& s, int j) {
    const int t = s.c + j * s.P;
    return TileJob{0, t % p.m_tiles, t / p.m_tiles, p.k_blocks, 0, 0};
  }
  static __device__ __forceinline__ bool job_ok(const Params& p, const TileJob& tj) {
    return tj.mb >= 0 && tj.mb < p.m_tiles && tj.nb >= 0 && tj.nb < p.n_tiles && tj.k_blocks > 0;
  }
  static __device__ __forceinline__ void load(const Params& p, int, uint8_t* a, uint8_t* b, uint32_t bar, int m0,
                                              int n0, int k0) {
    load_k_major(a, &p.a, bar, m0, k0);
    load_k_major(b, &p.b, bar, n0, k0);
  }
  static __device__ __forceinline__ uint64_t a_desc(int, uint32_t addr, int k) { return desc_k_major(addr, k); }
  static __device__ __forceinline__ uint64_t b_desc(int, uint32_t addr, int k) { return desc_k_major(addr, k); }
  static __device__ __forceinline__ uint32_t idesc(int) { return idesc_bf16_f32(P_TILE_M, BN, false, false); }
  static __device__ __forceinline__ void init(const Params& p, State&) { reset_status(p.ep); }
  static __device__ __forceinline__ void ahead(const Params& p, State& st, const TileJob&, int r) {
    if (MODE != TOK_EXP) return;
    st.y = r < p.ep.rows ? static_cast<long long>(p.ep.y[r]) : p.ep.ignore_index;
    st.z = r < p.ep.rows ? p.ep.ref[r] : 0.f;
  }
  static __device__ __forceinline__ void epilogue(const Params& p, State& st, const TileJob&, EpiCtx ctx, int m0,
                                                  int col0, uint32_t taddr) {
    ctx.out = &p.c;
    if constexpr (MODE == TOK_GRAD)
      TokEpi<MODE>::grad_tile(p.ep, ctx, m0, col0, taddr);
    else if constexpr (MODE == TOK_EXP)
      TokEpi<MODE>::exp_tile(p.ep, st, ctx, m0, col0, taddr);
    else
      TokEpi<MODE>::stats_tile(p.ep, ctx, m0, col0, taddr);
  }
};

template <int MODE, int EW = EPI_WARPS>
cudaError_t launch_tok_mode(const CUtensorMap& a, const CUtensorMap& b, const CUtensorMap& c, long long M, long long N,
                            long long K, const TokParams& ep, int num_sms, cudaStream_t s) {
  using Prob = TokProb<MODE>;
  typename Prob::Params p;
  p.a = a;
  p.b = b;
  p.c = c;
  p.m_tiles = static_cast<int>((M + P_TILE_M - 1) / P_TILE_M);
  p.n_tiles = static_cast<int>((N + BN - 1) / BN);
  p.k_blocks = static_cast<int>((K + BK - 1) / BK);
  p.ep = ep;
  const long long tiles = static_cast<long long>(p.m_tiles) * p.n_tiles;
  const int clusters = static_cast<int>(tiles < num_sms / 2 ? tiles : num_sms / 2);
  if (clusters <= 0) return cudaSuccess;
  auto kern = gemm_pair_kernel<Prob, EW>;
  constexpr int bytes = PairSmemLayoutT<EW>::kDynamicBytes;
  const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
  if (e != cudaSuccess) return e;
  return launch_k(kern, 2 * clusters, 32 * (EPI_WARP0 + EW), bytes, s, p);
}

// ----------------------------------------------------------------------------
// Few rows (decoding): the logits are one pass over W, bound by reading it, so
// the operands change sides. A tile is 128 MT vocabulary rows of W (the MMA's
// M, each read once, by one CTA) by all rows of H (its N = NT, zero-filled by
// TMA beyond the last), accumulated over d in TMEM; the ring of W blocks keeps
// 112 to 160 KB a SM on their way from HBM. The pair kernel's 256-row tiles
// would multiply 256 rows whatever their number and leave fewer bytes in
// flight: 7 rows of d = 7168 and V = 151655 took 517 us with it, 327 us here,
// 6.6 TB/s; from 97 rows on it is level or ahead (128 rows of d = 2048: 131 us
// against 133 when they were compared, 111 now).
// MT = 2 (NT = 32) halves the reads of H from L2 per byte of W: one row of d =
// 4096 and V = 151936 187 us against 204. With more rows the last tile's longer
// epilogue costs more than that gives (64 rows of d = 2048: 114 us against 112).
//   warp 0      TMA producer, warp 1 MMA issuer, warp 2 TMEM
//   warps 4-7   epilogue: TMEM lanes (vocabulary) into shared memory as
//               [32 rows][128]; a thread sums 32 columns of one row (no
//               shuffles), a warp stores a row's 512 bytes of logits
// The numbers and logits are laid out as the pair kernel's, and the kernels
// behind do not know which ran.
// ----------------------------------------------------------------------------
constexpr int kOutLd = 132;  // row stride of the logits in shared memory: 16-byte reads of 8 rows hit all banks once

template <int NT, int MT>
struct RowsCfg {
  static constexpr int kABytes = MT * 128 * BK * 2;
  static constexpr int kBBytes = NT * BK * 2;
  static constexpr int kStages = 211000 / (kABytes + kBBytes);
  static constexpr int kOut = kStages * (kABytes + kBBytes);
  static constexpr int kSums = kOut + 32 * kOutLd * 4;
  static constexpr int kBars = kSums + 128 * 16;
  static constexpr int kNumBars = 2 * kStages + 4 + 1;
  static constexpr int kMisc = kBars + kNumBars * 8;
  static constexpr int kTotal = kMisc + 16;
  static constexpr int kDynamicBytes = kTotal + 1024;
  static constexpr int kTmemCols = MT * NT <= 64 ? 128 : 256;  // two accumulators, a power of two
  static_assert(2 * MT * NT <= kTmemCols, "TMEM columns (few-rows kernel)");
  static_assert(kDynamicBytes <= 232448, "shared memory budget (few-rows kernel)");
};

struct RowsParams {
  CUtensorMap w, h;
  int tiles, k_blocks;
  int store_z;
  long long ldz;
  float* Z;
  TokParams ep;
};

__device__ __forceinline__ bool warp_wait(uint64_t* bar, uint32_t parity, volatile int* abort, int lane) {
  int ok = 0;
  if (lane == 0) ok = mbar_wait(bar, parity, abort) ? 1 : 0;
  return __shfl_sync(0xffffffffu, ok, 0) != 0;
}

// Barrier of the four epilogue warps: true if it is true in every thread.
__device__ __forceinline__ bool epilogue_all(bool ok) {
  int all;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t"
      "setp.ne.s32 p, %1, 0;\n\t"
      "bar.red.and.pred q, 1, 128, p;\n\t"
      "selp.s32 %0, 1, 0, q;\n\t}"
      : "=r"(all)
      : "r"(ok ? 1 : 0)
      : "memory");
  return all != 0;
}

template <int NT, int MT>
__global__ void __launch_bounds__(NUM_THREADS, 1) k_rows_logits(const __grid_constant__ RowsParams p) {
  using Cfg = RowsCfg<NT, MT>;
  constexpr int S = Cfg::kStages;
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw_addr = smem_u32(smem_raw);
  uint8_t* smem = smem_raw + (((raw_addr + 1023u) & ~1023u) - raw_addr);
  uint8_t* sA = smem;
  uint8_t* sB = smem + S * Cfg::kABytes;
  float* out = reinterpret_cast<float*>(smem + Cfg::kOut);
  float4* sums = reinterpret_cast<float4*>(smem + Cfg::kSums);
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + Cfg::kBars);
  uint64_t* empty = full + S;
  uint64_t* tfull = full + 2 * S;
  uint64_t* tempty = tfull + 2;
  uint64_t* drain = tempty + 2;
  uint32_t* tmem_holder = reinterpret_cast<uint32_t*>(smem + Cfg::kMisc);
  volatile int* abort = reinterpret_cast<volatile int*>(smem + Cfg::kMisc + 4);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

  if (threadIdx.x == 0) {
    for (int i = 0; i < S; ++i) {
      mbar_init(&full[i], 1);
      mbar_init(&empty[i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&tfull[i], 1);
      mbar_init(&tempty[i], EPI_WARPS);
    }
    mbar_init(drain, 1);
    *abort = 0;
    fence_mbarrier_init();
  }
  if (warp == 2) {
    tmem_alloc(tmem_holder, Cfg::kTmemCols);
    tmem_relinquish();
  }
  tc_fence_before_sync();
  __syncthreads();
  tc_fence_after_sync();
  const uint32_t tmem_base = *tmem_holder;
  grid_dep_wait();  // everything above is the CTA's own; below, memory of earlier kernels
  grid_dep_launch();

  if (warp == 0 && lane == 0) {
    int stage = 0;
    uint32_t phase = 0, armed = 0, armed_parity = 0;
    bool ok = p.ep.no_loads == 0;
    for (int t = blockIdx.x; t < p.tiles && ok; t += gridDim.x) {
      for (int kb = 0; kb < p.k_blocks; ++kb) {
        if (!mbar_wait(&empty[stage], phase ^ 1u, abort)) {
          report_timeout(abort, p.ep.flags);
          ok = false;
          break;
        }
        mbar_arrive_expect_tx(&full[stage], Cfg::kABytes + Cfg::kBBytes);
#pragma unroll
        for (int h = 0; h < MT; ++h)  // (a block past the vocabulary is all zeros)
          tma_load_2d(sA + stage * Cfg::kABytes + h * 128 * BK * 2, &p.w, &full[stage], kb * BK, (t * MT + h) * 128);
        tma_load_2d(sB + stage * Cfg::kBBytes, &p.h, &full[stage], kb * BK, 0);
        armed |= 1u << stage;
        armed_parity = (armed_parity & ~(1u << stage)) | (phase << stage);
        if (++stage == S) {
          stage = 0;
          phase ^= 1u;
        }
      }
    }
    if (!ok || *abort) {  // leaving early: the copies under way land before the block ends
      for (int i = 0; i < S; ++i)
        if (armed & (1u << i)) mbar_wait_drain(&full[i], (armed_parity >> i) & 1u, 100000000ull);
    }
  } else if (warp == 1 && lane == 0) {
    int stage = 0, acc = 0;
    uint32_t phase = 0, acc_phase = 0;
    bool ok = true, issued = false;
    constexpr uint32_t idesc = idesc_bf16_f32(128, NT, false, false);
    for (int t = blockIdx.x; t < p.tiles && ok; t += gridDim.x) {
      if (!mbar_wait(&tempty[acc], acc_phase ^ 1u, abort)) {
        report_timeout(abort, p.ep.flags);
        break;
      }
      tc_fence_after_sync();
      const uint32_t d_tmem = tmem_base + static_cast<uint32_t>(acc * MT * NT);
      for (int kb = 0; kb < p.k_blocks; ++kb) {
        if (!mbar_wait(&full[stage], phase, abort)) {
          report_timeout(abort, p.ep.flags);
          ok = false;
          break;
        }
        tc_fence_after_sync();
        const uint32_t a_addr = smem_u32(sA + stage * Cfg::kABytes);
        const uint32_t b_addr = smem_u32(sB + stage * Cfg::kBBytes);
#pragma unroll
        for (int k = 0; k < BK / 16; ++k) {
#pragma unroll
          for (int h = 0; h < MT; ++h)
            umma_bf16(d_tmem + h * NT, desc_k_major(a_addr + h * 128 * BK * 2, k), desc_k_major(b_addr, k), idesc,
                      (kb | k) != 0 ? 1u : 0u);
        }
        issued = true;
        umma_commit(&empty[stage]);
        if (++stage == S) {
          stage = 0;
          phase ^= 1u;
        }
      }
      if (!ok) break;
      umma_commit(&tfull[acc]);
      if (++acc == 2) {
        acc = 0;
        acc_phase ^= 1u;
      }
    }
    if (*abort && issued) {
      umma_commit(drain);
      mbar_wait_drain(drain, 0, 100000000ull);
    }
  } else if (warp >= EPI_WARP0) {
    const int q = warp & 3;
    const TokParams& e = p.ep;
    int acc = 0;
    uint32_t acc_phase = 0;
    reset_status(e);
    for (int t = blockIdx.x; t < p.tiles; t += gridDim.x) {
      // The four warps agree on whether the tile came (a wait that ran out in one ends the loop of
      // all, so that none is left at the barrier below); everyone has read the tile before by then.
      const bool came = warp_wait(&tfull[acc], acc_phase, abort, lane);
      if (!came && lane == 0) report_timeout(abort, e.flags);
      if (!epilogue_all(came)) break;
      tc_fence_after_sync();
      const uint32_t taddr = tmem_base + (static_cast<uint32_t>(q * 32) << 16) + static_cast<uint32_t>(acc * MT * NT);
#pragma unroll 1
      for (int g = 0, n0 = 0, h = 0; h < MT; ++g) {  // 32 rows of H by 128 of W at a time through shared memory
        const int part = t * MT + h, col0 = part * 128;
        if (g > 0) epilogue_all(true);  // what was there has been read
        {
          float v[32];
          tmem_ld_32x32b_x32(taddr + h * NT + n0, v);
#pragma unroll
          for (int c = 0; c < 32; ++c) out[c * kOutLd + q * 32 + lane] = v[c];
        }
        if (h == MT - 1 && n0 + 32 >= e.rows) {  // the accumulator is free for the tile after next
          tc_fence_before_sync();
          __syncwarp();
          if (lane == 0) mbar_arrive(&tempty[acc]);
        }
        epilogue_all(true);
        // this warp's 32 columns of row n0 + lane
        const int n = n0 + lane;
        const float* zr = out + lane * kOutLd + q * 32;
        Mst a{kMasked, 0.f, 0.f};
        const int vlim = e.V - col0 - q * 32;
        if (n < e.rows) {
          float v[32];
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            const float4 x = *reinterpret_cast<const float4*>(zr + 4 * j);
            v[4 * j] = x.x;
            v[4 * j + 1] = x.y;
            v[4 * j + 2] = x.z;
            v[4 * j + 3] = x.w;
          }
          if (vlim < 32) {
#pragma unroll
            for (int c = 0; c < 32; ++c)
              if (c >= vlim) v[c] = kMasked;
          }
          if (vlim > 0) add_columns(a, v, e.inv_t);
          if (!p.store_z) {
            const long long y = e.y[n], c = y - col0 - q * 32;
            if (c >= 0 && c < 32 && y < e.V && y != e.ignore_index) e.ztgt[n] = zr[c];
          }
        }
        sums[q * 32 + lane] = vlim > 0 ? make_float4(a.m, a.s, a.t, 1.f) : make_float4(-INFINITY, 0.f, 0.f, 0.f);
        if (p.store_z) {  // a warp a row: 512 bytes at a time
          const int n1 = e.rows - n0 < 32 ? e.rows - n0 : 32;
          for (int i = q; i < n1; i += 4)
            if (in_bounds(col0 + lane * 4 + 3, p.ldz, e.flags))
              *reinterpret_cast<float4*>(p.Z + static_cast<long long>(n0 + i) * p.ldz + col0 + lane * 4) =
                  *reinterpret_cast<const float4*>(out + i * kOutLd + lane * 4);
        }
        epilogue_all(true);
        if (q == 0 && n < e.rows && in_bounds(part, e.nparts, e.flags)) {  // the four warps' columns together
          const float4 x[4] = {sums[lane], sums[32 + lane], sums[64 + lane], sums[96 + lane]};
          const float M = fmaxf(fmaxf(x[0].x, x[1].x), fmaxf(x[2].x, x[3].x));
          RowSum all{0.f, 0.f, 0.f};
#pragma unroll
          for (int i = 0; i < 4; ++i) add_partial(all, x[i], M, e.inv_t);
          e.partials[static_cast<long long>(n) * e.nparts + part] = make_float4(M, all.s, all.t, all.c);
        }
        n0 += 32;
        if (n0 >= e.rows) {
          n0 = 0;
          ++h;
        }
      }
      if (++acc == 2) {
        acc = 0;
        acc_phase ^= 1u;
      }
    }
  }
  tc_fence_before_sync();
  __syncwarp();
  __syncthreads();
  tc_fence_after_sync();
  if (warp == 2) tmem_dealloc(tmem_base, Cfg::kTmemCols);
}

template <int NT, int MT>
cudaError_t launch_rows_nt(const CUtensorMap& h, const CUtensorMap& w, int store_z, float* Z, long long ldz,
                           long long V, long long d, const TokParams& ep, int num_sms, cudaStream_t s) {
  RowsParams p;
  p.w = w;
  p.h = h;
  p.tiles = static_cast<int>((V + MT * 128 - 1) / (MT * 128));
  p.k_blocks = static_cast<int>((d + BK - 1) / BK);
  p.store_z = store_z;
  p.ldz = ldz;
  p.Z = Z;
  p.ep = ep;
  const int grid = p.tiles < num_sms ? p.tiles : num_sms;
  auto kern = k_rows_logits<NT, MT>;
  const cudaError_t e =
      cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, RowsCfg<NT, MT>::kDynamicBytes);
  if (e != cudaSuccess) return e;
  return launch_k(kern, grid, NUM_THREADS, RowsCfg<NT, MT>::kDynamicBytes, s, p);
}

// ----------------------------------------------------------------------------
// Top-K list of a warp: 32 KPL keys in descending order, slot 32 j + lane. A
// key orders by (logit descending, index ascending): the logit's bits mapped
// to an ordered unsigned number above the complement of the index. 0 is empty.
// ----------------------------------------------------------------------------
using Key = unsigned long long;

__device__ __forceinline__ Key make_key(float z, uint32_t idx) {
  uint32_t u = __float_as_uint(z + 0.f);  // -0 counts as 0
  u = (u & 0x80000000u) ? ~u : (u | 0x80000000u);
  return (static_cast<Key>(u) << 32) | static_cast<uint32_t>(~idx);
}
__device__ __forceinline__ float key_value(Key k) {
  const uint32_t u = static_cast<uint32_t>(k >> 32);
  return __uint_as_float((u & 0x80000000u) ? (u & 0x7fffffffu) : ~u);
}
__device__ __forceinline__ uint32_t key_index(Key k) { return ~static_cast<uint32_t>(k); }

// Descending order of 32 keys, one per lane (bitonic sort).
__device__ __forceinline__ Key sort32(Key k, int lane) {
#pragma unroll
  for (int size = 2; size <= 32; size *= 2) {
#pragma unroll
    for (int stride = size / 2; stride > 0; stride /= 2) {
      const Key o = __shfl_xor_sync(0xffffffffu, k, stride);
      const bool low = (lane & stride) == 0, desc = (lane & size) == 0 || size == 32;
      k = (low == desc) == (o > k) ? o : k;
    }
  }
  return k;
}

template <int KPL>
struct TopList {
  Key slot[KPL];
  Key kth;   // candidates must exceed it: the key of slot K - 1, or a lower bound of it given at the start
  Key* buf;  // this warp's 64 entries in shared memory: candidates not merged yet
  int cnt;

  __device__ __forceinline__ void clear(Key* buffer, Key floor = 0) {
#pragma unroll
    for (int j = 0; j < KPL; ++j) slot[j] = 0;
    kth = floor;
    buf = buffer;
    cnt = 0;
  }
  __device__ __forceinline__ Key at(int i) const {  // slot i (warp-uniform), in every lane
    Key k = 0;
#pragma unroll
    for (int j = 0; j < KPL; ++j)
      if (j == (i >> 5)) k = slot[j];
    return __shfl_sync(0xffffffffu, k, i & 31);
  }
  // slot is bitonic (falls, then rises): into descending order.
  __device__ __forceinline__ void bitonic(int lane) {
#pragma unroll
    for (int stride = KPL / 2; stride > 0; stride /= 2) {
#pragma unroll
      for (int j = 0; j < KPL; ++j)
        if ((j & stride) == 0 && slot[j + stride] > slot[j]) {
          const Key o = slot[j];
          slot[j] = slot[j + stride];
          slot[j + stride] = o;
        }
    }
#pragma unroll
    for (int stride = 16; stride > 0; stride /= 2) {
#pragma unroll
      for (int j = 0; j < KPL; ++j) {
        const Key o = __shfl_xor_sync(0xffffffffu, slot[j], stride);
        slot[j] = ((lane & stride) == 0) == (o > slot[j]) ? o : slot[j];
      }
    }
  }
  __device__ __forceinline__ void raise(int K) {
    const Key k = at(K - 1);
    kth = k > kth ? k : kth;
  }
  // Up to 32 waiting candidates sorted and merged at once: of two falling
  // lists, the larger of each entry of one and its mirror image in the other
  // are the largest of both, and bitonic.
  __device__ __forceinline__ void merge_waiting(int K, int lane) {
    __syncwarp();
    Key k = lane < cnt ? buf[lane] : 0;
    const Key rest = 32 + lane < cnt ? buf[32 + lane] : 0;
    __syncwarp();
    k = sort32(k, lane);
    k = __shfl_sync(0xffffffffu, k, 31 - lane);
    slot[KPL - 1] = k > slot[KPL - 1] ? k : slot[KPL - 1];
    bitonic(lane);
    raise(K);
    if (32 + lane < cnt) buf[lane] = rest;
    cnt = cnt > 32 ? cnt - 32 : 0;
    __syncwarp();
  }
  // One candidate per lane (0: none); those that exceed kth wait until there are 32.
  __device__ __forceinline__ void offer(Key cand, int K, int lane) {
    const uint32_t mask = __ballot_sync(0xffffffffu, cand > kth);
    if (mask == 0) return;
    if (cand > kth) buf[cnt + __popc(mask & ((1u << lane) - 1u))] = cand;
    cnt += __popc(mask);
    if (cnt >= 32) merge_waiting(K, lane);
  }
  // What waits, then the lists of the block's warps, merged into everyone's list.
  template <int WARPS>
  __device__ __forceinline__ void finish(Key (*lists)[32 * KPL], int K, int warp, int lane) {
    if (cnt > 0) merge_waiting(K, lane);
#pragma unroll
    for (int j = 0; j < KPL; ++j) lists[warp][32 * j + lane] = slot[j];
    __syncthreads();
#pragma unroll
    for (int step = 1; step < WARPS; step *= 2) {
      if (warp % (2 * step) == 0) {
#pragma unroll
        for (int j = 0; j < KPL; ++j) {
          const Key o = lists[warp + step][32 * KPL - 1 - (32 * j + lane)];
          slot[j] = o > slot[j] ? o : slot[j];
        }
        bitonic(lane);
#pragma unroll
        for (int j = 0; j < KPL; ++j) lists[warp][32 * j + lane] = slot[j];
      }
      __syncthreads();
    }
#pragma unroll
    for (int j = 0; j < KPL; ++j) slot[j] = lists[0][32 * j + lane];
    raise(K);
  }
};

// The row's partial sums merged in a fixed order into lse, logp and entropy, and the
// top K alternatives. The K largest logits (ties to the lower index) lie in the
// K half tiles with the largest maxima (ties to the lower tile): before a half
// tile outside them come K others, each with an element before all of its own.
// So only K x 128 of the row's logits are read again, and of those only the
// ones that reach the K-th largest maximum are candidates.
// One block of WARPS warps per row. The sums are merged in an order that does
// not depend on WARPS (256 running sums, t mod 256, then lanes, then the eight
// groups of 32), so the results do not depend on how many rows a call or a
// chunk has.
template <int KPL, int WARPS>
__global__ void __launch_bounds__(32 * WARPS) k_score(const TokScoreArgs p) {
  grid_dep_wait();
  grid_dep_launch();
  constexpr int kMine = kGroups / WARPS;              // groups of this warp
  constexpr int kBlocks = kMine >= 4 ? 1 : 4 / kMine;  // blocks of 256 partials whose loads are in flight together
  __shared__ Key s_list[WARPS][32 * KPL];
  __shared__ Key s_wait[WARPS][64];
  __shared__ RowSum s_sum[kGroups];
  __shared__ float s_max[WARPS];
  const int lane = threadIdx.x & 31, warp = static_cast<int>(threadIdx.x >> 5);
  const int r = static_cast<int>(blockIdx.x);
  const float4* pr = p.partials + static_cast<long long>(r) * p.nparts;
  const int tiles = (p.V + EPI_COLS - 1) / EPI_COLS;  // half tiles that hold vocabulary columns
  const float* z = p.Z + static_cast<long long>(r) * p.ldz;
  TopList<KPL> top;
  top.clear(s_wait[warp]);
  float M = -INFINITY;
  for (int t0 = warp * 32 + lane; t0 - lane < tiles; t0 += 32 * kGroups * kBlocks) {
    float m[kBlocks][kMine];
#pragma unroll
    for (int b = 0; b < kBlocks; ++b) {
#pragma unroll
      for (int i = 0; i < kMine; ++i) {
        const int t = t0 + 32 * (b * kGroups + i * WARPS);
        m[b][i] = t < tiles ? pr[t].x : -INFINITY;
      }
    }
#pragma unroll
    for (int b = 0; b < kBlocks; ++b) {
#pragma unroll
      for (int i = 0; i < kMine; ++i) {
        const int t = t0 + 32 * (b * kGroups + i * WARPS);
        M = fmaxf(M, m[b][i]);
        if (p.K > 0) top.offer(t < tiles ? make_key(m[b][i], static_cast<uint32_t>(t)) : 0, p.K, lane);
      }
    }
  }
  M = warp_max(M);
  if (lane == 0) s_max[warp] = M;
  __syncthreads();
#pragma unroll
  for (int i = 0; i < WARPS; ++i) M = fmaxf(M, s_max[i]);
  RowSum sums[kMine];
#pragma unroll
  for (int i = 0; i < kMine; ++i) sums[i] = RowSum{0.f, 0.f, 0.f};
  for (int t0 = warp * 32 + lane; t0 - lane < tiles; t0 += 32 * kGroups) {
#pragma unroll
    for (int i = 0; i < kMine; ++i) {
      const int t = t0 + 32 * i * WARPS;
      if (t < tiles) add_partial(sums[i], pr[t], M, p.inv_t);
    }
  }
#pragma unroll
  for (int i = 0; i < kMine; ++i) {
    sums[i] = warp_add(sums[i]);
    if (lane == 0) s_sum[warp + i * WARPS] = sums[i];
  }
  __syncthreads();
  const RowSum acc = add_groups(s_sum);
  const float logs = log_sum(acc);
  if (threadIdx.x == 0) {
    if (p.lse != nullptr) p.lse[r] = fmaf(M, p.inv_t, logs);
    if (p.stats != nullptr) p.stats[r] = make_float2(M, logs);
    if (p.entropy != nullptr) p.entropy[r] = logs - acc.t / (acc.c + acc.s);
    const long long y = p.y[r];
    const bool given = y != p.ignore_index && y >= 0 && y < p.V;
    if (!given && y != p.ignore_index) atomicOr(p.flags, kFlagLabelRange);
    float lp = 0.f;
    if (given) lp = ((p.Z != nullptr ? z[y] : p.ztgt[r]) - M) * p.inv_t - logs;
    if (p.logp != nullptr) p.logp[r] = lp;
  }
  if (p.K == 0) return;
  top.template finish<WARPS>(s_list, p.K, warp, lane);
  TopList<KPL> best;
  const int ntop = tiles < p.K ? tiles : p.K;
  // with K half tiles, the K-th largest of their maxima bounds the K-th logit from below
  best.clear(s_wait[warp], ntop == p.K ? (top.at(p.K - 1) & 0xffffffff00000000ull) : 0);
  __syncthreads();  // s_list is written again below
  for (int i = warp; i < ntop; i += WARPS) {
    const int c = static_cast<int>(key_index(top.at(i))) * EPI_COLS + lane * 4;
    float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
    if (c < p.V && in_bounds(c + 3, p.ldz, p.flags)) v = *reinterpret_cast<const float4*>(z + c);
    best.offer(c < p.V ? make_key(v.x, c) : 0, p.K, lane);
    best.offer(c + 1 < p.V ? make_key(v.y, c + 1) : 0, p.K, lane);
    best.offer(c + 2 < p.V ? make_key(v.z, c + 2) : 0, p.K, lane);
    best.offer(c + 3 < p.V ? make_key(v.w, c + 3) : 0, p.K, lane);
  }
  best.template finish<WARPS>(s_list, p.K, warp, lane);
  if (warp != 0) return;
#pragma unroll
  for (int j = 0; j < KPL; ++j) {
    const int i = 32 * j + lane;
    if (i < p.K) {
      const long long at = static_cast<long long>(r) * p.K + i;
      p.top_logp[at] = (key_value(best.slot[j]) - M) * p.inv_t - logs;
      const uint32_t v = key_index(best.slot[j]);  // past V only if a row of NaN left the list short
      p.top_idx[at] = v < static_cast<uint32_t>(p.V) ? v : static_cast<uint32_t>(p.V - 1);
    }
  }
}

// One block per row: the row's scale, Ht = bf16(scale H), and, from logits kept
// since the forward (TILE), the gradient tile of TOK_GRAD: one pass over the row,
// 4 bytes read and 2 written a logit, in place of the logits GEMM (2 d flops a
// logit; 2048 rows of V = 151936: 302 us, 92% of the copy bandwidth, against 700
// at d = 2048). A row without upstream gradient is written without reading its
// logits.
template <bool TILE>
__global__ void __launch_bounds__(kRowThreads, 8) k_score_grad(const ScoreGradArgs p) {
  grid_dep_wait();
  grid_dep_launch();
  const int r = blockIdx.x, tid = threadIdx.x;
  if (r == 0 && p.st != nullptr) {  // what the label scan would do, without a launch of its own
    for (int i = tid; i < p.ncnt; i += kRowThreads) p.cnt[i] = 0;
    int bad = 0;
    for (long long i = tid; i < p.N; i += kRowThreads) {
      const long long v = p.y_all[i];
      bad |= v != p.ignore_index && (v < 0 || v >= p.V);
    }
    bad = __syncthreads_or(bad);
    if (tid == 0) {
      p.st->flags = (p.keep_flags ? p.st->flags : 0) | (bad ? kFlagLabelRange : 0);
      p.st->gscale = 1.f;
      p.st->lscale = 1.0;
    }
  }
  const Upstream u = upstream(r, p.y, p.ignore_index, p.V, p.g_logp, p.g_entropy, p.inv_t);
  const float entry = label_entry(u, p.logp[r], p.entropy, r), scale = row_scale(u, entry);
  const float label = scale == 1.f ? entry : 1.f;  // the label's entry of the tile
  if (tid == 0) {
    p.rowscale[r] = scale;
    p.label[r] = label;
  }
  if (p.Ht != nullptr) {
    const int groups = p.d / 8;
    const long long at = static_cast<long long>(r) * groups;
    scale_row(p.H + at, p.Ht + at, groups, scale, u.a != 0.f || u.e != 0.f, tid, kRowThreads);
  }
  if (!TILE) return;
  const float* z = p.Z + static_cast<long long>(r) * p.ldz;
  __nv_bfloat16* g = p.G + static_cast<long long>(r) * p.ldg;
  write_grad_row(grad_row(u, scale, p.stats, p.lse, p.entropy, r, p.inv_t), label, z, g, p.V, tid, kRowThreads);
}

// ----------------------------------------------------------------------------
// Distillation
// ----------------------------------------------------------------------------
__device__ __forceinline__ float teacher_value(const void* t, int bf16, long long i) {
  return bf16 ? __bfloat162float(static_cast<const __nv_bfloat16*>(t)[i]) : static_cast<const float*>(t)[i];
}

// Clears the status block and the dH part counters; k_distill_count adds into them.
__global__ void __launch_bounds__(1024) k_distill_init(DevStatus* st, int* cnt, int ncnt) {
  grid_dep_wait();
  grid_dep_launch();
  clear_status(st, cnt, ncnt, threadIdx.x, blockDim.x);
}

// Rows with at least one kept entry (an index in [0, V) whose teacher value is
// above -inf), and the range bit for an index that is neither kept nor
// ignore_index. One warp per row; the count is a sum of whole numbers, so the
// order of the atomics does not change it.
__global__ void __launch_bounds__(1024) k_distill_count(const int64_t* __restrict__ idx, const void* __restrict__ tv,
                                                        int t_bf16, long long N, int K, int V, long long ignore_index,
                                                        DevStatus* st) {
  grid_dep_wait();
  grid_dep_launch();
  __shared__ int s_cnt, s_bad;
  if (threadIdx.x == 0) s_cnt = s_bad = 0;
  __syncthreads();
  const int lane = threadIdx.x & 31;
  const long long nwarps = static_cast<long long>(gridDim.x) * (blockDim.x >> 5);
  for (long long r = (blockIdx.x * static_cast<long long>(blockDim.x) + threadIdx.x) >> 5; r < N; r += nwarps) {
    bool kept = false, bad = false;
    for (int k = lane; k < K; k += 32) {
      const long long v = idx[r * K + k];
      if (v == ignore_index) continue;
      if (v < 0 || v >= V)
        bad = true;
      else if (!(teacher_value(tv, t_bf16, r * K + k) == -INFINITY))
        kept = true;
    }
    const bool any = __any_sync(0xffffffffu, kept), anybad = __any_sync(0xffffffffu, bad);
    if (lane == 0) {
      if (any) atomicAdd(&s_cnt, 1);
      if (anybad) atomicOr(&s_bad, 1);
    }
  }
  __syncthreads();
  if (threadIdx.x == 0) {
    if (s_cnt) atomicAdd(reinterpret_cast<unsigned long long*>(&st->n_counted), static_cast<unsigned long long>(s_cnt));
    if (s_bad) atomicOr(&st->flags, kFlagLabelRange);
  }
}

// n, 1/n (1 for a sum) and the factor of the GEMMs behind, g T / n.
__device__ __forceinline__ double set_scales(const DistillArgs& p, long long counted, bool write) {
  const long long n = p.n_override >= 0 ? p.n_override : counted;
  const double weight = p.mean ? (n > 0 ? 1.0 / static_cast<double>(n) : 0.0) : 1.0;
  if (write) {
    const float up = p.grad_loss != nullptr ? *p.grad_loss : 1.f;
    p.st->n_valid = n;
    p.st->gscale = static_cast<float>(static_cast<double>(up) * weight / static_cast<double>(p.inv_t));
  }
  return weight;
}

// Writes the row's loss; the block that counts the call's last row sums them
// all in fp64, in an order that does not depend on which block that is. With
// one chunk n is known only then (whole numbers, so their order does not
// change it), and that block sets the scales.
__device__ __forceinline__ void finish_row(const DistillArgs& p, int r, float loss, bool kept) {
  __shared__ int s_last;
  __shared__ double s_sum[kRowThreads];
  const int tid = threadIdx.x;
  if (tid == 0) {
    p.row_loss[r] = loss;
    if (p.count_here && kept) atomicAdd(reinterpret_cast<unsigned long long*>(&p.st->n_counted), 1ull);
    __threadfence();
    s_last = atomicAdd(&p.st->rows_done, 1) == static_cast<int>(p.N - 1);
  }
  __syncthreads();
  if (!s_last) return;
  __threadfence();
  double sum = 0.0;
  for (long long i = tid; i < p.N; i += kRowThreads) sum += static_cast<double>(__ldcg(p.all_rows + i));
  s_sum[tid] = sum;
  __syncthreads();
  for (int w = kRowThreads / 2; w > 0; w >>= 1) {
    if (tid < w) s_sum[tid] += s_sum[tid + w];
    __syncthreads();
  }
  if (tid == 0) {
    const long long counted = __ldcg(&p.st->n_counted);
    *p.loss = static_cast<float>(s_sum[0] * set_scales(p, counted, p.count_here != 0));
  }
}

// dW's second operand: the row of H, or zeros where the row keeps no entry, as its
// zeros in G times a NaN in H would not be zero (4 bytes an element of H next to 6 an
// entry of G).
__device__ __forceinline__ void copy_row(const DistillArgs& p, int r, bool kept) {
  if (p.Ht == nullptr) return;
  const int groups = p.d / 8;
  const long long at = static_cast<long long>(r) * groups;
  for (int i = threadIdx.x; i < groups; i += kRowThreads)
    p.Ht[at + i] = kept ? p.H[at + i] : make_uint4(0u, 0u, 0u, 0u);
}

// One block per row of the chunk. The row's partial sums give lse; the K entries
// give the teacher's probabilities q and the row's loss
//   T^2 sum_k q_k (log q_k - z'_k + lse);
// with GRAD the row of the gradient tile is written in one pass over the
// stored logits,
//   G_v = m p_v - sum_k q_k [v = idx_k],   m = sum_k q_k,
// in fp32 with one rounding to bf16 (the operand type of the GEMMs behind
// it). The kept entries are written last, by one thread each: of entries with
// the same index the first writes, with the sum of their q.
template <bool GRAD>
__global__ void __launch_bounds__(kRowThreads, 8) k_distill_row(const DistillArgs p) {
  grid_dep_wait();
  grid_dep_launch();
  __shared__ float red[kRowThreads / 32];
  __shared__ RowSum s_sum[kGroups];
  __shared__ int s_idx[kMaxTop];
  __shared__ float s_q[kMaxTop];
  const int r = blockIdx.x, tid = threadIdx.x;
  const float* z = p.Z + static_cast<long long>(r) * p.ldz;
  __nv_bfloat16* g = GRAD ? p.G + static_cast<long long>(r) * p.ldg : nullptr;

  // several chunks: n is known since the count ran, and the first row of each sets the scales
  if (!p.count_here && r == 0 && tid == 0) set_scales(p, p.st->n_counted, true);

  // the teacher's entry of this thread
  const long long at = static_cast<long long>(r) * p.K + tid;
  int vi = -1;
  float tv = -INFINITY;
  if (tid < p.K) {
    const long long v = p.idx[at];
    if (v >= 0 && v < p.V && v != p.ignore_index) {
      tv = teacher_value(p.t, p.t_bf16, at);
      if (!(tv == -INFINITY)) vi = static_cast<int>(v);
    } else if (v != p.ignore_index && p.count_here) {
      atomicOr(&p.st->flags, kFlagLabelRange);
    }
  }
  const bool kept = __syncthreads_or(vi >= 0) != 0;
  if (!kept) {  // nothing of the teacher in this row: no loss, a zero gradient
    finish_row(p, r, 0.f, false);
    if (GRAD) {
      copy_row(p, r, false);
      for (int c = tid * 8; c < p.V; c += kRowThreads * 8) *reinterpret_cast<uint4*>(g + c) = make_uint4(0, 0, 0, 0);
    }
    return;
  }
  float q = 0.f, logq = 0.f;
  if (p.renormalize) {
    const float top = block_max(vi >= 0 ? tv : -INFINITY, red);
    const float e = vi >= 0 ? exp2f((tv - top) * p.inv_t * kLog2e) : 0.f;
    const float sum = block_sum(e, red);
    if (vi >= 0) {
      q = e / sum;
      logq = (tv - top) * p.inv_t - logf(sum);
    }
  } else if (vi >= 0) {
    q = expf(tv);
    logq = tv;
  }
  const float mass = block_sum(q, red);

  const float4* pr = p.partials + static_cast<long long>(r) * p.nparts;
  const int tiles = (p.V + EPI_COLS - 1) / EPI_COLS;
  float M = -INFINITY;
  for (int t = tid; t < tiles; t += kRowThreads) M = fmaxf(M, pr[t].x);
  M = block_max(M, red);
  RowSum acc{0.f, 0.f, 0.f};
  for (int t = tid; t < tiles; t += kRowThreads) add_partial(acc, pr[t], M, p.inv_t);
  acc = warp_add(acc);
  if ((tid & 31) == 0) s_sum[tid >> 5] = acc;
  if (tid < kMaxTop) {
    s_idx[tid] = vi;
    s_q[tid] = q;
  }
  __syncthreads();
  acc = add_groups(s_sum);
  const float logs = log_sum(acc);

  float zk = 0.f, term = 0.f;
  if (vi >= 0) {
    zk = z[vi];
    if (q > 0.f || q != q) term = q * (logq - (zk - M) * p.inv_t + logs);
  }
  const float loss = block_sum(term, red);
  finish_row(p, r, loss / (p.inv_t * p.inv_t), true);
  if (!GRAD) return;

  copy_row(p, r, true);
  const float k = p.inv_t * kLog2e, w = mass / (acc.c + acc.s);
  for (int c = tid * 8; c < p.V; c += kRowThreads * 8) {
    // columns past V (up to 7) lie inside the row's padding: never read by the GEMMs
    const float4 a = __ldcs(reinterpret_cast<const float4*>(z + c));
    const float4 b = __ldcs(reinterpret_cast<const float4*>(z + c + 4));
    uint4 o;
    o.x = pack_bf16x2(w * ex2_approx((a.x - M) * k), w * ex2_approx((a.y - M) * k));
    o.y = pack_bf16x2(w * ex2_approx((a.z - M) * k), w * ex2_approx((a.w - M) * k));
    o.z = pack_bf16x2(w * ex2_approx((b.x - M) * k), w * ex2_approx((b.y - M) * k));
    o.w = pack_bf16x2(w * ex2_approx((b.z - M) * k), w * ex2_approx((b.w - M) * k));
    *reinterpret_cast<uint4*>(g + c) = o;
  }
  __syncthreads();
  if (vi >= 0) {
    float sum = 0.f;
    bool first = true;
    for (int j = 0; j < p.K; ++j) {
      if (s_idx[j] != vi) continue;
      if (j < tid) first = false;
      sum += s_q[j];
    }
    if (first) g[vi] = __float2bfloat16_rn(w * ex2_approx((zk - M) * k) - sum);
  }
}

}  // namespace

// ----------------------------------------------------------------------------
// Launch wrappers
// ----------------------------------------------------------------------------
// Hidden size up to which epilogues that store little (bf16 exp tiles, or nothing) take eight warps: a tile of few k-blocks
// is bound by its epilogue, a tile of many by the MMA. 2048 rows of V = 151936, eight warps and four, us: exp tiles d = 64
// 128 and 182, 256 159 and 186, 512 217 and 215; statistics alone d = 64 140 and 196, 256 174 and 200, 512 212 and 209; with
// fp32 logits stored d = 256 272 and 253.
constexpr long long kShortK = 256;

cudaError_t launch_tok_logits(int mode, const CUtensorMap& a, const CUtensorMap& b, const CUtensorMap& c, long long M,
                              long long N, long long K, const TokParams& ep, int num_sms, cudaStream_t s) {
  switch (mode) {
    case TOK_STATS:
      return K <= kShortK ? launch_tok_mode<TOK_STATS, EPI_WARPS_SHORT>(a, b, c, M, N, K, ep, num_sms, s)
                          : launch_tok_mode<TOK_STATS>(a, b, c, M, N, K, ep, num_sms, s);
    case TOK_STATS_Z: return launch_tok_mode<TOK_STATS_Z>(a, b, c, M, N, K, ep, num_sms, s);
    case TOK_EXP:
      return K <= kShortK ? launch_tok_mode<TOK_EXP, EPI_WARPS_SHORT>(a, b, c, M, N, K, ep, num_sms, s)
                             : launch_tok_mode<TOK_EXP>(a, b, c, M, N, K, ep, num_sms, s);
    default: return launch_tok_mode<TOK_GRAD>(a, b, c, M, N, K, ep, num_sms, s);
  }
}

cudaError_t launch_rows_logits(const CUtensorMap& h, const CUtensorMap& w, int store_z, float* Z, long long ldz,
                               long long V, long long d, const TokParams& ep, int num_sms, cudaStream_t s) {
  switch (few_rows_box(ep.rows)) {
    case 32: return launch_rows_nt<32, 2>(h, w, store_z, Z, ldz, V, d, ep, num_sms, s);
    case 64: return launch_rows_nt<64, 1>(h, w, store_z, Z, ldz, V, d, ep, num_sms, s);
    default: return launch_rows_nt<96, 1>(h, w, store_z, Z, ldz, V, d, ep, num_sms, s);
  }
}

template <int WARPS>
cudaError_t launch_score_warps(const TokScoreArgs& p, cudaStream_t s) {
  if (p.K <= 32) return launch_k(k_score<1, WARPS>, p.rows, 32 * WARPS, 0, s, p);
  if (p.K <= 64) return launch_k(k_score<2, WARPS>, p.rows, 32 * WARPS, 0, s, p);
  return launch_k(k_score<kMaxTop / 32, WARPS>, p.rows, 32 * WARPS, 0, s, p);
}

// Warps of a row's block: with few rows the row's own latency counts, with
// many the GPU is full and every further warp is one more list to merge
// (microseconds at V = 151936 and K = 20 with 8 / 2 warps: 32 rows
// 12 / 18, 512 rows 20 / 24, 1024 rows 29 / 29, 4096 rows 82 / 59).
constexpr int kScoreRows8 = 512;

cudaError_t launch_score(const TokScoreArgs& p, cudaStream_t s) {
  if (p.rows <= 0) return cudaSuccess;
  return p.rows <= kScoreRows8 ? launch_score_warps<8>(p, s) : launch_score_warps<2>(p, s);
}

cudaError_t launch_score_grad(const ScoreGradArgs& p, int rows, cudaStream_t s) {
  if (rows <= 0) return cudaSuccess;
  return p.Z != nullptr ? launch_k(k_score_grad<true>, rows, kRowThreads, 0, s, p)
                        : launch_k(k_score_grad<false>, rows, kRowThreads, 0, s, p);
}

cudaError_t launch_distill_count(const int64_t* idx, const void* t, int t_bf16, long long N, int K, int V,
                                 long long ignore_index, DevStatus* st, int* cnt, int ncnt, int num_sms,
                                 cudaStream_t s) {
  const cudaError_t e = launch_k(k_distill_init, 1, 1024, 0, s, st, cnt, ncnt);
  if (e != cudaSuccess || N <= 0) return e;
  const long long want = (N + 31) / 32;
  const int grid = static_cast<int>(want < num_sms ? want : num_sms);
  return launch_k(k_distill_count, grid, 1024, 0, s, idx, t, t_bf16, N, K, V, ignore_index, st);
}

cudaError_t launch_distill_row(const DistillArgs& p, int rows, cudaStream_t s) {
  if (rows <= 0) return cudaSuccess;
  return p.G != nullptr ? launch_k(k_distill_row<true>, rows, kRowThreads, 0, s, p)
                        : launch_k(k_distill_row<false>, rows, kRowThreads, 0, s, p);
}

}  // namespace lce
