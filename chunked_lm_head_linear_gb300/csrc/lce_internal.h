// Internal interface between the C-ABI layer (lce_api.cu) and the kernels
// (lce_kernels.cu). Not part of the public header.
#pragma once

#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <cstdint>
#include <utility>

namespace lce {

// Programmatic dependent launch. Every kernel of the library starts with
// grid_dep_wait(): it returns once the grids it depends on (the previous
// kernel of the stream) have completed and their writes are visible, at once
// when the launch did not ask for programmatic serialization. grid_dep_launch()
// then lets the next kernel of the stream be scheduled; that kernel's own wait
// still holds its work back until this one has completed.
__device__ __forceinline__ void grid_dep_wait() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
__device__ __forceinline__ void grid_dep_launch() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }

// Every kernel of the library goes out with programmatic stream serialization,
// so that its launch and the scheduling of its blocks overlap the end of the
// kernel before it in the stream (its grid_dep_wait keeps the order).
template <typename... KArgs, typename... Args>
inline cudaError_t launch_k(void (*kern)(KArgs...), dim3 grid, dim3 block, size_t smem, cudaStream_t s,
                            Args&&... args) {
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = block;
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kern, std::forward<Args>(args)...);
}

// Device status bits (the workspace's flag word; the first two equal the
// public LCE_DEVICE_* bits).
constexpr int kFlagLabelRange = 1;
constexpr int kFlagTimeout = 2;
constexpr int kFlagBounds = 4;

// Bounds-checking debug build (compiled with -DLCE_CHECKS): every index a
// kernel computes into a plain global buffer, and every tile coordinate it
// hands to TMA, is checked before use; a bad one sets kFlagBounds in the
// device status word and the access is skipped (nothing traps). In the normal
// build the checks compile to nothing.
#if defined(LCE_CHECKS)
constexpr bool kChecks = true;
#else
constexpr bool kChecks = false;
#endif

// True if 0 <= i < n (always true without LCE_CHECKS).
__device__ __forceinline__ bool in_bounds(long long i, long long n, int* flags) {
  if constexpr (!kChecks) {
    return true;
  } else {
    if (i >= 0 && i < n) return true;
    if (flags != nullptr) atomicOr(flags, kFlagBounds);
    return false;
  }
}

// Device-side status block at the start of the workspace.
struct DevStatus {
  int flags;              // kFlag* bits
  int rows_done;          // distillation and the losses: rows (pairs) whose loss is written
  long long n_valid;      // denominator n actually used (count or override)
  long long n_counted;    // valid labels counted in this call
  float gscale;           // g / n (mean), g (sum); 0 when n == 0 under mean
  float pad1;
  double lscale;          // 1 / n (mean), 1 (sum); 0 when n == 0 under mean
};

enum FwdMode : int {
  FWD_STATS = 0,    // per-(row, vocab tile) max / sum-exp partials + target logit
  FWD_STATS_P = 1,  // FWD_STATS + exp-tile P = bf16(exp(z - ref_row)) stored for the backward
  FWD_GRAD = 2,     // gradient tile exp(z - lse) - onehot (valid rows), from a known lse
  FWD_REF = 3,      // row maximum over the first 128 words (one launch over the first tile)
  FWD_STATS_PX = 4, // exact FWD_STATS partials + the exp tile P = bf16(exp(z - ref_row)) (vocabulary shards:
                    // the statistics are exchanged before the tile's scale is known)
};

// An exp-tile entry may exceed the row reference by at most this many nats;
// beyond it the chunk falls back to the exact gradient tile (FWD_GRAD).
constexpr float kRefGuardSum = 1.0e26f;  // ~e^60: bound on a 32-column sum of exp(z - ref)
constexpr float kRefGuardLogit = 60.f;   // the same bound in nats, on lse - ref (vocabulary shards)

struct FwdParams {
  int mode;
  int rows;              // rows of this chunk
  int V;                 // vocabulary columns of this GEMM (a shard's size under vocabulary parallelism)
  int V_total;           // label range: labels in [0, V_total) are valid
  long long y_offset;    // label y sits in column y - y_offset (0 unless W is a vocabulary shard)
  int nparts;            // partials per row: two per 256-column vocabulary tile
  long long ignore_index;
  const int64_t* y;      // labels of this chunk
  float2* partials;      // [rows, nparts] (max, sum-exp) per 128-column half tile
  float* ztgt;           // [rows] logit of the label
  float* ref;            // [rows] row reference (FWD_REF output, FWD_STATS_P / FWD_STATS_PX input)
  const float* lse;      // [rows] (FWD_GRAD input)
  __nv_bfloat16* P;      // [rows, ldp] exp tile (FWD_STATS_P) or gradient tile (FWD_GRAD)
  long long ldp;
  int* flags;
  int* guard;            // FWD_STATS_P(X): set to 1 if some logit exceeds its row reference + guard
  const int* only_if;    // if non-null, the launch does nothing unless *only_if != 0
};

struct DhParams {
  int rows;              // rows of this chunk
  int N;                 // d
  int f32_out;           // 1: fp32 output (a partial dH to be summed across vocabulary shards)
  __nv_bfloat16* out;    // dH of this chunk, [rows, ld] (bf16, or fp32 when f32_out)
  long long ld;
  const float* rowscale; // optional per-row factor (nullptr: none)
  const DevStatus* st;   // gscale
  // The K = V reduction of a dH tile runs as `parts` tiles over fixed vocabulary
  // parts (dh_parts_for(V)); each stores its fp32 sum, and the last of them to
  // arrive adds the parts in part order and writes the tile.
  int parts;             // 1: one tile over the whole vocabulary; 0 (in): dh_parts_for(V)
  int tiles_n;           // 256-column blocks of d (tile index = row block * tiles_n + column block)
  float4* part_buf;      // [tiles, parts, 2 CTAs, 4 warps, 64 column groups, 32 lanes] fp32 part sums
  int* part_cnt;         // [tiles, 2, 4] arrivals per warp slice; zero before and after each launch
  long long part_slices; // counters (warp slices) the workspace holds (checked build)
  int block_major;       // the parts of each block run back to back on one cluster, in part order
  int split_rows;        // not 0: the parts are stored as they are, part s in rows [s split_rows, (s + 1) split_rows)
                         // of the fp32 output, and added behind the launch (launch_dh_sum)
};

// dH parts: the vocabulary's k-blocks (64 words each) are cut into at most
// kDhParts parts of ceil(kblocks / kDhParts) k-blocks. A function of V alone,
// so that every chunk size sums dH in the same order (dH is bitwise the same
// for every chunk size).
constexpr int kDhParts = 4;
inline int dh_kblocks_per_part(long long V) {
  const long long kb = (V + 63) / 64;
  return static_cast<int>((kb + kDhParts - 1) / kDhParts);
}
inline int dh_parts_for(long long V) {
  const long long kb = (V + 63) / 64;
  const long long per = dh_kblocks_per_part(V);
  return per > 0 ? static_cast<int>((kb + per - 1) / per) : 1;
}

// Time of a dW tile in units of one of its k-blocks (w_k of them): short ones are bound by their epilogue and by writing
// dW, in fp32 twice the bytes. Weighed as their k-blocks alone, short batches piled dW tiles onto the clusters that share no
// dH tile (64 rows of V = 151936, d = 4096 with four dH parts: 2344 us and 881). Backward of V = 151936, d = 2048 in us with
// a tile at: 128 rows (w_k 2) 4 280 to 302, 6 245, 8 275, 10 294; 256 rows 5 270, 6 256, 8 282, 10 301; 384 rows 7 371, 8
// 348, 10 381; 512 rows 9 404, 10 398, 11 410, 14 430; 768 rows 12 585, 13 574, 14 553. fp32: 256 rows 6 363, 8 345 to 357,
// 10 378; 512 rows 11 477, 14 463.
inline double dw_tile_cost(long long w_k, bool bf16) {
  if (w_k >= 14) return static_cast<double>(w_k);
  if (!bf16) return w_k >= 8 ? 14.0 : static_cast<double>(w_k + 4);
  return w_k > 12 ? 14.0 : w_k > 4 ? static_cast<double>(w_k + 2) : 6.0;
}

// dH parts where no such promise is made (the policy and preference losses). Each is stored as an fp32 tile of its own
// and a launch behind the GEMMs adds them. In k-blocks of time (0.31 us), a part takes its share of the kb there are and
// kDhStore more, the sum kDhSum and what it reads and writes; the fewest parts that stay within a tenth of the best are
// taken. With dW in the launch its tiles fill the clusters that have no part of dH, and the launch takes a cluster's fair
// share, or a part, whichever is longer. Short batches have few dH tiles, and four parts of V = 151936 run 594 k-blocks
// each on one cluster, 207 us whatever the rest takes; long ones do without parts. (Weighed with a bf16 dW; an fp32 one is
// within 3% of its best with the same: 128 rows of d = 2048 475 us of 454 to 559, 512 rows 695 of 662 to 719.) Without dW
// the clusters take the parts in rounds. Policy steps of a frozen W, V = 151936, us with the parts that a launch with dW
// would have, and with these: 256 x 2048 302 -> 245, 512 x 2048 531 -> 394, 512 x 4096 1128 -> 775, 2560 x 2048 2257 ->
// 1854, 2048 x 256 335 -> 309. clusters: two of the device's 152 SMs each (the workspace's size may not depend on it).
constexpr int kMaxDhParts = 32;
constexpr double kDhStore = 8.0, kDhSum = 10.0;
inline int dh_parts_balanced(long long rows, long long V, long long d, bool with_dw) {
  constexpr long long clusters = 76;
  const long long kb = (V + 63) / 64, cols = (d + 255) / 256, tiles = (rows + 255) / 256 * cols;
  const double k = static_cast<double>(kb);
  const double fair = (static_cast<double>(tiles) * k +
                       static_cast<double>((V + 255) / 256 * cols) * dw_tile_cost((rows + 63) / 64, true)) / clusters;
  const double bytes = 8.0 * static_cast<double>(rows) * static_cast<double>(d);  // of a part, written and read
  auto time = [&](int p) {
    const double part = p == 1 ? k : k / p + kDhStore;
    const double sum = p == 1 ? 0.0 : kDhSum + p * bytes / (5.0e12 * 0.31e-6);
    if (!with_dw) return static_cast<double>((tiles * p + clusters - 1) / clusters) * part + sum;
    return (part > fair ? part : fair) + sum;
  };
  double best = time(1);
  for (int p = 2; p <= kMaxDhParts; ++p) best = time(p) < best ? time(p) : best;
  long long parts = 1;
  while (parts < kMaxDhParts && time(static_cast<int>(parts)) > 1.1 * best) ++parts;
  const long long per = (kb + parts - 1) / parts;
  return static_cast<int>((kb + per - 1) / per);
}

struct DwParams {
  int rows;              // V
  int N;                 // d
  float* out;            // dW [V, ld]
  long long ld;
  int accumulate;        // 1: out += result
  const DevStatus* st;   // gscale
  int bf16_out;          // 1: bf16 output, stored once: bf16(add + result) (add null: bf16(result))
  const float* add;      // [V, ld] fp32, the sum over earlier chunks (bf16_out)
};

// Kernel launches (return cudaGetLastError()).
// Also zeroes guards[0, nguards) and cnt[0, ncnt) (the dH part counters).
cudaError_t launch_prepare(const int64_t* y, long long N, int V, long long ignore_index, int reduction,
                           long long n_override, const float* grad_loss, DevStatus* st, int* guards, int nguards,
                           int* cnt, int ncnt, cudaStream_t s);
// Logits GEMM of a chunk: z [M, N] = A [M, K] B [N, K]^T with the FwdEpi
// epilogue; a, b: K-major operand maps, c: the epilogue's store map (any valid
// map if the mode stores nothing).
// no_loads = 1 only for the timeout test (LCE_TEST_FORCE_TIMEOUT): no operand
// loads are issued, so the MMA issuer's bounded wait runs out.
cudaError_t launch_logits(const CUtensorMap& a, const CUtensorMap& b, const CUtensorMap& c, long long M, long long N,
                          long long K, const FwdParams& ep, int no_loads, int num_sms, cudaStream_t s);
// Backward GEMMs of a chunk in one launch: dH_c = G W (ah: G K-major, bh: W
// N-major, ch: dH store) and dW (+)= G^T B (aw: G M-major, bw: B N-major, cw:
// dW store / reduce-add). Only the dW rows [v_begin, v_end) are computed
// (v_end < 0: to V; v_begin a multiple of 256), and the dH tiles only if
// with_dh; every tile computed is the same as in the whole launch.
cudaError_t launch_backward(const CUtensorMap& ah, const CUtensorMap& bh, const CUtensorMap& ch, const CUtensorMap& aw,
                            const CUtensorMap& bw, const CUtensorMap& cw, long long rows, long long V, long long d,
                            const DhParams& h, const DwParams& w, int* flags, int num_sms, cudaStream_t s,
                            long long v_begin = 0, long long v_end = -1, bool with_dh = true);
// dH of `rows` rows: bf16(gscale rowscale sum_s part[s]), the parts [parts, split_rows, d] added in order.
cudaError_t launch_dh_sum(const float* part, int parts, long long split_rows, long long rows, int d,
                          const float* rowscale, const DevStatus* st, void* dH, cudaStream_t s);
cudaError_t launch_combine(const float2* partials, int nparts, int rows, const float* ztgt, const int64_t* y,
                           int V, long long ignore_index, float* lse, float* loss_i, cudaStream_t s);
// Per row of a chunk: lse, loss_i, alpha_i = exp(ref_i - lse_i) (1 if the chunk's guard is set,
// 0 for ignored rows), the label entry of the exp tile P, and Ht_i = bf16(alpha_i H_i) for the
// chunk's rows of H [rows, d] (the B operand of the dW GEMM). With only_if, the launch does
// nothing unless *only_if != 0.
cudaError_t launch_combine_exp(const float2* partials, int nparts, int rows, const float* ztgt, const int64_t* y,
                               int V, long long ignore_index, const float* ref, const int* guard, float* lse,
                               float* loss_i, float* alpha, __nv_bfloat16* P, long long ldp,
                               const __nv_bfloat16* H, int d, __nv_bfloat16* Ht, const int* only_if, int* flags,
                               cudaStream_t s);
// Vocabulary shards: per-row partial (max, sum-exp, target logit, has-target)
// of this shard, and the fixed-order merge of R shards' partials.
cudaError_t launch_shard_stats(const float2* partials, int nparts, int rows, const float* ztgt, const int64_t* y,
                               long long y_offset, int V_shard, int V_total, long long ignore_index, float4* stats,
                               cudaStream_t s);
cudaError_t launch_shard_merge(const float4* stats, int R, long long N, const int64_t* y, int V_total,
                               long long ignore_index, float* lse, float* loss_i, cudaStream_t s);
// Chunk rows of the stored-tile vocabulary-parallel backward (two launches):
// the merge of launch_shard_merge on stats [R, rows, 4] -> lse, setting *guard
// for a row whose label lies in the shard and whose lse exceeds its reference
// by more than kRefGuardLogit; then alpha_i = exp(ref_i - lse_i) (1 if *guard:
// the tile is then the exact gradient; 0 for ignored rows), the label entry of
// this shard's exp tile P when the label lies in the shard, and
// Ht_i = bf16(alpha_i H_i) for H [rows, d].
cudaError_t launch_vshard_scale(const float4* stats, int R, int rows, const int64_t* y, long long y_offset,
                                int V_shard, int V_total, long long ignore_index, const float* ref, int* guard,
                                float* lse, float* alpha, __nv_bfloat16* P, long long ldp, const __nv_bfloat16* H,
                                int d, __nv_bfloat16* Ht, int* flags, cudaStream_t s);
// Final zero-centred RMSNorm (lce_rmsnorm.cu). rmsnorm_bwd_blocks(N) partial
// rows of d floats are the backward's scratch.
int rmsnorm_bwd_blocks(long long N);
cudaError_t launch_rmsnorm_fwd(const void* x, const float* w, long long N, int d, float eps, void* H, float* rstd,
                               cudaStream_t s);
cudaError_t launch_rmsnorm_bwd(const void* x, const float* w, const float* rstd, const void* dH, long long N, int d,
                               void* dx, float* dw, float* part, cudaStream_t s);
// Layer norm (lce_layernorm.cu). x in bf16 or fp32; w and b in fp32 or bf16, either may be null.
struct LayerNormArgs {
  const void* x;           // [N, d]
  const void* w;           // [d] or null (ones)
  const void* b;           // [d] or null (zeros), forward only
  int x_f32, w_bf16;
  int no_cluster;          // backward: as where no cluster of sixteen fits (tests)
  long long N;
  int d;
  float eps;
  void* H;                 // [N, d] bf16 (forward)
  float* mean;             // [N]: out (or null) of the forward, in for the backward
  float* rstd;             // [N]
  const void* dH;          // [N, d] bf16 (backward)
  void* dx;                // [N, d] as x, or null
  float* dw;               // [d] or null
  float* db;               // [d] or null
  float* part;             // [2, layernorm_parts(N, d), d] partial sums of dw and db
};
int layernorm_parts(long long N, long long d);
cudaError_t launch_layernorm_fwd(const LayerNormArgs& p, int num_sms, cudaStream_t s);
cudaError_t launch_layernorm_bwd(const LayerNormArgs& p, int num_sms, cudaStream_t s);
// In-place x *= *g of n_bf16 bf16 values (a multiple of 8) and n_f32 fp32 values (a multiple of 4).
cudaError_t launch_scale(void* bf16, long long n_bf16, float* f32, long long n_f32, const float* g, int num_sms,
                         cudaStream_t s);
// The same of two bf16 arrays (multiples of 8), in one launch.
cudaError_t launch_scale_bf16(void* a, long long n_a, void* b, long long n_b, const float* g, int num_sms,
                              cudaStream_t s);
cudaError_t launch_finalize(const float* loss_i, long long N, const DevStatus* st, float* loss, cudaStream_t s);

// ----------------------------------------------------------------------------
// Token operators (lce_tokens.cu)
// ----------------------------------------------------------------------------
enum TokMode : int {
  TOK_STATS = 0,    // partial sums of each (row, half tile) and the label's logit
  TOK_STATS_Z = 1,  // the partial sums and the fp32 logits
  TOK_GRAD = 2,     // gradient tile of log-probability and entropy
  TOK_EXP = 3,      // exp tile exp((z - z_y) / T) of the label's logit z_y in bf16, and its sums
};

constexpr int kMaxTop = 128;  // most alternatives of a row, most teacher entries of a row

struct TokParams {
  int rows;              // rows of this chunk
  int V;
  int nparts;            // partials per row: two per 256-column vocabulary tile
  float inv_t;           // 1 / temperature
  long long ignore_index;
  const int64_t* y;      // labels of this chunk (TOK_STATS, TOK_GRAD)
  float4* partials;      // [rows, nparts] (m, s, t, c), see lce_tokens.cu
  float* ztgt;           // [rows] logit of the label (TOK_STATS, TOK_EXP)
  const float* lse;      // [rows] (TOK_GRAD; the next four too), used without stats
  const float2* stats;   // [rows] (max z, log sum exp((z - max)/T)), or null
  const float* entropy;  // [rows]
  const float* g_logp;   // [rows] upstream gradients
  const float* g_entropy;  // [rows] or null
  const float* rowscale;   // [rows] what the row's gradient tile is divided by
  const float* label;      // [rows] the label's entry of the tile
  int* flags;
  int reset;             // the first block clears *flags (the call's first launch; k_score reports bad labels)
  DevStatus* clear_st;   // not null: the first block clears the status block and cnt[0, ncnt) (distillation)
  int* cnt;
  int ncnt;
  int no_loads;          // timeout test only: no operand is loaded, so the waits run out
  const float* ref;      // [rows] the labels' logits from before the GEMM (TOK_EXP; the next two too)
  float* sums;           // [rows, nparts] sums of the exp tile, the label's column left out
  int* guard;            // set to 1 where a sum of a row with a given token is not below kExpGuard, or ref is further
                         // than kExpShift T from ztgt
  const int* only_if;    // not null: the launch does nothing unless *only_if != 0 (TOK_STATS, TOK_GRAD)
};

// An exp tile is used while its half tiles' sums stay below this: entries and sums are then finite, and what
// they are scaled by, 1 / (1 + their sum), is a normal number.
constexpr float kExpGuard = 1.0e26f;
// Nats by which the label's logit from before the GEMM may differ from the GEMM's own: the tile is against the one, the
// row's results against the other (a factor of e^8 leaves the sums finite). Only the coldest temperatures come near.
constexpr float kExpShift = 8.f;

struct TokScoreArgs {
  int rows, V, nparts, K;
  long long ldz;
  float inv_t;
  long long ignore_index;
  const int64_t* y;
  const float4* partials;
  const float* ztgt;     // Z null: the label logits
  const float* Z;        // [rows, ldz] fp32 logits, or null (K == 0)
  float* logp;           // [rows] or null, as the next three
  float* lse;            // [rows]
  float* entropy;        // [rows]
  float2* stats;         // [rows] (max z, log sum exp((z - max)/T))
  float* top_logp;       // [rows, K]
  int64_t* top_idx;      // [rows, K]
  int* flags;
};

struct ScoreGradArgs {
  int V, d;
  long long ldz, ldg;
  float inv_t;
  long long ignore_index;
  const int64_t* y;      // [rows], as the next six
  const float* logp;
  const float* lse;
  const float2* stats;     // or null: lse
  const float* entropy;
  const float* g_logp;
  const float* g_entropy;  // or null
  float* rowscale;         // [rows] out
  float* label;            // [rows] out: the label's entry of the tile
  const uint4* H;          // [rows, d] bf16
  uint4* Ht;               // [rows, d] bf16(rowscale H) out, or null
  const float* Z;        // [rows, ldz] logits of the forward, or null: no gradient tile
  __nv_bfloat16* G;      // [rows, ldg]
  // first chunk only (st not null): the status block for N labels y_all and upstream factors of
  // one, and the dH part counters cnt[0, ncnt) cleared
  DevStatus* st;
  int keep_flags;          // 1: an earlier launch of the call cleared the status bits and may have set some
  const int64_t* y_all;
  long long N;
  int* cnt;
  int ncnt;
};

struct DistillArgs {
  int V, K, nparts;
  int renormalize, mean, t_bf16;
  int count_here;        // one chunk: the rows themselves count the kept ones, and the last sets the scales
  long long ldz, ldg;
  float inv_t;
  long long ignore_index, n_override;
  const int64_t* idx;    // [rows, K] teacher entries of this chunk
  const void* t;         // [rows, K] their values, fp32 or bf16
  const float4* partials;
  const float* Z;        // [rows, ldz]
  __nv_bfloat16* G;      // [rows, ldg] gradient tile, or null (loss only)
  const uint4* H;        // [rows, d] bf16
  uint4* Ht;             // [rows, d] H with zeros in the rows that keep no entry, out, or null (no dW)
  int d;
  float* row_loss;       // [rows]
  const float* grad_loss;
  const float* all_rows;  // [N] row_loss of the whole call; the row finished last sums it into loss
  long long N;
  float* loss;
  DevStatus* st;
};

// Logits GEMM z [M, N] = A [M, K] B [N, K]^T with a token epilogue; c: store
// map of the logits (TOK_STATS_Z) or the gradient tile (TOK_GRAD).
cudaError_t launch_tok_logits(int mode, const CUtensorMap& a, const CUtensorMap& b, const CUtensorMap& c, long long M,
                              long long N, long long K, const TokParams& ep, int num_sms, cudaStream_t s);
// The same for at most kFewRows rows (ep.rows), by one pass over W (lce_tokens.cu); h: map of H with
// boxes of few_rows_box(rows) rows, w: K-major map of W; store_z: the logits too, else the label's.
constexpr int kFewRows = 96;
inline uint32_t few_rows_box(long long rows) { return static_cast<uint32_t>((rows + 31) / 32 * 32); }
cudaError_t launch_rows_logits(const CUtensorMap& h, const CUtensorMap& w, int store_z, float* Z, long long ldz,
                               long long V, long long d, const TokParams& ep, int num_sms, cudaStream_t s);
cudaError_t launch_score(const TokScoreArgs& p, cudaStream_t s);
// Per row: rowscale and Ht, and with Z the gradient tile too.
cudaError_t launch_score_grad(const ScoreGradArgs& p, int rows, cudaStream_t s);
// Clears the status block and cnt[0, ncnt), then counts the rows of idx [N, K] that keep an entry.
cudaError_t launch_distill_count(const int64_t* idx, const void* t, int t_bf16, long long N, int K, int V,
                                 long long ignore_index, DevStatus* st, int* cnt, int ncnt, int num_sms,
                                 cudaStream_t s);
cudaError_t launch_distill_row(const DistillArgs& p, int rows, cudaStream_t s);

// ----------------------------------------------------------------------------
// Losses on log-probabilities (lce_losses.cu)
// ----------------------------------------------------------------------------
// Rows of a chunk of the policy and preference losses: from the logits' partial
// sums (or the statistics found from them) to the row's factor a = dloss/dlogp
// over T, its scale, its row of dW's second operand and of the gradient tile.
struct LossRowArgs {
  int V, d, nparts;
  long long ldz, ldg;
  float inv_t;
  long long ignore_index;
  const int64_t* y;        // [rows] labels of this chunk
  const float4* partials;  // [rows, nparts]
  const float* ztgt;       // Z null: the label logits of the GEMM
  const float* Z;          // [rows, ldz] fp32 logits, or null: no gradient tile here
  __nv_bfloat16* G;        // [rows, ldg]
  const uint4* H;          // [rows, d] bf16
  uint4* Ht;               // [rows, d] bf16(scale H) out, or null (no dW)
  float* logp;             // [rows]: out (policy), in (preference)
  float2* stats;           // [rows] (max z, log sum exp((z - max)/T)): out (policy, or null), in (preference)
  float* rowscale;         // [rows] out, or null: no gradient (policy)
  float* label;            // [rows] out: the label's entry of the tile
  float* a;                // [rows] out: the upstream factor that a gradient epilogue reads, or null
  DevStatus* st;
  // from the exp tile (sums not null): used where *guard == 0, else the row comes from partials and ztgt
  const float* sums;       // [rows, nparts]
  const int* guard;
  const float* ref;        // [rows] the label logits that the tile's entries are against
  float* rest;             // [rows] sum of the row's entries but the label's: out, then in (preference)
};

struct PolicyArgs {
  LossRowArgs row;
  const float* advantages;  // [rows], as the next four
  const float* old_logp;    // or null: the ratio is 1
  const float* ref_logp;    // or null: no KL term
  const float* weights;     // or null: 1
  float* row_loss;          // [rows] out
  double* row64;            // [rows] out: the same, summed into the loss
  const double* all_rows;   // [N] of the whole call
  float clip_low, clip_high, dual_clip, kl_coef;
  int kl;
  // one chunk (loss not null): the row finished last counts the tokens, sums the rows' losses and sets the scales
  float* loss;
  const float* grad_loss;
  int mean;
  long long n_override;
  long long N;
};

// The pairs of the preference loss: sequences' log-probabilities, the pairs' losses and the factor of
// each sequence's tokens (without 1/n).
struct PairArgs {
  const void* cu;          // [2 P + 1] sequence bounds, int64 or int32
  int cu32;
  long long P, N;
  int V;
  long long ignore_index;
  const int64_t* y;        // [N]
  const float* logp;       // [N]
  const float* ref;        // [2 P] or null
  float beta, margin, smoothing;
  int kind, average;
  float* pair_loss;        // [P]
  float* seq_logp;         // [2 P]
  float* coef;             // [2 P]
  float* loss;
  const float* grad_loss;
  double weight;           // 1/n, or 1 for a sum
  DevStatus* st;
};

struct PreferenceArgs {
  LossRowArgs row;
  long long c0;            // first row of the chunk
  const void* cu;
  int cu32;
  long long P;
  const float* coef;       // [2 P]
};

// What the first launch of a call by exp tiles clears (st null: nothing).
struct LossClear {
  DevStatus* st;
  int* guards;
  int nguards;
  int* cnt;
  int ncnt;
};
// The labels' logits z_{i,y_i} of N rows (0 where none is given).
cudaError_t launch_label_logits(const void* H, const void* W, const int64_t* y, long long N, int d, int V,
                                long long ignore_index, float* z, const LossClear& clear, cudaStream_t s);
cudaError_t launch_policy_row(const PolicyArgs& p, int rows, cudaStream_t s);
cudaError_t launch_policy_total(const double* rows, long long N, const DevStatus* st, float* loss, cudaStream_t s);
cudaError_t launch_pairs(const PairArgs& p, cudaStream_t s);
// Preference loss: logp and stats (or, by an exp tile, rest) of rows; with_pairs: those of a whole call, whose pairs, at
// most kPairsHere, are done in the same launch.
constexpr int kPairsHere = 4;
cudaError_t launch_logp_rows(const LossRowArgs& p, const PairArgs& q, bool with_pairs, int rows, cudaStream_t s);
cudaError_t launch_preference_row(const PreferenceArgs& p, int rows, cudaStream_t s);

// GEMM tile geometry (must match the kernels): each CTA of a pair loads 128
// rows of a K-major operand per box and 64 rows of an MN-major one.
constexpr int kBoxRowsK = 128;
constexpr int kBoxRowsMN = 64;
constexpr int kTileN = 256;   // vocabulary tile of the logits GEMM (partials: two per tile)

}  // namespace lce
