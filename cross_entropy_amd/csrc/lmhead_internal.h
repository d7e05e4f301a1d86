// lmhead_internal.h -- launch descriptors shared by the C ABI (lmhead_api.hip)
// and the kernels (lmhead_kernels.hip, lmhead_distill.hip, lmhead_few.hip,
// lmhead_norm.hip).
// Not part of the public interface.
#pragma once

#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

namespace lmh {

constexpr int kTileRows = 256;   // output tile edge of every MMA kernel
constexpr int kNumCUs = 256;     // MI355X: 8 XCDs x 32 CUs

// Forward: token tiles x vocabulary splits of the tile kernel, then the merge.
struct FwdPlan {
  int n_tt = 0;          // token tiles of 256
  int n_vt = 0;          // vocabulary tiles of 256
  int S = 0;             // vocabulary splits (partials per token)
  int64_t part_ld = 0;   // tokens per split row of the partials array
  size_t bytes = 0;      // workspace bytes (partials)
};

// Row stride (elements) for a bf16 operand of the backward GEMMs holding rows
// of at least x elements: a multiple of 64 elements (128 bytes) whose
// quotient by 64 is odd. 256-row tiles of rows strided by a large power of
// two crowd onto few memory channels (measured: such tiles run ~20% slower).
inline int64_t spread_ld(int64_t x) { return (((x + 63) / 64) | 1) * 64; }

// Backward: the token x vocabulary plane is cut into blocks of at most
// Ct x Vb; each block's cotangent is one bf16 buffer dz [Ct][ld_dz], double
// buffered (4 bytes per element in all, like one float32 block, the stride
// padding included). The workspace also holds hidden^T [H_pad][ld_ht]
// (masked tokens zeroed) and W's last V % 64 rows zero-padded to 64 rows
// [64][H] (the dh GEMM's last vocabulary slice).
struct BwdPlan {
  int64_t Ct = 0, Vb = 0;      // block edges (tokens, vocabulary), multiples of 256
  int64_t n_tb = 0, n_vb = 0;  // blocks along tokens and vocabulary
  int64_t N_pad = 0, V_pad = 0, H_pad = 0;
  int64_t ld_dz = 0, ld_ht = 0;                   // row strides (spread_ld)
  size_t off_dz1 = 0, off_ht = 0, off_tail = 0;   // byte offsets in the workspace
  size_t off_ctr = 0;          // 8 int32 cotangent-tile counters per launch (n_tb * n_vb + 1 launches)
  size_t bytes = 0;            // total
  // bf16-gradient backward: float32 accumulators of the gradients across
  // blocks. With vocab_outer (N <= V) the blocks run vocabulary-major: dh
  // accumulates in acc_dh [N_pad][H] over the whole call and each vocabulary
  // block's dW in acc_dW [Vb][H]; otherwise token-major: dW in acc_dW
  // [V_pad][H] over the call and each token block's dh in acc_dh [Ct][H].
  bool vocab_outer = false;
  size_t off_acc_dh = 0, off_acc_dW = 0;
  size_t bytes_bf16 = 0;       // total with the accumulators
};

FwdPlan plan_forward(int64_t N, int64_t H, int64_t V, int most_splits = 128);
BwdPlan plan_backward(int64_t N, int64_t H, int64_t V, int64_t chunk_size);

struct FwdArgs {
  const uint16_t* hidden;
  const uint16_t* W;
  const int32_t* targets;
  int64_t N, H, V;
  int S, n_tt, n_vt;
  int64_t voff;   // global id of W's first row (vocabulary shard), 0 for the whole table
  int64_t Vtot;   // valid target ids are [0, Vtot)
  float sc;       // log2(e) / T
  float invT;     // 1 / T
  void* part;
  int64_t part_ld;
  float* logp;
  float* entropy;
  float* lse;
  float* rec;     // shard partial records [N][4] instead of logp/entropy/lse, or NULL
};

// Where a gradient tile of the bf16-gradient backward reads and writes.
enum SrcKind { kSrcNone = 0, kSrcF32 = 1, kSrcBf16 = 2 };
struct GradOut {
  const void* src = nullptr;
  int src_kind = kSrcNone;
  void* dst = nullptr;
  int dst_bf16 = 0;
};

// One backward launch: the gradient tiles of one block (n_dw + n_dh tiles,
// none if 0) and the cotangent tiles of the next (z_ntt * z_nvt, none if 0).
struct BwdStep {
  const uint16_t* hidden;
  const uint16_t* W;
  const int32_t* targets;
  int N, H, V;     // V: rows of W (the shard's vocabulary)
  int voff, Vtot;  // global id of W's first row; valid target ids are [0, Vtot)
  const float* lse;
  const float* entropy;
  const float* g_logp;
  const float* g_ent;
  float sc;     // log2(e) / T
  float invT;   // 1 / T
  const uint16_t* ht;   // hidden^T [H_pad][N_pad], masked tokens zeroed
  int64_t ld_ht;
  const uint16_t* W_tail;   // W rows v_tail .. V-1 padded with zero rows to 64, or NULL if V % 64 == 0
  int v_tail;               // V rounded down to a multiple of 64
  float* dh;
  float* dW;
  int64_t ld_dz;        // row stride of both dz buffers
  // gradient part
  const uint16_t* g_dz;
  int g_t0, g_Ct, g_v0, g_Vb, g_acc_dh, g_acc_dW;
  int n_dw, n_dh, n_ht;
  // cotangent part
  uint16_t* z_dz;
  int* z_ctr;   // this launch's 8 per-XCD tile counters (zero before the launch)
  int z_t0, z_Ct, z_v0, z_Vb, z_ntt, z_nvt;
  // bf16-gradient backward only (bwd_step_bf16_kernel): per gradient, where
  // this block's tiles read the values they add to (none, a float32
  // accumulator or the caller's bf16 gradient) and where they write the sum
  // (a float32 accumulator, or the caller's bf16 gradient, rounded once),
  // both pointing at the block's first row (row stride H). Masked tokens'
  // dh rows are stored as 0 when dh_dead_zero, else left as they are.
  GradOut o_dh, o_dW;
  int dh_dead_zero;
};

// Distillation (lmhead_distill.hip). K entries per token: ids [N][K], teacher
// logits [N][K] (float32 or bf16).
constexpr int kDistillMaxK = 1024;

struct DistillTopArgs {
  const uint16_t* hidden;
  const uint16_t* W;
  const int32_t* targets;     // or NULL
  const int32_t* ids;
  const void* teacher;
  bool t_f32;
  const float* teacher_lse;   // or NULL: softmax over the live entries
  int64_t N;
  int H, V, K;
  float T;
  float back_hi, back_lo;     // 1 / (sc T) in two words (sc = the base-2 scale of the records)
  const void* part;           // the forward's split records [S][part_ld][4]
  int64_t part_ld;
  int S;
  float* kl;
  float* logp;                // or NULL
  float* lse;
  float* logp_top;            // [N][K]
  int n_dot;                  // waves that take dot products (set by the launcher)
};

// What the backward forms per token before the tiles run: the combined
// log-prob cotangent ga and target id tgt that the tiles read, and K + 1
// special entries (id or -1, cotangent) that overwrite the tiles'.
struct DistillPrepArgs {
  const int32_t* targets;     // or NULL
  const int32_t* ids;
  const void* teacher;
  bool t_f32;
  const float* teacher_lse;
  int64_t N;
  int V, K;
  float T, invT;
  const float* logp;          // of the target; read where it is not among the ids
  const float* logp_top;
  const float* g_kl;          // or NULL
  const float* g_logp;        // or NULL
  int32_t* tgt;               // [N]
  float* ga;                  // [N]
  int32_t* ent_id;            // [N][K + 1]
  float* ent_val;             // [N][K + 1]
  // what the tiles need besides, in the same launch: n_ctr zeroed counters, and
  // W's last tail_rows rows with zero rows up to 64 (none if tail_rows is 0)
  int* ctr;
  int64_t n_ctr;
  const uint16_t* tail_in;
  uint16_t* tail_out;
  int tail_rows, H;
};

// A backward launch with its gradient tiles' K split: the dh tiles over the
// block's vocabulary, the dW tiles (w_splits > 1) over its tokens; or (part
// NULL, splits 1) neither.
struct DistillStep {
  BwdStep step;
  int splits, k_split;       // splits of the launch's dh tiles, of k_split vocabulary rows (a multiple of 64)
  float* part;               // [splits][g_Ct][H] float32
  int w_splits, w_k_split;   // splits of its dW tiles, of w_k_split tokens (a multiple of 64)
  float* w_part;             // [w_splits][g_Vb][H] float32
};

// Sum of the splits of one gradient's block of `rows` rows: part [splits][rows]
// [H] float32 (NULL: nothing to sum), to and from o.
struct SplitSum {
  const float* part;
  int splits, rows;
  GradOut o;
};

// What follows each launch: the special entries into the cotangent block that
// it formed (dz, or NULL), and the sums of its splits.
struct DistillPostArgs {
  const int32_t* ent_id;
  const float* ent_val;
  int K1;            // K + 1
  uint16_t* dz;
  int64_t ld_dz;
  int t0, Ct, v0, Vb;
  SplitSum dh, dW;
  int H, V;
  const int32_t* tgt;   // of dh's first row on
  int dead_zero;     // masked tokens' dh rows are written as 0, else left as they are
};

// The distillation for few tokens (lmhead_few.hip).
constexpr int kFewTokens = 256;

struct FewArgs {
  const uint16_t* hidden;
  const uint16_t* W;
  const int32_t* targets;   // forward: the hard targets or NULL; backward: what the preparation wrote
  int N, H, V;
  float sc, invT;           // log2(e) / T, 1 / T
  void* part;               // forward: split records [few_splits(V)][part_ld][4]
  int64_t part_ld;
  // backward
  const float* lse;
  const float* ga;
  const int32_t* ent_id;
  const float* ent_val;
  int K1;
  int padded;               // tokens rounded up to 32 or a multiple of 64
  uint16_t* dz_hi;          // [V][padded] each
  uint16_t* dz_lo;          // NULL above 64 tokens
  void* dW;
  bool add_dW;
  int tiles, splits, strips, dw_splits, dh_blocks;   // set by the launchers
  float* dh_part;           // [dh_splits][N][H]
  int dh_strips, dh_splits, dh_rows;
};

int few_splits(int64_t V);   // records per token of the forward
hipError_t launch_few_stats(FewArgs a, hipStream_t stream);
hipError_t launch_few_bwd(FewArgs a, bool bf16, hipStream_t stream);   // the cotangent, dW and the partials of dh

// The norm in front of the head (lmhead_norm.hip); rows of H elements.
constexpr int kNormMaxH = 16384;

struct NormFwdArgs {
  const void* x;
  const void* w;      // or NULL: ones
  const void* b;      // or NULL: zeros
  bool x_f32, y_f32, w_f32, rms;
  int64_t N;
  int H;
  float eps;
  void* y;
  float* mean;        // or NULL
  float* rstd;        // or NULL
};

struct NormBwdArgs {
  const void* x;
  const void* w;      // or NULL: ones
  const float* mean;  // not read for RMS
  const float* rstd;
  const void* dy;
  bool x_f32, y_f32, w_f32, rms;
  int64_t N;
  int H;
  void* dx;
  int row_blocks;     // workgroups that walk rows (norm_bwd_blocks)
  float* part;        // [row_blocks][2][H] partial sums of dw and db, or NULL: not wanted, or
  void* dw;           // these are summed in this launch (norm_by_columns), where not NULL
  void* db;
  bool g_f32, accumulate;
};

struct NormReduceArgs {
  const float* part;
  int blocks, H;
  bool g_f32, accumulate;
  void* dw;           // or NULL
  void* db;           // or NULL
};

int norm_bwd_blocks(int64_t N, int64_t H);   // workgroups (partial rows) of the norm's backward
bool norm_by_columns(int64_t N);             // whether dw and db are summed in its launch

// Kernel ids of the tracing facility (lmhead_trace.hip).
enum KernelId {
  kFwdStats = 0, kFwdMerge, kBwdStep, kTranspose, kFill, kPadRows, kBwdStepBf16,
  kDistillTop, kDistillPrep, kDistillStep, kDistillPost,
  kFewStats, kFewDz, kFewGrads, kNormFwd, kNormBwd, kNormReduce, kNumKernels
};
void trace_begin(hipStream_t stream);
void trace_end(int kernel, hipStream_t stream, double flops, double bytes);

hipError_t launch_fwd_stats(const FwdArgs& a, hipStream_t stream);   // the split records alone
hipError_t launch_fwd(const FwdArgs& a, hipStream_t stream);
// merge of P shard records [P][N] (float4 each) into logp / entropy / lse
hipError_t launch_merge(const float* partials, int P, int64_t N, const int32_t* targets, int64_t Vtot,
                        float invT, float* logp, float* entropy, float* lse, hipStream_t stream);
hipError_t launch_bwd_step(const BwdStep& st, hipStream_t stream);
hipError_t launch_bwd_step_bf16(const BwdStep& st, hipStream_t stream);
hipError_t launch_fill_zero(float* p, int64_t n, hipStream_t stream);
hipError_t launch_pad_rows(const uint16_t* in, int64_t R, int64_t C, int64_t R_pad, uint16_t* out,
                           hipStream_t stream);
hipError_t launch_transpose(const uint16_t* in, int64_t ld_in, int64_t R, int64_t C, int64_t R_pad,
                            int64_t C_pad, const int32_t* tgt, int64_t V, uint16_t* out,
                            int64_t ld_out, hipStream_t stream);
hipError_t launch_distill_top(DistillTopArgs a, hipStream_t stream);
hipError_t launch_distill_prep(const DistillPrepArgs& a, hipStream_t stream);
hipError_t launch_distill_step(const DistillStep& d, bool bf16, hipStream_t stream);
hipError_t launch_distill_post(const DistillPostArgs& a, hipStream_t stream);
hipError_t launch_norm_fwd(const NormFwdArgs& a, hipStream_t stream);
hipError_t launch_norm_bwd(const NormBwdArgs& a, hipStream_t stream);
hipError_t launch_norm_reduce(const NormReduceArgs& a, hipStream_t stream);

}  // namespace lmh
