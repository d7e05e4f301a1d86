// lmhead_api.hip -- the C ABI declared in include/lmhead_logps.h: argument
// checks, work planning and launches on the caller's stream.
//
// Planning follows the chunked head of the pages (SkyRL issue "[tx] support
// long sequence", "4. Chunked LM Head"; google/tunix pull request #2876,
// the chunk loop over flattened tokens):
//  * The forward holds no [tokens, vocab] transient. It runs one tile kernel
//    over all tokens, with the vocabulary cut into S splits so that the
//    launch fills the 256 CUs; S partial (max, exp-sum, exp-weighted sum,
//    target logit) records per token are merged by log-sum-exp.
//  * The backward holds the logits' cotangent as bf16 blocks of Ct tokens x
//    Vb vocabulary entries, double buffered so that the cotangent of the next
//    block is formed while the gradient GEMMs of the current one run (one
//    launch per block). chunk_size bounds the block: the two buffers, 4 bytes
//    per element, stay within one float32 [chunk_size, V] tensor, the
//    transient the pages' chunked head holds per chunk. Within that bound the
//    block shape is chosen to cut the dh / dW accumulation traffic and launch
//    count. The workspace also holds a bf16 transpose of the hidden states
//    (input-sized; the dW GEMM's K-contiguous operand) and W's last V % 64
//    rows padded to 64 (the dh GEMM reads W as it lies, 64 rows at a time).
#include <hip/hip_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstdarg>
#include <cstdio>
#include <cstring>
#include <mutex>
#include <string>

#include "../../include/lmhead_logps.h"
#include "lmhead_internal.h"

namespace lmh {

static int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }
static int64_t round_up(int64_t a, int64_t b) { return ceil_div(a, b) * b; }

FwdPlan plan_forward(int64_t N, int64_t H, int64_t V, int most_splits) {
  (void)H;
  FwdPlan p;
  p.n_tt = (int)lmh::ceil_div(N, kTileRows);
  p.n_vt = (int)lmh::ceil_div(V, kTileRows);
  const int s_max = (int)std::min<int64_t>(p.n_vt, most_splits);
  // makespan in tile-steps: rounds of resident workgroups x tiles per split
  auto cost = [&](int S) {
    return ceil_div((int64_t)p.n_tt * S, kNumCUs) * ceil_div(p.n_vt, S);
  };
  int64_t best = INT64_MAX;
  for (int S = 1; S <= s_max; ++S) best = std::min(best, cost(S));
  // among near-best split counts, prefer S near 6: an XCD's 32 concurrent
  // workgroups then cover ~5 token tiles x 6 vocabulary tiles, which share
  // the W and hidden tiles in its L2 about evenly (measured at N = 65536,
  // V = 151936: S = 5 or 6 beat 8 by 2%, 3 and 9 match 8, 2 and 16 lose 3%)
  int pick = 1;
  double pick_dist = 1e30;
  for (int S = 1; S <= s_max; ++S) {
    if ((double)cost(S) > 1.03 * (double)best) continue;
    const double dist = std::fabs(std::log2((double)S / 6.0));
    if (dist < pick_dist) {
      pick_dist = dist;
      pick = S;
    }
  }
  p.S = std::max(1, pick);
  p.part_ld = round_up(std::max<int64_t>(N, 1), 64);
  p.bytes = (size_t)round_up((int64_t)p.S * p.part_ld * 16, 256);
  return p;
}

BwdPlan plan_backward(int64_t N, int64_t H, int64_t V, int64_t chunk_size) {
  const int64_t T = kTileRows;
  N = std::max<int64_t>(N, 1);
  // elements of one dz buffer, stride padding included (two bf16 buffers, 4
  // bytes per element in all): at most chunk_size * V, and at least one
  // 256 x 256 tile.
  const double budget = std::max<double>((double)chunk_size * (double)V, (double)(T * spread_ld(T)));
  const int64_t n_pad = round_up(N, T);
  const int64_t v_pad = round_up(V, T);
  // model: the MFMA work is fixed; what the block shape changes is the f32
  // accumulation traffic of dh (one pass per vocabulary block) and dW (one
  // pass per token block), and the number of launches.
  const double hbm = 5.0e12;
  const double launch = 20e-6;
  BwdPlan best;
  double best_t = 1e300;
  for (int64_t ct = T; ct <= n_pad; ct += T) {
    // spread_ld(vb) = vb + 64 for vb a multiple of 256
    int64_t vb = ((int64_t)(budget / (double)ct) - 64) / T * T;
    vb = std::min(vb, v_pad);
    if (vb < T) break;
    const int64_t n_tb = ceil_div(N, ct);
    const int64_t n_vb = ceil_div(V, vb);
    const int64_t c2 = round_up(ceil_div(N, n_tb), T);   // even out the blocks
    const int64_t v2 = round_up(ceil_div(V, n_vb), T);
    const double traffic = (8.0 * N * H * n_vb + 8.0 * V * H * n_tb) / hbm;
    const double t = (double)(n_tb * n_vb + 1) * launch + traffic;
    if (t < best_t) {
      best_t = t;
      best.Ct = c2;
      best.Vb = v2;
      best.n_tb = n_tb;
      best.n_vb = n_vb;
    }
  }
  best.N_pad = round_up(N, T);
  best.V_pad = round_up(V, T);
  best.H_pad = round_up(H, T);
  best.ld_dz = spread_ld(best.Vb);
  best.ld_ht = spread_ld(best.N_pad);
  const size_t one = (size_t)round_up(best.Ct * best.ld_dz * 2, 256);
  best.off_dz1 = one;
  best.off_ht = 2 * one;
  best.off_tail = best.off_ht + (size_t)round_up(best.H_pad * best.ld_ht * 2, 256);
  best.off_ctr = best.off_tail + (size_t)round_up(64 * H * 2, 256);
  best.bytes = best.off_ctr + (size_t)round_up((best.n_tb * best.n_vb + 1) * 8 * 4, 256);
  // the bf16-gradient backward keeps the larger gradient per block and the
  // smaller one whole in float32
  best.vocab_outer = N <= V;
  const int64_t whole = best.vocab_outer ? best.N_pad : best.V_pad;
  const int64_t part = best.vocab_outer ? best.Vb : best.Ct;
  const size_t acc_whole = (size_t)round_up(whole * H * 4, 256);
  const size_t acc_part = (size_t)round_up(part * H * 4, 256);
  best.off_acc_dh = best.bytes;
  best.off_acc_dW = best.bytes + (best.vocab_outer ? acc_whole : acc_part);
  best.bytes_bf16 = best.bytes + acc_whole + acc_part;
  return best;
}

}  // namespace lmh

namespace {

thread_local std::string g_last_error;

int fail(int code, const char* fmt, ...) __attribute__((format(printf, 2, 3)));
int fail(int code, const char* fmt, ...) {
  char buf[512];
  va_list ap;
  va_start(ap, fmt);
  vsnprintf(buf, sizeof buf, fmt, ap);
  va_end(ap);
  g_last_error = buf;
  return code;
}

int ok() {
  g_last_error.clear();
  return LMH_OK;
}

int check_shape(int64_t N, int64_t H, int64_t V, int64_t chunk_size) {
  if (N < 0 || N >= (int64_t(1) << 31))
    return fail(LMH_ERR_SHAPE, "N must be in [0, 2^31), got %lld", (long long)N);
  if (H <= 0 || H >= (int64_t(1) << 20))
    return fail(LMH_ERR_SHAPE, "H must be in (0, 2^20), got %lld", (long long)H);
  if (V <= 0 || V >= (int64_t(1) << 31))
    return fail(LMH_ERR_SHAPE, "V must be in (0, 2^31), got %lld", (long long)V);
  if (chunk_size <= 0) return fail(LMH_ERR_CHUNK, "chunk_size must be > 0, got %lld", (long long)chunk_size);
  if (H % 64 != 0) return fail(LMH_ERR_UNSUPPORTED, "H must be a multiple of 64, got %lld", (long long)H);
  return LMH_OK;
}

// The backward's GEMMs read 256-row tiles of the cotangent block and of the
// transposed hidden states (row strides up to V_pad and N_pad elements)
// through 32-bit byte offsets from the tile's base: 256 * stride * 2 bytes
// must stay below 2^32.
int check_backward_size(int64_t N, int64_t V) {
  const int64_t lim = int64_t(1) << 23;
  if (lmh::round_up(std::max<int64_t>(N, 1), lmh::kTileRows) >= lim || lmh::round_up(V, lmh::kTileRows) >= lim)
    return fail(LMH_ERR_UNSUPPORTED, "bwd: N (%lld) and V (%lld) rounded up to 256 must stay below 2^23",
                (long long)N, (long long)V);
  return LMH_OK;
}

bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

// Base-2 scale of the tempered logits and the reciprocal temperature; at
// T = 1 these are log2(e) and 1 exactly, so the untempered entry points give
// the same bits as the tempered ones at T = 1.
float temper_scale(float temperature) { return (float)(1.4426950408889634 / (double)temperature); }
float inv_temperature(float temperature) { return (float)(1.0 / (double)temperature); }

int check_temperature(float temperature) {
  if (!(std::isfinite(temperature) && temperature > 0.0f))
    return fail(LMH_ERR_ARGS, "temperature must be finite and > 0, got %g", (double)temperature);
  if (!std::isfinite(temper_scale(temperature)) || !std::isfinite(inv_temperature(temperature)))
    return fail(LMH_ERR_ARGS, "temperature %g is too small: 1 / temperature overflows float32",
                (double)temperature);
  return LMH_OK;
}

}  // namespace

extern "C" {

const char* lmhead_logps_last_error(void) { return g_last_error.c_str(); }

const char* lmhead_logps_version(void) { return "lmhead_logps 0.1.0 (gfx950)"; }

int lmhead_logps_workspace_bytes(int64_t N, int64_t H, int64_t V, int64_t chunk_size,
                                 int with_backward, size_t* bytes_out) {
  if (bytes_out == nullptr) return fail(LMH_ERR_NULL, "bytes_out is NULL");
  const int rc = check_shape(N, H, V, chunk_size);
  if (rc != LMH_OK) return rc;
  if (with_backward) {
    const int rb = check_backward_size(N, V);
    if (rb != LMH_OK) return rb;
  }
  if (with_backward < 0 || with_backward > LMH_WS_BWD_BF16)
    return fail(LMH_ERR_ARGS, "with_backward must be 0, 1 or 2, got %d", with_backward);
  size_t b = lmh::plan_forward(N, H, V).bytes;
  if (with_backward) {
    const lmh::BwdPlan p = lmh::plan_backward(N, H, V, chunk_size);
    b = std::max(b, with_backward == LMH_WS_BWD_BF16 ? p.bytes_bf16 : p.bytes);
  }
  *bytes_out = b;
  return ok();
}

}  // extern "C"

namespace {

// Shard ranges: W holds rows [voff, voff + V) of a vocabulary of Vtot ids.
int check_shard(int64_t V, int64_t voff, int64_t Vtot) {
  if (voff < 0 || Vtot <= 0 || Vtot >= (int64_t(1) << 31) || voff > Vtot - V)
    return fail(LMH_ERR_SHAPE, "shard rows [%lld, %lld) must lie in a vocabulary [0, %lld) with 0 < %lld < 2^31",
                (long long)voff, (long long)(voff + V), (long long)Vtot, (long long)Vtot);
  return LMH_OK;
}

// The forward of W's rows [voff, voff + V); writes logp/entropy/lse, or with
// `rec` the merged partial record of this vocabulary range.
int fwd_impl(const char* who, const uint16_t* hidden, const uint16_t* W, const int32_t* targets,
             int64_t N, int64_t H, int64_t V, int64_t voff, int64_t Vtot, int64_t chunk_size,
             float temperature, float* logp, float* entropy, float* lse, float* rec,
             void* workspace, size_t workspace_bytes, void* stream) {
  int rc = check_shape(N, H, V, chunk_size);
  if (rc != LMH_OK) return rc;
  rc = check_shard(V, voff, Vtot);
  if (rc != LMH_OK) return rc;
  rc = check_temperature(temperature);
  if (rc != LMH_OK) return rc;
  if (N == 0) return ok();
  if (rec == nullptr) {
    if (!hidden || !W || !targets || !logp || !lse || !workspace)
      return fail(LMH_ERR_NULL, "%s: hidden, W, targets, logp, lse and workspace must be non-NULL", who);
    if (!aligned(hidden, 16) || !aligned(W, 16) || !aligned(workspace, 16) || !aligned(targets, 4) ||
        !aligned(logp, 4) || !aligned(lse, 4) || (entropy && !aligned(entropy, 4)))
      return fail(LMH_ERR_UNSUPPORTED, "%s: hidden, W and workspace need 16-byte alignment", who);
  } else {
    if (!hidden || !W || !targets || !workspace)
      return fail(LMH_ERR_NULL, "%s: hidden, W, targets, partial and workspace must be non-NULL", who);
    if (!aligned(hidden, 16) || !aligned(W, 16) || !aligned(workspace, 16) || !aligned(targets, 4) ||
        !aligned(rec, 16))
      return fail(LMH_ERR_UNSUPPORTED, "%s: hidden, W, partial and workspace need 16-byte alignment", who);
  }
  const lmh::FwdPlan p = lmh::plan_forward(N, H, V);
  if (workspace_bytes < p.bytes)
    return fail(LMH_ERR_WORKSPACE, "%s: workspace of %zu bytes, %zu needed", who, workspace_bytes, p.bytes);
  lmh::FwdArgs a{hidden, W, targets, N, H, V, p.S, p.n_tt, p.n_vt, voff, Vtot,
                 temper_scale(temperature), inv_temperature(temperature), workspace, p.part_ld,
                 logp, entropy, lse, rec};
  const hipError_t e = lmh::launch_fwd(a, static_cast<hipStream_t>(stream));
  if (e != hipSuccess) return fail(LMH_ERR_HIP, "%s: launch failed: %s", who, hipGetErrorString(e));
  return ok();
}

}  // namespace

extern "C" {

int lmhead_logps_fwd_temp(const uint16_t* hidden, const uint16_t* W, const int32_t* targets,
                          int64_t N, int64_t H, int64_t V, int64_t chunk_size, float temperature,
                          float* logp, float* entropy, float* lse, void* workspace,
                          size_t workspace_bytes, void* stream) {
  return fwd_impl("fwd", hidden, W, targets, N, H, V, 0, V, chunk_size, temperature, logp, entropy, lse,
                  nullptr, workspace, workspace_bytes, stream);
}

int lmhead_logps_fwd_shard(const uint16_t* hidden, const uint16_t* W_shard, const int32_t* targets,
                           int64_t N, int64_t H, int64_t V_shard, int64_t vocab_offset, int64_t V_total,
                           int64_t chunk_size, float temperature, float* partial, void* workspace,
                           size_t workspace_bytes, void* stream) {
  if (partial == nullptr && N > 0) return fail(LMH_ERR_NULL, "fwd_shard: partial must be non-NULL");
  return fwd_impl("fwd_shard", hidden, W_shard, targets, N, H, V_shard, vocab_offset, V_total, chunk_size,
                  temperature, nullptr, nullptr, nullptr, partial, workspace, workspace_bytes, stream);
}

int lmhead_logps_merge_shards(const float* partials, int64_t P, const int32_t* targets, int64_t N,
                              int64_t V_total, float temperature, float* logp, float* entropy,
                              float* lse, void* stream) {
  if (N < 0 || N >= (int64_t(1) << 31))
    return fail(LMH_ERR_SHAPE, "merge_shards: N must be in [0, 2^31), got %lld", (long long)N);
  if (P <= 0 || P > 65536) return fail(LMH_ERR_SHAPE, "merge_shards: P must be in [1, 65536], got %lld", (long long)P);
  if (V_total <= 0 || V_total >= (int64_t(1) << 31))
    return fail(LMH_ERR_SHAPE, "merge_shards: V_total must be in (0, 2^31), got %lld", (long long)V_total);
  int rc = check_temperature(temperature);
  if (rc != LMH_OK) return rc;
  if (N == 0) return ok();
  if (!partials || !targets || !logp || !lse)
    return fail(LMH_ERR_NULL, "merge_shards: partials, targets, logp and lse must be non-NULL");
  if (!aligned(partials, 16) || !aligned(targets, 4) || !aligned(logp, 4) || !aligned(lse, 4) ||
      (entropy && !aligned(entropy, 4)))
    return fail(LMH_ERR_UNSUPPORTED, "merge_shards: partials need 16-byte alignment");
  const hipError_t e = lmh::launch_merge(partials, (int)P, N, targets, V_total, inv_temperature(temperature),
                                         logp, entropy, lse, static_cast<hipStream_t>(stream));
  if (e != hipSuccess) return fail(LMH_ERR_HIP, "merge_shards: launch failed: %s", hipGetErrorString(e));
  return ok();
}

}  // extern "C"

// Scratch of the allocation-free forward (lmhead_logps_fwd_noalloc): the
// vocabulary-split partial records, in a fixed device array that every GPU
// the library runs on holds until the process ends. Host code never passes
// the array's name to a kernel (on the host it only stands in for the
// symbol): it passes the device address hipGetSymbolAddress returns, looked
// up once per device.
static __device__ __align__(256) char scratch[LMH_NOALLOC_SCRATCH_BYTES];

namespace {

constexpr int kMaxDevices = 64;
std::mutex g_scratch_mu;
void* g_scratch_ptr[kMaxDevices] = {};

// The address of `scratch` on the device the work runs on: the stream's
// device (the current device for the NULL stream). Looked up once per device,
// with that device current; the caller's current device is restored.
int scratch_address(hipStream_t stream, void** out) {
  int cur = -1;
  hipError_t e = hipGetDevice(&cur);
  if (e != hipSuccess) return fail(LMH_ERR_HIP, "fwd_noalloc: hipGetDevice failed: %s", hipGetErrorString(e));
  int dev = cur;
  if (stream != nullptr) {
    hipDevice_t sd = 0;
    e = hipStreamGetDevice(stream, &sd);
    if (e != hipSuccess)
      return fail(LMH_ERR_HIP, "fwd_noalloc: hipStreamGetDevice failed: %s", hipGetErrorString(e));
    dev = (int)sd;
  }
  if (dev < 0 || dev >= kMaxDevices)
    return fail(LMH_ERR_UNSUPPORTED, "fwd_noalloc: device %d is beyond the %d the library tracks", dev, kMaxDevices);
  std::lock_guard<std::mutex> lock(g_scratch_mu);
  if (g_scratch_ptr[dev] == nullptr) {
    if (dev != cur && (e = hipSetDevice(dev)) != hipSuccess)
      return fail(LMH_ERR_HIP, "fwd_noalloc: hipSetDevice(%d) failed: %s", dev, hipGetErrorString(e));
    void* p = nullptr;
    e = hipGetSymbolAddress(&p, HIP_SYMBOL(scratch));
    const hipError_t back = dev != cur ? hipSetDevice(cur) : hipSuccess;
    if (e != hipSuccess || p == nullptr)
      return fail(LMH_ERR_HIP, "fwd_noalloc: hipGetSymbolAddress(scratch) failed on device %d: %s", dev,
                  hipGetErrorString(e));
    if (back != hipSuccess)
      return fail(LMH_ERR_HIP, "fwd_noalloc: restoring device %d failed: %s", cur, hipGetErrorString(back));
    g_scratch_ptr[dev] = p;
  }
  *out = g_scratch_ptr[dev];
  return LMH_OK;
}

}  // namespace

extern "C" {

int lmhead_logps_fwd_noalloc(const uint16_t* hidden, const uint16_t* W, const int32_t* targets, int64_t N,
                             int64_t H, int64_t V, int64_t chunk_size, float temperature, float* logp,
                             float* entropy, float* lse, void* stream) {
  int rc = check_shape(N, H, V, chunk_size);
  if (rc != LMH_OK) return rc;
  rc = check_temperature(temperature);
  if (rc != LMH_OK) return rc;
  if (N == 0) return ok();
  const size_t need = lmh::plan_forward(N, H, V).bytes;
  if (need > (size_t)LMH_NOALLOC_SCRATCH_BYTES)
    return fail(LMH_ERR_WORKSPACE,
                "fwd_noalloc: N = %lld needs %zu bytes of scratch, beyond the fixed %zu (use lmhead_logps_fwd_temp "
                "with a workspace)",
                (long long)N, need, (size_t)LMH_NOALLOC_SCRATCH_BYTES);
  void* ws = nullptr;
  rc = scratch_address(static_cast<hipStream_t>(stream), &ws);
  if (rc != LMH_OK) return rc;
  return fwd_impl("fwd_noalloc", hidden, W, targets, N, H, V, 0, V, chunk_size, temperature, logp, entropy, lse,
                  nullptr, ws, (size_t)LMH_NOALLOC_SCRATCH_BYTES, stream);
}

}  // extern "C"

namespace {

// The distillation's part of a backward: its per-token preparation, launched
// before everything else, the special entries that overwrite each cotangent
// block once it is formed, and (k_split > 0) its launches with split gradient
// tiles. `bytes` is the whole workspace it needs.
struct DistillHook {
  lmh::DistillPrepArgs prep;
  int k_split, w_k_split;   // vocabulary rows of a dh split; tokens of a dW split (0: dW is not split)
  float* part;
  float* w_part;
  size_t bytes;
};

// One launch of the distillation's backward (gradients of one block if `grads`,
// the next block's cotangent if `forms`) and what follows it.
hipError_t launch_distill_block(const DistillHook& h, const lmh::BwdStep& st, bool bf16, bool grads, bool forms,
                                const lmh::BwdPlan& p, hipStream_t s) {
  lmh::DistillPostArgs a{};
  if (forms) {
    a.ent_id = h.prep.ent_id;
    a.ent_val = h.prep.ent_val;
    a.K1 = h.prep.K + 1;
    a.dz = st.z_dz;
    a.ld_dz = p.ld_dz;
    a.t0 = st.z_t0;
    a.Ct = st.z_Ct;
    a.v0 = st.z_v0;
    a.Vb = st.z_Vb;
  }
  lmh::DistillStep d{st, 1, 0, nullptr, 1, 0, nullptr};
  if (h.k_split > 0) {
    // the block may be shorter than the plan's: as many splits as it fills
    auto count = [&](int k, int split) { return grads && split > 0 ? (int)lmh::ceil_div(lmh::round_up(k, 64), split) : 1; };
    d.splits = count(st.g_Vb, h.k_split);
    d.k_split = h.k_split;
    d.part = h.part;
    d.w_splits = count(st.g_Ct, h.w_k_split);
    d.w_k_split = d.w_splits > 1 ? h.w_k_split : st.g_Ct;
    d.w_part = h.w_part;
    if (grads) {
      a.H = st.H;
      a.V = st.Vtot;
      a.tgt = st.targets + st.g_t0;
      a.dh.part = d.part;
      a.dh.splits = d.splits;
      a.dh.rows = st.g_Ct;
      if (bf16) {
        a.dh.o = st.o_dh;
        a.dead_zero = st.dh_dead_zero;
      } else {
        a.dh.o.src_kind = st.g_acc_dh ? lmh::kSrcF32 : lmh::kSrcNone;
        a.dh.o.src = a.dh.o.dst = st.dh + (int64_t)st.g_t0 * st.H;
        a.dead_zero = !st.g_acc_dh;
      }
    }
    if (grads && d.w_splits > 1) {
      a.dW.part = d.w_part;
      a.dW.splits = d.w_splits;
      a.dW.rows = st.g_Vb;
      if (bf16) {
        a.dW.o = st.o_dW;
      } else {
        a.dW.o.src_kind = st.g_acc_dW ? lmh::kSrcF32 : lmh::kSrcNone;
        a.dW.o.src = a.dW.o.dst = st.dW + (int64_t)st.g_v0 * st.H;
      }
    }
  }
  const hipError_t e = lmh::launch_distill_step(d, bf16, s);
  return e == hipSuccess ? lmh::launch_distill_post(a, s) : e;
}

// The backward of W's rows [voff, voff + V) of a vocabulary of Vtot ids.
// dh / dW are float32 (bf16_out false) or bf16 gradients (bf16_out true).
// With `distill`, targets and g_logp are what its preparation writes.
int bwd_impl(const char* who, const uint16_t* hidden, const uint16_t* W, const int32_t* targets, int64_t N,
             int64_t H, int64_t V, int64_t voff, int64_t Vtot, int64_t chunk_size, float temperature,
             const float* lse, const float* entropy, const float* g_logp, const float* g_ent, void* dh,
             void* dW, unsigned flags, bool bf16_out, void* workspace, size_t workspace_bytes, void* stream,
             const DistillHook* distill = nullptr) {
  int rc = check_shape(N, H, V, chunk_size);
  if (rc != LMH_OK) return rc;
  rc = check_shard(V, voff, Vtot);
  if (rc != LMH_OK) return rc;
  rc = check_temperature(temperature);
  if (rc != LMH_OK) return rc;
  if (flags & ~(unsigned)(LMH_BWD_ACCUMULATE_DH | LMH_BWD_ACCUMULATE_DW))
    return fail(LMH_ERR_ARGS, "%s: unknown flags 0x%x", who, flags);
  const bool acc_dh = (flags & LMH_BWD_ACCUMULATE_DH) != 0;
  const bool acc_dW = (flags & LMH_BWD_ACCUMULATE_DW) != 0;
  if (g_ent != nullptr && entropy == nullptr)
    return fail(LMH_ERR_ARGS, "%s: g_ent given without the forward's entropy", who);
  if (!dW) return fail(LMH_ERR_NULL, "%s: dW must be non-NULL", who);
  if (!aligned(dW, bf16_out ? 16 : 4))
    return fail(LMH_ERR_UNSUPPORTED, "%s: dW needs %d-byte alignment", who, bf16_out ? 16 : 4);
  rc = check_backward_size(N, V);
  if (rc != LMH_OK) return rc;
  hipStream_t s = static_cast<hipStream_t>(stream);
  if (N == 0) {
    if (acc_dW) return ok();   // nothing to add
    // bf16 zeros are 32-bit zeros two at a time (V * H is even: H % 64 == 0)
    const hipError_t e = lmh::launch_fill_zero(static_cast<float*>(dW), bf16_out ? V * H / 2 : V * H, s);
    if (e != hipSuccess) return fail(LMH_ERR_HIP, "%s: launch failed: %s", who, hipGetErrorString(e));
    return ok();
  }
  if (!hidden || !W || !targets || !lse || !dh || !workspace)
    return fail(LMH_ERR_NULL, "%s: hidden, W, targets, lse, dh, dW and workspace must be non-NULL", who);
  if (!aligned(hidden, 16) || !aligned(W, 16) || !aligned(workspace, 16) || !aligned(dh, 16))
    return fail(LMH_ERR_UNSUPPORTED, "%s: hidden, W, dh and workspace need 16-byte alignment", who);
  const lmh::BwdPlan p = lmh::plan_backward(N, H, V, chunk_size);
  const size_t need = distill ? distill->bytes : bf16_out ? p.bytes_bf16 : p.bytes;
  if (workspace_bytes < need)
    return fail(LMH_ERR_WORKSPACE, "%s: workspace of %zu bytes, %zu needed", who, workspace_bytes, need);
  char* ws = static_cast<char*>(workspace);
  uint16_t* dzbuf[2] = {reinterpret_cast<uint16_t*>(ws), reinterpret_cast<uint16_t*>(ws + p.off_dz1)};
  uint16_t* ht = reinterpret_cast<uint16_t*>(ws + p.off_ht);
  uint16_t* W_tail = reinterpret_cast<uint16_t*>(ws + p.off_tail);
  int* ctr = reinterpret_cast<int*>(ws + p.off_ctr);
  float* acc_h = reinterpret_cast<float*>(ws + p.off_acc_dh);
  float* acc_w = reinterpret_cast<float*>(ws + p.off_acc_dW);
  const int64_t v_tail = V / 64 * 64;
  const int64_t nb = p.n_tb * p.n_vb;
  // the cotangent-tile counters start at zero (a fill kernel, not a memset:
  // the call may be captured into a graph)
  hipError_t te;
  if (distill) {
    lmh::DistillPrepArgs prep = distill->prep;
    prep.ctr = ctr;
    prep.n_ctr = (nb + 1) * 8;
    prep.tail_in = W + v_tail * H;
    prep.tail_out = W_tail;
    prep.tail_rows = (int)(V - v_tail);
    prep.H = (int)H;
    te = lmh::launch_distill_prep(prep, s);
  } else {
    te = lmh::launch_fill_zero(reinterpret_cast<float*>(ctr), (nb + 1) * 8, s);
  }
  if (te == hipSuccess)
    te = lmh::launch_transpose(hidden, H, N, H, p.N_pad, p.H_pad, targets, Vtot, ht, p.ld_ht, s);
  if (te == hipSuccess && v_tail < V && !distill) te = lmh::launch_pad_rows(W + v_tail * H, V - v_tail, H, 64, W_tail, s);
  if (te != hipSuccess) return fail(LMH_ERR_HIP, "%s: launch failed: %s", who, hipGetErrorString(te));

  lmh::BwdStep st{};
  st.hidden = hidden;
  st.W = W;
  st.targets = targets;
  st.N = (int)N;
  st.H = (int)H;
  st.V = (int)V;
  st.voff = (int)voff;
  st.Vtot = (int)Vtot;
  st.lse = lse;
  st.entropy = entropy;
  st.g_logp = g_logp;
  st.g_ent = g_ent;
  st.sc = temper_scale(temperature);
  st.invT = inv_temperature(temperature);
  st.ht = ht;
  st.ld_ht = p.ld_ht;
  st.W_tail = v_tail < V ? W_tail : nullptr;
  st.v_tail = (int)v_tail;
  st.dh = bf16_out ? nullptr : static_cast<float*>(dh);
  st.dW = bf16_out ? nullptr : static_cast<float*>(dW);
  st.ld_dz = p.ld_dz;
  st.n_ht = (int)lmh::ceil_div(H, lmh::kTileRows);
  // blocks in a fixed order: token blocks outer (vocabulary blocks inner),
  // except for bf16 gradients with N <= V, which run vocabulary blocks outer
  // so that each vocabulary block's dW is complete (and rounded) before the
  // next starts. Launch j forms block j's cotangent and runs block j-1's GEMMs.
  const bool vocab_major = bf16_out && p.vocab_outer;
  auto block_of = [&](int64_t j, int64_t& tb, int64_t& vb) {
    if (vocab_major) {
      vb = j / p.n_tb;
      tb = j % p.n_tb;
    } else {
      tb = j / p.n_vb;
      vb = j % p.n_vb;
    }
  };
  uint16_t* dh16 = static_cast<uint16_t*>(dh);
  uint16_t* dW16 = static_cast<uint16_t*>(dW);
  for (int64_t j = 0; j <= nb; ++j) {
    st.z_ctr = ctr + j * 8;
    if (j >= 1) {
      int64_t tb, vb;
      block_of(j - 1, tb, vb);
      st.g_dz = dzbuf[(j - 1) & 1];
      st.g_t0 = (int)(tb * p.Ct);
      st.g_Ct = (int)std::min(p.Ct, N - tb * p.Ct);
      st.g_v0 = (int)(vb * p.Vb);
      st.g_Vb = (int)std::min(p.Vb, V - vb * p.Vb);
      st.g_acc_dh = vb > 0 || acc_dh;
      st.g_acc_dW = tb > 0 || acc_dW;
      st.n_dw = (int)(lmh::ceil_div(st.g_Vb, lmh::kTileRows) * st.n_ht);
      st.n_dh = (int)(lmh::ceil_div(st.g_Ct, lmh::kTileRows) * st.n_ht);
      if (bf16_out) {
        // each gradient sums its blocks in order (dW over token blocks, dh
        // over vocabulary blocks) in a float32 accumulator; its first block
        // starts from nothing (or the caller's bf16 values when adding) and
        // its last writes the caller's bf16 gradient
        const int64_t t0 = tb * p.Ct, v0 = vb * p.Vb;
        uint16_t* w_out = dW16 + v0 * H;
        float* w_acc = p.vocab_outer ? acc_w : acc_w + v0 * H;
        st.o_dW.src_kind = tb == 0 ? (acc_dW ? lmh::kSrcBf16 : lmh::kSrcNone) : lmh::kSrcF32;
        st.o_dW.src = tb == 0 ? static_cast<const void*>(w_out) : static_cast<const void*>(w_acc);
        st.o_dW.dst_bf16 = tb == p.n_tb - 1;
        st.o_dW.dst = st.o_dW.dst_bf16 ? static_cast<void*>(w_out) : static_cast<void*>(w_acc);
        uint16_t* h_out = dh16 + t0 * H;
        float* h_acc = p.vocab_outer ? acc_h + t0 * H : acc_h;
        st.o_dh.src_kind = vb == 0 ? (acc_dh ? lmh::kSrcBf16 : lmh::kSrcNone) : lmh::kSrcF32;
        st.o_dh.src = vb == 0 ? static_cast<const void*>(h_out) : static_cast<const void*>(h_acc);
        st.o_dh.dst_bf16 = vb == p.n_vb - 1;
        st.o_dh.dst = st.o_dh.dst_bf16 ? static_cast<void*>(h_out) : static_cast<void*>(h_acc);
        st.dh_dead_zero = st.o_dh.dst_bf16 && !acc_dh;
      }
    } else {
      st.g_dz = nullptr;
      st.n_dw = st.n_dh = 0;
    }
    if (j < nb) {
      int64_t tb, vb;
      block_of(j, tb, vb);
      st.z_dz = dzbuf[j & 1];
      st.z_t0 = (int)(tb * p.Ct);
      st.z_Ct = (int)std::min(p.Ct, N - tb * p.Ct);
      st.z_v0 = (int)(vb * p.Vb);
      st.z_Vb = (int)std::min(p.Vb, V - vb * p.Vb);
      st.z_ntt = (int)lmh::ceil_div(st.z_Ct, lmh::kTileRows);
      st.z_nvt = (int)lmh::ceil_div(st.z_Vb, lmh::kTileRows);
    } else {
      st.z_dz = nullptr;
      st.z_ntt = st.z_nvt = 0;
    }
    hipError_t e;
    if (distill == nullptr) {
      e = bf16_out ? lmh::launch_bwd_step_bf16(st, s) : lmh::launch_bwd_step(st, s);
    } else {
      e = launch_distill_block(*distill, st, bf16_out, j >= 1, j < nb, p, s);
    }
    if (e != hipSuccess) return fail(LMH_ERR_HIP, "%s: launch failed: %s", who, hipGetErrorString(e));
  }
  return ok();
}

}  // namespace

extern "C" {

int lmhead_logps_bwd_ex(const uint16_t* hidden, const uint16_t* W, const int32_t* targets,
                        int64_t N, int64_t H, int64_t V, int64_t chunk_size, float temperature,
                        const float* lse, const float* entropy, const float* g_logp,
                        const float* g_ent, float* dh, float* dW, unsigned flags, void* workspace,
                        size_t workspace_bytes, void* stream) {
  return bwd_impl("bwd", hidden, W, targets, N, H, V, 0, V, chunk_size, temperature, lse, entropy, g_logp, g_ent,
                  dh, dW, flags, false, workspace, workspace_bytes, stream);
}

int lmhead_logps_bwd_bf16(const uint16_t* hidden, const uint16_t* W, const int32_t* targets, int64_t N,
                          int64_t H, int64_t V, int64_t chunk_size, float temperature, const float* lse,
                          const float* entropy, const float* g_logp, const float* g_ent, uint16_t* dh,
                          uint16_t* dW, unsigned flags, void* workspace, size_t workspace_bytes, void* stream) {
  return bwd_impl("bwd_bf16", hidden, W, targets, N, H, V, 0, V, chunk_size, temperature, lse, entropy, g_logp,
                  g_ent, dh, dW, flags, true, workspace, workspace_bytes, stream);
}

int lmhead_logps_bwd_shard(const uint16_t* hidden, const uint16_t* W_shard, const int32_t* targets,
                           int64_t N, int64_t H, int64_t V_shard, int64_t vocab_offset, int64_t V_total,
                           int64_t chunk_size, float temperature, const float* lse, const float* entropy,
                           const float* g_logp, const float* g_ent, float* dh, float* dW_shard,
                           unsigned flags, void* workspace, size_t workspace_bytes, void* stream) {
  return bwd_impl("bwd_shard", hidden, W_shard, targets, N, H, V_shard, vocab_offset, V_total, chunk_size,
                  temperature, lse, entropy, g_logp, g_ent, dh, dW_shard, flags, false, workspace, workspace_bytes,
                  stream);
}

int lmhead_logps_fwd(const uint16_t* hidden, const uint16_t* W, const int32_t* targets, int64_t N,
                     int64_t H, int64_t V, int64_t chunk_size, float* logp, float* entropy,
                     float* lse, void* workspace, size_t workspace_bytes, void* stream) {
  return lmhead_logps_fwd_temp(hidden, W, targets, N, H, V, chunk_size, 1.0f, logp, entropy, lse,
                               workspace, workspace_bytes, stream);
}

int lmhead_logps_bwd_temp(const uint16_t* hidden, const uint16_t* W, const int32_t* targets,
                          int64_t N, int64_t H, int64_t V, int64_t chunk_size, float temperature,
                          const float* lse, const float* entropy, const float* g_logp,
                          const float* g_ent, float* dh, float* dW, void* workspace,
                          size_t workspace_bytes, void* stream) {
  return lmhead_logps_bwd_ex(hidden, W, targets, N, H, V, chunk_size, temperature, lse, entropy,
                             g_logp, g_ent, dh, dW, 0u, workspace, workspace_bytes, stream);
}

int lmhead_logps_bwd(const uint16_t* hidden, const uint16_t* W, const int32_t* targets, int64_t N,
                     int64_t H, int64_t V, int64_t chunk_size, const float* lse,
                     const float* entropy, const float* g_logp, const float* g_ent, float* dh,
                     float* dW, void* workspace, size_t workspace_bytes, void* stream) {
  return lmhead_logps_bwd_ex(hidden, W, targets, N, H, V, chunk_size, 1.0f, lse, entropy, g_logp,
                             g_ent, dh, dW, 0u, workspace, workspace_bytes, stream);
}

}  // extern "C"

// ---------------------------------------------------------------------------
// Distillation from a teacher's top logits.
namespace {

static_assert(lmh::kDistillMaxK == LMH_DISTILL_MAX_K && lmh::kNormMaxH == LMH_NORM_MAX_H, "limits in the header");

bool known_type(int type) { return type == LMH_TYPE_BF16 || type == LMH_TYPE_F32; }
uintptr_t type_size(int type) { return type == LMH_TYPE_F32 ? 4 : 2; }

int check_distill(int64_t N, int64_t H, int64_t V, int64_t K, int64_t chunk_size) {
  const int rc = check_shape(N, H, V, chunk_size);
  if (rc != LMH_OK) return rc;
  if (K < 1 || K > LMH_DISTILL_MAX_K)
    return fail(LMH_ERR_SHAPE, "K must be in [1, %d], got %lld", LMH_DISTILL_MAX_K, (long long)K);
  return LMH_OK;
}

// Where the distillation's arrays lie behind the head's own workspace.
struct DistillPlan {
  size_t fwd_bytes = 0;                                      // the forward: its split records alone
  size_t off_tgt = 0, off_ga = 0, off_id = 0, off_val = 0;   // the backward
  size_t off_part = 0, bytes = 0;                            // its dh splits; its total
  size_t off_w_part = 0;                                     // its dW splits
  int k_split = 0, w_k_split = 0;                            // 0: not split
  // few tokens: their own kernels
  bool few = false;
  size_t off_hi = 0, off_lo = 0;
  int dh_strips = 0, dh_rows = 0, dh_splits = 0;
};

// When the kernels for few tokens (lmhead_few.hip) run: they fetch W once per
// 64 tokens, where the 256 x 256 tiles fetch it once per 256 but spend a whole
// tile's time on what little there is. One tile of 64 tokens always; more, up
// to 256 tokens, where the vocabulary is small enough for the product of the
// two. Measured (us, few / tiles):
//   tokens  H     V       forward   backward
//   64      2560  151936  160/220   645/711
//   128     2560  151936  248/221   771/736
//   128     2560  32000   63/63     183/181
//   128     4096  16000   54/87     124/177
//   192     512   30000   30/28     83/76
//   192     2560  16000   50/62     136/138
//   256     2560  16000   62/62     159/142
//   256     2560  8000    38/62     95/123
//   256     512   8000    16/26     50/73
constexpr int64_t kFewRows = 49152;   // 64-token tiles times vocabulary
bool few_tokens(int64_t N, int64_t V) {
  return N <= 64 ? V < (int64_t(1) << 23) : N <= lmh::kFewTokens && lmh::ceil_div(N, 64) * V <= kFewRows;
}
// The chunk that the backward's blocks are sized by: chunk_size, but blocks hold
// at least two 256 x 256 cotangent tiles per CU (2^25 entries, 134 MB in both
// buffers, 0.05% of the card's memory). Below that a launch has less than a
// round of tiles, and the blocks' launches run one after the other. Measured (us
// at blocks of 8 / 32 / 64 / 128 / 256 MB): 2000 x 512 x 8000 423 / 188 / 147 /
// 132 / 131; 1357 x 1024 x 50257 1824 / 790 / 559 / 448 / 437; 16000 x 256 x 12000
// 4312 / 1279 / 880 / 549 / 476; 300 x 2048 x 100000 1804 / 756 / 615 / 611 / 621.
constexpr int64_t kLeastBlock = 2 * (int64_t)lmh::kNumCUs * lmh::kTileRows * lmh::kTileRows;
int64_t block_chunk(int64_t V, int64_t chunk_size) { return std::max(chunk_size, lmh::ceil_div(kLeastBlock, V)); }

// The backward holds the tokens' whole cotangent, as two bf16 words up to 64
// tokens and one above, which the block's size has to allow.
int64_t few_padded(int64_t N) { return N <= 32 ? 32 : lmh::round_up(N, 64); }
bool few_backward(int64_t N, int64_t V, int64_t chunk_size) {
  return few_tokens(N, V) && few_padded(N) / (N <= 64 ? 1 : 2) <= block_chunk(V, chunk_size);
}

// Splits of a launch's gradient tiles over their K (the block's vocabulary for
// dh, its tokens for dW). A launch holds the dh tiles, the dW tiles and (with
// more than one block) the next block's cotangent tiles, each of 1.05 us per 64
// of its K and 16 us around them on a CU (a dh tile of up to twice that: where
// few token tiles share its rows of W, it waits for memory); it takes all of
// them over the CUs, but no less than its longest gradient tile and a half. Small
// blocks have few tiles: 512 tokens, H 2560, V 151936 have 20 dh tiles that each
// walk 2374 slices, 2.5 ms alone (split, the whole call takes 1.26); 2000 tokens,
// H 512, V 8000 64 dW tiles of 32 slices. A split costs its tiles' 16 us and a float32
// partial of the block's gradient, written and read once at about 4 TB/s.
struct Splits {
  int dh, dW;
};
Splits grad_splits(const lmh::BwdPlan& p, int64_t H) {
  const double T = lmh::kTileRows;
  const double tt = (double)lmh::ceil_div(p.Ct, lmh::kTileRows), vt = (double)lmh::ceil_div(p.Vb, lmh::kTileRows);
  const double ht = (double)lmh::ceil_div(H, lmh::kTileRows);
  auto tile = [](double k) { return 1.05 * k / 64.0 + 16.0; };   // us
  const double z = p.n_tb * p.n_vb > 1 ? tile((double)H) : 0.0;
  Splits best{1, 1};
  double best_t = 1e300;
  for (int kd = 1; kd <= 64 && (kd == 1 || p.Vb / kd >= 512); ++kd)
    for (int kw = 1; kw <= 16 && (kw == 1 || p.Ct / kw >= 256); ++kw) {
      const double dh = tile((double)p.Vb / kd * (1.0 + 1.0 / tt)), dW = tile((double)p.Ct / kw);
      const double all = (tt * ht * kd * dh + vt * ht * kw * dW + tt * vt * z) / lmh::kNumCUs;
      const double part = ((kd > 1 || kw > 1 ? kd * tt : 0.0) + (kw > 1 ? kw * vt : 0.0)) * T * H * 8.0 / 4.0e6;
      const double t = std::max(std::max(all, z), 1.5 * std::max(dh, dW)) + part;
      if (t < best_t) {
        best_t = t;
        best = {kd, kw};
      }
    }
  return best;
}

// Up to a split per CU, since their records are merged by a wave per token
// here: with one token tile (N <= 256), 128 splits of 594 vocabulary tiles
// would take 5 tiles' time on half the CUs, 198 take 3.
lmh::FwdPlan plan_distill_forward(int64_t N, int64_t H, int64_t V) {
  if (!few_tokens(N, V)) return lmh::plan_forward(N, H, V, lmh::kNumCUs);
  lmh::FwdPlan p;
  p.S = lmh::few_splits(V);
  p.part_ld = lmh::round_up(std::max<int64_t>(N, 1), 64);
  p.bytes = (size_t)p.S * p.part_ld * 16;
  return p;
}

DistillPlan plan_distill(int64_t N, int64_t H, int64_t V, int64_t K, int64_t chunk_size, int kind) {
  DistillPlan d;
  const int64_t n = std::max<int64_t>(N, 1);
  auto room = [](int64_t bytes) { return (size_t)lmh::round_up(bytes, 256); };
  d.fwd_bytes = plan_distill_forward(N, H, V).bytes;
  if (kind == LMH_WS_FWD) {
    d.bytes = d.fwd_bytes;
    return d;
  }
  d.few = few_backward(n, V, chunk_size);
  lmh::BwdPlan p;
  if (!d.few) {
    p = lmh::plan_backward(N, H, V, block_chunk(V, chunk_size));
    d.off_tgt = kind == LMH_WS_BWD_BF16 ? p.bytes_bf16 : p.bytes;
  }
  d.off_ga = d.off_tgt + room(n * 4);
  d.off_id = d.off_ga + room(n * 4);
  d.off_val = d.off_id + room(n * (K + 1) * 4);
  d.off_part = d.off_val + room(n * (K + 1) * 4);
  if (d.few) {
    d.off_hi = d.off_part;
    d.off_lo = d.off_hi + room(V * few_padded(n) * 2);
    d.off_part = d.off_lo + (n <= 64 ? room(V * few_padded(n) * 2) : 0);
    // two workgroups a CU (three of up to 32 tokens), of at least 128 vocabulary rows
    // each; one split where the strips of a long row alone are more
    d.dh_strips = (int)lmh::ceil_div(H, 256);
    const int64_t wgs = (n <= 32 ? 3 : 2) * lmh::kNumCUs / (d.dh_strips * lmh::ceil_div(n, 64));
    const int64_t most = std::max<int64_t>(1, std::min<int64_t>(wgs, lmh::ceil_div(V, 128)));
    d.dh_rows = (int)lmh::round_up(lmh::ceil_div(V, most), 32);
    d.dh_splits = (int)lmh::ceil_div(V, d.dh_rows);
    d.bytes = d.off_part + room(d.dh_splits * n * H * 4);
    return d;
  }
  d.bytes = d.off_w_part = d.off_part;
  const Splits k = grad_splits(p, H);
  if (k.dh > 1 || k.dW > 1) {
    d.k_split = (int)lmh::round_up(lmh::ceil_div(p.Vb, k.dh), 64);
    d.off_w_part = d.off_part + room(lmh::ceil_div(lmh::round_up(p.Vb, 64), d.k_split) * p.Ct * H * 4);
    d.bytes = d.off_w_part;
    if (k.dW > 1) {
      d.w_k_split = (int)lmh::round_up(lmh::ceil_div(p.Ct, k.dW), 64);
      d.bytes += room(lmh::ceil_div(lmh::round_up(p.Ct, 64), d.w_k_split) * p.Vb * H * 4);
    }
  }
  return d;
}

}  // namespace

extern "C" {

int lmhead_logps_distill_workspace_bytes(int64_t N, int64_t H, int64_t V, int64_t K, int64_t chunk_size,
                                         int with_backward, size_t* bytes_out) {
  if (bytes_out == nullptr) return fail(LMH_ERR_NULL, "bytes_out is NULL");
  int rc = check_distill(N, H, V, K, chunk_size);
  if (rc != LMH_OK) return rc;
  if (with_backward < 0 || with_backward > LMH_WS_BWD_BF16)
    return fail(LMH_ERR_ARGS, "with_backward must be 0, 1 or 2, got %d", with_backward);
  if (with_backward && (rc = check_backward_size(N, V)) != LMH_OK) return rc;
  const DistillPlan d = plan_distill(N, H, V, K, chunk_size, with_backward);
  *bytes_out = std::max(d.fwd_bytes, d.bytes);
  return ok();
}

int lmhead_logps_distill_fwd(const uint16_t* hidden, const uint16_t* W, const int32_t* targets, const int32_t* ids,
                             const void* teacher, int teacher_type, const float* teacher_lse, int64_t N, int64_t H,
                             int64_t V, int64_t K, int64_t chunk_size, float temperature, float* kl, float* logp,
                             float* lse, float* logp_top, void* workspace, size_t workspace_bytes, void* stream) {
  int rc = check_distill(N, H, V, K, chunk_size);
  if (rc != LMH_OK) return rc;
  rc = check_temperature(temperature);
  if (rc != LMH_OK) return rc;
  if (!known_type(teacher_type)) return fail(LMH_ERR_ARGS, "distill_fwd: unknown teacher_type %d", teacher_type);
  if (logp != nullptr && targets == nullptr) return fail(LMH_ERR_ARGS, "distill_fwd: logp asked for without targets");
  if (N == 0) return ok();
  if (!hidden || !W || !ids || !teacher || !kl || !lse || !logp_top || !workspace)
    return fail(LMH_ERR_NULL,
                "distill_fwd: hidden, W, ids, teacher, kl, lse, logp_top and workspace must be non-NULL");
  if (!aligned(hidden, 16) || !aligned(W, 16) || !aligned(workspace, 16) || !aligned(targets, 4) || !aligned(ids, 4) ||
      !aligned(teacher, type_size(teacher_type)) || !aligned(teacher_lse, 4) || !aligned(kl, 4) || !aligned(logp, 4) ||
      !aligned(lse, 4) || !aligned(logp_top, 4))
    return fail(LMH_ERR_UNSUPPORTED,
                "distill_fwd: hidden, W and workspace need 16-byte alignment, the others that of their elements");
  const DistillPlan d = plan_distill(N, H, V, K, chunk_size, LMH_WS_FWD);
  if (workspace_bytes < d.bytes)
    return fail(LMH_ERR_WORKSPACE, "distill_fwd: workspace of %zu bytes, %zu needed", workspace_bytes, d.bytes);
  hipStream_t s = static_cast<hipStream_t>(stream);
  const lmh::FwdPlan p = plan_distill_forward(N, H, V);
  const float sc = temper_scale(temperature);
  // without hard targets the tile kernel still reads N ids to pick a logit by:
  // any will do, the pick is not used
  hipError_t e;
  if (few_tokens(N, V)) {
    lmh::FewArgs a{};
    a.hidden = hidden;
    a.W = W;
    a.targets = targets;
    a.N = (int)N;
    a.H = (int)H;
    a.V = (int)V;
    a.sc = sc;
    a.part = workspace;
    a.part_ld = p.part_ld;
    e = lmh::launch_few_stats(a, s);
  } else {
    lmh::FwdArgs a{hidden, W, targets != nullptr ? targets : ids, N, H, V, p.S, p.n_tt, p.n_vt, 0, V, sc,
                   inv_temperature(temperature), workspace, p.part_ld, nullptr, nullptr, nullptr, nullptr};
    e = lmh::launch_fwd_stats(a, s);
  }
  const double back = 1.0 / ((double)sc * (double)temperature);
  const float back_hi = (float)back;
  if (e == hipSuccess)
    e = lmh::launch_distill_top({hidden, W, targets, ids, teacher, teacher_type == LMH_TYPE_F32, teacher_lse, N,
                                 (int)H, (int)V, (int)K, temperature, back_hi, (float)(back - (double)back_hi),
                                 workspace, p.part_ld, p.S, kl, logp, lse, logp_top, 0}, s);
  if (e != hipSuccess) return fail(LMH_ERR_HIP, "distill_fwd: launch failed: %s", hipGetErrorString(e));
  return ok();
}

}  // extern "C"

namespace {

// The backward of few tokens, after every check.
hipError_t few_bwd(const DistillPlan& d, const lmh::DistillPrepArgs& prep, const uint16_t* hidden, const uint16_t* W,
                   int64_t H, float temperature, const float* lse, void* dh, void* dW, bool bf16, unsigned flags,
                   char* ws, hipStream_t s) {
  hipError_t e = lmh::launch_distill_prep(prep, s);
  if (e != hipSuccess) return e;
  lmh::FewArgs a{};
  a.hidden = hidden;
  a.W = W;
  a.targets = prep.tgt;
  a.N = (int)prep.N;
  a.H = (int)H;
  a.V = prep.V;
  a.sc = temper_scale(temperature);
  a.invT = prep.invT;
  a.lse = lse;
  a.ga = prep.ga;
  a.ent_id = prep.ent_id;
  a.ent_val = prep.ent_val;
  a.K1 = prep.K + 1;
  a.dz_hi = reinterpret_cast<uint16_t*>(ws + d.off_hi);
  a.dz_lo = prep.N <= 64 ? reinterpret_cast<uint16_t*>(ws + d.off_lo) : nullptr;
  a.padded = (int)few_padded(prep.N);
  a.dW = dW;
  a.add_dW = (flags & LMH_BWD_ACCUMULATE_DW) != 0;
  a.dh_part = reinterpret_cast<float*>(ws + d.off_part);
  a.dh_strips = d.dh_strips;
  a.dh_splits = d.dh_splits;
  a.dh_rows = d.dh_rows;
  e = lmh::launch_few_bwd(a, bf16, s);
  if (e != hipSuccess) return e;
  const bool add = (flags & LMH_BWD_ACCUMULATE_DH) != 0;
  lmh::DistillPostArgs post{};
  post.dh.part = a.dh_part;
  post.dh.splits = d.dh_splits;
  post.dh.rows = a.N;
  post.H = a.H;
  post.V = a.V;
  post.tgt = prep.tgt;
  post.dh.o.src_kind = !add ? lmh::kSrcNone : bf16 ? lmh::kSrcBf16 : lmh::kSrcF32;
  post.dh.o.src = post.dh.o.dst = dh;
  post.dh.o.dst_bf16 = bf16;
  post.dead_zero = !add;
  return lmh::launch_distill_post(post, s);
}

}  // namespace

extern "C" {

int lmhead_logps_distill_bwd(const uint16_t* hidden, const uint16_t* W, const int32_t* targets, const int32_t* ids,
                             const void* teacher, int teacher_type, const float* teacher_lse, int64_t N, int64_t H,
                             int64_t V, int64_t K, int64_t chunk_size, float temperature, const float* logp,
                             const float* lse, const float* logp_top, const float* g_kl, const float* g_logp,
                             void* dh, void* dW, int grad_type, unsigned flags, void* workspace,
                             size_t workspace_bytes, void* stream) {
  int rc = check_distill(N, H, V, K, chunk_size);
  if (rc != LMH_OK) return rc;
  rc = check_temperature(temperature);
  if (rc != LMH_OK) return rc;
  rc = check_backward_size(N, V);
  if (rc != LMH_OK) return rc;
  if (!known_type(teacher_type) || !known_type(grad_type))
    return fail(LMH_ERR_ARGS, "distill_bwd: unknown teacher_type %d or grad_type %d", teacher_type, grad_type);
  if (g_logp != nullptr && (targets == nullptr || logp == nullptr))
    return fail(LMH_ERR_ARGS, "distill_bwd: g_logp given without targets or without the forward's logp");
  const bool bf16 = grad_type == LMH_TYPE_BF16;
  DistillHook hook{};
  const int32_t* tgt = nullptr;
  const float* ga = nullptr;
  if (N > 0) {
    if (!hidden || !W || !ids || !teacher || !lse || !logp_top || !workspace || !dh || !dW)
      return fail(LMH_ERR_NULL,
                  "distill_bwd: hidden, W, ids, teacher, lse, logp_top, dh, dW and workspace must be non-NULL");
    if (flags & ~(unsigned)(LMH_BWD_ACCUMULATE_DH | LMH_BWD_ACCUMULATE_DW))
      return fail(LMH_ERR_ARGS, "distill_bwd: unknown flags 0x%x", flags);
    if (!aligned(hidden, 16) || !aligned(W, 16) || !aligned(dh, 16) || !aligned(targets, 4) || !aligned(ids, 4) || !aligned(teacher, type_size(teacher_type)) ||
        !aligned(teacher_lse, 4) || !aligned(logp, 4) || !aligned(lse, 4) || !aligned(logp_top, 4) ||
        !aligned(g_kl, 4) || !aligned(g_logp, 4) || !aligned(workspace, 16) || !aligned(dW, 16))
      return fail(LMH_ERR_UNSUPPORTED, "distill_bwd: a misaligned pointer");
    const DistillPlan d = plan_distill(N, H, V, K, chunk_size, bf16 ? LMH_WS_BWD_BF16 : LMH_WS_BWD);
    char* ws = static_cast<char*>(workspace);
    int32_t* w_tgt = reinterpret_cast<int32_t*>(ws + d.off_tgt);
    float* w_ga = reinterpret_cast<float*>(ws + d.off_ga);
    // a hard target without a cotangent takes no part
    hook.prep = {g_logp != nullptr ? targets : nullptr, ids, teacher, teacher_type == LMH_TYPE_F32, teacher_lse, N,
                 (int)V, (int)K, temperature, inv_temperature(temperature), logp, logp_top, g_kl, g_logp, w_tgt, w_ga,
                 reinterpret_cast<int32_t*>(ws + d.off_id), reinterpret_cast<float*>(ws + d.off_val),
                 nullptr, 0, nullptr, nullptr, 0, 0};
    if (d.few) {
      if (workspace_bytes < d.bytes)
        return fail(LMH_ERR_WORKSPACE, "distill_bwd: workspace of %zu bytes, %zu needed", workspace_bytes, d.bytes);
      const hipError_t e = few_bwd(d, hook.prep, hidden, W, H, temperature, lse, dh, dW, bf16, flags, ws,
                                   static_cast<hipStream_t>(stream));
      if (e != hipSuccess) return fail(LMH_ERR_HIP, "distill_bwd: launch failed: %s", hipGetErrorString(e));
      return ok();
    }
    hook.k_split = d.k_split;
    hook.w_k_split = d.w_k_split;
    hook.part = reinterpret_cast<float*>(ws + d.off_part);
    hook.w_part = reinterpret_cast<float*>(ws + d.off_w_part);
    hook.bytes = d.bytes;
    tgt = w_tgt;
    ga = w_ga;
  }
  return bwd_impl("distill_bwd", hidden, W, tgt, N, H, V, 0, V, block_chunk(V, chunk_size), temperature, lse, nullptr, ga, nullptr,
                  dh, dW, flags, bf16, workspace, workspace_bytes, stream, N > 0 ? &hook : nullptr);
}

}  // extern "C"

// ---------------------------------------------------------------------------
// The norm in front of the head.
namespace {

int check_norm(const char* who, int64_t N, int64_t H) {
  if (N < 0 || N >= (int64_t(1) << 31))
    return fail(LMH_ERR_SHAPE, "%s: N must be in [0, 2^31), got %lld", who, (long long)N);
  if (H <= 0) return fail(LMH_ERR_SHAPE, "%s: H must be > 0, got %lld", who, (long long)H);
  if (H > LMH_NORM_MAX_H)
    return fail(LMH_ERR_UNSUPPORTED, "%s: H must be at most %d, got %lld", who, LMH_NORM_MAX_H, (long long)H);
  return LMH_OK;
}

int check_norm_types(const char* who, int kind, int x_type, int y_type, int w_type) {
  if (kind != LMH_NORM_LAYER && kind != LMH_NORM_RMS) return fail(LMH_ERR_ARGS, "%s: unknown kind %d", who, kind);
  if (!known_type(x_type) || !known_type(y_type) || !known_type(w_type))
    return fail(LMH_ERR_ARGS, "%s: unknown type among x %d, y %d, weight %d", who, x_type, y_type, w_type);
  if (y_type == LMH_TYPE_F32 && x_type != LMH_TYPE_F32)
    return fail(LMH_ERR_ARGS, "%s: float32 y needs float32 x", who);
  return LMH_OK;
}

size_t norm_part_bytes(int64_t N, int64_t H) { return (size_t)lmh::norm_bwd_blocks(N, H) * 2 * (size_t)H * 4; }

}  // namespace

extern "C" {

int lmhead_logps_norm_workspace_bytes(int64_t N, int64_t H, size_t* bytes_out) {
  if (bytes_out == nullptr) return fail(LMH_ERR_NULL, "bytes_out is NULL");
  const int rc = check_norm("norm", N, H);
  if (rc != LMH_OK) return rc;
  *bytes_out = norm_part_bytes(N, H);
  return ok();
}

int lmhead_logps_norm_fwd(const void* x, int x_type, const void* weight, const void* bias, int w_type, int64_t N,
                          int64_t H, float eps, int kind, void* y, int y_type, float* mean, float* rstd,
                          void* stream) {
  int rc = check_norm("norm_fwd", N, H);
  if (rc != LMH_OK) return rc;
  rc = check_norm_types("norm_fwd", kind, x_type, y_type, w_type);
  if (rc != LMH_OK) return rc;
  if (!(eps >= 0.0f) || !std::isfinite(eps)) return fail(LMH_ERR_ARGS, "norm_fwd: eps must be finite and >= 0, got %g", (double)eps);
  if (N == 0) return ok();
  if (!x || !y) return fail(LMH_ERR_NULL, "norm_fwd: x and y must be non-NULL");
  if (!aligned(x, type_size(x_type)) || !aligned(y, type_size(y_type)) || !aligned(weight, type_size(w_type)) ||
      !aligned(bias, type_size(w_type)) || !aligned(mean, 4) || !aligned(rstd, 4))
    return fail(LMH_ERR_UNSUPPORTED, "norm_fwd: a pointer is not aligned to its elements");
  const hipError_t e = lmh::launch_norm_fwd({x, weight, bias, x_type == LMH_TYPE_F32, y_type == LMH_TYPE_F32,
                                             w_type == LMH_TYPE_F32, kind == LMH_NORM_RMS, N, (int)H, eps, y, mean,
                                             rstd}, static_cast<hipStream_t>(stream));
  if (e != hipSuccess) return fail(LMH_ERR_HIP, "norm_fwd: launch failed: %s", hipGetErrorString(e));
  return ok();
}

int lmhead_logps_norm_bwd(const void* x, int x_type, const void* weight, int w_type, int64_t N, int64_t H, int kind,
                          const float* mean, const float* rstd, const void* dy, int y_type, void* dx, void* dweight,
                          void* dbias, int g_type, unsigned flags, void* workspace, size_t workspace_bytes,
                          void* stream) {
  int rc = check_norm("norm_bwd", N, H);
  if (rc != LMH_OK) return rc;
  rc = check_norm_types("norm_bwd", kind, x_type, y_type, w_type);
  if (rc != LMH_OK) return rc;
  if (!known_type(g_type)) return fail(LMH_ERR_ARGS, "norm_bwd: unknown g_type %d", g_type);
  if (flags & ~(unsigned)LMH_BWD_ACCUMULATE_DW) return fail(LMH_ERR_ARGS, "norm_bwd: unknown flags 0x%x", flags);
  const bool accumulate = (flags & LMH_BWD_ACCUMULATE_DW) != 0;
  const bool sums = dweight != nullptr || dbias != nullptr;
  if (!aligned(dweight, type_size(g_type)) || !aligned(dbias, type_size(g_type)))
    return fail(LMH_ERR_UNSUPPORTED, "norm_bwd: a pointer is not aligned to its elements");
  const lmh::NormReduceArgs empty{nullptr, 0, (int)H, g_type == LMH_TYPE_F32, accumulate, dweight, dbias};
  hipStream_t s = static_cast<hipStream_t>(stream);
  if (N == 0) {
    if (!sums || accumulate) return ok();
    const hipError_t e = lmh::launch_norm_reduce(empty, s);
    if (e != hipSuccess) return fail(LMH_ERR_HIP, "norm_bwd: launch failed: %s", hipGetErrorString(e));
    return ok();
  }
  if (!x || !rstd || !dy || !dx || (kind == LMH_NORM_LAYER && !mean) || (sums && !workspace))
    return fail(LMH_ERR_NULL, "norm_bwd: x, mean (layer norm), rstd, dy, dx and workspace (for dweight, dbias) must be non-NULL");
  if (!aligned(x, type_size(x_type)) || !aligned(dx, type_size(x_type)) || !aligned(dy, type_size(y_type)) ||
      !aligned(weight, type_size(w_type)) || !aligned(mean, 4) || !aligned(rstd, 4) || (sums && !aligned(workspace, 16)))
    return fail(LMH_ERR_UNSUPPORTED, "norm_bwd: a pointer is not aligned to its elements (workspace: 16 bytes)");
  const size_t need = sums ? norm_part_bytes(N, H) : 0;
  if (workspace_bytes < need)
    return fail(LMH_ERR_WORKSPACE, "norm_bwd: workspace of %zu bytes, %zu needed", workspace_bytes, need);
  const bool columns = sums && lmh::norm_by_columns(N);
  const bool partial = sums && !columns;
  lmh::NormReduceArgs red = empty;
  red.part = partial ? static_cast<float*>(workspace) : nullptr;
  red.blocks = lmh::norm_bwd_blocks(N, H);
  hipError_t e = lmh::launch_norm_bwd({x, weight, mean, rstd, dy, x_type == LMH_TYPE_F32, y_type == LMH_TYPE_F32,
                                       w_type == LMH_TYPE_F32, kind == LMH_NORM_RMS, N, (int)H, dx, red.blocks,
                                       const_cast<float*>(red.part), columns ? dweight : nullptr,
                                       columns ? dbias : nullptr, red.g_f32, accumulate}, s);
  if (e == hipSuccess && partial) e = lmh::launch_norm_reduce(red, s);
  if (e != hipSuccess) return fail(LMH_ERR_HIP, "norm_bwd: launch failed: %s", hipGetErrorString(e));
  return ok();
}

}  // extern "C"

// ---------------------------------------------------------------------------
// The vocabulary table as an embedding.
namespace {

// A launch holds less than 2^32 threads: it has fewer workgroups of 256 than this.
constexpr int64_t kMostBlocks = int64_t(1) << 24;

static_assert(lmh::kMostBeams == LMH_BEAM_MAX_BEAMS && lmh::kMostCandidates == LMH_BEAM_MAX_CANDIDATES, "limits in the header");

int check_embed(const char* who, int64_t N, int64_t H, int64_t V) {
  if (N < 0 || N >= (int64_t(1) << 31))
    return fail(LMH_ERR_SHAPE, "%s: N must be in [0, 2^31), got %lld", who, (long long)N);
  if (H <= 0 || H >= (int64_t(1) << 20))
    return fail(LMH_ERR_SHAPE, "%s: H must be in (0, 2^20), got %lld", who, (long long)H);
  if (V <= 0 || V >= (int64_t(1) << 31))
    return fail(LMH_ERR_SHAPE, "%s: V must be in (0, 2^31), got %lld", who, (long long)V);
  return LMH_OK;
}

// The gradient's sort: words in classes by their lowest bits, 256 (one
// workgroup a CU) or as many as keep a class's counters within LDS.
struct EmbedPlan {
  bool few = false;
  int classes = lmh::kNumCUs, shift = 8, words = 0;
  size_t off_order = 0, off_pieces = 0, off_longs = 0, off_touched = 0, off_part = 0, bytes = 0;
};
EmbedPlan plan_embed(int64_t N, int64_t H, int64_t V, bool add) {
  EmbedPlan p;
  p.few = N <= lmh::kFewIds && (add || V <= lmh::kFewWords);
  static_assert(int64_t(lmh::kMostClasses) * lmh::kMostClassWords >= int64_t(1) << 23, "classes for the V that check_backward_size lets through");
  while (lmh::ceil_div(V, p.classes) > lmh::kMostClassWords) p.classes *= 2, ++p.shift;
  p.words = (int)lmh::ceil_div(V, p.classes);
  size_t at = 0;
  auto take = [&](int64_t bytes) {
    const size_t here = at;
    at += (size_t)lmh::round_up(bytes, 256);
    return here;
  };
  const bool sorted = !p.few;
  take(sorted ? 12 * (int64_t)p.classes : 0);
  p.off_order = take(sorted ? 4 * N : 0);
  p.off_pieces = take(sorted ? 16 * N : 0);
  p.off_longs = take(16 * (sorted ? N / lmh::kPiece + 1 : N));
  p.off_touched = take(sorted ? (int64_t)p.classes * p.words : 0);
  p.off_part = take(N > lmh::kPiece ? 2 * lmh::ceil_div(N, lmh::kPiece) * H * 4 : 0);
  p.bytes = at;
  return p;
}

}  // namespace

extern "C" {

int lmhead_logps_embed_workspace_bytes(int64_t N, int64_t H, int64_t V, size_t* bytes_out) {
  if (bytes_out == nullptr) return fail(LMH_ERR_NULL, "bytes_out is NULL");
  int rc = check_embed("embed", N, H, V);
  if (rc == LMH_OK) rc = check_backward_size(N, V);
  if (rc != LMH_OK) return rc;
  *bytes_out = std::max(plan_embed(N, H, V, false).bytes, plan_embed(N, H, V, true).bytes);
  return ok();
}

int lmhead_logps_embed_fwd(const void* W, int w_type, const int32_t* ids, int64_t N, int64_t H, int64_t V, float scale,
                           void* y, int y_type, void* stream) {
  const int rc = check_embed("embed_fwd", N, H, V);
  if (rc != LMH_OK) return rc;
  if (!known_type(w_type) || !known_type(y_type))
    return fail(LMH_ERR_ARGS, "embed_fwd: unknown type among W %d, y %d", w_type, y_type);
  if (!std::isfinite(scale)) return fail(LMH_ERR_ARGS, "embed_fwd: scale must be finite, got %g", (double)scale);
  // outputs that come near this have 512 groups, of four elements or eight, to a workgroup
  if (lmh::ceil_div(N * lmh::ceil_div(H, 4), 512) >= kMostBlocks)
    return fail(LMH_ERR_UNSUPPORTED, "embed_fwd: N (%lld) times H / 4, rounded up (%lld), must not exceed 2^33 - 512", (long long)N,
                (long long)lmh::ceil_div(H, 4));
  if (N == 0) return ok();
  if (!W || !ids || !y) return fail(LMH_ERR_NULL, "embed_fwd: W, ids and y must be non-NULL");
  if (!aligned(W, type_size(w_type)) || !aligned(ids, 4) || !aligned(y, type_size(y_type)))
    return fail(LMH_ERR_UNSUPPORTED, "embed_fwd: a pointer is not aligned to its elements");
  const hipError_t e = lmh::launch_embed_fwd({W, ids, w_type == LMH_TYPE_F32, y_type == LMH_TYPE_F32, N, (int)H, (int)V,
                                              scale, y}, static_cast<hipStream_t>(stream));
  if (e != hipSuccess) return fail(LMH_ERR_HIP, "embed_fwd: launch failed: %s", hipGetErrorString(e));
  return ok();
}

int lmhead_logps_embed_bwd(const int32_t* ids, const void* dy, int y_type, int64_t N, int64_t H, int64_t V, float scale,
                           void* dW, int g_type, unsigned flags, void* workspace, size_t workspace_bytes, void* stream) {
  int rc = check_embed("embed_bwd", N, H, V);
  if (rc == LMH_OK) rc = check_backward_size(N, V);
  if (rc != LMH_OK) return rc;
  if (!known_type(y_type) || !known_type(g_type))
    return fail(LMH_ERR_ARGS, "embed_bwd: unknown type among dy %d, dW %d", y_type, g_type);
  if (!std::isfinite(scale)) return fail(LMH_ERR_ARGS, "embed_bwd: scale must be finite, got %g", (double)scale);
  if (flags & ~(unsigned)LMH_BWD_ACCUMULATE_DW) return fail(LMH_ERR_ARGS, "embed_bwd: unknown flags 0x%x", flags);
  const bool add = (flags & LMH_BWD_ACCUMULATE_DW) != 0;
  if (N == 0 && add) return ok();
  const EmbedPlan p = plan_embed(N, H, V, add);
  if (!dW || (!workspace && p.bytes > 0) || (N > 0 && (!ids || !dy)))
    return fail(LMH_ERR_NULL, "embed_bwd: ids, dy, dW and workspace must be non-NULL");
  if (!aligned(ids, 4) || !aligned(dy, type_size(y_type)) || !aligned(dW, type_size(g_type)) || !aligned(workspace, 16))
    return fail(LMH_ERR_UNSUPPORTED, "embed_bwd: a pointer is not aligned to its elements (workspace: 16 bytes)");
  if (workspace_bytes < p.bytes)
    return fail(LMH_ERR_WORKSPACE, "embed_bwd: workspace of %zu bytes, %zu needed", workspace_bytes, p.bytes);
  char* ws = static_cast<char*>(workspace);
  lmh::EmbedBwdArgs a{};
  a.ids = ids;
  a.dy = dy;
  a.y_f32 = y_type == LMH_TYPE_F32;
  a.g_f32 = g_type == LMH_TYPE_F32;
  a.add = add;
  a.few = p.few;
  a.N = (int)N;
  a.H = (int)H;
  a.V = (int)V;
  a.scale = scale;
  a.dW = dW;
  a.classes = p.classes;
  a.class_shift = p.shift;
  a.class_words = p.words;
  a.counts = reinterpret_cast<int32_t*>(ws);
  a.order = reinterpret_cast<int32_t*>(ws + p.off_order);
  a.pieces = reinterpret_cast<int4*>(ws + p.off_pieces);
  a.longs = reinterpret_cast<int4*>(ws + p.off_longs);
  a.touched = reinterpret_cast<uint8_t*>(ws + p.off_touched);
  a.part = reinterpret_cast<float*>(ws + p.off_part);
  const hipError_t e = lmh::launch_embed_bwd(a, static_cast<hipStream_t>(stream));
  if (e != hipSuccess) return fail(LMH_ERR_HIP, "embed_bwd: launch failed: %s", hipGetErrorString(e));
  return ok();
}

}  // extern "C"

// ---------------------------------------------------------------------------
// Beam search on the head.
namespace {

int check_beam(int64_t N, int64_t H, int64_t V, int64_t beams, int64_t candidates) {
  const int rc = check_shape(N, H, V, 1);
  if (rc != LMH_OK) return rc;
  if (beams < 1 || beams > LMH_BEAM_MAX_BEAMS)
    return fail(LMH_ERR_SHAPE, "beams must be in [1, %d], got %lld", LMH_BEAM_MAX_BEAMS, (long long)beams);
  if (N % beams != 0)
    return fail(LMH_ERR_SHAPE, "N (%lld) must be a multiple of beams (%lld)", (long long)N, (long long)beams);
  if (candidates < 1 || candidates > LMH_BEAM_MAX_CANDIDATES)
    return fail(LMH_ERR_SHAPE, "candidates must be in [1, %d], got %lld", LMH_BEAM_MAX_CANDIDATES, (long long)candidates);
  if (N >= (int64_t(1) << 23) || beams * V >= (int64_t(1) << 31))
    return fail(LMH_ERR_UNSUPPORTED, "beam_step: N (%lld) must stay below 2^23 and beams * V (%lld) below 2^31",
                (long long)N, (long long)(beams * V));
  if (N / beams * (candidates + lmh::kSpare) >= kMostBlocks)   // workgroups that score
    return fail(LMH_ERR_UNSUPPORTED, "beam_step: N / beams * (candidates + 16) must stay below 2^24, got %lld",
                (long long)(N / beams * (candidates + lmh::kSpare)));
  return LMH_OK;
}

// When the streaming kernels run: they fetch W once per 128 rows, where the
// tiles take as long for one row as for 256. Measured (us, H 2560, streaming /
// tiles): 128 rows at 151936 words 200/205, at 32000 39/51, at 8000 22/48; 256
// rows at 151936 294/217, at 32000 73/52, at 8000 23/48.
bool few_beams(int64_t N, int64_t V) {
  return N <= 128 ? V < (int64_t(1) << 23) : N <= lmh::kFewTokens && V <= 24576;
}

struct BeamPlan {
  bool few = false;
  int splits = 0, n_tt = 0, n_vt = 0, per_section = 0;
  int64_t n_sections = 0, n_blocks = 0, ld = 0;
  size_t off_sections = 0, off_blocks = 0, off_lse = 0, off_chosen = 0, off_used = 0, off_exact = 0, bytes = 0;
};
BeamPlan plan_beam(int64_t N, int64_t H, int64_t V, int64_t beams) {
  BeamPlan p;
  p.few = few_beams(N, V);
  if (p.few) {
    const int rows = lmh::beam_few_rows(N, V);
    p.splits = (int)lmh::ceil_div(V, rows);
    p.n_sections = p.splits;
    p.per_section = rows / 16;
  } else {
    const lmh::FwdPlan f = lmh::plan_forward(N, H, V, lmh::kNumCUs);
    p.splits = f.S;
    p.n_tt = f.n_tt;
    p.n_vt = f.n_vt;
    p.n_sections = lmh::ceil_div(V, 128);
    p.per_section = 8;
  }
  p.n_blocks = lmh::ceil_div(V, 16);
  // the tiles store whole: rows to 256, words to 256 (sections and blocks of them)
  p.ld = lmh::round_up(std::max<int64_t>(N, 1), p.few ? 64 : lmh::kTileRows);
  const int64_t groups = N / beams;
  size_t at = 0;
  auto take = [&](int64_t bytes) {
    const size_t here = at;
    at += (size_t)lmh::round_up(bytes, 256);
    return here;
  };
  take(8 * p.splits * p.ld);
  p.off_sections = take(4 * std::max<int64_t>(p.n_sections, 2 * p.n_vt) * p.ld);
  p.off_blocks = take(4 * std::max<int64_t>(p.n_blocks, 16 * p.n_vt) * p.ld);
  p.off_lse = take(8 * N);
  p.off_chosen = take(4 * lmh::kMostKept * groups);
  p.off_used = take(4 * groups);
  p.off_exact = take(8 * 16 * lmh::kMostKept * groups);
  p.bytes = at;
  return p;
}

}  // namespace

extern "C" {

int lmhead_logps_beam_workspace_bytes(int64_t N, int64_t H, int64_t V, int64_t beams, int64_t candidates,
                                      size_t* bytes_out) {
  if (bytes_out == nullptr) return fail(LMH_ERR_NULL, "bytes_out is NULL");
  const int rc = check_beam(N, H, V, beams, candidates);
  if (rc != LMH_OK) return rc;
  *bytes_out = plan_beam(N, H, V, beams).bytes;
  return ok();
}

int lmhead_logps_beam_step(const uint16_t* hidden, const uint16_t* W, const float* scores, const int32_t* ended,
                           const int32_t* allowed, int64_t N, int64_t H, int64_t V, int64_t beams, int64_t candidates,
                           float temperature, float* top_scores, int32_t* top_ids, int32_t* top_parents, float* lse,
                           void* workspace, size_t workspace_bytes, void* stream) {
  int rc = check_beam(N, H, V, beams, candidates);
  if (rc == LMH_OK) rc = check_temperature(temperature);
  if (rc != LMH_OK) return rc;
  if (N == 0) return ok();
  if (!hidden || !W || !scores || !top_scores || !top_ids || !top_parents || !lse || !workspace)
    return fail(LMH_ERR_NULL, "beam_step: hidden, W, scores, top_scores, top_ids, top_parents, lse and workspace must be non-NULL");
  if (!aligned(hidden, 16) || !aligned(W, 16) || !aligned(workspace, 16) || !aligned(scores, 4) || !aligned(ended, 4) ||
      !aligned(allowed, 4) || !aligned(top_scores, 4) || !aligned(top_ids, 4) || !aligned(top_parents, 4) || !aligned(lse, 4))
    return fail(LMH_ERR_UNSUPPORTED,
                "beam_step: hidden, W and workspace need 16-byte alignment, the others that of their elements");
  const BeamPlan p = plan_beam(N, H, V, beams);
  if (workspace_bytes < p.bytes)
    return fail(LMH_ERR_WORKSPACE, "beam_step: workspace of %zu bytes, %zu needed", workspace_bytes, p.bytes);
  char* ws = static_cast<char*>(workspace);
  lmh::BeamArgs b{};
  b.hidden = hidden;
  b.W = W;
  b.scores = scores;
  b.ended = ended;
  b.allowed = allowed;
  b.mask_ld = lmh::ceil_div(V, 32);
  b.N = (int)N;
  b.H = (int)H;
  b.V = (int)V;
  b.beams = (int)beams;
  b.C = (int)candidates;
  b.keep = (int)candidates + lmh::kSpare;
  b.sc = temper_scale(temperature);
  b.invT = inv_temperature(temperature);
  b.rT = 1.0 / (double)temperature;
  b.back = 1.0 / ((double)b.sc * (double)temperature);
  b.few = p.few;
  b.splits = p.splits;
  b.n_tt = p.n_tt;
  b.n_vt = p.n_vt;
  b.n_sections = p.n_sections;
  b.n_blocks = p.n_blocks;
  b.per_section = p.per_section;
  b.ld = p.ld;
  b.records = reinterpret_cast<float2*>(ws);
  b.sections = reinterpret_cast<float*>(ws + p.off_sections);
  b.blocks = reinterpret_cast<float*>(ws + p.off_blocks);
  b.lse64 = reinterpret_cast<double*>(ws + p.off_lse);
  b.chosen = reinterpret_cast<uint32_t*>(ws + p.off_chosen);
  b.used = reinterpret_cast<int32_t*>(ws + p.off_used);
  b.exact = reinterpret_cast<double*>(ws + p.off_exact);
  b.top_scores = top_scores;
  b.top_ids = top_ids;
  b.top_parents = top_parents;
  b.lse = lse;
  const hipError_t e = lmh::launch_beam_step(b, static_cast<hipStream_t>(stream));
  if (e != hipSuccess) return fail(LMH_ERR_HIP, "beam_step: launch failed: %s", hipGetErrorString(e));
  return ok();
}

int lmhead_logps_beam_reorder(const void* states, void* out, const int32_t* parents, const int32_t* lengths,
                              int64_t planes, int64_t rows, int64_t beams, int64_t runs, int64_t steps,
                              int64_t step_bytes, void* stream) {
  if (beams < 1 || beams > LMH_BEAM_MAX_BEAMS)
    return fail(LMH_ERR_SHAPE, "beam_reorder: beams must be in [1, %d], got %lld", LMH_BEAM_MAX_BEAMS, (long long)beams);
  if (planes < 0 || rows < 0 || runs < 0 || steps < 0 || step_bytes < 0 || rows % beams != 0)
    return fail(LMH_ERR_SHAPE, "beam_reorder: planes, rows (a multiple of beams), runs, steps and step_bytes must be >= 0");
  if (planes == 0 || rows == 0 || runs == 0 || steps == 0 || step_bytes == 0) return ok();
  int64_t bytes = 1;
  for (int64_t n : {planes, rows, runs, steps, step_bytes})
    if (__builtin_mul_overflow(bytes, n, &bytes) || bytes >= (int64_t(1) << 43) || rows >= (int64_t(1) << 31))
      return fail(LMH_ERR_UNSUPPORTED, "beam_reorder: the states hold 2^43 bytes or more");
  const int64_t run = steps * step_bytes;
  if (run >= (int64_t(1) << 35) || rows >= (int64_t(1) << 30) ||
      lmh::round_up(lmh::reorder_blocks(planes, rows, beams, runs, run), 8) >= kMostBlocks)   // as launched
    return fail(LMH_ERR_UNSUPPORTED, "beam_reorder: a run of 2^35 bytes or more, 2^30 rows, or more than 2^24 - 8 workgroups");
  if (!states || !out || !parents) return fail(LMH_ERR_NULL, "beam_reorder: states, out and parents must be non-NULL");
  if (!aligned(parents, 4) || !aligned(lengths, 4))
    return fail(LMH_ERR_UNSUPPORTED, "beam_reorder: a pointer is not aligned to its elements");
  const uintptr_t a = reinterpret_cast<uintptr_t>(states), b = reinterpret_cast<uintptr_t>(out);
  if (a != b && (a < b ? b - a : a - b) < (uintptr_t)bytes)
    return fail(LMH_ERR_ARGS, "beam_reorder: out overlaps the states without being them");
  const hipError_t e = lmh::launch_beam_reorder({states, out, parents, lengths, planes, rows, (int)beams, runs, steps,
                                                 step_bytes, 0, 0, 0}, static_cast<hipStream_t>(stream));
  if (e != hipSuccess) return fail(LMH_ERR_HIP, "beam_reorder: launch failed: %s", hipGetErrorString(e));
  return ok();
}

}  // extern "C"
