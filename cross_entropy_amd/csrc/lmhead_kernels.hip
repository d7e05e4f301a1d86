// lmhead_kernels.hip -- gfx950 (CDNA4) kernels of the fused LM-head
// log-prob / entropy head.
//
// Method (google/tunix pull request #2913, the fused sharded log-prob head;
// SkyRL issue "[tx] support long sequence", "4. Chunked LM Head"):
//   forward : one pass over each tile of logits z = h W^T keeps, per token,
//             a running max, the exp-sum and the exp-weighted sum of z, and
//             picks the target logit by index compare (a one-hot select);
//             vocabulary splits are merged by log-sum-exp.
//   backward: the logits are recomputed tile by tile, their cotangent dz is
//             formed in one elementwise pass and rounded to bf16, and both
//             gradient matmuls (dh = dz W, dW = dz^T h) read that one dz.
//
// Every contraction runs on one MFMA tile core: a 256 x 256 output tile per
// 256-thread workgroup (4 wave64s as 2 x 2, each owning 128 x 128, its 256
// f32 accumulators in AGPRs), v_mfma_f32_16x16x32_bf16. One wave per SIMD
// halves the LDS fragment traffic per MFMA against two waves of 128 x 64,
// and the short 16x16 MFMA keeps accumulator traffic through the register
// file low; the wave hides its own latencies through the order in which it
// issues work (see mma_tile). K is staged through two 64-wide LDS slices
// filled by direct-to-LDS loads (global_load_lds_dwordx4), so no VGPRs hold
// staged data. Slice rows are 128 bytes with a 16-byte-chunk XOR swizzle,
// which keeps the fragment reads free of bank conflicts. An A operand stored
// MN-contiguous (W and the cotangent in the backward) is staged as it lies
// and read with transposed LDS reads; the hidden states enter the dW GEMM
// through a transposed copy.
//
// MFMA 16x16x32 register layout used throughout (wave64): lane l supplies
// row (l % 16) of A and column (l % 16) of B with the 8 K values
// 8*(l/16) .. 8*(l/16)+7; result register r of lane l holds
// D[4*(l/16) + r][l % 16].
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "lmhead_internal.h"
#include "lmhead_tile.h"

namespace lmh {

// ---------------------------------------------------------------------------
// Forward tile kernel. Workgroup (token tile tt, split s) walks vocabulary
// tiles s, s + S, s + 2S, ... for its 256 tokens (A = W rows = vocabulary,
// B = hidden rows = tokens) and writes one partial Stats per token and split.
// sc = log2(e) / T scores the tempered logits z / T in base 2; the target
// logit is kept untempered (the merge scales it). W holds the V vocabulary
// rows from global id voff on (a vocabulary shard; voff = 0 for the whole
// table): a target is picked here only when it falls inside that range.
// Lane l of wave (wm, wn) holds tokens wn * 128 + 16 j + l % 16 (j = 0..7)
// and, of each, 32 vocabulary rows of the wave's 128.
__global__ __launch_bounds__(kThreads) void fwd_stats_kernel(
    const uint16_t* __restrict__ hidden, const uint16_t* __restrict__ W,
    const int32_t* __restrict__ targets, int N, int H, int V, int voff, int S, int n_tt, int n_vt,
    float sc, float4* __restrict__ part, int64_t part_ld) {
  __shared__ __attribute__((aligned(16))) char lds[kLdsBytes];
  const int vid = xcd_remap(blockIdx.x, gridDim.x);
  if (vid >= n_tt * S) return;
  const int tt = vid / S;
  const int s = vid - tt * S;
  const int lane = threadIdx.x & 63;
  const int wave = threadIdx.x >> 6;
  const int wm = wave & 1;
  const int wn = wave >> 1;
  const int tok0 = tt * kTile;

  int tgt[kNB];
  Stats st[kNB];
#pragma unroll
  for (int j = 0; j < kNB; ++j) {
    const int tok = tok0 + wn * 128 + j * 16 + (lane & 15);
    const int t = tok < N ? targets[tok] : -1;
    tgt[j] = (t >= voff && t - voff < V) ? t - voff : -1;   // local row, or no hit
    st[j].m2 = kNegBig;
    st[j].s1 = 0.0f;
    st[j].s2 = 0.0f;
    st[j].zt = 0.0f;
  }

  const Operand ob{hidden + (int64_t)tok0 * H, H, min(kTile, N - tok0)};
  Pipe pipe;
  for (int vt = s; vt < n_vt; vt += S) {
    const int v0 = vt * kTile;
    const Operand oa{W + (int64_t)v0 * H, H, min(kTile, V - v0)};
    // one call site (a runtime chain flag): two inlined copies of the core
    // would merge 256 accumulator registers. Chained only into a tile of the
    // same shape (the next one is not the ragged last tile, or both are).
    const int v1 = v0 + S * kTile;
    const bool more = vt + S < n_vt && min(kTile, V - v1) == oa.rows;
    f32x4 acc[kNB][kNB];
    mma_tile<false, 96>(oa, ob, H, lds, acc, pipe, W + (int64_t)(more ? v1 : v0) * H, ob.base, more);

    const int vrow0 = v0 + wm * 128;
    // ragged last tile: rows past V take no part. Their logits are set to
    // kNegBig so they never win the max (unless the wave has no row left),
    // and their exponentials are zeroed outright: scaled by sc < 1 the
    // rounding error of kNegBig * sc alone would overflow exp2.
    const bool ragged = vrow0 + 128 > V;
#pragma unroll
    for (int j = 0; j < kNB; ++j) {
      float z[kNB][4];
#pragma unroll
      for (int i = 0; i < kNB; ++i) {
        pin_acc(acc[i][j]);
#pragma unroll
        for (int r = 0; r < 4; ++r) z[i][r] = acc[i][j][r];
      }
      if (ragged) {
#pragma unroll
        for (int i = 0; i < kNB; ++i)
#pragma unroll
          for (int r = 0; r < 4; ++r) z[i][r] = (vrow0 + acc_row(i, r, lane) < V) ? z[i][r] : kNegBig;
      }
      // target logit: one-hot select, only in waves whose rows hold a target
      const int tr = tgt[j] - vrow0;
      const bool hit = (tr >= 0) && (tr < 128);
      if (__any(hit)) {
        float zt = st[j].zt;
#pragma unroll
        for (int i = 0; i < kNB; ++i)
#pragma unroll
          for (int r = 0; r < 4; ++r) zt = (acc_row(i, r, lane) == tr) ? z[i][r] : zt;
        st[j].zt = zt;
      }
      float mx = z[0][0];
#pragma unroll
      for (int i = 0; i < kNB; ++i)
#pragma unroll
        for (int r = 0; r < 4; ++r) mx = nan_max(mx, z[i][r]);
      const float mnew = nan_max(st[j].m2, mx * sc);   // sc > 0: max commutes with the scaling
      const float dm = st[j].m2 - mnew;
      const float alpha = fast_exp2(dm);
      float s1 = alpha * st[j].s1;
      float s2 = alpha * (st[j].s2 + dm * st[j].s1);
      if (!ragged) {
#pragma unroll
        for (int i = 0; i < kNB; ++i)
#pragma unroll
          for (int r = 0; r < 4; ++r) {
            const float d = fmaf(z[i][r], sc, -mnew);
            const float e = fast_exp2(d);
            s1 += e;
            s2 = fmaf(e, d, s2);
          }
      } else {
#pragma unroll
        for (int i = 0; i < kNB; ++i)
#pragma unroll
          for (int r = 0; r < 4; ++r) {
            const bool live = vrow0 + acc_row(i, r, lane) < V;
            const float d = live ? fmaf(z[i][r], sc, -mnew) : 0.0f;
            const float e = live ? fast_exp2(d) : 0.0f;
            s1 += e;
            s2 = fmaf(e, d, s2);
          }
      }
      st[j].m2 = mnew;
      st[j].s1 = s1;
      st[j].s2 = s2;
      __builtin_amdgcn_sched_barrier(0);
    }
  }

  // lanes l, l ^ 16, l ^ 32, l ^ 48 hold other rows of the same tokens:
  // merge in a fixed order (the lower lane group's record first)
#pragma unroll
  for (int x = 16; x <= 32; x <<= 1) {
#pragma unroll
    for (int j = 0; j < kNB; ++j) {
      Stats o;
      o.m2 = __shfl_xor(st[j].m2, x);
      o.s1 = __shfl_xor(st[j].s1, x);
      o.s2 = __shfl_xor(st[j].s2, x);
      o.zt = __shfl_xor(st[j].zt, x);
      st[j] = (lane & x) == 0 ? merge_stats(st[j], o) : merge_stats(o, st[j]);
    }
  }
  // waves wm = 0 and wm = 1 hold the two vocabulary halves of the same tokens
  float4* xch = reinterpret_cast<float4*>(lds);
  if (wm == 1 && lane < 16) {
#pragma unroll
    for (int j = 0; j < kNB; ++j)
      xch[(wn * kNB + j) * 16 + lane] = make_float4(st[j].m2, st[j].s1, st[j].s2, st[j].zt);
  }
  __syncthreads();
  if (wm == 0 && lane < 16) {
#pragma unroll
    for (int j = 0; j < kNB; ++j) {
      const float4 q = xch[(wn * kNB + j) * 16 + lane];
      const Stats o{q.x, q.y, q.z, q.w};
      const Stats m = merge_stats(st[j], o);
      const int tok = tok0 + wn * 128 + j * 16 + lane;
      if (tok < N) part[(int64_t)s * part_ld + tok] = make_float4(m.m2, m.s1, m.s2, m.zt);
    }
  }
}

// Split merge: per token, the S partial records in order, by log-sum-exp
// (vocabulary splits of one launch, or vocabulary shards). invT = 1 / T
// tempers the target logit; Vtot bounds the valid target ids. With `rec`
// the merged record itself is written (a shard's partial) instead.
__global__ __launch_bounds__(256) void fwd_merge_kernel(
    const float4* __restrict__ part, int64_t part_ld, int S, const int32_t* __restrict__ targets,
    int N, int Vtot, float invT, float* __restrict__ logp, float* __restrict__ entropy,
    float* __restrict__ lse, float4* __restrict__ rec) {
  const int i = blockIdx.x * 256 + threadIdx.x;
  if (i >= N) return;
  float4 q = part[i];
  Stats a{q.x, q.y, q.z, q.w};
  for (int s = 1; s < S; ++s) {
    q = part[(int64_t)s * part_ld + i];
    a = merge_stats(a, Stats{q.x, q.y, q.z, q.w});
  }
  if (rec != nullptr) {
    rec[i] = make_float4(a.m2, a.s1, a.s2, a.zt);
    return;
  }
  const int t = targets[i];
  const bool valid = (t >= 0) && (t < Vtot);
  const float l2s = log2f(a.s1);
  // lse = m + ln(sum e^(z-m)); a +inf logit (and no NaN) leaves m = +inf and
  // s1 = NaN (inf - inf): the log-sum-exp is +inf
  const float l = a.m2 == INFINITY ? INFINITY : kLn2 * (a.m2 + l2s);
  const float h = kLn2 * (l2s - a.s2 / a.s1);        // lse - sum p z
  logp[i] = valid ? a.zt * invT - l : 0.0f;
  lse[i] = valid ? l : 0.0f;
  if (entropy != nullptr) entropy[i] = valid ? h : 0.0f;
}

__global__ __launch_bounds__(kThreads) void bwd_step_kernel(const BwdStep s) {
  __shared__ __attribute__((aligned(16))) char lds[kLdsBytes];
  __shared__ int z_tile;
  bwd_step<false>(s, lds, z_tile);
}

// The same launch writing bf16 gradients through float32 accumulators.
__global__ __launch_bounds__(kThreads) void bwd_step_bf16_kernel(const BwdStep s) {
  __shared__ __attribute__((aligned(16))) char lds[kLdsBytes];
  __shared__ int z_tile;
  bwd_step<true>(s, lds, z_tile);
}

// Transposed bf16 copy: out[c][r] = in[r][c] for r < R and c < C, 0 for the
// padding r in [R, R_pad) and c in [C, C_pad); with `tgt`, rows whose target
// id lies outside [0, V) are 0 too (masked tokens never reach the dW GEMM,
// whatever their hidden row holds: the select happens here, once).
// Grid: (R_pad / 64, C_pad / 64), 256 threads; 64 x 64 tiles through LDS.
__global__ __launch_bounds__(256) void transpose_kernel(
    const uint16_t* __restrict__ in, int64_t ld_in, int R, int C, const int32_t* __restrict__ tgt,
    int V, uint16_t* __restrict__ out, int64_t ld_out) {
  __shared__ uint32_t t[64][33];   // 64 rows x 64 bf16 (as 32 words) + 1 word pad
  const int r0 = blockIdx.x * 64;
  const int c0 = blockIdx.y * 64;
  const int tid = threadIdx.x;
  {
    const int rl = tid >> 2;          // 0..63
    const int cq = (tid & 3) * 16;    // 16 columns each
    const int r = r0 + rl;
    bool ok = (r < R) && (c0 + cq < C);
    if (ok && tgt != nullptr) {
      const int tv = tgt[r];
      ok = (tv >= 0) && (tv < V);
    }
    uint4 v0 = make_uint4(0u, 0u, 0u, 0u), v1 = make_uint4(0u, 0u, 0u, 0u);
    if (ok) {
      const uint4* src = reinterpret_cast<const uint4*>(in + (int64_t)r * ld_in + c0 + cq);
      v0 = src[0];
      v1 = src[1];
    }
    uint32_t* d = &t[rl][cq >> 1];
    d[0] = v0.x; d[1] = v0.y; d[2] = v0.z; d[3] = v0.w;
    d[4] = v1.x; d[5] = v1.y; d[6] = v1.z; d[7] = v1.w;
  }
  __syncthreads();
  {
    const int cl = tid >> 2;          // output row (input column) 0..63
    const int rq = (tid & 3) * 16;    // 16 input rows each
    uint32_t w[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const uint32_t a = t[rq + 2 * e][cl >> 1];
      const uint32_t b = t[rq + 2 * e + 1][cl >> 1];
      const uint32_t lo = (cl & 1) ? (a >> 16) : (a & 0xFFFFu);
      const uint32_t hi = (cl & 1) ? (b >> 16) : (b & 0xFFFFu);
      w[e] = lo | (hi << 16);
    }
    uint4* dst = reinterpret_cast<uint4*>(out + (int64_t)(c0 + cl) * ld_out + r0 + rq);
    dst[0] = make_uint4(w[0], w[1], w[2], w[3]);
    dst[1] = make_uint4(w[4], w[5], w[6], w[7]);
  }
}

// Row copy with zero padding: out[r][c] = in[r][c] for r < R, 0 for
// R <= r < R_pad (c < C, C % 8 == 0; both of row stride C). One 16-byte
// chunk per thread.
__global__ __launch_bounds__(256) void pad_rows_kernel(const uint16_t* __restrict__ in, int R, int C,
                                                       int R_pad, uint16_t* __restrict__ out) {
  const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
  const int cpr = C / 8;
  if (i >= (int64_t)R_pad * cpr) return;
  const int r = (int)(i / cpr);
  uint4 v = make_uint4(0u, 0u, 0u, 0u);
  if (r < R) v = reinterpret_cast<const uint4*>(in)[i];
  reinterpret_cast<uint4*>(out)[i] = v;
}

__global__ __launch_bounds__(256) void fill_zero_kernel(float* __restrict__ p, int64_t n) {
  const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
  const int64_t stride = (int64_t)gridDim.x * 256;
  for (int64_t k = i; k < n; k += stride) p[k] = 0.0f;
}

// ---------------------------------------------------------------------------
// Host-side launchers (called by the C ABI after argument checks).

static inline unsigned round8(long long x) { return (unsigned)((x + 7) / 8 * 8); }

hipError_t launch_fwd_stats(const FwdArgs& a, hipStream_t stream) {
  const long long wg = (long long)a.n_tt * a.S;
  const double N = (double)a.N, H = (double)a.H, V = (double)a.V;
  trace_begin(stream);
  hipLaunchKernelGGL(fwd_stats_kernel, dim3(round8(wg)), dim3(kThreads), 0, stream, a.hidden, a.W,
                     a.targets, (int)a.N, (int)a.H, (int)a.V, (int)a.voff, a.S, a.n_tt, a.n_vt, a.sc,
                     reinterpret_cast<float4*>(a.part), a.part_ld);
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  trace_end(kFwdStats, stream, 2.0 * N * H * V, 2.0 * (N + V) * H + 4.0 * N + 16.0 * a.S * N);
  return hipSuccess;
}

hipError_t launch_fwd(const FwdArgs& a, hipStream_t stream) {
  hipError_t e = launch_fwd_stats(a, stream);
  if (e != hipSuccess) return e;
  const double N = (double)a.N;
  trace_begin(stream);
  hipLaunchKernelGGL(fwd_merge_kernel, dim3((unsigned)((a.N + 255) / 256)), dim3(256), 0, stream,
                     reinterpret_cast<const float4*>(a.part), a.part_ld, a.S, a.targets, (int)a.N,
                     (int)a.Vtot, a.invT, a.logp, a.entropy, a.lse, reinterpret_cast<float4*>(a.rec));
  e = hipGetLastError();
  if (e != hipSuccess) return e;
  trace_end(kFwdMerge, stream, 0.0, 16.0 * a.S * N + 16.0 * N);
  return hipSuccess;
}

hipError_t launch_merge(const float* partials, int P, int64_t N, const int32_t* targets, int64_t Vtot,
                        float invT, float* logp, float* entropy, float* lse, hipStream_t stream) {
  trace_begin(stream);
  hipLaunchKernelGGL(fwd_merge_kernel, dim3((unsigned)((N + 255) / 256)), dim3(256), 0, stream,
                     reinterpret_cast<const float4*>(partials), N, P, targets, (int)N, (int)Vtot, invT,
                     logp, entropy, lse, nullptr);
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  trace_end(kFwdMerge, stream, 0.0, 16.0 * P * (double)N + 16.0 * (double)N);
  return hipSuccess;
}

template <bool BF16>
static hipError_t launch_bwd(const BwdStep& st, hipStream_t stream) {
  const int n_z = st.z_ntt * st.z_nvt;
  int per = 0;
  for (int x = 0; x < 8; ++x)
    per = max(per, ((x + 1) * st.n_dw / 8 - x * st.n_dw / 8) + ((x + 1) * st.n_dh / 8 - x * st.n_dh / 8) +
                       ((x + 1) * n_z / 8 - x * n_z / 8) + (n_z > 0 ? kStealSlots : 0));
  if (per == 0) return hipSuccess;
  const int n_g = st.n_dw + st.n_dh;
  const double H = (double)st.H;
  const double gc = (double)st.g_Ct, gv = (double)st.g_Vb;
  const double zc = (double)st.z_Ct, zv = (double)st.z_Vb;
  trace_begin(stream);
  if (BF16) hipLaunchKernelGGL(bwd_step_bf16_kernel, dim3(8 * per), dim3(kThreads), 0, stream, st);
  else hipLaunchKernelGGL(bwd_step_kernel, dim3(8 * per), dim3(kThreads), 0, stream, st);
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  // algorithmic (credited) work: 2 Ct Vb H for each of the dh and dW GEMMs;
  // the recomputed logits (2 Ct' Vb' H more) are executed but not counted.
  // Bytes: the dz block written once and read once, operand panels, f32 outputs
  const double fl = n_g ? 4.0 * gc * gv * H : 0.0;
  const double by = (n_g ? 2.0 * gc * gv + 2.0 * (gc + gv) * H +
                               4.0 * H * (gc * (1 + st.g_acc_dh) + gv * (1 + st.g_acc_dW)) : 0.0) +
                    (n_z ? 2.0 * zc * zv + 2.0 * (zc + zv) * H + 20.0 * zc : 0.0);
  trace_end(BF16 ? kBwdStepBf16 : kBwdStep, stream, fl, by);
  return hipSuccess;
}

hipError_t launch_bwd_step(const BwdStep& st, hipStream_t stream) { return launch_bwd<false>(st, stream); }
hipError_t launch_bwd_step_bf16(const BwdStep& st, hipStream_t stream) { return launch_bwd<true>(st, stream); }

hipError_t launch_transpose(const uint16_t* in, int64_t ld_in, int64_t R, int64_t C, int64_t R_pad,
                            int64_t C_pad, const int32_t* tgt, int64_t V, uint16_t* out,
                            int64_t ld_out, hipStream_t stream) {
  trace_begin(stream);
  hipLaunchKernelGGL(transpose_kernel, dim3((unsigned)(R_pad / 64), (unsigned)(C_pad / 64)), dim3(256),
                     0, stream, in, ld_in, (int)R, (int)C, tgt, (int)V, out, ld_out);
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  trace_end(kTranspose, stream, 0.0, 2.0 * (double)R * C + 2.0 * (double)R_pad * C_pad);
  return hipSuccess;
}

hipError_t launch_pad_rows(const uint16_t* in, int64_t R, int64_t C, int64_t R_pad, uint16_t* out,
                           hipStream_t stream) {
  const long long n = R_pad * (C / 8);
  if (n <= 0) return hipSuccess;
  trace_begin(stream);
  hipLaunchKernelGGL(pad_rows_kernel, dim3((unsigned)((n + 255) / 256)), dim3(256), 0, stream, in, (int)R,
                     (int)C, (int)R_pad, out);
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  trace_end(kPadRows, stream, 0.0, 2.0 * (double)R * C + 2.0 * (double)R_pad * C);
  return hipSuccess;
}

hipError_t launch_fill_zero(float* p, int64_t n, hipStream_t stream) {
  if (n <= 0) return hipSuccess;
  long long blocks = (n + 255) / 256;
  if (blocks > 4096) blocks = 4096;
  trace_begin(stream);
  hipLaunchKernelGGL(fill_zero_kernel, dim3((unsigned)blocks), dim3(256), 0, stream, p, n);
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  trace_end(kFill, stream, 0.0, 4.0 * (double)n);
  return hipSuccess;
}

}  // namespace lmh
