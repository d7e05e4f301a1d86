// lmhead_distill.hip -- distillation from a teacher's top logits on the head's
// never-stored logits, for gfx950: the parts beside the head's own tile
// kernels (lmhead_kernels.hip).
//
// With z = W h / T, lse = log sum exp z and, for the K teacher entries
// (id_k, t_k) of a token, s_k = z[id_k] - lse and q_k = softmax(t / T)_k over
// the live entries (or exp(t_k / T - teacher_lse)):
//
//   kl   = sum_k q_k (log q_k - s_k),   Q = sum_k q_k
//   dz_v = [ g_kl (Q p_v - sum_{id_k = v} q_k) + g_logp (1[v = target] - p_v) ] / T
//
// Away from the teacher's ids and the target, dz_v = -(g_logp - g_kl Q) p_v / T:
// the head's own cotangent under the log-prob cotangent g_logp - g_kl Q. So
// the forward takes the head's log-sum-exp record and adds K dot products a
// token (0.04% of its products at K = 64, V = 152k), and the backward runs the
// head's tiles with that combined cotangent and then overwrites the K + 1
// special entries of each token in the cotangent block, each formed in
// float32 and rounded to bf16 once (added to the tile's rounded entry instead,
// Q p - q would keep only the digits that bf16 left in p).
//
// The cotangent is bf16, as the head's is, also where the gradients are float32:
// the matrix units multiply bf16 at over ten times float32's rate. It is the only
// rounding beside the stored gradient's own: at 256 x 256 x 4096 float32 gradients
// are 1.6e-3 to 1.8e-3 off in norm (1e-6 from the products of the so rounded
// entries), bf16 ones 2.3e-3 to 2.4e-3, where storing them alone leaves 1.7e-3.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include <algorithm>

#include "lmhead_internal.h"
#include "lmhead_tile.h"

namespace lmh {
namespace {

__device__ __forceinline__ float teacher_at(const void* t, bool f32, int64_t i) {
  return f32 ? static_cast<const float*>(t)[i] : widen_bf16(static_cast<const uint16_t*>(t)[i]);
}

__device__ __forceinline__ float wave_sum(float v) {
#pragma unroll
  for (int x = 32; x >= 1; x >>= 1) v += __shfl_xor(v, x);
  return v;
}
__device__ __forceinline__ float wave_max(float v) {
#pragma unroll
  for (int x = 32; x >= 1; x >>= 1) v = nan_max(v, __shfl_xor(v, x));
  return v;
}

// A token's log q over its live entries is t_k / T - shift (a true division:
// t_k / T reaches the loss in full where the teacher's log-sum-exp is given,
// and a rounded reciprocal would add its error to it): shift is the
// teacher's own log-sum-exp, or that of the live entries (0 if none has any
// mass, whose q are then all 0). One wave; `t_of(k)` gives t_k / T, -inf for
// an entry that is not live.
template <class F>
__device__ __forceinline__ float teacher_shift(const float* teacher_lse, int64_t tok, int K, F t_of) {
  if (teacher_lse != nullptr) return teacher_lse[tok];
  const int lane = threadIdx.x & 63;
  float m = -INFINITY;
  for (int k = lane; k < K; k += 64) m = nan_max(m, t_of(k));
  m = wave_max(m);
  if (m == -INFINITY) return 0.0f;
  float s = 0.0f;
  for (int k = lane; k < K; k += 64) s += expf(t_of(k) - m);
  return m + logf(wave_sum(s));
}

// q of one entry: 0 at t = -inf whatever the shift is.
__device__ __forceinline__ float teacher_q(float t, float shift) { return t == -INFINITY ? 0.0f : expf(t - shift); }

// The K dot products W[id_k] . h of a token into s_z: a workgroup's waves take
// them eight at a time. Lane l holds 16-byte chunks l, l + 64, ... of the row;
// one load of h serves eight rows of W.
constexpr int kDotRows = 8;
__device__ __forceinline__ void distill_dots(const DistillTopArgs& a, int64_t tok, int lane, int wave, int n_waves,
                                             float* s_z) {
  const int K = a.K, H = a.H, V = a.V;
  const int32_t* ids = a.ids + tok * K;
  const uint4* h = reinterpret_cast<const uint4*>(a.hidden + tok * H);
  for (int k0 = wave * kDotRows; k0 < K; k0 += n_waves * kDotRows) {
    const uint4* w[kDotRows];
    float acc[kDotRows];
#pragma unroll
    for (int e = 0; e < kDotRows; ++e) {
      int id = ids[min(k0 + e, K - 1)];
      id = (id >= 0 && id < V) ? id : 0;   // a dead entry's dot product is not used
      w[e] = reinterpret_cast<const uint4*>(a.W + (int64_t)id * H);
      acc[e] = 0.0f;
    }
    for (int c = lane; c < H / 8; c += 64) {
      const uint4 x = h[c];
      const uint32_t xs[4] = {x.x, x.y, x.z, x.w};
      uint4 y[kDotRows];
#pragma unroll
      for (int e = 0; e < kDotRows; ++e) y[e] = w[e][c];
#pragma unroll
      for (int e = 0; e < kDotRows; ++e) {
        const uint32_t ys[4] = {y[e].x, y[e].y, y[e].z, y[e].w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          acc[e] = fmaf(__uint_as_float(xs[i] << 16), __uint_as_float(ys[i] << 16), acc[e]);
          acc[e] = fmaf(__uint_as_float(xs[i] & 0xFFFF0000u), __uint_as_float(ys[i] & 0xFFFF0000u), acc[e]);
        }
      }
    }
    // eight sums over 64 lanes: each of the first three steps halves the
    // number of rows a lane still carries, so they cost 7 exchanges and not 24
#pragma unroll
    for (int x = 32, n = 4; n >= 1; x >>= 1, n >>= 1) {
      const bool hi = (lane & x) != 0;
#pragma unroll
      for (int e = 0; e < n; ++e) {
        const float give = hi ? acc[e] : acc[e + n];
        const float keep = hi ? acc[e + n] : acc[e];
        acc[e] = keep + __shfl_xor(give, x);
      }
    }
    float z = acc[0];
#pragma unroll
    for (int x = 4; x >= 1; x >>= 1) z += __shfl_xor(z, x);
    // lane bits 5, 4, 3 now name the row
    const int e = ((lane >> 5) & 1) * 4 + ((lane >> 4) & 1) * 2 + ((lane >> 3) & 1);
    if ((lane & 7) == 0 && k0 + e < K) s_z[k0 + e] = z;
  }
}

// Forward tail, a workgroup per token: the first n_dot waves take the dot
// products, and the last merges the forward's split records and takes the
// teacher's shift, then forms the outputs. Bound by the fetch of the K rows
// of W (2 H bytes each), from the caches where teachers agree on frequent ids:
// 4096 tokens x 64 rows of 5 KB in 120 us (11 TB/s).
__global__ __launch_bounds__(320) void distill_top_kernel(const DistillTopArgs a) {
  __shared__ float s_z[kDistillMaxK];
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int last = (blockDim.x >> 6) - 1;
  const int n_dot = a.n_dot;
  const int K = a.K, V = a.V;
  for (int64_t tok = blockIdx.x; tok < a.N; tok += gridDim.x) {
    const int32_t* ids = a.ids + tok * K;
    auto live_of = [&](int k) { return ids[k] >= 0 && ids[k] < V; };
    auto t_of = [&](int k) { return live_of(k) ? teacher_at(a.teacher, a.t_f32, tok * K + k) / a.T : -INFINITY; };
    float lse = 0.0f, shift = 0.0f, zt = 0.0f;
    if (wave < n_dot) {
      distill_dots(a, tok, lane, wave, n_dot, s_z);
    }
    if (wave == last) {
      // a lane's records in split order, then across lanes by halves (the lower
      // lane's first), so the order is fixed
      Stats rec{kNegBig, 0.0f, 0.0f, 0.0f};
#pragma unroll 4
      for (int s = lane; s < a.S; s += 64) {
        const float4 q = reinterpret_cast<const float4*>(a.part)[s * a.part_ld + tok];
        rec = merge_stats(rec, Stats{q.x, q.y, q.z, q.w});
      }
#pragma unroll
      for (int x = 1; x < 64; x <<= 1) {
        const Stats o{__shfl_xor(rec.m2, x), __shfl_xor(rec.s1, x), __shfl_xor(rec.s2, x), __shfl_xor(rec.zt, x)};
        rec = (lane & x) == 0 ? merge_stats(rec, o) : merge_stats(o, rec);
      }
      // The records are in base 2 of logits scaled by the float32 sc ~ log2(e) / T:
      // back = 1 / (sc T) in two words takes the max back to natural units of z / T
      // without sc's rounding, which a loss of the size of the max's last digits
      // would show. A +inf logit (and no NaN) leaves m = +inf and s1 = NaN.
      lse = rec.m2 == INFINITY ? INFINITY : fmaf(rec.m2, a.back_hi, fmaf(rec.m2, a.back_lo, kLn2 * log2f(rec.s1)));
      zt = rec.zt;
      shift = teacher_shift(a.teacher_lse, tok, K, t_of);
    }
    __syncthreads();
    if (wave == last) {
      float kl = 0.0f;
      bool any = false;
      for (int k = lane; k < K; k += 64) {
        const bool live = live_of(k);
        any |= live;
        const float top = live ? s_z[k] / a.T - lse : 0.0f;
        const float t = t_of(k);
        const float q = teacher_q(t, shift);
        if (q != 0.0f) kl += q * ((t - shift) - top);
        a.logp_top[tok * K + k] = top;
      }
      kl = wave_sum(kl);
      const bool some = __any(any);
      if (lane == 0) {
        const int t = a.targets != nullptr ? a.targets[tok] : -1;
        const bool hard = t >= 0 && t < V;
        a.kl[tok] = kl;
        a.lse[tok] = (hard || some) ? lse : 0.0f;
        if (a.logp != nullptr) a.logp[tok] = hard ? zt / a.T - lse : 0.0f;
      }
    }
    __syncthreads();   // s_z is read before the next token's dot products
  }
}

// Backward, before the tiles. A wave per token forms what the head's tiles
// read (the combined log-prob cotangent and a target id, one of the special
// entries or -1 for a token without any) and the token's special entries:
// (id, cotangent), K + 1 of them, id -1 where there is none. An id
// that the teacher lists twice is formed once, at its first place, with the
// sum of its q in list order: K compares per entry from LDS, K^2 per token
// (4096 tokens, H 256, V 32000: 13 us of 421 at 64 entries, 84 of 485 at 256,
// 1210 of 1642 at 1024).
constexpr int kPrepWaves = 4;
__global__ __launch_bounds__(64 * kPrepWaves) void distill_prep_kernel(const DistillPrepArgs a) {
  extern __shared__ int lds[];   // per wave: the token's K ids (-1 for a missing entry), then its K q
  const int lane = threadIdx.x & 63;
  const int wave = threadIdx.x >> 6;
  const int K = a.K, V = a.V;
  const int64_t prep_blocks = (a.N + kPrepWaves - 1) / kPrepWaves;
  if (blockIdx.x >= prep_blocks) {   // the tiles' counters and padded rows
    const int64_t step = (gridDim.x - prep_blocks) * (int64_t)blockDim.x;
    const int64_t i0 = (blockIdx.x - prep_blocks) * (int64_t)blockDim.x + threadIdx.x;
    for (int64_t i = i0; i < a.n_ctr; i += step) a.ctr[i] = 0;
    const int64_t in = (int64_t)a.tail_rows * a.H / 8, n = a.tail_rows > 0 ? (int64_t)8 * a.H : 0;
    for (int64_t i = i0; i < n; i += step)
      reinterpret_cast<uint4*>(a.tail_out)[i] = i < in ? reinterpret_cast<const uint4*>(a.tail_in)[i] : make_uint4(0u, 0u, 0u, 0u);
    return;
  }
  int* s_id = lds + wave * 2 * K;
  float* s_q = reinterpret_cast<float*>(s_id + K);
  const int64_t tok = min((int64_t)blockIdx.x * kPrepWaves + wave, a.N - 1);   // a wave too many repeats the last token
  const int32_t* ids = a.ids + tok * K;
  const int target = a.targets != nullptr ? a.targets[tok] : -1;
  const bool hard = target >= 0 && target < V;
  const float g_kl = a.g_kl != nullptr ? a.g_kl[tok] : 0.0f;
  const float g_logp = (hard && a.g_logp != nullptr) ? a.g_logp[tok] : 0.0f;
  int first = K;   // the first live entry
  bool listed = false;
  for (int k = lane; k < K; k += 64) {
    const int id = ids[k];
    const bool live = id >= 0 && id < V;
    s_id[k] = live ? id : -1;
    if (live) first = min(first, k);
    listed |= hard && id == target;
  }
#pragma unroll
  for (int x = 32; x >= 1; x >>= 1) first = min(first, __shfl_xor(first, x));
  listed = __any(listed);
  // a token without a cotangent of its loss term, or without an entry, forms
  // none of the term (selected, so a NaN in the teacher's row under g_kl = 0, or
  // in g_kl under an empty row, stays out)
  const bool kd = g_kl != 0.0f && first < K;
  for (int k = lane; k < K; k += 64)
    s_q[k] = s_id[k] >= 0 && kd ? teacher_at(a.teacher, a.t_f32, tok * K + k) / a.T : -INFINITY;
  auto t_of = [&](int k) { return s_q[k]; };   // a lane's own entries: no wait between lanes is needed
  const float shift = kd ? teacher_shift(a.teacher_lse, tok, K, t_of) : 0.0f;
  float Q = 0.0f;
  for (int k = lane; k < K; k += 64) {
    const float q = teacher_q(s_q[k], shift);
    s_q[k] = q;
    Q += q;
  }
  Q = wave_sum(Q);
  const float gQ = kd ? g_kl * Q : 0.0f;
  __syncthreads();   // every lane's ids and q are read below
  auto cotangent = [&](float s, float q, bool is_target) {
    const float p = expf(s);
    float x = 0.0f;
    if (p != 0.0f) x = (kd ? g_kl * fmaf(Q, p, -q) : 0.0f) - g_logp * p;   // an entry of probability 0 has no such term
    else if (kd) x = -g_kl * q;
    return (is_target ? x + g_logp : x) * a.invT;
  };
  int32_t* e_id = a.ent_id + tok * (K + 1);
  float* e_val = a.ent_val + tok * (K + 1);
  for (int k = lane; k < K; k += 64) {
    const int id = s_id[k];
    int out = id;
    float q = 0.0f;
#pragma unroll 4
    for (int j = 0; j < K; ++j) {
      if (s_id[j] == id) {
        if (j < k) out = -1;
        q += s_q[j];
      }
    }
    e_id[k] = out;
    e_val[k] = out >= 0 ? cotangent(a.logp_top[tok * K + k], q, hard && id == target) : 0.0f;
  }
  if (lane == 0) {
    const bool extra = hard && !listed;
    e_id[K] = extra ? target : -1;
    e_val[K] = extra ? cotangent(a.logp != nullptr ? a.logp[tok] : 0.0f, 0.0f, true) : 0.0f;
    a.tgt[tok] = hard ? target : (first < K ? s_id[first] : -1);
    a.ga[tok] = g_logp - gQ;
  }
}

// dh tile of one split of the block's vocabulary: the head's dh tile over K =
// [k0, k0 + k_split) of it, written to its own float32 partial [Ct][H].
__device__ __forceinline__ void dh_split_tile(const DistillStep& d, int vid, char* lds) {
  const BwdStep& s = d.step;
  const int split = vid / s.n_dh;
  int mt, hb;
  raster(vid - split * s.n_dh, s.n_dh / s.n_ht, s.n_ht, 4, mt, hb);
  const int wave = threadIdx.x >> 6;
  const int wm = wave & 1;
  const int wn = wave >> 1;
  const int m0 = mt * kTile;
  const int h0 = hb * kTile;
  const int H = s.H;
  const int k0 = split * d.k_split;
  const int K = min(d.k_split, (s.g_Vb + kBK - 1) / kBK * kBK - k0);   // > 0: the host counts the splits
  // negative where the block's last slice lies in another split
  const int tail_k = s.W_tail != nullptr ? s.v_tail - s.g_v0 - k0 : -1;
  const Operand oa{s.W + (int64_t)(s.g_v0 + k0) * H + h0, H, min(kTile, H - h0),
                   s.W_tail != nullptr ? s.W_tail + h0 : nullptr, tail_k};
  const Operand ob{s.g_dz + (int64_t)m0 * s.ld_dz + k0, s.ld_dz, kTile};
  f32x4 acc[kNB][kNB];
  Pipe pipe;
  mma_tile<true, 64>(oa, ob, K, lds, acc, pipe, oa.base, ob.base, false);
  write_acc_t(d.part + (int64_t)split * s.g_Ct * H, H, h0 + wm * 128, H, m0 + wn * 128, s.g_Ct, false, s.targets, s.g_t0,
              s.Vtot, acc);
}

// Write one wave's 128 x 128 block of a dW tile as bf16 rows of H, through the
// (by then idle) slice ring, 64 rows at a time: a lane holds 4 rows of 16
// columns each, which as they lie take 256 stores of 2 bytes; turned they take
// 32 of 16 bytes, each covering 4 rows x 256 bytes.
constexpr int kTurnPitch = 256 + 16;
static_assert(4 * 64 * kTurnPitch <= kRingBytes, "staging fits in the slice ring");
__device__ __forceinline__ void write_acc_turned(uint16_t* __restrict__ out, int64_t ld, int r_base, int rows, int c_base,
                                                 int cols, char* lds, f32x4 (&acc)[kNB][kNB]) {
  const int lane = threadIdx.x & 63;
  char* mine = lds + wave_id() * 64 * kTurnPitch;
#pragma unroll
  for (int half = 0; half < 2; ++half) {
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int j = 0; j < kNB; ++j) {
        pin_acc(acc[4 * half + i][j]);
#pragma unroll
        for (int r = 0; r < 4; ++r)
          *reinterpret_cast<uint16_t*>(mine + acc_row(i, r, lane) * kTurnPitch + 2 * (16 * j + (lane & 15))) =
              round_bf16(acc[4 * half + i][j][r]);
      }
    wave_order();
#pragma unroll
    for (int q = 0; q < 16; ++q) {
      const int r = 4 * q + (lane >> 4);
      const uint4 v = *reinterpret_cast<const uint4*>(mine + r * kTurnPitch + 16 * (lane & 15));
      const int row = r_base + 64 * half + r, col = c_base + 8 * (lane & 15);
      if (row < rows && col < cols) *reinterpret_cast<uint4*>(out + (int64_t)row * ld + col) = v;
    }
    wave_order();   // the second half overwrites what the lanes have read
    __builtin_amdgcn_sched_barrier(0);
  }
}

// dW tile: the head's, with the writer above where a gradient's only block is
// written as bf16.
template <bool BF16>
__device__ __forceinline__ void dw_tile_turned(const BwdStep& s, int vid, char* lds) {
  int mt, hb;
  raster(vid, s.n_dw / s.n_ht, s.n_ht, 4, mt, hb);
  const int wave = threadIdx.x >> 6;
  const int wm = wave & 1;
  const int wn = wave >> 1;
  const int m0 = mt * kTile;
  const int h0 = hb * kTile;
  const int H = s.H;
  const Operand oa{s.g_dz + m0, s.ld_dz, kTile};
  const Operand ob{s.ht + (int64_t)h0 * s.ld_ht + s.g_t0, s.ld_ht, kTile};
  f32x4 acc[kNB][kNB];
  Pipe pipe;
  mma_tile<true, 64>(oa, ob, (s.g_Ct + kBK - 1) / kBK * kBK, lds, acc, pipe, oa.base, ob.base, false);
  if (s.o_dW.src_kind == kSrcNone && s.o_dW.dst_bf16) {
    write_acc_turned(static_cast<uint16_t*>(s.o_dW.dst), H, m0 + wm * 128, s.g_Vb, h0 + wn * 128, H, lds, acc);
  } else {
    write_acc_g(s.o_dW, H, m0 + wm * 128, s.g_Vb, h0 + wn * 128, H, acc);
  }
}

// dW tile of one split of the block's tokens, to its own float32 partial [Vb][H].
__device__ __forceinline__ void dw_split_tile(const DistillStep& d, int vid, char* lds) {
  const BwdStep& s = d.step;
  const int split = vid / s.n_dw;
  int mt, hb;
  raster(vid - split * s.n_dw, s.n_dw / s.n_ht, s.n_ht, 4, mt, hb);
  const int wave = threadIdx.x >> 6;
  const int wm = wave & 1;
  const int wn = wave >> 1;
  const int m0 = mt * kTile;
  const int h0 = hb * kTile;
  const int H = s.H;
  const int k0 = split * d.w_k_split;
  const int K = min(d.w_k_split, (s.g_Ct + kBK - 1) / kBK * kBK - k0);   // > 0: the host counts the splits
  const Operand oa{s.g_dz + (int64_t)k0 * s.ld_dz + m0, s.ld_dz, kTile};
  const Operand ob{s.ht + (int64_t)h0 * s.ld_ht + s.g_t0 + k0, s.ld_ht, kTile};
  f32x4 acc[kNB][kNB];
  Pipe pipe;
  mma_tile<true, 64>(oa, ob, K, lds, acc, pipe, oa.base, ob.base, false);
  write_acc(d.w_part + (int64_t)split * s.g_Vb * H, H, m0 + wm * 128, s.g_Vb, h0 + wn * 128, H, false, nullptr, 0, 0, acc);
}

// One backward launch: the head's (each XCD an eighth of the gradient tiles,
// the kind with the longer K first, then of the next block's cotangent tiles,
// the last off per-XCD counters and then off the others'), with the dW writer
// above, and with SPLIT the gradient tiles' K split: where a few tiles would
// otherwise run a whole vocabulary, or many tokens, in sequence while the chip
// idles. Bound by the matrix units: 4096 tokens, H 2560, V 151936 run at 1,360
// to 1,390 TFLOP/s in the middle launches (764 to 782 us each).
template <bool BF16, bool SPLIT>
__global__ __launch_bounds__(kThreads) void distill_step_kernel(const DistillStep d) {
  __shared__ __attribute__((aligned(16))) char lds[kLdsBytes];
  __shared__ int z_tile;
  const BwdStep& s = d.step;
  const int xcd = blockIdx.x & 7;
  const int loc = blockIdx.x >> 3;
  const int n_dh = s.n_dh * d.splits;
  const int n_dw = s.n_dw * d.w_splits;
  const int dw_lo = xcd * n_dw / 8;
  const int dw_cnt = (xcd + 1) * n_dw / 8 - dw_lo;
  const int dh_lo = xcd * n_dh / 8;
  const int dh_cnt = (xcd + 1) * n_dh / 8 - dh_lo;
  // dh tiles run K = Vb, dW tiles K = Ct, or a split of it
  const bool dh_first = SPLIT ? d.k_split > d.w_k_split : s.g_Vb > s.g_Ct;
  const int first_cnt = dh_first ? dh_cnt : dw_cnt;
  if (loc < dh_cnt + dw_cnt) {
    if ((loc < first_cnt) == dh_first) {
      const int vid = dh_lo + (dh_first ? loc : loc - dw_cnt);
      if constexpr (SPLIT) dh_split_tile(d, vid, lds);
      else dh_tile<BF16>(s, vid, lds);
    } else {
      const int vid = dw_lo + (dh_first ? loc - dh_cnt : loc);
      if (SPLIT && d.w_splits > 1) dw_split_tile(d, vid, lds);
      else if constexpr (BF16) dw_tile_turned<BF16>(s, vid, lds);
      else dw_tile<BF16>(s, vid, lds);
    }
    return;
  }
  const int n_z = s.z_ntt * s.z_nvt;
  if (n_z == 0) return;
  if (threadIdx.x == 0) z_tile = take_z_tile(s, xcd, n_z);
  __syncthreads();
  const int tile = z_tile;
  if (tile >= 0) dz_tile(s, tile, lds);
}

// Adds up the splits of a gradient's block in split order, onto what o reads
// and to where it writes (as the bf16-gradient backward's writers take it);
// with tgt a masked token's row is written as 0, or left as it is.
__device__ __forceinline__ void sum_splits(const SplitSum& a, int H, const int32_t* tgt, int V, bool dead_zero, int64_t i0,
                                           int64_t step) {
  const int h4 = H / 4;
  const int64_t n4 = (int64_t)a.rows * h4;
  for (int64_t i = i0; i < n4; i += step) {
    bool live = true;
    if (tgt != nullptr) {
      const int t = tgt[i / h4];
      live = t >= 0 && t < V;
      if (!live && !dead_zero) continue;
    }
    f32x4 v = {0.0f, 0.0f, 0.0f, 0.0f};
    if (live) {
      const f32x4* p = reinterpret_cast<const f32x4*>(a.part) + i;
      v = p[0];
#pragma unroll 8
      for (int k = 1; k < a.splits; ++k) v += p[k * n4];
      if (a.o.src_kind == kSrcF32) {
        v += static_cast<const f32x4*>(a.o.src)[i];
      } else if (a.o.src_kind == kSrcBf16) {
        const uint2 w = static_cast<const uint2*>(a.o.src)[i];
        v += f32x4{__uint_as_float(w.x << 16), __uint_as_float(w.x & 0xFFFF0000u), __uint_as_float(w.y << 16),
                   __uint_as_float(w.y & 0xFFFF0000u)};
      }
    }
    if (a.o.dst_bf16) {
      uint2 w;
      w.x = pack_bf16x2(v[0], v[1]);
      w.y = pack_bf16x2(v[2], v[3]);
      static_cast<uint2*>(a.o.dst)[i] = w;
    } else {
      static_cast<f32x4*>(a.o.dst)[i] = v;
    }
  }
}

// After each launch, on what it wrote: overwrites the special entries of tokens
// [t0, t0 + Ct) and vocabulary rows [v0, v0 + Vb) in their cotangent block, and
// adds up the splits of the gradients' blocks. A scatter of 2 bytes each into a
// block that the caches hold: 4.9 us a launch at 512 chunk x 4096 tokens x 64
// entries, a launch of its own, since every tile of the block comes before it.
__global__ __launch_bounds__(256) void distill_post_kernel(const DistillPostArgs a) {
  const int64_t step = (int64_t)gridDim.x * 256;
  const int64_t i0 = (int64_t)blockIdx.x * 256 + threadIdx.x;
  const int64_t n = a.dz != nullptr ? (int64_t)a.Ct * a.K1 : 0;
  for (int64_t i = i0; i < n; i += step) {
    const int64_t at = (int64_t)a.t0 * a.K1 + i;
    const int id = a.ent_id[at];
    const int v = id - a.v0;
    if (id >= 0 && v >= 0 && v < a.Vb) a.dz[i / a.K1 * a.ld_dz + v] = round_bf16(a.ent_val[at]);
  }
  if (a.dh.part != nullptr) sum_splits(a.dh, a.H, a.tgt, a.V, a.dead_zero != 0, i0, step);
  if (a.dW.part != nullptr) sum_splits(a.dW, a.H, nullptr, 0, false, i0, step);
}

}  // namespace

hipError_t launch_distill_top(DistillTopArgs a, hipStream_t stream) {
  a.n_dot = std::max(1, std::min(4, (a.K + kDotRows - 1) / kDotRows));
  // a wave of its own for the last wave's part while every workgroup is
  // resident at once and latency counts (1 token: 9.8 us instead of 14.4);
  // beyond, the waves are better spent on more tokens (4096: 200 us instead of 120)
  const int waves = a.n_dot + (a.N <= 2 * kNumCUs ? 1 : 0);
  const double N = (double)a.N, K = (double)a.K, H = (double)a.H;
  trace_begin(stream);
  hipLaunchKernelGGL(distill_top_kernel, dim3((unsigned)std::min<int64_t>(a.N, 1 << 20)), dim3(64 * waves), 0, stream, a);
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  trace_end(kDistillTop, stream, 2.0 * N * K * H, 2.0 * N * (K + 1) * H + N * K * (8 + (a.t_f32 ? 4 : 2)) + 32.0 * N);
  return hipSuccess;
}

hipError_t launch_distill_prep(const DistillPrepArgs& a, hipStream_t stream) {
  const double N = (double)a.N, K = (double)a.K;
  trace_begin(stream);
  const int64_t rest = std::max<int64_t>(a.n_ctr, a.tail_rows > 0 ? (int64_t)8 * a.H : 0);
  const int64_t blocks = (a.N + kPrepWaves - 1) / kPrepWaves + std::min<int64_t>((rest + 255) / 256, 256);
  hipLaunchKernelGGL(distill_prep_kernel, dim3((unsigned)blocks), dim3(64 * kPrepWaves),
                     (size_t)kPrepWaves * 2 * a.K * 4, stream, a);
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  trace_end(kDistillPrep, stream, 0.0, N * K * (14 + (a.t_f32 ? 4 : 2)) + 24.0 * N);
  return hipSuccess;
}

template <bool BF16, bool SPLIT>
static hipError_t launch_step(const DistillStep& d, hipStream_t stream) {
  const BwdStep& st = d.step;
  const int n_z = st.z_ntt * st.z_nvt, n_dh = st.n_dh * d.splits, n_dw = st.n_dw * d.w_splits;
  int per = 0;
  for (int x = 0; x < 8; ++x)
    per = std::max(per, ((x + 1) * n_dw / 8 - x * n_dw / 8) + ((x + 1) * n_dh / 8 - x * n_dh / 8) +
                            ((x + 1) * n_z / 8 - x * n_z / 8) + (n_z > 0 ? kStealSlots : 0));
  if (per == 0) return hipSuccess;
  const int n_g = st.n_dw + st.n_dh;
  const double H = (double)st.H;
  const double gc = (double)st.g_Ct, gv = (double)st.g_Vb, zc = (double)st.z_Ct, zv = (double)st.z_Vb;
  trace_begin(stream);
  hipLaunchKernelGGL((distill_step_kernel<BF16, SPLIT>), dim3(8 * per), dim3(kThreads), 0, stream, d);
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  trace_end(kDistillStep, stream, n_g ? 4.0 * gc * gv * H : 0.0,
            (n_g ? 2.0 * gc * gv + 2.0 * (gc + gv) * H + 4.0 * H * (gc * d.splits + gv * d.w_splits) : 0.0) +
                (n_z ? 2.0 * zc * zv + 2.0 * (zc + zv) * H + 20.0 * zc : 0.0));
  return hipSuccess;
}

hipError_t launch_distill_step(const DistillStep& d, bool bf16, hipStream_t stream) {
  if (d.part == nullptr) return bf16 ? launch_step<true, false>(d, stream) : launch_bwd_step(d.step, stream);
  return bf16 ? launch_step<true, true>(d, stream) : launch_step<false, true>(d, stream);
}

hipError_t launch_distill_post(const DistillPostArgs& a, hipStream_t stream) {
  const int64_t n = a.dz != nullptr ? (int64_t)a.Ct * a.K1 : 0;
  auto n4 = [&](const SplitSum& x) { return x.part != nullptr ? (int64_t)x.rows * (a.H / 4) : (int64_t)0; };
  const int64_t most = std::max(n, std::max(n4(a.dh), n4(a.dW)));
  if (most == 0) return hipSuccess;
  trace_begin(stream);
  hipLaunchKernelGGL(distill_post_kernel, dim3((unsigned)std::min<int64_t>((most + 255) / 256, 4096)), dim3(256), 0, stream, a);
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  trace_end(kDistillPost, stream, 0.0, 4.0 * (double)n + 16.0 * ((double)n4(a.dh) * (a.dh.splits + 1) + (double)n4(a.dW) * (a.dW.splits + 1)));
  return hipSuccess;
}

}  // namespace lmh
