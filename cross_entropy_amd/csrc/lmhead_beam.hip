// lmhead_beam.hip -- one step of beam search on the head's never-stored logits,
// and the reordering of the beams' states, for gfx950.
//
// With z = W h_r / T and lse_r = log sum exp z over the whole vocabulary, the
// candidates of a group of G beams are s_r + z_v - lse_r over its rows r and
// the words v that row r may take; the C best come out, equal ones by the
// lowest row and then the lowest word. The [rows, vocab] logits are never held:
//
//   logits  the head's tiles (or, for few rows, the streaming ones) keep the
//           log-sum-exp records and, of every 16 words, the largest logit that
//           is allowed, and of every section of such blocks the largest
//   select  a workgroup per group merges the records and takes the best
//           sections, then the best blocks of those: a candidate among the C
//           best lies in one of the C best blocks (each block before its own
//           holds a candidate before it)
//   score   the chosen blocks' logits once more, in 64 bits: the choice is then
//           free of the order of the tiles' float32 sums, which differs between
//           kernels and would decide between near candidates. kSpare blocks
//           more than C are looked at where their float32 maxima lie within
//           that error. The last workgroup of a group ranks its candidates.
//
// A row's log-sum-exp is the float32 one, corrected by what the 64-bit logit of
// its best candidate changes, which holds most of its mass as a rule. By that
// one alone, whatever else is chosen of the row: rows that are alike then keep
// scores that are alike, and ties between them are seen.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include <algorithm>

#include "lmhead_few.h"
#include "lmhead_internal.h"
#include "lmhead_tile.h"

namespace lmh {
namespace {

__device__ __forceinline__ float max_drop(float a, float b) { return fmaxf(a, b); }   // a NaN row is dropped by its log-sum-exp

// The bits of the 16 words from v (a multiple of 16) on that row tok may take.
__device__ __forceinline__ uint32_t allowed16(const BeamArgs& a, int64_t tok, int v) {
  return (uint32_t)a.allowed[tok * a.mask_ld + (v >> 5)] >> (v & 16);
}

// Few rows: the workgroup's 64 MB vocabulary rows, one record and one section.
template <int MB, int NB, bool MASK>
__global__ __launch_bounds__(256, 2) void beam_few_kernel(const FewArgs a, const BeamArgs b) {
  __shared__ __attribute__((aligned(16))) char lds[few_lds<NB>()];
  __shared__ float4 xch[4][16 * NB];
  const int lane = threadIdx.x & 63;
  const int wave = wave_id();
  const FewTile t = few_tile(a, xcd_remap(blockIdx.x, gridDim.x), a.splits);
  if (t.split < 0) return;
  const int r0 = (t.split * 4 + wave) * 16 * MB;
  const int V = a.V;
  const int q = lane >> 4;
  f32x4 acc[MB][NB];
  few_logits_of<MB, NB>(a, t, r0, lds, acc);
  float m2[NB], s1[NB], top[NB];
#pragma unroll
  for (int j = 0; j < NB; ++j) {
    const int tok = 16 * j + (lane & 15);
    const int at = t.tok0 + min(tok, t.n - 1);
    float mx = kNegBig;
    top[j] = -INFINITY;
#pragma unroll
    for (int i = 0; i < MB; ++i) {
      float best = -INFINITY;
      const int v0 = r0 + 16 * i;
      uint32_t bits = 0xFFFFu;
      if (MASK && v0 < V) bits = allowed16(b, at, v0);
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        const int row = v0 + 4 * q + r;
        if (row < V) {
          mx = nan_max(mx, acc[i][j][r]);
          if (!MASK || ((bits >> (4 * q + r)) & 1)) best = max_drop(best, acc[i][j][r]);
        }
      }
      best = max_drop(best, __shfl_xor(best, 16));
      best = max_drop(best, __shfl_xor(best, 32));
      if (q == 0 && v0 < V && tok < t.n) b.blocks[(int64_t)(v0 >> 4) * b.ld + t.tok0 + tok] = best;
      top[j] = max_drop(top[j], best);
    }
    const float m = nan_max(kNegBig, mx * a.sc);
    float s = 0.0f;
#pragma unroll
    for (int i = 0; i < MB; ++i)
#pragma unroll
      for (int r = 0; r < 4; ++r) s += r0 + acc_row(i, r, lane) < V ? fast_exp2(fmaf(acc[i][j][r], a.sc, -m)) : 0.0f;
    m2[j] = m;
    s1[j] = s;
  }
#pragma unroll
  for (int x = 16; x <= 32; x <<= 1)
#pragma unroll
    for (int j = 0; j < NB; ++j) {
      const float om = __shfl_xor(m2[j], x), os = __shfl_xor(s1[j], x);
      const float m = nan_max(m2[j], om);
      const float mine = s1[j] * fast_exp2(m2[j] - m), other = os * fast_exp2(om - m);
      m2[j] = m;
      s1[j] = mine + other;
    }
  if (lane < 16) {
#pragma unroll
    for (int j = 0; j < NB; ++j) xch[wave][16 * j + lane] = make_float4(m2[j], s1[j], top[j], 0.0f);
  }
  __syncthreads();
  const int tok = threadIdx.x;
  if (tok < 16 * NB && tok < t.n) {
    float4 p = xch[0][tok];
#pragma unroll
    for (int w = 1; w < 4; ++w) {
      const float4 o = xch[w][tok];
      const float m = nan_max(p.x, o.x);
      p.y = p.y * fast_exp2(p.x - m) + o.y * fast_exp2(o.x - m);
      p.x = m;
      p.z = max_drop(p.z, o.z);
    }
    b.records[(int64_t)t.split * b.ld + t.tok0 + tok] = make_float2(p.x, p.y);
    b.sections[(int64_t)t.split * b.ld + t.tok0 + tok] = p.z;
  }
}

// Many rows: the head's forward tiles; a section is a wave's 128 vocabulary rows.
template <bool MASK>
__global__ __launch_bounds__(kThreads) void beam_tile_kernel(const BeamArgs b) {
  __shared__ __attribute__((aligned(16))) char lds[kLdsBytes];
  const int vid = xcd_remap(blockIdx.x, gridDim.x);
  const int S = b.splits;
  if (vid >= b.n_tt * S) return;
  const int tt = vid / S;
  const int s = vid - tt * S;
  const int lane = threadIdx.x & 63;
  const int wave = threadIdx.x >> 6;
  const int wm = wave & 1;
  const int wn = wave >> 1;
  const int q = lane >> 4;
  const int tok0 = tt * kTile;
  const int N = b.N, H = b.H, V = b.V;
  const float sc = b.sc;
  float m2[kNB], s1[kNB];
#pragma unroll
  for (int j = 0; j < kNB; ++j) m2[j] = kNegBig, s1[j] = 0.0f;
  const Operand ob{b.hidden + (int64_t)tok0 * H, H, min(kTile, N - tok0)};
  Pipe pipe;
  for (int vt = s; vt < b.n_vt; vt += S) {
    const int v0 = vt * kTile;
    const Operand oa{b.W + (int64_t)v0 * H, H, min(kTile, V - v0)};
    const int v1 = v0 + S * kTile;
    const bool more = vt + S < b.n_vt && min(kTile, V - v1) == oa.rows;
    f32x4 acc[kNB][kNB];
    mma_tile<false, 96>(oa, ob, H, lds, acc, pipe, b.W + (int64_t)(more ? v1 : v0) * H, ob.base, more);
    const int vrow0 = v0 + wm * 128;
    const bool ragged = vrow0 + 128 > V;
#pragma unroll
    for (int j = 0; j < kNB; ++j) {
      const int tok = tok0 + wn * 128 + j * 16 + (lane & 15);
      uint32_t words[4] = {~0u, ~0u, ~0u, ~0u};
      if (MASK) {
        const int32_t* row = b.allowed + (int64_t)min(tok, N - 1) * b.mask_ld;
#pragma unroll
        for (int w = 0; w < 4; ++w) words[w] = (uint32_t)row[min((vrow0 >> 5) + w, (int)b.mask_ld - 1)];
      }
      float z[kNB][4];
#pragma unroll
      for (int i = 0; i < kNB; ++i) {
        pin_acc(acc[i][j]);
#pragma unroll
        for (int r = 0; r < 4; ++r) z[i][r] = acc[i][j][r];
      }
      if (ragged) {   // rows past V take no part
#pragma unroll
        for (int i = 0; i < kNB; ++i)
#pragma unroll
          for (int r = 0; r < 4; ++r) z[i][r] = (vrow0 + acc_row(i, r, lane) < V) ? z[i][r] : kNegBig;
      }
      float mx = z[0][0], top = -INFINITY;
      float best[kNB];
#pragma unroll
      for (int i = 0; i < kNB; ++i) {
        best[i] = -INFINITY;
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          mx = nan_max(mx, z[i][r]);
          bool in = !ragged || vrow0 + acc_row(i, r, lane) < V;
          if (MASK) in = in && ((words[i >> 1] >> (16 * (i & 1) + 4 * q + r)) & 1);
          best[i] = max_drop(best[i], in ? z[i][r] : -INFINITY);
        }
        best[i] = max_drop(best[i], __shfl_xor(best[i], 16));
        best[i] = max_drop(best[i], __shfl_xor(best[i], 32));
        top = max_drop(top, best[i]);
        const int vb = vrow0 + 16 * i;
        if (q == (i & 3) && vb < V && tok < N) b.blocks[(int64_t)(vb >> 4) * b.ld + tok] = best[i];
      }
      if (q == 0 && vrow0 < V && tok < N) b.sections[(int64_t)(vrow0 >> 7) * b.ld + tok] = top;
      const float mnew = nan_max(m2[j], mx * sc);
      float e = s1[j] * fast_exp2(m2[j] - mnew);
#pragma unroll
      for (int i = 0; i < kNB; ++i)
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          const float x = fast_exp2(fmaf(z[i][r], sc, -mnew));
          e += !ragged || vrow0 + acc_row(i, r, lane) < V ? x : 0.0f;
        }
      m2[j] = mnew;
      s1[j] = e;
      __builtin_amdgcn_sched_barrier(0);
    }
  }
#pragma unroll
  for (int x = 16; x <= 32; x <<= 1)
#pragma unroll
    for (int j = 0; j < kNB; ++j) {
      const float om = __shfl_xor(m2[j], x), os = __shfl_xor(s1[j], x);
      const float m = nan_max(m2[j], om);
      const float mine = s1[j] * fast_exp2(m2[j] - m), other = os * fast_exp2(om - m);
      m2[j] = m;
      s1[j] = mine + other;
    }
  float2* xch = reinterpret_cast<float2*>(lds);
  if (wm == 1 && lane < 16) {
#pragma unroll
    for (int j = 0; j < kNB; ++j) xch[(wn * kNB + j) * 16 + lane] = make_float2(m2[j], s1[j]);
  }
  __syncthreads();
  if (wm == 0 && lane < 16) {
#pragma unroll
    for (int j = 0; j < kNB; ++j) {
      const float2 o = xch[(wn * kNB + j) * 16 + lane];
      const float m = nan_max(m2[j], o.x);
      const int tok = tok0 + wn * 128 + j * 16 + lane;
      if (tok < N) b.records[(int64_t)s * b.ld + tok] = make_float2(m, s1[j] * fast_exp2(m2[j] - m) + o.y * fast_exp2(o.x - m));
    }
  }
}

// ---------------------------------------------------------------------------
// Keys: a float's order as an unsigned number, above the complement of its
// index, so that larger keys are better candidates and no two are equal.
__device__ __forceinline__ uint64_t key_of(float v, uint32_t index) {
  const uint32_t u = __float_as_uint(v);
  const uint32_t o = (u & 0x80000000u) ? ~u : (u | 0x80000000u);
  return ((uint64_t)o << 32) | (uint32_t)~index;
}
__device__ __forceinline__ float value_of(uint64_t key) {
  const uint32_t o = (uint32_t)(key >> 32);
  return __uint_as_float((o & 0x80000000u) ? (o & 0x7FFFFFFFu) : ~o);
}
__device__ __forceinline__ uint32_t index_of(uint64_t key) { return ~(uint32_t)key; }

constexpr int kSelThreads = 1024;
constexpr int kSelItems = 16;                                 // items of a thread at once
constexpr int kSelList = 4 * kSelItems * kMostKept + kMostKept;   // candidates that can pass the threshold, and those kept

// The `keep` largest keys of items 0 .. n - 1 into list[0 ..], sorted; returns
// how many there are. get(i) gives an item's key, 0 for none. Each group of
// four threads has a largest key, and the keep-th largest of those 256 is a
// threshold that at least `keep` items reach, and few more do.
struct Selection {
  uint64_t list[kSelList];
  uint64_t kept[kMostKept];
  uint64_t most[kSelThreads / 4];
  uint64_t limit;
  int count;
};
template <class F>
__device__ __forceinline__ int select_best(Selection& s, uint32_t n, int keep, F get) {
  const int tid = threadIdx.x;
  int have = 0;
  for (uint32_t base = 0; base < n; base += kSelThreads * kSelItems) {
    uint64_t key[kSelItems], most = 0;
#pragma unroll
    for (int k = 0; k < kSelItems; ++k) {
      const uint32_t i = base + tid + kSelThreads * k;
      key[k] = i < n ? get(i) : 0;
    }
#pragma unroll
    for (int k = 0; k < kSelItems; ++k) most = max(most, key[k]);
    most = max(most, (uint64_t)__shfl_xor((unsigned long long)most, 1));
    most = max(most, (uint64_t)__shfl_xor((unsigned long long)most, 2));
    if ((tid & 3) == 0) s.most[tid >> 2] = most;
    if (tid == 0) {
      s.limit = 0;
      s.count = have;
    }
    __syncthreads();
    if (tid < kSelThreads / 4) {
      const uint64_t mine = s.most[tid];
      int rank = 0;
#pragma unroll 8
      for (int k = 0; k < kSelThreads / 4; ++k) rank += s.most[k] > mine;
      if (rank == keep - 1) s.limit = mine;   // keys differ, so one has this rank, or (all zeros behind it) the limit stays 0
    }
    __syncthreads();
    uint64_t limit = max(s.limit, (uint64_t)1);
    if (have == keep) limit = max(limit, s.kept[keep - 1]);
    if (tid < have) s.list[tid] = s.kept[tid];
#pragma unroll
    for (int k = 0; k < kSelItems; ++k)
      if (key[k] >= limit) s.list[atomicAdd(&s.count, 1)] = key[k];
    __syncthreads();
    const int found = s.count;
    for (int i = tid; i < found; i += kSelThreads) {
      const uint64_t mine = s.list[i];
      int rank = 0;
      for (int k = 0; k < found; ++k) rank += s.list[k] > mine;
      if (rank < keep) s.kept[rank] = mine;
    }
    have = min(found, keep);
    __syncthreads();
  }
  return have;
}

__device__ __forceinline__ double wave_sum(double v) {
#pragma unroll
  for (int x = 32; x >= 1; x >>= 1) v += __shfl_xor(v, x);
  return v;
}

// A row that takes part: neither given up (a score that is not finite) nor ended.
__device__ __forceinline__ bool ended_row(const BeamArgs& b, int64_t tok) {
  return b.ended != nullptr && b.ended[tok] >= 0 && b.ended[tok] < b.V;
}
__device__ __forceinline__ bool finite(double v) { return fabs(v) < INFINITY; }

__global__ __launch_bounds__(kSelThreads) void beam_select_kernel(const BeamArgs b) {
  __shared__ Selection sel;
  __shared__ double base[kMostBeams];
  __shared__ float shift[kMostBeams], size[kMostBeams];
  __shared__ uint32_t section[kMostKept];
  __shared__ double ref;
  __shared__ float slack;
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int64_t group = blockIdx.x, row0 = group * b.beams;
  const int G = b.beams;
  for (int r = wave; r < G; r += kSelThreads / 64) {
    const int64_t tok = row0 + r;
    float m = kNegBig;
    for (int s = lane; s < b.splits; s += 64) m = nan_max(m, b.records[s * b.ld + tok].x);
#pragma unroll
    for (int x = 32; x >= 1; x >>= 1) m = nan_max(m, __shfl_xor(m, x));
    double sum = 0.0;
    for (int s = lane; s < b.splits; s += 64) {
      const float2 p = b.records[s * b.ld + tok];
      sum += (double)p.y * exp2((double)p.x - (double)m);
    }
    sum = wave_sum(sum);
    if (lane == 0) {
      const float score = b.scores[tok];
      // records are in base 2 of logits scaled by the float32 sc: back = 1 / (sc T) undoes both
      const double lse = m == INFINITY ? INFINITY : (double)m * b.back + log(sum);
      const bool part = finite(score) && !ended_row(b, tok);
      const bool live = part && finite(lse);
      base[r] = live ? (double)score - lse : -INFINITY;
      size[r] = live ? (float)((double)m * b.back) : 0.0f;
      b.lse64[tok] = lse;
      b.lse[tok] = part ? (float)lse : 0.0f;
    }
  }
  __syncthreads();
  if (tid == 0) {
    double best = -INFINITY;
    float most = 0.0f;
    for (int r = 0; r < G; ++r) {
      if (!finite(base[r])) continue;
      best = max(best, base[r] + (double)size[r]);
      most = max(most, fabsf(size[r]));
    }
    ref = best;
    slack = (most + b.invT) * 0x1p-13f;   // far more than the tiles' sums are off
  }
  __syncthreads();
  // values relative to about the best candidate, where float32 is finest
  if (tid < G) shift[tid] = finite(base[tid]) ? (float)(base[tid] - ref) : -INFINITY;
  __syncthreads();
  const int keep = b.keep;
  const uint32_t n_sec = (uint32_t)b.n_sections;   // beams * V stays below 2^31
  auto key = [&](float z, int r, uint32_t index) {
    const float x = shift[r];
    return x > -INFINITY && z > -INFINITY ? key_of(fmaf(z, b.invT, x), index) : (uint64_t)0;
  };
  const int n1 = select_best(sel, n_sec * G, keep, [&](uint32_t i) {
    const uint32_t s = i / (uint32_t)G, r = i - s * (uint32_t)G;
    return key(b.sections[(int64_t)s * b.ld + row0 + r], r, r * n_sec + s);
  });
  if (tid < n1) section[tid] = index_of(sel.kept[tid]);
  __syncthreads();
  const uint32_t per = b.per_section, n_blocks = (uint32_t)b.n_blocks;
  const int n2 = select_best(sel, (uint32_t)n1 * per, keep, [&](uint32_t i) {
    const uint32_t at = section[i / per];
    const uint32_t r = at / n_sec, blk = (at - r * n_sec) * per + i % per;
    return blk < n_blocks ? key(b.blocks[(int64_t)blk * b.ld + row0 + r], r, r * n_blocks + blk) : (uint64_t)0;
  });
  if (tid < n2) b.chosen[group * kMostKept + tid] = index_of(sel.kept[tid]);
  if (tid == 0) {
    int used = min(n2, b.C);
    while (used < n2 && value_of(sel.kept[used]) >= value_of(sel.kept[b.C - 1]) - slack) ++used;
    b.used[group] = used;
    b.ticket[group] = 0;
  }
}

// A workgroup per chosen block: its 16 logits in 64 bits. The last one of the
// group ranks the candidates.
constexpr int kScoreThreads = 256;
constexpr int kMostFound = 16 * kMostKept + kMostBeams;
__global__ __launch_bounds__(kScoreThreads) void beam_score_kernel(const BeamArgs b) {
  __shared__ double z_max[kMostKept], logsum[kMostBeams];
  __shared__ double value[kMostFound];
  __shared__ uint32_t index[kMostFound];
  __shared__ double limit;
  __shared__ int count, last;
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int64_t group = blockIdx.x / b.keep, row0 = group * b.beams;
  const int used = b.used[group];
  const int k = (int)(blockIdx.x - group * b.keep);
  if (k >= max(used, 1)) return;
  const int G = b.beams, V = b.V, H = b.H, C = b.C;
  if (k < used) {
    const uint32_t at = b.chosen[group * kMostKept + k];
    const int r = at / (uint32_t)b.n_blocks;
    const int v0 = (int)(at - (uint32_t)r * (uint32_t)b.n_blocks) * 16;
    const uint4* h = reinterpret_cast<const uint4*>(b.hidden + (row0 + r) * H);
    const uint4* w[4];
    double acc[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      w[e] = reinterpret_cast<const uint4*>(b.W + (int64_t)min(v0 + 4 * wave + e, V - 1) * H);
      acc[e] = 0.0;
    }
    for (int c = lane; c < H / 8; c += 64) {
      const uint4 x = h[c];
      const uint32_t xs[4] = {x.x, x.y, x.z, x.w};
      uint4 y[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) y[e] = w[e][c];
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const uint32_t ys[4] = {y[e].x, y[e].y, y[e].z, y[e].w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {   // a product of two bf16 is exact in float32 (but for its range: 64 bits)
          acc[e] = fma((double)__uint_as_float(xs[i] << 16), (double)__uint_as_float(ys[i] << 16), acc[e]);
          acc[e] = fma((double)__uint_as_float(xs[i] & 0xFFFF0000u), (double)__uint_as_float(ys[i] & 0xFFFF0000u), acc[e]);
        }
      }
    }
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const double z = wave_sum(acc[e]);
      if (lane == 0) b.exact[(group * kMostKept + k) * 16 + 4 * wave + e] = z;
    }
  }
  __threadfence();
  __syncthreads();
  if (tid == 0) last = atomicAdd(&b.ticket[group], 1) == max(used, 1) - 1;
  __syncthreads();
  if (!last) return;
  __threadfence();

  auto allowed = [&](int r, int64_t v) {
    return v < V && (b.allowed == nullptr || ((uint32_t)b.allowed[(row0 + r) * b.mask_ld + (v >> 5)] >> (v & 31)) & 1);
  };
  auto place = [&](int i, int& r, int64_t& v0) {
    const uint32_t at = b.chosen[group * kMostKept + i];
    r = at / (uint32_t)b.n_blocks;
    v0 = (int64_t)(at - (uint32_t)r * (uint32_t)b.n_blocks) * 16;
  };
  const double* exact = b.exact + group * kMostKept * 16;
  if (tid < used) {
    int r;
    int64_t v0;
    place(tid, r, v0);
    double m = -INFINITY;
    for (int e = 0; e < 16; ++e)
      if (allowed(r, v0 + e)) m = fmax(m, exact[16 * tid + e]);
    z_max[tid] = m;
  }
  if (tid == 0) {
    count = 0;
    limit = -INFINITY;
  }
  __syncthreads();
  if (tid < G) {
    double lse = b.lse64[row0 + tid];
    for (int i = 0; i < used; ++i) {
      int r;
      int64_t v0;
      place(i, r, v0);
      if (r != tid) continue;
      const double was = b.blocks[(v0 >> 4) * b.ld + row0 + r];
      lse += log1p(exp(z_max[i] / b.T - lse) - exp(was / b.T - lse));
      break;
    }
    logsum[tid] = lse;
  }
  __syncthreads();
  auto score_of = [&](int r, double z) { return (double)b.scores[row0 + r] + (z / b.T - logsum[r]); };
  // C blocks hold a candidate each that reaches the C-th largest of their best
  if (tid < used) {
    int r;
    int64_t v0;
    place(tid, r, v0);
    value[tid] = score_of(r, z_max[tid]);
  }
  __syncthreads();
  if (tid < used) {
    int rank = 0;
    for (int i = 0; i < used; ++i) rank += value[i] > value[tid] || (value[i] == value[tid] && i < tid);
    if (rank == C - 1) limit = value[tid];
  }
  __syncthreads();
  for (int i = tid; i < 16 * used; i += kScoreThreads) {
    int r;
    int64_t v0;
    place(i >> 4, r, v0);
    const int64_t v = v0 + (i & 15);
    if (!allowed(r, v)) continue;
    const double x = score_of(r, exact[i]);
    if (x > -INFINITY && x >= limit) {
      const int at = atomicAdd(&count, 1);
      value[at] = x;
      index[at] = (uint32_t)(r * (int64_t)V + v);
    }
  }
  for (int r = tid; r < G; r += kScoreThreads) {
    const float s = b.scores[row0 + r];
    if (!ended_row(b, row0 + r) || !finite(s)) continue;
    const int at = atomicAdd(&count, 1);
    value[at] = s;
    index[at] = (uint32_t)(r * (int64_t)V + b.ended[row0 + r]);
  }
  __syncthreads();
  const int found = count;
  for (int i = tid; i < found; i += kScoreThreads) {
    const double x = value[i];
    const uint32_t at = index[i];
    int rank = 0;
    for (int j = 0; j < found; ++j) rank += value[j] > x || (value[j] == x && index[j] < at);
    if (rank < C) {
      const int64_t to = group * C + rank;
      b.top_scores[to] = (float)x;
      b.top_ids[to] = (int32_t)(at % (uint32_t)V);
      b.top_parents[to] = (int32_t)(row0 + at / (uint32_t)V);
    }
  }
  for (int i = found + tid; i < C; i += kScoreThreads) {
    const int64_t to = group * C + i;
    b.top_scores[to] = -INFINITY;
    b.top_ids[to] = -1;
    b.top_parents[to] = -1;
  }
}

}  // namespace

hipError_t launch_beam_step(const BeamArgs& b, hipStream_t stream) {
  const double N = b.N, H = b.H, V = b.V;
  const int64_t groups = b.N / b.beams;
  trace_begin(stream);
  if (b.few) {
    FewArgs a{};
    a.hidden = b.hidden;
    a.W = b.W;
    a.N = b.N;
    a.H = b.H;
    a.V = b.V;
    a.sc = b.sc;
    a.tiles = (b.N + 63) / 64;
    a.splits = b.splits;
    with_sizes(few_blocks(b.V), b.N <= 16 ? 1 : b.N <= 32 ? 2 : 4, [&](auto mb, auto nb) {
      const dim3 grid(few_grid((int64_t)a.tiles * a.splits));
      if (b.allowed != nullptr) hipLaunchKernelGGL((beam_few_kernel<mb(), nb(), true>), grid, dim3(256), 0, stream, a, b);
      else hipLaunchKernelGGL((beam_few_kernel<mb(), nb(), false>), grid, dim3(256), 0, stream, a, b);
    });
  } else {
    const dim3 grid((unsigned)(((int64_t)b.n_tt * b.splits + 7) / 8 * 8));
    if (b.allowed != nullptr) hipLaunchKernelGGL((beam_tile_kernel<true>), grid, dim3(kThreads), 0, stream, b);
    else hipLaunchKernelGGL((beam_tile_kernel<false>), grid, dim3(kThreads), 0, stream, b);
  }
  hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  trace_end(kBeamLogits, stream, 2.0 * N * H * V, 2.0 * (N + V) * H + 8.0 * b.splits * N + 4.0 * N * (b.n_blocks + b.n_sections) +
                                                      (b.allowed != nullptr ? N * V / 8 : 0.0));
  trace_begin(stream);
  hipLaunchKernelGGL(beam_select_kernel, dim3((unsigned)groups), dim3(kSelThreads), 0, stream, b);
  e = hipGetLastError();
  if (e != hipSuccess) return e;
  trace_end(kBeamSelect, stream, 0.0, 8.0 * b.splits * N + 4.0 * N * b.n_sections);
  trace_begin(stream);
  hipLaunchKernelGGL(beam_score_kernel, dim3((unsigned)(b.keep * groups)), dim3(kScoreThreads), 0, stream, b);
  e = hipGetLastError();
  if (e != hipSuccess) return e;
  trace_end(kBeamScore, stream, 32.0 * groups * b.C * H, 34.0 * groups * b.C * H);
  return hipSuccess;
}

// ---------------------------------------------------------------------------
// Reordering: rows of `runs` runs of `run_bytes` each, of which the first
// lengths[parent] * step_bytes are in use (all without lengths). A thread owns
// the 16 bytes at one place of a run for the whole group, reads what the
// group's rows need of them and writes it: in place, every read of them comes
// before any write, without a wait between threads. Groups above kReorderRows
// rows go through LDS in place, and in batches of rows else.
namespace {

typedef uint32_t u32x4a __attribute__((ext_vector_type(4), aligned(1)));

__device__ __forceinline__ u32x4a load16(const char* p, int n) {
  if (n >= 16) return *reinterpret_cast<const u32x4a*>(p);
  u32x4a v = {0, 0, 0, 0};
#pragma unroll
  for (int k = 0; k < 16; ++k)
    if (k < n) v[k >> 2] |= (uint32_t)(uint8_t)p[k] << (8 * (k & 3));
  return v;
}
__device__ __forceinline__ void store16(char* p, int n, u32x4a v) {
  if (n >= 16) {
    *reinterpret_cast<u32x4a*>(p) = v;
    return;
  }
#pragma unroll
  for (int k = 0; k < 16; ++k)
    if (k < n) p[k] = (char)(v[k >> 2] >> (8 * (k & 3)));
}

constexpr int kReorderRows = 16;

// bytes in use of the run that row j of the group takes over from row `from`,
// 0 where it takes none
__device__ __forceinline__ int64_t used_bytes(const ReorderArgs& a, int64_t from) {
  if (a.lengths == nullptr) return a.run_bytes;
  const int64_t n = a.lengths[from];
  return (n < 0 ? 0 : n > a.steps ? a.steps : n) * a.step_bytes;
}

template <bool LDS>
__global__ __launch_bounds__(256) void beam_reorder_kernel(const ReorderArgs a) {
  extern __shared__ u32x4 held[];   // LDS: [threads][beams]
  const int64_t unit = (int64_t)blockIdx.x * blockDim.x + threadIdx.x;
  if (unit >= a.units) return;
  // unit = ((plane, group), run, place)
  const int64_t run_of = unit / a.places;
  const int64_t at = (unit - run_of * a.places) * 16;
  const int64_t pg = run_of / a.runs, run = run_of - pg * a.runs;
  const int64_t groups = a.rows / a.beams;
  const int64_t plane = pg / groups, group = pg - plane * groups;
  const int64_t row0 = group * a.beams, row_bytes = a.runs * a.run_bytes;
  const int64_t base = (plane * a.rows + row0) * row_bytes + run * a.run_bytes + at;
  const char* in = static_cast<const char*>(a.states) + base;
  char* out = static_cast<char*>(a.out) + base;
  const bool place = a.states == a.out;
  const int G = a.beams;
  // the bytes at this place that row j takes over, and from which row
  auto source = [&](int j, int& from) {
    const int64_t p = (int64_t)a.parents[row0 + j] - row0;
    from = (int)p;
    if (p < 0 || p >= G || (place && p == j)) return 0;
    const int64_t n = used_bytes(a, row0 + p) - at;
    return n <= 0 ? 0 : n >= 16 ? 16 : (int)n;
  };
  if (LDS) {
    u32x4* mine = held + (int64_t)threadIdx.x * G;
    for (int j = 0; j < G; ++j) {
      int from;
      const int n = source(j, from);
      if (n > 0) mine[j] = load16(in + from * row_bytes, n);
    }
    for (int j = 0; j < G; ++j) {
      int from;
      const int n = source(j, from);
      if (n > 0) store16(out + j * row_bytes, n, mine[j]);
    }
    return;
  }
  for (int j0 = 0; j0 < G; j0 += kReorderRows) {
    u32x4a v[kReorderRows];
    int n[kReorderRows];
#pragma unroll
    for (int j = 0; j < kReorderRows; ++j) {
      n[j] = 0;
      if (j0 + j >= G) continue;
      int from;
      n[j] = source(j0 + j, from);
      if (n[j] > 0) v[j] = load16(in + from * row_bytes, n[j]);
    }
#pragma unroll
    for (int j = 0; j < kReorderRows; ++j)
      if (n[j] > 0) store16(out + (j0 + j) * row_bytes, n[j], v[j]);
  }
}

}  // namespace

hipError_t launch_beam_reorder(ReorderArgs a, hipStream_t stream) {
  a.run_bytes = a.steps * a.step_bytes;
  a.places = (a.run_bytes + 15) / 16;
  a.units = a.planes * (a.rows / a.beams) * a.runs * a.places;
  if (a.units == 0) return hipSuccess;
  trace_begin(stream);
  if (a.states == a.out && a.beams > kReorderRows) {
    const int threads = 64;
    hipLaunchKernelGGL((beam_reorder_kernel<true>), dim3((unsigned)((a.units + threads - 1) / threads)), dim3(threads),
                       (size_t)threads * a.beams * 16, stream, a);
  } else {
    hipLaunchKernelGGL((beam_reorder_kernel<false>), dim3((unsigned)((a.units + 255) / 256)), dim3(256), 0, stream, a);
  }
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  trace_end(kBeamReorder, stream, 0.0, 2.0 * a.planes * a.rows * a.runs * (double)a.run_bytes);
  return hipSuccess;
}

}  // namespace lmh
