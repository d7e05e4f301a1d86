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
//           that error
//   rank    a workgroup per group orders the candidates of its blocks. A launch
//           of its own: the last of a group's scoring workgroups would do it
//           without, but each of them then makes its stores visible to the whole
//           card first, which takes longer
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
// Tiles of 16 NB tokens: up to 128, where the distillation's stop at 64. Bound by
// the read of W: 64 rows at H 2560, V 151936 (778 MB) take 154 us, 5.05 TB/s,
// as a copy; 4 rows at 1024 x 50257 (103 MB) 27 us, 3.8 TB/s, of which 6 are
// the launch's rise and fall.
template <int MB, int NB, bool MASK>
__global__ __launch_bounds__(256, 2) void beam_few_kernel(const FewArgs a, const BeamArgs b) {
  __shared__ __attribute__((aligned(16))) char lds[few_lds<NB>()];
  __shared__ float4 xch[4][16 * NB];
  const int lane = threadIdx.x & 63;
  const int wave = wave_id();
  const int vid = xcd_remap(blockIdx.x, gridDim.x), tok0 = vid % a.tiles * (16 * NB);
  const FewTile t{tok0, min(16 * NB, a.N - tok0), vid / a.tiles};
  if (t.split >= a.splits) return;
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

// Of four blocks' largest logits, of which a lane holds a part of each (the
// lanes of a row of 16 tokens four words each), the whole of one block in each
// quarter of the wave: quarter q gets block kQuarterBlock[q]. Three exchanges
// where a butterfly per block takes eight.
__device__ __forceinline__ float swap_max(float a, float b, bool halves) {
  typedef unsigned u32x2 __attribute__((ext_vector_type(2)));
  const unsigned x = __float_as_uint(a), y = __float_as_uint(b);
  const u32x2 r = halves ? __builtin_bit_cast(u32x2, __builtin_amdgcn_permlane32_swap(x, y, false, false))
                         : __builtin_bit_cast(u32x2, __builtin_amdgcn_permlane16_swap(x, y, false, false));
  return max_drop(__uint_as_float(r.x), __uint_as_float(r.y));
}
__device__ __forceinline__ float four_blocks(float b0, float b1, float b2, float b3) {
  return swap_max(swap_max(b0, b1, true), swap_max(b2, b3, true), false);
}
__device__ __forceinline__ int quarter_block(int q) { return (q & 1) * 2 + (q >> 1); }

// Four words of a row's mask, wherever they begin.
struct __attribute__((packed, aligned(4))) Words4 {
  uint32_t w[4];
};

// Many rows: the head's forward tiles; a section is a wave's 128 vocabulary
// rows. The arrays hold whole tiles of rows and of words, so every store is in
// place; what lies past N or V is not read. Bound by the matrix units: 1024
// rows at H 2560, V 151936 take 680 us (1,170 TFLOP/s) and with masks 727 to 768;
// the block maxima and statistics of a tile are a tenth of its time, on a
// SIMD's only wave.
template <bool MASK>
__global__ __launch_bounds__(kThreads) void beam_tile_kernel(
    const uint16_t* __restrict__ hidden, const uint16_t* __restrict__ W, const int32_t* __restrict__ allowed, int mask_ld, int N,
    int H, int V, int S, int n_tt, int n_vt, float sc, float2* __restrict__ records, float* __restrict__ sections,
    float* __restrict__ blocks, int ld) {
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
  float m2[kNB], s1[kNB];
#pragma unroll
  for (int j = 0; j < kNB; ++j) m2[j] = kNegBig, s1[j] = 0.0f;
  const Operand ob{hidden + (int64_t)tok0 * H, H, min(kTile, N - tok0)};
  Pipe pipe;
  for (int vt = s; vt < n_vt; vt += S) {
    const int v0 = vt * kTile;
    const Operand oa{W + (int64_t)v0 * H, H, min(kTile, V - v0)};
    const int v1 = v0 + S * kTile;
    const bool more = vt + S < n_vt && min(kTile, V - v1) == oa.rows;
    f32x4 acc[kNB][kNB];
    mma_tile<false, 96>(oa, ob, H, lds, acc, pipe, W + (int64_t)(more ? v1 : v0) * H, ob.base, more);
    const int vrow0 = v0 + wm * 128;
    const bool ragged = vrow0 + 128 > V;
    const int q = lane >> 4;
    const int tok = tok0 + wn * 128 + (lane & 15);
    float* to = blocks + (int64_t)((vrow0 >> 4) + quarter_block(q)) * ld + tok;
    float* sec = sections + (int64_t)(vrow0 >> 7) * ld + tok;
    // the masks of a row's 128 words: of the next row while one is looked at
    const int word0 = min(vrow0 >> 5, max(mask_ld - 4, 0));   // four words in place, of which `skip` come before
    const int skip = (vrow0 >> 5) - word0;
    auto masks_of = [&](int j) {
      const int32_t* row = allowed + (int64_t)min(tok + 16 * j, N - 1) * mask_ld + word0;
      if (mask_ld >= 4) return *reinterpret_cast<const Words4*>(row);
      Words4 w;
#pragma unroll
      for (int k = 0; k < 4; ++k) w.w[k] = k < mask_ld ? (uint32_t)row[min(k, mask_ld - 1)] : 0;
      return w;
    };
    Words4 ahead{};
    if (MASK) ahead = masks_of(0);
#pragma unroll
    for (int j = 0; j < kNB; ++j) {
      uint32_t words[4];
      if (MASK) {
        const Words4 now = ahead;
        if (j + 1 < kNB) ahead = masks_of(j + 1);
#pragma unroll
        for (int w = 0; w < 4; ++w) words[w] = now.w[w] >> (4 * q);
        if (skip > 0) {   // the last tile's
#pragma unroll
          for (int w = 0; w < 4; ++w) {
            uint32_t x = 0;
#pragma unroll
            for (int k = w + 1; k < 4; ++k) x = w + skip == k ? now.w[k] : x;
            words[w] = x >> (4 * q);
          }
        }
      }
      float z[kNB][4];
#pragma unroll
      for (int i = 0; i < kNB; ++i) {
        pin_acc(acc[i][j]);
#pragma unroll
        for (int r = 0; r < 4; ++r) z[i][r] = acc[i][j][r];
      }
      if (ragged) {   // rows past V take no part, whatever the bits of a mask say there: below every real logit, and
                      // in statistics that start at kNegBig nothing
#pragma unroll
        for (int i = 0; i < kNB; ++i)
#pragma unroll
          for (int r = 0; r < 4; ++r) z[i][r] = (vrow0 + acc_row(i, r, lane) < V) ? z[i][r] : -INFINITY;
      }
      float mx = z[0][0];
#pragma unroll
      for (int i = 0; i < kNB; ++i)
#pragma unroll
        for (int r = 0; r < 4; ++r) mx = nan_max(mx, z[i][r]);
      float whole[2];
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        float best[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int i = 4 * h + e;
          float x[4];
#pragma unroll
          for (int r = 0; r < 4; ++r) {
            x[r] = z[i][r];
            if (MASK) x[r] = (words[i >> 1] >> (16 * (i & 1) + r)) & 1 ? x[r] : -INFINITY;
          }
          best[e] = max_drop(max_drop(x[0], x[1]), max_drop(x[2], x[3]));
        }
        whole[h] = four_blocks(best[0], best[1], best[2], best[3]);
        to[(int64_t)(4 * h) * ld + 16 * j] = whole[h];
      }
      float top = max_drop(whole[0], whole[1]);
      top = swap_max(top, top, true);
      top = swap_max(top, top, false);
      if (q == 0) sec[16 * j] = top;
      const float mnew = nan_max(m2[j], mx * sc);
      float e = s1[j] * fast_exp2(m2[j] - mnew);
      if (!ragged) {
#pragma unroll
        for (int i = 0; i < kNB; ++i)
#pragma unroll
          for (int r = 0; r < 4; ++r) e += fast_exp2(fmaf(z[i][r], sc, -mnew));
      } else {
#pragma unroll
        for (int i = 0; i < kNB; ++i)
#pragma unroll
          for (int r = 0; r < 4; ++r) {
            const float x = fast_exp2(fmaf(z[i][r], sc, -mnew));
            e += vrow0 + acc_row(i, r, lane) < V ? x : 0.0f;
          }
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
      records[(int64_t)s * ld + tok0 + wn * 128 + j * 16 + lane] =
          make_float2(m, s1[j] * fast_exp2(m2[j] - m) + o.y * fast_exp2(o.x - m));
    }
  }
}

// ---------------------------------------------------------------------------
// Reductions over lanes on the vector unit (data-parallel primitives and lane
// swaps; __shfl_xor takes a trip through LDS for each step). Every lane of a
// group of W ends with the same bits: each step combines the same two values in
// both of the lanes that exchange them, lower half first where that matters.
struct Wide;
template <int CTRL, class T>
__device__ __forceinline__ T dpp_of(T v) {
  if constexpr (std::is_same_v<T, Wide>) {
    return {dpp_of<CTRL>(v.value), dpp_of<CTRL>(v.rest)};
  } else if constexpr (sizeof(T) == 4) {
    return __builtin_bit_cast(T, __builtin_amdgcn_mov_dpp(__builtin_bit_cast(int, v), CTRL, 0xF, 0xF, true));
  } else {
    const uint64_t u = __builtin_bit_cast(uint64_t, v);
    const uint32_t lo = __builtin_amdgcn_mov_dpp((int)(uint32_t)u, CTRL, 0xF, 0xF, true);
    const uint32_t hi = __builtin_amdgcn_mov_dpp((int)(uint32_t)(u >> 32), CTRL, 0xF, 0xF, true);
    return __builtin_bit_cast(T, (uint64_t)hi << 32 | lo);
  }
}
template <int HALF, class T, class F>
__device__ __forceinline__ T swapped(T v, F op) {
  typedef unsigned u32x2 __attribute__((ext_vector_type(2)));
  auto swap = [](uint32_t x) {
    return HALF == 32 ? __builtin_bit_cast(u32x2, __builtin_amdgcn_permlane32_swap(x, x, false, false))
                      : __builtin_bit_cast(u32x2, __builtin_amdgcn_permlane16_swap(x, x, false, false));
  };
  if constexpr (sizeof(T) == 4) {
    const u32x2 r = swap(__builtin_bit_cast(uint32_t, v));
    const uint32_t x = r.x, y = r.y;   // a bit_cast of r.y itself would read r.x
    return op(__builtin_bit_cast(T, x), __builtin_bit_cast(T, y));
  } else {
    const uint64_t u = __builtin_bit_cast(uint64_t, v);
    const u32x2 lo = swap((uint32_t)u), hi = swap((uint32_t)(u >> 32));
    return op(__builtin_bit_cast(T, (uint64_t)hi.x << 32 | lo.x), __builtin_bit_cast(T, (uint64_t)hi.y << 32 | lo.y));
  }
}
// op is commutative in its bits (a sum or a maximum of two values)
template <int W, class T, class F>
__device__ __forceinline__ T reduce(T v, F op) {
  v = op(v, dpp_of<0xB1>(v));                       // quad_perm 1 0 3 2
  v = op(v, dpp_of<0x4E>(v));                       // quad_perm 2 3 0 1
  if constexpr (W >= 8) v = op(v, dpp_of<0x141>(v));   // row_half_mirror
  if constexpr (W >= 16) v = op(v, dpp_of<0x140>(v));  // row_mirror
  if constexpr (W >= 32) v = swapped<16>(v, op);
  if constexpr (W >= 64) v = swapped<32>(v, op);
  return v;
}
struct Sum {
  template <class T>
  __device__ __forceinline__ T operator()(T a, T b) const { return a + b; }
};
struct Max {
  template <class T>
  __device__ __forceinline__ T operator()(T a, T b) const { return a > b ? a : b; }
  __device__ __forceinline__ double operator()(double a, double b) const { return fmax(a, b); }
};
struct NanMax {
  __device__ __forceinline__ float operator()(float a, float b) const { return nan_max(a, b); }
};

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

// The same of a double.
struct Wide {
  uint64_t value;
  uint32_t rest;
};
__device__ __forceinline__ bool operator>(const Wide& a, const Wide& b) {
  return a.value > b.value || (a.value == b.value && a.rest > b.rest);
}
__device__ __forceinline__ Wide key_of(double v, uint32_t index) {
  const uint64_t u = __double_as_longlong(v);
  return {(u >> 63) != 0 ? ~u : u | 1ull << 63, ~index};
}
__device__ __forceinline__ double value_of(const Wide& key) {
  const uint64_t o = key.value;
  return __longlong_as_double((o >> 63) != 0 ? o ^ 1ull << 63 : ~o);
}
__device__ __forceinline__ uint32_t index_of(const Wide& key) { return ~key.rest; }

// Key{} is none, and lies below all others.
template <class Key>
struct Limits;
template <>
struct Limits<uint64_t> {
  static constexpr uint64_t least = 1, above = ~(uint64_t)0;   // of the others; above all of them
};
template <>
struct Limits<Wide> {
  static constexpr Wide least{0, 1}, above{~(uint64_t)0, ~0u};
};

constexpr int kSelThreads = 1024;
constexpr int kSelTeams = 128;    // of 8 threads each
constexpr int kSelList = 2048;
constexpr int kSelHeld = 24576;   // items whose values LDS holds (96 KB)

// The `keep` largest keys of items 0 .. n - 1 into kept[0 ..], sorted; returns
// how many there are (keep, or all that are not none). key(i) gives an item's key. A thread looks at neighbouring items, a team at those of eight
// threads: rows in turn. Every team has a largest key, and the keep-th largest of
// those is a threshold that at least `keep` items reach, and few more do as a
// rule: those are ranked. Should more than the list holds reach it (most of the
// best items lie with few teams), the best are taken one after the other.
//
static_assert(kMostKept <= kSelTeams, "a threshold exists");
static_assert(kMostKept <= 2 * 64, "two waves look at the kept ones' logits");
template <class Key>
struct Selection {
  Key list[kSelList];
  Key most[kSelTeams];
  int rank[kSelTeams];
  Key kept[kMostKept];
  Key limit;
  int count;
};
template <class Key, class F>
__device__ __forceinline__ int select_best(Selection<Key>& s, uint32_t n, int keep, F key) {
  const int tid = threadIdx.x;
  constexpr int team = kSelThreads / kSelTeams;
  const uint32_t per = (n + kSelThreads - 1) / kSelThreads;
  const uint32_t i0 = min(n, tid * per), i1 = min(n, i0 + per);
  auto largest = [&](Key below) {
    Key most{};
#pragma unroll 4
    for (uint32_t i = i0; i < i1; ++i) {
      const Key k = key(i);
      most = below > k && k > most ? k : most;
    }
    return reduce<team>(most, Max());
  };
  Key below = Limits<Key>::above;
  int found = 0;
#pragma unroll 1
  for (int r = 0; r < keep; ++r) {   // once, unless the list runs over
    const Key most = largest(below);
    if (tid % team == 0) s.most[tid / team] = most;
    if (tid < kSelTeams) s.rank[tid] = 0;
    if (tid == 0) {
      s.limit = Limits<Key>::least;
      s.count = 0;
    }
    __syncthreads();
    {
      // the teams' ranks, 16 comparisons a thread
      const Key mine = s.most[tid % kSelTeams];
      int rank = 0;
#pragma unroll
      for (int k = 0; k < kSelTeams / team; ++k) rank += s.most[tid / kSelTeams * (kSelTeams / team) + k] > mine;
      if (rank > 0) atomicAdd(&s.rank[tid % kSelTeams], rank);
    }
    __syncthreads();
    const int want = found > kSelList ? 0 : keep - 1;
    if (tid < kSelTeams && s.rank[tid] == want && s.most[tid] > Key{}) s.limit = s.most[tid];
    __syncthreads();
    const Key limit = s.limit;
    if (found > kSelList) {
      if (tid == 0) s.kept[r] = limit;
      below = limit;
      __syncthreads();   // the limit has been read
      continue;
    }
#pragma unroll 4
    for (uint32_t i = i0; i < i1; ++i) {
      const Key k = key(i);
      if (limit > k) continue;
      const int at = atomicAdd(&s.count, 1);
      if (at < kSelList) s.list[at] = k;
    }
    __syncthreads();
    found = s.count;
    if (found <= kSelList) break;
    r = -1;   // one after the other, from the first
    __syncthreads();
  }
  if (found > kSelList) {
    __syncthreads();
    return keep;   // more than kSelList items are not none
  }
#pragma unroll 1
  for (int first = 0; first < found; first += kSelThreads / 16) {   // 16 threads a candidate
    const int i = first + (tid >> 4);
    const Key mine = i < found ? s.list[i] : Key{};
    int rank = 0;
#pragma unroll 2
    for (int k = tid & 15; k < found; k += 16) rank += s.list[k] > mine;
    rank = reduce<16>(rank, Sum());
    if (i < found && (tid & 15) == 0 && rank < keep) s.kept[rank] = mine;
  }
  __syncthreads();
  return min(found, keep);
}

__device__ __forceinline__ double wave_sum(double v) { return reduce<64>(v, Sum()); }
__device__ __forceinline__ bool finite(double v) { return fabs(v) < INFINITY; }
__device__ __forceinline__ bool ended_row(const BeamArgs& b, int64_t tok) {
  return b.ended != nullptr && b.ended[tok] >= 0 && b.ended[tok] < b.V;
}

// Bound by the chain of its steps (loads, records' sums, two choices of some ten
// barriers each), not by bytes: 12 us for one group of 4 beams at 50257 words,
// 15 for 8 of 8 at 151936, 28 for 64 of 16. One workgroup a group: a group's
// sections lie within 100 KB or so, and several would need a launch more.
__global__ __launch_bounds__(kSelThreads) void beam_select_kernel(const BeamArgs b) {
  __shared__ union {
    Selection<uint64_t> narrow;
    Selection<Wide> wide;
  } sel;
  __shared__ float held[kSelHeld];
  __shared__ double base[kMostBeams], lse64[kMostBeams];
  __shared__ float size[kMostBeams], shift[kMostBeams], scores[kMostBeams];
  __shared__ uint32_t sec_row[kMostKept], sec_block[kMostKept];
  __shared__ float unit;   // about the largest logit that counts
  __shared__ bool far;
  __shared__ double rec_sum[kSelThreads];
  __shared__ float rec_max[kSelThreads];
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int64_t group = blockIdx.x, row0 = group * b.beams;
  const uint32_t G = b.beams, n_sec = (uint32_t)b.n_sections, per = b.per_section, n_blocks = (uint32_t)b.n_blocks;
  const uint32_t n_a = n_sec * G;   // beams * V stays below 2^31: i / G is exact as a product with a reciprocal
  const uint32_t by_rows = G > 1 ? 0xFFFFFFFFu / G + 1 : 0, by_blocks = per > 1 ? 0xFFFFFFFFu / per + 1 : 0;
  auto quotient = [](uint32_t i, uint32_t recip) { return recip != 0 ? __umulhi(i, recip) : i; };
  const float* sections = b.sections + row0;
  auto section_at = [&](uint32_t i) {
    const uint32_t s = quotient(i, by_rows);
    return sections[(int64_t)s * b.ld + (i - s * G)];
  };
  // the sections' values, on their way while the records are merged
  constexpr int U = 4;
  float early[U];
#pragma unroll
  for (int k = 0; k < U; ++k) early[k] = section_at(min((uint32_t)tid + kSelThreads * k, n_a - 1));
  // records, rows side by side as they lie (a wave per row would fetch each line
  // for 8 bytes of it, for every row): a thread's of one row, then the row's
  {
    const uint32_t at_once = kSelThreads / G, mine = quotient(tid, by_rows), r = tid - mine * G;
    float m = kNegBig;
    double sum = 0.0;
    if (mine < at_once) {
#pragma unroll 1
      for (uint32_t s0 = mine; s0 < (uint32_t)b.splits; s0 += 4 * at_once) {
        float2 p[4];
        float mx = m;
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const uint32_t s = s0 + k * at_once;
          p[k] = b.records[(int64_t)min(s, (uint32_t)b.splits - 1) * b.ld + row0 + r];
          if (s >= (uint32_t)b.splits) p[k] = make_float2(kNegBig, 0.0f);
          mx = nan_max(mx, p[k].x);
        }
        sum *= (double)fast_exp2(m - mx);
#pragma unroll
        for (int k = 0; k < 4; ++k) sum += (double)p[k].y * (double)fast_exp2(p[k].x - mx);
        m = mx;
      }
    }
    rec_sum[tid] = sum;
    rec_max[tid] = m;
  }
  __syncthreads();
#pragma unroll 1
  for (int r = wave; r < (int)G; r += kSelThreads / 64) {
    const int64_t tok = row0 + r;
    const int at_once = kSelThreads / G;
    float m = kNegBig;
    for (int k = lane; k < at_once; k += 64) m = nan_max(m, rec_max[k * G + r]);
    const float mx = reduce<64>(m, NanMax());
    double sum = 0.0;
    for (int k = lane; k < at_once; k += 64) sum += rec_sum[k * G + r] * (double)fast_exp2(rec_max[k * G + r] - mx);
    sum = wave_sum(sum);
    if (lane == 0) {
      const float score = b.scores[tok];
      // records are in base 2 of logits scaled by the float32 sc: back = 1 / (sc T) undoes both
      const double lse = mx == INFINITY ? INFINITY : (double)mx * b.back + log(sum);
      const bool part = finite(score) && !ended_row(b, tok);
      const bool live = part && finite(lse);
      base[r] = live ? (double)score - lse : -INFINITY;
      size[r] = live ? (float)((double)mx * b.back) : 0.0f;
      scores[r] = score;
      lse64[r] = lse;
      b.lse64[tok] = lse;
      b.lse[tok] = part ? (float)lse : 0.0f;
    }
  }
#pragma unroll
  for (int k = 0; k < U; ++k)
    if (tid + kSelThreads * k < min(n_a, (uint32_t)kSelHeld)) held[tid + kSelThreads * k] = early[k];
#pragma unroll 1
  for (uint32_t i = tid + kSelThreads * U; i < min(n_a, (uint32_t)kSelHeld); i += kSelThreads * U) {
    float z[U];
#pragma unroll
    for (int k = 0; k < U; ++k) z[k] = section_at(min(i + kSelThreads * k, n_a - 1));
#pragma unroll
    for (int k = 0; k < U; ++k)
      if (i + kSelThreads * k < min(n_a, (uint32_t)kSelHeld)) held[i + kSelThreads * k] = z[k];
  }
  __syncthreads();
  if (wave == 0) {
    // values relative to about the best candidate, where float32 is finest
    const double mine = lane < (int)G ? base[lane] : -INFINITY;
    const float large = lane < (int)G ? size[lane] : 0.0f;
    const double ref = reduce<64>(mine + (double)large, Max());
    const float most = reduce<64>(fabsf(large), NanMax());
    if (lane < (int)G) shift[lane] = finite(mine) ? (float)(mine - ref) : -INFINITY;
    // a row that lies so far off that its float32 steps come near its own logits' sums' errors
    const bool any = __any(lane < (int)G && finite(mine) && ref - mine > 256.0 * (double)(fabsf(large) + b.invT));
    if (lane == 0) {
      unit = most + b.invT;
      far = any;
    }
  }
  __syncthreads();
  // key(r, index, z): of an item, by its row, index and largest logit; logit(r, value): that logit / T
  auto choose = [&](auto& sel, auto key, auto logit) {
    int kept = 0;
#pragma unroll 1
    for (int stage = 0; stage < 2; ++stage) {   // the sections, then the blocks of the best of them
      const uint32_t n = stage == 0 ? n_a : (uint32_t)kept * per;
      if (stage == 1) {
        if (tid < kept) {
          const uint32_t at = index_of(sel.kept[tid]), r = at / n_sec;
          sec_row[tid] = r;
          sec_block[tid] = (at - r * n_sec) * per;
        }
        __syncthreads();
#pragma unroll
        for (int k = 0; k < 2; ++k) {   // kMostKept sections of at most 20 blocks
          const uint32_t i = tid + kSelThreads * k;
          if (i >= n) continue;
          const uint32_t q = quotient(i, by_blocks), blk = sec_block[q] + (i - q * per);
          held[i] = blk < n_blocks ? b.blocks[(int64_t)blk * b.ld + row0 + sec_row[q]] : -INFINITY;
        }
        __syncthreads();
      }
      kept = select_best(sel, n, b.keep, [&](uint32_t i) {
        const uint32_t q = quotient(i, stage == 0 ? by_rows : by_blocks), rest = i - q * (stage == 0 ? G : per);
        const uint32_t r = stage == 0 ? rest : sec_row[q];
        const uint32_t index = stage == 0 ? r * n_sec + q : r * n_blocks + sec_block[q] + rest;
        return key(r, index, i < kSelHeld ? held[i] : section_at(i));
      });
    }
    // those of the first C, and of the spare ones that are as good within a slack that is far more than the tiles' sums
    // are off: a part of the largest logit, or of the kept ones where a mask leaves none as small
    if (tid < 2 * 64) {
      const float z = tid < kept ? fabsf(logit(index_of(sel.kept[tid]) / n_blocks, value_of(sel.kept[tid]))) : 0.0f;
      const float most = reduce<64>(z, [](float a, float b) { return fmaxf(a, b); });
      if (lane == 0) atomicMax(reinterpret_cast<int*>(&unit), __float_as_int(most + b.invT));   // none is negative
    }
    __syncthreads();
    const float slack = unit * 0x1p-13f;
    const bool in = tid < kept && (tid < b.C || value_of(sel.kept[tid]) >= value_of(sel.kept[b.C - 1]) - slack);
    if (in) b.chosen[group * kMostKept + tid] = index_of(sel.kept[tid]);
    const int used = __syncthreads_count(in);   // values fall, so these are the first ones
    if (tid == 0) b.used[group] = used;
  };
  // Rows whose scores lie far apart (a caller's -1e9 for beams that are to come
  // last) have keys of 64-bit scores, formed as rank forms them: float32 would not
  // tell the words of the lower rows apart. Select then takes 4 us longer (4 beams
  // at 50257 words), 25 (64 groups of 16 at 151936) or 44 (64 beams).
  if (!far) {
    choose(sel.narrow, [&](uint32_t r, uint32_t index, float z) {
      const float x = shift[r];
      return x > -INFINITY && z > -INFINITY ? key_of(fmaf(z, b.invT, x), index) : (uint64_t)0;
    }, [&](uint32_t r, float value) { return value - shift[r]; });
  } else {
    choose(sel.wide, [&](uint32_t r, uint32_t index, float z) {
      return base[r] > -INFINITY && z > -INFINITY ? key_of((double)scores[r] + ((double)z * b.rT - lse64[r]), index) : Wide{};
    }, [&](uint32_t r, double value) { return (float)(value - (double)scores[r] + lse64[r]); });
  }
}

// A workgroup per chosen block: its 16 logits in 64 bits, four a wave. Products
// of bf16 values are exact in float64, the sums off by 1e-16 of their terms. One
// trip to memory where there are few (4.6 us for 24 blocks of H 1024), gathered
// rows where there are many (27 us for 2048 blocks of H 2560, 6 TB/s with those
// that share rows).
__global__ __launch_bounds__(256) void beam_score_kernel(const BeamArgs b) {
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int64_t group = blockIdx.x / b.keep;
  const int k = (int)(blockIdx.x - group * b.keep);
  if (k >= b.used[group]) return;
  const int H8 = b.H / 8;
  const uint32_t at = b.chosen[group * kMostKept + k];
  const uint32_t r = at / (uint32_t)b.n_blocks;
  const int v0 = (int)(at - r * (uint32_t)b.n_blocks) * 16;
  const uint4* h = reinterpret_cast<const uint4*>(b.hidden + (group * b.beams + r) * b.H);
  const uint4* w[4];
  double acc[4];
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    w[e] = reinterpret_cast<const uint4*>(b.W + (int64_t)min(v0 + 4 * wave + e, b.V - 1) * b.H);
    acc[e] = 0.0;
  }
  constexpr int D = 3;
  for (int c = lane; c < H8; c += 64 * D) {
    uint4 x[D], y[D][4];
#pragma unroll
    for (int d = 0; d < D; ++d) {   // past the end: the last chunk of h times 0
      const int at = min(c + 64 * d, H8 - 1);
      x[d] = h[at];
#pragma unroll
      for (int e = 0; e < 4; ++e) y[d][e] = w[e][at];
    }
#pragma unroll
    for (int d = 0; d < D; ++d) {
      if (c + 64 * d >= H8) continue;
      const uint32_t xs[4] = {x[d].x, x[d].y, x[d].z, x[d].w};
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const uint32_t ys[4] = {y[d][e].x, y[d][e].y, y[d][e].z, y[d][e].w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          acc[e] = fma((double)__uint_as_float(xs[i] << 16), (double)__uint_as_float(ys[i] << 16), acc[e]);
          acc[e] = fma((double)__uint_as_float(xs[i] & 0xFFFF0000u), (double)__uint_as_float(ys[i] & 0xFFFF0000u), acc[e]);
        }
      }
    }
  }
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    const double z = wave_sum(acc[e]);
    if (lane == 0) b.exact[(group * kMostKept + k) * 16 + 4 * wave + e] = z;
  }
}

// A workgroup per group: the candidates of the chosen blocks, and the ended
// rows, in order: all pairs of the few that reach the C-th best block's maximum.
// A chain of steps like select's: 4.9 us for 8 candidates, 12 for 64 groups of 32.
constexpr int kRankThreads = 256;
constexpr int kMostFound = 16 * kMostKept + kMostBeams;
__global__ __launch_bounds__(kRankThreads) void beam_rank_kernel(const BeamArgs b) {
  __shared__ double z_max[kMostKept], logsum[kMostBeams], best[kMostKept];
  __shared__ uint32_t row_of[kMostKept], word_of[kMostKept];
  __shared__ int first[kMostBeams];
  __shared__ double value[kMostFound];
  __shared__ uint32_t index[kMostFound];
  __shared__ double limit;
  __shared__ int count;
  const int tid = threadIdx.x;
  const int64_t group = blockIdx.x, row0 = group * b.beams;
  const int G = b.beams, V = b.V, C = b.C, used = b.used[group];
  if (tid < G) first[tid] = kMostKept;
  if (tid == 0) {
    count = 0;
    limit = -INFINITY;
  }
  if (tid < used) {
    const uint32_t at = b.chosen[group * kMostKept + tid], r = at / (uint32_t)b.n_blocks;
    row_of[tid] = r;
    word_of[tid] = (at - r * (uint32_t)b.n_blocks) * 16;
  }
  __syncthreads();
  // sixteen lanes a block
  constexpr int rounds = (16 * kMostKept + kRankThreads - 1) / kRankThreads;
  double z[rounds];
#pragma unroll
  for (int q = 0; q < rounds; ++q) {
    const int i = q * kRankThreads + tid, k = i >> 4;
    z[q] = -INFINITY;
    if (k < used) {
      const uint32_t v = word_of[k] + (i & 15);
      const bool may = v < (uint32_t)V && (b.allowed == nullptr ||
                                           ((uint32_t)b.allowed[(row0 + row_of[k]) * b.mask_ld + (v >> 5)] >> (v & 31)) & 1);
      if (may) z[q] = b.exact[group * kMostKept * 16 + i];
    }
    const double m = reduce<16>(z[q], Max());
    if (k < used && (i & 15) == 0) {
      z_max[k] = m;
      atomicMin(&first[row_of[k]], k);
    }
  }
  __syncthreads();
  if (tid < G) {
    double lse = b.lse64[row0 + tid];
    const int k = first[tid];
    if (k < used) {
      // log1p(e^(z / T - lse) - e^(was / T - lse)); float32 carries it, being some 1e-6 at most
      const double was = b.blocks[(int64_t)(word_of[k] >> 4) * b.ld + row0 + tid];
      lse += (double)log1pf(expf((float)(was * b.rT - lse)) * expm1f((float)((z_max[k] - was) * b.rT)));
    }
    logsum[tid] = lse;
  }
  __syncthreads();
  auto score_of = [&](int r, double x) { return (double)b.scores[row0 + r] + (x * b.rT - logsum[r]); };
  // C blocks hold a candidate each that reaches the C-th largest of their best
  if (tid < used) best[tid] = score_of(row_of[tid], z_max[tid]);
  __syncthreads();
  if (tid < used) {
    const double mine = best[tid];
    int rank = 0;
#pragma unroll 8
    for (int i = 0; i < used; ++i) rank += best[i] > mine || (best[i] == mine && i < tid);
    if (rank == C - 1) limit = mine;
  }
  __syncthreads();
#pragma unroll
  for (int q = 0; q < rounds; ++q) {
    const int i = q * kRankThreads + tid, k = i >> 4;
    if (k >= used) continue;
    const double x = score_of(row_of[k], z[q]);
    if (x > -INFINITY && x >= limit) {
      const int at = atomicAdd(&count, 1);
      value[at] = x;
      index[at] = row_of[k] * (uint32_t)V + word_of[k] + (i & 15);
    }
  }
  if (tid < G) {
    const float s = b.scores[row0 + tid];
    if (ended_row(b, row0 + tid) && finite(s)) {
      const int at = atomicAdd(&count, 1);
      value[at] = s;
      index[at] = (uint32_t)tid * (uint32_t)V + (uint32_t)b.ended[row0 + tid];
    }
  }
  __syncthreads();
  const int found = count;
  for (int i = tid; i < found; i += kRankThreads) {
    const double x = value[i];
    const uint32_t at = index[i];
    int rank = 0;
#pragma unroll 8
    for (int j = 0; j < found; ++j) rank += value[j] > x || (value[j] == x && index[j] < at);
    if (rank < C) {
      const int64_t to = group * C + rank;
      b.top_scores[to] = (float)x;
      b.top_ids[to] = (int32_t)(at % (uint32_t)V);
      b.top_parents[to] = (int32_t)(row0 + at / (uint32_t)V);
    }
  }
  for (int i = found + tid; i < C; i += kRankThreads) {
    const int64_t to = group * C + i;
    b.top_scores[to] = -INFINITY;
    b.top_ids[to] = -1;
    b.top_parents[to] = -1;
  }
}

}  // namespace

// Vocabulary rows of a workgroup of the streaming kernels: above 64 tokens at
// most 128. 192 still leave registers for two workgroups a CU, but those of a
// large vocabulary then take two rounds, the second half empty (128 tokens, H
// 2560, V 151936: 198 us where 128 rows take 188 and 64 rows 237).
int beam_few_rows(int64_t N, int64_t V) { return N <= 64 ? few_rows(V) : std::min(few_rows(V), 128); }

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
    a.splits = b.splits;
    auto launch = [&](auto mb, auto nb) {
      a.tiles = (b.N + 16 * nb() - 1) / (16 * nb());
      const dim3 grid(few_grid((int64_t)a.tiles * a.splits));
      if (b.allowed != nullptr) hipLaunchKernelGGL((beam_few_kernel<mb(), nb(), true>), grid, dim3(256), 0, stream, a, b);
      else hipLaunchKernelGGL((beam_few_kernel<mb(), nb(), false>), grid, dim3(256), 0, stream, a, b);
    };
    constexpr std::integral_constant<int, 8> eight{};
    const int mb = beam_few_rows(b.N, b.V) / 64;
    if (b.N <= 64) with_sizes(mb, b.N <= 16 ? 1 : b.N <= 32 ? 2 : 4, launch);
    else if (mb == 2) launch(std::integral_constant<int, 2>{}, eight);
    else launch(std::integral_constant<int, 1>{}, eight);
  } else {
    const dim3 grid((unsigned)(((int64_t)b.n_tt * b.splits + 7) / 8 * 8));
    auto tiles = [&](auto mask) {
      hipLaunchKernelGGL((beam_tile_kernel<mask()>), grid, dim3(kThreads), 0, stream, b.hidden, b.W, b.allowed, (int)b.mask_ld, b.N,
                         b.H, b.V, b.splits, b.n_tt, b.n_vt, b.sc, b.records, b.sections, b.blocks, (int)b.ld);
    };
    b.allowed != nullptr ? tiles(std::true_type{}) : tiles(std::false_type{});
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
  hipLaunchKernelGGL(beam_score_kernel, dim3((unsigned)(b.keep * groups)), dim3(256), 0, stream, b);
  e = hipGetLastError();
  if (e != hipSuccess) return e;
  trace_end(kBeamScore, stream, 32.0 * groups * b.C * H, 34.0 * groups * b.C * H);
  trace_begin(stream);
  hipLaunchKernelGGL(beam_rank_kernel, dim3((unsigned)groups), dim3(kRankThreads), 0, stream, b);
  e = hipGetLastError();
  if (e != hipSuccess) return e;
  trace_end(kBeamRank, stream, 0.0, 140.0 * groups * b.C);
  return hipSuccess;
}

// ---------------------------------------------------------------------------
// Reordering: rows of `runs` runs of `run_bytes` each, of which the first
// lengths[parent] * step_bytes are in use (all without lengths). A wave takes 64
// places of 16 bytes, at which it first reads what up to 16 rows of the group
// take over, and then writes it. In place every read of a place so comes before
// any write: larger groups take several waves of a workgroup and a barrier
// between. Which row takes from which, and how much, is the same for all lanes.
// Bound by memory: 64 beams' caches of 34 MB, in use in part (1.30 GB read and
// written in place), 304 us, 4.3 TB/s; 24 states of 1024
// rows of 16 KB into other buffers (631 MB, parents read once for all their
// children) 118 us, 5.3 TB/s; a history of 512 words 2.4 us.
// Outputs larger than the near caches are stored past them (states 118 us instead
// of 128, caches 307 of 322); loads past them as well take 3% less at 1.3 GB but
// 10 to 30% more where the far cache still holds the states (64 MB: 21 us to 17).
namespace {

constexpr int kReorderRows = 16;

typedef uint32_t u32x4a __attribute__((ext_vector_type(4), aligned(1)));

// The first n < 16 bytes at p, the lowest byte first, and back.
__device__ __forceinline__ u32x4a load_bytes(const char* p, uint32_t n) {
  uint64_t lo = 0, hi = 0;
  for (uint32_t k = n; k-- > 0;) {
    hi = (hi << 8) | (lo >> 56);
    lo = (lo << 8) | (uint8_t)p[k];
  }
  return u32x4a{(uint32_t)lo, (uint32_t)(lo >> 32), (uint32_t)hi, (uint32_t)(hi >> 32)};
}
__device__ __forceinline__ void store_bytes(char* p, uint32_t n, u32x4a v) {
  uint64_t lo = v.x | (uint64_t)v.y << 32, hi = v.z | (uint64_t)v.w << 32;
  for (uint32_t k = 0; k < n; ++k) {
    p[k] = (char)lo;
    lo = (lo >> 8) | (hi << 56);
    hi >>= 8;
  }
}

// TAIL: bytes in use are no multiple of 16 everywhere; those of a row's last
// place are taken one by one.
template <int RB, int WR, bool TAIL, bool STREAM>
__global__ __launch_bounds__(256) void beam_reorder_kernel(const ReorderArgs a) {
  constexpr int CW = 4 / WR;   // waves side by side
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int part = wave % WR;
  const int G = a.beams;
  const bool place = a.states == a.out;
  // block = ((plane, group), places)
  const uint32_t block = (uint32_t)xcd_remap(blockIdx.x, gridDim.x), pg = block / a.blocks, groups = (uint32_t)(a.rows / G);
  if (pg >= a.planes * groups) return;
  const int64_t plane = pg / groups, row0 = (int64_t)(pg - (uint32_t)plane * groups) * G;
  const int64_t row_bytes = a.runs * a.run_bytes;
  const int64_t base = (plane * a.rows + row0) * row_bytes;
  const char* in = static_cast<const char*>(a.states) + base;
  char* out = static_cast<char*>(a.out) + base + part * RB * row_bytes;
  int from[RB];
  uint32_t whole[RB], rest[RB];   // places of a run that the row takes over, and bytes of one more
#pragma unroll
  for (int j = 0; j < RB; ++j) {
    const int row = part * RB + j;
    const int p = row < G ? (int)(a.parents[row0 + row] - row0) : -1;   // rows stay below 2^31
    const bool takes = p >= 0 && p < G && !(place && p == row);
    from[j] = takes ? p : 0;
    int64_t n = takes ? a.run_bytes : 0;
    if (takes && a.lengths != nullptr) {
      const int64_t len = a.lengths[row0 + p];
      n = (len < 0 ? 0 : len > a.steps ? a.steps : len) * a.step_bytes;
    }
    whole[j] = (uint32_t)(n >> 4);
    rest[j] = (uint32_t)n & 15;
  }
  const int64_t units = a.runs * a.places;
  const int64_t unit = (int64_t)(block - pg * a.blocks) * (64 * CW) + (wave / WR) * 64 + lane;
  uint32_t at = (uint32_t)unit;   // the place in the run; a run has less than 2^32
  int64_t offset = unit * 16;     // in the row
  if (a.runs > 1) {
    const int64_t run = units >> 32 ? unit / a.places : (int64_t)((uint32_t)unit / (uint32_t)a.places);
    at = (uint32_t)(unit - run * a.places);
    offset = run * a.run_bytes + (int64_t)at * 16;
  }
  if (unit >= units) at = ~0u;   // past the row: nothing is in use there
  u32x4a v[RB];
#pragma unroll
  for (int j = 0; j < RB; ++j) {
    if (j > 0 && from[j] == from[j - 1] && whole[j] == whole[j - 1] && rest[j] == rest[j - 1]) {
      v[j] = v[j - 1];   // children of one parent come one after the other
      continue;
    }
    const char* p = in + from[j] * row_bytes + offset;
    if (at < whole[j]) v[j] = *reinterpret_cast<const u32x4a*>(p);
    else if (TAIL && at == whole[j]) v[j] = load_bytes(p, rest[j]);
  }
  if (WR > 1 && place) __syncthreads();
#pragma unroll
  for (int j = 0; j < RB; ++j) {
    char* p = out + j * row_bytes + offset;
    if (at < whole[j]) {
      if (STREAM) __builtin_nontemporal_store(v[j], reinterpret_cast<u32x4a*>(p));
      else *reinterpret_cast<u32x4a*>(p) = v[j];
    }
    if (TAIL && at == whole[j]) store_bytes(p, rest[j], v[j]);
  }
}

}  // namespace

// Waves of a workgroup that share the group's rows, 16 each.
static int reorder_waves(int64_t beams) { return beams <= kReorderRows ? 1 : beams <= 2 * kReorderRows ? 2 : 4; }

int64_t reorder_blocks(int64_t planes, int64_t rows, int64_t beams, int64_t runs, int64_t run_bytes) {
  const int64_t at_once = 64 * (4 / reorder_waves(beams));
  return planes * (rows / beams) * ((runs * ((run_bytes + 15) / 16) + at_once - 1) / at_once);
}

hipError_t launch_beam_reorder(ReorderArgs a, hipStream_t stream) {
  a.run_bytes = a.steps * a.step_bytes;
  a.places = (a.run_bytes + 15) / 16;
  const int64_t groups = a.planes * (a.rows / a.beams), blocks = reorder_blocks(a.planes, a.rows, a.beams, a.runs, a.run_bytes);
  if (blocks == 0) return hipSuccess;
  a.blocks = (uint32_t)(blocks / groups);
  trace_begin(stream);
  const bool streamed = (double)a.planes * a.rows * a.runs * a.run_bytes > kStreamed;
  auto launch = [&](auto rb, auto wr) {
    const dim3 grid((unsigned)((blocks + 7) / 8 * 8));
    auto kind = [&](auto tail, auto past) {
      hipLaunchKernelGGL((beam_reorder_kernel<rb(), wr(), tail(), past()>), grid, dim3(256), 0, stream, a);
    };
    std::true_type yes;
    std::false_type no;
    if (a.step_bytes % 16 != 0) streamed ? kind(yes, yes) : kind(yes, no);
    else streamed ? kind(no, yes) : kind(no, no);
  };
  constexpr std::integral_constant<int, 1> one{};
  constexpr std::integral_constant<int, kReorderRows> most{};
  const int waves = reorder_waves(a.beams);
  if (a.beams <= 4) launch(std::integral_constant<int, 4>{}, one);
  else if (a.beams <= 8) launch(std::integral_constant<int, 8>{}, one);
  else if (waves == 1) launch(most, one);
  else if (waves == 2) launch(most, std::integral_constant<int, 2>{});
  else launch(most, std::integral_constant<int, 4>{});
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  trace_end(kBeamReorder, stream, 0.0, 2.0 * a.planes * a.rows * a.runs * (double)a.run_bytes);
  return hipSuccess;
}

}  // namespace lmh
