// lmhead_norm.hip -- the norm in front of the head (layer norm, or the RMS
// form without a mean), forward and backward, for gfx950.
//
//   mu = mean_j x_j (0 for RMS),  r = 1 / sqrt(mean_j (x_j - mu)^2 + eps)
//   xh = (x - mu) r,  y = xh w + b
//   g = dy w,  dx = r (g - mean_j g - xh mean_j (g xh))   (RMS: without mean g)
//   dw = sum_i dy_i xh_i,  db = sum_i dy_i
//
// Both passes are bound by HBM: every row is read once into registers, its
// statistics are taken there (the variance from the centred values, so a
// large mean costs no digits), and its outputs are written from there. All
// arithmetic is float32; bf16 outputs are rounded once, when stored.
//
// Measured (bf16, layer norm; a copy of 2 GB reaches 5.0 TB/s): 65536 x 2560
// forward 137 us (4.9 TB/s), backward 189 us (5.3 TB/s) and 5 us for the sums of
// the partial rows; 65536 x 256 12.5 and 24 us; one row 2.7 us forward.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include <algorithm>
#include <type_traits>

#include "lmhead_internal.h"

namespace lmh {
namespace {

// v_mul_legacy_f32: +0 when either factor is 0 (NaN and inf included), else IEEE.
// A zero of dy is to contribute 0 whatever lies beside it, at no cost; a NaN or an
// infinity of dy beside a 0 is to give NaN, and what it reaches is taken again.
extern "C" __device__ float lmh_norm_fmul_legacy(float, float) __asm("llvm.amdgcn.fmul.legacy");
__device__ __forceinline__ float mul0(float a, float b) { return lmh_norm_fmul_legacy(a, b); }

__device__ __forceinline__ float widen(uint16_t b) { return __uint_as_float((uint32_t)b << 16); }
template <bool F32>
__device__ __forceinline__ float element(const void* p, int64_t i) {
  return F32 ? static_cast<const float*>(p)[i] : widen(static_cast<const uint16_t*>(p)[i]);
}
__device__ __forceinline__ bool finite(float v) { return fabsf(v) < INFINITY; }

// a column's sum of dy xh over rows row, row + step, ..., IEEE's product for
// every element of dy but a zero
template <bool XF32, bool YF32>
__device__ float ieee_column(const NormBwdArgs& a, int j, int64_t row, int64_t step) {
  float u = 0.0f;
  for (; row < a.N; row += step) {
    const float dy = element<YF32>(a.dy, row * a.H + j);
    if (dy != 0.0f) u += dy * ((element<XF32>(a.x, row * a.H + j) - (a.rms ? 0.0f : a.mean[row])) * a.rstd[row]);
  }
  return u;
}
__device__ __forceinline__ uint16_t narrow(float x) { return __builtin_bit_cast(uint16_t, (__bf16)x); }
__device__ __forceinline__ uint32_t narrow2(float lo, float hi) {
  return (uint32_t)narrow(lo) | ((uint32_t)narrow(hi) << 16);
}

// Accesses of 8 and 16 bytes at element alignment: rows of an odd length
// start off any larger boundary, which global memory accepts (a split access
// costs a second request, where element-wide ones would cost up to eight).
template <int WORDS>
struct __attribute__((packed, aligned(2))) Raw {
  uint32_t w[WORDS];
};

// How a row of H elements lies over its threads: in groups of G elements,
// group i * threads + t being thread t's i-th, so that each load of a wave
// covers one piece of memory. G is 8 (16 bytes of bf16) where x is bf16 and 4
// (16 bytes) where it is float32; a thread holds 8 NV elements either way.
template <bool F32, int G>
struct Group {
  Raw<G * (F32 ? 4 : 2) / 4> raw;
  __device__ __forceinline__ float at(int k) const {
    if (F32) return __uint_as_float(raw.w[k]);
    const uint32_t w = raw.w[k / 2];
    return __uint_as_float((k & 1) ? (w & 0xFFFF0000u) : (w << 16));
  }
  __device__ __forceinline__ void set(const float (&v)[G]) {
#pragma unroll
    for (int k = 0; k < G; k += F32 ? 1 : 2) raw.w[F32 ? k : k / 2] = F32 ? __float_as_uint(v[k]) : narrow2(v[k], v[k + 1]);
  }
};

// A thread's part of a row as it lies in memory. Every thread issues all its
// loads before it uses any (groups past the last whole one reread that one;
// zero() drops them): a branch per group would wait for each load in turn. A
// last group of fewer elements is read by elements.
template <bool F32, int G, int NG>
struct Part {
  Group<F32, G> g[NG];
  __device__ __forceinline__ void load(const void* base, int64_t row, int H, int t, int threads) {
    const int whole = H / G;
    const char* p = static_cast<const char*>(base) + row * H * (F32 ? 4 : 2);
    constexpr int bytes = G * (F32 ? 4 : 2);
#pragma unroll
    for (int i = 0; i < NG; ++i) {
      const int c = min(i * threads + t, whole - 1);
      if (whole > 0) g[i].raw = *reinterpret_cast<const decltype(g[i].raw)*>(p + (int64_t)c * bytes);
    }
    if (H % G != 0) {
#pragma unroll
      for (int i = 0; i < NG; ++i) {
        if (i * threads + t != whole) continue;
        float v[G];
#pragma unroll
        for (int k = 0; k < G; ++k) {
          v[k] = 0.0f;
          if (k < H % G) v[k] = F32 ? reinterpret_cast<const float*>(p)[whole * G + k]
                                    : widen(reinterpret_cast<const uint16_t*>(p)[whole * G + k]);
        }
        g[i].set(v);
      }
    }
  }
  __device__ __forceinline__ void fill(float x) {
    float v[G];
#pragma unroll
    for (int k = 0; k < G; ++k) v[k] = x;
#pragma unroll
    for (int i = 0; i < NG; ++i) g[i].set(v);
  }
};

template <bool F32, int G, int NG>
__device__ __forceinline__ void store_part(void* base, int64_t row, int H, int t, int threads, const float (&v)[NG][G]) {
  const int whole = H / G;
  char* p = static_cast<char*>(base) + row * H * (F32 ? 4 : 2);
  constexpr int bytes = G * (F32 ? 4 : 2);
#pragma unroll
  for (int i = 0; i < NG; ++i) {
    const int c = i * threads + t;
    Group<F32, G> o;
    o.set(v[i]);
    if (c < whole) *reinterpret_cast<decltype(o.raw)*>(p + (int64_t)c * bytes) = o.raw;
  }
  if (H % G != 0) {
#pragma unroll
    for (int i = 0; i < NG; ++i) {
      if (i * threads + t != whole) continue;
#pragma unroll
      for (int k = 0; k < G - 1; ++k)
        if (k < H % G) {
          if (F32) reinterpret_cast<float*>(p)[whole * G + k] = v[i][k];
          else reinterpret_cast<uint16_t*>(p)[whole * G + k] = narrow(v[i][k]);
        }
    }
  }
}

// Sum over LANES lanes (16, 32 or 64) in a fixed order, on the vector unit alone
// up to 16 (data-parallel moves within rows of 16 lanes; then across rows).
// Every one of them gets the sum.
template <int CTRL, int ROWS>
__device__ __forceinline__ float dpp_add(float v) {
  const int o = __builtin_amdgcn_update_dpp(0, __float_as_int(v), CTRL, ROWS, 0xF, false);
  return v + __int_as_float(o);
}
template <int LANES>
__device__ __forceinline__ float lane_sum(float v) {
  v = dpp_add<0xB1, 0xF>(v);    // lanes ^ 1
  v = dpp_add<0x4E, 0xF>(v);    // lanes ^ 2
  v = dpp_add<0x141, 0xF>(v);   // the other four of eight
  v = dpp_add<0x140, 0xF>(v);   // the other eight of the row
  if (LANES == 32) v += __shfl_xor(v, 16);
  if (LANES == 64) {
    v = dpp_add<0x142, 0xA>(v);   // rows 1 and 3 add rows 0 and 2
    v = dpp_add<0x143, 0xC>(v);   // rows 2 and 3 add row 1's
    v = __int_as_float(__builtin_amdgcn_readlane(__float_as_int(v), 63));
  }
  return v;
}

// Sums of two values over the threads of a row: LANES lanes, or (WIDE, a block
// per row) the wave, then the waves' sums through LDS in order. The two halves
// of `s` alternate between calls, so one barrier a call is enough.
constexpr int kMaxWaves = 16;
constexpr int kWide = 0, kHuge = -1;   // LANES of a block per row: up to 512 threads, up to 1024
template <int LANES>
__device__ __forceinline__ void row_sum2(float& a, float& b, bool two, float (*s)[kMaxWaves][2], int& turn) {
  a = lane_sum<LANES <= 0 ? 64 : LANES>(a);
  if (two) b = lane_sum<LANES <= 0 ? 64 : LANES>(b);
  if (LANES <= 0) {
    const int waves = blockDim.x >> 6;
    if ((threadIdx.x & 63) == 0) {
      s[turn][threadIdx.x >> 6][0] = a;
      s[turn][threadIdx.x >> 6][1] = b;
    }
    __syncthreads();
    a = s[turn][0][0];
    b = s[turn][0][1];
    for (int i = 1; i < waves; ++i) {
      a += s[turn][i][0];
      b += s[turn][i][1];
    }
    turn ^= 1;
  }
}

// Forward: a row's threads (LANES lanes, or kWide the block) walk rows `step`
// apart, the weights in registers, the next row's loads in flight while the
// present one is worked on.
template <bool XF32, bool YF32, bool WF32, int NV, int LANES>
__global__ __launch_bounds__(LANES == kHuge ? 1024 : 512) void norm_fwd_kernel(const NormFwdArgs a) {
  constexpr int G = XF32 ? 4 : 8, NG = 8 * NV / G;
  __shared__ float s[2][kMaxWaves][2];
  constexpr bool WIDE = LANES <= 0;
  const int threads = WIDE ? blockDim.x : LANES;
  const int t = WIDE ? threadIdx.x : threadIdx.x % (WIDE ? 1 : LANES);
  const int per = WIDE ? 1 : blockDim.x / threads;
  const int64_t step = (int64_t)gridDim.x * per;
  const int H = a.H;
  const float inv = 1.0f / (float)H;
  int turn = 0;
  Part<WF32, G, NG> w, b;
  if (a.w != nullptr) w.load(a.w, 0, H, t, threads); else w.fill(1.0f);
  if (a.b != nullptr) b.load(a.b, 0, H, t, threads); else b.fill(0.0f);
  int64_t row = (int64_t)blockIdx.x * per + (WIDE ? 0 : threadIdx.x / threads);
  Part<XF32, G, NG> next;
  if (row < a.N) next.load(a.x, row, H, t, threads);
  for (; row < a.N; row += step) {
    float x[NG][G];
    bool in[NG][G];   // past the row's end nothing counts
#pragma unroll
    for (int i = 0; i < NG; ++i)
#pragma unroll
      for (int k = 0; k < G; ++k) {
        in[i][k] = G * (i * threads + t) + k < H;
        x[i][k] = in[i][k] ? next.g[i].at(k) : 0.0f;
      }
    if (row + step < a.N) next.load(a.x, row + step, H, t, threads);
    float mu = 0.0f, none = 0.0f;
    if (!a.rms) {
#pragma unroll
      for (int i = 0; i < NG; ++i)
#pragma unroll
        for (int k = 0; k < G; ++k) mu += x[i][k];
      row_sum2<LANES>(mu, none, false, s, turn);
      mu *= inv;
    }
    float q = 0.0f;
#pragma unroll
    for (int i = 0; i < NG; ++i)
#pragma unroll
      for (int k = 0; k < G; ++k) {
        x[i][k] -= mu;
        q = in[i][k] ? fmaf(x[i][k], x[i][k], q) : q;
      }
    row_sum2<LANES>(q, none, false, s, turn);
    const float r = 1.0f / sqrtf(fmaf(q, inv, a.eps));
#pragma unroll
    for (int i = 0; i < NG; ++i)
#pragma unroll
      for (int k = 0; k < G; ++k) x[i][k] = fmaf(x[i][k] * r, w.g[i].at(k), b.g[i].at(k));
    store_part<YF32, G, NG>(a.y, row, H, t, threads, x);
    if (t == 0) {
      if (a.mean != nullptr && !a.rms) a.mean[row] = mu;
      if (a.rstd != nullptr) a.rstd[row] = r;
    }
  }
}

// dw or db of one column, as norm_reduce_kernel and the columns' workgroups store it.
__device__ __forceinline__ void store_sum(void* out, bool f32, bool accumulate, int c, float u) {
  if (out == nullptr) return;
  if (f32) {
    float* o = static_cast<float*>(out) + c;
    *o = accumulate ? *o + u : u;
  } else {
    uint16_t* o = static_cast<uint16_t*>(out) + c;
    *o = narrow(accumulate ? widen(*o) + u : u);
  }
}

// dw and db of 32 columns over all rows, read from x and dy themselves: 8 lanes
// of 4 columns a row, each thread the rows blockDim / 8 apart, then the lanes of
// a column by halves and the waves in order.
constexpr int kSumCols = 32;
template <bool XF32, bool YF32>
__device__ __forceinline__ void norm_columns(const NormBwdArgs& a, int block, float* lds) {
  const int lane = threadIdx.x & 63;
  const int H = a.H;
  const int c = block * kSumCols + 4 * (lane & 7);
  float dw[4] = {0.0f, 0.0f, 0.0f, 0.0f}, db[4] = {0.0f, 0.0f, 0.0f, 0.0f};
  const int64_t step = blockDim.x / 8;
  const char* px = static_cast<const char*>(a.x) + (int64_t)c * (XF32 ? 4 : 2);
  const char* pg = static_cast<const char*>(a.dy) + (int64_t)c * (YF32 ? 4 : 2);
  const int64_t bx = (int64_t)H * (XF32 ? 4 : 2), bg = (int64_t)H * (YF32 ? 4 : 2);
  if (c + 3 < H) {
#pragma unroll 4
    for (int64_t row = threadIdx.x / 8; row < a.N; row += step) {
      Group<XF32, 4> x;
      Group<YF32, 4> g;
      x.raw = *reinterpret_cast<const decltype(x.raw)*>(px + row * bx);
      g.raw = *reinterpret_cast<const decltype(g.raw)*>(pg + row * bg);
      const float mu = a.rms ? 0.0f : a.mean[row], r = a.rstd[row];
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        dw[k] += mul0(g.at(k), (x.at(k) - mu) * r);
        db[k] += g.at(k);
      }
    }
  } else {
    for (int64_t row = threadIdx.x / 8; row < a.N; row += step) {
      const float mu = a.rms ? 0.0f : a.mean[row], r = a.rstd[row];
#pragma unroll
      for (int k = 0; k < 3; ++k) {
        if (c + k >= H) continue;
        const float x = XF32 ? reinterpret_cast<const float*>(px + row * bx)[k]
                             : widen(reinterpret_cast<const uint16_t*>(px + row * bx)[k]);
        const float g = YF32 ? reinterpret_cast<const float*>(pg + row * bg)[k]
                             : widen(reinterpret_cast<const uint16_t*>(pg + row * bg)[k]);
        dw[k] += mul0(g, (x - mu) * r);
        db[k] += g;
      }
    }
  }
#pragma unroll
  for (int k = 0; k < 4; ++k)
    if (__builtin_expect(!finite(db[k]), 0)) dw[k] = ieee_column<XF32, YF32>(a, c + k, threadIdx.x / 8, step);
  const int wave = threadIdx.x >> 6, waves = blockDim.x >> 6;
#pragma unroll
  for (int k = 0; k < 4; ++k) {
#pragma unroll
    for (int x = 8; x <= 32; x <<= 1) {
      dw[k] += __shfl_xor(dw[k], x);
      db[k] += __shfl_xor(db[k], x);
    }
    if (lane < 8) {
      lds[wave * 2 * kSumCols + 4 * lane + k] = dw[k];
      lds[wave * 2 * kSumCols + kSumCols + 4 * lane + k] = db[k];
    }
  }
  __syncthreads();
  const int col = block * kSumCols + threadIdx.x % kSumCols;
  if (threadIdx.x >= 2 * kSumCols || col >= H) return;
  float u = lds[threadIdx.x];
  for (int i = 1; i < waves; ++i) u += lds[i * 2 * kSumCols + threadIdx.x];
  store_sum(threadIdx.x < kSumCols ? a.dw : a.db, a.g_f32, a.accumulate, col, u);
}

// Backward: rows are walked likewise and each thread keeps its columns' sums
// of dw and db in registers; at the end the rows of a block are added through
// LDS in order and the block writes one partial row of each ([blocks][2][H]),
// which norm_reduce_kernel sums in block order; with few rows, workgroups past
// the rows' own sum the columns instead, and there are no partial rows. A zero in dy contributes a
// zero whatever x, the statistics and w hold there (mul0), so a masked token,
// whose dy row is 0, adds nothing and gets dx = 0 even where its x is NaN.
// The same product drops a NaN or an infinity of dy beside a 0 of xh or w: at the
// end a workgroup (or wave) that met one forms again what that reaches, as IEEE
// has it. Asking costs 0.1 us of a small call and 1% of a large one.
template <bool XF32, bool YF32, bool WF32, int NV, int LANES>
__global__ __launch_bounds__(LANES == kHuge ? 1024 : 512) void norm_bwd_kernel(const NormBwdArgs a) {
  constexpr int G = XF32 ? 4 : 8, NG = 8 * NV / G;
  extern __shared__ float lds[];   // [2][H]: the block's dw and db (LANES > 0); a columns' workgroup: [waves][2][32]
  if ((int)blockIdx.x >= a.row_blocks) {
    norm_columns<XF32, YF32>(a, (int)blockIdx.x - a.row_blocks, lds);
    return;
  }
  // 1024 threads have 128 registers each, which the sums would overflow: there
  // they live in LDS, each thread's at its own columns. Float32 rows still spill one
  // to four registers, outside the loop over rows: 4096 x 16384 take 168 us with float32
  // dy (4.8 TB/s), 148 with bf16 (4.5); bf16 rows 92 (4.4)
  constexpr bool kept = LANES == kHuge;
  __shared__ __attribute__((aligned(16))) float sums[2][kept ? kNormMaxH : 4];
  __shared__ float s[2][kMaxWaves][2];
  constexpr bool WIDE = LANES <= 0;
  const int threads = WIDE ? blockDim.x : LANES;
  const int t = WIDE ? threadIdx.x : threadIdx.x % (WIDE ? 1 : LANES);
  const int per = WIDE ? 1 : blockDim.x / threads;
  const int slot = WIDE ? 0 : threadIdx.x / threads;
  const int64_t step = (int64_t)a.row_blocks * per;
  const int H = a.H;
  const float inv = 1.0f / (float)H;
  int turn = 0;
  Part<WF32, G, NG> w;
  if (a.w != nullptr) w.load(a.w, 0, H, t, threads); else w.fill(1.0f);
  float dw[NG][G], db[NG][G];
#pragma unroll
  for (int i = 0; i < NG; ++i)
#pragma unroll
    for (int k = 0; k < G; ++k) {
      dw[i][k] = db[i][k] = 0.0f;
      if (kept) sums[0][G * (i * threads + t) + k] = sums[1][G * (i * threads + t) + k] = 0.0f;   // 16 a thread: within kNormMaxH
    }
  const int64_t first = (int64_t)blockIdx.x * per + slot;
  int64_t row = first;
  bool bad = false;   // something here is not finite
  Part<XF32, G, NG> nx;
  Part<YF32, G, NG> ng;
  float n_mu = 0.0f, n_r = 0.0f;
  auto fetch = [&](int64_t at) {
    nx.load(a.x, at, H, t, threads);
    ng.load(a.dy, at, H, t, threads);
    if (!a.rms) n_mu = a.mean[at];
    n_r = a.rstd[at];
  };
  if (row < a.N) fetch(row);
  for (; row < a.N; row += step) {
    float x[NG][G], g[NG][G];
    const float mu = n_mu, r = n_r;
#pragma unroll
    for (int i = 0; i < NG; ++i)
#pragma unroll
      for (int k = 0; k < G; ++k) {
        const bool in = G * (i * threads + t) + k < H;
        x[i][k] = nx.g[i].at(k);
        g[i][k] = in ? ng.g[i].at(k) : 0.0f;
      }
    if (row + step < a.N) fetch(row + step);
    float c1 = 0.0f, c2 = 0.0f;
#pragma unroll
    for (int i = 0; i < NG; ++i)
#pragma unroll
      for (int k = 0; k < G; ++k) {
        const float xh = (x[i][k] - mu) * r;
        if (kept) {
          const int j = G * (i * threads + t) + k;
          sums[0][j] += mul0(g[i][k], xh);
          sums[1][j] += g[i][k];
        } else {
          dw[i][k] += mul0(g[i][k], xh);
          db[i][k] += g[i][k];
        }
        const float gw = mul0(g[i][k], w.g[i].at(k));
        c1 += mul0(gw, xh);
        c2 += gw;
        x[i][k] = xh;
        g[i][k] = gw;
      }
    row_sum2<LANES>(c1, c2, !a.rms, s, turn);
    c1 *= inv;
    c2 = a.rms ? 0.0f : c2 * inv;
    bad |= !(finite(c1) && finite(c2)) || r == 0.0f;   // r is 0 beside an infinite x
#pragma unroll
    for (int i = 0; i < NG; ++i)
#pragma unroll
      for (int k = 0; k < G; ++k) x[i][k] = mul0(r, (g[i][k] - c2) - mul0(x[i][k], c1));
    store_part<XF32, G, NG>(a.dx, row, H, t, threads, x);
  }
#pragma unroll
  for (int i = 0; i < NG; ++i)
#pragma unroll
    for (int k = 0; k < G; ++k) bad |= !finite(kept ? sums[1][G * (i * threads + t) + k] : db[i][k]);
  if (__builtin_expect(WIDE ? __syncthreads_or(bad) : __any(bad), 0)) {
    int tc = t;
    int64_t from = first;
    asm volatile("" : "+v"(tc), "+v"(from));   // nothing of this is worth a register of the loop above
    // the columns with such a dy, whose db is not finite, and the rows with such a
    // dy or x, whose c1 is not or whose r is 0: element by element
    if (a.part != nullptr) {
#pragma unroll
      for (int i = 0; i < NG; ++i)
#pragma unroll
        for (int k = 0; k < G; ++k) {
          const int j = G * (i * threads + tc) + k;
          if (finite(kept ? sums[1][j] : db[i][k])) continue;
          const float u = ieee_column<XF32, YF32>(a, j, from, step);
          if (kept) sums[0][j] = u;
          else dw[i][k] = u;
        }
    }
    for (row = from; row < a.N; row += step) {
      const float mu = a.rms ? 0.0f : a.mean[row], r = a.rstd[row];
      auto each = [&](auto f) {   // f(column, dy, xh, dy weight)
#pragma unroll 1
        for (int e = 0; e < NG * G; ++e) {
          const int j = G * (e / G * threads + tc) + e % G;
          if (j >= H) continue;
          const float dy = element<YF32>(a.dy, row * H + j);
          const float wt = a.w != nullptr ? element<WF32>(a.w, j) : 1.0f;
          f(j, dy, (element<XF32>(a.x, row * H + j) - mu) * r, dy != 0.0f ? dy * wt : 0.0f);
        }
      };
      float c1 = 0.0f, c2 = 0.0f, some = 0.0f, none = 0.0f;
      each([&](int, float dy, float xh, float gw) {
        if (dy != 0.0f) {
          c1 += gw * xh;
          some = 1.0f;
        }
        c2 += gw;
      });
      row_sum2<LANES>(c1, c2, !a.rms, s, turn);
      row_sum2<LANES>(some, none, false, s, turn);
      c1 *= inv;
      c2 = a.rms ? 0.0f : c2 * inv;
      if (some == 0.0f || (finite(c1) && finite(c2) && r != 0.0f)) continue;   // masked, or no different above
      each([&](int j, float, float xh, float gw) {
        const float v = r * ((gw - c2) - xh * c1);
        if (XF32) static_cast<float*>(a.dx)[row * H + j] = v;
        else static_cast<uint16_t*>(a.dx)[row * H + j] = narrow(v);
      });
    }
  }
  if (a.part == nullptr) return;
  float* out = a.part + (int64_t)blockIdx.x * 2 * H;
  if (WIDE) {
    if (kept) {
#pragma unroll
      for (int i = 0; i < NG; ++i)
#pragma unroll
        for (int k = 0; k < G; ++k) {
          const int j = G * (i * threads + t) + k;
          dw[i][k] = sums[0][j];
          db[i][k] = sums[1][j];
        }
    }
    store_part<true, G, NG>(out, 0, H, t, threads, dw);
    store_part<true, G, NG>(out + H, 0, H, t, threads, db);
    return;
  }
  // the rows of a wave by halves, then the waves in order
  if (LANES < 64) {
#pragma unroll
    for (int i = 0; i < NG; ++i)
#pragma unroll
      for (int k = 0; k < G; ++k)
#pragma unroll
        for (int x = 32; x >= (WIDE ? 64 : LANES); x >>= 1) {
          dw[i][k] += __shfl_xor(dw[i][k], x);
          db[i][k] += __shfl_xor(db[i][k], x);
        }
  }
  const int waves = blockDim.x >> 6;
  const bool first_rows = (threadIdx.x & 63) < threads;
  for (int i0 = 0; i0 < waves; ++i0) {
    if (first_rows && (int)(threadIdx.x >> 6) == i0) {
#pragma unroll
      for (int i = 0; i < NG; ++i)
#pragma unroll
        for (int k = 0; k < G; ++k) {
          const int j = G * (i * threads + t) + k;
          if (j >= H) continue;
          if (i0 > 0) {
            dw[i][k] += lds[j];
            db[i][k] += lds[H + j];
          }
          if (i0 < waves - 1) {
            lds[j] = dw[i][k];
            lds[H + j] = db[i][k];
          } else {
            out[j] = dw[i][k];
            out[H + j] = db[i][k];
          }
        }
    }
    __syncthreads();
  }
}

// Sums the blocks' partial rows [blocks][2 H]: a workgroup takes 32 columns
// (128 bytes of each row), its 1024 threads as 128 groups of 8 that sum every
// 128th row four columns at a time; the groups' sums are then added in order,
// 8 at a time, and those 16 in order.
constexpr int kRedThreads = 1024, kRedCols = 32, kRedGroups = kRedThreads / (kRedCols / 4);
__global__ __launch_bounds__(kRedThreads) void norm_reduce_kernel(const NormReduceArgs a) {
  __shared__ float s[kRedGroups][kRedCols];
  __shared__ float s2[kRedGroups / 8][kRedCols];
  const int n = 2 * a.H;
  const int group = threadIdx.x / (kRedCols / 4);
  const int c4 = 4 * (threadIdx.x % (kRedCols / 4));
  const int j = blockIdx.x * kRedCols + c4;   // column of [dw | db]
  float v[4] = {0.0f, 0.0f, 0.0f, 0.0f};
  if (j + 3 < n) {
#pragma unroll 4
    for (int i = group; i < a.blocks; i += kRedGroups) {
      const Raw<4> p = *reinterpret_cast<const Raw<4>*>(a.part + (int64_t)i * n + j);
#pragma unroll
      for (int k = 0; k < 4; ++k) v[k] += __uint_as_float(p.w[k]);
    }
  } else {
    for (int i = group; i < a.blocks; i += kRedGroups)
      for (int k = 0; k < 4; ++k)
        if (j + k < n) v[k] += a.part[(int64_t)i * n + j + k];
  }
#pragma unroll
  for (int k = 0; k < 4; ++k) s[group][c4 + k] = v[k];
  __syncthreads();
  const int col = threadIdx.x % kRedCols, part = threadIdx.x / kRedCols;
  if (part < kRedGroups / 8) {
    float u = s[8 * part][col];
#pragma unroll
    for (int i = 1; i < 8; ++i) u += s[8 * part + i][col];
    s2[part][col] = u;
  }
  __syncthreads();
  const int at = blockIdx.x * kRedCols + col;
  if (part != 0 || at >= n) return;
  float u = s2[0][col];
#pragma unroll
  for (int i = 1; i < kRedGroups / 8; ++i) u += s2[i][col];
  store_sum(at < a.H ? a.dw : a.db, a.g_f32, a.accumulate, at < a.H ? at : at - a.H, u);
}

// How rows of H are laid over threads. Up to 1024 elements 16 to 64 lanes of a
// wave per row (no barrier); above that a block per row, the forward with 16
// elements a thread (two loads in flight beside the next row's two; 65536 x 2560
// bf16: 137 us, with 8 168) and the backward, whose sums take registers too,
// with 8 up to 4096.
struct Shape {
  int nv, lanes;
  int block, per;   // threads per block, rows per block
};
Shape shape_of(int64_t H, bool backward) {
  if (H <= 1024) {
    const int lanes = H <= 128 ? 16 : H <= 256 ? 32 : 64;
    return {H <= 512 ? 1 : 2, lanes, 256, 256 / lanes};
  }
  const int nv = H <= 4096 && backward ? 1 : 2;
  return {nv, H <= 8192 ? kWide : kHuge, (int)((H + 8 * nv * 64 - 1) / (8 * nv * 64)) * 64, 1};
}

template <class F>
void with_shape(const Shape& p, F f) {
  constexpr std::integral_constant<int, 1> one{};
  constexpr std::integral_constant<int, 2> two{};
  constexpr std::integral_constant<int, kWide> wide{};
  constexpr std::integral_constant<int, kHuge> huge{};
  if (p.lanes == 16) f(one, std::integral_constant<int, 16>{});
  else if (p.lanes == 32) f(one, std::integral_constant<int, 32>{});
  else if (p.lanes == 64 && p.nv == 1) f(one, std::integral_constant<int, 64>{});
  else if (p.lanes == 64) f(two, std::integral_constant<int, 64>{});
  else if (p.lanes == kWide && p.nv == 1) f(one, wide);
  else if (p.lanes == kWide) f(two, wide);
  else f(two, huge);
}

// The types of x, y and the weights (float32 y comes with float32 x only).
template <class F>
void with_types(bool x, bool y, bool w, F f) {
  std::true_type yes;
  std::false_type no;
  if (x && y) w ? f(yes, yes, yes) : f(yes, yes, no);
  else if (x) w ? f(yes, no, yes) : f(yes, no, no);
  else w ? f(no, no, yes) : f(no, no, no);
}

constexpr int kWavesPerCU = 32;

}  // namespace

// A row per wave or block while that leaves at most a workgroup per CU, then
// 4 rows each up to 16 waves per CU.
int norm_bwd_blocks(int64_t N, int64_t H) {
  const Shape p = shape_of(H, true);
  const int64_t full = kNumCUs * std::max(1, 16 * 64 / p.block);
  const int64_t rows = (N + p.per - 1) / p.per;
  return (int)std::max<int64_t>(1, std::min(rows, std::max<int64_t>(kNumCUs, std::min((rows + 3) / 4, full))));
}

hipError_t launch_norm_fwd(const NormFwdArgs& a, hipStream_t stream) {
  const Shape p = shape_of(a.H, false);
  const int64_t blocks = std::min<int64_t>((a.N + p.per - 1) / p.per, kNumCUs * (kWavesPerCU * 64 / p.block));
  trace_begin(stream);
  with_types(a.x_f32, a.y_f32, a.w_f32, [&](auto x, auto y, auto w) {
    with_shape(p, [&](auto nv, auto lanes) {
      hipLaunchKernelGGL((norm_fwd_kernel<x(), y(), w(), nv(), lanes()>), dim3((unsigned)blocks), dim3(p.block), 0,
                         stream, a);
    });
  });
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  const double n = (double)a.N * a.H;
  trace_end(kNormFwd, stream, 8.0 * n, n * ((a.x_f32 ? 4 : 2) + (a.y_f32 ? 4 : 2)) + 8.0 * a.N);
  return hipSuccess;
}

// Whether the columns' workgroups read x and dy again (one launch) instead of
// the rows' leaving partial sums (two). Measured in a graph (us, columns /
// partial sums, bf16): 64 rows of 256 2.9 / 7.3, of 2560 3.1 / 6.0; 256 rows of 1024
// 4.3 / 10.0, of 8192 8.9 / 13.6; 512 rows of 2560 8.3 / 9.6, of 16384 25.0 / 25.4;
// 1024 rows of 256 9.8 / 7.6, of 2560 14.5 / 11.6. A call that enqueues them
// one by one saves 3 us of the second launch besides.
constexpr int64_t kColumnRows = 512;
bool norm_by_columns(int64_t N) { return N <= kColumnRows; }

hipError_t launch_norm_bwd(const NormBwdArgs& a, hipStream_t stream) {
  const Shape p = shape_of(a.H, true);
  const bool columns = a.dw != nullptr || a.db != nullptr;
  const int blocks = a.row_blocks + (columns ? (a.H + kSumCols - 1) / kSumCols : 0);
  const size_t lds = columns ? (size_t)p.block * kSumCols / 8 : p.lanes <= 0 ? 0 : (size_t)2 * a.H * 4;
  trace_begin(stream);
  with_types(a.x_f32, a.y_f32, a.w_f32, [&](auto x, auto y, auto w) {
    with_shape(p, [&](auto nv, auto lanes) {
      hipLaunchKernelGGL((norm_bwd_kernel<x(), y(), w(), nv(), lanes()>), dim3(blocks), dim3(p.block), lds, stream, a);
    });
  });
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  const double n = (double)a.N * a.H;
  trace_end(kNormBwd, stream, 14.0 * n, n * (2 * (a.x_f32 ? 4 : 2) + (a.y_f32 ? 4 : 2)) + 8.0 * a.N);
  return hipSuccess;
}

hipError_t launch_norm_reduce(const NormReduceArgs& a, hipStream_t stream) {
  trace_begin(stream);
  hipLaunchKernelGGL(norm_reduce_kernel, dim3((unsigned)((2 * a.H + kRedCols - 1) / kRedCols)), dim3(kRedThreads), 0,
                     stream, a);
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  trace_end(kNormReduce, stream, 0.0, 8.0 * a.blocks * (double)a.H + 8.0 * a.H);
  return hipSuccess;
}

}  // namespace lmh
