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
#include <hip/hip_runtime.h>
#include <stdint.h>

#include <algorithm>
#include <type_traits>

#include "lmhead_internal.h"

namespace lmh {
namespace {

constexpr int kBlock = 256;   // 4 waves

// v_mul_legacy_f32: +0 when either factor is 0 (NaN and inf included), else IEEE
extern "C" __device__ float lmh_norm_fmul_legacy(float, float) __asm("llvm.amdgcn.fmul.legacy");
__device__ __forceinline__ float mul0(float a, float b) { return lmh_norm_fmul_legacy(a, b); }

// 16-byte accesses at element alignment: rows of an odd length start off any
// larger boundary, which global memory accepts (a split access costs a second
// request, where element-wide loads would cost eight).
struct __attribute__((packed, aligned(2))) Raw8h {
  uint32_t w[4];
};
struct __attribute__((packed, aligned(4))) Raw4f {
  float f[4];
};

__device__ __forceinline__ float widen(uint16_t b) { return __uint_as_float((uint32_t)b << 16); }
__device__ __forceinline__ uint16_t narrow(float x) { return __builtin_bit_cast(uint16_t, (__bf16)x); }
__device__ __forceinline__ uint32_t narrow2(float lo, float hi) {
  return (uint32_t)narrow(lo) | ((uint32_t)narrow(hi) << 16);
}

// A row of H elements over TPR threads, widened: thread t holds NV chunks of 8
// elements, v[i] being row chunk i * TPR + t, 0 past the row's end. Every
// thread issues all its loads before it uses any (chunks past the last whole
// one reread that one and are dropped): a branch per chunk would wait for each
// load in turn. A last chunk of less than 8 is read by elements afterwards.
template <bool F32, int TPR, int NV>
__device__ __forceinline__ void load_row(const void* row, int H, int t, float (&v)[NV][8]) {
  const int whole = H >> 3;
  if (whole > 0) {
    if (F32) {
      Raw4f a[NV], b[NV];
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        const Raw4f* p = reinterpret_cast<const Raw4f*>(static_cast<const float*>(row) + 8 * min(i * TPR + t, whole - 1));
        a[i] = p[0];
        b[i] = p[1];
      }
#pragma unroll
      for (int i = 0; i < NV; ++i)
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          v[i][k] = a[i].f[k];
          v[i][4 + k] = b[i].f[k];
        }
    } else {
      Raw8h a[NV];
#pragma unroll
      for (int i = 0; i < NV; ++i)
        a[i] = *reinterpret_cast<const Raw8h*>(static_cast<const uint16_t*>(row) + 8 * min(i * TPR + t, whole - 1));
#pragma unroll
      for (int i = 0; i < NV; ++i)
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          v[i][2 * k] = __uint_as_float(a[i].w[k] << 16);
          v[i][2 * k + 1] = __uint_as_float(a[i].w[k] & 0xFFFF0000u);
        }
    }
  }
#pragma unroll
  for (int i = 0; i < NV; ++i)
#pragma unroll
    for (int k = 0; k < 8; ++k) v[i][k] = i * TPR + t < whole ? v[i][k] : 0.0f;
  if ((H & 7) != 0) {
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      if (i * TPR + t != whole) continue;
#pragma unroll
      for (int k = 0; k < 7; ++k)
        if (k < (H & 7)) v[i][k] = F32 ? static_cast<const float*>(row)[8 * whole + k]
                                       : widen(static_cast<const uint16_t*>(row)[8 * whole + k]);
    }
  }
}

template <bool F32, int TPR, int NV>
__device__ __forceinline__ void store_row(void* row, int H, int t, const float (&v)[NV][8]) {
  const int whole = H >> 3;
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int c = i * TPR + t;
    if (c >= whole) continue;
    if (F32) {
      Raw4f a, b;
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        a.f[k] = v[i][k];
        b.f[k] = v[i][4 + k];
      }
      Raw4f* p = reinterpret_cast<Raw4f*>(static_cast<float*>(row) + 8 * c);
      p[0] = a;
      p[1] = b;
    } else {
      Raw8h a;
#pragma unroll
      for (int k = 0; k < 4; ++k) a.w[k] = narrow2(v[i][2 * k], v[i][2 * k + 1]);
      *reinterpret_cast<Raw8h*>(static_cast<uint16_t*>(row) + 8 * c) = a;
    }
  }
  if ((H & 7) != 0) {
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      if (i * TPR + t != whole) continue;
#pragma unroll
      for (int k = 0; k < 7; ++k)
        if (k < (H & 7)) {
          if (F32) static_cast<float*>(row)[8 * whole + k] = v[i][k];
          else static_cast<uint16_t*>(row)[8 * whole + k] = narrow(v[i][k]);
        }
    }
  }
}

// The weights of a thread's columns, in either type; `fill` where there are none.
template <int TPR, int NV>
__device__ __forceinline__ void load_weights(const void* w, bool f32, float fill, int H, int t, float (&v)[NV][8]) {
  if (w == nullptr) {
#pragma unroll
    for (int i = 0; i < NV; ++i)
#pragma unroll
      for (int k = 0; k < 8; ++k) v[i][k] = fill;
  } else if (f32) {
    load_row<true, TPR, NV>(w, H, t, v);
  } else {
    load_row<false, TPR, NV>(w, H, t, v);
  }
}

// Sums of two values over the threads of a row, in a fixed order: the wave by
// butterflies, then (a block per row) the four waves' sums through LDS. The
// two halves of `s` alternate between calls, so one barrier a call is enough.
template <int TPR>
__device__ __forceinline__ void row_sum2(float& a, float& b, float (*s)[4][2], int& turn) {
#pragma unroll
  for (int x = 32; x >= 1; x >>= 1) {
    a += __shfl_xor(a, x);
    b += __shfl_xor(b, x);
  }
  if (TPR > 64) {
    const int wave = threadIdx.x >> 6;
    if ((threadIdx.x & 63) == 0) {
      s[turn][wave][0] = a;
      s[turn][wave][1] = b;
    }
    __syncthreads();
    a = (s[turn][0][0] + s[turn][1][0]) + (s[turn][2][0] + s[turn][3][0]);
    b = (s[turn][0][1] + s[turn][1][1]) + (s[turn][2][1] + s[turn][3][1]);
    turn ^= 1;
  }
}

// Forward: a row's threads walk rows `step` apart, the weights in registers.
template <bool XF32, bool YF32, int TPR, int NV>
__global__ __launch_bounds__(kBlock) void norm_fwd_kernel(const NormFwdArgs a) {
  __shared__ float s[2][4][2];
  const int t = threadIdx.x % TPR;
  const int per = kBlock / TPR;
  const int64_t step = (int64_t)gridDim.x * per;
  const int H = a.H;
  const float inv = 1.0f / (float)H;
  int turn = 0;
  float w[NV][8], b[NV][8];
  load_weights<TPR, NV>(a.w, a.w_f32, 1.0f, H, t, w);
  load_weights<TPR, NV>(a.b, a.w_f32, 0.0f, H, t, b);
  for (int64_t row = (int64_t)blockIdx.x * per + threadIdx.x / TPR; row < a.N; row += step) {
    float x[NV][8];
    load_row<XF32, TPR, NV>(static_cast<const char*>(a.x) + row * H * (XF32 ? 4 : 2), H, t, x);
    float mu = 0.0f, z = 0.0f;
    if (!a.rms) {
#pragma unroll
      for (int v = 0; v < NV; ++v)
#pragma unroll
        for (int k = 0; k < 8; ++k) mu += x[v][k];
      row_sum2<TPR>(mu, z, s, turn);
      mu *= inv;
    }
    float q = 0.0f;
#pragma unroll
    for (int v = 0; v < NV; ++v)
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        const float d = x[v][k] - mu;
        const bool in = 8 * (v * TPR + t) + k < H;   // padding is not part of the variance
        q = in ? fmaf(d, d, q) : q;
      }
    row_sum2<TPR>(q, z, s, turn);
    const float r = 1.0f / sqrtf(fmaf(q, inv, a.eps));
#pragma unroll
    for (int v = 0; v < NV; ++v)
#pragma unroll
      for (int k = 0; k < 8; ++k) x[v][k] = fmaf((x[v][k] - mu) * r, w[v][k], b[v][k]);
    store_row<YF32, TPR, NV>(static_cast<char*>(a.y) + row * H * (YF32 ? 4 : 2), H, t, x);
    if (t == 0) {
      if (a.mean != nullptr && !a.rms) a.mean[row] = mu;
      if (a.rstd != nullptr) a.rstd[row] = r;
    }
  }
}

// Backward: a row's threads walk rows step apart and keep their columns' sums
// of dw and db in registers; at the end the rows of a block are added through
// LDS in order and the block writes one partial row of each ([blocks][2][H]),
// which norm_reduce_kernel sums in block order. A zero in dy contributes a
// zero whatever x, the statistics and w hold there (mul0), so a masked token,
// whose dy row is 0, adds nothing and gets dx = 0 even where its x is NaN.
template <bool XF32, bool YF32, int TPR, int NV>
__global__ __launch_bounds__(kBlock) void norm_bwd_kernel(const NormBwdArgs a) {
  extern __shared__ float lds[];   // [2][H]: the block's dw and db (TPR < 256)
  __shared__ float s[2][4][2];
  const int t = threadIdx.x % TPR;
  const int per = kBlock / TPR;
  const int slot = threadIdx.x / TPR;
  const int64_t step = (int64_t)gridDim.x * per;
  const int H = a.H;
  const float inv = 1.0f / (float)H;
  int turn = 0;
  float dw[NV][8], db[NV][8];
#pragma unroll
  for (int v = 0; v < NV; ++v)
#pragma unroll
    for (int k = 0; k < 8; ++k) dw[v][k] = db[v][k] = 0.0f;
  for (int64_t row = (int64_t)blockIdx.x * per + slot; row < a.N; row += step) {
    float x[NV][8], g[NV][8], w[NV][8];
    load_row<XF32, TPR, NV>(static_cast<const char*>(a.x) + row * H * (XF32 ? 4 : 2), H, t, x);
    load_row<YF32, TPR, NV>(static_cast<const char*>(a.dy) + row * H * (YF32 ? 4 : 2), H, t, g);
    load_weights<TPR, NV>(a.w, a.w_f32, 1.0f, H, t, w);   // reread: registers are dw's and db's
    const float mu = a.rms ? 0.0f : a.mean[row];
    const float r = a.rstd[row];
    float c1 = 0.0f, c2 = 0.0f;
#pragma unroll
    for (int v = 0; v < NV; ++v)
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        const float xh = (x[v][k] - mu) * r;
        dw[v][k] += mul0(g[v][k], xh);
        db[v][k] += g[v][k];
        const float gw = mul0(g[v][k], w[v][k]);
        c1 += mul0(gw, xh);
        c2 += gw;
        x[v][k] = xh;
        g[v][k] = gw;
      }
    row_sum2<TPR>(c1, c2, s, turn);
    c1 *= inv;
    c2 = a.rms ? 0.0f : c2 * inv;
#pragma unroll
    for (int v = 0; v < NV; ++v)
#pragma unroll
      for (int k = 0; k < 8; ++k) x[v][k] = mul0(r, (g[v][k] - c2) - mul0(x[v][k], c1));
    store_row<XF32, TPR, NV>(static_cast<char*>(a.dx) + row * H * (XF32 ? 4 : 2), H, t, x);
  }
  if (a.part == nullptr) return;
  float* out = a.part + (int64_t)blockIdx.x * 2 * H;
  if (TPR < kBlock) {
    for (int i = 0; i < per; ++i) {
      if (slot == i) {
#pragma unroll
        for (int v = 0; v < NV; ++v)
#pragma unroll
          for (int k = 0; k < 8; ++k) {
            const int j = 8 * (v * TPR + t) + k;
            if (j >= H) continue;
            if (i > 0) {
              dw[v][k] += lds[j];
              db[v][k] += lds[H + j];
            }
            if (i < per - 1) {
              lds[j] = dw[v][k];
              lds[H + j] = db[v][k];
            } else {
              out[j] = dw[v][k];
              out[H + j] = db[v][k];
            }
          }
      }
      __syncthreads();
    }
  } else {
    store_row<true, TPR, NV>(out, H, t, dw);
    store_row<true, TPR, NV>(out + H, H, t, db);
  }
}

// Sums the blocks' partial rows, 64 columns per workgroup, 16 waves each a
// sixteenth of the rows, joined in order.
constexpr int kRedWaves = 16;
__global__ __launch_bounds__(64 * kRedWaves) void norm_reduce_kernel(const NormReduceArgs a) {
  __shared__ float s[kRedWaves][64];
  const int lane = threadIdx.x & 63;
  const int wave = threadIdx.x >> 6;
  const int H = a.H;
  const int j = blockIdx.x * 64 + lane;   // column of [dw | db]
  const int lo = (int)((int64_t)wave * a.blocks / kRedWaves);
  const int hi = (int)((int64_t)(wave + 1) * a.blocks / kRedWaves);
  float v = 0.0f;
  if (j < 2 * H)
    for (int i = lo; i < hi; ++i) v += a.part[(int64_t)i * 2 * H + j];
  s[wave][lane] = v;
  __syncthreads();
  if (wave != 0 || j >= 2 * H) return;
  v = s[0][lane];
#pragma unroll
  for (int i = 1; i < kRedWaves; ++i) v += s[i][lane];
  void* out = j < H ? a.dw : a.db;
  const int c = j < H ? j : j - H;
  if (out == nullptr) return;
  if (a.g_f32) {
    float* o = static_cast<float*>(out) + c;
    *o = a.accumulate ? *o + v : v;
  } else {
    uint16_t* o = static_cast<uint16_t*>(out) + c;
    *o = narrow(a.accumulate ? widen(*o) + v : v);
  }
}

// Threads of a row and chunks of each: up to 2560 elements a wave per row
// (no barrier; up to 5 chunks, so the backward's 32 values per chunk and lane
// leave two waves per SIMD), above that a block per row.
template <class F>
hipError_t with_shape(int H, F f) {
#define LMH_NORM_CASE(tpr, nv) \
  if (H <= 8 * (tpr) * (nv)) return f(std::integral_constant<int, tpr>{}, std::integral_constant<int, nv>{});
  LMH_NORM_CASE(64, 1)
  LMH_NORM_CASE(64, 2)
  LMH_NORM_CASE(64, 3)
  LMH_NORM_CASE(64, 4)
  LMH_NORM_CASE(64, 5)
  LMH_NORM_CASE(256, 2)
  LMH_NORM_CASE(256, 3)
  LMH_NORM_CASE(256, 4)
  LMH_NORM_CASE(256, 6)
  LMH_NORM_CASE(256, 8)
#undef LMH_NORM_CASE
  return hipErrorInvalidValue;
}

template <bool XF32, bool YF32>
hipError_t fwd_typed(const NormFwdArgs& a, hipStream_t stream) {
  return with_shape(a.H, [&](auto tpr, auto nv) {
    const int per = kBlock / tpr();
    const int64_t blocks = std::min<int64_t>((a.N + per - 1) / per, 2048);
    hipLaunchKernelGGL((norm_fwd_kernel<XF32, YF32, tpr(), nv()>), dim3((unsigned)blocks), dim3(kBlock), 0, stream, a);
    return hipGetLastError();
  });
}

template <bool XF32, bool YF32>
hipError_t bwd_typed(const NormBwdArgs& a, int blocks, hipStream_t stream) {
  return with_shape(a.H, [&](auto tpr, auto nv) {
    const size_t lds = tpr() < kBlock ? (size_t)2 * a.H * 4 : 0;
    hipLaunchKernelGGL((norm_bwd_kernel<XF32, YF32, tpr(), nv()>), dim3(blocks), dim3(kBlock), lds, stream, a);
    return hipGetLastError();
  });
}

}  // namespace

int norm_bwd_blocks(int64_t N, int64_t H) {
  const int64_t per = H <= 2560 ? 4 : 1;
  return (int)std::max<int64_t>(1, std::min<int64_t>((N + 4 * per - 1) / (4 * per), 1024));
}

hipError_t launch_norm_fwd(const NormFwdArgs& a, hipStream_t stream) {
  trace_begin(stream);
  const hipError_t e = a.x_f32 ? (a.y_f32 ? fwd_typed<true, true>(a, stream) : fwd_typed<true, false>(a, stream))
                               : fwd_typed<false, false>(a, stream);
  if (e != hipSuccess) return e;
  const double n = (double)a.N * a.H;
  trace_end(kNormFwd, stream, 8.0 * n, n * ((a.x_f32 ? 4 : 2) + (a.y_f32 ? 4 : 2)) + 8.0 * a.N);
  return hipSuccess;
}

hipError_t launch_norm_bwd(const NormBwdArgs& a, int blocks, hipStream_t stream) {
  const double n = (double)a.N * a.H;
  trace_begin(stream);
  const hipError_t e = a.x_f32 ? (a.y_f32 ? bwd_typed<true, true>(a, blocks, stream)
                                          : bwd_typed<true, false>(a, blocks, stream))
                               : bwd_typed<false, false>(a, blocks, stream);
  if (e != hipSuccess) return e;
  trace_end(kNormBwd, stream, 14.0 * n, n * (2 * (a.x_f32 ? 4 : 2) + (a.y_f32 ? 4 : 2)) + 8.0 * a.N);
  return hipSuccess;
}

hipError_t launch_norm_reduce(const NormReduceArgs& a, hipStream_t stream) {
  trace_begin(stream);
  hipLaunchKernelGGL(norm_reduce_kernel, dim3((unsigned)((2 * a.H + 63) / 64)), dim3(64 * kRedWaves), 0, stream, a);
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  trace_end(kNormReduce, stream, 0.0, 8.0 * a.blocks * (double)a.H + 8.0 * a.H);
  return hipSuccess;
}

}  // namespace lmh
