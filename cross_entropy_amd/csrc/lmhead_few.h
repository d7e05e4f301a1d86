// lmhead_few.h -- the streaming logits of few tokens, shared by the
// distillation's kernels (lmhead_few.hip) and the beams' (lmhead_beam.hip).
// lmhead_few.hip describes the method and the register layout.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include <algorithm>
#include <type_traits>

#include "lmhead_internal.h"
#include "lmhead_tile.h"

namespace lmh {
namespace {

typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));

// acc[i][j] = W rows r0 + 16 i .. times tokens 16 j .., over K = H (a multiple
// of 64). A unit is 64 of K: quarter q of the lanes takes bytes 32 q .. of the
// 128 that a row has there, so a wave's two loads use each line whole. D units
// are in flight; loads past the end reread the last unit.
template <int MB, int NB, int D>
__device__ __forceinline__ void few_logits(const uint16_t* W, int V, const uint16_t* hidden, int N, int H, int r0,
                                           f32x4 (&acc)[MB][NB]) {
  const int lane = threadIdx.x & 63;
  const int col = lane & 15, q = lane >> 4;
  const char* pa[MB];
  const char* pb[NB];
#pragma unroll
  for (int i = 0; i < MB; ++i)
    pa[i] = reinterpret_cast<const char*>(W + (int64_t)min(r0 + 16 * i + col, V - 1) * H) + 32 * q;
#pragma unroll
  for (int j = 0; j < NB; ++j)
    pb[j] = reinterpret_cast<const char*>(hidden + (int64_t)min(16 * j + col, N - 1) * H) + 32 * q;
#pragma unroll
  for (int i = 0; i < MB; ++i)
#pragma unroll
    for (int j = 0; j < NB; ++j) acc[i][j] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
  bf16x8 a[D][MB][2], b[D][NB][2];
  const int units = H / 64;
  auto load = [&](int d, int u) {
    const int64_t at = 128 * (int64_t)min(u, units - 1);
#pragma unroll
    for (int i = 0; i < MB; ++i) {
      const bf16x8* p = reinterpret_cast<const bf16x8*>(pa[i] + at);
      a[d][i][0] = p[0];
      a[d][i][1] = p[1];
    }
#pragma unroll
    for (int j = 0; j < NB; ++j) {
      const bf16x8* p = reinterpret_cast<const bf16x8*>(pb[j] + at);
      b[d][j][0] = p[0];
      b[d][j][1] = p[1];
    }
  };
#pragma unroll
  for (int d = 0; d < D; ++d) load(d, d);
  for (int u = 0; u < units; u += D) {
#pragma unroll
    for (int d = 0; d < D; ++d) {
      if (u + d < units) {
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
          for (int i = 0; i < MB; ++i)
#pragma unroll
            for (int j = 0; j < NB; ++j)
              acc[i][j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(a[d][i][h], b[d][j][h], acc[i][j], 0, 0, 0);
      }
      load(d, u + d + D);
    }
  }
}

// The same for 32 and 64 tokens, hidden through LDS: from cache, each wave
// fetches up to 0.8 of W's bytes of hidden again, which bounds the pass (64
// tokens, H = 2560, V = 151936: 240 us against 147). The workgroup stages few_k
// of K of every token, the next chunk in registers meanwhile; rows are padded by
// 16 bytes, so the 16 tokens of a fragment read fall on 16 different bank
// groups. `lds` holds two chunks; every wave of the workgroup has to call, also
// one without rows.
template <int NB>
constexpr int few_k() { return 1024 / NB; }
template <int NB>
constexpr int few_pitch() { return 2 * few_k<NB>() + 16; }
template <int MB, int NB, int D>
__device__ __forceinline__ void few_logits_lds(const uint16_t* W, int V, const uint16_t* hidden, int N, int H, int r0,
                                               char* lds, f32x4 (&acc)[MB][NB]) {
  constexpr int kFewK = few_k<NB>(), kFewPitch = few_pitch<NB>(), UC = kFewK / 64, pieces = 8;
  constexpr int buffer = 16 * NB * kFewPitch, per = kFewK / 8, step = 256 / per;   // threads of a token's row; tokens at once
  const int lane = threadIdx.x & 63;
  const int col = lane & 15, q = lane >> 4;
  const char* pa[MB];
#pragma unroll
  for (int i = 0; i < MB; ++i)
    pa[i] = reinterpret_cast<const char*>(W + (int64_t)min(r0 + 16 * i + col, V - 1) * H) + 32 * q;
#pragma unroll
  for (int i = 0; i < MB; ++i)
#pragma unroll
    for (int j = 0; j < NB; ++j) acc[i][j] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
  const int units = H / 64, chunks = (units + UC - 1) / UC;
  bf16x8 a[D][MB][2];
  auto load = [&](int d, int u) {
    const int64_t at = 128 * (int64_t)min(u, units - 1);
#pragma unroll
    for (int i = 0; i < MB; ++i) {
      const bf16x8* p = reinterpret_cast<const bf16x8*>(pa[i] + at);
      a[d][i][0] = p[0];
      a[d][i][1] = p[1];
    }
  };
  // staging: thread t takes 16 bytes at 8 (t % per) of tokens t / per + step c
  u32x4 next[pieces];
  const int t_tok = threadIdx.x / per, t_k = 8 * (threadIdx.x % per);
  auto fetch = [&](int chunk) {
#pragma unroll
    for (int c = 0; c < pieces; ++c)
      next[c] = *reinterpret_cast<const u32x4*>(hidden + (int64_t)min(t_tok + step * c, N - 1) * H +
                                                min(chunk * kFewK + t_k, H - 8));
  };
  auto stage = [&](int chunk) {
#pragma unroll
    for (int c = 0; c < pieces; ++c)
      *reinterpret_cast<u32x4*>(lds + (chunk & 1) * buffer + (t_tok + step * c) * kFewPitch + 2 * t_k) = next[c];
  };
  fetch(0);
#pragma unroll
  for (int d = 0; d < D; ++d) load(d, d);
  stage(0);
  for (int chunk = 0; chunk < chunks; ++chunk) {
    fetch(min(chunk + 1, chunks - 1));
    __syncthreads();   // chunk is staged; chunk - 1, whose buffer is filled below, has been read
    const char* p = lds + (chunk & 1) * buffer + col * kFewPitch + 32 * q;
#pragma unroll
    for (int uc = 0; uc < UC; ++uc) {
      const int u = chunk * UC + uc;
      if (u < units) {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          bf16x8 b[NB];
#pragma unroll
          for (int j = 0; j < NB; ++j) b[j] = *reinterpret_cast<const bf16x8*>(p + 16 * j * kFewPitch + 128 * uc + 16 * h);
#pragma unroll
          for (int i = 0; i < MB; ++i)
#pragma unroll
            for (int j = 0; j < NB; ++j)
              acc[i][j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(a[uc % D][i][h], b[j], acc[i][j], 0, 0, 0);
        }
      }
      load(uc % D, u + D);
    }
    stage(chunk + 1);   // after the last, a copy of it that nobody reads
  }
}

// The token tile (up to 64 tokens) and the split of a workgroup: the tiles of a
// split are neighbours on one XCD, whose L2 then serves all but the first
// with the split's rows of W. split -1: a workgroup too many.
struct FewTile {
  int tok0, n, split;
};
__device__ __forceinline__ FewTile few_tile(const FewArgs& a, int vid, int splits) {
  const int tok0 = vid % a.tiles * 64;
  const int split = vid / a.tiles;
  return {tok0, min(64, a.N - tok0), split < splits ? split : -1};
}

template <int MB, int NB>
__device__ __forceinline__ void few_logits_of(const FewArgs& a, const FewTile& t, int r0, char* lds, f32x4 (&acc)[MB][NB]) {
  const uint16_t* hidden = a.hidden + (int64_t)t.tok0 * a.H;
  if constexpr (NB > 1) few_logits_lds<MB, NB, 2>(a.W, a.V, hidden, t.n, a.H, r0, lds, acc);
  else few_logits<MB, NB, 3>(a.W, a.V, hidden, t.n, a.H, r0, acc);
}
template <int NB>
constexpr int few_lds() { return NB > 1 ? 2 * 16 * NB * few_pitch<NB>() : 16; }

// Row blocks (of 16) per wave: as few as let two workgroups a CU cover the
// vocabulary at once, so that no CU is left a second round (V = 151936: 475
// workgroups of 5 blocks a wave take 143 us for one token, 594 of 4 take 162).
// Above V = 163840 a second round starts: the whole forward of one token takes
// 217 us at 200003 and 283 at 262144, where W at the copy's rate takes 205 and 268.
constexpr int kMostBlocks = 5;
int few_blocks(int64_t V) {
  return (int)std::max<int64_t>(1, std::min<int64_t>(kMostBlocks, (V + 128 * kNumCUs - 1) / (128 * kNumCUs)));
}

template <class F>
void with_sizes(int mb, int nb, F f) {
  auto rows = [&](auto n) {
    if (mb == 5) f(std::integral_constant<int, 5>{}, n);
    else if (mb == 4) f(std::integral_constant<int, 4>{}, n);
    else if (mb == 3) f(std::integral_constant<int, 3>{}, n);
    else if (mb == 2) f(std::integral_constant<int, 2>{}, n);
    else f(std::integral_constant<int, 1>{}, n);
  };
  if (nb == 4) rows(std::integral_constant<int, 4>{});
  else if (nb == 2) rows(std::integral_constant<int, 2>{});
  else rows(std::integral_constant<int, 1>{});
}

inline unsigned few_grid(int64_t n) { return (unsigned)((n + 7) / 8 * 8); }

}  // namespace

}  // namespace lmh
