// lmhead_few.hip -- the distillation head for few tokens, for gfx950.
//
// With few tokens every pass is bound by the vocabulary table: the forward
// reads W once (2 V H bytes), the backward reads it twice (for the logits and
// for dh) and writes dW once. The head's 256 x 256 tiles would spend 4 to 256
// times the products, and leave the chip waiting at their prologues and
// epilogues. Here waves stream W from memory through registers, for tiles of
// up to 64 tokens:
//
//   logits   a wave holds 16 MB vocabulary rows x 16 NB tokens and walks H, so a
//            row of W is loaded by one wave only
//   dW       (V x H, K = tokens) a wave keeps its columns of hidden^T in
//            registers and walks the vocabulary
//   dh       (tokens x H, K = V) a workgroup stages 32 rows of W and of the
//            cotangent in LDS and reads both transposed; the vocabulary is
//            split over workgroups, whose float32 partials are summed in order
//
// Up to 64 tokens the cotangent is held as two bf16 words (its rounding and
// what that left): its products then cost twice the matrix instructions, which
// are idle there, and carry 16 bits instead of 8. Above, it is one word, as the
// tiles' (a second would double what the gradients' kernels read of it).
//
// Measured with H = 2560, V = 151936 (778 MB of W; a copy reaches 5.0 TB/s): the
// forward's pass 143 us for one token and 147 us for 64 (5.4 TB/s); in the backward
// the cotangent 150-170 us, dh 135-190 us and dW 200-240 us, each paying for the
// write-back of the last one's stores: 2.33 GB in 0.55-0.6 ms, 4.1 TB/s.
//
// MFMA 16x16x32: lane l supplies row (l % 16) of A and column (l % 16) of B with
// 8 K values of its quarter l / 16; register r of lane l holds
// D[4 (l / 16) + r][l % 16]. Which 8 K values a quarter takes is free as long as
// A and B agree.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include <algorithm>

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

// Forward: the statistics of the workgroup's 64 MB vocabulary rows per token,
// as one record of the split (the workgroup).
template <int MB, int NB>
__global__ __launch_bounds__(256, 2) void few_stats_kernel(const FewArgs a) {
  __shared__ __attribute__((aligned(16))) char lds[few_lds<NB>()];
  __shared__ float4 xch[4][16 * NB];
  const int lane = threadIdx.x & 63;
  const int wave = wave_id();
  const FewTile t = few_tile(a, xcd_remap(blockIdx.x, gridDim.x), a.splits);
  if (t.split < 0) return;
  const int r0 = (t.split * 4 + wave) * 16 * MB;
  const int V = a.V;
  Stats st[NB];
#pragma unroll
  for (int j = 0; j < NB; ++j) st[j] = Stats{kNegBig, 0.0f, 0.0f, 0.0f};
  {
    int tgt[NB];
#pragma unroll
    for (int j = 0; j < NB; ++j) {
      const int tok = 16 * j + (lane & 15);
      tgt[j] = a.targets != nullptr ? a.targets[t.tok0 + min(tok, t.n - 1)] : -1;
      if (tgt[j] < 0 || tgt[j] >= V) tgt[j] = -1;
    }
    f32x4 acc[MB][NB];
    few_logits_of<MB, NB>(a, t, r0, lds, acc);
#pragma unroll
    for (int j = 0; j < NB; ++j) {
      // rows past V take no part: their logits never win the max, and their
      // exponentials are selected away
      float mx = kNegBig;
#pragma unroll
      for (int i = 0; i < MB; ++i)
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          const int row = r0 + acc_row(i, r, lane);
          if (row < V) mx = nan_max(mx, acc[i][j][r]);
          if (row == tgt[j]) st[j].zt = acc[i][j][r];
        }
      // sc > 0: max commutes with the scaling. Lanes without a row keep kNegBig: scaled by
      // an sc above 3.4e8 it would be -inf, whose merge with another such record is NaN.
      const float m = nan_max(kNegBig, mx * a.sc);
      float s1 = 0.0f, s2 = 0.0f;
#pragma unroll
      for (int i = 0; i < MB; ++i)
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          const bool in = r0 + acc_row(i, r, lane) < V;
          const float d = in ? fmaf(acc[i][j][r], a.sc, -m) : 0.0f;
          const float e = in ? fast_exp2(d) : 0.0f;
          s1 += e;
          s2 = fmaf(e, d, s2);
        }
      st[j].m2 = m;
      st[j].s1 = s1;
      st[j].s2 = s2;
    }
  }
#pragma unroll
  for (int x = 16; x <= 32; x <<= 1)
#pragma unroll
    for (int j = 0; j < NB; ++j) {
      const Stats o{__shfl_xor(st[j].m2, x), __shfl_xor(st[j].s1, x), __shfl_xor(st[j].s2, x), __shfl_xor(st[j].zt, x)};
      st[j] = (lane & x) == 0 ? merge_stats(st[j], o) : merge_stats(o, st[j]);
    }
  if (lane < 16) {
#pragma unroll
    for (int j = 0; j < NB; ++j) xch[wave][16 * j + lane] = make_float4(st[j].m2, st[j].s1, st[j].s2, st[j].zt);
  }
  __syncthreads();
  const int tok = threadIdx.x;
  if (tok < 16 * NB && tok < t.n) {
    Stats m{kNegBig, 0.0f, 0.0f, 0.0f};
#pragma unroll
    for (int w = 0; w < 4; ++w) {
      const float4 p = xch[w][tok];
      m = merge_stats(m, Stats{p.x, p.y, p.z, p.w});
    }
    reinterpret_cast<float4*>(a.part)[t.split * a.part_ld + t.tok0 + tok] = make_float4(m.m2, m.s1, m.s2, m.zt);
  }
}

// Backward: the cotangent of the workgroup's 64 MB vocabulary rows, formed in
// LDS as [row][token] pairs of bf16 words, the tokens' special entries
// overwriting theirs there, and stored as [V][padded tokens], high words and (up
// to 64 tokens) low words apart. Masked tokens and tokens past N are 0.
template <int MB, int NB>
__global__ __launch_bounds__(256, 2) void few_dz_kernel(const FewArgs a) {
  constexpr int NP = 16 * NB, rows = 64 * MB, tile = rows * NP * 2;
  // the logits' staging, then the two words' tiles in its place
  __shared__ __attribute__((aligned(16))) char lds[few_lds<NB>() > 2 * tile ? few_lds<NB>() : 2 * tile];
  uint16_t (*t_hi)[NP] = reinterpret_cast<uint16_t (*)[NP]>(lds);
  uint16_t (*t_lo)[NP] = reinterpret_cast<uint16_t (*)[NP]>(lds + tile);
  const int lane = threadIdx.x & 63;
  const int wave = wave_id();
  const FewTile t = few_tile(a, xcd_remap(blockIdx.x, gridDim.x), a.splits);
  if (t.split < 0) return;
  const int b0 = t.split * rows;
  const int w0 = wave * 16 * MB;
  const int V = a.V;
  auto put = [&](int row, int tok, float x) {
    const uint16_t hi = round_bf16(x);
    t_hi[row][tok] = hi;
    // the difference is exact; an infinity leaves nothing
    t_lo[row][tok] = (hi & 0x7FFF) == 0x7F80 ? (uint16_t)0 : round_bf16(x - widen_bf16(hi));
  };
  {
    f32x4 acc[MB][NB];
    few_logits_of<MB, NB>(a, t, b0 + w0, lds, acc);
    __syncthreads();
#pragma unroll
    for (int j = 0; j < NB; ++j) {
      const int tok = 16 * j + (lane & 15);
      const int at = t.tok0 + min(tok, t.n - 1);
      const int id = a.targets[at];
      const bool live = tok < t.n && id >= 0 && id < V;
      const float nlse = live ? -a.lse[at] * kLog2e : 0.0f;
      const float c0 = live ? -a.ga[at] * a.invT : 0.0f;
#pragma unroll
      for (int i = 0; i < MB; ++i)
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          // an entry of probability 0 has no such term, whatever c0 holds
          const float x = lmh_fmul_legacy(fast_exp2(fmaf(acc[i][j][r], a.sc, nlse)), c0);
          put(w0 + acc_row(i, r, lane), tok, live ? x : 0.0f);
        }
    }
  }
  __syncthreads();
  const int n = t.n * a.K1;
  const int32_t* ent_id = a.ent_id + (int64_t)t.tok0 * a.K1;
  for (int e = threadIdx.x; e < n; e += 256) {
    const int id = ent_id[e];
    if (id >= b0 && id < min(b0 + rows, V)) put(id - b0, e / a.K1, a.ent_val[(int64_t)t.tok0 * a.K1 + e]);
  }
  __syncthreads();
  constexpr int per_row = NP / 8;   // 16-byte chunks
  for (int c = threadIdx.x; c < rows * per_row; c += 256) {
    if (b0 + c / per_row >= V) break;
    const int64_t at = (int64_t)(b0 + c / per_row) * (a.padded / 8) + t.tok0 / 8 + c % per_row;
    reinterpret_cast<u32x4*>(a.dz_hi)[at] = reinterpret_cast<const u32x4*>(t_hi)[c];
    if (a.dz_lo != nullptr) reinterpret_cast<u32x4*>(a.dz_lo)[at] = reinterpret_cast<const u32x4*>(t_lo)[c];
  }
}

// dW[v][h] = sum_tok dz[v][tok] hidden[tok][h]. A wave holds 128 columns
// (64 above 64 tokens) of hidden^T as A operands (block pair c: columns 32 c + 8 q + (0..7) fall to
// quarter q, so a lane ends with 8 consecutive ones) and walks vocabulary
// groups of 16, the next group's cotangent in flight. Bound by the stores: the
// group's results turn in the wave's LDS, so that a store covers whole
// lines (4 rows x 256 bytes of bf16, 2 x 512 of float32) and not 16 pieces of 64.
template <int BL>
constexpr int few_ht_lds() { return 4 * 32 * (32 * BL + 16); }
template <int BL, bool BF16>
constexpr int few_dw_lds() { return std::max(4 * 16 * (16 * BL * (BF16 ? 2 : 4) + 16), few_ht_lds<BL>()); }
template <int KS, int BL, bool LO, bool BF16, bool ADD>
__device__ __forceinline__ void few_dw(const FewArgs& a, int vid, char* lds) {
  constexpr int NP = 32 * KS, cols = 16 * BL;
  constexpr int bytes = BF16 ? 2 : 4, pitch = cols * bytes + 16;
  constexpr int per_row = cols * bytes / 16, stores = 16 * per_row / 64;   // 16-byte pieces of a row; stores of a group
  const int lane = threadIdx.x & 63;
  const int col = lane & 15, q = lane >> 4;
  const int wave = wave_id();
  const int w = vid * 4 + wave;
  const int strip = w % a.strips, split = w / a.strips;
  if (split >= a.dw_splits) return;
  const int H = a.H, V = a.V;
  const int h0 = strip * cols;
  // hidden^T: 32 tokens at a time turn in the wave's LDS (masked tokens are 0,
  // whatever their rows hold)
  bf16x8 ht[BL][KS];
  constexpr int h_pitch = 2 * cols + 16, h_per = cols / 8, h_each = 32 * h_per / 64;
  static_assert(4 * 32 * h_pitch <= few_dw_lds<BL, BF16>(), "a wave's quarter holds 32 tokens");
  char* turn = lds + wave * (few_dw_lds<BL, BF16>() / 4);
#pragma unroll
  for (int k = 0; k < KS; ++k) {
    u32x4 x[h_each];
#pragma unroll
    for (int c = 0; c < h_each; ++c) {
      const int tok = 32 * k + (64 * c + lane) / h_per;
      const int at = min(tok, a.N - 1);
      const int id = a.targets[at];
      x[c] = *reinterpret_cast<const u32x4*>(a.hidden + (int64_t)at * H + min(h0 + 8 * (lane % h_per), H - 8));
      if (tok >= a.N || id < 0 || id >= V) x[c] = u32x4{0u, 0u, 0u, 0u};
    }
#pragma unroll
    for (int c = 0; c < h_each; ++c)
      *reinterpret_cast<u32x4*>(turn + (64 * c + lane) / h_per * h_pitch + 16 * (lane % h_per)) = x[c];
    wave_order();
    // a transposed read hands lane j the columns that lane j / 4 points at, element j % 4
#pragma unroll
    for (int b = 0; b < BL; ++b) {
      const char* p = turn + (8 * q + (col >> 2)) * h_pitch + 2 * (32 * (b >> 1) + 8 * (col & 3) + 4 * (b & 1));
      short8v v;
      v.s0123 = ds_read_tr(p);
      v.s4567 = ds_read_tr(p + 4 * h_pitch);
      ht[b][k] = __builtin_bit_cast(bf16x8, v);
    }
    wave_order();
  }
  const int groups = (V + 15) / 16;
  const int g_lo = (int)((int64_t)split * groups / a.dw_splits), g_hi = (int)((int64_t)(split + 1) * groups / a.dw_splits);
  bf16x8 hi[KS], lo[LO ? KS : 1];
  auto load = [&](int g) {
    const int64_t at = (int64_t)min(16 * g + col, V - 1) * NP + 8 * q;
#pragma unroll
    for (int k = 0; k < KS; ++k) {
      hi[k] = *reinterpret_cast<const bf16x8*>(a.dz_hi + at + 32 * k);
      if (LO) lo[k] = *reinterpret_cast<const bf16x8*>(a.dz_lo + at + 32 * k);
    }
  };
  char* mine = lds + wave * (few_dw_lds<BL, BF16>() / 4);
  auto group = [&](int g, bool checked) {
    f32x4 acc[BL];
#pragma unroll
    for (int b = 0; b < BL; ++b) acc[b] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
    for (int k = 0; k < KS; ++k) {
      if (LO) {
#pragma unroll
        for (int b = 0; b < BL; ++b) acc[b] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(ht[b][k], lo[LO ? k : 0], acc[b], 0, 0, 0);
      }
#pragma unroll
      for (int b = 0; b < BL; ++b) acc[b] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(ht[b][k], hi[k], acc[b], 0, 0, 0);
    }
    load(g + 1);
    if (ADD) {   // the sum is rounded once: the old values join in float32, where they lie
#pragma unroll
      for (int c = 0; c < BL / 2; ++c) {
        const int row = 16 * g + col;
        if (row >= V || h0 + 32 * c >= H) continue;
        const int64_t at = (int64_t)row * H + h0 + 32 * c + 8 * q;
        if (BF16) {
          const u32x4 o = *reinterpret_cast<const u32x4*>(static_cast<const uint16_t*>(a.dW) + at);
          acc[2 * c] += f32x4{__uint_as_float(o[0] << 16), __uint_as_float(o[0] & 0xFFFF0000u),
                              __uint_as_float(o[1] << 16), __uint_as_float(o[1] & 0xFFFF0000u)};
          acc[2 * c + 1] += f32x4{__uint_as_float(o[2] << 16), __uint_as_float(o[2] & 0xFFFF0000u),
                                  __uint_as_float(o[3] << 16), __uint_as_float(o[3] & 0xFFFF0000u)};
        } else {
          const f32x4* p = reinterpret_cast<const f32x4*>(static_cast<const float*>(a.dW) + at);
          acc[2 * c] += p[0];
          acc[2 * c + 1] += p[1];
        }
      }
    }
#pragma unroll
    for (int c = 0; c < BL / 2; ++c) {
      const f32x4 x = acc[2 * c], y = acc[2 * c + 1];
      char* p = mine + col * pitch + (32 * c + 8 * q) * bytes;
      if (BF16) {
        *reinterpret_cast<u32x4*>(p) =
            u32x4{pack_bf16x2(x[0], x[1]), pack_bf16x2(x[2], x[3]), pack_bf16x2(y[0], y[1]), pack_bf16x2(y[2], y[3])};
      } else {
        reinterpret_cast<f32x4*>(p)[0] = x;
        reinterpret_cast<f32x4*>(p)[1] = y;
      }
    }
    wave_order();
#pragma unroll
    for (int i = 0; i < stores; ++i) {
      const int r = (64 * i + lane) / per_row, piece = lane % per_row;
      const u32x4 v = *reinterpret_cast<const u32x4*>(mine + r * pitch + 16 * piece);
      if (checked && (16 * g + r >= V || h0 + 16 / bytes * piece >= H)) continue;
      *reinterpret_cast<u32x4*>(static_cast<char*>(a.dW) + ((int64_t)(16 * g + r) * H + h0) * bytes + 16 * piece) = v;
    }
    wave_order();
  };
  load(g_lo);
  const int whole = h0 + cols <= H ? min(g_hi, V / 16) : g_lo;   // groups whose every store lies inside
  for (int g = g_lo; g < whole; ++g) group(g, false);
  for (int g = max(g_lo, whole); g < g_hi; ++g) group(g, true);
}

// dh[tok][h] = sum_v dz[v][tok] W[v][h] over one split of the vocabulary and 256
// columns (64 a wave), as a float32 partial [split][N][H]. 32 vocabulary rows a
// step go through registers into LDS (two buffers); W's rows lie there as the
// tile core's MN-contiguous slices do, the cotangent's with 16 bytes of padding,
// so that the transposed reads of 16 lanes (4 rows x 32 bytes) meet no bank
// twice. Rows past the split are 0 in both operands.
template <int NB, bool LO>
constexpr int few_dh_lds() { return 2 * (32 * 512 + (LO ? 2 : 1) * 32 * (32 * NB + 16)); }
template <int NB, bool LO>
__device__ __forceinline__ void few_dh(const FewArgs& a, int vid, char* lds) {
  constexpr int NP = 16 * NB, pitch = 2 * NP + 16, words = LO ? 2 : 1;
  constexpr int w_bytes = 32 * 512, z_bytes = 32 * pitch, buf = w_bytes + words * z_bytes;
  static_assert(2 * buf == few_dh_lds<NB, LO>(), "two buffers");
  const int lane = threadIdx.x & 63;
  const int wave = wave_id();
  const FewTile t = few_tile(a, vid, a.dh_strips * a.dh_splits);
  if (t.split < 0) return;
  const int strip = t.split % a.dh_strips, split = t.split / a.dh_strips;
  const int H = a.H;
  const int h0 = strip * 256;
  const int v_lo = split * a.dh_rows, v_hi = min(v_lo + a.dh_rows, a.V);
  const int steps = (v_hi - v_lo + 31) / 32;   // > 0: the host counts the splits

  // staging: W row t / 32 + 8 c, 16-byte chunk t % 32; cotangent row t / (NP / 8)
  // (of the high words, then of the low ones)
  const int chunk = threadIdx.x & 31;
  const int w_col = min(h0 + 8 * chunk, H - 8);
  constexpr int z_per = NP / 8;                          // chunks of a cotangent row
  constexpr int z_n = words * 32 * z_per;                // chunks of the words
  constexpr int z_each = (z_n + 255) / 256;
  u32x4 sw2[2][4], sz2[2][z_each];   // two steps in flight
  const u32x4 none = {0u, 0u, 0u, 0u};
  auto fetch = [&](int step, u32x4 (&sw)[4], u32x4 (&sz)[z_each]) {
    const int v0 = v_lo + 32 * step;
#pragma unroll
    for (int c = 0; c < 4; ++c) {
      const int v = v0 + (threadIdx.x >> 5) + 8 * c;
      sw[c] = *reinterpret_cast<const u32x4*>(a.W + (int64_t)min(v, v_hi - 1) * H + w_col);
      if (v >= v_hi) sw[c] = none;
    }
#pragma unroll
    for (int c = 0; c < z_each; ++c) {
      const int i = threadIdx.x + 256 * c;
      const int v = v0 + (i / z_per) % 32;
      const uint16_t* src = i < 32 * z_per ? a.dz_hi : a.dz_lo;
      sz[c] = none;
      if (i < z_n && v < v_hi) sz[c] = *reinterpret_cast<const u32x4*>(src + (int64_t)v * a.padded + t.tok0 + 8 * (i % z_per));
    }
  };
  auto stage = [&](char* p, const u32x4 (&sw)[4], const u32x4 (&sz)[z_each]) {
#pragma unroll
    for (int c = 0; c < 4; ++c) {
      const int r = (threadIdx.x >> 5) + 8 * c;
      *reinterpret_cast<u32x4*>(p + r * 512 + ((chunk ^ swz_mn(r)) << 4)) = sw[c];
    }
#pragma unroll
    for (int c = 0; c < z_each; ++c) {
      const int i = threadIdx.x + 256 * c;
      if (i < z_n)
        *reinterpret_cast<u32x4*>(p + w_bytes + (i < 32 * z_per ? 0 : z_bytes) + (i / z_per) % 32 * pitch + 16 * (i % z_per)) = sz[c];
    }
  };
  // transposed reads: lane s of a 16-lane group points at K-row 8 q + s / 4 (+ 4
  // for the upper half) and 4 columns from 4 (s % 4) on
  const int s = lane & 15, q = lane >> 4;
  const int t_row = 8 * q + (s >> 2);
  const int t_x = swz_mn(t_row);
  const int t_chunk = wave * 8 + ((s & 3) >> 1);
  auto read = [&](const char* p0, const char* p1) {
    short8v v;
    v.s0123 = ds_read_tr(p0);
    v.s4567 = ds_read_tr(p1);
    return __builtin_bit_cast(bf16x8, v);
  };
  f32x4 acc[4][NB];
#pragma unroll
  for (int i = 0; i < 4; ++i)
#pragma unroll
    for (int j = 0; j < NB; ++j) acc[i][j] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
  auto turn = [&](int step, u32x4 (&sw)[4], u32x4 (&sz)[z_each]) {
    char* p = lds + (step & 1) * buf;
    stage(p, sw, sz);
    __syncthreads();   // one a step: a buffer is refilled two steps on, after every wave is past the step between
    if (step + 2 < steps) fetch(step + 2, sw, sz);
    bf16x8 fw[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const char* at = p + t_row * 512 + (((t_chunk + 2 * i) ^ t_x) << 4) + 8 * (s & 1);
      fw[i] = read(at, at + 4 * 512);   // 4 rows on, the swizzle is the same
    }
#pragma unroll
    for (int half = words - 1; half >= 0; --half)
#pragma unroll
      for (int j = 0; j < NB; ++j) {
        const char* at = p + w_bytes + half * z_bytes + t_row * pitch + 32 * j + 8 * (s & 3);
        const bf16x8 fz = read(at, at + 4 * pitch);
#pragma unroll
        for (int i = 0; i < 4; ++i) acc[i][j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(fw[i], fz, acc[i][j], 0, 0, 0);
      }
  };
  fetch(0, sw2[0], sz2[0]);
  if (steps > 1) fetch(1, sw2[1], sz2[1]);
  for (int step = 0; step < steps; step += 2) {
    turn(step, sw2[0], sz2[0]);
    if (step + 1 < steps) turn(step + 1, sw2[1], sz2[1]);
  }
#pragma unroll
  for (int j = 0; j < NB; ++j) {
    const int tok = 16 * j + s;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int h = h0 + 64 * wave + 16 * i + 4 * q;
      if (tok < t.n && h < H)
        *reinterpret_cast<f32x4*>(a.dh_part + ((int64_t)split * a.N + t.tok0 + tok) * H + h) = acc[i][j];
    }
  }
}

// Both products in one launch, dh's workgroups first (they read the end of W
// that the memory-side cache still holds); neither waits for the other, so
// each fills the other's tail. Ids are remapped within each part: a split's
// strips, and a strip's token tiles, share an XCD's L2.
template <int KS, int BL, bool LO, bool BF16, bool ADD>
__global__ __launch_bounds__(256, 2) void few_grads_kernel(const FewArgs a) {
  constexpr int NB = KS == 1 ? 2 : 4;
  constexpr int n_dw = few_dw_lds<BL, BF16>(), n_dh = few_dh_lds<NB, LO>();
  __shared__ __attribute__((aligned(16))) char lds[n_dw > n_dh ? n_dw : n_dh];
  const int bid = blockIdx.x;
  if (bid < a.dh_blocks) few_dh<NB, LO>(a, xcd_remap(bid, a.dh_blocks), lds);
  else few_dw<KS, BL, LO, BF16, ADD>(a, xcd_remap(bid - a.dh_blocks, gridDim.x - a.dh_blocks), lds);
}

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

}  // namespace

int few_splits(int64_t V) {
  const int rows = 64 * few_blocks(V);
  return (int)((V + rows - 1) / rows);
}

static unsigned few_grid(int64_t n) { return (unsigned)((n + 7) / 8 * 8); }

hipError_t launch_few_stats(FewArgs a, hipStream_t stream) {
  const double N = a.N, H = a.H, V = a.V;
  a.tiles = (a.N + 63) / 64;
  a.splits = few_splits(a.V);
  trace_begin(stream);
  with_sizes(few_blocks(a.V), a.N <= 16 ? 1 : a.N <= 32 ? 2 : 4, [&](auto mb, auto nb) {
    hipLaunchKernelGGL((few_stats_kernel<mb(), nb()>), dim3(few_grid((int64_t)a.tiles * a.splits)), dim3(256), 0, stream, a);
  });
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  trace_end(kFewStats, stream, 2.0 * N * H * V, 2.0 * (N + V) * H + 4.0 * N + 16.0 * a.splits * N);
  return hipSuccess;
}

// The cotangent, then dW and the partials of dh.
hipError_t launch_few_bwd(FewArgs a, bool bf16, hipStream_t stream) {
  const double N = a.N, H = a.H, V = a.V;
  const bool two = a.dz_lo != nullptr;
  a.tiles = (a.N + 63) / 64;
  a.splits = few_splits(a.V);
  trace_begin(stream);
  with_sizes(few_blocks(a.V), a.N <= 32 ? 2 : 4, [&](auto mb, auto n) {
    constexpr int NB = n() < 2 ? 2 : n();   // K of the gradient products is at least 32 tokens
    hipLaunchKernelGGL((few_dz_kernel<mb(), NB>), dim3(few_grid((int64_t)a.tiles * a.splits)), dim3(256), 0, stream, a);
  });
  hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  const double dz = (two ? 4.0 : 2.0) * a.padded * V;
  trace_end(kFewDz, stream, 0.0, 2.0 * (N + V) * H + dz);
  a.dh_blocks = few_grid((int64_t)a.tiles * a.dh_strips * a.dh_splits);
  // waves for dW: 8 a CU, but no less than 4 groups of 16 rows each
  const int cols = two ? 128 : 64;
  a.strips = (a.H + cols - 1) / cols;
  a.dw_splits = std::max(1, std::min((a.V + 63) / 64, 8 * kNumCUs / a.strips));
  const unsigned blocks = a.dh_blocks + few_grid(((int64_t)a.strips * a.dw_splits + 3) / 4);
  auto launch = [&](auto ks, auto bl, auto lo) {
    std::true_type yes;
    std::false_type no;
    auto typed = [&](auto half, auto add) {
      hipLaunchKernelGGL((few_grads_kernel<ks(), bl(), lo(), half(), add()>), dim3(blocks), dim3(256), 0, stream, a);
    };
    if (bf16) a.add_dW ? typed(yes, yes) : typed(yes, no);
    else a.add_dW ? typed(no, yes) : typed(no, no);
  };
  constexpr std::integral_constant<int, 4> four{};
  constexpr std::integral_constant<int, 8> eight{};
  trace_begin(stream);
  if (two && a.padded == 32) launch(std::integral_constant<int, 1>{}, eight, std::true_type{});
  else if (two) launch(std::integral_constant<int, 2>{}, eight, std::true_type{});
  else if (a.padded == 128) launch(four, four, std::false_type{});
  else if (a.padded == 192) launch(std::integral_constant<int, 6>{}, four, std::false_type{});
  else launch(eight, four, std::false_type{});
  e = hipGetLastError();
  if (e != hipSuccess) return e;
  trace_end(kFewGrads, stream, 4.0 * N * H * V, (bf16 ? 4.0 : 6.0) * V * H + 2.0 * dz + 4.0 * a.dh_splits * N * H);
  return hipSuccess;
}

}  // namespace lmh
