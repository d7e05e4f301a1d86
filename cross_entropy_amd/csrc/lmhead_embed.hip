// lmhead_embed.hip -- the vocabulary table as an embedding, for gfx950: the
// lookup with its scale, and the table's gradient.
//
//   y_i  = scale W[id_i]                      (0 for an id outside [0, V))
//   dW_v (+)= scale sum_{i: id_i = v} dy_i
//
// The gradient's sums run over the tokens of a word in the tokens' order, so
// the tokens are first sorted by word (stably), and no atomics take part in
// sums: results depend on the arguments alone.
//
//   sort   workgroup c owns the words v with v mod NC = c. Words that follow one
//          another fall to different workgroups, so a table sorted by frequency
//          loads them alike. Each scans all ids (its 16 waves a sixteenth each),
//          counts those of its words in LDS and those of lower classes (which is
//          where its part of the order begins: no word passes between
//          workgroups), and scans again to place its tokens.
//   rows   a word's tokens are cut into pieces of at most kPiece; a wave sums one
//          piece over 512 columns, straight into dW where it is the word's only
//          one, into a float32 partial row else. Rows without a token are zeroed.
//   join   partial rows of the words of several pieces, in order.
//
// All sums are float32; a bf16 gradient is rounded once, when stored.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include <algorithm>

#include "lmhead_internal.h"

namespace lmh {
namespace {

__device__ __forceinline__ uint16_t narrow(float x) { return __builtin_bit_cast(uint16_t, (__bf16)x); }
__device__ __forceinline__ uint32_t narrow2(float lo, float hi) {
  return (uint32_t)narrow(lo) | ((uint32_t)narrow(hi) << 16);
}

// Eight elements of a row, at their own alignment: rows of an odd length start
// off any larger boundary, which global memory accepts.
template <int WORDS>
struct __attribute__((packed, aligned(2))) Raw {
  uint32_t w[WORDS];
};
template <bool F32>
struct Eight {
  Raw<F32 ? 8 : 4> raw;
  // n < 8: the last elements of a row
  __device__ __forceinline__ void load(const void* row, int at, int n) {
    if (n >= 8) {
      raw = *reinterpret_cast<const Raw<F32 ? 8 : 4>*>(static_cast<const char*>(row) + (int64_t)at * (F32 ? 4 : 2));
      return;
    }
    uint32_t u[8];
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      u[k] = 0;
      if (k < n) u[k] = F32 ? static_cast<const uint32_t*>(row)[at + k] : static_cast<const uint16_t*>(row)[at + k];
    }
#pragma unroll
    for (int k = 0; k < (F32 ? 8 : 4); ++k) raw.w[k] = F32 ? u[k] : u[2 * k & 7] | (u[(2 * k + 1) & 7] << 16);
  }
  __device__ __forceinline__ float at(int k) const {
    if (F32) return __uint_as_float(raw.w[k]);
    const uint32_t w = raw.w[k / 2];
    return __uint_as_float((k & 1) ? (w & 0xFFFF0000u) : (w << 16));
  }
  __device__ __forceinline__ void set(const float (&v)[8]) {
#pragma unroll
    for (int k = 0; k < 8; k += F32 ? 1 : 2) raw.w[F32 ? k : k / 2] = F32 ? __float_as_uint(v[k]) : narrow2(v[k], v[k + 1]);
  }
  __device__ __forceinline__ void store(void* row, int at, int n) const {
    if (n >= 8) {
      *reinterpret_cast<Raw<F32 ? 8 : 4>*>(static_cast<char*>(row) + (int64_t)at * (F32 ? 4 : 2)) = raw;
      return;
    }
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      if (k >= n) break;
      if (F32) static_cast<uint32_t*>(row)[at + k] = raw.w[k];
      else static_cast<uint16_t*>(row)[at + k] = (uint16_t)(raw.w[k / 2] >> (16 * (k & 1)));
    }
  }
};

// Forward: a thread takes U groups of 8 elements, 256 apart in the row-major
// order of all of them.
template <bool WF32, bool YF32, int U>
__global__ __launch_bounds__(256) void embed_fwd_kernel(const EmbedFwdArgs a) {
  const int per = (a.H + 7) / 8;   // groups of a row
  const int64_t g0 = (int64_t)blockIdx.x * (256 * U);
  const int64_t row0 = g0 / per;
  const uint32_t off = (uint32_t)(g0 - row0 * per) + threadIdx.x;
  Eight<WF32> in[U];
  int64_t row[U];
  int col[U];
  bool live[U];
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const uint32_t local = off + 256 * u;
    const uint32_t r = local / (uint32_t)per;
    row[u] = row0 + r;
    col[u] = 8 * (int)(local - r * (uint32_t)per);
    const int id = a.ids[min(row[u], a.N - 1)];
    live[u] = id >= 0 && id < a.V;
    in[u].load(static_cast<const char*>(a.W) + (int64_t)(live[u] ? id : 0) * a.H * (WF32 ? 4 : 2), col[u], a.H - col[u]);
  }
#pragma unroll
  for (int u = 0; u < U; ++u) {
    if (row[u] >= a.N) continue;
    float v[8];
#pragma unroll
    for (int k = 0; k < 8; ++k) v[k] = live[u] ? in[u].at(k) * a.scale : 0.0f;
    Eight<YF32> out;
    out.set(v);
    out.store(static_cast<char*>(a.y) + row[u] * a.H * (YF32 ? 4 : 2), col[u], a.H - col[u]);
  }
}

constexpr int kSortWaves = 16;

// Exclusive sum over the workgroup's threads; total is the whole sum. `red`
// holds kSortWaves words.
__device__ __forceinline__ int block_scan(int x, int* red, int& total) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  int s = x;
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) {
    const int o = __shfl_up(s, d);
    if (lane >= d) s += o;
  }
  if (lane == 63) red[wave] = s;
  __syncthreads();
  int base = 0;
  total = 0;
  for (int w = 0; w < (int)(blockDim.x >> 6); ++w) {
    if (w < wave) base += red[w];
    total += red[w];
  }
  __syncthreads();
  return base + s - x;
}

template <int LC>
__global__ __launch_bounds__(64 * kSortWaves) void embed_sort_kernel(const EmbedBwdArgs a) {
  __shared__ int cnt[kSortWaves][LC];   // tokens of the class's word l in the wave's part, then where the wave's next goes
  __shared__ int red[kSortWaves];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int c = blockIdx.x, mask = a.classes - 1, shift = a.class_shift;
  const int lc = a.class_words;   // <= LC
  for (int i = tid; i < kSortWaves * LC; i += 64 * kSortWaves) (&cnt[0][0])[i] = 0;
  __syncthreads();
  const int part = (a.N + kSortWaves - 1) / kSortWaves;
  const int i0 = min(a.N, wave * part), i1 = min(a.N, i0 + part);
  int lower = 0;
#pragma unroll 4
  for (int i = i0 + lane; i < i1; i += 64) {
    const int id = a.ids[i];
    const bool live = id >= 0 && id < a.V;
    const int k = id & mask;
    lower += live && k < c;
    if (live && k == c) atomicAdd(&cnt[wave][id >> shift], 1);
  }
  int below;
  block_scan(lower, red, below);
  // the class's words in order: their tokens' places, and their pieces
  constexpr int per = (LC + 64 * kSortWaves - 1) / (64 * kSortWaves);
  int tot[per], n_tok = 0, n_pc = 0, n_lg = 0;
#pragma unroll
  for (int k = 0; k < per; ++k) {
    const int l = tid * per + k;
    tot[k] = 0;
    if (l < lc)
      for (int w = 0; w < kSortWaves; ++w) tot[k] += cnt[w][l];
    n_tok += tot[k];
    n_pc += (tot[k] + kPiece - 1) / kPiece;
    n_lg += tot[k] > kPiece;
  }
  int own, pieces, longs;
  int at = below + block_scan(n_tok, red, own);
  int pc = below + block_scan(n_pc, red, pieces);
  int lg = below / kPiece + block_scan(n_lg, red, longs);
#pragma unroll
  for (int k = 0; k < per; ++k) {
    const int l = tid * per + k;
    if (l >= lc) break;
    const int64_t v = ((int64_t)l << shift) + c;
    if (v < a.V) a.touched[(int64_t)c * lc + l] = tot[k] > 0;
    int to = at;
    for (int w = 0; w < kSortWaves; ++w) {
      const int n = cnt[w][l];
      cnt[w][l] = to;
      to += n;
    }
    const bool several = tot[k] > kPiece;
    if (several) a.longs[lg++] = make_int4(at, tot[k], (int)v, 0);
    for (int r = 0; r < tot[k]; r += kPiece)
      a.pieces[pc++] = make_int4(at + r, min(kPiece, tot[k] - r), (int)v,
                                 several ? 2 * ((at + r) / kPiece) + (r == 0) : -1);
    at += tot[k];
  }
  if (tid == 0) {
    a.counts[3 * c] = pieces;
    a.counts[3 * c + 1] = below;
    a.counts[3 * c + 2] = longs;
  }
  __syncthreads();
  // The wave's tokens to their places: a wave's counters are its own, and
  // tokens of one word among the 64 in flight go in lane order.
  for (int i = i0; i < i1; i += 64) {
    const int id = i + lane < i1 ? a.ids[i + lane] : -1;
    const bool mine = id >= 0 && id < a.V && (id & mask) == c;
    uint64_t todo = __ballot(mine);
    while (todo != 0) {
      const int word = __builtin_amdgcn_readlane(id, __builtin_ctzll(todo));
      const uint64_t same = __ballot(mine && id == word);
      const int to = cnt[wave][word >> shift];
      if (mine && id == word) a.order[to + __popcll(same & ((1ull << lane) - 1))] = i + lane;
      __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
      __builtin_amdgcn_wave_barrier();
      if (lane == 0) cnt[wave][word >> shift] = to + __popcll(same);
      __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
      __builtin_amdgcn_wave_barrier();
      todo &= ~same;
    }
  }
}

// scale times the sum, onto what the row holds where it is added to.
template <bool GF32>
__device__ __forceinline__ void put_row(const EmbedBwdArgs& a, int64_t v, int col, int n, float (&s)[8]) {
  char* row = static_cast<char*>(a.dW) + v * a.H * (GF32 ? 4 : 2);
  Eight<GF32> out;
  if (a.add) {
    out.load(row, col, n);
#pragma unroll
    for (int k = 0; k < 8; ++k) s[k] = fmaf(s[k], a.scale, out.at(k));
  } else {
#pragma unroll
    for (int k = 0; k < 8; ++k) s[k] *= a.scale;
  }
  out.set(s);
  out.store(row, col, n);
}

constexpr int kZeroRows = 8;   // rows that a wave looks at together

template <bool YF32, bool GF32>
__global__ __launch_bounds__(256) void embed_rows_kernel(const EmbedBwdArgs a) {
  __shared__ int first[kMostClasses + 1];   // pieces of the classes before
  __shared__ int red[4];
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int H = a.H;
  int total;
  {
    const int per = (a.classes + 255) / 256;
    int n = 0;
    for (int k = 0; k < per; ++k) n += tid * per + k < a.classes ? a.counts[3 * (tid * per + k)] : 0;
    int at = block_scan(n, red, total);
    for (int k = 0; k < per; ++k) {
      if (tid * per + k >= a.classes) break;
      first[tid * per + k] = at;
      at += a.counts[3 * (tid * per + k)];
    }
    __syncthreads();
  }
  const int chunks = (H + 511) / 512;
  const int64_t units = (int64_t)total * chunks;
  const int64_t waves = (int64_t)gridDim.x * 4, me = (int64_t)blockIdx.x * 4 + wave;
  for (int64_t u = me; u < units; u += waves) {
    const int g = (int)(u / chunks);
    int col = ((int)(u - (int64_t)g * chunks) * 64 + lane) * 8;
    const bool in = col < H;
    col = in ? col : 0;   // lanes past the row read along: every lane's token is read by the others
    int c = 0;   // the last class that begins at or before g
    for (int step = a.classes >> 1; step > 0; step >>= 1)
      if (first[c + step] <= g) c += step;
    const int4 p = a.pieces[a.counts[3 * c + 1] + g - first[c]];
    const int mine = a.order[p.x + min(lane, p.y - 1)];
    const int n = H - col;
    float s[8];
#pragma unroll
    for (int k = 0; k < 8; ++k) s[k] = 0.0f;
    auto row = [&](int t) { return static_cast<const char*>(a.dy) + (int64_t)__builtin_amdgcn_readlane(mine, t) * H * (YF32 ? 4 : 2); };
    constexpr int D = 4;
    int t = 0;
    for (; t + D <= p.y; t += D) {
      Eight<YF32> x[D];
#pragma unroll
      for (int d = 0; d < D; ++d) x[d].load(row(t + d), col, n);
#pragma unroll
      for (int d = 0; d < D; ++d)
#pragma unroll
        for (int k = 0; k < 8; ++k) s[k] += x[d].at(k);
    }
    for (; t < p.y; ++t) {
      Eight<YF32> x;
      x.load(row(t), col, n);
#pragma unroll
      for (int k = 0; k < 8; ++k) s[k] += x.at(k);
    }
    if (!in) continue;
    if (p.w < 0) {
      put_row<GF32>(a, p.z, col, n, s);
    } else {
      Eight<true> out;
      out.set(s);
      out.store(a.part + (int64_t)p.w * H, col, n);
    }
  }
  if (a.add) return;
  const int64_t groups = (a.V + kZeroRows - 1) / kZeroRows;
  for (int64_t u = me; u < groups; u += waves) {
    const int64_t v = u * kZeroRows + (lane & (kZeroRows - 1));
    bool empty = lane < kZeroRows && v < a.V;
    if (empty) empty = a.touched[(v & (a.classes - 1)) * a.class_words + (v >> a.class_shift)] == 0;
    uint64_t todo = __ballot(empty);
    while (todo != 0) {
      const int r = __builtin_ctzll(todo);
      todo &= todo - 1;
      char* row = static_cast<char*>(a.dW) + (u * kZeroRows + r) * H * (GF32 ? 4 : 2);
      Eight<GF32> none;
      const float zero[8] = {0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f};
      none.set(zero);
      for (int col = lane * 8; col < H; col += 512) none.store(row, col, H - col);
    }
  }
}

// A workgroup per class: the partial rows of its long words, in order.
template <bool GF32>
__global__ __launch_bounds__(256) void embed_join_kernel(const EmbedBwdArgs a) {
  const int c = blockIdx.x;
  const int n_long = a.counts[3 * c + 2], base = a.counts[3 * c + 1] / kPiece;
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int H = a.H, chunks = (H + 511) / 512;
  for (int u = wave; u < n_long * chunks; u += 4) {
    const int4 w = a.longs[base + u / chunks];
    const int col = (u % chunks * 64 + lane) * 8;
    const int n = H - col;
    if (n <= 0) continue;
    const int pieces = (w.y + kPiece - 1) / kPiece, slot = w.x / kPiece;
    Eight<true> x;
    x.load(a.part + (int64_t)(2 * slot + 1) * H, col, n);
    float s[8];
#pragma unroll
    for (int k = 0; k < 8; ++k) s[k] = x.at(k);
#pragma unroll 4
    for (int p = 1; p < pieces; ++p) {
      x.load(a.part + (int64_t)(2 * (slot + p)) * H, col, n);
#pragma unroll
      for (int k = 0; k < 8; ++k) s[k] += x.at(k);
    }
    put_row<GF32>(a, w.z, col, n, s);
  }
}

}  // namespace

hipError_t launch_embed_fwd(const EmbedFwdArgs& a, hipStream_t stream) {
  const int64_t groups = a.N * ((a.H + 7) / 8);
  const double N = (double)a.N, H = a.H;
  trace_begin(stream);
  auto launch = [&](auto w, auto y, auto u) {
    const int64_t blocks = (groups + 256 * u() - 1) / (256 * u());
    hipLaunchKernelGGL((embed_fwd_kernel<w(), y(), u()>), dim3((unsigned)blocks), dim3(256), 0, stream, a);
  };
  auto sized = [&](auto w, auto y) {
    if (groups <= 256 * 2 * kNumCUs) launch(w, y, std::integral_constant<int, 1>{});
    else launch(w, y, std::integral_constant<int, 4>{});
  };
  std::true_type yes;
  std::false_type no;
  if (a.w_f32) a.y_f32 ? sized(yes, yes) : sized(yes, no);
  else a.y_f32 ? sized(no, yes) : sized(no, no);
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  trace_end(kEmbedFwd, stream, N * H, N * H * ((a.w_f32 ? 4 : 2) + (a.y_f32 ? 4 : 2)) + 4.0 * N);
  return hipSuccess;
}

hipError_t launch_embed_bwd(const EmbedBwdArgs& a, hipStream_t stream) {
  const double N = (double)a.N, H = a.H, V = (double)a.V;
  trace_begin(stream);
  if (a.class_words <= 640)
    hipLaunchKernelGGL((embed_sort_kernel<640>), dim3(a.classes), dim3(64 * kSortWaves), 0, stream, a);
  else
    hipLaunchKernelGGL((embed_sort_kernel<kMostClassWords>), dim3(a.classes), dim3(64 * kSortWaves), 0, stream, a);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  trace_end(kEmbedSort, stream, 0.0, 24.0 * N + V);
  std::true_type yes;
  std::false_type no;
  const int chunks = (a.H + 511) / 512;
  const int64_t units = std::max<int64_t>((int64_t)a.N * chunks, a.add ? 0 : (a.V + kZeroRows - 1) / kZeroRows);
  trace_begin(stream);
  auto rows = [&](auto y, auto g) {
    const int64_t blocks = std::max<int64_t>(1, std::min<int64_t>((units + 3) / 4, 8 * kNumCUs));
    hipLaunchKernelGGL((embed_rows_kernel<y(), g()>), dim3((unsigned)blocks), dim3(256), 0, stream, a);
  };
  if (a.y_f32) a.g_f32 ? rows(yes, yes) : rows(yes, no);
  else a.g_f32 ? rows(no, yes) : rows(no, no);
  e = hipGetLastError();
  if (e != hipSuccess) return e;
  const double g = a.g_f32 ? 4.0 : 2.0;
  trace_end(kEmbedRows, stream, N * H, N * H * (a.y_f32 ? 4 : 2) + (a.add ? std::min(N, V) * 2.0 : V) * H * g);
  if (a.N <= kPiece) return hipSuccess;   // no word has several pieces
  trace_begin(stream);
  if (a.g_f32) hipLaunchKernelGGL((embed_join_kernel<true>), dim3(a.classes), dim3(256), 0, stream, a);
  else hipLaunchKernelGGL((embed_join_kernel<false>), dim3(a.classes), dim3(256), 0, stream, a);
  e = hipGetLastError();
  if (e != hipSuccess) return e;
  trace_end(kEmbedJoin, stream, 0.0, 12.0 * a.classes);
  return hipSuccess;
}

}  // namespace lmh
