// lmhead_embed.hip -- the vocabulary table as an embedding, for gfx950: the
// lookup with its scale, and the table's gradient.
//
//   y_i  = scale W[id_i]                      (0 for an id outside [0, V))
//   dW_v (+)= scale sum_{i: id_i = v} dy_i
//
// The gradient's sums run over the tokens of a word in the tokens' order, in
// pieces of at most kPiece tokens. The pieces' sums are added as eight runs of
// neighbouring ones, each in order, and then run by run. No atomics take part in
// sums: results depend on the arguments alone. Two ways lead there, with the same
// bits.
//
// Many tokens, sorted by word first (stably):
//   sort   workgroup c owns the words v with v mod NC = c. Words that follow one
//          another fall to different workgroups, so a table sorted by frequency
//          loads them alike. Each scans all ids (its 16 waves a sixteenth each),
//          counts those of its words in LDS and those of lower classes (which is
//          where its part of the order begins: no word passes between
//          workgroups), and scans again to place its tokens.
//   rows   a wave sums one piece over 64 groups of columns, straight into dW
//          where it is the word's only one, into a float32 partial row else, and
//          in between zeroes rows without a token.
//   join   partial rows of the words of several pieces, in order.
//
// Up to kFewIds tokens, counted: a workgroup per token looks at all ids for its
// own word and knows from the counts whether a piece begins with its token, of
// which tokens, and where the piece lies in the sorted order; other workgroups
// look for the words of 64 rows each and zero the rest. N^2 comparisons, but one
// launch, or two where a word may have several pieces.
//
// All sums are float32; a bf16 gradient is rounded once, when stored.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include <algorithm>
#include <type_traits>

#include "lmhead_internal.h"

namespace lmh {
namespace {

__device__ __forceinline__ uint16_t narrow(float x) { return __builtin_bit_cast(uint16_t, (__bf16)x); }
__device__ __forceinline__ uint32_t narrow2(float lo, float hi) {
  return (uint32_t)narrow(lo) | ((uint32_t)narrow(hi) << 16);
}

// G elements of a row, at their own alignment: rows of an odd length start off
// any larger boundary, which global memory accepts. G is 8 (16 bytes a lane)
// where both sides are bf16 and 4 (16 bytes of the float32 side) else, so that
// a wave's accesses cover whole lines of the larger side. TAIL: rows are no
// multiple of G, and their last elements are taken one by one.
template <int WORDS>
struct __attribute__((packed, aligned(2))) Raw {
  uint32_t w[WORDS];
};
template <bool F32, int G, bool TAIL>
struct Part {
  static constexpr int kWords = G * (F32 ? 4 : 2) / 4;
  typedef uint32_t Words __attribute__((ext_vector_type(kWords), aligned(2)));
  Raw<kWords> raw;
  // n < G: the last elements of a row. STREAM: past the caches, for what they
  // cannot hold anyway
  template <bool STREAM = false>
  __device__ __forceinline__ void load(const void* row, int at, int n) {
    if (!TAIL || n >= G) {
      const char* from = static_cast<const char*>(row) + (int64_t)at * (F32 ? 4 : 2);
      if constexpr (STREAM) {
        const Words w = __builtin_nontemporal_load(reinterpret_cast<const Words*>(from));
#pragma unroll
        for (int k = 0; k < kWords; ++k) raw.w[k] = w[k];
      } else {
        raw = *reinterpret_cast<const Raw<kWords>*>(from);
      }
      return;
    }
    uint32_t u[G];
#pragma unroll
    for (int k = 0; k < G; ++k) {
      u[k] = 0;
      if (k < n) u[k] = F32 ? static_cast<const uint32_t*>(row)[at + k] : static_cast<const uint16_t*>(row)[at + k];
    }
#pragma unroll
    for (int k = 0; k < kWords; ++k) raw.w[k] = F32 ? u[k] : u[2 * k % G] | (u[(2 * k + 1) % G] << 16);
  }
  __device__ __forceinline__ float at(int k) const {
    if (F32) return __uint_as_float(raw.w[k]);
    const uint32_t w = raw.w[k / 2];
    return __uint_as_float((k & 1) ? (w & 0xFFFF0000u) : (w << 16));
  }
  __device__ __forceinline__ void set(const float (&v)[G]) {
#pragma unroll
    for (int k = 0; k < G; k += F32 ? 1 : 2) raw.w[F32 ? k : k / 2] = F32 ? __float_as_uint(v[k]) : narrow2(v[k], v[k + 1]);
  }
  template <bool STREAM = false>
  __device__ __forceinline__ void store(void* row, int at, int n) const {
    if (!TAIL || n >= G) {
      char* to = static_cast<char*>(row) + (int64_t)at * (F32 ? 4 : 2);
      if constexpr (STREAM) {
        Words w;
#pragma unroll
        for (int k = 0; k < kWords; ++k) w[k] = raw.w[k];
        __builtin_nontemporal_store(w, reinterpret_cast<Words*>(to));
      } else {
        *reinterpret_cast<Raw<kWords>*>(to) = raw;
      }
      return;
    }
#pragma unroll
    for (int k = 0; k < G; ++k) {
      if (k >= n) break;
      if (F32) static_cast<uint32_t*>(row)[at + k] = raw.w[k];
      else static_cast<uint16_t*>(row)[at + k] = (uint16_t)(raw.w[k / 2] >> (16 * (k & 1)));
    }
  }
};

// Forward: a thread takes U groups of G elements, 256 apart in the row-major
// order of all of them: nothing is shared between rows, and any N and H fill the
// launch alike. Widening is exact, the product float32, and bf16 y rounded once.
// Bound by y's stores: 15237 rows of 4096 words (bf16 to float32, 250 MB of y
// and 54 MB of distinct rows) take 47 us, 6.5 TB/s, where a copy reaches 5.0 and
// a fill 6.7; 4099 x 1001 takes 6 us, one row 2.2. STREAM and U = 2 where y
// is larger than the caches near the units hold: 48 us, where plain stores take 87
// and one group a thread 51; smaller outputs are read from those caches next, and
// one group a thread spreads their few workgroups over all CUs.
template <bool WF32, bool YF32, bool TAIL, bool STREAM, int U>
__global__ __launch_bounds__(256) void embed_fwd_kernel(const EmbedFwdArgs a) {
  constexpr int G = WF32 || YF32 ? 4 : 8;
  const int per = (a.H + G - 1) / G;   // groups of a row
  const int64_t g0 = (int64_t)blockIdx.x * (256 * U);
  const int64_t row0 = g0 / per;
  const uint32_t off = (uint32_t)(g0 - row0 * per) + threadIdx.x;
  Part<WF32, G, TAIL> in[U];
  int64_t row[U];
  int col[U];
  bool live[U];
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const uint32_t local = off + 256 * u;
    const uint32_t r = local / (uint32_t)per;
    row[u] = row0 + r;
    col[u] = G * (int)(local - r * (uint32_t)per);
    const int id = a.ids[min(row[u], a.N - 1)];
    live[u] = id >= 0 && id < a.V;
    in[u].load(static_cast<const char*>(a.W) + (int64_t)(live[u] ? id : 0) * a.H * (WF32 ? 4 : 2), col[u], a.H - col[u]);
  }
#pragma unroll
  for (int u = 0; u < U; ++u) {
    if (row[u] >= a.N) continue;
    float v[G];
#pragma unroll
    for (int k = 0; k < G; ++k) v[k] = live[u] ? in[u].at(k) * a.scale : 0.0f;
    Part<YF32, G, TAIL> out;
    out.set(v);
    out.template store<STREAM>(static_cast<char*>(a.y) + row[u] * a.H * (YF32 ? 4 : 2), col[u], a.H - col[u]);
  }
}

constexpr int kSortWaves = 16;

// Exclusive sums over the workgroup's threads; total is the whole sum. `red`
// holds an entry per wave.
__device__ __forceinline__ int4 plus(int4 a, int4 b) { return make_int4(a.x + b.x, a.y + b.y, a.z + b.z, a.w + b.w); }
__device__ __forceinline__ int plus(int a, int b) { return a + b; }
__device__ __forceinline__ int4 minus(int4 a, int4 b) { return make_int4(a.x - b.x, a.y - b.y, a.z - b.z, a.w - b.w); }
__device__ __forceinline__ int minus(int a, int b) { return a - b; }
__device__ __forceinline__ int4 shfl_up(int4 v, int d) {
  return make_int4(__shfl_up(v.x, d), __shfl_up(v.y, d), __shfl_up(v.z, d), __shfl_up(v.w, d));
}
__device__ __forceinline__ int shfl_up(int v, int d) { return __shfl_up(v, d); }
template <class T, int W>
__device__ __forceinline__ T block_scan(T x, T (&red)[W], T& total) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  T s = x;
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) {
    const T o = shfl_up(s, d);
    if (lane >= d) s = plus(s, o);
  }
  if (lane == 63) red[wave] = s;
  __syncthreads();
  T base{};
  total = T{};
#pragma unroll
  for (int w = 0; w < W; ++w) {
    const T r = red[w];
    if (w < wave) base = plus(base, r);
    total = plus(total, r);
  }
  __syncthreads();
  return minus(plus(base, s), x);
}

__device__ __forceinline__ void wave_fence() {
  __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
  __builtin_amdgcn_wave_barrier();
}

// Tokens by word. `found` is what a wave found in its part of the ids, while it
// fits: it places them from there, and not from the ids again.
// N ids a workgroup, N / 16 a wave: bound by the vector unit above 8000 tokens
// or so (65536: 17 us, of 256 CUs that each look at all ids), by a chain of
// trips to memory and LDS below (4096: 6.8). A sort by digits reads the ids twice
// or more often, with a launch between, of 2 us at least each. LC: words of a
// class that LDS counts, 640 (up to 163840 words; 104 KB with 512 found tokens a
// wave) or kMostClassWords (152 KB with 192), which takes two words a thread and
// clears three times the counters: 65536 tokens of 163840 words 21 us, of 163841
// 37; 4096 tokens 8.7 and 10.0.
template <int LC>
__global__ __launch_bounds__(64 * kSortWaves) void embed_sort_kernel(const EmbedBwdArgs a) {
  __shared__ int cnt[kSortWaves][LC];   // tokens of the class's word l in the wave's part, then where the wave's next goes
  __shared__ int4 red[kSortWaves];
  constexpr int kFound = LC > 1024 ? 192 : 512;   // within 160 KB of LDS
  __shared__ int2 found[kSortWaves][kFound];      // (token, word)
  const int tid = threadIdx.x, lane = tid & 63;
  const int c = blockIdx.x, mask = a.classes - 1, shift = a.class_shift;
  // the part of the ids that a wave takes, turned by the class: workgroups side by side read different ones
  const int wave = __builtin_amdgcn_readfirstlane(((tid >> 6) + c) % kSortWaves);
  const int lc = a.class_words;   // <= LC
  for (int i = tid; i < kSortWaves * LC; i += 64 * kSortWaves) (&cnt[0][0])[i] = 0;
  __syncthreads();
  const int part = (a.N + kSortWaves - 1) / kSortWaves;
  const int i0 = min(a.N, wave * part), i1 = min(a.N, i0 + part);
  constexpr int D = 16;   // vectors of 64 ids in flight
  int lower = 0, n_found = 0;
  // whole batches are loaded without a bound, which costs as much as all the
  // rest: the scan is bound by the vector unit
  auto scan = [&](int i, auto vectors, auto whole) {
    constexpr int n = vectors();
    const int32_t* from = a.ids + i;
    int id[n];
#pragma unroll
    for (int d = 0; d < n; ++d) id[d] = whole() ? from[64 * d + lane] : a.ids[min(i + 64 * d + lane, i1 - 1)];
#pragma unroll
    for (int d = 0; d < n; ++d) {
      const bool live = (uint32_t)id[d] < (uint32_t)a.V && (whole() || i + 64 * d + lane < i1);
      const int k = id[d] & mask;
      lower += __popcll(__ballot(live && k < c));   // on the scalar unit
      const bool mine = live && k == c;
      const uint64_t all = __ballot(mine);
      if (all == 0) continue;
      const int at = n_found + __popcll(all & ((1ull << lane) - 1));
      if (mine) {
        atomicAdd(&cnt[wave][id[d] >> shift], 1);
        if (at < kFound) found[wave][at] = make_int2(i + 64 * d + lane, id[d]);
      }
      n_found += __popcll(all);
    }
  };
  int at_id = i0;
#pragma unroll 1
  for (; at_id + 64 * D <= i1; at_id += 64 * D) scan(at_id, std::integral_constant<int, D>{}, std::true_type{});
#pragma unroll 1
  for (; at_id < i1; at_id += 64 * 4) scan(at_id, std::integral_constant<int, 4>{}, std::false_type{});
  // the class's words in order: their tokens' places
  constexpr int per = (LC + 64 * kSortWaves - 1) / (64 * kSortWaves);
  __syncthreads();   // every wave's tokens are counted
  int of[per][kSortWaves], tot[per], n_tok = 0, n_pc = 0, n_lg = 0;
#pragma unroll
  for (int k = 0; k < per; ++k) {
    const int l = tid * per + k;
    tot[k] = 0;
#pragma unroll
    for (int w = 0; w < kSortWaves; ++w) {
      of[k][w] = l < lc ? cnt[w][l] : 0;
      tot[k] += of[k][w];
    }
    n_tok += tot[k];
    n_pc += (tot[k] + kPiece - 1) / kPiece;
    n_lg += tot[k] > kPiece;
  }
  // tokens, pieces and long words of the words before, and tokens of lower classes, in one go
  int4 sum, all;
  sum = block_scan(make_int4(n_tok, n_pc, n_lg, lane == 0 ? lower : 0), red, all);
  const int below = all.w, pieces = all.y, longs = all.z;
  int at = below + sum.x, pc = below + sum.y, lg = below / kPiece + sum.z;
  {
    int to = at;
#pragma unroll
    for (int k = 0; k < per; ++k) {
      const int l = tid * per + k;
#pragma unroll
      for (int w = 0; w < kSortWaves; ++w) {
        if (l < lc) cnt[w][l] = to;
        to += of[k][w];
      }
    }
  }
  __syncthreads();
  // the pieces, and which rows have a token: after the last barrier, none of
  // which then waits for these stores
  if (tid == 0) {
    a.counts[3 * c] = pieces;
    a.counts[3 * c + 1] = below;
    a.counts[3 * c + 2] = longs;
  }
#pragma unroll
  for (int k = 0; k < per; ++k) {
    const int l = tid * per + k;
    const int v = (l << shift) + c;
    if (l < lc && v < a.V) a.touched[(int64_t)c * lc + l] = tot[k] > 0;
    const bool several = tot[k] > kPiece;
    if (tot[k] > 0 && !several) a.pieces[pc] = make_int4(at, tot[k], v, -1);
    if (several) a.longs[lg++] = make_int4(at, tot[k], v, 0);
    // a long word's pieces are listed by the whole wave
    uint64_t todo = __ballot(several);
    while (todo != 0) {
      const int who = __builtin_ctzll(todo);
      todo &= todo - 1;
      const int from = __builtin_amdgcn_readlane(at, who), n = __builtin_amdgcn_readlane(tot[k], who);
      const int word = __builtin_amdgcn_readlane(v, who), to_pc = __builtin_amdgcn_readlane(pc, who);
      for (int r = lane * kPiece; r < n; r += 64 * kPiece)
        a.pieces[to_pc + r / kPiece] = make_int4(from + r, min(kPiece, n - r), word, 2 * ((from + r) / kPiece) + (r == 0));
    }
    pc += (tot[k] + kPiece - 1) / kPiece;
    at += tot[k];
  }
  // The wave's tokens to their places: a wave's counters are its own, and
  // tokens of one word among the 64 in flight go in lane order.
  auto place = [&](bool mine, int token, int id) {
    uint64_t todo = __ballot(mine);
    while (todo != 0) {
      const int word = __builtin_amdgcn_readlane(id, __builtin_ctzll(todo));
      const uint64_t same = __ballot(mine && id == word);
      const int to = cnt[wave][word >> shift];
      if (mine && id == word) a.order[to + __popcll(same & ((1ull << lane) - 1))] = token;
      wave_fence();
      if (lane == 0) cnt[wave][word >> shift] = to + __popcll(same);
      wave_fence();
      todo &= ~same;
    }
  };
  if (n_found <= kFound) {
    for (int k = 0; k < n_found; k += 64) {
      const int2 f = found[wave][min(k + lane, n_found - 1)];
      place(k + lane < n_found, f.x, f.y);
    }
    return;
  }
  // more than were kept (a word of every tenth token, say): all ids once more
#pragma unroll 1
  for (int i = i0; i < i1; i += 64 * D) {
    int id[D];
#pragma unroll
    for (int d = 0; d < D; ++d) id[d] = a.ids[min(i + 64 * d + lane, i1 - 1)];
#pragma unroll
    for (int d = 0; d < D; ++d)
      place(i + 64 * d + lane < i1 && (uint32_t)id[d] < (uint32_t)a.V && (id[d] & mask) == c, i + 64 * d + lane, id[d]);
  }
}

// scale times the sum, onto what the row holds where it is added to.
template <bool GF32, int G, bool TAIL>
__device__ __forceinline__ void put_row(void* dW, bool add, float scale, int H, int64_t v, int col, int n, float (&s)[G]) {
  char* row = static_cast<char*>(dW) + v * H * (GF32 ? 4 : 2);
  Part<GF32, G, TAIL> out;
  if (add) {
    out.load(row, col, n);
#pragma unroll
    for (int k = 0; k < G; ++k) s[k] = fmaf(s[k], scale, out.at(k));
  } else {
#pragma unroll
    for (int k = 0; k < G; ++k) s[k] *= scale;
  }
  out.set(s);
  out.store(row, col, n);
}

// Sums the rows row_of(0) .. row_of(count - 1) of dy over CB groups of columns
// (col, col + 64 G, ...) and stores them: into dW's row v, or (slot >= 0) into a
// partial row. A group past the row reads its beginning along and is not stored.
template <bool YF32, bool GF32, int G, bool TAIL, bool STREAM, bool STREAM_IN, int CB, class F>
__device__ __forceinline__ void sum_piece(const EmbedBwdArgs& a, int col, int count, int64_t v, int slot, F row_of) {
  const int H = a.H;
  int at[CB];
  float s[CB][G];
  Part<GF32, G, TAIL> old[CB];
  const bool add = a.add && slot < 0;
  char* into = static_cast<char*>(a.dW) + v * H * (GF32 ? 4 : 2);
#pragma unroll
  for (int c = 0; c < CB; ++c) {
    at[c] = col + 64 * G * c < H ? col + 64 * G * c : 0;
#pragma unroll
    for (int k = 0; k < G; ++k) s[c][k] = 0.0f;
    if (add) old[c].load(into, at[c], H - at[c]);
  }
  auto row = [&](int t) { return static_cast<const char*>(a.dy) + (int64_t)row_of(t) * H * (YF32 ? 4 : 2); };
  constexpr int D = 8 / CB;
  int t = 0;
  for (; t + D <= count; t += D) {
    Part<YF32, G, TAIL> x[D][CB];
#pragma unroll
    for (int d = 0; d < D; ++d)
#pragma unroll
      for (int c = 0; c < CB; ++c) x[d][c].template load<STREAM_IN>(row(t + d), at[c], H - at[c]);
#pragma unroll
    for (int d = 0; d < D; ++d)
#pragma unroll
      for (int c = 0; c < CB; ++c)
#pragma unroll
        for (int k = 0; k < G; ++k) s[c][k] += x[d][c].at(k);
  }
  for (; t < count; ++t) {
    Part<YF32, G, TAIL> x[CB];
#pragma unroll
    for (int c = 0; c < CB; ++c) x[c].template load<STREAM_IN>(row(t), at[c], H - at[c]);
#pragma unroll
    for (int c = 0; c < CB; ++c)
#pragma unroll
      for (int k = 0; k < G; ++k) s[c][k] += x[c].at(k);
  }
#pragma unroll
  for (int c = 0; c < CB; ++c) {
    if (col + 64 * G * c >= H) continue;
    const int n = H - at[c];
    if (slot >= 0) {
      Part<true, G, TAIL> out;
      out.set(s[c]);
      out.store(a.part + (int64_t)slot * H, at[c], n);
      continue;
    }
#pragma unroll
    for (int k = 0; k < G; ++k) s[c][k] = add ? fmaf(s[c][k], a.scale, old[c].at(k)) : s[c][k] * a.scale;
    Part<GF32, G, TAIL> out;
    out.set(s[c]);
    out.template store<STREAM>(into, at[c], n);
  }
}

// Zeroes the rows v of dW without a token (has(v) is 0 for them), as workgroup
// `me` of `blocks`: the table as it lies, 16 bytes a thread and 4 KB a
// workgroup at once, the workgroups side by side. Walked by rows, it takes 141
// us where this takes 115 (778 MB). The flags of the next kZeroAhead places are
// on their way while the last ones' are used.
constexpr int kZeroAhead = 8;
template <bool GF32, class F>
__device__ __forceinline__ void zero_rows(const EmbedBwdArgs& a, int me, int blocks, F has) {
  constexpr int size = GF32 ? 4 : 2;
  typedef uint32_t words __attribute__((ext_vector_type(4), aligned(2)));
  const uint32_t row_bytes = (uint32_t)a.H * size;
  const int64_t bytes = (int64_t)a.V * row_bytes;
  const uint32_t step = (uint32_t)blocks * 4096, step_rows = step / row_bytes, step_rest = step - step_rows * row_bytes;
  const uint32_t first = (uint32_t)me * 4096 + threadIdx.x * 16;
  uint32_t row = first / row_bytes, rest = first - row * row_bytes;   // of the next place whose flag is fetched
  int64_t at = first;
  uint32_t rows[kZeroAhead], rests[kZeroAhead];
  bool keep[kZeroAhead];
  auto fetch = [&]() {
#pragma unroll
    for (int k = 0; k < kZeroAhead; ++k) {
      rows[k] = row;
      rests[k] = rest;
      keep[k] = has((int)min(row, (uint32_t)a.V - 1)) != 0;
      row += step_rows;
      rest += step_rest;
      if (rest >= row_bytes) {
        rest -= row_bytes;
        ++row;
      }
    }
  };
  fetch();
  while (at < bytes) {
    uint32_t r[kZeroAhead], o[kZeroAhead];
    bool kept[kZeroAhead];
#pragma unroll
    for (int k = 0; k < kZeroAhead; ++k) {
      r[k] = rows[k];
      o[k] = rests[k];
      kept[k] = keep[k];
    }
    fetch();
#pragma unroll
    for (int k = 0; k < kZeroAhead; ++k, at += step) {
      if (at >= bytes) break;
      char* to = static_cast<char*>(a.dW) + at;
      if (o[k] + 16 <= row_bytes) {
        if (!kept[k]) __builtin_nontemporal_store(words{0, 0, 0, 0}, reinterpret_cast<words*>(to));
        continue;
      }
      // across the end of a row: element by element
      uint32_t v = r[k], left = row_bytes - o[k];
      bool full = kept[k];
      for (uint32_t e = 0; e < 16 && at + e < bytes; e += size) {
        if (left == 0) {
          full = has((int)++v) != 0;
          left = row_bytes;
        }
        if (!full) {
          if (GF32) *reinterpret_cast<uint32_t*>(to + e) = 0;
          else *reinterpret_cast<uint16_t*>(to + e) = 0;
        }
        left -= size;
      }
    }
  }
}

// The partial rows of a long word (first place in the order, tokens) over one
// wave's columns, by a workgroup: its waves take runs of neighbouring pieces,
// whose sums are added in order.
constexpr int kJoinWaves = 8;
static_assert(8 * kMostClasses <= 64 << 10, "LDS of embed_rows_kernel's classes");
template <bool GF32, bool TAIL>
__device__ __forceinline__ void join_row(const EmbedBwdArgs& a, int first, int tokens, int64_t v, int col, float4 (&xch)[kJoinWaves][64]) {
  constexpr int G = 4;
  const int H = a.H, lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const bool in = col < H;
  col = in ? col : 0;
  const int n = H - col;
  const int pieces = (tokens + kPiece - 1) / kPiece, slot = first / kPiece;
  const int run = (pieces + kJoinWaves - 1) / kJoinWaves, p0 = wave * run, p1 = min(pieces, p0 + run);
  float s[G] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll 8
  for (int p = p0; p < p1; ++p) {
    Part<true, G, TAIL> x;
    x.load(a.part + (int64_t)(2 * (slot + p) + (p == 0)) * H, col, n);
#pragma unroll
    for (int k = 0; k < G; ++k) s[k] += x.at(k);
  }
  xch[wave][lane] = make_float4(s[0], s[1], s[2], s[3]);
  __syncthreads();
  if (wave == 0 && in) {
#pragma unroll
    for (int w = 1; w < kJoinWaves; ++w) {
      const float4 o = xch[w][lane];
      s[0] += o.x;
      s[1] += o.y;
      s[2] += o.z;
      s[3] += o.w;
    }
    put_row<GF32, G, TAIL>(a.dW, a.add, a.scale, H, v, col, n, s);
  }
  __syncthreads();   // read before the next word's
}

constexpr int kRowGroups = 1;   // groups of columns that a wave sums at once
constexpr int kRowsPerCU = 5, kAddsPerCU = 8;   // workgroups that fit, zeroing rows beside them or adding
constexpr int kZeroBlocks = kNumCUs;   // those that zero rows, one a CU beside four that sum

// The first kZeroBlocks workgroups zero rows, unless dW is added to; the others
// sum pieces. Bound by memory where there is much of it: 65536 rows of 2560
// into 151936 rows take 247 us for 1.10 GB (4.4 TB/s; 336 MB of gathered rows of
// 5 KB, 778 MB of stores, 115 us of them by themselves), 131072 rows added to 34000
// rows 186 us for 1.0 GB (5.5 TB/s). 4096 rows added to 2250 take 13 us for 42 MB,
// a wave's one or two pieces one after the other. ADD has eight workgroups a CU
// (131072 rows 186 us where five take 195) and its classes' places in LDS, which
// saves a trip to memory a piece. Written, with zeroing beside, both make the
// frequent words' case slower (65536 rows 242 us, 253 with the places, 262 with
// eight) and the uniform one faster (262, 248, 222). 128 zeroing workgroups take
// 289 us, 512 300 (with uniform words).
template <bool YF32, bool GF32, bool TAIL, bool STREAM_IN, bool ADD>
__global__ __launch_bounds__(256, ADD ? kAddsPerCU : kRowsPerCU) void embed_rows_kernel(const EmbedBwdArgs a) {
  constexpr int G = YF32 || GF32 ? 4 : 8;
  extern __shared__ int first[];   // pieces of the classes before; ADD: and where the class's begin, less those
  __shared__ int red[4];
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  constexpr int zero_blocks = ADD ? 0 : kZeroBlocks;
  if (!ADD && (int)blockIdx.x < zero_blocks) {
    zero_rows<GF32>(a, blockIdx.x, kZeroBlocks, [&](int v) {
      return a.touched[(int64_t)(v & (a.classes - 1)) * a.class_words + (v >> a.class_shift)];
    });
    return;
  }
  int total;
  {
    const int per = a.classes / 256;
    int n = 0;
    for (int k = 0; k < per; ++k) n += a.counts[3 * (tid * per + k)];
    int at = block_scan(n, red, total);
    for (int k = 0; k < per; ++k) {
      const int c = tid * per + k;
      first[c] = at;
      if (ADD) first[a.classes + c] = a.counts[3 * c + 1] - at;
      at += a.counts[3 * c];
    }
    __syncthreads();
  }
  // piece g: the last class that begins at or before it, of the first 256 by
  // steps of `per` at once
  const int per = a.classes / 256;
  int mark[4];
#pragma unroll
  for (int k = 0; k < 4; ++k) mark[k] = first[(64 * k + lane) * per];
  auto piece = [&](int g) {
    if (g >= total) return make_int4(0, 1, 0, -1);
    int c = -1;
#pragma unroll
    for (int k = 0; k < 4; ++k) c += __popcll(__ballot(mark[k] <= g));
    c *= per;
    for (int step = per >> 1; step > 0; step >>= 1)
      if (first[c + step] <= g) c += step;
    return a.pieces[(ADD ? first[a.classes + c] : a.counts[3 * c + 1] - first[c]) + g];
  };
  auto tokens = [&](const int4& p) { return a.order[p.x + min(lane, p.y - 1)]; };
  const int chunks = (a.H + 64 * G * kRowGroups - 1) / (64 * G * kRowGroups);
  const int waves = ((int)gridDim.x - zero_blocks) * 4, me = ((int)blockIdx.x - zero_blocks) * 4 + wave;   // `chunks` waves at least
  const int step = waves / chunks;
  int g = me / chunks;
  const int col = ((me - g * chunks) * 64 * kRowGroups + lane) * G;
  if (g >= step || g >= total) return;
  // the piece after the next and the next one's tokens are on their way while a
  // piece is summed
  int4 p0 = piece(g), p1 = piece(g + step);
  int t0 = tokens(p0);
  for (; g < total; g += step) {
    const int4 p2 = piece(g + 2 * step);
    const int t1 = tokens(p1);
    sum_piece<YF32, GF32, G, TAIL, true, STREAM_IN, kRowGroups>(a, col, p0.y, p0.z, p0.w, [&](int t) { return __builtin_amdgcn_readlane(t0, t); });
    p0 = p1;
    p1 = p2;
    t0 = t1;
  }
}

// A class's long words; kJoinParts workgroups share their columns. Bound by the
// longest word's chain of pieces: 11 us for 65536 tokens with a word of 4000,
// 4.1 for 4096; 81 where 131072 tokens are one word.
constexpr int kJoinParts = 8;
template <bool GF32, bool TAIL>
__global__ __launch_bounds__(64 * kJoinWaves) void embed_join_kernel(const EmbedBwdArgs a) {
  __shared__ float4 xch[kJoinWaves][64];
  const int c = blockIdx.x / kJoinParts;
  const int n_long = a.counts[3 * c + 2], base = a.counts[3 * c + 1] / kPiece;
  const int chunks = (a.H + 255) / 256;
  for (int u = blockIdx.x % kJoinParts; u < n_long * chunks; u += kJoinParts) {
    const int4 w = a.longs[base + u / chunks];
    join_row<GF32, TAIL>(a, w.x, w.y, w.z, (u % chunks * 64 + (threadIdx.x & 63)) * 4, xch);
  }
}

// Few tokens, a workgroup per token: if a piece begins with it, its sum. Each
// wave looks at a fourth of the ids, 64 neighbours at a time. Bound by the chain
// ids, list, rows: 256 tokens of 256 columns take 5 us. Against sort, rows and
// join (H 2560, added): 1500 tokens 13 us to 20, 2048 16 to 19, 4096 31 to 23;
// kFewIds lies between.
constexpr int kFewPer = kFewIds / 256;
template <bool YF32, bool GF32, bool TAIL>
__global__ __launch_bounds__(256) void embed_few_kernel(const EmbedBwdArgs a) {
  constexpr int G = YF32 || GF32 ? 4 : 8;
  extern __shared__ uint32_t seen[];   // bits of the words that occur
  __shared__ int4 red[4];
  __shared__ int list[kPiece];
  const int tid = threadIdx.x;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int N = a.N;
  const int zero_blocks = (int)gridDim.x - N;   // the first ones, so that they spread over the CUs
  if ((int)blockIdx.x < zero_blocks) {
    for (int w = tid; w < (a.V + 31) / 32; w += 256) seen[w] = 0;
    __syncthreads();
    for (int i = tid; i < N; i += 256) {
      const int id = a.ids[i];
      if (id >= 0 && id < a.V) atomicOr(&seen[id >> 5], 1u << (id & 31));
    }
    __syncthreads();
    zero_rows<GF32>(a, blockIdx.x, zero_blocks, [&](int v) { return (seen[v >> 5] >> (v & 31)) & 1; });
    return;
  }
  const int i = (int)blockIdx.x - zero_blocks, word = a.ids[i];
  if (N > kPiece && tid == 0) a.longs[i] = make_int4(0, 0, 0, 0);   // thread 0 fills it below, if at all
  if (word < 0 || word >= a.V) return;
  const int lane = tid & 63, vectors = (N + 255) / 256, j0 = wave * vectors * 64;
  int id[kFewPer];
#pragma unroll
  for (int k = 0; k < kFewPer; ++k)
    if (k < vectors) id[k] = a.ids[min(j0 + 64 * k + lane, N - 1)];
#pragma unroll
  for (int k = 0; k < kFewPer; ++k) id[k] = k < vectors && j0 + 64 * k + lane < min(N, j0 + 64 * vectors) ? id[k] : -1;
  int same = 0, before = 0, less = 0;
#pragma unroll
  for (int k = 0; k < kFewPer; ++k) {
    same += __popcll(__ballot(id[k] == word));
    before += __popcll(__ballot(id[k] == word && j0 + 64 * k + lane < i));
    less += __popcll(__ballot(id[k] >= 0 && id[k] < word));
  }
  if (lane == 0) red[wave] = make_int4(same, before, less, 0);
  __syncthreads();
  int total = 0, ahead = 0, smaller = 0, rank = 0;
#pragma unroll
  for (int w = 0; w < 4; ++w) {
    const int4 r = red[w];
    if (w < wave) rank += r.x;
    total += r.x;
    ahead += r.y;
    smaller += r.z;
  }
  if (ahead % kPiece != 0) return;
#pragma unroll
  for (int k = 0; k < kFewPer; ++k) {
    const uint64_t all = __ballot(id[k] == word);
    if (all == 0) continue;
    const int at = rank + __popcll(all & ((1ull << lane) - 1)) - ahead;
    if (id[k] == word && at >= 0 && at < kPiece) list[at] = j0 + 64 * k + lane;
    rank += __popcll(all);
  }
  __syncthreads();
  const bool several = total > kPiece;
  if (several && ahead == 0 && tid == 0) a.longs[i] = make_int4(smaller, total, word, 0);
  const int count = min(kPiece, total - ahead);
  const int mine = list[min(lane, count - 1)];
  const int slot = several ? 2 * ((smaller + ahead) / kPiece) + (ahead == 0) : -1;
  for (int col = (wave * 64 + lane) * G; col - lane * G < a.H; col += 256 * G)
    sum_piece<YF32, GF32, G, TAIL, false, false, 1>(a, col, count, word, slot, [&](int t) { return __builtin_amdgcn_readlane(mine, t); });
}

// A workgroup per 64 tokens and 256 columns: the long words among them.
template <bool GF32, bool TAIL>
__global__ __launch_bounds__(64 * kJoinWaves) void embed_few_join_kernel(const EmbedBwdArgs a) {
  __shared__ float4 xch[kJoinWaves][64];
  const int lane = threadIdx.x & 63;
  const int chunks = (a.H + 255) / 256;
  const int block = blockIdx.x / chunks, col = ((int)(blockIdx.x - block * chunks) * 64 + lane) * 4;
  const int i = block * 64 + lane;
  const int4 w = i < a.N ? a.longs[i] : make_int4(0, 0, 0, 0);
  uint64_t todo = __ballot(w.y > 0);   // every wave looks at the same tokens
  while (todo != 0) {
    const int l = __builtin_ctzll(todo);
    todo &= todo - 1;
    join_row<GF32, TAIL>(a, __builtin_amdgcn_readlane(w.x, l), __builtin_amdgcn_readlane(w.y, l), __builtin_amdgcn_readlane(w.z, l), col, xch);
  }
}

}  // namespace

namespace {
template <class F>
void with_types(bool a, bool b, bool tail, F f) {
  std::true_type yes;
  std::false_type no;
  auto second = [&](auto x) {
    auto third = [&](auto y) { tail ? f(x, y, yes) : f(x, y, no); };
    b ? third(yes) : third(no);
  };
  a ? second(yes) : second(no);
}
}  // namespace

hipError_t launch_embed_fwd(const EmbedFwdArgs& a, hipStream_t stream) {
  const int G = a.w_f32 || a.y_f32 ? 4 : 8;
  const int64_t groups = a.N * ((a.H + G - 1) / G);
  const double N = (double)a.N, H = a.H;
  trace_begin(stream);
  with_types(a.w_f32, a.y_f32, a.H % G != 0, [&](auto w, auto y, auto tail) {
    auto launch = [&](auto stream_y, auto u) {
      const int64_t blocks = (groups + 256 * u() - 1) / (256 * u());
      hipLaunchKernelGGL((embed_fwd_kernel<w(), y(), tail(), stream_y(), u()>), dim3((unsigned)blocks), dim3(256), 0, stream, a);
    };
    if (N * H * (a.y_f32 ? 4 : 2) > kStreamed) launch(std::true_type{}, std::integral_constant<int, 2>{});
    else launch(std::false_type{}, std::integral_constant<int, 1>{});
  });
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  trace_end(kEmbedFwd, stream, N * H, N * H * ((a.w_f32 ? 4 : 2) + (a.y_f32 ? 4 : 2)) + 4.0 * N);
  return hipSuccess;
}

hipError_t launch_embed_bwd(const EmbedBwdArgs& a, hipStream_t stream) {
  const double N = (double)a.N, H = a.H, V = (double)a.V, g = a.g_f32 ? 4.0 : 2.0;
  const double rows_bytes = N * H * (a.y_f32 ? 4 : 2) + (a.add ? std::min(N, V) * 2.0 : V) * H * g;
  const int G = a.y_f32 || a.g_f32 ? 4 : 8;
  const bool tail = a.H % G != 0;
  const int chunks = (a.H + 64 * G * kRowGroups - 1) / (64 * G * kRowGroups), chunks4 = (a.H + 255) / 256;
  hipError_t e;
  if (a.few) {
    trace_begin(stream);
    const int blocks = a.N + (a.add ? 0 : (int)std::min<int64_t>(kZeroBlocks, ((int64_t)a.V * a.H * (int)g + 4095) / 4096));
    with_types(a.y_f32, a.g_f32, tail, [&](auto y, auto gf, auto t) {
      hipLaunchKernelGGL((embed_few_kernel<y(), gf(), t()>), dim3((unsigned)blocks), dim3(256), a.add ? 0 : (a.V + 31) / 32 * 4, stream, a);
    });
    e = hipGetLastError();
    if (e != hipSuccess) return e;
    trace_end(kEmbedFew, stream, N * H, rows_bytes);
    if (a.N <= kPiece) return hipSuccess;   // no word has several pieces
    trace_begin(stream);
    with_types(a.g_f32, false, a.H % 4 != 0, [&](auto gf, auto, auto t) {
      hipLaunchKernelGGL((embed_few_join_kernel<gf(), t()>), dim3((unsigned)((a.N + 63) / 64 * chunks4)), dim3(64 * kJoinWaves), 0,
                         stream, a);
    });
    e = hipGetLastError();
    if (e != hipSuccess) return e;
    trace_end(kEmbedJoin, stream, 0.0, 16.0 * N);
    return hipSuccess;
  }
  trace_begin(stream);
  if (a.class_words <= 640)
    hipLaunchKernelGGL((embed_sort_kernel<640>), dim3(a.classes), dim3(64 * kSortWaves), 0, stream, a);
  else
    hipLaunchKernelGGL((embed_sort_kernel<kMostClassWords>), dim3(a.classes), dim3(64 * kSortWaves), 0, stream, a);
  e = hipGetLastError();
  if (e != hipSuccess) return e;
  trace_end(kEmbedSort, stream, 0.0, 24.0 * N + V);
  const int64_t units = std::max<int64_t>((int64_t)a.N, 1) * chunks;
  const int64_t most = a.add ? kAddsPerCU * kNumCUs : kRowsPerCU * kNumCUs - kZeroBlocks;
  const int64_t blocks = std::max<int64_t>((chunks + 3) / 4, std::min<int64_t>((units + 3) / 4, most)) + (a.add ? 0 : kZeroBlocks);
  trace_begin(stream);
  with_types(a.y_f32, a.g_f32, tail, [&](auto y, auto gf, auto t) {
    auto launch = [&](auto past, auto add) {
      hipLaunchKernelGGL((embed_rows_kernel<y(), gf(), t(), past(), add()>), dim3((unsigned)blocks), dim3(256),
                         (add() ? 8 : 4) * a.classes, stream, a);
    };
    std::true_type yes;
    std::false_type no;
    // dy past the caches where the memory-side one does not hold it: 65536 rows of 5 KB (335 MB) added 113 us instead
    // of 128, but 16384 rows 38 instead of 28
    if (N * H * (a.y_f32 ? 4 : 2) > kMemoryCache) a.add ? launch(yes, yes) : launch(yes, no);
    else a.add ? launch(no, yes) : launch(no, no);
  });
  e = hipGetLastError();
  if (e != hipSuccess) return e;
  trace_end(kEmbedRows, stream, N * H, rows_bytes);
  trace_begin(stream);
  with_types(a.g_f32, false, a.H % 4 != 0, [&](auto gf, auto, auto t) {
    hipLaunchKernelGGL((embed_join_kernel<gf(), t()>), dim3(a.classes * kJoinParts), dim3(64 * kJoinWaves), 0, stream, a);
  });
  e = hipGetLastError();
  if (e != hipSuccess) return e;
  trace_end(kEmbedJoin, stream, 0.0, 12.0 * a.classes);
  return hipSuccess;
}

}  // namespace lmh
