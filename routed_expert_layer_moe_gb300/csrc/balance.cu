// Load-balance loss of the router, with per-expert counts, and its gradient.
//
// For a segment of n tokens with scores p_t that sum to one, c_e the ids equal to e and
// P_e = sum_t p_te:  loss = coef E / (K n^2) sum_e c_e P_e.  With v_e = coef E / (K n^2) c_e
// and the counts held constant, the gradient of a softmax row is p_j (v_j - sum_i v_i p_i);
// of a normalised sigmoid row that times 1 - sigmoid(l_j).  Adding a constant to v changes
// nothing, so v is taken less its mean: near balance the counts differ by a few percent, and the
// difference v_j - sum_i v_i p_i would otherwise lose those digits.
//
// Both directions read the logits once.  A token's row lies in the registers of a group of 8, 16
// or 32 lanes, so a warp works on up to four tokens at a time and its shuffles serve all of
// them, and the next rows are requested before this step's arithmetic.  65536 x 256 sigmoid scores:
// a warp per token and no request ahead took 64 and 52 us, held by the latency of one row at a
// time; groups of lanes 21.7 and 25.3 us (0.6 of the first for the rows of low sigmoids, see `scores`); 10 and 20 us is
// the memory's rate, 2-3 us of each go to start and end.
// The sums over tokens use no float
// atomics: the token range is cut into `ntiles` equal tiles, a tile meets the segments in
// pieces, and the piece of tile i in segment b is row i + b of the partial sums -- distinct for
// every piece, because along the tokens i and b only grow and at least one of them does from
// one piece to the next.  A second kernel adds each segment's rows in a fixed order.
#include <algorithm>
#include <type_traits>

#include "common.cuh"

namespace moe {
namespace {

constexpr int kWarps = 8;
constexpr int kThreads = 32 * kWarps;
constexpr int kFinishThreads = 512;  // of the second kernel
constexpr int kMinChunk = 8;         // experts of one of its CTAs at least: a 32-byte sector of a row
constexpr float kLog2e = 1.4426950408889634f;

// Tokens of one tile: about three tiles per SM, at least 32 (each tile costs the second kernel a row).
constexpr int kTilesPerSm = 3;
constexpr int kMaxTiles = 512;
constexpr int kMinTile = 32;
constexpr int kMaxCluster = 8;  // tiles of a batch that takes one launch
int tile_tokens(int T) {
  const int tiles = std::min(std::max(kTilesPerSm * device_info().sm_count, 1), kMaxTiles);
  return std::max((T + tiles - 1) / tiles, kMinTile);
}

// Rows of partial sums: a bound on the tiles that needs no device, plus the segments.
int64_t piece_rows(int64_t T, int nseq) {
  return std::min<int64_t>((T + kMinTile - 1) / kMinTile, kMaxTiles) + nseq;
}

struct Segments {
  const int32_t* off;  // null: one segment [0, T)
  int nseq, T;
  __device__ __forceinline__ int lo(int b) const { return off ? max(__ldg(off + b), 0) : 0; }
  __device__ __forceinline__ int hi(int b) const { return off ? min(__ldg(off + b + 1), T) : T; }
  // Offsets that a warp holds: v0, v1 = off[a + lane], off[a + 32 + lane] for the n <= 63 segments from a on.
  struct Window {
    int a = 0, n = 0, v0 = 0, v1 = 0;
    __device__ __forceinline__ int at(int i) const {  // off[a + i], the same i in every lane
      const int x = __shfl_sync(0xffffffffu, v0, i & 31), y = __shfl_sync(0xffffffffu, v1, i & 31);
      return i < 32 ? x : y;
    }
  };

  // The last segment that starts at or before t (the one that holds t, if any does), with its bounds.  For a t before
  // all segments: NEXT: the last one that starts where the first does (those before it are empty, so it is the
  // next with tokens, if any has); else any one, which does not hold t.  By a whole warp, the same t in every lane and t growing from call
  // to call: many places are looked at together, for one after the other each costs the memory's latency (six
  // of them for 48 segments), and kept for the next call: a tile that several short segments meet would pay
  // for each of them.
  template <bool NEXT>
  __device__ __forceinline__ int find(int t, Window& w, int& first, int& end) const {
    if (!off) {
      first = 0, end = T;
      return 0;
    }
    const int lane = threadIdx.x & 31;
    unsigned m0, m1;
    for (int pass = 0;; ++pass) {
      if (w.n == 0 || (w.a + w.n < nseq && w.at(w.n) <= t)) {
        int a = w.a, n = nseq - w.a;
        while (n > 63) {  // 32 steps through what is left
          const int step = (n + 31) / 32, i = lane * step;
          const bool before = i < n && __ldg(off + a + i) <= t;
          const int k = 31 - __clz(__ballot_sync(0xffffffffu, before) | 1u);  // the last place at or before t
          a += k * step;
          n = min(step, n - k * step);
        }
        w.a = a, w.n = min(63, nseq - a);
        w.v0 = lane <= w.n ? __ldg(off + a + lane) : 0;
        w.v1 = lane + 32 <= w.n ? __ldg(off + a + lane + 32) : 0;
      }
      m0 = __ballot_sync(0xffffffffu, lane < w.n && w.v0 <= t);
      m1 = __ballot_sync(0xffffffffu, lane + 32 < w.n && w.v1 <= t);
      if (!NEXT || m0 | m1 || pass) break;
      t = w.at(0);  // no segment starts at or before t: look up the first one's start instead
      w.n = 0;
    }
    const int k = m1 ? 63 - __clz(m1) : 31 - __clz(m0 | 1u);
    first = max(w.at(k), 0);
    end = min(w.at(k + 1), T);
    return w.a + k;
  }
};

// Over the L lanes of a group.
template <int L>
__device__ __forceinline__ float group_sum(float v) {
#pragma unroll
  for (int o = L / 2; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

template <int L>
__device__ __forceinline__ float group_max(float v) {
#pragma unroll
  for (int o = L / 2; o > 0; o >>= 1) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, o));
  return v;
}

// Expert of register j of lane `sub` of a group of L: VEC: float4 chunks, else single ones.
template <int L, bool VEC>
__device__ __forceinline__ int expert_of(int j, int sub) {
  return VEC ? (j >> 2) * 4 * L + sub * 4 + (j & 3) : j * L + sub;
}

// A lane's N values of a row, as pairs: the arithmetic is on pairs (fp32x2 instructions).
template <int N>
struct Row {
  float2 v[N / 2];
  __device__ __forceinline__ float get(int j) const { return j & 1 ? v[j / 2].y : v[j / 2].x; }
  __device__ __forceinline__ void set(int j, float x) {
    if (j & 1)
      v[j / 2].y = x;
    else
      v[j / 2].x = x;
  }
  __device__ __forceinline__ void fill(float x) {
#pragma unroll
    for (int i = 0; i < N / 2; ++i) v[i] = make_float2(x, x);
  }
};

// One token's logits (N L >= E); -inf past the last expert.  FULL: N L = E, float4 rows.  A masked token's
// are loaded too (and dropped before use): waiting for its mask first would put two memory
// latencies one after the other.
template <int N, int L, bool VEC, bool FULL>
__device__ __forceinline__ void load_row(const float* row, int E, int sub, Row<N>& l) {
  if constexpr (VEC) {
#pragma unroll
    for (int c = 0; c < N / 4; ++c) {
      const int e = c * 4 * L + sub * 4;
      float4 v = make_float4(-INFINITY, -INFINITY, -INFINITY, -INFINITY);
      if (FULL || e < E) v = __ldg(reinterpret_cast<const float4*>(row + e));
      l.v[2 * c] = make_float2(v.x, v.y), l.v[2 * c + 1] = make_float2(v.z, v.w);
    }
  } else {
#pragma unroll
    for (int j = 0; j < N; ++j) {
      const int e = j * L + sub;
      l.set(j, e < E ? __ldg(row + e) : -INFINITY);
    }
  }
}

// 2^x and 1/x with the special-function unit's own error (2 ulp and 1 ulp; results under 2^-126 are 0).  The
// scores' error is within 8e-8 of 64 bits so, against 1e-8 with expf and an IEEE division: fp32's own rounding.
__device__ __forceinline__ float fast_exp2(float x) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}

__device__ __forceinline__ float fast_rcp(float x) {
  float r;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}

// e^(l - the row's largest logit) in the lanes that `take` it (every lane of the warp takes part); returns this
// lane's part of their sum.
template <int N, int L>
__device__ __forceinline__ float exponentials(const Row<N>& l, bool take, Row<N>& a) {
  float m = -INFINITY;
#pragma unroll
  for (int i = 0; i < N / 2; ++i) m = fmaxf(m, fmaxf(l.v[i].x, l.v[i].y));
  m = group_max<L>(m);
  // the difference first: l log2 e - m log2 e as one multiply-add has the rounding of m log2 e in every term, which
  // is a power of two too many from |m| = 2^24 on and infinite for a row of the type's lowest value
  const float b = m == -INFINITY ? 0.0f : -m;
  float2 z = make_float2(0.0f, 0.0f);
#pragma unroll
  for (int i = 0; i < N / 2; ++i) {
    const float2 t = __fmul2_rn(__fadd2_rn(l.v[i], make_float2(b, b)), make_float2(kLog2e, kLog2e));
    const float2 e = make_float2(fast_exp2(t.x), fast_exp2(t.y));
    a.v[i] = take ? e : a.v[i];
    z = __fadd2_rn(z, e);
  }
  return z.x + z.y;
}

// Unnormalised scores a of the logits l of a token that takes part (live); returns this lane's part of their
// sum.  Sigmoid scores whose sum in every lane is below kLowSum are tiny or 0, but their ratios are not: the largest logit
// is below -51 there, sigmoid(l) = e^l to 2^-75 of it, and the scores are taken relative to the largest one
// instead (ratio).  In any other row some lane has kLowSum or more, next to which the at most 1024 scores below 2^-126
// that were taken as 0 are 2^-36.
constexpr float kLowSum = 0x1p-80f;

template <int N, int L, bool SIG>
__device__ __forceinline__ float scores(const Row<N>& l, bool live, Row<N>& a, bool& ratio) {
  ratio = false;
  if constexpr (!SIG) return exponentials<N, L>(l, true, a);
  float2 z2 = make_float2(0.0f, 0.0f);
#pragma unroll
  for (int i = 0; i < N / 2; ++i) {
    float2 t = __fmul2_rn(l.v[i], make_float2(-kLog2e, -kLog2e));
    t = __fadd2_rn(make_float2(fast_exp2(t.x), fast_exp2(t.y)), make_float2(1.0f, 1.0f));
    a.v[i] = make_float2(fast_rcp(t.x), fast_rcp(t.y));
    z2 = __fadd2_rn(z2, a.v[i]);
  }
  const float z = z2.x + z2.y;
  const unsigned low = __ballot_sync(0xffffffffu, live && z < kLowSum);
  if (low) {  // lanes of experts that are off, and rarely a whole row
    const unsigned group = (0xffffffffu >> (32 - L)) << (threadIdx.x & 31 & ~(L - 1));
    ratio = (low & group) == group;
    if (__any_sync(0xffffffffu, ratio)) {
      const float y = exponentials<N, L>(l, ratio, a);
      return ratio ? y : z;
    }
  }
  return z;
}

// 1 / the sum over the group; 0 for a row with nothing in it.
template <int L>
__device__ __forceinline__ float inverse_sum(float z) {
  z = group_sum<L>(z);
  return z == 0.0f ? 0.0f : 1.0f / z;
}

// What the calls write.
struct Outputs {
  float* loss;
  int32_t* counts;
  float* prob_sum;
  int32_t* tokens;
};

// ONE: a batch of at most kMaxCluster tiles and as many segments, the CTAs one cluster, which meets after
// the partial sums and adds each segment's rows itself: one launch, not two (128 tokens of 256
// experts: 18.4 us for the loss and its gradient, held by the host's launches).
template <int N, int L, bool VEC, bool SIG, bool FULL, bool ONE>
__global__ void __launch_bounds__(kThreads, N > 16 ? 2 : kTilesPerSm)
    balance_partial_kernel(const float* __restrict__ logits, const int32_t* __restrict__ ids,
                           const uint8_t* __restrict__ valid, Segments seg, int E, int K, int tile, float coef,
                           float* part_p, int32_t* part_c, int32_t* part_n, int32_t* done, Outputs out, int32_t* err) {
  extern __shared__ float smem[];
  float* red = smem;                                             // [kWarps][E]
  int32_t* cnt = reinterpret_cast<int32_t*>(smem + kWarps * E);  // [E]
  __shared__ int ntok;
  constexpr int G = 32 / L;  // tokens of a warp
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, sub = lane % L, grp = lane / L;
  const int t0 = blockIdx.x * tile, t1 = min(seg.T, t0 + tile);
  if (!ONE && blockIdx.x == 0)
    for (int b = threadIdx.x; b < seg.nseq; b += kThreads) done[b] = 0;  // the second kernel's counters
  grid_dependents_launch();  // the second kernel's CTAs may wait on the SMs
  int flags = 0;
  // u: this lane's token of the step at w; its row and ids are requested while the step before it is
  // worked on, those of a piece's first step while its segment is looked up (past the tile's end:
  // the last token's, which are not used)
  constexpr int Q = 32 / L;  // ids a lane counts: K <= 32
  bool next_valid = false;
  Row<N> next;
  int next_id[Q];
  auto request = [&](int u) {
    const int r = min(u, t1 - 1);
    next_valid = !valid || __ldg(valid + r);
    load_row<N, L, VEC, FULL>(logits + (size_t)r * E, E, sub, next);
#pragma unroll
    for (int q = 0; q < Q; ++q)
      if (sub + q * L < K) next_id[q] = __ldg(ids + (size_t)r * K + sub + q * L);
  };
  int t = t0;
  Segments::Window window;
  if (t < t1) request(t + warp * G + grp);
  while (t < t1) {
    int lo, hi;
    const int b = seg.find<true>(t, window, lo, hi);
    const int from = max(t, lo), end = min(t1, hi);  // from: past the tokens before the first segment
    if (end <= from) break;                          // past the last segment
    if (from != t) request(from + warp * G + grp);   // not the step that is on its way
    t = from;
    for (int e = threadIdx.x; e < E; e += kThreads) cnt[e] = 0;
    if (threadIdx.x == 0) ntok = 0;
    __syncthreads();
    Row<N> acc;
    acc.fill(0.0f);
    int mine = 0;
    for (int w = t + warp * G; w < end; w += kWarps * G) {  // the same steps for every lane of a warp
      const bool live = next_valid && w + grp < end;
      if (!__all_sync(0xffffffffu, live) && !live) next.fill(-INFINITY);
      Row<N> a;
      bool ratio;
      const float z = scores<N, L, SIG>(next, live, a, ratio);
      mine += live && sub == 0;
      int id[Q];
#pragma unroll
      for (int q = 0; q < Q; ++q) id[q] = next_id[q];
      if (w + kWarps * G < end) request(w + kWarps * G + grp);
#pragma unroll
      for (int q = 0; q < Q; ++q) {
        if (live && sub + q * L < K) {
          if ((unsigned)id[q] < (unsigned)E)
            atomicAdd(&cnt[id[q]], 1);
          else
            flags = MOE_FLAG_BAD_EXPERT;
        }
      }
      const float inv = inverse_sum<L>(z);
#pragma unroll
      for (int i = 0; i < N / 2; ++i) acc.v[i] = __ffma2_rn(a.v[i], make_float2(inv, inv), acc.v[i]);
    }
    if (end < t1) request(end + warp * G + grp);  // the next piece's first step
    if (mine) atomicAdd(&ntok, mine);
#pragma unroll
    for (int j = 0; j < N; ++j) {
      float sum = acc.get(j);
#pragma unroll
      for (int o = L; o < 32; o <<= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
      const int e = expert_of<L, VEC>(j, sub);
      if (grp == 0 && e < E) red[warp * E + e] = sum;
    }
    __syncthreads();
    const size_t row = (size_t)blockIdx.x + b;
    for (int e = threadIdx.x; e < E; e += kThreads) {
      float s = 0.0f;
#pragma unroll
      for (int w = 0; w < kWarps; ++w) s += red[w * E + e];
      part_p[row * E + e] = s;
      part_c[row * E + e] = cnt[e];
    }
    if (threadIdx.x == 0) part_n[row] = ntok;
    __syncthreads();
    t = end;
  }
  if (flags) atomicOr(err, flags);
  if constexpr (ONE) {
    cluster_sync_all();  // every CTA's rows are visible
    for (int b = blockIdx.x; b < seg.nseq; b += gridDim.x) {
      const int lo = seg.lo(b), hi = seg.hi(b);
      const int i0 = lo / tile, i1 = hi > lo ? (hi - 1) / tile : i0 - 1;
      int n = 0;
      for (int i = i0; i <= i1; ++i) n += __ldcg(part_n + i + b);
      float s = 0.0f;
      for (int e = threadIdx.x; e < E; e += kThreads) {
        float p = 0.0f;
        int c = 0;
#pragma unroll
        for (int k = 0; k < kMaxCluster; ++k) {
          if (i0 + k <= i1) {
            p += __ldcg(part_p + (size_t)(i0 + k + b) * E + e);
            c += __ldcg(part_c + (size_t)(i0 + k + b) * E + e);
          }
        }
        out.counts[(size_t)b * E + e] = c;
        out.prob_sum[(size_t)b * E + e] = p;
        s = fmaf((float)c, p, s);
      }
      s = group_sum<32>(s);
      __syncthreads();  // red is free
      if (lane == 0) red[warp] = s;
      __syncthreads();
      if (threadIdx.x == 0) {
        s = 0.0f;
#pragma unroll
        for (int w = 0; w < kWarps; ++w) s += red[w];
        const float fn = (float)max(n, 1);
        out.loss[b] = coef * (float)E / ((float)K * fn * fn) * s;
        out.tokens[b] = n;
      }
    }
  }
}

// One CTA per (segment, CHUNK experts): adds the segment's rows, ROWS at a time; the segment's last
// CTA adds the chunks' parts of the loss in order.  Each CTA is held by the latency of its loads: few
// segments of many rows take 8 experts and 64 rows (with 32 experts and 16 rows 456 rows of 512
// experts took 12.6 us, not 6.3), many segments of few rows the other way round (4.7 us for 48
// segments of 256 experts, not 9.2).
template <int CHUNK>
__global__ void __launch_bounds__(kFinishThreads)
    balance_finish_kernel(Segments seg, int E, int K, int tile, float coef, const float* part_p, const int32_t* part_c,
                          const int32_t* part_n, float* loss_part, int32_t* done, Outputs out) {
  constexpr int ROWS = kFinishThreads / CHUNK;
  grid_dependency_wait();
  grid_dependents_launch();
  __shared__ float sp[ROWS][CHUNK];
  __shared__ int sc[ROWS][CHUNK];
  __shared__ int sn[ROWS];
  const int b = blockIdx.y, col = threadIdx.x % CHUNK, g = threadIdx.x / CHUNK;
  int e = blockIdx.x * CHUNK + col;
  const int lo = seg.lo(b), hi = seg.hi(b);
  const int i0 = lo / tile, i1 = hi > lo ? (hi - 1) / tile : i0 - 1;
  float p = 0.0f;
  int c = 0, n = 0;
#pragma unroll 4
  for (int i = i0 + g; i <= i1; i += ROWS) {
    const size_t row = (size_t)i + b;
    if (e < E) {
      p += __ldcg(part_p + row * E + e);
      c += __ldcg(part_c + row * E + e);
    }
    if (col == 0) n += __ldcg(part_n + row);
  }
  sp[g][col] = p;
  sc[g][col] = c;
  if (col == 0) sn[g] = n;
  __syncthreads();
  if (threadIdx.x >= 32) return;
  // one warp: 32 / CHUNK groups of rows for each expert, then their sum
  const int lane = threadIdx.x;
  p = 0.0f, c = 0, n = 0;
#pragma unroll
  for (int i = g; i < ROWS; i += 32 / CHUNK) {
    p += sp[i][col];
    c += sc[i][col];
  }
#pragma unroll
  for (int i = lane; i < ROWS; i += 32) n += sn[i];
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    if (o >= CHUNK) {
      p += __shfl_xor_sync(0xffffffffu, p, o);
      c += __shfl_xor_sync(0xffffffffu, c, o);
    }
    n += __shfl_xor_sync(0xffffffffu, n, o);
  }
  if (lane >= CHUNK) e = E;  // the sums are there several times over
  if (e < E) {
    out.counts[(size_t)b * E + e] = c;
    out.prob_sum[(size_t)b * E + e] = p;
  }
  const float part = group_sum<32>(e < E ? (float)c * p : 0.0f);
  int last = 0;
  if (lane == 0) {
    loss_part[(size_t)b * gridDim.x + blockIdx.x] = part;
    __threadfence();
    last = atomicAdd(done + b, 1) == (int)gridDim.x - 1;
  }
  if (!__shfl_sync(0xffffffffu, last, 0)) return;
  __threadfence();
  float s = 0.0f;
  for (int i = lane; i < (int)gridDim.x; i += 32) s += __ldcg(loss_part + (size_t)b * gridDim.x + i);
  s = group_sum<32>(s);
  if (lane == 0) {
    const float fn = (float)max(n, 1);
    out.loss[b] = coef * (float)E / ((float)K * fn * fn) * s;
    out.tokens[b] = n;
  }
}

template <int N, int L, bool VEC, bool SIG, bool FULL>
__global__ void __launch_bounds__(kThreads, N > 16 ? 2 : kTilesPerSm)
    balance_backward_kernel(const float* __restrict__ logits, const uint8_t* __restrict__ valid, Segments seg, int E,
                            int K, int tile, float coef, const int32_t* __restrict__ counts,
                            const int32_t* __restrict__ tokens, const float* __restrict__ dloss,
                            float* __restrict__ dlogits) {
  grid_dependency_wait();
  constexpr int G = 32 / L;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, sub = lane % L, grp = lane / L;
  const int t0 = blockIdx.x * tile, t1 = min(seg.T, t0 + tile);
  Row<N> v;
  v.fill(0.0f);
  int lo = 0, hi = 0;  // the segment that v belongs to
  bool next_live = false;
  Row<N> next;
  auto request = [&](int t) {  // past the tile's end: the last token's row, which is not used
    const int r = min(t, t1 - 1);
    next_live = t < t1 && (!valid || __ldg(valid + r));
    load_row<N, L, VEC, FULL>(logits + (size_t)r * E, E, sub, next);
  };
  const int first = t0 + warp * G;
  if (first < t1) request(first + grp);
  for (int w = first; w < t1; w += kWarps * G) {  // the same steps for every lane of a warp
    const int t = w + grp;
    bool live = next_live;
    if (!__all_sync(0xffffffffu, live) && !live) next.fill(-INFINITY);
    Row<N> a;
    bool ratio;
    const float z = scores<N, L, SIG>(next, live, a, ratio);
    if (w + kWarps * G < t1) request(t + kWarps * G);
    const bool move = live && (t < lo || t >= hi);
    unsigned moving = __ballot_sync(0xffffffffu, move);
    if (moving) {
      int b = 0;
      do {  // the segments of the tokens that left theirs, one token after the other
        const int other = __shfl_sync(0xffffffffu, t, __ffs(moving) - 1);
        int slo, shi;
        Segments::Window window;
        const int s = seg.find<false>(other, window, slo, shi);
        const bool mine = move && (t == other || (t >= slo && t < shi));
        if (mine) {
          b = s;
          lo = slo, hi = shi;
          if (t < lo || t >= hi) lo = hi = 0;  // in no segment
        }
        moving &= ~__ballot_sync(0xffffffffu, mine);
      } while (moving);
      const bool fresh = move && hi > lo;
      Row<N> c;
      float sum = 0.0f;
#pragma unroll
      for (int j = 0; j < N; ++j) {
        const int e = expert_of<L, VEC>(j, sub);
        c.set(j, fresh && e < E ? (float)__ldg(counts + (size_t)b * E + e) : 0.0f);
        sum += c.get(j);
      }
      const float mean = group_sum<L>(sum) / (float)E;
      if (fresh) {
        const float fn = (float)max(__ldg(tokens + b), 1);
        const float scale = coef * (float)E / ((float)K * fn * fn) * __ldg(dloss + b);
#pragma unroll
        for (int j = 0; j < N; ++j) v.set(j, (c.get(j) - mean) * scale);
      }
    }
    live = live && t >= lo && t < hi;
    const float inv = inverse_sum<L>(z);
    float2 d2 = make_float2(0.0f, 0.0f);
    Row<N> g;  // the scores, then the gradient
#pragma unroll
    for (int i = 0; i < N / 2; ++i) {
      g.v[i] = __fmul2_rn(a.v[i], make_float2(inv, inv));
      d2 = __ffma2_rn(g.v[i], v.v[i], d2);
    }
    const float dot = group_sum<L>(d2.x + d2.y);
    if (t >= t1) continue;
    const float minus = ratio ? 0.0f : -1.0f;  // 1 - sigmoid(l) is 1 where the scores are ratios
#pragma unroll
    for (int i = 0; i < N / 2; ++i) {
      g.v[i] = __fmul2_rn(g.v[i], __fadd2_rn(v.v[i], make_float2(-dot, -dot)));
      if (SIG) g.v[i] = __fmul2_rn(g.v[i], __ffma2_rn(a.v[i], make_float2(minus, minus), make_float2(1.0f, 1.0f)));
    }
    if (!live) g.fill(0.0f);
    float* dst = dlogits + (size_t)t * E;
    if constexpr (VEC) {
#pragma unroll
      for (int c = 0; c < N / 4; ++c) {
        const int e = c * 4 * L + sub * 4;
        if (FULL || e < E)
          *reinterpret_cast<float4*>(dst + e) =
              make_float4(g.v[2 * c].x, g.v[2 * c].y, g.v[2 * c + 1].x, g.v[2 * c + 1].y);
      }
    } else {
#pragma unroll
      for (int j = 0; j < N; ++j) {
        const int e = j * L + sub;
        if (e < E) dst[e] = g.get(j);
      }
    }
  }
}

struct Work {
  float* part_p;
  int32_t* part_c;
  int32_t* part_n;
  float* loss_part;
  int32_t* done;
  size_t bytes;
};

Work carve(const moe_problem& p, int nseq, void* ws) {
  Work w{};
  uint8_t* base = static_cast<uint8_t*>(ws);
  const size_t rows = (size_t)piece_rows(p.T, nseq);
  size_t off = 0;
  auto take = [&](size_t bytes) {
    uint8_t* r = base + off;
    off += align_up(bytes, 256);
    return r;
  };
  w.part_p = reinterpret_cast<float*>(take(rows * p.E * 4));
  w.part_c = reinterpret_cast<int32_t*>(take(rows * p.E * 4));
  w.part_n = reinterpret_cast<int32_t*>(take(rows * 4));
  w.loss_part = reinterpret_cast<float*>(take((size_t)nseq * ((p.E + kMinChunk - 1) / kMinChunk) * 4));
  w.done = reinterpret_cast<int32_t*>(take((size_t)nseq * 4));
  w.bytes = off;
  return w;
}

// f(registers a lane, lanes a token, float4 rows, sigmoid, rows that fill the registers) with
// compile-time arguments.  float4 rows need E a multiple of 4 and 16-byte aligned arrays.
template <typename F>
int dispatch(int E, bool vec, int score, F f) {
  auto n = [&](auto v, auto s) {
    constexpr bool V = decltype(v)::value;
    auto full = [&](auto nn, auto l) {
      if constexpr (V) {
        if (E == decltype(nn)::value * decltype(l)::value) return f(nn, l, v, s, std::true_type());
      }
      return f(nn, l, v, s, std::false_type());
    };
    using std::integral_constant;
    if (E <= 32) return full(integral_constant<int, 4>(), integral_constant<int, 8>());
    if (E <= 64) return full(integral_constant<int, 8>(), integral_constant<int, 8>());
    if (E <= 128) return full(integral_constant<int, 16>(), integral_constant<int, 8>());
    if (E <= 256) return full(integral_constant<int, 16>(), integral_constant<int, 16>());
    if (E <= 512) return full(integral_constant<int, 16>(), integral_constant<int, 32>());
    return full(integral_constant<int, 32>(), integral_constant<int, 32>());
  };
  auto s = [&](auto v) {
    return score == MOE_SCORE_SIGMOID ? n(v, std::true_type()) : n(v, std::false_type());
  };
  return vec ? s(std::true_type()) : s(std::false_type());
}

}  // namespace

size_t balance_workspace_bytes(const moe_problem& p, int nseq) { return carve(p, nseq, nullptr).bytes; }

int launch_balance(const moe_problem& p, const float* logits, const int32_t* ids, const uint8_t* valid,
                   const int32_t* seq, int nseq, int score, float coef, float* loss, int32_t* counts,
                   float* prob_sum, int32_t* tokens, int32_t* err, void* ws, cudaStream_t st) {
  const Work w = carve(p, nseq, ws);
  const Segments seg{seq, nseq, p.T};
  const int tile = tile_tokens(p.T);
  const int tiles = p.T > 0 ? (p.T + tile - 1) / tile : 1;  // an empty batch: one CTA clears the counters
  const bool vec = p.E % 4 == 0 && aligned16(logits);
  const size_t smem = (size_t)(kWarps + 1) * p.E * 4;
  const Outputs out{loss, counts, prob_sum, tokens};
  const bool one = tiles <= kMaxCluster && nseq <= kMaxCluster;
  const int r = dispatch(p.E, vec, score, [&](auto n, auto l, auto v, auto s, auto full) {
    auto go = [&](auto o) {
      constexpr bool ONE = decltype(o)::value;
      auto kern = balance_partial_kernel<decltype(n)::value, decltype(l)::value, decltype(v)::value, decltype(s)::value,
                                         decltype(full)::value, ONE>;
      cudaLaunchAttribute attr{};
      cudaLaunchConfig_t cfg{};
      cfg.gridDim = dim3(tiles);
      cfg.blockDim = dim3(kThreads);
      cfg.dynamicSmemBytes = smem;
      cfg.stream = st;
      if (ONE) {  // a whole cluster: CTAs past the last token only meet the others
        int c = 1;
        while (c < tiles) c *= 2;
        attr.id = cudaLaunchAttributeClusterDimension;
        attr.val.clusterDim.x = c;
        attr.val.clusterDim.y = 1;
        attr.val.clusterDim.z = 1;
        cfg.gridDim = dim3(c);
        cfg.attrs = &attr;
        cfg.numAttrs = 1;
      }
      return cudaLaunchKernelEx(&cfg, kern, logits, ids, valid, seg, (int)p.E, (int)p.K, tile, coef, w.part_p, w.part_c,
                                w.part_n, w.done, out, err) == cudaSuccess
                 ? MOE_OK
                 : MOE_ERR_CUDA;
    };
    return one ? go(std::true_type()) : go(std::false_type());
  });
  if (r || one) return r;
  auto finish = [&](auto chunk) {
    constexpr int C = decltype(chunk)::value;
    cudaLaunchAttribute attr = overlap_attribute();
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3((p.E + C - 1) / C, nseq);
    cfg.blockDim = dim3(kFinishThreads);
    cfg.stream = st;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, balance_finish_kernel<C>, seg, (int)p.E, (int)p.K, tile, coef,
                              (const float*)w.part_p, (const int32_t*)w.part_c, (const int32_t*)w.part_n, w.loss_part,
                              w.done, out) == cudaSuccess
               ? MOE_OK
               : MOE_ERR_CUDA;
  };
  return tiles / nseq >= 32 ? finish(std::integral_constant<int, kMinChunk>()) : finish(std::integral_constant<int, 32>());
}

int launch_balance_backward(const moe_problem& p, const float* logits, const uint8_t* valid, const int32_t* seq,
                            int nseq, int score, float coef, const int32_t* counts, const int32_t* tokens,
                            const float* dloss, float* dlogits, cudaStream_t st) {
  if (p.T == 0) return MOE_OK;
  const Segments seg{seq, nseq, p.T};
  const int tile = tile_tokens(p.T);
  const int tiles = (p.T + tile - 1) / tile;
  const bool vec = p.E % 4 == 0 && aligned16(logits) && aligned16(dlogits);
  return dispatch(p.E, vec, score, [&](auto n, auto l, auto v, auto s, auto full) {
    auto kern = balance_backward_kernel<decltype(n)::value, decltype(l)::value, decltype(v)::value, decltype(s)::value,
                                  decltype(full)::value>;
    cudaLaunchAttribute attr = overlap_attribute();
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(tiles);
    cfg.blockDim = dim3(kThreads);
    cfg.stream = st;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kern, logits, valid, seg, (int)p.E, (int)p.K, tile, coef, counts, tokens, dloss,
                              dlogits) == cudaSuccess
               ? MOE_OK
               : MOE_ERR_CUDA;
  });
}

}  // namespace moe
