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
// time; groups of 8 lanes 22 and 24 us; 10 and 20 us is the memory's rate.
// The sums over tokens use no float
// atomics: the token range is cut into `ntiles` equal tiles, a tile meets the segments in
// pieces, and the piece of tile i in segment b is row i + b of the partial sums -- distinct for
// every piece, because along the tokens i and b only grow and at least one of them does from
// one piece to the next.  A second kernel adds each segment's rows in a fixed order.
#include <algorithm>
#include <climits>
#include <type_traits>

#include "common.cuh"

namespace moe {
namespace {

constexpr int kWarps = 8;
constexpr int kThreads = 32 * kWarps;
constexpr int kChunk = 8;         // experts of one CTA of the second kernel: a 32-byte sector of a row
constexpr int kFinishThreads = 512;
constexpr int kFinishRows = kFinishThreads / kChunk;  // partial rows it reads at a time
constexpr float kLog2e = 1.4426950408889634f;

// Tokens of one tile: about three tiles per SM, at least 32 (each tile costs the second kernel a row).
constexpr int kTilesPerSm = 3;
constexpr int kMaxTiles = 512;
constexpr int kMinTile = 32;
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
  // The last segment that starts at or before t (the one that holds t, if any does); 0 if none.
  __device__ __forceinline__ int find(int t) const {
    if (!off) return 0;
    int a = 0, z = nseq;
    while (z - a > 1) {
      const int m = (a + z) >> 1;
      if (__ldg(off + m) <= t)
        a = m;
      else
        z = m;
    }
    return a;
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

// One token's logits, N registers a lane (N L >= E); -inf past the last expert and, without
// `live`, everywhere.
template <int N, int L, bool VEC>
__device__ __forceinline__ void load_row(const float* row, int E, int sub, bool live, float (&l)[N]) {
  if constexpr (VEC) {
#pragma unroll
    for (int c = 0; c < N / 4; ++c) {
      const int e = c * 4 * L + sub * 4;
      float4 v = make_float4(-INFINITY, -INFINITY, -INFINITY, -INFINITY);
      if (live && e < E) v = __ldg(reinterpret_cast<const float4*>(row + e));
      l[4 * c] = v.x, l[4 * c + 1] = v.y, l[4 * c + 2] = v.z, l[4 * c + 3] = v.w;
    }
  } else {
#pragma unroll
    for (int j = 0; j < N; ++j) {
      const int e = j * L + sub;
      l[j] = live && e < E ? __ldg(row + e) : -INFINITY;
    }
  }
}

// 2^x and 1/x with the special-function unit's own error (2 ulp and 1 ulp; results under 2^-126 are 0, which
// no sum of scores notices).
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

// l -> unnormalised scores in place; returns 1 / their sum (0 for a row with nothing in it).
template <int N, int L, bool SIG>
__device__ __forceinline__ float scores(float (&l)[N]) {
  float z = 0.0f;
  if constexpr (SIG) {
#pragma unroll
    for (int j = 0; j < N; ++j) {
      l[j] = fast_rcp(1.0f + fast_exp2(-l[j] * kLog2e));
      z += l[j];
    }
  } else {
    float m = -INFINITY;
#pragma unroll
    for (int j = 0; j < N; ++j) m = fmaxf(m, l[j]);
    m = group_max<L>(m);
    const float b = m == -INFINITY ? 0.0f : m * kLog2e;
#pragma unroll
    for (int j = 0; j < N; ++j) {
      l[j] = fast_exp2(fmaf(l[j], kLog2e, -b));
      z += l[j];
    }
  }
  z = group_sum<L>(z);
  return z == 0.0f ? 0.0f : 1.0f / z;
}

template <int N, int L, bool VEC, bool SIG>
__global__ void __launch_bounds__(kThreads, N > 16 ? 2 : kTilesPerSm)
    balance_partial_kernel(const float* __restrict__ logits, const int32_t* __restrict__ ids,
                           const uint8_t* __restrict__ valid, Segments seg, int E, int K, int tile,
                           float* __restrict__ part_p, int32_t* __restrict__ part_c, int32_t* __restrict__ part_n,
                           int32_t* __restrict__ done, int32_t* err) {
  extern __shared__ float smem[];
  float* red = smem;                                             // [kWarps][E]
  int32_t* cnt = reinterpret_cast<int32_t*>(smem + kWarps * E);  // [E]
  __shared__ int ntok;
  constexpr int G = 32 / L;  // tokens of a warp
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, sub = lane % L, grp = lane / L;
  const int t0 = blockIdx.x * tile, t1 = min(seg.T, t0 + tile);
  if (blockIdx.x == 0)
    for (int b = threadIdx.x; b < seg.nseq; b += kThreads) done[b] = 0;  // the second kernel's counters
  int flags = 0;
  int t = max(t0, seg.lo(0));
  while (t < t1) {
    const int b = seg.find(t);
    const int end = min(t1, seg.hi(b));
    if (end <= t) break;  // past the last segment
    for (int e = threadIdx.x; e < E; e += kThreads) cnt[e] = 0;
    if (threadIdx.x == 0) ntok = 0;
    __syncthreads();
    float acc[N];
#pragma unroll
    for (int j = 0; j < N; ++j) acc[j] = 0.0f;
    int mine = 0;
    // u: this lane's token of the step at w; its row and ids are requested while the step before it
    // is worked on
    constexpr int Q = 32 / L;  // ids a lane counts: K <= 32
    bool next_live = false;
    float next[N];
    int next_id[Q];
    auto request = [&](int u) {
      next_live = u < end && !(valid && !__ldg(valid + u));
      load_row<N, L, VEC>(logits + (size_t)u * E, E, sub, next_live, next);
#pragma unroll
      for (int q = 0; q < Q; ++q)
        next_id[q] = next_live && sub + q * L < K ? __ldg(ids + (size_t)u * K + sub + q * L) : INT_MIN;
    };
    const int first = t + warp * G;
    if (first < end) request(first + grp);
    for (int w = first; w < end; w += kWarps * G) {  // the same steps for every lane of a warp
      float l[N];
      int id[Q];
#pragma unroll
      for (int j = 0; j < N; ++j) l[j] = next[j];
#pragma unroll
      for (int q = 0; q < Q; ++q) id[q] = next_id[q];
      mine += next_live && sub == 0;
      const bool live = next_live;
      if (w + kWarps * G < end) request(w + kWarps * G + grp);
#pragma unroll
      for (int q = 0; q < Q; ++q) {
        if (live && sub + q * L < K) {
          if (id[q] >= 0 && id[q] < E)
            atomicAdd(&cnt[id[q]], 1);
          else
            flags = MOE_FLAG_BAD_EXPERT;
        }
      }
      const float inv = scores<N, L, SIG>(l);
#pragma unroll
      for (int j = 0; j < N; ++j) acc[j] = fmaf(l[j], inv, acc[j]);
    }
    if (mine) atomicAdd(&ntok, mine);
#pragma unroll
    for (int j = 0; j < N; ++j) {
#pragma unroll
      for (int o = L; o < 32; o <<= 1) acc[j] += __shfl_xor_sync(0xffffffffu, acc[j], o);
      const int e = expert_of<L, VEC>(j, sub);
      if (grp == 0 && e < E) red[warp * E + e] = acc[j];
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
}

// One CTA per (segment, kChunk experts): adds the segment's rows; the segment's last CTA adds the
// chunks' parts of the loss in order.  Few CTAs work when there is one segment, each held by the
// latency of its loads, so a CTA takes 64 rows at a time (16 rows of 32 experts: 12.6 us for
// 456 rows of 512 experts).
__global__ void __launch_bounds__(kFinishThreads)
    balance_finish_kernel(Segments seg, int E, int K, int tile, float coef, const float* __restrict__ part_p,
                          const int32_t* __restrict__ part_c, const int32_t* __restrict__ part_n,
                          float* __restrict__ loss_part, int32_t* done, float* __restrict__ loss,
                          int32_t* __restrict__ counts, float* __restrict__ prob_sum, int32_t* __restrict__ tokens) {
  __shared__ float sp[kFinishRows][kChunk];
  __shared__ int sc[kFinishRows][kChunk];
  __shared__ int sn[kFinishRows];
  const int b = blockIdx.y, col = threadIdx.x % kChunk, g = threadIdx.x / kChunk;
  int e = blockIdx.x * kChunk + col;
  const int lo = seg.lo(b), hi = seg.hi(b);
  const int i0 = lo / tile, i1 = hi > lo ? (hi - 1) / tile : i0 - 1;
  float p = 0.0f;
  int c = 0, n = 0;
#pragma unroll 4
  for (int i = i0 + g; i <= i1; i += kFinishRows) {
    const size_t row = (size_t)i + b;
    if (e < E) {
      p += __ldg(part_p + row * E + e);
      c += __ldg(part_c + row * E + e);
    }
    if (col == 0) n += __ldg(part_n + row);
  }
  sp[g][col] = p;
  sc[g][col] = c;
  if (col == 0) sn[g] = n;
  __syncthreads();
  if (threadIdx.x >= 32) return;
  // one warp: four groups of rows for each expert, then their sum
  const int lane = threadIdx.x;
  p = 0.0f, c = 0;
#pragma unroll
  for (int i = 0; i < kFinishRows / 4; ++i) {
    p += sp[4 * i + g][col];
    c += sc[4 * i + g][col];
  }
  n = sn[lane] + sn[lane + 32];
  static_assert(kFinishRows == 64 && kChunk == 8, "the warp above covers 4 x 8 and 2 x 32 values");
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    if (o >= kChunk) {
      p += __shfl_xor_sync(0xffffffffu, p, o);
      c += __shfl_xor_sync(0xffffffffu, c, o);
    }
    n += __shfl_xor_sync(0xffffffffu, n, o);
  }
  if (lane >= kChunk) e = E;  // the sums are there four times over
  if (e < E) {
    counts[(size_t)b * E + e] = c;
    prob_sum[(size_t)b * E + e] = p;
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
    loss[b] = coef * (float)E / ((float)K * fn * fn) * s;
    tokens[b] = n;
  }
}

template <int N, int L, bool VEC, bool SIG>
__global__ void __launch_bounds__(kThreads, N > 16 ? 2 : kTilesPerSm)
    balance_backward_kernel(const float* __restrict__ logits, const uint8_t* __restrict__ valid, Segments seg, int E,
                            int K, int tile, float coef, const int32_t* __restrict__ counts,
                            const int32_t* __restrict__ tokens, const float* __restrict__ dloss,
                            float* __restrict__ dlogits) {
  constexpr int G = 32 / L;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, sub = lane % L, grp = lane / L;
  const int t0 = blockIdx.x * tile, t1 = min(seg.T, t0 + tile);
  float v[N];
#pragma unroll
  for (int j = 0; j < N; ++j) v[j] = 0.0f;
  int lo = 0, hi = 0;  // the segment that v belongs to
  auto is_live = [&](int t) { return t < t1 && !(valid && !__ldg(valid + t)); };
  const int first = t0 + warp * G;
  bool next_live = is_live(first + grp);
  float next[N];
  if (first < t1) load_row<N, L, VEC>(logits + (size_t)(first + grp) * E, E, sub, next_live, next);
  for (int w = first; w < t1; w += kWarps * G) {  // the same steps for every lane of a warp
    const int t = w + grp;
    bool live = next_live;
    float l[N];
#pragma unroll
    for (int j = 0; j < N; ++j) l[j] = next[j];
    if (w + kWarps * G < t1) {
      next_live = is_live(t + kWarps * G);
      load_row<N, L, VEC>(logits + (size_t)(t + kWarps * G) * E, E, sub, next_live, next);
    }
    const bool move = live && (t < lo || t >= hi);
    if (__any_sync(0xffffffffu, move)) {
      int b = 0;
      if (move) {
        b = seg.find(t);
        lo = seg.lo(b), hi = seg.hi(b);
        if (t < lo || t >= hi) lo = hi = 0;  // in no segment
      }
      const bool fresh = move && hi > lo;
      float c[N], sum = 0.0f;
#pragma unroll
      for (int j = 0; j < N; ++j) {
        const int e = expert_of<L, VEC>(j, sub);
        c[j] = fresh && e < E ? (float)__ldg(counts + (size_t)b * E + e) : 0.0f;
        sum += c[j];
      }
      const float mean = group_sum<L>(sum) / (float)E;
      if (fresh) {
        const float fn = (float)max(__ldg(tokens + b), 1);
        const float scale = coef * (float)E / ((float)K * fn * fn) * __ldg(dloss + b);
#pragma unroll
        for (int j = 0; j < N; ++j) v[j] = (c[j] - mean) * scale;
      }
    }
    live = live && t >= lo && t < hi;
    const float inv = scores<N, L, SIG>(l);
    float dot = 0.0f;
#pragma unroll
    for (int j = 0; j < N; ++j) dot = fmaf(l[j] * inv, v[j], dot);
    dot = group_sum<L>(dot);
    if (t >= t1) continue;
#pragma unroll
    for (int j = 0; j < N; ++j) {
      const float d = l[j] * inv * (v[j] - dot);
      l[j] = live ? (SIG ? d * (1.0f - l[j]) : d) : 0.0f;
    }
    float* dst = dlogits + (size_t)t * E;
    if constexpr (VEC) {
#pragma unroll
      for (int c = 0; c < N / 4; ++c) {
        const int e = c * 4 * L + sub * 4;
        if (e < E)
          *reinterpret_cast<float4*>(dst + e) = make_float4(l[4 * c], l[4 * c + 1], l[4 * c + 2], l[4 * c + 3]);
      }
    } else {
#pragma unroll
      for (int j = 0; j < N; ++j) {
        const int e = j * L + sub;
        if (e < E) dst[e] = l[j];
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
  w.loss_part = reinterpret_cast<float*>(take((size_t)nseq * ((p.E + kChunk - 1) / kChunk) * 4));
  w.done = reinterpret_cast<int32_t*>(take((size_t)nseq * 4));
  w.bytes = off;
  return w;
}

// f(registers a lane, lanes a token, float4 rows, sigmoid) with compile-time arguments.  float4
// rows need E a multiple of 4 and 16-byte aligned arrays.
template <typename F>
int dispatch(int E, bool vec, int score, F f) {
  auto n = [&](auto v, auto s) {
    using std::integral_constant;
    if (E <= 32) return f(integral_constant<int, 4>(), integral_constant<int, 8>(), v, s);
    if (E <= 64) return f(integral_constant<int, 8>(), integral_constant<int, 8>(), v, s);
    if (E <= 128) return f(integral_constant<int, 16>(), integral_constant<int, 8>(), v, s);
    if (E <= 256) return f(integral_constant<int, 16>(), integral_constant<int, 16>(), v, s);
    if (E <= 512) return f(integral_constant<int, 16>(), integral_constant<int, 32>(), v, s);
    return f(integral_constant<int, 32>(), integral_constant<int, 32>(), v, s);
  };
  auto s = [&](auto v) {
    return score == MOE_SCORE_SIGMOID ? n(v, std::true_type()) : n(v, std::false_type());
  };
  return vec ? s(std::true_type()) : s(std::false_type());
}

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

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
  const int r = dispatch(p.E, vec, score, [&](auto n, auto l, auto v, auto s) {
    auto kern = balance_partial_kernel<decltype(n)::value, decltype(l)::value, decltype(v)::value, decltype(s)::value>;
    kern<<<tiles, kThreads, smem, st>>>(
        logits, ids, valid, seg, p.E, p.K, tile, w.part_p, w.part_c, w.part_n, w.done, err);
    return cudaGetLastError() == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
  });
  if (r) return r;
  const dim3 grid((p.E + kChunk - 1) / kChunk, nseq);
  balance_finish_kernel<<<grid, kFinishThreads, 0, st>>>(seg, p.E, p.K, tile, coef, w.part_p, w.part_c, w.part_n,
                                                   w.loss_part, w.done, loss, counts, prob_sum, tokens);
  return cudaGetLastError() == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
}

int launch_balance_backward(const moe_problem& p, const float* logits, const uint8_t* valid, const int32_t* seq,
                            int nseq, int score, float coef, const int32_t* counts, const int32_t* tokens,
                            const float* dloss, float* dlogits, cudaStream_t st) {
  if (p.T == 0) return MOE_OK;
  const Segments seg{seq, nseq, p.T};
  const int tile = tile_tokens(p.T);
  const int tiles = (p.T + tile - 1) / tile;
  const bool vec = p.E % 4 == 0 && aligned16(logits) && aligned16(dlogits);
  return dispatch(p.E, vec, score, [&](auto n, auto l, auto v, auto s) {
    auto kern = balance_backward_kernel<decltype(n)::value, decltype(l)::value, decltype(v)::value, decltype(s)::value>;
    kern<<<tiles, kThreads, 0, st>>>(
        logits, valid, seg, p.E, p.K, tile, coef, counts, tokens, dloss, dlogits);
    return cudaGetLastError() == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
  });
}

}  // namespace moe
