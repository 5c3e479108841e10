// Load-balance loss of the router, with per-expert counts, and its gradient.
//
// For a segment of n tokens with scores p_t that sum to one, c_e the ids equal to e and
// P_e = sum_t p_te:  loss = coef E / (K n^2) sum_e c_e P_e.  With v_e = coef E / (K n^2) c_e
// and the counts held constant, the gradient of a softmax row is p_j (v_j - sum_i v_i p_i);
// of a normalised sigmoid row that times 1 - sigmoid(l_j).  Adding a constant to v changes
// nothing, so v is taken less its mean: near balance the counts differ by a few percent, and the
// difference v_j - sum_i v_i p_i would otherwise lose those digits.
//
// Both directions read the logits once, a warp per token, a row in registers; they are bound
// by HBM for large batches and by latency for small ones.  The sums over tokens use no float
// atomics: the token range is cut into `ntiles` equal tiles, a tile meets the segments in
// pieces, and the piece of tile i in segment b is row i + b of the partial sums -- distinct for
// every piece, because along the tokens i and b only grow and at least one of them does from
// one piece to the next.  A second kernel adds each segment's rows in tile order.
#include <algorithm>
#include <type_traits>

#include "common.cuh"

namespace moe {
namespace {

constexpr int kWarps = 8;
constexpr int kThreads = 32 * kWarps;
constexpr int kChunk = 32;  // experts of one CTA of the second kernel
constexpr float kLog2e = 1.4426950408889634f;

// Tokens of one tile: about two tiles per SM, at least one token a warp.
constexpr int kMaxTiles = 512;
int tile_tokens(int T) {
  const int tiles = std::min(std::max(2 * device_info().sm_count, 1), kMaxTiles);
  return std::max((T + tiles - 1) / tiles, kWarps);
}

// Rows of partial sums: a bound on the tiles that needs no device, plus the segments.
int64_t piece_rows(int64_t T, int nseq) {
  return std::min<int64_t>((T + kWarps - 1) / kWarps, kMaxTiles) + nseq;
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

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

__device__ __forceinline__ float warp_max(float v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, o));
  return v;
}

// Expert of register j of a lane: VEC: float4 chunks of 128 experts, else single ones of 32.
template <bool VEC>
__device__ __forceinline__ int expert_of(int j, int lane) {
  return VEC ? (j >> 2) * 128 + lane * 4 + (j & 3) : j * 32 + lane;
}

// One token's logits; -inf past the last expert.  N registers cover the experts: N * 32 >= E.
template <int N, bool VEC>
__device__ __forceinline__ void load_row(const float* row, int E, int lane, float (&l)[N]) {
  if constexpr (VEC) {
#pragma unroll
    for (int c = 0; c < N / 4; ++c) {
      const int e = c * 128 + lane * 4;
      float4 v = make_float4(-INFINITY, -INFINITY, -INFINITY, -INFINITY);
      if (e < E) v = __ldg(reinterpret_cast<const float4*>(row + e));
      l[4 * c] = v.x, l[4 * c + 1] = v.y, l[4 * c + 2] = v.z, l[4 * c + 3] = v.w;
    }
  } else {
#pragma unroll
    for (int j = 0; j < N; ++j) {
      const int e = j * 32 + lane;
      l[j] = e < E ? __ldg(row + e) : -INFINITY;
    }
  }
}

// l -> unnormalised scores in place; returns 1 / their sum (0 for a row with nothing in it).
template <int N, bool SIG>
__device__ __forceinline__ float scores(float (&l)[N]) {
  float z = 0.0f;
  if constexpr (SIG) {
#pragma unroll
    for (int j = 0; j < N; ++j) {
      l[j] = 1.0f / (1.0f + exp2f(-l[j] * kLog2e));
      z += l[j];
    }
  } else {
    float m = -INFINITY;
#pragma unroll
    for (int j = 0; j < N; ++j) m = fmaxf(m, l[j]);
    m = warp_max(m);
    const float b = m == -INFINITY ? 0.0f : m * kLog2e;
#pragma unroll
    for (int j = 0; j < N; ++j) {
      l[j] = exp2f(fmaf(l[j], kLog2e, -b));
      z += l[j];
    }
  }
  z = warp_sum(z);
  return z == 0.0f ? 0.0f : 1.0f / z;
}

template <int N, bool VEC, bool SIG>
__global__ void __launch_bounds__(kThreads)
    balance_partial_kernel(const float* __restrict__ logits, const int32_t* __restrict__ ids,
                           const uint8_t* __restrict__ valid, Segments seg, int E, int K, int tile,
                           float* __restrict__ part_p, int32_t* __restrict__ part_c, int32_t* __restrict__ part_n,
                           int32_t* __restrict__ done, int32_t* err) {
  extern __shared__ float smem[];
  float* red = smem;                                             // [kWarps][E]
  int32_t* cnt = reinterpret_cast<int32_t*>(smem + kWarps * E);  // [E]
  __shared__ int ntok;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
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
    for (int u = t + warp; u < end; u += kWarps) {
      if (valid && !__ldg(valid + u)) continue;
      ++mine;
      float l[N];
      load_row<N, VEC>(logits + (size_t)u * E, E, lane, l);
      if (lane < K) {
        const int id = __ldg(ids + (size_t)u * K + lane);
        if (id >= 0 && id < E)
          atomicAdd(&cnt[id], 1);
        else
          flags = MOE_FLAG_BAD_EXPERT;
      }
      const float inv = scores<N, SIG>(l);
#pragma unroll
      for (int j = 0; j < N; ++j) acc[j] = fmaf(l[j], inv, acc[j]);
    }
    if (lane == 0 && mine) atomicAdd(&ntok, mine);
#pragma unroll
    for (int j = 0; j < N; ++j) {
      const int e = expert_of<VEC>(j, lane);
      if (e < E) red[warp * E + e] = acc[j];
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

// One CTA per (segment, kChunk experts): adds the segment's rows, warps strided over them; the
// segment's last CTA adds the chunks' parts of the loss in order.
__global__ void __launch_bounds__(kThreads)
    balance_finish_kernel(Segments seg, int E, int K, int tile, float coef, const float* __restrict__ part_p,
                          const int32_t* __restrict__ part_c, const int32_t* __restrict__ part_n,
                          float* __restrict__ loss_part, int32_t* done, float* __restrict__ loss,
                          int32_t* __restrict__ counts, float* __restrict__ prob_sum, int32_t* __restrict__ tokens) {
  __shared__ float sp[kWarps][kChunk];
  __shared__ int sc[kWarps][kChunk];
  __shared__ int sn[kWarps];
  const int b = blockIdx.y, e = blockIdx.x * kChunk + (threadIdx.x & 31);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int lo = seg.lo(b), hi = seg.hi(b);
  const int i0 = lo / tile, i1 = hi > lo ? (hi - 1) / tile : i0 - 1;
  float p = 0.0f;
  int c = 0, n = 0;
#pragma unroll 4
  for (int i = i0 + warp; i <= i1; i += kWarps) {
    const size_t row = (size_t)i + b;
    if (e < E) {
      p += __ldg(part_p + row * E + e);
      c += __ldg(part_c + row * E + e);
    }
    n += __ldg(part_n + row);
  }
  sp[warp][lane] = p;
  sc[warp][lane] = c;
  if (lane == 0) sn[warp] = n;
  __syncthreads();
  if (warp != 0) return;
  p = 0.0f, c = 0, n = 0;
#pragma unroll
  for (int w = 0; w < kWarps; ++w) {
    p += sp[w][lane];
    c += sc[w][lane];
    n += sn[w];
  }
  if (e < E) {
    counts[(size_t)b * E + e] = c;
    prob_sum[(size_t)b * E + e] = p;
  }
  const float part = warp_sum(e < E ? (float)c * p : 0.0f);
  if (lane != 0) return;
  loss_part[(size_t)b * gridDim.x + blockIdx.x] = part;
  __threadfence();
  if (atomicAdd(done + b, 1) != (int)gridDim.x - 1) return;
  __threadfence();
  float s = 0.0f;
  for (int i = 0; i < (int)gridDim.x; ++i) s += __ldcg(loss_part + (size_t)b * gridDim.x + i);
  const float fn = (float)max(n, 1);
  loss[b] = coef * (float)E / ((float)K * fn * fn) * s;
  tokens[b] = n;
}

template <int N, bool VEC, bool SIG>
__global__ void __launch_bounds__(kThreads)
    balance_backward_kernel(const float* __restrict__ logits, const uint8_t* __restrict__ valid, Segments seg, int E,
                            int K, int tile, float coef, const int32_t* __restrict__ counts,
                            const int32_t* __restrict__ tokens, const float* __restrict__ dloss,
                            float* __restrict__ dlogits) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int t0 = blockIdx.x * tile, t1 = min(seg.T, t0 + tile);
  float v[N];
  int lo = 0, hi = 0;  // the segment that v belongs to
  for (int t = t0 + warp; t < t1; t += kWarps) {
    float l[N];
    bool live = !valid || __ldg(valid + t);
    if (live && (t < lo || t >= hi)) {
      const int b = seg.find(t);
      lo = seg.lo(b), hi = seg.hi(b);
      live = t >= lo && t < hi;
      if (live) {
        float sum = 0.0f;
#pragma unroll
        for (int j = 0; j < N; ++j) {
          const int e = expert_of<VEC>(j, lane);
          v[j] = e < E ? (float)__ldg(counts + (size_t)b * E + e) : 0.0f;
          sum += v[j];
        }
        const float mean = warp_sum(sum) / (float)E;
        const float fn = (float)max(__ldg(tokens + b), 1);
        const float scale = coef * (float)E / ((float)K * fn * fn) * __ldg(dloss + b);
#pragma unroll
        for (int j = 0; j < N; ++j) v[j] = (v[j] - mean) * scale;
      } else {
        lo = hi = 0;
      }
    }
    if (live) {
      load_row<N, VEC>(logits + (size_t)t * E, E, lane, l);
      float a[N];
      const float inv = scores<N, SIG>(l);
      float dot = 0.0f;
#pragma unroll
      for (int j = 0; j < N; ++j) {
        a[j] = l[j] * inv;
        dot = fmaf(a[j], v[j], dot);
      }
      dot = warp_sum(dot);
#pragma unroll
      for (int j = 0; j < N; ++j) l[j] = SIG ? a[j] * (v[j] - dot) * (1.0f - l[j]) : a[j] * (v[j] - dot);
    } else {
#pragma unroll
      for (int j = 0; j < N; ++j) l[j] = 0.0f;
    }
    float* dst = dlogits + (size_t)t * E;
    if constexpr (VEC) {
#pragma unroll
      for (int c = 0; c < N / 4; ++c) {
        const int e = c * 128 + lane * 4;
        if (e < E)
          *reinterpret_cast<float4*>(dst + e) = make_float4(l[4 * c], l[4 * c + 1], l[4 * c + 2], l[4 * c + 3]);
      }
    } else {
#pragma unroll
      for (int j = 0; j < N; ++j) {
        const int e = j * 32 + lane;
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

// f(registers a lane, float4 rows, sigmoid) with compile-time arguments.  float4 rows need E a
// multiple of 4 and 16-byte aligned arrays.
template <typename F>
int dispatch(int E, bool vec, int score, F f) {
  auto n = [&](auto v, auto s) {
    if (E <= 128) return f(std::integral_constant<int, 4>(), v, s);
    if (E <= 256) return f(std::integral_constant<int, 8>(), v, s);
    if (E <= 512) return f(std::integral_constant<int, 16>(), v, s);
    return f(std::integral_constant<int, 32>(), v, s);
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
  const int r = dispatch(p.E, vec, score, [&](auto n, auto v, auto s) {
    balance_partial_kernel<decltype(n)::value, decltype(v)::value, decltype(s)::value><<<tiles, kThreads, smem, st>>>(
        logits, ids, valid, seg, p.E, p.K, tile, w.part_p, w.part_c, w.part_n, w.done, err);
    return cudaGetLastError() == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
  });
  if (r) return r;
  const dim3 grid((p.E + kChunk - 1) / kChunk, nseq);
  balance_finish_kernel<<<grid, kThreads, 0, st>>>(seg, p.E, p.K, tile, coef, w.part_p, w.part_c, w.part_n,
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
  return dispatch(p.E, vec, score, [&](auto n, auto v, auto s) {
    balance_backward_kernel<decltype(n)::value, decltype(v)::value, decltype(s)::value><<<tiles, kThreads, 0, st>>>(
        logits, valid, seg, p.E, p.K, tile, coef, counts, tokens, dloss, dlogits);
    return cudaGetLastError() == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
  });
}

}  // namespace moe
