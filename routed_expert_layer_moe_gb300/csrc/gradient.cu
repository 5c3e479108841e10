// Gradients of the steps around the expert products: of the combine (step 5) and of the router's weights (step 1).
// The dispatch's gradient is the combine with weight 1 (combine.cu).
//
//   combine   out[t] = sum_k w[t,k] yg[row]  ->  gradient of yg[row] = w[t,k] dout[t], left as the pair of them: the
//             expert products multiply by w in fp32 instead of rounding w dout to bf16;  dw[t,k] = dout[t] . yg[row]
//   softmax   w_k = exp(l_k) / sum_j exp(l_j) over the K chosen  ->  dl_k = w_k (dw_k - sum_j w_j dw_j)
//   sigmoid   s_k = sigmoid(l_k), w_k = scale s_k [/ sum_j s_j]  ->  dl_k = s_k (1 - s_k) ds_k,
//             ds_k = scale dw_k, or scale (dw_k - sum_j r_j dw_j) / sum_j s_j with r_j = s_j / sum s
//
// Sums are fp32 in a fixed order; no atomics.
#include "common.cuh"

namespace moe {
namespace {

constexpr int kWarps = 8;   // records of a token that run at once
constexpr int kAhead = 4;   // 16-byte vectors a lane requests before it uses them

struct RouteArgs {
  const float* logits;
  const int32_t* ids;
  const float *w, *add;
  float* dlogits;  // [E] a token
  int E, K, score, renorm;
  float scale;
};

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) v += __shfl_xor_sync(0xffffffffu, v, off);
  return v;
}

// One token's row of dlogits, by a warp: lane k holds the k-th choice, d its dw (0 where there is none).
__device__ __forceinline__ void route_backward(const RouteArgs& r, int t, int lane, float d) {
  const size_t at = (size_t)t * r.E;
  int id = lane < r.K ? r.ids[(size_t)t * r.K + lane] : -1;
  if (id >= r.E || id < 0) id = -1, d = 0.0f;
  float dl;
  if (r.score == MOE_SCORE_SOFTMAX) {
    const float wk = id >= 0 ? r.w[(size_t)t * r.K + lane] : 0.0f;
    dl = wk * (d - warp_sum(wk * d));
  } else {
    // s and 1 - s from the exponential of -|l|, so that neither is lost where the other is next to 1
    const float l = id >= 0 ? r.logits[at + id] : 0.0f;
    const float e = expf(-fabsf(l)), z = 1.0f / (1.0f + e);
    const float s = id >= 0 ? (l >= 0.0f ? z : e * z) : 0.0f, rest = l >= 0.0f ? e * z : z;
    if (r.renorm) {
      const float sum = warp_sum(s), q = sum > 0.0f ? s / sum : 0.0f;
      dl = r.scale * q * rest * (d - warp_sum(q * d));
    } else {
      dl = r.scale * s * rest * d;
    }
  }
  // An expert that a token names twice gets both parts, in k order, at its first place.
  float total = dl;
  bool first = id >= 0;
  for (int k = 0; k < r.K; ++k) {
    const int other = __shfl_sync(0xffffffffu, id, k);
    const float part = __shfl_sync(0xffffffffu, dl, k);
    if (other != id || k == lane) continue;
    if (k < lane)
      first = false;
    else
      total += part;
  }
  for (int e = lane; e < r.E; e += 32) r.dlogits[at + e] = r.add ? r.add[at + e] : 0.0f;
  __syncwarp();
  if (first) r.dlogits[at + id] += total;
}

// A warp per token.
__global__ void __launch_bounds__(128) route_backward_kernel(const RouteArgs r, const float* __restrict__ dw, int T) {
  const int t = blockIdx.x * 4 + (threadIdx.x >> 5), lane = threadIdx.x & 31;
  if (t < T) route_backward(r, t, lane, lane < r.K ? dw[(size_t)t * r.K + lane] : 0.0f);
}

// A CTA per token, a warp per record: it reads the token's dout (the other records' warps find it in L1) and the
// record's yg, writes its dyg and sums its dot product with shuffles alone.  yg and dyg may be the same buffer, so
// yg does not go through the read-only path.  ROUTE: the token's dlogits follow from its dw in the same launch.
template <bool ROUTE>
__global__ void __launch_bounds__(32 * kWarps)
    combine_backward_kernel(const __nv_bfloat16* __restrict__ dout, const __nv_bfloat16* yg,
                            const int32_t* __restrict__ row_of, const float* __restrict__ w, __nv_bfloat16* dyg,
                            float* __restrict__ wg, float* __restrict__ dw, int nvec, int K, int KS, long long rows,
                            const RouteArgs r) {
  __shared__ float sums[32];
  grid_dependents_launch();  // the products' CTAs set up meanwhile
  const int t = blockIdx.x, lane = threadIdx.x & 31;
  const uint4* src = reinterpret_cast<const uint4*>(dout) + (size_t)t * nvec;
  for (int k = threadIdx.x >> 5; k < KS; k += blockDim.x >> 5) {
    const int row = row_of[(size_t)t * KS + k];
    float sum = 0.0f;
    if (row >= 0 && row < rows) {  // a record that was not placed has no part in the output
      if (lane == 0) wg[row] = k < K ? w[(size_t)t * K + k] : 1.0f;
      const bool dot = dw && k < K;
      const uint4* y = reinterpret_cast<const uint4*>(yg) + (size_t)row * nvec;
      uint4* dst = reinterpret_cast<uint4*>(dyg) + (size_t)row * nvec;
      for (int v0 = lane; v0 < nvec; v0 += 32 * kAhead) {
        uint4 a[kAhead], b[kAhead];
#pragma unroll
        for (int j = 0; j < kAhead; ++j)
          if (v0 + 32 * j < nvec) {
            a[j] = __ldg(src + v0 + 32 * j);
            b[j] = dot ? y[v0 + 32 * j] : make_uint4(0u, 0u, 0u, 0u);
          }
#pragma unroll
        for (int j = 0; j < kAhead; ++j)
          if (v0 + 32 * j < nvec) {
            const __nv_bfloat162* ha = reinterpret_cast<const __nv_bfloat162*>(&a[j]);
            const __nv_bfloat162* hb = reinterpret_cast<const __nv_bfloat162*>(&b[j]);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const float2 fa = __bfloat1622float2(ha[i]), fb = __bfloat1622float2(hb[i]);
              sum = fmaf(fa.x, fb.x, sum);
              sum = fmaf(fa.y, fb.y, sum);
            }
            dst[v0 + 32 * j] = a[j];
          }
      }
      sum = warp_sum(sum);
    }
    if (dw && k < K && lane == 0) dw[(size_t)t * K + k] = sum;
    if (ROUTE && k < K && lane == 0) sums[k] = sum;
  }
  if constexpr (ROUTE) {
    __syncthreads();
    if (threadIdx.x < 32) route_backward(r, t, lane, lane < K ? sums[lane] : 0.0f);
  }
}

}  // namespace

int launch_combine_backward(const moe_problem& p, const void* dout, const void* yg, const int32_t* row_of,
                            const float* w, void* dyg, float* wg, float* dw, cudaStream_t st, const RouteBackward* route) {
  if (p.T == 0) return MOE_OK;
  const int KS = p.K + p.has_shared;
  RouteArgs r{};
  if (route)
    r = {route->logits, route->ids, w, route->add, route->dlogits, p.E, p.K, route->score, route->renorm, route->scale};
  auto kern = route ? combine_backward_kernel<true> : combine_backward_kernel<false>;
  kern<<<p.T, 32 * std::min(KS, kWarps), 0, st>>>(static_cast<const __nv_bfloat16*>(dout),
                                                  static_cast<const __nv_bfloat16*>(yg), row_of, w,
                                                  static_cast<__nv_bfloat16*>(dyg), wg, dw, p.H / 8, p.K, KS,
                                                  grouped_rows(p), r);
  return cudaGetLastError() == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
}

int launch_route_backward(const moe_problem& p, const RouteBackward& route, const float* w, const float* dw,
                          cudaStream_t st) {
  if (p.T == 0) return MOE_OK;
  const RouteArgs r{route.logits, route.ids, w, route.add, route.dlogits, p.E, p.K, route.score, route.renorm, route.scale};
  route_backward_kernel<<<(p.T + 3) / 4, 128, 0, st>>>(r, dw, p.T);
  return cudaGetLastError() == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
}

}  // namespace moe
