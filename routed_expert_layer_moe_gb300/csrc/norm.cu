// The norms around the layer with the gate and the residual, and their gradient.
//
//   y = x + rs g (b rb w_post),  rb = 1 / sqrt(mean b^2 + eps)
//   xn = y ry w_pre,             ry = 1 / sqrt(mean y^2 + eps)
//
// Gradient, with bn = b rb, yn = y ry, q = dxn w_pre:
//   dx  = dy + ry (q - yn mean(q yn))
//   db  = rb (q2 - bn mean(q2 bn)),  q2 = rs g dx w_post
//   dw_post = rs sum_t g dx bn,  dw_pre = sum_t dxn yn
//   dg  = rs w_post sum_t dx bn (a gate per channel),  rs sum_h dx w_post bn (a gate per token)
//
// A CTA holds one row in registers, eight columns a vector, so each array is read and written
// once; the statistics are fp32 sums over the CTA.  Forward: a CTA per row.  Backward: CTAs
// walk the rows with a fixed stride and keep the sums over tokens in registers (one for
// dw_post and dg together: a per-channel gate leaves the sum over tokens), write them once, and a
// second kernel adds the CTAs' sums in order.
#include <algorithm>
#include <type_traits>

#include "common.cuh"

namespace moe {
namespace {

constexpr int kMaxH = 16384;
constexpr int kMaxThreads = 512;
constexpr int kMaxParts = 512;  // CTAs of the backward pass at most

// Eight consecutive columns c..c+7 of a row: 16-byte accesses (VEC: H a multiple of 8 and every
// array 16-byte aligned) or single ones within the row; zeros past its end.
template <bool VEC>
__device__ __forceinline__ void load8(const float* row, int c, int H, float (&v)[8]) {
  if constexpr (VEC) {
    const float4 a = *reinterpret_cast<const float4*>(row + c);
    const float4 b = *reinterpret_cast<const float4*>(row + c + 4);
    v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w, v[4] = b.x, v[5] = b.y, v[6] = b.z, v[7] = b.w;
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = c + i < H ? row[c + i] : 0.0f;
  }
}

template <bool VEC>
__device__ __forceinline__ void load8(const __nv_bfloat16* row, int c, int H, float (&v)[8]) {
  if constexpr (VEC) {
    const uint4 raw = *reinterpret_cast<const uint4*>(row + c);
    const __nv_bfloat162* h = reinterpret_cast<const __nv_bfloat162*>(&raw);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 f = __bfloat1622float2(h[i]);
      v[2 * i] = f.x;
      v[2 * i + 1] = f.y;
    }
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = c + i < H ? __bfloat162float(row[c + i]) : 0.0f;
  }
}

template <bool VEC>
__device__ __forceinline__ void store8(float* row, int c, int H, const float (&v)[8]) {
  if constexpr (VEC) {
    *reinterpret_cast<float4*>(row + c) = make_float4(v[0], v[1], v[2], v[3]);
    *reinterpret_cast<float4*>(row + c + 4) = make_float4(v[4], v[5], v[6], v[7]);
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (c + i < H) row[c + i] = v[i];
  }
}

template <bool VEC>
__device__ __forceinline__ void store8(__nv_bfloat16* row, int c, int H, const float (&v)[8]) {
  if constexpr (VEC) {
    uint4 raw;
    __nv_bfloat162* h = reinterpret_cast<__nv_bfloat162*>(&raw);
#pragma unroll
    for (int i = 0; i < 4; ++i) h[i] = __floats2bfloat162_rn(v[2 * i], v[2 * i + 1]);
    *reinterpret_cast<uint4*>(row + c) = raw;
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (c + i < H) row[c + i] = __float2bfloat16_rn(v[i]);
  }
}

__device__ __forceinline__ float to_float(float v) { return v; }
__device__ __forceinline__ float to_float(__nv_bfloat16 v) { return __bfloat162float(v); }

// Sums of N values over the CTA, in the same order in every thread.  `buf` [N][32] is free for
// the next use after one more barrier: the callers alternate between two.
template <int N>
__device__ __forceinline__ void cta_sum(float (&v)[N], float* buf) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, nwarps = blockDim.x >> 5;
#pragma unroll
  for (int i = 0; i < N; ++i) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v[i] += __shfl_xor_sync(0xffffffffu, v[i], o);
  }
  if (nwarps == 1) return;
  if (lane == 0) {
#pragma unroll
    for (int i = 0; i < N; ++i) buf[i * 32 + warp] = v[i];
  }
  __syncthreads();
#pragma unroll
  for (int i = 0; i < N; ++i) {
    v[i] = lane < nwarps ? buf[i * 32 + lane] : 0.0f;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v[i] += __shfl_xor_sync(0xffffffffu, v[i], o);
  }
}

template <typename T>
struct Args {
  const T *x, *block, *gate, *w_post, *w_pre, *dy, *dxn;
  T *y, *xn, *dx, *dblock;
  float* part;  // backward: [CTAs][2][H] sums over tokens
  float* dgate;
  int rows, H, gate_kind;
  float rs, eps;
};

template <typename T, int V, bool VEC>
__global__ void __launch_bounds__(kMaxThreads) block_norm_kernel(const Args<T> a) {
  __shared__ float buf[2][32];
  const int H = a.H, nt = blockDim.x;
  const size_t at = (size_t)blockIdx.x * H;
  float y[V][8];
#pragma unroll
  for (int j = 0; j < V; ++j) {
    const int c = (j * nt + threadIdx.x) * 8;
#pragma unroll
    for (int i = 0; i < 8; ++i) y[j][i] = 0.0f;
    if (c < H) load8<VEC>(a.x + at, c, H, y[j]);
  }
  if (a.block) {
    float b[V][8];
    float s[1] = {0.0f};
#pragma unroll
    for (int j = 0; j < V; ++j) {
      const int c = (j * nt + threadIdx.x) * 8;
      if (c < H) {
        load8<VEC>(a.block + at, c, H, b[j]);
#pragma unroll
        for (int i = 0; i < 8; ++i) s[0] = fmaf(b[j][i], b[j][i], s[0]);
      }
    }
    cta_sum(s, buf[0]);
    float f = a.rs * rsqrtf(s[0] / (float)H + a.eps);
    if (a.gate_kind == MOE_GATE_TOKEN) f *= to_float(a.gate[blockIdx.x]);
#pragma unroll
    for (int j = 0; j < V; ++j) {
      const int c = (j * nt + threadIdx.x) * 8;
      if (c < H) {
        float w[8];
        load8<VEC>(a.w_post, c, H, w);
        if (a.gate_kind == MOE_GATE_CHANNEL) {
          float g[8];
          load8<VEC>(a.gate, c, H, g);
#pragma unroll
          for (int i = 0; i < 8; ++i) w[i] *= g[i];
        }
#pragma unroll
        for (int i = 0; i < 8; ++i) y[j][i] = fmaf(f * w[i], b[j][i], y[j][i]);
      }
    }
  }
  if (a.y) {
#pragma unroll
    for (int j = 0; j < V; ++j) {
      const int c = (j * nt + threadIdx.x) * 8;
      if (c < H) store8<VEC>(a.y + at, c, H, y[j]);
    }
  }
  if (!a.xn) return;
  float s[1] = {0.0f};
#pragma unroll
  for (int j = 0; j < V; ++j) {
#pragma unroll
    for (int i = 0; i < 8; ++i) s[0] = fmaf(y[j][i], y[j][i], s[0]);  // zeros past the row's end
  }
  cta_sum(s, buf[1]);
  const float ry = rsqrtf(s[0] / (float)H + a.eps);
#pragma unroll
  for (int j = 0; j < V; ++j) {
    const int c = (j * nt + threadIdx.x) * 8;
    if (c < H) {
      float w[8];
      load8<VEC>(a.w_pre, c, H, w);
#pragma unroll
      for (int i = 0; i < 8; ++i) w[i] *= y[j][i] * ry;
      store8<VEC>(a.xn + at, c, H, w);
    }
  }
}

template <typename T, int V, bool VEC>
__global__ void __launch_bounds__(kMaxThreads) block_norm_backward_kernel(const Args<T> a) {
  __shared__ float buf[3][64];
  const int H = a.H, nt = blockDim.x;
  const float invH = 1.0f / (float)H;
  float acc_post[V][8], acc_pre[V][8];
#pragma unroll
  for (int j = 0; j < V; ++j) {
#pragma unroll
    for (int i = 0; i < 8; ++i) acc_post[j][i] = acc_pre[j][i] = 0.0f;
  }
  for (int r = blockIdx.x; r < a.rows; r += gridDim.x) {
    const size_t at = (size_t)r * H;
    const float gt = a.gate_kind == MOE_GATE_TOKEN ? to_float(a.gate[r]) : 1.0f;
    float y[V][8], b[V][8], d[V][8], q[V][8];
    float rb = 0.0f;
    float s[2] = {0.0f, 0.0f};
#pragma unroll
    for (int j = 0; j < V; ++j) {
      const int c = (j * nt + threadIdx.x) * 8;
#pragma unroll
      for (int i = 0; i < 8; ++i) y[j][i] = b[j][i] = d[j][i] = q[j][i] = 0.0f;
      if (c < H) {
        load8<VEC>(a.x + at, c, H, y[j]);
        if (a.block) load8<VEC>(a.block + at, c, H, b[j]);
        if (a.dy) load8<VEC>(a.dy + at, c, H, d[j]);
        if (a.dxn) load8<VEC>(a.dxn + at, c, H, q[j]);
      }
#pragma unroll
      for (int i = 0; i < 8; ++i) s[0] = fmaf(b[j][i], b[j][i], s[0]);
    }
    if (a.block) {
      float sb[1] = {s[0]};
      cta_sum(sb, buf[0]);
      rb = rsqrtf(sb[0] * invH + a.eps);
    }
    s[0] = 0.0f;
#pragma unroll
    for (int j = 0; j < V; ++j) {
      const int c = (j * nt + threadIdx.x) * 8;
      if (c < H) {
        if (a.block) {
          float w[8];
          load8<VEC>(a.w_post, c, H, w);
          if (a.gate_kind == MOE_GATE_CHANNEL) {
            float g[8];
            load8<VEC>(a.gate, c, H, g);
#pragma unroll
            for (int i = 0; i < 8; ++i) w[i] *= g[i];
          }
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            b[j][i] *= rb;
            y[j][i] = fmaf(a.rs * gt * w[i], b[j][i], y[j][i]);
          }
        }
        if (a.dxn) {
          float w[8];
          load8<VEC>(a.w_pre, c, H, w);
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            s[0] = fmaf(y[j][i], y[j][i], s[0]);
            s[1] = fmaf(q[j][i] * w[i], y[j][i], s[1]);
          }
        }
      }
    }
    float ry = 0.0f, m = 0.0f;
    if (a.dxn) {
      cta_sum(s, buf[1]);
      ry = rsqrtf(s[0] * invH + a.eps);
      m = s[1] * ry * ry * invH;  // mean(q yn) / y's factor: yn mean(q yn) = y m
    }
    float u[1] = {0.0f};
#pragma unroll
    for (int j = 0; j < V; ++j) {
      const int c = (j * nt + threadIdx.x) * 8;
      if (c < H) {
        if (a.dxn) {
          float w[8];
          load8<VEC>(a.w_pre, c, H, w);
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            acc_pre[j][i] = fmaf(q[j][i], y[j][i] * ry, acc_pre[j][i]);
            d[j][i] = fmaf(ry, fmaf(-y[j][i], m, q[j][i] * w[i]), d[j][i]);
          }
        }
        store8<VEC>(a.dx + at, c, H, d[j]);
        if (a.block) {
          float w[8];
          load8<VEC>(a.w_post, c, H, w);
          if (a.gate_kind == MOE_GATE_CHANNEL) {
            float g[8];
            load8<VEC>(a.gate, c, H, g);
#pragma unroll
            for (int i = 0; i < 8; ++i) w[i] *= g[i];
          }
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            const float db = d[j][i] * b[j][i];
            acc_post[j][i] = fmaf(gt, db, acc_post[j][i]);
            u[0] = fmaf(w[i], db, u[0]);
            d[j][i] *= a.rs * w[i];  // q2 without a token's gate
          }
        }
      }
    }
    if (a.block) {
      cta_sum(u, buf[2]);
      const float mean = a.rs * u[0] * invH, f = rb * gt;
#pragma unroll
      for (int j = 0; j < V; ++j) {
        const int c = (j * nt + threadIdx.x) * 8;
        if (c < H) {
#pragma unroll
          for (int i = 0; i < 8; ++i) d[j][i] = f * fmaf(-b[j][i], mean, d[j][i]);
          store8<VEC>(a.dblock + at, c, H, d[j]);
        }
      }
      if (a.dgate && a.gate_kind == MOE_GATE_TOKEN && threadIdx.x == 0) a.dgate[r] = a.rs * u[0];
    }
    __syncthreads();  // the next row writes the buffers again
  }
  float* part = a.part + (size_t)blockIdx.x * 2 * H;
#pragma unroll
  for (int j = 0; j < V; ++j) {
    const int c = (j * nt + threadIdx.x) * 8;
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (c + i < H) {
        part[c + i] = acc_post[j][i];
        part[H + c + i] = acc_pre[j][i];
      }
  }
}

// The CTAs' sums added in order; a thread per column, four groups of CTAs in flight.
template <typename T>
__global__ void __launch_bounds__(128) block_norm_reduce_kernel(const float* __restrict__ part, int parts, int H,
                                                               int gate_kind, const T* __restrict__ gate,
                                                               const T* __restrict__ w_post, float rs,
                                                               float* __restrict__ dgate,
                                                               float* __restrict__ dw_post,
                                                               float* __restrict__ dw_pre) {
  __shared__ float sum[4][32];
  const int c = blockIdx.x * 32 + (threadIdx.x & 31), g = threadIdx.x >> 5;
  const bool pre = blockIdx.y != 0;
  float s = 0.0f;
  if (c < H) {
#pragma unroll 8
    for (int i = g; i < parts; i += 4) s += __ldg(part + ((size_t)i * 2 + pre) * H + c);
  }
  sum[g][threadIdx.x & 31] = s;
  __syncthreads();
  if (g != 0 || c >= H) return;
  s = (sum[0][threadIdx.x] + sum[1][threadIdx.x]) + (sum[2][threadIdx.x] + sum[3][threadIdx.x]);
  if (pre) {
    if (dw_pre) dw_pre[c] = s;
  } else {
    const bool channel = gate_kind == MOE_GATE_CHANNEL;
    if (dw_post) dw_post[c] = rs * s * (channel ? to_float(gate[c]) : 1.0f);
    if (dgate && channel) dgate[c] = rs * s * to_float(w_post[c]);
  }
}

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

// f(vectors a thread, 16-byte accesses) and the CTA's threads: one vector a thread up to 512
// threads, then two, four.
template <typename F>
int dispatch(int H, bool vec, F f) {
  const int nvec = (H + 7) / 8;
  auto go = [&](auto v) {
    constexpr int V = decltype(v)::value;
    const int threads = (((nvec + V - 1) / V) + 31) / 32 * 32;
    return vec ? f(v, std::true_type(), threads) : f(v, std::false_type(), threads);
  };
  if (nvec <= 512) return go(std::integral_constant<int, 1>());
  if (nvec <= 1024) return go(std::integral_constant<int, 2>());
  return go(std::integral_constant<int, 4>());
}

int parts_of(int T) { return std::min(T, std::min(kMaxParts, std::max(2 * device_info().sm_count, 1))); }

template <typename T>
int forward(Args<T> a, cudaStream_t st) {
  const bool vec = a.H % 8 == 0 && aligned16(a.x) && aligned16(a.block) && aligned16(a.w_post) &&
                   aligned16(a.w_pre) && aligned16(a.y) && aligned16(a.xn) &&
                   (a.gate_kind != MOE_GATE_CHANNEL || aligned16(a.gate));
  return dispatch(a.H, vec, [&](auto v, auto w, int threads) {
    block_norm_kernel<T, decltype(v)::value, decltype(w)::value><<<a.rows, threads, 0, st>>>(a);
    return cudaGetLastError() == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
  });
}

template <typename T>
int backward(Args<T> a, float* dw_post, float* dw_pre, cudaStream_t st) {
  const bool vec = a.H % 8 == 0 && aligned16(a.x) && aligned16(a.block) && aligned16(a.w_post) &&
                   aligned16(a.w_pre) && aligned16(a.dy) && aligned16(a.dxn) && aligned16(a.dx) &&
                   aligned16(a.dblock) && (a.gate_kind != MOE_GATE_CHANNEL || aligned16(a.gate));
  const int parts = parts_of(a.rows);
  if (parts > 0) {
    const int r = dispatch(a.H, vec, [&](auto v, auto w, int threads) {
      block_norm_backward_kernel<T, decltype(v)::value, decltype(w)::value><<<parts, threads, 0, st>>>(a);
      return cudaGetLastError() == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
    });
    if (r) return r;
  }
  const dim3 grid((a.H + 31) / 32, 2);
  block_norm_reduce_kernel<T><<<grid, 128, 0, st>>>(a.part, parts, a.H, a.gate_kind, a.gate, a.w_post, a.rs,
                                                    a.block ? a.dgate : nullptr, a.block ? dw_post : nullptr,
                                                    a.w_pre ? dw_pre : nullptr);
  return cudaGetLastError() == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
}

template <typename T>
Args<T> make_args(const NormArgs& n) {
  Args<T> a{};
  a.x = static_cast<const T*>(n.x);
  a.block = static_cast<const T*>(n.block);
  a.gate = static_cast<const T*>(n.gate);
  a.w_post = static_cast<const T*>(n.w_post);
  a.w_pre = static_cast<const T*>(n.w_pre);
  a.dy = static_cast<const T*>(n.dy);
  a.dxn = static_cast<const T*>(n.dxn);
  a.y = static_cast<T*>(n.y);
  a.xn = static_cast<T*>(n.xn);
  a.dx = static_cast<T*>(n.dx);
  a.dblock = static_cast<T*>(n.dblock);
  a.part = static_cast<float*>(n.ws);
  a.dgate = n.dgate;
  a.rows = n.T;
  a.H = n.H;
  a.gate_kind = n.gate_kind;
  a.rs = n.res_scale;
  a.eps = n.eps;
  return a;
}

}  // namespace

size_t block_norm_workspace_bytes(int T, int H) {
  if (T < 0 || H < 1 || H > kMaxH) return 0;
  return std::max<size_t>((size_t)std::min(T, kMaxParts) * 2 * H * sizeof(float), 256);
}

int launch_block_norm(const NormArgs& n, cudaStream_t st) {
  if (n.T == 0) return MOE_OK;
  return n.dtype == MOE_F32 ? forward(make_args<float>(n), st) : forward(make_args<__nv_bfloat16>(n), st);
}

int launch_block_norm_backward(const NormArgs& n, float* dw_post, float* dw_pre, cudaStream_t st) {
  return n.dtype == MOE_F32 ? backward(make_args<float>(n), dw_post, dw_pre, st)
                            : backward(make_args<__nv_bfloat16>(n), dw_post, dw_pre, st);
}

}  // namespace moe
