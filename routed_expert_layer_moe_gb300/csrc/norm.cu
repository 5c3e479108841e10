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
// A CTA works on one row at a time, eight columns a vector, so each array is read and written
// once; the statistics are fp32 sums over the CTA.  Backward: CTAs walk the rows with a fixed
// stride and keep the sums over tokens in registers (one for dw_post and dg together: a
// per-channel gate leaves the sum over tokens), write them once, and a second kernel adds the
// CTAs' sums in order.  With a CTA's loads issued at the start
// of each row, memory idled through the row's two or three reductions: 8192 x 4096 bf16 took 67
// and 177 us, against 40 and 60 at the memory's rate.  So the rows to come are fetched into
// shared memory by asynchronous copies, DEPTH rows ahead; a thread copies and reads only its
// own columns, so these copies need no barrier.  Now 42 and 88 us: forward at the memory's rate (6.4 TB/s),
// backward (4.6 TB/s) held by its instructions and the latency of two reductions a row.  Rows that
// are not 16-byte aligned are read when wanted: 2018 x 6290 bf16 takes 75 us forward and 200
// backward, 15 and 23 at the memory's rate.
#include <algorithm>
#include <atomic>
#include <type_traits>

#include "common.cuh"

namespace moe {
namespace {

constexpr int kMaxH = 16384;
constexpr int kMaxT = 1 << 30;  // row numbers a few strides past the last one stay in 32 bits
constexpr int kMaxParts = 512;  // CTAs of the backward pass at most

// Eight consecutive columns as four pairs: the arithmetic is on pairs (fp32x2 instructions), for with
// single ones the backward kernel issued 690 instructions a row and warp and was bound by them.
struct V8 {
  float2 v[4];
};

__device__ __forceinline__ float2 pair(float a) { return make_float2(a, a); }
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) { return __ffma2_rn(a, b, c); }
__device__ __forceinline__ float2 mul2(float2 a, float2 b) { return __fmul2_rn(a, b); }

__device__ __forceinline__ V8 zeros() {
  V8 r;
#pragma unroll
  for (int i = 0; i < 4; ++i) r.v[i] = make_float2(0.0f, 0.0f);
  return r;
}

__device__ __forceinline__ V8 unpack(float4 a, float4 b) {
  V8 r;
  r.v[0] = make_float2(a.x, a.y), r.v[1] = make_float2(a.z, a.w);
  r.v[2] = make_float2(b.x, b.y), r.v[3] = make_float2(b.z, b.w);
  return r;
}

__device__ __forceinline__ V8 unpack(uint4 raw) {  // eight bf16
  const uint32_t w[4] = {raw.x, raw.y, raw.z, raw.w};
  V8 r;
#pragma unroll
  for (int i = 0; i < 4; ++i)
    r.v[i] = make_float2(__uint_as_float(w[i] << 16), __uint_as_float(w[i] & 0xFFFF0000u));
  return r;
}

__device__ __forceinline__ float to_float(float v) { return v; }
__device__ __forceinline__ float to_float(__nv_bfloat16 v) { return __bfloat162float(v); }
__device__ __forceinline__ void from_float(float* d, float v) { *d = v; }
__device__ __forceinline__ void from_float(__nv_bfloat16* d, float v) { *d = __float2bfloat16_rn(v); }

// The eight columns of the thread whose vector begins at c = 8 * (a number whose last five bits are the lane):
// c..c+7 by 16-byte accesses (VEC: H a multiple of 8 and every array 16-byte aligned), or by single ones the lane's
// of the warp's 256 columns with a stride of 32, so that a warp's access is one contiguous piece (4000 x 1111
// fp32 in both directions 71 us, 123 with columns c..c+7; 2018 x 6290 bf16 forward 75 and 103).  Zeros past
// the row's end.
template <bool VEC>
__device__ __forceinline__ int column(int c, int i) {
  return VEC ? c + i : (c & ~255) + ((c >> 3) & 31) + 32 * i;
}
template <bool VEC>
__device__ __forceinline__ bool inside(int c, int H) {  // one of a vector's columns may be in the row
  return (VEC ? c : c & ~255) < H;
}

template <bool VEC, typename T>
__device__ __forceinline__ V8 load8(const T* row, int c, int H) {
  if constexpr (VEC && sizeof(T) == 4) {
    return unpack(*reinterpret_cast<const float4*>(row + c), *reinterpret_cast<const float4*>(row + c + 4));
  } else if constexpr (VEC) {
    return unpack(*reinterpret_cast<const uint4*>(row + c));
  } else {
    V8 r;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int c0 = column<false>(c, 2 * i), c1 = column<false>(c, 2 * i + 1);
      r.v[i] = make_float2(c0 < H ? to_float(row[c0]) : 0.0f, c1 < H ? to_float(row[c1]) : 0.0f);
    }
    return r;
  }
}

// Eight values as two 16-byte parts, `plane` bytes apart, in shared memory.
__device__ __forceinline__ void put8(uint8_t* p, uint32_t plane, const V8& a) {
  *reinterpret_cast<float4*>(p) = make_float4(a.v[0].x, a.v[0].y, a.v[1].x, a.v[1].y);
  *reinterpret_cast<float4*>(p + plane) = make_float4(a.v[2].x, a.v[2].y, a.v[3].x, a.v[3].y);
}

__device__ __forceinline__ V8 get8(const uint8_t* p, uint32_t plane) {
  return unpack(*reinterpret_cast<const float4*>(p), *reinterpret_cast<const float4*>(p + plane));
}

template <bool VEC, typename T>
__device__ __forceinline__ void store8(T* row, int c, int H, const V8& a) {
  if constexpr (VEC && sizeof(T) == 4) {
    *reinterpret_cast<float4*>(row + c) = make_float4(a.v[0].x, a.v[0].y, a.v[1].x, a.v[1].y);
    *reinterpret_cast<float4*>(row + c + 4) = make_float4(a.v[2].x, a.v[2].y, a.v[3].x, a.v[3].y);
  } else if constexpr (VEC) {
    uint4 raw;
    __nv_bfloat162* h = reinterpret_cast<__nv_bfloat162*>(&raw);
#pragma unroll
    for (int i = 0; i < 4; ++i) h[i] = __float22bfloat162_rn(a.v[i]);
    *reinterpret_cast<uint4*>(row + c) = raw;
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int c0 = column<false>(c, 2 * i), c1 = column<false>(c, 2 * i + 1);
      if (c0 < H) from_float(row + c0, a.v[i].x);
      if (c1 < H) from_float(row + c1, a.v[i].y);
    }
  }
}

// Sums of N values over the CTA, in the same order in every thread.  `buf` [N][32] is free for
// the next use after one more barrier: the callers alternate between two.
template <int NT, int N>
__device__ __forceinline__ void cta_sum(float (&v)[N], float* buf) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, nwarps = (NT ? NT : blockDim.x) >> 5;
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
    if (nwarps == 8 || nwarps == 4) {  // a load or two and a tree of adds are shorter than the shuffles
      const float4 a = *reinterpret_cast<const float4*>(buf + i * 32), b = *reinterpret_cast<const float4*>(buf + i * 32 + 4);
      v[i] = (a.x + a.y) + (a.z + a.w);
      if (nwarps == 8) v[i] += (b.x + b.y) + (b.z + b.w);
    } else {
      v[i] = lane < nwarps ? buf[i * 32 + lane] : 0.0f;
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) v[i] += __shfl_xor_sync(0xffffffffu, v[i], o);
    }
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

__device__ __forceinline__ void cp_async16(void* smem_dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(smem_u32(smem_dst)), "l"(src) : "memory");
}

// The rows of N arrays on their way to one CTA: DEPTH rows ahead in shared memory (DEPTH = 0:
// read from global memory when wanted).  Vector j of a thread is columns (j * threads + thread) * 8.
// NT: the CTA's threads, or 0 where only the launch knows.
template <typename T, int V, bool VEC, int DEPTH, int N, int NT>
struct Rows {
  enum { PARTS = 8 * sizeof(T) / 16 };  // 16-byte parts of a vector, in planes of their own
  static constexpr bool kVec = VEC;
  const T* a[N];  // null: the array is not there
  int H;
  uint8_t* smem;

  static __device__ __forceinline__ uint32_t threads() { return NT ? NT : blockDim.x; }
  __device__ __forceinline__ uint8_t* at(int slot, int n, int part, int j) const {
    return smem + (uint32_t)slot * (N * PARTS * V * 16) * threads() + ((n * PARTS * V + part * V + j) * 16) * threads() +
           threadIdx.x * 16;
  }
  // Requests row r (if there is one) into a slot; every call is one group of copies.
  __device__ __forceinline__ void request(int r, int rows, int slot) const {
    if constexpr (DEPTH > 0) {
      if (r < rows) {
        const size_t row = (size_t)r * H;
#pragma unroll
        for (int n = 0; n < N; ++n) {
#pragma unroll
          for (int j = 0; j < V; ++j) {
            const int c = (j * threads() + threadIdx.x) * 8;
            if (a[n] && c < H) {
#pragma unroll
              for (int q = 0; q < PARTS; ++q)
                cp_async16(at(slot, n, q, j), reinterpret_cast<const uint8_t*>(a[n] + row + c) + 16 * q);
            }
          }
        }
      }
      asm volatile("cp.async.commit_group;" ::: "memory");
    }
  }
  // All but the last DEPTH - 1 - BUT requests have arrived (each thread waits for its own).
  template <int BUT>
  __device__ __forceinline__ void wait() const {
    if constexpr (DEPTH > 0) asm volatile("cp.async.wait_group %0;" ::"n"(DEPTH > BUT ? DEPTH - 1 - BUT : 0) : "memory");
  }
  __device__ __forceinline__ V8 get(int n, int r, int slot, int j) const {
    if constexpr (DEPTH == 0) {
      return load8<VEC>(a[n] + (size_t)r * H, (j * threads() + threadIdx.x) * 8, H);
    } else if constexpr (PARTS == 1) {
      return unpack(*reinterpret_cast<const uint4*>(at(slot, n, 0, j)));
    } else {
      return unpack(*reinterpret_cast<const float4*>(at(slot, n, 0, j)),
                    *reinterpret_cast<const float4*>(at(slot, n, 1, j)));
    }
  }
};

// w_post with a per-channel gate folded in.
template <bool VEC, typename T>
__device__ __forceinline__ V8 load_post(const Args<T>& a, int c) {
  V8 w = load8<VEC>(a.w_post, c, a.H);
  if (a.gate_kind == MOE_GATE_CHANNEL) {
    const V8 g = load8<VEC>(a.gate, c, a.H);
#pragma unroll
    for (int i = 0; i < 4; ++i) w.v[i] = mul2(w.v[i], g.v[i]);
  }
  return w;
}

// This thread's part of the sum of squares of array n in row r.
template <int V, typename R>
__device__ __forceinline__ float sum_squares(const R& in, int n, int r, int slot) {
  float2 s = pair(0.0f);
#pragma unroll
  for (int j = 0; j < V; ++j) {
    if (inside<R::kVec>((int)(j * in.threads() + threadIdx.x) * 8, in.H)) {
      const V8 b = in.get(n, r, slot, j);
#pragma unroll
      for (int i = 0; i < 4; ++i) s = fma2(b.v[i], b.v[i], s);
    }
  }
  return s.x + s.y;
}

// The sum over the block's row is needed before y, the sum over y after it.  The first is taken one
// row ahead, together with the second one of the row before: one reduction a row, not two.
template <typename T, int V, bool VEC, int DEPTH, int MAXT, int MINB, int NT>
__global__ void __launch_bounds__(MAXT, MINB) block_norm_kernel(const Args<T> a) {
  extern __shared__ __align__(16) uint8_t smem[];
  __shared__ __align__(16) float buf[2][64];
  const int H = a.H, nt = NT ? NT : blockDim.x;
  const float invH = 1.0f / (float)H;
  const Rows<T, V, VEC, DEPTH, 2, NT> in{{a.x, a.block}, H, smem};
#pragma unroll
  for (int d = 0; d < DEPTH; ++d) in.request(blockIdx.x + d * gridDim.x, a.rows, d);
  in.template wait<0>();
  float sb = 0.0f;  // sum of squares of the block's row
  if (a.block) {
    float v[1] = {sum_squares<V>(in, 1, blockIdx.x, 0)};
    cta_sum<NT>(v, buf[1]);
    sb = v[0];
  }
  int slot = 0, parity = 0;
  for (int r = blockIdx.x; r < a.rows; r += gridDim.x) {
    const size_t at = (size_t)r * H;
    const int next = r + gridDim.x, next_slot = DEPTH > 0 && slot + 1 < DEPTH ? slot + 1 : 0;
    float g = a.rs * rsqrtf(sb * invH + a.eps);
    if (a.gate_kind == MOE_GATE_TOKEN) g *= to_float(a.gate[r]);
    const float2 f = pair(g);
    V8 y[V];
    float2 s = pair(0.0f);
#pragma unroll
    for (int j = 0; j < V; ++j) {
      const int c = (j * nt + threadIdx.x) * 8;
      if (inside<VEC>(c, H)) {
        y[j] = in.get(0, r, slot, j);
        if (a.block) {
          const V8 b = in.get(1, r, slot, j), w = load_post<VEC>(a, c);
#pragma unroll
          for (int i = 0; i < 4; ++i) y[j].v[i] = fma2(f, mul2(w.v[i], b.v[i]), y[j].v[i]);
        }
        if (a.y) store8<VEC>(a.y + at, c, H, y[j]);
#pragma unroll
        for (int i = 0; i < 4; ++i) s = fma2(y[j].v[i], y[j].v[i], s);  // zeros past the row's end
      }
    }
    in.request(r + DEPTH * gridDim.x, a.rows, slot);
    in.template wait<0>();
    float v[2] = {s.x + s.y, 0.0f};
    if (a.block && next < a.rows) v[1] = sum_squares<V>(in, 1, next, next_slot);
    cta_sum<NT>(v, buf[parity]);
    sb = v[1];
    if (a.xn) {
      const float2 ry = pair(rsqrtf(v[0] * invH + a.eps));
#pragma unroll
      for (int j = 0; j < V; ++j) {
        const int c = (j * nt + threadIdx.x) * 8;
        if (inside<VEC>(c, H)) {
          V8 w = load8<VEC>(a.w_pre, c, H);
#pragma unroll
          for (int i = 0; i < 4; ++i) w.v[i] = mul2(w.v[i], mul2(y[j].v[i], ry));
          store8<VEC>(a.xn + at, c, H, w);
        }
      }
    }
    slot = next_slot;
    parity ^= 1;  // this row's buffer is written again after the next row's barrier
  }
}

// The reductions of a row: y^2 with q y, then the sum behind dblock with the next row's block^2.
template <typename T, int V, bool VEC, int DEPTH, int MAXT, int MINB, int NT>
__global__ void __launch_bounds__(MAXT, MINB) block_norm_backward_kernel(const Args<T> a) {
  extern __shared__ __align__(16) uint8_t smem[];
  __shared__ __align__(16) float buf[2][64];
  enum { X, B, DY, DXN };
  grid_dependents_launch();  // the second kernel's CTAs may wait on the SMs
  const int H = a.H, nt = NT ? NT : blockDim.x;
  const float invH = 1.0f / (float)H;
  const Rows<T, V, VEC, DEPTH, 4, NT> in{{a.x, a.block, a.dy, a.dxn}, H, smem};
  // Both weights in fp32, a channel's gate folded in, in this thread's own part of shared memory behind
  // the rows (when rows are fetched ahead): each is read twice a row, and loaded and unpacked from
  // global memory they took 33 of 163 us.
  uint8_t* const wmem = in.at(DEPTH, 0, 0, 0);
  const uint32_t plane = nt * 16u;
  if constexpr (DEPTH > 0) {
#pragma unroll
    for (int j = 0; j < V; ++j) {
      const int c = (j * nt + threadIdx.x) * 8;
      if (inside<VEC>(c, H)) {
        if (a.block) put8(wmem + 2 * j * plane, plane, load_post<VEC>(a, c));
        if (a.dxn) put8(wmem + (2 * V + 2 * j) * plane, plane, load8<VEC>(a.w_pre, c, H));
      }
    }
  }
  auto post_weight = [&](int j, int c) {
    if constexpr (DEPTH > 0) return get8(wmem + 2 * j * plane, plane);
    return load_post<VEC>(a, c);
  };
  auto pre_weight = [&](int j, int c) {
    if constexpr (DEPTH > 0) return get8(wmem + (2 * V + 2 * j) * plane, plane);
    return load8<VEC>(a.w_pre, c, H);
  };
  V8 acc_post[V], acc_pre[V];
#pragma unroll
  for (int j = 0; j < V; ++j) acc_post[j] = acc_pre[j] = zeros();
#pragma unroll
  for (int d = 0; d < DEPTH; ++d) in.request(blockIdx.x + d * gridDim.x, a.rows, d);
  in.template wait<0>();
  float sb = 0.0f;  // sum of squares of the block's row
  if (a.block) {
    float v[1] = {sum_squares<V>(in, B, blockIdx.x, 0)};
    cta_sum<NT>(v, buf[1]);
    sb = v[0];
    if (!a.dxn) __syncthreads();
  }
  int slot = 0;
  for (int r = blockIdx.x; r < a.rows; r += gridDim.x) {
    const size_t at = (size_t)r * H;
    const int next = r + gridDim.x, next_slot = DEPTH > 0 && slot + 1 < DEPTH ? slot + 1 : 0;
    const float gt = a.gate_kind == MOE_GATE_TOKEN ? to_float(a.gate[r]) : 1.0f;
    const float rb = rsqrtf(sb * invH + a.eps);
    V8 y[V];
    float2 s0 = pair(0.0f), s1 = pair(0.0f);  // sums of y^2 and of q y
#pragma unroll
    for (int j = 0; j < V; ++j) {
      const int c = (j * nt + threadIdx.x) * 8;
      if (inside<VEC>(c, H)) {
        y[j] = in.get(X, r, slot, j);
        if (a.block) {
          const V8 b = in.get(B, r, slot, j), w = post_weight(j, c);
          const float2 f = pair(a.rs * gt * rb);
#pragma unroll
          for (int i = 0; i < 4; ++i) y[j].v[i] = fma2(f, mul2(w.v[i], b.v[i]), y[j].v[i]);
        }
        if (a.dxn) {
          const V8 q = in.get(DXN, r, slot, j), w = pre_weight(j, c);
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            s0 = fma2(y[j].v[i], y[j].v[i], s0);
            s1 = fma2(mul2(q.v[i], w.v[i]), y[j].v[i], s1);
          }
        }
      }
    }
    float ry = 0.0f, m = 0.0f;
    if (a.dxn) {
      float sum[2] = {s0.x + s0.y, s1.x + s1.y};
      cta_sum<NT>(sum, buf[0]);
      ry = rsqrtf(sum[0] * invH + a.eps);
      m = -sum[1] * ry * ry * ry * invH;  // -ry yn mean(q yn) = y m
    }
    float2 u = pair(0.0f);
#pragma unroll
    for (int j = 0; j < V; ++j) {
      const int c = (j * nt + threadIdx.x) * 8;
      if (inside<VEC>(c, H)) {
        V8 d = a.dy ? in.get(DY, r, slot, j) : zeros();
        if (a.dxn) {
          const V8 q = in.get(DXN, r, slot, j), w = pre_weight(j, c);
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            acc_pre[j].v[i] = fma2(mul2(q.v[i], y[j].v[i]), pair(ry), acc_pre[j].v[i]);
            d.v[i] = fma2(pair(m), y[j].v[i], fma2(pair(ry), mul2(q.v[i], w.v[i]), d.v[i]));
          }
        }
        store8<VEC>(a.dx + at, c, H, d);
        if (a.block) {
          const V8 b = in.get(B, r, slot, j), w = post_weight(j, c);
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const float2 db = mul2(d.v[i], b.v[i]);
            acc_post[j].v[i] = fma2(pair(gt * rb), db, acc_post[j].v[i]);
            u = fma2(w.v[i], db, u);
            y[j].v[i] = mul2(d.v[i], w.v[i]);  // y is done with
          }
        }
      }
    }
    if (a.block) {
      in.template wait<1>();
      float sum[2] = {u.x + u.y, 0.0f};
      if (next < a.rows) sum[1] = sum_squares<V>(in, B, next, next_slot);
      cta_sum<NT>(sum, buf[1]);
      sb = sum[1];
      const float dg = a.rs * rb * sum[0];  // sum over the row of rs dx bn w_post
      const float2 f = pair(a.rs * rb * gt), mean = pair(-rb * rb * gt * dg * invH);
#pragma unroll
      for (int j = 0; j < V; ++j) {
        const int c = (j * nt + threadIdx.x) * 8;
        if (inside<VEC>(c, H)) {
          V8 b = in.get(B, r, slot, j);
#pragma unroll
          for (int i = 0; i < 4; ++i) b.v[i] = fma2(mean, b.v[i], mul2(f, y[j].v[i]));
          store8<VEC>(a.dblock + at, c, H, b);
        }
      }
      if (a.dgate && a.gate_kind == MOE_GATE_TOKEN && threadIdx.x == 0) a.dgate[r] = dg;
    }
    in.request(r + DEPTH * gridDim.x, a.rows, slot);
    slot = next_slot;
    if (!a.block) in.template wait<0>();
    if (!a.block || !a.dxn) __syncthreads();  // else a barrier on the other buffer lies between two uses of each
  }
  float* part = a.part + (size_t)blockIdx.x * 2 * H;
#pragma unroll
  for (int j = 0; j < V; ++j) {
    const int c = (j * nt + threadIdx.x) * 8;
    if (inside<VEC>(c, H)) {
      store8<VEC>(part, c, H, acc_post[j]);
      store8<VEC>(part + H, c, H, acc_pre[j]);
    }
  }
}

// The CTAs' sums added in a fixed order: a thread per column and group of CTAs.
constexpr int kReduceGroups = 16;

template <typename T>
__global__ void __launch_bounds__(32 * kReduceGroups)
    block_norm_reduce_kernel(const float* part, int parts, int H, int gate_kind,
                             const T* __restrict__ gate, const T* __restrict__ w_post, float rs,
                             float* __restrict__ dgate, float* __restrict__ dw_post, float* __restrict__ dw_pre) {
  __shared__ float sum[kReduceGroups][32];
  grid_dependency_wait();
  const int lane = threadIdx.x & 31, c = blockIdx.x * 32 + lane, g = threadIdx.x >> 5;
  const bool pre = blockIdx.y != 0;
  float s = 0.0f;
  if (c < H) {
#pragma unroll 8
    for (int i = g; i < parts; i += kReduceGroups) s += __ldcg(part + ((size_t)i * 2 + pre) * H + c);
  }
  sum[g][lane] = s;
  __syncthreads();
  if (g != 0 || c >= H) return;
  s = 0.0f;
#pragma unroll
  for (int i = 0; i < kReduceGroups; ++i) s += sum[i][lane];
  if (pre) {
    if (dw_pre) dw_pre[c] = s;
  } else {
    const bool channel = gate_kind == MOE_GATE_CHANNEL;
    if (dw_post) dw_post[c] = rs * s * (channel ? to_float(gate[c]) : 1.0f);
    if (dgate && channel) dgate[c] = rs * s * to_float(w_post[c]);
  }
}

constexpr int kReserved = 1024;  // shared memory that a CTA's static arrays and the system take

// How rows of H columns are shared out: vectors and threads, CTAs an SM holds, rows fetched ahead.
struct Shape {
  int v, threads, ctas, depth;
  size_t smem;
};

// A thread holds one vector when there are few rows, where a row's latency counts, or few columns; else
// two, and four beyond 8192 columns: the reductions, the addresses and the loop are then shared
// by 16 columns.  `arrays`: how many a row is read from; `weights`: fp32 rows kept in shared memory beside
// those fetched ahead; ctas1, ctas2: CTAs of 512 threads with one vector a thread and of 256 with two
// that an SM's registers hold (what the kernels are compiled for).
Shape shape_of(int H, int esz, bool vec, int arrays, int weights, int ctas1, int ctas2, int rows) {
  Shape s{};
  const int nvec = (H + 7) / 8;
  s.v = nvec > 1024 ? 4 : nvec > 512 || (nvec > 128 && rows > device_info().sm_count) ? 2 : 1;
  s.threads = ((nvec + s.v - 1) / s.v + 31) / 32 * 32;
  if (s.v == 2 && s.threads <= 256) s.threads = s.threads <= 128 ? 128 : 256;  // what addresses are compiled for
  s.ctas = s.v == 1 ? std::min(512 * ctas1 / s.threads, 24) : s.threads <= 256 ? 256 * ctas2 / s.threads : 1;
  const DeviceInfo& di = device_info();
  if (!vec || rows <= di.sm_count * s.ctas) return s;  // a row for each CTA: nothing to fetch ahead
  const size_t cols = (size_t)s.v * s.threads * 8;
  const size_t row = cols * esz * arrays, keep = cols * 4 * weights;
  const size_t room = (size_t)di.max_smem_optin - kReserved;
  for (int c = s.ctas; c >= 1; --c)
    for (int depth = 3; depth >= 2; --depth)
      if (row * depth + keep <= room / c - kReserved) {
        s.ctas = c, s.depth = depth, s.smem = row * depth + keep;
        return s;
      }
  return s;
}

// f(vectors a thread, 16-byte accesses, rows ahead, threads) with compile-time arguments; 512 threads: at most.
template <typename F>
int dispatch(const Shape& s, bool vec, F f) {
  using std::integral_constant;
  auto go = [&](auto v, auto t) {
    if (!vec) return f(v, std::false_type(), integral_constant<int, 0>(), t);
    if (s.depth == 3) return f(v, std::true_type(), integral_constant<int, 3>(), t);
    if (s.depth == 2) return f(v, std::true_type(), integral_constant<int, 2>(), t);
    return f(v, std::true_type(), integral_constant<int, 0>(), t);
  };
  if (s.v == 1) return go(integral_constant<int, 1>(), integral_constant<int, 512>());
  if (s.v == 2 && s.threads == 128) return go(integral_constant<int, 2>(), integral_constant<int, 128>());
  if (s.v == 2 && s.threads == 256) return go(integral_constant<int, 2>(), integral_constant<int, 256>());
  if (s.v == 2) return go(integral_constant<int, 2>(), integral_constant<int, 512>());
  return go(integral_constant<int, 4>(), integral_constant<int, 512>());
}

// A kernel's limit on dynamic shared memory is raised once per device, to all that a call may ask for: a call that set it
// to its own need could do so between another host thread's setting and launch.
template <auto kern>
bool raise_limit() {
  static std::atomic<bool> raised[64];
  int dev = 0;
  cudaGetDevice(&dev);
  const bool keep = dev >= 0 && dev < 64;
  if (keep && raised[dev].load(std::memory_order_acquire)) return true;
  if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, device_info().max_smem_optin - kReserved) !=
      cudaSuccess)
    return false;
  if (keep) raised[dev].store(true, std::memory_order_release);
  return true;
}

template <auto kern, typename T>
int launch(int grid, const Shape& s, const Args<T>& a, cudaStream_t st) {
  // 48 KB, the static memory counted in, is what a kernel has without asking
  if (s.smem > 40 * 1024 && !raise_limit<kern>()) return MOE_ERR_CUDA;
  kern<<<grid, s.threads, s.smem, st>>>(a);
  return cudaGetLastError() == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
}

constexpr int kForward1 = 3, kForward2 = 5, kBackward1 = 2, kBackward2 = 2;  // CTAs an SM holds, see shape_of

template <typename T>
int forward(Args<T> a, cudaStream_t st) {
  const bool vec = a.H % 8 == 0 && aligned16(a.x) && aligned16(a.block) && aligned16(a.w_post) &&
                   aligned16(a.w_pre) && aligned16(a.y) && aligned16(a.xn) &&
                   (a.gate_kind != MOE_GATE_CHANNEL || aligned16(a.gate));
  const Shape s = shape_of(a.H, (int)sizeof(T), vec, 2, 0, kForward1, kForward2, a.rows);
  const int grid = s.depth ? std::min(a.rows, s.ctas * device_info().sm_count) : a.rows;
  return dispatch(s, vec, [&](auto v, auto w, auto d, auto t) {
    constexpr int V = decltype(v)::value, MAXT = decltype(t)::value;
    constexpr int MINB = V == 1 ? kForward1 : MAXT <= 256 ? kForward2 * 256 / MAXT : 1;
    return launch<block_norm_kernel<T, V, decltype(w)::value, decltype(d)::value, MAXT, MINB, MAXT <= 256 ? MAXT : 0>>(
        grid, s, a, st);
  });
}

template <typename T>
int backward(Args<T> a, float* dw_post, float* dw_pre, cudaStream_t st) {
  const bool vec = a.H % 8 == 0 && aligned16(a.x) && aligned16(a.block) && aligned16(a.w_post) &&
                   aligned16(a.w_pre) && aligned16(a.dy) && aligned16(a.dxn) && aligned16(a.dx) &&
                   aligned16(a.dblock) && (a.gate_kind != MOE_GATE_CHANNEL || aligned16(a.gate));
  const Shape s = shape_of(a.H, (int)sizeof(T), vec, 4, 2, kBackward1, kBackward2, a.rows);
  const int parts = std::min({a.rows, kMaxParts, s.ctas * device_info().sm_count});
  const int r = dispatch(s, vec, [&](auto v, auto w, auto d, auto t) {
    constexpr int V = decltype(v)::value, MAXT = decltype(t)::value;
    constexpr int MINB = V == 1 ? kBackward1 : MAXT <= 256 ? kBackward2 * 256 / MAXT : 1;
    return launch<
        block_norm_backward_kernel<T, V, decltype(w)::value, decltype(d)::value, MAXT, MINB, MAXT <= 256 ? MAXT : 0>>(
        parts, s, a, st);
  });
  if (r) return r;
  const dim3 grid((a.H + 31) / 32, 2);
  cudaLaunchAttribute attr = overlap_attribute();
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(32 * kReduceGroups);
  cfg.stream = st;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, block_norm_reduce_kernel<T>, (const float*)a.part, parts, a.H, a.gate_kind, a.gate,
                            a.w_post, a.rs, a.block ? a.dgate : (float*)nullptr, a.block ? dw_post : (float*)nullptr,
                            a.w_pre ? dw_pre : (float*)nullptr) == cudaSuccess
             ? MOE_OK
             : MOE_ERR_CUDA;
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
  if (T < 0 || T > kMaxT || H < 1 || H > kMaxH) return 0;
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
