// Activation checkpoints in 8 bits: rows of E4M3 codes with one fp32 scale per 128 values, and back.
//
//   s = max |x| * fp32(1 / 448) over the group,  code = E4M3(x / s),  value = code * s
//
// The code is that of the exact quotient.  x * (1 / s) is within two units in the last place of it.  Where two codes
// meet, the low 19 mantissa bits are zero; so the nearest multiple m of eight units, moved by four units to the side of
// x - m s (exact in one fused multiply-add), lies between the same two codes as the quotient.  Eight instructions a value;
// with an IEEE division and its remainder in 64 bits where a middle is near, which bf16 values hit often, 8192 x 4096
// took 99 us to quantise, with this step taken only there 31.
#include "fp8.cuh"

namespace moe {
namespace {

constexpr int kThreads = 256;

// The same from the quotient and its remainder in 64 bits (24 x 24 bits: exact), for scales next to the ends of fp32.
__device__ __noinline__ float quotient_by_division(float x, float s) {
  const float q = __fdiv_rn(x, s);
  const uint32_t b = __float_as_uint(q);
  if ((b & 0x7FFFFu) || (b & 0x7FFFFFFFu) < 0x3A800000u) return q;  // no middle of two codes (the least is 2^-10)
  const double r = (double)x - (double)q * (double)s;
  if (r == 0.0) return q;
  return __uint_as_float((r > 0.0) == (q > 0.0f) ? b + 1u : b - 1u);  // one step to the side of the exact quotient
}

// A number with the exact quotient's E4M3 code.  inv = 1 / s, or 0 for a scale that is not within [2^-80, 2^100]: in
// between, the remainder of a quotient that has a code other than 0 loses nothing.
__device__ __forceinline__ float quotient(float x, float s, float inv) {
  const uint32_t m = (__float_as_uint(x * inv) + 4u) & ~7u;
  const float r = fmaf(-__uint_as_float(m), s, x);
  const int side = (int)(__float_as_uint(r) ^ m) >= 0 ? 4 : -4;  // the same sign as m: further from zero
  return __uint_as_float(r == 0.0f ? m : m + side);
}

__device__ __forceinline__ float inverse(float s) {
  return s >= 0x1p-80f && s <= 0x1p100f ? __frcp_rn(s) : 0.0f;
}

// Sixteen consecutive values of a 16-byte aligned array, and their largest magnitude (a NaN if there is one).
__device__ __forceinline__ float load16(const float* x, float (&v)[16]) {
  float4 a[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) a[i] = __ldg(reinterpret_cast<const float4*>(x) + i);
  float amax = 0.0f;
#pragma unroll
  for (int i = 0; i < 4; ++i) v[4 * i] = a[i].x, v[4 * i + 1] = a[i].y, v[4 * i + 2] = a[i].z, v[4 * i + 3] = a[i].w;
#pragma unroll
  for (int i = 0; i < 16; ++i) amax = fp8_amax(amax, v[i]);
  return amax;
}

__device__ __forceinline__ float load16(const __nv_bfloat16* x, float (&v)[16]) {
  const uint4 raw[2] = {__ldg(reinterpret_cast<const uint4*>(x)), __ldg(reinterpret_cast<const uint4*>(x) + 1)};
  const __nv_bfloat162* h = reinterpret_cast<const __nv_bfloat162*>(raw);
  __nv_bfloat162 m = __habs2(h[0]);
#pragma unroll
  for (int i = 1; i < 8; ++i) m = __hmax2_nan(m, __habs2(h[i]));
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const float2 f = __bfloat1622float2(h[i]);
    v[2 * i] = f.x, v[2 * i + 1] = f.y;
  }
  const float2 f = __bfloat1622float2(m);
  return fp8_amax(f.x, f.y);
}

template <typename T>
__device__ __forceinline__ T to_type(float v) {
  if constexpr (sizeof(T) == 4)
    return v;
  else
    return __float2bfloat16_rn(v);
}

// Rows of whole groups, 16-byte aligned: the groups of all rows lie one after the other.  Sixteen values a thread, eight
// threads a group; n16 is a multiple of 8, so a group's threads are all in range or all out of it.
template <typename T>
__global__ void __launch_bounds__(kThreads) quantize_kernel(const T* __restrict__ x, long long n16,
                                                            uint8_t* __restrict__ codes, float* __restrict__ scales) {
  const long long i = (long long)blockIdx.x * kThreads + threadIdx.x;
  float v[16], amax = 0.0f;
  if (i < n16) amax = load16(x + 16 * i, v);
#pragma unroll
  for (int off = 4; off > 0; off >>= 1) amax = fp8_amax(amax, __shfl_xor_sync(0xffffffffu, amax, off));
  if (i >= n16) return;
  const float s = fp8_scale(amax), inv = inverse(s);
  uint32_t c[4] = {0u, 0u, 0u, 0u};
  if (s == s) {
    if (inv != 0.0f) {
#pragma unroll
      for (int j = 0; j < 16; ++j) v[j] = quotient(v[j], s, inv);
    } else {
#pragma unroll 1
      for (int j = 0; j < 16; ++j) v[j] = quotient_by_division(v[j], s);
    }
#pragma unroll
    for (int j = 0; j < 4; ++j) c[j] = fp8_pair(v[4 * j], v[4 * j + 1]) | fp8_pair(v[4 * j + 2], v[4 * j + 3]) << 16;
  }
  reinterpret_cast<uint4*>(codes)[i] = make_uint4(c[0], c[1], c[2], c[3]);
  if ((i & 7) == 0) scales[i >> 3] = s;
}

template <typename T>
__global__ void __launch_bounds__(kThreads) dequantize_kernel(const uint8_t* __restrict__ codes,
                                                              const float* __restrict__ scales, long long n16,
                                                              T* __restrict__ out, bool wide) {
  const long long i = (long long)blockIdx.x * kThreads + threadIdx.x;
  if (i >= n16) return;
  const uint4 raw = __ldg(reinterpret_cast<const uint4*>(codes) + i);
  const uint32_t c[4] = {raw.x, raw.y, raw.z, raw.w};
  const float s = __ldg(scales + (i >> 3));
  float v[16];
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    const float2 f = fp8_unpair(c[j >> 1] >> (16 * (j & 1)));
    v[2 * j] = f.x * s, v[2 * j + 1] = f.y * s;
  }
  constexpr int N = sizeof(T);  // 16-byte pieces
  uint4 o[N];
  if constexpr (sizeof(T) == 4) {
#pragma unroll
    for (int j = 0; j < 16; ++j) reinterpret_cast<float*>(o)[j] = v[j];
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j) reinterpret_cast<__nv_bfloat162*>(o)[j] = __floats2bfloat162_rn(v[2 * j], v[2 * j + 1]);
  }
  uint4* dst = reinterpret_cast<uint4*>(out) + N * i;
#pragma unroll
  for (int j = 0; j < N; j += 2) {
    if (wide) {
      st_global_v8(dst + j, o[j], o[j + 1]);
    } else {
      dst[j] = o[j];
      dst[j + 1] = o[j + 1];
    }
  }
}

// Rows of any length: kLanes lanes a group, kEach values a lane, V of them side by side (1, 2 or 4, as the rows' length and
// the arrays' alignment allow).  Bound by its instructions: 4001 x 6290 fp32 took 54 us with a warp a group, 64-bit
// divisions and single values, 44 with pairs and 32-bit divisions.
constexpr int kLanes = 16, kEach = FP8_GROUP / kLanes;
template <int V>
__device__ __forceinline__ int at_lane(int lane, int j) {  // value j of a lane in its group
  return (lane + kLanes * (j / V)) * V + j % V;
}

template <int BYTES>
struct Piece;
template <>
struct Piece<1> { using type = uint8_t; };
template <>
struct Piece<2> { using type = uint16_t; };
template <>
struct Piece<4> { using type = uint32_t; };
template <>
struct Piece<8> { using type = uint2; };
template <>
struct Piece<16> { using type = uint4; };

template <typename T, int V>
__global__ void __launch_bounds__(kThreads) quantize_any_kernel(const T* __restrict__ x, uint32_t groups,
                                                                uint32_t per_row, long long cols,
                                                                uint8_t* __restrict__ codes, float* __restrict__ scales) {
  const uint32_t i = blockIdx.x * (kThreads / kLanes) + threadIdx.x / kLanes;
  const uint32_t gr = min(i, groups - 1);  // lanes behind the last group do its work again: shuffles are warp-wide
  const int lane = threadIdx.x % kLanes;
  const uint32_t row = gr / per_row;
  const long long col = (long long)(gr - row * per_row) * FP8_GROUP, at = row * cols + col;
  const int n = (int)min((long long)FP8_GROUP, cols - col);
  using In = typename Piece<V * sizeof(T)>::type;
  using Out = typename Piece<V>::type;
  float v[kEach], amax = 0.0f;
  In raw[kEach / V];
#pragma unroll
  for (int j = 0; j < kEach; j += V)
    if (at_lane<V>(lane, j) < n) raw[j / V] = __ldg(reinterpret_cast<const In*>(x + at + at_lane<V>(lane, j)));
#pragma unroll
  for (int j = 0; j < kEach; ++j) {
    v[j] = at_lane<V>(lane, j) < n ? (float)reinterpret_cast<const T*>(&raw[j / V])[j % V] : 0.0f;
    amax = fp8_amax(amax, v[j]);
  }
#pragma unroll
  for (int off = kLanes / 2; off > 0; off >>= 1) amax = fp8_amax(amax, __shfl_xor_sync(0xffffffffu, amax, off));
  const float s = fp8_scale(amax), inv = inverse(s);
  uint32_t c[kEach / 4] = {};
  if (s == s) {
    if (inv != 0.0f) {
#pragma unroll
      for (int j = 0; j < kEach; ++j) v[j] = quotient(v[j], s, inv);
    } else {
#pragma unroll 1
      for (int j = 0; j < kEach; ++j) v[j] = quotient_by_division(v[j], s);
    }
#pragma unroll
    for (int j = 0; j < kEach / 4; ++j) c[j] = fp8_pair(v[4 * j], v[4 * j + 1]) | fp8_pair(v[4 * j + 2], v[4 * j + 3]) << 16;
  }
#pragma unroll
  for (int j = 0; j < kEach; j += V)
    if (at_lane<V>(lane, j) < n) *reinterpret_cast<Out*>(codes + at + at_lane<V>(lane, j)) = (Out)(c[j / 4] >> (8 * (j % 4)));
  if (lane == 0) scales[gr] = s;
}

template <typename T, int V>
__global__ void __launch_bounds__(kThreads) dequantize_any_kernel(const uint8_t* __restrict__ codes,
                                                                  const float* __restrict__ scales, uint32_t groups,
                                                                  uint32_t per_row, long long cols, T* __restrict__ out) {
  const uint32_t i = blockIdx.x * (kThreads / kLanes) + threadIdx.x / kLanes;
  const uint32_t gr = min(i, groups - 1);  // lanes behind the last group do its work again: shuffles are warp-wide
  const int lane = threadIdx.x % kLanes;
  const uint32_t row = gr / per_row;
  const long long col = (long long)(gr - row * per_row) * FP8_GROUP, at = row * cols + col;
  const int n = (int)min((long long)FP8_GROUP, cols - col);
  using In = typename Piece<V>::type;
  using Out = typename Piece<V * sizeof(T)>::type;
  const float s = __ldg(scales + gr);
  In raw[kEach / V];
#pragma unroll
  for (int j = 0; j < kEach; j += V)
    if (at_lane<V>(lane, j) < n) raw[j / V] = __ldg(reinterpret_cast<const In*>(codes + at + at_lane<V>(lane, j)));
#pragma unroll
  for (int j = 0; j < kEach; j += V)
    if (at_lane<V>(lane, j) < n) {
      Out o;
#pragma unroll
      for (int e = 0; e < V; ++e)
        reinterpret_cast<T*>(&o)[e] = to_type<T>(fp8_unpair((uint32_t)raw[j / V] >> (8 * e)).x * s);
      *reinterpret_cast<Out*>(out + at + at_lane<V>(lane, j)) = o;
    }
}

// Values side by side that rows of `cols` values at these addresses let a lane take at once.
template <typename T>
int side_by_side(int64_t cols, const void* values, const void* codes) {
  const uintptr_t a = reinterpret_cast<uintptr_t>(values) / sizeof(T) | reinterpret_cast<uintptr_t>(codes) | (uintptr_t)cols;
  return a & 1 ? 1 : a & 2 ? 2 : 4;
}

template <typename T>
int quantize(int64_t rows, int64_t cols, const T* x, uint8_t* codes, float* scales, cudaStream_t st) {
  if (cols % FP8_GROUP == 0 && aligned16(x) && aligned16(codes)) {
    const long long n16 = rows * cols / 16;
    quantize_kernel<<<(unsigned)((n16 + kThreads - 1) / kThreads), kThreads, 0, st>>>(x, n16, codes, scales);
  } else {
    const uint32_t per_row = (uint32_t)((cols + FP8_GROUP - 1) / FP8_GROUP), groups = (uint32_t)(rows * per_row);
    const unsigned grid = (unsigned)(((long long)groups + kThreads / kLanes - 1) / (kThreads / kLanes));
    const int v = side_by_side<T>(cols, x, codes);
    auto kern = v == 4 ? quantize_any_kernel<T, 4> : v == 2 ? quantize_any_kernel<T, 2> : quantize_any_kernel<T, 1>;
    kern<<<grid, kThreads, 0, st>>>(x, groups, per_row, cols, codes, scales);
  }
  return cudaGetLastError() == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
}

template <typename T>
int dequantize(int64_t rows, int64_t cols, const uint8_t* codes, const float* scales, T* out, cudaStream_t st) {
  if (cols % FP8_GROUP == 0 && aligned16(out) && aligned16(codes)) {
    const long long n16 = rows * cols / 16;
    dequantize_kernel<<<(unsigned)((n16 + kThreads - 1) / kThreads), kThreads, 0, st>>>(
        codes, scales, n16, out, (reinterpret_cast<uintptr_t>(out) & 31u) == 0);
  } else {
    const uint32_t per_row = (uint32_t)((cols + FP8_GROUP - 1) / FP8_GROUP), groups = (uint32_t)(rows * per_row);
    const unsigned grid = (unsigned)(((long long)groups + kThreads / kLanes - 1) / (kThreads / kLanes));
    const int v = side_by_side<T>(cols, out, codes);
    auto kern = v == 4 ? dequantize_any_kernel<T, 4> : v == 2 ? dequantize_any_kernel<T, 2> : dequantize_any_kernel<T, 1>;
    kern<<<grid, kThreads, 0, st>>>(codes, scales, groups, per_row, cols, out);
  }
  return cudaGetLastError() == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
}

}  // namespace

int launch_fp8_quantize(int dtype, int64_t rows, int64_t cols, const void* x, uint8_t* codes, float* scales,
                        cudaStream_t st) {
  if (rows == 0 || cols == 0) return MOE_OK;
  return dtype == MOE_F32 ? quantize(rows, cols, static_cast<const float*>(x), codes, scales, st)
                          : quantize(rows, cols, static_cast<const __nv_bfloat16*>(x), codes, scales, st);
}

int launch_fp8_dequantize(int dtype, int64_t rows, int64_t cols, const uint8_t* codes, const float* scales, void* out,
                          cudaStream_t st) {
  if (rows == 0 || cols == 0) return MOE_OK;
  return dtype == MOE_F32 ? dequantize(rows, cols, codes, scales, static_cast<float*>(out), st)
                          : dequantize(rows, cols, codes, scales, static_cast<__nv_bfloat16*>(out), st);
}

}  // namespace moe
