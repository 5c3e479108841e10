// MXFP4 quantisation of rows and back.
//
// A row's length is a multiple of 32, so the blocks of all rows lie one after the other and
// the kernels work on the flat array: codes and scales of block i are at 16 i and at i.  Both are bound by
// HBM: 28672 x 4096 fp32 takes 86 us to quantise (6.2 TB/s) and 78 us back (6.8 TB/s).
#include "mx.cuh"

namespace moe {
namespace {

constexpr int kThreads = 256;

// Eight consecutive values of a 16-byte aligned array.
__device__ __forceinline__ void load8(const float* x, float (&v)[8]) {
  const float4 a = __ldg(reinterpret_cast<const float4*>(x));
  const float4 b = __ldg(reinterpret_cast<const float4*>(x) + 1);
  v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w, v[4] = b.x, v[5] = b.y, v[6] = b.z, v[7] = b.w;
}

__device__ __forceinline__ void load8(const __nv_bfloat16* x, float (&v)[8]) {
  const uint4 raw = __ldg(reinterpret_cast<const uint4*>(x));
  const __nv_bfloat162* h = reinterpret_cast<const __nv_bfloat162*>(&raw);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 f = __bfloat1622float2(h[i]);
    v[2 * i] = f.x;
    v[2 * i + 1] = f.y;
  }
}

__device__ __forceinline__ void store8(float* x, const float (&v)[8], bool wide) {
  const uint4 a = make_uint4(__float_as_uint(v[0]), __float_as_uint(v[1]), __float_as_uint(v[2]), __float_as_uint(v[3]));
  const uint4 b = make_uint4(__float_as_uint(v[4]), __float_as_uint(v[5]), __float_as_uint(v[6]), __float_as_uint(v[7]));
  if (wide) {
    st_global_v8(x, a, b);
  } else {
    reinterpret_cast<uint4*>(x)[0] = a;
    reinterpret_cast<uint4*>(x)[1] = b;
  }
}

__device__ __forceinline__ void store8(__nv_bfloat16* x, const float (&v)[8], bool) {
  uint4 raw;
  __nv_bfloat162* h = reinterpret_cast<__nv_bfloat162*>(&raw);
#pragma unroll
  for (int i = 0; i < 4; ++i) h[i] = __floats2bfloat162_rn(v[2 * i], v[2 * i + 1]);
  *reinterpret_cast<uint4*>(x) = raw;
}

// Eight values a thread, four threads a block.  n8 = values / 8 is a multiple of 4, so the four
// threads of a block are all in range or all out of it.
template <typename T>
__global__ void __launch_bounds__(kThreads) mx_quantize_kernel(const T* __restrict__ x, long long n8,
                                                               uint8_t* __restrict__ codes,
                                                               uint8_t* __restrict__ scales) {
  const long long i = (long long)blockIdx.x * kThreads + threadIdx.x;
  float v[8];
  float amax = 0.0f;
  if (i < n8) {
    load8(x + 8 * i, v);
#pragma unroll
    for (int j = 0; j < 8; ++j) amax = mx_amax(amax, v[j]);
  }
  amax = mx_amax(amax, __shfl_xor_sync(0xffffffffu, amax, 1));
  amax = mx_amax(amax, __shfl_xor_sync(0xffffffffu, amax, 2));
  if (i >= n8) return;
  const uint32_t s = mx_scale_byte(amax);
  reinterpret_cast<uint32_t*>(codes)[i] = mx_codes8(v, mx_inv_scale(s));
  if ((i & 3) == 0) scales[i >> 2] = (uint8_t)s;
}

template <typename T>
__global__ void __launch_bounds__(kThreads) mx_dequantize_kernel(const uint8_t* __restrict__ codes,
                                                                 const uint8_t* __restrict__ scales, long long n8,
                                                                 T* __restrict__ out) {
  const long long i = (long long)blockIdx.x * kThreads + threadIdx.x;
  if (i >= n8) return;
  const uint32_t c = __ldg(reinterpret_cast<const uint32_t*>(codes) + i);
  const float sc = mx_scale(__ldg(scales + (i >> 2)));
  float v[8];
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const __half2_raw h = __nv_cvt_fp4x2_to_halfraw2((__nv_fp4x2_storage_t)(c >> (8 * j)), __NV_E2M1);
    const float2 f = __half22float2(__half2(h));
    v[2 * j] = f.x * sc;
    v[2 * j + 1] = f.y * sc;
  }
  store8(out + 8 * i, v, (reinterpret_cast<uintptr_t>(out) & 31u) == 0);  // whole 32-byte sectors where they can be
}

}  // namespace

int launch_mx_quantize(int dtype, int64_t rows, int64_t cols, const void* x, uint8_t* codes, uint8_t* scales,
                       cudaStream_t st) {
  const long long n8 = rows * cols / 8;
  if (n8 == 0) return MOE_OK;
  const unsigned grid = (unsigned)((n8 + kThreads - 1) / kThreads);
  if (dtype == MOE_F32)
    mx_quantize_kernel<<<grid, kThreads, 0, st>>>(static_cast<const float*>(x), n8, codes, scales);
  else
    mx_quantize_kernel<<<grid, kThreads, 0, st>>>(static_cast<const __nv_bfloat16*>(x), n8, codes, scales);
  return cudaGetLastError() == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
}

int launch_mx_dequantize(int dtype, int64_t rows, int64_t cols, const uint8_t* codes, const uint8_t* scales,
                         void* out, cudaStream_t st) {
  const long long n8 = rows * cols / 8;
  if (n8 == 0) return MOE_OK;
  const unsigned grid = (unsigned)((n8 + kThreads - 1) / kThreads);
  if (dtype == MOE_F32)
    mx_dequantize_kernel<<<grid, kThreads, 0, st>>>(codes, scales, n8, static_cast<float*>(out));
  else
    mx_dequantize_kernel<<<grid, kThreads, 0, st>>>(codes, scales, n8, static_cast<__nv_bfloat16*>(out));
  return cudaGetLastError() == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
}

}  // namespace moe
