// Layer norm over the rows of a matrix, and its gradient.
//
//   y    = (x - mean) rstd w + b,   rstd = 1 / sqrt(mean((x - mean)^2) + eps)
//   xhat = (x - mean) rstd,  g = dy w
//   dx   = rstd (g - mean(g) - xhat mean(g xhat)),  dw = sum_rows dy xhat,  db = sum_rows dy
//
// Both passes are bound by bytes: the forward reads x and writes y, the
// backward reads x and dy and writes dx; 8 to 14 flops an element.  Every
// statistic is an fp32 sum in a fixed order (per thread, then across the
// threads of the row), the variance from centred values, so an offset that is
// large against the spread costs no digits.
#include "common.cuh"
#include "internal.h"

#include <cuda_fp16.h>

namespace muon {
namespace ln {

namespace {

template <typename T>
__device__ __forceinline__ float to_f(T v);
template <>
__device__ __forceinline__ float to_f<float>(float v) { return v; }
template <>
__device__ __forceinline__ float to_f<bf16>(bf16 v) { return __bfloat162float(v); }
template <>
__device__ __forceinline__ float to_f<__half>(__half v) { return __half2float(v); }

// The one rounding of a result to its storage type, to nearest even.
template <typename T>
__device__ __forceinline__ T from_f(float v);
template <>
__device__ __forceinline__ float from_f<float>(float v) { return v; }
template <>
__device__ __forceinline__ bf16 from_f<bf16>(float v) { return __float2bfloat16_rn(v); }
template <>
__device__ __forceinline__ __half from_f<__half>(float v) { return __float2half_rn(v); }

constexpr int kLoopThreads = 512;

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
  return v;
}

// Sum over the block, the same value in every thread; `buf` holds one float a
// warp and is free again on return.
__device__ __forceinline__ float block_sum(float v, float* buf) {
  v = warp_sum(v);
  if ((threadIdx.x & 31) == 0) buf[threadIdx.x >> 5] = v;
  __syncthreads();
  float s = 0.f;
  for (int w = 0; w < static_cast<int>(blockDim.x >> 5); ++w) s += buf[w];
  __syncthreads();
  return s;
}

// One row a block at a time, read again for every step: any width, any
// alignment.
template <typename T, typename P>
__global__ void __launch_bounds__(kLoopThreads) forward_loop_kernel(const FwdParams p) {
  __shared__ float buf[32];
  for (long long r = blockIdx.x; r < p.rows; r += gridDim.x) {
    const T* x = static_cast<const T*>(p.x) + r * p.ldx;
    T* y = static_cast<T*>(p.y) + r * p.ldy;
    float s = 0.f;
    for (int c = threadIdx.x; c < p.cols; c += blockDim.x) s += to_f(x[c]);
    const float mean = block_sum(s, buf) / p.cols;
    float q = 0.f;
    for (int c = threadIdx.x; c < p.cols; c += blockDim.x) {
      const float d = to_f(x[c]) - mean;
      q = fmaf(d, d, q);
    }
    const float rstd = 1.0f / sqrtf(block_sum(q, buf) / p.cols + p.eps);
    for (int c = threadIdx.x; c < p.cols; c += blockDim.x) {
      float v = (to_f(x[c]) - mean) * rstd;
      if (p.weight) v *= to_f(static_cast<const P*>(p.weight)[c]);
      if (p.bias) v += to_f(static_cast<const P*>(p.bias)[c]);
      y[c] = from_f<T>(v);
    }
    if (threadIdx.x == 0) {
      p.mean[r] = mean;
      p.rstd[r] = rstd;
    }
  }
}

// dx of one row a block at a time, read twice.
template <typename T, typename P>
__global__ void __launch_bounds__(kLoopThreads) backward_loop_kernel(const BwdParams p) {
  __shared__ float buf[32];
  for (long long r = blockIdx.x; r < p.rows; r += gridDim.x) {
    const T* x = static_cast<const T*>(p.x) + r * p.ldx;
    const T* dy = static_cast<const T*>(p.dy) + r * p.lddy;
    T* dx = static_cast<T*>(p.dx) + r * p.lddx;
    const float mean = p.mean[r], rstd = p.rstd[r];
    float s = 0.f, q = 0.f;
    for (int c = threadIdx.x; c < p.cols; c += blockDim.x) {
      float g = to_f(dy[c]);
      if (p.weight) g *= to_f(static_cast<const P*>(p.weight)[c]);
      s += g;
      q = fmaf(g, (to_f(x[c]) - mean) * rstd, q);
    }
    s = block_sum(s, buf) / p.cols;
    q = block_sum(q, buf) / p.cols;
    for (int c = threadIdx.x; c < p.cols; c += blockDim.x) {
      float g = to_f(dy[c]);
      if (p.weight) g *= to_f(static_cast<const P*>(p.weight)[c]);
      const float xhat = (to_f(x[c]) - mean) * rstd;
      dx[c] = from_f<T>(rstd * (g - s - xhat * q));
    }
  }
}

// Partial column sums of dy xhat and dy: block (i, j) takes 32 columns and the
// j-th of `parts` runs of rows, and writes partial j.
template <typename T>
__global__ void __launch_bounds__(256) column_kernel(const BwdParams p) {
  __shared__ float sw[8][33], sb[8][33];
  const int tx = threadIdx.x & 31, ty = threadIdx.x >> 5;
  const int c = blockIdx.x * 32 + tx;
  const long long per = (p.rows + p.parts - 1) / p.parts;
  const long long r0 = per * blockIdx.y;
  const long long r1 = r0 + per < p.rows ? r0 + per : p.rows;
  float w = 0.f, b = 0.f;
  if (c < p.cols) {
    for (long long r = r0 + ty; r < r1; r += 8) {
      const float d = to_f(static_cast<const T*>(p.dy)[r * p.lddy + c]);
      const float xhat = (to_f(static_cast<const T*>(p.x)[r * p.ldx + c]) - p.mean[r]) * p.rstd[r];
      w = fmaf(d, xhat, w);
      b += d;
    }
  }
  sw[ty][tx] = w;
  sb[ty][tx] = b;
  __syncthreads();
  if (ty == 0 && c < p.cols) {
    for (int k = 1; k < 8; ++k) {
      w += sw[k][tx];
      b += sb[k][tx];
    }
    float* out = p.partials + static_cast<long long>(blockIdx.y) * 2 * p.cols;
    out[c] = w;
    out[p.cols + c] = b;
  }
}

// dw and db from the partials, summed in their order; 32 columns a block.
template <typename P>
__global__ void __launch_bounds__(256) finish_kernel(const BwdParams p) {
  __shared__ float sw[8][33], sb[8][33];
  const int tx = threadIdx.x & 31, ty = threadIdx.x >> 5;
  const int c = blockIdx.x * 32 + tx;
  float w = 0.f, b = 0.f;
  if (c < p.cols) {
    for (int k = ty; k < p.parts; k += 8) {
      const float* in = p.partials + static_cast<long long>(k) * 2 * p.cols;
      w += in[c];
      b += in[p.cols + c];
    }
  }
  sw[ty][tx] = w;
  sb[ty][tx] = b;
  __syncthreads();
  if (ty == 0 && c < p.cols) {
    for (int k = 1; k < 8; ++k) {
      w += sw[k][tx];
      b += sb[k][tx];
    }
    if (p.dweight) static_cast<P*>(p.dweight)[c] = from_f<P>(w);
    if (p.dbias) static_cast<P*>(p.dbias)[c] = from_f<P>(b);
  }
}

template <typename T, typename P>
cudaError_t forward(const FwdParams& p, int sms, cudaStream_t s) {
  const long long want = static_cast<long long>(sms) * 4;
  forward_loop_kernel<T, P><<<static_cast<int>(p.rows < want ? p.rows : want), kLoopThreads, 0, s>>>(p);
  return cudaGetLastError();
}

template <typename T, typename P>
cudaError_t backward(const BwdParams& p, int sms, cudaStream_t s) {
  if (p.rows > 0) {
    const long long want = static_cast<long long>(sms) * 4;
    backward_loop_kernel<T, P><<<static_cast<int>(p.rows < want ? p.rows : want), kLoopThreads, 0, s>>>(p);
  }
  if (p.dweight || p.dbias) {
    if (p.parts > 0) column_kernel<T><<<dim3((p.cols + 31) / 32, p.parts), 256, 0, s>>>(p);
    finish_kernel<P><<<(p.cols + 31) / 32, 256, 0, s>>>(p);
  }
  return cudaGetLastError();
}

}  // namespace

// Partial column sums of a backward pass: runs of at least 64 rows, 64 of them at most.
int partial_count(long long rows, int cols, int sms) {
  (void)cols;
  (void)sms;
  const long long n = (rows + 63) / 64;
  return static_cast<int>(n < 64 ? n : 64);
}

cudaError_t launch_forward(const FwdParams& p, int dtype, int param_dtype, int sms, cudaStream_t s) {
  if (dtype == 1) return forward<float, float>(p, sms, s);
  if (dtype == 0)
    return param_dtype == 1 ? forward<bf16, float>(p, sms, s) : forward<bf16, bf16>(p, sms, s);
  return param_dtype == 1 ? forward<__half, float>(p, sms, s) : forward<__half, __half>(p, sms, s);
}

cudaError_t launch_backward(const BwdParams& p, int dtype, int param_dtype, int sms, cudaStream_t s) {
  if (dtype == 1) return backward<float, float>(p, sms, s);
  if (dtype == 0)
    return param_dtype == 1 ? backward<bf16, float>(p, sms, s) : backward<bf16, bf16>(p, sms, s);
  return param_dtype == 1 ? backward<__half, float>(p, sms, s) : backward<__half, __half>(p, sms, s);
}

}  // namespace ln
}  // namespace muon
