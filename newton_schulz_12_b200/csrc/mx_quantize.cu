// 4-bit microscaled (MX) matrices: E2M1 values in blocks of 32, one
// power-of-two scale byte a block (OCP Microscaling Formats v1.0: shared
// exponent floor(log2 amax) - 2, elements rounded to nearest even and held at
// the largest magnitude, 6).
//
//   byte  = max(0, E - 2), E the biased fp32 exponent of the block's largest
//           magnitude; 255 (NaN) when the block holds an infinity or a NaN
//   code  = e2m1(x 2^(127 - byte)): the product is exact (a power of two, and
//           2^(127 - byte) is a normal fp32 number for every byte but 255)
//
// Bound by bytes: one read of x gives the blocks along its rows, along its
// columns (the rows of the transpose), or both.
#include "common.cuh"
#include "internal.h"

#include <cuda_fp16.h>

namespace muon {
namespace mx {

namespace {

constexpr int kThreads = 256;
constexpr int kLd = kTile + 1;  // fp32 tile row: column and row reads without bank conflicts

__device__ __forceinline__ float as_float(float v) { return v; }
__device__ __forceinline__ float as_float(bf16 v) { return __bfloat162float(v); }
__device__ __forceinline__ float as_float(__half v) { return __half2float(v); }

template <typename T>
__device__ __forceinline__ T rounded(float v);
template <>
__device__ __forceinline__ float rounded<float>(float v) { return v; }
template <>
__device__ __forceinline__ bf16 rounded<bf16>(float v) { return __float2bfloat16_rn(v); }
template <>
__device__ __forceinline__ __half rounded<__half>(float v) { return __float2half_rn(v); }

// Scale byte of a block from the fp32 bits of its largest magnitude.
__device__ __forceinline__ uint32_t scale_byte(uint32_t amax_bits) {
  const int e = static_cast<int>(amax_bits >> 23);
  return e == 255 ? 255u : static_cast<uint32_t>(max(e - 2, 0));
}

// 2^(127 - byte); a block that is NaN by its scale gets codes of no meaning.
__device__ __forceinline__ float inverse_scale(uint32_t byte) {
  return __uint_as_float(byte == 255u ? 0u : (254u - byte) << 23);
}

// Eight values to eight codes, the first in the lowest four bits.
__device__ __forceinline__ uint32_t encode8(const float* v, float inv) {
  uint32_t r;
  asm("{\n\t.reg .b8 b0, b1, b2, b3;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b0, %2, %1;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b1, %4, %3;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b2, %6, %5;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b3, %8, %7;\n\t"
      "mov.b32 %0, {b0, b1, b2, b3};\n\t}"
      : "=r"(r)
      : "f"(v[0] * inv), "f"(v[1] * inv), "f"(v[2] * inv), "f"(v[3] * inv), "f"(v[4] * inv), "f"(v[5] * inv),
        "f"(v[6] * inv), "f"(v[7] * inv));
  return r;
}

// One block of 32 values, `step` floats apart: its 16 bytes of codes and its scale byte.
__device__ __forceinline__ uint4 encode_block(const float* v, int step, uint32_t& byte) {
  float f[32];
  uint32_t amax = 0;
#pragma unroll
  for (int i = 0; i < 32; ++i) {
    f[i] = v[i * step];
    amax = max(amax, __float_as_uint(f[i]) & 0x7FFFFFFFu);
  }
  byte = scale_byte(amax);
  const float inv = inverse_scale(byte);
  return make_uint4(encode8(f, inv), encode8(f + 8, inv), encode8(f + 16, inv), encode8(f + 24, inv));
}

template <typename T>
__global__ void __launch_bounds__(kThreads) quantize_kernel(const __grid_constant__ QuantParams p) {
  extern __shared__ float tile[];  // [kTile][kLd]
  __shared__ __align__(16) uint8_t sc[2][512];
  for (int t = blockIdx.x; t < p.ntiles; t += gridDim.x) {
    int i = 0;
    while (i + 1 < p.nmat && t >= p.mat[i + 1].tile_begin) ++i;
    const QuantMat& M = p.mat[i];
    const int local = t - M.tile_begin;
    const int tr = local / M.tiles_c, tc = local - tr * M.tiles_c;
    const int r0 = tr * kTile, c0 = tc * kTile;
    const T* x = static_cast<const T*>(M.x);
    for (int e = threadIdx.x; e < kTile * kTile; e += kThreads) {
      const int r = e / kTile, c = e - r * kTile;
      float v = 0.f;
      if (r0 + r < M.rows && c0 + c < M.cols) v = as_float(x[(r0 + r) * M.ldx + c0 + c]);
      tile[r * kLd + c] = v;
    }
    __syncthreads();
    if (M.row_data) {
      const long long stride = data_stride(M.cols);
      for (int b = threadIdx.x; b < 512; b += kThreads) {
        const int r = b >> 2, kb = b & 3;
        uint32_t byte;
        const uint4 q = encode_block(tile + r * kLd + 32 * kb, 1, byte);
        const bool in = r0 + r < M.rows && c0 + 32 * kb < M.cols;
        sc[0][(r & 31) * 16 + (r >> 5) * 4 + kb] = in ? static_cast<uint8_t>(byte) : 0;
        if (in)
          *reinterpret_cast<uint4*>(static_cast<uint8_t*>(M.row_data) + (r0 + r) * stride + (c0 >> 1) + 16 * kb) = q;
      }
    }
    if (M.col_data) {
      const long long stride = data_stride(M.rows);
      for (int b = threadIdx.x; b < 512; b += kThreads) {
        const int c = b & 127, kb = b >> 7;
        uint32_t byte;
        const uint4 q = encode_block(tile + 32 * kb * kLd + c, kLd, byte);
        const bool in = c0 + c < M.cols && r0 + 32 * kb < M.rows;
        sc[1][(c & 31) * 16 + (c >> 5) * 4 + kb] = in ? static_cast<uint8_t>(byte) : 0;
        if (in)
          *reinterpret_cast<uint4*>(static_cast<uint8_t*>(M.col_data) + (c0 + c) * stride + (r0 >> 1) + 16 * kb) = q;
      }
    }
    __syncthreads();
    const int tiles_r = (M.rows + kTile - 1) / kTile;
    if (M.row_data && threadIdx.x < 32)
      reinterpret_cast<uint4*>(static_cast<uint8_t*>(M.row_scales) + (static_cast<long long>(tr) * M.tiles_c + tc) * 512)[threadIdx.x] =
          reinterpret_cast<const uint4*>(sc[0])[threadIdx.x];
    if (M.col_data && threadIdx.x >= 32 && threadIdx.x < 64)
      reinterpret_cast<uint4*>(static_cast<uint8_t*>(M.col_scales) + (static_cast<long long>(tc) * tiles_r + tr) * 512)[threadIdx.x - 32] =
          reinterpret_cast<const uint4*>(sc[1])[threadIdx.x - 32];
    __syncthreads();
  }
}

// The value of a code (0 .. 15) in fp32.
__device__ __forceinline__ float decode(uint32_t code) {
  const uint32_t e = (code >> 1) & 3u, m = code & 1u;
  const float mag = e ? __uint_as_float((126u + e) << 23 | m << 22) : 0.5f * m;
  return code & 8u ? -mag : mag;
}

__device__ __forceinline__ float scale_value(uint32_t byte) {
  return byte == 255u ? __uint_as_float(0x7FC00000u) : byte ? __uint_as_float(byte << 23) : __uint_as_float(1u << 22);
}

template <typename T>
__global__ void __launch_bounds__(kThreads) dequantize_kernel(const __grid_constant__ DequantParams p) {
  for (int t = blockIdx.x; t < p.ntiles; t += gridDim.x) {
    int i = 0;
    while (i + 1 < p.nmat && t >= p.mat[i + 1].tile_begin) ++i;
    const DequantMat& M = p.mat[i];
    const int local = t - M.tile_begin;
    const int tr = local / M.tiles_c, tc = local - tr * M.tiles_c;
    const long long stride = data_stride(M.cols);
    const uint8_t* sc = static_cast<const uint8_t*>(M.scales) + static_cast<long long>(local) * 512;
    for (int e = threadIdx.x; e < kTile * kTile; e += kThreads) {
      const int r = e / kTile, c = e - r * kTile;
      const long long row = static_cast<long long>(tr) * kTile + r;
      const int col = tc * kTile + c;
      if (row >= M.rows || col >= M.cols) continue;
      const uint32_t two = static_cast<const uint8_t*>(M.data)[row * stride + (col >> 1)];
      const float s = scale_value(sc[(r & 31) * 16 + (r >> 5) * 4 + (c >> 5)]);
      static_cast<T*>(M.y)[row * M.cols + col] = rounded<T>(decode((two >> (4 * (col & 1))) & 15u) * s);
    }
  }
}

template <typename T>
cudaError_t quantize(const QuantParams& p, int sms, cudaStream_t s) {
  constexpr int smem = kTile * kLd * 4;
  static thread_local int configured_device = -1;
  int dev = 0;
  cudaGetDevice(&dev);
  if (configured_device != dev) {
    cudaError_t e = cudaFuncSetAttribute(quantize_kernel<T>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e != cudaSuccess) return e;
    configured_device = dev;
  }
  const int grid = p.ntiles < 3 * sms ? p.ntiles : 3 * sms;
  quantize_kernel<T><<<grid, kThreads, smem, s>>>(p);
  return cudaGetLastError();
}

template <typename T>
cudaError_t dequantize(const DequantParams& p, int sms, cudaStream_t s) {
  const int grid = p.ntiles < 8 * sms ? p.ntiles : 8 * sms;
  dequantize_kernel<T><<<grid, kThreads, 0, s>>>(p);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_quantize(const QuantParams& p, int dtype, int sms, cudaStream_t s) {
  if (p.ntiles <= 0) return cudaSuccess;
  return dtype == 1 ? quantize<float>(p, sms, s) : dtype == 0 ? quantize<bf16>(p, sms, s) : quantize<__half>(p, sms, s);
}

cudaError_t launch_dequantize(const DequantParams& p, int dtype, int sms, cudaStream_t s) {
  if (p.ntiles <= 0) return cudaSuccess;
  return dtype == 1 ? dequantize<float>(p, sms, s) : dtype == 0 ? dequantize<bf16>(p, sms, s) : dequantize<__half>(p, sms, s);
}

}  // namespace mx
}  // namespace muon
