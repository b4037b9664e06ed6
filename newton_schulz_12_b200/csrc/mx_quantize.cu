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
// columns (the rows of the transpose), or both.  A block of threads takes a
// tile of 128 x 128 values, which is a whole tile of scales either way.
#include "common.cuh"
#include "internal.h"

#include <cuda_fp16.h>

namespace muon {
namespace mx {

namespace {

constexpr int kThreads = 256;

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
__device__ __forceinline__ uint32_t encode8(const float* v, float inv = 1.f) {
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

// Two 16-bit values of one word: the larger magnitudes of two words side by
// side (a NaN stays one), and the fp32 bits of a magnitude.
template <typename T>
__device__ __forceinline__ uint32_t max_magnitudes(uint32_t a, uint32_t w);
template <>
__device__ __forceinline__ uint32_t max_magnitudes<bf16>(uint32_t a, uint32_t w) {
  const __nv_bfloat162 r = __hmax2_nan(*reinterpret_cast<const __nv_bfloat162*>(&a), __habs2(*reinterpret_cast<const __nv_bfloat162*>(&w)));
  return *reinterpret_cast<const uint32_t*>(&r);
}
template <>
__device__ __forceinline__ uint32_t max_magnitudes<__half>(uint32_t a, uint32_t w) {
  const __half2 r = __hmax2_nan(*reinterpret_cast<const __half2*>(&a), __habs2(*reinterpret_cast<const __half2*>(&w)));
  return *reinterpret_cast<const uint32_t*>(&r);
}
template <typename T>
__device__ __forceinline__ uint32_t magnitude_bits(uint32_t half);
template <>
__device__ __forceinline__ uint32_t magnitude_bits<bf16>(uint32_t half) { return half << 16; }
template <>
__device__ __forceinline__ uint32_t magnitude_bits<__half>(uint32_t half) {
  return __float_as_uint(__half2float(__ushort_as_half(static_cast<unsigned short>(half))));
}

// Two values of a word times their inverse scales.  bf16 multiplies in bf16: a
// power of two changes no digit, and what falls below its range rounds to code 0.
template <typename T>
__device__ __forceinline__ float2 scaled(uint32_t w, float i0, float i1);
template <>
__device__ __forceinline__ float2 scaled<bf16>(uint32_t w, float i0, float i1) {
  const __nv_bfloat162 p = __hmul2(*reinterpret_cast<const __nv_bfloat162*>(&w), __floats2bfloat162_rn(i0, i1));
  const uint32_t q = *reinterpret_cast<const uint32_t*>(&p);
  return make_float2(__uint_as_float(q << 16), __uint_as_float(q & 0xFFFF0000u));
}
template <>
__device__ __forceinline__ float2 scaled<__half>(uint32_t w, float i0, float i1) {
  const float2 v = __half22float2(*reinterpret_cast<const __half2*>(&w));
  return make_float2(v.x * i0, v.y * i1);
}

// The matrix that tile t belongs to.
template <typename Params>
__device__ __forceinline__ int matrix_of(const Params& p, int t) {
  int lo = 0, hi = p.nmat - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (t >= p.mat[mid].tile_begin)
      lo = mid;
    else
      hi = mid - 1;
  }
  return lo;
}

struct __align__(16) Chunk {
  uint4 q[2];
};

template <typename T>
struct __align__(16) Eight {
  T v[8];
};

// VEC: rows are aligned to 16 bytes and end on 8 values, so a thread reads
// eight at once; else the tile is read value by value.  COLS: the columns'
// blocks are wanted, too.  The tile waits in shared memory as it came for what
// reads it in another order.
template <typename T, bool VEC, bool COLS>
__global__ void __launch_bounds__(kThreads) quantize_kernel(const __grid_constant__ QuantParams p) {
  previous_kernel_done();
  extern __shared__ __align__(16) uint8_t smem[];
  T* tile = reinterpret_cast<T*>(smem);                                // COLS or !VEC: [kTile][kTile]
  uint4* codes = reinterpret_cast<uint4*>(tile + kTile * kTile);       // COLS: [column][4 blocks]
  __shared__ __align__(16) uint8_t sc[2][512];
  const QuantMat& M = p.mat[matrix_of(p, blockIdx.x)];
  const int local = blockIdx.x - M.tile_begin;
  const int tr = local / M.tiles_c, tc = local - tr * M.tiles_c;
  const int r0 = tr * kTile, c0 = tc * kTile;
  const T* x = static_cast<const T*>(M.x) + static_cast<long long>(r0) * M.ldx + c0;
  const int rows = min(kTile, M.rows - r0), cols = min(kTile, M.cols - c0);

  // A thread holds 32 bytes of a row, 16 or 8 values: a block of 32 values is two
  // or four neighbouring threads' (with 16 bytes, the scale's arithmetic and the
  // shuffles for it would be done twice as often: 42.2 us instead of 39.4 for 16384
  // x 4096 bf16, both forms; rows alone 29.2 instead of 26.8).
  constexpr int kPer = 32 / static_cast<int>(sizeof(T)), kSeg = kTile / kPer, kStep = kThreads / kSeg, kRows = kTile / kStep;
  const int seg = threadIdx.x & (kSeg - 1), first = threadIdx.x / kSeg;
  Chunk held[VEC ? kRows : 1];
  if (VEC) {
    if (rows == kTile && cols == kTile) {  // no conditions: all loads are under way at once
#pragma unroll
      for (int i = 0; i < kRows; ++i) {
        const uint4* at = reinterpret_cast<const uint4*>(x + (first + kStep * i) * M.ldx + kPer * seg);
        held[i].q[0] = at[0];
        held[i].q[1] = at[1];
      }
    } else {
#pragma unroll
      for (int i = 0; i < kRows; ++i) {
        const int r = first + kStep * i;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          held[i].q[h] = make_uint4(0, 0, 0, 0);
          const int c = kPer * seg + h * (kPer / 2);
          if (r < rows && c < cols) held[i].q[h] = *reinterpret_cast<const uint4*>(x + r * M.ldx + c);
        }
      }
    }
    if (COLS)
#pragma unroll
      for (int i = 0; i < kRows; ++i) {
        // every other four threads store their second half first: eight threads'
        // 16 bytes then lie in different banks (47.3 us without)
        uint4* dst = reinterpret_cast<uint4*>(tile) + ((first + kStep * i) * kSeg + seg) * 2;
        const bool swap = (threadIdx.x >> 2) & 1;
        dst[swap] = swap ? held[i].q[1] : held[i].q[0];
        dst[!swap] = swap ? held[i].q[0] : held[i].q[1];
      }
  } else {
    constexpr int kBatch = 16;
    const int c = threadIdx.x & 127, half = threadIdx.x >> 7;
    const bool full = rows == kTile && cols == kTile;
    for (int b = half; b < kTile; b += 2 * kBatch) {
      T v[kBatch];
      if (full) {
        const T* at = x + b * M.ldx + c;
#pragma unroll
        for (int i = 0; i < kBatch; ++i) v[i] = at[2 * i * M.ldx];
      } else {
#pragma unroll
        for (int i = 0; i < kBatch; ++i) {
          const int r = b + 2 * i;
          v[i] = r < rows && c < cols ? x[r * M.ldx + c] : rounded<T>(0.f);
        }
      }
#pragma unroll
      for (int i = 0; i < kBatch; ++i) tile[(b + 2 * i) * kTile + c] = v[i];
    }
  }
  if (COLS || !VEC) __syncthreads();

  if (M.row_data) {
    const long long stride = data_stride(M.cols);
    uint8_t* out = static_cast<uint8_t*>(M.row_data) + static_cast<long long>(r0) * stride + (c0 >> 1);
#pragma unroll
    for (int i = 0; i < kRows; ++i) {
      const int r = first + kStep * i;
      const Chunk e = VEC ? held[VEC ? i : 0] : reinterpret_cast<const Chunk*>(tile)[r * kSeg + seg];
      const uint32_t* w = reinterpret_cast<const uint32_t*>(&e);
      float f[kPer];
      uint32_t amax = 0, byte;
      if constexpr (sizeof(T) == 2) {
#pragma unroll
        for (int k = 0; k < 8; ++k) amax = max_magnitudes<T>(amax, w[k]);
        amax = max(amax & 0xFFFFu, amax >> 16);
        amax = max(amax, __shfl_xor_sync(0xFFFFFFFFu, amax, 1));
        byte = scale_byte(magnitude_bits<T>(amax));
        const float inv = inverse_scale(byte);
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          const float2 v = scaled<T>(w[k], inv, inv);
          f[2 * k] = v.x;
          f[2 * k + 1] = v.y;
        }
      } else {
#pragma unroll
        for (int k = 0; k < 8; ++k) amax = max(amax, w[k] & 0x7FFFFFFFu);
        amax = max(amax, __shfl_xor_sync(0xFFFFFFFFu, amax, 1));
        amax = max(amax, __shfl_xor_sync(0xFFFFFFFFu, amax, 2));
        byte = scale_byte(amax);
        const float inv = inverse_scale(byte);
#pragma unroll
        for (int k = 0; k < 8; ++k) f[k] = __uint_as_float(w[k]) * inv;
      }
      const int kb = seg * kPer / 32;  // the block within the tile's row
      const bool in = r < rows && 32 * kb < cols;
      if (in) {
        uint32_t* dst = reinterpret_cast<uint32_t*>(out + r * stride + seg * (kPer / 2));
        if constexpr (kPer == 16)
          *reinterpret_cast<uint2*>(dst) = make_uint2(encode8(f), encode8(f + 8));
        else
          *dst = encode8(f);
      }
      if (seg % (32 / kPer) == 0) sc[0][(r & 31) * 16 + (r >> 5) * 4 + kb] = in ? static_cast<uint8_t>(byte) : 0;
    }
  }
  if (COLS) {
    // Four blocks of a column lie side by side in `codes`, in an order without bank conflicts.
    auto put = [&](int c, int kb, uint32_t byte, const uint32_t (&q)[4]) {
      codes[c * 4 + (kb ^ ((c >> 1) & 3))] = make_uint4(q[0], q[1], q[2], q[3]);
      sc[1][(c & 31) * 16 + (c >> 5) * 4 + kb] = c < cols && 32 * kb < rows ? static_cast<uint8_t>(byte) : 0;
    };
    if constexpr (sizeof(T) == 2) {  // a thread takes a block of two neighbouring columns
      const int pair = threadIdx.x & 63, kb = threadIdx.x >> 6;
      const uint32_t src = smem_u32(tile) + (32 * kb * (kTile / 2) + pair) * 4;
      uint32_t w[32], amax = 0;
#pragma unroll
      for (int k = 0; k < 32; ++k)
        asm volatile("ld.shared.u32 %0, [%1];" : "=r"(w[k]) : "r"(src + k * (kTile / 2) * 4));
#pragma unroll
      for (int k = 0; k < 32; ++k) amax = max_magnitudes<T>(amax, w[k]);
      const uint32_t b0 = scale_byte(magnitude_bits<T>(amax & 0xFFFFu)), b1 = scale_byte(magnitude_bits<T>(amax >> 16));
      const float i0 = inverse_scale(b0), i1 = inverse_scale(b1);
      uint32_t q0[4], q1[4];
#pragma unroll
      for (int g = 0; g < 4; ++g) {
        float f0[8], f1[8];
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          const float2 v = scaled<T>(w[8 * g + k], i0, i1);
          f0[k] = v.x;
          f1[k] = v.y;
        }
        q0[g] = encode8(f0);
        q1[g] = encode8(f1);
      }
      put(2 * pair, kb, b0, q0);
      put(2 * pair + 1, kb, b1, q1);
    } else {
      for (int b = threadIdx.x; b < 512; b += kThreads) {
        const int c = b & 127, kb = b >> 7;
        float f[32];
        uint32_t amax = 0;
#pragma unroll
        for (int k = 0; k < 32; ++k) {
          f[k] = tile[(32 * kb + k) * kTile + c];
          amax = max(amax, __float_as_uint(f[k]) & 0x7FFFFFFFu);
        }
        const uint32_t byte = scale_byte(amax);
        const float inv = inverse_scale(byte);
        const uint32_t q[4] = {encode8(f, inv), encode8(f + 8, inv), encode8(f + 16, inv), encode8(f + 24, inv)};
        put(c, kb, byte, q);
      }
    }
  }
  __syncthreads();
  if (COLS) {
    const long long stride = data_stride(M.rows);
    uint8_t* out = static_cast<uint8_t*>(M.col_data) + static_cast<long long>(c0) * stride + (r0 >> 1);
    for (int b = threadIdx.x; b < 512; b += kThreads) {
      const int c = b >> 2, kb = b & 3;
      if (c < cols && 32 * kb < rows) *reinterpret_cast<uint4*>(out + c * stride + 16 * kb) = codes[c * 4 + (kb ^ ((c >> 1) & 3))];
    }
    const int tiles_r = (M.rows + kTile - 1) / kTile;
    if (threadIdx.x >= 32 && threadIdx.x < 64)
      reinterpret_cast<uint4*>(static_cast<uint8_t*>(M.col_scales) + (static_cast<long long>(tc) * tiles_r + tr) * 512)[threadIdx.x - 32] =
          reinterpret_cast<const uint4*>(sc[1])[threadIdx.x - 32];
  }
  if (M.row_data && threadIdx.x < 32)
    reinterpret_cast<uint4*>(static_cast<uint8_t*>(M.row_scales) + (static_cast<long long>(tr) * M.tiles_c + tc) * 512)[threadIdx.x] =
        reinterpret_cast<const uint4*>(sc[0])[threadIdx.x];
}

// Two codes of a byte to two values, exact in fp16.
__device__ __forceinline__ float2 decode2(uint32_t byte) {
  uint32_t h;
  asm("{\n\t.reg .b8 b;\n\tcvt.u8.u32 b, %1;\n\tcvt.rn.f16x2.e2m1x2 %0, b;\n\t}" : "=r"(h) : "r"(byte));
  return __half22float2(*reinterpret_cast<const __half2*>(&h));
}

__device__ __forceinline__ float scale_value(uint32_t byte) {
  return byte == 255u ? __uint_as_float(0x7FC00000u) : byte ? __uint_as_float(byte << 23) : __uint_as_float(1u << 22);
}

// A tile of 128 x 128 values a block; VEC: y's rows are aligned to 16 bytes and
// end on 8 values.  Else the values go through shared memory, so that a warp's
// stores of single values lie side by side.
template <typename T, bool VEC>
__global__ void __launch_bounds__(kThreads) dequantize_kernel(const __grid_constant__ DequantParams p) {
  previous_kernel_done();
  extern __shared__ __align__(16) uint8_t smem[];
  const DequantMat& M = p.mat[matrix_of(p, blockIdx.x)];
  const int local = blockIdx.x - M.tile_begin;
  const int tr = local / M.tiles_c, tc = local - tr * M.tiles_c;
  const long long stride = data_stride(M.cols);
  const int rows = min(kTile, M.rows - tr * kTile), cols = min(kTile, M.cols - tc * kTile);
  const uint8_t* sc = static_cast<const uint8_t*>(M.scales) + static_cast<long long>(local) * 512;
  const uint8_t* data = static_cast<const uint8_t*>(M.data) + static_cast<long long>(tr) * kTile * stride + tc * (kTile / 2);
  T* y = static_cast<T*>(M.y) + static_cast<long long>(tr) * kTile * M.cols + static_cast<long long>(tc) * kTile;
  const int oct = threadIdx.x & 15, first = threadIdx.x >> 4;
  uint32_t code[kTile / 16], byte[kTile / 16];
#pragma unroll
  for (int i = 0; i < kTile / 16; ++i) {
    const int r = first + 16 * i;
    code[i] = byte[i] = 0;
    if (r < rows && 8 * oct < cols) {
      code[i] = *reinterpret_cast<const uint32_t*>(data + r * stride + 4 * oct);
      byte[i] = sc[(r & 31) * 16 + (r >> 5) * 4 + (oct >> 2)];
    }
  }
#pragma unroll
  for (int i = 0; i < kTile / 16; ++i) {
    const int r = first + 16 * i;
    const float s = scale_value(byte[i]);
    Eight<T> out;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const float2 v = decode2(code[i] >> (8 * k));
      out.v[2 * k] = rounded<T>(v.x * s);
      out.v[2 * k + 1] = rounded<T>(v.y * s);
    }
    if (!VEC)
      reinterpret_cast<Eight<T>*>(smem)[r * 16 + oct] = out;
    else if (r < rows && 8 * oct < cols)
      *reinterpret_cast<Eight<T>*>(y + static_cast<long long>(r) * M.cols + 8 * oct) = out;
  }
  if (!VEC) {
    __syncthreads();
    const T* tile = reinterpret_cast<const T*>(smem);
    const int lane = threadIdx.x & 31;
    for (int r = threadIdx.x >> 5; r < rows; r += kThreads / 32) {
      T* dst = y + static_cast<long long>(r) * M.cols;
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const int c = lane + 32 * k;
        if (c < cols) dst[c] = tile[r * kTile + c];
      }
    }
  }
}

template <typename T, bool VEC, bool COLS>
cudaError_t quantize_as(const QuantParams& p, cudaStream_t s) {
  constexpr int smem = (COLS || !VEC ? kTile * kTile * static_cast<int>(sizeof(T)) : 0) + (COLS ? 8192 : 0);
  static thread_local int configured_device = -1;
  int dev = 0;
  cudaGetDevice(&dev);
  if (configured_device != dev) {
    cudaError_t e = cudaFuncSetAttribute(quantize_kernel<T, VEC, COLS>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e != cudaSuccess) return e;
    configured_device = dev;
  }
  return launch_after(quantize_kernel<T, VEC, COLS>, p.ntiles, kThreads, smem, s, 1, p);
}

// A launch reads eight values at once where all of its matrices allow it.
template <typename T>
cudaError_t quantize(const QuantParams& p, cudaStream_t s) {
  bool vec = true, cols = false;
  for (int i = 0; i < p.nmat; ++i) {
    const QuantMat& M = p.mat[i];
    vec = vec && M.cols % 8 == 0 && reinterpret_cast<uintptr_t>(M.x) % 16 == 0 && (M.rows <= 1 || M.ldx * sizeof(T) % 16 == 0);
    cols = cols || M.col_data;
  }
  if (vec) return cols ? quantize_as<T, true, true>(p, s) : quantize_as<T, true, false>(p, s);
  return cols ? quantize_as<T, false, true>(p, s) : quantize_as<T, false, false>(p, s);
}

template <typename T>
cudaError_t dequantize(const DequantParams& p, cudaStream_t s) {
  bool vec = true;
  for (int i = 0; i < p.nmat; ++i) vec = vec && p.mat[i].cols % 8 == 0 && reinterpret_cast<uintptr_t>(p.mat[i].y) % 16 == 0;
  if (vec) {
    return launch_after(dequantize_kernel<T, true>, p.ntiles, kThreads, 0, s, 1, p);
  }
  constexpr int smem = kTile * kTile * static_cast<int>(sizeof(T));
  static thread_local int configured_device = -1;
  int dev = 0;
  cudaGetDevice(&dev);
  if (configured_device != dev) {
    cudaError_t e = cudaFuncSetAttribute(dequantize_kernel<T, false>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e != cudaSuccess) return e;
    configured_device = dev;
  }
  return launch_after(dequantize_kernel<T, false>, p.ntiles, kThreads, smem, s, 1, p);
}

}  // namespace

cudaError_t launch_quantize(const QuantParams& p, int dtype, cudaStream_t s) {
  if (p.ntiles <= 0) return cudaSuccess;
  return dtype == 1 ? quantize<float>(p, s) : dtype == 0 ? quantize<bf16>(p, s) : quantize<__half>(p, s);
}

cudaError_t launch_dequantize(const DequantParams& p, int dtype, cudaStream_t s) {
  if (p.ntiles <= 0) return cudaSuccess;
  return dtype == 1 ? dequantize<float>(p, s) : dtype == 0 ? dequantize<bf16>(p, s) : dequantize<__half>(p, s);
}

}  // namespace mx
}  // namespace muon
