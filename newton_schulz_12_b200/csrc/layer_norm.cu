// Layer norm over the rows of a matrix, and its gradient.
//
//   y    = (x - mean) rstd w + b,   rstd = 1 / sqrt(mean((x - mean)^2) + eps)
//   xhat = (x - mean) rstd,  g = dy w
//   dx   = rstd (g - mean(g) - xhat mean(g xhat)),  dw = sum_rows dy xhat,  db = sum_rows dy
//
// Both passes are bound by bytes: the forward reads x and writes y, the
// backward reads x and dy and writes dx; 8 to 14 flops an element.  Every
// statistic is an fp32 sum in a fixed order (per thread, then across the
// threads of the row), the variance from centred values, so that nothing cancels
// in it.  The mean is an fp32 number: at an offset of 4096 spreads its rounding
// alone, half a unit, moves every y of the row by up to 2.4e-4 of a spread.
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
  previous_kernel_done();
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
  previous_kernel_done();
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

// dw and db from the partials, summed in a fixed order; 32 columns a block.
template <typename P>
__global__ void __launch_bounds__(1024) finish_kernel(const BwdParams p) {
  previous_kernel_done();
  __shared__ float sw[32][33], sb[32][33];
  const int tx = threadIdx.x & 31, ty = threadIdx.x >> 5;
  const int c = blockIdx.x * 32 + tx;
  float w = 0.f, b = 0.f;
  if (c < p.cols) {
#pragma unroll 4
    for (int k = ty; k < p.parts; k += 32) {
      const float* in = p.partials + static_cast<long long>(k) * 2 * p.cols;
      w += in[c];
      b += in[p.cols + c];
    }
  }
  sw[ty][tx] = w;
  sb[ty][tx] = b;
  __syncthreads();
  // thread (tx, ty) takes partial tx of column ty: one warp a column
  w = warp_sum(sw[tx][ty]);
  b = warp_sum(sb[tx][ty]);
  const int o = blockIdx.x * 32 + ty;
  if (tx == 0 && o < p.cols) {
    if (p.dweight) static_cast<P*>(p.dweight)[o] = from_f<P>(w);
    if (p.dbias) static_cast<P*>(p.dbias)[o] = from_f<P>(b);
  }
}

// ---------------------------------------------------------------------------
// Rows held on chip.  A row is the work of `tpr` threads (8, 16 or whole warps)
// with E = VEC * NV values each; a block has `groups` such groups and walks over
// the rows, two values an instruction (f32x2).
//
// RING: every thread copies its own values of the next rows into its own places
// of a ring in shared memory (cp.async: a thread waits for nobody else) and
// works on a row from registers.  Else a row is loaded straight into registers:
// for launches of few rows, which the ring's set-up costs more than it gives
// (1 x 768 bf16: 2.4 us against 4.7), and for 16-bit rows that start on no 16
// bytes, whose values would each take a 4-byte copy (16381 x 1021 bf16: 28.9 us
// against 42.3).
//
// What bounds it: bytes in flight first (about 40 KB an SM cover the latency),
// then the issue of instructions.  A row's sums cost the same for 8 values a
// thread as for 32, so a row takes as few warps as hold it.  The parameters are
// laid out in shared memory once, in the order in which threads read them: read
// from L1 as fp32, 32 bytes a lane, they kept it at 80 % of its throughput.
//
// VEC values are one 16-byte access where rows and results are aligned for it,
// else VEC = 1.
// ---------------------------------------------------------------------------
constexpr int kFwdE = 32, kFwdThreads = 512;  // values a thread, threads a block: at most
constexpr int kBwdE = 24, kBwdThreads = 384;  // with the column sums
constexpr int kMaxDepth = 4;                  // ring slots
constexpr int kSmemBudget = 212 * 1024;       // of an SM, for its blocks' rings and parameters

template <typename T, int VEC>
struct Pack;  // VEC values of one access
template <typename T>
struct Pack<T, 1> {
  T v[1];
};
template <typename T, int VEC>
struct __align__(16) Pack {
  T v[VEC];
};

// Partial column sums of dy xhat and dy, where rows are too wide to add them up
// on the way: block (i, j) takes 32 V columns, V a thread in one access, and the
// j-th of `parts` runs of rows, and writes partial j.
template <typename T, int V>
__global__ void __launch_bounds__(256) column_kernel(const BwdParams p) {
  previous_kernel_done();
  __shared__ float part[8][32 * V + 1];
  const int tx = threadIdx.x & 31, ty = threadIdx.x >> 5;
  const int c = (blockIdx.x * 32 + tx) * V;
  const long long per = (p.rows + p.parts - 1) / p.parts;
  const long long r0 = per * blockIdx.y;
  const long long r1 = r0 + per < p.rows ? r0 + per : p.rows;
  float w[V], b[V];
#pragma unroll
  for (int k = 0; k < V; ++k) w[k] = b[k] = 0.f;
  if (c < p.cols) {
    const T* x = static_cast<const T*>(p.x) + c;
    const T* dy = static_cast<const T*>(p.dy) + c;
#pragma unroll 4
    for (long long r = r0 + ty; r < r1; r += 8) {
      const Pack<T, V> xv = *reinterpret_cast<const Pack<T, V>*>(x + r * p.ldx);
      const Pack<T, V> dv = *reinterpret_cast<const Pack<T, V>*>(dy + r * p.lddy);
      const float mean = p.mean[r], rstd = p.rstd[r];
#pragma unroll
      for (int k = 0; k < V; ++k) {
        const float d = to_f(dv.v[k]);
        w[k] = fmaf(d, (to_f(xv.v[k]) - mean) * rstd, w[k]);
        b[k] += d;
      }
    }
  }
  float* out = p.partials + static_cast<long long>(blockIdx.y) * 2 * p.cols;
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    if (h) __syncthreads();
#pragma unroll
    for (int k = 0; k < V; ++k) part[ty][tx * V + k] = h ? b[k] : w[k];
    __syncthreads();
    for (int i = threadIdx.x; i < 32 * V; i += 256) {
      const int col = blockIdx.x * 32 * V + i;
      if (col >= p.cols) break;
      float v = part[0][i];
      for (int k = 1; k < 8; ++k) v += part[k][i];
      out[h * p.cols + col] = v;
    }
  }
}

// Two fp32 values in one register pair: the packed operations of common.cuh
// work on both at once, each rounded as alone.
typedef unsigned long long f32x2;

template <typename T>
__device__ __forceinline__ f32x2 widen(T lo, T hi) { return f2(to_f(lo), to_f(hi)); }

template <typename T>
__device__ __forceinline__ void narrow(f32x2 v, T* out);
template <>
__device__ __forceinline__ void narrow<float>(f32x2 v, float* out) { f2_split(v, out[0], out[1]); }
template <>
__device__ __forceinline__ void narrow<bf16>(f32x2 v, bf16* out) {
  float lo, hi;
  f2_split(v, lo, hi);
  *reinterpret_cast<__nv_bfloat162*>(out) = __floats2bfloat162_rn(lo, hi);
}
template <>
__device__ __forceinline__ void narrow<__half>(f32x2 v, __half* out) {
  float lo, hi;
  f2_split(v, lo, hi);
  *reinterpret_cast<__half2*>(out) = __floats2half2_rn(lo, hi);
}

// 1 / sqrt(v): the hardware's estimate (2 fp32 units) and one Newton step, left
// out where it would make a NaN of 0 or an infinity.  v y comes first: half of
// v itself would round where v is subnormal.
__device__ __forceinline__ float reciprocal_root(float v) {
  const float y = rsqrtf(v), z = y * fmaf(v * y, -0.5f * y, 1.5f);
  return v > 0.f && y > 0.f ? z : y;
}

// s / n, `inv` being 1 / n rounded: the product and one correction by its exact
// remainder (Markstein, IBM J. Res. Dev. 34, 1990), so that a mean that is an
// fp32 number comes out as that number.  The product alone is off by a unit for
// 896, 1792, 3584 ... columns: rows of one value were not 0.  (A division is as
// good and longer on a row's way: 2047 x 5003 fp32 24.1 us against 21.7.)
__device__ __forceinline__ float quotient(float s, float n, float inv) {
  const float m = s * inv, c = fmaf(fmaf(-m, n, s), inv, m);
  return fabsf(m) < __int_as_float(0x7F800000) ? c : m;  // infinities stay what they are
}

__device__ __forceinline__ float both(f32x2 v) {
  float lo, hi;
  f2_split(v, lo, hi);
  return lo + hi;
}

// This thread's places for one row a slot: slot s, vector j.
template <typename T, int VEC, int NV>
struct Ring {
  static constexpr int kPlace = VEC > 1 ? 16 : 4;
  static constexpr int kRow = NV * kPlace;  // bytes of a row a thread
  uint32_t base, vec;  // shared address of slot 0, vector 0; bytes from vector to vector
  int nv;              // vectors of the thread within the row: at t, t + tpr, ...

  __device__ __forceinline__ Ring(uint32_t start, int threads, int nv_)
      : base(start + threadIdx.x * kPlace), vec(threads * kPlace), nv(nv_) {}

  // Starts the copy of this thread's values of a row; `at`: its first value's
  // address (any valid one if it has none).  Vectors beyond the row, and all of
  // them where `in` is false, become zeros.
  __device__ __forceinline__ void start(int slot, const T* at, int tpr, bool in) const {
    uint32_t dst = base + static_cast<uint32_t>(slot * NV) * vec;
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const bool ok = in && j < nv;
      const T* src = at + (j < nv ? j * tpr * VEC : 0);
      if constexpr (VEC > 1)
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(ok ? 16 : 0) : "memory");
      else
        asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(dst), "l"(src), "r"(ok ? 4 : 0) : "memory");
      dst += vec;
    }
  }

  // The values of a slot's row, in fp32 pairs.
  __device__ __forceinline__ void read(int slot, f32x2 (&out)[VEC * NV / 2]) const {
    uint32_t src = base + static_cast<uint32_t>(slot * NV) * vec;
    if constexpr (VEC > 1) {
#pragma unroll
      for (int j = 0; j < NV; ++j) {
        uint4 r;
        asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(r.x), "=r"(r.y), "=r"(r.z), "=r"(r.w) : "r"(src));
        const Pack<T, VEC> v = *reinterpret_cast<const Pack<T, VEC>*>(&r);
#pragma unroll
        for (int i = 0; i < VEC; i += 2) out[(j * VEC + i) / 2] = widen<T>(v.v[i], v.v[i + 1]);
        src += vec;
      }
    } else {
      float v[NV];
#pragma unroll
      for (int j = 0; j < NV; ++j) {
        asm volatile("ld.shared.f32 %0, [%1];" : "=f"(v[j]) : "r"(src));
        src += vec;
      }
#pragma unroll
      for (int j = 0; j < NV; j += 2) out[j / 2] = f2(v[j], v[j + 1]);
    }
  }
};

// A value's access straight into a register, zero where `ok` is false.
// Predicated within one statement: with a branch around the load the zero would
// meet it in a register move that waits for it, so that a row's loads came one
// after the other (8192 x 8192 bf16, gradient: 229 us against 96).
template <typename T, int VEC>
__device__ __forceinline__ void load_pack(Pack<T, VEC>& out, const T* src, bool ok) {
  if constexpr (VEC > 1) {
    uint4 r;
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %5, 0;\n\t"
        "mov.u32 %0, 0;\n\tmov.u32 %1, 0;\n\tmov.u32 %2, 0;\n\tmov.u32 %3, 0;\n\t"
        "@p ld.global.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];\n\t}"
        : "=&r"(r.x), "=&r"(r.y), "=&r"(r.z), "=&r"(r.w)
        : "l"(src), "r"(static_cast<int>(ok)));
    out = *reinterpret_cast<const Pack<T, VEC>*>(&r);
  } else if constexpr (sizeof(T) == 2) {
    uint16_t r;
    asm volatile("{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %2, 0;\n\tmov.u16 %0, 0;\n\t@p ld.global.u16 %0, [%1];\n\t}"
                 : "=&h"(r)
                 : "l"(src), "r"(static_cast<int>(ok)));
    out.v[0] = *reinterpret_cast<const T*>(&r);
  } else {
    uint32_t r;
    asm volatile("{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %2, 0;\n\tmov.u32 %0, 0;\n\t@p ld.global.u32 %0, [%1];\n\t}"
                 : "=&r"(r)
                 : "l"(src), "r"(static_cast<int>(ok)));
    out.v[0] = *reinterpret_cast<const T*>(&r);
  }
}

// The thread's values of a row at `at`, in registers.
template <typename T, int VEC, int NV>
struct Held {
  Pack<T, VEC> raw[NV];
  __device__ __forceinline__ void load(const T* at, int tpr, int nv) {
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      load_pack(raw[j], at, j < nv);
      at += tpr * VEC;
    }
  }
  __device__ __forceinline__ void read(f32x2 (&out)[VEC * NV / 2]) const {
#pragma unroll
    for (int k = 0; k < VEC * NV / 2; ++k)
      out[k] = widen<T>(raw[2 * k / VEC].v[2 * k % VEC], raw[(2 * k + 1) / VEC].v[(2 * k + 1) % VEC]);
  }
};

__device__ __forceinline__ void ring_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
// All but the newest `n` rows of this thread have landed.
__device__ __forceinline__ void ring_wait(int n) {
  switch (n) {
    case 0: asm volatile("cp.async.wait_group 0;" ::: "memory"); break;
    case 1: asm volatile("cp.async.wait_group 1;" ::: "memory"); break;
    case 2: asm volatile("cp.async.wait_group 2;" ::: "memory"); break;
    default: asm volatile("cp.async.wait_group 3;" ::: "memory"); break;
  }
}

// A parameter vector in shared memory, in fp32: values 4 q .. 4 q + 3 of thread
// t of a row at float4 q * tpr + t, `fill` where there is none or beyond the
// row.  Eight float4 a thread are read before the first is written: one at a
// time, a launch of few rows waited for them about 9 us.
template <typename P, int VEC, int NV>
__device__ __forceinline__ void stage_params(float* dst, const void* src, float fill, int tpr, int cols) {
  constexpr int kBatch = 8;
  const P* __restrict__ par = static_cast<const P*>(src);
  const int total = VEC * NV / 4 * tpr;
  for (int e0 = threadIdx.x; e0 < total; e0 += kBatch * blockDim.x) {
    float v[kBatch][4];
#pragma unroll
    for (int i = 0; i < kBatch; ++i) {
      const int e = e0 + i * blockDim.x, q = e / tpr, t = e - q * tpr;
#pragma unroll
      for (int h = 0; h < 4; ++h) {
        const int k = 4 * q + h, c = (t + (k / VEC) * tpr) * VEC + k % VEC;
        v[i][h] = par && e < total && c < cols ? to_f(par[c]) : fill;
      }
    }
#pragma unroll
    for (int i = 0; i < kBatch; ++i) {
      const int e = e0 + i * blockDim.x;
      if (e < total) reinterpret_cast<float4*>(dst)[e] = make_float4(v[i][0], v[i][1], v[i][2], v[i][3]);
    }
  }
}

// Without a ring: a thread's values straight from memory (anything beyond the row).
template <typename P, int VEC, int NV>
__device__ __forceinline__ void load_params(f32x2* out, const void* src, float fill, int t, int tpr, int nv) {
  const P* par = static_cast<const P*>(src);
#pragma unroll
  for (int k = 0; k < VEC * NV / 2; ++k) {
    const int j0 = 2 * k / VEC, j1 = (2 * k + 1) / VEC;
    const int c0 = j0 < nv ? (t + j0 * tpr) * VEC + 2 * k % VEC : 0, c1 = j1 < nv ? (t + j1 * tpr) * VEC + (2 * k + 1) % VEC : 0;
    out[k] = par ? widen<P>(par[c0], par[c1]) : f2(fill, fill);
  }
}

__device__ __forceinline__ void read_params(const float* src, int q, int tpr, int t, f32x2& lo, f32x2& hi) {
  const float4 v = reinterpret_cast<const float4*>(src)[q * tpr + t];
  lo = f2(v.x, v.y);
  hi = f2(v.z, v.w);
}

// The thread's values to its columns of a row.
template <typename T, int VEC, int NV>
__device__ __forceinline__ void store_row(T* row, int t, int tpr, int nv, const f32x2* v) {
  T* at = row + t * VEC;
  if constexpr (VEC > 1) {
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      Pack<T, VEC> out;
#pragma unroll
      for (int i = 0; i < VEC; i += 2) narrow<T>(v[(j * VEC + i) / 2], out.v + i);
      if (j < nv) *reinterpret_cast<Pack<T, VEC>*>(at) = out;
      at += tpr * VEC;
    }
  } else {
#pragma unroll
    for (int j = 0; j < NV; j += 2) {
      __align__(8) T out[2];
      narrow<T>(v[j / 2], out);
      if (j < nv) at[0] = out[0];
      if (j + 1 < nv) at[tpr] = out[1];
      at += 2 * tpr;
    }
  }
}

// Sums over the threads of a row (the same order in every thread).  `buf` is
// one of two sets, used in turn: a set is written again only after the barrier
// of the other one, which every thread passes after its reads.  At most 16
// warps a row.
template <int N>
__device__ __forceinline__ void group_sum(float (&v)[N], float (*buf)[32], int tpr, int g, int t) {
  const int width = tpr < 32 ? tpr : 32;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1)
    if (o < width)
#pragma unroll
      for (int k = 0; k < N; ++k) v[k] += __shfl_xor_sync(0xFFFFFFFFu, v[k], o);
  if (tpr <= 32) return;
  const int nw = tpr >> 5, first = (g * tpr) >> 5;
  if ((t & 31) == 0)
#pragma unroll
    for (int k = 0; k < N; ++k) buf[k][first + (t >> 5)] = v[k];
  named_bar(1 + g, tpr);
#pragma unroll
  for (int k = 0; k < N; ++k) {
    v[k] = (t & 15) < nw ? buf[k][first + (t & 15)] : 0.f;  // both halves of a warp hold all of them
#pragma unroll
    for (int o = 8; o > 0; o >>= 1) v[k] += __shfl_xor_sync(0xFFFFFFFFu, v[k], o);
  }
}

// R rows of a group at a time: their sums overlap, and they share the reads of
// the parameters.
template <typename T, typename P, int VEC, int NV, int R, bool RING>
__global__ void __launch_bounds__(kFwdThreads) forward_kernel(const FwdParams p, int tpr, int groups, int depth) {
  previous_kernel_done();
  constexpr int E = VEC * NV;
  __shared__ float buf[2][R][32];
  extern __shared__ __align__(16) uint8_t smem[];
  const int g = threadIdx.x / tpr, t = threadIdx.x - g * tpr;
  const long long step = static_cast<long long>(gridDim.x) * groups * R;
  const int nv = max(0, (p.cols - t * VEC + tpr * VEC - 1) / (tpr * VEC));
  const float n = static_cast<float>(p.cols), inv = 1.0f / n;
  const T* x0 = static_cast<const T*>(p.x) + (nv ? t * VEC : 0);
  const Ring<T, VEC, NV> ring(smem_u32(smem), blockDim.x, nv);
  float* wsm = reinterpret_cast<float*>(smem + static_cast<size_t>(depth) * R * blockDim.x * ring.kRow);
  float* bsm = wsm + E * tpr;
  const long long first = static_cast<long long>(blockIdx.x) * groups * R;
  long long ahead = first + g * R;  // the next rows to start, and their slot
  int head = 0;
  auto start = [&] {
#pragma unroll
    for (int i = 0; i < R; ++i) {
      const bool in = ahead + i < p.rows;
      ring.start(head * R + i, in ? x0 + (ahead + i) * p.ldx : x0, tpr, in);
    }
    ring_commit();
    ahead += step;
    if (++head == depth) head = 0;
  };
  if constexpr (RING) {
    for (int i = 1; i < depth; ++i) start();
    stage_params<P, VEC, NV>(wsm, p.weight, 1.f, tpr, p.cols);
    stage_params<P, VEC, NV>(bsm, p.bias, 0.f, tpr, p.cols);
    __syncthreads();
  }
  int slot = 0;
  for (long long base = first; base < p.rows; base += step) {
    const long long r = base + g * R;
    f32x2 x[R][E / 2], wreg[RING ? 1 : E / 2], breg[RING ? 1 : E / 2];
    Held<T, VEC, NV> held[RING ? 1 : R];
    if constexpr (RING) {
      start();
      ring_wait(depth - 1);
    } else {
#pragma unroll
      for (int i = 0; i < R; ++i) held[i].load(x0 + (r + i < p.rows ? (r + i) * p.ldx : 0), tpr, r + i < p.rows ? nv : 0);
      load_params<P, VEC, NV>(wreg, p.weight, 1.f, t, tpr, nv);
      load_params<P, VEC, NV>(breg, p.bias, 0.f, t, tpr, nv);
    }
    float s[R], q[R];
#pragma unroll
    for (int i = 0; i < R; ++i) {
      if constexpr (RING)
        ring.read(slot * R + i, x[i]);
      else
        held[i].read(x[i]);
      f32x2 a = x[i][0];
#pragma unroll
      for (int k = 1; k < E / 2; ++k) a = f2_add(a, x[i][k]);
      s[i] = both(a);
    }
    if (RING && ++slot == depth) slot = 0;
    group_sum(s, buf[0], tpr, g, t);
#pragma unroll
    for (int i = 0; i < R; ++i) {
      s[i] = quotient(s[i], n, inv);
      const f32x2 m = f2(s[i], s[i]);
      f32x2 a = f2(0.f, 0.f);
#pragma unroll
      for (int k = 0; k < E / 2; ++k) {
        if (VEC > 1) {
          if (2 * k / VEC < nv) {
            x[i][k] = f2_sub(x[i][k], m);
            a = f2_fma(x[i][k], x[i][k], a);
          }
        } else {
          float lo, hi;
          f2_split(f2_sub(x[i][k], m), lo, hi);
          x[i][k] = f2(2 * k < nv ? lo : 0.f, 2 * k + 1 < nv ? hi : 0.f);
          a = f2_fma(x[i][k], x[i][k], a);
        }
      }
      q[i] = both(a);
    }
    group_sum(q, buf[1], tpr, g, t);
    f32x2 rr[R];
#pragma unroll
    for (int i = 0; i < R; ++i) {
      const float rstd = reciprocal_root(q[i] * inv + p.eps);
      rr[i] = f2(rstd, rstd);
      if (r + i < p.rows && t == 0) {
        p.mean[r + i] = s[i];
        p.rstd[r + i] = rstd;
      }
    }
#pragma unroll
    for (int k = 0; k < E / 4; ++k) {
      f32x2 w[2], b[2];
      if constexpr (RING) {
        read_params(wsm, k, tpr, t, w[0], w[1]);
        read_params(bsm, k, tpr, t, b[0], b[1]);
      } else {
        w[0] = wreg[2 * k], w[1] = wreg[2 * k + 1];
        b[0] = breg[2 * k], b[1] = breg[2 * k + 1];
      }
#pragma unroll
      for (int i = 0; i < R; ++i)
#pragma unroll
        for (int h = 0; h < 2; ++h) x[i][2 * k + h] = f2_fma(f2_mul(x[i][2 * k + h], rr[i]), w[h], b[h]);
    }
#pragma unroll
    for (int i = 0; i < R; ++i)
      if (r + i < p.rows) store_row<T, VEC, NV>(static_cast<T*>(p.y) + (r + i) * p.ldy, t, tpr, nv, x[i]);
  }
  if (RING) ring_wait(0);
}

// SUMS: each thread also adds up its columns' dy xhat and dy over the rows of
// its group; the block's groups are added in their order at the end and the
// block writes one partial.  Values beyond the row are zeros of dy, so they
// add nothing (where mean * rstd is beyond fp32, x = 0 there would make xhat
// infinite, and 0 times that a NaN: they take the mean then); rows beyond the
// matrix have rstd 0.
template <typename T, typename P, int VEC, int NV, int R, bool SUMS, bool RING>
__global__ void __launch_bounds__(SUMS ? kBwdThreads : kFwdThreads) backward_kernel(const BwdParams p, int tpr, int groups, int depth) {
  previous_kernel_done();
  constexpr int E = VEC * NV;
  __shared__ float buf[2][2 * R][32];
  extern __shared__ __align__(16) uint8_t smem[];
  const int g = threadIdx.x / tpr, t = threadIdx.x - g * tpr;
  const long long step = static_cast<long long>(gridDim.x) * groups * R;
  const int nv = max(0, (p.cols - t * VEC + tpr * VEC - 1) / (tpr * VEC));
  const float n = static_cast<float>(p.cols), inv = 1.0f / n;
  const T* x0 = static_cast<const T*>(p.x) + (nv ? t * VEC : 0);
  const T* g0 = static_cast<const T*>(p.dy) + (nv ? t * VEC : 0);
  const Ring<T, VEC, NV> rx(smem_u32(smem), blockDim.x, nv);
  const Ring<T, VEC, NV> rg(smem_u32(smem) + depth * R * blockDim.x * rx.kRow, blockDim.x, nv);
  float* wsm = reinterpret_cast<float*>(smem + static_cast<size_t>(depth) * 2 * R * blockDim.x * rx.kRow);
  const long long first = static_cast<long long>(blockIdx.x) * groups * R;
  long long ahead = first + g * R;
  int head = 0;
  float nmean[R], nrstd[R];  // the next rows'
  auto fetch = [&](long long r) {
#pragma unroll
    for (int i = 0; i < R; ++i) {
      const long long at = r + i < p.rows ? r + i : 0;
      nmean[i] = p.mean[at];
      nrstd[i] = p.rstd[at];
    }
  };
  fetch(ahead);
  auto start = [&] {
#pragma unroll
    for (int i = 0; i < R; ++i) {
      const bool in = ahead + i < p.rows;
      rx.start(head * R + i, in ? x0 + (ahead + i) * p.ldx : x0, tpr, in);
      rg.start(head * R + i, in ? g0 + (ahead + i) * p.lddy : g0, tpr, in);
    }
    ring_commit();
    ahead += step;
    if (++head == depth) head = 0;
  };
  if constexpr (RING) {
    for (int i = 1; i < depth; ++i) start();
    stage_params<P, VEC, NV>(wsm, p.weight, 1.f, tpr, p.cols);
    __syncthreads();
  }
  f32x2 dw[SUMS ? E / 2 : 1], db[SUMS ? E / 2 : 1];
  if (SUMS)
#pragma unroll
    for (int k = 0; k < E / 2; ++k) dw[k] = db[k] = f2(0.f, 0.f);
  int turn = 0, slot = 0;
  for (long long base = first; base < p.rows; base += step) {
    const long long r = base + g * R;
    f32x2 xhat[R][E / 2], d[R][E / 2], wreg[RING ? 1 : E / 2];
    Held<T, VEC, NV> hx[RING ? 1 : R], hg[RING ? 1 : R];
    if constexpr (RING) {
      start();
    } else {
#pragma unroll
      for (int i = 0; i < R; ++i) {
        const bool ok = r + i < p.rows;
        hx[i].load(x0 + (ok ? (r + i) * p.ldx : 0), tpr, ok ? nv : 0);
        hg[i].load(g0 + (ok ? (r + i) * p.lddy : 0), tpr, ok ? nv : 0);
      }
      load_params<P, VEC, NV>(wreg, p.weight, 1.f, t, tpr, nv);
    }
    f32x2 mean[R], rr[R];
#pragma unroll
    for (int i = 0; i < R; ++i) {
      const float rstd = r + i < p.rows ? nrstd[i] : 0.f;
      mean[i] = f2(nmean[i], nmean[i]);
      rr[i] = f2(rstd, rstd);
    }
    fetch(r + step);
    if constexpr (RING) ring_wait(depth - 1);
#pragma unroll
    for (int i = 0; i < R; ++i) {
      if constexpr (RING) {
        rx.read(slot * R + i, xhat[i]);
        rg.read(slot * R + i, d[i]);
      } else {
        hx[i].read(xhat[i]);
        hg[i].read(d[i]);
      }
    }
    if (RING && ++slot == depth) slot = 0;
#pragma unroll
    for (int i = 0; i < R; ++i) {
      float m, r1;
      f2_split(mean[i], m, r1);
      f2_split(rr[i], r1, r1);
      if (!(fabsf(m * r1) < __int_as_float(0x7F800000))) {  // hardly ever: beyond the row the mean, whose xhat is 0
#pragma unroll
        for (int k = 0; k < E / 2; ++k) {
          float lo, hi;
          f2_split(xhat[i][k], lo, hi);
          xhat[i][k] = f2((VEC > 1 ? 2 * k / VEC : 2 * k) < nv ? lo : m, (VEC > 1 ? 2 * k / VEC : 2 * k + 1) < nv ? hi : m);
        }
      }
    }
    f32x2 a[R], c[R];
#pragma unroll
    for (int i = 0; i < R; ++i) a[i] = c[i] = f2(0.f, 0.f);
#pragma unroll
    for (int k = 0; k < E / 4; ++k) {
      f32x2 w[2];
      if constexpr (RING)
        read_params(wsm, k, tpr, t, w[0], w[1]);
      else
        w[0] = wreg[2 * k], w[1] = wreg[2 * k + 1];
#pragma unroll
      for (int i = 0; i < R; ++i)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const int e = 2 * k + h;
          xhat[i][e] = f2_mul(f2_sub(xhat[i][e], mean[i]), rr[i]);
          if (SUMS) {
            dw[e] = f2_fma(d[i][e], xhat[i][e], dw[e]);
            db[e] = f2_add(db[e], d[i][e]);
          }
          d[i][e] = f2_mul(d[i][e], w[h]);
          a[i] = f2_add(a[i], d[i][e]);
          c[i] = f2_fma(d[i][e], xhat[i][e], c[i]);
        }
    }
    float s[2 * R];
#pragma unroll
    for (int i = 0; i < R; ++i) {
      s[2 * i] = both(a[i]);
      s[2 * i + 1] = both(c[i]);
    }
    group_sum(s, buf[turn], tpr, g, t);
    turn ^= 1;
#pragma unroll
    for (int i = 0; i < R; ++i) {
      const float sm = quotient(s[2 * i], n, inv), sq = s[2 * i + 1] * -inv;
      const f32x2 m = f2(sm, sm), q = f2(sq, sq);
#pragma unroll
      for (int k = 0; k < E / 2; ++k) d[i][k] = f2_mul(rr[i], f2_fma(xhat[i][k], q, f2_sub(d[i][k], m)));
      if (r + i < p.rows) store_row<T, VEC, NV>(static_cast<T*>(p.dx) + (r + i) * p.lddx, t, tpr, nv, d[i]);
    }
  }
  if (RING) ring_wait(0);
  if (SUMS && p.parts) {
    float* part = reinterpret_cast<float*>(smem);  // groups * tpr * E; the ring is done with
    float* out = p.partials + static_cast<long long>(blockIdx.x) * 2 * p.cols;
    const int span = tpr * E;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      __syncthreads();
#pragma unroll
      for (int k = 0; k < E / 2; ++k) {
        float lo, hi;
        f2_split(h ? db[k] : dw[k], lo, hi);
        part[g * span + (t + (2 * k / VEC) * tpr) * VEC + 2 * k % VEC] = lo;
        part[g * span + (t + ((2 * k + 1) / VEC) * tpr) * VEC + (2 * k + 1) % VEC] = hi;
      }
      __syncthreads();
      for (int c = threadIdx.x; c < p.cols; c += blockDim.x) {
        float v = part[c];
        for (int i = 1; i < groups; ++i) v += part[i * span + c];
        out[h * p.cols + c] = v;
      }
    }
  }
}

// Values a thread, threads a row and rows a block for rows of `cols`: the
// fewest warps that hold the row with at most `max_e` values a thread, then
// the fewest values (e = 0: no block of `max_threads` holds it).
struct Shape {
  int e, tpr, groups;
};

Shape shape_of(long long rows, int cols, int sms, int max_e, int max_threads) {
  Shape s{0, 0, 0};
  if (cols > max_threads * max_e) return s;
  const int need = (cols + max_e - 1) / max_e;
  s.tpr = cols <= 64 ? 8 : cols <= 128 ? 16 : (need + 31) / 32 * 32;
  s.e = ((cols + s.tpr - 1) / s.tpr + 7) / 8 * 8;
  s.groups = max_threads / s.tpr;
  if (s.tpr > 32 && s.groups > 15) s.groups = 15;  // named barriers
  // few rows: spread them over the SMs first; whole warps a block
  while (s.groups > 1 && (rows + s.groups - 1) / s.groups < 2 * sms && (s.groups / 2) * s.tpr >= 32) s.groups /= 2;
  if (s.tpr < 32) s.groups = s.groups * s.tpr / 32 * 32 / s.tpr;
  return s;
}

// Ring slots of a block, its shared memory, and its resident blocks an SM:
// asked once for a kernel and block.
struct Fit {
  int depth, smem, blocks;
};

template <auto kernel>
cudaError_t fit_of(int threads, int slot_bytes, int other_bytes, int least_bytes, Fit* fit) {
  static thread_local int device = -1, was_threads = 0, was_slot = 0, was_other = 0;
  static thread_local Fit was;
  int dev = 0;
  cudaGetDevice(&dev);
  if (dev != device || threads != was_threads || slot_bytes != was_slot || other_bytes != was_other) {
    cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmemBudget);
    if (e != cudaSuccess) return e;
    int n = 0;
    e = cudaOccupancyMaxActiveBlocksPerMultiprocessor(&n, kernel, threads, 0);  // by registers and threads
    if (e != cudaSuccess) return e;
    if (n < 1) return cudaErrorInvalidConfiguration;
    while (n > 1 && kSmemBudget / n < other_bytes + 3 * slot_bytes) --n;
    Fit f;
    f.depth = slot_bytes ? (kSmemBudget / n - other_bytes) / slot_bytes : 1;
    if (f.depth > kMaxDepth) f.depth = kMaxDepth;
    if (f.depth < 1) return cudaErrorInvalidConfiguration;
    f.smem = f.depth * slot_bytes + other_bytes;
    if (f.smem < least_bytes) f.smem = least_bytes;
    e = cudaOccupancyMaxActiveBlocksPerMultiprocessor(&f.blocks, kernel, threads, f.smem);
    if (e != cudaSuccess) return e;
    if (f.blocks < 1) return cudaErrorInvalidConfiguration;
    was = f;
    device = dev;
    was_threads = threads;
    was_slot = slot_bytes;
    was_other = other_bytes;
  }
  *fit = was;
  return cudaSuccess;
}

bool aligned(const void* p) { return reinterpret_cast<uintptr_t>(p) % 16 == 0; }
// Rows that all start on 16 bytes.
template <typename T>
bool aligned_rows(const void* p, long long ld, long long rows) {
  return aligned(p) && (rows <= 1 || ld * sizeof(T) % 16 == 0);
}

template <typename T, typename P, int VEC, int NV, int R, bool RING>
cudaError_t forward_with(const FwdParams& p, const Shape& h, int sms, cudaStream_t s) {
  const int threads = h.tpr * h.groups;
  Fit f;
  const cudaError_t e = fit_of<forward_kernel<T, P, VEC, NV, R, RING>>(
      threads, RING ? threads * R * Ring<T, VEC, NV>::kRow : 0, RING ? 2 * VEC * NV * h.tpr * 4 : 0, 0, &f);
  if (e != cudaSuccess) return e;
  const long long want = (p.rows + h.groups * R - 1) / (h.groups * R), most = static_cast<long long>(sms) * f.blocks;
  return launch_after(forward_kernel<T, P, VEC, NV, R, RING>, static_cast<int>(want < most ? want : most), threads, f.smem, s, 1, p,
                      h.tpr, h.groups, f.depth);
}

// Rows enough for the ring: four or more a group.
bool many_rows(long long rows, const Shape& h, int sms) { return rows >= 4ll * sms * h.groups; }

// Two rows a group at once where the registers and two slots allow it (8192 x
// 8192 bf16, 32 values a thread: 57.8 us against 71.6 with one).  Rows of up to
// 24 values a thread have 96 threads at most: their slots always fit.
template <typename T, typename P, int VEC, int NV>
cudaError_t forward_as(const FwdParams& p, const Shape& h, int sms, cudaStream_t s) {
  if constexpr (VEC > 1 || sizeof(T) == 4) {
    if (many_rows(p.rows, h, sms)) {
      if constexpr (VEC > 1 && VEC * NV <= 24) {
        return forward_with<T, P, VEC, NV, 2, true>(p, h, sms, s);
      } else {
        if constexpr (VEC > 1 && sizeof(T) == 2) {
          const int slot = h.tpr * h.groups * Ring<T, VEC, NV>::kRow, params = 2 * VEC * NV * h.tpr * 4;
          if (4 * slot + params <= kSmemBudget) return forward_with<T, P, VEC, NV, 2, true>(p, h, sms, s);
        }
        return forward_with<T, P, VEC, NV, 1, true>(p, h, sms, s);
      }
    }
  }
  return forward_with<T, P, VEC, NV, 1, false>(p, h, sms, s);
}

template <typename T, typename P>
cudaError_t forward(const FwdParams& p, int sms, cudaStream_t s) {
  constexpr int V = 16 / static_cast<int>(sizeof(T));
  const bool vec = p.cols % V == 0 && aligned_rows<T>(p.x, p.ldx, p.rows) && aligned_rows<T>(p.y, p.ldy, p.rows);
  // one-value accesses leave fewer registers
  const int max_e = vec || p.cols > 24 * kFwdThreads ? kFwdE : p.cols > 16 * kFwdThreads ? 24 : 16;
  const Shape h = shape_of(p.rows, p.cols, sms, max_e, kFwdThreads);
  switch (h.e) {
    case 8: return vec ? forward_as<T, P, V, 8 / V>(p, h, sms, s) : forward_as<T, P, 1, 8>(p, h, sms, s);
    case 16: return vec ? forward_as<T, P, V, 16 / V>(p, h, sms, s) : forward_as<T, P, 1, 16>(p, h, sms, s);
    case 24: return vec ? forward_as<T, P, V, 24 / V>(p, h, sms, s) : forward_as<T, P, 1, 24>(p, h, sms, s);
    case 32: return vec ? forward_as<T, P, V, 32 / V>(p, h, sms, s) : forward_as<T, P, 1, 32>(p, h, sms, s);
  }
  const long long want = static_cast<long long>(sms) * 4;
  return launch_after(forward_loop_kernel<T, P>, static_cast<int>(p.rows < want ? p.rows : want), kLoopThreads, 0, s, 1, p);
}

// Blocks of a backward launch that also adds up the columns: as many threads
// an SM as one full block has.
int column_blocks(long long rows, const Shape& h, int sms) {
  const long long want = (rows + h.groups - 1) / h.groups;
  const long long most = static_cast<long long>(sms) * (kBwdThreads / (h.tpr * h.groups));
  return static_cast<int>(want < most ? want : most);
}

// One-value accesses leave fewer registers: 16 values a thread where they hold the row.
Shape backward_shape(long long rows, int cols, int sms, bool vec) {
  return shape_of(rows, cols, sms, vec || cols > 16 * kBwdThreads ? kBwdE : 16, kBwdThreads);
}

// Runs of rows of column_kernel: at least 64 rows, 64 of them at most.
int column_runs(long long rows) {
  const long long n = (rows + 63) / 64;
  return static_cast<int>(n < 64 ? n : 64);
}

template <typename T, typename P, int VEC, int NV, int R, bool SUMS, bool RING>
cudaError_t backward_with(const BwdParams& p, const Shape& h, int sms, cudaStream_t s) {
  const int threads = h.tpr * h.groups;
  Fit f;
  const cudaError_t e = fit_of<backward_kernel<T, P, VEC, NV, R, SUMS, RING>>(
      threads, RING ? threads * 2 * R * Ring<T, VEC, NV>::kRow : 0, RING ? VEC * NV * h.tpr * 4 : 0,
      SUMS ? threads * VEC * NV * 4 : 0, &f);
  if (e != cudaSuccess) return e;
  long long blocks = SUMS ? column_blocks(p.rows, h, sms) : p.rows;
  if (!SUMS && blocks > static_cast<long long>(sms) * f.blocks) blocks = static_cast<long long>(sms) * f.blocks;
  return launch_after(backward_kernel<T, P, VEC, NV, R, SUMS, RING>, static_cast<int>(blocks), threads, f.smem, s, 1, p, h.tpr,
                      h.groups, f.depth);
}

template <typename T, typename P, int VEC, int NV, bool SUMS>
cudaError_t backward_as(const BwdParams& p, const Shape& h, int sms, cudaStream_t s) {
  constexpr int R = VEC > 1 && VEC * NV <= 16 ? 2 : 1;  // rows a group of the ring holds at once
  if constexpr (VEC > 1)
    if (many_rows(p.rows, h, sms)) return backward_with<T, P, VEC, NV, R, SUMS, true>(p, h, sms, s);
  return backward_with<T, P, VEC, NV, 1, SUMS, false>(p, h, sms, s);
}

template <typename T, typename P>
cudaError_t backward(BwdParams p, int sms, cudaStream_t s) {
  constexpr int V = 16 / static_cast<int>(sizeof(T));
  const bool vec = p.cols % V == 0 && aligned_rows<T>(p.x, p.ldx, p.rows) && aligned_rows<T>(p.dy, p.lddy, p.rows) &&
                   aligned_rows<T>(p.dx, p.lddx, p.rows);
  Shape h = backward_shape(p.rows, p.cols, sms, vec);
  const bool held = h.e != 0;  // rows whose columns are added up on the way
  if (p.parts) p.parts = held ? column_blocks(p.rows, h, sms) : column_runs(p.rows);
  if (!held) {
    h = shape_of(p.rows, p.cols, sms, kFwdE, kFwdThreads);
    h.groups = 1;
  }
  cudaError_t e = cudaSuccess;
  if (p.rows > 0) {
    if (held && h.e == 8)
      e = vec ? backward_as<T, P, V, 8 / V, true>(p, h, sms, s) : backward_as<T, P, 1, 8, true>(p, h, sms, s);
    else if (held && h.e == 16)
      e = vec ? backward_as<T, P, V, 16 / V, true>(p, h, sms, s) : backward_as<T, P, 1, 16, true>(p, h, sms, s);
    else if (held)
      e = vec ? backward_as<T, P, V, 24 / V, true>(p, h, sms, s) : backward_as<T, P, 1, 24, true>(p, h, sms, s);
    else if (h.e == 32)  // 9217 .. 16384 columns
      e = vec ? backward_as<T, P, V, 32 / V, false>(p, h, sms, s) : backward_as<T, P, 1, 32, false>(p, h, sms, s);
    else {
      const long long want = static_cast<long long>(sms) * 4;
      e = launch_after(backward_loop_kernel<T, P>, static_cast<int>(p.rows < want ? p.rows : want), kLoopThreads, 0, s, 1, p);
    }
  }
  if (e != cudaSuccess || !(p.dweight || p.dbias)) return e;
  if (!held && p.parts > 0) {
    e = vec ? launch_after(column_kernel<T, V>, dim3((p.cols + 32 * V - 1) / (32 * V), p.parts), 256, 0, s, 1, p)
            : launch_after(column_kernel<T, 1>, dim3((p.cols + 31) / 32, p.parts), 256, 0, s, 1, p);
    if (e != cudaSuccess) return e;
  }
  return launch_after(finish_kernel<P>, (p.cols + 31) / 32, 1024, 0, s, 1, p);
}

}  // namespace

// The most that either access width needs: one partial a block where the
// columns are added up on the way, else one a run of rows.
int partial_count(long long rows, int cols, int sms) {
  int most = 0;
  for (const bool vec : {false, true}) {
    const Shape h = backward_shape(rows, cols, sms, vec);
    const int n = h.e ? column_blocks(rows, h, sms) : column_runs(rows);
    if (n > most) most = n;
  }
  return most;
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
