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

// dw and db from the partials, summed in a fixed order; 32 columns a block.
template <typename P>
__global__ void __launch_bounds__(1024) finish_kernel(const BwdParams p) {
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
// Rows held in registers.  A row is the work of `tpr` threads (8, 16 or whole
// warps) with E = VEC * NV values each, a block has `groups` such groups and
// walks over the rows, with the next row's loads issued before this one is
// worked on.  VEC values are one 16-byte access where rows, parameters and
// results are aligned for it, else VEC = 1.  What bounds it beside the bytes is
// the issue of instructions: a row's sums cost the same for 8 values a thread
// as for 32, so a row takes as few warps as hold it.
// ---------------------------------------------------------------------------
constexpr int kFwdE = 32, kFwdThreads = 512;  // values a thread, threads a block: at most
constexpr int kBwdE = 24, kBwdThreads = 384;  // with the column sums: 168 registers a thread

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

// A streamed access, zeros where `ok` is false; it bypasses L1, which keeps the
// parameters.  Predicated within one statement: with a branch around the load
// the zeros would meet it in a register move that waits for it, so that a
// row's loads came one after the other (229 us instead of 96 for the gradient
// of 8192 x 8192 bf16).
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

template <typename T, int VEC, int NV>
struct Held {
  Pack<T, VEC> raw[NV];
  // `nv` vectors of the thread lie in the row: at t, t + tpr, ...
  __device__ __forceinline__ void load(const T* row, int t, int tpr, int nv) {
    const T* at = row + t * VEC;
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      load_pack(raw[j], at, j < nv);
      at += tpr * VEC;
    }
  }
  __device__ __forceinline__ float get(int k) const { return to_f(raw[k / VEC].v[k % VEC]); }
};

// A parameter vector's values of this thread's columns, `fill` where there is none.
template <typename P, int VEC, int NV>
__device__ __forceinline__ void load_params(float* out, const void* src, float fill, int t, int tpr, int nv) {
#pragma unroll
  for (int j = 0; j < NV; ++j) {
    const int c = (t + j * tpr) * VEC;
#pragma unroll
    for (int i = 0; i < VEC; ++i) out[j * VEC + i] = fill;
    if (src && j < nv) {
      constexpr int W = VEC == 1 ? 1 : 16 / static_cast<int>(sizeof(P));  // values an access of P
#pragma unroll
      for (int i = 0; i < VEC; i += W) {
        const Pack<P, W> w = *reinterpret_cast<const Pack<P, W>*>(static_cast<const P*>(src) + c + i);
#pragma unroll
        for (int q = 0; q < (W < VEC ? W : VEC); ++q) out[j * VEC + i + q] = to_f(w.v[q]);
      }
    }
  }
}

template <typename T, int VEC>
__device__ __forceinline__ void store(T* row, int c, const float* v) {
  Pack<T, VEC> out;
#pragma unroll
  for (int i = 0; i < VEC; ++i) out.v[i] = from_f<T>(v[i]);
  *reinterpret_cast<Pack<T, VEC>*>(row + c) = out;
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

template <typename T, typename P, int VEC, int NV>
__global__ void __launch_bounds__(kFwdThreads) forward_kernel(const FwdParams p, int tpr, int groups) {
  constexpr int E = VEC * NV;
  constexpr bool kKeep = E <= 8;     // parameters stay in registers
  constexpr bool kAhead = VEC > 1;   // one-value accesses have enough in flight, and no registers to spare
  __shared__ float buf[2][1][32];
  const int g = threadIdx.x / tpr, t = threadIdx.x - g * tpr;
  const long long step = static_cast<long long>(gridDim.x) * groups;
  const int nv = max(0, (p.cols - t * VEC + tpr * VEC - 1) / (tpr * VEC));
  float w[E], b[E];
  if (kKeep) {
    load_params<P, VEC, NV>(w, p.weight, 1.f, t, tpr, nv);
    load_params<P, VEC, NV>(b, p.bias, 0.f, t, tpr, nv);
  }
  const float inv = 1.0f / p.cols;
  Held<T, VEC, NV> next;
  long long r = static_cast<long long>(blockIdx.x) * groups + g;
  if (kAhead) next.load(static_cast<const T*>(p.x) + r * p.ldx, t, tpr, r < p.rows ? nv : 0);
  for (long long base = static_cast<long long>(blockIdx.x) * groups; base < p.rows; base += step) {
    r = base + g;
    const bool ok = r < p.rows;
    if (!kAhead) next.load(static_cast<const T*>(p.x) + r * p.ldx, t, tpr, ok ? nv : 0);
    float x[E];
    float s[1] = {0.f};
#pragma unroll
    for (int k = 0; k < E; ++k) {
      x[k] = next.get(k);
      s[0] += x[k];
    }
    if (kAhead) next.load(static_cast<const T*>(p.x) + (r + step) * p.ldx, t, tpr, r + step < p.rows ? nv : 0);
    group_sum(s, buf[0], tpr, g, t);
    const float mean = s[0] * inv;
    float q[1] = {0.f};
#pragma unroll
    for (int k = 0; k < E; ++k) {
      x[k] = k / VEC < nv ? x[k] - mean : 0.f;
      q[0] = fmaf(x[k], x[k], q[0]);
    }
    group_sum(q, buf[1], tpr, g, t);
    const float rstd = 1.0f / sqrtf(q[0] * inv + p.eps);
    if (!kKeep) {
      load_params<P, VEC, NV>(w, p.weight, 1.f, t, tpr, nv);
      load_params<P, VEC, NV>(b, p.bias, 0.f, t, tpr, nv);
    }
    T* y = static_cast<T*>(p.y) + r * p.ldy;
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      float v[VEC];
#pragma unroll
      for (int i = 0; i < VEC; ++i) v[i] = fmaf(x[j * VEC + i] * rstd, w[j * VEC + i], b[j * VEC + i]);
      if (ok && j < nv) store<T, VEC>(y, (t + j * tpr) * VEC, v);
    }
    if (ok && t == 0) {
      p.mean[r] = mean;
      p.rstd[r] = rstd;
    }
  }
}

// SUMS: each thread also adds up its columns' dy xhat and dy over the rows of
// its group; the block's groups are added in their order at the end and the
// block writes one partial.
template <typename T, typename P, int VEC, int NV, bool SUMS>
__global__ void __launch_bounds__(SUMS ? kBwdThreads : kFwdThreads) backward_kernel(const BwdParams p, int tpr, int groups) {
  constexpr int E = VEC * NV;
  __shared__ float buf[2][2][32];
  extern __shared__ float part[];  // SUMS: groups * tpr * E
  const int g = threadIdx.x / tpr, t = threadIdx.x - g * tpr;
  const long long step = static_cast<long long>(gridDim.x) * groups;
  const int nv = max(0, (p.cols - t * VEC + tpr * VEC - 1) / (tpr * VEC));
  constexpr bool kKeep = E <= 8;
  constexpr bool kAhead = VEC > 1;
  float w[E], dw[SUMS ? E : 1], db[SUMS ? E : 1];
  if (kKeep) load_params<P, VEC, NV>(w, p.weight, 1.f, t, tpr, nv);
  if (SUMS)
#pragma unroll
    for (int k = 0; k < E; ++k) dw[k] = db[k] = 0.f;
  const float inv = 1.0f / p.cols;
  Held<T, VEC, NV> nx, ng;
  float nmean = 0.f, nrstd = 0.f;
  auto fetch = [&](long long r) {
    const bool ok = r < p.rows;
    nx.load(static_cast<const T*>(p.x) + r * p.ldx, t, tpr, ok ? nv : 0);
    ng.load(static_cast<const T*>(p.dy) + r * p.lddy, t, tpr, ok ? nv : 0);
    nmean = ok ? p.mean[r] : 0.f;
    nrstd = ok ? p.rstd[r] : 0.f;
  };
  if (kAhead) fetch(static_cast<long long>(blockIdx.x) * groups + g);
  int turn = 0;
  for (long long base = static_cast<long long>(blockIdx.x) * groups; base < p.rows; base += step) {
    const long long r = base + g;
    const bool ok = r < p.rows;
    if (!kAhead) fetch(r);
    const float mean = nmean, rstd = nrstd;
    float xhat[E], d[E];
    if (!kKeep) load_params<P, VEC, NV>(w, p.weight, 1.f, t, tpr, nv);
    float s[2] = {0.f, 0.f};
#pragma unroll
    for (int k = 0; k < E; ++k) {
      xhat[k] = k / VEC < nv ? (nx.get(k) - mean) * rstd : 0.f;
      d[k] = ng.get(k);
      if (SUMS) {
        dw[k] = fmaf(d[k], xhat[k], dw[k]);
        db[k] += d[k];
      }
      d[k] *= w[k];
      s[0] += d[k];
      s[1] = fmaf(d[k], xhat[k], s[1]);
    }
    if (kAhead) fetch(r + step);
    group_sum(s, buf[turn], tpr, g, t);
    turn ^= 1;
    const float m = s[0] * inv, q = s[1] * inv;
    T* dx = static_cast<T*>(p.dx) + r * p.lddx;
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      float v[VEC];
#pragma unroll
      for (int i = 0; i < VEC; ++i) {
        const int k = j * VEC + i;
        v[i] = rstd * (d[k] - m - xhat[k] * q);
      }
      if (ok && j < nv) store<T, VEC>(dx, (t + j * tpr) * VEC, v);
    }
  }
  if (SUMS && p.parts) {
    float* out = p.partials + static_cast<long long>(blockIdx.x) * 2 * p.cols;
    const int span = tpr * E;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const float* mine = h ? db : dw;
      __syncthreads();
#pragma unroll
      for (int k = 0; k < E; ++k) part[g * span + (t + (k / VEC) * tpr) * VEC + k % VEC] = mine[k];
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

// Resident blocks of a kernel (registers bound it) at this block size.
template <typename K>
int blocks_per_sm(K kernel, int threads, size_t smem) {
  static thread_local int device = -1, cached_threads = 0, cached = 0;
  static thread_local size_t cached_smem = 0;
  int dev = 0;
  cudaGetDevice(&dev);
  if (dev != device || threads != cached_threads || smem != cached_smem) {
    int n = 0;
    if (cudaOccupancyMaxActiveBlocksPerMultiprocessor(&n, kernel, threads, smem) != cudaSuccess || n < 1) n = 1;
    device = dev;
    cached_threads = threads;
    cached_smem = smem;
    cached = n;
  }
  return cached;
}

bool aligned(const void* p) { return reinterpret_cast<uintptr_t>(p) % 16 == 0; }
// Rows that all start on 16 bytes.
template <typename T>
bool aligned_rows(const void* p, long long ld, long long rows) {
  return aligned(p) && (rows <= 1 || ld * sizeof(T) % 16 == 0);
}

template <typename T, typename P, int VEC, int NV>
cudaError_t forward_as(const FwdParams& p, const Shape& h, int sms, cudaStream_t s) {
  const int threads = h.tpr * h.groups;
  const long long want = (p.rows + h.groups - 1) / h.groups;
  long long most = sms;
  if (want > most) most = static_cast<long long>(sms) * blocks_per_sm(forward_kernel<T, P, VEC, NV>, threads, 0);
  forward_kernel<T, P, VEC, NV><<<static_cast<int>(want < most ? want : most), threads, 0, s>>>(p, h.tpr, h.groups);
  return cudaGetLastError();
}

template <typename T, typename P>
cudaError_t forward(const FwdParams& p, int sms, cudaStream_t s) {
  constexpr int V = 16 / static_cast<int>(sizeof(T));
  const bool vec = p.cols % V == 0 && aligned_rows<T>(p.x, p.ldx, p.rows) && aligned_rows<T>(p.y, p.ldy, p.rows) &&
                   aligned(p.weight) && aligned(p.bias);
  const Shape h = shape_of(p.rows, p.cols, sms, vec || p.cols > kFwdE / 2 * kFwdThreads ? kFwdE : kFwdE / 2, kFwdThreads);
  switch (h.e) {
    case 8: return vec ? forward_as<T, P, V, 8 / V>(p, h, sms, s) : forward_as<T, P, 1, 8>(p, h, sms, s);
    case 16: return vec ? forward_as<T, P, V, 16 / V>(p, h, sms, s) : forward_as<T, P, 1, 16>(p, h, sms, s);
    case 24: return vec ? forward_as<T, P, V, 24 / V>(p, h, sms, s) : forward_as<T, P, 1, 24>(p, h, sms, s);
    case 32: return vec ? forward_as<T, P, V, 32 / V>(p, h, sms, s) : forward_as<T, P, 1, 32>(p, h, sms, s);
  }
  const long long want = static_cast<long long>(sms) * 4;
  forward_loop_kernel<T, P><<<static_cast<int>(p.rows < want ? p.rows : want), kLoopThreads, 0, s>>>(p);
  return cudaGetLastError();
}

// Blocks of a backward launch that also adds up the columns: as many threads
// an SM as one full block has.
int column_blocks(long long rows, const Shape& h, int sms) {
  const long long want = (rows + h.groups - 1) / h.groups;
  const long long most = static_cast<long long>(sms) * (kBwdThreads / (h.tpr * h.groups));
  return static_cast<int>(want < most ? want : most);
}

template <typename T, typename P, int VEC, int NV, bool SUMS>
cudaError_t backward_as(const BwdParams& p, const Shape& h, int sms, cudaStream_t s) {
  const int threads = h.tpr * h.groups;
  const size_t smem = SUMS ? static_cast<size_t>(threads) * VEC * NV * 4 : 0;  // 36 KiB at most
  long long blocks = SUMS ? column_blocks(p.rows, h, sms) : p.rows;
  if (!SUMS && blocks > sms) blocks = sms;
  backward_kernel<T, P, VEC, NV, SUMS><<<static_cast<int>(blocks), threads, smem, s>>>(p, h.tpr, h.groups);
  return cudaGetLastError();
}

template <typename T, typename P>
cudaError_t backward(const BwdParams& p, int sms, cudaStream_t s) {
  constexpr int V = 16 / static_cast<int>(sizeof(T));
  Shape h = shape_of(p.rows, p.cols, sms, kBwdE, kBwdThreads);
  const bool held = h.e != 0;  // rows whose columns are added up on the way
  if (!held) {
    h = shape_of(p.rows, p.cols, sms, kFwdE, kFwdThreads);
    h.groups = 1;
  }
  const bool vec = p.cols % V == 0 && aligned_rows<T>(p.x, p.ldx, p.rows) && aligned_rows<T>(p.dy, p.lddy, p.rows) &&
                   aligned_rows<T>(p.dx, p.lddx, p.rows) && aligned(p.weight);
  cudaError_t e = cudaSuccess;
  if (p.rows > 0) {
    if (held && h.e == 8)
      e = vec ? backward_as<T, P, V, 8 / V, true>(p, h, sms, s) : backward_as<T, P, 1, 8, true>(p, h, sms, s);
    else if (held && h.e == 16)
      e = vec ? backward_as<T, P, V, 16 / V, true>(p, h, sms, s) : backward_as<T, P, 1, 16, true>(p, h, sms, s);
    else if (held)
      e = vec ? backward_as<T, P, V, 24 / V, true>(p, h, sms, s) : backward_as<T, P, 1, 24, true>(p, h, sms, s);
    else if (h.e == 24)  // 9217 .. 12288 columns
      e = vec ? backward_as<T, P, V, 24 / V, false>(p, h, sms, s) : backward_as<T, P, 1, 24, false>(p, h, sms, s);
    else if (h.e == 32)
      e = vec ? backward_as<T, P, V, 32 / V, false>(p, h, sms, s) : backward_as<T, P, 1, 32, false>(p, h, sms, s);
    else {
      const long long want = static_cast<long long>(sms) * 4;
      backward_loop_kernel<T, P><<<static_cast<int>(p.rows < want ? p.rows : want), kLoopThreads, 0, s>>>(p);
      e = cudaGetLastError();
    }
  }
  if (e != cudaSuccess || !(p.dweight || p.dbias)) return e;
  if (!held && p.parts > 0) column_kernel<T><<<dim3((p.cols + 31) / 32, p.parts), 256, 0, s>>>(p);
  finish_kernel<P><<<(p.cols + 31) / 32, 1024, 0, s>>>(p);
  return cudaGetLastError();
}

}  // namespace

// One partial a block where the columns are added up with the rows held in
// registers; for wider rows runs of at least 64 rows, 64 of them at most.
int partial_count(long long rows, int cols, int sms) {
  const Shape h = shape_of(rows, cols, sms, kBwdE, kBwdThreads);
  if (h.e) return column_blocks(rows, h, sms);
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
