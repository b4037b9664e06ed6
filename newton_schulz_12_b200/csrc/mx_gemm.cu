// C = A B^T of two 4-bit microscaled matrices on the tensor cores
// (tcgen05.mma kind::mxf4, one scale byte for every 32 values along k).
//
// Small products: a CTA holds a 128 x BN tile of C in tensor memory.  Warp 0
// copies the operands' data (128-byte swizzled boxes of 128 bytes = 256 values
// along k) and their scales (512-byte tiles of 128 rows x 4 blocks, already in
// the order that tcgen05.cp wants) into a ring; one thread of warp 1 copies each
// stage's scales on to tensor memory and issues the products; four warps
// convert and store the finished tile while the next one is computed in the
// second accumulator.  Where few tiles leave SMs idle (a token's row against a
// whole weight), a cluster of CTAs shares a tile, each with a run of k, and adds
// the partial sums up through distributed shared memory in rank order.
// (Large products: namespace pair below.)
#include "common.cuh"
#include "internal.h"

#include <cuda_fp16.h>

#include <mutex>

namespace muon {
namespace mx {

namespace {

constexpr int BM = 128;
constexpr int kStageK = 256;           // values of k a stage: 128 bytes of data a row
constexpr int kThreads = 192;          // copier, issuer, four epilogue warps
constexpr int kScaleTile = 512;        // bytes: 128 rows x 4 blocks

// Where a wait that runs out in a captured launch is recorded (see workspace_status).
__device__ int g_captured_status;
__device__ int g_taken_status;  // take_captured_status: what it held
__global__ void take_status_kernel() { g_taken_status = atomicExch(&g_captured_status, 0); }

template <int BN>
struct Cfg {
  static constexpr uint32_t kABytes = BM * 128;
  static constexpr uint32_t kBBytes = BN * 128;
  static constexpr uint32_t kScaleA = 2 * kScaleTile, kScaleB = 2 * kScaleTile;  // two tiles along k
  static constexpr uint32_t kStageBytes = kABytes + kBBytes + kScaleA + kScaleB;
  static constexpr int kStages = BN == 128 ? 5 : BN == 64 ? 7 : 8;
  static constexpr uint32_t kStageRow = 64 * 4 + 16;  // staging row: 64 values, padded against bank conflicts
  static constexpr uint32_t kStagingWarp = 32 * kStageRow;
  static constexpr int kBars = 2 * kStages + 5;       // full, empty per stage; tfull, tempty x 2; drain
  static constexpr size_t kSmem = 1024 + kStages * kStageBytes + 4 * kStagingWarp + kBars * 8 + 16;
  // tensor memory columns: two accumulators, then a slot of scales for each stage
  static constexpr uint32_t kScaleCol = 2 * BN;
  static constexpr uint32_t kSlotCols = 16;           // 4 columns a tile of scales: A's two, B's two
  static_assert(kScaleCol + kStages * kSlotCols <= 512, "tensor memory");
  static_assert(kSmem <= 232448, "shared memory");
  static_assert(kStageBytes % 1024 == 0, "swizzled boxes start on 1 KiB");
  static_assert(BM * (BN + 1) * 4 <= kStages * kStageBytes, "a tile's partial sums fit the ring");
};

__device__ __forceinline__ void tma_load_2d(uint32_t dst, const void* map, uint32_t bar, int c0, int c1) {
  asm volatile(
      "cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%3, %4}], [%2];" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(bar), "r"(c0), "r"(c1)
      : "memory");
}

__device__ __forceinline__ void bulk_load(uint32_t dst, const void* src, uint32_t bytes, uint32_t bar) {
  asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(dst),
               "l"(reinterpret_cast<uint64_t>(src)), "r"(bytes), "r"(bar)
               : "memory");
}

// Descriptors as two words: only the low one (the address) changes in the issue loop.
constexpr uint32_t kOperandHi = (1024u >> 4) | (1u << 14) | (2u << 29);  // 8-row groups 1 KiB apart, 128-byte swizzle
constexpr uint32_t kOperandLo = 1u << 16;
// One tile of scales (32 rows of 16 bytes) to four columns of tensor memory,
// the same in each quarter of the lanes: row 32 j + i of the operand is byte
// group j of lane i.
constexpr uint32_t kScaleHi = (128u >> 4) | (1u << 14);  // 8-row groups of 16-byte rows, no swizzle
__device__ __forceinline__ void scales_to_tmem(uint32_t taddr, uint32_t lo) {
  asm volatile(
      "{\n\t.reg .b64 d;\n\tmov.b64 d, {%1, %2};\n\t"
      "tcgen05.cp.cta_group::1.32x128b.warpx4 [%0], d;\n\t}" ::"r"(taddr), "r"(lo), "r"(kScaleHi)
      : "memory");
}

// Instruction descriptor of kind::mxf4: E2M1 operands, power-of-two scales,
// fp32 sums, M x N; `id` is the first of the two scale bytes in a column's four.
__host__ __device__ constexpr uint32_t idesc_mxf4(int m, int n, int id) {
  return (static_cast<uint32_t>(id) << 4) | (1u << 7) | (1u << 10) | (static_cast<uint32_t>(n >> 3) << 17) |
         (1u << 23) | (static_cast<uint32_t>(m >> 7) << 27) | (static_cast<uint32_t>(id) << 29);
}

template <int BN, int ID>
__device__ __forceinline__ void mma_mxf4(uint32_t d, uint32_t a_lo, uint32_t b_lo, uint32_t sa, uint32_t sb, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t.reg .b64 a, b;\n\t"
      "setp.ne.b32 p, %6, 0;\n\t"
      "mov.b64 a, {%1, %7};\n\tmov.b64 b, {%2, %7};\n\t"
      "tcgen05.mma.cta_group::1.kind::mxf4.block_scale.scale_vec::2X [%0], a, b, %3, [%4], [%5], p;\n\t}" ::"r"(d),
      "r"(a_lo), "r"(b_lo), "r"(idesc_mxf4(BM, BN, ID)), "r"(sa), "r"(sb), "r"(accumulate), "r"(kOperandHi)
      : "memory");
}

// Pair forms: the box lands in this CTA's shared memory and is credited to the
// barrier `cbar` of the pair's leader; a product takes 128 rows of A and half of
// B's rows from each CTA, and all scales that its rows need from its own tensor
// memory.
__device__ __forceinline__ void tma_load_2d_pair(uint32_t dst, const void* map, uint32_t cbar, int c0, int c1) {
  asm volatile(
      "cp.async.bulk.tensor.2d.cta_group::2.shared::cluster.global.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%3, %4}], [%2];" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(cbar), "r"(c0), "r"(c1)
      : "memory");
}
// A warp's lane quarter of tensor memory, 8 or 16 columns from `taddr`, one word a lane and column.
__device__ __forceinline__ void tmem_st_x8(uint32_t taddr, const uint32_t* r) {
  asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"r"(taddr), "r"(r[0]),
               "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7])
               : "memory");
}
__device__ __forceinline__ void tmem_st_x16(uint32_t taddr, const uint32_t* r) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16};" ::"r"(
          taddr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]), "r"(r[10]),
      "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
      : "memory");
}
__device__ __forceinline__ void tmem_st_wait() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }
template <int ID>
__device__ __forceinline__ void mma_mxf4_pair(uint32_t d, uint32_t a_lo, uint32_t b_lo, uint32_t sa, uint32_t sb, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t.reg .b64 a, b;\n\t"
      "setp.ne.b32 p, %6, 0;\n\t"
      "mov.b64 a, {%1, %7};\n\tmov.b64 b, {%2, %7};\n\t"
      "tcgen05.mma.cta_group::2.kind::mxf4.block_scale.scale_vec::2X [%0], a, b, %3, [%4], [%5], p;\n\t}" ::"r"(d),
      "r"(a_lo), "r"(b_lo), "r"(idesc_mxf4(256, 256, ID)), "r"(sa), "r"(sb), "r"(accumulate), "r"(kOperandHi)
      : "memory");
}
// Whether the phase with this parity is complete; does not wait.
__device__ __forceinline__ bool mbar_test(uint32_t bar, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "mbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(ok)
      : "r"(bar), "r"(parity)
      : "memory");
  return ok != 0;
}
// Arrives once on the barrier at this offset in both CTAs when every product issued so far is done.
__device__ __forceinline__ void commit_both(uint32_t bar) {
  asm volatile(
      "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;" ::"r"(bar),
      "h"(static_cast<uint16_t>(3))
      : "memory");
}

template <typename T>
__device__ __forceinline__ T rounded(float v);
template <>
__device__ __forceinline__ float rounded<float>(float v) { return v; }
template <>
__device__ __forceinline__ bf16 rounded<bf16>(float v) { return __float2bfloat16_rn(v); }
template <>
__device__ __forceinline__ __half rounded<__half>(float v) { return __float2half_rn(v); }

// CTAs that share a tile of 128 x bn, bn 32 or 64: as many as find an SM and a
// stage along k each, 8 at most (16 x 4096 x 4096: 13.0 -> 6.4 us, 1 x 8192 x
// 8192: 22.2 -> 11.8 us.  Of 128 x 128 tiles the partial sums cost more than the
// split gives: 1024^3 12 us against 6).
int split_of(int m, int n, int k, int bn, int sms) {
  const long long tiles = static_cast<long long>((m + BM - 1) / BM) * ((n + bn - 1) / bn);
  const int stages = (k + kStageK - 1) / kStageK;
  int c = 1;
  while (c < 8 && tiles * c * 2 <= sms && c * 2 <= stages) c *= 2;
  return c;
}

// A warp's 32 rows x CW columns from their staging rows to C, cut at its edges.
template <typename T, int CW>
__device__ __forceinline__ void store_chunk(T* out, const ProductParams& p, const uint8_t* stg, uint32_t stg_row, long long row0,
                                            long long col0, int lane, bool vec) {
  constexpr int kVec = 16 / static_cast<int>(sizeof(T));
  if (vec && col0 + CW <= p.n) {
    constexpr int per_row = CW / kVec;
#pragma unroll
    for (int e = lane; e < 32 * per_row; e += 32) {
      const int r = e / per_row, u = e % per_row;
      if (row0 + r < p.m)
        *reinterpret_cast<uint4*>(out + (row0 + r) * p.ldo + col0 + u * kVec) =
            *reinterpret_cast<const uint4*>(stg + r * stg_row + u * 16);
    }
  } else {  // value by value, eight under way at a time
    const int rows = p.m - row0 < 32 ? static_cast<int>(p.m - row0) : 32;
    constexpr int kPer = CW / 32, kBatch = 8 / kPer;
    bool in[kPer];
#pragma unroll
    for (int k = 0; k < kPer; ++k) in[k] = col0 + lane + 32 * k < p.n;
    T* dst = out + row0 * p.ldo + col0 + lane;
    for (int r0 = 0; r0 < rows; r0 += kBatch) {
      T v[kBatch][kPer];
#pragma unroll
      for (int i = 0; i < kBatch; ++i)
#pragma unroll
        for (int k = 0; k < kPer; ++k) v[i][k] = reinterpret_cast<const T*>(stg + (r0 + i) * stg_row)[lane + 32 * k];
#pragma unroll
      for (int i = 0; i < kBatch; ++i) {
#pragma unroll
        for (int k = 0; k < kPer; ++k)
          if (r0 + i < rows && in[k]) dst[32 * k] = v[i][k];
        dst += p.ldo;
      }
    }
  }
}

// SPLIT: one tile a cluster, each CTA a run of k; else the CTAs walk over the tiles.
template <int BN, typename T, bool TRANS, bool SPLIT>
__global__ void __launch_bounds__(kThreads, 1) product_kernel(const __grid_constant__ ProductParams p) {
  previous_kernel_done();
  using C = Cfg<BN>;
  constexpr int S = C::kStages;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  uint8_t* staging = smem + S * C::kStageBytes;
  uint64_t* bars = reinterpret_cast<uint64_t*>(staging + 4 * C::kStagingWarp);
  uint32_t* tmem_holder = reinterpret_cast<uint32_t*>(bars + C::kBars);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_holder + 1);
  volatile int* stages_copied = abort_flag + 1;  // started, by the end of the copier's loop
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t bar0 = smem_u32(bars), smem0 = smem_u32(smem);
  auto full_bar = [&](int s) { return bar0 + 8u * s; };
  auto empty_bar = [&](int s) { return bar0 + 8u * (S + s); };
  auto tfull_bar = [&](int a) { return bar0 + 8u * (2 * S + a); };
  auto tempty_bar = [&](int a) { return bar0 + 8u * (2 * S + 2 + a); };
  const uint32_t drain_bar = bar0 + 8u * (2 * S + 4);

  if (threadIdx.x == 0) {
    for (int s = 0; s < S; ++s) {
      mbar_init(full_bar(s), 1);
      mbar_init(empty_bar(s), 1);
    }
    for (int a = 0; a < 2; ++a) {
      mbar_init(tfull_bar(a), 1);
      mbar_init(tempty_bar(a), 4);
    }
    mbar_init(drain_bar, 1);
    *abort_flag = 0;
    fence_barrier_init();
  }
  if (warp == 1) {
    tmem_alloc(smem_u32(tmem_holder), 512);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_holder;

  WaitCtl ctl;
  ctl.abort_flag = abort_flag;
  ctl.status = p.status ? p.status : &g_captured_status;
  ctl.timeout_ns = p.timeout_ns;
  ctl.where = 0;
  ctl.peer_abort = 0;
  const unsigned long long drain_ns = p.timeout_ns < 50000000ull ? p.timeout_ns : 50000000ull;

  const int tiles_m = (p.m + BM - 1) / BM, tiles_n = (p.n + BN - 1) / BN;
  const int tiles = tiles_m * tiles_n;
  const int kiters = (p.k + kStageK - 1) / kStageK;
  const int ktiles = (p.k + 127) / 128;  // scale tiles along k
  const int share = SPLIT ? p.split : 1, rank = SPLIT ? static_cast<int>(cluster_ctarank()) : 0;
  const int first = blockIdx.x / share, stride = gridDim.x / share;
  const int it0 = SPLIT ? kiters * rank / share : 0, it1 = SPLIT ? kiters * (rank + 1) / share : kiters;

  if (warp == 0) {
    if (lane == 0) {
      int stage = 0, copied = 0;
      uint32_t phase = 0;
      bool ok = true, withhold = p.inject == 1 && blockIdx.x == 0;
      for (int t = first; t < tiles && ok; t += stride) {
        const int tm = t % tiles_m, tn = t / tiles_m;
        const uint8_t* sa0 = static_cast<const uint8_t*>(p.a_scales) + static_cast<long long>(tm) * ktiles * kScaleTile;
        const uint8_t* sb0 = static_cast<const uint8_t*>(p.b_scales) + static_cast<long long>(tn * BN / 128) * ktiles * kScaleTile;
        for (int it = it0; it < it1; ++it) {
          if (!mbar_wait(empty_bar(stage), phase ^ 1u, ctl)) {
            ok = false;
            break;
          }
          const uint32_t sbytes = static_cast<uint32_t>(min(2, ktiles - 2 * it)) * kScaleTile;  // this stage's, along k
          mbar_arrive_expect_tx(full_bar(stage), C::kABytes + C::kBBytes + 2 * sbytes);
          ++copied;
          const uint32_t a = smem0 + stage * C::kStageBytes, b = a + C::kABytes, sa = b + C::kBBytes, sb = sa + C::kScaleA;
          if (!withhold) tma_load_2d(a, &p.a, full_bar(stage), it * 128, tm * BM);
          withhold = false;
          tma_load_2d(b, &p.b, full_bar(stage), it * 128, tn * BN);
          bulk_load(sa, sa0 + static_cast<long long>(2 * it) * kScaleTile, sbytes, full_bar(stage));
          bulk_load(sb, sb0 + static_cast<long long>(2 * it) * kScaleTile, sbytes, full_bar(stage));
          if (++stage == S) {
            stage = 0;
            phase ^= 1u;
          }
        }
      }
      *stages_copied = copied;
    }
    __syncwarp();
  } else if (warp == 1) {
    if (lane == 0) {
      int stage = 0, acc = 0;
      uint32_t phase = 0, acc_phase = 0;
      bool ok = true, ready = false;
      const uint32_t a0 = kOperandLo | (smem0 >> 4), s0 = (smem0 + C::kABytes + C::kBBytes) >> 4;
      for (int t = first; t < tiles && ok; t += stride) {
        if (!mbar_wait(tempty_bar(acc), acc_phase ^ 1u, ctl)) break;
        tc_fence_after();
        const uint32_t d = tmem + static_cast<uint32_t>(acc * BN);
        const uint32_t group = static_cast<uint32_t>((t / tiles_m) * BN % 128) / 32;  // first 32 rows of B in its scale tile
        uint32_t accumulate = 0;
        for (int it = it0; it < it1; ++it) {
          // full again: the products that last read this stage's operands and scales are done
          if (!ready && !mbar_wait(full_bar(stage), phase, ctl)) {
            ok = false;
            break;
          }
          tc_fence_after();
          const uint32_t off = static_cast<uint32_t>(stage) * (C::kStageBytes >> 4);
          const uint32_t a = a0 + off, b = a + (C::kABytes >> 4), sa = s0 + off, sb = sa + (C::kScaleA >> 4);
          const uint32_t ta = tmem + C::kScaleCol + static_cast<uint32_t>(stage) * C::kSlotCols, tb = ta + 8;
          const uint32_t empty = empty_bar(stage);
          const int left = p.k - it * kStageK;
          scales_to_tmem(ta, sa);
          scales_to_tmem(tb, sb);
          if (left > 128) {
            scales_to_tmem(ta + 4, sa + (kScaleTile >> 4));
            scales_to_tmem(tb + 4, sb + (kScaleTile >> 4));
          }
          mma_mxf4<BN, 0>(d, a, b, ta, tb + group, accumulate);
          accumulate = 1;
          if (++stage == S) {
            stage = 0;
            phase ^= 1u;
          }
          ready = mbar_test(full_bar(stage), phase);  // while the products are issued
          if (left > 64) mma_mxf4<BN, 2>(d, a + 2, b + 2, ta, tb + group, 1);
          if (left > 128) mma_mxf4<BN, 0>(d, a + 4, b + 4, ta + 4, tb + 4 + group, 1);
          if (left > 192) mma_mxf4<BN, 2>(d, a + 6, b + 6, ta + 4, tb + 4 + group, 1);
          tc_commit(empty);
        }
        if (!ok) break;
        tc_commit(tfull_bar(acc));
        if (++acc == 2) {
          acc = 0;
          acc_phase ^= 1u;
        }
      }
      tc_commit(drain_bar);
      mbar_wait_drain(drain_bar, 0, drain_ns > 1000000ull ? drain_ns : 1000000ull);
    }
    __syncwarp();
  } else if constexpr (SPLIT) {
    // this CTA's partial sums over the ring (all its products are done), in the order in which C is written
    const int quarter = warp & 3, row = quarter * 32 + lane;
    const bool ok = mbar_wait(tfull_bar(0), 0, ctl);
    if (__all_sync(0xFFFFFFFFu, ok)) {
      tc_fence_after();
      float* part = reinterpret_cast<float*>(smem) + (TRANS ? row : row * (BN + 1));
#pragma unroll
      for (int c0 = 0; c0 < BN; c0 += 32) {
        uint32_t r[32];
        tmem_ld_32x32(tmem + (static_cast<uint32_t>(quarter * 32) << 16) + static_cast<uint32_t>(c0), r);
        tmem_ld_wait();
#pragma unroll
        for (int j = 0; j < 32; ++j) part[(c0 + j) * (TRANS ? BM : 1)] = __uint_as_float(r[j]);
      }
    }
  } else {
    const int quarter = warp & 3;
    uint8_t* stg = staging + quarter * C::kStagingWarp;
    T* out = static_cast<T*>(p.out);
    constexpr int kVec = 16 / sizeof(T);
    const bool vec = (reinterpret_cast<uintptr_t>(out) % 16 == 0) && (p.ldo % kVec == 0);
    int acc = 0;
    uint32_t acc_phase = 0;
    for (int t = first; t < tiles; t += stride) {
      const int tm = t % tiles_m, tn = t / tiles_m;
      const bool ok = mbar_wait(tfull_bar(acc), acc_phase, ctl);
      if (!__all_sync(0xFFFFFFFFu, ok)) break;
      tc_fence_after();
      const long long row0 = static_cast<long long>(tm) * BM + quarter * 32;
      constexpr int CW = BN < 64 ? BN : 64;
      for (int c0 = 0; c0 < BN; c0 += CW) {
        const long long col0 = static_cast<long long>(tn) * BN + c0;
#pragma unroll
        for (int h = 0; h < CW / 32; ++h) {
          uint32_t r[32];
          tmem_ld_32x32(tmem + (static_cast<uint32_t>(quarter * 32) << 16) + static_cast<uint32_t>(acc * BN + c0 + 32 * h), r);
          tmem_ld_wait();
          if (TRANS) {
            if (row0 + lane < p.m)
              for (int j = 0; j < 32; ++j)
                if (col0 + 32 * h + j < p.n) out[(col0 + 32 * h + j) * p.ldo + row0 + lane] = rounded<T>(__uint_as_float(r[j]));
          } else {
            T* mine = reinterpret_cast<T*>(stg + lane * C::kStageRow) + 32 * h;
#pragma unroll
            for (int j = 0; j < 32; j += kVec) {
              T v[kVec];
#pragma unroll
              for (int q = 0; q < kVec; ++q) v[q] = rounded<T>(__uint_as_float(r[j + q]));
              *reinterpret_cast<uint4*>(mine + j) = *reinterpret_cast<const uint4*>(v);
            }
          }
        }
        if (!TRANS) {
          __syncwarp();
          store_chunk<T, CW>(out, p, stg, C::kStageRow, row0, col0, lane, vec);
          __syncwarp();
        }
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(tempty_bar(acc));
      if (++acc == 2) {
        acc = 0;
        acc_phase ^= 1u;
      }
    }
  }
  tc_fence_before();
  if constexpr (SPLIT) {
    cluster_sync();  // every CTA's partial sums are written
    if (warp >= 2) {
      // a CTA adds up every share-th column (TRANS) or row, the partial sums in
      // rank order; four of them, or of a row's 32 columns, a thread at a time
      T* out = static_cast<T*>(p.out);
      const int tm = first % tiles_m, tn = first / tiles_m;
      const int rows = min(static_cast<long long>(BM), p.m - static_cast<long long>(tm) * BM), cols = min(BN, p.n - tn * BN);
      const long long row0 = static_cast<long long>(tm) * BM, col0 = static_cast<long long>(tn) * BN;
      auto add_up = [&](const uint32_t (&at)[4], float (&v)[4]) {
        for (int q = 0; q < share; ++q) {
          const uint32_t base = cluster_addr(smem0, static_cast<uint32_t>(q));
          float w[4];
#pragma unroll
          for (int i = 0; i < 4; ++i) asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(w[i]) : "r"(base + at[i]));
#pragma unroll
          for (int i = 0; i < 4; ++i) v[i] = q ? v[i] + w[i] : w[i];
        }
      };
      uint32_t at[4];
      float v[4];
      if (TRANS) {
        const int row = threadIdx.x - 64;
        for (int c0 = rank; c0 < cols; c0 += 4 * share) {
#pragma unroll
          for (int i = 0; i < 4; ++i) at[i] = static_cast<uint32_t>(min(c0 + i * share, BN - 1) * BM + row) * 4u;
          add_up(at, v);
#pragma unroll
          for (int i = 0; i < 4; ++i)
            if (c0 + i * share < cols && row < rows) out[(col0 + c0 + i * share) * p.ldo + row0 + row] = rounded<T>(v[i]);
        }
      } else {
        constexpr int kPer = BN / 32, kRows = 4 / kPer;  // a row's accesses of a thread; rows at a time
        for (int r0 = rank + share * (warp - 2); r0 < rows; r0 += 4 * kRows * share) {
#pragma unroll
          for (int i = 0; i < 4; ++i)
            at[i] = static_cast<uint32_t>(min(r0 + 4 * share * (i / kPer), BM - 1) * (BN + 1) + lane + 32 * (i % kPer)) * 4u;
          add_up(at, v);
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const int r = r0 + 4 * share * (i / kPer), c = lane + 32 * (i % kPer);
            if (r < rows && c < cols) out[(row0 + r) * p.ldo + col0 + c] = rounded<T>(v[i]);
          }
        }
      }
    }
    cluster_sync();  // nobody leaves while its sums are read
  } else {
    __syncthreads();
  }
  // A wait ran out: the last stages may still be landing, also where their copier
  // had finished.
  if (threadIdx.x == 0 && *abort_flag) {
    const int copied = *stages_copied;
    for (int i = max(0, copied - S); i < copied; ++i) mbar_wait_drain(full_bar(i % S), (i / S) & 1, drain_ns);
  }
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

// ---------------------------------------------------------------------------
// Large products: a pair of CTAs holds a 256 x 256 tile of C (128 rows each), so
// that each SM reads half of B's tile from its shared memory and 8 KiB feed a
// step of 128 cycles.  Two accumulators of 256 columns and the slots of scales do
// not fit the 512 columns of tensor memory side by side: the accumulators share
// up to 128 columns, which the epilogue reads first, and the next tile starts once
// they are read.
//
// Four warps carry each stage's scales from shared to tensor memory.  tcgen05.cp
// does it, too, but takes its turn with the products: six copies a stage made
// 8192^3 take 244 us instead of 208.
// ---------------------------------------------------------------------------
namespace pair {

constexpr int BN = 256;
constexpr int kEpiWarps = 8;
constexpr int kThreads = 64 + 32 * kEpiWarps + 128;  // copier, issuer, epilogue, scales
constexpr uint32_t kABytes = BM * 128, kBBytes = BN / 2 * 128;
constexpr uint32_t kScaleA = 2 * kScaleTile, kScaleB = 4 * kScaleTile;  // a stage: two tiles along k; B's 256 rows in both CTAs
constexpr uint32_t kStageBytes = kABytes + kBBytes + kScaleA + kScaleB;
constexpr uint32_t kSlotCols = 8 + 16;
constexpr int kChunk = 64;

template <typename T>
struct Cfg {
  static constexpr int kStages = sizeof(T) == 4 ? 4 : 5;
  static constexpr uint32_t kScaleCol = 512 - kStages * kSlotCols;  // a slot of scales for each stage
  static constexpr uint32_t kAcc1 = kScaleCol - BN;                 // the second accumulator: columns kAcc1 .. 255 are shared
  static_assert(BN - kAcc1 <= 2 * kChunk, "the shared columns lie in the two chunks read first");
  static constexpr uint32_t kRow = kChunk * sizeof(T) + 16;  // staging row, padded against bank conflicts
  static constexpr int kBars = 4 * kStages + 4;              // full, empty, scales landed, scales ready; tfull x 2; early; drain
  static constexpr size_t kSmem = 1024 + kStages * kStageBytes + kEpiWarps * 32 * kRow + kBars * 8 + 16;
  static_assert(kSmem <= 232448, "shared memory");
};

// Tile t of the launch: runs of 8 tile rows, column by column, so that tiles
// that run together share operands in L2.
__device__ __forceinline__ void tile_of(int t, int tiles_m, int tiles_n, int& tm, int& tn) {
  const int run = 8 * tiles_n, r = t / run, rest = t - r * run;
  const int rows = min(8, tiles_m - 8 * r);
  tn = rest / rows;
  tm = 8 * r + rest - tn * rows;
}

template <typename T>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kThreads, 1)
    pair_kernel(const __grid_constant__ ProductParams p) {
  previous_kernel_done();
  using C = Cfg<T>;
  constexpr int S = C::kStages;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  uint8_t* staging = smem + S * kStageBytes;
  uint64_t* bars = reinterpret_cast<uint64_t*>(staging + kEpiWarps * 32 * C::kRow);
  uint32_t* tmem_holder = reinterpret_cast<uint32_t*>(bars + C::kBars);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_holder + 1);
  volatile int* stages_copied = abort_flag + 1;  // started, by the end of this CTA's copier's loop
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int rank = static_cast<int>(cluster_ctarank());
  const uint32_t peer = static_cast<uint32_t>(rank ^ 1);
  const int first = blockIdx.x >> 1, npairs = gridDim.x >> 1;
  const uint32_t bar0 = smem_u32(bars), smem0 = smem_u32(smem);
  auto full_bar = [&](int s) { return bar0 + 8u * s; };
  auto empty_bar = [&](int s) { return bar0 + 8u * (S + s); };
  auto tfull_bar = [&](int a) { return bar0 + 8u * (2 * S + a); };
  const uint32_t early_bar = bar0 + 8u * (2 * S + 2);
  const uint32_t drain_bar = bar0 + 8u * (2 * S + 3);
  auto landed_bar = [&](int s) { return bar0 + 8u * (2 * S + 4 + s); };
  auto ready_bar = [&](int s) { return bar0 + 8u * (3 * S + 4 + s); };

  if (threadIdx.x == 0) {
    for (int s = 0; s < S; ++s) {
      mbar_init(full_bar(s), 1);
      mbar_init(empty_bar(s), 1);
      mbar_init(landed_bar(s), 1);
      mbar_init(ready_bar(s), 8);  // the leader's: the scale warps of both CTAs
    }
    for (int a = 0; a < 2; ++a) mbar_init(tfull_bar(a), 1);
    mbar_init(early_bar, 2 * kEpiWarps);  // the leader's: the epilogue warps of both CTAs
    mbar_init(drain_bar, 1);
    *abort_flag = 0;
    fence_barrier_init();
  }
  if (warp == 1) {
    tmem_alloc_pair(smem_u32(tmem_holder), 512);
    tmem_relinquish_pair();
  }
  if (warp == 0 && lane == 0) {
    tma_prefetch_map(&p.a);
    tma_prefetch_map(&p.b);
    tma_prefetch_map(&p.sa);
    tma_prefetch_map(&p.sb);
  }
  tc_fence_before();
  cluster_sync();
  tc_fence_after();
  const uint32_t tmem = *tmem_holder;

  WaitCtl ctl;
  ctl.abort_flag = abort_flag;
  ctl.status = p.status ? p.status : &g_captured_status;
  ctl.timeout_ns = p.timeout_ns;
  ctl.where = 0;
  ctl.peer_abort = cluster_addr(smem_u32(const_cast<int*>(abort_flag)), peer);
  const unsigned long long drain_ns = p.timeout_ns < 50000000ull ? p.timeout_ns : 50000000ull;

  const int tiles_m = (p.m + 2 * BM - 1) / (2 * BM), tiles_n = (p.n + BN - 1) / BN;
  const int tiles = tiles_m * tiles_n;
  const int kiters = (p.k + kStageK - 1) / kStageK;

  if (warp == 0) {
    // copies, in both CTAs
    if (lane == 0) {
      int stage = 0, copied = 0;
      uint32_t phase = 0;
      bool ok = true, withhold = p.inject == 1 && blockIdx.x == 0;
      for (int t = first; t < tiles && ok; t += npairs) {
        int tm, tn;
        tile_of(t, tiles_m, tiles_n, tm, tn);
        for (int it = 0; it < kiters; ++it) {
          if (!mbar_wait(empty_bar(stage), phase ^ 1u, ctl)) {
            ok = false;
            break;
          }
          const uint32_t fbar = cluster_addr(full_bar(stage), 0);
          // what lies beyond a matrix comes as zeros and counts
          if (rank == 0) mbar_arrive_expect_tx(full_bar(stage), 2 * (kABytes + kBBytes));
          mbar_arrive_expect_tx(landed_bar(stage), kScaleA + kScaleB);
          ++copied;
          const uint32_t a = smem0 + stage * kStageBytes, b = a + kABytes, sa = b + kBBytes, sb = sa + kScaleA;
          tma_load_2d(sa, &p.sa, landed_bar(stage), it * 256, 2 * tm + rank);
          tma_load_2d(sb, &p.sb, landed_bar(stage), it * 256, 2 * tn);
          if (!withhold) tma_load_2d_pair(a, &p.a, fbar, it * 128, (2 * tm + rank) * BM);
          withhold = false;
          tma_load_2d_pair(b, &p.b, fbar, it * 128, tn * BN + rank * (BN / 2));
          if (++stage == S) {
            stage = 0;
            phase ^= 1u;
          }
        }
      }
      *stages_copied = copied;
    }
    __syncwarp();
  } else if (warp == 1) {
    if (lane == 0 && rank == 0) {
      // One thread issues everything: what it spends between two stages, the
      // tensor cores wait for.
      int stage = 0;
      uint32_t phase = 0;
      bool ok = true, ready = false;
      // this stage's operand descriptor and scales in tensor memory
      const uint32_t a0 = kOperandLo | (smem0 >> 4), t0 = tmem + C::kScaleCol;
      uint32_t a = a0, ta = t0;
      for (int t = first, k = 0; t < tiles && ok; t += npairs, ++k) {
        // the tile before last is read out and the shared columns of the last one too
        if (k > 0 && !mbar_wait(early_bar, static_cast<uint32_t>(k - 1) & 1u, ctl)) break;
        tc_fence_after();
        const uint32_t d = tmem + (k & 1 ? C::kAcc1 : 0u);
        uint32_t accumulate = 0;
        int left = p.k;
        for (int it = 0; it < kiters; ++it, left -= kStageK) {
          // full again: the products that last read this stage's operands and scales are done
          if (!ready && (!mbar_wait(full_bar(stage), phase, ctl) || !mbar_wait(ready_bar(stage), phase, ctl))) {
            ok = false;
            break;
          }
          tc_fence_after();
          const uint32_t b = a + (kABytes >> 4), tb = ta + 8, empty = empty_bar(stage);
          mma_mxf4_pair<0>(d, a, b, ta, tb, accumulate);
          accumulate = 1;
          // the next stage's addresses, and whether it is there, while the first product runs
          const bool wrap = stage + 1 == S;
          const uint32_t next_a = wrap ? a0 : a + (kStageBytes >> 4), next_ta = wrap ? t0 : ta + kSlotCols;
          stage = wrap ? 0 : stage + 1;
          phase ^= wrap ? 1u : 0u;
          ready = mbar_test(full_bar(stage), phase) && mbar_test(ready_bar(stage), phase);
          if (left > 192) {
            mma_mxf4_pair<2>(d, a + 2, b + 2, ta, tb, 1);
            mma_mxf4_pair<0>(d, a + 4, b + 4, ta + 4, tb + 8, 1);
            mma_mxf4_pair<2>(d, a + 6, b + 6, ta + 4, tb + 8, 1);
          } else {
            if (left > 64) mma_mxf4_pair<2>(d, a + 2, b + 2, ta, tb, 1);
            if (left > 128) mma_mxf4_pair<0>(d, a + 4, b + 4, ta + 4, tb + 8, 1);
          }
          commit_both(empty);
          a = next_a;
          ta = next_ta;
        }
        if (!ok) break;
        commit_both(tfull_bar(k & 1));
      }
      tc_commit_pair(drain_bar);
      mbar_wait_drain(drain_bar, 0, drain_ns > 1000000ull ? drain_ns : 1000000ull);
    }
    __syncwarp();
  } else if (warp >= 2 + kEpiWarps) {
    // scales of each stage, in both CTAs: a warp a lane quarter, all with the same words
    const uint32_t mine = static_cast<uint32_t>((warp & 3) * 32) << 16;
    int stage = 0;
    uint32_t phase = 0;
    bool ok = true;
    for (int t = first; t < tiles && ok; t += npairs) {
      for (int it = 0; it < kiters; ++it) {
        ok = __all_sync(0xFFFFFFFFu, mbar_wait(landed_bar(stage), phase, ctl));
        if (!ok) break;
        tc_fence_after();  // the products that last read this slot are done: the stage was empty
        const uint8_t* sa = smem + stage * kStageBytes + kABytes + kBBytes + 16 * lane;
        const uint8_t* sb = sa + kScaleA;
        uint32_t r[24];
        auto take = [&](int at, const uint8_t* src) { *reinterpret_cast<uint4*>(r + at) = *reinterpret_cast<const uint4*>(src); };
        take(0, sa);
        take(4, sa + kScaleTile);
        take(8, sb);  // B: 128 rows, the next 128; then the same of the second tile along k
        take(12, sb + 2 * kScaleTile);
        take(16, sb + kScaleTile);
        take(20, sb + 3 * kScaleTile);
        const uint32_t ta = tmem + mine + C::kScaleCol + static_cast<uint32_t>(stage) * kSlotCols;
        tmem_st_x8(ta, r);
        tmem_st_x16(ta + 8, r + 8);
        tmem_st_wait();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive_remote(cluster_addr(ready_bar(stage), 0));
        if (++stage == S) {
          stage = 0;
          phase ^= 1u;
        }
      }
    }
  } else {
    // two warps a lane quarter, alternate chunks, those with the shared columns first
    const int quarter = warp & 3, half = (warp - 2) >> 2;
    constexpr uint32_t kRow = C::kRow;
    uint8_t* stg = staging + (warp - 2) * 32 * kRow;
    T* out = static_cast<T*>(p.out);
    constexpr int kVec = 16 / static_cast<int>(sizeof(T));
    const bool vec = (reinterpret_cast<uintptr_t>(out) % 16 == 0) && (p.ldo % kVec == 0);
    const uint32_t early = cluster_addr(early_bar, 0);
    for (int t = first, k = 0; t < tiles; t += npairs, ++k) {
      int tm, tn;
      tile_of(t, tiles_m, tiles_n, tm, tn);
      const bool ok = mbar_wait(tfull_bar(k & 1), (k >> 1) & 1, ctl);
      if (!__all_sync(0xFFFFFFFFu, ok)) break;
      tc_fence_after();
      const long long row0 = static_cast<long long>(2 * tm + rank) * BM + quarter * 32;
#pragma unroll 1
      for (int i = half; i < BN / kChunk; i += 2) {
        const int c0 = (k & 1 ? i : BN / kChunk - 1 - i) * kChunk;
        const long long col0 = static_cast<long long>(tn) * BN + c0;
        uint32_t r[2][32];
        const uint32_t ta = tmem + (static_cast<uint32_t>(quarter * 32) << 16) + (k & 1 ? C::kAcc1 : 0u) + static_cast<uint32_t>(c0);
        tmem_ld_32x32(ta, r[0]);
        tmem_ld_32x32(ta + 32, r[1]);
        tmem_ld_wait();
        if (i == half) {  // this warp has left the tile before and the shared columns
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive_remote(early);
        }
        if (row0 >= p.m || col0 >= p.n) continue;
        T* mine = reinterpret_cast<T*>(stg + lane * kRow);
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
          for (int j = 0; j < 32; j += kVec) {
            T v[kVec];
#pragma unroll
            for (int q = 0; q < kVec; ++q) v[q] = rounded<T>(__uint_as_float(r[h][j + q]));
            *reinterpret_cast<uint4*>(mine + 32 * h + j) = *reinterpret_cast<const uint4*>(v);
          }
        __syncwarp();
        store_chunk<T, kChunk>(out, p, stg, kRow, row0, col0, lane, vec);
        __syncwarp();
      }
    }
  }
  tc_fence_before();
  cluster_sync();
  if (*abort_flag) {  // in both CTAs or in neither (whoever gives up sets both)
    // A wait ran out: the last stages may still be landing, also where their
    // copier had finished.  The leader's barriers count the operands of both;
    // stages that only the partner has started are armed for its half now.
    if (threadIdx.x == 0) {
      const int copied = *stages_copied;
      for (int i = max(0, copied - S); i < copied; ++i) {
        if (rank == 0) mbar_wait_drain(full_bar(i % S), (i / S) & 1, drain_ns);
        mbar_wait_drain(landed_bar(i % S), (i / S) & 1, drain_ns);
      }
      if (rank == 0) {
        int theirs;
        asm volatile("ld.shared::cluster.s32 %0, [%1];"
                     : "=r"(theirs)
                     : "r"(cluster_addr(smem_u32(const_cast<int*>(stages_copied)), 1)));
        for (int i = copied; i < theirs; ++i) {
          mbar_arrive_expect_tx(full_bar(i % S), kABytes + kBBytes);
          mbar_wait_drain(full_bar(i % S), (i / S) & 1, drain_ns);
        }
      }
    }
    __syncwarp();
    cluster_sync();
  }
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc_pair(tmem, 512);
  }
}

template <typename T>
cudaError_t launch(const ProductParams& p, int sms, cudaStream_t s) {
  static thread_local int configured_device = -1, resident = 0;
  int dev = 0;
  cudaGetDevice(&dev);
  if (configured_device != dev) {
    cudaError_t e = cudaFuncSetAttribute(pair_kernel<T>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                         static_cast<int>(Cfg<T>::kSmem));
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(sms / 2 * 2, 1, 1);
    cfg.blockDim = dim3(kThreads, 1, 1);
    cfg.dynamicSmemBytes = Cfg<T>::kSmem;
    e = cudaOccupancyMaxActiveClusters(&resident, pair_kernel<T>, &cfg);
    if (e != cudaSuccess) return e;
    configured_device = dev;
  }
  const long long tiles = static_cast<long long>((p.m + 2 * BM - 1) / (2 * BM)) * ((p.n + BN - 1) / BN);
  long long pairs = sms / 2;
  if (resident > 0 && pairs > resident) pairs = resident;
  if (pairs > tiles) pairs = tiles;
  return launch_after(pair_kernel<T>, static_cast<int>(2 * pairs), kThreads, Cfg<T>::kSmem, s, 1, p);
}

}  // namespace pair

template <int BN, typename T, bool TRANS, bool SPLIT>
cudaError_t launch_one(const ProductParams& p, int sms, cudaStream_t s) {
  static thread_local int configured_device = -1;
  int dev = 0;
  cudaGetDevice(&dev);
  if (configured_device != dev) {
    cudaError_t e = cudaFuncSetAttribute(product_kernel<BN, T, TRANS, SPLIT>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                         static_cast<int>(Cfg<BN>::kSmem));
    if (e != cudaSuccess) return e;
    configured_device = dev;
  }
  const long long tiles = static_cast<long long>((p.m + BM - 1) / BM) * ((p.n + BN - 1) / BN);
  const long long blocks = SPLIT ? tiles * p.split : tiles < sms ? tiles : sms;
  return launch_after(product_kernel<BN, T, TRANS, SPLIT>, static_cast<int>(blocks), kThreads, Cfg<BN>::kSmem, s,
                      SPLIT ? p.split : 1, p);
}

template <int BN, typename T, bool TRANS>
cudaError_t launch_tiles(ProductParams p, int sms, cudaStream_t s) {
  p.split = split_of(p.m, p.n, p.k, BN, sms);
  return p.split > 1 ? launch_one<BN, T, TRANS, true>(p, sms, s) : launch_one<BN, T, TRANS, false>(p, sms, s);
}

template <typename T>
cudaError_t launch_typed(const ProductParams& p, int sms, cudaStream_t s) {
  switch (product_tile_n(p.m, p.n, p.k, sms)) {
    case 256: return pair::launch<T>(p, sms, s);
    case 32: return p.transposed ? launch_tiles<32, T, true>(p, sms, s) : launch_tiles<32, T, false>(p, sms, s);
    case 64: return p.transposed ? launch_tiles<64, T, true>(p, sms, s) : launch_tiles<64, T, false>(p, sms, s);
    default: return launch_one<128, T, false, false>(p, sms, s);
  }
}

}  // namespace

// 32 or 64 where the smaller side has so few rows.  Else 256 (pairs of CTAs) or
// 128 (one CTA), whichever takes less time: measured, about 6.0 us + 0.345 us a
// wave and stage along k for pairs, 3.7 us + 0.46 us for single CTAs (512 x 512 x
// 1024: 7.4 against 5.5 us; x 8192: 17.2 against 18.4; 2048^3: 9.4 against 12.0).
int product_tile_n(int m, int n, int k, int sms) {
  if (n <= 64) return n <= 32 ? 32 : 64;
  auto waves = [](long long tiles, long long at_once) { return (tiles + at_once - 1) / at_once; };
  const long long pairs = waves(static_cast<long long>((m + 255) / 256) * ((n + 255) / 256), sms / 2);
  const long long single = waves(static_cast<long long>((m + 127) / 128) * ((n + 127) / 128), sms);
  const long long stages = (k + kStageK - 1) / kStageK;
  return 460 + 69 * pairs * stages <= 92 * single * stages ? 256 : 128;
}

cudaError_t launch_product(const ProductParams& p, int dtype, int sms, cudaStream_t s) {
  return dtype == 1 ? launch_typed<float>(p, sms, s) : dtype == 0 ? launch_typed<bf16>(p, sms, s) : launch_typed<__half>(p, sms, s);
}

// The word is taken in one step on the device, so that a wait that runs out
// meanwhile (a graph on another stream) is not lost.
cudaError_t take_captured_status(cudaStream_t s, int* value) {
  static std::mutex mu;  // one g_taken_status a device
  std::lock_guard<std::mutex> lk(mu);
  take_status_kernel<<<1, 1, 0, s>>>();
  cudaError_t e = cudaGetLastError();
  if (e == cudaSuccess) e = cudaMemcpyFromSymbolAsync(value, g_taken_status, sizeof(int), 0, cudaMemcpyDeviceToHost, s);
  return e == cudaSuccess ? cudaStreamSynchronize(s) : e;
}

}  // namespace mx
}  // namespace muon
