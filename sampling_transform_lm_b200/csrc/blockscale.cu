// sts_block_scaled_product: C[m, n] = sum_k A[m, k] B[n, k] of two matrices held
// in 8-bit floating point with a scale for each block of 128 along k:
//
//   C[m, n] = sum_kb a[m, kb] b[n, kb] ( sum_{k in block kb} A[m, k] B[n, k] )
//
// with b[n, kb] per row, or shared by 128 rows; then / tau_m, + C.
//
// The inner sums run on the tensor cores (tcgen05 kind::f8f6f4, fp32
// accumulators in tensor memory); scales differ from block to block, so each
// block's 128 x NT products leave tensor memory once and are scaled and summed
// in fp32 registers. That takes NT / 2 FMAs a thread and block beside the
// tensor cores' 2 NT clocks, so it hides behind them as long as both have
// accumulators to work on: 2 (NT = 256) or 4 of them alternate.
//
// B's rows (a head's vocabulary) are the 128 rows of the tensor core's tile and
// A's rows (tokens) its NT columns, NT = 16 .. 256:
//   - a few tokens take a narrow tile, and then the kernel only streams B;
//   - a thread owns one n and NT / 2 rows m of C, so the 32 lanes of a warp
//     write 128 (fp32) consecutive bytes of C and need no staging;
//   - b[n, kb] is a register, a[m, kb] a broadcast from shared memory, whatever
//     the strides of the scales are (4-byte asynchronous copies bring them).
//
// One CTA per SM, 320 threads:
//   warp 0      producer: TMA loads of B 128 x 128 and A NT x 128 bytes into a
//               ring (128-byte swizzle), and the block's scales into a second
//   warp 1      one thread issues 4 tcgen05.mma (K = 32 each) per block
//   warps 2..9  scale and sum; warp w reads tensor memory lanes 32 (w % 4)..
//               and one half of the columns
// Tiles are walked persistently, 16 tiles of A's rows for one of B's, so that
// B is read from L2. Where there are too few tiles for the SMs, a cluster of 2,
// 4 or 8 CTAs shares a tile: each takes a stretch of k, the sums meet in
// distributed shared memory and are added in the order of k.
#include <cooperative_groups.h>

#include "sts_device.cuh"

namespace sts {
namespace {

namespace cg = cooperative_groups;

constexpr int kThreads = 320;
constexpr int kSumWarps = 8;
constexpr int kRowsB = 128;
constexpr int kBlock = 128;  // k per scale, and bytes per row of a stage
constexpr int kGroup = 16;   // tiles of A's rows per raster group
constexpr int kScaleSlots = 8;
constexpr int kMaxSplit = 8;

template <int NT>
struct Shape {
  static constexpr int kBufs = NT == 256 ? 2 : 4;
  static constexpr uint32_t kTmemCols = NT * kBufs;
  static constexpr uint32_t kBytesB = kRowsB * kBlock;
  static constexpr uint32_t kBytesA = NT * kBlock;
  static constexpr uint32_t kStage = kBytesB + kBytesA;
  static constexpr int kStages = (int)(196608u / kStage) < 10 ? (int)(196608u / kStage) : 10;
  static constexpr uint32_t kSlot = (NT + kRowsB) * 4;
  static constexpr size_t kSmem = 1024 + (size_t)kStages * kStage + kScaleSlots * kSlot + 512;
  static_assert(kSmem <= 227 * 1024, "shared memory of one CTA");
  static_assert((size_t)kStages * kStage >= (size_t)kRowsB * NT * 4, "a split's sums fit the ring");
};

struct ProductArgs {
  int M, N, K, kb;  // kb: blocks along k
  int tiles_m, tiles_n;
  const float* a_scale;
  int64_t a_sr, a_sk;
  const float* b_scale;
  int64_t b_sr, b_sk;
  int b_shared;  // 1: one scale per 128 rows of B
  uint32_t idesc;
  const float* tau;
  void* C;
  int64_t ldc;
  int accumulate;
  int split;  // CTAs per tile (cluster size)
  int* err;
};

// D[tmem] (+)= A[smem] . B[smem]^T, 8-bit inputs, fp32 accumulate, one CTA.
__device__ __forceinline__ void umma_f8(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc,
                                        uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}\n" ::"r"(d_tmem),
      "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate)
      : "memory");
}

// Instruction descriptor, kind::f8f6f4: fp32 accumulator (bits 4-5 = 1), the
// formats of the 128-row operand in bits 7-9 and of the other in bits 10-12
// (0 e4m3, 1 e5m2), both K-major, N >> 3 in bits 17-22, M >> 4 in bits 24-28.
uint32_t idesc_f8(bool rows_e5, bool cols_e5, int M, int N) {
  return (1u << 4) | ((rows_e5 ? 1u : 0u) << 7) | ((cols_e5 ? 1u : 0u) << 10) |
         ((uint32_t)(N >> 3) << 17) | ((uint32_t)(M >> 4) << 24);
}

__device__ __forceinline__ void tmem_ld_x8(uint32_t taddr, uint32_t* r) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
        "=r"(r[7])
      : "r"(taddr));
}

__device__ __forceinline__ void tmem_ld_x16(uint32_t taddr, uint32_t* r) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, "
      "%12, %13, %14, %15}, [%16];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
        "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]),
        "=r"(r[14]), "=r"(r[15])
      : "r"(taddr));
}

template <int N>
__device__ __forceinline__ void tmem_ld(uint32_t taddr, uint32_t (&r)[N]) {
  if constexpr (N == 8)
    tmem_ld_x8(taddr, r);
  else if constexpr (N == 16)
    tmem_ld_x16(taddr, r);
  else
    tmem_ld_32x32b_x32(taddr, r);
}

// 4 bytes global -> shared, or 4 zero bytes where !live (src is not read then).
__device__ __forceinline__ void copy4(uint32_t dst, const float* src, bool live) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(dst), "l"(src),
               "r"(live ? 4 : 0)
               : "memory");
}

// Arrives on `bar` (once per thread, counted at its init) when this thread's
// copies so far have landed.
__device__ __forceinline__ void copies_arrive(uint32_t bar) {
  asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(bar) : "memory");
}

__device__ __forceinline__ void tile_coords(int t, int tiles_m, int tiles_n, int& tm, int& tn) {
  const int64_t per = (int64_t)kGroup * tiles_n;
  const int g = (int)(t / per);
  const int first = g * kGroup;
  const int gm = min(kGroup, tiles_m - first);
  const int r = (int)(t - g * per);
  tm = first + r % gm;
  tn = r / gm;
}

__device__ __forceinline__ void put(float* c, float v) { *c = v; }
__device__ __forceinline__ void put(__nv_bfloat16* c, float v) { *c = __float2bfloat16_rn(v); }

// One element of C from its finished sum.
template <typename O>
__device__ __forceinline__ void finish(const ProductArgs& p, int m, int n, float v) {
  if (p.tau) v = __fdiv_rn(v, __ldg(p.tau + m));
  O* c = static_cast<O*>(p.C) + (int64_t)m * p.ldc + n;
  if (p.accumulate) v += (float)*c;
  put(c, v);
}

template <int NT, typename O>
__global__ void __launch_bounds__(kThreads, 1)
    product_kernel(const __grid_constant__ CUtensorMap map_b,
                   const __grid_constant__ CUtensorMap map_a, const ProductArgs p) {
  using S = Shape<NT>;
  constexpr int kBufs = S::kBufs, kStages = S::kStages;
  constexpr int kHalf = NT / 2;
  constexpr int kChunk = kHalf < 32 ? kHalf : 32;
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw_s = smem_u32(smem_raw);
  uint8_t* smem = smem_raw + ((1024u - (raw_s & 1023u)) & 1023u);

  uint8_t* sB = smem;
  uint8_t* sA = sB + kStages * S::kBytesB;
  float* sS = reinterpret_cast<float*>(sA + kStages * S::kBytesA);
  uint64_t* full = reinterpret_cast<uint64_t*>(reinterpret_cast<uint8_t*>(sS) +
                                               kScaleSlots * S::kSlot);
  uint64_t* empty = full + kStages;
  uint64_t* sfull = empty + kStages;
  uint64_t* sempty = sfull + kScaleSlots;
  uint64_t* tfull = sempty + kScaleSlots;
  uint64_t* tempty = tfull + kBufs;
  uint64_t* drain = tempty + kBufs;
  uint32_t* tmem_holder = reinterpret_cast<uint32_t*>(drain + 1);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_holder + 1);

  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;
  const int tiles = p.tiles_m * p.tiles_n;
  // this CTA's stretch of k, and its first tile and tile stride
  const int part = blockIdx.x % p.split;
  const int kb0 = (int)((int64_t)p.kb * part / p.split);
  const int kb1 = (int)((int64_t)p.kb * (part + 1) / p.split);
  const int tile0 = blockIdx.x / p.split;
  const int step = gridDim.x / p.split;

  if (threadIdx.x == 0) {
    for (int s = 0; s < kStages; ++s) {
      mbar_init(smem_u32(&full[s]), 1);
      mbar_init(smem_u32(&empty[s]), 1);
    }
    for (int s = 0; s < kScaleSlots; ++s) {
      mbar_init(smem_u32(&sfull[s]), 32);
      mbar_init(smem_u32(&sempty[s]), kSumWarps);
    }
    for (int b = 0; b < kBufs; ++b) {
      mbar_init(smem_u32(&tfull[b]), 1);
      mbar_init(smem_u32(&tempty[b]), kSumWarps);
    }
    mbar_init(smem_u32(drain), 1);
    *abort_flag = 0;
    fence_barrier_init();
    fence_proxy_async_smem();
  }
  if (warp == 0 && lane == 0) {
    tma_prefetch_desc(&map_b);
    tma_prefetch_desc(&map_a);
  }
  if (warp == 1) {
    tmem_alloc(smem_u32(tmem_holder), S::kTmemCols);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem_base = *tmem_holder;

  // this thread's sums (warps 2..9): row n of the tile, kHalf columns m
  float acc[kHalf];
  const int quarter = warp & 3;
  const int half = warp >= 6 ? 1 : 0;
  int last_tm = 0, last_tn = 0;
  bool have = false;

  if (warp == 0) {
    // ------------------------------------------------------------ producer
    uint32_t stage = 0, phase = 0, slot = 0, sphase = 0;
    long long issued = 0;
    bool ok = true;
    for (int t = tile0; ok && t < tiles; t += step) {
      int tm, tn;
      tile_coords(t, p.tiles_m, p.tiles_n, tm, tn);
      for (int kb = kb0; kb < kb1; ++kb) {
        if (!mbar_wait(smem_u32(&empty[stage]), phase ^ 1u, abort_flag, p.err)) {
          ok = false;
          break;
        }
        if (lane == 0) {
          const uint32_t fb = smem_u32(&full[stage]);
          mbar_arrive_expect_tx(fb, S::kStage);
          tma_load_2d(smem_u32(sB + stage * S::kBytesB), &map_b, fb, kb * kBlock, tn * kRowsB);
          tma_load_2d(smem_u32(sA + stage * S::kBytesA), &map_a, fb, kb * kBlock, tm * NT);
        }
        __syncwarp();
        ++issued;
        if (++stage == kStages) {
          stage = 0;
          phase ^= 1u;
        }
        if (!mbar_wait(smem_u32(&sempty[slot]), sphase ^ 1u, abort_flag, p.err)) {
          ok = false;
          break;
        }
        const uint32_t dst = smem_u32(sS) + slot * S::kSlot;
#pragma unroll
        for (int i = 0; i < (NT + 31) / 32; ++i) {
          const int j = i * 32 + lane, m = tm * NT + j;
          if (j < NT) {
            const bool live = m < p.M;
            copy4(dst + j * 4, p.a_scale + (live ? m * p.a_sr + kb * p.a_sk : 0), live);
          }
        }
        if (p.b_shared) {
          if (lane == 0) copy4(dst + NT * 4, p.b_scale + tn * p.b_sr + kb * p.b_sk, true);
        } else {
#pragma unroll
          for (int i = 0; i < kRowsB / 32; ++i) {
            const int j = i * 32 + lane, n = tn * kRowsB + j;
            const bool live = n < p.N;
            copy4(dst + (NT + j) * 4, p.b_scale + (live ? n * p.b_sr + kb * p.b_sk : 0), live);
          }
        }
        copies_arrive(smem_u32(&sfull[slot]));
        if (++slot == kScaleSlots) {
          slot = 0;
          sphase ^= 1u;
        }
      }
    }
    // Our own loads must have landed before the CTA may exit.
    asm volatile("cp.async.wait_all;" ::: "memory");
    if (lane == 0) {
      for (int s = 0; s < kStages; ++s) {
        if (issued > s) {
          const long long last = ((issued - 1 - s) / kStages) * kStages + s;
          mbar_wait_drain(smem_u32(&full[s]), (uint32_t)((last / kStages) & 1));
        }
      }
    }
    __syncwarp();
  } else if (warp == 1) {
    // ------------------------------------------------------------ MMA issuer
    uint32_t stage = 0, phase = 0, buf = 0, bphase = 0;
    bool ok = true;
    for (int t = tile0; ok && t < tiles; t += step) {
      for (int kb = kb0; kb < kb1; ++kb) {
        if (!mbar_wait(smem_u32(&tempty[buf]), bphase ^ 1u, abort_flag, p.err) ||
            !mbar_wait(smem_u32(&full[stage]), phase, abort_flag, p.err)) {
          ok = false;
          break;
        }
        tc_fence_after();
        if (lane == 0) {
          const uint32_t rows = smem_u32(sB + stage * S::kBytesB);
          const uint32_t cols = smem_u32(sA + stage * S::kBytesA);
#pragma unroll
          for (int kk = 0; kk < kBlock / 32; ++kk)
            umma_f8(tmem_base + buf * NT, desc_kmajor_sw128(rows + kk * 32),
                    desc_kmajor_sw128(cols + kk * 32), p.idesc, kk != 0 ? 1u : 0u);
          umma_commit(smem_u32(&empty[stage]));
          umma_commit(smem_u32(&tfull[buf]));
        }
        __syncwarp();
        if (++stage == kStages) {
          stage = 0;
          phase ^= 1u;
        }
        if (++buf == kBufs) {
          buf = 0;
          bphase ^= 1u;
        }
      }
    }
    // Every MMA this thread issued must be complete before TMEM is freed.
    if (lane == 0) {
      umma_commit(smem_u32(drain));
      mbar_wait_drain(smem_u32(drain), 0);
    }
    __syncwarp();
  } else {
    // ------------------------------------------------------------ scale and sum
    uint32_t slot = 0, sphase = 0, buf = 0, bphase = 0;
    bool ok = true;
    for (int t = tile0; ok && t < tiles; t += step) {
      int tm, tn;
      tile_coords(t, p.tiles_m, p.tiles_n, tm, tn);
#pragma unroll
      for (int j = 0; j < kHalf; ++j) acc[j] = 0.f;
      for (int kb = kb0; kb < kb1; ++kb) {
        if (!mbar_wait(smem_u32(&sfull[slot]), sphase, abort_flag, p.err) ||
            !mbar_wait(smem_u32(&tfull[buf]), bphase, abort_flag, p.err)) {
          ok = false;
          break;
        }
        tc_fence_after();
        const float* sa = sS + slot * (S::kSlot / 4) + half * kHalf;
        const float* sb = sS + slot * (S::kSlot / 4) + NT;
        const float b = sb[p.b_shared ? 0 : quarter * 32 + lane];
        const uint32_t taddr = tmem_base + ((uint32_t)(quarter * 32) << 16) + buf * NT + half * kHalf;
#pragma unroll
        for (int c0 = 0; c0 < kHalf; c0 += kChunk) {
          uint32_t r[kChunk];
          tmem_ld<kChunk>(taddr + c0, r);
          tmem_ld_wait();
#pragma unroll
          for (int j = 0; j < kChunk; j += 4) {
            const float4 a = *reinterpret_cast<const float4*>(sa + c0 + j);
            acc[c0 + j] = fmaf(__uint_as_float(r[j]), a.x * b, acc[c0 + j]);
            acc[c0 + j + 1] = fmaf(__uint_as_float(r[j + 1]), a.y * b, acc[c0 + j + 1]);
            acc[c0 + j + 2] = fmaf(__uint_as_float(r[j + 2]), a.z * b, acc[c0 + j + 2]);
            acc[c0 + j + 3] = fmaf(__uint_as_float(r[j + 3]), a.w * b, acc[c0 + j + 3]);
          }
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) {
          mbar_arrive(smem_u32(&tempty[buf]));
          mbar_arrive(smem_u32(&sempty[slot]));
        }
        if (++slot == kScaleSlots) {
          slot = 0;
          sphase ^= 1u;
        }
        if (++buf == kBufs) {
          buf = 0;
          bphase ^= 1u;
        }
      }
      if (!ok) break;
      if (p.split == 1) {
        const int n = tn * kRowsB + quarter * 32 + lane;
        const int m0 = tm * NT + half * kHalf;
        if (n < p.N) {
#pragma unroll
          for (int j = 0; j < kHalf; ++j)
            if (m0 + j < p.M) finish<O>(p, m0 + j, n, acc[j]);
        }
      } else {
        last_tm = tm;
        last_tn = tn;
        have = true;
      }
    }
  }

  if (p.split > 1) {
    // One tile per cluster. Every stage has been read by now (the sums wait for
    // the last MMA), so the ring holds the sums: [column][row of the tile].
    __syncthreads();
    float* sums = reinterpret_cast<float*>(smem);
    if (warp >= 2 && have) {
#pragma unroll
      for (int j = 0; j < kHalf; ++j)
        sums[(half * kHalf + j) * kRowsB + quarter * 32 + lane] = acc[j];
    }
    cg::cluster_group cluster = cg::this_cluster();
    cluster.sync();
    if (warp >= 2 && have) {
      const int c1 = NT / p.split * (part + 1);
      const int n = last_tn * kRowsB + quarter * 32 + lane;
      for (int j = NT / p.split * part + half; j < c1; j += 2) {
        const int m = last_tm * NT + j;
        if (m >= p.M) break;
        float v = 0.f;
        for (int q = 0; q < p.split; ++q)
          v += cluster.map_shared_rank(sums, q)[j * kRowsB + quarter * 32 + lane];
        if (n < p.N) finish<O>(p, m, n, v);
      }
    }
    cluster.sync();
  }
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem_base, S::kTmemCols);
  }
}

template <int NT, typename O>
cudaError_t launch(const CUtensorMap& mb, const CUtensorMap& ma, const ProductArgs& p, int grid,
                   cudaStream_t st) {
  auto kern = product_kernel<NT, O>;
  cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                       (int)Shape<NT>::kSmem);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3((unsigned)grid);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = Shape<NT>::kSmem;
  cfg.stream = st;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeClusterDimension;
  at[0].val.clusterDim.x = (unsigned)p.split;
  at[0].val.clusterDim.y = 1;
  at[0].val.clusterDim.z = 1;
  cfg.attrs = at;
  cfg.numAttrs = p.split > 1 ? 1 : 0;
  e = cudaLaunchKernelEx(&cfg, kern, mb, ma, p);
  const cudaError_t last = cudaGetLastError();
  return e != cudaSuccess ? e : last;
}

template <int NT>
cudaError_t launch_out(bool bf16, const CUtensorMap& mb, const CUtensorMap& ma,
                       const ProductArgs& p, int grid, cudaStream_t st) {
  return bf16 ? launch<NT, __nv_bfloat16>(mb, ma, p, grid, st)
              : launch<NT, float>(mb, ma, p, grid, st);
}

constexpr int64_t kMost = (int64_t(1) << 31) - 1024;

sts_status check_operand(const sts_block_operand* o, int64_t K, bool rows_only) {
  if (!o) return STS_ERR_NULL;
  if (o->dtype != STS_DTYPE_E4M3 && o->dtype != STS_DTYPE_E5M2) return STS_ERR_DTYPE;
  if (o->rows < 0 || o->rows > kMost) return STS_ERR_SHAPE;
  if (o->block_rows != 1 && (rows_only || o->block_rows != kRowsB)) return STS_ERR_SHAPE;
  if (o->scale_stride_r < 0 || o->scale_stride_k < 0) return STS_ERR_SHAPE;
  if (o->rows == 0) return STS_OK;
  if (!o->q || !o->scale) return STS_ERR_NULL;
  // TMA: 16-byte rows from a 16-byte boundary
  if ((reinterpret_cast<uintptr_t>(o->q) & 15u) != 0 || o->ld < K || o->ld % 16 != 0 ||
      o->ld >= (int64_t(1) << 40))
    return STS_ERR_SHAPE;
  if ((reinterpret_cast<uintptr_t>(o->scale) & 3u) != 0) return STS_ERR_SHAPE;
  return STS_OK;
}

}  // namespace
}  // namespace sts

using namespace sts;

extern "C" sts_status sts_block_scaled_product(const sts_block_operand* A,
                                               const sts_block_operand* B, int64_t K,
                                               const float* temperature, void* C, int c_dtype,
                                               int64_t ldc, int accumulate, void* ws,
                                               size_t ws_bytes, sts_stream_t stream) {
  if (K < 1 || K > kMost) return STS_ERR_SHAPE;
  if (c_dtype != STS_DTYPE_F32 && c_dtype != STS_DTYPE_BF16) return STS_ERR_DTYPE;
  if (accumulate && c_dtype != STS_DTYPE_F32) return STS_ERR_DTYPE;
  sts_status s = check_operand(A, K, true);
  if (s != STS_OK) return s;
  s = check_operand(B, K, false);
  if (s != STS_OK) return s;
  if (A->rows > 1 && ldc < B->rows) return STS_ERR_SHAPE;
  if (ws && ((reinterpret_cast<uintptr_t>(ws) & 255u) != 0 || ws_bytes < sizeof(WsHeader)))
    return STS_ERR_WORKSPACE;
  if (A->rows == 0 || B->rows == 0) return STS_OK;
  if (!C) return STS_ERR_NULL;
  if ((reinterpret_cast<uintptr_t>(C) % (c_dtype == STS_DTYPE_F32 ? 4u : 2u)) != 0)
    return STS_ERR_SHAPE;
  int sms = 0;
  s = current_device(&sms);
  if (s != STS_OK) return s;

  const int64_t M = A->rows, N = B->rows;
  const int NT = M <= 16 ? 16 : M <= 32 ? 32 : M <= 64 ? 64 : M <= 128 ? 128 : 256;
  ProductArgs p{};
  p.M = (int)M;
  p.N = (int)N;
  p.K = (int)K;
  p.kb = (int)((K + kBlock - 1) / kBlock);
  const int64_t tiles_m = (M + NT - 1) / NT, tiles_n = (N + kRowsB - 1) / kRowsB;
  if (tiles_m * tiles_n > kMost) return STS_ERR_SHAPE;
  p.tiles_m = (int)tiles_m;
  p.tiles_n = (int)tiles_n;
  p.a_scale = A->scale;
  p.a_sr = A->scale_stride_r;
  p.a_sk = A->scale_stride_k;
  p.b_scale = B->scale;
  p.b_sr = B->scale_stride_r;
  p.b_sk = B->scale_stride_k;
  p.b_shared = B->block_rows == kRowsB ? 1 : 0;
  p.idesc = idesc_f8(B->dtype == STS_DTYPE_E5M2, A->dtype == STS_DTYPE_E5M2, kRowsB, NT);
  p.tau = temperature;
  p.C = C;
  p.ldc = ldc;
  p.accumulate = accumulate ? 1 : 0;
  const int64_t tiles = tiles_m * tiles_n;
  p.split = 1;
  while (p.split < kMaxSplit && tiles * p.split * 2 <= sms && p.kb >= p.split * 2 * 4) p.split *= 2;
  const int grid = (int)(p.split > 1 ? tiles * p.split : (tiles < sms ? tiles : sms));

  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  if (ws) {
    WsHeader* hdr = static_cast<WsHeader*>(ws);
    if (cudaMemsetAsync(&hdr->bad_row_code, 0xFF, sizeof(hdr->bad_row_code), st) != cudaSuccess ||
        cudaMemsetAsync(&hdr->err, 0, sizeof(hdr->err), st) != cudaSuccess)
      return STS_ERR_CUDA;
    p.err = &hdr->err;
  }
  CUtensorMap ma, mb;
  if (!tensor_map_2d(&mb, B->q, CU_TENSOR_MAP_DATA_TYPE_UINT8, (uint64_t)K, (uint64_t)N,
                     (uint64_t)B->ld, kBlock, kRowsB) ||
      !tensor_map_2d(&ma, A->q, CU_TENSOR_MAP_DATA_TYPE_UINT8, (uint64_t)K, (uint64_t)M,
                     (uint64_t)A->ld, kBlock, (uint32_t)NT))
    return STS_ERR_CUDA;
  const LaunchMark mark = launch_begin(STS_KERNEL_BLOCK_PRODUCT, st);
  const bool bf = c_dtype == STS_DTYPE_BF16;
  const cudaError_t e = NT == 16    ? launch_out<16>(bf, mb, ma, p, grid, st)
                        : NT == 32  ? launch_out<32>(bf, mb, ma, p, grid, st)
                        : NT == 64  ? launch_out<64>(bf, mb, ma, p, grid, st)
                        : NT == 128 ? launch_out<128>(bf, mb, ma, p, grid, st)
                                    : launch_out<256>(bf, mb, ma, p, grid, st);
  launch_end(mark, st);
  return e == cudaSuccess ? STS_OK : STS_ERR_CUDA;
}
