// sts_block_scaled_product: C[m, n] = sum_k A[m, k] B[n, k] of two matrices held
// in 8-bit floating point with a scale for each block of 128 along k:
//
//   C[m, n] = sum_kb a[m, kb] b[n, kb] ( sum_{k in block kb} A[m, k] B[n, k] )
//
// with b[n, kb] per row, or shared by 128 rows; then times 1 / tau_m, + C.
//
// The inner sums run on the tensor cores (tcgen05 kind::f8f6f4, fp32
// accumulators in tensor memory). Scales differ from block to block, so each
// block's 128 x NT products leave tensor memory once and are scaled and summed
// in fp32 registers. A thread's row is a lane of tensor memory, so a scale that
// belongs to the rows is one register, while one that differs from column to
// column is read from shared memory by every warp. Hence two forms:
//   wide    A's rows are the 128 lanes, B's rows the 256 columns. With b shared
//           by 128 rows a block costs a thread 64 packed FMAs; with b per row 32
//           reads of four scales and 64 packed products more. C leaves through
//           swizzled shared memory by TMA (a store or an fp32 reduction).
//   narrow  B's rows are the lanes, A's rows the NT = 16 .. 128 columns: it
//           streams B once. The 32 lanes of a warp write consecutive elements of
//           C. A tile has as many rows of B (16 to 128) as gives every SM the
//           same share of them.
//
// One CTA per SM, 384 threads:
//   warp 0       TMA loads of both operands into a ring of stages of 128 bytes
//                of k (128-byte swizzle)
//   warp 1       4 tcgen05.mma (K = 32 each) per block into one of two groups of
//                accumulators (one block a group if wide, 2 or 4 if narrow)
//   warp 2       the blocks' scales, into a ring of their own (4-byte
//                asynchronous copies: any strides)
//   warps 4..11  scale and sum; warp w reads lanes 32 (w % 4).. and one half of
//                the columns
// Tiles are walked persistently, 16 tiles of A's rows for one of B's, so that
// operands are read from L2. Where there are too few tiles for the SMs, a
// cluster of 2, 4 or 8 CTAs shares a tile: each takes a stretch of k, the sums
// meet in distributed shared memory and are added in the order of k.
//
// What bounds it. Narrow: HBM. 1 x 151,936 x 4,096 takes 93 to 97 us, 6.4 to 6.7
// TB/s; 77 x 50,021 x 2,048 43 us, 2.6 times its bytes, where three rounds of
// tiles of 16 blocks each end in a write of C. Wide: the sums. 4,096 x 152,064 x
// 5,120 takes 3.16 to 3.19 ms in a short burst at full clocks (2.0 PFLOP/s), 3.6
// to 3.7 back to back under the power cap (1.7 to 1.8), for 5,160 blocks an SM,
// 0.61 us a block in the burst. Alone, the products take 0.29 us of a block, the
// loads 0.26, both together 0.37 (they share the bandwidth of shared memory),
// reading tensor memory and handing blocks over 0.34, the FMAs 0.12 more, the
// writing of C 10 %. With a scale per row of both, 32,768 x 2,048 x 4,001 takes 435
// to 446 us in a burst, 490 to 510 back to back; that form spills 12 bytes.
// Sixteen warps of sums (96 registers), 32 columns a read (spills) and waiting by
// polling were each slower by 1 to 20 %.
#include <atomic>
#include <cstring>

#include <cooperative_groups.h>

#include "sts_device.cuh"

namespace sts {
namespace {

namespace cg = cooperative_groups;

constexpr int kThreads = 384;
constexpr int kSumWarps = 8;
constexpr int kLanes = 128;  // rows of the tensor core's tile
constexpr int kBlock = 128;  // k per scale, and bytes per row of a stage
constexpr int kGroup = 16;   // tiles of A's rows per raster group
constexpr int kMaxSplit = 8;
constexpr int kStaging = 2048;  // one of a warp's two staging buffers: 32 rows x 64 bytes

// kUniform: the columns' scales are shared by 128 of them (wide, b shared).
template <int NT, bool kWide, bool kUniform>
struct Shape {
  static_assert(!kUniform || kWide, "a uniform column scale is the wide form's");
  // blocks that change hands together: the accumulators of a group are waited
  // for, read and given back at once (a handover costs the sums some 300 clocks:
  // 1 x 2,368 x 65,536 took 174 us block by block, by fours it takes 98)
  static constexpr int kGroupBlocks = kWide ? 1 : NT == 128 ? 2 : 4;
  static constexpr int kBufs = 2;  // groups of accumulators
  static constexpr uint32_t kTmemCols = NT * kGroupBlocks * kBufs;
  static constexpr uint32_t kLaneBytes = kLanes * kBlock;
  static constexpr uint32_t kColBytes = NT * kBlock;
  static constexpr uint32_t kStage = kLaneBytes + kColBytes;
  static constexpr int kStages = kWide ? (kUniform ? 4 : 3) : (NT == 128 ? 6 : 8);
  static constexpr int kSlots = 4;  // of a group's scales
  static constexpr int kColScales = kUniform ? 4 : NT;  // floats of a block's scales beyond the lanes' 128
  static constexpr uint32_t kBlockScales = kLanes + kColScales;
  static constexpr uint32_t kSlot = kBlockScales * kGroupBlocks * 4;
  static constexpr uint32_t kStagingBytes = kWide ? kSumWarps * 2 * kStaging : 0;
  static constexpr int kBars = 2 * kStages + 2 * kSlots + 2 * kBufs + 1;
  static constexpr size_t kSmem = (size_t)kStages * kStage + kStagingBytes + kSlots * kSlot + kBars * 8 + 8 + kSumWarps * 4;
  // a split's sums: a line for each m of C (wide: a lane, narrow: a column), n
  // along it; 16 bytes more a line, against bank conflicts
  static constexpr int kLines = kWide ? kLanes : NT, kLong = kWide ? NT : kLanes;
  static constexpr int kPitch = kLong + 4;
  static_assert(kSmem <= 227 * 1024, "shared memory of one CTA");
  static_assert((size_t)kStages * kStage >= (size_t)kLines * kPitch * 4, "a split's sums fit the ring");
};

struct ProductArgs {
  int M, N, kb;         // kb: blocks along k
  int lane_n, col_n;    // rows of the two operands (lanes: A if wide, else B)
  int height;           // rows of the lanes' operand per tile (128 if wide)
  int tiles_l, tiles_c;
  const float* lane_scale;
  int64_t lane_sr, lane_sk;
  int lane_shift;       // row >> lane_shift is the row of its scale
  const float* col_scale;
  int64_t col_sr, col_sk;
  uint32_t idesc;
  const float* tau;
  void* C;
  int64_t ldc;
  int accumulate;
  int split;            // CTAs per tile (cluster size)
  int tma_cols;         // columns of C in the pieces that TMA writes (wide; 0: none)
  int give_up;          // a block that acts as if its first wait had given up, or -1
  int* err;
};

// The issuing helpers below take `mine`: every lane of the warp calls them, so
// that control flow and operands stay uniform, and the elected lane acts.
__device__ __forceinline__ uint32_t elected() {
  uint32_t e;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "elect.sync _|p, 0xFFFFFFFF;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}\n"
      : "=r"(e));
  return e;
}

// D[tmem] (+)= A[smem] . B[smem]^T over a block of 128 bytes of k: four MMAs of
// 8-bit inputs, fp32 accumulate, one CTA; the first overwrites D. A
// descriptor's low bits are the address in units of 16 bytes.
__device__ __forceinline__ void umma_block(uint32_t mine, uint32_t d_tmem, uint64_t a_desc,
                                           uint64_t b_desc, uint32_t idesc) {
  asm volatile(
      "{\n\t.reg .pred q, no, yes;\n\t.reg .b64 a1, b1, a2, b2, a3, b3;\n\t"
      "setp.ne.b32 q, %4, 0;\n\t"
      "setp.ne.b32 no, 0, 0;\n\t"
      "setp.eq.b32 yes, 0, 0;\n\t"
      "add.u64 a1, %1, 2;\n\tadd.u64 b1, %2, 2;\n\t"
      "add.u64 a2, %1, 4;\n\tadd.u64 b2, %2, 4;\n\t"
      "add.u64 a3, %1, 6;\n\tadd.u64 b3, %2, 6;\n\t"
      "@q tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, no;\n\t"
      "@q tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], a1, b1, %3, yes;\n\t"
      "@q tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], a2, b2, %3, yes;\n\t"
      "@q tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], a3, b3, %3, yes;\n\t}\n" ::"r"(d_tmem),
      "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(mine)
      : "memory");
}

// Arrives on `bar` when every tcgen05 op issued so far by the elected lane is done.
__device__ __forceinline__ void commit(uint32_t mine, uint32_t bar) {
  asm volatile(
      "{\n\t.reg .pred q;\n\tsetp.ne.b32 q, %1, 0;\n\t"
      "@q tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n\t}\n" ::"r"(bar),
      "r"(mine)
      : "memory");
}

// Two boxes into shared memory; `bar` counts their bytes.
__device__ __forceinline__ void load_stage(uint32_t mine, uint32_t bar, uint32_t bytes,
                                           uint32_t dst_l, const CUtensorMap* map_l, int32_t y_l,
                                           uint32_t dst_c, const CUtensorMap* map_c, int32_t y_c,
                                           int32_t x) {
  asm volatile(
      "{\n\t.reg .pred q;\n\tsetp.ne.b32 q, %9, 0;\n\t"
      "@q mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;\n\t"
      "@q cp.async.bulk.tensor.2d.shared::cluster.global.mbarrier::complete_tx::bytes"
      " [%2], [%3, {%8, %4}], [%0];\n\t"
      "@q cp.async.bulk.tensor.2d.shared::cluster.global.mbarrier::complete_tx::bytes"
      " [%5], [%6, {%8, %7}], [%0];\n\t}\n" ::"r"(bar),
      "r"(bytes), "r"(dst_l), "l"(reinterpret_cast<uint64_t>(map_l)), "r"(y_l), "r"(dst_c),
      "l"(reinterpret_cast<uint64_t>(map_c)), "r"(y_c), "r"(x), "r"(mine)
      : "memory");
}

// Instruction descriptor, kind::f8f6f4: fp32 accumulator (bits 4-5 = 1), the
// formats of the lanes' operand in bits 7-9 and of the columns' in bits 10-12
// (0 e4m3, 1 e5m2), both K-major, N >> 3 in bits 17-22, M >> 4 in bits 24-28.
uint32_t idesc_f8(bool rows_e5, bool cols_e5, int M, int N) {
  return (1u << 4) | ((rows_e5 ? 1u : 0u) << 7) | ((cols_e5 ? 1u : 0u) << 10) |
         ((uint32_t)(N >> 3) << 17) | ((uint32_t)(M >> 4) << 24);
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


// 32 lanes x kN consecutive columns of tensor memory; complete after tmem_wait.
template <int kN>
__device__ __forceinline__ void tmem_ld(uint32_t taddr, uint32_t (&r)[kN]) {
  static_assert(kN == 8 || kN == 16, "");
  if constexpr (kN == 8) {
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]),
                   "=r"(r[6]), "=r"(r[7])
                 : "r"(taddr));
  } else {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, "
        "%11, %12, %13, %14, %15}, [%16];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
          "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]),
          "=r"(r[14]), "=r"(r[15])
        : "r"(taddr));
  }
}

// Keeps what uses these registers below this point.
template <int kN>
__device__ __forceinline__ void tmem_tie(uint32_t (&r)[kN]) {
#pragma unroll
  for (int i = 0; i < kN; i += 8)
    asm volatile("" : "+r"(r[i]), "+r"(r[i + 1]), "+r"(r[i + 2]), "+r"(r[i + 3]), "+r"(r[i + 4]),
                 "+r"(r[i + 5]), "+r"(r[i + 6]), "+r"(r[i + 7]));
}

// Waits for this thread's loads from tensor memory.
template <int kN>
__device__ __forceinline__ void tmem_wait(uint32_t (&r)[kN]) {
  asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
  tmem_tie<kN>(r);
}

// Two fp32 in one register pair; one instruction for both, rounded each.
__device__ __forceinline__ uint64_t pair(float x, float y) {
  uint64_t p;
  asm("mov.b64 %0, {%1, %2};" : "=l"(p) : "f"(x), "f"(y));
  return p;
}
__device__ __forceinline__ uint64_t pair(uint32_t x, uint32_t y) {
  uint64_t p;
  asm("mov.b64 %0, {%1, %2};" : "=l"(p) : "r"(x), "r"(y));
  return p;
}
__device__ __forceinline__ float2 unpair(uint64_t p) {
  float2 v;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(v.x), "=f"(v.y) : "l"(p));
  return v;
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t d;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(a), "l"(b), "l"(c));
  return d;
}
__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b) {
  uint64_t d;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}

// acc += w (s, the columns' scales b where they differ), kN columns in pairs.
template <bool kUniform, int kN>
__device__ __forceinline__ void sum_columns(uint64_t* acc, const uint32_t (&w)[kN], const float4* b,
                                            uint64_t s2) {
#pragma unroll
  for (int j = 0; j < kN / 4; ++j) {
    uint64_t x = s2, y = s2;
    if constexpr (!kUniform) {
      x = mul2(pair(b[j].x, b[j].y), s2);
      y = mul2(pair(b[j].z, b[j].w), s2);
    }
    acc[2 * j] = fma2(pair(w[4 * j], w[4 * j + 1]), x, acc[2 * j]);
    acc[2 * j + 1] = fma2(pair(w[4 * j + 2], w[4 * j + 3]), y, acc[2 * j + 1]);
  }
}

// Tile t: groups of kGroup tiles of A's rows, all of B's tiles within a group.
template <bool kWide>
__device__ __forceinline__ void tile_coords(const ProductArgs& p, int t, int& tl, int& tc) {
  const int na = kWide ? p.tiles_l : p.tiles_c, nb = kWide ? p.tiles_c : p.tiles_l;
  const int64_t per = (int64_t)kGroup * nb;
  const int g = (int)(t / per);
  const int first = g * kGroup;
  const int ga = min(kGroup, na - first);
  const int r = (int)(t - g * per);
  const int ta = first + r % ga, tb = r / ga;
  tl = kWide ? ta : tb;
  tc = kWide ? tb : ta;
}

__device__ __forceinline__ void put(float* c, float v) { *c = v; }
__device__ __forceinline__ void put(__nv_bfloat16* c, float v) { *c = __float2bfloat16_rn(v); }

// One element of C from its finished sum (already over the temperature).
template <typename O>
__device__ __forceinline__ void finish(const ProductArgs& p, int m, int n, float v) {
  O* c = static_cast<O*>(p.C) + (int64_t)m * p.ldc + n;
  if (p.accumulate) v += (float)*c;
  put(c, v);
}

// NaN over rows x cols (0 or fewer: nothing) of C, by one warp.
template <typename O>
__device__ __forceinline__ void blank(O* c, int64_t ldc, int rows, int cols) {
#pragma unroll 1
  for (int m = 0; m < rows; ++m)
#pragma unroll 1
    for (int n = (int)threadIdx.x & 31; n < cols; n += 32)
      put(c + m * ldc + n, __int_as_float(0x7fc00000));
}

// 1 / tau_m, by which row m's sums are multiplied: a division an element would
// take longer than the multiplication of two blocks, and round once less.
__device__ __forceinline__ float over_tau(const ProductArgs& p, int m) {
  return p.tau ? __frcp_rn(__ldg(p.tau + m)) : 1.f;
}

// The wide form's sums may take 208 registers a thread, its other warps 64: 128 x
// 64 + 256 x 208 = 61,440 of the launch's 384 x 168 = 64,512. Each is called at
// one place by whole warpgroups, inside the branch that needs it (code that
// follows both branches is bound to the smaller number: the exchange of a split's
// sums there spilled, and took 15 us).
template <bool kWide>
__device__ __forceinline__ void give_registers() {
  if constexpr (kWide) asm volatile("setmaxnreg.dec.sync.aligned.u32 64;");
}
template <bool kWide>
__device__ __forceinline__ void take_registers() {
  if constexpr (kWide) asm volatile("setmaxnreg.inc.sync.aligned.u32 208;");
}

template <int NT, bool kWide, bool kUniform, typename O>
__global__ void __launch_bounds__(kThreads, 1)
    product_kernel(const __grid_constant__ CUtensorMap map_l,
                   const __grid_constant__ CUtensorMap map_c,
                   const __grid_constant__ CUtensorMap map_out, const ProductArgs p) {
  using S = Shape<NT, kWide, kUniform>;
  constexpr int kBufs = S::kBufs, kStages = S::kStages, kSlots = S::kSlots;
  constexpr int kHalf = NT / 2;
  constexpr int kG = S::kGroupBlocks;
  // columns in flight from tensor memory, twice (beside the sums, and the
  // columns' scales where they differ)
  constexpr int kMostChunk = kWide && !kUniform ? 8 : 16;
  constexpr int kChunk = kHalf < kMostChunk ? kHalf : kMostChunk;
  extern __shared__ __align__(1024) uint8_t smem[];

  uint8_t* sL = smem;
  uint8_t* sC = sL + kStages * S::kLaneBytes;
  uint8_t* staging = sC + kStages * S::kColBytes;
  float* sS = reinterpret_cast<float*>(staging + S::kStagingBytes);
  uint64_t* full = reinterpret_cast<uint64_t*>(reinterpret_cast<uint8_t*>(sS) + kSlots * S::kSlot);
  uint64_t* empty = full + kStages;
  uint64_t* sfull = empty + kStages;
  uint64_t* sempty = sfull + kSlots;
  uint64_t* tfull = sempty + kSlots;
  uint64_t* tempty = tfull + kBufs;
  uint64_t* drain = tempty + kBufs;
  uint32_t* tmem_holder = reinterpret_cast<uint32_t*>(drain + 1);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_holder + 1);
  int* stopped = reinterpret_cast<int*>(tmem_holder + 2);  // the tile at which a warp of sums gave up

  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;
  const int tiles = p.tiles_l * p.tiles_c;
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
    for (int s = 0; s < kSlots; ++s) {
      mbar_init(smem_u32(&sfull[s]), 32);
      mbar_init(smem_u32(&sempty[s]), kSumWarps);
    }
    for (int b = 0; b < kBufs; ++b) {
      mbar_init(smem_u32(&tfull[b]), 1);
      mbar_init(smem_u32(&tempty[b]), kSumWarps);
    }
    mbar_init(smem_u32(drain), 1);
    // the ring's swizzle needs 1,024-byte stages; without them nothing runs
    const int bad = (smem_u32(smem) & 1023u) != 0        ? (int)STS_ERR_OVERFLOW
                    : (int)blockIdx.x == p.give_up ? (int)STS_ERR_TIMEOUT
                                                   : 0;
    *abort_flag = bad != 0 ? 1 : 0;
    for (int w = 0; w < kSumWarps; ++w) stopped[w] = bad != 0 ? tile0 : tiles;
    if (bad != 0 && p.err) atomicCAS(p.err, 0, bad);
    fence_barrier_init();
    fence_proxy_async_smem();
  }
  if (warp == 0 && lane == 0) {
    tma_prefetch_desc(&map_l);
    tma_prefetch_desc(&map_c);
    if (kWide && p.tma_cols > 0) tma_prefetch_desc(&map_out);
  }
  if (warp == 1) {
    tmem_alloc(smem_u32(tmem_holder), S::kTmemCols);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem_base = *tmem_holder;
  const bool start_ok = *abort_flag == 0;

  const int quarter = warp & 3;
  const int half = warp >= 8 ? 1 : 0;

  // Warps 0 and 1 have 512 clocks (wide) for a block: their loops go through one
  // turn of the rings at a time, so that barriers, addresses and phases are
  // constants, and count blocks through the tiles' ends.
  const int mine_tiles = tile0 < tiles ? (tiles - tile0 + step - 1) / step : 0;
  const int blocks = mine_tiles * (kb1 - kb0);
  if (warp < 4) {
  give_registers<kWide>();
  if (warp == 0) {
    // ------------------------------------------------------------ operands
    const uint32_t mine = elected();
    const uint32_t bytes = (uint32_t)(p.height + NT) * kBlock;
    int t = tile0, kb = kb0, tl = 0, tc = 0;
    if (t < tiles) tile_coords<kWide>(p, t, tl, tc);
    bool ok = start_ok;
    int done = 0;
    for (uint32_t phase = 1; ok && done < blocks; phase ^= 1u) {
#pragma unroll
      for (int s = 0; s < kStages; ++s) {
        if (done >= blocks) break;
        if (!mbar_wait_soon(smem_u32(&empty[s]), phase, abort_flag, p.err)) {
          ok = false;
          break;
        }
        load_stage(mine, smem_u32(&full[s]), bytes, smem_u32(sL + s * S::kLaneBytes), &map_l,
                   tl * p.height, smem_u32(sC + s * S::kColBytes), &map_c, tc * NT, kb * kBlock);
        ++done;
        if (++kb == kb1) {
          kb = kb0;
          t += step;
          if (t < tiles) tile_coords<kWide>(p, t, tl, tc);
        }
      }
    }
    // Our own loads must have landed before the CTA may exit.
    for (int s = 0; s < kStages; ++s)
      if (done > s) mbar_wait_drain(smem_u32(&full[s]), (uint32_t)((done - 1 - s) / kStages) & 1u);
  } else if (warp == 1) {
    // ------------------------------------------------------------ MMA issuer
    const uint32_t mine = elected();
    const uint64_t rows0 = desc_kmajor_sw128(smem_u32(sL)), cols0 = desc_kmajor_sw128(smem_u32(sC));
    bool ok = start_ok;
    int done = 0;
    if constexpr (kG == 1) {
      // stages and accumulators repeat together after this many blocks
      constexpr int kTurn = kStages % kBufs == 0 ? kStages : kStages * kBufs;
      // phases at the start of a turn; within it they change as the rings wrap
      for (uint32_t fphase = 0, tphase = 1; ok && done < blocks;
           fphase ^= (kTurn / kStages) & 1, tphase ^= (kTurn / kBufs) & 1) {
#pragma unroll
        for (int i = 0; i < kTurn; ++i) {
          const int s = i % kStages, b = i % kBufs;
          if (done >= blocks) break;
          if (!mbar_wait_soon(smem_u32(&tempty[b]), tphase ^ ((i / kBufs) & 1), abort_flag, p.err) ||
              !mbar_wait_soon(smem_u32(&full[s]), fphase ^ ((i / kStages) & 1), abort_flag, p.err)) {
            ok = false;
            break;
          }
          tc_fence_after();
          umma_block(mine, tmem_base + b * NT, rows0 + s * (S::kLaneBytes >> 4),
                     cols0 + s * (S::kColBytes >> 4), p.idesc);
          commit(mine, smem_u32(&tfull[b]));
          commit(mine, smem_u32(&empty[s]));
          ++done;
        }
      }
    } else {
      uint32_t s = 0, fphase = 0, b = 0, tphase = 1;
      int kb = kb0;
      while (ok && done < blocks) {
        if (!mbar_wait_soon(smem_u32(&tempty[b]), tphase, abort_flag, p.err)) break;
        tc_fence_after();
        const int n = min(kG, kb1 - kb);  // a tile's last group may be smaller
        for (int i = 0; i < n; ++i) {
          if (!mbar_wait_soon(smem_u32(&full[s]), fphase, abort_flag, p.err)) {
            ok = false;
            break;
          }
          tc_fence_after();
          umma_block(mine, tmem_base + (b * kG + i) * NT, rows0 + s * (S::kLaneBytes >> 4),
                     cols0 + s * (S::kColBytes >> 4), p.idesc);
          commit(mine, smem_u32(&empty[s]));
          ++done;
          if (++s == (uint32_t)kStages) {
            s = 0;
            fphase ^= 1u;
          }
        }
        if (!ok) break;  // a group that is not whole is not handed over
        commit(mine, smem_u32(&tfull[b]));
        kb += n;
        if (kb == kb1) kb = kb0;
        if (++b == (uint32_t)kBufs) {
          b = 0;
          tphase ^= 1u;
        }
      }
    }
    // Every MMA this warp issued must be complete before TMEM is freed.
    commit(mine, smem_u32(drain));
    mbar_wait_drain(smem_u32(drain), 0);
  } else if (warp == 2) {
    // ------------------------------------------------------------ scales
    uint32_t slot = 0, sphase = 0;
    bool ok = start_ok;
    for (int t = tile0; ok && t < tiles; t += step) {
      int tl, tc;
      tile_coords<kWide>(p, t, tl, tc);
      // this thread's rows of both operands: where their scales start, or null
      const float* ls[kLanes / 32];
      const float* cs[S::kColScales < 32 ? 1 : S::kColScales / 32];
#pragma unroll
      for (int i = 0; i < kLanes / 32; ++i) {
        const int j = i * 32 + lane, row = tl * p.height + j;
        ls[i] = j < p.height && row < p.lane_n
                    ? p.lane_scale + (int64_t)(row >> p.lane_shift) * p.lane_sr
                    : nullptr;
      }
      if constexpr (kUniform) {
        const int row = tc * NT + lane * kBlock;
        cs[0] = lane < NT / kBlock && row < p.col_n
                    ? p.col_scale + (int64_t)(row / kBlock) * p.col_sr
                    : nullptr;
      } else {
#pragma unroll
        for (int i = 0; i < (NT + 31) / 32; ++i) {
          const int j = i * 32 + lane, row = tc * NT + j;
          cs[i] = j < NT && row < p.col_n ? p.col_scale + (int64_t)row * p.col_sr : nullptr;
        }
      }
      for (int kg = kb0; kg < kb1; kg += kG) {
        if (!mbar_wait_soon(smem_u32(&sempty[slot]), sphase ^ 1u, abort_flag, p.err)) {
          ok = false;
          break;
        }
#pragma unroll
        for (int g = 0; g < kG; ++g) {
          const int kb = kg + g;
          if (kb >= kb1) break;
          const uint32_t dst = smem_u32(sS) + slot * S::kSlot + g * (S::kBlockScales * 4);
#pragma unroll
          for (int i = 0; i < kLanes / 32; ++i)
            copy4(dst + (i * 32 + lane) * 4, ls[i] ? ls[i] + kb * p.lane_sk : p.lane_scale,
                  ls[i] != nullptr);
          if constexpr (kUniform) {
            if (lane < NT / kBlock)
              copy4(dst + (kLanes + lane) * 4, cs[0] ? cs[0] + kb * p.col_sk : p.col_scale,
                    cs[0] != nullptr);
          } else {
#pragma unroll
            for (int i = 0; i < (NT + 31) / 32; ++i)
              if (i * 32 + lane < NT)
                copy4(dst + (kLanes + i * 32 + lane) * 4,
                      cs[i] ? cs[i] + kb * p.col_sk : p.col_scale, cs[i] != nullptr);
          }
        }
        copies_arrive(smem_u32(&sfull[slot]));
        if (++slot == kSlots) {
          slot = 0;
          sphase ^= 1u;
        }
      }
    }
    asm volatile("cp.async.wait_all;" ::: "memory");  // before the CTA may exit
  }
    if (p.split > 1) {  // the sums' exchange (below) has two of these
      cg::this_cluster().sync();
      cg::this_cluster().sync();
    }
  } else {
    // ------------------------------------------------------------ scale and sum
    take_registers<kWide>();
    uint64_t acc[kHalf / 2];  // this thread's sums: its lane's row, kHalf columns, in pairs
    uint32_t slot = 0, sphase = 0, buf = 0, bphase = 0;
    uint32_t sel = 0;
    bool ok = start_ok;
    for (int t = tile0; ok && t < tiles; t += step) {
      int tl, tc;
      tile_coords<kWide>(p, t, tl, tc);
#pragma unroll
      for (int j = 0; j < kHalf / 2; ++j) acc[j] = 0;
      constexpr int kPer = kHalf / kChunk, kSteps = kG * kPer;
      if constexpr (kG == 1) {
        // a block at a time, the next kChunk columns on their way while kChunk are summed
        uint32_t r[2][kChunk];
        for (int kb = kb0; kb < kb1; ++kb) {
          if (!mbar_wait_soon(smem_u32(&sfull[slot]), sphase, abort_flag, p.err)) {
            ok = false;
            break;
          }
          const float* sl = sS + slot * (S::kSlot / 4);
          const float* sc = sl + kLanes + (kUniform ? half : half * kHalf);
          float s = sl[quarter * 32 + lane];
          if constexpr (kUniform) s *= sc[0];
          const uint64_t s2 = pair(s, s);
          if (!mbar_wait_soon(smem_u32(&tfull[buf]), bphase, abort_flag, p.err)) {
            ok = false;
            break;
          }
          tc_fence_after();
          const uint32_t taddr =
              tmem_base + ((uint32_t)(quarter * 32) << 16) + buf * NT + half * kHalf;
          tmem_ld<kChunk>(taddr, r[0]);
#pragma unroll
          for (int c = 0; c < kPer; ++c) {
            uint32_t(&w)[kChunk] = r[c & 1];
            float4 b[kUniform ? 1 : kChunk / 4];
            if constexpr (!kUniform) {  // on their way while tensor memory answers
#pragma unroll
              for (int j = 0; j < kChunk / 4; ++j)
                b[j] = *reinterpret_cast<const float4*>(sc + c * kChunk + 4 * j);
            }
            tmem_wait<kChunk>(w);
            if (c + 1 < kPer) {
              tmem_ld<kChunk>(taddr + (c + 1) * kChunk, r[(c + 1) & 1]);
            } else {  // everything is in registers: the accumulator is free
              tc_fence_before();
              __syncwarp();
              if (lane == 0) mbar_arrive(smem_u32(&tempty[buf]));
            }
            sum_columns<kUniform, kChunk>(acc + c * kChunk / 2, w, b, s2);
          }
          __syncwarp();
          if (lane == 0) mbar_arrive(smem_u32(&sempty[slot]));
          if (++slot == kSlots) {
            slot = 0;
            sphase ^= 1u;
          }
          if (++buf == kBufs) {
            buf = 0;
            bphase ^= 1u;
          }
        }
      } else {
        // A group's columns in steps of kChunk, two steps from tensor memory at a
        // time: the next one is on its way while one is summed.
        static_assert(kSteps % 2 == 0, "steps go in pairs");
        static_assert(!kUniform, "groups are the narrow form's: every column has a scale of its own");
        uint32_t r[2][kChunk];
        const uint32_t lane_addr = tmem_base + ((uint32_t)(quarter * 32) << 16) + half * kHalf;
        for (int kb = kb0; kb < kb1; kb += kG) {
          ok = mbar_wait_soon(smem_u32(&sfull[slot]), sphase, abort_flag, p.err) &&
               mbar_wait_soon(smem_u32(&tfull[buf]), bphase, abort_flag, p.err);
          if (!ok) break;
          tc_fence_after();
          const int live = min(kG, kb1 - kb);  // blocks of the group
          auto load = [&](int step) {
            tmem_ld<kChunk>(lane_addr + (buf * kG + step / kPer) * NT + step % kPer * kChunk, r[step & 1]);
          };
          load(0);
          load(1);
          float sl[kG];
#pragma unroll
          for (int g = 0; g < kG; ++g) {
            const float* at = sS + slot * (S::kSlot / 4) + g * S::kBlockScales;
            sl[g] = at[quarter * 32 + lane];
          }
#pragma unroll
          for (int st = 0; st < kSteps; ++st) {
            const int g = st / kPer, c = st % kPer;
            float4 b[kChunk / 4];  // on their way while tensor memory answers
            const float* at = sS + slot * (S::kSlot / 4) + g * S::kBlockScales + kLanes + half * kHalf;
#pragma unroll
            for (int j = 0; j < kChunk / 4; ++j)
              b[j] = *reinterpret_cast<const float4*>(at + c * kChunk + 4 * j);
            if (st % 2 == 0) {
              tmem_wait<kChunk>(r[0]);
              tmem_tie<kChunk>(r[1]);
              if (st + 2 >= kSteps) {  // the group is in registers
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(smem_u32(&tempty[buf]));
              }
            }
            if (g < live) {
              const uint64_t s2 = pair(sl[g], sl[g]);
              uint32_t(&w)[kChunk] = r[st & 1];
              sum_columns<false, kChunk>(acc + c * kChunk / 2, w, b, s2);
            }
            if (st + 2 < kSteps) load(st + 2);
          }
          __syncwarp();
          if (lane == 0) mbar_arrive(smem_u32(&sempty[slot]));
          if (++slot == kSlots) {
            slot = 0;
            sphase ^= 1u;
          }
          if (++buf == kBufs) {
            buf = 0;
            bphase ^= 1u;
          }
        }
      }
      if (!ok) {
        if (lane == 0) stopped[warp - 4] = t;
        break;
      }
      if (p.split > 1) {
        // one tile a cluster: its sums are joined below
      } else if constexpr (!kWide) {
        const int row = quarter * 32 + lane;
        const int n = tl * p.height + row;
        const int m0 = tc * NT + half * kHalf;
        const bool mine = row < p.height && n < p.N;
        // the columns' 1 / tau, one a lane (a load for each column as it is
        // written would be waited for each time)
        float inv[(kHalf + 31) / 32];
#pragma unroll
        for (int i = 0; i < (kHalf + 31) / 32; ++i) {
          const int m = m0 + i * 32 + lane;
          inv[i] = i * 32 + lane < kHalf && m < p.M ? over_tau(p, m) : 1.f;
        }
#pragma unroll
        for (int j = 0; j < kHalf; ++j) {
          if (m0 + j >= p.M) break;  // the same in every lane
          const float2 v = unpair(acc[j / 2]);
          const float x = (j % 2 ? v.y : v.x) * __shfl_sync(0xFFFFFFFFu, inv[j / 32], j % 32);
          if (mine) finish<O>(p, m0 + j, n, x);
        }
      } else {
        // 32 rows x 64 bytes at a time: a thread's row in 16-byte pieces, piece
        // i of row r at i ^ (r / 2) % 4 (64-byte swizzle, no bank conflicts)
        constexpr int kCols = 64 / (int)sizeof(O);
        const int m0 = tl * kLanes + quarter * 32, m = m0 + lane;
        const float inv = m < p.M ? over_tau(p, m) : 0.f;
        uint8_t* mine = staging + (warp - 4) * 2 * kStaging;
#pragma unroll
        for (int c = 0; c < kHalf / kCols; ++c) {
          const int n0 = tc * NT + half * kHalf + c * kCols;
          if (n0 < p.N && m0 < p.M) {  // the same in every thread of the warp
            const uint32_t buf_s = smem_u32(mine + sel * kStaging);
            if (lane == 0) bulk_wait_read<1>();
            __syncwarp();
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              uint32_t w[4];
              if constexpr (sizeof(O) == 4) {
                const float2 x = unpair(acc[c * 8 + 2 * i]), y = unpair(acc[c * 8 + 2 * i + 1]);
                w[0] = __float_as_uint(x.x * inv);
                w[1] = __float_as_uint(x.y * inv);
                w[2] = __float_as_uint(y.x * inv);
                w[3] = __float_as_uint(y.y * inv);
              } else {
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                  const float2 x = unpair(acc[c * 16 + 4 * i + k]);
                  w[k] = pack_bf16x2(x.x * inv, x.y * inv);
                }
              }
              st_shared_v4(buf_s + lane * 64 + ((i ^ ((lane >> 1) & 3)) << 4), w[0], w[1], w[2], w[3]);
            }
            if (n0 < p.tma_cols) {
              fence_proxy_async_smem();
              __syncwarp();
              if (lane == 0) {
                if (p.accumulate)
                  tma_reduce_add_2d(&map_out, buf_s, n0, m0);
                else
                  tma_store_2d(&map_out, buf_s, n0, m0);
                bulk_commit();
              }
              sel ^= 1u;  // (the other way's piece has been read when its turn is over)
            } else {  // what TMA cannot address of C: 64 bytes of a row per 16 or 32 lanes
              __syncwarp();
              constexpr int kRows = 32 / kCols;  // rows per step
              const int col = lane % kCols;
              for (int r = lane / kCols; r < 32; r += kRows) {
                const O v = *reinterpret_cast<const O*>(
                    mine + sel * kStaging + r * 64 +
                    (((col * (int)sizeof(O) / 16) ^ ((r >> 1) & 3)) << 4) + (col * (int)sizeof(O)) % 16);
                if (m0 + r < p.M && n0 + col < p.N) finish<O>(p, m0 + r, n0 + col, (float)v);
              }
              __syncwarp();
            }
          }
        }
      }
    }
    if (kWide && lane == 0) bulk_wait_all();
    __syncwarp();
    if (p.split > 1) {
      // One tile per cluster. Every stage has been read by now (the sums wait
      // for the last MMA), so the ring holds the sums, a line for each m.
      float* sums = reinterpret_cast<float*>(smem);
      const int row = quarter * 32 + lane;
      if constexpr (kWide) {
        float4* mine = reinterpret_cast<float4*>(sums + row * S::kPitch + half * kHalf);
#pragma unroll
        for (int j = 0; j < kHalf / 4; ++j) {
          const float2 x = unpair(acc[2 * j]), y = unpair(acc[2 * j + 1]);
          mine[j] = make_float4(x.x, x.y, y.x, y.y);
        }
      } else {
#pragma unroll
        for (int j = 0; j < kHalf / 2; ++j) {
          const float2 v = unpair(acc[j]);
          sums[(half * kHalf + 2 * j) * S::kPitch + row] = v.x;
          sums[(half * kHalf + 2 * j + 1) * S::kPitch + row] = v.y;
        }
      }
    }
    if (p.split > 1) {
      float* sums = reinterpret_cast<float*>(smem);
      cg::cluster_group cluster = cg::this_cluster();
      cluster.sync();
      {
        int last_l, last_c;
        tile_coords<kWide>(p, tile0, last_l, last_c);
        // the CTAs divide the lines; the parts are added in the order of k
        for (int j = part + p.split * (warp - 4); j < S::kLines; j += p.split * kSumWarps) {
          const int m = (kWide ? last_l * kLanes : last_c * NT) + j;
          if (m >= p.M) break;
          const float inv = over_tau(p, m);
          const int n0 = kWide ? last_c * NT : last_l * p.height;
          const int end = min(kWide ? S::kLong : p.height, p.N - n0);
          // 128 elements of a line; what every part has of them is on its way
          // before the first is added
#pragma unroll 1
          for (int i = lane * 4; i < S::kLong; i += 128) {
            float4 x[kMaxSplit];
#pragma unroll
            for (int q = 0; q < kMaxSplit; ++q)
              if (q < p.split)
                x[q] = *reinterpret_cast<const float4*>(cluster.map_shared_rank(sums, q) + j * S::kPitch + i);
            float v[4] = {x[0].x, x[0].y, x[0].z, x[0].w};
#pragma unroll
            for (int q = 1; q < kMaxSplit; ++q) {
              if (q < p.split) {
                v[0] += x[q].x;
                v[1] += x[q].y;
                v[2] += x[q].z;
                v[3] += x[q].w;
              }
            }
#pragma unroll
            for (int u = 0; u < 4; ++u)
              if (i + u < end) finish<O>(p, m, n0 + i + u, v[u] * inv);
          }
        }
      }
      cluster.sync();
    }
  }

  __syncthreads();
  if (*abort_flag != 0 && warp >= 4) {
    // After a wait that gave up, this warp's share of the tile that it was at and
    // of those to come is unknown; of a split, the whole tile, which by now every
    // other part has written.
    for (int t = p.split > 1 ? tile0 : stopped[warp - 4]; t < tiles; t += step) {
      int tl, tc;
      tile_coords<kWide>(p, t, tl, tc);
      const int l0 = tl * p.height + quarter * 32, l = min(32, p.height - quarter * 32);
      const int c0 = tc * NT + half * kHalf;
      const int m0 = kWide ? l0 : c0, n0 = kWide ? c0 : l0;
      blank(static_cast<O*>(p.C) + (int64_t)m0 * p.ldc + n0, p.ldc, min(kWide ? l : kHalf, p.M - m0),
            min(kWide ? kHalf : l, p.N - n0));
    }
  }
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem_base, S::kTmemCols);
  }
}

struct Maps {
  CUtensorMap lanes, cols, out;
};

template <int NT, bool kWide, bool kUniform, typename O>
cudaError_t launch(const Maps& maps, const ProductArgs& p, int grid, cudaStream_t st) {
  using S = Shape<NT, kWide, kUniform>;
  auto kern = product_kernel<NT, kWide, kUniform, O>;
  cudaError_t e =
      cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)S::kSmem);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3((unsigned)grid);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = S::kSmem;
  cfg.stream = st;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeClusterDimension;
  at[0].val.clusterDim.x = (unsigned)p.split;
  at[0].val.clusterDim.y = 1;
  at[0].val.clusterDim.z = 1;
  cfg.attrs = at;
  cfg.numAttrs = p.split > 1 ? 1 : 0;
  e = cudaLaunchKernelEx(&cfg, kern, maps.lanes, maps.cols, maps.out, p);
  const cudaError_t last = cudaGetLastError();
  return e != cudaSuccess ? e : last;
}

template <typename O>
cudaError_t launch_out(int NT, bool uniform, const Maps& maps, const ProductArgs& p, int grid,
                       cudaStream_t st) {
  switch (NT) {
    case 16: return launch<16, false, false, O>(maps, p, grid, st);
    case 32: return launch<32, false, false, O>(maps, p, grid, st);
    case 64: return launch<64, false, false, O>(maps, p, grid, st);
    case 128: return launch<128, false, false, O>(maps, p, grid, st);
    default:
      return uniform ? launch<256, true, true, O>(maps, p, grid, st)
                     : launch<256, true, false, O>(maps, p, grid, st);
  }
}

constexpr int64_t kMost = (int64_t(1) << 31) - 1024;

std::atomic<int64_t> g_give_up{-1};  // sts_probe_product_timeout

// Which form. Above 128 rows of A the wide one, up to 64 the narrow one (at 33 to
// 64 rows the two take the same time at the median of 207 shapes where TMA can
// write C; where it cannot, the wide one takes 1.6 times the narrow one's). Between
// them the wide one where TMA can: it took 0.7 of the narrow one's time at the
// median of 276 shapes (128 x 2,048 x 2,048 12.4 us, narrow 18.5; 100 x 151,936 x
// 4,096 125, narrow 202; 96 x 8,000 x 8,192 22.5, narrow 43.7), more only where
// there is little work (128 x 300 x 1,024 14.4, narrow 12.4). Where C leaves by
// ordinary stores, by the rounds of tiles that each takes over the SMs: a round of
// the wide form's takes about as long as its blocks along k and 12 more (its
// results leave while nothing is multiplied), of the narrow form's as its blocks
// and 2 more. 77 x 50,021 x 2,048: wide 49.1, narrow 43.1; x 4,096 68.0 and 70.5; x
// 8,192 106 and 121 (with a scale per row of B x 4,096 83 and 70: there the wide
// form's blocks cost more than the estimate has it).
bool wide_form(int64_t M, int64_t N, int64_t kb, int sms, bool tma) {
  if (M > 128) return true;
  if (M <= 64) return false;
  if (tma) return true;
  const int64_t wide = ((N + 255) / 256 + sms - 1) / sms;
  const int64_t narrow = (N + (int64_t)kLanes * sms - 1) / ((int64_t)kLanes * sms);
  return wide * (kb + 12) < narrow * (kb + 2);
}

// Rows of B in the narrow form's smallest tile: 1 x 512 x 16,384 takes 13.4 us, with
// 32 rows 16.5 (with 64, and 8 parts a tile, 10.3).
constexpr int kMinHeight = 16;

// Clusters of `size` blocks that the current device holds at once. A block takes
// an SM whatever its form, and a cluster lies within one of the device's groups of
// SMs, so there are fewer than sms / size: 74 of 2, 33 of 4 and 15 of 8 on a B200
// of 148 SMs.
int clusters_held(int size, int sms) {
  constexpr int kDevices = 64;
  static std::atomic<int> held[kDevices][kMaxSplit + 1];
  int device = 0;
  if (cudaGetDevice(&device) != cudaSuccess || device >= kDevices) return sms / size;
  int n = held[device][size].load(std::memory_order_relaxed);
  if (n > 0) return n;
  using S = Shape<256, true, true>;
  auto kern = product_kernel<256, true, true, float>;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3((unsigned)size);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = S::kSmem;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeClusterDimension;
  at[0].val.clusterDim.x = (unsigned)size;
  at[0].val.clusterDim.y = 1;
  at[0].val.clusterDim.z = 1;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)S::kSmem) !=
          cudaSuccess ||
      cudaOccupancyMaxActiveClusters(&n, kern, &cfg) != cudaSuccess || n < 1) {
    cudaGetLastError();  // the launch does not answer for it
    return sms / size;
  }
  held[device][size].store(n, std::memory_order_relaxed);
  return n;
}

sts_status check_operand(const sts_block_operand* o, int64_t K, bool rows_only) {
  if (!o) return STS_ERR_NULL;
  if (o->dtype != STS_DTYPE_E4M3 && o->dtype != STS_DTYPE_E5M2) return STS_ERR_DTYPE;
  if (o->rows < 0 || o->rows > kMost) return STS_ERR_SHAPE;
  if (o->block_rows != 1 && (rows_only || o->block_rows != kBlock)) return STS_ERR_SHAPE;
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

extern "C" void sts_probe_product_timeout(int64_t block) {
  g_give_up.store(block >= 0 && block <= kMost ? block : -1, std::memory_order_relaxed);
}

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
  if ((reinterpret_cast<uintptr_t>(C) % (c_dtype == STS_DTYPE_F32 ? 4u : 2u)) != 0 ||
      (reinterpret_cast<uintptr_t>(temperature) & 3u) != 0)
    return STS_ERR_SHAPE;
  int sms = 0;
  s = current_device(&sms);
  if (s != STS_OK) return s;

  const int64_t M = A->rows, N = B->rows;
  const bool bf = c_dtype == STS_DTYPE_BF16;
  const int64_t cs = bf ? 2 : 4;
  const bool tma = (reinterpret_cast<uintptr_t>(C) & 15u) == 0 && ldc * cs % 16 == 0 &&
                   ldc < (int64_t(1) << 37);  // it can address C's rows
  const bool wide = wide_form(M, N, (K + kBlock - 1) / kBlock, sms, tma);
  const int NT = wide ? 256 : M <= 16 ? 16 : M <= 32 ? 32 : M <= 64 ? 64 : 128;
  const sts_block_operand* L = wide ? A : B;  // the lanes' operand
  const sts_block_operand* R = wide ? B : A;  // the columns'
  const bool uniform = wide && B->block_rows == kBlock;
  ProductArgs p{};
  p.M = (int)M;
  p.N = (int)N;
  p.kb = (int)((K + kBlock - 1) / kBlock);
  p.lane_n = (int)L->rows;
  p.col_n = (int)R->rows;
  p.height = kLanes;
  if (!wide) {
    // as many rounds of tiles as 128 rows each would take, and equal tiles (1 x
    // 32,768 x 4,096: 26.4 us, with tiles of 64 rows 31.0, of 16 89.0; 1 x 2,048 x
    // 4,096: 12.4, of 64 rows and 4 parts 9.1, of 128 12.4)
    const int64_t rounds = (N + (int64_t)kLanes * sms - 1) / ((int64_t)kLanes * sms);
    p.height = (int)((N + rounds * sms - 1) / (rounds * sms));
    if (p.height < kMinHeight) p.height = kMinHeight;
  }
  const int64_t tiles_l = (L->rows + p.height - 1) / p.height, tiles_c = (R->rows + NT - 1) / NT;
  if (tiles_l * tiles_c > kMost) return STS_ERR_SHAPE;
  p.tiles_l = (int)tiles_l;
  p.tiles_c = (int)tiles_c;
  p.lane_scale = L->scale;
  p.lane_sr = L->scale_stride_r;
  p.lane_sk = L->scale_stride_k;
  p.lane_shift = L->block_rows == kBlock ? 7 : 0;
  p.col_scale = R->scale;
  p.col_sr = R->scale_stride_r;
  p.col_sk = R->scale_stride_k;
  p.idesc = idesc_f8(L->dtype == STS_DTYPE_E5M2, R->dtype == STS_DTYPE_E5M2, kLanes, NT);
  p.tau = temperature;
  p.C = C;
  p.ldc = ldc;
  p.accumulate = accumulate ? 1 : 0;
  p.give_up = (int)g_give_up.load(std::memory_order_relaxed);
  const int64_t tiles = tiles_l * tiles_c;
  // a stretch of k for each of 2, 4 or 8 CTAs while the device holds all tiles'
  // clusters at once, none below 4 blocks. 300 x 512 x 16,384 (6 tiles): 8 parts
  // 18.5 us, 4 24.7, whole 61.5; 300 x 2,048 x 8,192 (24): 4 parts 18.6, 2 26.8,
  // whole 35.2. Where the last clusters would wait for the first, 1 x 256 x 16,384
  // (16): 4 parts 12.4, 8 16.5; 300 x 1,536 x 16,384 (18): 4 parts 26.7, 8 34.1
  p.split = 1;
  while (p.split < kMaxSplit && tiles * p.split * 2 <= sms && p.kb >= p.split * 2 * 4 &&
         tiles <= clusters_held(p.split * 2, sms))
    p.split *= 2;
  const int grid = (int)(p.split > 1 ? tiles * p.split : (tiles < sms ? tiles : sms));

  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  if (ws) {
    WsHeader* hdr = static_cast<WsHeader*>(ws);
    if (cudaMemsetAsync(&hdr->bad_row_code, 0xFF, sizeof(hdr->bad_row_code), st) != cudaSuccess ||
        cudaMemsetAsync(&hdr->err, 0, sizeof(hdr->err), st) != cudaSuccess)
      return STS_ERR_CUDA;
    p.err = &hdr->err;
  }
  Maps maps;
  std::memset(&maps, 0, sizeof(maps));
  if (!tensor_map_2d(&maps.lanes, L->q, CU_TENSOR_MAP_DATA_TYPE_UINT8, (uint64_t)K,
                     (uint64_t)L->rows, (uint64_t)L->ld, kBlock, (uint32_t)p.height,
                     CU_TENSOR_MAP_SWIZZLE_128B) ||
      !tensor_map_2d(&maps.cols, R->q, CU_TENSOR_MAP_DATA_TYPE_UINT8, (uint64_t)K,
                     (uint64_t)R->rows, (uint64_t)R->ld, kBlock, (uint32_t)NT,
                     CU_TENSOR_MAP_SWIZZLE_128B))
    return STS_ERR_CUDA;
  if (wide && tma) {
    if (!tensor_map_2d(&maps.out, C, bf ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT32,
                       (uint64_t)N, (uint64_t)M, (uint64_t)(ldc * cs), (uint32_t)(64 / cs), 32,
                       CU_TENSOR_MAP_SWIZZLE_64B))
      return STS_ERR_CUDA;
    // TMA ends a row at whole 16 bytes: the last piece of rows that end elsewhere
    // would reach over what lies behind them
    const int64_t piece = 64 / cs;
    p.tma_cols = (int)(N * cs % 16 == 0 ? N : N / piece * piece);
  }
  const LaunchMark mark = launch_begin(STS_KERNEL_BLOCK_PRODUCT, st);
  const cudaError_t e = bf ? launch_out<__nv_bfloat16>(NT, uniform, maps, p, grid, st)
                           : launch_out<float>(NT, uniform, maps, p, grid, st);
  launch_end(mark, st);
  return e == cudaSuccess ? STS_OK : STS_ERR_CUDA;
}
