// sts_block_quantize: a matrix to 8-bit floating point with one fp32 scale per
// block of 1 x 128 or 128 x 128 elements.
//
// For a block with largest finite magnitude a, and top the largest code of the
// 8-bit type (448 for e4m3, 57344 for e5m2):
//   scale = a / top, or 1 when that quotient is 0   (IEEE fp32 division)
//   code  = x (1 / scale), the reciprocal and the product rounded to fp32 (x /
//           scale where scale is below 2^-126, whose reciprocal may not exist),
//           limited to +-top, rounded to nearest even in the 8-bit type; NaN for
//           an x that is not finite
// (a division an element would be bound by its instructions, not by HBM: 1.29
// ms for 151,936 x 4,096 bf16), so that code * scale is x within half a step of the 8-bit type (2^-4
// relative for e4m3 in its normal range). Entries that are not finite do not
// enter the scale, so they cost their neighbours no precision, and stay
// visible as NaN in every product that they take part in.
//
// Nothing is used twice: the kernels are bound by HBM. Each block is read once
// into registers (8 elements a load), its maximum is taken there, and the codes
// leave 8 bytes a thread:
//   rows1    x's K is contiguous, blocks of 1 x 128: 16 lanes hold a block, the
//            maximum is four shuffles. No shared memory, no barrier.
//   rows128  x's K is contiguous, blocks of 128 x 128: 256 threads hold a block.
//   cols     x's rows are contiguous (a transposed view): 256 threads hold 128
//            x 128 elements; the codes cross shared memory, so that both the
//            reads along x's rows and the writes along K are whole lines.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_fp8.h>

#include "sts_internal.h"

namespace sts {
namespace {

constexpr int kBlock = 128;
constexpr int kThreads = 256;

__device__ __forceinline__ float to_f32(float v) { return v; }
__device__ __forceinline__ float to_f32(__nv_bfloat16 v) { return __bfloat162float(v); }
__device__ __forceinline__ float to_f32(__half v) { return __half2float(v); }

// 8 consecutive elements from p, `live` of them present (the others 0).
template <typename T, bool kVec>
__device__ __forceinline__ void load8(const T* p, int live, float (&v)[8]) {
  if (kVec && live >= 8) {
    constexpr int kWords = (int)sizeof(T) * 8 / 16;
    union {
      uint4 w[kWords];
      T e[8];
    } u;
#pragma unroll
    for (int i = 0; i < kWords; ++i) u.w[i] = __ldg(reinterpret_cast<const uint4*>(p) + i);
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = to_f32(u.e[i]);
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = i < live ? to_f32(p[i]) : 0.f;
  }
}

constexpr float kLargest = 3.402823466e+38f;

// The largest finite |v|, 0 without one.
__device__ __forceinline__ float largest8(const float (&v)[8]) {
  float m = 0.f;
#pragma unroll
  for (int i = 0; i < 8; ++i) m = fmaxf(m, fabsf(v[i]));  // a NaN is passed over
  if (m > kLargest) {  // an infinity among them
    m = 0.f;
#pragma unroll
    for (int i = 0; i < 8; ++i) m = fmaxf(m, fabsf(v[i]) <= kLargest ? fabsf(v[i]) : 0.f);
  }
  return m;
}

// A block's scale, and what its entries are multiplied by.
struct Scale {
  float s, inv;
};

template <bool kE5>
__device__ __forceinline__ Scale block_scale(float amax) {
  Scale r;
  r.s = __fdiv_rn(amax, kE5 ? 57344.f : 448.f);
  r.s = r.s > 0.f ? r.s : 1.f;
  r.inv = __frcp_rn(r.s);
  return r;
}

template <bool kE5>
__device__ __forceinline__ uint32_t code2(float a, float b) {
  return (uint32_t)__nv_cvt_float2_to_fp8x2(make_float2(a, b), __NV_SATFINITE,
                                            kE5 ? __NV_E5M2 : __NV_E4M3);
}

template <bool kE5>
__device__ __forceinline__ uint2 code8(const float (&v)[8], const Scale& sc) {
  float y[8];
  if (sc.s >= 1.17549435e-38f) {
#pragma unroll
    for (int i = 0; i < 8; ++i) y[i] = v[i] * sc.inv;
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) y[i] = __fdiv_rn(v[i], sc.s);
  }
  // the conversion limits what is too large, infinities included: NaN for those
  // (inf times a reciprocal is inf; a finite entry gives at most about top)
  float m = 0.f;
#pragma unroll
  for (int i = 0; i < 8; ++i) m = fmaxf(m, fabsf(y[i]));
  if (m > kLargest) {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (fabsf(y[i]) > kLargest) y[i] = __int_as_float(0x7fc00000);
  }
  uint2 w;
  w.x = code2<kE5>(y[0], y[1]) | (code2<kE5>(y[2], y[3]) << 16);
  w.y = code2<kE5>(y[4], y[5]) | (code2<kE5>(y[6], y[7]) << 16);
  return w;
}

__device__ __forceinline__ void store8(uint8_t* q, uint2 w, int live, bool vec) {
  if (vec && live >= 8) {
    *reinterpret_cast<uint2*>(q) = w;
    return;
  }
#pragma unroll
  for (int i = 0; i < 8; ++i)
    if (i < live) q[i] = (uint8_t)((i < 4 ? w.x : w.y) >> (8 * (i & 3)));
}

struct QuantArgs {
  const void* x;
  int64_t R, K, ld;  // ld: stride of the dimension that is not contiguous (elements)
  uint8_t* q;
  int64_t q_ld;
  float* scale;
  int64_t scale_ld;
  int64_t row_blocks, k_blocks;
  bool q_vec;  // q rows start on 8-byte boundaries
};

// 1 x 128 blocks along contiguous K: 16 lanes a block, kUnroll blocks in flight
// for each group of lanes.
template <typename T, bool kE5, bool kVec>
__global__ void __launch_bounds__(kThreads) rows1_kernel(const QuantArgs a) {
  constexpr int kUnroll = sizeof(T) == 2 ? 4 : 2;
  const int sub = threadIdx.x & 15;
  const int64_t total = a.R * a.k_blocks;
  const int64_t groups = (int64_t)gridDim.x * (kThreads / 16);
  for (int64_t first = (int64_t)blockIdx.x * (kThreads / 16) + (threadIdx.x >> 4); first < total;
       first += groups * kUnroll) {
    float v[kUnroll][8];
    int64_t row[kUnroll];
    int64_t kb[kUnroll];
    int live[kUnroll];
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
      const int64_t b = first + u * groups;
      live[u] = 0;
      if (b < total) {
        if (total <= 0xFFFFFFFFll) {  // a 32-bit division wherever it will do
          row[u] = (int64_t)((uint32_t)b / (uint32_t)a.k_blocks);
        } else {
          row[u] = b / a.k_blocks;
        }
        kb[u] = b - row[u] * a.k_blocks;
        const int64_t left = a.K - (kb[u] * kBlock + sub * 8);
        live[u] = left >= 8 ? 8 : (left > 0 ? (int)left : 0);
        if (live[u] > 0)
          load8<T, kVec>(static_cast<const T*>(a.x) + row[u] * a.ld + kb[u] * kBlock + sub * 8,
                         live[u], v[u]);
      }
    }
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
      const bool mine = first + u * groups < total;
      float m = 0.f;
      if (live[u] > 0) m = largest8(v[u]);
      // the 16 lanes of a group agree on `first`, but the two groups of a warp
      // may leave the loop apart: only this group's lanes take part
      const uint32_t lanes = 0xFFFFu << (threadIdx.x & 16);
#pragma unroll
      for (int o = 8; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(lanes, m, o));
      if (!mine) continue;
      const Scale s = block_scale<kE5>(m);
      if (sub == 0) a.scale[row[u] * a.scale_ld + kb[u]] = s.s;
      if (live[u] > 0)
        store8(a.q + row[u] * a.q_ld + kb[u] * kBlock + sub * 8, code8<kE5>(v[u], s), live[u],
               a.q_vec);
    }
  }
}

// The largest of m over the 256 threads of the block.
__device__ __forceinline__ float block_max(float m, float* warp_max) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xFFFFFFFFu, m, o));
  if ((threadIdx.x & 31) == 0) warp_max[threadIdx.x >> 5] = m;
  __syncthreads();
#pragma unroll
  for (int w = 0; w < kThreads / 32; ++w) m = fmaxf(m, warp_max[w]);
  return m;
}

// 128 x 128 blocks along contiguous K: one block per thread block, thread t
// holds 8 columns of the rows t / 16 + 16 i.
template <typename T, bool kE5, bool kVec>
__global__ void __launch_bounds__(kThreads) rows128_kernel(const QuantArgs a) {
  __shared__ float warp_max[kThreads / 32];
  const int64_t rb = (int64_t)blockIdx.x / a.k_blocks;
  const int64_t kb = (int64_t)blockIdx.x - rb * a.k_blocks;
  const int64_t k = kb * kBlock + (threadIdx.x & 15) * 8;
  const int64_t left = a.K - k;
  const int live = left >= 8 ? 8 : (left > 0 ? (int)left : 0);
  const int64_t r0 = rb * kBlock + (threadIdx.x >> 4);
  float v[8][8];
  float m = 0.f;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int64_t r = r0 + 16 * i;
    load8<T, kVec>(static_cast<const T*>(a.x) + r * a.ld + k, r < a.R ? live : 0, v[i]);
  }
#pragma unroll
  for (int i = 0; i < 8; ++i) m = fmaxf(m, largest8(v[i]));
  const Scale s = block_scale<kE5>(block_max(m, warp_max));
  if (threadIdx.x == 0) a.scale[rb * a.scale_ld + kb] = s.s;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int64_t r = r0 + 16 * i;
    if (r < a.R) store8(a.q + r * a.q_ld + k, code8<kE5>(v[i], s), live, a.q_vec);
  }
}

// x's rows are contiguous: element (r, k) at x[r + k * ld]. 128 x 128 elements
// per thread block; thread t holds the 8 rows 8 (t % 16).. of the 8 columns
// 8 (t / 16)... The codes cross shared memory as [row][16 groups of 8 k], the
// group index exclusive-ored with row / 8 so that neither side meets a bank
// conflict.
template <typename T, bool kE5, bool kVec, bool kSquare>
__global__ void __launch_bounds__(kThreads) cols_kernel(const QuantArgs a) {
  __shared__ float warp_max[kThreads / 32];
  __shared__ float row_max[16][kBlock + 1];
  __shared__ uint2 codes[kBlock][16];
  const int64_t rb = (int64_t)blockIdx.x % a.row_blocks;
  const int64_t kb = (int64_t)blockIdx.x / a.row_blocks;
  const int oct = threadIdx.x & 15, kg = threadIdx.x >> 4;
  const int64_t r = rb * kBlock + oct * 8;
  const int64_t k = kb * kBlock + kg * 8;
  const int64_t left = a.R - r;
  const int live = left >= 8 ? 8 : (left > 0 ? (int)left : 0);
  float v[8][8];  // [k][r]
#pragma unroll
  for (int i = 0; i < 8; ++i)
    load8<T, kVec>(static_cast<const T*>(a.x) + (k + i) * a.ld + r, k + i < a.K ? live : 0, v[i]);
  Scale s[kSquare ? 1 : 8];
  if constexpr (kSquare) {
    float m = 0.f;
#pragma unroll
    for (int i = 0; i < 8; ++i) m = fmaxf(m, largest8(v[i]));
    s[0] = block_scale<kE5>(block_max(m, warp_max));
    if (threadIdx.x == 0) a.scale[rb * a.scale_ld + kb] = s[0].s;
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      float w[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) w[i] = v[i][j];
      row_max[kg][oct * 8 + j] = largest8(w);
    }
    __syncthreads();
    if (threadIdx.x < kBlock) {
      float m = 0.f;
#pragma unroll
      for (int g = 0; g < 16; ++g) m = fmaxf(m, row_max[g][threadIdx.x]);
      const Scale sc = block_scale<kE5>(m);
      row_max[0][threadIdx.x] = sc.s;
      row_max[1][threadIdx.x] = sc.inv;
      const int64_t row = rb * kBlock + threadIdx.x;
      if (row < a.R) a.scale[row * a.scale_ld + kb] = sc.s;
    }
    __syncthreads();
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      s[j].s = row_max[0][oct * 8 + j];
      s[j].inv = row_max[1][oct * 8 + j];
    }
  }
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    float w[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) w[i] = v[i][j];
    codes[oct * 8 + j][kg ^ oct] = code8<kE5>(w, s[kSquare ? 0 : j]);
  }
  __syncthreads();
  const int64_t kk = kb * kBlock + oct * 8;  // now 16 lanes write a row's 128 codes
  const int64_t kleft = a.K - kk;
  const int klive = kleft >= 8 ? 8 : (kleft > 0 ? (int)kleft : 0);
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int row = kg + 16 * i;
    if (rb * kBlock + row < a.R)
      store8(a.q + (rb * kBlock + row) * a.q_ld + kk, codes[row][oct ^ (row >> 3)], klive, a.q_vec);
  }
}

template <typename T, bool kE5, bool kVec>
cudaError_t launch(const QuantArgs& a, bool transposed, int block_rows, int sms, cudaStream_t st) {
  if (!transposed && block_rows == 1) {
    constexpr int64_t per = kThreads / 16;
    const int64_t want = (a.R * a.k_blocks + per - 1) / per;
    const int64_t most = (int64_t)sms * 16;  // 2,048 threads an SM, two blocks deep
    rows1_kernel<T, kE5, kVec><<<(int)(want < most ? want : most), kThreads, 0, st>>>(a);
    return cudaGetLastError();
  }
  const unsigned grid = (unsigned)(a.row_blocks * a.k_blocks);
  if (!transposed)
    rows128_kernel<T, kE5, kVec><<<grid, kThreads, 0, st>>>(a);
  else if (block_rows == 1)
    cols_kernel<T, kE5, kVec, false><<<grid, kThreads, 0, st>>>(a);
  else
    cols_kernel<T, kE5, kVec, true><<<grid, kThreads, 0, st>>>(a);
  return cudaGetLastError();
}

template <typename T>
cudaError_t launch_t(const QuantArgs& a, bool e5, bool transposed, int block_rows, int sms,
                     cudaStream_t st) {
  // 16-byte loads need 16-byte rows; any other layout is read element by element
  const bool vec = (reinterpret_cast<uintptr_t>(a.x) & 15u) == 0 &&
                   (a.ld * (int64_t)sizeof(T)) % 16 == 0;
  if (vec)
    return e5 ? launch<T, true, true>(a, transposed, block_rows, sms, st)
              : launch<T, false, true>(a, transposed, block_rows, sms, st);
  return e5 ? launch<T, true, false>(a, transposed, block_rows, sms, st)
            : launch<T, false, false>(a, transposed, block_rows, sms, st);
}

}  // namespace
}  // namespace sts

using namespace sts;

extern "C" sts_status sts_block_quantize(int64_t R, int64_t K, const void* x, int x_dtype,
                                         int64_t stride_r, int64_t stride_k, int block_rows,
                                         int q_dtype, void* q, int64_t q_ld, float* scale,
                                         int64_t scale_ld, sts_stream_t stream) {
  if (x_dtype != STS_DTYPE_F32 && x_dtype != STS_DTYPE_BF16 && x_dtype != STS_DTYPE_F16)
    return STS_ERR_DTYPE;
  if (q_dtype != STS_DTYPE_E4M3 && q_dtype != STS_DTYPE_E5M2) return STS_ERR_DTYPE;
  constexpr int64_t kMost = (int64_t(1) << 31) - 1;
  if (R < 0 || R > kMost || K < 1 || K > kMost) return STS_ERR_SHAPE;
  if (block_rows != 1 && block_rows != kBlock) return STS_ERR_SHAPE;
  const bool transposed = stride_k != 1;
  if (transposed && stride_r != 1) return STS_ERR_SHAPE;
  const int64_t ld = transposed ? stride_k : stride_r;
  // a single row (or column) has no stride to speak of
  if ((transposed ? K : R) > 1 && ld < (transposed ? R : K)) return STS_ERR_SHAPE;
  const int64_t k_blocks = (K + kBlock - 1) / kBlock;
  if (q_ld < K || scale_ld < k_blocks) return STS_ERR_SHAPE;
  if (R == 0) return STS_OK;
  if (!x || !q || !scale) return STS_ERR_NULL;
  QuantArgs a{};
  a.x = x;
  a.R = R;
  a.K = K;
  a.ld = ld;
  a.q = static_cast<uint8_t*>(q);
  a.q_ld = q_ld;
  a.scale = scale;
  a.scale_ld = scale_ld;
  a.row_blocks = (R + kBlock - 1) / kBlock;
  a.k_blocks = k_blocks;
  a.q_vec = (reinterpret_cast<uintptr_t>(q) & 7u) == 0 && q_ld % 8 == 0;
  if (a.row_blocks * k_blocks > kMost) return STS_ERR_SHAPE;
  int sms = 0;
  const sts_status ds = current_device(&sms);
  if (ds != STS_OK) return ds;
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  const LaunchMark mark = launch_begin(STS_KERNEL_BLOCK_QUANTIZE, st);
  const bool e5 = q_dtype == STS_DTYPE_E5M2;
  const cudaError_t e =
      x_dtype == STS_DTYPE_F32    ? launch_t<float>(a, e5, transposed, block_rows, sms, st)
      : x_dtype == STS_DTYPE_BF16 ? launch_t<__nv_bfloat16>(a, e5, transposed, block_rows, sms, st)
                                  : launch_t<__half>(a, e5, transposed, block_rows, sms, st);
  launch_end(mark, st);
  return e == cudaSuccess ? STS_OK : STS_ERR_CUDA;
}
