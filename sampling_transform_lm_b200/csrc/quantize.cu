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
// ms for 151,936 x 4,096 bf16), so that code * scale is x within half a step of
// the 8-bit type (2^-4 relative for e4m3 in its normal range). The reciprocal's
// rounding shows where x / scale lies within 2^-23 of the middle between two
// codes, as quotients of bf16 values often do: 0.05 % of the codes of 151,936 x
// 4,096 are then the other neighbour. Entries that are not finite do not
// enter the scale, so they cost their neighbours no precision, and stay
// visible as NaN in every product that they take part in.
//
// Nothing is used twice: HBM bounds the kernels, as long as they stay under some
// 8 instructions an element. Each block is read once, 16 bytes a load, and kept
// as it was read; the maximum is taken on packed pairs, and the codes leave 8
// bytes a store:
//   rows1    x's K is contiguous, blocks of 1 x 128: 4 lanes hold a block, 32
//            elements each, so that the scale's division is paid once in 32. No
//            shared memory, no barrier.
//   rows128  x's K is contiguous, blocks of 128 x 128: 256 threads hold a block.
//   cols     x's rows are contiguous (a transposed view): 256 threads hold 128
//            x 128 elements; the codes cross shared memory, so that both the
//            reads along x's rows and the writes along K are whole lines.
// 151,936 x 4,096 bf16 takes 319 to 330 us in 1 x 128 blocks, 326 to 350 in 128 x
// 128 (5.3 to 5.9 TB/s, 81 to 90 % of a measured copy), fp32 32,768 x 4,096 97 us;
// rows that are no multiple of 16 bytes are read element by element (32,768 x
// 4,001: fp32 166 us, bf16 168). cols holds two to three thread blocks an SM, too
// few to hide its three barriers: 32,768 x 4,001, transposed, bf16 90 to 94 us
// (4.2 to 4.4 TB/s), in 128 x 128 blocks 85, fp32 127, fp16 104 (its 1 x 128 form
// spills some 120 bytes).
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_fp8.h>

#include "sts_internal.h"

namespace sts {
namespace {

constexpr int kBlock = 128;
constexpr int kThreads = 256;

constexpr float kLargest = 3.402823466e+38f;

// 8 consecutive elements, as they were read. Absent ones are 0.
template <typename T>
struct Octet {
  static constexpr int kWords = (int)sizeof(T) / 2;
  uint4 w[kWords];

  template <bool kVec>
  __device__ __forceinline__ void load(const T* p, int live) {
    if (kVec && live >= 8) {
#pragma unroll
      for (int i = 0; i < kWords; ++i) w[i] = __ldg(reinterpret_cast<const uint4*>(p) + i);
    } else {
      union {
        uint4 q[kWords];
        T e[8];
      } u;
#pragma unroll
      for (int i = 0; i < kWords; ++i) u.q[i] = make_uint4(0, 0, 0, 0);
#pragma unroll
      for (int i = 0; i < 8; ++i)
        if (i < live) u.e[i] = p[i];
#pragma unroll
      for (int i = 0; i < kWords; ++i) w[i] = u.q[i];
    }
  }
  __device__ __forceinline__ void get(float (&v)[8]) const;
  __device__ __forceinline__ float at(int j) const {  // j a constant where it is called
    float v[8];
    get(v);
    return v[j];
  }
};

__device__ __forceinline__ void words(const uint4& w, uint32_t (&u)[4]) {
  u[0] = w.x;
  u[1] = w.y;
  u[2] = w.z;
  u[3] = w.w;
}

template <>
__device__ __forceinline__ void Octet<float>::get(float (&v)[8]) const {
  uint32_t u[4];
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    words(w[h], u);
#pragma unroll
    for (int i = 0; i < 4; ++i) v[4 * h + i] = __uint_as_float(u[i]);
  }
}
template <>
__device__ __forceinline__ void Octet<__nv_bfloat16>::get(float (&v)[8]) const {
  uint32_t u[4];
  words(w[0], u);
#pragma unroll
  for (int i = 0; i < 4; ++i) {  // a bf16 is the upper half of its fp32
    v[2 * i] = __uint_as_float(u[i] << 16);
    v[2 * i + 1] = __uint_as_float(u[i] & 0xFFFF0000u);
  }
}
template <>
__device__ __forceinline__ void Octet<__half>::get(float (&v)[8]) const {
  uint32_t u[4];
  words(w[0], u);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&u[i]));
    v[2 * i] = f.x;
    v[2 * i + 1] = f.y;
  }
}

// Element-wise largest |.| of octets (a NaN is passed over), on packed pairs.
template <typename T>
struct Largest;

template <>
struct Largest<float> {
  float m[8];
  __device__ __forceinline__ Largest() {
#pragma unroll
    for (int i = 0; i < 8; ++i) m[i] = 0.f;
  }
  __device__ __forceinline__ void add(const Octet<float>& o) {
    float v[8];
    o.get(v);
#pragma unroll
    for (int i = 0; i < 8; ++i) m[i] = fmaxf(m[i], fabsf(v[i]));
  }
  __device__ __forceinline__ void get(float (&v)[8]) const {
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = m[i];
  }
};

template <typename P>
struct LargestPairs {
  P m[4];
  __device__ __forceinline__ LargestPairs() {
    const uint32_t zero = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) m[i] = *reinterpret_cast<const P*>(&zero);
  }
  template <typename T>
  __device__ __forceinline__ void add(const Octet<T>& o) {
    uint32_t u[4];
    words(o.w[0], u);
#pragma unroll
    for (int i = 0; i < 4; ++i) m[i] = __hmax2(m[i], __habs2(*reinterpret_cast<const P*>(&u[i])));
  }
};
template <>
struct Largest<__nv_bfloat16> : LargestPairs<__nv_bfloat162> {
  __device__ __forceinline__ void get(float (&v)[8]) const {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 f = __bfloat1622float2(m[i]);
      v[2 * i] = f.x;
      v[2 * i + 1] = f.y;
    }
  }
};
template <>
struct Largest<__half> : LargestPairs<__half2> {
  __device__ __forceinline__ void get(float (&v)[8]) const {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 f = __half22float2(m[i]);
      v[2 * i] = f.x;
      v[2 * i + 1] = f.y;
    }
  }
};

__device__ __forceinline__ float most(const float (&v)[8]) {
  return fmaxf(fmaxf(fmaxf(v[0], v[1]), fmaxf(v[2], v[3])),
               fmaxf(fmaxf(v[4], v[5]), fmaxf(v[6], v[7])));
}

// The largest finite |.| of kN octets; `inf` where an infinity is among them
// (they are then looked through once more without it).
template <typename T, int kN>
__device__ __forceinline__ float largest_of(const Octet<T> (&o)[kN], bool& inf) {
  Largest<T> l;
#pragma unroll
  for (int i = 0; i < kN; ++i) l.add(o[i]);
  float v[8];
  l.get(v);
  float m = most(v);
  inf = m > kLargest;
  if (inf) {
    m = 0.f;
#pragma unroll
    for (int i = 0; i < kN; ++i) {
      o[i].get(v);
#pragma unroll
      for (int j = 0; j < 8; ++j) m = fmaxf(m, fabsf(v[j]) <= kLargest ? fabsf(v[j]) : 0.f);
    }
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

// Codes of 8 entries; `inf`: infinities may be among them.
template <bool kE5>
__device__ __forceinline__ uint2 code8(const float (&v)[8], const Scale& sc, bool inf) {
  float y[8];
  if (sc.s >= 1.17549435e-38f) {
#pragma unroll
    for (int i = 0; i < 8; ++i) y[i] = v[i] * sc.inv;
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) y[i] = __fdiv_rn(v[i], sc.s);
  }
  if (inf) {  // the conversion would limit them to +-top
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (fabsf(v[i]) > kLargest) y[i] = __int_as_float(0x7fc00000);
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
  int width;   // rows1: blocks along K per thread block
  bool q_vec;  // q rows start on 8-byte boundaries
};

// 1 x 128 blocks along contiguous K: 4 lanes a block, 64 blocks a thread block
// (`width` of them, a power of two, along K and 64 / width rows). Lane i of the
// four holds the 16-byte pieces i, i + 4, ..
template <typename T, bool kE5, bool kVec>
__global__ void __launch_bounds__(kThreads) rows1_kernel(const QuantArgs a) {
  const int sub = threadIdx.x & 3, at = threadIdx.x >> 2;
  const int64_t r = (int64_t)blockIdx.x * (64 / a.width) + at / a.width;
  for (int64_t kb = (int64_t)blockIdx.y * a.width + at % a.width;; kb += (int64_t)gridDim.y * a.width) {
    // the four lanes of a block agree; whole warps leave together
    const bool mine = r < a.R && kb < a.k_blocks;
    if (__ballot_sync(0xFFFFFFFFu, mine) == 0) break;
    const int64_t k = kb * kBlock + sub * 8;
    const T* x = static_cast<const T*>(a.x) + r * a.ld + k;
    const int left = mine ? (int)min(a.K - k, (int64_t)kBlock) : 0;
    Octet<T> o[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) o[i].template load<kVec>(x + 32 * i, left - 32 * i);
    bool inf;
    float m = largest_of(o, inf);
    m = fmaxf(m, __shfl_xor_sync(0xFFFFFFFFu, m, 1));
    m = fmaxf(m, __shfl_xor_sync(0xFFFFFFFFu, m, 2));
    if (!mine) continue;
    const Scale s = block_scale<kE5>(m);
    if (sub == 0) a.scale[r * a.scale_ld + kb] = s.s;
    uint8_t* q = a.q + r * a.q_ld + k;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      float v[8];
      o[i].get(v);
      store8(q + 32 * i, code8<kE5>(v, s, inf), left - 32 * i, a.q_vec);
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
__global__ void __launch_bounds__(kThreads, sizeof(T) == 2 ? 3 : 2) rows128_kernel(const QuantArgs a) {
  __shared__ float warp_max[kThreads / 32];
  const int64_t rb = (int64_t)blockIdx.x / a.k_blocks;
  const int64_t kb = (int64_t)blockIdx.x - rb * a.k_blocks;
  const int64_t k = kb * kBlock + (threadIdx.x & 15) * 8;
  const int64_t left = a.K - k;
  const int live = left >= 8 ? 8 : (left > 0 ? (int)left : 0);
  const int64_t r0 = rb * kBlock + (threadIdx.x >> 4);
  Octet<T> o[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int64_t r = r0 + 16 * i;
    o[i].template load<kVec>(static_cast<const T*>(a.x) + r * a.ld + k, r < a.R ? live : 0);
  }
  bool inf;
  const float m = largest_of(o, inf);
  const Scale s = block_scale<kE5>(block_max(m, warp_max));
  if (threadIdx.x == 0) a.scale[rb * a.scale_ld + kb] = s.s;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int64_t r = r0 + 16 * i;
    float v[8];
    o[i].get(v);
    if (r < a.R) store8(a.q + r * a.q_ld + k, code8<kE5>(v, s, inf), live, a.q_vec);
  }
}

// x's rows are contiguous: element (r, k) at x[r + k * ld]. 128 x 128 elements
// per thread block; thread t holds the 8 rows 8 (t % 16).. of the 8 columns
// 8 (t / 16)... The codes cross shared memory as [row][16 groups of 8 k], the
// group index exclusive-ored with row / 8 so that neither side meets a bank
// conflict.
template <typename T, bool kE5, bool kVec, bool kSquare>
__global__ void __launch_bounds__(kThreads, sizeof(T) == 2 ? 3 : 2) cols_kernel(const QuantArgs a) {
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
  Octet<T> o[8];  // [k]: 8 rows each
#pragma unroll
  for (int i = 0; i < 8; ++i)
    o[i].template load<kVec>(static_cast<const T*>(a.x) + (k + i) * a.ld + r, k + i < a.K ? live : 0);
  Scale s[kSquare ? 1 : 8];
  bool inf;
  if constexpr (kSquare) {
    const float m = largest_of(o, inf);
    s[0] = block_scale<kE5>(block_max(m, warp_max));
    if (threadIdx.x == 0) a.scale[rb * a.scale_ld + kb] = s[0].s;
  } else {
    Largest<T> l;  // of each of the 8 rows
#pragma unroll
    for (int i = 0; i < 8; ++i) l.add(o[i]);
    float m[8];
    l.get(m);
    inf = most(m) > kLargest;
    if (inf) {
#pragma unroll
      for (int j = 0; j < 8; ++j) m[j] = 0.f;
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        float v[8];
        o[i].get(v);
#pragma unroll
        for (int j = 0; j < 8; ++j) m[j] = fmaxf(m[j], fabsf(v[j]) <= kLargest ? fabsf(v[j]) : 0.f);
      }
    }
#pragma unroll
    for (int j = 0; j < 8; ++j) row_max[kg][oct * 8 + j] = m[j];
    __syncthreads();
    if (threadIdx.x < kBlock) {
      float x = 0.f;
#pragma unroll
      for (int g = 0; g < 16; ++g) x = fmaxf(x, row_max[g][threadIdx.x]);
      const Scale sc = block_scale<kE5>(x);
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
    for (int i = 0; i < 8; ++i) w[i] = o[i].at(j);
    codes[oct * 8 + j][kg ^ oct] = code8<kE5>(w, s[kSquare ? 0 : j], inf);
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
cudaError_t launch(const QuantArgs& a, bool transposed, int block_rows, cudaStream_t st) {
  if (!transposed && block_rows == 1) {
    const int64_t rows = 64 / a.width;
    const int64_t along = (a.k_blocks + a.width - 1) / a.width;
    const dim3 grid((unsigned)((a.R + rows - 1) / rows), (unsigned)(along < 65535 ? along : 65535));
    rows1_kernel<T, kE5, kVec><<<grid, kThreads, 0, st>>>(a);
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
cudaError_t launch_t(const QuantArgs& a, bool e5, bool transposed, int block_rows,
                     cudaStream_t st) {
  // 16-byte loads need 16-byte rows; any other layout is read element by element
  const bool vec = (reinterpret_cast<uintptr_t>(a.x) & 15u) == 0 &&
                   (a.ld * (int64_t)sizeof(T)) % 16 == 0;
  if (vec)
    return e5 ? launch<T, true, true>(a, transposed, block_rows, st)
              : launch<T, false, true>(a, transposed, block_rows, st);
  return e5 ? launch<T, true, false>(a, transposed, block_rows, st)
            : launch<T, false, false>(a, transposed, block_rows, st);
}

// Rows of bytes in memory, at least their width apart.
struct Rows {
  uintptr_t at;
  int64_t n;
  uintptr_t pitch, width;
  uintptr_t end() const { return at + (uintptr_t)(n - 1) * pitch + width; }
};

// Whether a row of one meets a row of the other. Rows of one pitch, side by side
// (codes and their scales in one record), and rows that lie apart are told at once.
bool meet(Rows a, Rows b) {
  if (a.n < 1 || b.n < 1 || a.end() <= b.at || b.end() <= a.at) return false;
  if (a.n > 1 && b.n > 1 && a.pitch == b.pitch) {
    const uintptr_t p = a.pitch, d = b.at >= a.at ? (b.at - a.at) % p : (p - (a.at - b.at) % p) % p;
    if (d >= a.width && d + b.width <= p) return false;
  }
  if (b.n < a.n) {
    const Rows c = a;
    a = b;
    b = c;
  }
  for (int64_t i = 0; i < a.n; ++i) {
    const uintptr_t from = a.at + (uintptr_t)i * a.pitch, to = from + a.width;
    if (to <= b.at) continue;
    // the last of b's rows that starts before this one ends
    const uintptr_t j = b.n > 1 ? (to - 1 - b.at) / b.pitch : 0;
    const uintptr_t last = j < (uintptr_t)b.n ? j : (uintptr_t)b.n - 1;
    if (b.at + last * b.pitch + b.width > from) return true;
  }
  return false;
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
  const unsigned es = x_dtype == STS_DTYPE_F32 ? 4 : 2;
  if (reinterpret_cast<uintptr_t>(x) % es != 0 || (reinterpret_cast<uintptr_t>(scale) & 3u) != 0)
    return STS_ERR_SHAPE;
  // blocks are written while others are still to be read
  const int64_t scale_rows = block_rows == 1 ? R : (R + kBlock - 1) / kBlock;
  const Rows in{reinterpret_cast<uintptr_t>(x), transposed ? K : R, (uintptr_t)ld * es,
                (uintptr_t)(transposed ? R : K) * es};
  const Rows codes{reinterpret_cast<uintptr_t>(q), R, (uintptr_t)q_ld, (uintptr_t)K};
  const Rows scales{reinterpret_cast<uintptr_t>(scale), scale_rows, (uintptr_t)scale_ld * 4,
                    (uintptr_t)k_blocks * 4};
  if (meet(in, codes) || meet(in, scales) || meet(codes, scales)) return STS_ERR_SHAPE;
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
  // as many blocks along K as leave at most an eighth of them without work
  a.width = 64;
  while (a.width > 1 && ((k_blocks + a.width - 1) / a.width * a.width - k_blocks) * 8 > k_blocks)
    a.width /= 2;
  a.q_vec = (reinterpret_cast<uintptr_t>(q) & 7u) == 0 && q_ld % 8 == 0;
  if (a.row_blocks * k_blocks > kMost) return STS_ERR_SHAPE;
  int sms = 0;
  const sts_status ds = current_device(&sms);
  if (ds != STS_OK) return ds;
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  const LaunchMark mark = launch_begin(STS_KERNEL_BLOCK_QUANTIZE, st);
  const bool e5 = q_dtype == STS_DTYPE_E5M2;
  const cudaError_t e =
      x_dtype == STS_DTYPE_F32    ? launch_t<float>(a, e5, transposed, block_rows, st)
      : x_dtype == STS_DTYPE_BF16 ? launch_t<__nv_bfloat16>(a, e5, transposed, block_rows, st)
                                  : launch_t<__half>(a, e5, transposed, block_rows, st);
  launch_end(mark, st);
  return e == cudaSuccess ? STS_OK : STS_ERR_CUDA;
}
