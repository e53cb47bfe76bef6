// Log probabilities of given tokens, entropy and top alternatives of rows of
// logits, and their gradient.
//
// With z the logits of one row, tau its temperature, M = max_i z_i and
// d_i = (z_i - M) / tau:
//   S        = sum_i exp(d_i)
//   log_sum  = ln S,   lse = M / tau + log_sum
//   logprob  = d_y - log_sum                        for each given token y
//   entropy  = ln S - (sum_i exp(d_i) d_i) / S
//   top n    = the first n tokens in (z descending, id ascending) order
// and for L with dL/dlogprob_j = g_j, dL/dentropy = h, dL/dtop_j = g'_j:
//   dL/dz_i  = (1 / tau) [ sum_{j: y_j = i} g_j - p_i (G + h (ln p_i + entropy)) ]
// where G is the sum of every g_j and g'_j whose token has a probability.
//
// One pass over the row in each direction; HBM bounds both. The forward's
// running sums are taken against a fixed base b instead of a running maximum:
//   x_i = c z_i - b,  c = log2(e) / tau,  S' = sum 2^x_i,  S'_1 = sum 2^x_i x_i
// Any base gives the same quotients, so b is c times the maximum of the first
// chunk of 2,048 to 8,192 elements and moves, a thread at a time, only when an
// element, or the bound of the alternatives (below), exceeds it by more than a
// factor of 2 (a larger x would carry a larger rounding into the terms that
// matter, and from 128 on 2^x is infinite). An element costs a clamp, an FMA, an
// exponential and two sums; fp32 logits a second FMA, for what c's rounding
// leaves (16-bit logits are themselves rounded by 2^-9 or 2^-11; there c's 2^-24
// is a temperature half a step off, put right in log_sum by its derivative). The clamp keeps x at -200 or above (2^-200 is 0 in
// fp32), so that masked logits put no 0 * inf into S'_1. Each thread's sums
// (fp32, two of each) are joined in float64. Rows whose largest c z_i leaves
// fp32's exact range, 2^20 (nothing but masks of the type's lowest value, say),
// form x from differences of logits instead.
//
// The alternatives ride in the same loop: a lower bound of the n-th largest
// element (the n-th largest of group maxima of the first chunk, tightened as
// the row goes on) is compared with the maximum of each 4 or 8 elements, and
// only what lies above it is kept as a 64-bit key (monotone logit bits above
// the inverted id, so that the order of keys is the order of alternatives).
// Keys that outgrow the buffer (ascending rows, rows of equal logits) are
// dropped and the row's share is searched again digit by digit.
//
// The logits come by bulk copies into two buffers of shared memory a block, so
// that the next chunk is on its way while one is summed, without a register
// spent on it; the last warp to have read a buffer orders its next chunk.
//
// A row is a thread block's, or, where there are too few rows to fill the
// GPU, that of a cluster of 2, 4 or 8 blocks, each with a stretch of the
// vocabulary; the first block joins their results over distributed shared
// memory. One launch, no workspace, nothing shared between calls.
//
// What it takes. The gradient: 4,096 rows of 152,064 bf16 logits 390 us in short
// bursts, 398 to 416 back to back (6.0 to 6.4 TB/s, 91 to 97 % of a measured copy);
// to fp32 645 to 655 (6.9 GB; the form spills 32 bytes). Rows of logits and result
// on different 16-byte boundaries: 555 for types of one width, 2,100 for bf16 to
// fp32, whose elements are then stored one by one. The forward: the same rows 275 to
// 290 us without alternatives, 303 to 315 with 8, 451 with 64 (HBM: 190); 2,048
// rows of 151,936 fp32 with 20 258 to 276 (190). It issues 2.7 to 3 instructions a clock (some 10 an element, and
// one exponential, which alone would take as long as the bytes do); 64
// alternatives cost 2,400 instructions a row and warp more, in ranking them at
// each doubling of the row. Packed fp32 operations lost more in moves than they
// saved, loads by registers waited for memory, and a prefetch of them spilled.
#include <cmath>
#include <type_traits>

#include <cooperative_groups.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "sts_device.cuh"

namespace sts {
namespace {

namespace cg = cooperative_groups;

constexpr int kThreads = 256;     // of the gradient, and of the forward for long rows
constexpr int kUnroll = 4;       // 16-byte loads in flight per thread
constexpr int kBuffers = 2;      // of one chunk each: threads x kUnroll x 16 bytes
constexpr int kMaxTop = 64;      // alternatives per row
constexpr int kMaxGiven = 512;   // given tokens per row
constexpr int kMaxParts = 8;     // portable cluster size
constexpr int kKeyCap = 1024;    // keys kept between two tightenings
// Rows up to this long have blocks of 128 threads, so that more of them are in
// flight: 8,192 rows of 1,024 fp32 take 62 us (256 threads: 104), of 16,000 bf16 101
// (123); one row of 151,936 fp32 23 us (18.5), 4,096 rows of 152,064 bf16 the same.
// A few hundred rows of tens of thousands would be faster with 256 threads (500 of
// 30,000 bf16: 24.7 us, 20.5).
constexpr int64_t kShortRow = 65536;
constexpr double kLog2eD = 1.4426950408889634074;
constexpr double kLn2 = 0.69314718055994530942;
constexpr float kNegInf = -INFINITY;

// log2(e) / tau, finite for every tau > 0
__device__ __forceinline__ double exponent_scale(float tau) {
  return fmin(kLog2eD / (double)tau, 3.402823466e+38);
}

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// The larger one, NaN where either is NaN.
__device__ __forceinline__ float max_nan(float a, float b) {
  float y;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(y) : "f"(a), "f"(b));
  return y;
}

__device__ __forceinline__ float to_f32(float v) { return v; }
__device__ __forceinline__ float to_f32(__nv_bfloat16 v) { return __bfloat162float(v); }
__device__ __forceinline__ float to_f32(__half v) { return __half2float(v); }
__device__ __forceinline__ void from_f32(float v, float& o) { o = v; }
__device__ __forceinline__ void from_f32(float v, __nv_bfloat16& o) { o = __float2bfloat16_rn(v); }
__device__ __forceinline__ void from_f32(float v, __half& o) { o = __float2half_rn(v); }

// 16 bytes of logits.
template <typename T>
struct Vec {
  static constexpr int kN = 16 / (int)sizeof(T);
  uint4 w;
  __device__ __forceinline__ void none() {  // all -inf
    constexpr uint32_t k = std::is_same<T, float>::value           ? 0xFF800000u
                           : std::is_same<T, __nv_bfloat16>::value ? 0xFF80FF80u
                                                                   : 0xFC00FC00u;
    w = make_uint4(k, k, k, k);
  }
  __device__ __forceinline__ void f32(float (&v)[kN]) const;
  __device__ __forceinline__ float at(int k) const {  // one element, chosen at run time
    constexpr int kPer = 4 / (int)sizeof(T);
    const int i = k / kPer;
    const uint32_t u = i == 0 ? w.x : i == 1 ? w.y : i == 2 ? w.z : w.w;
    if constexpr (kPer == 1) return __uint_as_float(u);
    const uint16_t h = (uint16_t)(u >> ((k & 1) * 16));
    return to_f32(*reinterpret_cast<const T*>(&h));
  }
};

template <>
__device__ __forceinline__ void Vec<float>::f32(float (&v)[4]) const {
  v[0] = __uint_as_float(w.x);
  v[1] = __uint_as_float(w.y);
  v[2] = __uint_as_float(w.z);
  v[3] = __uint_as_float(w.w);
}
template <>
__device__ __forceinline__ void Vec<__nv_bfloat16>::f32(float (&v)[8]) const {
  const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {  // a bf16 is the upper half of its fp32
    v[2 * i] = __uint_as_float(u[i] << 16);
    v[2 * i + 1] = __uint_as_float(u[i] & 0xFFFF0000u);
  }
}
template <>
__device__ __forceinline__ void Vec<__half>::f32(float (&v)[8]) const {
  const __half2* h = reinterpret_cast<const __half2*>(&w);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 f = __half22float2(h[i]);
    v[2 * i] = f.x;
    v[2 * i + 1] = f.y;
  }
}
// The largest element of kM vectors, NaN where one is NaN.
template <typename P, int kM>
__device__ __forceinline__ P largest_pairs(const uint4* w) {
  P m[4];
#pragma unroll
  for (int u = 0; u < kM; ++u) {
    const P* h = reinterpret_cast<const P*>(w + u);
#pragma unroll
    for (int i = 0; i < 4; ++i) m[i] = u == 0 ? h[i] : __hmax2_nan(m[i], h[i]);
  }
  return __hmax2_nan(__hmax2_nan(m[0], m[1]), __hmax2_nan(m[2], m[3]));
}
template <typename T, int kM>
__device__ __forceinline__ float largest(const Vec<T> (&v)[kM]) {
  uint4 w[kM];
#pragma unroll
  for (int u = 0; u < kM; ++u) w[u] = v[u].w;
  if constexpr (std::is_same<T, float>::value) {
    float m = kNegInf;
#pragma unroll
    for (int u = 0; u < kM; ++u)
      m = max_nan(max_nan(m, max_nan(__uint_as_float(w[u].x), __uint_as_float(w[u].y))),
                  max_nan(__uint_as_float(w[u].z), __uint_as_float(w[u].w)));
    return m;
  } else if constexpr (std::is_same<T, __nv_bfloat16>::value) {
    const float2 f = __bfloat1622float2(largest_pairs<__nv_bfloat162, kM>(w));
    return max_nan(f.x, f.y);
  } else {
    const float2 f = __half22float2(largest_pairs<__half2, kM>(w));
    return max_nan(f.x, f.y);
  }
}

// fp32 bits as an unsigned number of the same order; -0 counts as +0.
__device__ __forceinline__ uint32_t order_bits(float z) {
  const uint32_t b = __float_as_uint(z + 0.f);
  return b ^ (((int32_t)b >> 31) | 0x80000000u);
}
__device__ __forceinline__ float order_value(uint32_t k) {
  return __uint_as_float(k ^ ((k & 0x80000000u) ? 0x80000000u : 0xFFFFFFFFu));
}
__device__ __forceinline__ uint64_t token_key(float z, uint32_t id) {
  return ((uint64_t)order_bits(z) << 32) | (uint32_t)~id;
}
__device__ __forceinline__ float key_logit(uint64_t k) { return order_value((uint32_t)(k >> 32)); }
__device__ __forceinline__ uint32_t key_id(uint64_t k) { return ~(uint32_t)k; }

struct FwdArgs {
  const void* z;
  int64_t ld;
  int64_t T;
  int V, parts, stretch;  // stretch: vocabulary entries per part
  const int64_t* tokens;
  int64_t tokens_ld;
  int m;
  const float* tau;
  int n;
  float* logprob;
  float *logit_max, *log_sum, *lse, *entropy;
  int32_t* flags;
  int64_t* top_id;
  float* top_logprob;
};

struct Share {  // what one block found in its stretch
  double s0, s1;
  double e;  // the exponent of their base
  int bad;
  int found;
};

template <int kT>
struct FwdSmem {
  uint4 ring[kBuffers][kT * kUnroll];
  uint64_t full[kBuffers];
  uint32_t read[kBuffers];  // warps that have read the buffer
  int abort;
  uint64_t keys[kKeyCap];
  uint64_t top[kMaxTop];
  uint64_t lists[kMaxParts][kMaxTop];
  Share share[kMaxParts];  // [0]: this block's; all of them in the joining block
  float group_max[kT];
  double red0[kT / 32], red1[kT / 32];
  double rede[kT / 32];
  float cut, chunk_max, log_sum;
  uint32_t count;
  uint32_t hist[256];
  uint32_t digit, above;
  uint32_t ties[kT / 32];
};

// Keys across a warp into descending order, lane 0 first.
__device__ __forceinline__ uint64_t sort_warp(uint64_t k) {
  const int lane = (int)threadIdx.x & 31;
#pragma unroll
  for (int size = 2; size <= 32; size *= 2) {
#pragma unroll
    for (int step = size / 2; step > 0; step /= 2) {
      const uint64_t o = __shfl_xor_sync(0xFFFFFFFFu, k, step);
      const bool larger = ((lane & step) == 0) == ((lane & size) == 0);  // this lane keeps it
      k = (o > k) == larger ? o : k;
    }
  }
  return k;
}

// The n largest of keys[0, c) (all different, none 0), in descending order, to
// out; keys[0, c rounded up to 32) is left as sorted runs of 32. Every thread of
// the block takes part; the barriers before and after are the caller's. A key's
// place is its own within its run and, by bisection, the number of larger keys
// in each other run: some 150 + 35 c / 32 instructions a key, beside the 4 c of
// comparing all with all.
template <int kT>
__device__ __forceinline__ void rank_keys(uint64_t* keys, int c, int n, uint64_t* out) {
  const int runs = (c + 31) / 32;
  for (int r = (int)threadIdx.x / 32; r < runs; r += kT / 32) {
    const int i = r * 32 + ((int)threadIdx.x & 31);
    keys[i] = sort_warp(i < c ? keys[i] : 0ull);
  }
  __syncthreads();
  for (int i = threadIdx.x; i < runs * 32; i += kT) {
    const uint64_t k = keys[i];
    if (k == 0ull) continue;
    int above = i & 31;
    for (int r = 0; r < runs && above < n; ++r) {
      if (r == i / 32) continue;
      const uint64_t* run = keys + r * 32;
      int at = 0;  // of the run's keys, the first that is not larger
#pragma unroll
      for (int step = 16; step > 0; step /= 2) at += run[at + step - 1] > k ? step : 0;
      above += at + (run[at] > k ? 1 : 0);
    }
    if (above < n) out[above] = k;
  }
}

// c = log2(e) / tau in two parts, and whether the thread's base is far: x = c (z - base)
struct Factor {
  float hi, lo;
  bool far;
};

// One thread's running sums against its base (a logit), in two halves.
struct Sums {
  float s0[2], s1[2];
  float base;   // x = 0 there
  float b;      // c base, rounded once: what the sums are really against
  float least;  // logits below it count as this one
};
constexpr float kLowest = -3.402823466e+38f;  // the base before anything was seen
constexpr float kFar = 1048576.f;  // c base beyond it: far (its rounding would be an exponent's size)

// The exponent of the sums' base, exactly: x = c z - this (far: c (z - base)).
__device__ __forceinline__ double base_exponent(const Sums& s, bool far, double c) {
  return far ? __dmul_rn(c, (double)s.base) : (double)s.b;
}

__device__ __forceinline__ void shift(Sums& s, float to, float b, float by, const Factor& c) {
  const float f = ex2(fmaxf(by, -200.f));
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    s.s1[h] = f == 0.f ? 0.f : fmaf(by, s.s0[h], s.s1[h]) * f;
    s.s0[h] *= f;
  }
  s.base = to;
  s.b = b;
  s.least = fmaxf(to - 200.f / c.hi, kLowest);
}

// Moves the base (upwards; the sums are 0 where it is kLowest), and the thread
// between the near and the far form as the new base has it.
__device__ __forceinline__ void rebase(Sums& s, float to, Factor& c) {
  const float b = to * c.hi;
  const bool far = !(fabsf(b) < kFar) || !(200.f / c.hi < 1e30f);
  float by;  // the old base's exponent over the new one's: 0 or less
  if (far)
    by = c.far ? (s.base - to) * c.hi : -fmaf(to, c.lo, fmaf(to, c.hi, -s.b));
  else
    by = c.far ? fmaf(s.base, c.lo, fmaf(s.base, c.hi, -b)) : s.b - b;
  shift(s, to, b, by, c);
  c.far = far;
}

template <bool kFarForm, bool kTwo>
__device__ __forceinline__ void add(Sums& s, int h, float z, const Factor& c) {
  float x;
  if (kFarForm) {
    const float d = z - s.base;
    // (a masked logit may give NaN here, -inf times both parts of c: fmaxf drops it)
    x = fmaxf(fmaf(d, c.lo, d * c.hi), -200.f);
  } else {
    const float y = fmaxf(z, s.least);
    x = fmaf(y, c.hi, -s.b);
    if (kTwo) x = fmaf(y, c.lo, x);
  }
  const float e = ex2(x);
  s.s0[h] += e;
  s.s1[h] = fmaf(e, x, s.s1[h]);
}

template <int kT>
__device__ __forceinline__ void keep(FwdSmem<kT>& sm, float z, uint32_t id) {
  const uint32_t at = atomicAdd(&sm.count, 1u);
  if (at < (uint32_t)kKeyCap) sm.keys[at] = token_key(z, id);
}

template <int kT>
__device__ __forceinline__ void keep_above(FwdSmem<kT>& sm, float z, uint32_t id, float cut,
                                           bool or_equal) {
  if (z > cut || (or_equal && z == cut && z > kNegInf)) keep(sm, z, id);
}

// The n largest of the stretch, digit by digit, for rows whose keys did not
// fit: four histograms fix the n-th largest logit, then everything above it is
// collected, and the ties at it in order of their ids.
template <typename T, int kT>
__device__ __noinline__ int search_again(FwdSmem<kT>& sm, const T* z, int len, uint32_t id0, int n) {
  uint32_t prefix = 0, want = (uint32_t)n;
  for (int shift = 24; shift >= 0; shift -= 8) {
    __syncthreads();
    for (int i = threadIdx.x; i < 256; i += kT) sm.hist[i] = 0;
    __syncthreads();
    const uint32_t mask = shift == 24 ? 0u : 0xFFFFFFFFu << (shift + 8);
    for (int i = threadIdx.x; i < (len + 31) / 32 * 32; i += kT) {
      bool in = false;
      uint32_t digit = 0;
      if (i < len) {
        const float v = to_f32(z[i]);
        const uint32_t b = order_bits(v);
        in = v > kNegInf && (b & mask) == (prefix & mask);
        digit = (b >> shift) & 255u;
      }
      const uint32_t same = __match_any_sync(0xFFFFFFFFu, in ? digit : 256u);
      if (in && (__ffs((int)same) - 1) == (int)(threadIdx.x & 31))
        atomicAdd(&sm.hist[digit], (uint32_t)__popc(same));
    }
    __syncthreads();
    if (threadIdx.x == 0) {
      uint32_t seen = 0;
      int b = 255;
      for (; b > 0; --b) {
        if (seen + sm.hist[b] >= want) break;
        seen += sm.hist[b];
      }
      sm.digit = (uint32_t)b;
      sm.above = seen;
    }
    __syncthreads();
    prefix |= sm.digit << shift;
    want -= min(want, sm.above);
  }
  // prefix: the n-th largest logit (or less, where fewer are there); `want` ties
  __syncthreads();
  if (threadIdx.x == 0) sm.count = 0;
  __syncthreads();
  uint32_t ties = 0;
  for (int i0 = 0; i0 < len; i0 += kT) {
    const int i = i0 + (int)threadIdx.x;
    bool tie = false;
    float v = kNegInf;
    if (i < len) {
      v = to_f32(z[i]);
      const uint32_t b = order_bits(v);
      if (v > kNegInf && b > prefix) keep(sm, v, id0 + (uint32_t)i);
      tie = v > kNegInf && b == prefix;
    }
    if (ties < want) {  // the same in every thread
      const uint32_t ballot = __ballot_sync(0xFFFFFFFFu, tie);
      if ((threadIdx.x & 31) == 0) sm.ties[threadIdx.x >> 5] = (uint32_t)__popc(ballot);
      __syncthreads();
      uint32_t before = ties, all = ties;
      for (int w = 0; w < kT / 32; ++w) {
        if (w < (int)(threadIdx.x >> 5)) before += sm.ties[w];
        all += sm.ties[w];
      }
      before += (uint32_t)__popc(ballot & ((1u << (threadIdx.x & 31)) - 1u));
      if (tie && before < want) keep(sm, v, id0 + (uint32_t)i);
      ties = all;
      __syncthreads();
    }
  }
  __syncthreads();
  return (int)min(sm.count, (uint32_t)kKeyCap);
}

// The first bound, from one chunk (m: the maximum of this thread's vectors):
// sm.cut is the n-th largest of `groups` group maxima, and sm.chunk_max the
// largest; -inf where fewer than n groups hold anything. NaN counts as nothing.
template <int kT>
__device__ __forceinline__ void first_bound(FwdSmem<kT>& sm, float m, int groups, int n) {
  const int tid = threadIdx.x;
  const int per_group = kT / groups;
  for (int o = 1; o < per_group; o *= 2) m = fmaxf(m, __shfl_xor_sync(0xFFFFFFFFu, m, o));
  if ((tid & (per_group - 1)) == 0) sm.group_max[tid / per_group] = m;
  if (tid == 0) sm.cut = kNegInf;
  __syncthreads();
  // per_group lanes share a group's count of those above it
  const int mine = tid / per_group, sub = tid & (per_group - 1);
  const float v = sm.group_max[mine];
  int above = 0;
#pragma unroll 4
  for (int j = sub; j < groups; j += per_group) {
    const float o = sm.group_max[j];
    above += (o > v || (o == v && j < mine)) ? 1 : 0;
  }
  for (int o = 1; o < per_group; o *= 2) above += __shfl_xor_sync(0xFFFFFFFFu, above, o);
  if (v > kNegInf && sub == 0) {
    if (above == n - 1) sm.cut = v;
    if (above == 0) sm.chunk_max = v;
  }
  __syncthreads();
}

template <typename T, int kT>
__global__ void __launch_bounds__(kT, 1024 / kT) forward_kernel(const FwdArgs a) {
  extern __shared__ __align__(128) uint8_t smem_raw[];
  FwdSmem<kT>& sm = *reinterpret_cast<FwdSmem<kT>*>(smem_raw);
  constexpr int kN = Vec<T>::kN;
  constexpr int kChunk = kT * kUnroll;  // vectors
  constexpr bool kTwo = sizeof(T) == 4;  // c in two parts
  const int parts = a.parts;
  const int64_t row = (int64_t)blockIdx.x / parts;
  const int part = (int)((int64_t)blockIdx.x - row * parts);
  const int tid = threadIdx.x;
  const int n = max(a.n, 1);  // the first alternative gives the maximum
  const int v0 = (int)min((int64_t)part * a.stretch, (int64_t)a.V);
  const int len = min(a.stretch, a.V - v0);
  const T* z = static_cast<const T*>(a.z) + row * a.ld + v0;
  // [0, head): up to the first 16-byte boundary; [head, head + body kN): vectors
  const int head = min((int)((16u - (uint32_t)(reinterpret_cast<uintptr_t>(z) & 15u)) % 16u) /
                           (int)sizeof(T), len);
  const int body = (len - head) / kN;
  const int tail0 = head + body * kN;
  const T* zb = z + head;

  // chunk number i of the stretch into its buffer
  auto order = [&](int i) {
    const int i0 = i * kChunk, n16 = min(kChunk, body - i0);
    const uint32_t bar = smem_u32(&sm.full[i % kBuffers]);
    mbar_arrive_expect_tx(bar, (uint32_t)n16 * 16u);
    bulk_load(smem_u32(sm.ring[i % kBuffers]), zb + (int64_t)i0 * kN, (uint32_t)n16 * 16u, bar);
  };
  const int chunks = (body + kChunk - 1) / kChunk;
  if (tid == 0) {
    sm.count = 0;
    sm.abort = 0;
    for (int b = 0; b < kBuffers; ++b) {
      mbar_init(smem_u32(&sm.full[b]), 1);
      sm.read[b] = 0;
    }
    fence_barrier_init();
    fence_proxy_async_smem();
    for (int i = 0; i < min(kBuffers, chunks); ++i) order(i);
  }
  const float tau = a.tau ? a.tau[row] : 1.f;  // on its way while the barriers are made
  __syncthreads();
  const bool tau_ok = tau > 0.f && tau < INFINITY;
  const double cd = exponent_scale(tau_ok ? tau : 1.f);
  Factor c;
  c.hi = (float)cd;
  c.lo = (float)(cd - (double)c.hi);
  c.far = true;  // until a maximum shows that it is not

  // the block's first given tokens and their logits, while the row arrives
  const T* zrow = static_cast<const T*>(a.z) + row * a.ld;
  int64_t token = -1;
  float token_logit = kNegInf;
  if (part == 0 && tid < a.m) {
    token = a.tokens[row * a.tokens_ld + tid];
    if (token >= 0 && token < a.V) token_logit = to_f32(zrow[token]);
  }

  Sums s{{0.f, 0.f}, {0.f, 0.f}, kLowest, 0.f, kLowest};
  float cut = kNegInf;   // nothing at or below it can be an alternative any more
  float seen = kNegInf;  // only to catch NaN and inf: the maximum of what was looked at closely
  int groups = 32;       // group maxima for the first bound: 2 n at least
  while (groups < 2 * n && groups < kT) groups *= 2;

  bool bound = false;  // a finite bound has been found (the same in every thread)
  // the keys are about n by the first chunk, n more for each doubling of the row
  int next_tighten = n > 16 ? 2 : 4;
  bool late = false;  // a copy that never came
  for (int it = 0; it < max(chunks, 1); ++it) {
    const int i0 = it * kChunk, buf = it % kBuffers;
    Vec<T> v[kUnroll];
    if (it < chunks) {
      late |= !mbar_wait_soon(smem_u32(&sm.full[buf]), (uint32_t)(it / kBuffers) & 1u, &sm.abort, nullptr);
      if (i0 + kChunk <= body) {
#pragma unroll
        for (int u = 0; u < kUnroll; ++u) v[u].w = sm.ring[buf][u * kT + tid];
      } else {
#pragma unroll
        for (int u = 0; u < kUnroll; ++u) {
          if (i0 + u * kT + tid < body)
            v[u].w = sm.ring[buf][u * kT + tid];
          else
            v[u].none();
        }
      }
    } else {  // a stretch without a whole vector
#pragma unroll
      for (int u = 0; u < kUnroll; ++u) v[u].none();
    }
    const float vmax = largest(v);  // NaN where one is
    bool equal = false;  // whether ties with the bound still count
    float raise = kNegInf;  // where this thread's base moves to
    if (!bound) {
      first_bound(sm, vmax, groups, n);
      if (sm.cut > kNegInf) {
        bound = true;
        equal = true;  // the n elements of the bound are of this very chunk
        cut = sm.cut;
        // the base: the chunk's maximum
        raise = fmaxf(fminf(sm.chunk_max, -kLowest), s.base);
      }
      __syncthreads();  // group_max, cut and chunk_max are free again
    } else if (it >= next_tighten && a.n > 1) {
      next_tighten *= n > 16 ? 2 : 4;
      __syncthreads();
      const int cnt = (int)min(sm.count, (uint32_t)kKeyCap);
      const bool whole = sm.count <= (uint32_t)kKeyCap;
      if (whole && cnt > n) {
        rank_keys<kT>(sm.keys, cnt, n, sm.top);
        __syncthreads();
        if (tid < n) sm.keys[tid] = sm.top[tid];
        if (tid == 0) sm.count = (uint32_t)n;
        cut = fmaxf(cut, key_logit(sm.top[n - 1]));
        // what lies below the bound is not looked at, so no base stays behind it
        if ((cut - s.base) * c.hi > 1.f && cut < INFINITY) raise = cut;
      }
      __syncthreads();
    }
    if (raise > kNegInf) rebase(s, raise, c);
    // Something above the bound (or at it while ties count; without one, above
    // -inf), or a NaN: the warp looks at the thread's elements together, a lane each, in the
    // buffer (rare: about n elements for each doubling of the row). The thread
    // moves its base first.
    const bool look = equal ? !(vmax < cut) : !(vmax <= cut);
    uint32_t lookers = __ballot_sync(0xFFFFFFFFu, look);
    if (lookers != 0u) {
      if (look) {
        seen = max_nan(seen, vmax);
        if ((vmax - s.base) * c.hi > 1.f && vmax < INFINITY) rebase(s, vmax, c);
      }
      const int lane = tid & 31;
      do {
        const int owner = (tid & ~31) + __ffs((int)lookers) - 1;
        lookers &= lookers - 1u;
        const int i = lane / kN * kT + owner;  // of the chunk's vectors
        if (lane < kUnroll * kN && i0 + i < body) {
          const float f = to_f32(reinterpret_cast<const T*>(&sm.ring[buf][i])[lane % kN]);
          keep_above(sm, f, (uint32_t)(v0 + head + (i0 + i) * kN + lane % kN), cut, equal);
        }
      } while (lookers != 0u);
      __syncwarp();
    }
    if ((tid & 31) == 0 && it + kBuffers < chunks) {
      __threadfence_block();
      if (atomicAdd(&sm.read[buf], 1u) == (uint32_t)(kT / 32 - 1)) {
        sm.read[buf] = 0;
        __threadfence_block();
        fence_proxy_async_smem();
        order(it + kBuffers);
      }
    }
    __syncwarp();
    if (!c.far) {
#pragma unroll
      for (int u = 0; u < kUnroll; ++u) {
        float f[kN];
        v[u].f32(f);
#pragma unroll
        for (int k = 0; k < kN; ++k) add<false, kTwo>(s, k & 1, f[k], c);
      }
    } else {
      for (int u = 0; u < kUnroll; ++u) {
#pragma unroll 1
        for (int k = 0; k < kN; ++k) {
          Vec<T> x = v[0];
#pragma unroll
          for (int i = 1; i < kUnroll; ++i)
            if (u == i) x = v[i];
          add<true, kTwo>(s, 0, x.at(k), c);
        }
      }
    }
  }
  if (late && (tid & 31) == 0)  // no copy may outlive the block
    for (int i = max(0, chunks - kBuffers); i < chunks; ++i)
      mbar_wait_drain(smem_u32(&sm.full[i % kBuffers]), (uint32_t)(i / kBuffers) & 1u);
  // the elements outside the vectors: ids below (head) or above (tail) all others
  for (int i = tid; i < head + (len - tail0); i += kT) {
    const int at = i < head ? i : tail0 + (i - head);
    const float f = to_f32(z[at]);
    seen = max_nan(seen, f);
    keep_above(sm, f, (uint32_t)(v0 + at), cut, true);
    if ((f - s.base) * c.hi > 1.f && f < INFINITY) rebase(s, f, c);
    if (c.far)
      add<true, kTwo>(s, 0, f, c);
    else
      add<false, kTwo>(s, 0, f, c);
  }

  // ---- join the block's sums (float64) and find its n largest
  {
    const double own = base_exponent(s, c.far, cd);
    double e = own;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) e = fmax(e, __shfl_xor_sync(0xFFFFFFFFu, e, o));
    if ((tid & 31) == 0) sm.rede[tid >> 5] = e;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < kT / 32; ++w) e = fmax(e, sm.rede[w]);
    double s0 = (double)s.s0[0] + (double)s.s0[1], s1 = (double)s.s1[0] + (double)s.s1[1];
    if (own != e) {
      const double by = own - e;
      const double f = by < -300.0 ? 0.0 : exp2(by);
      s1 = f == 0.0 ? 0.0 : (s1 + by * s0) * f;
      s0 *= f;
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
      s0 += __shfl_xor_sync(0xFFFFFFFFu, s0, o);
      s1 += __shfl_xor_sync(0xFFFFFFFFu, s1, o);
    }
    if ((tid & 31) == 0) {
      sm.red0[tid >> 5] = s0;
      sm.red1[tid >> 5] = s1;
    }
    const int bad = __syncthreads_or(late || seen != seen || seen == INFINITY);
    if (tid == 0) {
      s0 = s1 = 0.0;
      for (int w = 0; w < kT / 32; ++w) {
        s0 += sm.red0[w];
        s1 += sm.red1[w];
      }
      sm.share[0].s0 = s0;
      sm.share[0].s1 = s1;
      sm.share[0].e = e;
      sm.share[0].bad = bad;
    }
  }
  int cnt = (int)min(sm.count, (uint32_t)kKeyCap);
  if (sm.count > (uint32_t)kKeyCap)  // the same in every thread: a barrier has passed
    cnt = search_again<T, kT>(sm, z, len, (uint32_t)v0, n);
  rank_keys<kT>(sm.keys, cnt, n, sm.top);
  if (tid == 0) sm.share[0].found = min(cnt, n);

  // ---- join the cluster's blocks
  int found;
  double s0, s1;
  double e;
  int bad;
  if (parts > 1) {
    cg::cluster_group cluster = cg::this_cluster();
    cluster.sync();
    if (part == 0) {
      for (int i = tid; i < parts * n; i += kT) {
        const int p = i / n, j = i - p * n;
        sm.lists[p][j] = cluster.map_shared_rank(&sm, p)->top[j];
      }
      if (tid > 0 && tid < parts) sm.share[tid] = cluster.map_shared_rank(&sm, tid)->share[0];
    }
    cluster.sync();  // the others' shared memory is no longer read
    if (part != 0) return;
    e = sm.share[0].e;
    for (int p = 1; p < parts; ++p) e = fmax(e, sm.share[p].e);
    s0 = s1 = 0.0;
    bad = 0;
    found = 0;
    for (int p = 0; p < parts; ++p) {
      const Share sh = sm.share[p];
      const double by = sh.e - e;
      const double f = by < -300.0 ? 0.0 : exp2(by);
      s0 += sh.s0 * f;
      s1 += f == 0.0 ? 0.0 : (sh.s1 + by * sh.s0) * f;
      bad |= sh.bad;
      found += sh.found;
    }
    found = min(found, n);
    // each list is in order: a key's place is its own and, in every other list,
    // the number of keys above it
    for (int i = tid; i < parts * n; i += kT) {
      const int p = i / n, j = i - p * n;
      if (j >= sm.share[p].found) continue;
      const uint64_t k = sm.lists[p][j];
      int above = j;
      for (int q = 0; q < parts && above < n; ++q) {
        if (q == p) continue;
        int lo_ = 0, hi_ = sm.share[q].found;
        while (lo_ < hi_) {
          const int mid = (lo_ + hi_) >> 1;
          if (sm.lists[q][mid] > k)
            lo_ = mid + 1;
          else
            hi_ = mid;
        }
        above += lo_;
      }
      if (above < n) sm.top[above] = k;
    }
    __syncthreads();
  } else {
    __syncthreads();
    found = sm.share[0].found;
    s0 = sm.share[0].s0;
    s1 = sm.share[0].s1;
    e = sm.share[0].e;
    bad = sm.share[0].bad;
  }
  const uint64_t* top = sm.top;

  // ---- the row's results: the sums' logarithm and the rest by one warp
  int reason = (tau_ok ? 0 : STS_ROW_BAD_TEMPERATURE) | (bad ? STS_ROW_BAD_LOGIT : 0);
  {
    int out = 0;
    for (int j = tid; j < a.m; j += kT) {
      const int64_t y = j == tid ? token : a.tokens[row * a.tokens_ld + j];
      out |= (y < -1 || y >= a.V) ? 1 : 0;
    }
    if (__syncthreads_or(out)) reason |= STS_ROW_BAD_TARGET;
  }
  const float nan = __int_as_float(0x7fc00000);
  const bool empty = reason == 0 && found == 0;
  const float zmax = found > 0 ? key_logit(top[0]) : kNegInf;
  if (tid < 32) {
    // S = sum 2^(c (z - zmax)), where c is what the sums were formed with; by:
    // what their base is off that. What c is off cd moves ln S by d ln S / dc.
    const bool near = fabsf(zmax * c.hi) < kFar;
    const double cs = kTwo || !near ? cd : (double)c.hi;
    const double by = found > 0 ? e - __dmul_rn(cs, (double)zmax) : 0.0;
    const double mean = s1 / s0 + by;  // of c (z - zmax)
    const double ln_total = log(s0 * exp2(by)) + kLn2 * (cd / cs - 1.0) * mean;
    const float log_sum = reason ? nan : empty ? kNegInf : (float)ln_total;
    if (tid == 0) {
      sm.log_sum = log_sum;
      if (a.logit_max) a.logit_max[row] = reason ? nan : zmax;
      if (a.log_sum) a.log_sum[row] = log_sum;
      if (a.lse)
        a.lse[row] = reason ? nan : empty ? kNegInf : (float)((double)zmax / (double)tau + ln_total);
      if (a.entropy) {
        const double h = ln_total - kLn2 * (cd / cs) * mean;
        a.entropy[row] = reason ? nan : empty ? 0.f : (float)fmax(h, 0.0);
      }
      if (a.flags)
        a.flags[row] = reason ? (STS_ROW_INVALID | reason) : empty ? STS_ROW_EMPTY : 0;
    }
  }
  __syncthreads();
  const float log_sum = sm.log_sum;
  for (int j = tid; j < a.m; j += kT) {
    const int64_t y = j == tid ? token : a.tokens[row * a.tokens_ld + j];
    float lp = nan;
    if (!reason) {
      if (y < 0)
        lp = 0.f;
      else if (empty)
        lp = kNegInf;
      else
        lp = __fdiv_rn((j == tid ? token_logit : to_f32(zrow[y])) - zmax, tau) - log_sum;
    }
    a.logprob[row * a.m + j] = lp;
  }
  for (int j = tid; j < a.n; j += kT) {
    const bool has = !reason && j < found;
    a.top_id[row * a.n + j] = has ? (int64_t)key_id(top[j]) : -1;
    a.top_logprob[row * a.n + j] =
        reason ? nan : has ? __fdiv_rn(key_logit(top[j]) - zmax, tau) - log_sum : kNegInf;
  }
}

// ---------------------------------------------------------------- gradient

struct BwdArgs {
  const void* z;
  int64_t ld;
  int64_t T;
  int V, parts, stretch;
  const int64_t* tokens;
  int64_t tokens_ld;
  int m;
  const float* tau;
  int n;
  const float *logit_max, *log_sum, *entropy;
  const int32_t* flags;
  const int64_t* top_id;
  const float *grad, *grad_entropy, *grad_top;
  void* out;
  int64_t out_ld;
};

struct BwdSmem {
  int64_t id[kMaxGiven + kMaxTop];
  float g[kMaxGiven + kMaxTop];
  float z[kMaxGiven + kMaxTop];
  double part[kThreads / 32];
};

// kN results to p (kN output elements, 16-byte rows where kVecOut).
template <typename O, int kN>
__device__ __forceinline__ void store_vec(O* p, const float (&v)[kN]) {
  union {
    O o[kN];
    uint4 w[(kN * sizeof(O) + 15) / 16];
    uint2 h;
  } u;
#pragma unroll
  for (int i = 0; i < kN; ++i) from_f32(v[i], u.o[i]);
  if constexpr (kN * sizeof(O) == 8) {
    *reinterpret_cast<uint2*>(p) = u.h;
  } else {
#pragma unroll
    for (int i = 0; i < (int)(kN * sizeof(O) / 16); ++i) reinterpret_cast<uint4*>(p)[i] = u.w[i];
  }
}

// The same where the output's 16-byte boundaries lie `skip` bytes into each
// lane's 16 bytes (the same in every lane): a lane stores the 16 bytes from its
// own boundary on, the rest of its vector and the start of the next lane's; the
// first lane's start and the last one's rest go element by element. Every lane
// of the warp calls it; `mine`: it has a vector (those that have come first).
template <typename O, int kN>
__device__ __forceinline__ void store_shifted(O* p, const float (&v)[kN], int skip, bool mine) {
  static_assert(kN * sizeof(O) == 16, "16 bytes a lane");
  union {
    O o[kN];
    uint32_t w[4];
  } u;
#pragma unroll
  for (int i = 0; i < kN; ++i) from_f32(v[i], u.o[i]);
  uint32_t c[8];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    c[i] = u.w[i];
    c[i + 4] = __shfl_down_sync(0xFFFFFFFFu, u.w[i], 1);
  }
  const int lane = (int)threadIdx.x & 31;
  const bool next = __shfl_down_sync(0xFFFFFFFFu, mine ? 1 : 0, 1) != 0 && lane < 31;
  if (!mine) return;
  if (next) {
    const int bits = (skip & 3) * 8;
    uint32_t d[5];
#pragma unroll
    for (int i = 0; i < 5; ++i) {
      const uint32_t lo = (skip & 4) ? c[i + 1 < 8 ? i + 1 : 7] : c[i];
      const uint32_t hi = (skip & 4) ? c[i + 3 < 8 ? i + 3 : 7] : c[i + 2];
      d[i] = (skip & 8) ? hi : lo;
    }
    uint4 w;
    w.x = __funnelshift_r(d[0], d[1], bits);
    w.y = __funnelshift_r(d[1], d[2], bits);
    w.z = __funnelshift_r(d[2], d[3], bits);
    w.w = __funnelshift_r(d[3], d[4], bits);
    *reinterpret_cast<uint4*>(reinterpret_cast<uint8_t*>(p) + skip) = w;
  }
#pragma unroll
  for (int i = 0; i < kN; ++i) {
    const bool start = i * (int)sizeof(O) < skip;
    if (start ? lane == 0 : !next) p[i] = u.o[i];
  }
}

struct RowCoef {
  float zmax, c, lo, l2s;  // x = (z - zmax) (c + lo) - l2s, p = 2^x
  float a, b;              // dz = p (a + b x)
};

// p and a + b x
__device__ __forceinline__ float2 factors_of(float z, const RowCoef& k) {
  // c d comes first: where it leaves fp32 (masked tokens, low temperatures) x is
  // -inf whatever lo d is, or NaN, which fmaxf drops. Added to lo d, which may be
  // +inf, the exact product of the FMA would not count.
  const float d = z - k.zmax;
  const float x = fmaxf(fmaf(d, k.lo, fmaf(d, k.c, -k.l2s)), -200.f);
  return make_float2(ex2(x), fmaf(k.b, x, k.a));
}
__device__ __forceinline__ float grad_of(float z, const RowCoef& k) {
  const float2 f = factors_of(z, k);
  return f.x * f.y;
}

template <typename T, typename O>
__global__ void __launch_bounds__(kThreads, 4) backward_kernel(const BwdArgs a) {
  __shared__ BwdSmem sm;
  constexpr int kN = Vec<T>::kN;
  const int parts = a.parts;
  const int64_t row = (int64_t)blockIdx.x / parts;
  const int part = (int)((int64_t)blockIdx.x - row * parts);
  const int tid = threadIdx.x;
  const int v0 = (int)min((int64_t)part * a.stretch, (int64_t)a.V);
  const int len = min(a.stretch, a.V - v0);
  const T* zrow = static_cast<const T*>(a.z) + row * a.ld;
  O* orow = static_cast<O*>(a.out) + row * a.out_ld;
  const T* z = zrow + v0;
  O* out = orow + v0;
  const int head = min((int)((16u - (uint32_t)(reinterpret_cast<uintptr_t>(z) & 15u)) % 16u) /
                           (int)sizeof(T), len);
  const int body = (len - head) / kN;
  const int tail0 = head + body * kN;
  const T* zb = z + head;
  O* ob = out + head;
  constexpr uintptr_t kOutAlign = kN * sizeof(O) >= 16 ? 15u : 7u;
  const bool vec_out = (reinterpret_cast<uintptr_t>(ob) & kOutAlign) == 0;
  const int skip = (int)((16u - (uint32_t)(reinterpret_cast<uintptr_t>(ob) & 15u)) & 15u);

  // what the row needs first is asked for at once, not one after the other: its
  // scalars, its tokens and its first logits
  const int32_t flags = a.flags[row];
  const float tau_in = a.tau ? a.tau[row] : 1.f;
  const float zmax = a.logit_max[row], log_sum = a.log_sum[row];
  const double h = a.grad_entropy ? (double)a.grad_entropy[row] : 0.0;
  const double entropy = a.grad_entropy ? (double)a.entropy[row] : 0.0;
  Vec<T> v[kUnroll];
  auto load = [&](int i0) {
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
      const int i = i0 + u * kThreads + tid;
      // not __ldg: the output may be the logits themselves
      if (i < body) v[u].w = *reinterpret_cast<const uint4*>(zb + (int64_t)i * kN);
    }
  };
  load(0);
  const bool live = (flags & (STS_ROW_INVALID | STS_ROW_EMPTY)) == 0;

  // the tokens that get a share, with their logits: read before any block of
  // the row writes, since the gradient may take the logits' place
  const int given = a.grad ? a.m : 0;
  const int count = given + (a.grad_top ? a.n : 0);
  double sum = 0.0;
  for (int j = tid; j < count; j += kThreads) {
    int64_t id;
    float g;
    if (j < given) {
      id = a.tokens[row * a.tokens_ld + j];
      g = a.grad[row * a.m + j];
    } else {
      id = a.top_id[row * a.n + (j - given)];
      g = a.grad_top[row * a.n + (j - given)];
    }
    float zv = kNegInf;
    if (id >= 0 && id < a.V) zv = to_f32(zrow[id]);
    const bool valid = zv > kNegInf;
    sm.id[j] = valid ? id : -1;
    sm.g[j] = g;
    sm.z[j] = zv;
    if (valid) sum += (double)g;
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xFFFFFFFFu, sum, o);
  if ((tid & 31) == 0) sm.part[tid >> 5] = sum;
  if (parts > 1)
    cg::this_cluster().sync();
  else
    __syncthreads();
  sum = 0.0;
  for (int w = 0; w < kThreads / 32; ++w) sum += sm.part[w];

  RowCoef k{0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
  float tau = 1.f;
  if (live) {
    tau = tau_in;
    k.zmax = zmax;
    const double cd = exponent_scale(tau);
    k.c = (float)cd;
    k.lo = (float)(cd - (double)k.c);
    k.l2s = (float)((double)log_sum * kLog2eD);
    const double ca = -(sum + (h != 0.0 ? h * entropy : 0.0)) / (double)tau;
    const double cb = -h * kLn2 / (double)tau;
    k.a = (float)ca;
    k.b = (float)cb;
    // Temperatures below some 1e-36 take them out of fp32, where a probability of
    // 0 would meet an infinity: 2^100 of them then goes over to p, by way of x
    // (x + 100 is at most 100, and -200 still gives 0).
    if (!(fabsf(k.a) + 200.f * fabsf(k.b) < 1e38f)) {
      k.a = (float)((ca - 100.0 * cb) * 0x1p-100);
      k.b = (float)(cb * 0x1p-100);
      k.l2s -= 100.f;
    }
  }

  for (int i0 = 0; i0 < body; i0 += kThreads * kUnroll) {
    if (i0 > 0) load(i0);
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
      const int i = i0 + u * kThreads + tid;
      if (i - (tid & 31) >= body) break;  // no lane of the warp has one
      float f[kN];
#pragma unroll
      for (int j = 0; j < kN; ++j) f[j] = 0.f;
      if (live && i < body) {
        v[u].f32(f);
#pragma unroll
        for (int j = 0; j < kN; ++j) f[j] = grad_of(f[j], k);
      }
      O* p = ob + (int64_t)i * kN;
      if (vec_out) {
        if (i < body) store_vec<O, kN>(p, f);
      } else if constexpr (sizeof(O) == sizeof(T)) {
        store_shifted<O, kN>(p, f, skip, i < body);
      } else if (i < body) {
#pragma unroll
        for (int j = 0; j < kN; ++j) from_f32(f[j], p[j]);
      }
    }
  }
  for (int i = tid; i < head + (len - tail0); i += kThreads) {
    const int at = i < head ? i : tail0 + (i - head);
    from_f32(live ? grad_of(to_f32(z[at]), k) : 0.f, out[at]);
  }
  if (!live || count == 0) return;
  __syncthreads();  // the tokens' own elements are written again, whole, by their first mention
  for (int j = tid; j < count; j += kThreads) {
    const int64_t id = sm.id[j];
    if (id < v0 || id >= (int64_t)v0 + len) continue;
    double g = 0.0;
    bool first = true;
    for (int i = 0; i < count; ++i) {
      if (sm.id[i] != id) continue;
      if (i < j) {
        first = false;
        break;
      }
      g += (double)sm.g[i];
    }
    if (first) {  // in float64: both terms may be beyond fp32 and their sum 0
      const float2 f = factors_of(sm.z[j], k);
      from_f32((float)(g / (double)tau + (double)f.x * (double)f.y), orow[id]);
    }
  }
}

// ---------------------------------------------------------------- launches

// Parts per row: 1, 2, 4 or 8, none much shorter than one round of the loop; a
// block's cost is its bytes and 32 KB more. The gradient and the forward's short
// rows: as many waves of blocks as there are, four (of 128 threads seven) an SM:
// 700 rows of 152,064 bf16, gradient, 4 parts 80.8 us, 2 82.6, 1 89.8; 400 rows 4
// parts 50.0, 1 49.2, 2 56.8; 333 rows of 32,771 fp32, forward, 2 parts 28.7, 4
// 39.9. The forward's long rows are bound by instructions: as many blocks as the
// busiest SM gets, the slower the fewer threads that SM has: 100 rows of 152,064
// bf16 4 parts 23 us, 8 31, 2 25; 700 rows 1 part 70, 2 82. Of some 200 to 500 rows it
// divides too many (400 rows: 2 parts 54.5 us, 1 part 45.2): over 762 shapes the
// forward takes 1.12 of the best choice's time, 1.9 at most.
int parts_for(int64_t T, int64_t V, int elem, int sms, int threads, bool forward) {
  const int64_t round = (int64_t)threads * kUnroll * (16 / elem);
  int best = 1;
  double least = 0.0;
  for (int parts = 1; parts <= kMaxParts && (parts == 1 || V > round * (parts / 2)); parts *= 2) {
    const bool busiest = forward && threads == 256;
    const int64_t slots = busiest ? sms : (int64_t)sms * (threads == 128 ? 7 : 4);
    const int64_t turns = (T * parts + slots - 1) / slots;
    double cost = (double)turns * ((double)V * elem / parts + 32768.0);
    if (busiest) {
      const int64_t held = turns * threads;  // threads of the busiest SM
      cost /= held >= 1024 ? 1.0 : held >= 768 ? 0.9 : held >= 512 ? 0.7 : 0.4;
    }
    if (parts == 1 || cost < least) {
      best = parts;
      least = cost;
    }
  }
  return best;
}

template <typename K, typename A>
cudaError_t launch_rows(K kernel, const A& a, cudaStream_t st, int threads = kThreads,
                        size_t smem = 0) {
  if (smem > 48 * 1024) {
    const cudaError_t e =
        cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
    if (e != cudaSuccess) return e;
  }
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3((unsigned)(a.T * a.parts));
  cfg.blockDim = dim3((unsigned)threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeClusterDimension;
  at[0].val.clusterDim.x = (unsigned)a.parts;
  at[0].val.clusterDim.y = 1;
  at[0].val.clusterDim.z = 1;
  cfg.attrs = at;
  cfg.numAttrs = a.parts > 1 ? 1 : 0;
  const cudaError_t e = cudaLaunchKernelEx(&cfg, kernel, a);
  const cudaError_t last = cudaGetLastError();
  return e != cudaSuccess ? e : last;
}

int elem_size(int dtype) {
  return dtype == STS_DTYPE_F32 ? 4 : dtype == STS_DTYPE_BF16 || dtype == STS_DTYPE_F16 ? 2 : 0;
}

template <typename T>
cudaError_t launch_forward(const FwdArgs& a, int threads, cudaStream_t st) {
  return threads == 128 ? launch_rows(forward_kernel<T, 128>, a, st, 128, sizeof(FwdSmem<128>))
                        : launch_rows(forward_kernel<T, 256>, a, st, 256, sizeof(FwdSmem<256>));
}

constexpr int64_t kMost = (int64_t(1) << 31) - 1;

bool aligned(const void* p, int bytes) {
  return reinterpret_cast<uintptr_t>(p) % (unsigned)bytes == 0;
}

// Host checks shared by both directions; *done where there is nothing to do.
sts_status check_token_rows(const sts_token_rows* r, bool* done) {
  *done = false;
  if (!r) return STS_ERR_NULL;
  const int es = elem_size(r->dtype);
  if (!es) return STS_ERR_DTYPE;
  if (r->T < 0 || r->T > kMost / kMaxParts || r->V < 1 || r->V > kMost - 1024) return STS_ERR_SHAPE;
  if (r->m < 0 || r->m > kMaxGiven || r->top_n < 0 || r->top_n > kMaxTop) return STS_ERR_SHAPE;
  if (r->T > 1 && (r->ld < r->V || r->tokens_ld < r->m)) return STS_ERR_SHAPE;
  if (r->T == 0) {
    *done = true;
    return STS_OK;
  }
  if (!r->logits || (r->m > 0 && !r->tokens)) return STS_ERR_NULL;
  if (!aligned(r->logits, es) || (r->m > 0 && !aligned(r->tokens, 8)) || !aligned(r->temperature, 4))
    return STS_ERR_SHAPE;
  return STS_OK;
}

bool aligned_stats(const sts_token_stats* s) {
  return aligned(s->logit_max, 4) && aligned(s->log_sum, 4) && aligned(s->lse, 4) &&
         aligned(s->entropy, 4) && aligned(s->flags, 4) && aligned(s->top_id, 8) &&
         aligned(s->top_logprob, 4);
}

}  // namespace
}  // namespace sts

using namespace sts;

extern "C" sts_status sts_token_logprobs(const sts_token_rows* rows, float* logprob,
                                         const sts_token_stats* stats, sts_stream_t stream) {
  bool done = false;
  const sts_status cs = check_token_rows(rows, &done);
  if (cs != STS_OK || done) return cs;
  if (!stats || (rows->m > 0 && !logprob)) return STS_ERR_NULL;
  if (rows->top_n > 0 && (!stats->top_id || !stats->top_logprob)) return STS_ERR_NULL;
  if (!aligned_stats(stats) || !aligned(logprob, 4)) return STS_ERR_SHAPE;
  int sms = 0;
  const sts_status ds = current_device(&sms);
  if (ds != STS_OK) return ds;
  FwdArgs a{};
  a.z = rows->logits;
  a.ld = rows->ld;
  a.T = rows->T;
  a.V = (int)rows->V;
  const int threads = rows->V <= kShortRow ? 128 : 256;
  a.parts = parts_for(rows->T, rows->V, elem_size(rows->dtype), sms, threads, true);
  a.stretch = (int)(((rows->V + a.parts - 1) / a.parts + 63) / 64 * 64);
  a.tokens = rows->tokens;
  a.tokens_ld = rows->tokens_ld;
  a.m = (int)rows->m;
  a.tau = rows->temperature;
  a.n = (int)rows->top_n;
  a.logprob = logprob;
  a.logit_max = stats->logit_max;
  a.log_sum = stats->log_sum;
  a.lse = stats->lse;
  a.entropy = stats->entropy;
  a.flags = stats->flags;
  a.top_id = stats->top_id;
  a.top_logprob = stats->top_logprob;
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  const LaunchMark mark = launch_begin(STS_KERNEL_TOKEN_LOGPROBS, st);
  const cudaError_t e = rows->dtype == STS_DTYPE_F32    ? launch_forward<float>(a, threads, st)
                        : rows->dtype == STS_DTYPE_BF16 ? launch_forward<__nv_bfloat16>(a, threads, st)
                                                        : launch_forward<__half>(a, threads, st);
  launch_end(mark, st);
  return e == cudaSuccess ? STS_OK : STS_ERR_CUDA;
}

namespace sts {
namespace {

template <typename T>
cudaError_t launch_backward(const BwdArgs& a, int out_dtype, cudaStream_t st) {
  return out_dtype == STS_DTYPE_F32    ? launch_rows(backward_kernel<T, float>, a, st)
         : out_dtype == STS_DTYPE_BF16 ? launch_rows(backward_kernel<T, __nv_bfloat16>, a, st)
                                       : launch_rows(backward_kernel<T, __half>, a, st);
}

}  // namespace
}  // namespace sts

extern "C" sts_status sts_token_logprobs_backward(const sts_token_rows* rows,
                                                  const sts_token_stats* saved,
                                                  const float* grad_logprob,
                                                  const float* grad_entropy, const float* grad_top,
                                                  void* dlogits, int dlogits_dtype,
                                                  int64_t dlogits_ld, sts_stream_t stream) {
  const int os = elem_size(dlogits_dtype);
  if (!os) return STS_ERR_DTYPE;
  bool done = false;
  const sts_status cs = check_token_rows(rows, &done);
  if (cs != STS_OK) return cs;
  if (rows->T > 1 && dlogits_ld < rows->V) return STS_ERR_SHAPE;
  if (done) return STS_OK;
  if (!saved || !saved->logit_max || !saved->log_sum || !saved->flags || !dlogits)
    return STS_ERR_NULL;
  if (grad_entropy && !saved->entropy) return STS_ERR_NULL;
  if (grad_top && rows->top_n > 0 && !saved->top_id) return STS_ERR_NULL;
  if (!aligned(dlogits, os) || !aligned_stats(saved) || !aligned(grad_logprob, 4) ||
      !aligned(grad_entropy, 4) || !aligned(grad_top, 4))
    return STS_ERR_SHAPE;
  // the gradient may take the logits' own place, and no other part of them
  const int es = elem_size(rows->dtype);
  const uintptr_t z0 = reinterpret_cast<uintptr_t>(rows->logits);
  const uintptr_t o0 = reinterpret_cast<uintptr_t>(dlogits);
  const uintptr_t z1 = z0 + (uintptr_t)(((rows->T - 1) * (rows->T > 1 ? rows->ld : 0) + rows->V) * es);
  const uintptr_t o1 = o0 + (uintptr_t)(((rows->T - 1) * (rows->T > 1 ? dlogits_ld : 0) + rows->V) * os);
  if (z0 < o1 && o0 < z1 &&
      !(z0 == o0 && rows->dtype == dlogits_dtype && (rows->T == 1 || rows->ld == dlogits_ld)))
    return STS_ERR_SHAPE;
  int sms = 0;
  const sts_status ds = current_device(&sms);
  if (ds != STS_OK) return ds;
  BwdArgs a{};
  a.z = rows->logits;
  a.ld = rows->ld;
  a.T = rows->T;
  a.V = (int)rows->V;
  a.parts = parts_for(rows->T, rows->V, es, sms, kThreads, false);
  a.stretch = (int)(((rows->V + a.parts - 1) / a.parts + 63) / 64 * 64);
  a.tokens = rows->tokens;
  a.tokens_ld = rows->tokens_ld;
  a.m = (int)rows->m;
  a.tau = rows->temperature;
  a.n = (int)rows->top_n;
  a.logit_max = saved->logit_max;
  a.log_sum = saved->log_sum;
  a.entropy = saved->entropy;
  a.flags = saved->flags;
  a.top_id = saved->top_id;
  a.grad = rows->m > 0 ? grad_logprob : nullptr;
  a.grad_entropy = grad_entropy;
  a.grad_top = rows->top_n > 0 ? grad_top : nullptr;
  a.out = dlogits;
  a.out_ld = dlogits_ld;
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  const LaunchMark mark = launch_begin(STS_KERNEL_TOKEN_GRAD, st);
  const cudaError_t e = rows->dtype == STS_DTYPE_F32 ? launch_backward<float>(a, dlogits_dtype, st)
                        : rows->dtype == STS_DTYPE_BF16
                            ? launch_backward<__nv_bfloat16>(a, dlogits_dtype, st)
                            : launch_backward<__half>(a, dlogits_dtype, st);
  launch_end(mark, st);
  return e == cudaSuccess ? STS_OK : STS_ERR_CUDA;
}
