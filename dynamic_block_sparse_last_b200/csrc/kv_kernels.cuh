// kv_kernels.cuh -- the paged key/value cache: rows quantised as they are
// written to their slots, and read back.
//
// A row is the d values of one token in one head: scale = M / c, code =
// round(c x / M), M = max|x|; c = 127 (int8) or 448 (e4m3).  The quotient is
// formed by one multiplication with c / M (error below 2^-21 of it) and only
// where that leaves the rounding open, near a value half way between two codes,
// by the correctly rounded division (c x) / M, so the code is that of the
// division for every row at about a third of its instructions.
//
// Bound: memory, each byte once.  A block takes 64 neighbouring tokens and a
// group of heads: it looks the tokens' slots up once, into shared memory, and
// then moves rows in 16-byte vectors, several rows in flight per thread.
#pragma once

#include <type_traits>

#include "ptx.cuh"
#include "rope_kernel.cuh"

namespace fpk {

constexpr int kKvTokens = 64;    // tokens of a block
constexpr int kKvThreads = 256;

struct KvGeom {
  void *pool[2];       // K, V  [pages][heads][page][d]
  float *scale[2];     // [pages][heads][page]
  int64_t pages;
  int page, page_shift, heads;
};

struct KvWriteParams {
  KvGeom g;
  const void *in[2];   // null: not written
  int64_t tok[2], head[2];
  const int64_t *slots;
  int T, group;        // heads of a block
  int *err;
};

struct KvReadParams {
  KvGeom g;
  void *out[2];
  int64_t tok[2], head[2];
  const int *table, *cu, *first;
  int max_pages, nseq, T, group;
  int *err;
};

// kinds of cache rows
enum { kKvBf16 = 0, kKvF16 = 1, kKvInt8 = 3, kKvE4m3 = 4 };
template <int KIND>
struct KvCode {
  static constexpr bool kQuant = KIND == kKvInt8 || KIND == kKvE4m3;
  static constexpr int kBytes = kQuant ? 1 : 2;
  static constexpr float kTop = KIND == kKvInt8 ? 127.f : 448.f;
};

// Four codes of the quotients y (c x / M by multiplication), exact ones where
// the rounding is open.
template <int KIND>
__device__ __forceinline__ uint32_t kv_codes4(const float *x, float inv, float M) {
  constexpr float C = KvCode<KIND>::kTop;
  float y[4];
  bool open = false;
  if constexpr (KIND == kKvInt8) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      y[i] = x[i] * inv;
      // |y| <= 127.0001, off by at most 127 * 2^-21 = 6.1e-5
      open |= fabsf(fabsf(y[i] - rintf(y[i])) - 0.5f) < 1e-4f;
    }
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      y[i] = x[i] * inv;
      // Half way between two normal codes the 20 bits below the kept 3 are
      // 0x80000 (2^-24 of the value a step); below 2^-6 the codes are 2^-9
      // apart, and the division is always made.
      const uint32_t low = __float_as_uint(y[i]) & 0xfffffu;
      open |= (low - (0x80000u - 64u)) < 128u || (fabsf(y[i]) < 0.015625f && y[i] != 0.f);
    }
  }
  if (open) {
#pragma unroll
    for (int i = 0; i < 4; ++i) y[i] = __fdiv_rn(C * x[i], M);
  }
  if constexpr (KIND == kKvInt8) {
    uint32_t w = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) w |= (static_cast<uint32_t>(__float2int_rn(y[i])) & 0xffu) << (8 * i);
    return w;
  } else {
    uint16_t lo, hi;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(lo) : "f"(y[1]), "f"(y[0]));
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(hi) : "f"(y[3]), "f"(y[2]));
    return static_cast<uint32_t>(lo) | (static_cast<uint32_t>(hi) << 16);
  }
}

// Values of four codes.
template <int KIND>
__device__ __forceinline__ void kv_values4(uint32_t w, float *x) {
  if constexpr (KIND == kKvInt8) {
#pragma unroll
    for (int i = 0; i < 4; ++i) x[i] = static_cast<float>(static_cast<int8_t>(w >> (8 * i)));
  } else {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      uint32_t h;
      asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"(static_cast<uint16_t>(w >> (16 * i))));
      const float2 f = __half22float2(*reinterpret_cast<const __half2 *>(&h));
      x[2 * i] = f.x;
      x[2 * i + 1] = f.y;
    }
  }
}

// grid (ceil(T / 64), head groups); d = D; T: type of the input rows
template <int KIND, typename T, int D>
__global__ void __launch_bounds__(kKvThreads) k_kv_write(const KvWriteParams P) {
  constexpr int V = RopeVec<T>::kElems;      // elements of a lane
  constexpr int L = D / V;                   // lanes of a row
  constexpr int R = kKvThreads / L;          // rows of the block at a time
  __shared__ int64_t slot_sh[kKvTokens];
  const int t0 = blockIdx.x * kKvTokens, nt = min(kKvTokens, P.T - t0);
  if (threadIdx.x < kKvTokens) {
    int64_t s = threadIdx.x < nt ? P.slots[t0 + threadIdx.x] : -1;
    if (s >= (P.g.pages << P.g.page_shift)) {
      s = -1;
      atomicOr(P.err, kDevErrRange);
    }
    slot_sh[threadIdx.x] = s;
  }
  __syncthreads();
  const int h0 = blockIdx.y * P.group, nh = min(P.group, P.g.heads - h0);
  const int lane = threadIdx.x % L, r0 = threadIdx.x / L;
  const int rows = kKvTokens * nh;  // a multiple of R: whole warps take part in the row maxima
  for (int r = r0; r < rows; r += R) {
    const int tt = r % kKvTokens, h = h0 + r / kKvTokens;
    const int64_t slot = slot_sh[tt];
    uint4 raw[2];
#pragma unroll
    for (int w = 0; w < 2; ++w)
      if (slot >= 0 && P.in[w])
        raw[w] = *reinterpret_cast<const uint4 *>(static_cast<const T *>(P.in[w]) + (t0 + tt) * P.tok[w] +
                                                  h * P.head[w] + lane * V);
      else
        raw[w] = make_uint4(0, 0, 0, 0);
    const int64_t pg = slot >> P.g.page_shift;
    const int64_t row = ((pg * P.g.heads + h) << P.g.page_shift) + (slot & (P.g.page - 1));
#pragma unroll
    for (int w = 0; w < 2; ++w) {
      if (!P.in[w]) continue;
      float x[V];
      RopeVec<T>::unpack(raw[w], x);
      if constexpr (KvCode<KIND>::kQuant) {
        // the largest magnitude of the row, as bits: a NaN's are above an
        // infinity's, so anything not finite is seen
        uint32_t mb = 0;
#pragma unroll
        for (int i = 0; i < V; ++i) mb = max(mb, __float_as_uint(x[i]) & 0x7fffffffu);
#pragma unroll
        for (int o = L / 2; o > 0; o >>= 1) mb = max(mb, __shfl_xor_sync(0xffffffffu, mb, o));
        const float M = __uint_as_float(mb);
        const bool finite = mb < 0x7f800000u;
        uint32_t code[V / 4] = {};
        if (finite && mb != 0) {
          if (M > 1e-30f && M < 1e30f) {
            const float inv = __fdiv_rn(KvCode<KIND>::kTop, M);
#pragma unroll
            for (int i = 0; i < V; i += 4) code[i / 4] = kv_codes4<KIND>(x + i, inv, M);
          } else {  // c / M or c x would leave fp32: the row times 2^100 or 2^-100, which the quotient does not see
            const float f = M < 1.f ? 1.2676506002282294e30f : 7.888609052210118e-31f;
            float z[V];
#pragma unroll
            for (int i = 0; i < V; ++i) z[i] = x[i] * f;
            const float M2 = M * f, inv2 = __fdiv_rn(KvCode<KIND>::kTop, M2);
#pragma unroll
            for (int i = 0; i < V; i += 4) code[i / 4] = kv_codes4<KIND>(z + i, inv2, M2);
          }
        }
        if (slot >= 0) {
          uint8_t *dst = static_cast<uint8_t *>(P.g.pool[w]) + row * D + lane * V;
          if constexpr (V == 8) *reinterpret_cast<uint2 *>(dst) = make_uint2(code[0], code[1]);
          else *reinterpret_cast<uint32_t *>(dst) = code[0];
          if (lane == 0)
            P.g.scale[w][row] = finite ? __fdiv_rn(M, KvCode<KIND>::kTop) : __uint_as_float(0x7fc00000u);
        }
      } else if (slot >= 0) {
        using C = typename std::conditional<KIND == kKvBf16, __nv_bfloat16, __half>::type;
        C *dst = static_cast<C *>(P.g.pool[w]) + row * D + lane * V;
        if constexpr (V == 8) {
          *reinterpret_cast<uint4 *>(dst) = RopeVec<C>::pack(x);
        } else {
          C y[4];
#pragma unroll
          for (int i = 0; i < 4; ++i) y[i] = rope_from_float<C>(x[i]);
          *reinterpret_cast<uint2 *>(dst) = *reinterpret_cast<const uint2 *>(y);
        }
      }
    }
  }
}

// The sequence of packed row t: the last s with cu[s] <= t (cu non-decreasing,
// cu[0] <= t < cu[nseq]).
__device__ __forceinline__ int kv_find_seq(const int *cu, int nseq, int t) {
  int lo = 0, hi = nseq;  // cu[lo] <= t < cu[hi]
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (cu[mid] <= t) lo = mid;
    else hi = mid;
  }
  return lo;
}

// grid (ceil(T / 64), head groups); T: type of the output rows
template <int KIND, typename T, int D>
__global__ void __launch_bounds__(kKvThreads) k_kv_read(const KvReadParams P) {
  constexpr int VO = RopeVec<T>::kElems;     // output elements of a 16-byte vector
  constexpr int V = 8;                       // elements of a lane
  constexpr int L = D / V;
  constexpr int R = kKvThreads / L;
  __shared__ int64_t slot_sh[kKvTokens];
  const int t0 = blockIdx.x * kKvTokens, nt = min(kKvTokens, P.T - t0);
  if (threadIdx.x < kKvTokens) {
    const int t = t0 + threadIdx.x;
    int64_t slot = -1;
    if (threadIdx.x < nt && t >= P.cu[0] && t < P.cu[P.nseq]) {
      const int s = kv_find_seq(P.cu, P.nseq, t);
      const int64_t p = (int64_t)(P.first ? P.first[s] : 0) + (t - P.cu[s]);
      bool ok = p >= 0 && (p >> P.g.page_shift) < P.max_pages;
      if (ok) {
        const int pg = P.table[(int64_t)s * P.max_pages + (p >> P.g.page_shift)];
        ok = pg >= 0 && pg < P.g.pages;
        slot = ok ? ((int64_t)pg << P.g.page_shift) + (p & (P.g.page - 1)) : -1;
      }
      if (!ok) atomicOr(P.err, kDevErrRange);
    }
    slot_sh[threadIdx.x] = slot;
  }
  __syncthreads();
  const int h0 = blockIdx.y * P.group, nh = min(P.group, P.g.heads - h0);
  const int lane = threadIdx.x % L, r0 = threadIdx.x / L;
  const int rows = kKvTokens * nh;
#pragma unroll 2
  for (int r = r0; r < rows; r += R) {
    const int tt = r % kKvTokens, h = h0 + r / kKvTokens;
    const int64_t slot = slot_sh[tt];
    if (slot < 0) continue;
    const int64_t row = (((slot >> P.g.page_shift) * P.g.heads + h) << P.g.page_shift) + (slot & (P.g.page - 1));
#pragma unroll
    for (int w = 0; w < 2; ++w) {
      if (!P.out[w]) continue;
      float x[V];
      if constexpr (KvCode<KIND>::kQuant) {
        const uint2 c = *reinterpret_cast<const uint2 *>(static_cast<const uint8_t *>(P.g.pool[w]) + row * D + lane * V);
        const float s = P.g.scale[w][row];
        kv_values4<KIND>(c.x, x);
        kv_values4<KIND>(c.y, x + 4);
#pragma unroll
        for (int i = 0; i < V; ++i) x[i] *= s;
      } else {
        using C = typename std::conditional<KIND == kKvBf16, __nv_bfloat16, __half>::type;
        RopeVec<C>::unpack(*reinterpret_cast<const uint4 *>(static_cast<const C *>(P.g.pool[w]) + row * D + lane * V), x);
      }
      T *dst = static_cast<T *>(P.out[w]) + (t0 + tt) * P.tok[w] + h * P.head[w] + lane * V;
#pragma unroll
      for (int i = 0; i < V; i += VO) *reinterpret_cast<uint4 *>(dst + i) = RopeVec<T>::pack(x + i);
    }
  }
}

}  // namespace fpk
