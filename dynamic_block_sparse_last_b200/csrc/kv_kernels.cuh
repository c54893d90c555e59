// kv_kernels.cuh -- the paged key/value cache: rows quantised as they are
// written to their slots, and read back.
//
// A row is the d values of one token in one head: scale = M / c, code =
// round(c x / M), M = max|x|; c = 127 (int8) or 448 (e4m3).
//
// The code without a division per element: with v = c / M to 2^-21.9, the quotient
// q = c x / M lies between x v (1 - 2^-20) and x v (1 + 2^-20), both within 2^-19.4 of
// it (relative to q), and rounding is monotone, so where both round to the same code
// that is q's code.  Where they do not, a border t of two codes lies between them.  For
// bf16 and fp16 rows q then is t, and the even code is the answer, since a quotient that
// is not a border is further than 2^-19 from it: with x = b 2^i, M = a 2^j, a, b < 2^11,
//   int8  q = 127 b 2^n / a, t = T / 2 (T odd, < 2^8): q - t = (254 b 2^n - a T) / 2a; if
//         not 0, at least 1/2a, 1/(aT) of t, for n >= 0, else 2^n / 2a, 1/(254 b) of q;
//   e4m3  q = 7 b 2^n / a, t = T 2^k (T odd, < 2^5): at least 2^min(n,k) / a, which is
//         1/(7 b) of q or 1/(aT) of t.
// fp32 rows take the correctly rounded division there.
//
// Bound: memory, each byte once.  A block takes some neighbouring tokens and a
// group of heads: it looks the tokens' slots up once, into shared memory, and
// then moves rows in 16-byte vectors, several rows in flight per thread.  Measured
// over 8 heads of 128: 43.7 K bf16 tokens to e4m3 in 65 us (4.2 TB/s; the integer pipe
// is 61% busy, with a division per element it took 136 us), back in 47 us (5.8 TB/s);
// 131072 int8 tokens back in 131 us (6.2 TB/s).
#pragma once

#include <type_traits>

#include "ptx.cuh"
#include "rope_kernel.cuh"

namespace fpk {

constexpr int kKvTokens = 32;    // most tokens of a block (kv_split)
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
  int tok_shift;       // log2 of its tokens
  int *err;
};

struct KvReadParams {
  KvGeom g;
  void *out[2];
  int64_t tok[2], head[2];
  const int *table, *cu, *first;
  int max_pages, nseq, T, group, tok_shift;
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

// Four codes, packed: those of x vlo and of x vhi.
template <int KIND>
__device__ __forceinline__ uint32_t kv_codes4(const float *x, float v) {
  if constexpr (KIND == kKvInt8) {
    // x v + 1.5 2^23, rounded once: the integer (half to even) in the low bits
    const uint64_t v2 = f2_pack(v, v), big = f2_pack(12582912.f, 12582912.f);
    float y[4];
    f2_unpack(f2_fma(f2_pack(x[0], x[1]), v2, big), y[0], y[1]);
    f2_unpack(f2_fma(f2_pack(x[2], x[3]), v2, big), y[2], y[3]);
    const uint32_t lo = __byte_perm(__float_as_uint(y[0]), __float_as_uint(y[1]), 0x0040);
    const uint32_t hi = __byte_perm(__float_as_uint(y[2]), __float_as_uint(y[3]), 0x0040);
    return __byte_perm(lo, hi, 0x5410);
  } else {
    const uint64_t v2 = f2_pack(v, v);
    float y[4];
    f2_unpack(f2_mul(f2_pack(x[0], x[1]), v2), y[0], y[1]);
    f2_unpack(f2_mul(f2_pack(x[2], x[3]), v2), y[2], y[3]);
    uint32_t w;
    asm("{\n\t.reg .b16 l, h;\n\tcvt.rn.satfinite.e4m3x2.f32 l, %2, %1;\n\tcvt.rn.satfinite.e4m3x2.f32 h, %4, %3;\n\t"
        "mov.b32 %0, {l, h};\n\t}"
        : "=r"(w)
        : "f"(y[0]), "f"(y[1]), "f"(y[2]), "f"(y[3]));
    return w;
  }
}

// One code of a correctly rounded quotient.
template <int KIND>
__device__ __forceinline__ uint32_t kv_code_exact(float x, float M) {
  const float y = __fdiv_rn(KvCode<KIND>::kTop * x, M);
  if constexpr (KIND == kKvInt8) return static_cast<uint32_t>(__float2int_rn(y)) & 0xffu;
  uint16_t c;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(c) : "f"(0.f), "f"(y));
  return c & 0xffu;
}

// The codes of one lane's elements of a row (EXACT: rows of fp32).
template <int KIND, int V, bool EXACT>
__device__ __forceinline__ void kv_quantise(const float *x, float M, uint32_t *code) {
  const float v = __fdividef(KvCode<KIND>::kTop, M);  // 1e-30 < M < 1e30
  const float vlo = v * (1.f - 9.5367431640625e-07f), vhi = v * (1.f + 9.5367431640625e-07f);
#pragma unroll
  for (int i = 0; i < V; i += 4) {
    const uint32_t lo = kv_codes4<KIND>(x + i, vlo), hi = kv_codes4<KIND>(x + i, vhi);
    if constexpr (EXACT) {
      code[i / 4] = lo;
      if (lo != hi) {
        uint32_t w = 0;
#pragma unroll
        for (int e = 0; e < 4; ++e) w |= kv_code_exact<KIND>(x[i + e], M) << (8 * e);
        code[i / 4] = w;
      }
    } else {
      // the even code of each byte's two (the same one mostly): hi where lo is odd
      const uint32_t odd = (lo & 0x01010101u) * 255u;
      code[i / 4] = (hi & odd) | (lo & ~odd);
    }
  }
}

// The largest magnitude of a lane's 16 bytes, as fp32 bits: a NaN's are above an
// infinity's, so anything not finite is seen.
template <typename T>
__device__ __forceinline__ uint32_t kv_max_bits(const uint4 &r) {
  if constexpr (sizeof(T) == 4) {
    return max(max(r.x & 0x7fffffffu, r.y & 0x7fffffffu), max(r.z & 0x7fffffffu, r.w & 0x7fffffffu));
  } else {
    constexpr uint32_t A = 0x7fff7fffu;
    return __vmaxu2(__vmaxu2(r.x & A, r.y & A), __vmaxu2(r.z & A, r.w & A));  // pairs of 16-bit magnitudes
  }
}
template <typename T, int L>
__device__ __forceinline__ float kv_row_max(const uint4 &r) {
  uint32_t m = kv_max_bits<T>(r);
#pragma unroll
  for (int o = L / 2; o > 0; o >>= 1) {
    const uint32_t y = __shfl_xor_sync(0xffffffffu, m, o);
    if constexpr (sizeof(T) == 4) m = max(m, y);
    else m = __vmaxu2(m, y);
  }
  if constexpr (sizeof(T) == 4) return __uint_as_float(m);
  m = max(m & 0xffffu, m >> 16);
  if constexpr (std::is_same<T, __half>::value) return __half2float(__ushort_as_half(static_cast<unsigned short>(m)));
  return __uint_as_float(m << 16);
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

// grid (ceil(T / tokens of a block), head groups); d = D; T: type of the input rows
template <int KIND, typename T, int D>
__global__ void __launch_bounds__(kKvThreads) k_kv_write(const KvWriteParams P) {
  constexpr int V = RopeVec<T>::kElems;      // elements of a lane
  constexpr int L = D / V;                   // lanes of a row
  constexpr int R = kKvThreads / L;          // rows of the block at a time (two a thread measured the same)
  __shared__ int64_t slot_sh[kKvTokens];
  const int tokens = 1 << P.tok_shift;
  const int t0 = blockIdx.x << P.tok_shift;
  if (threadIdx.x < tokens) {
    int64_t s = t0 + (int)threadIdx.x < P.T ? P.slots[t0 + threadIdx.x] : -1;
    if (s >= (P.g.pages << P.g.page_shift)) {
      s = -1;
      atomicOr(P.err, kDevErrRange);
    }
    slot_sh[threadIdx.x] = s;
  }
  __syncthreads();
  const int h0 = blockIdx.y * P.group, nh = min(P.group, P.g.heads - h0);
  const int lane = threadIdx.x % L, r0 = threadIdx.x / L;
  const int rows = tokens * nh;
  for (int base = 0; base < rows; base += R) {  // whole warps take part in the row maxima
    const int r = base + r0, tt = r & (tokens - 1), h = h0 + (r >> P.tok_shift);
    const int64_t slot = r < rows ? slot_sh[tt] : -1;
    const int64_t row = slot < 0 ? -1 : (((slot >> P.g.page_shift) * P.g.heads + h) << P.g.page_shift) + (slot & (P.g.page - 1));
    uint4 raw[2];
#pragma unroll
    for (int w = 0; w < 2; ++w) {
      raw[w] = make_uint4(0, 0, 0, 0);
      if (slot >= 0 && P.in[w])
        raw[w] = *reinterpret_cast<const uint4 *>(static_cast<const T *>(P.in[w]) + (t0 + tt) * P.tok[w] + h * P.head[w] +
                                                  lane * V);
    }
    float Ms[2];
    if constexpr (KvCode<KIND>::kQuant) {
      // the two scales, one division for both: lane w makes one
      float M = 0.f;
      int64_t at = -1;
      int kv = 0;
#pragma unroll
      for (int w = 0; w < 2; ++w) {
        Ms[w] = kv_row_max<T, L>(raw[w]);
        if (lane == w && P.in[w]) {
          M = Ms[w];
          at = row;
          kv = w;
        }
      }
      if (at >= 0) P.g.scale[kv][at] = M < INFINITY ? __fdiv_rn(M, KvCode<KIND>::kTop) : __uint_as_float(0x7fc00000u);
    }
#pragma unroll
    for (int w = 0; w < 2; ++w) {
      if (!P.in[w]) continue;
      float x[V];
      RopeVec<T>::unpack(raw[w], x);
      if constexpr (KvCode<KIND>::kQuant) {
        constexpr bool kExact = sizeof(T) == 4;
        const float M = Ms[w];
        uint32_t code[V / 4] = {};
        if (M > 1e-30f && M < 1e30f) {
          kv_quantise<KIND, V, kExact>(x, M, code);
        } else if (M > 0.f && M < INFINITY) {
          // c / M would leave fp32: the row times 2^100 or 2^-100, which the quotient does not see
          const float f = M < 1.f ? 1.2676506002282294e30f : 7.888609052210118e-31f;
          float z[V];
#pragma unroll
          for (int i = 0; i < V; ++i) z[i] = x[i] * f;
          kv_quantise<KIND, V, kExact>(z, M * f, code);
        }
        if (row >= 0) {
          uint8_t *dst = static_cast<uint8_t *>(P.g.pool[w]) + row * D + lane * V;
          if constexpr (V == 8) *reinterpret_cast<uint2 *>(dst) = make_uint2(code[0], code[1]);
          else *reinterpret_cast<uint32_t *>(dst) = code[0];
        }
      } else if (row >= 0) {
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

// grid (ceil(T / tokens of a block), head groups); T: type of the output rows
template <int KIND, typename T, int D>
__global__ void __launch_bounds__(kKvThreads) k_kv_read(const KvReadParams P) {
  constexpr int VO = RopeVec<T>::kElems;     // output elements of a 16-byte vector
  constexpr int V = 8;                       // elements of a lane
  constexpr int L = D / V;
  constexpr int R = kKvThreads / L;
  constexpr int U = KvCode<KIND>::kQuant ? 4 : 2;  // rows in flight
  __shared__ int64_t slot_sh[kKvTokens];
  const int tokens = 1 << P.tok_shift;
  const int t0 = blockIdx.x << P.tok_shift;
  if (threadIdx.x < tokens) {
    const int t = t0 + threadIdx.x;
    int64_t slot = -1;
    if (t < P.T && t >= P.cu[0] && t < P.cu[P.nseq]) {
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
  const int rows = tokens * nh;
  using Raw = typename std::conditional<KvCode<KIND>::kQuant, uint2, uint4>::type;
  for (int base = 0; base < rows; base += U * R) {
    Raw raw[U][2];
    float sc[U][2];
    bool have[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int r = base + u * R + r0, tt = r & (tokens - 1), h = h0 + (r >> P.tok_shift);
      const int64_t slot = r < rows ? slot_sh[tt] : -1;
      have[u] = slot >= 0;
      const int64_t row = (((slot >> P.g.page_shift) * P.g.heads + h) << P.g.page_shift) + (slot & (P.g.page - 1));
#pragma unroll
      for (int w = 0; w < 2; ++w)
        if (have[u] && P.out[w]) {
          raw[u][w] = *reinterpret_cast<const Raw *>(static_cast<const uint8_t *>(P.g.pool[w]) +
                                                     (row * D + lane * V) * KvCode<KIND>::kBytes);
          if constexpr (KvCode<KIND>::kQuant) sc[u][w] = P.g.scale[w][row];
        }
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int r = base + u * R + r0, tt = r & (tokens - 1), h = h0 + (r >> P.tok_shift);
#pragma unroll
      for (int w = 0; w < 2; ++w) {
        if (!have[u] || !P.out[w]) continue;
        float x[V];
        if constexpr (KvCode<KIND>::kQuant) {
          kv_values4<KIND>(raw[u][w].x, x);
          kv_values4<KIND>(raw[u][w].y, x + 4);
#pragma unroll
          for (int i = 0; i < V; ++i) x[i] *= sc[u][w];
        } else {
          using C = typename std::conditional<KIND == kKvBf16, __nv_bfloat16, __half>::type;
          RopeVec<C>::unpack(raw[u][w], x);
        }
        T *dst = static_cast<T *>(P.out[w]) + (t0 + tt) * P.tok[w] + h * P.head[w] + lane * V;
#pragma unroll
        for (int i = 0; i < V; i += VO) *reinterpret_cast<uint4 *>(dst + i) = RopeVec<T>::pack(x + i);
      }
    }
  }
}

}  // namespace fpk
