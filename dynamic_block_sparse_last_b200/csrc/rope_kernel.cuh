// rope_kernel.cuh -- rotary positions on sm_100a, any layout, part of the head.
//
// Pair (a, b) of frequency f at position p, x = p f, amplitude m:
//   a' = m (a cos x - b sin x),  b' = m (b cos x + a sin x).
// The angle is kept in turns as 64-bit fixed point: F = round(f / (2 pi) 2^64)
// is made on the host, and p F mod 2^64 is the fraction of a turn, off by at
// most |p| 2^-65 turns (2^-34 at p = 2^31) where an fp32 product p f would be
// off by whole turns at long contexts.  Its top 32 bits, as a signed number,
// are the angle in [-1/2, 1/2) turns, rounded to fp32 (2^-25 turns) for
// sincospi.
//
// Bound: memory, 2 x size bytes an element.  A thread holds the sines and
// cosines of one slot (VEC pairs of one token) in registers and walks the heads
// of its group, so the 64-bit products and the sines are paid once for up to
// Hq + Hkv heads and no table is read; a slot is two 16-byte vectors of a head.
// Measured: 131072 tokens of 32 + 8 bf16 heads of 128 in 412 us, 6.5 TB/s (0.99 of the
// measured copy); 64 tokens in 2.7 us.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <stdint.h>

namespace fpk {

constexpr int kRopeMaxPairs = 128;

struct RopeSide {
  const void *in;
  void *out;
  int64_t in_tok, in_head, out_tok, out_head;
  int heads;
};

struct RopeParams {
  RopeSide side[2];  // q, k
  const int *pos;
  int T, rot, d;
  int slots;         // slots of a token: rotated, then passed through
  int rot_slots;
  int group;         // heads of a thread
  int copy_tail;     // some output is not its own input
  float amp, sign;   // sign: -1 for the inverse
  unsigned long long turn[kRopeMaxPairs];
};

template <typename T>
struct RopeVec;
template <>
struct RopeVec<float> {
  static constexpr int kElems = 4;
  static __device__ __forceinline__ void unpack(const uint4 &r, float *x) {
    x[0] = __uint_as_float(r.x); x[1] = __uint_as_float(r.y);
    x[2] = __uint_as_float(r.z); x[3] = __uint_as_float(r.w);
  }
  static __device__ __forceinline__ uint4 pack(const float *x) {
    return make_uint4(__float_as_uint(x[0]), __float_as_uint(x[1]), __float_as_uint(x[2]), __float_as_uint(x[3]));
  }
};
template <>
struct RopeVec<__nv_bfloat16> {
  static constexpr int kElems = 8;
  static __device__ __forceinline__ void unpack(const uint4 &r, float *x) {
    const uint32_t w[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      x[2 * i] = __uint_as_float(w[i] << 16);
      x[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    }
  }
  static __device__ __forceinline__ uint4 pack(const float *x) {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const __nv_bfloat162 v = __floats2bfloat162_rn(x[2 * i], x[2 * i + 1]);
      w[i] = *reinterpret_cast<const uint32_t *>(&v);
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
  }
};
template <>
struct RopeVec<__half> {
  static constexpr int kElems = 8;
  static __device__ __forceinline__ void unpack(const uint4 &r, float *x) {
    const uint32_t w[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 f = __half22float2(*reinterpret_cast<const __half2 *>(&w[i]));
      x[2 * i] = f.x;
      x[2 * i + 1] = f.y;
    }
  }
  static __device__ __forceinline__ uint4 pack(const float *x) {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const __half2 v = __floats2half2_rn(x[2 * i], x[2 * i + 1]);
      w[i] = *reinterpret_cast<const uint32_t *>(&v);
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
  }
};

// cos and sin (times amplitude, sine signed) of one pair's angle.
__device__ __forceinline__ void rope_angle(const RopeParams &P, int pos, int pair, float &c, float &s) {
  const unsigned long long t = static_cast<unsigned long long>(static_cast<long long>(pos)) * P.turn[pair];
  const float x = static_cast<float>(static_cast<int>(t >> 32)) * 4.656612873077393e-10f;  // 2^-31: half turns
  float sn, cs;
  sincospif(x, &sn, &cs);
  c = P.amp * cs;
  s = P.amp * P.sign * sn;
}

// Rows of 16-byte vectors.  grid (ceil(T * slots / 256), head groups).
template <typename T, bool HALF>
__global__ void __launch_bounds__(256) k_rope(const __grid_constant__ RopeParams P) {
  constexpr int V = RopeVec<T>::kElems;
  const int64_t gid = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (gid >= (int64_t)P.T * P.slots) return;
  const int t = (int)(gid / P.slots), sl = (int)(gid - (int64_t)t * P.slots);
  const bool turn = sl < P.rot_slots;
  if (!turn && !P.copy_tail) return;
  // element offsets of the slot's two vectors, and their pairs
  int e0, e1;
  if (!turn) {
    e0 = P.rot + 2 * V * (sl - P.rot_slots);
    e1 = e0 + V;
  } else if (HALF) {
    e0 = V * sl;
    e1 = P.rot / 2 + V * sl;
  } else {
    e0 = 2 * V * sl;
    e1 = e0 + V;
  }
  float c[V], s[V];
  if (turn) {
    const int p = P.pos[t];
#pragma unroll
    for (int i = 0; i < V; ++i) rope_angle(P, p, V * sl + i, c[i], s[i]);
  }
  const int h0 = blockIdx.y * P.group, h1 = min(h0 + P.group, P.side[0].heads + P.side[1].heads);
  constexpr int U = 4;  // heads in flight
  for (int h = h0; h < h1; h += U) {
    uint4 r0[U], r1[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      if (h + u >= h1) break;
      const int k = h + u >= P.side[0].heads;
      const RopeSide &S = P.side[k];
      const T *in = static_cast<const T *>(S.in) + t * S.in_tok + (h + u - (k ? P.side[0].heads : 0)) * S.in_head;
      r0[u] = *reinterpret_cast<const uint4 *>(in + e0);
      r1[u] = *reinterpret_cast<const uint4 *>(in + e1);
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      if (h + u >= h1) break;
      const int k = h + u >= P.side[0].heads;
      const RopeSide &S = P.side[k];
      T *out = static_cast<T *>(S.out) + t * S.out_tok + (h + u - (k ? P.side[0].heads : 0)) * S.out_head;
      if (turn) {
        float x[2 * V], y[2 * V];
        RopeVec<T>::unpack(r0[u], x);
        RopeVec<T>::unpack(r1[u], x + V);
#pragma unroll
        for (int i = 0; i < V; ++i) {
          const int ia = HALF ? i : 2 * i, ib = HALF ? V + i : 2 * i + 1;
          y[ia] = fmaf(x[ia], c[i], -x[ib] * s[i]);
          y[ib] = fmaf(x[ib], c[i], x[ia] * s[i]);
        }
        r0[u] = RopeVec<T>::pack(y);
        r1[u] = RopeVec<T>::pack(y + V);
      }
      *reinterpret_cast<uint4 *>(out + e0) = r0[u];
      *reinterpret_cast<uint4 *>(out + e1) = r1[u];
    }
  }
}

template <typename T>
__device__ __forceinline__ float rope_to_float(T x);
template <>
__device__ __forceinline__ float rope_to_float(float x) { return x; }
template <>
__device__ __forceinline__ float rope_to_float(__nv_bfloat16 x) { return __bfloat162float(x); }
template <>
__device__ __forceinline__ float rope_to_float(__half x) { return __half2float(x); }
template <typename T>
__device__ __forceinline__ T rope_from_float(float x);
template <>
__device__ __forceinline__ float rope_from_float(float x) { return x; }
template <>
__device__ __forceinline__ __nv_bfloat16 rope_from_float(float x) { return __float2bfloat16(x); }
template <>
__device__ __forceinline__ __half rope_from_float(float x) { return __float2half(x); }

// Any even sizes and element alignment: a slot is one pair, or two elements
// passed through.
template <typename T, bool HALF>
__global__ void __launch_bounds__(256) k_rope_any(const __grid_constant__ RopeParams P) {
  const int64_t gid = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (gid >= (int64_t)P.T * P.slots) return;
  const int t = (int)(gid / P.slots), sl = (int)(gid - (int64_t)t * P.slots);
  const bool turn = sl < P.rot_slots;
  if (!turn && !P.copy_tail) return;
  const int e0 = turn && HALF ? sl : 2 * sl, e1 = turn && HALF ? P.rot / 2 + sl : 2 * sl + 1;
  float c = 1.f, s = 0.f;
  if (turn) rope_angle(P, P.pos[t], sl, c, s);
  const int h0 = blockIdx.y * P.group, h1 = min(h0 + P.group, P.side[0].heads + P.side[1].heads);
  for (int h = h0; h < h1; ++h) {
    const int k = h >= P.side[0].heads;
    const RopeSide &S = P.side[k];
    const int hh = h - (k ? P.side[0].heads : 0);
    const T *in = static_cast<const T *>(S.in) + t * S.in_tok + hh * S.in_head;
    T *out = static_cast<T *>(S.out) + t * S.out_tok + hh * S.out_head;
    const T ra = in[e0], rb = in[e1];
    if (turn) {
      const float a = rope_to_float<T>(ra), b = rope_to_float<T>(rb);
      out[e0] = rope_from_float<T>(fmaf(a, c, -b * s));
      out[e1] = rope_from_float<T>(fmaf(b, c, a * s));
    } else {
      out[e0] = ra;
      out[e1] = rb;
    }
  }
}

}  // namespace fpk
