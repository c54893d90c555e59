// tree_tc.cuh -- attention of drafted tokens over the paged cache for more
// than 32 query rows of a KV head (trees, grouped heads): tcgen05.
//
// The mathematics, the work split and the join are those of tree_kernels.cuh.  A
// CTA (one per SM) works on 128-row query tiles and 128-token K/V tiles:
//   warps 0-3, 4-7  two softmax groups, a thread per query row
//   warps 8-11      K/V: codes -> fp16 operands (fp16 holds them exactly), V's
//                   tokens behind the sequence -> zeros
//   warp 12         tensor memory and the MMAs (one thread)
//   warp 13         TMA producer: pages -> ring of raw tiles
//   warps 14, 15    idle (registers come in whole warpgroups)
// More than 128 rows (PAIR): the groups hold two query tiles and share every K/V
// tile.  Up to 128 rows: the groups hold the same query tile and take alternate K/V
// tiles, each with its own reference, sum and O, and are added at the end; a softmax
// takes longer than the memory needs for a tile, and so two are under way.
// Operands of bf16 and fp16 caches are multiplied where TMA put them.
// TMEM: S_t at 128 t, O_t at 256 + 128 t; P, in 16 bits, over the first half of S.
//
// A byte of K and V serves up to 256 rows, 2 (bf16) to 4 (8 bits) flops a row: up to
// 128 rows the bound is memory, with 256 rows over an 8-bit cache it is the tensor
// pipe and, as much, the exponentials (128 x 256 of them a tile at 16 a clock are
// 2048 clocks, as many as its products take).
//
// Softmax: 32 scores of a row at a time, each read once from tensor memory: their
// largest, then the exponentials, P written over columns of S that are read already
// (whole rows in registers spilled, and with 192 KB of operands there is no L1 to
// spill to).  Where a row's unit moves (Units in tree_kernels.cuh), the P of the tile
// that is already written is scaled in fp32 and rounded again, which changes only what
// becomes smaller than the type's smallest normal number.
// Sums are of the unrounded exponentials.
//
// Measured (32 query heads, 8 KV heads of 128): 64 drafted tokens over 131072 cached in
// bf16 in 172 us (799 TFLOP/s), in e4m3 in 235 to 243 us; 16 drafted tokens for 8
// sequences of up to 32768 in bf16 in 142 us, 5.4 TB/s (157 to 160 us, 4.8 TB/s, after
// seconds under load).  Of 256 rows over 8 bits a tile took about 6200 clocks when that took
// 220 us (units move more often since): softmax 4100, then the wait for PV and QK; the products need
// 2048, shared memory (Q twice, K and V twice, the conversion's traffic) about 2560.
//
// The K/V warps read shared memory that TMA filled and not global memory: the
// proxy fence before they hand an operand to the tensor core, and the barrier's
// release, wait for all of a thread's loads in flight (3600 clocks a tile measured
// with a prefetch in registers).
#pragma once

#include "tree_kernels.cuh"

namespace fpk {

constexpr int kTcBN = 128;

constexpr int kTcThreads = 512;

template <int KIND, int D, bool PAIR>
struct TcCfg {
  static constexpr bool kQuant = KvCode<KIND>::kQuant;
  static constexpr int BM = PAIR ? 256 : 128;
  static constexpr int kOp = 128 * D * 2;                 // bytes of a 128-row 16-bit operand tile
  static constexpr int RB = D * KvCode<KIND>::kBytes;     // bytes of a cached row
  static constexpr int kBoxB = RB < 128 ? RB : 128;
  static constexpr int kRaw = 128 * RB;                   // bytes of a raw K (or V) tile
  static constexpr int kRow16 = RB / 16;                  // 16-byte pieces of a row
  static constexpr int kStages = D == 128 ? 2 : 3;        // raw tiles in flight
  // Operand buffers: the raw tiles themselves when not quantised; else one, two where
  // they fit (V first: its conversion would wait for the product before it).
  static constexpr int kOpsK = !kQuant ? kStages : D == 64 ? 2 : 1;
  static constexpr int kOpsV = !kQuant ? kStages : D == 64 || !PAIR ? 2 : 1;
  static constexpr int kQOff = 0, kKOff = (PAIR ? 2 : 1) * kOp, kVOff = kKOff + kOpsK * kOp;
  static constexpr int kRkOff = kQuant ? kVOff + kOpsV * kOp : kKOff, kRvOff = kQuant ? kRkOff + kStages * kRaw : kVOff;
  static constexpr int kEnd = kRvOff + kStages * kRaw;
  static constexpr int kRsOff = kEnd;                     // raw scales [stage][K, V][128] fp32
  static constexpr int kSmem = kRsOff + (kQuant ? kStages * 1024 : 0) + 1024;
  static constexpr int kSc = 4;                           // scale ring
};

__device__ __forceinline__ void fence_async_shared() { asm volatile("fence.proxy.async.shared::cta;" ::: "memory"); }
__device__ __forceinline__ void sts128(uint32_t a, uint32_t x, uint32_t y, uint32_t z, uint32_t w) {
  asm volatile("st.shared.v4.b32 [%0], {%1,%2,%3,%4};" ::"r"(a), "r"(x), "r"(y), "r"(z), "r"(w) : "memory");
}

// tcgen05.mma with the shared-memory descriptors given as the low word (address
// and leading offset) and the high word that all of an operand's steps share, so
// that the issuing thread holds no 64-bit descriptor per step.
__device__ __forceinline__ void tc_mma_ss(uint32_t d, uint32_t a_lo, uint32_t a_hi, uint32_t b_lo, uint32_t b_hi,
                                          uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t.reg .b64 a, b;\n\tsetp.ne.b32 p, %6, 0;\n\tmov.b64 a, {%1, %2};\n\tmov.b64 b, {%3, %4};\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], a, b, %5, p;\n\t}\n" ::"r"(d),
      "r"(a_lo), "r"(a_hi), "r"(b_lo), "r"(b_hi), "r"(idesc), "r"(accumulate)
      : "memory");
}
__device__ __forceinline__ void tc_mma_ts(uint32_t d, uint32_t a_tmem, uint32_t b_lo, uint32_t b_hi, uint32_t idesc,
                                          uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t.reg .b64 b;\n\tsetp.ne.b32 p, %5, 0;\n\tmov.b64 b, {%2, %3};\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], b, %4, p;\n\t}\n" ::"r"(d),
      "r"(a_tmem), "r"(b_lo), "r"(b_hi), "r"(idesc), "r"(accumulate)
      : "memory");
}

__device__ __forceinline__ void tc_st16(uint32_t taddr, const uint32_t (&r)[16]) {
  asm volatile("tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(taddr),
               "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
               "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
               : "memory");
}

__device__ __forceinline__ void tc_ld16(uint32_t taddr, uint32_t (&r)[16]) {
  asm volatile("tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
                 "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
               : "r"(taddr));
}
__device__ __forceinline__ void tc_ld_wait16(uint32_t (&r)[16]) {
  asm volatile("tcgen05.wait::ld.sync.aligned;"
               : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]), "+r"(r[6]), "+r"(r[7]), "+r"(r[8]),
                 "+r"(r[9]), "+r"(r[10]), "+r"(r[11]), "+r"(r[12]), "+r"(r[13]), "+r"(r[14]), "+r"(r[15])::"memory");
}
// Two packed 16-bit values times a power of two, which may be below fp16's range (the values
// are up to 2^15, so the products need not be).
template <int KIND>
__device__ __forceinline__ uint32_t tc_scale2(uint32_t x, float by) {
  if constexpr (KIND == kKvBf16) {
    return pack_bf16x2(__uint_as_float(x << 16) * by, __uint_as_float(x & 0xffff0000u) * by);
  } else {
    const float2 f = __half22float2(*reinterpret_cast<const __half2 *>(&x));
    return pack_f16x2(f.x * by, f.y * by);
  }
}

// Instruction descriptor as idesc_bf16, operand format 0 = fp16 or 1 = bf16.
__host__ __device__ constexpr uint32_t tc_idesc(int M, int N, int b_mn_major, uint32_t fmt) {
  return (1u << 4) | (fmt << 7) | (fmt << 10) | (static_cast<uint32_t>(b_mn_major) << 16) |
         (static_cast<uint32_t>(N >> 3) << 17) | (static_cast<uint32_t>(M >> 4) << 24);
}

// Offset of 16-byte chunk c (0 .. D/8-1) of row r in a swizzled operand tile.
__device__ __forceinline__ uint32_t tc_off(int r, int c) {
  return (c >> 3) * 16384 + r * 128 + (((c & 7) ^ (r & 7)) << 4);
}
// The same in a raw tile of quantised rows (128 or 64 bytes).
template <int RB>
__device__ __forceinline__ uint32_t tc_raw_off(int r, int c) {
  if constexpr (RB == 128) return r * 128 + ((c ^ (r & 7)) << 4);
  else return r * 64 + ((c ^ ((r >> 1) & 3)) << 4);
}

// Which of the 32 tokens from position pos on the sequence's new token i sees.
__device__ __forceinline__ uint32_t tc_sees(const TreeParams &P, const TreeSeq &q, int i, int pos, int prefix) {
  const int in = q.len - pos, w0 = pos - prefix;  // tokens to the end; the first one's place among the new ones
  if (in <= 0) return 0u;
  unsigned long long v;
  if (P.mask) {
    const unsigned long long *m = P.mask + (int64_t)(q.row0 + i) * P.W;
    if (w0 < 0) {
      v = w0 <= -32 ? ~0ull : ((1ull << -w0) - 1) | (m[0] << -w0);
    } else {
      const int k = w0 >> 6, sh = w0 & 63;
      v = m[k] >> sh;  // in > 0: word k exists
      if (sh > 32 && k + 1 < P.W) v |= m[k + 1] << (64 - sh);
    }
  } else {
    const int upto = i + 1 - w0;  // new tokens 0 .. i
    v = upto >= 32 ? ~0ull : upto <= 0 ? 0ull : (1ull << upto) - 1;
  }
  if (in < 32) v &= (1ull << in) - 1;
  return (uint32_t)v;
}

// Eight bf16 elements of a query row, which LR lanes hold, as fp16, the row divided by
// the power of two below its largest magnitude; returns that power.
template <int LR>
__device__ __forceinline__ float tc_q_f16(uint4 &x) {
  float f[8];
  RopeVec<__nv_bfloat16>::unpack(x, f);
  float mx = 0.f;
#pragma unroll
  for (int e = 0; e < 8; ++e) mx = fmaxf(mx, fabsf(f[e]));
#pragma unroll
  for (int o = LR / 2; o > 0; o >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
  const int e = tree_q_exp(mx);
  const float inv = pow2i(-e);
  x = make_uint4(pack_f16x2(f[0] * inv, f[1] * inv), pack_f16x2(f[2] * inv, f[3] * inv), pack_f16x2(f[4] * inv, f[5] * inv),
                 pack_f16x2(f[6] * inv, f[7] * inv));
  return pow2i(e);
}

// Adds the non-finite values of the new tokens that row token i sees to its columns
// [c0, c1) of the stored result (16-bit when half >= 0: bf16 0, fp16 1; else fp32),
// which makes them what they are whatever the finite rest is.  The rare path: not
// inlined, so that it costs the usual one no registers.
template <int KIND, int D>
__device__ __noinline__ void tc_fixup(const TreeParams &P, const void *v_pool, int s, int j, int row0, int i, int len, int n,
                                      int pos_a, int pos_b, int c0, int c1, void *dst, int half) {
  TreeSeq q;
  q.row0 = row0;
  for (int jj = 0; jj < n; ++jj) {
    const int pos = len - n + jj;
    if (pos < pos_a || pos >= pos_b || !tree_sees(P, q, i, jj)) continue;
    for (int c = c0; c < c1; ++c) {
      const float y = tree_v_value<KIND, D>(P, v_pool, s, j, pos, c);
      if (fabsf(y) < INFINITY) continue;
      if (half < 0) static_cast<float *>(dst)[c] += y;
      else if (half) static_cast<__half *>(dst)[c] = __float2half(__half2float(static_cast<__half *>(dst)[c]) + y);
      else static_cast<__nv_bfloat16 *>(dst)[c] = __float2bfloat16(__bfloat162float(static_cast<__nv_bfloat16 *>(dst)[c]) + y);
    }
  }
}

// The 128 x D elements of a raw tile of codes as an fp16 operand tile; CLEAN: rows
// from `left` on become 0, and NaN codes of rows from `fresh` on (which raise bad).
// Eight neighbouring lanes take four 16-byte pieces of rows r and r ^ 5: in the
// swizzle, both the pieces read and the two halves written then lie in eight
// different bank groups.  A thread's rows are 32 apart, so its addresses are three
// and constants.
template <typename C, int KIND, bool CLEAN>
__device__ __forceinline__ void tc_convert(uint32_t raw, uint32_t op, int ct, int fresh, int left, int &bad) {
  const int c = ct & 3, row = (((ct >> 3) & 3) | ((ct >> 5) << 3)) ^ (((ct >> 2) & 1) * 5);
  const uint32_t r0 = raw + tc_raw_off<C::RB>(row, c), a0 = op + tc_off(row, 2 * c), a1 = a0 ^ 16;
  const uint32_t r1 = r0 ^ 64;  // the row's second 64 bytes (128-byte rows)
#pragma unroll
  for (int it = 0; it < 4; ++it)
#pragma unroll
    for (int cc = 0; cc < C::kRow16 / 4; ++cc) {
      const uint4 v = lds128((cc ? r1 : r0) + it * 32 * C::RB);
      uint32_t x[4] = {v.x, v.y, v.z, v.w}, y[8];
      if constexpr (CLEAN) {
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          if (row + 32 * it >= left) x[e] = 0u;
          else if (row + 32 * it >= fresh) x[e] = tree_clean<KIND>(x[e], bad);
        }
      }
#pragma unroll
      for (int e = 0; e < 4; ++e) tree_codes4<KIND>(KIND == kKvInt8 ? x[e] ^ 0x80808080u : x[e], y[2 * e], y[2 * e + 1]);
      sts128(a0 + it * 4096 + cc * 16384, y[0], y[1], y[2], y[3]);
      sts128(a1 + it * 4096 + cc * 16384, y[4], y[5], y[6], y[7]);
    }
}

template <int KIND, int D, bool PAIR>
__global__ void __launch_bounds__(kTcThreads, 1)
    k_tree_tc(const __grid_constant__ CUtensorMap tm_k, const __grid_constant__ CUtensorMap tm_v,
              const __grid_constant__ TreeParams P, const void *v_pool) {
  using C = TcCfg<KIND, D, PAIR>;
  constexpr int kMma = 12, kTma = 13;
  constexpr int kQWarps = PAIR ? 4 : 8;   // warps that write a query tile
  extern __shared__ uint8_t smem_raw[];
  __shared__ __align__(8) uint64_t bar_q[2], bar_rkf[C::kStages], bar_rke[C::kStages], bar_rvf[C::kStages],
      bar_rve[C::kStages], bar_kfull[C::kOpsK], bar_kempty[C::kOpsK], bar_vfull[C::kOpsV], bar_vempty[C::kOpsV], bar_sfull[2],
      bar_pfull[2], bar_odone[2], bar_scfull[C::kSc], bar_scempty[C::kSc];
  __shared__ __align__(16) float sc_k[C::kSc][kTcBN], sc_v[C::kSc][kTcBN], sc_l[C::kSc][kTcBN];  // sc_l: log2 of sc_v,
  __shared__ float sc_m[C::kSc][4];                                                                      // and bounds of 32
  __shared__ float row_scale[PAIR ? 2 : 1][128], x_m[2][128], x_l[2][128];
  __shared__ long long warp_sum[kTcThreads / 32];
  __shared__ TreeShare share;
  __shared__ uint32_t tmem_sh;
  __shared__ int abort_sh, bad_sh;  // bad_sh stays raised: it only asks the segments' ends to look

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t base = (smem_u32(smem_raw) + 1023u) & ~1023u;
  if (threadIdx.x == 0) {
    abort_sh = 0;
    bad_sh = 0;
    for (int i = 0; i < 2; ++i) {
      mbar_init(smem_u32(&bar_q[i]), kQWarps);
      mbar_init(smem_u32(&bar_sfull[i]), 1);
      mbar_init(smem_u32(&bar_pfull[i]), 4);
      mbar_init(smem_u32(&bar_odone[i]), 1);
    }
    for (int i = 0; i < C::kStages; ++i) {
      mbar_init(smem_u32(&bar_rkf[i]), 1);
      mbar_init(smem_u32(&bar_rke[i]), 4);
      mbar_init(smem_u32(&bar_rvf[i]), 1);
      mbar_init(smem_u32(&bar_rve[i]), 4);
    }
    for (int i = 0; i < C::kOpsK; ++i) {
      mbar_init(smem_u32(&bar_kfull[i]), 4);
      mbar_init(smem_u32(&bar_kempty[i]), 1);
    }
    for (int i = 0; i < C::kOpsV; ++i) {
      mbar_init(smem_u32(&bar_vfull[i]), 4);
      mbar_init(smem_u32(&bar_vempty[i]), 1);
    }
    for (int i = 0; i < C::kSc; ++i) {
      mbar_init(smem_u32(&bar_scfull[i]), 1);
      mbar_init(smem_u32(&bar_scempty[i]), PAIR ? 8 : 4);
    }
    fence_mbar_init();
  }
  if (warp == kMma) {
    tmem_alloc(smem_u32(&tmem_sh), 512);
    tmem_relinquish();
  }
  tree_share<kTcThreads>(P, C::BM, kTcBN, &share, warp_sum);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const uint32_t tmem = tmem_sh;
  volatile int *abort_flag = &abort_sh;
  TreeWalk w;
  bool more = w.start(P, share, C::BM, kTcBN);
  const uint32_t sq = base + C::kQOff, sk = base + C::kKOff, sv = base + C::kVOff;

  if (warp == kMma) {
    // ------------------------------------------------------------ MMA issuer
    // Items i of a segment: query tile i & 1 with K/V tile i / 2 (PAIR), or K/V tile
    // i for group i & 1.  Order: QK(0), QK(1), PV(0), QK(2), PV(1), QK(3), ...
    if (lane == 0) {
      constexpr uint32_t fmt = KIND == kKvBf16 ? 1u : 0u;
      constexpr uint32_t id_qk = tc_idesc(128, 128, 0, fmt), id_pv = tc_idesc(128, D, 1, fmt);
      // an operand is below 64 KB from its ring's start: adding to the low words never carries out of the address field
      const uint32_t dq_lo = (uint32_t)umma_desc_sw128(sq, 16, 1024), dk_lo = (uint32_t)umma_desc_sw128(sk, 16, 1024),
                     dv_lo = (uint32_t)umma_desc_sw128(sv, 16384, 1024),
                     desc_hi = (uint32_t)(umma_desc_sw128(sq, 16, 1024) >> 32);
      int u0 = 0, seg = 0, npv[2] = {0, 0};  // tiles before the segment, segments, PV products (barrier phases)
      bool ok = true;
      for (; more && ok; u0 += w.b - w.a, more = w.next(P, C::BM, kTcBN), ++seg) {
        const int I = (w.b - w.a) * (PAIR ? 2 : 1);
        for (int t = 0; t < (PAIR ? 2 : 1) && ok; ++t) ok = mbar_wait(smem_u32(&bar_q[t]), seg & 1, abort_flag, P.err);
        for (int i = 0; i < I + 2 && ok; ++i) {
          const int t = i & 1;
          if (i >= 2) {
            const int u = u0 + (PAIR ? (i - 2) >> 1 : i - 2), st = u % C::kOpsV;
            if ((!PAIR || t == 0) && !mbar_wait(smem_u32(&bar_vfull[st]), (u / C::kOpsV) & 1, abort_flag, P.err)) { ok = false; break; }
            if (!mbar_wait(smem_u32(&bar_pfull[t]), npv[t] & 1, abort_flag, P.err)) { ok = false; break; }
            tc_fence_after();
            const uint32_t dv = dv_lo + ((st * C::kOp) >> 4);
            const bool acc = i >= 4;  // the group's first product of the segment starts O
#pragma unroll
            for (int kk = 0; kk < 8; ++kk)
              tc_mma_ts(tmem + 256 + t * 128, tmem + t * 128 + kk * 8, dv + ((kk * 2048) >> 4), desc_hi, id_pv, acc || kk > 0);
            tc_commit(smem_u32(&bar_odone[t]));
            ++npv[t];
            if (!PAIR || t == 1) tc_commit(smem_u32(&bar_vempty[st]));
          }
          if (i < I) {
            const int u = u0 + (PAIR ? i >> 1 : i), st = u % C::kOpsK;
            // K of an unquantised cache is used as TMA left it
            const uint32_t full = C::kQuant ? smem_u32(&bar_kfull[st]) : smem_u32(&bar_rkf[st]);
            if ((!PAIR || t == 0) && !mbar_wait(full, (u / C::kOpsK) & 1, abort_flag, P.err)) { ok = false; break; }
            tc_fence_after();
            const uint32_t dq = dq_lo + (((PAIR ? t : 0) * C::kOp) >> 4), dk = dk_lo + ((st * C::kOp) >> 4);
#pragma unroll
            for (int kk = 0; kk < D / 16; ++kk) {
              const uint32_t off = ((kk >> 2) * 16384 + (kk & 3) * 32) >> 4;
              tc_mma_ss(tmem + t * 128, dq + off, desc_hi, dk + off, desc_hi, id_qk, kk > 0);
            }
            tc_commit(smem_u32(&bar_sfull[t]));
            if (!PAIR || t == 1) tc_commit(smem_u32(&bar_kempty[st]));
          }
        }
      }
    }
  } else if (warp == kTma) {
    // ------------------------------------------------------------ producer
    // A tile is 128 / min(page, 64) pieces, each of one page; lane i moves piece i.
    const int piece = min(P.page, 64), pieces = kTcBN / piece;
    int u = 0;
    bool ok = true;
    for (; more && ok; more = w.next(P, C::BM, kTcBN)) {
      const int *tab = P.table + (int64_t)w.s * P.max_pages;
      int pg = 0;
      const int p0 = w.a * kTcBN + lane * piece;
      if (lane < pieces && p0 < w.q.len) pg = tab[p0 >> P.page_shift];
      for (int t = w.a; t < w.b; ++t, ++u) {
        const int pos = t * kTcBN + lane * piece, st = u % C::kStages;
        const bool mine = lane < pieces && pos < w.q.len;
        int id = pg;
        const int nx = pos + kTcBN;  // the next tile's page, ahead of its use
        if (t + 1 < w.b && lane < pieces && nx < w.q.len) pg = tab[nx >> P.page_shift];
        if (mine && (id < 0 || id >= P.pages)) {
          id = 0;
          atomicOr(P.err, kDevErrRange);
        }
        const int row = ((id * P.Hkv + w.j) << P.page_shift) + (pos & (P.page - 1));
        const int n = __popc(__ballot_sync(0xffffffffu, mine)) * piece;
        const uint32_t ph = ((u / C::kStages) - 1) & 1;
        // K and its scales
        if (u >= C::kStages) ok = mbar_wait(C::kQuant ? smem_u32(&bar_rke[st]) : smem_u32(&bar_kempty[st]), ph, abort_flag, P.err);
        if (!__all_sync(0xffffffffu, ok)) { ok = false; break; }
        const uint32_t kf = smem_u32(&bar_rkf[st]), vf = smem_u32(&bar_rvf[st]);
        if (lane == 0) mbar_expect_tx(kf, n * (C::RB + (C::kQuant ? 8 : 0)));
        __syncwarp();
        if (mine) {
          const uint32_t dst = base + C::kRkOff + st * C::kRaw + lane * piece * C::kBoxB;
#pragma unroll
          for (int x = 0; x < C::RB / C::kBoxB; ++x) tma_load_2d(dst + x * 16384, &tm_k, x * 128, row, kf);
          if constexpr (C::kQuant) {
            const uint32_t sd = base + C::kRsOff + st * 1024 + lane * piece * 4;
            bulk_load(sd, P.scale[0] + row, piece * 4, kf);
            bulk_load(sd + 512, P.scale[1] + row, piece * 4, kf);
          }
        }
        // V
        if (u >= C::kStages) ok = mbar_wait(C::kQuant ? smem_u32(&bar_rve[st]) : smem_u32(&bar_vempty[st]), ph, abort_flag, P.err);
        if (!__all_sync(0xffffffffu, ok)) { ok = false; ++u; break; }
        if (lane == 0) mbar_expect_tx(vf, n * C::RB);
        __syncwarp();
        if (mine) {
          const uint32_t dst = base + C::kRvOff + st * C::kRaw + lane * piece * C::kBoxB;
#pragma unroll
          for (int x = 0; x < C::RB / C::kBoxB; ++x) tma_load_2d(dst + x * 16384, &tm_v, x * 128, row, vf);
        }
      }
    }
    // nothing may end with copies in flight; after an abandoned wait nobody else waits for them
    if (!ok)
      for (int v = max(u - C::kStages, 0); v < u; ++v) {
        const unsigned long long t0 = globaltimer();
        while (!(mbar_try_wait(smem_u32(&bar_rkf[v % C::kStages]), (v / C::kStages) & 1) &&
                 mbar_try_wait(smem_u32(&bar_rvf[v % C::kStages]), (v / C::kStages) & 1)) &&
               globaltimer() - t0 < kWaitLimitNs) {
        }
      }
  } else if (warp >= 8 && warp < kMma) {
    // ------------------------------------------------------------ K and V
    const int cw = warp - 8, ct = threadIdx.x - 256;
    int u = 0, bad = 0;
    bool ok = true;
    for (; more && ok; more = w.next(P, C::BM, kTcBN)) {
      for (int t = w.a; t < w.b; ++t, ++u) {
        const int rst = u % C::kStages, kst = u % C::kOpsK, vst = u % C::kOpsV;
        const uint32_t rph = (u / C::kStages) & 1, kph = ((u / C::kOpsK) - 1) & 1, vph = ((u / C::kOpsV) - 1) & 1;
        const int left = w.q.len - t * kTcBN, fresh = left - w.q.n;  // tokens to the end; before the first new one
        if constexpr (C::kQuant) {
          ok = mbar_wait(smem_u32(&bar_rkf[rst]), rph, abort_flag, P.err);
          if (cw == 0) {
            // the scales of four tokens a lane
            const int ss = u % C::kSc;
            if (ok && u >= C::kSc) ok = mbar_wait(smem_u32(&bar_scempty[ss]), ((u / C::kSc) - 1) & 1, abort_flag, P.err);
            const uint4 a = lds128(base + C::kRsOff + rst * 1024 + lane * 16), b = lds128(base + C::kRsOff + rst * 1024 + 512 + lane * 16);
            float ks[4] = {__uint_as_float(a.x), __uint_as_float(a.y), __uint_as_float(a.z), __uint_as_float(a.w)};
            float vs[4] = {__uint_as_float(b.x), __uint_as_float(b.y), __uint_as_float(b.z), __uint_as_float(b.w)};
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              if (4 * lane + e >= left) {
                ks[e] = 1.f;
                vs[e] = 0.f;
              }
              // a new token's NaN scale: added at the end for the rows that see it
              if (4 * lane + e >= fresh && !(fabsf(vs[e]) < INFINITY)) {
                vs[e] = 0.f;
                bad = 1;
              }
            }
            *reinterpret_cast<float4 *>(&sc_k[ss][4 * lane]) = make_float4(ks[0], ks[1], ks[2], ks[3]);
            *reinterpret_cast<float4 *>(&sc_v[ss][4 * lane]) = make_float4(vs[0], vs[1], vs[2], vs[3]);
            const float4 lv = make_float4(tree_log2(vs[0]), tree_log2(vs[1]), tree_log2(vs[2]), tree_log2(vs[3]));
            *reinterpret_cast<float4 *>(&sc_l[ss][4 * lane]) = lv;
            float lm = fmaxf(fmaxf(lv.x, lv.y), fmaxf(lv.z, lv.w));
#pragma unroll
            for (int x = 1; x < 8; x <<= 1) lm = fmaxf(lm, __shfl_xor_sync(0xffffffffu, lm, x));
            if ((lane & 7) == 0) sc_m[ss][lane >> 3] = TreeUnit<KIND>::bound(lm);
            if (bad) bad_sh = 1;
            __syncwarp();
            if (lane == 0) mbar_arrive(smem_u32(&bar_scfull[ss]));
          }
          if (ok && u >= C::kOpsK) ok = mbar_wait(smem_u32(&bar_kempty[kst]), kph, abort_flag, P.err);
          if (!__all_sync(0xffffffffu, ok)) { ok = false; break; }
          tc_convert<C, KIND, false>(base + C::kRkOff + rst * C::kRaw, sk + kst * C::kOp, ct, 0, 0, bad);
          fence_async_shared();
          __syncwarp();
          if (lane == 0) {
            mbar_arrive(smem_u32(&bar_kfull[kst]));
            mbar_arrive(smem_u32(&bar_rke[rst]));
          }
          ok = mbar_wait(smem_u32(&bar_rvf[rst]), rph, abort_flag, P.err);
          if (ok && u >= C::kOpsV) ok = mbar_wait(smem_u32(&bar_vempty[vst]), vph, abort_flag, P.err);
          if (!__all_sync(0xffffffffu, ok)) { ok = false; break; }
          if (fresh < kTcBN) tc_convert<C, KIND, true>(base + C::kRvOff + rst * C::kRaw, sv + vst * C::kOp, ct, fresh, left, bad);
          else tc_convert<C, KIND, false>(base + C::kRvOff + rst * C::kRaw, sv + vst * C::kOp, ct, 0, 0, bad);
          if (bad) bad_sh = 1;
          fence_async_shared();
          __syncwarp();
          if (lane == 0) {
            mbar_arrive(smem_u32(&bar_vfull[vst]));
            mbar_arrive(smem_u32(&bar_rve[rst]));
          }
        } else {
          ok = __all_sync(0xffffffffu, mbar_wait(smem_u32(&bar_rvf[rst]), rph, abort_flag, P.err));
          if (!ok) break;
          if (fresh < kTcBN) {
            const int r0 = max(fresh, 0);
            for (int idx = ct; idx < (kTcBN - r0) * C::kRow16; idx += 128) {
              const int row = r0 + idx / C::kRow16, c = idx % C::kRow16;
              const uint32_t at = sv + vst * C::kOp + tc_off(row, c);
              if (row >= left) {
                sts128(at, 0u, 0u, 0u, 0u);
              } else {
                const uint4 v = lds128(at);
                int any = 0;
                const uint32_t x0 = tree_clean<KIND>(v.x, any), x1 = tree_clean<KIND>(v.y, any), x2 = tree_clean<KIND>(v.z, any),
                               x3 = tree_clean<KIND>(v.w, any);
                if (any) {
                  sts128(at, x0, x1, x2, x3);
                  bad_sh = 1;
                }
              }
            }
            fence_async_shared();
          }
          __syncwarp();
          if (lane == 0) mbar_arrive(smem_u32(&bar_vfull[vst]));
        }
      }
    }
  } else if (warp < 8) {
    // ------------------------------------------------------------ softmax
    const int t = warp >> 2, row = (warp & 3) * 32 + lane;
    const uint32_t lane_off = ((uint32_t)((warp & 3) * 32)) << 16;
    const uint32_t s_tm = tmem + t * 128 + lane_off, o_tm = tmem + 256 + lane_off;
    if (threadIdx.x == 0) P.desc[blockIdx.x].n = 0;
    long long at = share.begin;
    int u0 = 0, n = 0;  // tiles before the segment; items of this group so far (barrier phases)
    bool ok = true;     // after an abandoned wait the warps only keep the barriers below company
    for (; more; at += w.b - w.a, u0 += w.b - w.a, more = w.next(P, C::BM, kTcBN)) {
      const int prefix = w.q.len - w.q.n, rbase = w.m * C::BM, R = min(C::BM, w.q.n * P.g - rbase);
      // Q: a warp writes its share of the query tile's rows, 16 bytes a lane, all of
      // its rows under way at once; a lane works out where one row is
      if (ok) {
        constexpr int RW = 128 / kQWarps, LR = D / 8, NB = RW * LR / 32;  // rows of the warp, lanes of a row, loads of a lane
        const int first = (PAIR ? (warp & 3) : warp) * RW, unit0 = PAIR ? t * 128 : 0;
        long long off = -1;
        if (lane < RW && unit0 + first + lane < R) {
          const int gr = rbase + unit0 + first + lane, tok = gr / P.g;
          off = (w.q.row0 + tok) * P.q_tok + (w.j * P.g + gr - tok * P.g) * P.q_head;
        }
        uint4 x[NB];
#pragma unroll
        for (int i = 0; i < NB; ++i) {
          const long long o = __shfl_sync(0xffffffffu, off, i * (32 / LR) + lane / LR);
          x[i] = make_uint4(0, 0, 0, 0);
          if (o >= 0) x[i] = *reinterpret_cast<const uint4 *>(static_cast<const uint16_t *>(P.q) + o + (lane % LR) * 8);
        }
#pragma unroll
        for (int i = 0; i < NB; ++i) {
          const int r = first + i * (32 / LR) + lane / LR;
          float fac = 1.f;
          if (C::kQuant && !P.q_f16) fac = tc_q_f16<LR>(x[i]);
          const uint32_t dst = sq + (PAIR ? t * C::kOp : 0) + tc_off(r, lane % LR);
          sts128(dst, x[i].x, x[i].y, x[i].z, x[i].w);
          if (lane % LR == 0) row_scale[PAIR ? t : 0][r] = tree_row_scale(fac, P.scale2);
        }
        fence_async_shared();
      }
      if constexpr (PAIR) named_sync(1 + t, 128);
      else named_sync(1, 256);
      if (lane == 0) mbar_arrive(smem_u32(&bar_q[PAIR ? t : 0]));
      const int trow = (PAIR ? t * 128 : 0) + row;               // row of the unit
      const int grow = rbase + trow;                             // row of the sequence
      const bool have = trow < R;
      const bool live = (PAIR ? t * 128 : 0) + (warp & 3) * 32 < R;  // the warp has rows at all
      const int tk = min(grow / P.g, w.q.n - 1);
      const float rs = row_scale[PAIR ? t : 0][row];
      float m_ref = -INFINITY, l = 0.f;  // the row's unit (log2) and its sum in it
      const int L = w.b - w.a, cnt = PAIR ? L : (L - t + 1) / 2;  // tiles of this group
      for (int j = 0; j < cnt && ok; ++j, ++n) {
        const int tile = PAIR ? j : 2 * j + t, u = u0 + tile, ss = u % C::kSc;
        ok = mbar_wait(smem_u32(&bar_sfull[t]), n & 1, abort_flag, P.err);
        if (C::kQuant && ok) ok = mbar_wait(smem_u32(&bar_scfull[ss]), (u / C::kSc) & 1, abort_flag, P.err);
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) break;
        tc_fence_after();
        if (live) {
        const int pos0 = (w.a + tile) * kTcBN;
        float alpha = 1.f, sum = 0.f;
        bool moved = false;
        // compiled once for tiles that every row sees whole and once for the others
        auto rows_of_tile = [&](auto tail_tag) __attribute__((always_inline)) {
          constexpr bool tail = decltype(tail_tag)::value;
          const uint64_t rs2 = f2_pack(rs, rs);
          using U = TreeUnit<KIND>;
          uint64_t acc[4] = {0ull, 0ull, 0ull, 0ull};
#pragma unroll 1  // four copies of this and the other roles' code do not fit the instruction cache (295 -> 236 us)
          for (int hh = 0; hh < 4; ++hh) {
            uint32_t rr[32], pk[16];
            tmem_ld32(s_tm + 32 * hh, rr);
            tmem_ld_wait(rr);
            if constexpr (C::kQuant) {
#pragma unroll
              for (int e = 0; e < 32; e += 4) {
                const float4 k4 = *reinterpret_cast<const float4 *>(&sc_k[ss][hh * 32 + e]);
                const uint64_t a = f2_mul(f2_pack(__uint_as_float(rr[e]), __uint_as_float(rr[e + 1])), f2_pack(k4.x, k4.y));
                const uint64_t b = f2_mul(f2_pack(__uint_as_float(rr[e + 2]), __uint_as_float(rr[e + 3])), f2_pack(k4.z, k4.w));
                float x0, x1;
                f2_unpack(a, x0, x1);
                rr[e] = __float_as_uint(x0);
                rr[e + 1] = __float_as_uint(x1);
                f2_unpack(b, x0, x1);
                rr[e + 2] = __float_as_uint(x0);
                rr[e + 3] = __float_as_uint(x1);
              }
            }
            if constexpr (tail) {  // after K's scale, which may be a NaN
              const uint32_t vis = tc_sees(P, w.q, tk, pos0 + 32 * hh, prefix);
#pragma unroll
              for (int e = 0; e < 32; ++e)
                if (!((vis >> e) & 1u)) rr[e] = 0xff800000u;
            }
            float mx4[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) mx4[e] = __uint_as_float(rr[e]);
#pragma unroll
            for (int e = 4; e < 32; ++e) mx4[e & 3] = fmaxf(mx4[e & 3], __uint_as_float(rr[e]));
            const float top = fmaxf(fmaxf(mx4[0], mx4[1]), fmaxf(mx4[2], mx4[3])) * rs;  // rs > 0
            float lim = -(U::kLift + U::kSlack);
            if constexpr (C::kQuant) lim = sc_m[ss][hh];
            if (__any_sync(0xffffffffu, top + lim > m_ref)) {
              // the unit moves, by whole powers of two: the sums scale exactly, and so do the
              // P of the chunks before as far as their type goes
              float key = C::kQuant ? -INFINITY : top;
              if constexpr (C::kQuant) {
#pragma unroll
                for (int e = 0; e < 32; e += 4) {
                  const float4 l4 = *reinterpret_cast<const float4 *>(&sc_l[ss][hh * 32 + e]);
                  key = fmaxf(key, fmaf(__uint_as_float(rr[e]), rs, l4.x));
                  key = fmaxf(key, fmaf(__uint_as_float(rr[e + 1]), rs, l4.y));
                  key = fmaxf(key, fmaf(__uint_as_float(rr[e + 2]), rs, l4.z));
                  key = fmaxf(key, fmaf(__uint_as_float(rr[e + 3]), rs, l4.w));
                }
              }
              const float to = U::at(key, top);
              const bool mine = to > m_ref + U::kSlack;
              const float by = mine ? tree_pow2(m_ref - to) : 1.f;
              m_ref = mine ? to : m_ref;
              moved |= mine;
              alpha *= by;
              const uint64_t by2 = f2_pack(by, by);
#pragma unroll
              for (int e = 0; e < 4; ++e) acc[e] = f2_mul(acc[e], by2);
              if (hh > 0 && __any_sync(0xffffffffu, mine)) {
                tmem_st_wait();
#pragma unroll 1
                for (int k = 0; k < hh; ++k) {
                  tc_ld16(s_tm + 16 * k, pk);
                  tc_ld_wait16(pk);
#pragma unroll
                  for (int e = 0; e < 16; ++e) pk[e] = tc_scale2<KIND>(pk[e], by);
                  tc_st16(s_tm + 16 * k, pk);
                }
              }
            }
            // P, packed, over columns of S that are read already
            const float ref = m_ref == -INFINITY ? 0.f : m_ref;
            const uint64_t nm2 = f2_pack(-ref, -ref);
#pragma unroll
            for (int e = 0; e < 32; e += 4) {
              [[maybe_unused]] float4 v4;
              if constexpr (C::kQuant) v4 = *reinterpret_cast<const float4 *>(&sc_v[ss][hh * 32 + e]);
#pragma unroll
              for (int q = 0; q < 4; q += 2) {
                float x0, x1;
                f2_unpack(f2_fma(f2_pack(__uint_as_float(rr[e + q]), __uint_as_float(rr[e + q + 1])), rs2, nm2), x0, x1);
                uint64_t p2 = f2_pack(ex2(x0), ex2(x1));
                acc[(e + q) / 2 & 3] = f2_add(acc[(e + q) / 2 & 3], p2);
                if constexpr (C::kQuant) p2 = f2_mul(p2, q ? f2_pack(v4.z, v4.w) : f2_pack(v4.x, v4.y));
                float p0, p1;
                f2_unpack(p2, p0, p1);
                pk[(e + q) / 2] = KIND == kKvBf16 ? pack_bf16x2(p0, p1) : pack_f16x2(p0, p1);
              }
            }
            tc_st16(s_tm + 16 * hh, pk);
          }
          float a0, a1;
          f2_unpack(f2_add(f2_add(acc[0], acc[1]), f2_add(acc[2], acc[3])), a0, a1);
          sum = a0 + a1;
        };
        if (pos0 + kTcBN > prefix) rows_of_tile(std::true_type{});
        else rows_of_tile(std::false_type{});
        l = l * alpha + sum;
        // S was signalled after the group's product before had completed: O is stable here
        if (j > 0 && __any_sync(0xffffffffu, moved)) {
#pragma unroll 1
          for (int c = 0; c < D; c += 32) {
            uint32_t o[32];
            tmem_ld32(o_tm + t * 128 + c, o);
            tmem_ld_wait(o);
#pragma unroll
            for (int e = 0; e < 32; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * alpha);
            tmem_st32(o_tm + t * 128 + c, o);
          }
        }
        tmem_st_wait();
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) {
          mbar_arrive(smem_u32(&bar_pfull[t]));
          if (C::kQuant) mbar_arrive(smem_u32(&bar_scempty[ss]));
        }
      }
      // ---- the end of the segment
      if (ok && cnt > 0) ok = mbar_wait(smem_u32(&bar_odone[t]), (n - 1) & 1, abort_flag, P.err);
      ok = __all_sync(0xffffffffu, ok);
      if constexpr (!PAIR) {
        x_m[t][row] = m_ref;
        x_l[t][row] = l;
        named_sync(2, 256);
      }
      if (!ok) continue;
      tc_fence_after();
      // O_0 f0 + O_1 f1 over columns [c0, c1): PAIR: this group's rows; else both groups' parts of the same rows
      float f0, f1 = 0.f, M = m_ref, Ls = l;
      if constexpr (PAIR) {
        f0 = 1.f;
      } else {
        const float m0 = x_m[0][row], m1 = x_m[1][row];
        M = fmaxf(tree_top(m0, x_l[0][row]), tree_top(m1, x_l[1][row]));
        const float ref = M == -INFINITY ? 0.f : M;
        f0 = tree_pow2(m0 - ref);
        f1 = tree_pow2(m1 - ref);
        Ls = x_l[0][row] * f0 + x_l[1][row] * f1;
      }
      const bool whole = w.a == 0 && w.b == w.q.nt;
      const int slot = 2 * blockIdx.x + (w.a == 0 ? 1 : 0);
      if (whole) {
        const float inv = Ls == 0.f ? 0.f : 1.f / Ls;
        f0 *= inv;
        f1 *= inv;
      }
      const int h = w.j * P.g + grow % P.g;
      const int c0 = PAIR ? 0 : t * (D / 2), c1 = PAIR ? D : c0 + D / 2;
      if (live) {
#pragma unroll 1
        for (int col = c0; col < c1; col += 32) {
          uint32_t o[32];
          tmem_ld32(o_tm + (PAIR ? t * 128 : 0) + col, o);
          tmem_ld_wait(o);
#pragma unroll
          for (int e = 0; e < 32; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * f0);
          if (!PAIR && L > 1) {
            uint32_t o1[32];
            tmem_ld32(o_tm + 128 + col, o1);
            tmem_ld_wait(o1);
#pragma unroll
            for (int e = 0; e < 32; ++e) o[e] = __float_as_uint(fmaf(__uint_as_float(o1[e]), f1, __uint_as_float(o[e])));
          }
          if (have) {
            if (whole) {
              uint16_t *dst = static_cast<uint16_t *>(P.out) + (w.q.row0 + tk) * P.o_tok + h * P.o_head + col;
#pragma unroll
              for (int e = 0; e < 32; e += 8) {
                uint32_t y[4];
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                  const float a = __uint_as_float(o[e + 2 * q]), b = __uint_as_float(o[e + 2 * q + 1]);
                  y[q] = P.q_f16 ? pack_f16x2(a, b) : pack_bf16x2(a, b);
                }
                *reinterpret_cast<uint4 *>(dst + e) = make_uint4(y[0], y[1], y[2], y[3]);
              }
            } else {
              float *dst = P.part + ((int64_t)slot * C::BM + trow) * D + col;
#pragma unroll
              for (int e = 0; e < 32; e += 4)
                *reinterpret_cast<float4 *>(dst + e) = make_float4(__uint_as_float(o[e]), __uint_as_float(o[e + 1]),
                                                                   __uint_as_float(o[e + 2]), __uint_as_float(o[e + 3]));
            }
          }
          __syncwarp();  // the next load from tensor memory takes the warp together
        }
      }
      if (have && *(volatile int *)&bad_sh) {
        void *dst = whole ? static_cast<void *>(static_cast<uint16_t *>(P.out) + (w.q.row0 + tk) * P.o_tok + h * P.o_head)
                          : static_cast<void *>(P.part + ((int64_t)slot * C::BM + trow) * D);
        tc_fixup<KIND, D>(P, v_pool, w.s, w.j, w.q.row0, tk, w.q.len, w.q.n, w.a * kTcBN, w.b * kTcBN, c0, c1, dst,
                          whole ? P.q_f16 : -1);
      }
      if (have && (PAIR || t == 0)) {
        if (whole) {
          if (P.lse) P.lse[(int64_t)h * P.T + w.q.row0 + tk] = Ls == 0.f ? -INFINITY : (M + log2f(Ls)) * kLn2;
        } else {
          float *ml = P.part_ml + ((int64_t)slot * C::BM + trow) * 2;
          ml[0] = M;
          ml[1] = Ls;
        }
      }
      if (w.a == 0 && !whole && threadIdx.x == 0) {
        TreeDesc d = {};
        d.seq_row0 = w.q.row0;
        d.n = w.q.n;
        d.j = w.j;
        d.row_tile0 = rbase;
        d.last = tree_last_cta(share, at, w.q.nt);
        P.desc[blockIdx.x] = d;
      }
    }
  }
  __syncwarp();  // the roles' branches leave lanes apart; what follows takes whole warps
  tc_fence_before();
  __syncthreads();
  if (warp == kMma) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

}  // namespace fpk
