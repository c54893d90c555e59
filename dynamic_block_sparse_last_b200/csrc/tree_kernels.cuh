// tree_kernels.cuh -- attention of drafted tokens over the paged cache, for
// up to 32 query rows at a time (mma.sync), and the join of split sequences.
//
//   out_i = sum_p softmax_p(scale q_i . k_p) v_p
// over the cached tokens p that new token i sees: all of the prefix, and the
// new tokens that its mask names.
//
// Rows: the n new tokens of a sequence times the g query heads of one KV head
// share that head's K and V, so a row tile is 16 * MT of those n g rows (row r:
// token r / g, head r % g) and every K/V byte is read once per tile.
//
// Bound: memory.  A K/V byte serves 16 or 32 rows, 32-64 flops a byte over a
// bf16 cache, well below what mma.sync sustains; so K and V stream through a
// ring of TMA tiles (64 to 128 tokens) and each warp takes 16 or 32 tokens of a tile.
// With 16 or 32 rows a tcgen05 tile (128 rows at least) would be mostly padding, and
// its accumulators would have to come back through tensor memory.
//
// Work split: all (sequence, row tile, KV head) units of ceil(len / BN) tiles each
// are cut into shares of equal length, one per CTA, whatever the lengths are
// (tree_share); every CTA finds its share from the lengths on the device, so nothing
// is planned on the host.  A unit inside
// one share is finished there; the parts of the others go to the workspace (at
// most two per CTA) and k_tree_join adds them up in a fixed order.
//
// Measured (32 query heads, 8 KV heads of 128): 64 sequences of up to 16384 tokens,
// one new token each, over bf16 in 365 us, 6.4 TB/s (0.97 of the measured copy); over
// int8 in 235 us, 5.1 TB/s (250 to 256 us after seconds under load, as the clock falls):
// there a warp's chain of conversion, product, softmax and product is what two warps
// a scheduler do not hide (issue slots 49% busy).
//
// Operand order: a matrix product does not mind the order of its inner index,
// so K is taken in the order in which a thread's 16-byte shared-memory reads
// bring it (Q's registers follow), and V's columns likewise: no ldmatrix, no
// transposition through shared memory.  Quantised K and V are multiplied as
// their codes, which fp16 holds exactly; K's scale goes to the scores and V's
// to the probabilities.  bf16 queries over a quantised
// cache are brought to fp16 by a power of two per row, exactly (elements below
// 2^-14 of the row's largest lose bits from 2^-25 of it on).
//
// Units: a row's weights w_p = 2^(s_p - m) times V's scale (1 where there is none) and its sum of
// 2^(s_p - m) are taken in one unit 2^m, m a whole number.  It moves only when a weight
// of the row passes 2^(kLift + kSlack), and then so that the row's largest is at most
// 2^kLift; sum and O are rescaled exactly.  It is the row's own: what a row does not
// see, or sees without weight, whatever V row it has, moves nothing of it: a bound that
// takes a row's largest score with the largest of some tokens' scales only says when to
// look at the products themselves.  Parts are
// added up relative to the row's sum, not to their units, which V's scales may set
// far apart (tree_top).
//
// Rounding: the products take P (times V's scale) in 16 bits, bf16 over bf16 caches and
// fp16 elsewhere, off by at most 2^-8 or 2^-11 of each: as much again as
// out's own rounding has.  fp16 has that down to 2^-17 of the row's largest (of the same
// processor), and an absolute 2^-28 of that largest below it (kLift).  With many tokens these errors average out; where one token
// dominates a row they are common to its columns.  The sums are of the unrounded
// values: sums of the rounded ones would make a dominated row exact, but they would bring
// P's rounding into lse and double the bound of the others.
#pragma once

#include <type_traits>

#include "kv_kernels.cuh"
#include "ptx.cuh"

namespace fpk {

constexpr float kLn2 = 0.6931471805599453f;

struct TreeDesc {       // a unit split over several CTAs, written by the first of them
  int seq_row0, n, j;   // first row of q / out, new tokens, KV head (n = 0: no such unit)
  int row_tile0;        // first of its rows
  int last;             // the CTA that holds its last tile
  int pad[3];
};

struct TreeParams {
  const float *scale[2];
  const int *table, *kv_len, *cu;
  const unsigned long long *mask;
  const void *q;
  void *out;
  float *lse;
  float *part;     // [2 C][BM][D]
  float *part_ml;  // [2 C][BM][2]
  TreeDesc *desc;  // [C]
  int *err;
  int64_t q_tok, q_head, o_tok, o_head, pages;
  int max_pages, nseq, T, max_q, W, Hq, Hkv, g, page, page_shift, q_f16;
  float scale2;    // scale * log2(e)
};

// A sequence's share of the work.
struct TreeSeq {
  int row0, n, len, nt, mt;
};
__device__ __forceinline__ TreeSeq tree_seq(const TreeParams &P, int s, int BM, int BN, bool report) {
  TreeSeq q;
  q.row0 = P.cu[s];
  q.n = P.cu[s + 1] - q.row0;
  q.len = P.kv_len[s];
  q.nt = q.mt = 0;
  if (q.n == 0) return q;
  const bool ok = q.n > 0 && q.n <= P.max_q && q.row0 >= 0 && q.row0 <= P.T - q.n && q.len >= q.n &&
                  (int64_t)q.len <= ((int64_t)P.max_pages << P.page_shift);
  if (!ok) {
    if (report) atomicOr(P.err, kDevErrRange);
    q.n = 0;
    return q;
  }
  q.nt = (q.len + BN - 1) / BN;
  q.mt = (q.n * P.g + BM - 1) / BM;
  return q;
}

struct TreeShare {
  long long begin, end, chunk;   // tiles of this CTA (laid end to end); tiles per CTA
  long long rem;                 // its first tile's place among those of sequence s
  int s, aligned;
};

// This CTA's share, found by all of its threads together.  Tiles are laid end to
// end and cut evenly; but starting a second unit costs a CTA about as much as a few
// tiles, so where a share of up to kTreeSlack tiles more gives every unit CTAs of its
// own (ceil(nt / chunk) of them, no more than there are in all), units are cut by
// themselves.
constexpr int kTreeSlack = 4;
template <int NT>
__device__ __forceinline__ void tree_share(const TreeParams &P, int BM, int BN, TreeShare *sh, long long *warp_sum) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int per = (P.nseq + NT - 1) / NT;
  const int s0 = min(tid * per, P.nseq), s1 = min(s0 + per, P.nseq);
  __shared__ unsigned long long cand[(kTreeSlack + 2) / 2][NT / 32];
  long long own = 0;
  for (int s = s0; s < s1; ++s) {
    const TreeSeq q = tree_seq(P, s, BM, BN, blockIdx.x == 0);
    own += (long long)q.nt * q.mt * P.Hkv;
  }
  long long inc = own;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long long v = __shfl_up_sync(0xffffffffu, inc, o);
    if (lane >= o) inc += v;
  }
  if (lane == 31) warp_sum[warp] = inc;
  __syncthreads();
  long long before = 0, total = 0;
  for (int w = 0; w < NT / 32; ++w) {
    if (w < warp) before += warp_sum[w];
    total += warp_sum[w];
  }
  inc += before;
  long long chunk = (total + gridDim.x - 1) / gridDim.x;
  long long at = inc - own, me = (long long)blockIdx.x * chunk;
  bool aligned = false;
  // with one tile a CTA the units are apart already; with more units than CTAs they cannot be
  if (chunk > 1 && (long long)P.nseq * P.Hkv <= gridDim.x) {
    // the CTAs that each longer share needs, capped so that two sums fit one word
    constexpr int NC = kTreeSlack + 1, NW = (NC + 1) / 2;
    unsigned long long want[NW], all[NW], upto[NW];
#pragma unroll
    for (int w = 0; w < NW; ++w) want[w] = 0;
    for (int s = s0; s < s1; ++s) {
      const TreeSeq q = tree_seq(P, s, BM, BN, false);
#pragma unroll
      for (int k = 0; k < NC; ++k)
        want[k / 2] += min((q.nt + chunk + k - 1) / (chunk + k) * q.mt * P.Hkv, 1ll << 20) << (32 * (k & 1));
    }
#pragma unroll
    for (int w = 0; w < NW; ++w) upto[w] = want[w];
#pragma unroll
    for (int o = 1; o < 32; o <<= 1)
#pragma unroll
      for (int w = 0; w < NW; ++w) {
        const unsigned long long v = __shfl_up_sync(0xffffffffu, upto[w], o);
        if (lane >= o) upto[w] += v;
      }
    if (lane == 31) {
#pragma unroll
      for (int w = 0; w < NW; ++w) cand[w][warp] = upto[w];
    }
    __syncthreads();
#pragma unroll
    for (int w = 0; w < NW; ++w) {
      all[w] = 0;
      for (int k = 0; k < NT / 32; ++k) {
        if (k < warp) upto[w] += cand[w][k];
        all[w] += cand[w][k];
      }
    }
#pragma unroll
    for (int k = 0; k < NC; ++k) {
      const int sh32 = 32 * (k & 1);
      if (!aligned && (uint32_t)(all[k / 2] >> sh32) <= gridDim.x) {
        aligned = true;
        chunk += k;
        own = (uint32_t)(want[k / 2] >> sh32);
        at = (uint32_t)(upto[k / 2] >> sh32) - own;
        total = (uint32_t)(all[k / 2] >> sh32);
        me = blockIdx.x;
      }
    }
  }
  if (tid == 0) {
    sh->chunk = chunk;
    sh->aligned = aligned;
    sh->begin = aligned ? 0 : min(me, total);
    sh->end = aligned ? 0 : min(me + chunk, total);
  }
  __syncthreads();
  if (me < total && me >= at && me < at + own) {
    for (int s = s0; s < s1; ++s) {
      const TreeSeq q = tree_seq(P, s, BM, BN, false);
      const long long cut = q.nt > 0 ? (q.nt + chunk - 1) / chunk : 0;
      const long long c = (aligned ? cut : q.nt) * q.mt * P.Hkv;
      if (me < at + c) {
        sh->s = s;
        sh->rem = me - at;
        if (aligned) {
          const long long u = (me - at) / cut, part = (me - at) - u * cut;
          sh->rem = u * q.nt + part * chunk;
          sh->end = min(chunk, q.nt - part * chunk);
        }
        break;
      }
      at += c;
    }
  }
  __syncthreads();
}

// The CTA with the last tile of a unit of nt tiles that begins, at tile `at` of all, in this one.
__device__ __forceinline__ int tree_last_cta(const TreeShare &sh, long long at, int nt) {
  return sh.aligned ? (int)(blockIdx.x + (nt - 1) / sh.chunk) : (int)((at + nt - 1) / sh.chunk);
}

// The segments of a share: consecutive tiles of one unit.
struct TreeWalk {
  TreeSeq q;
  int s, m, j, a, b;    // sequence, row tile, KV head, tiles [a, b) of the unit
  int left;             // tiles of the share from this segment on (a share is below 2^31: a sequence's tokens are)
  __device__ __forceinline__ bool start(const TreeParams &P, const TreeShare &sh, int BM, int BN) {
    left = (int)min(sh.end - sh.begin, 0x7fffffffll);
    if (left <= 0) return false;
    s = sh.s;
    q = tree_seq(P, s, BM, BN, false);
    const long long u = sh.rem / q.nt;
    a = (int)(sh.rem - u * q.nt);
    m = (int)(u / P.Hkv);
    j = (int)(u - (long long)m * P.Hkv);
    b = min(q.nt, a + left);
    return true;
  }
  __device__ __forceinline__ bool next(const TreeParams &P, int BM, int BN) {
    left -= b - a;
    if (left <= 0) return false;
    if (++j == P.Hkv) {
      j = 0;
      if (++m == q.mt) {
        m = 0;
        do {
          q = tree_seq(P, ++s, BM, BN, false);
        } while (q.nt == 0);  // left > 0: another sequence has tiles
      }
    }
    a = 0;
    b = min(q.nt, left);
    return true;
  }
};

// Whether row token i of the sequence sees new token jj (0 <= jj < n).
__device__ __forceinline__ bool tree_sees(const TreeParams &P, const TreeSeq &q, int i, int jj) {
  if (!P.mask) return jj <= i;
  return (P.mask[(int64_t)(q.row0 + i) * P.W + (jj >> 6)] >> (jj & 63)) & 1ull;
}

// One cached value of V as fp32 (the rare path of non-finite drafted values).
template <int KIND, int D>
__device__ __forceinline__ float tree_v_value(const TreeParams &P, const void *pool, int s, int j, int pos, int col) {
  const int pg = P.table[(int64_t)s * P.max_pages + (pos >> P.page_shift)];
  if (pg < 0 || pg >= P.pages) return 0.f;
  const int64_t row = (((int64_t)pg * P.Hkv + j) << P.page_shift) + (pos & (P.page - 1));
  if constexpr (KvCode<KIND>::kQuant) {
    float x[4];
    kv_values4<KIND>(static_cast<const uint8_t *>(pool)[row * D + col], x);
    return x[0] * P.scale[1][row];
  } else {
    using C = typename std::conditional<KIND == kKvBf16, __nv_bfloat16, __half>::type;
    return rope_to_float<C>(static_cast<const C *>(pool)[row * D + col]);
  }
}

__device__ __forceinline__ uint32_t prmt(uint32_t a, uint32_t b, uint32_t sel) {
  uint32_t r;
  asm("prmt.b32 %0, %1, %2, %3;" : "=r"(r) : "r"(a), "r"(b), "r"(sel));
  return r;
}
__device__ __forceinline__ uint32_t hsub2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("sub.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}
__device__ __forceinline__ uint32_t pack_f16x2(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}

// Four codes as two fp16 pairs.  int8 (with the sign bit flipped beforehand,
// so b + 128): as the low byte of 1024 + u in fp16, minus 1152: exact.
template <int KIND>
__device__ __forceinline__ void tree_codes4(uint32_t w, uint32_t &lo, uint32_t &hi) {
  if constexpr (KIND == kKvInt8) {
    lo = hsub2(prmt(w, 0x64646464u, 0x4140u), 0x64806480u);
    hi = hsub2(prmt(w, 0x64646464u, 0x4342u), 0x64806480u);
  } else {
    asm("{\n\t.reg .b16 l, h;\n\tmov.b32 {l, h}, %2;\n\t"
        "cvt.rn.f16x2.e4m3x2 %0, l;\n\tcvt.rn.f16x2.e4m3x2 %1, h;\n\t}"
        : "=r"(lo), "=r"(hi)
        : "r"(w));
  }
}

template <int KIND>
__device__ __forceinline__ void tree_mma(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  if constexpr (KIND == kKvBf16)
    asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                 : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
                 : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
  else
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                 : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
                 : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// 16 bytes of one cached V row with its non-finite values set to 0 (they are
// added for the rows that see them at the end); *bad is raised when there were any.
template <int KIND>
__device__ __forceinline__ uint32_t tree_clean(uint32_t w, int &bad) {
  if constexpr (KIND == kKvInt8) {
    return w;
  } else if constexpr (KIND == kKvE4m3) {
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (((w >> (8 * i)) & 0x7fu) == 0x7fu) {
        w &= ~(0xffu << (8 * i));
        bad = 1;
      }
    return w;
  } else {
    constexpr uint32_t E = KIND == kKvBf16 ? 0x7f80u : 0x7c00u;
    if ((w & E) == E) {
      w &= 0xffff0000u;
      bad = 1;
    }
    if (((w >> 16) & E) == E) {
      w &= 0xffffu;
      bad = 1;
    }
    return w;
  }
}

__device__ __forceinline__ float pow2i(int e) { return __int_as_float((127 + e) << 23); }  // -126 <= e <= 127
// 2^d of a whole number d <= 127, 0 below fp32's normal range.
__device__ __forceinline__ float tree_pow2(float d) { return d < -126.f ? 0.f : pow2i((int)d); }

// What a row's weights are taken in (see Units above).
template <int KIND>
struct TreeUnit {
  // fp16: up to 2^15 of its 2^15.99, and the largest weight above 2^3 when the unit is set, so that
  // 2^-17 of it is still a normal number and 2^-28 of it half of the last step.  A unit that moves
  // costs time, mostly above 32 rows: 64 drafted tokens over 128K in e4m3 take 228 us with 0 + 14,
  // 243 with 4 + 11, 253 with 9 + 6.
  // bf16: up to 2^-24, so that sums over 2^24 tokens do not overflow whatever V is, and 2^-86 of the
  // largest weight is still a normal number; s - m near 40 is off by 2^-19, far below bf16's steps.
  static constexpr float kLift = KIND == kKvBf16 ? -40.f : 4.f;
  static constexpr float kSlack = KIND == kKvBf16 ? 16.f : 11.f;
  // Over V rows of next to nothing 2^(s - m) stays below 2^(kFar + kLift + kSlack), and its sum over 2^30
  // tokens below 2^127; V scales from 2^-kFar on set their unit themselves.
  static constexpr float kFar = 82.f;
  // the unit of a row whose largest product is 2^key and whose largest score is top
  static __device__ __forceinline__ float at(float key, float top) { return ceilf(fmaxf(key, top - kFar)) - kLift; }
  // log2 of the largest of some V scales, as the bound takes it
  static __device__ __forceinline__ float bound(float lv) { return fmaxf(lv, -kFar) - (kLift + kSlack); }
};

// The power of two (log2) below the sum l of a row in units of 2^m; -inf for 0.
__device__ __forceinline__ float tree_top(float m, float l) {
  return l == 0.f ? -INFINITY : m + (float)((int)((__float_as_uint(l) >> 23) & 0xffu) - 127);
}
// What a row's products are multiplied by, above 0 and finite whatever the softmax scale and the
// row's own power of two are, so that a hidden score stays -inf and a row of zeros (its power is
// 2^-126) scores 0.
__device__ __forceinline__ float tree_row_scale(float power, float scale2) {
  return fminf(fmaxf(power * scale2, 1.1754944e-38f), 3.4028235e38f);
}
// The power of two by which a bf16 query row of largest magnitude mx is divided for fp16, which
// leaves it below 4; 0 for a row that is not finite.
__device__ __forceinline__ int tree_q_exp(float mx) {
  const int e = (int)(__float_as_uint(mx) >> 23) - 127;  // mx in [2^e, 2^(e+1))
  return e > 127 ? 0 : min(max(e, -126), 126);
}
// log2 of a V scale; -inf for one that sets no unit (0, or not finite).
__device__ __forceinline__ float tree_log2(float v) { return v > 0.f && v < INFINITY ? __log2f(v) : -INFINITY; }

// A barrier of some warps of the block; each takes part as a whole, so its lanes meet first.
__device__ __forceinline__ void named_sync(int id, int threads) {
  __syncwarp();
  asm volatile("bar.sync %0, %1;" ::"r"(id), "r"(threads) : "memory");
}
__device__ __forceinline__ void bulk_load(uint32_t dst, const void *src, uint32_t bytes, uint32_t bar) {
  asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(dst),
               "l"(src), "r"(bytes), "r"(bar)
               : "memory");
}
__device__ __forceinline__ uint4 lds128(uint32_t a) {
  uint4 v;
  asm volatile("ld.shared.v4.b32 {%0,%1,%2,%3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(a));
  return v;
}
__device__ __forceinline__ uint2 lds64(uint32_t a) {
  uint2 v;
  asm volatile("ld.shared.v2.b32 {%0,%1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(a));
  return v;
}

template <int KIND, int D, int MT>
struct TreeCfg {
  static constexpr bool kQuant = KvCode<KIND>::kQuant;
  static constexpr int BM = 16 * MT;
  // Two CTAs per SM of four warps, up to 200 registers a thread; 32 rows of 128-wide
  // heads, whose O alone is 128 registers: one of eight warps.  Where there is room a
  // warp takes 32 tokens at a time (quantised caches, where its work per byte is
  // larger, and 64-wide heads): two independent halves hide each other's latency.
  static constexpr bool kBig = MT == 2 && D == 128;
  static constexpr int kWarps = kBig ? 8 : 4;
  static constexpr int kCtas = kBig ? 1 : 2;
  static constexpr int kThreads = (kBig ? kWarps + 4 : kWarps + 1) * 32;  // the producer; kBig: in a warpgroup of its own
  // Registers when kBig: the block starts with 168 a thread (384 threads), and 2 x 128 x 216 + 128 x 56 = 62464 <= 384 x 168.
  static constexpr int kRegs = 216, kRegsTma = 56;
  static constexpr int TOK = (kQuant && MT == 1) || D == 64 ? 32 : 16;  // tokens of a warp in a tile
  // Q in registers, except where they are short: read again for every 32 tokens then
  // (int8 decode batch, 64 sequences of up to 16384 tokens: 231 us against 243)
  static constexpr bool kQReg = MT == 1 && !(kQuant && D == 128);
  static constexpr int BN = kWarps * TOK;                 // tokens of a tile
  static constexpr int RB = D * KvCode<KIND>::kBytes;     // bytes of a cached row
  static constexpr int kBoxB = RB < 128 ? RB : 128;       // bytes of a box row
  static constexpr int kBoxes = RB / kBoxB;
  static constexpr int E = 16 / KvCode<KIND>::kBytes;     // elements of 16 bytes
  static constexpr int kSteps = D / 16;
  static constexpr int VE = (kQuant && D == 128) ? 16 : 8;  // V columns of a thread's read
  static constexpr int kTile = BN * RB;                   // K (or V) bytes of a tile
  static constexpr int kStage = 2 * kTile;
  static constexpr int kStageAll = kStage + (kQuant ? 2 * BN * 4 : 0);  // with the scales
  // as many as leave room for Q, obuf and the other CTA (227 KB an SM), 6 at most
  static constexpr int kFit = (kBig ? 200000 : 99000) / kStageAll, kStages = kFit > 6 ? 6 : kFit;
  static constexpr int kScaleOff = kStages * kStage;      // [stage][K, V][BN] fp32
  static constexpr int kQOff = kScaleOff + (kQuant ? kStages * 2 * BN * 4 : 0);  // [MT][steps][32] uint4
  static constexpr int kLd = D + 4;                       // row pitch of obuf (fp32)
  static constexpr int kOOff = kQOff + MT * kSteps * 512;
  static constexpr int kSmem = kOOff + BM * kLd * 4 + 1024;
};

// Shared address of the 16-byte chunk `ch` of row r of a tile (TMA swizzle:
// 128-byte rows by row mod 8, 64-byte rows by row / 2 mod 4; 256-byte rows are
// two boxes of 128).
template <typename C>
__device__ __forceinline__ uint32_t tree_chunk(uint32_t tile, int r, int ch) {
  if constexpr (C::kBoxB == 128)
    return tile + (ch >> 3) * (C::BN * 128) + r * 128 + (((ch & 7) ^ (r & 7)) << 4);
  else
    return tile + r * 64 + ((ch ^ ((r >> 1) & 3)) << 4);
}

template <int KIND, int D, int MT>
__global__ void __launch_bounds__((TreeCfg<KIND, D, MT>::kThreads), (TreeCfg<KIND, D, MT>::kCtas))
    k_tree(const __grid_constant__ CUtensorMap tm_k, const __grid_constant__ CUtensorMap tm_v,
           const __grid_constant__ TreeParams P, const void *v_pool) {
  using C = TreeCfg<KIND, D, MT>;
  extern __shared__ uint8_t smem_raw[];
  __shared__ __align__(8) uint64_t bar_full[C::kStages], bar_empty[C::kStages];
  __shared__ long long warp_sum[C::kThreads / 32];
  __shared__ TreeShare share;
  __shared__ float red_m[C::kWarps][C::BM], red_l[C::kWarps][C::BM], row_scale[C::BM], fin_m[C::BM], fin_l[C::BM];
  __shared__ int abort_sh, bad_sh;

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t base = (smem_u32(smem_raw) + 1023u) & ~1023u;
  if (threadIdx.x == 0) {
    abort_sh = 0;
    bad_sh = 0;
    for (int i = 0; i < C::kStages; ++i) {
      mbar_init(smem_u32(&bar_full[i]), 1);
      mbar_init(smem_u32(&bar_empty[i]), C::kWarps);
    }
    fence_mbar_init();
  }
  tree_share<C::kThreads>(P, C::BM, C::BN, &share, warp_sum);
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  volatile int *abort_flag = &abort_sh;
  TreeWalk w;
  bool more = w.start(P, share, C::BM, C::BN);

  if (warp >= C::kWarps) {
    // ------------------------------------------------------------ producer
    if constexpr (C::kBig) asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(C::kRegsTma));
    if (warp > C::kWarps) return;
    // A tile is BN / min(page, 64) pieces, each of one page; lane i moves piece i.
    const int piece = min(P.page, 64), pieces = C::BN / piece;
    if (lane == 0) {
      tma_prefetch_map(&tm_k);
      tma_prefetch_map(&tm_v);
    }
    int u = 0;
    bool ok = true;
    for (; more && ok; more = w.next(P, C::BM, C::BN)) {
      const int *tab = P.table + (int64_t)w.s * P.max_pages;
      int pg = 0;
      const int p0 = w.a * C::BN + lane * piece;
      if (lane < pieces && p0 < w.q.len) pg = tab[p0 >> P.page_shift];
      for (int t = w.a; t < w.b; ++t, ++u) {
        const int pos = t * C::BN + lane * piece;
        const bool mine = lane < pieces && pos < w.q.len;
        const int now = pg;
        const int nx = pos + C::BN;  // the next tile's page, ahead of its use
        if (t + 1 < w.b && lane < pieces && nx < w.q.len) pg = tab[nx >> P.page_shift];
        const int st = u % C::kStages;
        if (u >= C::kStages) ok = mbar_wait(smem_u32(&bar_empty[st]), ((u / C::kStages) - 1) & 1, abort_flag, P.err);
        if (!__all_sync(0xffffffffu, ok)) {
          ok = false;
          break;
        }
        const int n = __popc(__ballot_sync(0xffffffffu, mine));
        const uint32_t bar = smem_u32(&bar_full[st]);
        if (lane == 0) mbar_expect_tx(bar, n * piece * (2 * C::RB + (C::kQuant ? 8 : 0)));
        __syncwarp();
        if (mine) {
          int id = now;
          if (id < 0 || id >= P.pages) {
            id = 0;
            atomicOr(P.err, kDevErrRange);
          }
          const int row = ((id * P.Hkv + w.j) << P.page_shift) + (pos & (P.page - 1));
          const uint32_t dst = base + st * C::kStage + lane * piece * C::kBoxB;
#pragma unroll
          for (int x = 0; x < C::kBoxes; ++x) {
            tma_load_2d(dst + x * C::BN * 128, &tm_k, x * 128, row, bar);
            tma_load_2d(dst + C::kTile + x * C::BN * 128, &tm_v, x * 128, row, bar);
          }
          if constexpr (C::kQuant) {
            const uint32_t sd = base + C::kScaleOff + st * 2 * C::BN * 4 + lane * piece * 4;
            bulk_load(sd, P.scale[0] + row, piece * 4, bar);
            bulk_load(sd + C::BN * 4, P.scale[1] + row, piece * 4, bar);
          }
        }
      }
    }
    // a CTA may not end with copies in flight: the consumers wait for every
    // tile; after an abandoned wait nothing reads them, so wait here
    if (!ok)
      for (int i = 0; i < C::kStages; ++i)
        if (u - 1 - i >= 0) {
          const int v = u - 1 - i;
          const unsigned long long t0 = globaltimer();
          while (!mbar_try_wait(smem_u32(&bar_full[v % C::kStages]), (v / C::kStages) & 1) &&
                 globaltimer() - t0 < kWaitLimitNs) {
          }
        }
    return;
  }

  // -------------------------------------------------------------- consumers
  if constexpr (C::kBig) asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(C::kRegs));
  const int q4 = lane >> 2, c4 = lane & 3;
  const uint32_t qbase = base + C::kQOff;
  float *obuf = reinterpret_cast<float *>(smem_raw + (base - smem_u32(smem_raw)) + C::kOOff);
  constexpr int NC = C::kWarps * 32;
  int u = 0;
  if (threadIdx.x == 0) P.desc[blockIdx.x].n = 0;
  long long at = share.begin;  // tile index of the segment's first tile
  for (; more; at += w.b - w.a, more = w.next(P, C::BM, C::BN)) {
    const int prefix = w.q.len - w.q.n, rbase = w.m * C::BM, R = min(C::BM, w.q.n * P.g - rbase);
    // Q fragments: a warp takes a row, a lane 4 neighbouring elements, which are one
    // thread's (a0, a2) or (a1, a3) of one step; a warp's rows are under way at once
    constexpr int RW = C::BM / C::kWarps;
    long long off = -1;  // of row warp + lane * kWarps
    if (lane < RW && warp + lane * C::kWarps < R) {
      const int gr = rbase + warp + lane * C::kWarps, i = gr / P.g;
      off = (w.q.row0 + i) * P.q_tok + (w.j * P.g + gr - i * P.g) * P.q_head;
    }
    uint2 qx[RW];
#pragma unroll
    for (int k = 0; k < RW; ++k) {
      const long long o = __shfl_sync(0xffffffffu, off, k);
      qx[k] = make_uint2(0u, 0u);
      if (o >= 0 && lane < D / 4) qx[k] = *reinterpret_cast<const uint2 *>(static_cast<const uint16_t *>(P.q) + o + 4 * lane);
    }
#pragma unroll
    for (int k = 0; k < RW; ++k) {
      const int r = warp + k * C::kWarps;
      uint32_t lo = qx[k].x, hi = qx[k].y;
      float fac = 1.f;
      if (C::kQuant && !P.q_f16) {
        float x[4] = {__uint_as_float(lo << 16), __uint_as_float(lo & 0xffff0000u), __uint_as_float(hi << 16),
                      __uint_as_float(hi & 0xffff0000u)};
        float mx = fmaxf(fmaxf(fabsf(x[0]), fabsf(x[1])), fmaxf(fabsf(x[2]), fabsf(x[3])));
        mx = redux_max_f32(mx);
        const int e = tree_q_exp(mx);
        fac = pow2i(e);
        const float inv = pow2i(-e);
        lo = pack_f16x2(x[0] * inv, x[1] * inv);
        hi = pack_f16x2(x[2] * inv, x[3] * inv);
      }
      if (lane < D / 4) {
        const int chunk = 4 * lane / C::E, jj = (4 * lane % C::E) / 4, step = (chunk >> 2) * (C::E / 4) + jj;
        const int dl = (r & 7) * 4 + (chunk & 3);
        const uint32_t dst = qbase + (((r >> 4) * C::kSteps + step) * 32 + dl) * 16 + ((r >> 3) & 1) * 4;
        asm volatile("st.shared.b32 [%0], %1;\n\tst.shared.b32 [%0+8], %2;" ::"r"(dst), "r"(lo), "r"(hi) : "memory");
      }
      if (lane == 0) row_scale[r] = tree_row_scale(fac, P.scale2);
    }
    named_sync(1, NC);
    uint32_t qf[C::kQReg ? C::kSteps : 1][4];
    if constexpr (C::kQReg) {
#pragma unroll
      for (int k = 0; k < C::kSteps; ++k) {
        const uint4 x = lds128(qbase + (k * 32 + lane) * 16);
        qf[k][0] = x.x; qf[k][1] = x.y; qf[k][2] = x.z; qf[k][3] = x.w;
      }
    }
    float rs[MT][2];
#pragma unroll
    for (int mt = 0; mt < MT; ++mt) {
      rs[mt][0] = row_scale[16 * mt + q4];
      rs[mt][1] = row_scale[16 * mt + 8 + q4];
    }
    float o[MT][D / 8][4];
    float m[MT][2], l[MT][2];
#pragma unroll
    for (int mt = 0; mt < MT; ++mt) {
#pragma unroll
      for (int i = 0; i < D / 8; ++i)
#pragma unroll
        for (int e = 0; e < 4; ++e) o[mt][i][e] = 0.f;
      m[mt][0] = m[mt][1] = -INFINITY;
      l[mt][0] = l[mt][1] = 0.f;
    }
    int bad = 0;
    for (int t = w.a; t < w.b; ++t, ++u) {
      const int st = u % C::kStages;
      // after an abandoned wait the warps still walk to the end together (the
      // barriers below have no time limit of their own); the results are lost
      if (!__all_sync(0xffffffffu, mbar_wait(smem_u32(&bar_full[st]), (u / C::kStages) & 1, abort_flag, P.err))) break;
      const uint32_t kt = base + st * C::kStage, vt = kt + C::kTile;
      constexpr int NT = C::TOK / 8, NB = C::TOK / 16;  // 8-token tiles of S, 16-token steps of P V
      const int key0 = warp * C::TOK;
      const int pos0 = t * C::BN + key0;
      // compiled once for tokens that every row sees and once for the others
      auto step = [&](auto tail_tag) __attribute__((always_inline)) {
        constexpr bool tail = decltype(tail_tag)::value;
        // ---- scores
        float s[MT][NT][4];
#pragma unroll
        for (int mt = 0; mt < MT; ++mt)
#pragma unroll
          for (int i = 0; i < NT; ++i)
#pragma unroll
            for (int e = 0; e < 4; ++e) s[mt][i][e] = 0.f;
#pragma unroll
        for (int h = 0; h < C::RB / 64; ++h) {
          uint32_t kw[NT][4];
#pragma unroll
          for (int i = 0; i < NT; ++i) {
            const uint4 x = lds128(tree_chunk<C>(kt, key0 + 8 * i + q4, c4 + 4 * h));
            kw[i][0] = x.x; kw[i][1] = x.y; kw[i][2] = x.z; kw[i][3] = x.w;
          }
#pragma unroll
          for (int jj = 0; jj < C::E / 4; ++jj) {
            const int step = h * (C::E / 4) + jj;
            uint32_t b[NT][2];
#pragma unroll
            for (int i = 0; i < NT; ++i) {
              if constexpr (C::kQuant) {
                tree_codes4<KIND>(KIND == kKvInt8 ? kw[i][jj] ^ 0x80808080u : kw[i][jj], b[i][0], b[i][1]);
              } else {
                b[i][0] = kw[i][2 * jj];
                b[i][1] = kw[i][2 * jj + 1];
              }
            }
#pragma unroll
            for (int mt = 0; mt < MT; ++mt) {
              uint32_t a[4];
              if constexpr (C::kQReg) {
#pragma unroll
                for (int e = 0; e < 4; ++e) a[e] = qf[step][e];
              } else {
                const uint4 x = lds128(qbase + ((mt * C::kSteps + step) * 32 + lane) * 16);
                a[0] = x.x; a[1] = x.y; a[2] = x.z; a[3] = x.w;
              }
#pragma unroll
              for (int i = 0; i < NT; ++i) tree_mma<KIND>(s[mt][i], a, b[i][0], b[i][1]);
            }
          }
        }
        // ---- scales and masks; a thread has tokens 8i + 2c, 8i + 2c + 1 of rows q, q + 8
        [[maybe_unused]] float vs[2 * NT];
        [[maybe_unused]] const uint32_t sc = base + C::kScaleOff + st * 2 * C::BN * 4 + (key0 + 2 * c4) * 4;
        if constexpr (C::kQuant) {
#pragma unroll
          for (int i = 0; i < NT; ++i) {
            const uint2 k = lds64(sc + 32 * i);
#pragma unroll
            for (int mt = 0; mt < MT; ++mt)
#pragma unroll
              for (int e = 0; e < 4; ++e) s[mt][i][e] *= __uint_as_float(e & 1 ? k.y : k.x) * rs[mt][e >> 1];
            const uint2 v = lds64(sc + C::BN * 4 + 32 * i);
            vs[2 * i] = __uint_as_float(v.x);
            vs[2 * i + 1] = __uint_as_float(v.y);
          }
        } else {
#pragma unroll
          for (int mt = 0; mt < MT; ++mt)
#pragma unroll
            for (int i = 0; i < NT; ++i)
#pragma unroll
              for (int e = 0; e < 4; ++e) s[mt][i][e] *= rs[mt][e >> 1];
        }
        [[maybe_unused]] uint32_t hide = 0;  // bit ((mt * NT + i) * 4 + e): not visible
        if constexpr (tail) {
#pragma unroll
          for (int mt = 0; mt < MT; ++mt)
#pragma unroll
            for (int hh = 0; hh < 2; ++hh) {
              const int i = min((rbase + 16 * mt + 8 * hh + q4) / P.g, w.q.n - 1);
#pragma unroll
              for (int k = 0; k < 2 * NT; ++k) {
                const int pos = pos0 + 8 * (k >> 1) + 2 * c4 + (k & 1), e = 2 * hh + (k & 1);
                const bool vis = pos < prefix || (pos < w.q.len && tree_sees(P, w.q, i, pos - prefix));
                if (!vis) {
                  s[mt][k >> 1][e] = -INFINITY;
                  hide |= 1u << ((mt * NT + (k >> 1)) * 4 + e);
                }
              }
            }
          if constexpr (C::kQuant) {
#pragma unroll
            for (int k = 0; k < 2 * NT; ++k)
              if (pos0 + 8 * (k >> 1) + 2 * c4 + (k & 1) >= w.q.len) vs[k] = 0.f;
          }
        }
        // ---- weights in the rows' units.  In the common case no thread's values ask for
        // more than a vote; only then do the four lanes of a row agree on its unit.
        using U = TreeUnit<KIND>;
        float lim = -(U::kLift + U::kSlack);
        if constexpr (C::kQuant) {
          float vmx = vs[0];
#pragma unroll
          for (int k = 1; k < 2 * NT; ++k) vmx = fmaxf(vmx, vs[k]);
          lim = U::bound(__log2f(vmx));
        }
        float mxl[MT][2];
        bool ask = false;
#pragma unroll
        for (int mt = 0; mt < MT; ++mt)
#pragma unroll
          for (int hh = 0; hh < 2; ++hh) {
            float mx = fmaxf(s[mt][0][2 * hh], s[mt][0][2 * hh + 1]);
#pragma unroll
            for (int i = 1; i < NT; ++i) mx = fmaxf(mx, fmaxf(s[mt][i][2 * hh], s[mt][i][2 * hh + 1]));
            mxl[mt][hh] = mx;
            ask |= mx + lim > m[mt][hh];
          }
        if (__any_sync(0xffffffffu, ask)) {
          [[maybe_unused]] float lv[2 * NT];
          if constexpr (C::kQuant) {
#pragma unroll
            for (int k = 0; k < 2 * NT; ++k) lv[k] = tree_log2(vs[k]);
          }
#pragma unroll
          for (int mt = 0; mt < MT; ++mt) {
            float al[2];
#pragma unroll
            for (int hh = 0; hh < 2; ++hh) {
              float top = mxl[mt][hh], key = C::kQuant ? -INFINITY : top;
              if constexpr (C::kQuant) {
#pragma unroll
                for (int k = 0; k < 2 * NT; ++k) key = fmaxf(key, s[mt][k >> 1][2 * hh + (k & 1)] + lv[k]);
              }
#pragma unroll
              for (int x = 1; x < 4; x <<= 1) {
                top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, x));
                key = fmaxf(key, __shfl_xor_sync(0xffffffffu, key, x));
              }
              const float to = U::at(key, top);
              al[hh] = 1.f;
              if (to > m[mt][hh] + U::kSlack) {
                al[hh] = tree_pow2(m[mt][hh] - to);
                m[mt][hh] = to;
              }
              l[mt][hh] *= al[hh];
            }
#pragma unroll
            for (int i = 0; i < D / 8; ++i)
#pragma unroll
              for (int e = 0; e < 4; ++e) o[mt][i][e] *= al[e >> 1];
          }
        }
        uint32_t pa[MT][NB][4];
#pragma unroll
        for (int mt = 0; mt < MT; ++mt)
#pragma unroll
          for (int hh = 0; hh < 2; ++hh) {
            const float ref = m[mt][hh] == -INFINITY ? 0.f : m[mt][hh];
            float sum = 0.f;
#pragma unroll
            for (int i = 0; i < NT; ++i) {
              float p0 = ex2(s[mt][i][2 * hh] - ref), p1 = ex2(s[mt][i][2 * hh + 1] - ref);
              sum += p0 + p1;
              if constexpr (C::kQuant) {
                p0 *= vs[2 * i];
                p1 *= vs[2 * i + 1];
                if constexpr (tail) {  // a hidden token's scale may be a NaN
                  if ((hide >> ((mt * NT + i) * 4 + 2 * hh)) & 1u) p0 = 0.f;
                  if ((hide >> ((mt * NT + i) * 4 + 2 * hh + 1)) & 1u) p1 = 0.f;
                }
              }
              pa[mt][i >> 1][2 * (i & 1) + hh] = KIND == kKvBf16 ? pack_bf16x2(p0, p1) : pack_f16x2(p0, p1);
            }
            l[mt][hh] += sum;
          }
        // ---- O += P V
#pragma unroll
        for (int kb = 0; kb < NB; ++kb)
#pragma unroll
          for (int x = 0; x < C::kBoxes; ++x) {
            constexpr int VW = C::VE * KvCode<KIND>::kBytes / 4;
            uint32_t vw[4][VW];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const int r = key0 + 16 * kb + 8 * (e >> 1) + 2 * c4 + (e & 1);
              if constexpr (VW == 4) {
                const uint4 y = lds128(tree_chunk<C>(vt, r, q4 + 8 * x));
                vw[e][0] = y.x; vw[e][1] = y.y; vw[e][2] = y.z; vw[e][3] = y.w;
              } else {
                const uint2 y = lds64(tree_chunk<C>(vt, r, q4 >> 1) + (q4 & 1) * 8);
                vw[e][0] = y.x; vw[e][1] = y.y;
              }
            }
            if constexpr (tail) {
#pragma unroll
              for (int e = 0; e < 4; ++e) {
                const int pos = pos0 + 16 * kb + 8 * (e >> 1) + 2 * c4 + (e & 1);
#pragma unroll
                for (int k = 0; k < VW; ++k) {
                  if (pos >= w.q.len) vw[e][k] = 0u;
                  else if (pos >= prefix) vw[e][k] = tree_clean<KIND>(vw[e][k], bad);
                }
              }
              __syncwarp();  // the products take the warp together
            }
            if constexpr (C::kQuant) {
#pragma unroll
              for (int k = 0; k < C::VE / 4; ++k) {
                uint32_t b0[4], b1[4];  // columns 4k .. 4k+3
                const uint32_t fl = KIND == kKvInt8 ? 0x80808080u : 0u;
                tree_codes4<KIND>(prmt(vw[0][k], vw[1][k], 0x5140u) ^ fl, b0[0], b0[1]);
                tree_codes4<KIND>(prmt(vw[0][k], vw[1][k], 0x7362u) ^ fl, b0[2], b0[3]);
                tree_codes4<KIND>(prmt(vw[2][k], vw[3][k], 0x5140u) ^ fl, b1[0], b1[1]);
                tree_codes4<KIND>(prmt(vw[2][k], vw[3][k], 0x7362u) ^ fl, b1[2], b1[3]);
#pragma unroll
                for (int i = 0; i < 4; ++i)
#pragma unroll
                  for (int mt = 0; mt < MT; ++mt) tree_mma<KIND>(o[mt][4 * k + i], pa[mt][kb], b0[i], b1[i]);
              }
            } else {
#pragma unroll
              for (int k = 0; k < 4; ++k)
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                  const uint32_t sel = i ? 0x7632u : 0x5410u;
                  const uint32_t b0 = prmt(vw[0][k], vw[1][k], sel), b1 = prmt(vw[2][k], vw[3][k], sel);
#pragma unroll
                  for (int mt = 0; mt < MT; ++mt) tree_mma<KIND>(o[mt][8 * x + 2 * k + i], pa[mt][kb], b0, b1);
                }
            }
          }
      };
      if (pos0 + C::TOK > prefix) step(std::true_type{});
      else step(std::false_type{});
      __syncwarp();
      if (lane == 0) mbar_arrive(smem_u32(&bar_empty[st]));
    }
    // ---- join the warps
#pragma unroll
    for (int mt = 0; mt < MT; ++mt)
#pragma unroll
      for (int hh = 0; hh < 2; ++hh) {
        l[mt][hh] += __shfl_xor_sync(0xffffffffu, l[mt][hh], 1);
        l[mt][hh] += __shfl_xor_sync(0xffffffffu, l[mt][hh], 2);
        if (c4 == 0) {
          red_m[warp][16 * mt + 8 * hh + q4] = m[mt][hh];
          red_l[warp][16 * mt + 8 * hh + q4] = l[mt][hh];
        }
      }
    if (bad) bad_sh = 1;
    named_sync(1, NC);
    float f[MT][2];
#pragma unroll
    for (int mt = 0; mt < MT; ++mt)
#pragma unroll
      for (int hh = 0; hh < 2; ++hh) {
        const int r = 16 * mt + 8 * hh + q4;
        float M = tree_top(red_m[0][r], red_l[0][r]);
#pragma unroll
        for (int k = 1; k < C::kWarps; ++k) M = fmaxf(M, tree_top(red_m[k][r], red_l[k][r]));
        const float ref = M == -INFINITY ? 0.f : M;
        float L = 0.f;
#pragma unroll
        for (int k = 0; k < C::kWarps; ++k) L += red_l[k][r] * tree_pow2(red_m[k][r] - ref);
        f[mt][hh] = tree_pow2(m[mt][hh] - ref);
        if (warp == 0 && c4 == 0) {
          fin_m[r] = M;
          fin_l[r] = L;
        }
      }
    // O in kWarps parts; in step k a warp adds its values of part (warp + k) mod kWarps:
    // no two warps at the same part, and each part's sum in a fixed order
    for (int k = 0; k < C::kWarps; ++k) {
      const int mine = (warp + k) & (C::kWarps - 1);
#pragma unroll
      for (int mt = 0; mt < MT; ++mt)
#pragma unroll
        for (int x = 0; x < C::kBoxes; ++x)
#pragma unroll
          for (int i = 0; i < C::VE; i += 4)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              const int quarter = D == 128 ? (C::VE * x + i) / 4 : (i / 4) * 2 + e;  // of a row's columns
              if (mine != (C::kBig ? mt * 4 + quarter : quarter)) continue;
#pragma unroll
              for (int hh = 0; hh < 2; ++hh) {
                float4 *dst = reinterpret_cast<float4 *>(obuf + (16 * mt + 8 * hh + q4) * C::kLd + 64 * x + C::VE * (2 * c4 + e) + i);
                float4 v = k == 0 ? make_float4(0.f, 0.f, 0.f, 0.f) : *dst;
                const int oi = C::VE * x + i, oe = 2 * hh + e;
                v.x = fmaf(o[mt][oi][oe], f[mt][hh], v.x);
                v.y = fmaf(o[mt][oi + 1][oe], f[mt][hh], v.y);
                v.z = fmaf(o[mt][oi + 2][oe], f[mt][hh], v.z);
                v.w = fmaf(o[mt][oi + 3][oe], f[mt][hh], v.w);
                *dst = v;
              }
            }
      named_sync(1, NC);
    }
    // ---- out, or this CTA's part of it
    const bool whole = w.a == 0 && w.b == w.q.nt;
    const int slot = 2 * blockIdx.x + (w.a == 0 ? 1 : 0);
    const int fixup = bad_sh;
    for (int x = threadIdx.x; x < R * (D / 4); x += NC) {
      const int r = x / (D / 4), col = 4 * (x % (D / 4));
      const int i = (rbase + r) / P.g, h = w.j * P.g + (rbase + r) % P.g;
      float4 v = *reinterpret_cast<const float4 *>(obuf + r * C::kLd + col);
      const float L = fin_l[r];
      if (whole) {
        const float inv = L == 0.f ? 0.f : 1.f / L;
        v.x *= inv; v.y *= inv; v.z *= inv; v.w *= inv;
      }
      if (fixup) {
        float *vv = reinterpret_cast<float *>(&v);
        for (int jj = 0; jj < w.q.n; ++jj) {
          const int pos = prefix + jj;
          if (pos < w.a * C::BN || pos >= w.b * C::BN || !tree_sees(P, w.q, i, jj)) continue;
          for (int e = 0; e < 4; ++e) {
            const float y = tree_v_value<KIND, D>(P, v_pool, w.s, w.j, pos, col + e);
            if (!(fabsf(y) < INFINITY)) vv[e] += y;
          }
        }
      }
      if (whole) {
        uint2 y;
        if (P.q_f16) y = make_uint2(pack_f16x2(v.x, v.y), pack_f16x2(v.z, v.w));
        else y = make_uint2(pack_bf16x2(v.x, v.y), pack_bf16x2(v.z, v.w));
        *reinterpret_cast<uint2 *>(static_cast<uint16_t *>(P.out) + (w.q.row0 + i) * P.o_tok + h * P.o_head + col) = y;
        if (col == 0 && P.lse) P.lse[(int64_t)h * P.T + w.q.row0 + i] = L == 0.f ? -INFINITY : (fin_m[r] + log2f(L)) * kLn2;
      } else {
        *reinterpret_cast<float4 *>(P.part + ((int64_t)slot * C::BM + r) * D + col) = v;
        if (col == 0) {
          P.part_ml[((int64_t)slot * C::BM + r) * 2] = fin_m[r];
          P.part_ml[((int64_t)slot * C::BM + r) * 2 + 1] = L;
        }
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
    named_sync(1, NC);  // obuf and the Q fragments are free again
    if (threadIdx.x == 0) bad_sh = 0;
  }
}

// Adds up the parts of the units that several CTAs share, in the order of the
// CTAs.  grid (C, row groups), a warp per row (D = 64: two rows), a lane per 4
// columns.  A latency, not a bandwidth: so the first 16 parts are under way before
// their weights 2^(m - M) are known, which the lanes work out a part each (M: the
// largest tree_top of the row's parts).
template <int D>
__global__ void __launch_bounds__(256) k_tree_join(const __grid_constant__ TreeParams P, int BM) {
  constexpr int G = D / 4, RPB = 256 / G, NP = 16;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const TreeDesc d = P.desc[blockIdx.x];
  if (d.n == 0) return;
  const int R = min(BM, d.n * P.g - d.row_tile0);
  const int r = blockIdx.y * RPB + threadIdx.x / G, gl = threadIdx.x % G, col = 4 * gl;
  if (r >= R) return;
  const int c0 = blockIdx.x, parts = d.last - c0 + 1;
  const unsigned gm = G == 32 ? 0xffffffffu : 0xffffu << (threadIdx.x & 16);
  auto row_of = [&](int k) { return (int64_t)(2 * (c0 + k) + (k == 0 ? 1 : 0)) * BM + r; };
  auto ml_of = [&](int k) {
    return k < parts ? *reinterpret_cast<const float2 *>(P.part_ml + row_of(k) * 2) : make_float2(-INFINITY, 0.f);
  };
  float4 v[NP];
  auto load = [&](int k0) {
#pragma unroll
    for (int k = 0; k < NP; ++k)
      v[k] = k0 + k < parts ? *reinterpret_cast<const float4 *>(P.part + row_of(k0 + k) * D + col) : make_float4(0.f, 0.f, 0.f, 0.f);
  };
  load(0);
  const float2 first = ml_of(gl);
  float M = tree_top(first.x, first.y);
  for (int k = gl + G; k < parts; k += G) {
    const float2 ml = ml_of(k);
    M = fmaxf(M, tree_top(ml.x, ml.y));
  }
#pragma unroll
  for (int o = G / 2; o > 0; o >>= 1) M = fmaxf(M, __shfl_xor_sync(gm, M, o));
  const float ref = M == -INFINITY ? 0.f : M;
  float L = 0.f;
  float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
  for (int k0 = 0; k0 < parts; k0 += G) {
    const float2 ml = k0 == 0 ? first : ml_of(k0 + gl);
    const float f = tree_pow2(ml.x - ref);
    float lsum = ml.y * f;
#pragma unroll
    for (int o = G / 2; o > 0; o >>= 1) lsum += __shfl_xor_sync(gm, lsum, o);
    L += lsum;
    for (int kk = 0; kk < G && k0 + kk < parts; kk += NP) {
      if (k0 + kk > 0) load(k0 + kk);
#pragma unroll
      for (int k = 0; k < NP; ++k) {
        const float fk = __shfl_sync(gm, f, kk + k, G);  // 0 behind the last part
        acc.x = fmaf(v[k].x, fk, acc.x);
        acc.y = fmaf(v[k].y, fk, acc.y);
        acc.z = fmaf(v[k].z, fk, acc.z);
        acc.w = fmaf(v[k].w, fk, acc.w);
      }
    }
  }
  const float inv = L == 0.f ? 0.f : 1.f / L;
  const int i = (d.row_tile0 + r) / P.g, h = d.j * P.g + (d.row_tile0 + r) % P.g;
  uint2 y;
  if (P.q_f16) y = make_uint2(pack_f16x2(acc.x * inv, acc.y * inv), pack_f16x2(acc.z * inv, acc.w * inv));
  else y = make_uint2(pack_bf16x2(acc.x * inv, acc.y * inv), pack_bf16x2(acc.z * inv, acc.w * inv));
  *reinterpret_cast<uint2 *>(static_cast<uint16_t *>(P.out) + (d.seq_row0 + i) * P.o_tok + h * P.o_head + col) = y;
  if (col == 0 && P.lse) P.lse[(int64_t)h * P.T + d.seq_row0 + i] = L == 0.f ? -INFINITY : (M + log2f(L)) * kLn2;
}

}  // namespace fpk
