// fp_decode.cu -- host side of include/fp_decode.h: argument checks, the
// rotary frequencies, tensor maps and launches.
#include <atomic>
#include <cmath>
#include <cstdint>
#include <new>

#include "decode_sizes.h"
#include "fp_decode.h"
#include "fp_internal.h"
#include "kv_kernels.cuh"
#include "rope_kernel.cuh"
#include "tree_kernels.cuh"
#include "tree_tc.cuh"

using namespace fpk;

struct fp_rope {
  int d, rot, layout;
  float amp;
  double freq[kRopeMaxPairs];
  unsigned long long turn[kRopeMaxPairs];
};

struct fp_kv {
  KvGeom g;
  int dtype, d, device;
  CUtensorMap map[2];
};

namespace {

bool multiple_of(const void *p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }
int status() { return cudaGetLastError() == cudaSuccess ? FP_OK : FP_ERR_CUDA; }

// Multiprocessors of the current device, looked up once per device.
int sms() {
  static std::atomic<int> n[128];
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 128) return 0;
  int v = n[dev].load(std::memory_order_relaxed);
  if (!v) {
    if (cudaDeviceGetAttribute(&v, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess) return 0;
    n[dev].store(v, std::memory_order_relaxed);
  }
  return v;
}

int size_of(int dtype) {
  switch (dtype) {
    case FP_DT_BF16:
    case FP_DT_F16: return 2;
    case FP_DT_F32: return 4;
    case FP_DT_INT8:
    case FP_DT_E4M3: return 1;
  }
  return 0;
}

// A tensor of rows that start on 16-byte boundaries.
bool rows_ok(const void *p, int64_t tok, int64_t head, int size) {
  return p && multiple_of(p, 16) && (tok * size) % 16 == 0 && (head * size) % 16 == 0;
}

}  // namespace

// ---------------------------------------------------------------------------
// Rotary positions
// ---------------------------------------------------------------------------
namespace {

template <typename T>
int launch_rope(RopeParams &P, int layout, bool wide, cudaStream_t st) {
  const int heads = P.side[0].heads + P.side[1].heads;
  const int V = wide ? 16 / (int)sizeof(T) : 1;
  P.rot_slots = P.rot / 2 / V;
  P.slots = P.rot_slots + (P.d - P.rot) / 2 / V;
  const int64_t blocks = ((int64_t)P.T * P.slots + 255) / 256;
  // Few tokens: the heads are spread over blocks until there are about 16 per
  // multiprocessor, two rounds of what fits (5000 fp32 tokens of 20 heads: 22.3 us
  // with 4, 18.2 with 8, 16.0 with 16, 17.6 with 32).
  int64_t groups = (16 * (int64_t)sms() + blocks - 1) / blocks;
  if (groups > heads) groups = heads;
  P.group = (int)((heads + groups - 1) / groups);
  const dim3 grid((unsigned)blocks, (unsigned)((heads + P.group - 1) / P.group));
  if (wide) {
    if (layout == FP_ROPE_HALF) k_rope<T, true><<<grid, 256, 0, st>>>(P);
    else k_rope<T, false><<<grid, 256, 0, st>>>(P);
  } else {
    if (layout == FP_ROPE_HALF) k_rope_any<T, true><<<grid, 256, 0, st>>>(P);
    else k_rope_any<T, false><<<grid, 256, 0, st>>>(P);
  }
  return status();
}

}  // namespace

extern "C" {

int fp_rope_create(int d, int rot, int layout, double theta, int scaling, double factor, double orig_len, double low,
                   double high, double amplitude, fp_rope **out) {
  if (!out) return FP_ERR_ARG;
  *out = nullptr;
  if (d < 2 || d > 512 || (d & 1) || rot < 2 || (rot & 1) || rot > d || rot > 2 * kRopeMaxPairs) return FP_ERR_ARG;
  if (layout != FP_ROPE_HALF && layout != FP_ROPE_INTERLEAVED) return FP_ERR_ARG;
  if (scaling < FP_ROPE_NONE || scaling > FP_ROPE_RAMP) return FP_ERR_ARG;
  if (!(theta > 1.0) || !std::isfinite(theta) || !(amplitude > 0.0) || !std::isfinite((float)amplitude)) return FP_ERR_ARG;
  if (!(factor > 0.0) || !std::isfinite(factor)) return FP_ERR_ARG;
  if (scaling == FP_ROPE_BASE && rot <= 2) return FP_ERR_ARG;
  if (scaling == FP_ROPE_BANDS || scaling == FP_ROPE_RAMP)
    if (!(orig_len > 0.0) || !(low > 0.0) || !(high > low) || !std::isfinite(high) || !std::isfinite(orig_len))
      return FP_ERR_ARG;
  fp_rope *r = new (std::nothrow) fp_rope();
  if (!r) return FP_ERR_CUDA;
  r->d = d;
  r->rot = rot;
  r->layout = layout;
  r->amp = (float)amplitude;
  const long double two_pi = 6.283185307179586476925286766559L;
  long double base = theta;
  if (scaling == FP_ROPE_BASE) base *= powl(factor, (long double)rot / (rot - 2));
  double lo = 0, hi = 0;  // RAMP: between which pairs the frequencies pass over
  if (scaling == FP_ROPE_RAMP) {
    auto at = [&](double turns) { return rot * std::log(orig_len / ((double)two_pi * turns)) / (2 * std::log(theta)); };
    lo = std::fmax(std::floor(at(high)), 0.0);
    hi = std::fmin(std::ceil(at(low)), rot - 1.0);
  }
  bool ok = true;
  const long double step = powl(base, -2.0L / rot);
  long double power = 1.0L;  // step^i, off by at most i 2^-63 of itself
  for (int i = 0; i < rot / 2; ++i, power *= step) {
    long double f = power;
    if (scaling == FP_ROPE_LINEAR) f /= factor;
    if (scaling == FP_ROPE_BANDS) {
      long double w = ((long double)orig_len * f / two_pi - low) / (high - low);
      w = w < 0 ? 0 : (w > 1 ? 1 : w);
      f = f * w + f / factor * (1 - w);
    }
    if (scaling == FP_ROPE_RAMP) {
      long double w = (i - lo) / std::fmax(hi - lo, 0.001);
      w = w < 0 ? 0 : (w > 1 ? 1 : w);
      f = f * (1 - w) + f / factor * w;
    }
    ok = ok && std::isfinite((double)f);
    r->freq[i] = (double)f;
    long double turns = f / two_pi;
    turns -= floorl(turns);
    const long double fixed = roundl(ldexpl(turns, 64));
    r->turn[i] = fixed >= 18446744073709551616.0L ? 0ull : (unsigned long long)fixed;
  }
  if (!ok) {
    delete r;
    return FP_ERR_ARG;
  }
  *out = r;
  return FP_OK;
}

void fp_rope_free(fp_rope *r) { delete r; }

int fp_rope_freqs(const fp_rope *r, double *freqs) {
  if (!r || !freqs) return FP_ERR_ARG;
  for (int i = 0; i < r->rot / 2; ++i) freqs[i] = r->freq[i];
  return FP_OK;
}

int fp_rope_apply(const fp_rope *r, const void *q_in, int64_t q_in_tok, int64_t q_in_head, const void *k_in,
                  int64_t k_in_tok, int64_t k_in_head, void *q_out, int64_t q_out_tok, int64_t q_out_head,
                  void *k_out, int64_t k_out_tok, int64_t k_out_head, int dtype, int T, int Hq, int Hkv,
                  const int32_t *pos, int inverse, void *stream) {
  if (!r || T < 0 || Hq < 0 || Hkv < 0 || (int64_t)Hq + Hkv > 65535) return FP_ERR_ARG;
  if (dtype != FP_DT_BF16 && dtype != FP_DT_F16 && dtype != FP_DT_F32) return FP_ERR_ARG;
  if (T == 0 || Hq + Hkv == 0) return FP_OK;
  const int size = size_of(dtype);
  RopeParams P;
  P.side[0] = RopeSide{q_in, q_out, q_in_tok, q_in_head, q_out_tok, q_out_head, Hq};
  P.side[1] = RopeSide{k_in, k_out, k_in_tok, k_in_head, k_out_tok, k_out_head, Hkv};
  bool wide = (r->rot / 2) % (16 / size) == 0 && ((r->d - r->rot) / 2) % (16 / size) == 0;
  P.copy_tail = 0;
  for (const RopeSide &s : P.side) {
    if (!s.heads) continue;
    if (!s.in || !s.out || !multiple_of(s.in, size) || !multiple_of(s.out, size)) return FP_ERR_ARG;
    wide = wide && rows_ok(s.in, s.in_tok, s.in_head, size) && rows_ok(s.out, s.out_tok, s.out_head, size);
    if (s.in == s.out) {  // in place: the same strides, or the rows would overlap
      if (s.in_tok != s.out_tok || s.in_head != s.out_head) return FP_ERR_ARG;
    } else {
      P.copy_tail = 1;
    }
  }
  if (!pos || !multiple_of(pos, 4)) return FP_ERR_ARG;
  if (!sms()) return FP_ERR_CUDA;
  P.pos = pos;
  P.T = T;
  P.rot = r->rot;
  P.d = r->d;
  P.amp = r->amp;
  P.sign = inverse ? -1.f : 1.f;
  for (int i = 0; i < r->rot / 2; ++i) P.turn[i] = r->turn[i];
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  if (dtype == FP_DT_BF16) return launch_rope<__nv_bfloat16>(P, r->layout, wide, st);
  if (dtype == FP_DT_F16) return launch_rope<__half>(P, r->layout, wide, st);
  return launch_rope<float>(P, r->layout, wide, st);
}

}  // extern "C"

// ---------------------------------------------------------------------------
// Paged key/value cache
// ---------------------------------------------------------------------------
namespace {

bool on_device(const fp_kv *kv) {
  int dev = -1;
  return cudaGetDevice(&dev) == cudaSuccess && dev == kv->device;
}

template <int KIND, typename T>
int launch_kv_write(const KvWriteParams &P, int d, dim3 grid, cudaStream_t st) {
  if (d == 128) k_kv_write<KIND, T, 128><<<grid, kKvThreads, 0, st>>>(P);
  else k_kv_write<KIND, T, 64><<<grid, kKvThreads, 0, st>>>(P);
  return status();
}
template <int KIND, typename T>
int launch_kv_read(const KvReadParams &P, int d, dim3 grid, cudaStream_t st) {
  if (d == 128) k_kv_read<KIND, T, 128><<<grid, kKvThreads, 0, st>>>(P);
  else k_kv_read<KIND, T, 64><<<grid, kKvThreads, 0, st>>>(P);
  return status();
}
template <typename P>
int launch_kv(int kind, int dtype, const P &p, int d, dim3 grid, cudaStream_t st) {
#define FPK_KV_TYPES(K)                                                                   \
  if (kind == K) {                                                                        \
    if constexpr (std::is_same<P, KvWriteParams>::value) {                                \
      if (dtype == FP_DT_BF16) return launch_kv_write<K, __nv_bfloat16>(p, d, grid, st);  \
      if (dtype == FP_DT_F16) return launch_kv_write<K, __half>(p, d, grid, st);          \
      return launch_kv_write<K, float>(p, d, grid, st);                                   \
    } else {                                                                              \
      if (dtype == FP_DT_BF16) return launch_kv_read<K, __nv_bfloat16>(p, d, grid, st);   \
      if (dtype == FP_DT_F16) return launch_kv_read<K, __half>(p, d, grid, st);           \
      return launch_kv_read<K, float>(p, d, grid, st);                                    \
    }                                                                                     \
  }
  FPK_KV_TYPES(kKvBf16)
  FPK_KV_TYPES(kKvF16)
  FPK_KV_TYPES(kKvInt8)
  FPK_KV_TYPES(kKvE4m3)
#undef FPK_KV_TYPES
  return FP_ERR_ARG;
}

}  // namespace

extern "C" {

int fp_kv_create(void *k_pool, void *v_pool, float *k_scale, float *v_scale, int dtype, int64_t pages, int page,
                 int Hkv, int d, fp_kv **out) {
  if (!out) return FP_ERR_ARG;
  *out = nullptr;
  if (dtype != FP_DT_BF16 && dtype != FP_DT_F16 && dtype != FP_DT_INT8 && dtype != FP_DT_E4M3) return FP_ERR_ARG;
  const bool quant = dtype == FP_DT_INT8 || dtype == FP_DT_E4M3;
  if (page != 16 && page != 32 && page != 64 && page != 128) return FP_ERR_ARG;
  if ((d != 64 && d != 128) || Hkv <= 0 || Hkv > 65535 || pages <= 0) return FP_ERR_ARG;
  if (pages > (int64_t)INT32_MAX / Hkv / page) return FP_ERR_ARG;
  if (!k_pool || !v_pool || !multiple_of(k_pool, 16) || !multiple_of(v_pool, 16)) return FP_ERR_ARG;
  if (quant ? (!k_scale || !v_scale || !multiple_of(k_scale, 16) || !multiple_of(v_scale, 16)) : (k_scale || v_scale))
    return FP_ERR_ARG;
  fp_kv *kv = new (std::nothrow) fp_kv();
  if (!kv) return FP_ERR_CUDA;
  kv->g.pool[0] = k_pool;
  kv->g.pool[1] = v_pool;
  kv->g.scale[0] = k_scale;
  kv->g.scale[1] = v_scale;
  kv->g.pages = pages;
  kv->g.page = page;
  kv->g.page_shift = page == 16 ? 4 : page == 32 ? 5 : page == 64 ? 6 : 7;
  kv->g.heads = Hkv;
  kv->dtype = dtype;
  kv->d = d;
  const uint32_t row = d * size_of(dtype), box = row < 128 ? row : 128;
  const uint64_t rows = (uint64_t)pages * Hkv * page;
  if (cudaGetDevice(&kv->device) != cudaSuccess ||
      !make_byte_map(&kv->map[0], k_pool, row, rows, box, page < 64 ? page : 64) ||
      !make_byte_map(&kv->map[1], v_pool, row, rows, box, page < 64 ? page : 64)) {
    delete kv;
    return FP_ERR_CUDA;
  }
  *out = kv;
  return FP_OK;
}

void fp_kv_free(fp_kv *kv) { delete kv; }

int fp_kv_write(const fp_kv *kv, const void *k, int64_t k_tok, int64_t k_head, const void *v, int64_t v_tok,
                int64_t v_head, int dtype, int T, const int64_t *slots, void *stream) {
  if (!kv || T < 0) return FP_ERR_ARG;
  if (dtype != FP_DT_BF16 && dtype != FP_DT_F16 && dtype != FP_DT_F32) return FP_ERR_ARG;
  if (T == 0) return FP_OK;
  if (!k && !v) return FP_ERR_ARG;
  const int size = size_of(dtype);
  if (k && !rows_ok(k, k_tok, k_head, size)) return FP_ERR_ARG;
  if (v && !rows_ok(v, v_tok, v_head, size)) return FP_ERR_ARG;
  if (!slots || !multiple_of(slots, 8)) return FP_ERR_ARG;
  if (!on_device(kv)) return FP_ERR_ARG;
  if (!sms()) return FP_ERR_CUDA;
  KvWriteParams P;
  P.g = kv->g;
  P.in[0] = k;
  P.in[1] = v;
  P.tok[0] = k_tok;
  P.tok[1] = v_tok;
  P.head[0] = k_head;
  P.head[1] = v_head;
  P.slots = slots;
  P.T = T;
  const KvSplit split = kv_split(kv->g.heads, T, sms());
  P.group = split.group;
  P.tok_shift = split.shift;
  P.err = library_error_word();
  if (!P.err) return FP_ERR_CUDA;
  return launch_kv(kv->dtype, dtype, P, kv->d, dim3(split.blocks, split.groups), static_cast<cudaStream_t>(stream));
}

int fp_kv_read(const fp_kv *kv, const int32_t *block_table, int max_pages, const int32_t *cu, const int32_t *first,
               int nseq, int T, void *k, int64_t k_tok, int64_t k_head, void *v, int64_t v_tok, int64_t v_head,
               int dtype, void *stream) {
  if (!kv || T < 0 || nseq < 0 || max_pages < 0) return FP_ERR_ARG;
  if (dtype != FP_DT_BF16 && dtype != FP_DT_F16 && dtype != FP_DT_F32) return FP_ERR_ARG;
  if (T == 0 || nseq == 0) return FP_OK;
  if (!k && !v) return FP_ERR_ARG;
  const int size = size_of(dtype);
  if (k && !rows_ok(k, k_tok, k_head, size)) return FP_ERR_ARG;
  if (v && !rows_ok(v, v_tok, v_head, size)) return FP_ERR_ARG;
  if (!block_table || !cu || !multiple_of(block_table, 4) || !multiple_of(cu, 4) || !multiple_of(first, 4))
    return FP_ERR_ARG;
  if (!on_device(kv)) return FP_ERR_ARG;
  if (!sms()) return FP_ERR_CUDA;
  KvReadParams P;
  P.g = kv->g;
  P.out[0] = k;
  P.out[1] = v;
  P.tok[0] = k_tok;
  P.tok[1] = v_tok;
  P.head[0] = k_head;
  P.head[1] = v_head;
  P.table = block_table;
  P.cu = cu;
  P.first = first;
  P.max_pages = max_pages;
  P.nseq = nseq;
  P.T = T;
  const KvSplit split = kv_split(kv->g.heads, T, sms());
  P.group = split.group;
  P.tok_shift = split.shift;
  P.err = library_error_word();
  if (!P.err) return FP_ERR_CUDA;
  return launch_kv(kv->dtype, dtype, P, kv->d, dim3(split.blocks, split.groups), static_cast<cudaStream_t>(stream));
}

}  // extern "C"

// ---------------------------------------------------------------------------
// Attention of drafted tokens over the cache
// ---------------------------------------------------------------------------
namespace {

bool tree_shape_ok(int nseq, int max_q, int Hq, int Hkv, int d) {
  return nseq >= 0 && max_q >= 1 && max_q <= 256 && Hkv > 0 && Hq > 0 && Hq % Hkv == 0 && Hq / Hkv <= 256 &&
         (d == 64 || d == 128);
}

constexpr int kTreeLeastBN = 64;  // the shortest of all kernels' token tiles
static_assert(sizeof(TreeDesc) == kTreeDescBytes, "the workspace's descriptors");

// Raises a kernel's shared-memory limit, once in a context; `where` is the kernel's
// own record of the contexts it was raised in, by device.
template <typename K>
bool allow_smem(K kernel, int bytes, std::atomic<void *> (&where)[128]) {
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 128) return false;
  void *ctx = library_context();
  if (ctx && where[dev].load(std::memory_order_relaxed) == ctx) return true;
  if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes) != cudaSuccess) return false;
  where[dev].store(ctx, std::memory_order_relaxed);
  return true;
}

// The parts of split units are added up by a launch of its own, which may be
// set up while the first one still runs.
template <int D>
int launch_join(const TreeParams &P, int bm, int ctas, cudaStream_t st) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(ctas, (bm + 1024 / D - 1) / (1024 / D));
  cfg.blockDim = dim3(256);
  cfg.stream = st;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, k_tree_join<D>, P, bm) == cudaSuccess ? FP_OK : FP_ERR_CUDA;
}

template <int KIND, int D, int MT>
int launch_tree(const fp_kv *kv, const TreeParams &P, int ctas, cudaStream_t st) {
  using C = TreeCfg<KIND, D, MT>;
  static std::atomic<void *> raised[128];
  if (!allow_smem(k_tree<KIND, D, MT>, C::kSmem, raised)) return FP_ERR_CUDA;
  k_tree<KIND, D, MT><<<ctas, C::kThreads, C::kSmem, st>>>(kv->map[0], kv->map[1], P, kv->g.pool[1]);
  const int rc = status();
  return rc ? rc : launch_join<D>(P, C::BM, ctas, st);
}

template <int KIND, int D, bool PAIR>
int launch_tree_tc(const fp_kv *kv, const TreeParams &P, int ctas, cudaStream_t st) {
  using C = TcCfg<KIND, D, PAIR>;
  static std::atomic<void *> raised[128];
  if (!allow_smem(k_tree_tc<KIND, D, PAIR>, C::kSmem, raised)) return FP_ERR_CUDA;
  k_tree_tc<KIND, D, PAIR><<<ctas, kTcThreads, C::kSmem, st>>>(kv->map[0], kv->map[1], P, kv->g.pool[1]);
  const int rc = status();
  return rc ? rc : launch_join<D>(P, C::BM, ctas, st);
}

template <int KIND, int D>
int launch_tree_kind(const fp_kv *kv, const TreeParams &P, int bm, int ctas, cudaStream_t st) {
  switch (bm) {
    case 16: return launch_tree<KIND, D, 1>(kv, P, ctas, st);
    case 32: return launch_tree<KIND, D, 2>(kv, P, ctas, st);
    case 128: return launch_tree_tc<KIND, D, false>(kv, P, ctas, st);
    default: return launch_tree_tc<KIND, D, true>(kv, P, ctas, st);
  }
}
template <int KIND>
int launch_tree_kind(const fp_kv *kv, const TreeParams &P, int bm, int ctas, cudaStream_t st) {
  return kv->d == 128 ? launch_tree_kind<KIND, 128>(kv, P, bm, ctas, st) : launch_tree_kind<KIND, 64>(kv, P, bm, ctas, st);
}

}  // namespace

extern "C" {

size_t fp_tree_attn_workspace(int nseq, int max_q, int Hq, int Hkv, int d) {
  if (!tree_shape_ok(nseq, max_q, Hq, Hkv, d)) return 0;
  if (!sms()) return 0;
  return tree_workspace(max_q * (Hq / Hkv), d, sms());
}

int fp_tree_attn(const fp_kv *kv, const void *q, int64_t q_tok, int64_t q_head, int dtype, int T, int Hq,
                 const int32_t *block_table, int max_pages, const int32_t *kv_len, const int32_t *cu_q, int nseq,
                 int max_q, const uint64_t *mask, float scale, void *out, int64_t o_tok, int64_t o_head, float *lse,
                 void *work, size_t work_bytes, void *stream) {
  if (!kv || T < 0 || max_pages < 0 || !tree_shape_ok(nseq, max_q, Hq, kv->g.heads, kv->d)) return FP_ERR_ARG;
  if ((int64_t)max_pages * kv->g.page > (int64_t)1 << 30) return FP_ERR_ARG;  // positions are 32-bit in the kernels
  if (dtype != FP_DT_BF16 && dtype != FP_DT_F16) return FP_ERR_ARG;
  if ((kv->dtype == FP_DT_BF16 || kv->dtype == FP_DT_F16) && kv->dtype != dtype) return FP_ERR_ARG;
  if (!(scale > 0.f) || !std::isfinite(scale)) return FP_ERR_ARG;
  if (T == 0 || nseq == 0) return FP_OK;
  if (!rows_ok(q, q_tok, q_head, 2) || !rows_ok(out, o_tok, o_head, 2)) return FP_ERR_ARG;
  if (!block_table || !kv_len || !cu_q || !multiple_of(block_table, 4) || !multiple_of(kv_len, 4) ||
      !multiple_of(cu_q, 4) || !multiple_of(mask, 8) || !multiple_of(lse, 4))
    return FP_ERR_ARG;
  if (!work || !multiple_of(work, 16)) return FP_ERR_ARG;
  if (!on_device(kv)) return FP_ERR_ARG;
  if (!sms()) return FP_ERR_CUDA;
  const int g = Hq / kv->g.heads, bm = tree_bm(max_q * g);
  const int most = tree_ctas(bm, kv->d, sms());
  const TreeWork w = tree_work(most, bm, kv->d);
  if (work_bytes < w.bytes) return FP_ERR_ARG;
  // no more CTAs than there can be tiles
  const double tiles = (double)nseq * ((max_q * g + bm - 1) / bm) * kv->g.heads *
                       std::ceil((double)max_pages * kv->g.page / kTreeLeastBN);
  const int ctas = tiles < most ? (tiles < 1 ? 1 : (int)tiles) : most;
  TreeParams P;
  P.scale[0] = kv->g.scale[0];
  P.scale[1] = kv->g.scale[1];
  P.table = block_table;
  P.kv_len = kv_len;
  P.cu = cu_q;
  P.mask = reinterpret_cast<const unsigned long long *>(mask);
  P.q = q;
  P.out = out;
  P.lse = lse;
  char *base = static_cast<char *>(work);
  P.part = reinterpret_cast<float *>(base + w.part);
  P.part_ml = reinterpret_cast<float *>(base + w.ml);
  P.desc = reinterpret_cast<TreeDesc *>(base + w.desc);
  P.err = library_error_word();
  if (!P.err) return FP_ERR_CUDA;
  P.q_tok = q_tok;
  P.q_head = q_head;
  P.o_tok = o_tok;
  P.o_head = o_head;
  P.pages = kv->g.pages;
  P.max_pages = max_pages;
  P.nseq = nseq;
  P.T = T;
  P.max_q = max_q;
  P.W = (max_q + 63) / 64;
  P.Hq = Hq;
  P.Hkv = kv->g.heads;
  P.g = g;
  P.page = kv->g.page;
  P.page_shift = kv->g.page_shift;
  P.q_f16 = dtype == FP_DT_F16;
  P.scale2 = std::fmin(scale * 1.4426950408889634f, 3.4028235e38f);
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  switch (kv->dtype) {
    case FP_DT_BF16: return launch_tree_kind<kKvBf16>(kv, P, bm, ctas, st);
    case FP_DT_F16: return launch_tree_kind<kKvF16>(kv, P, bm, ctas, st);
    case FP_DT_INT8: return launch_tree_kind<kKvInt8>(kv, P, bm, ctas, st);
    default: return launch_tree_kind<kKvE4m3>(kv, P, bm, ctas, st);
  }
}

}  // extern "C"
