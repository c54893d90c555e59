// decode_sizes.h -- grids and workspaces of the calls of fp_decode.h from their sizes
// and the device's multiprocessors: plain arithmetic, no CUDA.
#pragma once

#include <stddef.h>
#include <stdint.h>

#include <initializer_list>

namespace fpk {

// Tokens and heads of a block of fp_kv_write and fp_kv_read: 32 tokens of all heads, so
// that the slots are looked up once for them, while that makes about eight blocks per
// multiprocessor (enough to fill it); with less work, fewer heads, and then 16 tokens.
struct KvSplit {
  int shift, group;          // log2 of the tokens, heads
  unsigned blocks, groups;   // the grid
};
inline KvSplit kv_split(int heads, int T, int sms) {
  KvSplit s;
  const int64_t want = 8 * (int64_t)(sms > 0 ? sms : 1);
  s.shift = 5;
  int64_t blocks = ((int64_t)T + 31) / 32;
  if (blocks * heads < want) {
    s.shift = 4;
    blocks = ((int64_t)T + 15) / 16;
  }
  int64_t groups = (want + blocks - 1) / blocks;
  if (groups > heads) groups = heads;
  s.group = (int)((heads + groups - 1) / groups);
  s.blocks = (unsigned)blocks;
  s.groups = (unsigned)((heads + s.group - 1) / s.group);
  return s;
}

inline size_t round_up(size_t x) { return (x + 255) / 256 * 256; }

// Query rows of a unit of fp_tree_attn for at most `rows` rows of a KV head, and the CTAs
// that go with it.
inline int tree_bm(int rows) { return rows <= 16 ? 16 : rows <= 32 ? 32 : rows <= 128 ? 128 : 256; }
inline int tree_ctas(int bm, int d, int sms) { return bm == 16 || (bm == 32 && d == 64) ? 2 * sms : sms; }

constexpr size_t kTreeDescBytes = 32;
struct TreeWork {
  size_t part, ml, desc, bytes;
};
inline TreeWork tree_work(int ctas, int bm, int d) {
  TreeWork w;
  w.part = 0;
  w.ml = round_up((size_t)2 * ctas * bm * d * 4);
  w.desc = w.ml + round_up((size_t)2 * ctas * bm * 8);
  w.bytes = w.desc + round_up((size_t)ctas * kTreeDescBytes);
  return w;
}

// Bytes that serve every call of at most `rows` rows: fewer rows may take more CTAs.
inline size_t tree_workspace(int rows, int d, int sms) {
  size_t most = 0;
  for (const int bm : {16, 32, 128, 256}) {
    if (bm > tree_bm(rows)) break;
    const size_t b = tree_work(tree_ctas(bm, d, sms), bm, d).bytes;
    if (b > most) most = b;
  }
  return most;
}

}  // namespace fpk
