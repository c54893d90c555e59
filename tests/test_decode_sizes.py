"""Grids and workspaces of the serving calls (csrc/decode_sizes.h), compiled for the host."""
import ctypes
import os
import subprocess

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "dynamic_block_sparse_last_b200", "csrc")

SHIM = """
#include "decode_sizes.h"
extern "C" size_t need(int rows, int d, int sms) {      // what a call of exactly these rows checks for
  const int bm = fpk::tree_bm(rows);
  return fpk::tree_work(fpk::tree_ctas(bm, d, sms), bm, d).bytes;
}
extern "C" void split(int heads, int T, int sms, int64_t *out) {
  const fpk::KvSplit s = fpk::kv_split(heads, T, sms);
  out[0] = s.shift; out[1] = s.group; out[2] = s.blocks; out[3] = s.groups;
}
extern "C" size_t space(int rows, int d, int sms) { return fpk::tree_workspace(rows, d, sms); }
"""


@pytest.fixture(scope="module")
def sizes(tmp_path_factory):
    at = tmp_path_factory.mktemp("sizes")
    (at / "shim.cpp").write_text(SHIM)
    subprocess.check_call(["g++", "-std=c++17", "-O1", "-Wall", "-Werror", "-shared", "-fPIC", "-I" + CSRC, str(at / "shim.cpp"),
                           "-o", str(at / "shim.so")])
    lib = ctypes.CDLL(str(at / "shim.so"))
    lib.need.restype = lib.space.restype = ctypes.c_size_t
    return lib


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("sms", [1, 7, 132, 148, 160])
def test_a_workspace_serves_every_call_with_fewer_rows(sizes, d, sms):
    most = 0
    for rows in [*range(1, 300), 1000, 65536]:
        most = max(most, sizes.need(rows, d, sms))
        assert sizes.space(rows, d, sms) == most


@pytest.mark.parametrize("sms", [0, 1, 132, 148])
@pytest.mark.parametrize("heads", [1, 2, 3, 8, 40, 65535])
def test_cache_blocks_cover_every_token_and_head_once(sizes, sms, heads):
    """Also on a device whose multiprocessors could not be counted (0), where the calls return an error."""
    out = (ctypes.c_int64 * 4)()
    for T in [1, 15, 16, 17, 33, 500, 4737, 131072, 2 ** 31 - 1]:
        sizes.split(heads, T, sms, out)
        shift, group, blocks, groups = out
        assert shift in (4, 5) and 1 <= group <= heads
        assert (blocks - 1) << shift < T <= blocks << shift
        assert (groups - 1) * group < heads <= groups * group
