"""The calls of include/fp_decode.h without a GPU: what they refuse on the host
before any CUDA call, and the rotary frequencies against their formulas."""
import ctypes
import math

import numpy as np
import pytest


@pytest.fixture(scope="module")
def fp():
    from dynamic_block_sparse_last_b200 import build
    build.build()
    from dynamic_block_sparse_last_b200 import fp as mod
    return mod


ROPE_OK = dict(d=128, rot=128, layout=0, theta=1e4, scaling=0, factor=1.0, orig_len=0.0, low=0.0, high=0.0, amplitude=1.0)


@pytest.mark.parametrize("bad", [
    dict(d=0), dict(d=127), dict(d=514, rot=2), dict(rot=0), dict(rot=3), dict(rot=130), dict(d=512, rot=258),
    dict(layout=2), dict(theta=1.0), dict(theta=float("nan")), dict(theta=float("inf")), dict(scaling=5), dict(scaling=-1),
    dict(factor=0.0), dict(factor=float("inf")), dict(amplitude=0.0), dict(amplitude=1e39), dict(scaling=2, rot=2),
    dict(scaling=3, orig_len=0.0, low=1.0, high=4.0), dict(scaling=3, orig_len=8192.0, low=4.0, high=4.0),
    dict(scaling=3, orig_len=8192.0, low=0.0, high=4.0), dict(scaling=4, orig_len=4096.0, low=32.0, high=1.0),
    dict(scaling=4, orig_len=float("inf"), low=1.0, high=32.0)], ids=str)
def test_rope_create_refuses(fp, bad):
    h = ctypes.c_void_p(1)
    assert fp.lib().fp_rope_create(*{**ROPE_OK, **bad}.values(), ctypes.byref(h)) == fp.FP_ERR_ARG
    assert h.value is None
    assert fp.lib().fp_rope_create(*ROPE_OK.values(), None) == fp.FP_ERR_ARG


def reference_freqs(rot, theta, scaling, factor=1.0, orig=0.0, low=0.0, high=0.0):
    if scaling == 2:
        theta = theta * factor ** (rot / (rot - 2))
    out = []
    for i in range(rot // 2):
        f = theta ** (-2.0 * i / rot)
        if scaling == 1:
            f /= factor
        elif scaling == 3:
            n = orig / (2 * math.pi / f)      # original length over the wavelength
            if n <= low:
                f = f / factor
            elif n < high:
                w = (n - low) / (high - low)
                f = f * w + f * (1 - w) / factor
        elif scaling == 4:
            c = [rot * math.log(orig / (n * 2 * math.pi)) / (2 * math.log(theta)) for n in (high, low)]
            a, b = max(math.floor(c[0]), 0), min(math.ceil(c[1]), rot - 1)
            u = min(max((i - a) / max(b - a, 0.001), 0.0), 1.0)
            f = f * (1 - u) + f * u / factor
        out.append(f)
    return np.array(out)


@pytest.mark.parametrize("rot", [2, 16, 64, 96, 128, 256])
@pytest.mark.parametrize("scaling,args", [(0, {}), (1, dict(factor=4.0)), (2, dict(factor=8.0)),
                                          (3, dict(factor=8.0, orig_len=8192.0, low=1.0, high=4.0)),
                                          (4, dict(factor=32.0, orig_len=4096.0, low=1.0, high=32.0))])
@pytest.mark.parametrize("theta", [1e4, 5e5])
def test_rope_frequencies(fp, rot, scaling, args, theta):
    if scaling == 2 and rot == 2:
        return
    r = fp.Rope(256, rot_dim=rot, theta=theta, scaling=scaling, **args)
    ref = reference_freqs(rot, theta, scaling, args.get("factor", 1.0), args.get("orig_len", 0.0), args.get("low", 0.0),
                          args.get("high", 0.0))
    # each frequency is a power, a product and a quotient in fp64: a few times 2^-53, and a power's error grows
    # with the logarithm of its value (below 2^5 here)
    assert np.all(np.abs(r.freqs() - ref) <= 2.0 ** -46 * ref)
    assert r.freqs()[0] == 1.0 or scaling in (1, 3, 4)


def rope_args(fp, h, **bad):
    a = dict(r=h, q=4096, qt=128, qh=1280, k=8192, kt=128, kh=1280, qo=4096, qot=128, qoh=1280, ko=8192, kot=128,
             koh=1280, dtype=fp.FP_DT_BF16, T=10, Hq=4, Hkv=2, pos=16, inverse=0, stream=None)
    a.update(bad)
    return list(a.values())


def test_rope_apply_refuses(fp):
    h = fp.Rope(128).handle
    call = fp.lib().fp_rope_apply
    for bad in (dict(r=None), dict(T=-1), dict(Hq=-1), dict(Hkv=-1), dict(Hq=65536), dict(dtype=3), dict(dtype=-1),
                dict(q=None), dict(ko=None), dict(q=4097, qo=4097), dict(pos=None), dict(pos=18),
                dict(qot=256), dict(koh=128)):  # in place with other strides
        assert call(*rope_args(fp, h, **bad)) == fp.FP_ERR_ARG, bad
    assert call(*rope_args(fp, h, T=0)) == fp.FP_OK
    assert call(*rope_args(fp, h, Hq=0, Hkv=0)) == fp.FP_OK


KV_OK = dict(k=4096, v=8192, ks=None, vs=None, dtype=0, pages=8, page=16, Hkv=2, d=128)


@pytest.mark.parametrize("bad", [
    dict(k=None), dict(v=None), dict(k=4104), dict(v=8200), dict(dtype=2), dict(dtype=5), dict(dtype=3),
    dict(dtype=4, ks=16), dict(dtype=3, ks=16, vs=8), dict(ks=16), dict(pages=0), dict(pages=-1), dict(page=8),
    dict(page=48), dict(page=256), dict(Hkv=0), dict(Hkv=65536), dict(d=96), dict(d=256), dict(pages=1 << 27),
    dict(pages=1 << 40)], ids=str)
def test_kv_create_refuses(fp, bad):
    h = ctypes.c_void_p(1)
    assert fp.lib().fp_kv_create(*{**KV_OK, **bad}.values(), ctypes.byref(h)) == fp.FP_ERR_ARG
    assert h.value is None


def test_calls_refuse_null_handles(fp):
    L = fp.lib()
    assert L.fp_kv_create(*KV_OK.values(), None) == fp.FP_ERR_ARG
    assert L.fp_kv_write(None, 16, 128, 128, 16, 128, 128, 0, 1, 16, None) == fp.FP_ERR_ARG
    assert L.fp_kv_read(None, 16, 1, 16, None, 1, 1, 16, 128, 128, 16, 128, 128, 0, None) == fp.FP_ERR_ARG
    assert L.fp_tree_attn(None, 16, 128, 128, 0, 1, 4, 16, 1, 16, 16, 1, 1, None, 0.1, 16, 128, 128, None, 16, 1 << 30,
                          None) == fp.FP_ERR_ARG
    assert L.fp_rope_freqs(None, None) == fp.FP_ERR_ARG
    L.fp_rope_free(None)
    L.fp_kv_free(None)


@pytest.mark.parametrize("args", [(-1, 1, 4, 2, 128), (1, 0, 4, 2, 128), (1, 257, 4, 2, 128), (1, 1, 3, 2, 128),
                                  (1, 1, 0, 1, 128), (1, 1, 4, 0, 128), (1, 1, 4, 2, 96), (1, 1, 1024, 2, 128)])
def test_tree_workspace_refuses(fp, args):
    assert fp.lib().fp_tree_attn_workspace(*args) == 0
    with pytest.raises(fp.FpError):
        fp.fp_tree_attn_workspace(*args)


def test_error_code_has_a_message(fp):
    assert "range" in fp.fp_strerror(fp.FP_ERR_RANGE)


def test_binding_refuses_cpu_tensors(fp):
    import torch
    x = torch.zeros(2, 3, 128, dtype=torch.bfloat16)
    with pytest.raises(fp.FpError) as e:
        fp.Rope(128).apply(x, x, x, x, torch.zeros(3, dtype=torch.int32))
    assert e.value.code == fp.FP_ERR_ARG
    with pytest.raises(fp.FpError):
        fp.KvCache(torch.zeros(2, 2, 16, 128, dtype=torch.bfloat16), torch.zeros(2, 2, 16, 128, dtype=torch.bfloat16))
