"""fp_rope_apply on the GPU against the rotation in fp64.

Tolerance of one element, y = m (a cos x -+ b sin x), counted from the
arithmetic: the result is rounded once (half a step of its type), and before
that in fp32 the angle is off by at most 2^-25 half turns (pi 2^-25 radians),
sine and cosine by 2 units of 2^-24, the amplitude, the two products and the
sum by 2^-24 each: below 2^-21 of m (|a| + |b|) together.
"""
import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu

TYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}


@pytest.fixture(scope="module")
def fp():
    from dynamic_block_sparse_last_b200 import fp as mod
    assert torch.cuda.is_available(), "CUDA device required"
    return mod


def turned(x, pos, freqs, rot, layout, amp, inverse):
    """(exact result in fp64, |a| + |b| of each element's pair times amp)."""
    y = x.double()
    ang = pos.double()[:, None] * torch.from_numpy(freqs).to(x.device)
    c, s = amp * ang.cos(), amp * ang.sin() * (-1 if inverse else 1)
    out, size = y.clone(), y.abs() * 0
    h = rot // 2
    ia, ib = (slice(0, h), slice(h, rot)) if layout == 0 else (slice(0, rot, 2), slice(1, rot, 2))
    a, b = y[..., ia], y[..., ib]
    out[..., ia], out[..., ib] = a * c - b * s, b * c + a * s
    size[..., ia] = size[..., ib] = amp * (a.abs() + b.abs())
    return out, size


def check(got, x, pos, rope, amp, inverse):
    ref, size = turned(x, pos, rope.freqs(), rope.rot_dim, rope.layout, amp, inverse)
    bound = torch.finfo(got.dtype).eps / 2 * (ref.abs() + 2.0 ** -21 * size) + 2.0 ** -21 * size
    if got.dtype == torch.float16:
        bound = bound + 2.0 ** -25  # half a step of fp16's subnormals
    off = (got.double() - ref).abs()
    assert bool((off <= bound).all()), float((off - bound).max())
    assert torch.equal(got[..., rope.rot_dim:], x[..., rope.rot_dim:])


def rand(shape, dtype, seed):
    return torch.randn(shape, generator=torch.Generator("cuda").manual_seed(seed), device="cuda").to(dtype)


@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("layout", [0, 1])
@pytest.mark.parametrize("T,Hq,Hkv,d,rot", [(1, 1, 1, 64, 64), (3, 32, 8, 128, 128), (257, 5, 1, 128, 64), (64, 8, 2, 96, 32),
                                           (33, 3, 3, 80, 20), (7, 2, 1, 256, 256), (19, 1, 0, 512, 6), (5, 0, 4, 2, 2),
                                           (2000, 9, 3, 128, 96)])
def test_against_fp64(fp, dtype, layout, T, Hq, Hkv, d, rot):
    rope = fp.Rope(d, rot_dim=rot, layout=layout, theta=5e5)
    q = rand((Hq, T, d), TYPES[dtype], 1) if Hq else None
    k = rand((Hkv, T, d), TYPES[dtype], 2) if Hkv else None
    pos = torch.randint(0, 1 << 20, (T,), device="cuda", dtype=torch.int32)
    for inverse in (False, True):
        outs = [None if x is None else torch.full_like(x, float("nan")) for x in (q, k)]
        rope.apply(q, k, outs[0], outs[1], pos, inverse=inverse)
        for x, y in ((q, outs[0]), (k, outs[1])):
            if x is not None:
                check(y, x, pos, rope, 1.0, inverse)
    assert fp.fp_get_device_error() == fp.FP_OK


def test_far_and_negative_positions(fp):
    rope = fp.Rope(128, theta=1e4)
    edge = [0, 1, -1, 2 ** 31 - 1, -2 ** 31, 2 ** 30 + 7, 10 ** 9, -12345]
    pos = torch.tensor(edge, device="cuda", dtype=torch.int32)
    q = rand((2, len(edge), 128), torch.float32, 3)
    out = torch.empty_like(q)
    rope.apply(q, None, out, None, pos)
    # the fp64 angle of the oracle itself is off by up to 2^31 2^-53: taken in
    # exact integers instead, from the frequencies as fractions of a turn
    from decimal import Decimal, getcontext
    getcontext().prec = 60
    two_pi = Decimal("6.283185307179586476925286766559005768394338798750211641949889")
    turns = [[float((Decimal(p) * (Decimal(10000) ** (Decimal(-2 * i) / 128)) / two_pi) % 1) for i in range(64)] for p in edge]
    ang = torch.tensor(turns, device="cuda", dtype=torch.float64) * 2 * np.pi
    a, b = q.double()[..., :64], q.double()[..., 64:]
    ref = torch.cat([a * ang.cos() - b * ang.sin(), b * ang.cos() + a * ang.sin()], -1)
    size = (a.abs() + b.abs()).repeat(1, 1, 2)
    # 64-bit fixed point: |p| 2^-65 turns more, and 2^-32 turns where the top half is cut off
    assert bool(((out.double() - ref).abs() <= 2.0 ** -24 * ref.abs() + (2.0 ** -21 + 2.0 ** -29) * size).all())


@pytest.mark.parametrize("scaling,args", [(1, dict(factor=4.0)), (2, dict(factor=8.0)),
                                          (3, dict(factor=8.0, orig_len=8192.0, low=1.0, high=4.0)),
                                          (4, dict(factor=32.0, orig_len=4096.0, low=1.0, high=32.0, amplitude=1.3466))])
def test_scaled(fp, scaling, args):
    rope = fp.Rope(128, theta=1e4, scaling=scaling, **args)
    q, k = rand((4, 100, 128), torch.float32, 4), rand((2, 100, 128), torch.float32, 5)
    pos = torch.randint(0, 131072, (100,), device="cuda", dtype=torch.int32)
    qo, ko = torch.empty_like(q), torch.empty_like(k)
    rope.apply(q, k, qo, ko, pos)
    amp = float(np.float32(args.get("amplitude", 1.0)))
    check(qo, q, pos, rope, amp, False)
    check(ko, k, pos, rope, amp, False)


@pytest.mark.parametrize("layout", [0, 1])
@pytest.mark.parametrize("rot", [128, 64])
def test_strided_rows_in_place_and_untouched_neighbours(fp, layout, rot):
    """q and k as slices of fused token-major rows, rotated in place: equal to the
    contiguous call, and the value heads beside them are not written."""
    T, Hq, Hkv, d = 77, 6, 2, 128
    x = rand((T, Hq + 2 * Hkv, d), torch.bfloat16, 6)
    keep = x.clone()
    rope = fp.Rope(d, rot_dim=rot, layout=layout)
    pos = torch.randint(0, 4096, (T,), device="cuda", dtype=torch.int32)
    q, k = x[:, :Hq].transpose(0, 1), x[:, Hq:Hq + Hkv].transpose(0, 1)
    qc, kc = q.contiguous(), k.contiguous()
    qo, ko = torch.empty_like(qc), torch.empty_like(kc)
    rope.apply(qc, kc, qo, ko, pos)
    rope.apply(q, k, q, k, pos)
    assert torch.equal(q, qo) and torch.equal(k, ko)
    assert torch.equal(x[:, Hq + Hkv:], keep[:, Hq + Hkv:])


def test_rows_off_16_bytes_take_the_other_path_with_equal_results(fp):
    T, d = 40, 64
    x = rand((3, T, d + 2), torch.bfloat16, 7)
    q = x[..., 1:d + 1]                      # rows 2 bytes off, 132 bytes apart
    pos = torch.arange(T, device="cuda", dtype=torch.int32) + 1000
    rope = fp.Rope(d)
    a, b = torch.empty(3, T, d, device="cuda", dtype=torch.bfloat16), torch.empty(3, T, d, device="cuda", dtype=torch.bfloat16)
    rope.apply(q, None, a, None, pos)
    rope.apply(q.contiguous(), None, b, None, pos)
    assert torch.equal(a, b)


@pytest.mark.parametrize("layout", [0, 1])
def test_inverse_is_the_gradient(fp, layout):
    """sum(w * rope(x)) has the gradient rope^T w: against the formula's and against
    differences (the map is linear, so a difference of any step is exact up to rounding)."""
    T, H, d, rot = 9, 2, 64, 32
    rope = fp.Rope(d, rot_dim=rot, layout=layout, amplitude=1.25)
    x, w = rand((H, T, d), torch.float32, 8), rand((H, T, d), torch.float32, 9)
    pos = torch.randint(0, 10000, (T,), device="cuda", dtype=torch.int32)
    g = torch.empty_like(w)
    rope.apply(w, None, g, None, pos, inverse=True)
    check(g, w, pos, rope, 1.25, True)
    r = np.random.RandomState(0)
    for _ in range(20):
        h, t, i = r.randint(H), r.randint(T), r.randint(d)
        ys = []
        for step in (2.0, -2.0):
            z = x.clone()
            z[h, t, i] += step
            y = torch.empty_like(z)
            rope.apply(z, None, y, None, pos)
            ys.append(y)
        slope = float(((ys[0] - ys[1]).double() * w.double()).sum() / 4.0)
        # two outputs change; each is off by 2^-21 of its pair's size (below 2 * 10) and weighted by |w| < 6
        assert abs(slope - float(g[h, t, i])) < 2 * 2.0 ** -21 * 20 * 6


def test_agrees_with_the_pooling_epilogue(fp):
    """The same rotation as fp_rope_pool (fp32 tables of the same angles): at most one
    bf16 step apart, plus the tables' rounding."""
    S, Hq, Hkv, d = 300, 4, 2, 128
    q, k = rand((Hq, S, d), torch.bfloat16, 10), rand((Hkv, S, d), torch.bfloat16, 11)
    rope = fp.Rope(d, theta=5e5)
    ang = torch.arange(S, device="cuda").double()[:, None] * torch.from_numpy(rope.freqs()).cuda()
    n = -(-S // 128)
    outs = [torch.empty_like(q), torch.empty_like(k), torch.empty(Hq, n, d, device="cuda"), torch.empty(Hkv, n, d, device="cuda")]
    fp.fp_rope_pool(q, k, ang.cos().float().contiguous(), ang.sin().float().contiguous(), S, Hq, Hkv, d, 128, *outs)
    qo, ko = torch.empty_like(q), torch.empty_like(k)
    rope.apply(q, k, qo, ko, torch.arange(S, device="cuda", dtype=torch.int32))
    for x, a, b in ((q, qo, outs[0]), (k, ko, outs[1])):
        y = x.double().abs()
        size = (y[..., :64] + y[..., 64:]).repeat(1, 1, 2)
        assert bool(((a.double() - b.double()).abs() <= 2.0 ** -7 * a.double().abs() + 2.0 ** -20 * size).all())


def test_nan_and_infinity_stay_in_their_pair(fp):
    q = rand((1, 4, 64), torch.float32, 12)
    q[0, 1, 3] = float("nan")
    q[0, 2, 40] = float("inf")
    out = torch.empty_like(q)
    fp.Rope(64).apply(q, None, out, None, torch.arange(4, device="cuda", dtype=torch.int32))
    bad = ~torch.isfinite(out[0])
    want = torch.zeros_like(bad)
    want[1, [3, 35]] = True
    want[2, [8, 40]] = True
    assert torch.equal(bad, want)


def test_captured_and_replayed_with_new_positions(fp):
    rope = fp.Rope(128)
    q, pos = rand((4, 16, 128), torch.bfloat16, 13), torch.arange(16, device="cuda", dtype=torch.int32)
    out, eager = torch.empty_like(q), torch.empty_like(q)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        rope.apply(q, None, out, None, pos)
    for shift in (0, 500):
        pos.copy_(torch.arange(16, device="cuda", dtype=torch.int32) + shift)
        g.replay()
        rope.apply(q, None, eager, None, pos)
        assert torch.equal(out, eager)


def test_refusals_of_the_binding(fp):
    rope = fp.Rope(64)
    q, pos = rand((2, 8, 64), torch.bfloat16, 14), torch.zeros(8, device="cuda", dtype=torch.int32)
    out = torch.empty_like(q)
    for args in ((None, None, None, None, pos), (q, None, None, None, pos), (q, None, out, None, pos.long()),
                 (q, None, out, None, pos[:4]), (q, None, out.float(), None, pos), (q[..., :32], None, out, None, pos),
                 (q, None, out.transpose(0, 1), None, pos), (q.transpose(1, 2), None, out, None, pos),
                 (q.double(), None, out.double(), None, pos), (q, None, out, None, pos.cpu())):
        with pytest.raises(fp.FpError) as e:
            rope.apply(*args)
        assert e.value.code == fp.FP_ERR_ARG
