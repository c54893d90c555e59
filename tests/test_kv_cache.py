"""The paged key/value cache (fp_kv_write, fp_kv_read) on the GPU against its
definition in fp64.

For bf16 and fp16 rows the quotient c x / M is a ratio of two numbers of at most
18 and 11 bits, so no quotient but an exact tie lies within 2^-13 of the border
of two codes, relative to it, and the codes are compared exactly; for fp32 rows
they are compared with the fp32 quotient, which the definition names.  A value
read back is code * scale: half a step of its type, 2^-24 for the scale and
2^-24 for the product.
"""
import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu

TYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
CODES = {"int8": (torch.int8, 127.0), "e4m3": (torch.float8_e4m3fn, 448.0)}


@pytest.fixture(scope="module")
def fp():
    from dynamic_block_sparse_last_b200 import fp as mod
    assert torch.cuda.is_available(), "CUDA device required"
    return mod


def rand(shape, dtype, seed):
    g = torch.Generator("cuda").manual_seed(seed)
    x = torch.randn(shape, generator=g, device="cuda")
    return (x * torch.exp2(12 * torch.rand(shape[:-1] + (1,), generator=g, device="cuda") - 8)).to(dtype)


def pools(kind, pages, hkv, page, d):
    """Pools filled with a pattern that no write makes (bytes 0x5a, scales -7)."""
    if kind in CODES:
        dt = CODES[kind][0]
        p = [torch.full((pages, hkv, page, d), 0x5a, dtype=torch.uint8, device="cuda").view(dt) for _ in range(2)]
        return p + [torch.full((pages, hkv, page), -7.0, device="cuda") for _ in range(2)]
    return [torch.full((pages, hkv, page, 2 * d), 0x5a, dtype=torch.uint8, device="cuda").view(TYPES[kind])
            for _ in range(2)] + [None, None]


def raw(p):
    return p.view(torch.uint8)


def codes_of(x, kind, wide):
    """(codes as fp32, scale) of rows x; the quotient in fp64, or in fp32 when not wide."""
    dt, c = CODES[kind]
    y = x.double() if wide else x.float()
    M = y.abs().amax(-1, keepdim=True)
    z = torch.where(M > 0, c * y / M, torch.zeros_like(y))
    code = z.round() if kind == "int8" else z.to(dt)
    return code.float(), (M.double() / c).squeeze(-1)


@pytest.mark.parametrize("kind", ["int8", "e4m3", "bf16", "f16"])
@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("d,page,hkv,T", [(128, 16, 1, 1), (128, 64, 8, 333), (64, 32, 3, 130), (64, 128, 2, 64), (128, 128, 5, 65)])
def test_write(fp, kind, dtype, d, page, hkv, T):
    pages = -(-T // page) + 4
    p = pools(kind, pages, hkv, page, d)
    before = [raw(x).clone() for x in p[:2]]
    kv = fp.KvCache(*p)
    k, v = rand((hkv, T, d), TYPES[dtype], 1), rand((hkv, T, d), TYPES[dtype], 2)
    k[:, 0] = 0                                             # a row of zeros
    if T > 2:
        k[:, 1] = 0
        k[:, 1, 5] = 1.0                                    # a single value
        v[:, 2, ::2] = v[:, 2, 1:2] * 0.5                   # exact ties at half of the largest
    slots = torch.randperm(pages * page, device="cuda")[:T]
    kv.write(k, v, slots)
    pg, off = slots // page, slots % page
    for w, x in enumerate((k, v)):
        xt = x.transpose(0, 1)                              # [T, hkv, d]
        if kind in CODES:
            code, scale = codes_of(xt, kind, dtype != "f32")
            got = raw(p[w])[pg, :, off].view(CODES[kind][0]).float()
            assert torch.equal(got, code)
            gs = p[2 + w][pg, :, off].double()
            assert bool(((gs - scale.double()).abs() <= 2.0 ** -24 * scale.double()).all())
            other = torch.ones(pages, page, dtype=torch.bool, device="cuda")
            other[pg, off] = False
            assert bool((p[2 + w].transpose(1, 2)[other] == -7.0).all())
        else:
            got = raw(p[w])[pg, :, off].view(TYPES[kind])
            assert torch.equal(got, xt.to(TYPES[kind]))
        # nothing but the slots is written
        now = raw(p[w]).clone()
        now[pg, :, off] = before[w][pg, :, off]
        assert torch.equal(now, before[w])
    assert fp.fp_get_device_error() == fp.FP_OK


@pytest.mark.parametrize("kind", ["int8", "e4m3"])
def test_every_quotient_near_a_border(fp, kind):
    """Rows whose quotients run over the borders of all codes and one step of the input type to
    either side: where the division decides."""
    d = 128
    dt, c = CODES[kind]
    if kind == "int8":
        edge = torch.arange(-127, 127, dtype=torch.float64) + 0.5
    else:
        all_codes = torch.arange(0, 127, dtype=torch.uint8).view(dt).double()
        edge = (all_codes[1:] + all_codes[:-1]) / 2
    for M in (1.0, 127.0, 448.0, 3.0, 0.337890625, 5e-20, 6e20):
        x = (edge * M / c).float()
        x = torch.cat([x, torch.nextafter(x, x * 2), torch.nextafter(x, x * 0)])
        rows = []
        for i in range(0, len(x), d - 1):
            part = x[i:i + d - 1]
            rows.append(torch.cat([torch.tensor([M], dtype=torch.float32), part, torch.zeros(d - 1 - len(part))]))
        k = torch.stack(rows)[None].cuda()
        T = k.shape[1]
        p = pools(kind, 2, 1, 64, d)
        fp.KvCache(*p).write(k, None, torch.arange(T, device="cuda"))
        code, _ = codes_of(k.transpose(0, 1), kind, False)
        assert torch.equal(raw(p[0])[0, 0, :T].view(dt).float(), code[:, 0]), M


@pytest.mark.parametrize("kind", ["int8", "e4m3"])
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
def test_every_ratio_of_16_bit_mantissas(fp, kind, dtype):
    """All mantissas b over those of M (all of bf16's 128, 48 of fp16's 1024, the ones with the most borders
    among them), over the binades that reach a code other than 0: exact ties and all that is near one."""
    bits = {"bf16": 8, "f16": 11}[dtype]
    one = 1 << (bits - 1)
    tops = range(one, 2 * one)
    if dtype == "f16":
        tops = sorted({one, 2 * one - 1, 127 * 8 + 0, 127 * 16 - one, 254 * 8 // 2} | set(range(one, 2 * one, 23)))
        tops = [t for t in tops if one <= t < 2 * one]
    b = torch.arange(one, 2 * one, dtype=torch.float64)
    binades = range(0, 10 if kind == "int8" else 20)
    x = torch.cat([b * 2.0 ** -(k + bits - 1) for k in binades])     # below 2
    if dtype == "f16":
        x = x.half().double().unique()                              # fp16's subnormals repeat
    rows = []
    for a in tops:
        M = a / one
        y = x[x <= M]
        y = torch.cat([y, torch.zeros(-len(y) % 127)]).view(-1, 127)
        rows.append(torch.cat([torch.full((len(y), 1), M, dtype=torch.float64), y], 1))
    k = torch.cat(rows).to(TYPES[dtype])
    assert torch.equal(k.double(), torch.cat(rows))                 # the rows are what they are meant to be
    k = k.cuda()
    k[::2, 1:] *= -1
    T, page = len(k), 128
    pages = -(-T // page)
    p = pools(kind, pages, 1, page, 128)
    fp.KvCache(*p).write(k[None], None, torch.arange(T, device="cuda"))
    code, _ = codes_of(k, kind, True)
    assert torch.equal(raw(p[0]).view(-1, 128)[:T].view(CODES[kind][0]).float(), code)


def test_extreme_and_non_finite_rows(fp):
    d, page = 128, 16
    p = pools("int8", 1, 1, page, d)
    kv = fp.KvCache(*p)
    k = torch.randn(1, 8, d, device="cuda")
    k[0, 0] *= 3e38 / k[0, 0].abs().max()
    k[0, 1] *= 1e-37 / k[0, 1].abs().max()
    k[0, 2, 3] = float("nan")
    k[0, 3, 4] = float("inf")
    k[0, 4, 5] = -float("inf")
    kv.write(k, k, torch.arange(8, device="cuda"))
    out = torch.empty(1, 8, d, device="cuda")
    kv.read(torch.zeros(1, 1, dtype=torch.int32, device="cuda"), torch.tensor([0, 8], dtype=torch.int32, device="cuda"), out, None)
    assert bool(torch.isnan(out[0, 2:5]).all())
    fine = [0, 1, 5, 6, 7]
    M = k[0, fine].abs().amax(-1, keepdim=True).double()
    # half a code, and the roundings of scale and product (the smallest row's scale has 2^-149 steps)
    assert bool(((out[0, fine].double() - k[0, fine].double()).abs() <= M / 254 * (1 + 2.0 ** -20) + 127 * 2.0 ** -149).all())


@pytest.mark.parametrize("kind", ["int8", "e4m3"])
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
def test_non_finite_and_extreme_16_bit_rows(fp, kind, dtype):
    d, dt = 64, TYPES[dtype]
    top, low = (3e38, 1e-38) if dtype == "bf16" else (6e4, 2e-6)
    p = pools(kind, 1, 2, 16, d)
    kv = fp.KvCache(*p)
    k = rand((2, 9, d), torch.float32, 10)
    k[:, 0] *= top / k[:, 0].abs().amax(-1, keepdim=True)
    k[:, 1] *= low / k[:, 1].abs().amax(-1, keepdim=True)
    k = k.to(dt)
    k[0, 2, 63], k[1, 3, 0], k[0, 4, 17], k[1, 4, 18] = float("nan"), float("inf"), -float("inf"), float("nan")
    kv.write(k, k, torch.arange(9, device="cuda"))
    out = torch.empty(2, 9, d, device="cuda")
    kv.read(torch.zeros(1, 1, dtype=torch.int32, device="cuda"), torch.tensor([0, 9], dtype=torch.int32, device="cuda"), out, None)
    bad = ~torch.isfinite(k).all(-1)
    assert bool(torch.isnan(out[bad]).all()) and bool(torch.isfinite(out[~bad]).all())
    code, _ = codes_of(k.transpose(0, 1), kind, True)
    got = raw(p[0])[0].view(CODES[kind][0])[:, :9].float()
    assert torch.equal(got[~bad], code.transpose(0, 1)[~bad]) and float(got[bad].abs().max()) == 0


@pytest.mark.parametrize("kind", ["int8", "e4m3", "bf16", "f16"])
@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("d,page", [(128, 16), (64, 64), (128, 128)])
def test_read(fp, kind, dtype, d, page):
    """Ragged sequences (an empty one among them), from a start inside a page, with rows behind the last
    sequence left as they were."""
    hkv, lens, first = 3, [1, 0, 200, 63, 130], [5, 0, 0, 17, 100]
    width = max(-(-(a + b) // page) for a, b in zip(lens, first)) + 1
    pages = 5 * width
    p = pools(kind, pages, hkv, page, d)
    kv = fp.KvCache(*p)
    for w in range(2):
        if kind in CODES:
            raw(p[w]).copy_(torch.randint(0, 120, p[w].shape, device="cuda", dtype=torch.uint8))
            p[2 + w].copy_(torch.rand_like(p[2 + w]))
        else:
            p[w].copy_(torch.randn(p[w].shape, device="cuda"))
    table = torch.randperm(pages, device="cuda").to(torch.int32).view(5, width)
    cu = [0]
    for n in lens:
        cu.append(cu[-1] + n)
    T = cu[-1] + 9
    dt = TYPES[dtype]
    k = torch.full((T, hkv, d), 3.0, device="cuda", dtype=dt).transpose(0, 1)   # token-major
    v = torch.full((hkv, T, d), 3.0, device="cuda", dtype=dt)
    kv.read(table, torch.tensor(cu, dtype=torch.int32, device="cuda"), k, v,
            first=torch.tensor(first, dtype=torch.int32, device="cuda"))
    assert fp.fp_get_device_error() == fp.FP_OK
    for w, got in enumerate((k, v)):
        assert bool((got[:, cu[-1]:] == 3.0).all())
        for s, n in enumerate(lens):
            pos = torch.arange(n, device="cuda") + first[s]
            pg, off = table[s].long()[pos // page], pos % page
            ref = raw(p[w])[pg, :, off].view(p[w].dtype).double()
            if kind in CODES:
                ref = ref * p[2 + w][pg, :, off].double()[..., None]
            off_by = (got[:, cu[s]:cu[s + 1]].transpose(0, 1).double() - ref).abs()
            assert bool((off_by <= (torch.finfo(dt).eps / 2 + 2.0 ** -23) * ref.abs() + 2.0 ** -25 * (dt == torch.float16)).all())


def test_padding_bad_slots_and_bad_tables(fp):
    hkv, page, d, pages = 2, 16, 64, 4
    p = pools("bf16", pages, hkv, page, d)
    before = raw(p[0]).clone()
    kv = fp.KvCache(*p)
    k = rand((hkv, 5, d), torch.bfloat16, 3)
    kv.write(k, None, torch.tensor([-1, -2 ** 62, 3, -5, -1], device="cuda"))
    assert fp.fp_get_device_error() == fp.FP_OK
    now = raw(p[0]).clone()
    assert torch.equal(now.view(torch.bfloat16)[0, :, 3], k[:, 2])
    now[0, :, 3] = before[0, :, 3]
    assert torch.equal(now, before)
    assert torch.equal(raw(p[1]), before)                      # v was not given
    kv.write(k, None, torch.tensor([pages * page, 2 ** 62, pages * page - 1, -1, 2 ** 40], device="cuda"))
    assert fp.fp_get_device_error() == fp.FP_ERR_RANGE
    assert fp.fp_get_device_error() == fp.FP_OK
    assert torch.equal(p[0][pages - 1, :, page - 1], k[:, 2])
    # a page outside the cache, and positions behind the table or before its start
    out = torch.full((hkv, 40, d), 9.0, device="cuda", dtype=torch.bfloat16)
    table = torch.tensor([[0, pages], [-1, 1]], dtype=torch.int32, device="cuda")
    cu = torch.tensor([0, 20, 40], dtype=torch.int32, device="cuda")
    kv.read(table, cu, out, None)
    assert fp.fp_get_device_error() == fp.FP_ERR_RANGE
    assert torch.equal(out[:, :16], p[0][0]) and bool((out[:, 16:36] == 9.0).all())
    assert torch.equal(out[:, 36:], p[0][1, :, :4])
    out.fill_(9.0)
    kv.read(table[:1, :1].contiguous(), torch.tensor([0, 4], dtype=torch.int32, device="cuda"), out, None,
            first=torch.tensor([-2], dtype=torch.int32, device="cuda"))
    assert fp.fp_get_device_error() == fp.FP_ERR_RANGE
    assert bool((out[:, :2] == 9.0).all()) and torch.equal(out[:, 2:4], p[0][0, :, :2])
    kv.read(table[:1, :1].contiguous(), torch.tensor([0, 4], dtype=torch.int32, device="cuda"), out, None,
            first=torch.tensor([2 ** 31 - 2], dtype=torch.int32, device="cuda"))
    assert fp.fp_get_device_error() == fp.FP_ERR_RANGE


def test_pools_past_32_bits(fp):
    """Rows whose byte offset passes 2^32."""
    hkv, page, d = 8, 128, 128
    pages = (1 << 32) // (hkv * page * d) + 3
    pool = [torch.zeros(pages, hkv, page, d, dtype=torch.int8, device="cuda") for _ in range(2)]
    scale = [torch.zeros(pages, hkv, page, device="cuda") for _ in range(2)]
    kv = fp.KvCache(*pool, *scale)
    T = 200
    k, v = rand((hkv, T, d), torch.bfloat16, 4), rand((hkv, T, d), torch.bfloat16, 5)
    slots = pages * page - 1 - torch.arange(T, device="cuda")
    kv.write(k, v, slots)
    table = torch.tensor([[pages - 2, pages - 1]], dtype=torch.int32, device="cuda")
    ko, vo = torch.empty(hkv, 256, d, device="cuda"), torch.empty(hkv, 256, d, device="cuda")
    kv.read(table, torch.tensor([0, 256], dtype=torch.int32, device="cuda"), ko, vo)
    for x, y in ((k, ko), (v, vo)):
        code, s = codes_of(x.transpose(0, 1), "int8", True)
        ref = (code.double() * s.double()[..., None]).transpose(0, 1).flip(1)
        assert bool(((y[:, 56:].double() - ref).abs() <= 2.0 ** -22 * ref.abs()).all())
    assert float(pool[0][:pages - 2].view(-1)[:1 << 20].abs().max()) == 0
    assert fp.fp_get_device_error() == fp.FP_OK


def test_round_trip_into_a_prefill(fp):
    """What is read back has the layout that the packed prefill takes: the sparse prefill over K and V
    from the cache equals the one over the same values handed over directly."""
    lens, Hq, Hkv, d = [300, 129], 4, 2, 128
    T = sum(lens)
    q, k, v = (rand((h, T, d), torch.bfloat16, 6 + i) for i, h in enumerate((Hq, Hkv, Hkv)))
    k, v = k / 8, v / 8
    p = pools("e4m3", 12, Hkv, 64, d)
    kv = fp.KvCache(*p)
    table = torch.randperm(12, device="cuda")[:10].to(torch.int32).view(2, 5)
    pos = torch.cat([torch.arange(n, device="cuda") for n in lens])
    seq = torch.repeat_interleave(torch.arange(2, device="cuda"), torch.tensor(lens, device="cuda"))
    kv.write(k, v, table.long()[seq, pos // 64] * 64 + pos % 64)
    ko, vo = torch.empty_like(k), torch.empty_like(v)
    kv.read(table, torch.tensor([0, 300, 429], dtype=torch.int32, device="cuda"), ko, vo)
    direct = []
    for x in (k, v):
        code, s = codes_of(x.transpose(0, 1), "e4m3", True)
        direct.append((code.double() * s.double()[..., None]).float().to(torch.bfloat16).transpose(0, 1).contiguous())
    for got, want in ((ko, direct[0]), (vo, direct[1])):
        assert bool(((got.float() - want.float()).abs() <= 2.0 ** -7 * want.float().abs()).all())
    outs = []
    for kk, vv in ((ko, vo), direct):
        vl = fp.Varlen([0, 300, 429], Hq, Hkv, d, 128)
        vl.build_index(q, kk, 1.0, 0.1, fp.FP_QK_BF16)
        out = torch.empty_like(q)
        vl.sparse_attn(q, kk, vv, out)
        outs.append(out.float())
    torch.cuda.synchronize()
    # the operands differ by one bf16 step in at most a few places (2^-24 of scale and product before rounding)
    assert float((outs[0] - outs[1]).abs().max()) <= 2.0 ** -6 * float(outs[1].abs().max())


def test_refusals_of_the_binding(fp):
    p = pools("int8", 2, 2, 16, 64)
    kv = fp.KvCache(*p)
    k = rand((2, 4, 64), torch.bfloat16, 8)
    slots = torch.arange(4, device="cuda")
    for args in ((None, None, slots), (k[:1], None, slots), (k, None, slots.int()), (k, None, slots[:3]), (k, k.float(), slots),
                 (k.double(), None, slots), (k, None, slots.cpu()), (k.transpose(1, 2), None, slots)):
        with pytest.raises(fp.FpError):
            kv.write(*args)
    table, cu = torch.zeros(1, 1, dtype=torch.int32, device="cuda"), torch.tensor([0, 4], dtype=torch.int32, device="cuda")
    for args in ((table, cu, None, None), (table.long(), cu, k, None), (table, cu[:1], k, None), (table[0], cu, k, None),
                 (table, cu.long(), k, None)):
        with pytest.raises(fp.FpError):
            kv.read(*args)
    with pytest.raises(fp.FpError):
        fp.KvCache(p[0], p[1])                                  # int8 without scales
    with pytest.raises(fp.FpError):
        fp.KvCache(p[0], p[1], p[2][:1], p[3])
    x = rand((2, 5, 64), torch.bfloat16, 9).view(-1)[4:4 + 2 * 4 * 64].view(2, 4, 64)  # rows 8 bytes off
    with pytest.raises(fp.FpError):
        kv.write(x, None, slots)


@pytest.mark.parametrize("kind", ["int8", "bf16"])
def test_calls_without_tokens(fp, kind):
    """No tokens, as a step without new ones has it (empty tensors have no address): nothing happens."""
    hkv, d = 2, 64
    p = pools(kind, 2, hkv, 16, d)
    before = [raw(x).clone() for x in p[:2]]
    kv = fp.KvCache(*p)
    k = torch.empty(hkv, 0, d, device="cuda", dtype=torch.bfloat16)
    none = torch.empty(0, device="cuda")
    kv.write(k, k, none.long())
    kv.write(k, None, none.long())
    table, cu = torch.zeros(1, 1, dtype=torch.int32, device="cuda"), torch.zeros(2, dtype=torch.int32, device="cuda")
    kv.read(table, cu, k, k)
    kv.read(table, cu, None, k)
    kv.read(table[:0], cu[:1], rand((hkv, 3, d), torch.bfloat16, 11), None)
    q = torch.empty(4, 0, d, device="cuda", dtype=torch.bfloat16)
    pos = none.int()
    fp.Rope(d).apply(q, k, q, k, pos)
    work = torch.empty(fp.fp_tree_attn_workspace(1, 1, 4, hkv, d), dtype=torch.uint8, device="cuda")
    fp.fp_tree_attn(q, kv, table, cu[:1], cu, 1, torch.empty(0, 1, dtype=torch.int64, device="cuda"), 0.125, torch.empty_like(q), work,
                    lse=torch.empty(4, 0, device="cuda"))
    torch.cuda.synchronize()
    assert fp.fp_get_device_error() == fp.FP_OK
    assert all(torch.equal(raw(x), y) for x, y in zip(p[:2], before))
