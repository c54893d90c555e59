"""fp_tree_attn on the GPU against attention in fp64 over the same cached values.

Tolerance, counted from the arithmetic, with A = sum_p P_p |v_p| of an element
(P the exact probabilities, v the dequantised values):
  scores     a product of d terms accumulated in fp32 (each addition off by at
             most 2^-23 of the sum of magnitudes Z = scale sum_i |q_i k_i|),
             times scales and log2(e): dS = (d + 8) 2^-23 max Z, and 2^-22 for
             the exponential; a probability is off by 2 (dS + 2^-22) of itself,
             numerator and sum together
  products   probabilities are rounded to bf16 (2^-8; bf16 caches) or fp16
             (2^-11), over quantised caches after V's scale came in, off by 2^-25
             of the largest scale where they are too small for fp16
  sums       at most len / 16 + 400 additions in fp32, 2^-23 each
  result     half a step of its type.
"""
import math
import random

import pytest
import torch

pytestmark = pytest.mark.gpu

TYPES = {"bf16": torch.bfloat16, "f16": torch.float16}
CODES = {"int8": (torch.int8, 127.0), "e4m3": (torch.float8_e4m3fn, 448.0)}
KINDS = [("bf16", "bf16"), ("f16", "f16"), ("int8", "bf16"), ("int8", "f16"), ("e4m3", "bf16"), ("e4m3", "f16")]


@pytest.fixture(scope="module")
def fp():
    from dynamic_block_sparse_last_b200 import fp as mod
    assert torch.cuda.is_available(), "CUDA device required"
    return mod


class Case:
    """A cache with shuffled pages (unused slots hold NaN patterns), new tokens and masks."""

    def __init__(self, kind, dtype, d, page, Hkv, g, lens, news, masked=False, seed=0, size=1.0, max_q=None, masks=None):
        self.kind, self.dtype, self.d, self.page, self.Hkv, self.g = kind, TYPES[dtype], d, page, Hkv, g
        self.lens, self.news, self.Hq, self.B = lens, news, Hkv * g, len(lens)
        gen = torch.Generator("cuda").manual_seed(seed)
        width = max(1, max(-(-n // page) for n in lens)) + 1
        self.pages = self.B * width + 2
        order = torch.randperm(self.pages, generator=gen, device="cuda")
        self.table = order[:self.B * width].view(self.B, width).to(torch.int32).contiguous()
        shape = (self.pages, Hkv, page, d)
        self.pool, self.scale = [], []
        for _ in range(2):
            if kind in CODES:
                self.pool.append(torch.full(shape, 0x7f, dtype=torch.uint8, device="cuda").view(CODES[kind][0]))
                self.scale.append(torch.full(shape[:3], float("nan"), device="cuda"))
            else:
                self.pool.append(torch.full(shape, float("nan"), device="cuda", dtype=TYPES[kind]))
                self.scale.append(None)
        for s, n in enumerate(lens):
            p = torch.arange(n, device="cuda")
            pg, off = self.table[s].long()[p // page], p % page
            for w in range(2):
                x = size * torch.randn(n, Hkv, d, generator=gen, device="cuda")
                x = x * (0.25 + 2 * torch.rand(n, Hkv, 1, generator=gen, device="cuda"))
                self.put(w, pg, off, x)
        T = sum(news)
        self.T, self.max_q = T, max_q or max(1, max(news))
        self.cu = torch.tensor([sum(news[:i]) for i in range(len(news) + 1)], dtype=torch.int32, device="cuda")
        self.len = torch.tensor(lens, dtype=torch.int32, device="cuda")
        self.q = (2 * torch.randn(max(T, 1), self.Hq, d, generator=gen, device="cuda")).to(self.dtype)[:T].transpose(0, 1)
        self.bits = None
        if masked:
            r = random.Random(seed)
            self.bits = masks or [self.tree(n, r) for n in news]
            words = (self.max_q + 63) // 64
            rows = [[b >> 64 * k & (1 << 64) - 1 for k in range(words)] for seq in self.bits for b in seq]
            self.mask = torch.tensor([[x - (1 << 64) if x >> 63 else x for x in row] for row in rows], dtype=torch.int64).cuda()
        else:
            self.mask = None
        self.k_scale = d ** -0.5

    @staticmethod
    def tree(n, r):
        seen = []
        for i in range(n):
            up = r.randint(-1, i - 1) if i else -1
            seen.append((seen[up] if up >= 0 else 0) | 1 << i)
        return seen

    def put(self, w, pg, off, x):
        if self.kind in CODES:
            dt, c = CODES[self.kind]
            M = x.abs().amax(-1, keepdim=True)
            y = c * x / M
            code = (y.round() if self.kind == "int8" else y).to(dt)
            self.pool[w].view(torch.uint8)[pg, :, off] = code.contiguous().view(torch.uint8)
            self.scale[w][pg, :, off] = (M / c).squeeze(-1)
        else:
            self.pool[w][pg, :, off] = x.to(self.pool[w].dtype)

    def values(self, s, w):
        """fp64 values [len, Hkv, d] of sequence s."""
        p = torch.arange(self.lens[s], device="cuda")
        pg, off = self.table[s].long()[p // self.page], p % self.page
        x = self.pool[w].view(torch.uint8)[pg, :, off].view(self.pool[w].dtype).double()
        return x if self.scale[w] is None else x * self.scale[w][pg, :, off].double()[..., None]

    def visible(self, s):
        n, L = self.news[s], self.lens[s]
        vis = torch.ones(n, L, dtype=torch.bool)
        for i in range(n):
            for j in range(n):
                vis[i, L - n + j] = bool(self.bits[s][i] >> j & 1) if self.bits is not None else j <= i
        return vis.cuda()

    def reference(self):
        """out, its bound, lse, its bound: [Hq, T(, d)] in fp64."""
        out = torch.zeros(self.Hq, self.T, self.d, dtype=torch.float64, device="cuda")
        bound = torch.zeros_like(out)
        lse = torch.full((self.Hq, self.T), -math.inf, dtype=torch.float64, device="cuda")
        lb = torch.zeros_like(lse)
        up = 2.0 ** -8 if self.kind == "bf16" else 2.0 ** -11
        for s in range(self.B):
            n, L, c = self.news[s], self.lens[s], int(self.cu[s])
            if n == 0:
                continue
            k, v, vis = self.values(s, 0), self.values(s, 1), self.visible(s)
            some = vis.any(1)
            for h in range(self.Hq):
                kh, vh = k[:, h // self.g], v[:, h // self.g]
                q = self.q[h, c:c + n].double()
                z = (q @ kh.T) * self.k_scale
                size = (q.abs() @ torch.nan_to_num(kh, 0, 0, 0).abs().T * self.k_scale).masked_fill(~vis, 0).amax(1)
                z = z.masked_fill(~vis, -math.inf)
                top = z.amax(1, keepdim=True)
                e = torch.exp(z - torch.where(some[:, None], top, torch.zeros_like(top)))
                P = e / e.sum(1, keepdim=True)
                P = torch.where(vis & some[:, None], P, torch.zeros_like(P))
                # values that are not visible have no effect, NaN included
                finite = torch.isfinite(vh)
                o = P @ torch.where(finite, vh, torch.zeros_like(vh))
                A = P @ torch.where(finite, vh, torch.zeros_like(vh)).abs()
                dS = ((self.d + 8) * 2.0 ** -23 * size + 2.0 ** -22)[:, None]
                small = L * 2.0 ** -25 * torch.where(finite, vh, torch.zeros_like(vh)).abs().max() if self.kind != "bf16" else 0.0
                out[h, c:c + n] = o
                bound[h, c:c + n] = (up + 2 * dS + (L / 16 + 400) * 2.0 ** -23) * A + small
                lse[h, c:c + n] = torch.where(some, torch.logsumexp(z, 1), torch.full_like(top[:, 0], -math.inf))
                lb[h, c:c + n] = dS[:, 0] + (L / 16 + 400) * 2.0 ** -23
        u = torch.finfo(self.dtype).eps / 2
        bound = bound * (1 + u) + u * out.abs() + (2.0 ** -25 if self.dtype == torch.float16 else 0)
        return out, bound, lse, lb + 2.0 ** -22 * lse.abs().nan_to_num(0, 0, 0)

    def run(self, fp, work=None, out=None, lse=None, stream=None):
        kv = fp.KvCache(*self.pool, *self.scale)
        if work is None:
            work = torch.empty(fp.fp_tree_attn_workspace(self.B, self.max_q, self.Hq, self.Hkv, self.d), dtype=torch.uint8,
                               device="cuda").fill_(0xff)
        if out is None:
            out = torch.full((self.Hq, self.T, self.d), float("nan"), device="cuda", dtype=self.dtype)
        if lse is None:
            lse = torch.full((self.Hq, self.T), float("nan"), device="cuda")
        fp.fp_tree_attn(self.q, kv, self.table, self.len, self.cu, self.max_q, self.mask, self.k_scale, out, work, lse=lse,
                        stream=stream)
        return out, lse

    def check(self, fp, **kw):
        out, lse = self.run(fp, **kw)
        assert fp.fp_get_device_error() == fp.FP_OK
        ref, bound, rl, lb = self.reference()
        off = (out.double() - ref).abs()
        assert bool((off <= bound).all()), ("out", float((off - bound).nan_to_num(1e9).max()), float((off / bound).nan_to_num(1e9).max()))
        none = rl == -math.inf
        assert bool((lse[none] == -math.inf).all())
        lo = (lse.double() - rl).abs()[~none]
        assert bool((lo <= lb[~none]).all()), ("lse", float((lo / lb[~none]).nan_to_num(1e9).max()))
        return out, lse


@pytest.mark.parametrize("kind,dtype", KINDS)
@pytest.mark.parametrize("d,page", [(128, 16), (128, 64), (64, 32), (64, 128), (128, 128)])
def test_one_token(fp, kind, dtype, d, page):
    """The plain decode step: lengths of 1, around page and tile borders, long ones."""
    Case(kind, dtype, d, page, 2, 4, [1, 2, 15, 16, 17, 63, 64, 65, 128, 500, 1999], [1] * 11, seed=1).check(fp)


@pytest.mark.parametrize("kind,dtype", KINDS)
@pytest.mark.parametrize("g", [1, 3, 8, 32])
def test_group_sizes(fp, kind, dtype, g):
    Case(kind, dtype, 128, 32, 2, g, [300, 7, 1000], [1, 1, 1], seed=2).check(fp)


@pytest.mark.parametrize("kind,dtype", KINDS)
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("masked", [False, True])
def test_ragged_new_tokens(fp, kind, dtype, d, masked):
    """Sequences without new tokens among them, and one that is new from its first token on."""
    Case(kind, dtype, d, 64, 3, 2, [0, 70, 9, 640, 129, 33], [0, 5, 9, 0, 7, 1], masked=masked, seed=3).check(fp)


@pytest.mark.parametrize("kind,dtype", KINDS)
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("n,g", [(16, 2), (33, 1), (64, 4), (40, 8), (65, 3), (256, 1), (130, 5)])
def test_many_rows(fp, kind, dtype, d, n, g):
    """Row tiles of every size; masks of more than one word."""
    Case(kind, dtype, d, 64, 2, g, [n + 500, n, n + 77], [n, n, max(1, n // 3)], masked=True, seed=4).check(fp)


@pytest.mark.parametrize("kind,dtype", [("bf16", "bf16"), ("int8", "bf16"), ("e4m3", "f16")])
@pytest.mark.parametrize("n,g", [(1, 4), (7, 4), (64, 4)])
def test_long(fp, kind, dtype, n, g):
    """Few sequences, long enough to be split over all processors."""
    Case(kind, dtype, 128, 128, 2, g, [50001, 33], [n, min(n, 33)], masked=n > 1, seed=5).check(fp)


@pytest.mark.parametrize("kind,dtype", KINDS)
@pytest.mark.parametrize("g", [1, 4, 16])
def test_rows_that_see_nothing(fp, kind, dtype, g):
    """Empty masks with and without a prefix: 0 and -inf where nothing is left."""
    masks = [[0, 0b10, 0, 0b1000], [0, 0, 0b111], [0]]
    Case(kind, dtype, 128, 16, 2, g, [4, 40, 1], [4, 3, 1], masked=True, masks=masks, seed=6).check(fp)


@pytest.mark.parametrize("kind,dtype", KINDS)
@pytest.mark.parametrize("n,g", [(4, 2), (12, 2), (24, 4)])
def test_non_finite_values_in_masked_places(fp, kind, dtype, n, g):
    """NaN and infinities of one drafted token change only the rows that see it."""
    c = Case(kind, dtype, 128, 16, 2, g, [100 + n, n], [n, n], masked=True, seed=7,
             masks=[[1 << i for i in range(n)]] * 2)
    clean, clean_lse = c.check(fp)
    vis = torch.zeros(c.T, dtype=torch.bool, device="cuda")
    for s in range(2):
        pos = c.lens[s] - n + 1 + s                            # drafted token 1 + s: seen by itself only
        pg, off = int(c.table[s][pos // 16]), pos % 16
        for w in range(2):
            if kind in CODES:
                c.scale[w][pg, :, off] = float("nan")
            else:
                c.pool[w][pg, :, off, 3::5] = float("nan")
                c.pool[w][pg, :, off, 4::5] = float("inf")
                c.pool[w][pg, :, off, 5::5] = -float("inf")
        vis[s * n + 1 + s] = True
    out, lse = c.run(fp)
    assert torch.equal(out[:, ~vis], clean[:, ~vis]) and torch.equal(lse[:, ~vis], clean_lse[:, ~vis])
    assert bool(torch.isnan(out[:, vis]).all()) and bool(torch.isnan(lse[:, vis]).all())


@pytest.mark.parametrize("kind", ["bf16", "f16"])
@pytest.mark.parametrize("n,g", [(4, 2), (24, 4)])
def test_infinite_value_of_a_visible_drafted_token(fp, kind, n, g):
    c = Case(kind, kind, 64, 16, 1, g, [60 + n], [n], masked=True, seed=8, masks=[[1 << i for i in range(n)]])
    clean, _ = c.run(fp)
    pos = 60 + 2
    c.pool[1][int(c.table[0][pos // 16]), :, pos % 16, 7] = float("inf")
    c.pool[1][int(c.table[0][pos // 16]), :, pos % 16, 9] = -float("inf")
    out, _ = c.run(fp)
    want = clean.clone()
    want[:, 2, 7] = float("inf")
    want[:, 2, 9] = -float("inf")
    assert torch.equal(out, want)


@pytest.mark.parametrize("kind,dtype", KINDS)
@pytest.mark.parametrize("size", [1e-3, 30.0])
def test_sizes_of_values(fp, kind, dtype, size):
    """Scores that are all alike, and scores far apart; V scales over many binades."""
    c = Case(kind, dtype, 128, 64, 1, 4, [777, 130], [3, 1], seed=9, size=size)
    if kind in CODES:
        c.scale[1].mul_(torch.exp2(torch.randint(-6, 7, c.scale[1].shape, device="cuda").float()))
    c.check(fp)


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
def test_query_sizes_over_a_quantised_cache(fp, dtype):
    """Query rows far from 1, zero rows among them; bf16 ones beyond fp16's range, over keys that are nearly zero."""
    c = Case("int8", dtype, 128, 64, 2, 2, [200, 90], [5, 5], seed=10)
    f = [2.0 ** -12, 1.0, 0.0, 2.0, 2.0 ** -3] if dtype == "f16" else [2.0 ** -100, 2.0 ** 60, 0.0, 2.0 ** 58, 2.0 ** -20]
    c.q = (c.q.float() * torch.tensor(f * 2, device="cuda")[None, :, None]).to(c.dtype)
    if dtype == "bf16":
        c.scale[0].mul_(2.0 ** -60)
    c.check(fp)


def test_results_do_not_change_from_run_to_run(fp):
    for n, g in ((1, 4), (9, 3), (64, 4)):
        c = Case("e4m3", "bf16", 128, 64, 4, g, [20000, 300, 4500], [n] * 3, masked=n > 1, seed=11)
        a, la = c.run(fp)
        for _ in range(3):
            b, lb = c.run(fp)
            assert torch.equal(a, b) and torch.equal(la, lb)


def test_strides_and_rows_behind_the_last_sequence(fp):
    for n, g in ((3, 2), (20, 4)):
        c = Case("bf16", "bf16", 128, 16, 2, g, [150, 40], [n, n - 1], seed=12)
        dense, dl = c.run(fp)
        T = c.T + 5
        wide = torch.randn(T, c.Hq + 3, 160, device="cuda").to(torch.bfloat16)
        wide[:c.T, :c.Hq, :128] = c.q.transpose(0, 1)
        outw = torch.full((T, c.Hq, 136), 7.0, device="cuda", dtype=torch.bfloat16)
        lse = torch.full((c.Hq, T), 7.0, device="cuda")
        q, out = wide[:, :c.Hq, :128].transpose(0, 1), outw[:, :, :128].transpose(0, 1)
        kv = fp.KvCache(*c.pool, *c.scale)
        work = torch.empty(fp.fp_tree_attn_workspace(2, n, c.Hq, 2, 128), dtype=torch.uint8, device="cuda")
        fp.fp_tree_attn(q, kv, c.table, c.len, c.cu, n, None, c.k_scale, out, work, lse=lse)
        assert torch.equal(out[:, :c.T], dense) and torch.equal(lse[:, :c.T], dl)
        assert bool((outw[c.T:] == 7.0).all()) and bool((outw[:, :, 128:] == 7.0).all()) and bool((lse[:, c.T:] == 7.0).all())
        # without lse
        out2 = torch.empty_like(dense)
        fp.fp_tree_attn(c.q, kv, c.table, c.len, c.cu, n, None, c.k_scale, out2, work)
        assert torch.equal(out2, dense)


@pytest.mark.parametrize("n,g", [(2, 2), (20, 4)])
def test_bad_tables_are_not_followed(fp, n, g):
    def fresh():
        return Case("bf16", "bf16", 128, 16, 2, g, [100, 90, 80], [n, n, n], seed=13)

    c = fresh()
    good, _ = c.check(fp)
    width = c.table.shape[1]
    for change in (lambda c: c.len.__setitem__(1, n - 1), lambda c: c.len.__setitem__(1, -5),
                   lambda c: c.len.__setitem__(1, width * 16 + 1), lambda c: c.len.__setitem__(1, 2 ** 31 - 1),
                   lambda c: setattr(c, "max_q", n - 1) if n > 1 else None):
        c = fresh()
        change(c)
        left_out = [0, 1, 2] if c.max_q < n else [1]
        out = torch.full((c.Hq, c.T, 128), 5.0, device="cuda", dtype=torch.bfloat16)
        lse = torch.full((c.Hq, c.T), 5.0, device="cuda")
        c.run(fp, out=out, lse=lse)
        assert fp.fp_get_device_error() == fp.FP_ERR_RANGE
        for s in range(3):
            rows = slice(s * n, (s + 1) * n)
            assert bool((out[:, rows] == 5.0).all()) if s in left_out else torch.equal(out[:, rows], good[:, rows])
    for cu in ([0, n, 2 * n, 3 * n + 1], [0, n, n - 1, 2 * n - 1], [-1, n - 1, 2 * n - 1, 3 * n - 1]):
        c = fresh()
        c.cu = torch.tensor(cu, dtype=torch.int32, device="cuda")
        c.run(fp)
        assert fp.fp_get_device_error() == fp.FP_ERR_RANGE
    for bad in (c.pages, -1, 2 ** 31 - 1):
        c = fresh()
        c.table[1, 2] = bad
        out, _ = c.run(fp)
        assert fp.fp_get_device_error() == fp.FP_ERR_RANGE
        assert torch.equal(out[:, :n], good[:, :n]) and torch.equal(out[:, 2 * n:], good[:, 2 * n:])


@pytest.mark.parametrize("n,g", [(1, 4), (24, 4)])
def test_captured_and_replayed_with_new_lengths(fp, n, g):
    """A step captured once, replayed as the conversation grows; and two graphs with a workspace each."""
    c = Case("int8", "bf16", 128, 16, 2, g, [700, 300], [n, n], seed=14)
    work = [torch.empty(fp.fp_tree_attn_workspace(2, n, c.Hq, 2, 128), dtype=torch.uint8, device="cuda") for _ in range(2)]
    out = [torch.empty(c.Hq, c.T, 128, device="cuda", dtype=torch.bfloat16) for _ in range(2)]
    lse = [torch.empty(c.Hq, c.T, device="cuda") for _ in range(2)]
    graphs = []
    for i in range(2):
        g_ = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g_):
            c.run(fp, work=work[i], out=out[i], lse=lse[i])
        graphs.append(g_)
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for lens in ([700, 300], [699, n], [n + 130, 299]):
        c.lens = lens
        c.len.copy_(torch.tensor(lens, dtype=torch.int32))
        torch.cuda.synchronize()
        for _ in range(5):
            for i in range(2):
                with torch.cuda.stream(streams[i]):
                    graphs[i].replay()
        torch.cuda.synchronize()
        eager, el = c.check(fp)
        for i in range(2):
            assert torch.equal(out[i], eager) and torch.equal(lse[i], el)


def test_another_stream(fp):
    c = Case("bf16", "bf16", 128, 64, 2, 4, [5000], [4], seed=15)
    want, _ = c.run(fp)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        out, _ = c.run(fp)
    s.synchronize()
    assert torch.equal(out, want)
    out2, _ = c.run(fp, stream=s)      # named by argument; the buffers were made on the current stream
    torch.cuda.synchronize()
    assert torch.equal(out2, want)


@pytest.mark.parametrize("kind", ["bf16", "int8", "e4m3"])
def test_a_decode_step_end_to_end(fp, kind):
    """Rotate, write, attend: three conversations grow by drafted trees, as a serving loop does it, against
    the same in fp64 from the unrotated tokens."""
    torch.manual_seed(16)
    Hq, Hkv, d, page, lens, news = 8, 2, 128, 16, [50, 3, 200], [4, 1, 6]
    g = Hq // Hkv
    rope = fp.Rope(d, theta=5e5)
    shape = (40, Hkv, page, d)
    dt = torch.bfloat16 if kind == "bf16" else CODES[kind][0]
    pool = [torch.zeros(shape, dtype=torch.uint8 if kind != "bf16" else dt, device="cuda").view(dt) for _ in range(2)]
    scale = [torch.zeros(shape[:3], device="cuda") if kind != "bf16" else None for _ in range(2)]
    kv = fp.KvCache(*pool, *scale)
    table = torch.randperm(40, device="cuda")[:39].to(torch.int32).view(3, 13)

    def slots(first, count):
        pos = torch.cat([torch.arange(n, device="cuda") + f for f, n in zip(first, count)])
        seq = torch.repeat_interleave(torch.arange(3, device="cuda"), torch.tensor(count, device="cuda"))
        return pos.to(torch.int32), table.long()[seq, pos // page] * page + pos % page

    def rows(T):     # a fused projection's output
        return torch.randn(T, Hq + 2 * Hkv, d, device="cuda").to(torch.bfloat16)

    def heads(x):
        return x[:, :Hq].transpose(0, 1), x[:, Hq:Hq + Hkv].transpose(0, 1), x[:, Hq + Hkv:].transpose(0, 1)

    # the prompt
    x0, (pos0, sl0) = rows(sum(lens)), slots([0] * 3, lens)
    keep0 = x0.clone()
    _, k, v = heads(x0)
    rope.apply(None, k, None, k, pos0)
    kv.write(k, v, sl0)
    # the drafted trees: a token's position is its depth, its slot its place in the draft
    bits = [[1, 0b11, 0b101, 0b1011], [1], [1, 0b11, 0b111, 0b1001, 0b11001, 0b100001]]
    depth = [[bin(b).count("1") - 1 for b in seq] for seq in bits]
    x1 = rows(sum(news))
    keep1 = x1.clone()
    pos1 = torch.tensor([L + e for L, seq in zip(lens, depth) for e in seq], dtype=torch.int32, device="cuda")
    q, k, v = heads(x1)
    rope.apply(q, k, q, k, pos1)
    kv.write(k, v, slots(lens, news)[1])
    mask = torch.tensor([[b] for seq in bits for b in seq], dtype=torch.int64, device="cuda")
    total = [a + b for a, b in zip(lens, news)]
    cu = torch.tensor([0, 4, 5, 11], dtype=torch.int32, device="cuda")
    out = torch.empty(11, Hq, d, device="cuda", dtype=torch.bfloat16).transpose(0, 1)
    work = torch.empty(fp.fp_tree_attn_workspace(3, 6, Hq, Hkv, d), dtype=torch.uint8, device="cuda")
    fp.fp_tree_attn(q, kv, table, torch.tensor(total, dtype=torch.int32, device="cuda"), cu, 6, mask, d ** -0.5, out, work)
    assert fp.fp_get_device_error() == fp.FP_OK

    f = torch.from_numpy(rope.freqs()).cuda()

    def rot(x, pos):
        a = pos.double()[:, None, None] * f
        lo, hi = x[..., :64], x[..., 64:]
        return torch.cat([lo * a.cos() - hi * a.sin(), hi * a.cos() + lo * a.sin()], -1)

    for s in range(3):
        a, b = sum(lens[:s]), sum(news[:s])
        y0, y1 = keep0[a:a + lens[s]].double(), keep1[b:b + news[s]].double()
        kk = torch.cat([rot(y0[:, Hq:Hq + Hkv], pos0[a:a + lens[s]]), rot(y1[:, Hq:Hq + Hkv], pos1[b:b + news[s]])])
        vv = torch.cat([y0[:, Hq + Hkv:], y1[:, Hq + Hkv:]])
        qq = rot(y1[:, :Hq], pos1[b:b + news[s]])
        vis = torch.ones(news[s], total[s], dtype=torch.bool, device="cuda")
        for i in range(news[s]):
            for j in range(news[s]):
                vis[i, lens[s] + j] = bool(bits[s][i] >> j & 1)
        for h in range(Hq):
            z = (qq[:, h] @ kk[:, h // g].T * d ** -0.5).masked_fill(~vis, -math.inf)
            P = torch.softmax(z, 1)
            ref = P @ vv[:, h // g]
            # rotated q and k are rounded to bf16 (2^-8), k and v to codes: half a step of 1/127 of the row's
            # largest (int8) or 2^-4 of the value (e4m3); scores move by dz, probabilities by 2 dz of themselves
            zq = qq[:, h].abs() @ kk[:, h // g].abs().T * d ** -0.5
            kmax, vmax = kk[:, h // g].abs().amax(1), vv[:, h // g].abs().amax(1)
            ek = {"bf16": 0 * zq, "int8": (qq[:, h].abs().sum(1)[:, None] * kmax * d ** -0.5) / 254, "e4m3": zq * 2.0 ** -4}[kind]
            ev = {"bf16": 0, "int8": P @ (vmax / 254)[:, None].expand(-1, d), "e4m3": P @ vv[:, h // g].abs() * 2.0 ** -4}[kind]
            dz = (2 * 2.0 ** -8 * zq + ek).masked_fill(~vis, 0).amax(1)[:, None]
            A = P @ vv[:, h // g].abs()
            bound = (torch.expm1(2 * dz) + 2.0 ** -7) * A + ev * torch.exp(2 * dz) + 2.0 ** -8 * ref.abs() + 1e-5
            assert bool(((out[h, b:b + news[s]].double() - ref).abs() <= bound).all())


@pytest.mark.parametrize("kind,dtype", [("bf16", "bf16"), ("e4m3", "f16")])
@pytest.mark.parametrize("n,g,count,Hkv", [(1, 2, 700, 1), (2, 16, 130, 3), (20, 4, 170, 2), (64, 4, 40, 2)])
def test_more_sequences_than_processors(fp, kind, dtype, n, g, count, Hkv):
    """Several units to a CTA, more sequences than a block has threads, empty ones among them."""
    r = random.Random(19)
    news = [r.choice([0, n, n, max(1, n // 2)]) for _ in range(count)]
    lens = [m + r.choice([0, 3, 64, 130, 200]) for m in news]
    Case(kind, dtype, 64, 16, Hkv, g, lens, news, masked=n > 1, seed=19, max_q=n).check(fp)


@pytest.mark.parametrize("kind,dtype", [("f16", "f16"), ("int8", "bf16")])
@pytest.mark.parametrize("n,g", [(1, 4), (6, 4), (32, 4), (64, 4)])
def test_lengths_that_fill_their_tiles(fp, kind, dtype, n, g):
    Case(kind, dtype, 128, 128, 2, g, [64, 128, 256, 384, 1024], [n] * 5, masked=True, seed=20).check(fp)


@pytest.mark.parametrize("n,g", [(3, 4), (40, 2)])
def test_sequences_that_share_pages_and_masks_with_bits_past_the_draft(fp, n, g):
    """Two sequences over the same prefix pages give what they give over copies of them; bits of a mask
    from the draft's length on mean nothing."""
    c = Case("bf16", "bf16", 128, 16, 2, g, [160 + n, 160 + n], [n, n], masked=True, seed=21, max_q=64)
    for w in range(2):
        for p in range(10):
            c.pool[w][c.table[1, p].long()] = c.pool[w][c.table[0, p].long()]
    want, wl = c.check(fp)
    c.table[1, :10] = c.table[0, :10]
    c.mask = c.mask | (-1 << n)
    out, lse = c.run(fp)
    assert torch.equal(out, want) and torch.equal(lse, wl)


def test_cache_past_32_bits(fp):
    """Pages whose byte offset passes 2^32."""
    c = Case("int8", "bf16", 128, 128, 8, 2, [300], [2], seed=17)
    pages = (1 << 32) // (8 * 128 * 128) + 8
    pool = [torch.empty(pages, 8, 128, 128, dtype=torch.int8, device="cuda") for _ in range(2)]
    scale = [torch.empty(pages, 8, 128, device="cuda") for _ in range(2)]
    shift = pages - c.pages
    want, _ = c.run(fp)
    for w in range(2):
        pool[w][shift:] = c.pool[w]
        scale[w][shift:] = c.scale[w]
    c.pool, c.scale = pool, scale
    c.table += shift
    out, _ = c.run(fp)
    assert torch.equal(out, want)
    assert fp.fp_get_device_error() == fp.FP_OK


def test_refusals_of_the_binding(fp):
    c = Case("bf16", "bf16", 128, 16, 2, 2, [40], [2], masked=True, seed=18)
    kv = fp.KvCache(*c.pool)
    work = torch.empty(fp.fp_tree_attn_workspace(1, 2, 4, 2, 128), dtype=torch.uint8, device="cuda")
    out = torch.empty(4, 2, 128, device="cuda", dtype=torch.bfloat16)
    ok = dict(q=c.q, kv=kv, block_table=c.table, kv_len=c.len, cu_q=c.cu, max_q=2, mask=c.mask, scale=0.1, out=out, work=work)
    fp.fp_tree_attn(**ok)
    for bad in (dict(q=c.q.half()), dict(q=c.q[:3], out=out[:3]), dict(q=c.q[:, :1]), dict(out=out.float()), dict(out=out[:, :1]),
                dict(block_table=c.table.long()), dict(block_table=c.table[0]), dict(kv_len=c.len.long()), dict(cu_q=c.cu[:1]),
                dict(mask=c.mask.int()), dict(mask=c.mask[:1]), dict(max_q=0), dict(max_q=257), dict(max_q=100),
                dict(scale=float("nan")), dict(scale=0.0), dict(scale=-1.0), dict(scale=float("inf")), dict(work=work[:-256]), dict(work=work[8:]), dict(work=work.cpu()),
                dict(lse=torch.empty(4, 1, device="cuda")), dict(kv_len=c.len.cpu())):
        with pytest.raises(fp.FpError) as e:
            fp.fp_tree_attn(**{**ok, **bad})
        assert e.value.code == fp.FP_ERR_ARG, bad
    wide = torch.zeros(1, (1 << 26) + 1, dtype=torch.int32, device="cuda")
    with pytest.raises(fp.FpError):
        fp.fp_tree_attn(**{**ok, "block_table": wide})   # positions past 2^30
    h = fp.KvCache(c.pool[0].half(), c.pool[1].half())
    with pytest.raises(fp.FpError):
        fp.fp_tree_attn(**{**ok, "kv": h})          # bf16 queries over an fp16 cache
    torch.cuda.synchronize()
    assert fp.fp_get_device_error() == fp.FP_OK


@pytest.mark.parametrize("kind,dtype", [("bf16", "bf16"), ("e4m3", "f16")])
@pytest.mark.parametrize("n", [33, 47, 63, 65, 97, 127, 129, 161, 200, 255])
def test_rows_that_end_inside_a_warp(fp, kind, dtype, n):
    """Units whose last warp has rows for some of its lanes only, finished by one processor and split over several."""
    Case(kind, dtype, 128, 64, 1, 1, [n + 40, n + 3000], [n, n], masked=True, seed=22).check(fp)
