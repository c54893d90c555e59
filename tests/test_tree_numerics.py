"""fp_tree_attn where its 16-bit probabilities and fp32 sums are pressed: scores that jump, V rows of very
different sizes, values near the ends of their type, query rows of zeros.

Tolerance: that of test_tree_attn.py, with the error of small probabilities counted token by token.  A product
takes w = p (p times V's scale over a quantised cache) in 16 bits, and fp16 holds w to 2^-25 of the
unit it is taken in, which is set so that the row's largest w of the same processor is above 2^3: 2^-28 of that largest w.
P of a tile is rounded again when the unit moves, up to three times: 2^-26 for each visible token.  Tokens that are
not visible do not enter.
"""
import math

import pytest
import torch

from .test_tree_attn import CODES, KINDS, Case, fp  # noqa: F401

pytestmark = pytest.mark.gpu

# new tokens and query heads a KV head: each kernel form (up to 16, 32, 128 and 256 rows)
ROWS = [(4, 2), (12, 2), (32, 2), (64, 4)]


class Pressed(Case):
    """A case whose scores and values are given: every query row is its gain times the first unit vector, a cached key the
    score (in log2 units) times it."""

    def __init__(self, kind, dtype, n, g, scores, values, gains=(1.0, 0.5), masks=None, d=128, Hkv=1, news=None):
        """scores [B][len], values(s, len, Hkv, d) -> rows."""
        news = news or [n] * len(scores)
        super().__init__(kind, dtype, d, 16, Hkv, g, [len(x) for x in scores], news, masked=masks is not None, masks=masks)
        self.k_scale = math.log(2.0) / 8
        q = torch.zeros(self.T, self.Hq, d, device="cuda")
        r = torch.arange(self.T * self.Hq, device="cuda")
        q[..., 0] = 8 * torch.tensor(gains, device="cuda")[r % len(gains)].view(self.T, self.Hq)
        self.q = q.to(self.dtype).transpose(0, 1)
        for s, x in enumerate(scores):
            p = torch.arange(len(x), device="cuda")
            pg, off = self.table[s].long()[p // 16], p % 16
            k = torch.zeros(len(x), Hkv, d, device="cuda")
            k[..., 0] = torch.as_tensor(x, dtype=torch.float32, device="cuda")[:, None]
            self.put(0, pg, off, k)
            self.put(1, pg, off, values(s, len(x), Hkv, d))

    def put(self, w, pg, off, x):
        if self.kind in CODES and bool((x.abs().amax(-1) == 0).any()):
            x = x.clone()
            super().put(w, pg, off, torch.where((x.abs().amax(-1, keepdim=True) == 0), torch.ones_like(x), x))
            zero = x.abs().amax(-1) == 0
            code = self.pool[w].view(torch.uint8)[pg, :, off]
            code[zero] = 0
            self.pool[w].view(torch.uint8)[pg, :, off] = code
            sc = self.scale[w][pg, :, off]
            sc[zero] = 0
            self.scale[w][pg, :, off] = sc
        else:
            super().put(w, pg, off, x)

    def reference(self):
        return tight(self)


def tight(c):
    """out, its bound, lse, its bound: [Hq, T(, d)] in fp64."""
    out = torch.zeros(c.Hq, c.T, c.d, dtype=torch.float64, device="cuda")
    bound = torch.zeros_like(out)
    lse = torch.full((c.Hq, c.T), -math.inf, dtype=torch.float64, device="cuda")
    lb = torch.zeros_like(lse)
    up = 2.0 ** -8 if c.kind == "bf16" else 2.0 ** -11
    for s in range(c.B):
        n, L, at = c.news[s], c.lens[s], int(c.cu[s])
        if n == 0:
            continue
        k, v, vis = c.values(s, 0), c.values(s, 1), c.visible(s)
        some = vis.any(1)
        for h in range(c.Hq):
            kh, vh = k[:, h // c.g], v[:, h // c.g]
            q = c.q[h, at:at + n].double()
            z = (q @ kh.T) * c.k_scale
            size = (q.abs() @ kh.abs().T * c.k_scale).masked_fill(~vis, 0).amax(1)
            z = z.masked_fill(~vis, -math.inf)
            top = torch.where(some, z.amax(1), torch.zeros_like(z[:, 0]))[:, None]
            e = torch.exp(z - top)
            P = e / e.sum(1, keepdim=True).clamp(min=1e-300)
            A = P @ vh.abs()
            dS = ((c.d + 8) * 2.0 ** -23 * size + 2.0 ** -20)[:, None]
            if c.kind == "bf16":
                small = 0.0
            elif c.kind == "f16":
                small = 2.0 ** -26 * P.amax(1, keepdim=True) * (vis.double() @ vh.abs())
            else:
                small = 2.0 ** -26 * vis.sum(1, keepdim=True) * (P * vh.abs().amax(1)).amax(1, keepdim=True)
            out[h, at:at + n] = P @ vh
            bound[h, at:at + n] = (up + 2 * dS + (L / 16 + 400) * 2.0 ** -23) * A + small
            lse[h, at:at + n] = torch.where(some, torch.logsumexp(z, 1), torch.full_like(top[:, 0], -math.inf))
            lb[h, at:at + n] = dS[:, 0] + (L / 16 + 400) * 2.0 ** -23
    u = torch.finfo(c.dtype).eps / 2
    tiny = 2.0 ** -25 if c.dtype == torch.float16 else 2.0 ** -134
    bound = bound * (1 + u) + u * out.abs() + tiny
    bound[out.abs() + bound >= torch.finfo(c.dtype).max] = math.inf  # a result that the type does not hold is infinite
    return out, bound, lse, lb + 2.0 ** -22 * lse.abs().nan_to_num(0, 0, 0)


def normal(seed, size=1.0):
    def make(s, n, Hkv, d):
        g = torch.Generator("cuda").manual_seed(seed + s)
        return size * torch.randn(n, Hkv, d, generator=g, device="cuda")
    return make


@pytest.mark.parametrize("kind,dtype", KINDS)
@pytest.mark.parametrize("n,g", ROWS)
@pytest.mark.parametrize("plateau", [10.875, 13.875])
@pytest.mark.parametrize("jump", [24.25, 26.0, 31.5, 38.0])
def test_scores_that_jump_after_a_plateau(fp, kind, dtype, n, g, jump, plateau):
    """Every 128 tokens: 32 low scores, 64 on a plateau (log2), then one far above it.  Only the plateau has values
    in all columns but the last, where the others have theirs, so that the rows are alike in size."""
    x = torch.zeros(512 + n)
    for a in range(0, 512, 128):
        x[a + 32:a + 96] = plateau
        x[a + 96 + a // 16] = jump

    def values(s, m, Hkv, d):
        v = torch.zeros(m, Hkv, d, device="cuda")
        on = (x[:m] == plateau).cuda()
        v[on, :, :-1] = 1.0
        v[~on, :, -1] = 1.0
        return v
    Pressed(kind, dtype, n, g, [x.tolist(), x[:128 + n].tolist()], values).check(fp)


@pytest.mark.parametrize("kind,dtype", [("int8", "bf16"), ("e4m3", "bf16"), ("e4m3", "f16")])
@pytest.mark.parametrize("n,g", ROWS)
@pytest.mark.parametrize("size", [12, 22, 24, 30])
def test_hidden_values_of_any_size_have_no_effect(fp, kind, dtype, n, g, size):
    """A drafted token that only itself sees, its V row 2^size times the others': the other rows give what they give
    without it, and its own is right too."""
    masks = [[(1 << i) | (0 if i == 2 else 1) for i in range(n)]] * 2
    res = []
    for big in (0, size):
        c = Case(kind, dtype, 128, 16, 2, g, [70 + n, n], [n, n], masked=True, masks=masks, seed=31)
        for s in range(2):
            pos = c.lens[s] - n + 2
            c.scale[1][int(c.table[s][pos // 16]), :, pos % 16] *= 2.0 ** big
        c.reference = lambda c=c: tight(c)
        res.append(c.check(fp))
    other = [i for i in range(2 * n) if i % n != 2]
    assert torch.equal(res[0][0][:, other], res[1][0][:, other]) and torch.equal(res[0][1][:, other], res[1][1][:, other])


@pytest.mark.parametrize("kind,dtype", KINDS)
@pytest.mark.parametrize("n,g", ROWS)
def test_large_values_of_tokens_without_weight(fp, kind, dtype, n, g):
    """Small V rows carry the weight; beside them V rows 2^24 times as large (2^8 in fp16, which has no more) whose
    probability is 2^-100."""
    x = torch.zeros(300 + n)
    x[5::7] = -100.0
    far = 2.0 ** (8 if kind == "f16" else 24)

    def values(s, m, Hkv, d):
        v = 2.0 ** -6 * normal(41)(s, m, Hkv, d)
        v[5:300:7] *= far
        return v
    Pressed(kind, dtype, n, g, [x.tolist()], values, gains=(1.0,)).check(fp)


@pytest.mark.parametrize("kind,dtype", KINDS)
@pytest.mark.parametrize("n,g", ROWS)
@pytest.mark.parametrize("above", [18.25, 23.5])
def test_many_small_probabilities_beside_a_large_one(fp, kind, dtype, n, g, above):
    """Every eighth token takes nearly all of the weight and has no values: the others' probabilities are far below
    fp16's smallest normal number, and all of the result."""
    x = torch.zeros(2000 + n)
    x[::8] = above

    def values(s, m, Hkv, d):
        v = 1 + normal(51)(s, m, Hkv, d).abs()
        v[::8] = 0
        return 256 * v
    Pressed(kind, dtype, n, g, [x.tolist()], values, gains=(1.0, 0.875)).check(fp)


@pytest.mark.parametrize("n,g", ROWS)
@pytest.mark.parametrize("d", [64, 128])
def test_largest_bf16_values(fp, n, g, d):
    """V rows of up to 2^126 while the scores rise by 39 (log2) from tile to tile and within them: results that the type holds."""
    scores = []
    for s in range(40):
        x = torch.zeros(300 + n)
        x[40:] = 30.0
        x[100:] = 38.5
        x[200:] = 76.0
        scores.append(x.tolist())

    def values(s, m, Hkv, d):
        return 2.0 ** 126 * normal(61)(s, m, Hkv, d).clamp(-1, 1)
    c = Pressed("bf16", "bf16", n, g, scores, values, d=d, Hkv=8, gains=(1.0, 0.5, 0.25))
    c.check(fp)


@pytest.mark.parametrize("kind", ["int8", "e4m3"])
@pytest.mark.parametrize("n,g", ROWS)
@pytest.mark.parametrize("scale", [2.0 ** -30, 2.0 ** -100, 3e38])
def test_query_rows_of_zeros_and_scales_of_any_size(fp, kind, n, g, scale):
    """Rows of zeros see their tokens alike, whatever the scale is; masks hide some."""
    c = Case(kind, "bf16", 128, 16, 1, g, [90 + n, n], [n, n], masked=True, seed=71)
    c.q = torch.zeros_like(c.q)
    c.k_scale = scale
    c.reference = lambda: tight(c)
    c.check(fp)


@pytest.mark.parametrize("kind,dtype", KINDS)
@pytest.mark.parametrize("n,g", ROWS)
@pytest.mark.parametrize("size", [1.0, 30.0])
def test_long_caches_counted_token_by_token(fp, kind, dtype, n, g, size):
    """Ordinary and far-apart scores over a cache that all processors share, V scales over many binades."""
    c = Case(kind, dtype, 128, 64, 1, g, [20011, 300], [n, n - 1], masked=True, seed=81, size=size)
    if kind in CODES:
        c.scale[1].mul_(torch.exp2(torch.randint(-20, 7, c.scale[1].shape, device="cuda").float()))
    c.reference = lambda: tight(c)
    c.check(fp)


def test_a_workspace_for_the_longest_drafts_serves_shorter_ones(fp):
    for d in (64, 128):
        for g in (1, 3, 4, 16, 40, 256):
            size = 0
            for max_q in (1, 2, 4, 5, 8, 9, 16, 33, 64, 65, 256):
                now = fp.fp_tree_attn_workspace(3, max_q, 2 * g, 2, d)
                assert now >= size, (d, g, max_q)
                size = now
    c = Case("int8", "bf16", 128, 16, 2, 4, [300, 77], [1, 1], seed=91, max_q=1)
    work = torch.empty(fp.fp_tree_attn_workspace(2, 8, 8, 2, 128), dtype=torch.uint8, device="cuda")
    c.check(fp, work=work)


@pytest.mark.parametrize("kind", ["int8", "e4m3"])
@pytest.mark.parametrize("n,g", ROWS)
def test_largest_bf16_queries(fp, kind, n, g):
    """Query rows whose largest element is 2^127 or more, under a softmax scale that brings their scores back."""
    c = Case(kind, "bf16", 128, 16, 1, g, [90 + n, n], [n, n], masked=True, seed=101)
    c.q = (c.q.double() * 2.0 ** 125).clamp(-3.3e38, 3.3e38).to(torch.bfloat16)
    assert bool((c.q.float().abs().amax(-1) >= 2.0 ** 127).any())
    c.k_scale *= 2.0 ** -125
    c.reference = lambda: tight(c)
    c.check(fp)


@pytest.mark.parametrize("kind", ["int8", "e4m3"])
@pytest.mark.parametrize("n,g", ROWS)
@pytest.mark.parametrize("size", [-80, -60, 60, 80])
def test_v_scales_at_the_ends_of_their_range(fp, kind, n, g, size):
    """All V scales near 2^size, scores far apart: the results are those at 2^0, times 2^size."""
    c = Case(kind, "bf16", 128, 64, 1, g, [1500 + n, 200], [n, n - 1], masked=True, seed=111, size=3.0)
    for pool in c.scale[1:]:                     # powers of two, so that the results scale exactly
        pool.copy_(torch.exp2(torch.log2(pool).floor()).nan_to_num(1.0))
        pool.mul_(2.0 ** (size - math.log2(float(pool.min()))))
    c.reference = lambda: tight(c)
    c.check(fp)


@pytest.mark.parametrize("kind,dtype", [("bf16", "bf16"), ("int8", "bf16"), ("e4m3", "bf16")])
@pytest.mark.parametrize("n,g", ROWS)
def test_tokens_far_below_one_that_holds_zeros(fp, kind, dtype, n, g):
    """All of a result from probabilities of 2^-60, the likely tokens' V rows being zeros."""
    x = torch.zeros(700 + n)
    x[::9] = 60.0

    def values(s, m, Hkv, d):
        v = normal(121)(s, m, Hkv, d)
        v[::9] = 0
        return v
    Pressed(kind, dtype, n, g, [x.tolist()], values, gains=(1.0, 0.5)).check(fp)
