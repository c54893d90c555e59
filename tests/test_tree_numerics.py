"""fp_tree_attn where scores jump.

Tolerance: that of test_tree_attn.py without its share for probabilities that are small for fp16: those below
2^-14 of the largest carry no values here.
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
            out[h, at:at + n] = P @ vh
            bound[h, at:at + n] = (up + 2 * dS + (L / 16 + 400) * 2.0 ** -23) * A
            lse[h, at:at + n] = torch.where(some, torch.logsumexp(z, 1), torch.full_like(top[:, 0], -math.inf))
            lb[h, at:at + n] = dS[:, 0] + (L / 16 + 400) * 2.0 ** -23
    u = torch.finfo(c.dtype).eps / 2
    tiny = 2.0 ** -25 if c.dtype == torch.float16 else 2.0 ** -134
    bound = bound * (1 + u) + u * out.abs() + tiny
    return out, bound, lse, lb + 2.0 ** -22 * lse.abs().nan_to_num(0, 0, 0)


@pytest.mark.parametrize("kind,dtype", KINDS)
@pytest.mark.parametrize("n,g", ROWS)
@pytest.mark.parametrize("jump", [24.25, 26.0])
def test_scores_that_jump_after_a_plateau(fp, kind, dtype, n, g, jump):
    """Every 128 tokens: 32 low scores, 64 on a plateau of 13.875 (log2), then one far above it.  Only the plateau has values."""
    x = torch.zeros(512 + n)
    for a in range(0, 512, 128):
        x[a + 32:a + 96] = 13.875
        x[a + 96 + a // 16] = jump

    def values(s, m, Hkv, d):
        v = torch.zeros(m, Hkv, d, device="cuda")
        v[(x[:m] == 13.875).cuda()] = 1.0
        return v
    Pressed(kind, dtype, n, g, [x.tolist(), x[:128 + n].tolist()], values).check(fp)
