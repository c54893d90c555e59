"""What the serving operators compute and how they are called, case by case.

Three groups of operators that follow a prefill: rotary positions (``rope``),
the paged key/value cache that is quantised as it is written and read back
(``kv``), and the attention of drafted tokens over that cache (``tree``).  For
each case this file makes the inputs, runs one pass in the plain form (``own``
false: elementary torch operations in fp32, rounded once at the end) or through
the library (``own`` true), counts the work that the pass cannot do without,
and gives the exact result in fp64.

Formulas
  rope   pair (a, b) of one head at position p, frequency f_i, amplitude m:
         a' = m (a cos(p f_i) - b sin(p f_i)),  b' = m (b cos(p f_i) + a sin(p f_i));
         the inverse turns by -p f_i, which is the gradient of the forward call.
  kv     a row is one token's d values of one head: scale = max|x| / c with
         c = 127 (int8) or 448 (e4m3), code = round((c x) / max|x|), all codes 0
         for a row of zeros; read back as code * scale.  bf16 caches keep the row.
  tree   token i of a sequence with n new tokens and L cached ones (its own
         included) sees key p when p < L - n, or when bit p - (L - n) of its mask
         is set; out = softmax(scale q.k) v over those, lse = log sum exp.
"""
import math
import random

import torch

own = False

DT = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
CODE = {"int8": (torch.int8, 127.0), "e4m3": (torch.float8_e4m3fn, 448.0)}
SIZE = {"bf16": 2, "f16": 2, "f32": 4, "int8": 1, "e4m3": 1}


# ------------------------------------------------------------------ cases
def listed():
    return [
        # one decode step of a batch of 64 conversations: q and k are slices of the fused projection's rows
        {"name": "rope_step_64", "op": "rope", "tokens": 64, "hq": 32, "hkv": 8, "d": 128, "rot": 128, "dtype": "bf16",
         "layout": "half", "scaling": "bands", "inverse": False, "fused": True, "far": 131072},
        # the whole prompt of a 128K prefill, head-major as the sparse prefill reads it
        {"name": "rope_prompt_128k", "op": "rope", "tokens": 131072, "hq": 32, "hkv": 8, "d": 128, "rot": 128,
         "dtype": "bf16", "layout": "half", "scaling": "ramp", "inverse": False, "fused": False, "far": 131072},
        # the gradient of a partial, interleaved rotation of an odd number of fp32 training tokens
        {"name": "rope_grad_partial_4999", "op": "rope", "tokens": 4999, "hq": 16, "hkv": 4, "d": 128, "rot": 64,
         "dtype": "f32", "layout": "interleaved", "scaling": "none", "inverse": True, "fused": True, "far": 1000000},
        # a step that appends one to eight tokens for each of 64 sequences and reads them back
        {"name": "kv_step_int8_64", "op": "kv", "seqs": 64, "most": 8, "hkv": 8, "d": 128, "page": 16, "kind": "int8",
         "dtype": "bf16", "write": True, "read": True, "behind": 4096},
        # a ragged batch of prompts written to pages and read back for the next chunk's prefill
        {"name": "kv_prompt_e4m3_32k", "op": "kv", "seqs": 7, "most": 9000, "hkv": 8, "d": 128, "page": 64, "kind": "e4m3",
         "dtype": "bf16", "write": True, "read": True, "behind": 0},
        # an unquantised cache, written only: one odd fp16 prompt with 64-wide heads
        {"name": "kv_write_f16_16k", "op": "kv", "seqs": 1, "most": 16411, "hkv": 4, "d": 64, "page": 32, "kind": "f16",
         "dtype": "f16", "write": True, "read": False, "behind": 0},
        # a cached 128K prefix brought back for a re-prefill
        {"name": "kv_read_int8_128k", "op": "kv", "seqs": 1, "most": 131072, "hkv": 8, "d": 128, "page": 128, "kind": "int8",
         "dtype": "bf16", "write": False, "read": True, "behind": 0},
        # the smallest call: one token of one short conversation
        {"name": "tree_one_777", "op": "tree", "seqs": 1, "least": 777, "most": 777, "new": 1, "hq": 32, "hkv": 8, "d": 128,
         "page": 16, "kind": "bf16", "dtype": "bf16", "mask": False, "lse": False},
        # a decode batch of 64 ragged conversations over an int8 cache
        {"name": "tree_batch64_int8_16k", "op": "tree", "seqs": 64, "least": 100, "most": 16384, "new": 1, "hq": 32, "hkv": 8,
         "d": 128, "page": 64, "kind": "int8", "dtype": "bf16", "mask": False, "lse": True},
        # small trees of 7 drafted tokens over an fp16 cache with 64-wide heads, three query heads to a kv head
        {"name": "tree_draft7_f16_9k", "op": "tree", "seqs": 5, "least": 1000, "most": 9001, "new": 7, "hq": 12, "hkv": 4,
         "d": 64, "page": 32, "kind": "f16", "dtype": "f16", "mask": True, "lse": True},
        # trees of 16 drafted tokens for eight long conversations
        {"name": "tree_draft16_bf16_32k", "op": "tree", "seqs": 8, "least": 8000, "most": 32768, "new": 16, "hq": 32, "hkv": 8,
         "d": 128, "page": 64, "kind": "bf16", "dtype": "bf16", "mask": True, "lse": False},
        # one tree of 64 drafted tokens over a 128K fp8 cache
        {"name": "tree_draft64_e4m3_128k", "op": "tree", "seqs": 1, "least": 131072, "most": 131072, "new": 64, "hq": 32,
         "hkv": 8, "d": 128, "page": 128, "kind": "e4m3", "dtype": "bf16", "mask": True, "lse": True},
    ]


def _spread(rng, lo, hi):
    """A whole number from lo to hi, spread evenly over its logarithm."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.5)))))))


def draw(rng):
    op = rng.choice(["rope", "kv", "tree"])
    d = rng.choice([64, 128, 128])
    hkv = rng.choice([1, 2, 4, 8])
    if op == "rope":
        hq = hkv * rng.randint(1, 8 if hkv < 8 else 4)
        rot = rng.choice([d, d, d // 2, d // 4])
        dtype = rng.choice(["bf16", "bf16", "f16", "f32"])
        most = max(1, int(131072 * 40 * 256 / ((hq + hkv) * d * SIZE[dtype])))
        return {"op": "rope", "tokens": _spread(rng, 1, min(131072, most)), "hq": hq, "hkv": hkv, "d": d, "rot": rot,
                "dtype": dtype, "layout": rng.choice(["half", "interleaved"]),
                "scaling": rng.choice(["none", "linear", "base", "bands", "ramp"]), "inverse": rng.random() < 0.3,
                "fused": rng.random() < 0.5, "far": rng.choice([8192, 131072, 1000000])}
    kind = rng.choice(["int8", "e4m3", "bf16", "f16"])
    dtype = kind if kind in DT else rng.choice(["bf16", "f16"])
    page = rng.choice([16, 32, 64, 128])
    if op == "kv":
        seqs = _spread(rng, 1, 64)
        most = _spread(rng, 1, max(1, 131072 // seqs))
        write = rng.random() < 0.7
        return {"op": "kv", "seqs": seqs, "most": most, "hkv": hkv, "d": d, "page": page, "kind": kind, "dtype": dtype,
                "write": write, "read": not write or kind in CODE or rng.random() < 0.5, "behind": rng.choice([0, 0, 333])}
    seqs = _spread(rng, 1, 64)
    hq = hkv * rng.randint(1, 8 if hkv < 8 else 4)
    new = _spread(rng, 1, 64)
    most = _spread(rng, max(64, new), max(64, new, min(131072, 400000 // seqs, 134217728 * 2 // (seqs * hq * new))))
    return {"op": "tree", "seqs": seqs, "least": max(new, most // rng.choice([1, 4, 40])), "most": most, "new": new,
            "hq": hq, "hkv": hkv, "d": d, "page": page, "kind": kind, "dtype": dtype,
            "mask": new > 1 and rng.random() < 0.7, "lse": rng.random() < 0.5}


# ------------------------------------------------------------------ inputs
def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _scaling(c):
    """Frequency scaling: (kind, base, factor, original length, low, high, amplitude)."""
    return {"none": (10000.0, 1.0, 0.0, 0.0, 0.0, 1.0), "linear": (10000.0, 4.0, 0.0, 0.0, 0.0, 1.0),
            "base": (10000.0, 8.0, 0.0, 0.0, 0.0, 1.0), "bands": (500000.0, 8.0, 8192.0, 1.0, 4.0, 1.0),
            "ramp": (10000.0, 32.0, 4096.0, 1.0, 32.0, 0.1 * math.log(32.0) + 1.0)}[c["scaling"]]


def _rope_inputs(c, seed):
    g = _gen(seed)
    T, hq, hkv, d, dt = c["tokens"], c["hq"], c["hkv"], c["d"], DT[c["dtype"]]
    if c["fused"]:  # rows of the fused projection: q, k and v heads of a token side by side
        x = torch.randn(T, hq + 2 * hkv, d, generator=g, device="cuda").to(dt)
        q, k = x[:, :hq].transpose(0, 1), x[:, hq:hq + hkv].transpose(0, 1)
    else:
        q = torch.randn(hq, T, d, generator=g, device="cuda").to(dt)
        k = torch.randn(hkv, T, d, generator=g, device="cuda").to(dt)
    if T > 1024 and not c["fused"]:  # one prompt from a random start
        start = torch.randint(0, max(1, c["far"] - T + 1), (1,), generator=g, device="cuda", dtype=torch.int32)
        pos = torch.arange(T, device="cuda", dtype=torch.int32) + start
    else:
        pos = torch.randint(0, c["far"], (T,), generator=g, device="cuda", dtype=torch.int32)
    return {"case": c, "q": q, "k": k, "pos": pos.to(torch.int32),
            "q_out": torch.empty(hq, T, d, device="cuda", dtype=dt), "k_out": torch.empty(hkv, T, d, device="cuda", dtype=dt)}


def _lengths(n, lo, hi, salt):
    """n lengths from lo to hi, the first of them hi: the same for every seed, so that outputs keep their shape."""
    r = random.Random(salt)
    return [hi] + [r.randint(lo, hi) for _ in range(n - 1)]


def _kv_lengths(c):
    return _lengths(c["seqs"], max(1, c["most"] // 4), c["most"], 1)


def _tree_lengths(c):
    """(new tokens, cached tokens) of the sequences."""
    n = _lengths(c["seqs"], (c["new"] + 1) // 2 if c["mask"] else c["new"], c["new"], 2)
    return n, [max(a, b) for a, b in zip(_lengths(c["seqs"], c["least"], c["most"], 3), n)]


def _on_gpu(x):
    return torch.tensor(x, dtype=torch.int64).cuda()


def _table(lens, page, g):
    """A block table of shuffled pages for sequences of these lengths, and the number of pages."""
    need = (lens + page - 1) // page
    width = int(need.max())
    pages = int(need.sum()) + 3
    order = torch.randperm(pages, generator=g, device="cuda")
    at = torch.cumsum(need, 0) - need
    col = torch.arange(width, device="cuda")
    idx = (at[:, None] + col).clamp(max=pages - 1)
    return torch.where(col < need[:, None], order[idx], torch.zeros_like(idx)).to(torch.int32).contiguous(), pages


def _cu(n):
    return torch.cat([torch.zeros(1, device="cuda", dtype=torch.int64), torch.cumsum(n, 0)]).to(torch.int32)


def _pools(pages, hkv, page, d, kind):
    if kind in CODE:
        return ([torch.zeros(pages, hkv, page, d, device="cuda", dtype=CODE[kind][0]) for _ in range(2)]
                + [torch.zeros(pages, hkv, page, device="cuda") for _ in range(2)])
    return [torch.zeros(pages, hkv, page, d, device="cuda", dtype=DT[kind]) for _ in range(2)] + [None, None]


def _encode(x, kind):
    """Codes and scales of the rows of x (fp32)."""
    dt, c = CODE[kind]
    big = x.abs().amax(-1, keepdim=True)
    y = torch.where(big > 0, c * x / big, torch.zeros_like(x))
    return (y.round() if kind == "int8" else y).to(dt), (big / c).squeeze(-1)


def _fill(pool, scale, kind, g, spread):
    """Rows as a model leaves them: normal values, the size varying from token to token."""
    at = list(range(0, pool.shape[0], max(1, (1 << 25) // pool[0].numel()))) + [pool.shape[0]]
    for a, b in zip(at, at[1:]):
        part = pool[a:b]
        x = torch.randn(part.shape, generator=g, device="cuda") * (1 + spread * torch.rand(part.shape[:3], generator=g, device="cuda")[..., None])
        if kind in CODE:
            code, s = _encode(x, kind)
            part.view(torch.int8).copy_(code.view(torch.int8))
            scale[a:b].copy_(s)
        else:
            part.copy_(x)


def _kv_inputs(c, seed):
    g = _gen(seed)
    counts = _kv_lengths(c)
    n, T = _on_gpu(counts), sum(counts)
    first = (torch.rand(c["seqs"], generator=g, device="cuda") * (c["behind"] + 1)).floor().to(torch.int64)
    table, pages = _table(first + n, c["page"], g)
    cu = _cu(n)
    st = {"case": c, "table": table, "cu": cu, "first": first.to(torch.int32)}
    st["pools"] = _pools(pages, c["hkv"], c["page"], c["d"], c["kind"])
    dt = DT[c["dtype"]]
    if c["write"]:
        seq = torch.repeat_interleave(torch.arange(c["seqs"], device="cuda"), n)
        p = torch.arange(T, device="cuda") - cu.long()[seq] + first[seq]
        st["slots"] = table.long()[seq, p // c["page"]] * c["page"] + p % c["page"]
        size = 0.25 + 4 * torch.rand(T, 1, 1, generator=g, device="cuda")
        x = (torch.randn(T, 2 * c["hkv"], c["d"], generator=g, device="cuda") * size).to(dt)
        st["k"], st["v"] = x[:, :c["hkv"]].transpose(0, 1), x[:, c["hkv"]:].transpose(0, 1)
    else:
        for i in range(2):
            _fill(st["pools"][i], st["pools"][2 + i], c["kind"], g, 3.0)
    if c["read"]:
        st["k_out"] = torch.empty(c["hkv"], T, c["d"], device="cuda", dtype=dt)
        st["v_out"] = torch.empty(c["hkv"], T, c["d"], device="cuda", dtype=dt)
    return st


def _tree_words(news, most, seed):
    """Random trees: every drafted token hangs on an earlier one or on the prefix; bit j of row i: token i sees token j."""
    r, words = random.Random(seed), (most + 63) // 64
    rows = []
    for n in news:
        seen = []
        for i in range(n):
            up = r.randint(-1, i - 1) if i else -1
            seen.append((seen[up] if up >= 0 else 0) | 1 << i)
        for bits in seen:
            w = [bits >> 64 * k & (1 << 64) - 1 for k in range(words)]
            rows.append([x - (1 << 64) if x >> 63 else x for x in w])
    return torch.tensor(rows, dtype=torch.int64).cuda()


def _tree_inputs(c, seed):
    g = _gen(seed)
    counts, cached = _tree_lengths(c)
    n, lens, T = _on_gpu(counts), _on_gpu(cached), sum(counts)
    table, pages = _table(lens, c["page"], g)
    cu = _cu(n)
    st = {"case": c, "table": table, "cu": cu, "len": lens.to(torch.int32), "T": T}
    st["pools"] = _pools(pages, c["hkv"], c["page"], c["d"], c["kind"])
    for i in range(2):
        _fill(st["pools"][i], st["pools"][2 + i], c["kind"], g, 1.0)
    dt = DT[c["dtype"]]
    st["q"] = (2 * torch.randn(T, c["hq"], c["d"], generator=g, device="cuda")).to(dt).transpose(0, 1)
    st["out"] = torch.empty(T, c["hq"], c["d"], device="cuda", dtype=dt).transpose(0, 1)
    st["lse"] = torch.empty(c["hq"], T, device="cuda") if c["lse"] else None
    st["mask"] = _tree_words(counts, c["new"], seed) if c["mask"] else None
    return st


def prepare(case, seed):
    st = {"rope": _rope_inputs, "kv": _kv_inputs, "tree": _tree_inputs}[case["op"]](case, seed)
    if own:  # the handles and the workspace that a serving program makes once
        from dynamic_block_sparse_last_b200 import fp
        if case["op"] == "rope":
            base, factor, length, low, high, amp = _scaling(case)
            kinds = {"none": fp.FP_ROPE_NONE, "linear": fp.FP_ROPE_LINEAR, "base": fp.FP_ROPE_BASE,
                     "bands": fp.FP_ROPE_BANDS, "ramp": fp.FP_ROPE_RAMP}
            st["rope"] = fp.Rope(case["d"], rot_dim=case["rot"], theta=base, scaling=kinds[case["scaling"]], factor=factor,
                                 orig_len=length, low=low, high=high, amplitude=amp,
                                 layout=fp.FP_ROPE_HALF if case["layout"] == "half" else fp.FP_ROPE_INTERLEAVED)
        else:
            st["kv"] = fp.KvCache(*st["pools"])
            if case["op"] == "tree":
                size = fp.fp_tree_attn_workspace(case["seqs"], case["new"], case["hq"], case["hkv"], case["d"])
                st["work"] = torch.empty(size, device="cuda", dtype=torch.uint8)
    return st


# ------------------------------------------------------------------ the plain form and the library's calls
def _freqs(c):
    """The rot/2 frequencies of a case, fp64."""
    base, factor, length, low, high, _ = _scaling(c)
    rot = c["rot"]
    i = torch.arange(rot // 2, device="cuda", dtype=torch.float64)
    if c["scaling"] == "base":
        base = base * factor ** (rot / (rot - 2))
    f = base ** (-2 * i / rot)
    if c["scaling"] == "linear":
        return f / factor
    if c["scaling"] == "bands":  # by the turns that a frequency makes within the original length
        keep = ((length * f / (2 * math.pi) - low) / (high - low)).clamp(0, 1)
        return f * keep + f / factor * (1 - keep)
    if c["scaling"] == "ramp":  # by the index, between those that make `high` and `low` turns
        at = [rot * math.log(length / (2 * math.pi * t)) / (2 * math.log(base)) for t in (high, low)]
        a, b = max(math.floor(at[0]), 0), min(math.ceil(at[1]), rot - 1)
        away = ((i - a) / max(b - a, 0.001)).clamp(0, 1)
        return f * (1 - away) + f / factor * away
    return f


def _rope_plain(st):
    c = st["case"]
    rot, amp = c["rot"], _scaling(c)[5]
    angle = st["pos"].double()[:, None] * _freqs(c)
    cos, sin = (amp * angle.cos()).float(), (amp * angle.sin() * (-1 if c["inverse"] else 1)).float()
    got = []
    for x in (st["q"], st["k"]):
        y = x.float()
        if c["layout"] == "half":
            a, b = y[..., :rot // 2], y[..., rot // 2:rot]
        else:
            a, b = y[..., :rot:2], y[..., 1:rot:2]
        turned = (a * cos - b * sin, b * cos + a * sin)
        turned = torch.cat(turned, -1) if c["layout"] == "half" else torch.stack(turned, -1).flatten(-2)
        got.append(torch.cat([turned, y[..., rot:]], -1).to(x.dtype))
    return got


def _rows_of(pool, scale, page, off):
    """fp32 values of the cache rows (page, off), which may have any shape: [..., heads, d]."""
    x = pool.view(torch.int8)[page, :, off].view(pool.dtype).float()
    return x if scale is None else x * scale[page, :, off][..., None]


def _kv_plain(st):
    c, pools = st["case"], st["pools"]
    if c["write"]:
        page, off = st["slots"] // c["page"], st["slots"] % c["page"]
        for i, x in enumerate((st["k"], st["v"])):
            x = x.transpose(0, 1)
            if c["kind"] in CODE:
                x, pools[2 + i][page, :, off] = _encode(x.float(), c["kind"])
            pools[i].view(torch.int8)[page, :, off] = x.contiguous().view(torch.int8)
    if not c["read"]:
        return pools[:2]
    cu = st["cu"].long()
    n = cu[1:] - cu[:-1]
    T = st["k_out"].shape[1]
    seq = torch.repeat_interleave(torch.arange(c["seqs"], device="cuda"), n, output_size=T)
    p = torch.arange(T, device="cuda") - cu[seq] + st["first"].long()[seq]
    page = st["table"].long()[seq, p // c["page"]]
    for i, o in enumerate((st["k_out"], st["v_out"])):
        o.copy_(_rows_of(pools[i], pools[2 + i], page, p % c["page"]).transpose(0, 1))
    return [st["k_out"], st["v_out"]]


def _tree_plain(st):
    c, pools = st["case"], st["pools"]
    B, N, hkv, d, g, T = c["seqs"], c["new"], c["hkv"], c["d"], c["hq"] // c["hkv"], st["T"]
    cu, lens = st["cu"].long(), st["len"].long()
    n = cu[1:] - cu[:-1]
    L = c["most"]
    p = torch.arange(L, device="cuda")
    page = st["table"].long()[:, (p // c["page"]).clamp(max=st["table"].shape[1] - 1)]
    k = _rows_of(pools[0], pools[2], page, (p % c["page"]).expand(B, L))        # [B, L, hkv, d]
    v = _rows_of(pools[1], pools[3], page, (p % c["page"]).expand(B, L))
    i = torch.arange(N, device="cuda")
    row = (cu[:-1, None] + i).clamp(max=T - 1)                                   # [B, N] packed rows
    q = st["q"].float().transpose(0, 1)[row].view(B, N, hkv, g, d)
    j = p[None] - (lens - n)[:, None]                                            # [B, L] index among the new tokens
    if st["mask"] is None:
        own_part = j[:, None] <= i[:, None]
    else:
        jj = j.clamp(0, N - 1)
        words = st["mask"][row]                                                  # [B, N, W]
        own_part = (torch.gather(words, 2, (jj >> 6)[:, None].expand(B, N, L)) >> (jj & 63)[:, None]) & 1 > 0
    seen = ((j < 0)[:, None] | own_part) & (p[None] < lens[:, None])[:, None]    # [B, N, L]
    s = torch.matmul(q.permute(0, 2, 3, 1, 4).reshape(B, hkv, g * N, d), k.permute(0, 2, 3, 1)) * d ** -0.5
    s = s.view(B, hkv, g, N, L).masked_fill_(~seen[:, None, None], -math.inf)
    top = s.amax(-1, keepdim=True)
    e = torch.exp(s - torch.where(top == -math.inf, torch.zeros_like(top), top))
    total = e.sum(-1, keepdim=True)
    o = torch.matmul(e.view(B, hkv, g * N, L), v.permute(0, 2, 1, 3)).view(B, hkv, g, N, d)
    o = torch.where(total > 0, o / total, torch.zeros_like(o)).permute(0, 3, 1, 2, 4).reshape(B, N, c["hq"], d)
    have = i[None] < n[:, None]
    st["out"].copy_(o[have].transpose(0, 1))
    if st["lse"] is None:
        return [st["out"]]
    lse = (top + total.log()).squeeze(-1).permute(0, 3, 1, 2).reshape(B, N, c["hq"])
    st["lse"].copy_(lse[have].transpose(0, 1))
    return [st["out"], st["lse"]]


def run(state):
    c = state["case"]
    if not own:
        return {"rope": _rope_plain, "kv": _kv_plain, "tree": _tree_plain}[c["op"]](state)
    if c["op"] == "rope":
        state["rope"].apply(state["q"], state["k"], state["q_out"], state["k_out"], state["pos"], inverse=c["inverse"])
        return [state["q_out"], state["k_out"]]
    kv = state["kv"]
    if c["op"] == "kv":
        if c["write"]:
            kv.write(state["k"], state["v"], state["slots"])
        if not c["read"]:
            return state["pools"][:2]
        kv.read(state["table"], state["cu"], state["k_out"], state["v_out"], first=state["first"])
        return [state["k_out"], state["v_out"]]
    from dynamic_block_sparse_last_b200 import fp
    fp.fp_tree_attn(state["q"], kv, state["table"], state["len"], state["cu"], c["new"], state["mask"], c["d"] ** -0.5,
                    state["out"], state["work"], lse=state["lse"])
    return [state["out"]] if state["lse"] is None else [state["out"], state["lse"]]


# ------------------------------------------------------------------ work
def work(case):
    c = case
    if c["op"] == "rope":
        n = c["tokens"] * (c["hq"] + c["hkv"]) * c["d"]
        return {"bytes": 2 * n * SIZE[c["dtype"]] + 4 * c["tokens"], "flops": 3 * n * c["rot"] / c["d"]}
    row = c["hkv"] * c["d"]
    cell = 2 * (row * SIZE[c["kind"]] + (4 * c["hkv"] if c["kind"] in CODE else 0))  # a cached token: K and V
    if c["op"] == "kv":
        T = sum(_kv_lengths(c))
        a_way = 2 * row * SIZE[c["dtype"]] + cell
        return {"bytes": T * ((a_way + 8 if c["write"] else 0) + (a_way if c["read"] else 0)), "flops": 4 * T * row}
    n, cached = _tree_lengths(c)
    return {"bytes": sum(cached) * cell + sum(n) * c["hq"] * (2 * c["d"] * SIZE[c["dtype"]] + (4 if c["lse"] else 0)),
            "flops": 4 * c["hq"] * c["d"] * sum(a * b for a, b in zip(n, cached))}


# ------------------------------------------------------------------ the definition in 64 bits
def _exact_rope(st):
    c = st["case"]
    rot, amp = c["rot"], _scaling(c)[5]
    turn = torch.polar(torch.full((c["tokens"], rot // 2), amp, device="cuda", dtype=torch.float64),
                       torch.outer(st["pos"].double(), _freqs(c)))
    turn = turn.conj() if c["inverse"] else turn

    def one(x):
        y = x.double()
        head, tail = y[:, :rot], y[:, rot:]
        pairs = head.reshape(-1, 2, rot // 2).transpose(1, 2) if c["layout"] == "half" else head.reshape(-1, rot // 2, 2)
        z = torch.view_as_real(torch.view_as_complex(pairs.contiguous()) * turn)
        return torch.cat([(z.transpose(1, 2) if c["layout"] == "half" else z).reshape(-1, rot), tail], 1)
    return [torch.stack([one(x[h]) for h in range(x.shape[0])]) for x in (st["q"], st["k"])]


def _exact_cell(pool, scale, page, h, at):
    """fp64 values of one head's cache rows at the flat slots `at`."""
    x = pool[:, h].reshape(-1, pool.shape[-1]).view(torch.int8).index_select(0, at).view(pool.dtype).double()
    return x if scale is None else x * scale[:, h].reshape(-1).index_select(0, at).double()[:, None]


def _exact_kv(st):
    c = st["case"]
    P, cu, got = c["page"], st["cu"].tolist(), []
    if c["write"]:
        dt, top = CODE.get(c["kind"], (None, None))
        for i, x in enumerate((st["k"], st["v"])):
            y = x.double()
            if dt is not None:
                big = y.abs().max(-1, keepdim=True).values
                y = torch.nan_to_num(top * y / big)
                y = (torch.round(y) if c["kind"] == "int8" else y.to(dt).double()) * (big / top)
            if not c["read"]:  # the pools, whole
                pool = st["pools"][i].double().transpose(0, 1).reshape(c["hkv"], -1, c["d"])
                pool[:, st["slots"]] = y
                y = pool.view(c["hkv"], -1, P, c["d"]).transpose(0, 1)
            got.append(y)  # what was written is what is read back, in order
        return got
    for i in range(2):
        out = torch.empty(c["hkv"], cu[-1], c["d"], device="cuda", dtype=torch.float64)
        for s in range(c["seqs"]):
            p = torch.arange(cu[s + 1] - cu[s], device="cuda") + int(st["first"][s])
            at = st["table"][s].long()[p // P] * P + p % P
            for h in range(c["hkv"]):
                out[h, cu[s]:cu[s + 1]] = _exact_cell(st["pools"][i], st["pools"][2 + i], P, h, at)
        got.append(out)
    return got


def _exact_tree(st):
    c = st["case"]
    P, d, g, cu, lens = c["page"], c["d"], c["hq"] // c["hkv"], st["cu"].tolist(), st["len"].tolist()
    out = torch.zeros(c["hq"], st["T"], d, device="cuda", dtype=torch.float64)
    lse = torch.full((c["hq"], st["T"]), -math.inf, device="cuda", dtype=torch.float64)
    for s, L in enumerate(lens):
        n = cu[s + 1] - cu[s]
        p = torch.arange(L, device="cuda")
        at = st["table"][s].long()[p // P] * P + p % P
        hide = torch.zeros(n, L, device="cuda", dtype=torch.bool)
        if st["mask"] is None:
            hide[:, L - n:] = torch.ones(n, n, device="cuda", dtype=torch.bool).triu(1)
        else:
            for j in range(n):
                hide[:, L - n + j] = (st["mask"][cu[s]:cu[s + 1], j // 64] >> (j % 64)) & 1 == 0
        for h in range(c["hkv"]):
            k, v = (_exact_cell(st["pools"][i], st["pools"][2 + i], P, h, at) for i in (0, 1))
            for x in range(h * g, (h + 1) * g):
                z = (st["q"][x, cu[s]:cu[s + 1]].double() @ k.T / math.sqrt(d)).masked_fill(hide, -math.inf)
                out[x, cu[s]:cu[s + 1]] = torch.softmax(z, 1) @ v
                lse[x, cu[s]:cu[s + 1]] = torch.logsumexp(z, 1)
    return [out] if st["lse"] is None else [out, lse]


def exact(case, seed):
    st = {"rope": _rope_inputs, "kv": _kv_inputs, "tree": _tree_inputs}[case["op"]](case, seed)
    return {"rope": _exact_rope, "kv": _exact_kv, "tree": _exact_tree}[case["op"]](st)
