"""Measured cases of a decoder step's operators between its projections and its next token.

Four operators: rotary positions (half and interleaved layouts, a part of the
head, frequencies scaled for long contexts); writing a step's keys and values
into the paged cache with that rotation applied on the way, into pages of
values or of 4-bit codes; attention over pages of 4-bit codes, of the newest
token(s) and of prompt chunks; and drawing the next token from logits by
temperature, top-k, top-p and min-p with given random numbers.

A page of 4-bit codes holds, for each head, an affine matrix [tokens, head size]
in groups of 64: first the codes (element 2j in the low half of byte j, 2j+1 in
the high half), then a bf16 scale s and offset b for each group. A value is s*q + b.

``own`` False computes the plain forms below in elementary torch operations,
``own`` True calls the package. ``exact`` computes the definitions in 64 bits.
"""
import math

import numpy as np
import torch

own = False

_DT = {"bf16": torch.bfloat16, "f32": torch.float32}


# ---------------------------------------------------------------- the cases
def listed():
    return [
        # the query of one new token far into a context, whole heads in halves
        dict(name="rotary_one_token", op="rotary", dtype="bf16", rows=1, heads=16, D=128, dim=128, pairs=False, base=1e4,
             factor=1.0, context=0, top=262144, slack=512),
        # all heads of a long prompt, pairs of neighbours in half of the head, frequencies stretched 8 times by parts
        dict(name="rotary_prompt", op="rotary", dtype="bf16", rows=16384, heads=40, D=128, dim=64, pairs=True, base=5e5,
             factor=8.0, context=8192, top=65536, slack=0),
        # one user's next token into pages of bf16
        dict(name="write_one_token", op="write", dtype="bf16", bits=16, lens="777", new="1", hq=16, hkv=2, D=128, dim=128,
             pairs=False, base=1e4, factor=1.0, context=0, page=16, layers=2, slack=0),
        # a serving batch in fp32, three to five speculated tokens each, neighbours rotated in a part of the head
        dict(name="write_batch_f32", op="write", dtype="f32", bits=16, lens=_text(_spread(i, 40, 32768) + 5 for i in range(40)),
             new=_text(3 + i % 3 for i in range(40)), hq=12, hkv=4, D=96, dim=32, pairs=True, base=1e4, factor=4.0, context=0,
             page=64, layers=1, slack=4),
        # ragged prompts into pages of 4-bit codes, one of them with no new token; the pages' new values are read back
        dict(name="write_prompts_4bit", op="write", dtype="bf16", bits=4, lens="3001,129,9000,1,700,40", new="3001,129,4111,1,350,0",
             hq=32, hkv=8, D=128, dim=128, pairs=False, base=5e5, factor=8.0, context=8192, page=64, layers=1, slack=0),
        # one user's next token, short context
        dict(name="decode4_one_short", op="decode", dtype="bf16", lens="777", n_q=1, hq=16, hkv=2, D=128, page=16, layers=2,
             window=0, sinks=0, slack=0),
        # a serving batch with two speculated tokens each, contexts from none to 32K, windowed with first tokens kept
        dict(name="decode4_batch_window", op="decode", dtype="f32", lens=_text(_spread(i, 24, 32768) for i in range(24)), n_q=2,
             hq=8, hkv=2, D=64, page=32, layers=2, window=4096, sinks=4, slack=8),
        # a few very long contexts
        dict(name="decode4_long", op="decode", dtype="bf16", lens="262143,131072,200001", n_q=1, hq=32, hkv=8, D=128, page=64,
             layers=1, window=0, sinks=0, slack=0),
        # the last 2,048-token chunk of a 32K prompt
        dict(name="prefill4_chunk", op="prefill", dtype="bf16", lens="32768", q="2048", hq=16, hkv=2, D=128, page=64, layers=1,
             window=0, sinks=0, slack=512),
        # one user's next token from a large vocabulary
        dict(name="sample_one", op="sample", dtype="f32", rows=1, V=131072, temperature="0.8", top_k="50", top_p="0.95",
             min_p="0", masked=0.0, slack=0),
        # a serving batch in which every user has settings of their own
        dict(name="sample_batch", op="sample", dtype="f32", rows=64, V=131072, temperature="0.7,1,0,1.3", top_k="0,0,5,1000,50",
             top_p="0.9,1,0.95", min_p="0,0.02", masked=0.0, slack=0),
        # a large batch of bf16 logits of an odd vocabulary, half of it ruled out, drawn from all that is left
        dict(name="sample_masked_bf16", op="sample", dtype="bf16", rows=331, V=32771, temperature="1", top_k="0", top_p="1",
             min_p="0", masked=0.5, slack=5),
    ]


def _spread(i, n, top):
    """Length i of n: none, one, then spread over the logarithm up to top (odd values mostly)."""
    if i == 0:
        return 0
    return max(1, int(top ** (i / (n - 1)))) | (1 if i < n - 1 else 0)


def _text(values):
    return ",".join(str(i) for i in values)


def _open(case):
    """The case with its lists as lists."""
    c = dict(case)
    for k in ("lens", "new", "q"):
        if k in c:
            c[k] = [int(i) for i in c[k].split(",")]
    for k in ("temperature", "top_k", "top_p", "min_p"):
        if k in c:
            kind = int if k == "top_k" else float
            c[k] = [kind(i) for i in c[k].split(",")]
    return c


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _draw_rotary(rng, D):
    half = D // 2
    dim = rng.choice([D, D, 2 * max(1, half // 2), 2 * rng.randint(1, half)])
    return dict(dim=dim, pairs=rng.random() < 0.5, base=rng.choice([1e4, 1e6, 5e5]), factor=rng.choice([1.0, 1.0, 4.0, 8.0]),
                context=rng.choice([0, 4096, 8192]))


def draw(rng):
    op = rng.choice(["rotary", "rotary", "write", "write", "write", "decode", "decode", "decode", "prefill", "sample", "sample",
                     "sample"])
    if op == "rotary":
        D = rng.choice([64, 80, 96, 128, 128, 256])
        heads = rng.choice([1, 5, 8, 16, 40])
        dtype = rng.choice(["bf16", "bf16", "f32"])
        most = 16384 * 40 * 128 // (heads * D * (1 if dtype == "bf16" else 2))
        return dict(op=op, dtype=dtype, rows=_log(rng, 1, min(65536, most)), heads=heads, D=D, **_draw_rotary(rng, D),
                    top=rng.choice([100, 32768, 1000000]), slack=rng.choice([0, 8, 512]))
    if op == "write":
        bits = rng.choice([16, 4, 4])
        dtype = rng.choice(["bf16", "bf16", "f32"])
        D = rng.choice([64, 128, 128, 256]) if bits == 4 else rng.choice([64, 80, 96, 128, 128, 256])
        hkv, group = rng.choice([1, 2, 4, 8]), rng.choice([1, 2, 4, 8])
        B = _log(rng, 1, 64)
        most = max(1, 4096 * 48 * 128 // ((group + 2) * hkv * D * B * (1 if dtype == "bf16" else 2)))
        top = rng.choice([1, 4, min(4096, most)])
        new = [0 if rng.random() < 0.05 else _log(rng, 1, max(1, min(top, most))) for _ in range(B)]
        new[0] = max(1, new[0])
        past = [rng.choice([0, _log(rng, 1, 30000)]) for _ in range(B)]
        return dict(op=op, dtype=dtype, bits=bits, lens=_text(a + b for a, b in zip(past, new)), new=_text(new), hq=hkv * group,
                    hkv=hkv, D=D, **_draw_rotary(rng, D), page=rng.choice([16, 32, 64, 128]), layers=1,
                    slack=rng.choice([0, 8, 64]))
    if op in ("decode", "prefill"):
        dtype = rng.choice(["bf16", "bf16", "f32"] if op == "decode" else ["bf16", "bf16", "bf16", "f32"])
        D = rng.choice([64, 128, 128, 256])
        hkv, group = rng.choice([1, 2, 4, 8]), rng.choice([1, 2, 3, 4, 8])
        c = dict(op=op, dtype=dtype, hq=hkv * group, hkv=hkv, D=D, page=rng.choice([16, 32, 64, 128]), layers=1,
                 window=rng.choice([0, 0, 100, 1024, 4096]), sinks=rng.choice([0, 4, 33]), slack=rng.choice([0, 8, 64]))
        if op == "decode":
            B = _log(rng, 1, 40)
            budget = 593216 * 8 * 128 // (hkv * D * (1 if dtype == "bf16" else 4))
            top = max(2, min(262144 if B <= 3 else 65536, budget // B))
            lens = [0 if rng.random() < 0.05 else _log(rng, 1, top) for _ in range(B)]
            lens[0] = max(lens[0], top // 3)
            return dict(c, lens=_text(lens), n_q=rng.choice([1, 1, 2, 4, 5, 8]))
        q, lens = [], []
        B = rng.choice([1, 1, 2, 5])
        room = (2048 * 31744 * 16 * 128 if dtype == "bf16" else 2.0e11) / (c["hq"] * D)
        for _ in range(B):
            n = _log(rng, 9, 4096 if dtype == "bf16" else 500)
            past = rng.choice([0, 0, _log(rng, 1, 28000 if dtype == "bf16" else 1500)])
            cost = n * (past + n / 2)
            if cost > room / B:
                n = max(9, int(n * room / B / cost))
            q.append(n)
            lens.append(n + past)
        return dict(c, lens=_text(lens), q=_text(q))
    V = _log(rng, 100, 200000)
    return dict(op=op, dtype=rng.choice(["bf16", "f32", "f32"]), rows=_log(rng, 1, max(1, min(400, 64 * 131072 // V))), V=V,
                temperature=_text(rng.choice([0, 0.3, 0.7, 1.0, 1.0, 1.7]) for _ in range(5)),
                top_k=_text(rng.choice([0, 0, 1, 7, 50, 1000]) for _ in range(3)),
                top_p=_text(rng.choice([1.0, 1.0, 0.95, 0.9, 0.5]) for _ in range(4)),
                min_p=_text(rng.choice([0, 0, 0.01, 0.1]) for _ in range(2)), masked=rng.choice([0.0, 0.0, 0.3, 0.98]),
                slack=rng.choice([0, 3, 8]))


# ---------------------------------------------------------------- inputs
def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(int(seed) * 7919 + 29)


def _rows(n, cols, slack, dtype, g, scale=1.0):
    """[n, cols] as the leading columns of wider rows (a slice of a fused projection)."""
    x = torch.randn((n, cols + slack), dtype=dtype, device="cuda", generator=g)
    return (x.mul_(scale) if scale != 1.0 else x)[:, :cols]


def _angles_of(c):
    """Angle a position of each rotated pair, in 64 bits."""
    i = np.arange(c["dim"] // 2, dtype=np.float64)
    f = c["base"] ** (-2.0 * i / c["dim"])
    if c["context"]:  # frequencies of many turns within the context stay, those of few are stretched
        keep = np.clip((f * c["context"] / (2 * math.pi) - 1.0) / 31.0, 0.0, 1.0)
        return f * (keep + (1.0 - keep) / c["factor"])
    return f / c["factor"]


def _magnitude(c):
    return 0.1 * math.log(c["factor"]) + 1.0


def _rotary_of(c, st):
    st["angles"] = torch.from_numpy(_angles_of(c)).cuda()
    st["magnitude"] = _magnitude(c)
    if own:
        import bounded_expert_cache_gb300 as bec
        st["rot"] = bec.Rotary(c["dim"], base=c["base"], interleaved=c["pairs"], factor=c["factor"], context=c["context"],
                               turns=(1.0, 32.0), magnitude=st["magnitude"])


def _codes_meta(pool, D):
    """The codes [..., tokens, D/2] and the scales and offsets [..., tokens, D/64, 2] of a pool of 4-bit pages."""
    page = pool.shape[-2]
    flat = pool.flatten(-2)
    codes = flat[..., :page * D // 2].unflatten(-1, (page, D // 2))
    meta = flat[..., page * D // 2:].view(torch.bfloat16).unflatten(-1, (page, D // 64, 2))
    return codes, meta


def _quantise(x):
    """The codes [..., D/2] and scales and offsets [..., D/64, 2] of values [..., D] in fp32."""
    g = x.unflatten(-1, (-1, 64))
    b = g.amin(-1, keepdim=True).bfloat16()
    s = ((g.amax(-1, keepdim=True) - b.float()) / 15.0).bfloat16()
    q = torch.round((g - b.float()) / torch.where(s > 0, s, torch.ones_like(s)).float()).clamp(0, 15)
    q = torch.where(s > 0, q, torch.zeros_like(q)).to(torch.uint8).flatten(-2)
    return q[..., 0::2] | (q[..., 1::2] << 4), torch.cat([s, b], dim=-1)


def _values(codes, meta):
    """fp32 values [..., D]."""
    q = torch.stack([codes & 15, codes >> 4], dim=-1).flatten(-2).float().unflatten(-1, (-1, 64))
    return (q * meta[..., :1].float() + meta[..., 1:].float()).flatten(-2)


def _pool(c, n_pages, g):
    shape = (c["layers"], n_pages, c["hkv"], c["page"])
    if c.get("bits", 4) == 16:
        return torch.randn(shape + (c["D"],), dtype=_DT[c["dtype"]], device="cuda", generator=g)
    pool = torch.empty(shape + (c["D"] * 9 // 16,), dtype=torch.uint8, device="cuda")
    step = max(1, 2 ** 26 // (c["hkv"] * c["page"] * c["D"]))
    for layer in range(c["layers"]):
        for p in range(0, n_pages, step):
            part = pool[layer, p:p + step]
            codes, meta = _codes_meta(part, c["D"])
            x = torch.randn(part.shape[:-1] + (c["D"],), device="cuda", generator=g)
            codes[...], meta[...] = _quantise(x)
    return pool


def prepare(case, seed):
    g = _gen(seed)
    c = _open(case)
    return {"rotary": _prepare_rotary, "write": _prepare_kv, "decode": _prepare_kv, "prefill": _prepare_kv,
            "sample": _prepare_sample}[c["op"]](c, g)


def _prepare_rotary(c, g):
    st = dict(c)
    st["x"] = _rows(c["rows"], c["heads"] * c["D"], c["slack"], _DT[c["dtype"]], g).unflatten(1, (c["heads"], c["D"]))
    start = torch.randint(0, c["top"], (1,), device="cuda", generator=g)
    st["pos"] = ((start + torch.arange(c["rows"], device="cuda")) % c["top"]).to(torch.int32)
    st["out"] = torch.empty((c["rows"], c["heads"], c["D"]), dtype=_DT[c["dtype"]], device="cuda")
    _rotary_of(c, st)
    return st


def _prepare_kv(c, g):
    B, page = len(c["lens"]), c["page"]
    need = [-(-n // page) for n in c["lens"]]
    n_pages = sum(need) + 3
    order = torch.randperm(n_pages, device="cuda", generator=g).to(torch.int32)  # a pool in use is fragmented
    host = torch.full((B + 1, max(need) + 1), -1, dtype=torch.int32)
    pages = order.cpu()
    at = 0
    for b, n in enumerate(need):  # the batch's sequences sit in the table in another order than the batch's
        host[B - b, :n] = pages[at:at + n]
        at += n
    ref = torch.zeros(n_pages, dtype=torch.int32, device="cuda")
    ref[order[:at].long()] = 1
    st = dict(c, table=host.cuda(), seqs=torch.arange(B, 0, -1, dtype=torch.int32, device="cuda"), ref=ref)
    st["host_lens"] = c["lens"]
    st["lens"] = torch.tensor([0] + c["lens"][::-1], dtype=torch.int32, device="cuda")
    dtype = _DT[c["dtype"]]
    st["k"], st["v"] = _pool(c, n_pages, g), _pool(c, n_pages, g)
    rows = {"write": c.get("new"), "prefill": c.get("q")}.get(c["op"]) or [c["n_q"]] * B
    st["host_rows"] = rows
    cu = [0]
    for n in rows:
        cu.append(cu[-1] + n)
    st["cu"] = torch.tensor(cu, dtype=torch.int32, device="cuda")
    st["layer"] = c["layers"] - 1
    hq, hkv, D = c["hq"], c["hkv"], c["D"]
    if c["op"] == "write":  # one fused projection's rows
        x = _rows(cu[-1], (hq + 2 * hkv) * D, c["slack"], dtype, g)
        st["q"] = x[:, :hq * D].unflatten(1, (hq, D))
        st["new_k"] = x[:, hq * D:(hq + hkv) * D].unflatten(1, (hkv, D))
        st["new_v"] = x[:, (hq + hkv) * D:].unflatten(1, (hkv, D))
        _rotary_of(c, st)
    else:  # queries a little sharper than unit normal, as a slice of wider rows
        st["q"] = _rows(cu[-1], hq * D, c["slack"], dtype, g, 1.5).unflatten(1, (hq, D))
    st["out"] = torch.empty((cu[-1], hq, D), dtype=dtype, device="cuda")
    if own:
        import bounded_expert_cache_gb300 as bec
        st["kv"] = bec.KvCache(k=st["k"], v=st["v"], table=st["table"], lens=st["lens"], ref=st["ref"],
                               **({"dtype": dtype} if c.get("bits", 4) == 4 else {}))
    return st


def _prepare_sample(c, g):
    n, V, dtype = c["rows"], c["V"], _DT[c["dtype"]]
    z = torch.randn((n, V + c["slack"]), device="cuda", generator=g).mul_(2.0)
    # a few likely tokens above the bulk
    at = torch.randint(0, V, (n, 24), device="cuda", generator=g)
    z.scatter_add_(1, at, torch.empty((n, 24), device="cuda").uniform_(2.0, 11.0, generator=g))
    z = z.to(dtype)
    if c["masked"] > 0:  # tokens that a grammar rules out
        z.masked_fill_(torch.rand((n, V + c["slack"]), device="cuda", generator=g) < c["masked"], -math.inf)
    st = dict(c, logits=z[:, :V], u=torch.rand((n,), device="cuda", generator=g))
    for k, kind in (("temperature", torch.float32), ("top_k", torch.int32), ("top_p", torch.float32), ("min_p", torch.float32)):
        st[k] = torch.tensor([c[k][i % len(c[k])] for i in range(n)], dtype=kind, device="cuda")
    return st


# ---------------------------------------------------------------- one pass
def run(state):
    return {"rotary": _run_rotary, "write": _run_write, "decode": _run_attn, "prefill": _run_attn,
            "sample": _run_sample}[state["op"]](state)


def _turned(st, x, pos):
    """x [rows, heads, D] in fp32, its leading `dim` columns turned to `pos`."""
    dim = st["dim"]
    a = pos.double()[:, None] * st["angles"][None, :]  # far positions need 64 bits
    c, s = (torch.cos(a) * st["magnitude"]).float()[:, None], (torch.sin(a) * st["magnitude"]).float()[:, None]
    x = x.float()
    if st["pairs"]:
        u, w = x[..., 0:dim:2], x[..., 1:dim:2]
        y = torch.stack([u * c - w * s, w * c + u * s], dim=-1).flatten(-2)
    else:
        u, w = x[..., :dim // 2], x[..., dim // 2:dim]
        y = torch.cat([u * c - w * s, w * c + u * s], dim=-1)
    return torch.cat([y, x[..., dim:]], dim=-1)


def _run_rotary(st):
    if own:
        import bounded_expert_cache_gb300 as bec
        return bec.rotary(st["x"], st["pos"], st["rot"], out=st["out"])
    return _turned(st, st["x"], st["pos"]).to(st["x"].dtype)


def _places(st):
    """Sequence, position, page and place within it of every new token."""
    new = (st["cu"][1:] - st["cu"][:-1]).long()
    who = torch.repeat_interleave(torch.arange(new.numel(), device="cuda"), new)
    s = st["seqs"].long()[who]
    at = st["lens"].long()[s] - st["cu"][1:].long()[who] + torch.arange(who.numel(), device="cuda")
    return at, st["table"][s, at // st["page"]].long(), at % st["page"]


def _run_write(st):
    layer = st["layer"]
    if own:
        kv = st["kv"]
        q = kv.write_rotary(layer, st["q"], st["new_k"], st["new_v"], st["seqs"], st["cu"], st["rot"], q_out=st["out"])
        if st["bits"] == 16:
            return q, st["k"], st["v"]
        k, v = kv.read(layer, st["seqs"], st["cu"], st["q"].shape[0])
        return q, k, v
    at, page, place = _places(st)
    q, k, v = _turned(st, st["q"], at).to(st["q"].dtype), _turned(st, st["new_k"], at), st["new_v"].float()
    if st["bits"] == 16:
        st["k"][layer, page, :, place] = k.to(st["k"].dtype)
        st["v"][layer, page, :, place] = v.to(st["v"].dtype)
        return q, st["k"], st["v"]
    back = []
    for pool, x in ((st["k"], k), (st["v"], v)):
        codes, meta = _codes_meta(pool[layer], st["D"])
        codes[page, :, place], meta[page, :, place] = _quantise(x)
        back.append(_values(codes[page, :, place], meta[page, :, place]).to(st["q"].dtype))
    return (q, *back)


def _run_attn(st):
    if own:
        kv = st["kv"]
        if st["op"] == "decode":
            return kv.attn_decode(st["layer"], st["q"], st["seqs"], st["n_q"], out=st["out"], window=st["window"],
                                  sinks=st["sinks"])
        return kv.attn_prefill(st["layer"], st["q"], st["seqs"], st["cu"], out=st["out"], window=st["window"],
                               sinks=st["sinks"])
    hq, hkv, D, page = st["hq"], st["hkv"], st["D"], st["page"]
    out = torch.zeros_like(st["out"])
    kc, km = _codes_meta(st["k"][st["layer"]], D)
    vc, vm = _codes_meta(st["v"][st["layer"]], D)
    at = 0
    for b, (n, m) in enumerate(zip(st["host_lens"], st["host_rows"])):  # (contexts of very different lengths)
        q = st["q"][at:at + m].float()
        if n > 0:
            pages = st["table"][len(st["host_lens"]) - b, :-(-n // page)].long()
            k = _values(kc[pages], km[pages]).transpose(0, 1).reshape(hkv, -1, D)[:, :n]
            v = _values(vc[pages], vm[pages]).transpose(0, 1).reshape(hkv, -1, D)[:, :n]
            step = max(1, min(m, 2 ** 29 // (hq * n)))  # rows at a time: 2 GB of scores
            for r0 in range(0, m, step):
                r1 = min(m, r0 + step)
                pos = torch.arange(n - m + r0, n - m + r1, device="cuda")
                j = torch.arange(n, device="cuda")
                see = j[None, :] <= pos[:, None]
                if st["window"]:
                    see &= (pos[:, None] - j[None, :] < st["window"]) | (j[None, :] < st["sinks"])
                qs = q[r0:r1].view(r1 - r0, hkv, hq // hkv, D).permute(1, 2, 0, 3)
                s = (qs @ k[:, None].transpose(-1, -2)) / math.sqrt(D)
                s = s.masked_fill(~see, float("-inf"))
                top = s.amax(-1, keepdim=True)
                p = torch.exp(s - torch.where(torch.isinf(top), torch.zeros_like(top), top))
                total = p.sum(-1, keepdim=True)
                o = (p @ v[:, None]) / torch.where(total > 0, total, torch.ones_like(total))
                out[at + r0:at + r1] = o.permute(2, 0, 1, 3).reshape(r1 - r0, hq, D).to(out.dtype)
        at += m
    return out


def _run_sample(st):
    if own:
        import bounded_expert_cache_gb300 as bec
        return bec.sample(st["logits"], st["u"], temperature=st["temperature"], top_k=st["top_k"], top_p=st["top_p"],
                          min_p=st["min_p"])
    # in 64 bits: which token a random number falls on is decided by sums over the vocabulary
    z, V = st["logits"].double(), st["V"]
    top = z.amax(-1, keepdim=True)
    t = st["temperature"].double()[:, None]
    w = torch.exp((z - top.clamp(min=-1e300)) / torch.where(t > 0, t, torch.ones_like(t)))
    w, order = torch.sort(torch.where(t > 0, w, ((z == top) & (top > -math.inf)).double()), dim=-1, descending=True, stable=True)
    # (equal logits have equal weights, and weights keep the order of logits until they are 0)
    place = torch.arange(V, device="cuda")[None, :]
    k = st["top_k"].long()[:, None]
    w = torch.where((k > 0) & (place >= k) | (t <= 0) & (place >= 1), torch.zeros_like(w), w)
    before = torch.cumsum(w, dim=-1) - w
    p = st["top_p"].double()[:, None]
    keep = (p >= 1) | (place == 0) | (before < p * w.sum(-1, keepdim=True))
    keep &= w >= st["min_p"].double()[:, None].clamp(max=1.0)
    w = torch.zeros_like(w).scatter_(1, order, torch.where(keep, w, torch.zeros_like(w)))
    sums = torch.cumsum(w, dim=-1)
    total = sums[:, -1:]
    token = torch.searchsorted(sums, st["u"].double()[:, None] * total, right=True).clamp(max=V - 1)
    prob = w.gather(1, token) / torch.where(total > 0, total, torch.ones_like(total))
    # (a row in which nothing is left has no token)
    return torch.where(total > 0, token, -torch.ones_like(token))[:, 0].to(torch.int32), prob[:, 0].float()


# ---------------------------------------------------------------- the least work
def _visible(n, m, window, sinks):
    """Visible (row, key) pairs of one sequence and the keys some row sees."""
    pairs = 0
    for i in range(max(0, m - n), m):
        pos = n - m + i
        if not window or pos < window:
            pairs += pos + 1
        else:
            pairs += window + min(sinks, pos - window + 1)
    low = 0 if not window else max(0, max(0, n - m) - window + 1)
    return pairs, n - low + min(sinks, low) if n else 0


def work(case):
    c = _open(case)
    es = {"bf16": 2, "f32": 4}[c["dtype"]]
    if c["op"] == "rotary":
        n = c["rows"] * c["heads"] * c["D"]
        return {"bytes": 2 * n * es + 4 * c["rows"], "flops": 3 * c["rows"] * c["heads"] * c["dim"]}
    if c["op"] == "write":
        rows = sum(c["new"])
        kv = 2 * rows * c["hkv"] * c["D"]
        held = kv * 9 // 16 if c["bits"] == 4 else kv * es
        back = held + kv * es if c["bits"] == 4 else 0  # the values that are read back
        return {"bytes": 2 * rows * c["hq"] * c["D"] * es + kv * es + held + back,
                "flops": 3 * rows * (c["hq"] + c["hkv"]) * c["dim"]}
    if c["op"] == "sample":
        return {"bytes": c["rows"] * (c["V"] * es + 28), "flops": 2 * c["rows"] * c["V"]}
    nbytes = flops = 0
    for b, n in enumerate(c["lens"]):
        m = c["q"][b] if c["op"] == "prefill" else c["n_q"]
        pairs, keys = _visible(n, m, c["window"], c["sinks"])
        nbytes += keys * c["hkv"] * c["D"] * 2 * 9 // 16 + 2 * m * c["hq"] * c["D"] * es
        flops += 4 * pairs * c["hq"] * c["D"]
    return {"bytes": nbytes, "flops": flops}


# ---------------------------------------------------------------- the definitions in 64 bits
def exact(case, seed):
    c = _open(case)
    st = prepare(case, seed)
    return {"rotary": _exact_rotary, "write": _exact_write, "decode": _exact_attn, "prefill": _exact_attn,
            "sample": _exact_sample}[c["op"]](st)


def _exact_turn(st, x, pos):
    """Each pair as a complex number times e^(i angle)."""
    y = x.double().clone()
    dim = st["dim"]
    first = slice(0, dim, 2) if st["pairs"] else slice(0, dim // 2)
    second = slice(1, dim, 2) if st["pairs"] else slice(dim // 2, dim)
    z = torch.complex(y[..., first], y[..., second])
    angle = torch.outer(pos.double(), torch.tensor(_angles_of(st), device="cuda"))
    z = z * torch.polar(torch.full_like(angle, _magnitude(st)), angle)[:, None]
    y[..., first], y[..., second] = z.real, z.imag
    return y


def _exact_rotary(st):
    return _exact_turn(st, st["x"], st["pos"])


def _exact_codes(x):
    """The values that the 4-bit codes of x [rows, heads, D] stand for."""
    g = x.reshape(x.shape[0], x.shape[1], -1, 64)
    low = g.min(-1, keepdim=True).values.float().bfloat16().double()
    step = ((g.max(-1, keepdim=True).values - low) / 15).float().bfloat16().double()
    code = torch.where(step > 0, ((g - low) / torch.where(step > 0, step, 1.0)).round().clamp(0, 15), 0.0)
    return (low + step * code).reshape(x.shape)


def _exact_write(st):
    pos = []
    for n, m in zip(st["host_lens"], st["host_rows"]):
        pos += range(n - m, n)
    pos = torch.tensor(pos, device="cuda")
    q, k, v = _exact_turn(st, st["q"], pos), _exact_turn(st, st["new_k"], pos), st["new_v"].double()
    if st["bits"] == 4:
        return q, _exact_codes(k), _exact_codes(v)
    pools = []
    for pool, x in ((st["k"], k), (st["v"], v)):
        pool = pool.double()
        row = 0
        for b, (n, m) in enumerate(zip(st["host_lens"], st["host_rows"])):
            where = torch.arange(n - m, n, device="cuda")
            pages = st["table"][len(st["host_lens"]) - b].long()[where // st["page"]]
            pool[st["layer"]][pages, :, where % st["page"]] = x[row:row + m]
            row += m
        pools.append(pool)
    return (q, *pools)


def _exact_attn(st):
    B, hq, hkv, D, page = len(st["host_lens"]), st["hq"], st["hkv"], st["D"], st["page"]
    pairs = sum(_visible(n, m, 0, 0)[0] for n, m in zip(st["host_lens"], st["host_rows"]))
    if 4.0 * pairs * hq * D > 4e12:
        return None
    out = torch.zeros(st["out"].shape, dtype=torch.float64, device="cuda")
    group = hq // hkv

    def held(pool, h, where, place):  # fp64 values of one head's tokens
        flat = pool[st["layer"], :, h].reshape(pool.shape[1], -1)
        codes = flat[:, :page * D // 2].reshape(-1, page, D // 2)[where, place].long()
        meta = flat[:, page * D // 2:].reshape(-1, page, D // 64, 2, 2)[where, place].long()
        meta = ((meta[..., 1] * 256 + meta[..., 0]) << 16).to(torch.int32).view(torch.float32).double()  # bf16 bits
        q = torch.empty((codes.shape[0], D), dtype=torch.float64, device="cuda")
        q[:, 0::2], q[:, 1::2] = codes % 16, codes // 16
        return q * meta[..., 0].repeat_interleave(64, 1) + meta[..., 1].repeat_interleave(64, 1)

    start = 0
    for b in range(B):
        n, m = st["host_lens"][b], st["host_rows"][b]
        tok = torch.arange(n, device="cuda")
        where = st["table"][B - b].long()[tok // page] if n else tok
        for h in range(hkv if n else 0):
            kh, vh = held(st["k"], h, where, tok % page), held(st["v"], h, where, tok % page)
            for r in range(0, m, 2048):
                rows = torch.arange(r, min(m, r + 2048), device="cuda")
                back = (n - m + rows)[:, None] - tok[None, :]  # how far behind the row's own position
                hidden = back < 0
                if st["window"] > 0:
                    hidden = hidden | ((back >= st["window"]) & (tok >= st["sinks"])[None, :])
                for head in range(h * group, (h + 1) * group):
                    z = torch.einsum("rd,nd->rn", st["q"][start + rows, head].double(), kh) * (D ** -0.5)
                    z[hidden] = -math.inf
                    z = torch.softmax(z, dim=1)
                    z[hidden.all(dim=1)] = 0.0
                    out[start + rows, head] = z @ vh
        start += m
    return out


def _exact_sample(st):
    """Row by row on the host: sort, keep, walk along the vocabulary."""
    tokens, probs = [], []
    for r in range(st["rows"]):
        z = st["logits"][r].double().cpu().numpy()
        u = float(st["u"][r])
        temperature, k, p, floor = (float(st[x][r]) for x in ("temperature", "top_k", "top_p", "min_p"))
        order = np.lexsort((np.arange(z.size), -z))
        if z[order[0]] == -math.inf:
            tokens.append(-1)
            probs.append(0.0)
            continue
        if temperature <= 0:
            tokens.append(int(order[0]))
            probs.append(1.0)
            continue
        if k > 0:
            order = order[:int(k)]
        weight = np.exp((z[order] - z[order[0]]) / temperature)
        sums = np.cumsum(weight)
        if p < 1:
            n = 1 + int(np.count_nonzero(sums[:-1] < p * sums[-1]))
            order, weight = order[:n], weight[:n]
        kept = weight >= min(floor, 1.0)
        order, weight = order[kept], weight[kept]
        walk = np.argsort(order)
        order, weight = order[walk], weight[walk]
        sums = np.cumsum(weight)
        i = min(int(np.count_nonzero(sums <= u * sums[-1])), order.size - 1)
        tokens.append(int(order[i]))
        probs.append(weight[i] / sums[-1])
    return torch.tensor(tokens, dtype=torch.int32), torch.tensor(probs, dtype=torch.float64)
