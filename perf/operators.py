"""Measured cases of the decoder operators around the routed FFN layer.

Four operators: a linear layer with 4-bit weights and group scales, attention
of the newest token(s) over a paged KV cache, attention of prompt chunks over
the same cache (causal, with an optional sliding window beside a few first
tokens that stay visible), and the bookkeeping of the cache's pages (fork,
reserve with copy-on-write, write, free, compact).

``own`` False computes the plain forms below in elementary torch operations,
``own`` True calls the package. ``exact`` computes the definitions in 64 bits.
"""
import math

import torch

own = False

Q4_0, I4_G64 = 1, 2  # weight formats, numbered as in the package
_DT = {"bf16": torch.bfloat16, "f32": torch.float32}


# ---------------------------------------------------------------- the cases
def listed():
    return [
        # fused q/k/v projection of one new token (16 + 2 + 2 heads of 128)
        dict(name="linear_one_token", op="linear", quant=Q4_0, T=1, N=2560, K=2048, x="bf16", y="bf16",
             bias=False, slack=0),
        # projection of a step of four speculated tokens, fp32 stream, odd row count
        dict(name="linear_four_tokens_affine", op="linear", quant=I4_G64, T=4, N=4099, K=2816, x="f32",
             y="f32", bias=True, slack=8),
        # output head over a large vocabulary for a batch of sequences
        dict(name="linear_vocabulary", op="linear", quant=Q4_0, T=24, N=131072, K=2048, x="bf16", y="f32",
             bias=False, slack=0),
        # one user's next token, short context
        dict(name="decode_one_short", op="decode", dtype="bf16", lens="777", n_q=1, hq=16, hkv=2, D=128,
             page=16, layers=2, window=0, sinks=0, slack=0),
        # a serving batch with four speculated tokens each, contexts from none to 32K
        dict(name="decode_ragged_batch", op="decode", dtype="bf16",
             lens=_text(_spread(i, 40, 32768) for i in range(40)), n_q=4, hq=16, hkv=2, D=256, page=64, layers=1,
             window=0, sinks=0, slack=16),
        # a few very long contexts
        dict(name="decode_long", op="decode", dtype="bf16", lens="262143,131072,200001", n_q=1, hq=32,
             hkv=8, D=128, page=32, layers=1, window=0, sinks=0, slack=0),
        # fp32 stream, windowed with four first tokens kept
        dict(name="decode_window_f32", op="decode", dtype="f32", lens="5000,17,1,0,20011,4096,1300,999,33",
             n_q=1, hq=12, hkv=4, D=96, page=16, layers=2, window=1024, sinks=4, slack=4),
        # the eighth 4096-token chunk of a 32K prompt
        dict(name="prefill_chunk", op="prefill", dtype="bf16", lens="32768", q="4096", hq=16, hkv=2, D=128,
             page=64, layers=1, window=0, sinks=0, slack=512),
        # ragged prompts in one call, windowed with first tokens kept
        dict(name="prefill_window_ragged", op="prefill", dtype="bf16", lens="3001,129,9000,1,700",
             q="3001,129,1111,1,350", hq=32, hkv=4, D=64, page=16, layers=2, window=1024, sinks=4, slack=0),
        # a short fp32 prompt
        dict(name="prefill_short_f32", op="prefill", dtype="f32", lens="131,300", q="131,40", hq=8, hkv=8, D=80,
             page=16, layers=1, window=0, sinks=0, slack=0),
        # 8 prompts branched into 4 continuations each, one decode step written, branches freed
        dict(name="pages_branch", op="branch", dtype="bf16", prompts=8, branches=4, prompt_len=1500, n_new=1, hkv=2,
             D=128, page=64, layers=8, free_every=3),
        # a fragmented pool brought together
        dict(name="pages_compact", op="compact", dtype="bf16", seqs=48, pages=3000, fill=45, hkv=2, D=128, page=64,
             layers=10),
    ]


def _spread(i, n, top):
    """Length i of n: none, one, then spread over the logarithm up to top (odd values mostly)."""
    if i == 0:
        return 0
    return max(1, int(top ** (i / (n - 1)))) | (1 if i < n - 1 else 0)


def _text(ints):
    return ",".join(str(i) for i in ints)


def _open(case):
    """The case with its lists of lengths as lists."""
    return {k: [int(i) for i in v.split(",")] if k in ("lens", "q") else v for k, v in case.items()}


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["linear", "linear", "decode", "decode", "decode", "prefill", "prefill", "branch", "compact"])
    if op == "linear":
        quant = rng.choice([Q4_0, I4_G64])
        g = 32 if quant == Q4_0 else 64
        K = g * _log(rng, 2, 8192 // g)
        N = _log(rng, 16, max(16, min(131072, 131072 * 2048 // K)))
        return dict(op=op, quant=quant, T=_log(rng, 1, 24), N=N, K=K, x=rng.choice(["bf16", "f32"]),
                    y=rng.choice(["bf16", "f32"]), bias=rng.random() < 0.5, slack=rng.choice([0, 0, 8, 24]))
    if op == "decode":
        dtype = rng.choice(["bf16", "bf16", "f32"])
        D = rng.choice([64, 80, 96, 128, 128, 256])
        hkv, group = rng.choice([1, 2, 4, 8]), rng.choice([1, 2, 3, 4, 8])
        B = _log(rng, 1, 64)
        budget = 593216 * 8 * 128 // (hkv * D * (1 if dtype == "bf16" else 4))
        top = max(2, min(262144 if B <= 3 else 65536, budget // B))
        lens = [0 if rng.random() < 0.05 else _log(rng, 1, top) for _ in range(B)]
        lens[0] = max(lens[0], top // 3)
        return dict(op=op, dtype=dtype, lens=_text(lens), n_q=rng.choice([1, 1, 2, 4, 5, 8]), hq=hkv * group, hkv=hkv, D=D,
                    page=rng.choice([16, 32, 64, 128]), layers=1 if sum(lens) > 100000 else 2,
                    window=rng.choice([0, 0, 100, 1024, 4096]), sinks=rng.choice([0, 4, 33]),
                    slack=rng.choice([0, 8, 64]))
    if op == "prefill":
        dtype = rng.choice(["bf16", "bf16", "bf16", "f32"])
        D = rng.choice([64, 80, 96, 128, 128])
        hkv, group = rng.choice([1, 2, 4, 8]), rng.choice([1, 2, 3, 4, 8])
        B = rng.choice([1, 1, 2, 5])
        q, lens, room = [], [], (4096 * 30720 * 16 if dtype == "bf16" else 2.0e9) / (hkv * group)
        for _ in range(B):
            n = _log(rng, 9, 4096 if dtype == "bf16" else 500)
            past = rng.choice([0, 0, _log(rng, 1, 28000 if dtype == "bf16" else 1500)])
            cost = n * (past + n / 2)
            if cost > room / B:
                n = max(9, int(n * room / B / cost))
            q.append(n)
            lens.append(n + past)
        return dict(op=op, dtype=dtype, lens=_text(lens), q=_text(q), hq=hkv * group, hkv=hkv, D=D,
                    page=rng.choice([16, 32, 64, 128]), layers=1, window=rng.choice([0, 0, 200, 1024, 4096]),
                    sinks=rng.choice([0, 4, 33]), slack=rng.choice([0, 8, 512]))
    dtype = rng.choice(["bf16", "bf16", "f32"])
    hkv, D, page = rng.choice([1, 2, 4]), rng.choice([64, 80, 128]), rng.choice([16, 32, 64])
    if op == "branch":
        return dict(op=op, dtype=dtype, prompts=_log(rng, 1, 8), branches=rng.choice([1, 2, 3, 4]),
                    prompt_len=_log(rng, 1, 1500), n_new=rng.choice([1, 1, 4, 70]), hkv=hkv, D=D, page=page,
                    layers=rng.choice([1, 3, 8]), free_every=rng.choice([2, 3, 5]))
    layers = rng.choice([1, 4, 10])
    size = hkv * D * page * layers * (2 if dtype == "bf16" else 4)
    return dict(op=op, dtype=dtype, seqs=_log(rng, 2, 48),
                pages=_log(rng, 40, max(41, min(6000, 3000 * 2 * 128 * 64 * 10 * 2 // size))), fill=rng.choice([20, 45, 70]),
                hkv=hkv, D=D, page=page, layers=layers)


# ---------------------------------------------------------------- inputs
def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(int(seed) * 7919 + 17)


def _randn(shape, dtype, g, scale=1.0):
    x = torch.randn(shape, dtype=torch.float32 if dtype == torch.float32 else torch.bfloat16, device="cuda", generator=g)
    return x.mul_(scale) if scale != 1.0 else x


def _rows(n, cols, slack, dtype, g, scale=1.0):
    """[n, cols] as the leading columns of wider rows (a slice of a fused projection)."""
    return _randn((n, cols + slack), dtype, g, scale)[:, :cols]


def _pool(case, n_pages, g):
    shape = (case["layers"], n_pages, case["hkv"], case["page"], case["D"])
    k = _randn(shape, _DT[case["dtype"]], g)
    v = _randn(shape, _DT[case["dtype"]], g)
    return k, v


def _cache(st):
    """The package's cache object over this state's tensors."""
    import bounded_expert_cache_gb300 as bec
    return bec.KvCache(k=st["k"], v=st["v"], table=st["table"], lens=st["lens"], ref=st["ref"])


def prepare(case, seed):
    g = _gen(seed)
    return {"linear": _prepare_linear, "decode": _prepare_attn, "prefill": _prepare_attn, "branch": _prepare_branch,
            "compact": _prepare_compact}[case["op"]](_open(case), g)


def _prepare_linear(c, g):
    N, K = c["N"], c["K"]
    codes = torch.randint(0, 256, (N, K // 2), dtype=torch.uint8, device="cuda", generator=g)
    if c["quant"] == Q4_0:
        meta = torch.empty((N, K // 32), device="cuda").uniform_(1e-3, 2e-2, generator=g).half()
    else:
        s = torch.empty((N, K // 64), device="cuda").uniform_(1e-3, 2e-2, generator=g)
        b = -s * torch.empty_like(s).uniform_(7.0, 8.0, generator=g)
        meta = torch.stack([s, b], dim=-1).bfloat16()
    w = torch.cat([codes.reshape(-1), meta.reshape(-1).view(torch.uint8)])  # quant plane, then metadata plane
    st = dict(c, w=w, xin=_rows(c["T"], K, c["slack"], _DT[c["x"]], g),
              bvec=_randn((N,), torch.float32, g) if c["bias"] else None)
    st["out"] = torch.empty((c["T"], N), dtype=_DT[c["y"]], device="cuda")
    return st


def _prepare_attn(c, g):
    B, page = len(c["lens"]), c["page"]
    need = [-(-n // page) for n in c["lens"]]
    n_pages = sum(need) + 3
    order = torch.randperm(n_pages, device="cuda", generator=g).to(torch.int32)  # a pool in use is fragmented
    table = torch.full((B + 1, max(need) + 1), -1, dtype=torch.int32, device="cuda")
    # the batch's sequences sit in the table in another order than the batch's
    seqs = torch.arange(B, 0, -1, dtype=torch.int32, device="cuda")
    lens = torch.zeros(B + 1, dtype=torch.int32, device="cuda")
    at = 0
    for b, n in enumerate(need):
        table[B - b, :n] = order[at:at + n]
        at += n
    lens[1:] = torch.tensor(c["lens"][::-1], dtype=torch.int32)
    ref = torch.zeros(n_pages, dtype=torch.int32, device="cuda")
    ref[order[:at].long()] = 1
    st = dict(c, table=table, seqs=seqs, ref=ref)
    st["host_lens"] = list(c["lens"])
    st["lens"] = lens
    st["k"], st["v"] = _pool(c, n_pages, g)
    q = c["q"] if c["op"] == "prefill" else [c["n_q"]] * B
    st["host_q"] = q
    cu = [0]
    for n in q:
        cu.append(cu[-1] + n)
    st["cu"] = torch.tensor(cu, dtype=torch.int32, device="cuda")
    # queries a little sharper than unit normal, as a slice of wider rows
    st["q"] = _rows(cu[-1], c["hq"] * c["D"], c["slack"], _DT[c["dtype"]], g, 1.5).unflatten(1, (c["hq"], c["D"]))
    st["out"] = torch.empty((cu[-1], c["hq"], c["D"]), dtype=_DT[c["dtype"]], device="cuda")
    st["layer"] = c["layers"] - 1
    if own:
        st["kv"] = _cache(st)
    return st


def _lists(c):
    """Sequence ids of a branch case: prompts 0..n-1, their branches after them."""
    n, m = c["prompts"], c["branches"]
    src = [p for p in range(n) for _ in range(m)]
    dst = [n + i for i in range(n * m)]
    # one prompt in two goes on itself beside its branches
    step = [p for p in range(0, n, 2)] + dst
    new = [c["n_new"] + (i % 2) for i in range(len(step))]
    done = dst[::c["free_every"]]
    return src, dst, step, new, done


def _prepare_branch(c, g):
    n, m, page = c["prompts"], c["branches"], c["page"]
    src, dst, step, new, done = _lists(c)
    lens_h = [max(1, c["prompt_len"] - 13 * p) for p in range(n)]
    need = [-(-x // page) for x in lens_h]
    n_pages = sum(need) + len(step) * (2 + -(-max(new) // page)) + 2
    width = max(need) + 2 + -(-max(new) // page)
    order = torch.randperm(n_pages, device="cuda", generator=g).to(torch.int32)
    table = torch.full((n + n * m, width), -1, dtype=torch.int32, device="cuda")
    lens = torch.zeros(n + n * m, dtype=torch.int32, device="cuda")
    at = 0
    for p in range(n):
        table[p, :need[p]] = order[at:at + need[p]]
        lens[p] = lens_h[p]
        at += need[p]
    ref = torch.zeros(n_pages, dtype=torch.int32, device="cuda")
    ref[order[:at].long()] = 1
    st = dict(c, table=table, lens=lens, ref=ref, n_pages=n_pages)
    st["saved"] = [t.clone() for t in (table, lens, ref)]
    st["k"], st["v"] = _pool(c, n_pages, g)
    i32 = dict(dtype=torch.int32, device="cuda")
    st["src"], st["dst"] = torch.tensor(src, **i32), torch.tensor(dst, **i32)
    st["step"], st["new"], st["done"] = torch.tensor(step, **i32), torch.tensor(new, **i32), torch.tensor(done, **i32)
    cu = [0]
    for x in new:
        cu.append(cu[-1] + x)
    st["cu"] = torch.tensor(cu, **i32)
    st["host_new"], st["host_step"] = new, step
    width_kv = c["hkv"] * c["D"]
    kv = [_rows(cu[-1], 2 * width_kv, 64, _DT[c["dtype"]], g) for _ in range(c["layers"])]
    st["new_k"] = [t[:, :width_kv].unflatten(1, (c["hkv"], c["D"])) for t in kv]
    st["new_v"] = [t[:, width_kv:].unflatten(1, (c["hkv"], c["D"])) for t in kv]
    if own:
        st["kv"] = _cache(st)
    return st


def _prepare_compact(c, g):
    S, P, page = c["seqs"], c["pages"], c["page"]
    live = max(S, P * c["fill"] // 100)
    order = torch.randperm(P, device="cuda", generator=g)[:live].to(torch.int32)
    per = [live // S + (1 if s < live % S else 0) for s in range(S)]
    table = torch.full((S + 2, max(per) + 1), -1, dtype=torch.int32, device="cuda")
    lens = torch.zeros(S + 2, dtype=torch.int32, device="cuda")
    ref = torch.zeros(P, dtype=torch.int32, device="cuda")
    at = 0
    for s in range(S):
        table[s, :per[s]] = order[at:at + per[s]]
        lens[s] = per[s] * page - (s % page)
        at += per[s]
    ref[order.long()] = 1
    # sequence S shares the whole pages of sequence 0
    whole = max(0, per[0] - 1)
    table[S, :whole] = table[0, :whole]
    lens[S] = whole * page
    ref[table[0, :whole].long()] += 1
    st = dict(c, table=table, lens=lens, ref=ref)
    st["saved"] = [t.clone() for t in (table, lens, ref)]
    st["k"], st["v"] = _pool(c, P, g)
    if own:
        st["kv"] = _cache(st)
    return st


# ---------------------------------------------------------------- one pass
def run(state):
    return {"linear": _run_linear, "decode": _run_attn, "prefill": _run_attn, "branch": _run_branch,
            "compact": _run_compact}[state["op"]](state)


def _run_linear(st):
    if own:
        import bounded_expert_cache_gb300 as bec
        return bec.quant_linear(st["xin"], st["w"], st["quant"], st["N"], bias=st["bvec"], y=st["out"])
    N, K = st["N"], st["K"]
    codes = st["w"][:N * K // 2]
    meta = st["w"][N * K // 2:]
    if st["quant"] == Q4_0:
        b = codes.view(N, K // 32, 16)
        q = torch.cat([b & 15, b >> 4], dim=-1).float() - 8.0
        w = q * meta.view(torch.float16).view(N, K // 32, 1).float()
    else:
        b = codes.view(N, K // 64, 32)
        q = torch.stack([b & 15, b >> 4], dim=-1).view(N, K // 64, 64).float()
        sb = meta.view(torch.bfloat16).view(N, K // 64, 2).float()
        w = q * sb[..., :1] + sb[..., 1:]
    y = st["xin"].float() @ w.view(N, K).t()
    if st["bvec"] is not None:
        y = y + st["bvec"]
    return y.to(_DT[st["y"]])


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
    at = 0
    for b, (n, m) in enumerate(zip(st["host_lens"], st["host_q"])):
        q = st["q"][at:at + m].float()
        if n > 0:
            pages = st["table"][len(st["host_lens"]) - b, :-(-n // page)].long()
            k = st["k"][st["layer"], pages].transpose(0, 1).reshape(hkv, -1, D)[:, :n].float()
            v = st["v"][st["layer"], pages].transpose(0, 1).reshape(hkv, -1, D)[:, :n].float()
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


def _restore(st):
    for t, s in zip((st["table"], st["lens"], st["ref"]), st["saved"]):
        t.copy_(s)


def _plain_pages(lens, page):
    return (lens + page - 1) // page


def _plain_fork(st):
    src, dst = st["src"].long(), st["dst"].long()
    table, lens, ref = st["table"], st["lens"], st["ref"]
    rows = table[src]
    ref.add_(torch.bincount(rows[rows >= 0].long(), minlength=ref.numel()).to(torch.int32))
    table[dst] = rows
    lens[dst] = lens[src]


def _plain_reserve(st):
    table, lens, ref, page = st["table"], st["lens"], st["ref"], st["page"]
    s, new = st["step"].long(), st["new"].long()
    n = lens[s].long()
    have, then = _plain_pages(n, page), _plain_pages(n + new, page)
    last = table[s, (have - 1).clamp(min=0)].long()
    partial = (n % page != 0) & (new > 0)
    same = (last[:, None] == last[None, :]) & partial[:, None] & partial[None, :]
    before = torch.tril(same, -1).sum(1)  # sharers listed earlier
    cow = partial & (ref[last.clamp(min=0)] - before > 1)
    need = cow.long() + then - have
    first = torch.cumsum(need, 0) - need
    total = int(need.sum())
    free = torch.nonzero(ref == 0).view(-1)[:total]
    who = torch.repeat_interleave(torch.arange(s.numel(), device="cuda"), need)
    entry = have[who] + torch.arange(total, device="cuda") - first[who] - cow.long()[who]
    table[s[who], entry] = free.to(torch.int32)
    ref.sub_(torch.bincount(last[cow], minlength=ref.numel()).to(torch.int32))
    ref[free] = 1
    old, fresh = last[cow], free[first[cow]]
    filled = (torch.arange(page, device="cuda")[None, :] < (n % page)[cow][:, None])[None, :, None, :, None]
    for pool in (st["k"], st["v"]):
        pool[:, fresh] = torch.where(filled, pool[:, old], pool[:, fresh])
    lens[s] = (n + new).to(torch.int32)


def _plain_write(st, layer):
    s, new = st["step"].long(), st["new"].long()
    who = torch.repeat_interleave(torch.arange(s.numel(), device="cuda"), new)
    at = st["lens"][s].long()[who] - new[who] + torch.arange(who.numel(), device="cuda") - st["cu"].long()[who]
    pages = st["table"][s[who], at // st["page"]].long()
    st["k"][layer, pages, :, at % st["page"]] = st["new_k"][layer]
    st["v"][layer, pages, :, at % st["page"]] = st["new_v"][layer]


def _plain_free(st):
    done = st["done"].long()
    rows = st["table"][done]
    st["ref"].sub_(torch.bincount(rows[rows >= 0].long(), minlength=st["ref"].numel()).to(torch.int32))
    st["table"][done] = -1
    st["lens"][done] = 0


def _run_branch(st):
    _restore(st)
    if own:
        kv = st["kv"]
        kv.fork(st["src"], st["dst"])
        kv.reserve(st["step"], st["new"])
        for layer in range(st["layers"]):
            kv.write(layer, st["new_k"][layer], st["new_v"][layer], st["step"], st["cu"])
        kv.free(st["done"])
    else:
        _plain_fork(st)
        _plain_reserve(st)
        for layer in range(st["layers"]):
            _plain_write(st, layer)
        _plain_free(st)
    return st["table"], st["lens"], st["ref"], st["k"], st["v"]


def _run_compact(st):
    _restore(st)
    if own:
        st["kv"].compact()
    else:
        table, ref = st["table"], st["ref"]
        live = ref > 0
        n = int(live.sum())
        dst = torch.nonzero(~live[:n]).view(-1)
        src = torch.nonzero(live[n:]).view(-1) + n
        for pool in (st["k"], st["v"]):
            pool[:, dst] = pool[:, src]
        to = torch.arange(ref.numel(), dtype=torch.int32, device="cuda")
        to[src] = dst.to(torch.int32)
        table.copy_(torch.where(table >= 0, to[table.clamp(min=0).long()], table))
        ref[dst] = ref[src]
        ref[src] = 0
    return st["table"], st["lens"], st["ref"], st["k"], st["v"]


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
    es = {"bf16": 2, "f32": 4}
    if c["op"] == "linear":
        N, K, T = c["N"], c["K"], c["T"]
        return {"bytes": N * K * 9 // 16 + T * K * es[c["x"]] + T * N * es[c["y"]] + (4 * N if c["bias"] else 0),
                "flops": 2 * T * N * K}
    e = es[c["dtype"]]
    if c["op"] in ("decode", "prefill"):
        q = c["q"] if c["op"] == "prefill" else [c["n_q"]] * len(c["lens"])
        pairs = keys = 0
        for n, m in zip(c["lens"], q):
            a, b = _visible(n, m, c["window"], c["sinks"])
            pairs, keys = pairs + a, keys + b
        return {"bytes": keys * 2 * c["hkv"] * c["D"] * e + 2 * sum(q) * c["hq"] * c["D"] * e
                + 4 * sum(-(-n // c["page"]) for n in c["lens"]),
                "flops": 4 * pairs * c["hq"] * c["D"]}
    token = 2 * c["layers"] * c["hkv"] * c["D"] * e
    if c["op"] == "branch":
        src, dst, step, new, done = _lists(c)
        lens = [max(1, c["prompt_len"] - 13 * p) for p in range(c["prompts"])]
        copied = 0
        for p in range(c["prompts"]):
            sharers = c["branches"] + (1 if p % 2 == 0 else 0)
            copied += lens[p] % c["page"] * min(sharers, c["branches"])
        ints = sum(-(-lens[s] // c["page"]) for s in src) * 4 * 3
        return {"bytes": 2 * token * (copied + sum(new)) + ints, "flops": 0}
    P = c["pages"]
    live = max(c["seqs"], P * c["fill"] // 100)
    moved = live * (P - live) // P  # live pages above the new end, on average
    return {"bytes": 2 * token * c["page"] * moved + 4 * 2 * P + 8 * live, "flops": 0}


# ---------------------------------------------------------------- definitions in 64 bits
def exact(case, seed):
    st = prepare(case, seed)
    return {"linear": _exact_linear, "decode": _exact_attn, "prefill": _exact_attn, "branch": _exact_branch,
            "compact": _exact_compact}[case["op"]](st)


def _exact_linear(st):
    """Weight by weight from the packed bytes: element k's nibble and its group's numbers."""
    N, K = st["N"], st["K"]
    k = torch.arange(K, device="cuda")
    if st["quant"] == Q4_0:
        byte, high = k // 32 * 16 + k % 16, k % 32 >= 16
    else:
        byte, high = k // 2, k % 2 == 1
    x = st["xin"].double()
    y = torch.empty((st["T"], N), dtype=torch.float64, device="cuda")
    codes = st["w"][:N * K // 2].view(N, K // 2)
    tail = st["w"][N * K // 2:].view(N, -1)
    for n0 in range(0, N, 8192):
        raw = codes[n0:n0 + 8192][:, byte].to(torch.int16)
        nib = torch.where(high, raw.div(16, rounding_mode="floor"), raw.remainder(16)).double()
        m = tail[n0:n0 + 8192].contiguous()
        if st["quant"] == Q4_0:
            w = (nib - 8.0) * m.view(torch.float16).double()[:, k // 32]
        else:
            m = m.view(torch.bfloat16).double()
            w = nib * m[:, k // 64 * 2] + m[:, k // 64 * 2 + 1]
        y[:, n0:n0 + 8192] = torch.einsum("tk,nk->tn", x, w)
    if st["bvec"] is not None:
        y += st["bvec"].double()[None]
    return y


def _exact_attn(st):
    """Head by head over each sequence's tokens, gathered one by one through the page table."""
    D, page, hq, group = st["D"], st["page"], st["hq"], st["hq"] // st["hkv"]
    B = len(st["host_lens"])
    out = torch.zeros(st["out"].shape, dtype=torch.float64, device="cuda")
    start = 0
    for b in range(B):
        n, m = st["host_lens"][b], st["host_q"][b]
        tok = torch.arange(n, device="cuda")
        where = st["table"][B - b].long()[tok // page] if n else tok
        for h in range(hq if n else 0):
            kh = st["k"][st["layer"], :, h // group][where, tok % page].double()
            vh = st["v"][st["layer"], :, h // group][where, tok % page].double()
            for r in range(0, m, 2048):
                rows = torch.arange(r, min(m, r + 2048), device="cuda")
                back = (n - m + rows)[:, None] - tok[None, :]  # how far behind the row's own position
                hidden = back < 0
                if st["window"] > 0:
                    hidden = hidden | ((back >= st["window"]) & (tok >= st["sinks"])[None, :])
                z = torch.einsum("rd,nd->rn", st["q"][start + rows, h].double(), kh) * (D ** -0.5)
                z[hidden] = -math.inf
                z = torch.softmax(z, dim=1)
                z[hidden.all(dim=1)] = 0.0
                out[start + rows, h] = z @ vh
        start += m
    return out


def _exact_branch(st):
    """The bookkeeping page by page on the host."""
    page, (table, lens, ref) = st["page"], [t.tolist() for t in st["saved"]]
    k, v = st["k"], st["v"]
    for s, d in zip(st["src"].tolist(), st["dst"].tolist()):
        for i, p in enumerate(table[s]):
            table[d][i] = p
            if p >= 0:
                ref[p] += 1
        lens[d] = lens[s]

    def lowest():
        p = ref.index(0)
        ref[p] = 1
        return p

    copies = []
    at = 0
    for s, n_new in zip(st["host_step"], st["host_new"]):
        n = lens[s]
        e = n // page
        if n % page and ref[table[s][e]] > 1:
            old = table[s][e]
            ref[old] -= 1
            table[s][e] = lowest()
            copies.append((old, table[s][e], n % page))
        for i in range(-(-n // page), -(-(n + n_new) // page)):
            table[s][i] = lowest()
        lens[s] = n + n_new
    for old, fresh, filled in copies:
        for pool in (k, v):
            pool[:, fresh, :, :filled] = pool[:, old, :, :filled]
    for s, n_new in zip(st["host_step"], st["host_new"]):
        for i in range(n_new):
            t = lens[s] - n_new + i
            for layer in range(st["layers"]):
                k[layer, table[s][t // page], :, t % page] = st["new_k"][layer][at]
                v[layer, table[s][t // page], :, t % page] = st["new_v"][layer][at]
            at += 1
    for s in st["done"].tolist():
        for i, p in enumerate(table[s]):
            if p >= 0:
                ref[p] -= 1
            table[s][i] = -1
        lens[s] = 0
    i32 = dict(dtype=torch.int32, device="cuda")
    return torch.tensor(table, **i32), torch.tensor(lens, **i32), torch.tensor(ref, **i32), k, v


def _exact_compact(st):
    table, lens, ref = [t.tolist() for t in st["saved"]]
    live = sum(1 for r in ref if r)
    move, hole = {}, 0
    for p in range(live, len(ref)):
        if ref[p]:
            while ref[hole]:
                hole += 1
            move[p] = hole
            ref[hole], ref[p] = ref[p], 0
    for p, h in move.items():
        for pool in (st["k"], st["v"]):
            pool[:, h].copy_(pool[:, p])
    table = [[move.get(p, p) for p in row] for row in table]
    i32 = dict(dtype=torch.int32, device="cuda")
    return torch.tensor(table, **i32), torch.tensor(lens, **i32), torch.tensor(ref, **i32), st["k"], st["v"]
