"""GPU tests of attention over pages of 4-bit codes, against 64 bits, and of a
decoding step of the cache's calls together."""
import random

import pytest
import torch

from test_gpu_kv import BF16, F32, U8, U24, gen, i32, randn, worst
from test_gpu_rotary import codes_of, rounding, split, turned

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def bec():
    import bounded_expert_cache_gb300 as m
    return m


class Codes:
    """A cache of codes whose pages are scattered, with rubbish (codes 15, scales and offsets NaN) wherever no token lies."""

    def __init__(self, bec, lens, page, hkv, D, dtype, seed, layers=2, layer=1, extra=5):
        g = gen(seed)
        need = [-(-n // page) for n in lens]
        P = sum(need) + extra
        order = torch.randperm(P, device="cuda", generator=g)
        S, W = len(lens) + 2, max(need) + 2
        table = torch.full((S, W), -1, dtype=torch.int32, device="cuda")
        held = torch.zeros(S, dtype=torch.int32, device="cuda")
        ref = torch.zeros(P, dtype=torch.int32, device="cuda")
        self.seqs = i32(S - 1 - b for b in range(len(lens)))
        k, v = (torch.full((layers, P, hkv, page, D * 9 // 16), 255, dtype=torch.uint8, device="cuda") for _ in range(2))
        self.k, self.v = [], []  # (scale, code - 8, offset of centred codes), 64 bits, [n, hkv, D]
        at = 0
        for b, n in enumerate(lens):
            row, pages = S - 1 - b, order[at:at + need[b]]
            at += need[b]
            table[row, :need[b]] = pages.int()
            held[row] = n
            ref[pages] = 1
            j = torch.arange(n, device="cuda")
            for pool, parts in ((k, self.k), (v, self.v)):
                codes, meta = codes_of(torch.randn((n, hkv, D), device="cuda", generator=g) + 0.3)
                if n:
                    cc, mm = split(pool[layer], D)
                    cc[pages[j // page], :, j % page] = codes
                    mm[pages[j // page], :, j % page] = meta
                parts.append(self.parts(codes, meta))
        self.layer, self.page, self.D = layer, page, D
        self.kv = bec.KvCache(k, v, table, held, ref, dtype)

    @staticmethod
    def parts(codes, meta):
        q = torch.stack([codes & 15, codes >> 4], -1).flatten(-2).double() - 8
        s, b = (meta[..., i].double().repeat_interleave(64, -1) for i in (0, 1))
        return s, q, b + 8 * s

    def poison(self, b, j, what="v", word=0x7FC0):
        """The scale of token j's first group becomes NaN (or another bf16)."""
        p = int(self.kv.table[self.seqs[b], j // self.page])
        pool = self.kv.k if what == "k" else self.kv.v
        split(pool[self.layer], self.D)[1].view(torch.int16)[p, :, j % self.page, 0, 0] = word
        for part in (self.k if what == "k" else self.v)[b][::2]:
            part[j, :, :64] = float("nan")


U11 = 2.0 ** -11  # of f16 (11-bit significand)


def rows_ref(q, K, V, n, window, sinks, scale, dtype, chunk=False):
    """64-bit rows of one sequence and their tolerance."""
    half = chunk and dtype == BF16 and q.shape[2] <= 128  # the tensor-core kernel: values and numerators are f16
    m, hq, D = q.shape
    (ks, kq, kb), (vs, vq, vb) = K, V
    g = hq // ks.shape[1]
    out = torch.zeros((m, hq, D), dtype=torch.float64, device="cuda")
    tol = torch.full_like(out, 1e-30)
    for i in range(m):
        p = n - m + i
        if p < 0:
            continue
        see = torch.arange(p + 1, device="cuda")
        if window:
            see = see[(p - see < window) | (see < sinks)]
        x = q[i].double()
        wide = lambda t: t[see].repeat_interleave(g, 1)  # noqa: E731
        s = torch.einsum("hd,jhd->hj", x, wide(ks * kq + kb)) * scale
        w = torch.softmax(s, dim=1)
        out[i] = torch.einsum("hj,jhd->hd", w, wide(vs * vq + vb))
        A = torch.einsum("hj,jhd->hd", w, wide((vs * vq).abs() + vb.abs()))
        R = torch.einsum("hj,jhd->hd", w, wide((vs * vq).abs()))
        # a score: products of codes exact, sums and the scales' and offsets'
        # products in fp32, twice the unit for the matrix units' sums; the same in
        # the quotient and above it; the exponential and the sums. bf16: a
        # numerator times its scale and the result are rounded
        mag = torch.einsum("hd,jhd->hj", x.abs(), wide((ks * kq).abs() + kb.abs())).nan_to_num(0).amax(1) * scale
        delta = 2 * (D + 16) * U24 * mag
        t = (2 * delta[:, None] + (64 + len(see) / 8) * 2 * U24) * A
        if half:
            # a key's value is rounded by u11 of itself, which moves a score by up to
            # u11 sum |x k| and every weight by a factor e^(+-2 of that), in the
            # quotient and above it; a value and a numerator are rounded by u11 each
            off = U11 * torch.einsum("hd,jhd->hj", x.abs(), wide((ks * kq + kb).abs())).nan_to_num(0).amax(1) * scale
            t = t + (torch.expm1(2 * off)[:, None] + 2.01 * U11) * A + 1.01 * U8 * out[i].abs()
        elif dtype == BF16:
            t = t + 1.01 * U8 * R + 1.01 * U8 * out[i].abs()
        tol[i] = t + 1e-30
    return out, tol


def check(pool, q, out, lens, ms, window, sinks, scale, chunk=False):
    at = 0
    for b, (n, m) in enumerate(zip(lens, ms)):
        ref, tol = rows_ref(q[at:at + m], pool.k[b], pool.v[b], n, window, sinks, scale, q.dtype, chunk)
        assert worst(out[at:at + m], ref, tol) <= 1.0, (b, n, m)
        at += m


DECODE = [
    # lens, n_q, hkv, group, D, page, window, sinks
    ([1], 1, 1, 1, 64, 16, 0, 0),
    ([0, 1, 2, 15, 16, 17], 1, 2, 8, 128, 16, 0, 0),
    ([255, 256, 257, 0, 1000], 1, 2, 4, 128, 64, 0, 0),
    ([3, 700, 1, 64], 4, 2, 8, 128, 32, 0, 0),
    ([5, 2000], 8, 1, 8, 128, 16, 0, 0),
    ([300, 31], 2, 4, 3, 192, 16, 0, 0),
    ([700, 0, 65], 1, 2, 5, 64, 128, 0, 0),
    ([513, 2], 4, 1, 8, 256, 64, 0, 0),
    ([900], 8, 1, 16, 256, 32, 0, 0),
    ([1000, 40], 1, 1, 64, 64, 256, 0, 0),
    ([640, 100], 8, 1, 64, 64, 16, 0, 0),
    ([1500, 90, 257], 1, 2, 8, 128, 16, 100, 4),
    ([1500, 90, 257], 4, 2, 2, 64, 64, 128, 0),
    ([2000, 1999, 33], 4, 1, 8, 128, 32, 1, 1),
    ([2000, 10], 2, 2, 4, 192, 16, 200, 500),
    ([1300, 260], 8, 2, 4, 256, 128, 90, 33),
    ([4000, 1], 1, 1, 8, 128, 16, 1024, 2000),
    ([3, 5], 8, 2, 1, 128, 16, 2, 0),
]


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("case", range(len(DECODE)))
def test_decode_over_codes_matches_64_bit(bec, dtype, case):
    lens, n_q, hkv, group, D, page, window, sinks = DECODE[case]
    pool = Codes(bec, lens, page, hkv, D, dtype, 10 + case)
    hq, rows = hkv * group, len(lens) * n_q
    slack = [0, 8, 40][case % 3]
    q = randn((rows, hq * D + slack), dtype, gen(1000 + case), 1.5)[:, :hq * D].unflatten(1, (hq, D))
    frame = torch.full((rows, hq * D + slack), 7.0, dtype=dtype, device="cuda")
    out = frame[:, :hq * D].unflatten(1, (hq, D))
    scale = D ** -0.5 if case % 2 else 0.2
    pool.kv.attn_decode(1, q, pool.seqs, n_q, out=out, scale=scale, window=window, sinks=sinks)
    pool.kv.check_errors()
    check(pool, q, out, lens, [n_q] * len(lens), window, sinks, scale)
    assert (frame[:, hq * D:] == 7.0).all()
    again = pool.kv.attn_decode(1, q, pool.seqs, n_q, scale=scale, window=window, sinks=sinks)
    assert torch.equal(out, again)


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_decode_over_codes_many_sequences(bec, dtype):
    rng = random.Random(3)
    lens = [rng.choice([0, 0, 1, 3, 20]) for _ in range(600)]
    lens[417] = 3000
    pool = Codes(bec, lens, 16, 1, 64, dtype, 3)
    q = randn((600, 4, 64), dtype, gen(4))
    out = pool.kv.attn_decode(1, q, pool.seqs)
    pool.kv.check_errors()
    check(pool, q, out, lens, [1] * 600, 0, 0, 0.125)


PREFILL = [
    # lens, ms, hkv, group, D, page, window, sinks
    ([1], [1], 1, 1, 64, 16, 0, 0),
    ([130, 1, 0], [130, 1, 0], 2, 4, 128, 16, 0, 0),
    ([700, 33], [200, 33], 1, 8, 128, 64, 0, 0),
    ([300, 20, 129], [100, 20, 65], 2, 2, 64, 32, 0, 0),
    ([260], [257], 1, 3, 192, 16, 0, 0),
    ([300, 40], [90, 3], 2, 1, 256, 64, 0, 0),
    ([900, 257], [300, 257], 1, 4, 128, 16, 100, 4),
    ([640, 140], [300, 140], 2, 8, 64, 128, 64, 0),
    ([500], [40], 1, 2, 256, 32, 7, 300),
    ([5, 3], [9, 3], 1, 2, 128, 16, 0, 0),  # rows before their sequence
    ([2000, 700], [5, 300], 2, 7, 128, 256, 0, 0),
    ([3000], [17], 1, 8, 128, 32, 0, 0),
]


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("case", range(len(PREFILL)))
def test_prefill_over_codes_matches_64_bit(bec, dtype, case):
    lens, ms, hkv, group, D, page, window, sinks = PREFILL[case]
    pool = Codes(bec, lens, page, hkv, D, dtype, 30 + case)
    hq, rows = hkv * group, sum(ms)
    slack = [0, 8, 40][case % 3]
    q = randn((rows, hq * D + slack), dtype, gen(2000 + case), 1.5)[:, :hq * D].unflatten(1, (hq, D))
    frame = torch.full((rows, hq * D + slack), 7.0, dtype=dtype, device="cuda")
    out = frame[:, :hq * D].unflatten(1, (hq, D))
    cu = i32([sum(ms[:i]) for i in range(len(ms) + 1)])
    scale = D ** -0.5 if case % 2 else 0.2
    pool.kv.attn_prefill(1, q, pool.seqs, cu, out=out, scale=scale, window=window, sinks=sinks)
    pool.kv.check_errors()
    check(pool, q, out, lens, ms, window, sinks, scale, chunk=True)
    assert (frame[:, hq * D:] == 7.0).all()
    again = pool.kv.attn_prefill(1, q, pool.seqs, cu, scale=scale, window=window, sinks=sinks)
    assert torch.equal(out, again)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("D", [64, 128])
def test_prefill_over_codes_many_chunks(bec, dtype, D):
    rng = random.Random(5)
    lens = [rng.choice([0, 1, 2, 5, 30]) for _ in range(500)]
    lens[77] = 1500
    ms = [min(n, rng.choice([0, 1, 3, 30])) for n in lens]
    ms[77] = 400
    pool = Codes(bec, lens, 16, 1, D, dtype, 3)
    q = randn((sum(ms), 3, D), dtype, gen(4))
    cu = i32([sum(ms[:i]) for i in range(len(ms) + 1)])
    out = pool.kv.attn_prefill(1, q, pool.seqs, cu)
    pool.kv.check_errors()
    check(pool, q, out, lens, ms, 0, 0, D ** -0.5, chunk=True)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("D", [64, 128, 192, 256])
@pytest.mark.parametrize("what,word", [("v", 0x7FC0), ("v", 0x7F80), ("k", 0x7FC0)])
def test_hidden_tokens_of_codes_do_not_reach_a_row(bec, dtype, D, what, word):
    """NaN or infinite scales at tokens that some rows see: those rows become NaN, the others stay."""
    n, m = 300, 40
    pool = Codes(bec, [n, 50], 16, 1, D, dtype, 6)
    q = randn((2 * m, 2, D), dtype, gen(7))
    cu = i32([0, m, 2 * m])
    args = dict(scale=D ** -0.5, window=100, sinks=3)
    before = pool.kv.attn_prefill(1, q, pool.seqs, cu, **args)
    tokens = [2, 190, 280]
    for j in tokens:
        pool.poison(0, j, what, word)
    seen = torch.tensor([any(j <= p and (p - j < 100 or j < 3) for j in tokens) for p in range(n - m, n)], device="cuda")
    hide = torch.tensor([not s for s in seen.tolist()], device="cuda")
    assert seen.all() or hide.any()
    for j in (2, 190):  # now only the third is left to be seen: the first is a first token, the second leaves the window midway
        p = int(pool.kv.table[pool.seqs[0], j // 16])
        if j == 2:
            fresh = Codes(bec, [n, 50], 16, 1, D, dtype, 6)
            for mine, other in ((pool.kv.k, fresh.kv.k), (pool.kv.v, fresh.kv.v)):
                mine[:, p] = other[:, p]
    out = pool.kv.attn_prefill(1, q, pool.seqs, cu, **args)
    pool.kv.check_errors()
    for i in range(m):
        p = n - m + i
        bad = any(j <= p and p - j < 100 for j in (190, 280))
        cols = slice(0, 64) if what == "v" else slice(0, D)
        got = out[i]
        if bad:
            assert not torch.isfinite(got[:, cols].float()).any()
            assert what == "k" or torch.equal(got[:, 64:], before[i][:, 64:])
        else:
            assert torch.equal(got, before[i]), i
    assert torch.equal(out[m:], before[m:])
    # the newest tokens of the decoding call: of 8, those from 295 on see what the window leaves
    dec = pool.kv.attn_decode(1, q[m - 8:m], pool.seqs[:1], 8, **args)
    assert torch.equal(torch.isfinite(dec.float()), torch.isfinite(out[m - 8:m].float()))


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_codes_with_large_and_tiny_scores(bec, dtype):
    """Scores of some hundred times the usual spread, and queries of zero."""
    pool = Codes(bec, [700, 300], 16, 2, 128, dtype, 12)
    q = randn((2, 8, 128), dtype, gen(3), 200.0)
    q[1] = 0.0
    out = pool.kv.attn_decode(1, q, pool.seqs)
    check(pool, q, out, [700, 300], [1, 1], 0, 0, 128 ** -0.5)
    pre = pool.kv.attn_prefill(1, q, pool.seqs, i32([0, 1, 2]))
    check(pool, q, pre, [700, 300], [1, 1], 0, 0, 128 ** -0.5, chunk=True)


def test_codes_past_32_bit_offsets(bec):
    """The last pages of a pool of 4.6 GB a tensor."""
    D, page, hkv = 256, 256, 8
    P = 15700  # x 8 heads x 36,864 bytes
    pool = torch.empty((1, P, hkv, page, D * 9 // 16), dtype=torch.uint8, device="cuda")
    kv = bec.KvCache(pool, pool.clone(), torch.full((2, 4), -1, dtype=torch.int32, device="cuda"),
                     torch.zeros(2, dtype=torch.int32, device="cuda"), torch.zeros(P, dtype=torch.int32, device="cuda"), BF16)
    kv.table[1, :2] = i32([P - 1, P - 2])
    kv.ref[P - 2:] = 1
    kv.lens[1] = 300
    x = randn((300, hkv, D), BF16, gen(2))
    rot = bec.Rotary(D)
    q = kv.write_rotary(0, x, x, x, i32([1]), i32([0, 300]), rot)
    k, v = kv.read(0, i32([1]), i32([0, 300]), 300)
    kv.check_errors()
    y, _ = turned(x, torch.arange(300, device="cuda"), rot)
    span = y.unflatten(-1, (-1, 64)).abs().amax(-1)
    assert ((k.double() - y).abs() <= (span * 2 / 15 * 0.6 + span * 4 * U8).repeat_interleave(64, -1)).all()
    # attention over what read gives back
    kk, vv = (t.double().transpose(0, 1) for t in (k, v))
    for out, rows in ((kv.attn_decode(0, q[-2:], i32([1]), 2), (298, 299)), (kv.attn_prefill(0, q, i32([1]), i32([0, 300])), range(300))):
        for i, p in enumerate(rows):
            s = torch.einsum("hd,hjd->hj", q[p].double(), kk[:, :p + 1]) * D ** -0.5
            w = torch.softmax(s, 1)
            ref = torch.einsum("hj,hjd->hd", w, vv[:, :p + 1])
            # (k and v were read back as bf16: a score is off by that, too)
            off = 2 * U8 * torch.einsum("hd,hjd->hj", q[p].double().abs(), kk[:, :p + 1].abs()).amax(1) * D ** -0.5 / 8
            A = torch.einsum("hj,hjd->hd", w, vv[:, :p + 1].abs())
            assert ((out[i].double() - ref).abs() <= (2 * off[:, None] + 4 * U8) * A.amax(-1, keepdim=True) + 1e-6).all()


@pytest.mark.parametrize("kind", ["decode", "prefill"])
@pytest.mark.parametrize("dtype,D", [(BF16, 64), (BF16, 128), (BF16, 256), (F32, 128)])
@pytest.mark.parametrize("copies,window", [(0, 0), (0, 200), (1, 0), (5, 0)])
def test_attention_over_codes_whose_wait_times_out_leaves_the_cache_usable(bec, kind, dtype, D, copies, window):
    # several tiles a CTA: the hook stops it between them
    lens = [160000, 80000, 70]
    pool = Codes(bec, lens, 16, 2, D, dtype, 21)
    ms = [1] * 3 if kind == "decode" else [300, 129, 70]
    q = randn((sum(ms), 4, D), dtype, gen(5))
    cu = i32([sum(ms[:i]) for i in range(4)])

    def call():
        if kind == "decode":
            return pool.kv.attn_decode(1, q, pool.seqs, window=window)
        return pool.kv.attn_prefill(1, q, pool.seqs, cu, window=window)
    want = call()
    pool.kv.check_errors()
    bec.KvCache.debug_attn_wait_timeout(2_000_000, copies)
    call()
    with pytest.raises(bec.MoeError) as e:
        pool.kv.check_errors()
    assert e.value.status == 5
    assert torch.equal(call(), want)
    pool.kv.check_errors()


def test_refusals_of_attention_over_codes(bec):
    pool = Codes(bec, [40], 16, 2, 64, BF16, 2)
    kv, seqs = pool.kv, pool.seqs
    q = torch.zeros((1, 4, 64), dtype=BF16, device="cuda")
    with pytest.raises(TypeError):
        kv.attn_decode(1, q.float(), seqs)
    with pytest.raises(TypeError):
        kv.attn_prefill(1, q.view(torch.uint8), seqs, i32([0, 1]))
    with pytest.raises(bec.MoeError):
        kv.attn_decode(1, q, seqs, scale=0.0)
    with pytest.raises(bec.MoeError):
        kv.attn_decode(2, q, seqs)
    kv.attn_decode(1, q, i32([77]))
    with pytest.raises(bec.MoeError):
        kv.check_errors()
    kv.attn_prefill(1, q, seqs, i32([1, 1]))
    with pytest.raises(bec.MoeError):
        kv.check_errors()
    kv.table[seqs[0], 1] = 10 ** 6  # a page that is not there
    for call in (lambda: kv.attn_decode(1, q, seqs), lambda: kv.attn_prefill(1, q, seqs, i32([0, 1]))):
        call()
        with pytest.raises(bec.MoeError):
            kv.check_errors()


# ---------------------------------------------------------------- together
@pytest.mark.parametrize("dtype,bits", [(BF16, 4), (F32, 4), (BF16, 0)])
def test_step_in_a_graph_on_another_stream(bec, dtype, bits):
    """Reserve, rotate and write, attend, project to a vocabulary, draw: captured once, replayed with other contents."""
    D, hkv, hq, V, n = 128, 2, 8, 5000, 3
    g = gen(1)
    kv = bec.KvCache.empty(1, 60, hkv, 16, D, 4, 20, dtype=dtype, bits=bits)
    plain = bec.KvCache.empty(1, 60, hkv, 16, D, 4, 20, dtype=dtype, bits=bits)
    rot = bec.Rotary(D, factor=4.0, context=64)
    seqs = i32([2, 0, 3])
    ones, cu = i32([1, 1, 1]), i32(range(n + 1))
    x = torch.empty((n, hq + 2 * hkv, D), dtype=dtype, device="cuda")
    u = torch.empty((n,), device="cuda")
    head = torch.randn((hq * D, V), device="cuda", generator=g) * 0.2
    token, prob = torch.empty((n,), dtype=torch.int32, device="cuda"), torch.empty((n,), device="cuda")

    def step(cache, token, prob):
        cache.reserve(seqs, ones)
        q = cache.write_rotary(0, x[:, :hq], x[:, hq:hq + hkv], x[:, hq + hkv:], seqs, cu, rot)
        a = cache.attn_decode(0, q, seqs)
        z = a.flatten(1).float() @ head
        bec.sample(z, u, 0.9, 40, 0.95, token=token, prob=prob)
        return a, z

    prompt = randn((37 + 5 + 16, hq + 2 * hkv, D), dtype, g)
    for cache in (kv, plain):
        cache.reserve(seqs, i32([37, 5, 16]))
        pcu = i32([0, 37, 42, 58])
        q = cache.write_rotary(0, prompt[:, :hq], prompt[:, hq:hq + hkv], prompt[:, hq + hkv:], seqs, pcu, rot)
        cache.attn_prefill(0, q, seqs, pcu)
        cache.check_errors()
    x.copy_(randn(x.shape, dtype, g))
    u.uniform_(generator=g)
    step(kv, token, prob)  # (warm up, also on the other cache)
    step(plain, token, prob)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        a, z = step(kv, token, prob)
    mine, share = torch.empty_like(token), torch.empty_like(prob)
    for _ in range(20):  # across ends of pages
        x.copy_(randn(x.shape, dtype, g))
        u.uniform_(generator=g)
        torch.cuda.synchronize()
        with torch.cuda.stream(side):
            graph.replay()
        side.synchronize()
        want, logits = step(plain, mine, share)
        torch.cuda.synchronize()
        assert torch.equal(a, want) and torch.equal(token, mine) and torch.equal(prob, share)
    kv.check_errors()
    plain.check_errors()
    assert torch.equal(kv.lens, plain.lens) and torch.equal(kv.table, plain.table)
    assert torch.equal(kv.k, plain.k) and torch.equal(kv.v, plain.v)


@pytest.mark.parametrize("call", ["rotary", "write", "read", "sample"])
def test_results_of_the_calls_stream(bec, call):
    """A result that a call makes itself is its stream's memory."""
    side = torch.cuda.Stream()
    rot = bec.Rotary(64)
    kv = bec.KvCache.empty(1, 4, 1, 16, 64, 2, 2, dtype=BF16, bits=4)
    kv.reserve(i32([0]), i32([2]))
    x = torch.ones((2, 1, 64), dtype=BF16, device="cuda")
    z, u = torch.zeros((2, 9), device="cuda"), torch.zeros((2,), device="cuda")
    seqs, cu = i32([0]), i32([0, 2])
    made = {"rotary": lambda s: bec.rotary(x, i32([0, 1]), rot, stream=s), "write": lambda s: kv.write_rotary(0, x, x, x, seqs, cu, rot, stream=s),
            "read": lambda s: kv.read(0, seqs, cu, 2, stream=s)[0], "sample": lambda s: bec.sample(z, u, stream=s)[1]}[call]
    torch.cuda.synchronize()
    want = made(None)
    torch.cuda.synchronize()
    got = made(side)
    side.synchronize()
    assert torch.equal(got, want)
    # its memory goes back to that stream: a new tensor there may take it, one of the current stream does not
    at = got.data_ptr()
    del got
    with torch.cuda.stream(side):
        taken = [torch.empty_like(want) for _ in range(4)]
    assert at in [t.data_ptr() for t in taken]
