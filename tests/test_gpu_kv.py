"""GPU tests of the paged KV cache, attention over it and the 4-bit linear
layer, each against a plain 64-bit implementation."""
import math
import random

import pytest
import torch

pytestmark = pytest.mark.gpu

Q4_0, I4_G64 = 1, 2
BF16, F32 = torch.bfloat16, torch.float32
U24, U8 = 2.0 ** -24, 2.0 ** -8  # unit roundoffs of fp32 and bf16 (24- and 8-bit significands)


@pytest.fixture(scope="module")
def bec():
    import bounded_expert_cache_gb300 as m
    return m


def gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def i32(x):
    return torch.tensor(list(x), dtype=torch.int32, device="cuda")


def randn(shape, dtype, g, scale=1.0):
    return (torch.randn(shape, device="cuda", generator=g) * scale).to(dtype)


def worst(got, ref, tol):
    """Largest error in units of the tolerance; NaN and infinities have to be the same in both."""
    got, ref = got.double(), ref.double()
    odd = ~torch.isfinite(ref)
    assert torch.equal(torch.isnan(got), torch.isnan(ref)), "NaN in other places"
    assert torch.equal(got[odd & ~torch.isnan(ref)], ref[odd & ~torch.isnan(ref)])
    ratio = ((got - ref).abs() / tol)[~odd]
    return ratio.max().item() if ratio.numel() else 0.0


# ---------------------------------------------------------------- linear
def pack(N, K, quant, g):
    """Packed bytes of a random matrix and (group factor, integer code, group offset) in 64 bits."""
    codes = torch.randint(0, 16, (N, K), device="cuda", generator=g)
    if quant == Q4_0:
        d = torch.empty((N, K // 32), device="cuda").uniform_(-2e-2, 2e-2, generator=g).half()
        blk = codes.view(N, K // 32, 2, 16)
        raw = (blk[:, :, 0] | (blk[:, :, 1] << 4)).to(torch.uint8)
        scale = d.double().repeat_interleave(32, 1)
        parts = (scale, codes.double() - 8, torch.zeros_like(scale))
        meta = d
    else:
        s = torch.empty((N, K // 64), device="cuda").uniform_(1e-3, 2e-2, generator=g).to(BF16)
        b = (-s.float() * torch.empty_like(s, dtype=F32).uniform_(7, 8, generator=g)).to(BF16)
        raw = (codes[:, 0::2] | (codes[:, 1::2] << 4)).to(torch.uint8)
        parts = (s.double().repeat_interleave(64, 1), codes.double(), b.double().repeat_interleave(64, 1))
        meta = torch.stack([s, b], -1)
    w = torch.cat([raw.reshape(-1), meta.contiguous().view(torch.uint8).reshape(-1)])
    return w, parts


LINEAR = [
    # T, N, K
    (1, 1, 64), (1, 17, 128), (2, 8, 64), (3, 33, 192), (1, 2560, 2048), (4, 515, 1088), (5, 130, 4096),
    (8, 1000, 512), (9, 67, 2816), (16, 129, 1024), (17, 48, 704), (24, 2051, 2048), (33, 16, 8192), (70, 301, 320),
    (129, 64, 64),
]


@pytest.mark.parametrize("quant", [Q4_0, I4_G64])
@pytest.mark.parametrize("xt,yt", [(BF16, BF16), (BF16, F32), (F32, F32), (F32, BF16)])
def test_quant_linear_matches_64_bit(bec, quant, xt, yt):
    for i, (T, N, K) in enumerate(LINEAR):
        g = gen(100 * i + quant)
        w, (s, q, b) = pack(N, K, quant, g)
        slack = [0, 8, 24][i % 3]
        x = randn((T, K + slack), xt, g)[:, :K]
        bias = randn((N,), F32, g) if i % 2 else None
        frame = torch.full((T, N + 3), 7.0, dtype=yt, device="cuda")
        y = frame[:, 1:N + 1] if i % 4 == 3 else frame[:, :N]
        bec.quant_linear(x, w, quant, N, bias=bias, y=y)
        W = s * q + b
        ref = x.double() @ W.t()
        # every product is exact, a sum of n fp32 additions in any order is
        # within n u of the summed magnitudes; the matrix units' sums and the
        # factors double that; a bf16 result rounds once
        mag = x.double().abs() @ (s.abs() * q.abs() + b.abs()).t()
        if bias is not None:
            ref = ref + bias.double()
            mag = mag + bias.double().abs()
        tol = 2 * (K / 32 + 80) * U24 * mag + (U8 * ref.abs() if yt == BF16 else 0) * 1.01 + 1e-30
        assert worst(y, ref, tol) <= 1.0, (T, N, K)
        assert (frame[:, N + 1:] == 7.0).all() and (i % 4 != 3 or (frame[:, 0] == 7.0).all()), "outside of y"


@pytest.mark.parametrize("group", ["q4_0_single_block", "large_values"])
def test_quant_linear_edges(bec, group):
    g = gen(5)
    if group == "q4_0_single_block":
        # one block of 32: the format's smallest row, every code once or twice
        w, (s, q, b) = pack(3, 32, Q4_0, g)
        x = randn((2, 32), BF16, g)
        y = bec.quant_linear(x, w, Q4_0, 3)
        ref = x.double() @ (s * q).t()
        assert worst(y, ref, U8 * ref.abs() * 1.01 + 200 * U24 * (x.double().abs() @ (s * q).abs().t())) <= 1
    else:
        # activations near the ends of bf16's range: sums stay in fp32
        w, (s, q, b) = pack(40, 256, I4_G64, g)
        for mag in (1e30, 1e-30):
            x = randn((3, 256), F32, g, mag)
            y = bec.quant_linear(x, w, I4_G64, 40)
            ref = x.double() @ (s * q + b).t()
            m = x.double().abs() @ (s * q + b.abs()).t()
            assert worst(y, ref, 2 * 88 * U24 * m) <= 1
    assert bec.quant_linear(torch.empty((0, 256), device="cuda", dtype=BF16), pack(4, 256, Q4_0, g)[0], Q4_0,
                            4).shape == (0, 4)


@pytest.mark.parametrize("quant", [Q4_0, I4_G64])
@pytest.mark.parametrize("xt", [BF16, F32])
@pytest.mark.parametrize("T,N,K", [(1, 40, 256), (3, 515, 1088), (24, 300, 2048), (24, 70, 8192), (50, 33, 192)])
def test_quant_linear_infinite_and_large_activations(bec, quant, xt, T, N, K):
    """Infinities and NaN in x give what weight times x gives; sums of codes times x that pass fp32's range do not
    reach outputs that stay within it."""
    g = gen(T + K)
    w, (s, q, b) = pack(N, K, quant, g)
    W = s * q + b
    bias = randn((N,), F32, g)
    x = randn((T, K), xt, g).abs()
    for t in range(T):  # every kind of token beside each other
        kind = t % 5
        if kind == 0:  # group sums of codes overflow, outputs do not
            x[t, :64] *= 1.2e37 if quant == Q4_0 else 1.5e36
        elif kind == 1:
            x[t, K // 2] = float("inf")
        elif kind == 2:
            x[t, 5], x[t, K - 1] = float("inf"), -float("inf")
        elif kind == 3:
            x[t, 70 % K] = float("nan")
    for yt in (F32, BF16):
        y = bec.quant_linear(x, w, quant, N, bias=bias, y=torch.empty((T, N), dtype=yt, device="cuda"))
        # an infinity times a weight of zero is a NaN: products one by one, not a library's sums
        ref = torch.stack([(W * r[None]).sum(1) for r in x.double()]) + bias.double()
        mag = x.double().abs() @ (s.abs() * q.abs() + b.abs()).t() + bias.double().abs()
        tol = 2 * (K / 32 + 80) * U24 * mag + (U8 * ref.abs() if yt == BF16 else 0) * 1.01 + 1e-30
        assert torch.isfinite(ref[::5]).all() and ref[0].abs().max() > 1e35
        assert worst(y, ref, tol) <= 1.0


@pytest.mark.parametrize("quant,xt", [(Q4_0, BF16), (I4_G64, F32)])
def test_quant_linear_more_tokens_than_a_grid_has_blocks(bec, quant, xt):
    T, N, K = 65535 * 24 + 50, 17, 64
    g = gen(6)
    w, (s, q, b) = pack(N, K, quant, g)
    x = randn((T, K + 8), xt, g)[:, :K]
    frame = torch.full((T, N + 1), 7.0, dtype=xt, device="cuda")
    y = bec.quant_linear(x, w, quant, N, y=frame[:, :N])
    W = s * q + b
    for t0 in range(0, T, 2 ** 18):
        r = x[t0:t0 + 2 ** 18].double()
        ref, mag = r @ W.t(), r.abs() @ (s.abs() * q.abs() + b.abs()).t()
        tol = 2 * (K / 32 + 80) * U24 * mag + (U8 * ref.abs() if xt == BF16 else 0) * 1.01 + 1e-30
        assert worst(y[t0:t0 + 2 ** 18], ref, tol) <= 1.0, t0
    assert (frame[:, N] == 7.0).all()


def test_quant_linear_refusals(bec):
    g = gen(1)
    w, _ = pack(16, 64, Q4_0, g)
    x = randn((2, 64), BF16, g)
    with pytest.raises(bec.MoeError, match="quant"):
        bec.quant_linear(x, torch.zeros(16 * 36, dtype=torch.uint8, device="cuda"), bec.Q8_0, 16)
    with pytest.raises(ValueError):
        bec.quant_linear(x, w, Q4_0, 17)
    with pytest.raises(ValueError):
        bec.quant_linear(x.t(), w, Q4_0, 16)
    with pytest.raises(TypeError):
        bec.quant_linear(x.half(), w, Q4_0, 16)
    with pytest.raises(bec.MoeError, match="group"):
        bec.quant_linear(randn((2, 32), BF16, g), pack(16, 32, Q4_0, g)[0], I4_G64, 16)
    with pytest.raises(bec.MoeError, match="aligned"):
        bec.quant_linear(randn((2, 65), BF16, g)[:, :64], w, Q4_0, 16)
    with pytest.raises(bec.MoeError, match="aligned"):
        bec.quant_linear(x, torch.zeros(577, dtype=torch.uint8, device="cuda")[1:], Q4_0, 16)


# ---------------------------------------------------------------- attention
class Pool:
    """A cache whose pages are scattered, with garbage (NaN) wherever no token lies."""

    def __init__(self, bec, lens, page, hkv, D, dtype, seed, layers=2, layer=1, extra=5):
        g = gen(seed)
        need = [-(-n // page) for n in lens]
        P = sum(need) + extra
        order = torch.randperm(P, device="cuda", generator=g)
        S, W = len(lens) + 2, max(need) + 2
        self.table = torch.full((S, W), -1, dtype=torch.int32, device="cuda")
        self.lens = torch.zeros(S, dtype=torch.int32, device="cuda")
        self.ref = torch.zeros(P, dtype=torch.int32, device="cuda")
        self.seqs = i32(S - 1 - b for b in range(len(lens)))
        shape = (layers, P, hkv, page, D)
        k = torch.full(shape, float("nan"), dtype=dtype, device="cuda")
        v = torch.full(shape, float("nan"), dtype=dtype, device="cuda")
        self.tok_k, self.tok_v = [], []
        at = 0
        for b, n in enumerate(lens):
            row = S - 1 - b
            pages = order[at:at + need[b]]
            at += need[b]
            self.table[row, :need[b]] = pages.int()
            self.lens[row] = n
            self.ref[pages] = 1
            tk, tv = randn((n, hkv, D), dtype, g), randn((n, hkv, D), dtype, g)
            self.tok_k.append(tk)
            self.tok_v.append(tv)
            j = torch.arange(n, device="cuda")
            if n:
                k[layer, pages[j // page], :, j % page] = tk
                v[layer, pages[j // page], :, j % page] = tv
        self.layer, self.page = layer, page
        self.kv = bec.KvCache(k, v, self.table, self.lens, self.ref)

    def set_token(self, b, j, k=None, v=None):
        row = self.seqs[b].item()
        p = self.table[row, j // self.page].item()
        for pool, toks, val in ((self.kv.k, self.tok_k, k), (self.kv.v, self.tok_v, v)):
            if val is not None:
                pool[self.layer, p, :, j % self.page] = val
                toks[b][j] = val


def attn_ref(q, k, v, n, window, sinks, scale, dtype):
    """64-bit rows of one sequence (q [m, hq, D], k and v [n, hkv, D]) and their tolerance."""
    m, hq, D = q.shape
    hkv = k.shape[1]
    out = torch.zeros((m, hq, D), dtype=torch.float64, device="cuda")
    tol = torch.full_like(out, 1e-30)
    for i in range(m):
        p = n - m + i
        if p < 0:
            continue
        see = list(range(p + 1))
        if window:
            see = [j for j in see if p - j < window or j < sinks]
        see = torch.tensor(see, device="cuda")
        kk = k[see].double().repeat_interleave(hq // hkv, 1)
        vv = v[see].double().repeat_interleave(hq // hkv, 1)
        qq = q[i].double()
        s = torch.einsum("hd,jhd->hj", qq, kk) * scale
        w = torch.softmax(s, dim=1)
        out[i] = torch.einsum("hj,jhd->hd", w, vv)
        A = torch.einsum("hj,jhd->hd", w, vv.abs())
        # a score's error, in and below the quotient; the exponential and the
        # sums; for bf16 the numerators' and the result's rounding
        delta = (D + 8) * U24 * 2 * (scale * torch.einsum("hd,jhd->hj", qq.abs(), kk.abs())).amax(1)
        t = (2 * delta[:, None] + (64 + len(see) / 8) * 2 * U24) * A
        if dtype == BF16:
            t = t + U8 * A + 1.01 * U8 * out[i].abs()
        tol[i] = t + 1e-30
    return out, tol


def check_attn(pool, q, out, lens, ms, window, sinks, scale):
    at = 0
    for b, (n, m) in enumerate(zip(lens, ms)):
        ref, tol = attn_ref(q[at:at + m], pool.tok_k[b], pool.tok_v[b], n, window, sinks, scale, q.dtype)
        assert worst(out[at:at + m], ref, tol) <= 1.0, (b, n, m)
        at += m


DECODE = [
    # lens, n_q, hkv, group, D, page, window, sinks
    ([1], 1, 1, 1, 64, 16, 0, 0),
    ([0, 1, 2, 15, 16, 17], 1, 2, 8, 128, 16, 0, 0),
    ([127, 128, 129, 0, 1000], 1, 2, 4, 128, 64, 0, 0),
    ([3, 700, 1, 64], 4, 2, 8, 128, 32, 0, 0),
    ([5, 2000], 8, 1, 8, 128, 16, 0, 0),
    ([300, 31], 2, 4, 3, 96, 16, 0, 0),
    ([700, 0, 65], 1, 2, 5, 80, 128, 0, 0),
    ([513, 2], 4, 1, 8, 256, 64, 0, 0),
    ([900], 8, 1, 16, 256, 32, 0, 0),
    ([77, 400], 3, 3, 7, 200, 16, 0, 0),
    ([1000, 40], 1, 1, 64, 64, 256, 0, 0),
    ([640, 100], 8, 1, 64, 8, 16, 0, 0),
    ([1500, 90, 257], 1, 2, 8, 128, 16, 100, 4),
    ([1500, 90, 257], 4, 2, 2, 64, 64, 128, 0),
    ([2000, 1999, 33], 4, 1, 8, 128, 32, 1, 1),
    ([2000, 10], 2, 2, 4, 128, 16, 200, 500),
    ([1300, 260], 8, 2, 4, 256, 128, 90, 33),
    ([4000, 1], 1, 1, 8, 128, 16, 1024, 2000),
]


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("case", range(len(DECODE)))
def test_attn_decode_matches_64_bit(bec, dtype, case):
    lens, n_q, hkv, group, D, page, window, sinks = DECODE[case]
    pool = Pool(bec, lens, page, hkv, D, dtype, 10 + case)
    hq, rows = hkv * group, len(lens) * n_q
    slack = [0, 8, 40][case % 3]
    g = gen(1000 + case)
    q = randn((rows, hq * D + slack), dtype, g, 2.0)[:, :hq * D].unflatten(1, (hq, D))
    frame = torch.full((rows, hq * D + slack), 7.0, dtype=dtype, device="cuda")
    out = frame[:, :hq * D].unflatten(1, (hq, D))
    scale = D ** -0.5 if case % 2 else 0.3
    pool.kv.attn_decode(1, q, pool.seqs, n_q, out=out, scale=scale, window=window, sinks=sinks)
    pool.kv.check_errors()
    check_attn(pool, q, out, lens, [n_q] * len(lens), window, sinks, scale)
    assert (frame[:, hq * D:] == 7.0).all()
    # the same again, bit for bit: no result depends on arrival order
    again = pool.kv.attn_decode(1, q, pool.seqs, n_q, scale=scale, window=window, sinks=sinks)
    assert torch.equal(out, again)


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_attn_decode_many_sequences(bec, dtype):
    # more sequences than a block's threads, most of them empty or tiny, one long
    rng = random.Random(3)
    lens = [rng.choice([0, 0, 1, 3, 20]) for _ in range(600)]
    lens[417] = 3000
    pool = Pool(bec, lens, 16, 1, 64, dtype, 3)
    q = randn((600, 4, 64), dtype, gen(4))
    out = pool.kv.attn_decode(1, q, pool.seqs)
    pool.kv.check_errors()
    check_attn(pool, q, out, lens, [1] * 600, 0, 0, 0.125)


PREFILL = [
    # (len, rows) per sequence, hkv, group, D, page, window, sinks
    ([(1, 1)], 1, 1, 64, 16, 0, 0),
    ([(130, 130), (5, 0), (1, 1), (300, 40)], 2, 4, 128, 16, 0, 0),
    ([(257, 257)], 1, 8, 128, 64, 0, 0),
    ([(700, 129), (65, 65)], 2, 1, 64, 32, 0, 0),
    ([(500, 100)], 1, 3, 96, 128, 0, 0),
    ([(333, 333)], 2, 2, 80, 16, 0, 0),
    ([(400, 150)], 1, 5, 256, 64, 0, 0),
    ([(150, 90), (20, 33)], 1, 2, 200, 16, 0, 0),   # the second has rows before its first token
    ([(600, 600)], 1, 4, 128, 16, 64, 4),
    ([(900, 300), (100, 100)], 2, 8, 64, 64, 128, 0),
    ([(1000, 200)], 1, 16, 128, 32, 1, 1),
    ([(640, 640)], 1, 2, 128, 256, 150, 300),
    ([(1400, 70)], 4, 2, 112, 16, 500, 130),
    ([(200, 200)], 1, 64, 32, 16, 0, 0),
]


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("case", range(len(PREFILL)))
def test_attn_prefill_matches_64_bit(bec, dtype, case):
    pairs, hkv, group, D, page, window, sinks = PREFILL[case]
    lens, ms = [p[0] for p in pairs], [p[1] for p in pairs]
    pool = Pool(bec, lens, page, hkv, D, dtype, 50 + case)
    hq, rows = hkv * group, sum(ms)
    slack = [8, 0, 64][case % 3]
    g = gen(2000 + case)
    q = randn((rows, hq * D + slack), dtype, g, 2.0)[:, :hq * D].unflatten(1, (hq, D))
    frame = torch.full((rows, hq * D + slack), 7.0, dtype=dtype, device="cuda")
    out = frame[:, :hq * D].unflatten(1, (hq, D))
    cu = [0]
    for m in ms:
        cu.append(cu[-1] + m)
    scale = D ** -0.5
    pool.kv.attn_prefill(1, q, pool.seqs, i32(cu), out=out, window=window, sinks=sinks)
    pool.kv.check_errors()
    check_attn(pool, q, out, lens, ms, window, sinks, scale)
    assert (frame[:, hq * D:] == 7.0).all()


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("D", [8, 40, 120])
@pytest.mark.parametrize("tokens", [0, 1024])
def test_attn_prefill_many_chunks(bec, dtype, D, tokens):
    """More chunks than a block's threads, rows of 16 but not 32 bytes; with a long one, run ends fall into it."""
    rng = random.Random(D)
    lens = [rng.choice([0, 0, 1, 3, 20]) for _ in range(500)]
    ms = [min(n, rng.choice([0, 1, 20])) for n in lens]
    lens[411], ms[411] = 1000 + tokens, 100
    pool = Pool(bec, lens, 16, 1, D, dtype, 5)
    q = randn((sum(ms), 3, D), dtype, gen(6))
    cu = [0]
    for m in ms:
        cu.append(cu[-1] + m)
    out = pool.kv.attn_prefill(1, q, pool.seqs, i32(cu))
    pool.kv.check_errors()
    check_attn(pool, q, out, lens, ms, 0, 0, D ** -0.5)
    assert torch.equal(out, pool.kv.attn_prefill(1, q, pool.seqs, i32(cu)))


@pytest.mark.parametrize("D", [64, 128])
def test_attn_prefill_long_context_beside_rows_before_their_sequence(bec, D):
    """Rows without a token take no part in the work: the others' units are cut into many parts all the same."""
    lens, ms = [20000, 0], [64, 20000]
    pool = Pool(bec, lens, 64, 2, D, BF16, 12)
    q = randn((sum(ms), 32, D), BF16, gen(13))
    out = torch.full_like(q, 7.0)
    pool.kv.attn_prefill(1, q, pool.seqs, i32([0, 64, 20064]), out=out)
    pool.kv.check_errors()
    check_attn(pool, q[:64], out[:64], lens[:1], ms[:1], 0, 0, D ** -0.5)
    assert (out[64:] == 0).all()
    # the scratch is as it was: the next call's parts meet as well
    again = pool.kv.attn_prefill(1, q[:64].contiguous(), pool.seqs[:1].contiguous(), i32([0, 64]))
    check_attn(pool, q[:64], again, lens[:1], ms[:1], 0, 0, D ** -0.5)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf")])
def test_hidden_tokens_do_not_reach_a_row(bec, dtype, D, bad):
    """A token a row does not see may hold anything; rows that see it get what the formula gives."""
    lens, ms, window, sinks = [300, 90], [200, 90], 60, 2
    pool = Pool(bec, lens, 16, 2, D, dtype, 7)
    # values only: a value's infinity or NaN reaches exactly the rows that see it
    for b, j in ((0, 299), (0, 180), (0, 50), (1, 40)):
        pool.set_token(b, j, v=torch.full((2, D), bad))
    # one column of one head, and a key (hidden from most rows)
    one = pool.tok_v[0][250].clone()
    one[1, 5] = bad
    pool.set_token(0, 250, v=one)
    q = randn((290, 4, D), dtype, gen(8))
    out = pool.kv.attn_prefill(1, q, pool.seqs, i32([0, 200, 290]), window=window, sinks=sinks)
    pool.kv.check_errors()
    check_attn(pool, q, out, lens, ms, window, sinks, D ** -0.5)
    # decode: positions 292..299 of the first sequence, 82..89 of the second
    pool.set_token(0, 295, v=torch.full((2, D), bad))
    qd = randn((16, 4, D), dtype, gen(9))
    out = pool.kv.attn_decode(1, qd, pool.seqs, 8, window=window, sinks=sinks)
    check_attn(pool, qd, out, lens, [8, 8], window, sinks, D ** -0.5)
    # a NaN key hidden from the row
    pool.set_token(1, 10, k=torch.full((2, D), float("nan")))
    out = pool.kv.attn_decode(1, qd[8:], pool.seqs[1:].contiguous(), 8, window=window, sinks=sinks)
    check_attn_one(pool, 1, qd[8:], out, 90, 8, window, sinks, D ** -0.5)


def check_attn_one(pool, b, q, out, n, m, window, sinks, scale):
    ref, tol = attn_ref(q, pool.tok_k[b], pool.tok_v[b], n, window, sinks, scale, q.dtype)
    assert worst(out, ref, tol) <= 1.0


@pytest.mark.parametrize("dtype,D", [(BF16, 64), (BF16, 128), (BF16, 256), (F32, 64)])
@pytest.mark.parametrize("window,sinks", [(0, 0), (150000, 300)])
def test_hidden_values_of_a_long_context(bec, dtype, D, window, sinks):
    """Infinities and NaN among the values that only some rows see, 200,000 tokens in: their cost is that of the
    tiles they lie in, the other rows and the sequence behind are as ever."""
    lens, ms = [200000, 90], [140, 90]
    pool = Pool(bec, lens, 64, 1, D, dtype, 41)
    # near the rows' own positions, a whole token and single columns; at the window's far end; the second sequence
    for b, j, bad in ((0, 199900, float("nan")), (0, 49920, float("inf")), (1, 60, -float("inf"))):
        pool.set_token(b, j, v=torch.full((1, D), bad))
    for j, col, bad in ((199990, 3, float("inf")), (199870, 3, -float("inf")), (199995, D - 1, -float("inf")),
                        (50010, 9, float("nan"))):
        one = pool.tok_v[0][j].clone()
        one[0, col] = bad
        pool.set_token(0, j, v=one)
    q = randn((230, 2, D), dtype, gen(42))
    # the rows that see a bad value give it its weight: weights that fp32 holds
    out = pool.kv.attn_prefill(1, q, pool.seqs, i32([0, 140, 230]), window=window, sinks=sinks, scale=0.02)
    pool.kv.check_errors()
    check_attn(pool, q, out, lens, ms, window, sinks, 0.02)


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_attn_large_and_tiny_scores(bec, dtype):
    """Scores far apart, and a running maximum that grows along the cache."""
    pool = Pool(bec, [700], 16, 1, 128, dtype, 21)
    for j in range(0, 700, 50):
        pool.set_token(0, j, k=(pool.tok_k[0][j].float() * (1 + j / 40)).to(dtype))
    q = randn((300, 8, 128), dtype, gen(22), 4.0)
    out = pool.kv.attn_prefill(1, q, pool.seqs, i32([0, 300]))
    check_attn(pool, q, out, [700], [300], 0, 0, 128 ** -0.5)
    out = pool.kv.attn_decode(1, q[:4].contiguous(), pool.seqs, 4)
    check_attn(pool, q[:4], out, [700], [4], 0, 0, 128 ** -0.5)


def test_attention_past_32_bit_offsets(bec):
    # a pool of more than 2^32 bytes and 2^31 elements per tensor; the sequence lies at its end
    P, hkv, page, D = 18000, 8, 128, 128
    k = torch.empty((1, P, hkv, page, D), dtype=BF16, device="cuda")
    v = torch.empty_like(k)
    assert k.numel() > 2 ** 31
    table = torch.full((1, 4), -1, dtype=torch.int32, device="cuda")
    pages = [P - 1, P - 7, 17000]
    table[0, :3] = i32(pages)
    ref = torch.zeros(P, dtype=torch.int32, device="cuda")
    ref[pages] = 1
    kv = bec.KvCache(k, v, table, i32([300]), ref)
    g = gen(31)
    tk, tv = randn((300, hkv, D), BF16, g), randn((300, hkv, D), BF16, g)
    kv.write(0, tk, tv, i32([0]), i32([0, 300]))
    kv.check_errors()
    q = randn((60, 16, D), BF16, g)
    out = kv.attn_prefill(0, q, i32([0]), i32([0, 60]))
    ref_o, tol = attn_ref(q, tk, tv, 300, 0, 0, D ** -0.5, BF16)
    assert worst(out, ref_o, tol) <= 1.0
    out = kv.attn_decode(0, q[52:].contiguous(), i32([0]), 8)
    assert worst(out, ref_o[52:], tol[52:]) <= 1.0
    # a page moved over the whole pool
    kv.copy_pages(i32([P - 1]), i32([3]))
    assert torch.equal(k[0, 3], k[0, P - 1])


def test_attn_prefill_more_rows_than_31_bits(bec):
    """A chunk of more than 2^31 (token, head) rows: its last tokens are the sequence's, those before see nothing."""
    m, n, heads, D = 2 ** 31 // 64 + 3, 40, 64, 8
    if torch.cuda.mem_get_info()[0] < 2 * m * heads * D * 4 + 2 ** 33:
        pytest.skip("needs 146 GB of device memory")
    pool = Pool(bec, [n], 16, 1, D, F32, 61)
    q = torch.empty((m, heads, D), dtype=F32, device="cuda")
    q[-n:] = randn((n, heads, D), F32, gen(62))
    out = torch.full((m, heads, D), 7.0, dtype=F32, device="cuda")
    pool.kv.attn_prefill(1, q, pool.seqs, i32([0, m]), out=out)
    pool.kv.check_errors()
    for part in out[:-n].split(2 ** 21):
        assert part.abs().max().item() == 0.0
    check_attn(pool, q[-n:], out[-n:], [n], [n], 0, 0, D ** -0.5)
    del q, out
    torch.cuda.empty_cache()


def test_attention_refusals(bec):
    pool = Pool(bec, [50, 20], 16, 2, 64, BF16, 1)
    kv, q = pool.kv, randn((2, 4, 64), BF16, gen(1))
    with pytest.raises(bec.MoeError, match="layer"):
        kv.attn_decode(2, q, pool.seqs)
    with pytest.raises(bec.MoeError, match="n_q"):
        kv.attn_decode(1, randn((18, 4, 64), BF16, gen(1)), pool.seqs, 9)
    with pytest.raises(bec.MoeError, match="multiple"):
        kv.attn_decode(1, randn((2, 3, 64), BF16, gen(1)), pool.seqs)
    with pytest.raises(bec.MoeError, match="window"):
        kv.attn_decode(1, q, pool.seqs, window=-1)
    with pytest.raises(bec.MoeError, match="scale"):
        kv.attn_decode(1, q, pool.seqs, scale=float("nan"))
    with pytest.raises(ValueError):
        kv.attn_decode(1, q, pool.seqs, 2)
    with pytest.raises(TypeError):
        kv.attn_decode(1, q.float(), pool.seqs)
    with pytest.raises(bec.MoeError, match="aligned"):
        kv.attn_decode(1, randn((2, 4 * 64 + 1), BF16, gen(1))[:, :256].unflatten(1, (4, 64)), pool.seqs)
    with pytest.raises(bec.MoeError, match="page_tokens"):
        bec.KvCache.empty(1, 4, 1, 24, 64, 1, 4)
    with pytest.raises(bec.MoeError, match="head_dim"):
        bec.KvCache.empty(1, 4, 1, 16, 60, 1, 4)
    # found on the device: recorded, reported once, outputs of good rows as ever
    kv.attn_decode(1, q, i32([99, pool.seqs[1].item()]))
    with pytest.raises(bec.MoeError, match="MOE_ERR_ARG"):
        kv.check_errors()
    kv.check_errors()
    kv.attn_prefill(1, q, pool.seqs, i32([0, 5, 2]))
    with pytest.raises(bec.MoeError, match="MOE_ERR_ARG"):
        kv.check_errors()
    # no rows, no sequences
    assert kv.attn_prefill(1, q[:0], pool.seqs, i32([0, 0, 0])).shape == (0, 4, 64)
    assert kv.attn_decode(1, q[:0], i32([])).shape == (0, 4, 64)
    kv.check_errors()


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("cu", [[0, 2, 5], [1, 3, 6], [0, 6, 6]])
def test_attn_prefill_chunks_cover_all_rows(bec, dtype, cu):
    pool = Pool(bec, [40, 9], 16, 2, 64, dtype, 6)
    q = randn((6, 4, 64), dtype, gen(2))
    pool.kv.attn_prefill(1, q, pool.seqs, i32(cu))
    if cu == [0, 6, 6]:
        pool.kv.check_errors()
    else:
        with pytest.raises(bec.MoeError, match="MOE_ERR_ARG"):
            pool.kv.check_errors()


@pytest.mark.parametrize("D", [64, 256])
def test_attn_prefill_rows_without_any_sequence_are_refused(bec, D):
    kv = Pool(bec, [5], 16, 2, D, BF16, 1).kv
    q = randn((6, 4, D), BF16, gen(2))
    with pytest.raises(bec.MoeError, match="without a sequence"):
        kv.attn_prefill(1, q, i32([]), i32([0]))
    assert kv.attn_prefill(1, q[:0], i32([]), i32([0])).shape == (0, 4, D)
    kv.check_errors()


@pytest.mark.parametrize("kind", ["decode", "prefill"])
@pytest.mark.parametrize("dtype,D", [(BF16, 64), (BF16, 128), (BF16, 256), (F32, 96)])
@pytest.mark.parametrize("copies,window", [(0, 0), (0, 200), (1, 0), (7, 0)])
def test_attention_whose_wait_times_out_leaves_the_cache_usable(bec, kind, dtype, D, copies, window):
    """Copies stop after 0, 1 or 7 tiles of a CTA, waits are limited to about 1 ms: an error, no fault; the same call then
    succeeds, twice, so nothing of the first is left in the scratch."""
    lens, ms = ([60000, 3, 700], [8, 8, 8]) if kind == "decode" else ([6000, 3, 700], [6000, 3, 500])
    pool = Pool(bec, lens, 64, 2, D, dtype, 71)
    q = randn((sum(ms), 8, D), dtype, gen(72))
    cu = i32([0, ms[0], ms[0] + ms[1], sum(ms)])

    def call():
        if kind == "decode":
            return pool.kv.attn_decode(1, q, pool.seqs, 8, window=window, sinks=4)
        return pool.kv.attn_prefill(1, q, pool.seqs, cu, window=window, sinks=4)

    good = call()
    pool.kv.check_errors()
    pool.kv.debug_attn_wait_timeout(2_000_000, copies)
    call()
    with pytest.raises(bec.MoeError) as e:
        pool.kv.check_errors()
    assert e.value.status == 5  # MOE_ERR_TIMEOUT
    for _ in range(2):
        assert torch.equal(call(), good)
        pool.kv.check_errors()
    at = sum(ms[:2])
    ref, tol = attn_ref(q[at:], pool.tok_k[2], pool.tok_v[2], lens[2], window, 4, D ** -0.5, dtype)
    assert worst(good[at:], ref, tol) <= 1.0


def test_attention_wait_hook_refusals(bec):
    for args in ((-1, 0), (5, -2)):
        with pytest.raises(bec.MoeError, match="copies"):
            bec.KvCache.debug_attn_wait_timeout(*args)


def test_a_single_row_of_an_odd_stride(bec):
    """The stride of a row that has no next one does not matter."""
    pool = Pool(bec, [50], 16, 2, 64, BF16, 1)
    wide = randn((3, 4 * 64 + 1), BF16, gen(1))
    q = wide[:1, :256].unflatten(1, (4, 64))
    out = torch.zeros((3, 259), dtype=BF16, device="cuda")[:1, :256].unflatten(1, (4, 64))
    want = pool.kv.attn_decode(1, q.contiguous(), pool.seqs)
    assert torch.equal(pool.kv.attn_decode(1, q, pool.seqs, out=out), want) and torch.equal(out, want)
    assert torch.equal(pool.kv.attn_prefill(1, q, pool.seqs, i32([0, 1]), out=out), out)
    check_attn(pool, q, out, [50], [1], 0, 0, 0.125)
    rows = wide[:1, :128].unflatten(1, (2, 64))
    pool.kv.write(1, rows, rows, pool.seqs, i32([0, 1]))
    pool.kv.check_errors()
    page = pool.table[pool.seqs[0], 3].item()
    assert torch.equal(pool.kv.k[1, page, :, 1], rows[0]) and torch.equal(pool.kv.v[1, page, :, 1], rows[0])
    w, (s, c, b) = pack(16, 64, Q4_0, gen(1))
    x = randn((2, 67), BF16, gen(2))[:1, :64]
    ref = x.double() @ (s * c).t()
    assert worst(bec.quant_linear(x, w, Q4_0, 16), ref,
                 U8 * ref.abs() * 1.01 + 200 * U24 * (x.double().abs() @ (s * c).abs().t())) <= 1


# ---------------------------------------------------------------- pages
class Model:
    """The cache's bookkeeping on the host, page by page, with the tokens each page holds."""

    def __init__(self, kv):
        self.kv = kv
        self.table, self.lens, self.ref = kv.table.tolist(), kv.lens.tolist(), kv.ref.tolist()
        self.k, self.v = kv.k.cpu().clone(), kv.v.cpu().clone()
        self.page = kv.k.shape[3]

    def pages(self, n):
        return -(-n // self.page)

    def fork(self, src, dst):
        lens = [self.lens[s] for s in src]
        for s, d, n in zip(src, dst, lens):
            self.lens[d] = n
            for i in range(self.pages(n)):
                self.table[d][i] = self.table[s][i]
                self.ref[self.table[s][i]] += 1

    def reserve(self, seqs, new):
        free = [p for p, r in enumerate(self.ref) if r == 0]
        copies = []
        for s, a in zip(seqs, new):
            n = self.lens[s]
            if a and n % self.page and self.ref[self.table[s][n // self.page]] > 1:
                old, p = self.table[s][n // self.page], free.pop(0)
                self.ref[old] -= 1
                self.ref[p] = 1
                self.table[s][n // self.page] = p
                copies.append((old, p, n % self.page))
            for i in range(self.pages(n), self.pages(n + a)):
                p = free.pop(0)
                self.ref[p] = 1
                self.table[s][i] = p
            self.lens[s] += a
        for old, p, f in copies:
            self.k[:, p, :, :f] = self.k[:, old, :, :f]
            self.v[:, p, :, :f] = self.v[:, old, :, :f]

    def write(self, layer, k, v, seqs, cu):
        for i, s in enumerate(seqs):
            for r in range(cu[i], cu[i + 1]):
                t = self.lens[s] - (cu[i + 1] - r)
                p = self.table[s][t // self.page]
                self.k[layer, p, :, t % self.page] = k[r]
                self.v[layer, p, :, t % self.page] = v[r]

    def free(self, seqs):
        for s in seqs:
            for i in range(self.pages(self.lens[s])):
                self.ref[self.table[s][i]] -= 1
                self.table[s][i] = -1
            self.lens[s] = 0

    def compact(self):
        live = sum(r > 0 for r in self.ref)
        src = [p for p in range(live, len(self.ref)) if self.ref[p]]
        dst = [p for p in range(live) if not self.ref[p]]
        to = dict(zip(src, dst))
        for s, d in to.items():
            self.k[:, d], self.v[:, d] = self.k[:, s].clone(), self.v[:, s].clone()
            self.ref[d], self.ref[s] = self.ref[s], 0
        self.table = [[to.get(p, p) for p in row] for row in self.table]

    def check(self):
        assert self.kv.lens.tolist() == self.lens
        assert self.kv.table.tolist() == self.table
        assert self.kv.ref.tolist() == self.ref
        assert torch.equal(self.kv.k.cpu(), self.k) and torch.equal(self.kv.v.cpu(), self.v)


@pytest.mark.parametrize("dtype,page,hkv,D,pages", [(BF16, 16, 2, 64, 400), (F32, 32, 1, 24, 150), (BF16, 64, 3, 8, 4500)])
def test_page_calls_match_a_host_model(bec, dtype, page, hkv, D, pages):
    rng = random.Random(pages)
    S, layers = 40, 2
    kv = bec.KvCache.empty(layers, pages, hkv, page, D, S, max_pages=pages // 4, dtype=dtype)
    kv.k.copy_(randn(kv.k.shape, dtype, gen(1)))
    kv.v.copy_(randn(kv.v.shape, dtype, gen(2)))
    m = Model(kv)
    g = gen(3)
    for step in range(30):
        used = [s for s in range(S) if m.lens[s]]
        idle = [s for s in range(S) if not m.lens[s]]
        op = rng.choice(["grow", "grow", "fork", "free", "compact"])
        if op == "grow":
            seqs = rng.sample(range(S), rng.randint(1, S // 2))
            new = [rng.choice([0, 1, 1, 3, page, 2 * page + 5]) for _ in seqs]
            if sum(m.pages(a) + 2 for a in new) > m.ref.count(0) or any(
                    m.pages(m.lens[s] + a) > pages // 4 for s, a in zip(seqs, new)):
                continue
            kv.reserve(i32(seqs), i32(new))
            m.reserve(seqs, new)
            cu = [0]
            for a in new:
                cu.append(cu[-1] + a)
            for layer in range(layers):
                fused = randn((cu[-1], 2 * hkv * D + 8), dtype, g)
                k = fused[:, :hkv * D].unflatten(1, (hkv, D))
                v = fused[:, hkv * D:2 * hkv * D].unflatten(1, (hkv, D))
                kv.write(layer, k, v, i32(seqs), i32(cu))
                m.write(layer, k.cpu(), v.cpu(), seqs, cu)
        elif op == "fork" and used and idle:
            dst = rng.sample(idle, rng.randint(1, min(6, len(idle))))
            src = [rng.choice(used + dst[:1]) for _ in dst]
            kv.fork(i32(src), i32(dst))
            m.fork(src, dst)
        elif op == "free" and used:
            seqs = rng.sample(used, rng.randint(1, max(1, len(used) // 2)))
            kv.free(i32(seqs))
            m.free(seqs)
        elif op == "compact":
            kv.compact()
            m.compact()
        kv.check_errors()
        m.check()


def test_copy_on_write_keeps_one_owner(bec):
    """Sharers of one partial page: with an unlisted one all copy; with all listed the last keeps it."""
    for listed, copies in (([1, 2], 2), ([0, 1, 2], 2), ([2], 1)):
        kv = bec.KvCache.empty(1, 16, 1, 16, 8, 4, 4)
        kv.reserve(i32([0]), i32([20]))
        kv.fork(i32([0, 0]), i32([1, 2]))
        m = Model(kv)
        kv.reserve(i32(listed), i32([1] * len(listed)))
        m.reserve(listed, [1] * len(listed))
        kv.check_errors()
        m.check()
        assert sum(r > 0 for r in m.ref) == 2 + copies


def test_page_calls_refuse_and_change_nothing(bec):
    kv = bec.KvCache.empty(1, 8, 1, 16, 64, 4, max_pages=5)
    kv.reserve(i32([0, 1]), i32([40, 30]))  # 3 + 2 pages
    kv.check_errors()
    m = Model(kv)

    def refused(status, call):
        call()
        kv.reserve(i32([1]), i32([1]))  # does nothing while the failure is pending
        kv.compact()
        with pytest.raises(bec.MoeError, match=status):
            kv.check_errors()
        kv.check_errors()
        m.check()

    refused("CAPACITY", lambda: kv.reserve(i32([0, 2]), i32([8, 64])))   # 4 pages of 3
    refused("CAPACITY", lambda: kv.reserve(i32([0]), i32([41])))         # 81 tokens in rows of 80
    refused("ARG", lambda: kv.reserve(i32([2, 2]), i32([1, 1])))
    refused("ARG", lambda: kv.reserve(i32([4]), i32([1])))
    refused("ARG", lambda: kv.reserve(i32([2]), i32([-1])))
    refused("ARG", lambda: kv.fork(i32([0]), i32([1])))
    refused("ARG", lambda: kv.fork(i32([0, 1]), i32([2, 2])))
    refused("ARG", lambda: kv.fork(i32([-1]), i32([2])))
    refused("ARG", lambda: kv.free(i32([0, 0])))
    refused("ARG", lambda: kv.copy_pages(i32([0]), i32([8])))
    rows = randn((41, 1, 64), BF16, gen(1))
    refused("STATE", lambda: kv.write(0, rows, rows, i32([0]), i32([0, 41])))
    kv.fork(i32([0]), i32([3]))
    m.fork([0], [3])
    refused("STATE", lambda: kv.write(0, rows[:1], rows[:1], i32([0]), i32([0, 1])))
    with pytest.raises(bec.MoeError, match="n outside"):
        kv.free(torch.zeros(9000, dtype=torch.int32, device="cuda"))
    kv.reserve(i32([]), i32([]))
    kv.free(i32([]))
    kv.check_errors()
    m.check()


@pytest.mark.parametrize("n,each", [(32, 2 ** 30), (64, 2 ** 30), (64, 2 ** 30 - 15)])
def test_reserve_of_more_pages_than_32_bits_count(bec, n, each):
    """Requests that each fit their table row, 2^31 and 2^32 pages together (or a few less than a whole page's)."""
    W = 2 ** 26
    k = torch.zeros((1, 8, 1, 16, 8), dtype=BF16, device="cuda")
    table = torch.empty((n, W), dtype=torch.int32, device="cuda")
    kv = bec.KvCache(k, k.clone(), table, i32([0] * n), i32([0] * 8))
    kv.reserve(i32(range(n)), i32([each] * n))
    with pytest.raises(bec.MoeError, match="CAPACITY"):
        kv.check_errors()
    assert kv.lens.tolist() == [0] * n and kv.ref.tolist() == [0] * 8
    # a request behind them that fits is granted alone
    table[1, :2] = -1
    kv.reserve(i32([1]), i32([20]))
    kv.check_errors()
    assert kv.lens.tolist() == [0, 20] + [0] * (n - 2) and table[1, :2].tolist() == [0, 1]


@pytest.mark.parametrize("n,bad", [(3, 1), (600, 599), (2200, 0), (2200, 700), (2200, 2199)])
@pytest.mark.parametrize("which", ["src", "dst"])
def test_copy_pages_with_one_bad_id_copies_nothing(bec, n, bad, which):
    """Lists good but for one entry, short ones and more work than the GPU holds blocks at once."""
    kv = bec.KvCache.empty(2, 4500, 2, 16, 64, 1, 4)
    kv.k.copy_(randn(kv.k.shape, BF16, gen(1)))
    kv.v.copy_(randn(kv.v.shape, BF16, gen(2)))
    k, v = kv.k.clone(), kv.v.clone()
    lists = dict(src=torch.arange(n, dtype=torch.int32, device="cuda"),
                 dst=torch.arange(2250, 2250 + n, dtype=torch.int32, device="cuda"))
    good = lists[which][bad].item()
    for wrong in (-1, 4500, 2 ** 31 - 1):
        lists[which][bad] = wrong
        kv.copy_pages(lists["src"], lists["dst"])
        with pytest.raises(bec.MoeError, match="MOE_ERR_ARG"):
            kv.check_errors()
        assert torch.equal(kv.k, k) and torch.equal(kv.v, v)
    lists[which][bad] = good
    kv.copy_pages(lists["src"], lists["dst"])
    kv.check_errors()
    k[:, 2250:2250 + n], v[:, 2250:2250 + n] = k[:, :n], v[:, :n]
    assert torch.equal(kv.k, k) and torch.equal(kv.v, v)


@pytest.mark.parametrize("n", [5, 8, 9, 100, 255, 20000])
@pytest.mark.parametrize("where", [0.0, 0.5, 1.0])
@pytest.mark.parametrize("kind", ["shared", "long", "id"])
def test_write_leaves_out_what_is_wrong_and_writes_the_rest(bec, n, where, kind):
    """One token a sequence, up to more blocks than the GPU holds at once; one entry of the list is bad."""
    kv = bec.KvCache.empty(1, n + 5, 1, 16, 8, n + 2, 1)
    for at in range(0, n, 8192):
        seqs = torch.arange(at, min(n, at + 8192), dtype=torch.int32, device="cuda")
        kv.reserve(seqs, torch.ones_like(seqs))
    bad = int(where * (n - 1))
    seqs = torch.arange(n, dtype=torch.int32, device="cuda")
    rows = torch.arange(n + 1, dtype=torch.int32, device="cuda")  # cu
    if kind == "shared":
        kv.fork(seqs[bad:bad + 1].clone(), i32([n]))
    elif kind == "long":
        rows[bad + 1:] += 1
    else:
        seqs[bad] = n + 2
    pages = kv.table[:n, 0].long()
    for step in range(3):
        k, v = randn((n + 1, 1, 8), BF16, gen(step)), randn((n + 1, 1, 8), BF16, gen(9 + step))
        m = n + (kind == "long")
        old_k, old_v = kv.k.clone(), kv.v.clone()
        kv.write(0, k[:m], v[:m], seqs, rows)
        first_k, first_v = kv.k.clone(), kv.v.clone()
        kv.write(0, v[:m], k[:m], seqs, rows)  # does nothing while the failure is pending
        with pytest.raises(bec.MoeError, match="MOE_ERR_ARG" if kind == "id" else "MOE_ERR_STATE"):
            kv.check_errors()
        kv.check_errors()
        good = torch.arange(n, device="cuda") != bad
        src = rows[:n].long()[good]
        old_k[0, pages[good], :, 0], old_v[0, pages[good], :, 0] = k[src], v[src]
        assert torch.equal(first_k, old_k) and torch.equal(first_v, old_v)
        assert torch.equal(kv.k, old_k) and torch.equal(kv.v, old_v)


@pytest.mark.parametrize("cu", [[0, 20, 41], [0, 20, 30, 50], [0, 20, 40, 45], [-1, 20, 40],
                                [0, 40, 2 ** 31 - 1]])
def test_write_of_chunks_that_pass_the_rows(bec, cu):
    """40 rows; chunks that need more are left as they were and recorded, the others are written."""
    n = len(cu) - 1
    kv = bec.KvCache.empty(1, 40, 1, 16, 8, n, 8)
    seqs = i32(range(n))
    kv.reserve(seqs, i32([60] * n))
    kv.check_errors()
    k, v = randn((40, 1, 8), BF16, gen(1)), randn((40, 1, 8), BF16, gen(2))
    ref_k, ref_v = kv.k.clone(), kv.v.clone()
    kv.write(0, k, v, seqs, i32(cu))
    with pytest.raises(bec.MoeError, match="MOE_ERR_ARG"):
        kv.check_errors()
    for b in range(n):
        if cu[b] < 0 or cu[b + 1] > 40:
            continue
        for r in range(cu[b], cu[b + 1]):
            t = 60 - (cu[b + 1] - r)
            p = kv.table[b, t // 16].item()
            ref_k[0, p, :, t % 16], ref_v[0, p, :, t % 16] = k[r], v[r]
    assert torch.equal(kv.k, ref_k) and torch.equal(kv.v, ref_v)


@pytest.mark.parametrize("call", ["decode", "prefill", "linear"])
def test_new_results_are_of_the_calls_stream(bec, call):
    """Memory that the current stream has yet to read is not written by a call on another one."""
    pool = Pool(bec, [50] * 256, 16, 8, 128, BF16, 1)
    q = randn((256, 64, 128), BF16, gen(1))
    w, _ = pack(8192, 64, Q4_0, gen(2))
    x = randn((256, 64), BF16, gen(3))
    cu, side = i32(range(257)), torch.cuda.Stream()

    def run():
        if call == "decode":
            return pool.kv.attn_decode(1, q, pool.seqs, stream=side)
        if call == "prefill":
            return pool.kv.attn_prefill(1, q, pool.seqs, cu, stream=side)
        return bec.quant_linear(x, w, Q4_0, 8192, stream=side)

    torch.cuda.synchronize()
    run()  # a first launch loads the kernel, which waits for the device
    torch.cuda.synchronize()
    torch.cuda.empty_cache()
    # two blocks of the results' size; the second is free again at once as far as the current stream goes
    was = torch.randn((256, 8192)).bfloat16()
    copy = torch.empty(was.shape, dtype=BF16, device="cuda")
    mine = torch.empty(was.shape, dtype=BF16, device="cuda")
    mine.copy_(was)
    torch.cuda._sleep(200_000_000)  # about 0.1 s
    copy.copy_(mine)
    del mine
    out = run()
    torch.cuda.synchronize()
    assert torch.equal(copy.cpu(), was)
    assert torch.isfinite(out).all()


def test_scratch_is_zero_on_whichever_stream_comes_first(bec):
    k = torch.zeros((1, 8, 1, 16, 64), dtype=BF16, device="cuda")
    v, table = torch.zeros_like(k), torch.full((2, 4), -1, dtype=torch.int32, device="cuda")
    lens, ref, seqs, new = i32([0, 0]), i32([0] * 8), i32([1]), i32([40])
    side = torch.cuda.Stream()
    kv = bec.KvCache(k, v, table, lens, ref)
    n = kv.work.numel()
    torch.cuda.synchronize()
    kv.reserve(seqs, i32([0]), stream=side)  # a first launch loads the kernels, which waits for the device
    torch.cuda.synchronize()
    del kv
    torch.cuda.empty_cache()
    junk = torch.full((n,), 255, dtype=torch.uint8, device="cuda")
    torch.cuda.synchronize()
    del junk
    torch.cuda._sleep(200_000_000)
    kv = bec.KvCache(k, v, table, lens, ref)
    kv.reserve(seqs, new, stream=side)
    side.synchronize()
    assert lens.tolist() == [0, 40] and table[1].tolist() == [0, 1, 2, -1]
    kv.check_errors()


def test_decode_step_in_a_graph_on_another_stream(bec):
    """reserve, write and attention captured once and replayed as the sequences grow."""
    dtype, hkv, hq, D, page = BF16, 2, 8, 64, 16
    kv = bec.KvCache.empty(1, 64, hkv, page, D, 3, 16, dtype=dtype)
    kv.k.fill_(float("nan"))
    kv.v.fill_(float("nan"))
    seqs, ones, cu = i32([2, 0]), i32([1, 1]), i32([0, 1, 2])
    qkv = torch.zeros((2, (hq + 2 * hkv) * D), dtype=dtype, device="cuda")
    q = qkv[:, :hq * D].unflatten(1, (hq, D))
    k = qkv[:, hq * D:(hq + hkv) * D].unflatten(1, (hkv, D))
    v = qkv[:, (hq + hkv) * D:].unflatten(1, (hkv, D))
    out = torch.zeros((2, hq, D), dtype=dtype, device="cuda")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())

    def step():
        kv.reserve(seqs, ones, stream=side)
        kv.write(0, k, v, seqs, cu, stream=side)
        kv.attn_decode(0, q, seqs, out=out, stream=side)

    g = gen(17)
    toks = [[], []]
    with torch.cuda.stream(side):
        qkv.copy_(randn(qkv.shape, dtype, g))
        step()  # first use outside of the capture
    side.synchronize()
    hist = [(k.clone(), v.clone())]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        step()
    for i in range(40):
        qkv.copy_(randn(qkv.shape, dtype, g))
        hist.append((k.clone(), v.clone()))
        graph.replay()
        torch.cuda.synchronize()
        for b in range(2):
            tk = torch.stack([h[0][b] for h in hist])
            tv = torch.stack([h[1][b] for h in hist])
            ref, tol = attn_ref(q[b:b + 1], tk, tv, len(hist), 0, 0, D ** -0.5, dtype)
            assert worst(out[b:b + 1], ref, tol) <= 1.0
    kv.check_errors()
    assert kv.lens.tolist() == [41, 0, 41]
    assert kv.token_bytes == 2 * hkv * D * 2
