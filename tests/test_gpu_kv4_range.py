"""GPU tests of attention over pages of 4-bit codes far from magnitudes of 1: powers of two that
rows, tiles and units are divided by, weights far below a row's largest, and units of many kinds
in one call, against 64 bits."""
import pytest
import torch

pytestmark = pytest.mark.gpu

BF16, F32 = torch.bfloat16, torch.float32
U24, U11, U8 = 2.0 ** -24, 2.0 ** -11, 2.0 ** -8  # unit roundoffs of fp32, f16 and bf16
PAGE = 16


@pytest.fixture(scope="module")
def bec():
    import bounded_expert_cache_gb300 as m
    return m


def gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def i32(x):
    return torch.tensor(list(x), dtype=torch.int32, device="cuda")


def coded(x):
    """Bytes of a token's and head's codes, its scales and offsets as bytes, and the parts in 64 bits, of fp32 [n, hkv, D]."""
    g = x.unflatten(-1, (-1, 64))
    b = g.amin(-1, keepdim=True).bfloat16()
    s = ((g.amax(-1, keepdim=True) - b.float()) / 15.0).bfloat16()
    q = torch.where(s > 0, torch.round((g - b.float()) / torch.where(s > 0, s, torch.ones_like(s)).float()).clamp(0, 15), torch.zeros_like(g))
    codes = q.to(torch.uint8).flatten(-2)
    wide = lambda t: t.double().expand(g.shape).flatten(-2)  # noqa: E731
    parts = (wide(s), q.double().flatten(-2) - 8, wide(b) + 8 * wide(s))
    return codes[..., 0::2] | (codes[..., 1::2] << 4), torch.cat([s, b], -1).contiguous().view(torch.uint8).flatten(-2), parts


class Pool:
    """A cache of codes of the sequences' keys and values (lists of fp32 [n, hkv, D]), page after page."""

    def __init__(self, bec, keys, values, dtype):
        self.lens = [k.shape[0] for k in keys]
        hkv, D = keys[0].shape[1:]
        need = [-(-n // PAGE) for n in self.lens]
        P, S = sum(need) + 1, len(keys)
        first = torch.tensor([sum(need[:b]) for b in range(S)])
        table = torch.full((S, max(need) + 1), -1, dtype=torch.int32)
        for b in range(S):
            table[b, :need[b]] = torch.arange(need[b]) + first[b]
        ref = torch.ones(P, dtype=torch.int32, device="cuda")
        ref[P - 1] = 0
        pools, parts = [], []
        at = torch.cat([torch.arange(n) + first[b] * PAGE for b, n in enumerate(self.lens)]).cuda()
        for xs in (keys, values):
            codes, meta, whole = coded(torch.cat(xs))
            flat = torch.zeros((P * PAGE, hkv, D // 2), dtype=torch.uint8, device="cuda")
            flat[at] = codes
            flat_meta = torch.zeros((P * PAGE, hkv, D // 16), dtype=torch.uint8, device="cuda")
            flat_meta[at] = meta
            blocks = [t.unflatten(0, (P, PAGE)).transpose(1, 2).reshape(P, hkv, -1) for t in (flat, flat_meta)]
            pools.append(torch.cat(blocks, -1).view(1, P, hkv, PAGE, D * 9 // 16).contiguous())
            parts.append([tuple(p[b] for p in [t.split(self.lens) for t in whole]) for b in range(S)])
        self.k, self.v = parts
        self.D, self.dtype = D, dtype
        self.kv = bec.KvCache(pools[0], pools[1], table.cuda(), i32(self.lens), ref, dtype)
        self.seqs = i32(range(S))


def expected(pool, b, q, scale, window, sinks, chunk):
    """Rows of the sequence's newest tokens in 64 bits, and their tolerance, [m, hq, D]."""
    (ks, kq, kb), (vs, vq, vb) = pool.k[b], pool.v[b]
    m, hq, D = q.shape
    n, hkv = ks.shape[:2]
    x = q.double().unflatten(1, (hkv, hq // hkv))
    K, V = ks * kq + kb, vs * vq + vb
    p, j = torch.arange(n - m, n, device="cuda")[:, None], torch.arange(n, device="cuda")[None]
    see = (j <= p) & ((p - j < window) | (j < sinks) if window else torch.ones_like(j, dtype=torch.bool))
    hidden = ~see[:, None, None, :]
    s = (torch.einsum("mhgd,jhd->mhgj", x, K) * scale).masked_fill(hidden, -float("inf"))
    w = torch.softmax(s, -1)
    over = lambda t: torch.einsum("mhgj,jhd->mhgd", w, t)  # noqa: E731
    out, A, R = over(V), over((vs * vq).abs() + vb.abs()), over((vs * vq).abs())
    reach = lambda t: (torch.einsum("mhgd,jhd->mhgj", x.abs(), t.abs()) * scale).masked_fill(hidden, 0).amax(-1, keepdim=True)  # noqa: E731
    # a score: products in fp32 or exact, sums in fp32, twice the unit for the matrix units';
    # the same in the quotient and above it; the exponential, and the sums of n terms
    delta = 2 * (D + 16) * U24 * reach((ks * kq).abs() + kb.abs())
    if chunk and pool.dtype == BF16 and D <= 128:
        # a key's value is rounded to f16, u11 of itself, which moves every weight by up to
        # e^(+-2 of a score's error); a value and a numerator are rounded to f16 once each, a numerator
        # below 2^-24 of the row's largest by half of f16's last step there
        t = (torch.expm1(2 * delta + 2 * U11 * reach(K)) + 2.01 * U11) * A
        most = V.abs()
    else:
        t = torch.expm1(2 * delta) * A
        most = 8 * vs.abs()
        if pool.dtype == BF16:
            # the numerator times the scale is rounded to f16, likewise
            t = t + 1.01 * U11 * R
    t = t + (64 + n / 8) * 2 * U24 * A
    if pool.dtype == BF16:
        t = t + 1.01 * U8 * out.abs()
        least = see.sum(-1)[:, None, None] * 2.0 ** -35
        top = torch.stack([most[r].amax(0) for r in see]).unflatten(-1, (D,)) if window else most.cummax(0).values[n - m:]
        # (the weights' sum is at least the largest weight)
        t = t + (least * top)[:, :, None, :]
    return out.flatten(1, 2), t.flatten(1, 2) + 1e-300


def check(pool, kind, q, ms, scale, window=0, sinks=0):
    cu = i32([sum(ms[:i]) for i in range(len(ms) + 1)])
    if kind == "decode":
        out = pool.kv.attn_decode(0, q, pool.seqs, ms[0], scale=scale, window=window, sinks=sinks)
    else:
        out = pool.kv.attn_prefill(0, q, pool.seqs, cu, scale=scale, window=window, sinks=sinks)
    pool.kv.check_errors()
    at = 0
    for b, m in enumerate(ms):
        ref, tol = expected(pool, b, q[at:at + m], scale, window, sinks, kind == "prefill")
        got = out[at:at + m].double()
        assert torch.isfinite(got).all(), (b, "not finite")
        ratio = ((got - ref).abs() / tol).max().item()
        assert ratio <= 1.0, (b, m, ratio)
        at += m
    return out


def made(bec, lens, hkv, D, dtype, seed, k=1.0, v=1.0):
    """Random keys and values times k and v (numbers, or tensors of [n, D] for one sequence)."""
    g = gen(seed)
    rand = lambda n, f: (torch.randn((n, hkv, D), device="cuda", generator=g) + 0.3) * (f if not torch.is_tensor(f) else f[:, None, None])  # noqa: E731
    keys, values = [rand(n, k) for n in lens], [rand(n, v) for n in lens]
    return Pool(bec, keys, values, dtype)


def queries(rows, hq, D, dtype, seed, f=1.0):
    return (torch.randn((rows, hq, D), device="cuda", generator=gen(seed)) * f).to(dtype)


CALLS = [("decode", 64), ("decode", 128), ("decode", 256), ("prefill", 64), ("prefill", 128), ("prefill", 192)]
SIZES = [(4, 300), (4, 40)]


def chunks(kind, lens):
    return [4] * len(lens) if kind == "decode" else [min(n, 140) for n in lens]


# ---------------------------------------------------------------- scores beyond fp32's smallest
@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("kind,D", CALLS)
@pytest.mark.parametrize("q,k,scale", [(2.0 ** -70, 2.0 ** -70, 0.1), (2.0 ** -110, 2.0 ** -20, 1e-30), (2.0 ** -115, 1.0, 1e-37)])
def test_scores_that_are_nothing_weigh_evenly(bec, dtype, kind, D, q, k, scale):
    lens = [300, 40]
    pool = made(bec, lens, 2, D, dtype, 1, k=k)
    ms = chunks(kind, lens)
    check(pool, kind, queries(sum(ms), 4, D, dtype, 2, q), ms, scale)
    check(pool, kind, queries(sum(ms), 4, D, dtype, 2, q), ms, scale, window=30, sinks=3)


# ---------------------------------------------------------------- magnitudes
@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("kind,D", CALLS)
@pytest.mark.parametrize("q,k,v", [(16, -12, -70), (-70, 16, 16), (-12, -70, 60), (16, -90, -100), (60, -70, -12), (-60, 95, 100), (0, 0, 0)])
def test_queries_keys_and_values_of_any_magnitude(bec, dtype, kind, D, q, k, v):
    lens = [300, 40]
    pool = made(bec, lens, 2, D, dtype, 3, k=2.0 ** k, v=2.0 ** v)
    ms = chunks(kind, lens)
    check(pool, kind, queries(sum(ms), 8, D, dtype, 4, 2.0 ** q), ms, D ** -0.5 * 2.0 ** -(q + k))


# ---------------------------------------------------------------- queries' and keys' columns, and rows, of different magnitudes
@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("kind,D", [c for c in CALLS if c[1] > 64])
def test_columns_of_queries_and_keys_that_make_up_for_each_other(bec, dtype, kind, D):
    lens = [300, 40]
    pool = made(bec, lens, 2, D, dtype, 5)
    g = gen(5)
    keys = [torch.randn((n, 2, D), device="cuda", generator=g) for n in lens]
    values = [torch.randn((n, 2, D), device="cuda", generator=g) for n in lens]
    for x in keys:
        x[..., 64:] *= 2.0 ** -20
    pool = Pool(bec, keys, values, dtype)
    ms = chunks(kind, lens)
    q = queries(sum(ms), 8, D, F32, 6)
    q[..., :64] *= 2.0 ** -20
    check(pool, kind, q.to(dtype), ms, 2.0 ** 20 * D ** -0.5)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("kind,D", CALLS)
def test_rows_of_queries_of_different_magnitudes(bec, dtype, kind, D):
    """Some rows' queries are 2^-22 of their neighbours' and see keys that the others do not tell apart."""
    lens = [300, 40]
    pool = made(bec, lens, 2, D, dtype, 7, k=2.0 ** 20)
    ms = chunks(kind, lens)
    q = queries(sum(ms), 8, D, F32, 8, 2.0 ** -20)
    q[1::2] = 0
    q[1::2, :, 0] = 4.0
    check(pool, kind, q.to(dtype), ms, D ** -0.5)


# ---------------------------------------------------------------- values
@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("kind,D", [c for c in CALLS if c[1] > 64])
def test_groups_of_values_2_20_apart(bec, dtype, kind, D):
    lens = [300, 40]
    g = gen(9)
    keys = [torch.randn((n, 2, D), device="cuda", generator=g) for n in lens]
    values = [torch.randn((n, 2, D), device="cuda", generator=g) + 0.3 for n in lens]
    for x in values:
        x[..., 64:] *= 2.0 ** -20
    pool = Pool(bec, keys, values, dtype)
    ms = chunks(kind, lens)
    check(pool, kind, queries(sum(ms), 8, D, dtype, 10), ms, D ** -0.5)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("kind,D", CALLS)
@pytest.mark.parametrize("exponents,window", [((0, 10, 20), 0), ((20, 10, 0), 100), ((0, 20, 5), 100), ((-60, -70, -50), 0), ((0, 3, 6, 1, 9), 0)])
def test_values_whose_size_changes_from_tile_to_tile(bec, dtype, kind, D, exponents, window):
    n = 128 * len(exponents)
    f = torch.tensor([2.0 ** e for e in exponents], device="cuda").repeat_interleave(128)
    pool = made(bec, [n], 2, D, dtype, 11, v=f)
    ms = [8 if kind == "decode" else n]
    check(pool, kind, queries(ms[0], 4, D, dtype, 12), ms, D ** -0.5, window, 2 if window else 0)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("kind,D", CALLS)
@pytest.mark.parametrize("what", ["keys", "values"])
def test_tiles_of_zeros_and_of_small_keys(bec, dtype, kind, D, what):
    n = 384
    f = torch.tensor([0.0, 1.0, 2.0 ** -14] if what == "keys" else [0.0, 2.0 ** -30, 0.0], device="cuda").repeat_interleave(128)
    pool = made(bec, [n], 2, D, dtype, 13, **{"k" if what == "keys" else "v": f})
    ms = [8 if kind == "decode" else n]
    check(pool, kind, queries(ms[0], 4, D, dtype, 14), ms, D ** -0.5)


# ---------------------------------------------------------------- weights
@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("kind,D", CALLS)
@pytest.mark.parametrize("bits", [20, 24, 27])
@pytest.mark.parametrize("at", [0, 1000, 2047])
def test_many_tokens_far_below_the_largest(bec, dtype, kind, D, bits, at):
    """One token outweighs each of the others by 2^bits, and its values are zeros. Heads enough for one block to see it all."""
    n, hkv = 2048, 152
    keys = torch.zeros((n, hkv, D), device="cuda")
    keys[at, :, 0::64] = 15.0  # (exact in codes)
    values = torch.rand((n, hkv, D), device="cuda", generator=gen(15)) + 0.5
    values[at] = 0.0
    pool = Pool(bec, [keys], [values], dtype)
    q = torch.zeros((2, hkv, D), dtype=dtype, device="cuda")
    q[..., 0] = 1.0
    check(pool, kind, q, [2], bits * 0.6931471805599453 / 15.0)


# ---------------------------------------------------------------- units of many kinds in one call
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("lone", [7, 15])
def test_chunks_of_one_and_two_row_tiles_whose_queries_differ(bec, D, lone):
    """Chunks of 200 rows between `lone` of 100: the second row tile has work in every eighth unit of a block or so."""
    n_seqs = 152 * 4 * (lone + 1)
    two = [b % (lone + 1) == 0 for b in range(n_seqs)]
    ms = [200 if t else 100 for t in two]
    g = gen(16)
    T = sum(ms)
    k, v = (torch.randn((T, 1, D), device="cuda", generator=g) for _ in range(2))
    kv = bec.KvCache.empty(1, sum(-(-m // PAGE) for m in ms), 1, PAGE, D, n_seqs, 16, bits=4)
    seqs = i32(range(n_seqs))
    for s in range(0, n_seqs, 8000):
        kv.reserve(seqs[s:s + 8000].contiguous(), i32(ms[s:s + 8000]))
    cu = torch.tensor([0] + ms).cumsum(0).int().cuda()
    kv.write(0, k.bfloat16(), v.bfloat16(), seqs, cu)
    kv.check_errors()
    # a chunk's queries are 2^16, 2^18 or 2^20 times the usual ones, in turn
    size = torch.tensor([2.0 ** (16 + 2 * ((b // (lone + 1)) % 3)) for b in range(n_seqs)]).repeat_interleave(torch.tensor(ms)).cuda()
    x = torch.randn((T, 1, D), device="cuda", generator=g)
    scale = D ** -0.5 * 2.0 ** -18
    q = (x * size[:, None, None]).bfloat16()
    got = kv.attn_prefill(0, q, seqs, cu, scale=scale)
    kv.check_errors()
    # the same rows of chunks of 200 alone
    alone = torch.tensor([b for b in range(n_seqs) if two[b]])
    rows = torch.cat([torch.arange(int(cu[b]), int(cu[b + 1])) for b in alone]).cuda()
    want = kv.attn_prefill(0, q[rows].contiguous(), alone.int().cuda(), i32(range(0, 200 * len(alone) + 1, 200)), scale=scale)
    kv.check_errors()
    a, b = got[rows].float(), want.float()
    # (how the work is cut may move a sum's last bit, and so a result by one step of bf16)
    assert ((a - b).abs() <= 2 * U8 * b.abs() + 1e-4 * b.abs().max()).all(), (a - b).abs().max().item()


@pytest.mark.parametrize("bits", [4, 0])
@pytest.mark.parametrize("D", [64, 128])
def test_nan_of_many_short_units(bec, bits, D):
    """Units of one and two row tiles, each with a NaN among its values that its last rows see: those and no others are NaN."""
    lone, hkv = 7, 2
    n_seqs = 152 * 3 * (lone + 1)
    ms = [200 if b % (lone + 1) == 0 else 40 for b in range(n_seqs)]
    T = sum(ms)
    g = gen(17)
    k, v = (torch.randn((T, hkv, D), device="cuda", generator=g).bfloat16() for _ in range(2))
    cu = torch.tensor([0] + ms).cumsum(0)
    # token 3/4 through each chunk; in every third none
    bad = torch.tensor([int(cu[b]) + ms[b] * 3 // 4 for b in range(n_seqs) if b % 3])
    v[bad.cuda()] = float("nan")
    kv = bec.KvCache.empty(1, sum(-(-m // PAGE) for m in ms), hkv, PAGE, D, n_seqs, 16, bits=bits)
    seqs = i32(range(n_seqs))
    kv.reserve(seqs, i32(ms))
    cu = cu.int().cuda()
    kv.write(0, k, v, seqs, cu)
    q = torch.randn((T, hkv, D), device="cuda", generator=g).bfloat16()
    want = torch.zeros(T, dtype=torch.bool)
    first = cu.tolist()
    for b in range(n_seqs):
        if b % 3:
            want[first[b] + ms[b] * 3 // 4:first[b + 1]] = True
    for _ in range(10):
        out = kv.attn_prefill(0, q, seqs, cu)
        assert torch.equal(torch.isnan(out).all(-1).all(-1).cpu(), want)
        assert torch.equal(torch.isnan(out).any(-1).any(-1).cpu(), want)
    kv.check_errors()
