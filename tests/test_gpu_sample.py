"""GPU tests of sampling against its definition in 64 bits on the host."""
import numpy as np
import pytest
import torch

from test_gpu_kv import gen

pytestmark = pytest.mark.gpu
BF16, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module")
def bec():
    import bounded_expert_cache_gb300 as m
    return m


def outcomes(z, u, temperature, k, p, floor):
    """(token, probability) of a row, and of it with its sums off by what weights may be: about 2^-31 of themselves and 2^-43."""
    z = np.where(np.isnan(z), -np.inf, z)
    order = np.lexsort((np.arange(z.size), -z))
    top = z[order[0]]
    if top == -np.inf:
        return [(-1, 0.0)]
    if not temperature > 0 or k == 1:
        return [(int(order[0]), 1.0)]
    with np.errstate(invalid="ignore", over="ignore"):
        weight = np.where(z[order] == top, 1.0, np.exp((z[order] - top) / temperature))
    weight[(z[order] == -np.inf) | ((top == np.inf) & (z[order] != top))] = 0.0  # infinite logits share it all
    if k > 0:
        weight = np.where(np.arange(z.size) < k, weight, 0.0)
    got = []
    eps = 2.0 ** -29 + z.size * 2.0 ** -43
    for a in ((0,) if p >= 1 else (0, -eps, eps)):
        w = weight
        if p < 1:
            before = np.cumsum(w) - w
            w = np.where((before < p * (1 + a) * w.sum()) | (np.arange(z.size) == 0), w, 0.0)
        for f in ((0,) if floor <= 0 else (0, -eps, eps)):
            x = np.where(w >= min(floor, 1.0) * (1 + f), w, 0.0) if floor > 0 else w
            x[0] = w[0]
            by_index = np.zeros_like(x)
            by_index[order] = x
            sums = np.cumsum(by_index)
            for b in (0, -eps, eps):
                i = int(np.searchsorted(sums, u * sums[-1] * (1 + b), side="right"))
                i = min(i, int(np.nonzero(by_index)[0][-1]))
                got.append((i, by_index[i] / sums[-1]))
    return got


def check(bec, z, u, temperature=1.0, top_k=0, top_p=1.0, min_p=0.0):
    token, prob = bec.sample(z, u, temperature, top_k, top_p, min_p)
    n = z.shape[0]
    cols = [x.tolist() if isinstance(x, torch.Tensor) else [x] * n for x in (temperature, top_k, top_p, min_p)]
    zs = z.double().cpu().numpy()
    odd = 0
    for r in range(n):
        t, p, f = (np.float64(np.float32(cols[i][r])) for i in (0, 2, 3))  # (settings are fp32)
        k = cols[1][r]
        want = outcomes(zs[r], float(u[r]), t, int(k), p, f)
        mine = int(token[r])
        assert mine in [w[0] for w in want], (r, mine, want[0])
        odd += mine != want[0][0]
        near = [w[1] for w in want if w[0] == mine]
        # fp32's rounding, and weights and their sum
        assert min(abs(float(prob[r]) - w) for w in near) <= 2.0 ** -23 * max(near) + 2.0 ** -40, r
    assert odd <= max(1, n // 100)
    # the same again, whatever the rest of the batch
    again = bec.sample(z, u, temperature, top_k, top_p, min_p)
    assert torch.equal(token, again[0]) and torch.equal(prob, again[1])
    if n > 1:
        one = bec.sample(z[n - 1:], u[n - 1:], *[c[n - 1:] if isinstance(c, torch.Tensor) else c for c in (temperature, top_k, top_p, min_p)])
        assert torch.equal(token[n - 1:], one[0]) and torch.equal(prob[n - 1:], one[1])
    return token, prob


def logits(n, V, dtype, seed, slack=0, scale=2.0):
    g = gen(seed)
    z = torch.randn((n, V + slack), device="cuda", generator=g) * scale
    at = torch.randint(0, V, (n, 9), device="cuda", generator=g)
    z.scatter_add_(1, at, torch.rand((n, 9), device="cuda", generator=g) * 8)
    return z.to(dtype)[:, :V], torch.rand((n,), device="cuda", generator=g)


SETTINGS = [
    # temperature, top_k, top_p, min_p
    (1.0, 0, 1.0, 0.0), (0.7, 50, 1.0, 0.0), (1.3, 0, 0.9, 0.0), (1.0, 0, 1.0, 0.05), (0.8, 40, 0.95, 0.02), (2.0, 1000, 0.5, 0.0),
    (0.05, 3, 0.99, 0.0), (1.0, 0, 0.999999, 0.0), (30.0, 0, 0.7, 0.0), (1.0, 2, 1e-9, 0.0), (1.0, 10 ** 6, 0.3, 0.0),
]


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("n,V,slack", [(1, 1, 0), (3, 2, 1), (5, 37, 0), (4, 511, 3), (7, 4097, 1), (40, 1000, 5), (2, 32771, 8),
                                       (160, 4500, 0), (1, 131072, 0), (3, 50001, 2), (1, 450001, 1), (1, 2 ** 20, 0)])
def test_sample_matches_64_bit(bec, dtype, n, V, slack):
    for i, s in enumerate(SETTINGS if V < 400000 else SETTINGS[2:5]):
        z, u = logits(n, V, dtype, 100 * i + n, slack)
        check(bec, z, u, *s)


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_sample_settings_of_each_row(bec, dtype):
    z, u = logits(66, 9001, dtype, 5)
    col = lambda v, t: torch.tensor([v[i % len(v)] for i in range(66)], dtype=t, device="cuda")  # noqa: E731
    check(bec, z, u, col([1.0, 0.0, 0.5, -1.0, float("nan"), 1.5, 0.9], F32), col([0, 5, 1, -3, 9000, 9001, 2 ** 31 - 1], torch.int32),
          col([1.0, 0.9, 0.0, 2.0, -1.0, 0.5], F32), col([0.0, 0.1, -1.0, 1.0, 7.0], F32))


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("V", [9, 5000, 40000, 131072])
@pytest.mark.parametrize("kind", ["equal", "two values", "coarse", "signed zeros"])
def test_sample_ties(bec, dtype, V, kind):
    """Equal logits: a cut inside them goes by the index, and shares are exact."""
    z, u = logits(6, V, dtype, 3)
    if kind == "equal":
        z = torch.full_like(z, -3.25)
    elif kind == "two values":
        z = (z > 1).to(dtype)
    elif kind == "coarse":
        z = (z.float() * 2).round().div(2).to(dtype)
    else:
        z = torch.where(z > 0, 0.0, -0.0).to(dtype)
    u[0], u[1] = 0.0, 1 - 2.0 ** -24
    for s in SETTINGS:
        check(bec, z, u, *s)
    if kind in ("equal", "signed zeros"):
        for k in (1, 2, V // 2 + 1, V):
            token, prob = bec.sample(z, u, 1.0, k)
            want = torch.floor(u.double() * k).to(torch.int32)
            assert torch.equal(token, want)
            assert torch.allclose(prob, torch.full_like(prob, 1.0 / k), rtol=2.0 ** -23, atol=0)


@pytest.mark.parametrize("V", [5000, 60000])
@pytest.mark.parametrize("steps", [3, 700, 200000])
def test_sample_thousands_of_near_ties(bec, V, steps):
    """Logits a few last bits apart: the end lies among thousands of tokens of one bin, and is looked for round by round."""
    rng = np.random.default_rng(V + steps)
    ulp = rng.integers(0, steps, (12, V))
    z = torch.from_numpy((np.float32(1.0) + ulp.astype(np.float32) * np.float32(2.0 ** -23)).astype(np.float32)).cuda()
    u = torch.from_numpy(rng.uniform(0, 1, 12).astype(np.float32)).cuda()
    p = torch.tensor([0.001, 0.01, 0.03, 0.3, 0.5, 0.9, 0.99, 0.9999, 1.0, 0.02, 0.6, 0.5], device="cuda")
    check(bec, z, u, top_p=p)
    k = torch.tensor([0, 1, 2, 900, 2047, 2048, 2049, 4000, V - 1, V, 3000, 1000], device="cuda", dtype=torch.int32)
    check(bec, z, u, top_k=k)
    check(bec, z, u, 0.5, top_k=k, top_p=p)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("V", [70, 20000])
def test_sample_infinities_and_nan(bec, dtype, V):
    inf, nan = float("inf"), float("nan")
    low = torch.finfo(dtype).min
    z, u = logits(12, V, dtype, 8)
    z[0] = -inf  # nothing left
    z[1] = nan
    z[2] = -inf
    z[2, 60] = -5.0  # one left
    z[3] = low
    z[4, 1:] = low
    z[5, 7] = inf
    z[6, 7:12] = inf
    z[7, ::2] = nan
    z[8, :60] = -inf
    z[9] = torch.finfo(dtype).max
    z[10, 5] = torch.finfo(dtype).max
    z[10, 6] = low
    for s in SETTINGS + [(1e-38, 0, 1.0, 0.0), (1e-42, 4, 0.9, 0.0), (1e38, 0, 0.9, 0.0), (inf, 0, 1.0, 0.0), (inf, 3, 0.5, 0.0)]:
        token, prob = check(bec, z, u, *s)
        assert token[:3].tolist() == [-1, -1, 60] and prob[:3].tolist() == [0.0, 0.0, 1.0]
        assert int(token[5]) == 7 and 7 <= int(token[6]) < 12 and (s[0] > 1e30 or int(token[10]) == 5)


def test_sample_given_numbers_at_their_ends(bec):
    z, _ = logits(4, 3000, F32, 2)
    u = torch.tensor([0.0, 2.0 ** -149, 1 - 2.0 ** -24, 0.5], device="cuda")
    check(bec, z, u)
    check(bec, z, u, 1.0, 7)
    # the distribution is the weights': every token's share of evenly spread numbers
    n = 20000
    zz = torch.tensor([[0.0, 1.0, 2.0, -float("inf"), 1.0]], device="cuda").expand(n, 5)
    token, _ = bec.sample(zz, (torch.arange(n, device="cuda") + 0.5) / n)
    share = torch.bincount(token.long(), minlength=5).double() / n
    want = torch.softmax(zz[0].double(), 0).cpu()
    assert ((share.cpu() - want).abs() <= 1.0 / n).all()


def test_sample_of_the_calls_tensors(bec):
    """Rows of a wider tensor at odd places, outputs given, no row."""
    z, u = logits(5, 1000, BF16, 6, slack=7)
    token, prob = torch.full((5,), 9, dtype=torch.int32, device="cuda"), torch.full((5,), 9.0, device="cuda")
    t, p = bec.sample(z, u, token=token, prob=prob)
    assert t is token and p is prob
    want = bec.sample(z.contiguous(), u)
    assert torch.equal(token, want[0]) and torch.equal(prob, want[1])
    frame = torch.cat([torch.zeros((5, 3), dtype=BF16, device="cuda"), z], 1)
    assert torch.equal(bec.sample(frame[:, 3:], u)[0], want[0])
    t, p = bec.sample(z[:0], u[:0])
    assert t.shape == (0,) and p.shape == (0,)
    with pytest.raises(bec.MoeError, match="V outside"):
        bec.sample(torch.zeros((1, 2 ** 20 + 1), device="cuda"), u[:1])


def test_sample_in_a_graph_and_on_streams(bec):
    z, u = logits(8, 30000, F32, 4)
    k = torch.full((8,), 20, dtype=torch.int32, device="cuda")
    token, prob = torch.empty((8,), dtype=torch.int32, device="cuda"), torch.empty((8,), device="cuda")
    bec.sample(z, u, 0.9, k, 0.95, token=token, prob=prob)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        bec.sample(z, u, 0.9, k, 0.95, token=token, prob=prob)
    for seed in (5, 6):
        z2, u2 = logits(8, 30000, F32, seed)
        z.copy_(z2)
        u.copy_(u2)
        k.fill_(seed)
        graph.replay()
        torch.cuda.synchronize()
        want = bec.sample(z2, u2, 0.9, k, 0.95)
        assert torch.equal(token, want[0]) and torch.equal(prob, want[1])
    # two calls at once share nothing
    other = torch.cuda.Stream()
    torch.cuda.synchronize()
    results = [bec.sample(z, u, 0.9, k, 0.95, stream=s) for _ in range(4) for s in (side, other)]
    torch.cuda.synchronize()
    assert all(torch.equal(r[0], want[0]) and torch.equal(r[1], want[1]) for r in results)
