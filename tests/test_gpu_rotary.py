"""GPU tests of rotary positions and of writes and reads of the paged cache,
against the formulas in 64 bits."""
import math

import pytest
import torch

from test_gpu_kv import BF16, F32, U8, U24, gen, i32, randn, worst

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def bec():
    import bounded_expert_cache_gb300 as m
    return m


def turned(x, pos, rot):
    """x [rows, heads, D] turned in 64 bits, and the tolerance of an fp32 rotation (without the result's rounding)."""
    x = x.double()
    y, tol = x.clone(), torch.zeros_like(x)
    h = rot.dim // 2
    a = slice(0, rot.dim, 2) if rot.interleaved else slice(0, h)
    b = slice(1, rot.dim, 2) if rot.interleaved else slice(h, rot.dim)
    angle = pos.double()[:, None] * torch.tensor(rot.angles, dtype=torch.float64, device="cuda")
    c, s = torch.cos(angle)[:, None] * rot.magnitude, torch.sin(angle)[:, None] * rot.magnitude
    y[..., a], y[..., b] = x[..., a] * c - x[..., b] * s, x[..., b] * c + x[..., a] * s
    # the angle: its turns in 64 bits (a quotient and a product of doubles), what is
    # left of them rounded to fp32 (pi u); sine and cosine within two units; the
    # magnitude, two products and a sum
    off = angle.abs()[:, None] * 2.0 ** -50 + (math.pi + 2 + 1 + 3) * U24
    m = abs(rot.magnitude) * (x[..., a].abs() + x[..., b].abs()) * off
    tol[..., a], tol[..., b] = m, m
    return y, tol


def rounding(y, dtype):
    return (U8 * 1.01 * y.abs() if dtype == BF16 else 0) + 1e-37


ROTARY = [
    # rows, heads, D, dim, interleaved
    (1, 16, 128, 128, False), (1, 1, 8, 2, True), (3, 5, 64, 64, True), (7, 3, 80, 80, False), (5, 2, 96, 32, False),
    (9, 4, 128, 64, True), (2, 40, 128, 100, False), (6, 1, 256, 256, False), (4, 7, 72, 36, False), (33, 2, 16, 6, True),
    (1300, 3, 64, 64, False), (1300, 2, 128, 96, True), (700, 40, 40, 26, False), (2500, 1, 24, 18, True),
]


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("case", range(len(ROTARY)))
def test_rotary_matches_64_bit(bec, dtype, case):
    rows, heads, D, dim, interleaved = ROTARY[case]
    g = gen(case)
    rot = bec.Rotary(dim, base=[1e4, 5e5][case % 2], interleaved=interleaved, factor=[1.0, 8.0][case // 2 % 2],
                     context=[0, 8192][case // 4 % 2], magnitude=[1.0, 1.2, -0.5][case % 3])
    slack = [0, 8, 40][case % 3]
    x = randn((rows, heads * D + slack), dtype, g)[:, :heads * D].unflatten(1, (heads, D))
    top = [100, 70000, 2 ** 31 - 1][case % 3]
    pos = torch.randint(-top, top, (rows,), device="cuda", generator=g).to(torch.int32)
    pos[0] = [0, 2 ** 31 - 1, -2 ** 31][case % 3]
    frame = torch.full((rows, heads * D + slack), 7.0, dtype=dtype, device="cuda")
    out = frame[:, :heads * D].unflatten(1, (heads, D))
    before = x.clone()
    assert bec.rotary(x, pos, rot, out=out) is out
    y, tol = turned(x, pos, rot)
    assert worst(out, y, tol + rounding(y, dtype)) <= 1.0
    assert torch.equal(out[..., dim:], x[..., dim:]) and torch.equal(x, before)
    assert (frame[:, heads * D:] == 7.0).all()
    # into a new tensor and in place, bit for bit the same
    assert torch.equal(bec.rotary(x, pos, rot), out)
    bec.rotary(x, pos, rot, out=x)
    assert torch.equal(x, out)


def test_rotary_keeps_far_positions_apart(bec):
    """One radian a position: at 10^6 an fp32 angle would be off by a sixteenth."""
    rot = bec.Rotary(2, base=2.0)
    pos = i32([10 ** 6, 10 ** 6 + 1, 2 ** 31 - 1, -10 ** 6])
    x = torch.zeros((4, 1, 8), device="cuda")
    x[:, 0, 0] = 1.0
    y = bec.rotary(x, pos, rot)
    for i, p in enumerate(pos.tolist()):
        assert abs(y[i, 0, 0].item() - math.cos(p)) < 1e-6 + abs(p) * 2.0 ** -50
        assert abs(y[i, 0, 1].item() - math.sin(p)) < 1e-6 + abs(p) * 2.0 ** -50


def test_rotary_of_given_angles_and_of_no_rows(bec):
    rot = bec.Rotary(6, angles=[0.0, -2.5, 400.0], interleaved=True)
    x = randn((5, 2, 8), F32, gen(1))
    pos = i32(range(5))
    y, tol = turned(x, pos, rot)
    assert worst(bec.rotary(x, pos, rot), y, tol + 1e-37) <= 1.0
    assert bec.rotary(x[:0], pos[:0], rot).shape == (0, 2, 8)


def test_rotary_infinities_stay_in_their_pairs(bec):
    rot = bec.Rotary(8)
    x = torch.ones((1, 2, 16), device="cuda")
    x[0, 0, 2] = float("inf")
    x[0, 1, 9] = float("nan")
    y = bec.rotary(x, i32([3]), rot)
    odd = ~torch.isfinite(y)
    assert odd.nonzero().tolist() == [[0, 0, 2], [0, 0, 6], [0, 1, 9]]


# ---------------------------------------------------------------- pages
def codes_of(x):
    """Expected codes [..., D/2] (bytes) and metadata [..., D/64] (words) of fp32 values [..., D]."""
    g = x.unflatten(-1, (-1, 64))
    fine = (g.abs() <= 2.0 ** 126).all(-1, keepdim=True)
    safe = torch.where(fine, g, torch.zeros_like(g))
    b = safe.amin(-1, keepdim=True).bfloat16()
    s = ((safe.amax(-1, keepdim=True) - b.float()) / 15.0).bfloat16()
    s = torch.where(s > 0, s, torch.zeros_like(s))
    q = torch.round((safe - b.float()) / torch.where(s > 0, s, torch.ones_like(s)).float()).clamp(0, 15)
    q = torch.where(fine & (s > 0), q, torch.zeros_like(q)).to(torch.uint8).flatten(-2)
    nan = torch.full_like(s, float("nan"))
    meta = torch.cat([torch.where(fine, s, nan), torch.where(fine, b, nan)], -1)
    return q[..., 0::2] | (q[..., 1::2] << 4), meta


def split(pool, D):
    """Codes [..., tokens, D/2] and metadata [..., tokens, D/64, 2] of a pool of pages of codes."""
    page = pool.shape[-2]
    flat = pool.flatten(-2)
    return (flat[..., :page * D // 2].unflatten(-1, (page, D // 2)),
            flat[..., page * D // 2:].view(BF16).unflatten(-1, (page, D // 64, 2)))


def values_of(codes, meta):
    q = torch.stack([codes & 15, codes >> 4], -1).flatten(-2).double().unflatten(-1, (-1, 64))
    return (q * meta[..., :1].double() + meta[..., 1:].double()).flatten(-2)


class Cache:
    """A cache whose pages hold rubbish (NaN where they can) until they are written."""

    def __init__(self, bec, dtype, bits, D, page, hkv, seqs=4, pages=40, width=16, layers=2):
        self.kv = bec.KvCache.empty(layers, pages, hkv, page, D, seqs, width, dtype=dtype, bits=bits)
        for t in (self.kv.k, self.kv.v):
            t.view(torch.uint8).fill_(255)
        self.D, self.page, self.bits = D, page, bits

    def at(self, s, j):
        return int(self.kv.table[s, j // self.page]), j % self.page


WRITE = [
    # bits, D, dim, interleaved, page, hkv, group
    (0, 64, 64, False, 16, 2, 4), (0, 80, 26, False, 32, 1, 3), (0, 128, 64, True, 64, 4, 1), (0, 24, 24, False, 16, 3, 2),
    (4, 64, 64, False, 16, 2, 4), (4, 128, 128, False, 64, 2, 8), (4, 192, 50, True, 16, 1, 2), (4, 256, 106, False, 32, 3, 1),
    (4, 128, 2, False, 128, 1, 1),
]


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("case", range(len(WRITE)))
def test_write_rotary_and_read(bec, dtype, case):
    bits, D, dim, interleaved, page, hkv, group = WRITE[case]
    hq = hkv * group
    c = Cache(bec, dtype, bits, D, page, hkv)
    kv, g = c.kv, gen(50 + case)
    rot = bec.Rotary(dim, interleaved=interleaved, magnitude=1.1)
    ids, held = [3, 0, 2], [0, 0, 0]
    for counts, pad in (([37, 1, 0], 0), ([1, 5, 18], 3), ([1, 1, 1], 0)):
        rows = sum(counts) + pad  # rows behind the last sequence belong to none
        kv.reserve(i32(ids), i32(counts))
        cu = i32([0] + [sum(counts[:i + 1]) for i in range(3)])
        x = randn((rows, (hq + 2 * hkv) * D + 8), dtype, g)
        q, k, v = (x[:, a * D:b * D].unflatten(1, (-1, D)) for a, b in ((0, hq), (hq, hq + hkv), (hq + hkv, hq + 2 * hkv)))
        out = torch.full((rows, hq, D), 7.0, dtype=dtype, device="cuda")
        kv.write_rotary(1, q, k, v, i32(ids), cu, rot, q_out=out)
        kv.check_errors()
        n = sum(counts)
        pos = i32([held[i] + j for i in range(3) for j in range(counts[i])])
        y, tol = turned(q[:n], pos, rot)
        assert worst(out[:n], y, tol + rounding(y, dtype)) <= 1.0
        assert (out[n:] == 7.0).all()
        # the pages: k within a rotation's error (codes: a step more where that crosses a border), v exactly
        where = [c.at(ids[i], held[i] + j) for i in range(3) for j in range(counts[i])]
        p, t = i32([w[0] for w in where]).long(), i32([w[1] for w in where]).long()
        ky, ktol = turned(k[:n], pos, rot)
        back = [torch.full((rows, hkv, D), 7.0, dtype=dtype, device="cuda") for _ in range(2)]
        kv.read(1, i32(ids), cu, rows, *back)
        kv.check_errors()
        assert all((b[n:] == 7.0).all() for b in back)
        if bits == 0:
            assert worst(kv.k[1, p, :, t], ky, ktol + rounding(ky, dtype)) <= 1.0
            assert torch.equal(kv.v[1, p, :, t], v[:n])
            assert torch.equal(back[0][:n], kv.k[1, p, :, t]) and torch.equal(back[1][:n], v[:n])
        else:
            (kc, km), (vc, vm) = split(kv.k[1], D), split(kv.v[1], D)
            codes, meta = codes_of(v[:n].float())
            assert torch.equal(vc[p, :, t], codes) and torch.equal(vm[p, :, t], meta)
            # of the rotated keys: offsets and scales within a bf16 step of the formula's, values within half a step and what these are off
            got, lo = values_of(kc[p, :, t], km[p, :, t]), ky.unflatten(-1, (-1, 64))
            span = (lo.amax(-1, keepdim=True) - lo.amin(-1, keepdim=True))
            edge = lo.abs().amax(-1, keepdim=True)
            bound = (span / 15 * (0.5 + 8 * U8) + U8 * edge * 2).expand_as(lo).flatten(-2) + 4 * ktol
            assert ((got - ky).abs() <= bound).all()
            for b, (cc, mm) in zip(back, ((kc, km), (vc, vm))):
                val = values_of(cc[p, :, t], mm[p, :, t])
                assert worst(b[:n], val, 2 * U24 * val.abs() + 2 * U24 * edge.amax() + rounding(val, dtype)) <= 1.0
        held = [h + m for h, m in zip(held, counts)]
    # q in place
    q2 = q.clone()
    kv.write_rotary(1, q2, k, v, i32(ids), cu, rot, q_out=q2)
    assert torch.equal(q2[:n], out[:n])
    kv.check_errors()


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_codes_of_every_kind_of_group(bec, dtype):
    """Constant, tiny, large, one-sided, ties between codes, infinities and NaN."""
    inf, nan = float("inf"), float("nan")
    D, kinds = 128, []
    g = gen(9)
    base = torch.randn((64,), device="cuda", generator=g)
    kinds += [base * 0 + 0.7, base * 0, base * 1e-30, base * 1e30, base.abs() + 100, -base.abs(), base * 1e-40, base * 8e37 / base.abs().max()]
    kinds += [torch.arange(64, device="cuda") / 4.0, torch.arange(64, device="cuda") % 2 * 15.0 - 3]
    for odd in (inf, -inf, nan, 3e38, -3e38):
        t = base.clone()
        t[17] = odd
        kinds.append(t)
    x = torch.stack(kinds).to(dtype)
    n = x.shape[0]
    k = torch.cat([x, x.flip(0)], 1)[:, None]  # two groups a head, kinds beside others
    c = Cache(bec, dtype, 4, D, 16, 1, seqs=1)
    c.kv.reserve(i32([0]), i32([n]))
    c.kv.write(0, k, k, i32([0]), i32([0, n]))
    c.kv.check_errors()
    p = c.kv.table[0, torch.arange(n, device="cuda") // 16].long()
    t = torch.arange(n, device="cuda") % 16
    codes, meta = codes_of(k.float())
    for pool in (c.kv.k, c.kv.v):
        got_c, got_m = split(pool[0], D)
        assert torch.equal(got_c[p, :, t], codes)
        assert torch.equal(got_m[p, :, t].view(torch.int16), meta.view(torch.int16)) or torch.equal(
            torch.nan_to_num(got_m[p, :, t].float(), nan=5e9), torch.nan_to_num(meta.float(), nan=5e9))
    back, _ = c.kv.read(0, i32([0]), i32([0, n]), n)
    want = values_of(codes, meta)
    assert torch.equal(torch.isnan(back), torch.isnan(want))
    ok = ~torch.isnan(want)
    assert worst(back[ok], want[ok], 3 * U24 * want[ok].abs() + 3 * U24 * k.double().nan_to_num(0, 0, 0).abs().amax(-1, keepdim=True).expand_as(want)[ok]
                 + rounding(want[ok], dtype)) <= 1.0


def test_write_rotary_leaves_out_what_is_wrong(bec):
    """As write: a shared page, a chunk longer than its sequence, an id out of range; their rows of q_out stay."""
    c = Cache(bec, BF16, 4, 64, 16, 1, seqs=6)
    kv, g = c.kv, gen(3)
    rot = bec.Rotary(64)
    x = randn((4, 1, 64), BF16, g)
    kv.reserve(i32([0, 1, 2]), i32([20, 20, 1]))
    kv.fork(i32([1]), i32([3]))
    before = kv.k.clone(), kv.v.clone()
    out = torch.full_like(x, 7.0)
    # sequence 1 shares its pages, 2 has one token for two rows, 99 does not exist, 0 is fine
    for ids, cu, good in (([1, 2, 99, 0], [0, 1, 3, 3, 4], [3]), ([99, 0], [0, 1, 2], [1]), ([0, 1], [0, 1, 9], [0])):
        out.fill_(7.0)
        kv.k.copy_(before[0])
        kv.v.copy_(before[1])
        kv.write_rotary(1, x, x, x, i32(ids), i32(cu), rot, q_out=out)
        with pytest.raises(bec.MoeError):
            kv.check_errors()
        changed = (kv.k != before[0]).any(-1).any(-1).flatten()
        written = changed.nonzero().numel()
        assert written == len(good)
        stayed = [i for i in range(4) if i not in good]
        assert (out[stayed] == 7.0).all() and not (out[good] == 7.0).all()
    # a pending failure stops the next write
    kv.write_rotary(1, x, x, x, i32([99, 99, 99, 99]), i32([0, 1, 2, 3, 4]), rot)
    out.fill_(7.0)
    kv.k.copy_(before[0])
    kv.write_rotary(1, x[:1], x[:1], x[:1], i32([0]), i32([0, 1]), rot, q_out=out[:1])
    assert (out == 7.0).all() and torch.equal(kv.k, before[0])
    with pytest.raises(bec.MoeError):
        kv.check_errors()


def test_read_of_what_is_not_held_is_an_error(bec):
    c = Cache(bec, F32, 0, 16, 16, 1)
    c.kv.reserve(i32([0]), i32([3]))
    k = torch.full((5, 1, 16), 7.0, device="cuda")
    for ids, cu in (([0], [0, 5]), ([9], [0, 1]), ([0], [0, 9])):
        c.kv.read(0, i32(ids), i32(cu), 5, k, k.clone())
        with pytest.raises(bec.MoeError):
            c.kv.check_errors()
        assert (k == 7.0).all()
    # shared pages are read
    c.kv.write(0, k[:3], k[:3], i32([0]), i32([0, 3]))
    c.kv.fork(i32([0]), i32([1]))
    back, _ = c.kv.read(0, i32([1, 0]), i32([0, 2, 3]), 3)
    c.kv.check_errors()
    assert (back == 7.0).all()


@pytest.mark.parametrize("bits", [0, 4])
def test_many_short_chunks(bec, bits):
    """More chunks than a block finds at once, most of them of one row or none."""
    n, D = 3000, 64
    counts = [(i * 7) % 3 for i in range(n)]
    rows = sum(counts)
    c = Cache(bec, BF16, bits, D, 16, 1, seqs=n, pages=n, width=2)
    g = gen(8)
    rot = bec.Rotary(D)
    kv = c.kv
    ids = torch.randperm(n, generator=torch.Generator().manual_seed(1)).tolist()
    kv.reserve(i32(ids), i32(counts))
    cu = torch.zeros(n + 1, dtype=torch.int32, device="cuda")
    cu[1:] = torch.cumsum(i32(counts), 0)
    x = randn((rows, 3, D), BF16, g)
    out = kv.write_rotary(0, x[:, :1], x[:, 1:2], x[:, 2:], i32(ids), cu, rot)
    kv.check_errors()
    pos = i32([j for m in counts for j in range(m)])
    y, tol = turned(x[:, :1], pos, rot)
    assert worst(out, y, tol + rounding(y, BF16)) <= 1.0
    _, v = kv.read(0, i32(ids), cu, rows)
    if bits == 0:
        assert torch.equal(v, x[:, 2:])
    else:
        val = values_of(*codes_of(x[:, 2:].float()))
        assert worst(v, val, 4 * U24 * x.double().abs().amax() + rounding(val, BF16)) <= 1.0


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_copy_on_write_and_moves_of_pages_of_codes(bec, dtype):
    """Branches of a prompt whose last page is partly filled, compacted, keep their values."""
    D, page = 128, 32
    c = Cache(bec, dtype, 4, D, page, 2, seqs=5, pages=60)
    kv, g = c.kv, gen(4)
    x = randn((77, 2, D), dtype, g)
    kv.reserve(i32([4]), i32([30]))
    for layer in range(2):
        kv.write(layer, x[:30], x[:30], i32([4]), i32([0, 30]))
    kv.reserve(i32([0]), i32([77]))
    for layer in range(2):
        kv.write(layer, x, x * 2, i32([0]), i32([0, 77]))
    kv.fork(i32([0, 0]), i32([1, 2]))
    kv.reserve(i32([1, 0]), i32([1, 2]))
    y = randn((3, 2, D), dtype, g)
    for layer in range(2):
        kv.write(layer, y, y, i32([1, 0]), i32([0, 1, 3]))
    kv.free(i32([4]))
    kv.compact()
    kv.check_errors()
    assert torch.nonzero(kv.ref).max() < int((kv.ref > 0).sum())
    want = values_of(*codes_of(x.float())), values_of(*codes_of((x * 2).float())), values_of(*codes_of(y.float()))
    for s, n, tail in ((1, 78, want[2][:1]), (0, 79, want[2][1:]), (2, 77, None)):
        for layer in range(2):
            k, v = kv.read(layer, i32([s]), i32([0, n]), n)
            for got, w in ((k, want[0]), (v, want[1])):
                w = w if tail is None else torch.cat([w, tail])
                assert worst(got, w, 4 * U24 * w.abs().amax() + rounding(w, dtype)) <= 1.0, (s, layer)
    kv.check_errors()


def test_rotary_refusals_on_a_cache(bec):
    kv = bec.KvCache.empty(1, 4, 1, 16, 64, 2, 2, dtype=BF16, bits=4)
    q, k = torch.zeros((2, 4, 64), dtype=BF16, device="cuda"), torch.zeros((2, 1, 64), dtype=BF16, device="cuda")
    seqs, cu = i32([0]), i32([0, 2])
    with pytest.raises(bec.MoeError, match="dim"):
        kv.write_rotary(0, q, k, k, seqs, cu, bec.Rotary(66))
    with pytest.raises(bec.MoeError, match="layer"):
        kv.write_rotary(1, q, k, k, seqs, cu, bec.Rotary(64))
    with pytest.raises(bec.MoeError, match="layer"):
        kv.read(-1, seqs, cu, 2)
    odd = torch.zeros((2, 4 * 64 + 4), dtype=BF16, device="cuda")[:, 4:].unflatten(1, (4, 64))
    with pytest.raises(bec.MoeError, match="16-byte"):
        kv.write_rotary(0, odd, k, k, seqs, cu, bec.Rotary(64))
    with pytest.raises(bec.MoeError, match="16-byte"):
        bec.rotary(odd, i32([0, 1]), bec.Rotary(64))
    kv.check_errors()
