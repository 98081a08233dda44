"""Host-side tests of rotary positions, 4-bit caches and sampling in
include/moekv.h and its binding (no GPU): structure layouts, host arithmetic,
refusals that need no device, devices of calls."""
import ctypes as C
import math
import os
import subprocess
from fractions import Fraction

import pytest
import torch

from test_kv_binding import Fake, kvmod, world  # noqa: F401  (fixtures)
from test_kv_host import geometry, native  # noqa: F401

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
BF16, F32, I32, U8 = torch.bfloat16, torch.float32, torch.int32, torch.uint8


@pytest.mark.parametrize("name,struct", [("moe_rotary_t", "RotaryT"), ("moe_sampling_t", "SamplingT")])
def test_structures_match_header(native, tmp_path, name, struct):  # noqa: F811
    cls = getattr(native, struct)
    lines = ["#include <stdio.h>", "#include <stddef.h>", '#include "moekv.h"', "int main(void) {",
             '  printf("size %%zu\\n", sizeof(%s));' % name, '  printf("flag %d\\n", (int)MOE_KV_I4);']
    lines += ['  printf("%s %%zu\\n", offsetof(%s, %s));' % (f, name, f) for f, _ in cls._fields_]
    src, exe = tmp_path / "layout.c", tmp_path / "layout"
    src.write_text("\n".join(lines + ["  return 0;", "}"]) + "\n")
    r = subprocess.run(["gcc", "-std=c11", "-I", os.path.join(ROOT, "include"), str(src), "-o", str(exe)],
                       capture_output=True, text=True)
    assert r.returncode == 0, r.stderr
    got = dict(line.split() for line in subprocess.run([str(exe)], capture_output=True, text=True, check=True).stdout.splitlines())
    assert int(got["size"]) == C.sizeof(cls) and int(got["flag"]) == native.KV_I4
    for f, _ in cls._fields_:
        assert int(got[f]) == getattr(cls, f).offset, f


# ---------------------------------------------------------------- rotary: host arithmetic
def angles_of(native, *args):  # noqa: F811
    out = (C.c_double * (args[0] // 2))()
    assert native.lib.moe_rotary_angles(*args, out) == 0
    return list(out)


def test_angles_are_the_formula(native):  # noqa: F811
    assert angles_of(native, 8, 10000.0, 1.0, 0, 0.0, 0.0) == [10000.0 ** (-2.0 * i / 8) for i in range(4)]
    assert angles_of(native, 6, 500.0, 4.0, 0, 0.0, 0.0) == pytest.approx([500.0 ** (-i / 3) / 4 for i in range(3)], rel=1e-15)
    # by parts: turns within 4,096 tokens decide
    plain = angles_of(native, 64, 1e4, 1.0, 0, 0.0, 0.0)
    mixed = angles_of(native, 64, 1e4, 8.0, 4096, 1.0, 32.0)
    kinds = set()
    for f, g in zip(plain, mixed):
        turns = f * 4096 / (2 * math.pi)
        if turns >= 32:
            assert g == f
            kinds.add("kept")
        elif turns <= 1:
            assert g == pytest.approx(f / 8, rel=1e-15)
            kinds.add("stretched")
        else:
            keep = (turns - 1) / 31
            assert g == pytest.approx(f * (keep + (1 - keep) / 8), rel=1e-14)
            kinds.add("between")
    assert kinds == {"kept", "stretched", "between"}


def test_turns_are_fractions_of_64_bits(native):  # noqa: F811
    angles = [0.0, 1.0, 2 * math.pi * 0.25, -1.0, 7.5, 1e-9, 123456.75]
    out = (C.c_uint64 * len(angles))()
    assert native.lib.moe_rotary_turns((C.c_double * len(angles))(*angles), len(angles), out) == 0
    two_pi = Fraction(2 * 884279719003555, 281474976710656)  # the double nearest 2 pi
    for a, t in zip(angles, out):
        turn = Fraction(a) / two_pi
        off = abs(Fraction(t, 2 ** 64) - (turn - math.floor(turn)))
        # the quotient's and the difference's rounding; whole turns are the same angle
        assert min(off, 1 - off) <= Fraction(2) ** -52 * max(1, abs(turn)), a


@pytest.mark.parametrize("args,why", [((7, 1e4, 1.0, 0, 0.0, 1.0), b"even"), ((0, 1e4, 1.0, 0, 0.0, 1.0), b"even"),
                                      ((8, 0.0, 1.0, 0, 0.0, 1.0), b"base"), ((8, math.inf, 1.0, 0, 0.0, 1.0), b"base"),
                                      ((8, 1e4, 0.0, 0, 0.0, 1.0), b"factor"), ((8, 1e4, math.nan, 0, 0.0, 1.0), b"factor"),
                                      ((8, 1e4, 2.0, -1, 0.0, 1.0), b"context"), ((8, 1e4, 2.0, 64, 2.0, 2.0), b"turns_high")])
def test_angles_refusals(native, args, why):  # noqa: F811
    out = (C.c_double * 8)()
    assert native.lib.moe_rotary_angles(*args, out) == 1 and why in native.lib.moe_last_error(None)
    assert native.lib.moe_rotary_angles(8, 1e4, 1.0, 0, 0.0, 1.0, None) == 1


def test_turns_refusals(native):  # noqa: F811
    one, out = (C.c_double * 2)(1.0, math.inf), (C.c_uint64 * 2)(5, 5)
    assert native.lib.moe_rotary_turns(one, 2, out) == 1 and b"finite" in native.lib.moe_last_error(None)
    assert list(out) == [5, 5]
    assert native.lib.moe_rotary_turns(one, -1, out) == 1
    assert native.lib.moe_rotary_turns(None, 1, out) == 1
    assert native.lib.moe_rotary_turns(None, 0, None) == 0


@pytest.mark.parametrize("change,why", [(dict(xt=2), b"neither"), (dict(D=12), b"head_dim"), (dict(D=264), b"head_dim"),
                                        (dict(rot=None), b"NULL"), (dict(turns=None), b"NULL"), (dict(turns=4100), b"8-byte"),
                                        (dict(dim=130), b"dim"), (dict(dim=7), b"dim"), (dict(dim=0), b"dim"),
                                        (dict(interleaved=2), b"interleaved"), (dict(magnitude=math.nan), b"magnitude"),
                                        (dict(rows=-1), b"n_rows"), (dict(rows=2 ** 30 + 1), b"n_rows"), (dict(heads=0), b"n_heads"),
                                        (dict(pos=None), b"NULL"), (dict(x=None), b"NULL"), (dict(x=4104), b"16-byte"),
                                        (dict(ldx=1028), b"16-byte"), (dict(ldy=1000), b"smaller")])
def test_rotary_refusals(native, change, why):  # noqa: F811
    c = dict(rot=True, turns=4096, dim=128, interleaved=0, magnitude=1.0, pos=4096, x=4096, xt=native.BF16, ldx=1024, rows=3,
             heads=8, D=128, y=8192, ldy=1024)
    c.update(change)
    rot = C.byref(native.RotaryT(c["turns"], c["dim"], c["interleaved"], c["magnitude"])) if c["rot"] else None
    st = native.lib.moe_rotary(rot, c["pos"], c["x"], c["xt"], c["ldx"], c["rows"], c["heads"], c["D"], c["y"], c["ldy"], None)
    assert st == 1 and why in native.lib.moe_last_error(None)


def test_rotary_of_no_rows_is_no_work(native):  # noqa: F811
    assert native.lib.moe_rotary(C.byref(native.RotaryT(4096, 8, 0, 1.0)), None, None, 0, 0, 0, 1, 8, None, 0, None) == 0


# ---------------------------------------------------------------- caches of 4-bit codes
@pytest.mark.parametrize("change", [dict(dtype=16, head_dim=80), dict(dtype=17, head_dim=8), dict(dtype=18), dict(dtype=32),
                                    dict(dtype=17, head_dim=320)])
def test_bad_geometry_of_codes_is_refused(native, change):  # noqa: F811
    kv, n = geometry(native, **change), C.c_int64()
    assert native.lib.moe_kv_work_bytes(C.byref(kv), C.byref(n)) == 1
    assert native.lib.moe_kv_read(C.byref(kv), 0, None, 0, None, 0, None, None, 1, 1, None) == 1
    assert native.lib.moe_kv_write_rotary(C.byref(kv), 0, None, None, 0, 1, None, 0, None, 0, None, 0, None, None, 1, 1, None) == 1


def codes_cache(kvmod, D=128, page=16, dtype=BF16, device=0):  # noqa: F811
    pool = (2, 10, 2, page, D * 9 // 16)
    kv = kvmod.KvCache.__new__(kvmod.KvCache)
    kv.k, kv.v = Fake(pool, U8, device), Fake(pool, U8, device)
    kv.raw, kv._ref = kvmod.N.KvT(), None
    kv._device, kv._kv_heads, kv._dim, kv._dtype = device, 2, D, dtype
    return kv


def rotation(kvmod, device=0, dim=64):  # noqa: F811
    rot = kvmod.Rotary.__new__(kvmod.Rotary)
    rot._device, rot._ref, rot.dim = device, "rot", dim
    return rot


def test_pages_of_codes_need_their_shape_and_type(kvmod):  # noqa: F811
    def make(last, dtype=BF16, k=U8):
        return kvmod.KvCache(Fake((2, 10, 2, 16, last), k), Fake((2, 10, 2, 16, last), k), Fake((4, 8), I32), Fake((4,), I32),
                             Fake((10,), I32), dtype)
    with pytest.raises(TypeError):
        make(72, None)
    with pytest.raises(TypeError):
        make(72, torch.float16)
    with pytest.raises(TypeError):
        make(64, F32, BF16)
    for last in (64, 45, 71):
        with pytest.raises(ValueError):
            make(last)
    with pytest.raises(ValueError):
        kvmod.KvCache.empty(1, 4, 1, 16, 96, 1, 4, bits=4)
    with pytest.raises(ValueError):
        kvmod.KvCache.empty(1, 4, 1, 16, 64, 1, 4, bits=8)


def test_token_bytes_of_codes(kvmod):  # noqa: F811
    assert codes_cache(kvmod).token_bytes == 2 * 2 * 2 * 128 * 9 // 16


@pytest.mark.parametrize("device", [0, 1])
def test_calls_run_on_their_tensors_device(kvmod, world, device):  # noqa: F811
    kv, rot = codes_cache(kvmod, device=device), rotation(kvmod, device)
    q, k = Fake((5, 8, 128), BF16, device), Fake((5, 2, 128), BF16, device)
    seqs, cu = Fake((2,), I32, device), Fake((3,), I32, device)
    assert kv.write_rotary(1, q, k, k, seqs, cu, rot, q_out=q) is q
    kv.read(1, seqs, cu, 5, k, k)
    kvmod.rotary(q, Fake((5,), I32, device), rot, out=q)
    z, u = Fake((5, 100), F32, device), Fake((5,), F32, device)
    kvmod.sample(z, u, top_p=u, token=Fake((5,), I32, device), prob=u)
    assert [(c[0], c[1]) for c in world["lib"].calls] == [
        ("moe_kv_write_rotary", device), ("moe_kv_read", device), ("moe_rotary", device), ("moe_sample", device)]


def test_tensors_of_another_device_are_refused(kvmod, world):  # noqa: F811
    kv, rot = codes_cache(kvmod), rotation(kvmod)
    q, k = Fake((5, 8, 128), BF16), Fake((5, 2, 128), BF16)
    seqs, cu, pos = Fake((2,), I32), Fake((3,), I32), Fake((5,), I32)
    z, u, token = Fake((5, 100), F32), Fake((5,), F32), Fake((5,), I32)
    other = {"q": Fake((5, 8, 128), BF16, 1), "k": Fake((5, 2, 128), BF16, 1), "rot": rotation(kvmod, 1), "pos": Fake((5,), I32, 1),
             "u": Fake((5,), F32, 1), "token": Fake((5,), I32, 1)}
    for call in (lambda: kv.write_rotary(0, other["q"], k, k, seqs, cu, rot, q_out=q),
                 lambda: kv.write_rotary(0, q, other["k"], k, seqs, cu, rot, q_out=q),
                 lambda: kv.write_rotary(0, q, k, k, seqs, cu, rot, q_out=other["q"]),
                 lambda: kv.write_rotary(0, q, k, k, seqs, cu, other["rot"], q_out=q),
                 lambda: kv.read(0, seqs, cu, 5, other["k"], k),
                 lambda: kvmod.rotary(q, other["pos"], rot, out=q),
                 lambda: kvmod.rotary(q, pos, other["rot"], out=q),
                 lambda: kvmod.rotary(q, pos, rot, out=other["q"]),
                 lambda: kvmod.sample(z, other["u"], token=token, prob=u),
                 lambda: kvmod.sample(z, u, min_p=other["u"], token=token, prob=u),
                 lambda: kvmod.sample(z, u, token=other["token"], prob=u)):
        with pytest.raises(ValueError, match="cuda:0"):
            call()
    assert not world["lib"].calls


def test_shapes_and_types_that_the_binding_refuses(kvmod, world):  # noqa: F811
    kv, rot = codes_cache(kvmod), rotation(kvmod)
    q, k = Fake((5, 8, 128), BF16), Fake((5, 2, 128), BF16)
    seqs, cu, pos = Fake((2,), I32), Fake((3,), I32), Fake((5,), I32)
    z, u, token = Fake((5, 100), F32), Fake((5,), F32), Fake((5,), I32)
    for call in (lambda: kv.write_rotary(0, q, Fake((4, 2, 128), BF16), k, seqs, cu, rot, q_out=q),
                 lambda: kv.write_rotary(0, Fake((6, 8, 128), BF16), k, k, seqs, cu, rot, q_out=Fake((6, 8, 128), BF16)),
                 lambda: kv.write_rotary(0, q, k, k, seqs, cu, rot, q_out=Fake((5, 4, 128), BF16)),
                 lambda: kv.write_rotary(0, q, k, k, seqs, cu, "rot", q_out=q),
                 lambda: kv.write(0, Fake((5, 2, 72), U8), k, seqs, cu),
                 lambda: kv.read(0, seqs, cu, 4, k, k),
                 lambda: kv.read(0, seqs, cu, 5, Fake((5, 2, 128), F32), k),
                 lambda: kvmod.rotary(Fake((5, 1024), BF16), pos, rot),
                 lambda: kvmod.rotary(Fake((5, 8, 128), torch.float16), pos, rot, out=q),
                 lambda: kvmod.rotary(q, Fake((4,), I32), rot, out=q),
                 lambda: kvmod.rotary(q, Fake((5,), torch.int64), rot, out=q),
                 lambda: kvmod.rotary(q, pos, None, out=q),
                 lambda: kvmod.sample(Fake((500,), F32), u),
                 lambda: kvmod.sample(Fake((5, 100), F32, stride=(200, 2)), u),
                 lambda: kvmod.sample(Fake((5, 100), torch.float16), u),
                 lambda: kvmod.sample(z, Fake((4,), F32), token=token, prob=u),
                 lambda: kvmod.sample(z, u, top_k=u, token=token, prob=u),
                 lambda: kvmod.sample(z, u, temperature=token, token=token, prob=u)):
        with pytest.raises((ValueError, TypeError)):
            call()
    assert not world["lib"].calls


@pytest.mark.parametrize("dim", [0, 1, 7])
def test_rotations_of_an_odd_size_are_refused(kvmod, dim):  # noqa: F811
    with pytest.raises(ValueError):
        kvmod.Rotary(dim)
    with pytest.raises(ValueError):
        kvmod.Rotary(8, angles=[1.0, 2.0])


# ---------------------------------------------------------------- sampling
@pytest.mark.parametrize("change,why", [(dict(zt=2), b"neither"), (dict(V=0), b"V outside"), (dict(V=2 ** 20 + 1, ld=2 ** 21), b"V outside"),
                                        (dict(rows=-1), b"rows"), (dict(rows=2 ** 24 + 1), b"rows"), (dict(by=None), b"NULL"),
                                        (dict(z=None), b"NULL"), (dict(u=None), b"NULL"), (dict(token=None), b"NULL"),
                                        (dict(ld=99), b"smaller"), (dict(z=4098), b"aligned"), (dict(u=4098), b"aligned"),
                                        (dict(prob=4097), b"aligned"), (dict(t=4097), b"aligned")])
def test_sample_refusals(native, change, why):  # noqa: F811
    c = dict(z=4096, zt=native.F32, ld=100, rows=3, V=100, u=4096, by=True, token=4096, prob=4096, t=None)
    c.update(change)
    by = C.byref(native.SamplingT(1.0, 1.0, 0.0, 0, c["t"], None, None, None)) if c["by"] else None
    assert native.lib.moe_sample(c["z"], c["zt"], c["ld"], c["rows"], c["V"], c["u"], by, c["token"], c["prob"], None) == 1
    assert why in native.lib.moe_last_error(None)


def test_sample_of_no_rows_is_no_work(native):  # noqa: F811
    assert native.lib.moe_sample(None, 0, 0, 0, 5, None, C.byref(native.SamplingT()), None, None, None) == 0


@pytest.mark.parametrize("magnitude,fine", [(1e39, False), (-math.inf, False), (3e38, True), (-0.5, True)])
def test_magnitude_must_be_finite_in_fp32(native, magnitude, fine):  # noqa: F811
    rot = native.RotaryT(4096, 8, 0, magnitude)
    st = native.lib.moe_rotary(C.byref(rot), None, None, 0, 0, 0, 1, 8, None, 0, None)
    assert (st == 0) == fine
    assert fine or b"magnitude" in native.lib.moe_last_error(None)
