"""Host-side tests of include/moekv.h (no GPU): structure layout, argument
checks that need no device."""
import ctypes as C
import os
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def native():
    import __graft_entry__
    __graft_entry__.build()
    from bounded_expert_cache_gb300 import _native
    return _native


def test_kv_structure_matches_header(native, tmp_path):
    lines = ["#include <stdio.h>", "#include <stddef.h>", '#include "moekv.h"', "int main(void) {",
             '  printf("size %zu\\n", sizeof(moe_kv_t));']
    lines += ['  printf("%s %%zu\\n", offsetof(moe_kv_t, %s));' % (f, f) for f, _ in native.KvT._fields_]
    src = tmp_path / "layout.c"
    src.write_text("\n".join(lines + ["  return 0;", "}"]) + "\n")
    exe = tmp_path / "layout"
    r = subprocess.run(["gcc", "-std=c11", "-I", os.path.join(ROOT, "include"), str(src), "-o", str(exe)],
                       capture_output=True, text=True)
    assert r.returncode == 0, r.stderr
    got = dict(line.split() for line in subprocess.run([str(exe)], capture_output=True, text=True,
                                                       check=True).stdout.splitlines())
    assert int(got["size"]) == C.sizeof(native.KvT)
    for f, _ in native.KvT._fields_:
        assert int(got[f]) == getattr(native.KvT, f).offset, f


def geometry(native, **kw):
    base = dict(n_layers=2, n_pages=10, n_kv_heads=2, page_tokens=16, head_dim=64, dtype=native.BF16, max_seqs=4,
                max_pages=8)
    base.update(kw)
    return native.KvT(**base)


@pytest.mark.parametrize("change", [dict(n_layers=0), dict(n_pages=0), dict(n_kv_heads=0), dict(page_tokens=8),
                                    dict(page_tokens=24), dict(page_tokens=512), dict(head_dim=0), dict(head_dim=12),
                                    dict(head_dim=264), dict(dtype=2), dict(max_seqs=0), dict(max_seqs=65537),
                                    dict(max_pages=0), dict(max_pages=2 ** 28)])
def test_bad_geometry_is_refused(native, change):
    kv = geometry(native, **change)
    n = C.c_int64()
    assert native.lib.moe_kv_work_bytes(C.byref(kv), C.byref(n)) == 1
    assert b"moe_kv_work_bytes" in native.lib.moe_last_error(None)
    # and by the calls themselves, before any pointer is used
    assert native.lib.moe_kv_compact(C.byref(kv), None) == 1
    assert native.lib.moe_attn_decode(C.byref(kv), 0, None, 0, None, 1, 1, 4, 1.0, 0, 0, None, 0, None) == 1


def test_null_arguments_are_refused(native):
    n = C.c_int64()
    assert native.lib.moe_kv_work_bytes(None, C.byref(n)) == 1
    kv = geometry(native)
    assert native.lib.moe_kv_work_bytes(C.byref(kv), None) == 1
    for call in (lambda: native.lib.moe_kv_fork(C.byref(kv), None, None, 1, None),
                 lambda: native.lib.moe_kv_reserve(C.byref(kv), None, None, 1, None),
                 lambda: native.lib.moe_kv_free(C.byref(kv), None, 1, None),
                 lambda: native.lib.moe_kv_check_errors(C.byref(kv), None)):
        assert call() == 1
        assert b"NULL" in native.lib.moe_last_error(None)


@pytest.mark.parametrize("args,why", [
    ((0, 16, 64, 1, 64, 1, 0, 16), b"quant"),      # Q8_0 is not a 4-bit format
    ((1, 0, 64, 1, 64, 1, 0, 16), b"N < 1"),
    ((1, 16, 40, 1, 40, 1, 0, 16), b"group"),
    ((2, 16, 96, 1, 96, 1, 0, 16), b"group"),
    ((1, 16, 64, 3, 64, 1, 0, 16), b"neither"),
    ((1, 16, 64, 1, 64, -1, 0, 16), b"T < 0"),
    ((1, 16, 64, 1, 64, 1, 0, 16), b"NULL"),
])
def test_quant_linear_arguments(native, args, why):
    quant, N, K, xt, ldx, T, yt, ldy = args
    st = native.lib.moe_quant_linear(None, quant, N, K, None, xt, ldx, T, None, None, yt, ldy, None)
    assert st == 1 and why in native.lib.moe_last_error(None)


def test_quant_linear_no_tokens_is_no_work(native):
    assert native.lib.moe_quant_linear(None, 1, 16, 64, None, 1, 64, 0, None, None, 0, 16, None) == 0


@pytest.mark.parametrize("N,K,refused", [(16, 2 ** 25, True), (128, 2 ** 26, True), (1, 2 ** 31 - 64, True),
                                         (2 ** 31 - 512, 64, True), (2 ** 31 - 1, 64, True), (16, 2 ** 25 - 64, False),
                                         (2 ** 31 - 513, 64, False)])
def test_quant_linear_sizes_that_offsets_hold(native, N, K, refused):
    """Sizes that pass stop at the NULL pointers instead."""
    st = native.lib.moe_quant_linear(None, 2, N, K, None, 1, K, 1, None, None, 0, N, None)
    why = native.lib.moe_last_error(None)
    assert st == 1 and (b"above" if refused else b"NULL") in why
