"""Host-side tests of the KV cache's Python binding (no GPU): which device a
call is made on, and that its tensors are all there. Stand-ins take the place
of tensors on several devices, of the library and of the device guard."""
import contextlib
import math

import pytest
import torch


@pytest.fixture(scope="module")
def kvmod():
    import __graft_entry__
    __graft_entry__.build()
    from bounded_expert_cache_gb300 import kv
    return kv


class Fake:
    """What the binding asks of a tensor."""

    def __init__(self, shape, dtype, device=0, stride=None):
        self.shape, self.dtype, self.index = torch.Size(shape), dtype, device
        self.strides = stride or tuple(math.prod(shape[i + 1:]) for i in range(len(shape)))
        self.device = torch.device("cuda", device) if device >= 0 else torch.device("cpu")
        self.is_cuda = device >= 0

    def get_device(self):
        return self.index

    def dim(self):
        return len(self.shape)

    def numel(self):
        return math.prod(self.shape)

    def stride(self, i=None):
        return self.strides if i is None else self.strides[i]

    def is_contiguous(self):
        return True

    def element_size(self):
        return self.dtype.itemsize

    def data_ptr(self):
        return 4096


class Library:
    """Records (name, current device, arguments) and succeeds."""

    def __init__(self, world):
        self.world, self.calls = world, []

    def __getattr__(self, name):
        def call(*args):
            self.calls.append((name, self.world["device"], args))
            return 0
        return call


@pytest.fixture
def world(kvmod, monkeypatch):
    w = {"device": 0}

    @contextlib.contextmanager
    def device(index):
        before, w["device"] = w["device"], index
        yield
        w["device"] = before

    w["lib"] = Library(w)
    monkeypatch.setattr(kvmod, "lib", w["lib"])
    monkeypatch.setattr(kvmod, "_current_device", lambda: w["device"])
    monkeypatch.setattr(kvmod, "_raw_stream", lambda index: 1000 + index)
    monkeypatch.setattr(torch.cuda, "device", device)
    return w


def cache(kvmod, device):
    c = object.__new__(kvmod.KvCache)
    c._device, c._kv_heads, c._dim, c._dtype, c._ref = device, 2, 64, torch.bfloat16, None
    return c


def calls_of(c, device, other=None):
    """Every call on the cache; `other` names the tensor that is on another device."""
    def t(name, shape, dtype):
        return Fake(shape, dtype, device if name != other else device + 1)

    def ints(name, n):
        return t(name, (n,), torch.int32)

    def rows(name, heads):
        return t(name, (3, heads, 64), torch.bfloat16)

    return dict(
        fork=lambda: c.fork(ints("src", 3), ints("dst", 3)),
        reserve=lambda: c.reserve(ints("seqs", 3), ints("n_new", 3)),
        write=lambda: c.write(0, rows("k", 2), rows("v", 2), ints("seqs", 3), ints("cu", 4)),
        free=lambda: c.free(ints("seqs", 3)),
        copy_pages=lambda: c.copy_pages(ints("src", 3), ints("dst", 3)),
        attn_decode=lambda: c.attn_decode(0, rows("q", 4), ints("seqs", 3), out=rows("out", 4)),
        attn_prefill=lambda: c.attn_prefill(0, rows("q", 4), ints("seqs", 3), ints("cu", 4), out=rows("out", 4)),
    )


@pytest.mark.parametrize("device", [0, 1])
def test_calls_are_made_on_the_caches_device(kvmod, world, device):
    c = cache(kvmod, device)
    for current in (0, 1):
        world["device"] = current
        for call in calls_of(c, device).values():
            call()
        c.compact()
        c.check_errors()
    calls = world["lib"].calls
    assert len(calls) == 18 and all(at == device for _, at, _ in calls)
    assert all(args[-1] == 1000 + device for _, _, args in calls)  # that device's current stream
    assert world["device"] == 1  # as before the calls


@pytest.mark.parametrize("call,other", [("fork", "src"), ("fork", "dst"), ("reserve", "seqs"), ("reserve", "n_new"),
                                        ("write", "k"), ("write", "v"), ("write", "seqs"), ("write", "cu"),
                                        ("free", "seqs"), ("copy_pages", "src"), ("copy_pages", "dst"),
                                        ("attn_decode", "q"), ("attn_decode", "seqs"), ("attn_decode", "out"),
                                        ("attn_prefill", "q"), ("attn_prefill", "seqs"), ("attn_prefill", "cu"),
                                        ("attn_prefill", "out")])
def test_tensors_of_another_device_are_refused(kvmod, world, call, other):
    with pytest.raises(ValueError, match=f"{other} must be on cuda:0"):
        calls_of(cache(kvmod, 0), 0, other)[call]()
    with pytest.raises(TypeError, match="CUDA"):  # and of none
        calls_of(cache(kvmod, -2), -2, other)[call]()
    assert not world["lib"].calls


def test_linear_is_made_on_its_tensors_device(kvmod, world):
    x, w = Fake((2, 64), torch.bfloat16, 1), Fake((16 * 36,), torch.uint8, 1)
    y, bias = Fake((2, 16), torch.float32, 1), Fake((16,), torch.float32, 1)
    kvmod.quant_linear(x, w, 1, 16, bias=bias, y=y)
    (name, at, args), = world["lib"].calls
    assert name == "moe_quant_linear" and at == 1 and args[-1] == 1001 and world["device"] == 0
    for bad in ("w", "y", "bias"):
        t = dict(w=w, y=y, bias=bias)
        t[bad] = Fake(t[bad].shape, t[bad].dtype, 0)
        with pytest.raises(ValueError, match=f"^{bad} must be"):
            kvmod.quant_linear(x, t["w"], 1, 16, bias=t["bias"], y=t["y"])
    assert len(world["lib"].calls) == 1


@pytest.mark.parametrize("size", [2 ** 31, 2 ** 32 + 8, 2 ** 40])
def test_windows_past_32_bits_are_not_cut_to_their_low_half(kvmod, world, size):
    c = cache(kvmod, 0)
    q, seqs, cu = Fake((3, 4, 64), torch.bfloat16), Fake((3,), torch.int32), Fake((4,), torch.int32)
    c.attn_decode(0, q, seqs, out=q, window=size, sinks=size)
    c.attn_prefill(0, q, seqs, cu, out=q, window=size, sinks=size)
    for _, _, args in world["lib"].calls:
        assert args.count(2 ** 31 - 1) == 2 and size not in args
