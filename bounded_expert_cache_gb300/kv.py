"""Paged key-value cache, attention over it, rotary positions, the 4-bit linear layer and sampling: the
binding of include/moekv.h. PyTorch supplies device memory and streams; every
step runs in the library's CUDA kernels.
"""
from __future__ import annotations

import ctypes as C
import math
from typing import Optional

import torch

from . import _native as N
from ._native import lib
from .api import MoeError

_raw_stream = torch._C._cuda_getCurrentRawStream
_current_device = torch._C._cuda_getDevice


# These calls take microseconds on the device, so the binding keeps its own
# share small: plain integers for pointers, no temporary ctypes objects.
def _ok(st: int):
    if st != N.MOE_OK:
        raise MoeError(st, (lib.moe_last_error(None) or b"").decode(errors="replace"))


def _dtype_id(dtype: torch.dtype) -> int:
    if dtype == torch.float32:
        return N.F32
    if dtype == torch.bfloat16:
        return N.BF16
    raise TypeError(f"expected float32 or bfloat16 (got {dtype})")


def _elsewhere(t: torch.Tensor, name: str, device: int):
    """The error for a tensor that is not on the call's device."""
    if not t.is_cuda:
        return TypeError(f"{name} must be a CUDA tensor")
    return ValueError(f"{name} must be on cuda:{device} (is on cuda:{t.get_device()})")


_MOST = 2 ** 31 - 1  # a window or a count of first tokens beyond it hides no more, and keeps no more, than this


def _run(device: int, fn, *args):
    """The library launches on the current device: make it the tensors' one for the call."""
    if _current_device() == device:
        st = fn(*args)
    else:
        with torch.cuda.device(device):
            st = fn(*args)
    if st != N.MOE_OK:
        _ok(st)


def _new(shape, dtype, device, stream) -> torch.Tensor:
    """A result of a call on `stream`, from that stream's memory: a block that other streams' work may still use
    must not be written by this one."""
    if stream is None:
        return torch.empty(shape, dtype=dtype, device=device)
    with torch.cuda.stream(stream):
        return torch.empty(shape, dtype=dtype, device=device)


def _ints(t: torch.Tensor, name: str, device: int, n: Optional[int] = None) -> int:
    """Entries of an index list."""
    if t.dtype != torch.int32 or t.dim() != 1 or not t.is_contiguous():
        raise TypeError(f"{name} must be a contiguous one-dimensional int32 CUDA tensor")
    if t.get_device() != device:
        raise _elsewhere(t, name, device)
    have = t.shape[0]
    if n is not None and have != n:
        raise ValueError(f"{name} must hold {n} entries (got {have})")
    return have


def _head_rows(t: torch.Tensor, name: str, heads: Optional[int], dim: int, dtype: torch.dtype, device: int) -> int:
    """Row stride (elements) of [rows, heads, dim] whose rows are dense but may lie apart."""
    if t.dtype != dtype:
        raise TypeError(f"{name} must be a {dtype} CUDA tensor")
    if t.get_device() != device:
        raise _elsewhere(t, name, device)
    shape = t.shape
    if len(shape) != 3 or shape[2] != dim or (heads is not None and shape[1] != heads):
        raise ValueError(f"{name} must be [rows, {heads if heads is not None else 'heads'}, {dim}] "
                         f"(got {tuple(shape)})")
    rows, head, one = t.stride()
    if one != 1 or (shape[1] > 1 and head != dim):
        raise ValueError(f"the heads of a row of {name} must be dense")
    return rows if shape[0] > 1 else shape[1] * dim  # (a single row's stride leads nowhere)


class Rotary:
    """Rotary positions of the leading ``dim`` columns of a head (``moe_rotary_t``).

    Pairs are halves of those columns, or with ``interleaved`` neighbours. Frequency i
    is base^(-2i/dim) radians a position; for long contexts it is divided by ``factor``:
    every one with context 0, else those of at most turns[0] turns within ``context``
    tokens, less and less up to those of turns[1] turns, which stay: linearly in the turns
    (a rule that is linear in i instead needs ``angles``). ``angles``
    gives the dim / 2 frequencies themselves instead. Results are scaled by ``magnitude``.
    """

    def __init__(self, dim: int, base: float = 10000.0, interleaved: bool = False, factor: float = 1.0, context: int = 0,
                 turns=(1.0, 32.0), magnitude: float = 1.0, angles=None, device=None):
        if dim < 2 or dim % 2:
            raise ValueError("dim must be an even number of at least 2")
        n = dim // 2
        radians, fractions = (C.c_double * n)(), (C.c_uint64 * n)()
        if angles is None:
            _ok(lib.moe_rotary_angles(dim, base, factor, context, turns[0], turns[1], radians))
        else:
            if len(angles) != n:
                raise ValueError(f"angles must hold {n} entries (got {len(angles)})")
            radians[:] = [float(a) for a in angles]
        _ok(lib.moe_rotary_turns(radians, n, fractions))
        self.dim, self.interleaved, self.magnitude = dim, bool(interleaved), float(magnitude)
        self.angles = list(radians)
        # (a copy from pageable memory has been taken when the call returns, and is there before later work on any stream)
        self.turns = torch.frombuffer(fractions, dtype=torch.int64).to(device or torch.device("cuda"))
        if not self.turns.is_cuda:
            raise TypeError("a rotation's device must be a CUDA device")
        self.raw = N.RotaryT(self.turns.data_ptr(), dim, int(self.interleaved), self.magnitude)
        self._ref = C.byref(self.raw)
        self._device = self.turns.device.index


def _rotation(rot, device: int):
    if not isinstance(rot, Rotary):
        raise TypeError("the rotation must be a Rotary")
    if rot._device != device:
        raise ValueError(f"the rotation must be on cuda:{device} (is on cuda:{rot._device})")
    return rot._ref


def rotary(x: torch.Tensor, pos: torch.Tensor, rot: Rotary, out: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """x [rows, heads, head_dim] (float32 or bfloat16, rows may lie apart) turned to pos (int32 [rows]).

    ``out`` may be x itself. Runs on the current stream, or on ``stream``.
    """
    if x.dim() != 3 or not x.is_cuda:
        raise ValueError("x must be a [rows, heads, head_dim] CUDA tensor")
    xt = _dtype_id(x.dtype)
    device = x.get_device()
    rows, heads, dim = x.shape
    _ints(pos, "pos", device, rows)
    ldx = _head_rows(x, "x", heads, dim, x.dtype, device)
    if out is None:
        out = _new(x.shape, x.dtype, x.device, stream)
    elif out.shape != x.shape:
        raise ValueError("out must have x's shape")
    _run(device, lib.moe_rotary, _rotation(rot, device), pos.data_ptr(), x.data_ptr(), xt, ldx, rows, heads, dim, out.data_ptr(),
         _head_rows(out, "out", heads, dim, x.dtype, device), _raw_stream(device) if stream is None else stream.cuda_stream)
    return out


class KvCache:
    """Device arrays of a paged key-value cache (``moe_kv_t``).

    Either over tensors that the caller has (k, v: [layers, pages, kv_heads,
    page_tokens, head_dim]; table: int32 [max_seqs, max_pages]; lens: int32
    [max_seqs]; ref: int32 [pages]) or, with :meth:`empty`, over new ones.
    Pages of 4-bit codes are uint8 [layers, pages, kv_heads, page_tokens,
    head_dim * 9 / 16], where the last two dimensions together are a head's codes
    and behind them its scales and offsets; ``dtype`` is then the type of queries,
    results and new tokens.
    Sequence ids are rows of ``table``; every list of them is an int32 CUDA
    tensor, so that a captured step can be replayed with other contents.

    Calls run on the current stream, or on ``stream``; a result that a call
    makes itself is then that stream's. Inputs have to be ready there, and they
    and the cache have to live until the call has run.
    """

    def __init__(self, k: torch.Tensor, v: torch.Tensor, table: torch.Tensor, lens: torch.Tensor, ref: torch.Tensor,
                 dtype: Optional[torch.dtype] = None):
        for t, name, dims in ((k, "k", 5), (v, "v", 5), (table, "table", 2), (lens, "lens", 1), (ref, "ref", 1)):
            if not t.is_cuda or t.dim() != dims or not t.is_contiguous():
                raise TypeError(f"{name} must be a contiguous CUDA tensor of {dims} dimensions")
        codes = k.dtype == torch.uint8
        if dtype is None and codes:
            raise TypeError("pages of codes need the dtype of queries and new tokens")
        if dtype is not None and not codes and dtype != k.dtype:
            raise TypeError("dtype must be that of k and v")
        dtype = dtype or k.dtype
        kind = _dtype_id(dtype) | (N.KV_I4 if codes else 0)
        if k.shape != v.shape or k.dtype != v.dtype:
            raise ValueError("k and v must have one shape and type")
        if any(t.dtype != torch.int32 for t in (table, lens, ref)):
            raise TypeError("table, lens and ref must be int32")
        if lens.numel() != table.shape[0] or ref.numel() != k.shape[1]:
            raise ValueError("lens needs one entry per table row, ref one per page")
        if any(t.device != k.device for t in (v, table, lens, ref)):
            raise ValueError("the cache's tensors must be on one device")
        self.k, self.v, self.table, self.lens, self.ref = k, v, table, lens, ref
        L, P, Hkv, page, D = k.shape
        if codes:
            if D % 36:
                raise ValueError("the last dimension of pages of codes must be head_dim * 9 / 16, head_dim a multiple of 64")
            D = D * 16 // 9
        self.raw = N.KvT(k.data_ptr(), v.data_ptr(), table.data_ptr(), lens.data_ptr(), ref.data_ptr(), None, 0, L, P,
                         Hkv, page, D, kind, table.shape[0], table.shape[1])
        self._ref = C.byref(self.raw)
        self._device = k.device.index
        self._kv_heads, self._dim, self._dtype = Hkv, D, dtype
        n = C.c_int64()
        _run(self._device, lib.moe_kv_work_bytes, self._ref, C.byref(n))
        self.work = torch.zeros(n.value, dtype=torch.uint8, device=k.device)
        self.raw.work, self.raw.work_bytes = self.work.data_ptr(), n.value
        # the scratch is the cache's own: zero before a first call on whichever stream
        with torch.cuda.device(k.device):
            if not torch.cuda.is_current_stream_capturing():
                torch.cuda.current_stream().synchronize()

    def _st(self, stream) -> int:
        return _raw_stream(self._device) if stream is None else stream.cuda_stream

    @classmethod
    def empty(cls, n_layers, n_pages, n_kv_heads, page_tokens, head_dim, max_seqs, max_pages,
              dtype=torch.bfloat16, device=None, bits: int = 0) -> "KvCache":
        """bits: 4 for pages of 4-bit codes; 0 for pages of ``dtype``."""
        if bits not in (0, 4):
            raise ValueError("bits must be 0 (pages of dtype) or 4")
        if bits and head_dim % 64:
            raise ValueError("head_dim must be a multiple of 64 in a cache of 4-bit codes")
        dev = device or torch.device("cuda")
        shape = (n_layers, n_pages, n_kv_heads, page_tokens, head_dim * 9 // 16 if bits else head_dim)
        held = dict(dtype=torch.uint8 if bits else dtype, device=dev)
        i32 = dict(dtype=torch.int32, device=dev)
        return cls(torch.zeros(shape, **held), torch.zeros(shape, **held),
                   torch.full((max_seqs, max_pages), -1, **i32), torch.zeros(max_seqs, **i32),
                   torch.zeros(n_pages, **i32), dtype)

    @property
    def token_bytes(self) -> int:
        """Bytes of one token over all layers: kv_bytes_per_token of static_budget."""
        L, _, Hkv, _, D = self.k.shape
        return 2 * L * Hkv * D * self.k.element_size()

    def fork(self, src, dst, stream=None):
        """dst[i] becomes a sequence of src[i]'s tokens, sharing its pages."""
        n = _ints(src, "src", self._device)
        _ints(dst, "dst", self._device, n)
        _run(self._device, lib.moe_kv_fork, self._ref, src.data_ptr(), dst.data_ptr(), n, self._st(stream))

    def reserve(self, seqs, n_new, stream=None):
        """Pages for n_new[i] more tokens of seqs[i]; their lengths grow by it."""
        n = _ints(seqs, "seqs", self._device)
        _ints(n_new, "n_new", self._device, n)
        _run(self._device, lib.moe_kv_reserve, self._ref, seqs.data_ptr(), n_new.data_ptr(), n, self._st(stream))

    def write(self, layer, k, v, seqs, cu, stream=None):
        """Rows cu[i]..cu[i+1]-1 of k and v [rows, kv_heads, head_dim] become the newest tokens of seqs[i]."""
        n = _ints(seqs, "seqs", self._device)
        _ints(cu, "cu", self._device, n + 1)
        ldk = _head_rows(k, "k", self._kv_heads, self._dim, self._dtype, self._device)
        ldv = _head_rows(v, "v", self._kv_heads, self._dim, self._dtype, self._device)
        rows = k.shape[0]
        if rows != v.shape[0]:
            raise ValueError("k and v must have as many rows")
        _run(self._device, lib.moe_kv_write, self._ref, layer, k.data_ptr(), ldk, v.data_ptr(), ldv, seqs.data_ptr(),
             cu.data_ptr(), n, rows, self._st(stream))

    def write_rotary(self, layer, q, k, v, seqs, cu, rot, q_out=None, stream=None):
        """write with k turned to its tokens' positions on the way, and q [rows, heads, head_dim] into q_out.

        Returns q_out (new if None; it may be q itself). Rows of no sequence are left as they are in it.
        """
        n = _ints(seqs, "seqs", self._device)
        _ints(cu, "cu", self._device, n + 1)
        ldk = _head_rows(k, "k", self._kv_heads, self._dim, self._dtype, self._device)
        ldv = _head_rows(v, "v", self._kv_heads, self._dim, self._dtype, self._device)
        q_out, ldq, ldqo = self._q_out(q, q_out, stream, "q_out")
        rows, heads = q.shape[:2]
        if rows != v.shape[0] or rows != k.shape[0]:
            raise ValueError("q, k and v must have as many rows")
        _run(self._device, lib.moe_kv_write_rotary, self._ref, layer, _rotation(rot, self._device), q.data_ptr(), ldq, heads,
             q_out.data_ptr(), ldqo, k.data_ptr(), ldk, v.data_ptr(), ldv, seqs.data_ptr(), cu.data_ptr(), n, rows,
             self._st(stream))
        return q_out

    def read(self, layer, seqs, cu, rows, k=None, v=None, stream=None):
        """The newest cu[i+1]-cu[i] tokens of seqs[i] as rows cu[i].. of k and v [rows, kv_heads, head_dim].

        Returns k and v (new ones of ``rows`` rows if None). Rows of no sequence are left as they are.
        """
        n = _ints(seqs, "seqs", self._device)
        _ints(cu, "cu", self._device, n + 1)
        shape = (rows, self._kv_heads, self._dim)
        k = _new(shape, self._dtype, self.k.device, stream) if k is None else k
        v = _new(shape, self._dtype, self.k.device, stream) if v is None else v
        if k.shape != shape or v.shape != shape:
            raise ValueError(f"k and v must be {list(shape)}")
        ldk = _head_rows(k, "k", self._kv_heads, self._dim, self._dtype, self._device)
        ldv = _head_rows(v, "v", self._kv_heads, self._dim, self._dtype, self._device)
        _run(self._device, lib.moe_kv_read, self._ref, layer, k.data_ptr(), ldk, v.data_ptr(), ldv, seqs.data_ptr(),
             cu.data_ptr(), n, rows, self._st(stream))
        return k, v

    def free(self, seqs, stream=None):
        """Drop sequences; pages that no other sequence names become free."""
        n = _ints(seqs, "seqs", self._device)
        _run(self._device, lib.moe_kv_free, self._ref, seqs.data_ptr(), n, self._st(stream))

    def compact(self, stream=None):
        """Move the pages in use to the lowest ids."""
        _run(self._device, lib.moe_kv_compact, self._ref, self._st(stream))

    def copy_pages(self, src, dst, stream=None):
        """Copy whole pages src[i] -> dst[i] in every layer; table and ref are untouched."""
        n = _ints(src, "src", self._device)
        _ints(dst, "dst", self._device, n)
        _run(self._device, lib.moe_kv_copy_pages, self._ref, src.data_ptr(), dst.data_ptr(), n, self._st(stream))

    def check_errors(self, stream=None):
        """Synchronise, raise what kernels recorded on this cache, and clear it."""
        _run(self._device, lib.moe_kv_check_errors, self._ref, self._st(stream))

    @staticmethod
    def debug_attn_wait_timeout(wait_cycles: int, copies: int):
        """The next attention call of this thread runs into its bounded waits (a test hook)."""
        _ok(lib.moe_debug_attn_wait_timeout(wait_cycles, copies))

    def _q_out(self, q, out, stream, name="out"):
        """out (new if None) and the row strides of q and out."""
        ldq = _head_rows(q, "q", None, self._dim, self._dtype, self._device)
        if out is None:
            out = _new(q.shape, q.dtype, q.device, stream)
        elif out.shape != q.shape:
            raise ValueError(f"{name} must have q's shape")
        return out, ldq, _head_rows(out, name, None, self._dim, self._dtype, self._device)

    def attn_decode(self, layer, q, seqs, n_q=1, out=None, scale=None, window=0, sinks=0, stream=None):
        """Attention of the newest n_q tokens of each sequence: q [len(seqs) * n_q, heads, head_dim]."""
        n = _ints(seqs, "seqs", self._device)
        out, ldq, ldo = self._q_out(q, out, stream)
        rows, heads, dim = q.shape
        if rows != n * n_q:
            raise ValueError(f"q must have {n} x {n_q} rows (got {rows})")
        _run(self._device, lib.moe_attn_decode, self._ref, layer, q.data_ptr(), ldq, seqs.data_ptr(), n, n_q, heads,
             1.0 / math.sqrt(dim) if scale is None else scale, min(window, _MOST), min(sinks, _MOST), out.data_ptr(),
             ldo, self._st(stream))
        return out

    def attn_prefill(self, layer, q, seqs, cu, out=None, scale=None, window=0, sinks=0, stream=None):
        """Attention of chunks: rows cu[i]..cu[i+1]-1 of q are the newest tokens of seqs[i]."""
        n = _ints(seqs, "seqs", self._device)
        _ints(cu, "cu", self._device, n + 1)
        out, ldq, ldo = self._q_out(q, out, stream)
        rows, heads, dim = q.shape
        _run(self._device, lib.moe_attn_prefill, self._ref, layer, q.data_ptr(), ldq, seqs.data_ptr(), cu.data_ptr(), n,
             rows, heads, 1.0 / math.sqrt(dim) if scale is None else scale, min(window, _MOST), min(sinks, _MOST),
             out.data_ptr(), ldo, self._st(stream))
        return out


def quant_linear(x: torch.Tensor, w: torch.Tensor, quant: int, n_out: int, bias: Optional[torch.Tensor] = None,
                 y: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """y = x W^T (+ bias) for a 4-bit matrix W [n_out, K] in split-plane layout.

    x: [T, K] float32 or bfloat16 (rows may lie apart); w: uint8 with
    n_out*K/2 quant bytes and n_out*K/16 scale bytes; quant: Q4_0 or I4_G64;
    bias: float32 [n_out]; y: [T, n_out] float32 or bfloat16 (a new tensor of
    x's type if None).
    """
    if x.dim() != 2 or not x.is_cuda or (x.shape[1] > 1 and x.stride(1) != 1):
        raise ValueError("x must be a [T, K] CUDA tensor with dense rows")
    T, K = x.shape
    xt = _dtype_id(x.dtype)
    device = x.get_device()
    if w.dtype != torch.uint8 or w.get_device() != device or not w.is_contiguous() or w.numel() != n_out * K * 9 // 16:
        raise ValueError(f"w must be {n_out * K * 9 // 16} contiguous uint8 CUDA bytes on x's device")
    if bias is not None and (bias.dtype != torch.float32 or bias.get_device() != device or not bias.is_contiguous()
                             or bias.numel() != n_out):
        raise ValueError(f"bias must be a contiguous float32 CUDA tensor of {n_out} entries on x's device")
    if y is None:
        y = _new((T, n_out), x.dtype, x.device, stream)
    elif y.shape != (T, n_out) or y.get_device() != device or (n_out > 1 and y.stride(1) != 1):
        raise ValueError(f"y must be a [{T}, {n_out}] CUDA tensor with dense rows on x's device")
    ldx = x.stride(0) if T > 1 else K
    ldy = y.stride(0) if T > 1 else n_out
    _run(device, lib.moe_quant_linear, w.data_ptr(), quant, n_out, K, x.data_ptr(), xt, ldx, T,
         None if bias is None else bias.data_ptr(), y.data_ptr(), _dtype_id(y.dtype), ldy,
         _raw_stream(device) if stream is None else stream.cuda_stream)
    return y


def _column(t: torch.Tensor, name: str, dtype: torch.dtype, rows: int, device: int) -> int:
    """Address of one value a row."""
    if t.dtype != dtype or t.shape != (rows,) or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous {dtype} CUDA tensor of {rows} entries")
    if t.get_device() != device:
        raise _elsewhere(t, name, device)
    return t.data_ptr()


def sample(logits: torch.Tensor, u: torch.Tensor, temperature=1.0, top_k=0, top_p=1.0, min_p=0.0, token=None, prob=None,
           stream=None):
    """Draw one token of each row of logits [rows, V] (float32 or bfloat16, rows may lie apart) with u [rows] in [0, 1).

    temperature, top_p and min_p are numbers or float32 CUDA tensors [rows], top_k an
    integer or an int32 one. Kept are the top_k largest logits, of these the fewest
    with top_p of their weight, of these those of at least min_p times the largest's.
    The token is the first, by index, up to which their weights exceed u times the sum.
    Returns (token int32 [rows], prob float32 [rows]), new ones if None.
    """
    if logits.dim() != 2 or not logits.is_cuda:
        raise ValueError("logits must be a [rows, V] CUDA tensor with dense rows")
    zt = _dtype_id(logits.dtype)
    device = logits.get_device()
    rows, V = logits.shape
    ld, one = logits.stride()
    if one != 1 and V > 1:
        raise ValueError("logits must be a [rows, V] CUDA tensor with dense rows")
    by = N.SamplingT()
    if hasattr(temperature, "data_ptr"):
        by.temperatures = _column(temperature, "temperature", torch.float32, rows, device)
    else:
        by.temperature = float(temperature)
    if hasattr(top_k, "data_ptr"):
        by.top_ks = _column(top_k, "top_k", torch.int32, rows, device)
    else:
        by.top_k = min(max(int(top_k), 0), _MOST)
    if hasattr(top_p, "data_ptr"):
        by.top_ps = _column(top_p, "top_p", torch.float32, rows, device)
    else:
        by.top_p = float(top_p)
    if hasattr(min_p, "data_ptr"):
        by.min_ps = _column(min_p, "min_p", torch.float32, rows, device)
    else:
        by.min_p = float(min_p)
    at = _column(u, "u", torch.float32, rows, device)
    token = _new((rows,), torch.int32, logits.device, stream) if token is None else token
    prob = _new((rows,), torch.float32, logits.device, stream) if prob is None else prob
    _run(device, lib.moe_sample, logits.data_ptr(), zt, ld if rows > 1 else V, rows, V, at, C.byref(by),
         _column(token, "token", torch.int32, rows, device), _column(prob, "prob", torch.float32, rows, device),
         _raw_stream(device) if stream is None else stream.cuda_stream)
    return token, prob
