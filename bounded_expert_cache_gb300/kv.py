"""Paged key-value cache, attention over it and the 4-bit linear layer: the
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


class KvCache:
    """Device arrays of a paged key-value cache (``moe_kv_t``).

    Either over tensors that the caller has (k, v: [layers, pages, kv_heads,
    page_tokens, head_dim]; table: int32 [max_seqs, max_pages]; lens: int32
    [max_seqs]; ref: int32 [pages]) or, with :meth:`empty`, over new ones.
    Sequence ids are rows of ``table``; every list of them is an int32 CUDA
    tensor, so that a captured step can be replayed with other contents.

    Calls run on the current stream, or on ``stream``; a result that a call
    makes itself is then that stream's. Inputs have to be ready there, and they
    and the cache have to live until the call has run.
    """

    def __init__(self, k: torch.Tensor, v: torch.Tensor, table: torch.Tensor, lens: torch.Tensor, ref: torch.Tensor):
        for t, name, dims in ((k, "k", 5), (v, "v", 5), (table, "table", 2), (lens, "lens", 1), (ref, "ref", 1)):
            if not t.is_cuda or t.dim() != dims or not t.is_contiguous():
                raise TypeError(f"{name} must be a contiguous CUDA tensor of {dims} dimensions")
        _dtype_id(k.dtype)
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
        self.raw = N.KvT(k.data_ptr(), v.data_ptr(), table.data_ptr(), lens.data_ptr(), ref.data_ptr(), None, 0, L, P,
                         Hkv, page, D, _dtype_id(k.dtype), table.shape[0], table.shape[1])
        self._ref = C.byref(self.raw)
        self._device = k.device.index
        self._kv_heads, self._dim, self._dtype = Hkv, D, k.dtype
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
              dtype=torch.bfloat16, device=None) -> "KvCache":
        dev = device or torch.device("cuda")
        shape = (n_layers, n_pages, n_kv_heads, page_tokens, head_dim)
        i32 = dict(dtype=torch.int32, device=dev)
        return cls(torch.zeros(shape, dtype=dtype, device=dev), torch.zeros(shape, dtype=dtype, device=dev),
                   torch.full((max_seqs, max_pages), -1, **i32), torch.zeros(max_seqs, **i32),
                   torch.zeros(n_pages, **i32))

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

    def _q_out(self, q, out, stream):
        """out (new if None) and the row strides of q and out."""
        ldq = _head_rows(q, "q", None, self._dim, self._dtype, self._device)
        if out is None:
            out = _new(q.shape, q.dtype, q.device, stream)
        elif out.shape != q.shape:
            raise ValueError("out must have q's shape")
        return out, ldq, _head_rows(out, "out", None, self._dim, self._dtype, self._device)

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
