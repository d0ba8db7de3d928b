"""The paged 4-bit cache: its handle and the calls that write and read it.

Like the rest of the binding this marshals arguments only: dl_paged_append, dl_paged_attn and
dl_paged_select carry the C names of include/dl.h and take torch tensors.  All tensors of a call
lie on one device; the call runs on that device's current stream unless `stream` names another, whose
memory the results then are that the call makes itself.
The tensors are checked in csrc/paged_call.c (in Python the checks took longer than a small call).
"""
from __future__ import annotations

import ctypes
from typing import Optional

import torch

from . import Rope, _check, _empty, dl_paged_kv, lib

_PAGES = (16, 32, 64, 128, 256)
_native = None


def _calls():
    """The compiled side of the calls, bound to the loaded library."""
    global _native
    if _native is None:
        L = lib()
        try:
            from . import _paged_call as m
        except ImportError as e:
            raise RuntimeError("_paged_call is not built for this interpreter (run __graft_entry__.build() or python "
                               "row_decode_step_gb300/_build.py, with a host compiler and Python.h)") from e
        m.bind(*(ctypes.cast(f, ctypes.c_void_p).value for f in (L.dl_paged_append, L.dl_paged_attn, L.dl_paged_select)),
               torch.float32, torch.int32, torch.uint8)
        _native = m
    return _native


def dl_paged_kv_bytes(n_pages: int, page: int, n_kv: int, head_dim: int):
    """(bytes of the pool, bytes of the mean plane)."""
    pb, mb = ctypes.c_size_t(), ctypes.c_size_t()
    _check(lib().dl_paged_kv_bytes(n_pages, page, n_kv, head_dim, ctypes.byref(pb), ctypes.byref(mb)))
    return pb.value, mb.value


class PagedKV:
    """A pool of pages: uint8 [n_pages][n_kv][page/16][18 * head_dim], and the pages' mean keys
    (float16 [n_pages][n_kv][head_dim]) where pages are to be selected from it."""

    def __init__(self, pool: torch.Tensor, page: int, head_dim: int, k_mean: Optional[torch.Tensor] = None):
        if page not in _PAGES or head_dim not in (64, 128):
            raise ValueError("pages of 16, 32, 64, 128 or 256 keys and heads of 64 or 128 channels, got %r and %r"
                             % (page, head_dim))
        if pool.dtype != torch.uint8 or pool.dim() != 4 or not pool.is_contiguous() or \
                tuple(pool.shape[2:]) != (page // 16, 18 * head_dim):
            raise ValueError("pool must be contiguous uint8 [n_pages][n_kv][%d][%d]" % (page // 16, 18 * head_dim))
        if k_mean is not None:
            if k_mean.dtype != torch.float16 or not k_mean.is_contiguous() or \
                    tuple(k_mean.shape) != (pool.shape[0], pool.shape[1], head_dim):
                raise ValueError("k_mean must be contiguous float16 [n_pages][n_kv][head_dim]")
            if k_mean.device != pool.device:
                raise ValueError("k_mean must be on the pool's device")
        self.pool, self.k_mean, self.page, self.head_dim = pool, k_mean, int(page), int(head_dim)
        self.n_pages, self.n_kv = int(pool.shape[0]), int(pool.shape[1])
        self.device, self.dev = pool.device, pool.get_device()
        self.c = dl_paged_kv(pool.data_ptr(), None if k_mean is None else k_mean.data_ptr(), self.n_pages, self.page,
                             self.n_kv, self.head_dim)
        self.addr = ctypes.addressof(self.c)

    @classmethod
    def empty(cls, n_pages: int, n_kv: int, page: int, head_dim: int, means: bool = False, device="cuda"):
        pool = torch.empty(n_pages, n_kv, page // 16, 18 * head_dim, dtype=torch.uint8, device=device)
        mean = torch.empty(n_pages, n_kv, head_dim, dtype=torch.float16, device=device) if means else None
        return cls(pool, page, head_dim, mean)


def _call(f, kv: PagedKV, stream, *args) -> None:
    """The call on the cache's device, on its current stream or `stream`."""
    dev = kv.dev
    if dev < 0:
        raise ValueError("the cache must lie on a CUDA device")
    s = torch._C._cuda_getCurrentRawStream(dev) if stream is None else stream.cuda_stream
    if dev == torch._C._cuda_getDevice():
        rc = f(kv.addr, dev, *args, s)
    else:
        with torch.cuda.device(dev):
            rc = f(kv.addr, dev, *args, s)
    if rc:
        _check(rc)


def dl_paged_append(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, pos: torch.Tensor, tables: torch.Tensor,
                    rope: Rope, kv: PagedKV, n_q: int, row_seq: Optional[torch.Tensor] = None,
                    bias: Optional[torch.Tensor] = None, q_out: Optional[torch.Tensor] = None,
                    k_out: Optional[torch.Tensor] = None, v_out: Optional[torch.Tensor] = None,
                    status: Optional[torch.Tensor] = None, stream=None) -> None:
    """Rotate the rows' q (into q_out, or in place) and k and store k and v in their pages; k_out and
    v_out receive the values the cache now holds."""
    _call(_calls().append, kv, stream, q, k, v, pos, tables, ctypes.addressof(rope.c), rope.table, n_q, row_seq, bias, q_out,
          k_out, v_out, status)


def dl_paged_attn_workspace_size(n_q: int, n_kv: int, head_dim: int) -> int:
    b = ctypes.c_size_t()
    _check(lib().dl_paged_attn_workspace_size(n_q, n_kv, head_dim, ctypes.byref(b)))
    return b.value


def paged_attn_workspace(n_q: int, n_kv: int, head_dim: int, device="cuda") -> torch.Tensor:
    """A zeroed workspace of dl_paged_attn for these heads, whatever the rows and lengths; calls whose
    kernels may overlap want one each."""
    with torch.cuda.device(device):
        n = dl_paged_attn_workspace_size(n_q, n_kv, head_dim)
    return torch.zeros(n, dtype=torch.uint8, device=device)


def dl_paged_attn(q: torch.Tensor, kv: PagedKV, tables: torch.Tensor, seqlen: torch.Tensor, workspace: torch.Tensor,
                  n_q: int, out: Optional[torch.Tensor] = None, lse: Optional[torch.Tensor] = None,
                  row_begin: Optional[torch.Tensor] = None, max_rows: int = 1, pages: Optional[torch.Tensor] = None,
                  status: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """Attention of the rows over their sequences' pages (all, or those that `pages` lists)."""
    if out is None:
        out = _empty(q.shape[0], n_q * kv.head_dim, dtype=torch.float32, device=kv.device, stream=stream)
    _call(_calls().attn, kv, stream, q, tables, seqlen, workspace, n_q, out, lse, row_begin, max_rows, pages, status)
    return out


def dl_paged_select(q: torch.Tensor, kv: PagedKV, tables: torch.Tensor, seqlen: torch.Tensor, n_q: int,
                    pages: Optional[torch.Tensor] = None, top_k: int = 64, n_sink: int = 1, n_local: int = 2,
                    status: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """The pages worth reading of every row and KV head (int32 [rows][n_kv][n_sink + top_k + n_local],
    ascending, -1 past them), for dl_paged_attn's `pages`."""
    if pages is None:
        pages = _empty(q.shape[0], kv.n_kv, n_sink + top_k + n_local, dtype=torch.int32, device=kv.device, stream=stream)
    _call(_calls().select, kv, stream, q, tables, seqlen, n_q, pages, top_k, n_sink, n_local, status)
    return pages
