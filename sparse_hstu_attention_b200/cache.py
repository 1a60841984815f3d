"""Paged 4-bit history cache for serving (include/hstu_cache.h).

Argument marshalling only, as in the package's other bindings: every step runs
in the library's CUDA kernels.  A serving loop keeps the users' histories
cached and brings only new rows, history events and candidates:

    tables = cache.allocate_tables(B, max_pages, num_pages, page_size=64, device="cuda")
    pages = [cache.allocate_pages(num_pages, H, d, 64, "cuda") for _ in layers]
    ...
    slots = cache.plan(tables, seq_offsets, num_targets, total_tokens=T)   # once a step
    for each layer:
        cache.append(k, v, slots, pages[l], tables)
        out = cache.attend(q, k, v, seq_offsets, num_targets, pages[l], tables,
                           contextual_len=32, K1=1024, K2=128, alpha=128 ** -0.5, N=16384.0,
                           max_new=most_rows)  # of any sequence of this step
    cache.get_error(tables)   # when the program synchronises anyway

Row b of the tables is a user slot; a step's batch has B sequences, one per
slot, of any number of rows (none for a slot with nothing new).  There is no
gradient: the outputs are new tensors outside autograd.  Attention with a relative
attention bias has no cached form.

Calls run on the tensors' own device, on its current stream unless `stream` is
given, and allocate only their outputs (and plan and attend their scratch), from
the memory of the stream they run on.  They can be captured into a CUDA graph and
replayed with other lengths, counts and offsets in the same tensors: nothing about
them is read on the host.
"""
from __future__ import annotations

import struct
from typing import Optional

import torch

from . import SLAError, _abi

__all__ = ["CacheTables", "allocate_tables", "allocate_pages", "plan", "slot_map", "append",
           "read", "attend", "get_error"]

_HEADER = 64  # int32 words before the lengths: word 0 the status, word 16 the free count


def _pad(n: int) -> int:
    return (n + 63) // 64 * 64


class CacheTables:
    """Lengths, free pages and block table of B user slots, in one contiguous
    CUDA int32 buffer (`buf.clone()` copies the whole state): a header of 64
    words (word 0 the status, word 16 the number of free pages), lengths [B],
    free_pages [num_pages], block_table [B, max_pages], each part starting at a
    multiple of 64 words."""

    __slots__ = ("buf", "device", "B", "max_pages", "num_pages", "page_size", "_c")

    def __init__(self, buf: torch.Tensor, B: int, max_pages: int, num_pages: int,
                 page_size: int):
        if buf.dtype is not torch.int32 or not buf.is_cuda or not buf.is_contiguous():
            raise TypeError("buf must be a contiguous CUDA int32 tensor")
        if B < 1 or max_pages < 1 or num_pages < 1:
            raise ValueError("B, max_pages and num_pages must be at least 1")
        if page_size not in (16, 32, 64) or max(B, max_pages, num_pages) >= 1 << 31:
            raise ValueError("page_size must be 16, 32 or 64, the sizes below 2^31")
        n = self.words(B, max_pages, num_pages)
        if buf.numel() < n:
            raise ValueError(f"buf has {buf.numel()} words, needs {n}")
        self.buf, self.device = buf, buf.device
        self.B, self.max_pages, self.num_pages, self.page_size = B, max_pages, num_pages, page_size
        p = buf.data_ptr()
        free = p + 4 * (_HEADER + _pad(B))
        self._c = _abi.CacheTablesC(B, max_pages, num_pages, page_size, p, p + 64,
                                    p + 4 * _HEADER, free, free + 4 * _pad(num_pages))

    @staticmethod
    def words(B: int, max_pages: int, num_pages: int) -> int:
        return _HEADER + _pad(B) + _pad(num_pages) + B * max_pages

    @property
    def status(self) -> torch.Tensor:
        return self.buf[0:1]

    @property
    def free_count(self) -> torch.Tensor:
        return self.buf[16:17]

    @property
    def lengths(self) -> torch.Tensor:
        return self.buf[_HEADER:_HEADER + self.B]

    @property
    def free_pages(self) -> torch.Tensor:
        at = _HEADER + _pad(self.B)
        return self.buf[at:at + self.num_pages]

    @property
    def block_table(self) -> torch.Tensor:
        at = _HEADER + _pad(self.B) + _pad(self.num_pages)
        return self.buf[at:at + self.B * self.max_pages].view(self.B, self.max_pages)


def allocate_tables(B: int, max_pages: int, num_pages: int, *, page_size: int = 64,
                    device="cuda") -> CacheTables:
    """Tables of an empty cache: all lengths 0, all pages free (page 0 on top)."""
    buf = torch.zeros(CacheTables.words(B, max_pages, num_pages), dtype=torch.int32,
                      device=device)
    t = CacheTables(buf, B, max_pages, num_pages, page_size)
    t.free_count.fill_(num_pages)
    t.free_pages.copy_(torch.arange(num_pages - 1, -1, -1, dtype=torch.int32))
    return t


def allocate_pages(num_pages: int, H: int, d: int, page_size: int = 64,
                   device="cuda") -> torch.Tensor:
    """One layer's pages: uint8 [num_pages, H, page_size * (d + 8)]; their
    contents need not be initialised."""
    return torch.empty((num_pages, H, page_size * (d + 8)), dtype=torch.uint8, device=device)


def _launch(device: torch.device, stream, where: str, call, *args):
    """call(*args, stream) with the tensors' device current (the library
    launches there); raises on a status other than OK."""
    i = device.index
    if i == torch._C._cuda_getDevice():
        code = call(*args, _stream(stream, i))
    else:
        with torch.cuda.device(device):
            code = call(*args, _stream(stream, i))
    if code != _abi.OK:
        raise SLAError(code, where)


def _stream(stream, index: int) -> int:
    # torch.cuda.current_stream() builds a Stream object, 2 us a call
    return torch._C._cuda_getCurrentRawStream(index) if stream is None else stream.cuda_stream


def _i32(t: Optional[torch.Tensor], n: int, name: str, device) -> Optional[int]:
    if t is None:
        return None
    if t.dtype is not torch.int32 or t.device != device or not t.is_contiguous():
        raise TypeError(f"{name} must be a contiguous int32 tensor on {device}")
    if t.numel() != n:
        raise ValueError(f"{name} must have {n} elements, got {t.numel()}")
    return t.data_ptr()


def _rows(t: torch.Tensor, name: str, T: int, H: int, d: int, device) -> int:
    """Checks a bf16 [T, H, d] tensor; returns its row stride."""
    if t.dtype is not torch.bfloat16 or t.device != device:
        raise TypeError(f"{name} must be a bfloat16 tensor on {device}")
    if t.shape != (T, H, d):
        raise ValueError(f"{name} must be [{T}, {H}, {d}], got {tuple(t.shape)}")
    row, head, dim = t.stride()
    if T > 0 and (dim != 1 or (H > 1 and head != d)):
        raise ValueError(f"{name}: heads and head_dim must be dense (stride (*, {d}, 1))")
    return row if T > 1 else H * d


def _pages(pages: torch.Tensor, tables: CacheTables):
    """(H, d, page stride in bytes) of a pages tensor."""
    if pages.dtype is not torch.uint8 or pages.device != tables.device or pages.dim() != 3:
        raise TypeError("pages must be a uint8 tensor [num_pages, H, page_size * (d + 8)] on the "
                        "tables' device")
    P, H, n = pages.shape
    ps = tables.page_size
    d = n // ps - 8
    if P != tables.num_pages or H < 1 or d < 1 or n != ps * (d + 8):
        raise ValueError(f"pages must be [{tables.num_pages}, H, {ps} * (d + 8)], got "
                         f"{tuple(pages.shape)}")
    page, head, byte = pages.stride()
    if byte != 1 or (H > 1 and head != n):
        raise ValueError("pages: the heads of a page must be dense")
    return H, d, page if P > 1 else H * n


def plan(tables: CacheTables, seq_offsets: torch.Tensor, num_targets: Optional[torch.Tensor] = None,
         *, total_tokens: int, release: Optional[torch.Tensor] = None,
         slots: Optional[torch.Tensor] = None, workspace: Optional[torch.Tensor] = None,
         stream=None) -> torch.Tensor:
    """One step's pages, slots and lengths (include/hstu_cache.h,
    hstu_cache_plan), written into `tables`; returns slots, int64
    [total_tokens], -1 for candidates and for rows behind seq_offsets[B].
    seq_offsets: int32 [B + 1]; num_targets: int32 [B], the trailing candidates
    of each sequence; release: int32 [B], non-zero empties the slot first."""
    dev = tables.device
    o = _i32(seq_offsets, tables.B + 1, "seq_offsets", dev)
    nt = _i32(num_targets, tables.B, "num_targets", dev)
    rel = _i32(release, tables.B, "release", dev)
    slots = _slots_out(slots, total_tokens, dev, stream)
    lib = _abi.load()
    ws = _workspace(workspace, lib.hstu_cache_plan_workspace_bytes(tables.B, total_tokens), dev,
                    stream)
    _launch(dev, stream, "hstu_cache_plan", lib.hstu_cache_plan, tables._c, o, nt, rel,
            total_tokens, slots.data_ptr(), None if ws is None else ws.data_ptr(),
            0 if ws is None else ws.numel())
    return slots


def _workspace(workspace: Optional[torch.Tensor], need: int, dev, stream):
    """The given workspace, checked, or a new one; None if the call needs none."""
    if workspace is None:
        if need == 0:
            return None
        workspace = _new(torch.uint8, dev, stream, need, out=False)
    elif workspace.dtype != torch.uint8 or workspace.device != dev or \
            not workspace.is_contiguous() or workspace.numel() < need:
        raise ValueError(f"workspace must be a contiguous uint8 tensor of {need} bytes on {dev}")
    return workspace


def _new(dtype, device, stream, *size, out: bool = True) -> torch.Tensor:
    """A tensor that a call allocates: from the memory of the stream that writes it, since
    what another stream has just released may still be in use there.  An output is then
    kept from reuse until the current stream, where the caller goes on, is done too."""
    if stream is None:  # (the sizes one by one: a tuple of them costs 1 us)
        return torch.empty(*size, dtype=dtype, device=device)
    with torch.cuda.stream(stream):
        t = torch.empty(*size, dtype=dtype, device=device)
    if out:
        t.record_stream(torch.cuda.current_stream(device))
    return t


def _slots_out(slots, total_tokens, dev, stream):
    if slots is None:
        return _new(torch.int64, dev, stream, total_tokens)
    _slots(slots, dev)
    if slots.numel() != total_tokens:
        raise ValueError(f"slots must have {total_tokens} elements")
    return slots


def _slots(slots, dev):
    if slots.dtype != torch.int64 or slots.device != dev or slots.dim() != 1 or \
            not slots.is_contiguous():
        raise TypeError(f"slots must be a contiguous int64 vector on {dev}")


def slot_map(tables: CacheTables, seq_offsets: torch.Tensor, *, total_tokens: int,
             slots: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """Slots of the last seq_offsets[b + 1] - seq_offsets[b] cached tokens of
    every sequence (e.g. to read whole histories back)."""
    dev = tables.device
    o = _i32(seq_offsets, tables.B + 1, "seq_offsets", dev)
    slots = _slots_out(slots, total_tokens, dev, stream)
    _launch(dev, stream, "hstu_cache_slot_map", _abi.load().hstu_cache_slot_map, tables._c, o,
            total_tokens, slots.data_ptr())
    return slots


def _pack(layout: struct.Struct, *values) -> bytes:
    try:
        return layout.pack(*values)
    except (struct.error, OverflowError) as e:
        raise ValueError(f"an argument is out of range ({e})") from None


def append(k: torch.Tensor, v: torch.Tensor, slots: torch.Tensor, pages: torch.Tensor,
           tables: CacheTables, *, stream=None) -> None:
    """Quantise the rows of k and v ([T, H, d] bf16) into `pages` at `slots`
    (rows with a negative slot are skipped)."""
    H, d, stride = _pages(pages, tables)
    dev = tables.device
    _slots(slots, dev)
    T = slots.numel()
    k_rs, v_rs = _rows(k, "k", T, H, d, dev), _rows(v, "v", T, H, d, dev)
    r = _pack(_abi.CACHE_ROWS, H, d, T, slots.data_ptr(), pages.data_ptr(), stride, k.data_ptr(),
              v.data_ptr(), k_rs, v_rs)
    _launch(dev, stream, "hstu_cache_append", _abi.load().hstu_cache_append_packed, tables._c, r)


def read(slots: torch.Tensor, pages: torch.Tensor, tables: CacheTables, *,
         k: Optional[torch.Tensor] = None, v: Optional[torch.Tensor] = None, stream=None):
    """The rows that `slots` hold, as bf16 (k, v) [T, H, d]; zeros for a
    negative slot."""
    H, d, stride = _pages(pages, tables)
    dev = tables.device
    _slots(slots, dev)
    T = slots.numel()
    k_rs = v_rs = H * d
    if k is None:
        k = _new(torch.bfloat16, dev, stream, T, H, d)
    else:
        k_rs = _rows(k, "k", T, H, d, dev)
    if v is None:
        v = _new(torch.bfloat16, dev, stream, T, H, d)
    else:
        v_rs = _rows(v, "v", T, H, d, dev)
    r = _pack(_abi.CACHE_ROWS, H, d, T, slots.data_ptr(), pages.data_ptr(), stride, k.data_ptr(),
              v.data_ptr(), k_rs, v_rs)
    _launch(dev, stream, "hstu_cache_read", _abi.load().hstu_cache_read_packed, tables._c, r)
    return k, v


def attend(q: torch.Tensor, k: Optional[torch.Tensor], v: Optional[torch.Tensor],
           seq_offsets: torch.Tensor, num_targets: Optional[torch.Tensor], pages: torch.Tensor,
           tables: CacheTables, *, contextual_len: int, K1: int, K2: int, alpha: float, N: float,
           max_new: Optional[int] = None, out: Optional[torch.Tensor] = None,
           workspace: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """SLA HSTU attention of the step's rows over the cached histories; returns
    out [T, H, d] bf16 (rows behind seq_offsets[B] are left as they were).  The
    step's history rows are in the cache already (plan, append); a candidate
    sees the history and, through its own row of k and v, itself.  k and v may
    be None when num_targets is.  max_new: a bound on the rows of any sequence, checked
    on the device.  Give it: it chooses the kernel and the launch's size.  Left out it is
    the whole batch's rows, and single events of many users then run as if one user might
    have them all (64 users, 4 heads of 128: 26 us instead of 9)."""
    H, d, stride = _pages(pages, tables)
    dev = tables.device
    T = q.shape[0]
    q_rs = _rows(q, "q", T, H, d, dev)
    k_ptr = v_ptr = k_rs = v_rs = 0
    if num_targets is not None:
        if k is None or v is None:
            raise ValueError("candidates (num_targets) need their rows of k and v")
        k_rs, v_rs = _rows(k, "k", T, H, d, dev), _rows(v, "v", T, H, d, dev)
        k_ptr, v_ptr = k.data_ptr(), v.data_ptr()
    o_rs = H * d
    if out is None:
        out = _new(torch.bfloat16, dev, stream, T, H, d)
    else:
        o_rs = _rows(out, "out", T, H, d, dev)
    p = _pack(_abi.CACHE_ATTEND, H, d, T, T if max_new is None else int(max_new),
              _i32(seq_offsets, tables.B + 1, "seq_offsets", dev),
              _i32(num_targets, tables.B, "num_targets", dev) or 0, int(contextual_len), int(K1),
              int(K2), alpha, N, q.data_ptr(), k_ptr, v_ptr, q_rs, k_rs, v_rs, pages.data_ptr(),
              stride, out.data_ptr(), o_rs)
    lib = _abi.load()
    ws = _workspace(workspace, lib.hstu_cache_attend_workspace_bytes_packed(tables._c, p), dev,
                    stream)
    _launch(dev, stream, "hstu_cache_attend", lib.hstu_cache_attend_packed, tables._c, p,
            None if ws is None else ws.data_ptr(), 0 if ws is None else ws.numel())
    return out


def get_error(tables: CacheTables, stream=None) -> int:
    """Synchronise `stream` (default: the current one) and return the tables'
    status (0 = no error)."""
    with torch.cuda.device(tables.device):
        return int(_abi.load().hstu_cache_get_error(tables._c,
                                                    _stream(stream, tables.device.index)))
