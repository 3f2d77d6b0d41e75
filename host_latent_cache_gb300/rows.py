"""The device row cache and the 8-bit norm with torch tensors.

Latent rows that stay on the GPU, in bf16, compact (8-bit) or 4-bit rows
behind a page table: `RowCache` writes raw token rows into them (norm,
rotation, encoding), reads rows back, and attends to the 4-bit ones.
`norm_q8` makes the 8-bit rows that the indexer keys are.  PyTorch is used for
memory and streams only; every step runs in the CUDA library.

Calls run on the current stream of the tensors' device.  Arguments that the
kernels do not take as they are (another type, device, shape or layout) raise
ValueError; nothing is copied or converted on the way.
"""
from __future__ import annotations

import ctypes
import threading
import weakref
from typing import Optional, Sequence

import torch

from . import ess

FORMATS = {"bf16": ess.ESS_ROW_BF16, "compact": ess.ESS_ROW_COMPACT, "q4": ess.ESS_ROW_Q4}
PAIRS = {"adjacent": ess.ESS_ROPE_ADJACENT, "halves": ess.ESS_ROPE_HALVES}
LATENT, ROPE, ROW = 512, 64, 576
TILE = 128   # values per scale of norm_q8
MOST = (1 << 31) - 1   # of a size that the C calls take as int32


_BF16, _I32, _I64 = torch.bfloat16, torch.int32, torch.int64


def _need(ok: bool, what: str) -> None:
    if not ok:
        raise ValueError(what)


def _is(t, dtype, shape, index: int) -> bool:
    """t is a contiguous tensor of this type and shape on this CUDA device."""
    return (isinstance(t, torch.Tensor) and t.dtype is dtype and t.shape == shape and t.is_cuda
            and t.get_device() == index and t.is_contiguous())


def _is_rows(t, dtype, shape, index: int) -> bool:
    """The same, with contiguous rows at any stride."""
    return (isinstance(t, torch.Tensor) and t.dtype is dtype and t.shape == shape and t.is_cuda
            and t.get_device() == index
            and (t.is_contiguous() or t.stride(1) == 1 or shape[1] <= 1))


def _refuse(t, name: str, dtype, shape, index: int) -> None:
    what = (f"{t.dtype} {tuple(t.shape)} on {t.device}, strides {t.stride()}"
            if isinstance(t, torch.Tensor) else repr(type(t)))
    raise ValueError(f"{name}: {dtype} {tuple(shape)} on cuda:{index} with contiguous "
                     f"values is needed, not {what}")


def _check(t, name: str, dtype, shape, index: int) -> None:
    if not _is(t, dtype, shape, index):
        _refuse(t, name, dtype, shape, index)


def _check_rows(t, name: str, dtype, shape, index: int) -> None:
    if not _is_rows(t, dtype, shape, index):
        _refuse(t, name, dtype, shape, index)


def _row_stride(t) -> int:
    """Elements from row to row; of a single row, any that the kernels take."""
    n, dim = t.shape
    return t.stride(0) if n > 1 else -(-dim // 8) * 8


class _OnDevice:
    """Makes a device current for a call and puts the old one back; costs
    nothing when it is current already.  Yields the device's current stream."""

    __slots__ = ("index", "old")

    def __init__(self, index: int):
        self.index = index

    def __enter__(self) -> int:
        self.old = torch._C._cuda_getDevice()
        if self.old != self.index:
            torch.cuda.set_device(self.index)
        return torch._C._cuda_getCurrentRawStream(self.index)

    def __exit__(self, *exc):
        if self.old != self.index:
            torch.cuda.set_device(self.old)
        return False


class _Workspace:
    """What the eager calls on one stream of a device share, whichever cache makes
    them: the largest workspace any of them needed, and a lock that keeps a call's
    two launches together on the stream."""

    __slots__ = ("buf", "lock", "__weakref__")

    def __init__(self):
        self.buf = None
        self.lock = threading.Lock()


_workspaces = weakref.WeakValueDictionary()   # (device index, stream): as long as a cache uses it
_workspaces_lock = threading.Lock()


def release_workspaces() -> None:
    """Give up the workspaces that caches keep for their streams; the next call on
    a stream takes a new one."""
    with _workspaces_lock:
        kept = list(_workspaces.values())
    for ws in kept:
        with ws.lock:
            ws.buf = None


class RowCache:
    """A caller's tensor of cache rows, uint8 [n_rows][row bytes], with the
    calls on it.  `status` is a device int32 that keeps the first device-side
    error of the calls (see `poll`)."""

    def __init__(self, rows: torch.Tensor, fmt: str, page: int = 64):
        _need(fmt in FORMATS, f"format {fmt!r} is none of {', '.join(FORMATS)}")
        _need(1 <= page <= MOST, "a page has at least one row, and no more than 2^31 - 1")
        self.fmt, self.page = fmt, int(page)
        self._f = FORMATS[fmt]
        _need(isinstance(rows, torch.Tensor) and rows.is_cuda and rows.dim() == 2,
              "rows: a CUDA tensor [n_rows][row bytes] is needed")
        self.rows = rows
        self.n_rows = rows.shape[0]
        self.device = rows.device
        self._index = rows.get_device()
        _check(rows, "rows", torch.uint8, (self.n_rows, ess.ess_row_bytes(self._f)), self._index)
        self.status = torch.zeros(1, dtype=torch.int32, device=self.device)
        with _OnDevice(self._index):
            if not torch._C._cuda_isCurrentStreamCapturing():
                torch.cuda.current_stream().synchronize()   # any stream may use it from here on
        self._freq = (None, None)
        self._ws = {}       # by stream, shared with the other caches that run on it
        self._bytes = {}    # by shape

    def poll(self) -> int:
        """The first device-side error that is there, cleared.  Waits for the calls on
        the current stream; what a call that still runs on another stream reports
        is kept for a later poll."""
        with _OnDevice(self._index) as stream:
            taken = torch.empty(1, dtype=torch.int32, device=self.device)
            ess.ess_status_take(self.status, taken, stream)
            return int(taken.item())

    def _freqs(self, inv_freq: Sequence[float]):
        key = tuple(map(float, inv_freq))   # numbers: a tensor's entries may change later
        old, freq = self._freq
        if old != key:
            _need(len(key) == ROPE // 2, f"inv_freq has {len(key)} entries, not {ROPE // 2}")
            freq = (ctypes.c_double * len(key))(*key)
            self._freq = (key, freq)
        return freq

    def write(self, kv, slots, gamma=None, eps: float = 1e-6, pos=None, inv_freq=None,
              pairs: str = "adjacent") -> None:
        """Rows kv bf16 [n][576] (any row stride that is a multiple of 8) into
        the rows `slots` int64 [n] (negative: not written): the first 512
        values normed when gamma bf16 [512] is given, the last 64 rotated by
        pos int32 [n] when inv_freq (32 radians per position) is given."""
        at = self._index
        _need(isinstance(slots, torch.Tensor) and slots.dim() == 1, "slots: [n] is needed")
        n = slots.shape[0]
        _check(slots, "slots", _I64, (n,), at)
        _check_rows(kv, "kv", _BF16, (n, ROW), at)
        _need(pairs in PAIRS, f"pairs {pairs!r} is none of {', '.join(PAIRS)}")
        if gamma is not None:
            _check(gamma, "gamma", _BF16, (LATENT,), at)
        freq = None
        if inv_freq is None:
            pos = None
        else:
            freq = self._freqs(inv_freq)
            _check(pos, "pos", _I32, (n,), at)
        with _OnDevice(self._index) as stream:
            ess.ess_cache_write(kv, _row_stride(kv), n, gamma, eps, freq, pos, PAIRS[pairs], slots,
                                self.rows, self.n_rows, self._f, self.status, stream)

    def read(self, slots, out=None):
        """The rows `slots` int64 [n] as bf16 [n][576]; zeros for a negative slot."""
        at = self._index
        _need(isinstance(slots, torch.Tensor) and slots.dim() == 1, "slots: [n] is needed")
        n = slots.shape[0]
        _check(slots, "slots", _I64, (n,), at)
        if out is None:
            out = torch.empty((n, ROW), dtype=_BF16, device=self.device)
        else:
            _check(out, "out", _BF16, (n, ROW), at)
        with _OnDevice(self._index) as stream:
            ess.ess_cache_read(self.rows, self.n_rows, self._f, slots, n, out, self.status, stream)
        return out

    def workspace(self, batch: int, ways: int, heads: int) -> torch.Tensor:
        """A workspace for `attend`; one for each stream, or captured graph,
        that may run beside another."""
        n = ess.ess_cache_mla_bytes(batch, ways, heads)
        buf = torch.empty(n + 256, dtype=torch.uint8, device=self.device)
        off = (-buf.data_ptr()) % 256
        return buf[off:off + n]

    def attend(self, q, page_table, T, sm_scale: float, tokens=None, out=None, lse=None,
               workspace=None):
        """Attention of q bf16 [batch][ways][heads][576] over the cached tokens
        of each request (page_table int32 [batch][max_pages], T int32
        [batch]), or over tokens int32 [batch][ways][k].  Returns (out bf16
        [batch][ways][heads][512], lse float32 [batch][ways][heads]).  Without
        `workspace` all caches keep one for each current stream (see
        `release_workspaces`), and a captured call takes one from its graph's
        memory.  Threads may call it at once without `workspace`; calls that are
        given one are ordered by the caller.  An empty batch, list (k = 0) or page
        table is taken: queries without a token get zeros and lse = -infinity."""
        at = self._index
        _need(isinstance(q, torch.Tensor) and q.dim() == 4, "q: [batch][ways][heads][576] is needed")
        batch, ways, heads, _ = q.shape
        _check(q, "q", _BF16, (batch, ways, heads, ROW), at)
        _need(isinstance(page_table, torch.Tensor) and page_table.dim() == 2,
              "page_table: [batch][max_pages] is needed")
        max_pages = page_table.shape[1]
        _check(page_table, "page_table", _I32, (batch, max_pages), at)
        _check(T, "T", _I32, (batch,), at)
        k = 0
        if tokens is not None:
            _need(isinstance(tokens, torch.Tensor) and tokens.dim() == 3,
                  "tokens: [batch][ways][k] is needed")
            k = tokens.shape[2]
            _check(tokens, "tokens", _I32, (batch, ways, k), at)
        _need(max_pages <= MOST and k <= MOST, "more than 2^31 - 1 pages or listed tokens")
        if out is None:
            out = torch.empty((batch, ways, heads, LATENT), dtype=_BF16, device=self.device)
        else:
            _check(out, "out", _BF16, (batch, ways, heads, LATENT), at)
        if lse is None:
            lse = torch.empty((batch, ways, heads), dtype=torch.float32, device=self.device)
        else:
            _check(lse, "lse", torch.float32, (batch, ways, heads), at)
        if workspace is not None:
            _need(_is(workspace, torch.uint8, (workspace.numel(),), at)
                  if isinstance(workspace, torch.Tensor) else False,
                  f"workspace: contiguous uint8 [bytes] on cuda:{at} is needed")
        if batch == 0:
            return out, lse
        page = self.page
        if k == 0 and tokens is not None:      # as a list that holds nothing
            k = 1
            tokens = torch.full((batch, ways, 1), -1, dtype=_I32, device=self.device)
        if max_pages == 0:                     # as one page that is not there
            max_pages = page = 1
            page_table = torch.full((batch, 1), -1, dtype=_I32, device=self.device)
        with _OnDevice(at) as stream:
            if workspace is None:
                if torch._C._cuda_isCurrentStreamCapturing():
                    workspace = self.workspace(batch, ways, heads)
                else:
                    kept = self._ws.get(stream) or self._share(stream)
                    with kept.lock:
                        self._attend(q, page_table, max_pages, page, T, batch, ways, heads,
                                     tokens, k, sm_scale, out, lse,
                                     self._enough(kept, batch, ways, heads), stream)
                    return out, lse
            self._attend(q, page_table, max_pages, page, T, batch, ways, heads, tokens, k, sm_scale,
                         out, lse, workspace, stream)
        return out, lse

    def _share(self, stream: int) -> _Workspace:
        with _workspaces_lock:
            kept = _workspaces.get((self._index, stream))
            if kept is None:
                kept = _workspaces[self._index, stream] = _Workspace()
            self._ws[stream] = kept
        return kept

    def _enough(self, kept: _Workspace, batch: int, ways: int, heads: int) -> torch.Tensor:
        need = self._bytes.get((batch, ways, heads))
        if need is None:
            need = self._bytes[batch, ways, heads] = ess.ess_cache_mla_bytes(batch, ways, heads)
        if kept.buf is None or kept.buf.numel() < need:
            kept.buf = self.workspace(batch, ways, heads)
        return kept.buf

    def _attend(self, q, page_table, max_pages, page, T, batch, ways, heads, tokens, k, sm_scale,
                out, lse, workspace, stream) -> None:
        ess.ess_cache_mla(q, self.rows, self.n_rows, self._f, page_table, max_pages, page, T,
                          batch, ways, heads, tokens, k, sm_scale, out, lse, workspace,
                          workspace.numel(), self.status, stream)


def norm_q8(x, gamma, eps: float = 1e-6, residual=None, residual_out=None, codes=None,
            scales=None):
    """Root-mean-square norm of x (+ residual), bf16 [n][dim] at any row stride
    that is a multiple of 8, with e4m3 output: (codes float8_e4m3fn [n][dim],
    scales float32 [n][ceil(dim / 128)], x + residual as bf16 or None).
    residual_out may be x or residual."""
    _need(isinstance(x, torch.Tensor) and x.dim() == 2 and x.is_cuda,
          "x: a CUDA tensor [n][dim] is needed")
    n, dim = x.shape
    at = x.get_device()
    _need(dim <= MOST, "more than 2^31 - 1 values a row")
    _check_rows(x, "x", _BF16, (n, dim), at)
    _check(gamma, "gamma", _BF16, (dim,), at)
    r_stride = 0
    if residual is not None:
        _check_rows(residual, "residual", _BF16, (n, dim), at)
        r_stride = _row_stride(residual)
        if residual_out is None:
            residual_out = (torch.empty((n, dim), dtype=_BF16, device=x.device) if r_stride == dim else
                            torch.empty_strided((n, dim), (r_stride, 1), dtype=_BF16,
                                                device=x.device))
        else:
            _check_rows(residual_out, "residual_out", _BF16, (n, dim), at)
            _need(_row_stride(residual_out) == r_stride,
                  "residual_out and residual have one row stride")
    else:
        _need(residual_out is None, "residual_out without a residual")
    groups = -(-dim // TILE)
    if codes is None:
        codes = torch.empty((n, dim), dtype=torch.float8_e4m3fn, device=x.device)
    else:
        _check(codes, "codes", torch.float8_e4m3fn, (n, dim), at)
    if scales is None:
        scales = torch.empty((n, groups), dtype=torch.float32, device=x.device)
    else:
        _check(scales, "scales", torch.float32, (n, groups), at)
    with _OnDevice(at) as stream:
        ess.ess_norm_quant(x, _row_stride(x), residual, r_stride, gamma, eps, n, dim, residual_out,
                           codes, scales, stream)
    return codes, scales, residual_out
