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
from typing import Optional, Sequence

import torch

from . import ess

FORMATS = {"bf16": ess.ESS_ROW_BF16, "compact": ess.ESS_ROW_COMPACT, "q4": ess.ESS_ROW_Q4}
PAIRS = {"adjacent": ess.ESS_ROPE_ADJACENT, "halves": ess.ESS_ROPE_HALVES}
LATENT, ROPE, ROW = 512, 64, 576
TILE = 128   # values per scale of norm_q8


def _need(ok: bool, what: str) -> None:
    if not ok:
        raise ValueError(what)


def _tensor(t, name: str, dtype, shape, device, rows_apart: bool = False) -> None:
    """t is a tensor of this type, shape and device; contiguous, or (rows_apart)
    with contiguous rows at any stride."""
    _need(isinstance(t, torch.Tensor) and t.dtype == dtype, f"{name}: a {dtype} tensor is needed")
    _need(t.device == device, f"{name} is on {t.device}, not on {device}")
    _need(tuple(t.shape) == tuple(shape), f"{name} has shape {tuple(t.shape)}, not {tuple(shape)}")
    if rows_apart:
        _need(t.stride(-1) == 1 or t.shape[-1] <= 1 or t.numel() == 0,
              f"{name}: the values of a row are next to one another")
    else:
        _need(t.is_contiguous(), f"{name} is not contiguous")


def _on(device):
    """The call runs on this device's current stream, whatever the current device."""
    return torch.cuda.device(device)


class RowCache:
    """A caller's tensor of cache rows, uint8 [n_rows][row bytes], with the
    calls on it.  `status` is a device int32 that keeps the first device-side
    error of the calls (see `poll`)."""

    def __init__(self, rows: torch.Tensor, fmt: str, page: int = 64):
        _need(fmt in FORMATS, f"format {fmt!r} is none of {', '.join(FORMATS)}")
        _need(page >= 1, "a page has at least one row")
        self.fmt, self.page = fmt, int(page)
        self._f = FORMATS[fmt]
        _need(isinstance(rows, torch.Tensor) and rows.is_cuda and rows.dim() == 2,
              "rows: a CUDA tensor [n_rows][row bytes] is needed")
        _tensor(rows, "rows", torch.uint8, (rows.shape[0], ess.ess_row_bytes(self._f)), rows.device)
        self.rows = rows
        self.n_rows = rows.shape[0]
        self.device = rows.device
        self.status = torch.zeros(1, dtype=torch.int32, device=self.device)
        self._freq = (None, None)
        self._ws = {}

    def poll(self) -> int:
        """The first device-side error since the last poll (synchronous), cleared."""
        code = int(self.status.item())
        self.status.zero_()
        return code

    def _freqs(self, inv_freq: Optional[Sequence[float]]):
        if inv_freq is None:
            return None
        key = tuple(inv_freq)
        if self._freq[0] != key:
            _need(len(key) == ROPE // 2, f"inv_freq has {len(key)} entries, not {ROPE // 2}")
            self._freq = (key, (ctypes.c_double * len(key))(*key))
        return self._freq[1]

    def write(self, kv, slots, gamma=None, eps: float = 1e-6, pos=None, inv_freq=None,
              pairs: str = "adjacent") -> None:
        """Rows kv bf16 [n][576] (any row stride that is a multiple of 8) into
        the rows `slots` int64 [n] (negative: not written): the first 512
        values normed when gamma bf16 [512] is given, the last 64 rotated by
        pos int32 [n] when inv_freq (32 radians per position) is given."""
        dev = self.device
        n = slots.shape[0]
        _tensor(kv, "kv", torch.bfloat16, (n, ROW), dev, rows_apart=True)
        _tensor(slots, "slots", torch.int64, (n,), dev)
        _need(pairs in PAIRS, f"pairs {pairs!r} is none of {', '.join(PAIRS)}")
        if gamma is not None:
            _tensor(gamma, "gamma", torch.bfloat16, (LATENT,), dev)
        freq = self._freqs(inv_freq)
        if freq is not None:
            _need(pos is not None, "a rotation needs pos")
            _tensor(pos, "pos", torch.int32, (n,), dev)
        stride = kv.stride(0) if n > 1 else max(ROW, kv.stride(0) // 8 * 8)
        with _on(dev):
            ess.ess_cache_write(kv, stride, n, gamma, eps, freq, pos if freq is not None else None,
                                PAIRS[pairs], slots, self.rows, self.n_rows, self._f, self.status)

    def read(self, slots, out=None):
        """The rows `slots` int64 [n] as bf16 [n][576]; zeros for a negative slot."""
        n = slots.shape[0]
        _tensor(slots, "slots", torch.int64, (n,), self.device)
        if out is None:
            out = torch.empty((n, ROW), dtype=torch.bfloat16, device=self.device)
        else:
            _tensor(out, "out", torch.bfloat16, (n, ROW), self.device)
        with _on(self.device):
            ess.ess_cache_read(self.rows, self.n_rows, self._f, slots, n, out, self.status)
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
        `workspace` the cache keeps one for each current stream."""
        dev = self.device
        _need(isinstance(q, torch.Tensor) and q.dim() == 4, "q: [batch][ways][heads][576] is needed")
        batch, ways, heads, _ = q.shape
        _tensor(q, "q", torch.bfloat16, (batch, ways, heads, ROW), dev)
        _need(isinstance(page_table, torch.Tensor) and page_table.dim() == 2,
              "page_table: [batch][max_pages] is needed")
        max_pages = page_table.shape[1]
        _tensor(page_table, "page_table", torch.int32, (batch, max_pages), dev)
        _tensor(T, "T", torch.int32, (batch,), dev)
        k = 0
        if tokens is not None:
            _need(isinstance(tokens, torch.Tensor) and tokens.dim() == 3,
                  "tokens: [batch][ways][k] is needed")
            k = tokens.shape[2]
            _tensor(tokens, "tokens", torch.int32, (batch, ways, k), dev)
        if out is None:
            out = torch.empty((batch, ways, heads, LATENT), dtype=torch.bfloat16, device=dev)
        else:
            _tensor(out, "out", torch.bfloat16, (batch, ways, heads, LATENT), dev)
        if lse is None:
            lse = torch.empty((batch, ways, heads), dtype=torch.float32, device=dev)
        else:
            _tensor(lse, "lse", torch.float32, (batch, ways, heads), dev)
        with _on(dev):
            stream = torch.cuda.current_stream().cuda_stream
            if workspace is None:
                key = (stream, batch, ways, heads)
                workspace = self._ws.get(key)
                if workspace is None:
                    workspace = self._ws[key] = self.workspace(batch, ways, heads)
            ess.ess_cache_mla(q, self.rows, self.n_rows, self._f, page_table, max_pages, self.page,
                              T, batch, ways, heads, tokens, k, sm_scale, out, lse, workspace,
                              workspace.numel(), self.status, stream)
        return out, lse


def norm_q8(x, gamma, eps: float = 1e-6, residual=None, residual_out=None, codes=None,
            scales=None):
    """Root-mean-square norm of x (+ residual), bf16 [n][dim] at any row stride
    that is a multiple of 8, with e4m3 output: (codes float8_e4m3fn [n][dim],
    scales float32 [n][ceil(dim / 128)], x + residual as bf16 or None).
    residual_out may be x or residual."""
    _need(isinstance(x, torch.Tensor) and x.dim() == 2 and x.is_cuda, "x: a CUDA tensor [n][dim] is needed")
    n, dim = x.shape
    dev = x.device
    _tensor(x, "x", torch.bfloat16, (n, dim), dev, rows_apart=True)
    _tensor(gamma, "gamma", torch.bfloat16, (dim,), dev)
    apart = lambda t: t.stride(0) if n > 1 else max(dim, t.stride(0) // 8 * 8)
    r_stride = 0
    if residual is not None:
        _tensor(residual, "residual", torch.bfloat16, (n, dim), dev, rows_apart=True)
        r_stride = apart(residual)
        if residual_out is None:
            residual_out = torch.empty_strided((n, dim), (r_stride, 1), dtype=torch.bfloat16,
                                               device=dev)
        else:
            _tensor(residual_out, "residual_out", torch.bfloat16, (n, dim), dev, rows_apart=True)
            _need(apart(residual_out) == r_stride, "residual_out and residual have one row stride")
    else:
        _need(residual_out is None, "residual_out without a residual")
    groups = -(-dim // TILE)
    if codes is None:
        codes = torch.empty((n, dim), dtype=torch.float8_e4m3fn, device=dev)
    else:
        _tensor(codes, "codes", torch.float8_e4m3fn, (n, dim), dev)
    if scales is None:
        scales = torch.empty((n, groups), dtype=torch.float32, device=dev)
    else:
        _tensor(scales, "scales", torch.float32, (n, groups), dev)
    with _on(dev):
        ess.ess_norm_quant(x, apart(x), residual, r_stride, gamma, eps, n, dim, residual_out, codes,
                           scales)
    return codes, scales, residual_out
