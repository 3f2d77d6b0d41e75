"""8-bit quantisation and products with torch tensors.

`quant_q8` turns bf16 values into e4m3 codes with power-of-two scales, of 128
values of a row (activations) or of 128 x 128 values (weights); `Weight8` holds
a weight so quantised and multiplies 8-bit activations, as `quant_q8` or
`rows.norm_q8` make them, with it.  PyTorch is used for memory and streams only;
every step runs in the CUDA library.

Calls run on the current stream of the tensors' device.  Arguments that the
kernels do not take as they are (another type, device, shape or layout) raise
ValueError; nothing is copied or converted on the way.
"""
from __future__ import annotations

import torch

from . import ess
from .rows import (MOST, TILE, _BF16, _OnDevice, _check, _check_rows, _need, _new_status,
                   _row_stride, _take_status)

E4M3 = torch.float8_e4m3fn


def _groups(values: int) -> int:
    return -(-values // TILE)


def quant_q8(x, square: bool = False, codes=None, scales=None):
    """x bf16 [n][dim] at any row stride that is a multiple of 8 as (codes
    float8_e4m3fn [n][dim], scales float32): scales of 128 values of a row, [n][ceil(dim
    / 128)], or with `square` of 128 x 128 values, [ceil(n / 128)][ceil(dim / 128)]."""
    _need(isinstance(x, torch.Tensor) and x.dim() == 2 and x.is_cuda,
          "x: a CUDA tensor [n][dim] is needed")
    n, dim = x.shape
    at = x.get_device()
    _need(1 <= dim <= MOST and n <= MOST, "1 to 2^31 - 1 rows and values a row")
    _check_rows(x, "x", _BF16, (n, dim), at)
    shape = (_groups(n) if square else n, _groups(dim))
    if codes is None:
        codes = torch.empty((n, dim), dtype=E4M3, device=x.device)
    else:
        _check(codes, "codes", E4M3, (n, dim), at)
    if scales is None:
        scales = torch.empty(shape, dtype=torch.float32, device=x.device)
    else:
        _check(scales, "scales", torch.float32, shape, at)
    with _OnDevice(at) as stream:
        ess.ess_quant(x, _row_stride(x), n, dim, int(bool(square)), codes, scales, stream)
    return codes, scales


class Weight8:
    """A weight in 8 bits: codes float8_e4m3fn [outs][ins] and scales float32
    [ceil(outs / 128)][ceil(ins / 128)], powers of two, as `quant_q8(w, square=True)`
    gives them.  `status` is a device int32 that keeps the first device-side error of
    the products (see `poll`)."""

    def __init__(self, codes, scales):
        _need(isinstance(codes, torch.Tensor) and codes.is_cuda and codes.dim() == 2,
              "codes: a CUDA tensor [outs][ins] is needed")
        self.outs, self.ins = codes.shape
        self._index = codes.get_device()
        _need(1 <= self.outs <= MOST and 16 <= self.ins <= MOST and self.ins % 16 == 0,
              "outs of at least 1, and ins that are a multiple of 16")
        _check(codes, "codes", E4M3, (self.outs, self.ins), self._index)
        _check(scales, "scales", torch.float32, (_groups(self.outs), _groups(self.ins)),
               self._index)
        self.codes, self.scales = codes, scales
        self.device = codes.device
        self.status = _new_status(self._index)

    @classmethod
    def of(cls, w) -> "Weight8":
        """The weight w bf16 [outs][ins], quantised."""
        return cls(*quant_q8(w, square=True))

    def product(self, codes, scales, out=None, dtype=_BF16):
        """out [n][outs] = activations (codes float8_e4m3fn [n][ins], scales float32
        [n][ceil(ins / 128)]) times the transposed weight, in `dtype` (bf16 or float32),
        or into `out` of either type at any row stride."""
        at = self._index
        _need(isinstance(codes, torch.Tensor) and codes.dim() == 2, "codes: [n][ins] is needed")
        n = codes.shape[0]
        _check(codes, "codes", E4M3, (n, self.ins), at)
        _check(scales, "scales", torch.float32, (n, _groups(self.ins)), at)
        if out is None:
            if dtype is not _BF16 and dtype is not torch.float32:
                raise ValueError(f"results are bf16 or float32, not {dtype}")
            out = torch.empty((n, self.outs), dtype=dtype, device=self.device)
        else:
            dtype = out.dtype if isinstance(out, torch.Tensor) else _BF16
            if dtype is not _BF16 and dtype is not torch.float32:
                raise ValueError(f"results are bf16 or float32, not {dtype}")
            _check_rows(out, "out", dtype, (n, self.outs), at)
            _need(n < 2 or out.stride(0) >= self.outs, "out: rows that do not overlap are needed")
        with _OnDevice(at) as stream:
            ess.ess_product(codes, scales, n, self.codes, self.scales, self.outs, self.ins, out,
                            out.stride(0) if n > 1 else self.outs, int(dtype is torch.float32),
                            self.status, stream)
        return out

    def poll(self) -> int:
        """The first device-side error that is there, cleared.  Waits for the calls on
        the current stream."""
        return _take_status(self.status, self._index)
