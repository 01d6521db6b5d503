"""Helpers of the layer operators' tests: inputs, plain forms in binary64, and
error bounds.  u = 2^-24 is binary32's unit roundoff; half(y) is half a unit in
the last place of the output's type at y."""
from __future__ import annotations

import numpy as np
import torch

from _util import spacing

U = 2.0 ** -24
TORCH = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32,
         "e4m3": torch.float8_e4m3fn}
LEAST = 2.0 ** -96


def randn(seed: int, *shape) -> torch.Tensor:
    g = torch.Generator()
    g.manual_seed(seed)
    return torch.randn(*shape, generator=g, dtype=torch.float64)


def placed(t: torch.Tensor, pad: int = 0, shift: int = 0, fill: float = float("nan")):
    """A CUDA copy of the matrix t inside a wider buffer: `pad` elements after
    each row, `shift` before the first.  Returns (view, buffer)."""
    rows, cols = t.shape
    buf = torch.full((shift + rows * (cols + pad),), fill, dtype=torch.float32,
                     device="cuda").to(t.dtype)
    view = buf[shift:].view(rows, cols + pad)[:, :cols]
    view.copy_(t)
    return view, buf


def untouched(buf: torch.Tensor, rows: int, cols: int, pad: int, shift: int) -> bool:
    """Whether everything around the matrix still holds NaN."""
    if not buf.is_floating_point() and "float8" not in str(buf.dtype):
        raise TypeError
    b = buf.float()
    edges = [b[:shift].reshape(-1), b[shift:].view(rows, cols + pad)[:, cols:].reshape(-1)]
    return all(bool(torch.isnan(e).all()) for e in edges)


def f64(t: torch.Tensor) -> np.ndarray:
    return t.detach().float().cpu().double().numpy()


def half(y: np.ndarray, dtype: str) -> np.ndarray:
    return 0.5 * spacing(y, dtype)


def e4m3_step(t: np.ndarray) -> np.ndarray:
    """Distance between E4M3 neighbours at |t|."""
    a = np.maximum(np.abs(t), 2.0 ** -6)
    return np.exp2(np.floor(np.log2(a)) - 3)


def assert_within(got: np.ndarray, want: np.ndarray, bound: np.ndarray, what: str):
    bad = ~(np.abs(got - want) <= bound)
    if bad.any():
        i = tuple(int(x) for x in np.argwhere(bad)[0])
        raise AssertionError("%s: %d of %d outside the bound; first at %s: got %r want %r bound %r"
                             % (what, int(bad.sum()), bad.size, i, got[i], want[i],
                                np.broadcast_to(bound, want.shape)[i]))
