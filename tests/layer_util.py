"""Padded device matrices for the tests of the operators around the einsums (no arithmetic of
the method): a matrix inside wider, longer storage whose other elements must stay as they were."""

import numpy as np
import torch

DEV = "cuda"
BF, F32, E4, E8 = torch.bfloat16, torch.float32, torch.float8_e4m3fn, torch.float8_e8m0fnu
HALF = {BF: 2.0 ** -8, F32: 2.0 ** -24, E4: 2.0 ** -4}     # half a step, relative


def up(v, step):
    return -(-v // step) * step


class Padded:
    """`t`: [rows, cols] with ld = cols rounded up to `step`, plus `pad`, and a row behind.  What
    is not the matrix holds NaN of every type: it may neither be written nor reach a result."""

    def __init__(self, rows, cols, dtype, pad=0, step=8, value=None):
        self.rows, self.cols = rows, cols
        ld = up(cols, step) + up(pad, step)
        size = torch.empty((), dtype=dtype).element_size()
        self.bytes = torch.full(((rows + 1) * ld * size,), 0xff, dtype=torch.uint8, device=DEV)
        self.whole = self.bytes.view(dtype).view(rows + 1, ld)
        self.t = self.whole[:rows, :cols]
        if value is not None:
            self.t.copy_(value.to(DEV) if isinstance(value, torch.Tensor) else torch.as_tensor(value, device=DEV))

    def check_rest(self, what):
        size = self.t.element_size()
        b = self.bytes.view(self.rows + 1, -1)
        assert bool((b[self.rows] == 0xff).all()), f"{what}: the row behind was written"
        assert bool((b[:, self.cols * size:] == 0xff).all()), f"{what}: columns behind were written"


def f64(t):
    return t.detach().cpu().to(torch.float32).numpy().astype(np.float64)


def randn(shape, seed, std=1.0, dtype=F32):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(shape, generator=g) * std).to(dtype)


def uneven(rows, cols, seed, dtype):
    """Rows and columns of very different magnitude."""
    g = torch.Generator().manual_seed(seed)
    v = torch.randn((rows, cols), generator=g) * torch.exp(2 * torch.randn((rows, 1), generator=g))
    v = v * torch.where(torch.rand((1, cols), generator=g) < 0.02, 40.0, 1.0)
    return v.to(dtype)


def within(got, ref, tol, what):
    got, ref = np.asarray(got, np.float64), np.asarray(ref, np.float64)
    bad = ~(np.abs(got - ref) <= tol)
    assert not bad.any(), (f"{what}: {bad.sum()} of {bad.size} off, first at {np.argwhere(bad)[0]}: "
                           f"{got[tuple(np.argwhere(bad)[0])]} for {ref[tuple(np.argwhere(bad)[0])]}")
