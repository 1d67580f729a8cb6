"""GPU tests of the operators around the einsums at the ends of their ranges: scales and rows near
the types' limits, several calls in flight, many experts, the kernels for large products on values
as they come.  Tolerances as in test_gpu_layer.py: u = 2^-24 is half a step of fp32."""

import numpy as np
import pytest
import torch

from layer_util import BF, DEV, E4, E8, F32, HALF, Padded, f64, randn, uneven, within
from oracle import layer as ol, numerics

pytestmark = pytest.mark.gpu
EPS = 1e-5
U = 2.0 ** -24


@pytest.fixture(scope="module")
def ctx():
    import collective_overlap_amd as cce
    c = cce.Context(0)
    yield c
    torch.cuda.synchronize()
    c.close()


@pytest.mark.parametrize("rows,cols", [(3000, 4096), (600, 16392)])
def test_norm_backward_on_two_streams_with_workspaces_of_its_own(ctx, rows, cols):
    """No workspace given: calls of one shape on the current stream and on a side stream, in flight
    together, have memory of their own, so each gives the bits of a run alone."""
    import collective_overlap_amd as cce
    w = (1 + randn((cols,), 1, 0.2)).to(BF).to(DEV)
    x, d = ([randn((rows, cols), s + i, 1, BF).to(DEV) for i in range(2)] for s in (2, 4))
    dx, dw = [torch.empty_like(t) for t in x], [torch.empty(cols, device=DEV) for _ in x]
    want = []
    for i in range(2):
        cce.cce_rmsnorm_backward(ctx, x[i], w, d[i], dx[i], dw[i], EPS)
        torch.cuda.synchronize()
        want.append((dx[i].clone(), dw[i].clone()))
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    for step in range(6):
        for t in dx + dw:
            t.zero_()
        torch.cuda.synchronize()
        for i, s in (((0, None), (1, side)) if step % 2 else ((1, side), (0, None))):
            cce.cce_rmsnorm_backward(ctx, x[i], w, d[i], dx[i], dw[i], EPS, stream=s)
        torch.cuda.synchronize()
        for i in range(2):
            assert torch.equal(dw[i], want[i][1]) and torch.equal(dx[i], want[i][0]), f"step {step}, call {i}"
