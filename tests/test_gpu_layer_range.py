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


# ---- the 8-bit product -------------------------------------------------------------------
EVERY_PRODUCT_KERNEL = [(4, 4104, 400), (12, 4100, 272), (12, 8200, 272), (20, 2600, 272), (25, 8210, 272),
                        (40, 200, 1040), (130, 1000, 1040), (2100, 2060, 272), (4090, 4104, 272)]


def _e8(exponents):
    return (exponents + 127).to(torch.uint8).view(E8).to(DEV)


@pytest.mark.parametrize("m,n,k", EVERY_PRODUCT_KERNEL)
@pytest.mark.parametrize("ot", [BF, F32])
@pytest.mark.parametrize("scales", ["opposite", "ends"])
def test_scales_at_the_ends_of_their_range_give_the_product_in_range(ctx, m, n, k, ot, scales):
    """Scales of a and b up to 2^125 that cancel (opposite), and rows whose two scales together are
    2^-116 to 2^120 (ends), with values up to 256 in a and down to 2^-9 in b: integers in [-2, 2] or
    [-1, 1] times one power of two per row, so every sum is exact in fp32 and within its range, in
    each kernel."""
    import collective_overlap_amd as cce
    g = torch.Generator().manual_seed(m + n)
    kb, nb, top = -(-k // 128), -(-n // 128), 2 if scales == "opposite" else 1
    a, b = (torch.randint(-top, top + 1, (r, k), generator=g).float().to(DEV) for r in (m, n))
    if scales == "opposite":
        column = torch.randint(-125, 126, (1, kb), generator=g)
        total = torch.randint(-2, 3, (m, 1), generator=g)
    else:
        column = torch.randint(-1, 2, (1, kb), generator=g)
        total = torch.tensor([-116, -100, 0, 100, 120])[torch.randint(0, 5, (m, 1), generator=g)]
    ea, eb = total - column, column.expand(nb, kb)
    a, b = (a * (256 / top)).to(E4), (b * 2.0 ** -9).to(E4)
    c = torch.empty((m, -(-n // 8) * 8), device=DEV, dtype=ot)[:, :n]
    cce.cce_block_scaled_gemm(ctx, a, _e8(ea), b, _e8(eb), c)
    want = (a.double() @ b.double().t().contiguous()) * torch.exp2(total.double()).to(DEV)
    want = want.float().to(ot)
    assert torch.equal(c, want), f"{int((c != want).sum())} of {want.numel()} differ"
    if scales == "ends":
        s = _e8(ea)
        s.view(torch.uint8)[m // 2, 1] = 255
        cce.cce_block_scaled_gemm(ctx, a, s, b, _e8(eb), c)
        other = torch.arange(m, device=DEV) != m // 2
        assert bool(torch.isnan(c[m // 2]).all()) and torch.equal(c[other], want[other])


def test_the_largest_values_times_small_ones(ctx):
    """bf16's largest value quantises to 256 * 2^120; its product with weights of 2^-100 is in range."""
    import collective_overlap_amd as cce
    x = torch.full((3, 256), 3.3895e38, dtype=BF, device=DEV)
    w = torch.full((128, 256), 2.0 ** -100, device=DEV)
    q, s = torch.empty((3, 256), device=DEV, dtype=E4), torch.empty((3, 2), device=DEV, dtype=E8)
    b, t = torch.empty((128, 256), device=DEV, dtype=E4), torch.empty((1, 2), device=DEV, dtype=E8)
    cce.cce_quantize_blocks(ctx, x, q, s, 1)
    cce.cce_quantize_blocks(ctx, w, b, t, 128)
    c = torch.empty((3, 128), device=DEV)
    cce.cce_block_scaled_gemm(ctx, q, s, b, t, c)
    assert bool((c == 256 * 2.0 ** 28).all()), c[0, 0].item()


@pytest.mark.parametrize("m,n,k", [(4, 4104, 32), (20, 2600, 32), (40, 200, 32), (130, 1000, 32), (2100, 2060, 32)])
def test_gelu_of_fp32_results_is_fp32(ctx, m, n, k):
    """Sums that are exact in fp32 (multiples of 1/16, to beyond 6 on both sides), so that the error
    is GELU's own, relative to the result: the exponent x^2 / 2 is rounded twice, with a factor off
    by 0.22 u, 1.2 x^2 u; the reciprocal in erfc's argument by 3 u, which counts threefold at x = 0;
    a polynomial of degree 8 and its coefficients 5 u; the exponential 2 u, the products 3 u.  (An
    erf good to 1.5e-7 is off by 3e-3, 50000 u, at x = -4.)"""
    import collective_overlap_amd as cce
    g = torch.Generator().manual_seed(m)
    a, b = (torch.randint(-2, 3, (r, k), generator=g).float().to(DEV).to(E4) for r in (m, n))
    c, y = (torch.empty((m, -(-n // 8) * 8), device=DEV)[:, :n] for _ in range(2))
    sa, sb = _e8(torch.randint(-4, 1, (m, 1), generator=g)), _e8(torch.zeros(-(-n // 128), 1))
    cce.cce_block_scaled_gemm(ctx, a, sa, b, sb, c)
    cce.cce_block_scaled_gemm(ctx, a, sa, b, sb, y, gelu=True)
    x = c.double()
    assert torch.equal(x, (a.double() @ b.double().t().contiguous()) * sa.float().double())
    ref = 0.5 * x * torch.special.erfc(-x * 2 ** -0.5)
    tol = (1.2 * x * x + 20) * U * ref.abs() + 1e-37
    bad = ~((y.double() - ref).abs() <= tol)
    assert not bool(bad.any()), (int(bad.sum()), x[bad][0].item(), y[bad][0].item(), ref[bad][0].item())


# ---- the products grouped by expert --------------------------------------------------------
def test_few_rows_of_many_experts_times_a_wide_shared_matrix(ctx):
    """1024 rows of 256 experts and 2^20 columns: 20 million tiles that there could be, for a grid
    that takes them in turn.  One matrix for all experts, so one product is the reference."""
    import collective_overlap_amd as cce
    rows, n, k, experts = 1024, 1 << 20, 16, 256
    g = torch.Generator(device=DEV).manual_seed(1)
    a = torch.randint(-3, 4, (rows, k), generator=g, device=DEV).to(BF)
    w = torch.randint(-3, 4, (n, k), generator=g, device=DEV).to(BF)
    off = torch.arange(experts + 1, device=DEV) * 4
    off[1:9] = torch.tensor([0, 1, 1, 20, 20, 21, 25, 32], device=DEV)
    c = torch.full((rows, n), 5.0, device=DEV, dtype=BF)
    cce.cce_ragged_gemm(ctx, a, w.expand(experts, n, k), off, c)
    wt = w.float().t().contiguous()
    for i in range(0, rows, 128):
        assert torch.equal(c[i:i + 128], (a[i:i + 128].float() @ wt).to(BF)), f"rows from {i}"


@pytest.mark.parametrize("ot", [BF, F32])
def test_product_of_the_most_rows(ctx, ot):
    """2^30 rows, the documented most, of 16 and 8 columns."""
    import collective_overlap_amd as cce
    m, n, k = 1 << 30, 8, 16
    pick = torch.tensor([0, 255, 256, (1 << 29) + 1, (1 << 30) - 257, (1 << 30) - 1], device=DEV)
    g = torch.Generator(device=DEV).manual_seed(1)
    a = torch.zeros((m, k), device=DEV, dtype=torch.uint8).view(E4)
    some = torch.randint(-3, 4, (len(pick), k), generator=g, device=DEV).float()
    a.view(torch.uint8)[pick] = some.to(E4).view(torch.uint8)
    b = torch.randint(1, 4, (n, k), generator=g, device=DEV).float()
    s = torch.full((m, 1), 127, device=DEV, dtype=torch.uint8).view(E8)
    c = torch.empty((m, n), device=DEV, dtype=ot)
    cce.cce_block_scaled_gemm(ctx, a, s, b.to(E4), _e8(torch.zeros(1, 1)), c)
    want = (some.double() @ b.double().t().contiguous()).to(ot)
    assert torch.equal(c[pick], want)
    assert sum(int(torch.count_nonzero(x)) for x in c.split(1 << 26)) == int(torch.count_nonzero(want))


# ---- the row-wise operators ------------------------------------------------------------------
@pytest.mark.parametrize("cols", [(1 << 31) - 8, (1 << 31) - 131])
def test_one_row_of_nearly_two_to_the_31_columns(ctx, cols):
    """The widest row that can be asked for: the last lanes' columns pass 2^31.  Zeros but for a few
    columns, so that the sums are exact: the norm's error is that of its root and products."""
    import collective_overlap_amd as cce
    pick = torch.tensor([0, 7, 8, 4097, (1 << 30) - 1, 1 << 30, cols - 2050, cols - 9, cols - 1], device=DEV)
    v = 2.0 ** torch.arange(9, dtype=torch.float64)
    v = v * torch.tensor([1, -1, 1, 1, -1, 1, -1, 1, 1])
    def row(dtype):
        return torch.zeros((1, (1 << 31) - 8), device=DEV, dtype=torch.uint8).view(dtype)[:, :cols] if dtype == E4 else \
            torch.zeros((1, (1 << 31) - 8), device=DEV, dtype=dtype)[:, :cols]
    x = row(BF)
    x[0, pick] = v.to(BF).to(DEV)
    rstd = 1 / np.sqrt(float((v * v).sum()) / cols + EPS)
    for br in (1, 128):
        q, s = row(E4), torch.zeros((1, -(-cols // 128)), device=DEV, dtype=torch.uint8).view(E8)
        cce.cce_quantize_blocks(ctx, x, q, s, br)
        got = q[0, pick].float().double().cpu() * s[0, pick // 128].float().double().cpu()
        assert torch.equal(got, v), (br, got)
        assert int(torch.count_nonzero(q.view(torch.uint8))) == len(pick)
        del q, s
    w = torch.ones((1 << 31) - 8, device=DEV, dtype=BF)[:cols]
    out = row(BF)
    cce.cce_rmsnorm(ctx, x, w, out, EPS)
    within(f64(out[0, pick]), (v * rstd).numpy(), (2.0 ** -8 + 8 * U) * np.abs((v * rstd).numpy()), "out")
    assert int(torch.count_nonzero(out)) == len(pick)
    q, s = row(E4), torch.zeros((1, -(-cols // 128)), device=DEV, dtype=torch.uint8).view(E8)
    cce.cce_rmsnorm(ctx, x, w, q, EPS, scales=s)
    got = q[0, pick].float().double().cpu().numpy() * s[0, pick // 128].float().double().cpu().numpy()
    within(got, (v * rstd).numpy(), (2.0 ** -4 + 8 * U) * np.abs((v * rstd).numpy()), "e4m3")
    assert int(torch.count_nonzero(q.view(torch.uint8))) == len(pick)
    del q, s
    # dout = x: the mean of w dout n and n are exact but for the root; dweight = x n
    dx, dw = out, torch.full((cols,), 3.0, device=DEV)
    cce.cce_rmsnorm_backward(ctx, x, w, x, dx, dw, EPS)
    n = (v * rstd).numpy()
    mean = float((v.numpy() * n).sum()) / cols
    mag = (np.abs(v.numpy()) + np.abs(n) * mean) * rstd
    within(f64(dx[0, pick]), (v.numpy() - n * mean) * rstd, (2.0 ** -8 + 24 * U) * mag, "dx")
    within(f64(dw[pick]), v.numpy() * n, 12 * U * np.abs(v.numpy() * n), "dweight")
    assert int(torch.count_nonzero(dw)) == len(pick) and int(torch.count_nonzero(dx)) == len(pick)


@pytest.mark.parametrize("cols", [40, 128, 200, 600, 1000, 2000, 4096, 8000, 12288, 16392])
@pytest.mark.parametrize("xt", [BF, F32])
@pytest.mark.parametrize("d_residual", [False, True])
def test_norm_backward_of_overflowing_infinite_and_nan_rows(ctx, cols, xt, d_residual):
    """A row whose squares pass fp32's range has a norm of zero, so no gradient passes it, also
    where the sum of w dout x overflows; a row with an infinity has n = NaN there and 0 elsewhere,
    so its mean and its dx are NaN, and dweight in that column; a NaN makes the row NaN, and
    dweight.  Other rows keep theirs."""
    import collective_overlap_amd as cce
    rows = 70
    x, d = randn((rows, cols), 1, 1, xt), randn((rows, cols), 2, 1, xt)
    x[3] = 3e38 * torch.sign(x[3]) * (1 if xt == F32 else 0.99)
    d[3] = 1e30 * torch.sign(x[3])
    x[37] = 1e25
    x[41, cols // 2] = float("inf")
    w = (1 + randn((cols,), 3, 0.2)).to(DEV)
    r = randn((rows, cols), 4, 1, xt).to(DEV) if d_residual else None
    dx, dw = torch.empty((rows, cols), device=DEV, dtype=xt), torch.empty(cols, device=DEV)
    cce.cce_rmsnorm_backward(ctx, x.to(DEV), w, d.to(DEV), dx, dw, EPS, d_residual=r)
    for i in (3, 37):
        assert torch.equal(dx[i], r[i] if d_residual else torch.zeros_like(dx[i])), i
    assert bool(torch.isnan(dx[41]).all())
    other = [i for i in range(rows) if i not in (3, 37, 41)]
    ref, _ = ol.rmsnorm_backward(f64(x[other]), f64(w), f64(d[other]), EPS, None if r is None else f64(r[other]))
    got = f64(dx[other])
    assert np.linalg.norm(got - ref) <= (HALF[xt] + 4 * cols * U) * np.linalg.norm(ref)
    column = torch.arange(cols, device=DEV) == cols // 2
    assert bool(torch.isnan(dw[column]).all())
    some = [i for i in range(rows) if i != 41]
    x64 = f64(x)
    x64[[3, 37]] = 0.0
    _, refw = ol.rmsnorm_backward(x64[some], f64(w), np.where(np.abs(f64(d[some])) > 1e29, 0, f64(d[some])), EPS)
    keep = ~column.cpu().numpy()
    assert np.linalg.norm((f64(dw) - refw)[keep]) <= 1e-5 * np.linalg.norm(refw[keep])
    x[41, cols // 2], x[5, 1] = 1.0, float("nan")
    cce.cce_rmsnorm_backward(ctx, x.to(DEV), w, d.to(DEV), dx, dw, EPS, d_residual=r)
    bad = torch.isnan(dx).any(1).cpu()
    assert bool(torch.isnan(dx[5]).all()) and int(bad.sum()) == 1 and bool(torch.isnan(dw).all())


@pytest.mark.parametrize("rows,cols", [(300, 100), (40, 700), (30, 4104), (20, 16400)])
def test_norm_backward_without_the_weight_gradient_allocates_nothing(ctx, rows, cols):
    import collective_overlap_amd as cce
    x, d, dx, dx2 = (randn((rows, -(-cols // 8) * 8), s, 1, BF).to(DEV)[:, :cols] for s in range(4))
    w, dw = torch.ones(cols, device=DEV), torch.empty(cols, device=DEV)
    cce.cce_rmsnorm_backward(ctx, x, w, d, dx2, dw, EPS)
    torch.cuda.synchronize()
    torch.cuda.reset_peak_memory_stats()
    before = torch.cuda.memory_allocated()
    cce.cce_rmsnorm_backward(ctx, x, w, d, dx, None, EPS)
    torch.cuda.synchronize()
    assert torch.cuda.max_memory_allocated() == before and torch.equal(dx, dx2)


# ---- the kernels for large products, on values as they come ----------------------------------
def _quantised(ctx, rows, cols, block_rows, pad, value):
    """Quantised by the call under test elsewhere, inside wider storage full of NaN."""
    import collective_overlap_amd as cce
    x = torch.empty((rows, -(-cols // 8) * 8), device=DEV)[:, :cols].copy_(value.to(DEV))
    q = Padded(rows, cols, E4, pad, 16)
    s = Padded(-(-rows // block_rows), -(-cols // 128), E8, 3, 1)
    cce.cce_quantize_blocks(ctx, x, q.t, s.t, block_rows)
    wide = s.t.float().double().repeat_interleave(block_rows, 0)[:rows].repeat_interleave(128, 1)[:, :cols]
    return q, s, q.t.float().double() * wide


@pytest.mark.parametrize("m,n,k", [(1500, 1030, 400), (2000, 1100, 4240), (4090, 4104, 272), (5000, 3600, 1040)])
@pytest.mark.parametrize("gelu", [False, True])
def test_large_products_of_uneven_values(ctx, m, n, k, gelu):
    """128 x 128 and 256 x 256 tiles of the 8-bit instruction: what it leaves out of its sums of 64
    products is at most 2^-12 of the sum of their magnitudes (test_gpu_layer.py), GELU has a slope
    of at most 1.13 and is off by 4e-7 |c|, and the result is rounded to bf16."""
    import collective_overlap_amd as cce
    a, sa, wa = _quantised(ctx, m, k, 1, 16, uneven(m, k, m, F32))
    b, sb, wb = _quantised(ctx, n, k, 128, 32, randn((n, k), n, 0.05))
    c = Padded(m, n, BF, 8)
    cce.cce_block_scaled_gemm(ctx, a.t, sa.t, b.t, sb.t, c.t, gelu=gelu)
    torch.cuda.synchronize()
    c.check_rest("c")
    wbt = wb.t().contiguous()
    ref, mag = wa @ wbt, wa.abs() @ wbt.abs()
    tol = mag * 2.0 ** -12
    if gelu:
        tol = 1.13 * tol + 4e-7 * ref.abs()
        ref = torch.special.ndtr(ref) * ref
    bad = ~((c.t.double() - ref).abs() <= tol + 2.0 ** -8 * ref.abs())
    assert not bool(bad.any()), f"{int(bad.sum())} of {bad.numel()} off"


@pytest.mark.parametrize("m,n,k", [(1500, 1030, 400), (4090, 4104, 272)])
def test_a_nan_scale_of_a_large_product_stays_in_its_row_or_block(ctx, m, n, k):
    import collective_overlap_amd as cce
    a, sa, _ = _quantised(ctx, m, k, 1, 16, uneven(m, k, m, F32))
    b, sb, _ = _quantised(ctx, n, k, 128, 32, randn((n, k), n, 0.05))
    want, c = (torch.empty((m, -(-n // 8) * 8), device=DEV, dtype=BF)[:, :n] for _ in range(2))
    cce.cce_block_scaled_gemm(ctx, a.t, sa.t, b.t, sb.t, want)
    row = torch.arange(m, device=DEV) == m // 2
    block = (torch.arange(n, device=DEV) // 128) == 3
    for s, i, j in ((sa, m // 2, 2), (sb, 3, 1)):
        bytes_ = s.t.view(torch.uint8)
        keep = bytes_[i, j].item()
        bytes_[i, j] = 255
        cce.cce_block_scaled_gemm(ctx, a.t, sa.t, b.t, sb.t, c)
        bytes_[i, j] = keep
        hit = row[:, None].expand(m, n) if s is sa else block[None].expand(m, n)
        assert bool(torch.isnan(c[hit]).all()) and torch.equal(c[~hit], want[~hit])


@pytest.mark.parametrize("experts,rows,n,k", [(200, 600, 1000, 203), (70, 150, 5000, 64), (1000, 3000, 264, 40)])
@pytest.mark.parametrize("ot", [BF, F32])
def test_few_rows_of_many_experts(ctx, experts, rows, n, k, ot):
    """More than 64 experts and more tiles than workgroups, uneven experts, empty ones, rows of no
    expert: integers, so every sum is exact.  What lies behind a row of a and b is NaN."""
    import collective_overlap_amd as cce
    g = torch.Generator().manual_seed(experts)
    a = Padded(rows, k, BF, 8, value=torch.randint(-3, 4, (rows, k), generator=g).float())
    b = torch.full((experts, n, -(-k // 8) * 8 + 8), float("nan"), device=DEV, dtype=BF)[:, :, :k]
    b.copy_(torch.randint(-3, 4, (experts, n, k), generator=g).float())
    off = torch.randint(2, rows - 3, (experts + 1,), generator=g).sort().values
    off[5:9] = off[9]
    c = Padded(rows, n, ot, 8, value=torch.full((rows, n), 5.0))
    cce.cce_ragged_gemm(ctx, a.t, b, off.to(DEV), c.t)
    torch.cuda.synchronize()
    c.check_rest("c")
    want = torch.full((rows, n), 5.0, device=DEV)
    for e in range(experts):
        lo, hi = int(off[e]), int(off[e + 1])
        if hi > lo:
            want[lo:hi] = (a.t[lo:hi].double() @ b[e].double().t().contiguous()).float()
    assert torch.equal(c.t, want.to(ot))


def test_a_temporary_workspace_for_a_stream_given_as_a_handle(ctx):
    """A stream as torch gives it, its handle, and the default stream's (0), from another current one."""
    import collective_overlap_amd as cce
    x, d = randn((500, 2048), 1, 1, BF).to(DEV), randn((500, 2048), 2, 1, BF).to(DEV)
    w, dx = torch.ones(2048, device=DEV), torch.empty_like(x)
    want = torch.empty(2048, device=DEV)
    cce.cce_rmsnorm_backward(ctx, x, w, d, dx, want, EPS)
    side, other = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(other):
        got = [torch.zeros(2048, device=DEV) for _ in range(4)]
        torch.cuda.synchronize()
        for g, s in zip(got, (side, side.cuda_stream, 0, None)):
            cce.cce_rmsnorm_backward(ctx, x, w, d, dx, g, EPS, stream=s)
            torch.cuda.synchronize()
            assert torch.cuda.current_stream() == other
    assert all(torch.equal(g, want) for g in got)
