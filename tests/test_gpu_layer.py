"""GPU parity of the norm, the block quantisation and the 8-bit product against the float64
oracle, at the sizes where they can go wrong, and the operators in a row as a layer runs them.

Tolerances, from the formats: u = 2^-24 is half a step of fp32.  A row's sum of squares of
non-negative terms is off by at most (longest chain of additions) u relative; with 64 threads or
more to a row the chain is at most 8 ceil(cols / 512) + 16 (8 values per vector, the vectors of a
thread, the joins).  The root halves it; division, root, reciprocal and the two products add at
most 6 u.  A result of type t is then rounded once: half a step of t."""

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


def chain(cols):
    return 8 * -(-cols // 512) + 16


def norm_tol(cols):
    return (0.5 * chain(cols) + 6) * U


SHAPES = [(1, 8), (3, 1), (5, 7), (2, 64), (4, 127), (4, 128), (3, 129), (7, 1000), (2, 2048), (3, 4096),
          (2, 5005), (3, 8192), (5, 12288), (2, 16384), (2, 16392), (2, 40001), (300, 520), (4100, 96), (1501, 250), (33, 256)]


@pytest.mark.parametrize("rows,cols", SHAPES)
@pytest.mark.parametrize("xt,wt,ot", [(BF, BF, BF), (F32, F32, F32), (BF, F32, F32), (F32, BF, BF)])
@pytest.mark.parametrize("residual", [False, True])
def test_norm(ctx, rows, cols, xt, wt, ot, residual):
    import collective_overlap_amd as cce
    pad = 8 if cols % 3 else 0
    x = Padded(rows, cols, xt, pad, value=uneven(rows, cols, cols, xt))
    w = (1 + randn((cols,), 1, 0.3)).to(wt).to(DEV)
    out = Padded(rows, cols, ot, pad)
    res = res_out = None
    r = x.t.cpu()
    if residual:
        res = Padded(rows, cols, xt, 0, value=uneven(rows, cols, cols + 1, xt))
        res_out = Padded(rows, cols, xt, 16)
        r = (r.float() + res.t.cpu().float()).to(xt)
    cce.cce_rmsnorm(ctx, x.t, w, out.t, EPS, residual=res.t if res else None,
                    residual_out=res_out.t if res else None)
    torch.cuda.synchronize()
    out.check_rest("out")
    if residual:
        res_out.check_rest("residual_out")
        assert torch.equal(res_out.t.cpu(), r), "residual_out"
    ref = ol.rmsnorm(f64(r), f64(w), EPS)
    within(f64(out.t), ref, (norm_tol(cols) + HALF[ot]) * np.abs(ref) * 1.01 + 1e-37, "out")


@pytest.mark.parametrize("rows,cols", SHAPES)
@pytest.mark.parametrize("xt", [BF, F32])
@pytest.mark.parametrize("residual", [False, True])
def test_norm_to_e4m3(ctx, rows, cols, xt, residual):
    import collective_overlap_amd as cce
    x = Padded(rows, cols, xt, 0, value=uneven(rows, cols, cols, xt))
    w = (1 + randn((cols,), 1, 0.3)).to(xt).to(DEV)
    res = Padded(rows, cols, xt, 8, value=uneven(rows, cols, cols + 1, xt)) if residual else None
    out = Padded(rows, cols, E4, 8)
    scales = Padded(rows, -(-cols // 128), E8, 3, step=1)
    cce.cce_rmsnorm(ctx, x.t, w, out.t, EPS, residual=res.t if res else None, scales=scales.t)
    torch.cuda.synchronize()
    out.check_rest("out")
    scales.check_rest("scales")
    r = x.t.cpu() if res is None else (x.t.cpu().float() + res.t.cpu().float()).to(xt)
    y = ol.rmsnorm(f64(r), f64(w), EPS)
    tol = norm_tol(cols)
    s = f64(scales.t)
    top = np.stack([np.abs(y[:, j:j + 128]).max(1) for j in range(0, cols, 128)], 1)
    # the smallest power of two that fits, except where the fp32 norm may sit on the other side
    assert np.all(top <= 448 * s * (1 + 4 * tol)) and np.all((s == 2.0 ** -126) | (top >= 224 * s * (1 - 4 * tol)))
    wide = ol.expand(s, y.shape, 1)
    within(f64(out.t) * wide, y, (HALF[E4] + 2 * tol) * np.abs(y) + 2.0 ** -10 * wide, "e4m3 values")


def test_norm_of_zero_and_of_large_rows(ctx):
    """A row of zeros stays zero (scale 2^-126 in 8 bits); rows near the type's limits keep their
    squares finite up to 1e18; a NaN or an infinity stays in its row."""
    import collective_overlap_amd as cce
    cols = 640
    x = randn((6, cols), 3).to(DEV)
    x[0] = 0
    x[1] *= 1e17
    x[2] *= 1e-20
    x[3, 5] = float("nan")
    x[4, 9] = float("inf")
    w = torch.ones(cols, device=DEV)
    out = torch.empty((6, cols), device=DEV)
    q, s = torch.empty((6, cols), device=DEV, dtype=E4), torch.empty((6, 5), device=DEV, dtype=E8)
    cce.cce_rmsnorm(ctx, x, w, out, EPS)
    cce.cce_rmsnorm(ctx, x, w, q, EPS, scales=s)
    torch.cuda.synchronize()
    ref = ol.rmsnorm(f64(x[[0, 1, 2, 5]]), f64(w), EPS)
    within(f64(out[[0, 1, 2, 5]]), ref, (norm_tol(cols) + U) * np.abs(ref) * 1.01 + 1e-37, "finite rows")
    assert bool(torch.isnan(out[3]).all()) and bool(torch.isnan(out[4]).any())
    got, sc = f64(q), f64(s)
    assert np.all(got[0] == 0) and np.all(sc[0] == 2.0 ** -126)
    assert np.isnan(sc[3]).all() and np.isfinite(sc[[0, 1, 2, 5]]).all()


@pytest.mark.parametrize("rows,cols", SHAPES + [(2100, 264), (700, 4104)])
@pytest.mark.parametrize("xt,wt", [(BF, BF), (F32, F32), (BF, F32)])
@pytest.mark.parametrize("d_residual,want_dw", [(False, True), (True, True), (True, False)])
def test_norm_backward(ctx, rows, cols, xt, wt, d_residual, want_dw):
    """Against the formula in float64; the gradient's two terms are of similar size, so the
    tolerance is taken on the sum of their magnitudes."""
    import collective_overlap_amd as cce
    x = Padded(rows, cols, xt, 0, value=uneven(rows, cols, cols, xt))
    w = (1 + randn((cols,), 1, 0.3)).to(wt).to(DEV)
    dout = Padded(rows, cols, xt, 16, value=randn((rows, cols), 5, 0.7, xt))
    dres = Padded(rows, cols, xt, 8, value=randn((rows, cols), 6, 0.7, xt)) if d_residual else None
    dx = Padded(rows, cols, xt, 8)
    dw = torch.full((cols + 8,), 3.0, device=DEV)
    cce.cce_rmsnorm_backward(ctx, x.t, w, dout.t, dx.t, dw[:cols] if want_dw else None, EPS,
                             d_residual=dres.t if dres else None)
    torch.cuda.synchronize()
    dx.check_rest("dx")
    X, W, D = f64(x.t), f64(w), f64(dout.t)
    R = f64(dres.t) if dres else None
    ref, refw = ol.rmsnorm_backward(X, W, D, EPS, R)
    root = np.sqrt(np.mean(X * X, axis=1, keepdims=True) + EPS)
    n, g = X / root, np.abs(W * D)
    mag = (g + np.abs(n) * np.mean(g * np.abs(n), axis=1, keepdims=True)) / root + (0 if R is None else np.abs(R))
    # the mean of w dy n: a chain of additions and its products, on top of twice the norm's error
    within(f64(dx.t), ref, (chain(cols) + 3 * norm_tol(cols) / U + 8) * U * mag + HALF[xt] * np.abs(ref), "dx")
    if want_dw:
        # a column's sum over the rows: at most rows additions
        magw = np.sum(np.abs(D * n), axis=0)
        within(f64(dw[:cols]), refw, (rows + norm_tol(cols) / U + 4) * U * magw, "dweight")
    assert bool((dw[cols if want_dw else 0:] == 3.0).all())


def test_norm_backward_of_no_rows_gives_zero_weight_gradient(ctx):
    import collective_overlap_amd as cce
    e = torch.empty((0, 72), device=DEV)
    dw = torch.full((72,), 3.0, device=DEV)
    cce.cce_rmsnorm_backward(ctx, e, torch.ones(72, device=DEV), e, torch.empty_like(e), dw)
    torch.cuda.synchronize()
    assert bool((dw == 0).all())


def test_norm_gradient_is_that_of_differences(ctx):
    """dx and dweight against differences of the forward call itself, in fp32 with a step that
    balances truncation (h^2) and rounding (u / h): agreement to 2e-2 of the gradient's norm."""
    import collective_overlap_amd as cce
    rows, cols, h = 3, 24, 2.0 ** -8
    x, w, d = randn((rows, cols), 1).to(DEV), (1 + randn((cols,), 2, 0.3)).to(DEV), randn((rows, cols), 3).to(DEV)
    dx, dw = torch.empty_like(x), torch.empty_like(w)
    cce.cce_rmsnorm_backward(ctx, x, w, d, dx, dw)

    def loss(x, w):
        y = torch.empty_like(x)
        cce.cce_rmsnorm(ctx, x, w, y)
        return (y.double() * d.double()).sum().item()

    num = np.zeros((rows, cols))
    for i in range(rows):
        for j in range(cols):
            e = torch.zeros_like(x)
            e[i, j] = h
            num[i, j] = (loss(x + e, w) - loss(x - e, w)) / (2 * h)
    assert np.linalg.norm(num - f64(dx)) <= 2e-2 * np.linalg.norm(num)
    numw = np.zeros(cols)
    for j in range(cols):
        e = torch.zeros_like(w)
        e[j] = h
        numw[j] = (loss(x, w + e) - loss(x, w - e)) / (2 * h)
    assert np.linalg.norm(numw - f64(dw)) <= 2e-2 * np.linalg.norm(numw)


# ---- quantisation -------------------------------------------------------------------
@pytest.mark.parametrize("rows,cols", [(1, 1), (1, 128), (3, 130), (129, 100), (128, 128), (257, 1000), (40, 8200)])
@pytest.mark.parametrize("xt", [BF, F32])
@pytest.mark.parametrize("block_rows", [1, 128])
def test_quantize(ctx, rows, cols, xt, block_rows):
    """Dividing by a power of two is exact, so values and scales equal the oracle's."""
    import collective_overlap_amd as cce
    v = uneven(rows, cols, rows, xt)
    if rows > 2:
        v[1] = 0
    x = Padded(rows, cols, xt, 8, value=v)
    q = Padded(rows, cols, E4, 16)
    s = Padded(-(-rows // block_rows), -(-cols // 128), E8, 1, step=1)
    cce.cce_quantize_blocks(ctx, x.t, q.t, s.t, block_rows)
    torch.cuda.synchronize()
    q.check_rest("q")
    s.check_rest("scales")
    qr, sr = ol.quantize(f64(v), block_rows)
    np.testing.assert_array_equal(f64(s.t), sr)
    np.testing.assert_array_equal(f64(q.t), qr)


def test_quantize_special_values(ctx):
    import collective_overlap_amd as cce
    v = torch.zeros((12, 128))
    v[0, 3] = 448.0
    v[1, 3] = 448.0001
    v[2] = torch.linspace(-448, 448, 128)
    v[3, 0], v[3, 1] = 2.0 ** -126, 2.0 ** -149
    v[4, 0] = 3.4028e38
    v[5, 0], v[5, 1] = float("inf"), 1.0
    v[6, 7], v[6, 8] = float("nan"), 2.0
    v[7, 0], v[7, 1], v[7, 2] = 448.0, 2.0 ** -9, 2.0 ** -10
    v[8, 0] = -0.0
    v[9] = 1e-42
    v[10, 0], v[10, 1] = 1.75 * 2.0 ** 20, float(np.float32(1.75 * 2.0 ** 20) * (1 + 2.0 ** -22))
    v[11, 0] = 1.75 * 2.0 ** -118
    x = v.to(DEV)
    for br in (1, 128):
        rows = range(12) if br == 1 else [i for i in range(12) if i not in (5, 6)]
        xx = x[list(rows)].contiguous()
        q = torch.empty(xx.shape, device=DEV, dtype=E4)
        s = torch.empty((-(-len(xx) // br), 1), device=DEV, dtype=E8)
        cce.cce_quantize_blocks(ctx, xx, q, s, br)
        torch.cuda.synchronize()
        qr, sr = ol.quantize(f64(xx), br)
        np.testing.assert_array_equal(f64(s), sr)
        np.testing.assert_array_equal(f64(q), qr)


# ---- the 8-bit product ----------------------------------------------------------------
def operands(m, n, k, seed, pad=0):
    """Quantised operands as the oracle makes them, on the device."""
    (qa, sa), (qb, sb) = ol.quantize(f64(uneven(m, k, seed, F32)), 1), ol.quantize(f64(randn((n, k), seed + 1, 0.05)), 128)
    dev = [Padded(m, k, E4, pad, 16, torch.from_numpy(qa)), Padded(*sa.shape, E8, 1, 1, torch.from_numpy(sa).float()),
           Padded(n, k, E4, 2 * pad, 16, torch.from_numpy(qb)), Padded(*sb.shape, E8, 0, 1, torch.from_numpy(sb).float())]
    return (qa, sa, qb, sb), dev


PRODUCTS = [(1, 1, 16), (1, 64, 128), (1, 1000, 4096), (2, 130, 272), (4, 4096, 1040), (8, 520, 2048), (16, 256, 512),
            (17, 129, 144), (32, 1000, 528), (33, 200, 640), (64, 640, 256), (65, 72, 4224), (128, 128, 128),
            (129, 300, 384), (255, 257, 400), (333, 1000, 2064), (512, 384, 1024), (1030, 520, 272), (12, 4100, 400), (20, 2600, 1040), (9, 8200, 272),
            (25, 8210, 1040), (32, 2049, 144)]


@pytest.mark.parametrize("m,n,k", PRODUCTS)
@pytest.mark.parametrize("ot", [BF, F32])
@pytest.mark.parametrize("gelu", [False, True])
def test_block_scaled_gemm(ctx, m, n, k, ot, gelu):
    """fp32 results: the products are exact, so the error is that of at most K additions, K u
    times the sum of the magnitudes.  bf16 results: half a step, and what the 8-bit instruction
    leaves out of its sums of 64 products: less than 2^-16 of the largest for each of them, so at
    most 2^-10 of the largest and 2^-12 of a sum of magnitudes that is over four times that.  GELU
    has a slope of at most 1.13 and the error function 1.5e-7 (4e-7 |c| with its other roundings)."""
    import collective_overlap_amd as cce
    (qa, sa, qb, sb), (a, da, b, db) = operands(m, n, k, m + n, 16)
    c = Padded(m, n, ot, 8)
    cce.cce_block_scaled_gemm(ctx, a.t, da.t, b.t, db.t, c.t, gelu=gelu)
    torch.cuda.synchronize()
    c.check_rest("c")
    ref, mag = ol.block_scaled_product(qa, sa, qb, sb)
    tol = (k * U if ot == F32 else 2.0 ** -12) * mag
    if gelu:
        tol = 1.13 * tol + 4e-7 * np.abs(ref)
        ref = numerics.gelu(ref)
    within(f64(c.t), ref, tol + HALF[ot] * np.abs(ref), "c")
    if ot == F32 and not gelu:
        e = np.linalg.norm(f64(c.t) - ref) / np.linalg.norm(ref)
        assert e <= 2e-6, e


@pytest.mark.parametrize("m,n,k", [(1, 300, 4096), (16, 100, 640), (100, 200, 1024), (300, 520, 528), (1500, 2100, 400)])
@pytest.mark.parametrize("ot", [BF, F32])
def test_block_scaled_gemm_of_small_integers_is_exact(ctx, m, n, k, ot):
    """Integers in [-4, 4] and scales of 1/4 to 4: every sum is a multiple of 1/16 below 2^24 / 16,
    exact in fp32 whatever the order, then rounded once."""
    import collective_overlap_amd as cce
    rng = np.random.default_rng(m)
    qa, qb = rng.integers(-4, 5, (m, k)).astype(float), rng.integers(-4, 5, (n, k)).astype(float)
    kb = -(-k // 128)
    sa, sb = 2.0 ** rng.integers(-2, 3, (m, kb)), 2.0 ** rng.integers(-2, 3, (-(-n // 128), kb))
    a, b = (torch.from_numpy(t).to(DEV).to(E4) for t in (qa, qb))
    da, db = (torch.from_numpy(t).float().to(DEV).to(E8) for t in (sa, sb))
    c = torch.empty((m, -(-n // 8) * 8), device=DEV, dtype=ot)[:, :n]
    cce.cce_block_scaled_gemm(ctx, a, da, b, db, c)
    torch.cuda.synchronize()
    ref, _ = ol.block_scaled_product(qa, sa, qb, sb)
    want = torch.from_numpy(ref).float().to(ot)
    assert torch.equal(c.cpu(), want), f"{int((c.cpu() != want).sum())} of {want.numel()} differ"


@pytest.mark.parametrize("m", [1, 20, 300])
@pytest.mark.parametrize("ot", [BF, F32])
def test_block_scaled_gemm_edges(ctx, m, ot):
    """A contraction of length 0 gives zeros; a block whose scale is NaN gives NaN in its row (a)
    or its 128 columns (b) and nowhere else."""
    import collective_overlap_amd as cce
    n, k = 200, 384
    z = torch.empty((m, n), device=DEV, dtype=ot).fill_(7)
    cce.cce_block_scaled_gemm(ctx, torch.empty((m, 0), device=DEV, dtype=E4), torch.empty((m, 0), device=DEV, dtype=E8),
                              torch.empty((n, 0), device=DEV, dtype=E4), torch.empty((2, 0), device=DEV, dtype=E8), z, gelu=True)
    _, (a, da, b, db) = operands(m, n, k, 3)
    for where in ("a", "b"):
        s = (da if where == "a" else db).t
        keep = s.clone()
        s[0, 1] = float("nan")
        c = torch.empty((m, n), device=DEV, dtype=ot)
        cce.cce_block_scaled_gemm(ctx, a.t, da.t, b.t, db.t, c)
        torch.cuda.synchronize()
        nan = torch.isnan(c)
        if where == "a":
            assert bool(nan[0].all()) and not bool(nan[1:].any())
        else:
            assert bool(nan[:, :128].all()) and not bool(nan[:, 128:].any())
        s.copy_(keep)
    assert bool((z == 0).all())


@pytest.mark.parametrize("m,n,k,ot", [
    (40, 200, 16400, F32),        # few 64 x 64 tiles: waves along the contraction
    (700, 500, 16016, F32),       # 64 x 64 tiles, scales in two panels
    (2100, 2060, 31888, F32),     # 128 x 128 tiles, three panels
    (1500, 1030, 16016, BF),      # 128 x 128 tiles of the 8-bit instruction
    (4096, 4112, 16016, BF),      # 256 x 256 tiles
    (4090, 4096, 272, BF),
    (8, 4104, 16400, BF),
])
@pytest.mark.parametrize("scale_ld", [0, 3])
def test_every_product_kernel_is_exact_on_small_integers(ctx, m, n, k, ot, scale_ld):
    """Integers in [-2, 2] and scales of 1/2 to 2: sums of multiples of 1/4 below 2^22 are exact in
    fp32 whatever the order, and in the fp64 product on the device; a contraction longer than the
    124 blocks whose scales are held at a time, scale rows on words and off them."""
    import collective_overlap_amd as cce
    g = torch.Generator(device=DEV).manual_seed(m)
    kb, nb = -(-k // 128), -(-n // 128)
    a = torch.randint(-2, 3, (m, k), generator=g, device=DEV).float().to(E4)
    b = torch.randint(-2, 3, (n, k), generator=g, device=DEV).float().to(E4)
    def scales(rows):
        s = torch.exp2(torch.randint(-1, 2, (rows, kb), generator=g, device=DEV).float())
        t = torch.empty((rows, -(-kb // 4) * 4 + scale_ld), device=DEV, dtype=E8)[:, :kb]
        t.copy_(s.to(E8))
        return t
    sa, sb = scales(m), scales(nb)
    c = torch.empty((m, -(-n // 8) * 8), device=DEV, dtype=ot)[:, :n]
    cce.cce_block_scaled_gemm(ctx, a, sa, b, sb, c)
    wa = a.float().double() * sa.float().double().repeat_interleave(128, 1)[:, :k]
    wb = b.float().double() * sb.float().double().repeat_interleave(128, 1)[:, :k].repeat_interleave(128, 0)[:n]
    want = (wa @ wb.t().contiguous()).float().to(ot)
    assert torch.equal(c, want), f"{int((c != want).sum())} of {want.numel()} differ"


def test_more_rows_than_one_launch_takes(ctx):
    """134 million rows of 8: more workgroups than a launch may have."""
    import collective_overlap_amd as cce
    rows = (1 << 27) + 70_003
    x = torch.zeros((rows, 8), device=DEV, dtype=BF)
    pick = torch.tensor([0, 1, (1 << 24) - 1, 1 << 24, (1 << 27) - 1, 1 << 27, rows - 2, rows - 1], device=DEV)
    x[pick] = randn((len(pick), 8), 1, 1, BF).to(DEV)
    w = torch.ones(8, device=DEV, dtype=BF)
    out, q, s = torch.empty_like(x), torch.empty((rows, 8), device=DEV, dtype=E4), torch.empty((rows, 1), device=DEV, dtype=E8)
    cce.cce_rmsnorm(ctx, x, w, out, EPS)
    cce.cce_quantize_blocks(ctx, x, q, s, 1)
    torch.cuda.synchronize()
    X = f64(x[pick])
    ref = ol.rmsnorm(X, np.ones(8), EPS)
    within(f64(out[pick]), ref, (norm_tol(8) + HALF[BF]) * np.abs(ref) * 1.01, "out")
    qr, sr = ol.quantize(X, 1)
    np.testing.assert_array_equal(f64(q[pick]), qr)
    np.testing.assert_array_equal(f64(s[pick]), sr)
    assert int(torch.count_nonzero(out)) == int(torch.count_nonzero(x))
    del out
    dx, dw = torch.empty_like(x), torch.empty(8, device=DEV)
    cce.cce_rmsnorm_backward(ctx, x, w, x, dx, dw, EPS)
    torch.cuda.synchronize()
    rdx, rdw = ol.rmsnorm_backward(X, np.ones(8), X, EPS)
    n = X / np.sqrt(np.mean(X * X, axis=1, keepdims=True) + EPS)
    mag = (np.abs(X) + np.abs(n) * np.mean(np.abs(X * n), axis=1, keepdims=True)) * np.abs(n / X)
    within(f64(dx[pick]), rdx, (chain(8) + 3 * norm_tol(8) / U + 8) * U * mag + HALF[BF] * np.abs(rdx), "dx")
    # (adding a row of zeros is exact: the sums are those of the picked rows)
    within(f64(dw), rdw, (len(pick) + norm_tol(8) / U + 4) * U * np.abs(X * n).sum(0), "dweight")


def test_tensors_beyond_four_gibibytes(ctx):
    """Rows past 2^32 bytes of the norm, its backward pass, the quantisation and the product."""
    import collective_overlap_amd as cce
    rows, cols, last = 1_100_000, 2048, 50
    x = torch.zeros((rows, cols), device=DEV, dtype=BF)
    x[-last:] = randn((last, cols), 1, 1, BF).to(DEV)
    w = (1 + randn((cols,), 2, 0.2)).to(BF).to(DEV)
    q, s = torch.empty((rows, cols), device=DEV, dtype=E4), torch.empty((rows, cols // 128), device=DEV, dtype=E8)
    out, dx, dw = torch.empty_like(x), torch.empty_like(x), torch.empty(cols, device=DEV)
    cce.cce_rmsnorm(ctx, x, w, out, EPS)
    cce.cce_rmsnorm_backward(ctx, x, w, x, dx, dw, EPS)
    cce.cce_quantize_blocks(ctx, x, q, s, 1)
    b, sb = torch.empty((64, cols), device=DEV, dtype=E4), torch.empty((1, cols // 128), device=DEV, dtype=E8)
    cce.cce_quantize_blocks(ctx, randn((64, cols), 3, 0.05).to(DEV), b, sb, 128)
    torch.cuda.synchronize()
    X, W = f64(x[-last:]), f64(w)
    ref = ol.rmsnorm(X, W, EPS)
    within(f64(out[-last:]), ref, (norm_tol(cols) + HALF[BF]) * np.abs(ref) * 1.01, "out")
    rdx, rdw = ol.rmsnorm_backward(X, W, X, EPS)
    n = X / np.sqrt(np.mean(X * X, axis=1, keepdims=True) + EPS)
    within(f64(dw), rdw, (rows + norm_tol(cols) / U) * U * np.abs(X * n).sum(0), "dweight")
    assert np.linalg.norm(f64(dx[-last:]) - rdx) <= 1e-2 * np.linalg.norm(rdx)
    qr, sr = ol.quantize(X, 1)
    np.testing.assert_array_equal(f64(q[-last:]), qr)
    np.testing.assert_array_equal(f64(s[-last:]), sr)
    del out, dx
    qq = torch.zeros((2 * rows, cols), device=DEV, dtype=E4)
    ss = torch.ones((2 * rows, cols // 128), device=DEV).to(E8)
    assert qq.numel() > 1 << 32
    qq[-last:], ss[-last:] = q[-last:], s[-last:]
    for ot in (BF, F32):
        c = torch.empty((2 * rows, 64), device=DEV, dtype=ot)
        cce.cce_block_scaled_gemm(ctx, qq, ss, b, sb, c)
        torch.cuda.synchronize()
        ref, mag = ol.block_scaled_product(qr, sr, f64(b), f64(sb))
        within(f64(c[-last:]), ref, (cols * U if ot == F32 else 2.0 ** -12) * mag + HALF[ot] * np.abs(ref), "c")
        assert not bool(c[:-last].any())


# ---- together -----------------------------------------------------------------------------
def _layer(cce, ctx, t, stream=None):
    """Norm with the residual's addition and an 8-bit output, product with GELU, quantisation,
    second product, backward of the norm: as a layer runs them."""
    cce.cce_rmsnorm(ctx, t["x"], t["w"], t["q"], EPS, residual=t["res"], residual_out=t["r"], scales=t["s"], stream=stream)
    cce.cce_block_scaled_gemm(ctx, t["q"], t["s"], t["b1"], t["sb1"], t["h"], gelu=True, stream=stream)
    cce.cce_quantize_blocks(ctx, t["h"], t["qh"], t["sh"], 1, stream=stream)
    cce.cce_block_scaled_gemm(ctx, t["qh"], t["sh"], t["b2"], t["sb2"], t["y"], stream=stream)
    cce.cce_rmsnorm_backward(ctx, t["r"], t["w"], t["y"], t["dx"], t["dw"], EPS, d_residual=t["y"], workspace=t["ws"], stream=stream)
    cce.cce_ragged_gemm(ctx, t["h"], t["we"], t["off"], t["c"], stream=stream)
    cce.cce_ragged_gemm_dgrad(ctx, t["c"], t["we"], t["off"], t["dh"], stream=stream)
    cce.cce_ragged_gemm_wgrad(ctx, t["c"], t["h"], t["off"], t["dwe"], stream=stream)


def _tensors(rows, hidden, ffn, seed):
    import collective_overlap_amd as cce
    e = torch.empty
    ctx = cce.Context(0)
    t = dict(x=randn((rows, hidden), seed, 1, BF).to(DEV), res=randn((rows, hidden), seed + 1, 1, BF).to(DEV),
             w=(1 + randn((hidden,), seed + 2, 0.2)).to(BF).to(DEV), r=e((rows, hidden), device=DEV, dtype=BF),
             q=e((rows, hidden), device=DEV, dtype=E4), s=e((rows, -(-hidden // 128)), device=DEV, dtype=E8),
             b1=e((ffn, hidden), device=DEV, dtype=E4), sb1=e((-(-ffn // 128), -(-hidden // 128)), device=DEV, dtype=E8),
             h=e((rows, ffn), device=DEV, dtype=BF), qh=e((rows, ffn), device=DEV, dtype=E4),
             sh=e((rows, -(-ffn // 128)), device=DEV, dtype=E8),
             b2=e((hidden, ffn), device=DEV, dtype=E4), sb2=e((-(-hidden // 128), -(-ffn // 128)), device=DEV, dtype=E8),
             y=e((rows, hidden), device=DEV, dtype=BF), dx=e((rows, hidden), device=DEV, dtype=BF),
             dw=e((hidden,), device=DEV),
             we=randn((3, hidden, ffn), seed + 3, 0.05, BF).to(DEV),
             off=torch.tensor([0, rows // 3, rows // 3, rows], device=DEV),
             c=torch.zeros((rows, hidden), device=DEV, dtype=BF), dh=torch.zeros((rows, ffn), device=DEV, dtype=BF),
             dwe=e((3, hidden, ffn), device=DEV),
             ws=e(cce.cce_rmsnorm_backward_workspace((rows, hidden)), device=DEV, dtype=torch.uint8))
    for q, s, shape in (("b1", "sb1", (ffn, hidden)), ("b2", "sb2", (hidden, ffn))):
        cce.cce_quantize_blocks(ctx, randn(shape, seed + 4, 0.05).to(DEV), t[q], t[s], 128)
    torch.cuda.synchronize()
    ctx.close()
    return t


OUTS = ("r", "q", "s", "h", "qh", "sh", "y", "dx", "dw", "c", "dh", "dwe")


def _bits(t):
    return [t[k].clone().view(torch.uint8) for k in OUTS]


@pytest.mark.parametrize("rows,hidden,ffn", [(1, 256, 512), (70, 384, 640), (515, 512, 1024)])
def test_layer_against_the_oracle(ctx, rows, hidden, ffn):
    """The chain against float64 on the values each step really had, each step's own tolerance."""
    import collective_overlap_amd as cce
    t = _tensors(rows, hidden, ffn, 11)
    _layer(cce, ctx, t)
    torch.cuda.synchronize()
    h, mag = ol.block_scaled_product(f64(t["q"]), f64(t["s"]), f64(t["b1"]), f64(t["sb1"]))
    ref = numerics.gelu(h)
    within(f64(t["h"]), ref, 1.13 * 2.0 ** -12 * mag + 4e-7 * np.abs(h) + HALF[BF] * np.abs(ref), "first product")
    qh, sh = ol.quantize(f64(t["h"]), 1)
    np.testing.assert_array_equal(f64(t["qh"]), qh)
    y, mag = ol.block_scaled_product(qh, sh, f64(t["b2"]), f64(t["sb2"]))
    within(f64(t["y"]), y, 2.0 ** -12 * mag + HALF[BF] * np.abs(y), "second product")
    c = ol.ragged(f64(t["h"]), f64(t["we"]), t["off"].tolist(), np.zeros((rows, hidden)))
    cm = ol.ragged(np.abs(f64(t["h"])), np.abs(f64(t["we"])), t["off"].tolist(), np.zeros((rows, hidden)))
    within(f64(t["c"]), c, ffn * U * cm + HALF[BF] * np.abs(c), "experts")


def test_layer_on_another_stream_and_twice_at_once(ctx):
    """Two layers on two streams with their own tensors, after their inputs are ready: the bits of
    each are those of a run alone."""
    import collective_overlap_amd as cce
    ts = [_tensors(200 + 60 * i, 384, 512, 20 + i) for i in range(2)]
    want = []
    for t in ts:
        _layer(cce, ctx, t)
        torch.cuda.synchronize()
        want.append(_bits(t))
        for k in OUTS:
            t[k].view(torch.uint8).zero_()
    ctxs = [cce.Context(0), cce.Context(0)]
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    for _ in range(3):
        for t, s, c in zip(ts, streams, ctxs):
            _layer(cce, c, t, stream=s)
    torch.cuda.synchronize()
    for t, w in zip(ts, want):
        assert all(torch.equal(a, b) for a, b in zip(_bits(t), w))
    for c in ctxs:
        c.close()


def test_layer_captured_and_replayed(ctx):
    """Two graphs, replayed in turn with eager work between, new inputs before each replay."""
    import collective_overlap_amd as cce
    ts = [_tensors(130, 384, 512, 30), _tensors(3, 256, 640, 31)]
    graphs = []
    for t in ts:
        _layer(cce, ctx, t)
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            _layer(cce, ctx, t)
        graphs.append(g)
    for step in range(3):
        for t, g in zip(ts, graphs):
            t["x"].copy_(randn(t["x"].shape, 50 + step, 1, BF).to(DEV))
            rows = t["x"].shape[0]
            t["off"].copy_(torch.tensor([0, (step * rows) // 3, rows // 2 + step // 2, rows]))
            _layer(cce, ctx, t)
            torch.cuda.synchronize()
            want = _bits(t)
            for k in OUTS:
                if k not in ("c", "dh"):
                    t[k].view(torch.uint8).zero_()
            g.replay()
            torch.cuda.synchronize()
            assert all(torch.equal(a, b) for a, b in zip(_bits(t), want)), f"replay {step}"
            (torch.ones(1000, device=DEV) * 2).sum().item()


def test_profile_names_the_new_launches(ctx):
    import collective_overlap_amd as cce
    t = _tensors(8, 256, 512, 40)
    ctx.set_profiling(True)
    _layer(cce, ctx, t)
    torch.cuda.synchronize()
    kinds = [r["kind"] for r in ctx.read_profile()]
    ctx.set_profiling(False)
    assert kinds == ["norm", "gemm", "quantize", "gemm", "norm", "gemm", "gemm", "gemm"]
