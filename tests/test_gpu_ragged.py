"""GPU parity of the products grouped by expert (forward and both gradients) against the float64
oracle: experts without rows, rows of no expert, one row, one expert with all, odd extents and
wide rows.  bf16 products are exact in fp32, so the error is that of the additions: at most
(contraction length) half steps of fp32 times the sum of the magnitudes, then one rounding."""

import numpy as np
import pytest
import torch

from layer_util import BF, DEV, F32, HALF, Padded, f64, randn, within
from oracle import layer as ol

pytestmark = pytest.mark.gpu
U = 2.0 ** -24


@pytest.fixture(scope="module")
def ctx():
    import collective_overlap_amd as cce
    c = cce.Context(0)
    yield c
    torch.cuda.synchronize()
    c.close()


CASES = {   # rows, N, K, offsets
    "one row": (1, 8, 8, [0, 1]),
    "one row of many experts": (1, 72, 40, [0, 0, 0, 1, 1]),
    "no rows": (0, 24, 16, [0, 0, 0]),
    "none owned": (9, 24, 16, [4, 4, 4]),
    "rows before, between and behind": (100, 40, 72, [3, 20, 20, 77]),
    "decode": (16, 520, 264, [0, 1, 1, 3, 3, 3, 4, 12, 12, 15, 16]),
    "even": (512, 256, 128, [0, 128, 256, 384, 512]),
    "all to one": (300, 136, 200, [0, 0, 300, 300]),
    "odd": (733, 331, 77, [0, 65, 129, 130, 600, 733]),
    "wide": (200, 640, 1032, [0, 100, 200]),
    "large": (2500, 600, 528, [0, 1100, 1101, 1400, 1400, 2500]),
    "many experts": (700, 64, 64, list(range(0, 701, 5))),
}


def build(case, pad):
    rows, n, k, off = CASES[case]
    e = len(off) - 1
    a = Padded(rows, k, BF, pad, value=randn((rows, k), 1, 1, BF))
    c = Padded(rows, n, BF, 0, value=randn((rows, n), 2, 1, BF))
    ld = -(-k // 8) * 8 + pad
    w = torch.full((e, n + 1, ld), float("nan"), dtype=BF, device=DEV)
    b = w[:, :n, :k]
    b.copy_(randn((e, n, k), 3, 0.2, BF).to(DEV))
    return rows, n, k, off, a, b, c, torch.tensor(off, device=DEV)


@pytest.mark.parametrize("case", list(CASES))
@pytest.mark.parametrize("ot", [BF, F32])
@pytest.mark.parametrize("pad", [0, 8])
def test_forward(ctx, case, ot, pad):
    import collective_overlap_amd as cce
    rows, n, k, off, a, b, _, o = build(case, pad)
    out = Padded(rows, n, ot, pad, value=randn((rows, n), 4))
    before = f64(out.t)
    print(f"[gpu] ragged forward {case}", flush=True)
    cce.cce_ragged_gemm(ctx, a.t, b, o, out.t)
    torch.cuda.synchronize()
    out.check_rest("c")
    ref = ol.ragged(f64(a.t), f64(b), off, before)
    mag = ol.ragged(np.abs(f64(a.t)), np.abs(f64(b)), off, np.zeros((rows, n)))
    within(f64(out.t), ref, k * U * mag + np.where(mag > 0, HALF[ot], 0) * np.abs(ref), "c")


@pytest.mark.parametrize("case", list(CASES))
@pytest.mark.parametrize("ot", [BF, F32])
@pytest.mark.parametrize("pad", [0, 8])
def test_dgrad(ctx, case, ot, pad):
    import collective_overlap_amd as cce
    rows, n, k, off, _, b, c, o = build(case, pad)
    out = Padded(rows, k, ot, pad, value=randn((rows, k), 4))
    before = f64(out.t)
    print(f"[gpu] ragged dgrad {case}", flush=True)
    cce.cce_ragged_gemm_dgrad(ctx, c.t, b, o, out.t)
    torch.cuda.synchronize()
    out.check_rest("da")
    ref = ol.ragged_dgrad(f64(c.t), f64(b), off, before)
    mag = ol.ragged_dgrad(np.abs(f64(c.t)), np.abs(f64(b)), off, np.zeros((rows, k)))
    within(f64(out.t), ref, n * U * mag + np.where(mag > 0, HALF[ot], 0) * np.abs(ref), "da")


@pytest.mark.parametrize("case", list(CASES))
@pytest.mark.parametrize("ot", [BF, F32])
@pytest.mark.parametrize("pad", [0, 8])
def test_wgrad(ctx, case, ot, pad):
    import collective_overlap_amd as cce
    rows, n, k, off, a, _, c, o = build(case, pad)
    ld = -(-k // 8) * 8 + pad
    whole = torch.full((len(off) - 1, n + 1, ld), 9.0, dtype=ot, device=DEV)
    print(f"[gpu] ragged wgrad {case}", flush=True)
    cce.cce_ragged_gemm_wgrad(ctx, c.t, a.t, o, whole[:, :n, :k])
    torch.cuda.synchronize()
    assert bool((whole[:, n:] == 9).all()) and bool((whole[:, :, k:] == 9).all())
    ref = ol.ragged_wgrad(f64(c.t), f64(a.t), off)
    mag = ol.ragged_wgrad(np.abs(f64(c.t)), np.abs(f64(a.t)), off)
    within(f64(whole[:, :n, :k]), ref, max(rows, 1) * U * mag + HALF[ot] * np.abs(ref), "db")


@pytest.mark.parametrize("rows,n,k,experts", [(1030, 520, 264, 3), (40, 264, 520, 7), (3000, 1032, 640, 4)])
def test_small_integers_are_exact(ctx, rows, n, k, experts):
    """Integers in [-3, 3]: every sum is exact in fp32, so all three results equal the oracle's."""
    import collective_overlap_amd as cce
    rng = np.random.default_rng(rows)
    a, b, c = (rng.integers(-3, 4, s).astype(float) for s in ((rows, k), (experts, n, k), (rows, n)))
    off = [0] + sorted(rng.integers(0, rows + 1, experts - 1).tolist()) + [rows]
    ta, tb, tc = (torch.from_numpy(t).to(BF).to(DEV) for t in (a, b, c))
    o = torch.tensor(off, device=DEV)
    y, da, db = (torch.empty(s, device=DEV) for s in ((rows, n), (rows, k), (experts, n, k)))
    cce.cce_ragged_gemm(ctx, ta, tb, o, y)
    cce.cce_ragged_gemm_dgrad(ctx, tc, tb, o, da)
    cce.cce_ragged_gemm_wgrad(ctx, tc, ta, o, db)
    torch.cuda.synchronize()
    assert np.array_equal(f64(y), ol.ragged(a, b, off, np.zeros((rows, n))))
    assert np.array_equal(f64(da), ol.ragged_dgrad(c, b, off, np.zeros((rows, k))))
    assert np.array_equal(f64(db), ol.ragged_wgrad(c, a, off))


def test_a_nan_stays_with_its_row_and_expert(ctx):
    """A NaN or an infinity in rows of one expert (or of none) reaches no other expert's results."""
    import collective_overlap_amd as cce
    rows, n, k, off = 50, 72, 40, [2, 20, 20, 33]
    a, b, c = randn((rows, k), 1, 1, BF).to(DEV), randn((3, n, k), 2, 1, BF).to(DEV), randn((rows, n), 3, 1, BF).to(DEV)
    a[0], a[40], a[25] = float("nan"), float("inf"), float("nan")
    c[1], c[49], c[25] = float("nan"), float("inf"), float("nan")
    o = torch.tensor(off, device=DEV)
    y, da, db = torch.zeros((rows, n), device=DEV), torch.zeros((rows, k), device=DEV), torch.empty((3, n, k), device=DEV)
    cce.cce_ragged_gemm(ctx, a, b, o, y)
    cce.cce_ragged_gemm_dgrad(ctx, c, b, o, da)
    cce.cce_ragged_gemm_wgrad(ctx, c, a, o, db)
    torch.cuda.synchronize()
    for t in (y, da):
        bad = torch.isnan(t).any(1).cpu()
        assert bool(bad[25]) and int(bad.sum()) == 1
    assert not bool(torch.isnan(db[:2]).any()) and bool(torch.isnan(db[2]).any())


def test_offsets_outside_the_rows_act_as_the_nearest(ctx):
    import collective_overlap_amd as cce
    rows, n, k = 40, 24, 32
    a, b = randn((rows, k), 1, 1, BF).to(DEV), randn((2, n, k), 2, 1, BF).to(DEV)
    got, want = torch.zeros((rows, n), device=DEV), torch.zeros((rows, n), device=DEV)
    cce.cce_ragged_gemm(ctx, a, b, torch.tensor([-5, 17, 1 << 40], device=DEV), got)
    cce.cce_ragged_gemm(ctx, a, b, torch.tensor([0, 17, 40], device=DEV), want)
    torch.cuda.synchronize()
    assert torch.equal(got, want)


def test_decreasing_offsets_act_as_the_ones_before(ctx):
    """No row has two experts: the same bits as the offsets raised to their running maximum."""
    import collective_overlap_amd as cce
    rows, n, k = 300, 72, 80
    a, b, c = randn((rows, k), 1, 1, BF).to(DEV), randn((4, n, k), 2, 1, BF).to(DEV), randn((rows, n), 3, 1, BF).to(DEV)
    got = []
    for off in ([10, 200, 90, 250, 240], [10, 200, 200, 250, 250]):
        o = torch.tensor(off, device=DEV)
        y, da, db = torch.zeros((rows, n), device=DEV), torch.zeros((rows, k), device=DEV), torch.empty_like(b)
        cce.cce_ragged_gemm(ctx, a, b, o, y)
        cce.cce_ragged_gemm_dgrad(ctx, c, b, o, da)
        cce.cce_ragged_gemm_wgrad(ctx, c, a, o, db)
        torch.cuda.synchronize()
        got.append((y, da, db))
    for x, y in zip(*got):
        assert torch.equal(x, y)


def test_shared_weights_as_a_broadcast_input(ctx):
    """One matrix for all experts (stride 0 between them) in the forward form and in dgrad."""
    import collective_overlap_amd as cce
    rows, n, k = 60, 40, 48
    a, w = randn((rows, k), 1, 1, BF).to(DEV), randn((1, n, k), 2, 1, BF).to(DEV)
    o = torch.tensor([0, 10, 60], device=DEV)
    y1, y2 = torch.empty((rows, n), device=DEV), torch.empty((rows, n), device=DEV)
    cce.cce_ragged_gemm(ctx, a, w.expand(2, n, k), o, y1)
    cce.cce_ragged_gemm(ctx, a, w.repeat(2, 1, 1), o, y2)
    torch.cuda.synchronize()
    assert torch.equal(y1, y2)


@pytest.mark.parametrize("rows,n,k,experts,top", [
    (6200, 2832, 2840, 8, 3),      # 256 x 256 tiles
    (6200, 2833, 2843, 8, 3),      # 256 x 256 tiles, odd extents
    (9000, 2816, 4096, 20, 3),     # 256 x 256 tiles, most experts part of a tile
    (4096, 1024, 4096, 4, 3),      # 128 x 128 tiles, whole
    (5000, 1100, 4104, 4, 3),      # 128 x 128 tiles, ragged
    (3000, 700, 520, 2, 3),
    (6000, 64, 72, 1, 2),          # 64 x 64, four groups, a long sum over the rows
    (500, 1000, 8200, 5, 2),
])
def test_every_tile_size_is_exact_on_small_integers(ctx, rows, n, k, experts, top):
    """Integers: every sum is below 2^24, so exact in fp32 and in the fp64 product on the device."""
    import collective_overlap_amd as cce
    g = torch.Generator(device=DEV).manual_seed(rows)
    def empty(*shape, dtype=F32):       # rows on multiples of 8
        return torch.empty((*shape[:-1], -(-shape[-1] // 8) * 8), device=DEV, dtype=dtype)[..., :shape[-1]]
    def ints(*shape):
        return empty(*shape, dtype=BF).copy_(torch.randint(-top, top + 1, shape, generator=g, device=DEV))
    a, b, c = ints(rows, k), ints(experts, n, k), ints(rows, n)
    cut = sorted(torch.randint(0, rows - 5, (experts - 1,), generator=g, device=DEV).tolist())
    off = [3] + [max(3, x) for x in cut] + [rows - 2]
    o = torch.tensor(off, device=DEV)
    y, da, db = empty(rows, n).fill_(5.0), empty(rows, k).fill_(5.0), empty(experts, n, k)
    cce.cce_ragged_gemm(ctx, a, b, o, y)
    cce.cce_ragged_gemm_dgrad(ctx, c, b, o, da)
    cce.cce_ragged_gemm_wgrad(ctx, c, a, o, db)
    ry, rda = torch.full((rows, n), 5.0, device=DEV), torch.full((rows, k), 5.0, device=DEV)
    for e, (lo, hi) in enumerate(zip(off[:-1], off[1:])):
        w = b[e].double()
        ry[lo:hi] = (a[lo:hi].double() @ w.t().contiguous()).float()
        rda[lo:hi] = (c[lo:hi].double() @ w).float()
        assert torch.equal(db[e], (c[lo:hi].double().t().contiguous() @ a[lo:hi].double()).float()), f"db {e}"
    assert torch.equal(y, ry) and torch.equal(da, rda)


@pytest.mark.parametrize("counts", [[256] * 22, [256] * 32 + [0], [1] * 3 + [5800], [256] * 33, [300] * 17, [257] * 19,
                                    [2048, 100, 2048, 1500]])
def test_large_tiles_of_many_counts(ctx, counts):
    """Counts of tiles (12 to a row of them) on both sides of a round of the compute units, one
    round, two; experts of exactly a tile's rows, of one more, of one."""
    import collective_overlap_amd as cce
    rows, n, k, e = sum(counts), 3000, 136, len(counts)
    g = torch.Generator(device=DEV).manual_seed(e)
    a = torch.randint(-3, 4, (rows, k), generator=g, device=DEV).to(BF)
    b = torch.randint(-3, 4, (e, n, k), generator=g, device=DEV).to(BF)
    c = torch.randint(-3, 4, (rows, k), generator=g, device=DEV).to(BF)
    off = torch.tensor([0] + counts, device=DEV).cumsum(0)
    y, da = torch.full((rows, n), 5.0, device=DEV), torch.full((rows, n), 5.0, device=DEV)
    cce.cce_ragged_gemm(ctx, a, b, off, y)
    bt = b.transpose(1, 2).contiguous()                    # [e, k, n]: the gradient has n columns
    cce.cce_ragged_gemm_dgrad(ctx, c, bt, off, da)
    for i, (lo, hi) in enumerate(zip(off[:-1].tolist(), off[1:].tolist())):
        assert torch.equal(y[lo:hi], (a[lo:hi].double() @ bt[i].double()).float()), f"expert {i}"
        assert torch.equal(da[lo:hi], (c[lo:hi].double() @ bt[i].double()).float()), f"gradient, expert {i}"


def test_rows_beyond_four_gibibytes(ctx):
    """Operands of over 2^32 bytes: the last expert's rows are addressed past 32 bits."""
    import collective_overlap_amd as cce
    rows, n, k = 1_100_000, 64, 2048
    a = torch.zeros((rows, k), device=DEV, dtype=BF)
    assert a.numel() * 2 > 1 << 32
    a[:100], a[-100:] = randn((100, k), 1, 1, BF).to(DEV), randn((100, k), 2, 1, BF).to(DEV)
    b = randn((2, n, k), 3, 0.2, BF).to(DEV)
    o = torch.tensor([0, 70, rows], device=DEV)
    y, c = torch.empty((rows, n), device=DEV), torch.zeros((rows, n), device=DEV, dtype=BF)
    c[-50:] = randn((50, n), 4, 1, BF).to(DEV)
    da, db = torch.empty_like(a), torch.empty((2, n, k), device=DEV)
    cce.cce_ragged_gemm(ctx, a, b, o, y)
    cce.cce_ragged_gemm_dgrad(ctx, c, b, o, da)
    cce.cce_ragged_gemm_wgrad(ctx, c, a, o, db)
    torch.cuda.synchronize()
    A, B, C = f64(a[-100:]), f64(b[1]), f64(c[-50:])
    within(f64(y[-100:]), A @ B.T, k * U * (np.abs(A) @ np.abs(B).T), "c")
    within(f64(da[-50:]), C @ B, n * U * (np.abs(C) @ np.abs(B)) + HALF[BF] * np.abs(C @ B), "da")
    within(f64(db[1]), C.T @ A[-50:], 50 * U * (np.abs(C).T @ np.abs(A[-50:])), "db")
    assert not bool(y[200:-200].any()) and not bool(da[200:-200].any()) and not bool(db[0].any())
