"""CPU tests of what the norm, quantisation, 8-bit product and ragged product entry points
refuse: in the binding (dtypes, shapes, host tensors) and at the C ABI (extents, alignment,
overlaps, NULLs, workspace).  No GPU is needed: every call here is refused, or has nothing
to do, before the context is used."""

import ctypes

import pytest
import torch

import collective_overlap_amd as cce
from collective_overlap_amd import _lib
from collective_overlap_amd._lib import cce_mat

BF, F32, E4, E8 = torch.bfloat16, torch.float32, torch.float8_e4m3fn, torch.float8_e8m0fnu


class _Ctx:
    device = 0
    handle = None


def _t(shape, dtype=BF):
    return torch.empty(shape, dtype=dtype)


# ---- the binding -----------------------------------------------------------------
def _norm(**kw):
    a = dict(x=_t((4, 64)), weight=_t((64,)), out=_t((4, 64)))
    a.update(kw)
    x, w, out = a.pop("x"), a.pop("weight"), a.pop("out")
    return cce.cce_rmsnorm(_Ctx(), x, w, out, **a)


@pytest.mark.parametrize("kw,match", [
    (dict(), "cuda:0"),
    (dict(residual=_t((4, 64), F32)), "residual"),
    (dict(residual=_t((4, 63))), "residual"),
    (dict(out=_t((4, 56))), "out"),
    (dict(weight=_t((63,))), "weight"),
    (dict(weight=_t((128,))[::2]), "contiguous"),
    (dict(out=_t((4, 64), E4)), "scales go with"),
    (dict(scales=_t((4, 1), E8)), "scales go with"),
    (dict(out=_t((4, 64), E4), scales=_t((4, 1), torch.uint8)), "scales"),
    (dict(out=_t((4, 64), E4), scales=_t((4, 2), E8)), "scales"),
    (dict(x=_t((4, 128))[:, ::2]), "unit column stride"),
])
def test_norm_binding_refuses(kw, match):
    with pytest.raises(ValueError, match=match):
        _norm(**kw)


def test_norm_binding_refuses_other_dtypes():
    with pytest.raises(TypeError, match="unsupported dtype"):
        cce.cce_rmsnorm(_Cuda(), _Fake((4, 64), torch.float16), _Fake((64,), BF), _Fake((4, 64), BF))


class _Cuda(_Ctx):
    device = None


class _Fake:
    """A tensor that says it is on the GPU: only its description is read before a refusal."""

    def __init__(self, shape, dtype):
        self._t = torch.empty(shape, dtype=dtype)
        self.device = torch.device("cuda", 0)

    def get_device(self):
        return 0

    def __getattr__(self, name):
        return getattr(self._t, name)


@pytest.mark.parametrize("kw,match", [
    (dict(), "cuda:0"),
    (dict(dout=_t((4, 64), F32)), "dout"),
    (dict(dx=_t((4, 72))), "dx"),
    (dict(dweight=_t((64,))), "dweight"),
    (dict(dweight=_t((63,), F32)), "dweight"),
    (dict(d_residual=_t((5, 64))), "d_residual"),
])
def test_norm_backward_binding_refuses(kw, match):
    a = dict(dout=_t((4, 64)), dx=_t((4, 64)), dweight=_t((64,), F32), d_residual=None)
    a.update(kw)
    with pytest.raises(ValueError, match=match):
        cce.cce_rmsnorm_backward(_Ctx(), _t((4, 64)), _t((64,)), a["dout"], a["dx"], a["dweight"],
                                 d_residual=a["d_residual"])


@pytest.mark.parametrize("x,q,s,block_rows,match", [
    (_t((4, 64)), _t((4, 64), E4), _t((4, 1), E8), 1, "cuda:0"),
    (_t((4, 64)), _t((4, 64)), _t((4, 1), E8), 1, "q must be"),
    (_t((4, 64)), _t((4, 64), E4), _t((4, 1), F32), 1, "scales"),
    (_t((4, 64)), _t((4, 64), E4), _t((4, 1), E8), 128, "scales"),
    (_t((4, 64)), _t((4, 64), E4), _t((4, 1), E8), 64, "block_rows"),
])
def test_quantize_binding_refuses(x, q, s, block_rows, match):
    with pytest.raises(ValueError, match=match):
        cce.cce_quantize_blocks(_Ctx(), x, q, s, block_rows)


def test_block_scaled_gemm_binding_refuses():
    a, b, c = _t((4, 256), E4), _t((8, 256), E4), _t((4, 8))
    sa, sb = _t((4, 2), E8), _t((1, 2), E8)
    with pytest.raises(ValueError, match="cuda:0"):
        cce.cce_block_scaled_gemm(_Ctx(), a, sa, b, sb, c)
    with pytest.raises(ValueError, match="a and b"):
        cce.cce_block_scaled_gemm(_Ctx(), a, sa, _t((8, 256)), sb, c)
    with pytest.raises(ValueError, match="b_scales"):
        cce.cce_block_scaled_gemm(_Ctx(), a, sa, b, _t((8, 2), E8), c)
    with pytest.raises(ValueError, match="a_scales"):
        cce.cce_block_scaled_gemm(_Ctx(), a, _t((4, 2), F32), b, sb, c)


def test_ragged_binding_refuses():
    a, b, c = _t((4, 16)), _t((2, 8, 16)), _t((4, 8))
    off = torch.zeros(3, dtype=torch.int64)
    for f, args in ((cce.cce_ragged_gemm, (a, b, off, c)), (cce.cce_ragged_gemm_dgrad, (c, b, off, a)),
                    (cce.cce_ragged_gemm_wgrad, (c, a, off, b))):
        with pytest.raises(ValueError, match="cuda:0"):
            f(_Ctx(), *args)
        bad = [off.int() if t is off else t for t in args]
        with pytest.raises(ValueError, match="offsets"):
            f(_Ctx(), *bad)
        bad = [off[:2] if t is off else t for t in args]
        with pytest.raises(ValueError, match="offsets"):
            f(_Ctx(), *bad)
    with pytest.raises(ValueError, match="a and b"):
        cce.cce_ragged_gemm(_Ctx(), a.float(), b, off, c)
    with pytest.raises(ValueError, match="experts, N, K"):
        cce.cce_ragged_gemm(_Ctx(), a, b[0], off, c)


# ---- the C ABI -------------------------------------------------------------------
@pytest.fixture(scope="module")
def L():
    return _lib.lib()


CTX = ctypes.create_string_buffer(4096)     # stands in for a context: never read by a refused call
P = 1 << 20                                  # stands in for a device address: never dereferenced
F, B, Q = _lib.CCE_F32, _lib.CCE_BF16, _lib.CCE_E4M3
EINVAL, EUNS, EWS = _lib.CCE_EINVAL, _lib.CCE_EUNSUPPORTED, _lib.CCE_EWORKSPACE


def _call(f, names, base, change):
    a = dict(base)
    a.update(change)
    return f(*[a[n] for n in names])


NORM = ["ctx", "x_t", "x", "xm", "res", "ld_res", "ro", "ld_ro", "w", "w_t", "eps", "out", "out_t", "ld_out",
        "s", "ld_s", "flags", "stream"]
NORM_BASE = dict(ctx=CTX, x_t=B, x=P, xm=cce_mat(4, 64, 64), res=None, ld_res=64, ro=None, ld_ro=64, w=2 * P, w_t=B,
                 eps=1e-5, out=3 * P, out_t=B, ld_out=64, s=None, ld_s=1, flags=0, stream=None)


@pytest.mark.parametrize("change,status", [
    (dict(ctx=None), EINVAL), (dict(flags=1), EINVAL), (dict(x_t=7), EINVAL), (dict(x_t=Q), EINVAL),
    (dict(w_t=Q), EINVAL), (dict(out_t=5), EINVAL), (dict(eps=0.0), EINVAL), (dict(eps=-1.0), EINVAL),
    (dict(eps=float("nan")), EINVAL), (dict(eps=float("inf")), EINVAL), (dict(eps=1e-60), EINVAL),
    (dict(x=None), EINVAL), (dict(w=None), EINVAL), (dict(out=None), EINVAL), (dict(ro=4 * P), EINVAL),
    (dict(s=4 * P), EINVAL), (dict(out_t=Q), EINVAL), (dict(out_t=Q, s=4 * P, ld_s=0), EINVAL),
    (dict(x=P + 8), EUNS), (dict(w=2 * P + 2), EUNS), (dict(ld_out=68), EUNS), (dict(ld_out=56), EINVAL),
    (dict(xm=cce_mat(-1, 64, 64)), EINVAL), (dict(xm=cce_mat(4, 64, 60)), EINVAL),
    (dict(xm=cce_mat(1 << 32, 64, 64)), EUNS), (dict(res=4 * P, ld_res=32), EINVAL),
    (dict(out=P + 128), EINVAL), (dict(res=4 * P, ro=4 * P), EINVAL), (dict(res=4 * P, ro=P), EINVAL),
    (dict(out_t=Q, s=3 * P + 16, ld_s=1), EINVAL), (dict(out=2 * P + 64), EINVAL),
])
def test_norm_abi_refuses(L, change, status):
    assert _call(L.cce_rmsnorm, NORM, NORM_BASE, change) == status


BWD = ["ctx", "x_t", "x", "xm", "w", "w_t", "dout", "ld_dout", "dres", "ld_dres", "eps", "dx", "ld_dx", "dw", "ws",
       "wsb", "flags", "stream"]
BWD_BASE = dict(ctx=CTX, x_t=B, x=P, xm=cce_mat(4, 64, 64), w=2 * P, w_t=F, dout=3 * P, ld_dout=64, dres=None,
                ld_dres=64, eps=1e-5, dx=4 * P, ld_dx=64, dw=5 * P, ws=6 * P, wsb=1 << 20, flags=0, stream=None)


@pytest.mark.parametrize("change,status", [
    (dict(ctx=None), EINVAL), (dict(flags=2), EINVAL), (dict(x_t=Q), EINVAL), (dict(eps=0.0), EINVAL),
    (dict(ws=None), EWS), (dict(wsb=16), EWS), (dict(ws=6 * P + 4), EUNS), (dict(dout=None), EINVAL),
    (dict(dx=None), EINVAL), (dict(dx=P), EINVAL), (dict(dw=4 * P), EINVAL), (dict(dw=5 * P + 4), EUNS),
    (dict(ws=5 * P + 64), EINVAL), (dict(ld_dx=12), EINVAL), (dict(ld_dout=65), EUNS),
    (dict(dres=7 * P, ld_dres=8), EINVAL),
])
def test_norm_backward_abi_refuses(L, change, status):
    assert _call(L.cce_rmsnorm_backward, BWD, BWD_BASE, change) == status


def test_norm_backward_workspace_query(L):
    nb = ctypes.c_size_t()
    assert L.cce_rmsnorm_backward_workspace(cce_mat(4, 64, 64), None) == EINVAL
    assert L.cce_rmsnorm_backward_workspace(cce_mat(4, 64, 60), ctypes.byref(nb)) == EINVAL
    for shape in ((1, 1), (4, 64), (8192, 12288), (3, 100001)):
        need = cce.cce_rmsnorm_backward_workspace(shape)
        assert 4 * shape[1] <= need <= 16 * shape[0] * shape[1] + 4096 + 4 * shape[1] * 512
    assert cce.cce_rmsnorm_backward_workspace((0, 64)) == 0


QUANT = ["ctx", "x_t", "x", "xm", "br", "q", "ld_q", "s", "ld_s", "flags", "stream"]
QUANT_BASE = dict(ctx=CTX, x_t=F, x=P, xm=cce_mat(4, 64, 64), br=1, q=2 * P, ld_q=64, s=3 * P, ld_s=1, flags=0,
                  stream=None)


@pytest.mark.parametrize("change,status", [
    (dict(ctx=None), EINVAL), (dict(br=2), EINVAL), (dict(x_t=Q), EINVAL), (dict(flags=1), EINVAL),
    (dict(q=None), EINVAL), (dict(s=None), EINVAL), (dict(ld_q=60), EINVAL), (dict(ld_q=68), EUNS),
    (dict(ld_s=0), EINVAL), (dict(q=P), EINVAL), (dict(s=2 * P + 3), EINVAL),
])
def test_quantize_abi_refuses(L, change, status):
    assert _call(L.cce_quantize_blocks, QUANT, QUANT_BASE, change) == status


G8 = ["ctx", "out_t", "a", "am", "sa", "ld_sa", "b", "bm", "sb", "ld_sb", "c", "cm", "flags", "stream"]
G8_BASE = dict(ctx=CTX, out_t=B, a=P, am=cce_mat(4, 256, 256), sa=2 * P, ld_sa=2, b=3 * P, bm=cce_mat(8, 256, 256),
               sb=4 * P, ld_sb=2, c=5 * P, cm=cce_mat(4, 8, 8), flags=0, stream=None)


@pytest.mark.parametrize("change,status", [
    (dict(ctx=None), EINVAL), (dict(out_t=Q), EINVAL), (dict(flags=1), EINVAL), (dict(a=None), EINVAL),
    (dict(sa=None), EINVAL), (dict(sb=None), EINVAL), (dict(c=None), EINVAL), (dict(ld_sa=1), EINVAL),
    (dict(am=cce_mat(4, 240, 256)), EINVAL), (dict(cm=cce_mat(4, 16, 16)), EINVAL), (dict(cm=cce_mat(3, 8, 8)), EINVAL),
    (dict(am=cce_mat(4, 248, 256), bm=cce_mat(8, 248, 256)), EUNS), (dict(am=cce_mat(4, 256, 264)), EUNS),
    (dict(bm=cce_mat(8, 256, 1 << 21)), EUNS), (dict(c=P + 512), EINVAL), (dict(c=2 * P), EINVAL),
    (dict(b=3 * P + 8), EUNS),
])
def test_block_scaled_gemm_abi_refuses(L, change, status):
    assert _call(L.cce_block_scaled_gemm, G8, G8_BASE, change) == status


RAG = ["ctx", "out_t", "e", "off", "p0", "m0", "p1", "m1", "stride", "p2", "m2", "flags", "stream"]
A, W, C = cce_mat(6, 32, 32), cce_mat(16, 32, 32), cce_mat(6, 16, 16)
RAG_BASE = dict(ctx=CTX, out_t=B, e=3, off=4 * P, p0=P, m0=A, p1=2 * P, m1=W, stride=512, p2=3 * P, m2=C, flags=0,
                stream=None)


@pytest.mark.parametrize("change,status", [
    (dict(ctx=None), EINVAL), (dict(out_t=Q), EINVAL), (dict(flags=2), EINVAL), (dict(e=0), EINVAL),
    (dict(e=65537), EUNS), (dict(off=None), EINVAL), (dict(off=4 * P + 4), EUNS), (dict(p0=None), EINVAL),
    (dict(p1=None), EINVAL), (dict(p2=None), EINVAL), (dict(stride=511), EUNS), (dict(stride=-8), EINVAL),
    (dict(m0=cce_mat(6, 24, 32)), EINVAL), (dict(m2=cce_mat(5, 16, 16)), EINVAL), (dict(m2=cce_mat(6, 8, 16)), EINVAL),
    (dict(p2=P + 64), EINVAL), (dict(p2=4 * P - 16), EINVAL), (dict(p2=2 * P + 2048), EINVAL),
    (dict(m0=cce_mat(6, 32, 2 << 20)), EUNS),
])
def test_ragged_abi_refuses(L, change, status):
    assert _call(L.cce_ragged_gemm, RAG, RAG_BASE, change) == status


@pytest.mark.parametrize("change,status", [
    (dict(stride=256), EINVAL), (dict(stride=0), EINVAL), (dict(p2=P), EINVAL), (dict(p2=4 * P - 2048), EINVAL),
    (dict(m2=cce_mat(16, 24, 32)), EINVAL),
])
def test_ragged_wgrad_abi_refuses(L, change, status):
    names = ["ctx", "out_t", "e", "off", "p0", "m0", "p1", "m1", "p2", "m2", "stride", "flags", "stream"]
    base = dict(ctx=CTX, out_t=F, e=3, off=4 * P, p0=P, m0=C, p1=2 * P, m1=A, p2=3 * P, m2=W, stride=512, flags=0,
                stream=None)
    assert _call(L.cce_ragged_gemm_wgrad, names, base, change) == status


def test_nothing_to_do_is_ok(L):
    """Zero extents: CCE_OK before the context is used."""
    assert _call(L.cce_rmsnorm, NORM, NORM_BASE, dict(xm=cce_mat(0, 64, 64))) == 0
    assert _call(L.cce_rmsnorm, NORM, NORM_BASE, dict(xm=cce_mat(4, 0, 0), x=None, w=None, out=None)) == 0
    assert _call(L.cce_rmsnorm_backward, BWD, BWD_BASE, dict(xm=cce_mat(0, 64, 64), dw=None, ws=None, wsb=0)) == 0
    assert _call(L.cce_quantize_blocks, QUANT, QUANT_BASE, dict(xm=cce_mat(0, 64, 64))) == 0
    assert _call(L.cce_block_scaled_gemm, G8, G8_BASE, dict(am=cce_mat(0, 256, 256), cm=cce_mat(0, 8, 8))) == 0
    assert _call(L.cce_ragged_gemm, RAG, RAG_BASE, dict(m0=cce_mat(0, 32, 32), m2=cce_mat(0, 16, 16))) == 0


def test_norm_backward_without_the_weight_gradient_needs_no_workspace(L):
    """The call gets past the workspace's check, to that of the overlap."""
    for ws, wsb in ((None, 0), (6 * P, 16)):
        assert _call(L.cce_rmsnorm_backward, BWD, BWD_BASE, dict(dw=None, ws=ws, wsb=wsb, dx=P)) == EINVAL
        assert _call(L.cce_rmsnorm_backward, BWD, BWD_BASE, dict(ws=ws, wsb=wsb, dx=P)) == EWS
