"""Refusals of the operators around an fp8 linear layer: every argument check
of the C entry points runs before any HIP call, and the binding's own checks
run on host tensors (nothing is launched)."""
import ctypes as C
import os

import pytest
import torch

import fp8_tensor_scaled_quantize_amd as fp8mi
from fp8_tensor_scaled_quantize_amd import _lib

OK, NULL, ENUM, SHAPE, STRIDE, UNSUP, HIP, ARG = range(8)
FAKE = 0x10000


@pytest.fixture(scope="module")
def L():
    if not os.path.exists(_lib.LIB_PATH):
        pytest.skip("libfp8mi.so not built")
    return _lib.lib()


def eps_ptr(v=1e-6):
    return C.byref(C.c_float(v))


NAN_EPS = float("nan")


@pytest.mark.parametrize("kw,status", [
    (dict(dt=3), ENUM), (dict(fmt=2), ENUM), (dict(wdt=7), ENUM), (dict(scaling=2), ENUM),
    (dict(rows=-1), SHAPE), (dict(ld=7), SHAPE), (dict(ld_res=7), SHAPE), (dict(ld_sum=7, sum_out=FAKE), SHAPE),
    (dict(ld_out=7), SHAPE), (dict(ld=1 << 61), SHAPE), (dict(ld_res=1 << 61), SHAPE),
    (dict(cols=32769, ld=32769, ld_res=32769, ld_out=32769), UNSUP),
    (dict(x=None), NULL), (dict(out=None), NULL), (dict(eps=None), NULL),
    (dict(eps=-1.0), ARG), (dict(eps=NAN_EPS), ARG),
    (dict(scale=None), ARG), (dict(ring=FAKE, h=4), ARG), (dict(scale=None, ring=FAKE, h=0), SHAPE),
    (dict(scaling=1), ARG), (dict(scaling=1, scale=None, ring=FAKE, h=4), ARG), (dict(scaling=1, scale=None), NULL),
    (dict(x=FAKE + 1), ARG), (dict(res=FAKE + 1), ARG), (dict(w=FAKE + 1), ARG), (dict(sum_out=FAKE + 1), ARG),
    (dict(scale=FAKE + 2), ARG), (dict(sinv=FAKE + 2), ARG), (dict(amax=FAKE + 2), ARG), (dict(rstd=FAKE + 2), ARG),
])
def test_rmsnorm_rejects(L, kw, status):
    a = dict(x=FAKE, dt=2, rows=4, cols=8, ld=8, res=FAKE, ld_res=8, w=FAKE, wdt=2, eps=1e-6, fmt=0, out=FAKE,
             ld_out=8, scaling=0, scale=FAKE, ring=None, h=0, sinv=None, amax=None, sum_out=None, ld_sum=8, rstd=None)
    a.update(kw)
    a["eps"] = None if a["eps"] is None else eps_ptr(a["eps"])
    assert L.fp8_rmsnorm(*a.values(), None) == status
    assert L.fp8mi_last_error()


def test_rmsnorm_grad_rejects(L):
    need = L.fp8_rmsnorm_grad_workspace_bytes(4, 8)
    base = dict(dy=FAKE, dt=2, rows=4, cols=8, ld=8, h=FAKE, ld_h=8, w=FAKE, wdt=2, rstd=FAKE, ds=FAKE, ld_ds=8,
                dx=FAKE, ld_dx=8, dw=FAKE, ws=FAKE, wsb=need)

    def call(**kw):
        return L.fp8_rmsnorm_grad(*{**base, **kw}.values(), None)

    assert call(dt=5) == ENUM and call(wdt=-1) == ENUM
    assert call(rows=-1) == SHAPE and call(ld=7) == SHAPE and call(ld_h=7) == SHAPE
    assert call(ld_ds=7) == SHAPE and call(ld_dx=7) == SHAPE and call(ld_dx=1 << 61) == SHAPE
    assert call(cols=40000, ld=40000) == UNSUP
    for name in ("dy", "h", "rstd", "dx", "ws"):
        assert call(**{name: None}) == NULL, name
    for name in ("dy", "h", "w", "ds", "dx"):
        assert call(**{name: FAKE + 1}) == ARG, name
    for name in ("rstd", "dw", "ws"):
        assert call(**{name: FAKE + 2}) == ARG, name
    assert call(wsb=need - 1) == ARG
    assert call(dy=None, cols=0, h=None, dx=None, rstd=None, ws=None, wsb=0) == OK  # nothing to do


def test_rmsnorm_grad_workspace(L):
    f = L.fp8_rmsnorm_grad_workspace_bytes
    assert f(0, 8) == 0 and f(8, 0) == 0 and f(-1, 8) == 0
    for rows, cols in ((1, 1), (7, 1535), (8192, 1536), (100000, 4096)):
        assert 4 * cols <= f(rows, cols) <= 4 * cols * min(rows, 1024)


def test_binding_checks_norm_arguments():
    x, w = torch.zeros(4, 8, dtype=torch.bfloat16), torch.ones(8)
    one = torch.ones(1)
    with pytest.raises(ValueError, match="device"):
        fp8mi.fp8_rmsnorm(x, w, scale=one)
    with pytest.raises(ValueError, match="2-D"):
        fp8mi.fp8_rmsnorm(x.t(), w, scale=one)
    with pytest.raises(ValueError, match="residual"):
        fp8mi.fp8_rmsnorm(x, w, scale=one, residual=x.float())
    with pytest.raises(ValueError, match="sum_out"):
        fp8mi.fp8_rmsnorm(x, w, scale=one, sum_out=x[:2])
    with pytest.raises(ValueError, match="weight"):
        fp8mi.fp8_rmsnorm(x, w[:7], scale=one)
    with pytest.raises(ValueError, match="scale_inv_out"):
        fp8mi.fp8_rmsnorm(x, w, row_scaled=True)
    with pytest.raises(ValueError, match="neither"):
        fp8mi.fp8_rmsnorm(x, w, row_scaled=True, scale=one, scale_inv_out=torch.ones(4))
    with pytest.raises(ValueError, match="scale_inv_out"):
        fp8mi.fp8_rmsnorm(x, w, row_scaled=True, scale_inv_out=torch.ones(3))
    with pytest.raises(ValueError, match="rstd_out"):
        fp8mi.fp8_rmsnorm(x, w, scale=one, rstd_out=torch.ones(4, dtype=torch.float64))
    with pytest.raises(ValueError, match="out"):
        fp8mi.fp8_rmsnorm(x, w, scale=one, out=torch.zeros(4, 7, dtype=torch.uint8))
    with pytest.raises(ValueError, match="h must be"):
        fp8mi.fp8_rmsnorm_grad(x, x.float(), w, torch.ones(4))
    with pytest.raises(ValueError, match="rstd"):
        fp8mi.fp8_rmsnorm_grad(x, x, w, torch.ones(5))
    with pytest.raises(ValueError, match="dweight"):
        fp8mi.fp8_rmsnorm_grad(x, x, w, torch.ones(4), dweight=torch.ones(8, dtype=torch.bfloat16))


@pytest.mark.parametrize("kw,status", [
    (dict(act=4), ENUM), (dict(act=-1), ENUM), (dict(act=32), ENUM), (dict(rows=4), ENUM), (dict(bdt=3), ENUM),
    (dict(rdt=3), ENUM), (dict(cdt=0), ENUM), (dict(cdt=4, cs=FAKE), UNSUP),
    (dict(M=-1), SHAPE), (dict(K=-16), SHAPE), (dict(N=33, act=19, ldc=40, ldz=40), SHAPE), (dict(ldc=31), SHAPE),
    (dict(lda=48), SHAPE), (dict(ldb=48), SHAPE), (dict(ldr=31), SHAPE), (dict(ldz=31), SHAPE), (dict(ldz=1 << 61), SHAPE),
    (dict(ldc=1 << 62), SHAPE), (dict(lda=1 << 60), SHAPE),
    (dict(a=None), NULL), (dict(b=None), NULL), (dict(c=None), NULL), (dict(rows=1, sa=None), NULL),
    (dict(rows=2, sb=None), NULL),
    (dict(cs=FAKE), ARG), (dict(cdt=3), ARG), (dict(cdt=3, cs=FAKE, ring=FAKE, h=4), ARG),
    (dict(cdt=3, ring=FAKE, h=0), SHAPE), (dict(c=FAKE + 1), ARG), (dict(z=FAKE + 1), ARG), (dict(res=FAKE + 1), ARG),
    (dict(bias=FAKE + 1), ARG), (dict(sa=FAKE + 2), ARG), (dict(sb=FAKE + 2), ARG),
    (dict(K=40), UNSUP), (dict(lda=72), UNSUP), (dict(a=FAKE + 8), UNSUP), (dict(b=FAKE + 8), UNSUP),
    (dict(M=1 << 23), UNSUP), (dict(M=1 << 20, lda=4096), UNSUP),
])
def test_mm_act_rejects(L, kw, status):
    a = dict(a=FAKE, lda=64, b=FAKE, ldb=64, M=32, N=32, K=64, sa=FAKE, sb=FAKE, rows=0, bias=FAKE, bdt=2, act=2,
             res=FAKE, rdt=2, ldr=32, z=FAKE, ldz=32, c=FAKE, cdt=2, ldc=32, cs=None, ring=None, h=0, csi=None, cam=None)
    a.update(kw)
    assert L.fp8_mm_act(*a.values(), None) == status
    assert L.fp8mi_last_error()


def test_mm_act_empty_is_noop(L):
    z = [None, 64, None, 64, 0, 32, 64, None, None, 0, None, 0, 2, None, 0, 0, None, 0, None, 2, 32, None, None, 0, None,
         None, None]
    assert L.fp8_mm_act(*z) == OK


@pytest.mark.parametrize("kw,status", [
    (dict(act=0), ARG), (dict(act=4), ENUM), (dict(act=-3), ENUM), (dict(dt=0), UNSUP), (dict(dt=5), ENUM),
    (dict(fmt=2), ENUM), (dict(act=18, cols=9), SHAPE), (dict(rows=-1), SHAPE), (dict(ld=7), SHAPE), (dict(ldz=7), SHAPE),
    (dict(ldr=7), SHAPE), (dict(ldt=3), SHAPE), (dict(ldz=1 << 62), SHAPE), (dict(dy=None), NULL), (dict(z=None), NULL),
    (dict(o=None), NULL), (dict(ot=None), NULL), (dict(ws=None), NULL), (dict(wsb=63), ARG), (dict(ws=FAKE + 4), ARG),
    (dict(db=FAKE + 1), ARG), (dict(s=None), ARG), (dict(ring=FAKE, h=4), ARG), (dict(s=FAKE + 2), ARG),
    (dict(dy=FAKE + 1), ARG), (dict(z=FAKE + 1), ARG), (dict(am=FAKE + 2), ARG),
])
def test_act_grad_rejects(L, kw, status):
    assert L.fp8_bias_grad_workspace_bytes(4, 8) == 64
    a = dict(dy=FAKE, dt=2, rows=4, cols=8, ld=8, z=FAKE, ldz=8, act=2, fmt=1, o=FAKE, ldr=8, ot=FAKE, ldt=4, s=FAKE,
             ring=None, h=0, si=None, am=None, db=FAKE, ws=FAKE, wsb=64)
    a.update(kw)
    assert L.fp8_act_grad(*a.values(), None) == status
    assert L.fp8mi_last_error()


def test_binding_checks_mm_act_arguments():
    a, b = torch.zeros(4, 16, dtype=torch.uint8), torch.zeros(6, 16, dtype=torch.uint8)
    with pytest.raises(ValueError, match="device"):
        fp8mi.fp8_mm_act(a, b)
    with pytest.raises(ValueError, match="K mismatch"):
        fp8mi.fp8_mm_act(a, b[:, :8])
    with pytest.raises(ValueError, match="activation"):
        fp8mi.fp8_mm_act(a, b, act="tanh")
    with pytest.raises(ValueError, match="even"):
        fp8mi.fp8_mm_act(a, b[:5], gated=True)
    with pytest.raises(ValueError, match="a_scale_inv"):
        fp8mi.fp8_mm_act(a, b, a_scale_inv=torch.ones(3))
    with pytest.raises(ValueError, match="b_scale_inv"):
        fp8mi.fp8_mm_act(a, b, b_scale_inv=torch.ones(6, dtype=torch.float64))
    with pytest.raises(ValueError, match="bias"):
        fp8mi.fp8_mm_act(a, b, bias=torch.ones(4))
    with pytest.raises(ValueError, match="residual"):
        fp8mi.fp8_mm_act(a, b, gated=True, residual=torch.zeros(4, 6))
    with pytest.raises(ValueError, match="z_out"):
        fp8mi.fp8_mm_act(a, b, z_out=torch.zeros(4, 6))
    with pytest.raises(ValueError, match="E4M3"):
        fp8mi.fp8_mm_act(a, b, out_fmt=fp8mi.E5M2)
    with pytest.raises(ValueError, match="out must be bfloat16"):
        fp8mi.fp8_mm_act(a, b, out=torch.zeros(4, 6))
    with pytest.raises(ValueError, match="1-byte"):
        fp8mi.fp8_mm_act(a.float(), b)


def test_binding_checks_act_grad_arguments():
    dy, z = torch.zeros(4, 8, dtype=torch.bfloat16), torch.zeros(4, 8, dtype=torch.bfloat16)
    one = torch.ones(1)
    with pytest.raises(ValueError, match="device"):
        fp8mi.fp8_act_grad(dy, z, "gelu", scale=one)
    with pytest.raises(ValueError, match="does not fit"):
        fp8mi.fp8_act_grad(dy, z, "gelu", gated=True, scale=one)
    with pytest.raises(ValueError, match="z must be bfloat16"):
        fp8mi.fp8_act_grad(dy, z.float(), "gelu", scale=one)
    with pytest.raises(ValueError, match="out_t"):
        fp8mi.fp8_act_grad(dy, z, "gelu", scale=one, out_t=torch.zeros(4, 8, dtype=torch.uint8))
    with pytest.raises(ValueError, match="bias_grad_out"):
        fp8mi.fp8_act_grad(dy, z, "gelu", scale=one, bias_grad_out=torch.zeros(7, dtype=torch.bfloat16))


def test_interleave_gated():
    g, v = torch.arange(6).reshape(3, 2), torch.arange(10, 16).reshape(3, 2)
    w = fp8mi.interleave_gated(g, v)
    assert torch.equal(w[0::2], g) and torch.equal(w[1::2], v)
    assert torch.equal(fp8mi.interleave_gated(g[:, 0], v[:, 0]), torch.tensor([0, 10, 2, 12, 4, 14]))
    with pytest.raises(ValueError):
        fp8mi.interleave_gated(g, v[:2])
