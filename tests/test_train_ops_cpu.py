"""Refusals of the operators that end a training step: every argument check of
the C entry points runs before any HIP call, and the binding's own checks run on
host tensors (nothing is launched)."""
import ctypes as C
import os
import struct

import numpy as np
import pytest
import torch

import fp8_tensor_scaled_quantize_amd as fp8mi
import train_ref as R
from fp8_tensor_scaled_quantize_amd import _lib

OK, NULL, ENUM, SHAPE, STRIDE, UNSUP, HIP, ARG = range(8)
FAKE = 0x10000


@pytest.fixture(scope="module")
def L():
    if not os.path.exists(_lib.LIB_PATH):
        pytest.skip("libfp8mi.so not built")
    return _lib.lib()


def tensor(param=FAKE, grad=FAKE, master=0, m=FAKE, v=FAKE, ms=0, vs=0, n=10, pdt=2, gdt=2, bits=32, wd=0.0):
    return struct.pack("@7Pq3if", param, grad, master, m, v, ms, vs, n, pdt, gdt, bits, wd)


def hyper(lr=1e-3, b1=0.9, b2=0.95, eps=1e-8, step=1, words=0, lr_device=0, scale=0, seed=0):
    return struct.pack("@4dq3PI4x", lr, b1, b2, eps, step, words, lr_device, scale, seed)


NAN = float("nan")


@pytest.mark.parametrize("kw,status", [
    (dict(pdt=3), ENUM), (dict(gdt=-1), ENUM), (dict(bits=16), ENUM), (dict(n=-1), SHAPE), (dict(n=1 << 60), SHAPE),
    (dict(param=0), NULL), (dict(grad=0), NULL), (dict(m=0), NULL), (dict(v=0), NULL),
    (dict(bits=8), NULL), (dict(bits=8, ms=FAKE), NULL), (dict(ms=FAKE), ARG), (dict(vs=FAKE), ARG),
    (dict(pdt=0, master=FAKE), ARG), (dict(param=FAKE + 1), ARG), (dict(grad=FAKE + 1), ARG), (dict(master=FAKE + 2), ARG),
    (dict(m=FAKE + 2), ARG), (dict(v=FAKE + 2), ARG), (dict(bits=8, ms=FAKE + 2, vs=FAKE), ARG), (dict(wd=-0.1), ARG),
    (dict(wd=NAN), ARG),
])
def test_adamw_rejects_tensors(L, kw, status):
    assert L.fp8_adamw_step(tensor() + tensor(**kw), 2, hyper(), None) == status
    assert L.fp8mi_last_error()


@pytest.mark.parametrize("kw,status", [
    (dict(b1=1.0), ARG), (dict(b1=-0.1), ARG), (dict(b2=NAN), ARG), (dict(eps=-1.0), ARG), (dict(lr=NAN), ARG),
    (dict(lr=-1.0), ARG), (dict(step=0), ARG), (dict(step=-3), ARG), (dict(step=1 << 31), ARG), (dict(step=1, words=FAKE), ARG),
    (dict(lr_device=FAKE), ARG), (dict(step=0, words=FAKE + 2), ARG), (dict(scale=FAKE + 1), ARG),
])
def test_adamw_rejects_hyper_parameters(L, kw, status):
    assert L.fp8_adamw_step(tensor(), 1, hyper(**kw), None) == status


def test_adamw_rejects_lists(L):
    assert L.fp8_adamw_step(None, 1, hyper(), None) == NULL and L.fp8_adamw_step(tensor(), 1, None, None) == NULL
    assert L.fp8_adamw_step(tensor(), -1, hyper(), None) == SHAPE
    assert L.fp8_adamw_step(None, 0, hyper(), None) == OK


def test_grad_norm_rejects(L):
    def t(p=FAKE, n=10000, dt=2):
        return struct.pack("@Pqi4x", p, n, dt)

    need = L.fp8_grad_norm_workspace_bytes(t() + t(), 2)
    assert need == 2 * 3 * 8 and L.fp8_grad_norm_workspace_bytes(None, 0) == 0

    def call(table=t(), count=1, limit=1.0, out=FAKE, clip=FAKE, ws=FAKE, nbytes=need):
        return L.fp8_grad_norm(table, count, C.byref(C.c_float(limit)), out, clip, ws, nbytes, None)

    assert call(count=-1) == SHAPE and call(table=None) == NULL and call(table=t(n=-1)) == SHAPE
    assert call(table=t(dt=4)) == ENUM and call(table=t(p=0)) == NULL and call(table=t(p=FAKE + 1)) == ARG
    assert call(limit=-1.0) == ARG and call(limit=NAN) == ARG and call(out=FAKE + 2) == ARG and call(clip=FAKE + 2) == ARG
    assert call(ws=None) == NULL and call(ws=FAKE + 4) == ARG and call(nbytes=8) == ARG


def test_sizes_beyond_a_grid(L):
    """A grid holds fewer than 2^32 threads: sizes that would need more are refused before anything is read."""
    assert L.fp8_adamw_step(tensor(n=(1 << 33) + 1), 1, hyper(), None) == SHAPE

    def norm(*sizes):
        table = b"".join(struct.pack("@Pqi4x", FAKE, n, 2) for n in sizes)
        return L.fp8_grad_norm(table, len(sizes), None, FAKE, FAKE, None, 0, None)

    assert norm((1 << 38) + 1) == SHAPE and norm(1 << 37, (1 << 37) + 1) == SHAPE
    assert norm(1 << 37, 1 << 37) == NULL  # allowed: only the workspace is missing
    for f in (L.fp8_cross_entropy_workspace_bytes, L.fp8_cross_entropy_grad_workspace_bytes):
        assert f(1, (1 << 28) + 1, 16) == 0 and f(1, 1 << 28, 16) > 0


def test_binding_refuses_lists():
    f32 = lambda n=4: torch.zeros(n)  # noqa: E731

    def step(p=None, g=None, m=None, v=None, t=1, **kw):
        fp8mi.fp8_adamw_step(p or [f32()], g or [f32()], m or [f32()], v or [f32()], t, **kw)

    for kw, text in [
        (dict(g=[f32(5)]), "elements"), (dict(g=[f32(), f32()]), "grads for"), (dict(m=[f32(3)]), "elements"),
        (dict(p=[torch.zeros(4, 4).t()], g=[f32(16)], m=[f32(16)], v=[f32(16)]), "contiguous"),
        (dict(p=[torch.zeros(4, dtype=torch.int32)]), "params must be"), (dict(g=[torch.zeros(4, dtype=torch.uint8)]), "grads must be"),
        (dict(m=[torch.zeros(4, dtype=torch.bfloat16)]), "states must be float32"), (dict(masters=[]), "one entry per"),
        (dict(masters=[torch.zeros(4, dtype=torch.float16)]), "masters must be float32"), (dict(masters=[f32(5)]), "elements"),
        (dict(exp_avg_scales=[f32(1)]), "8-bit states"), (dict(exp_avg_scales=[f32(1)], exp_avg_sq_scales=[f32(1)]), "1-byte"),
        (dict(m=[torch.zeros(4, dtype=torch.uint8)], v=[torch.zeros(4, dtype=torch.uint8)], exp_avg_scales=[f32(2)],
              exp_avg_sq_scales=[f32(1)]), "scales"),
        (dict(weight_decay=[0.1, 0.2]), "weight decays"), (dict(t=torch.zeros(1, dtype=torch.int32)), "device step"),
        (dict(t=torch.zeros(4, dtype=torch.int64)), "device step"), (dict(lr=f32(1)), "lr on the device"),
        (dict(grad_scale=torch.zeros(1, dtype=torch.float64)), "grad_scale"), (dict(), "host tensor"),
    ]:
        with pytest.raises(ValueError, match=text):
            step(**kw)
    with pytest.raises(ValueError, match="host tensor"):
        fp8mi.fp8_grad_norm([f32()])
    with pytest.raises(ValueError, match="no gradients"):
        fp8mi.fp8_grad_norm([])
    with pytest.raises(ValueError, match="contiguous"):
        fp8mi.fp8_grad_norm([torch.zeros(4, 4).t()])


def test_reference_grid_and_numbers():
    """The reference's E4M3 grid holds every code, its uniforms are uniform."""
    codes = np.arange(127)
    k, f, step = R.grid(R.decode_e4m3(codes))
    assert (f == 0).all() and (k * step == R.decode_e4m3(codes)).all()
    for u in R.uniforms(1 << 16, 3, 4, 5):
        assert abs(u.mean() - 0.5) < 5 * 0.289 / 256 and abs((u < 0.25).mean() - 0.25) < 5 * 0.433 / 256


# ------------------------------------------------------------------ cross entropy
def xent_args(**kw):
    a = dict(a=FAKE, lda=64, b=FAKE, ldb=64, M=8, N=100, K=64, sa=FAKE, sb=FAKE, rows=0, t=FAKE, bits=64, loss=FAKE, lse=FAKE,
             mean=FAKE, ws=FAKE, wsb=1 << 40)
    a.update(kw)
    return a


COMMON = [
    (dict(M=-1), SHAPE), (dict(N=0), SHAPE), (dict(K=0), SHAPE), (dict(K=24, lda=32, ldb=32), UNSUP),
    (dict(K=65552, lda=65552, ldb=65552), UNSUP), (dict(M=(1 << 20) + 1), UNSUP), (dict(M=1 << 20, K=1024, lda=1024, ldb=1024), UNSUP),
    (dict(N=1 << 31), UNSUP), (dict(bits=16), ENUM), (dict(a=None), NULL), (dict(b=None), NULL), (dict(t=None), NULL),
    (dict(lda=48), SHAPE), (dict(ldb=48), SHAPE), (dict(lda=72), UNSUP), (dict(ldb=72), UNSUP), (dict(lda=(1 << 22) + 16), UNSUP), (dict(ldb=(1 << 22) + 16), UNSUP),
    (dict(a=FAKE + 8), UNSUP), (dict(b=FAKE + 8), UNSUP), (dict(t=FAKE + 4), ARG), (dict(bits=32, t=FAKE + 2), ARG),
    (dict(sa=FAKE + 2), ARG), (dict(sb=FAKE + 1), ARG), (dict(ws=None), NULL), (dict(wsb=100), ARG), (dict(ws=FAKE + 8), ARG),
]


@pytest.mark.parametrize("kw,status", COMMON + [
    (dict(rows=4), ENUM), (dict(rows=-1), ENUM), (dict(rows=1, sa=None), NULL), (dict(rows=2, sb=None), NULL),
    (dict(loss=None), NULL), (dict(lse=None), NULL), (dict(loss=FAKE + 2), ARG), (dict(lse=FAKE + 2), ARG), (dict(mean=FAKE + 2), ARG),
])
def test_cross_entropy_rejects(L, kw, status):
    assert L.fp8_cross_entropy(*xent_args(**kw).values(), None) == status
    assert L.fp8mi_last_error()


@pytest.mark.parametrize("kw,status", COMMON + [
    (dict(lse=None), NULL), (dict(dloss=None), NULL), (dict(dloss=FAKE + 2), ARG), (dict(lse=FAKE + 1), ARG), (dict(drows=2), ENUM),
    (dict(ld_da=63), SHAPE), (dict(ld_db=63), SHAPE), (dict(da=FAKE + 1), ARG), (dict(db=FAKE + 1), ARG),
])
def test_cross_entropy_grad_rejects(L, kw, status):
    a = xent_args(dloss=FAKE, drows=0, da=FAKE, ld_da=64, db=FAKE, ld_db=64)
    a.update(kw)
    order = ("a", "lda", "b", "ldb", "M", "N", "K", "sa", "sb", "t", "bits", "lse", "dloss", "drows", "da", "ld_da", "db", "ld_db",
             "ws", "wsb")
    assert L.fp8_cross_entropy_grad(*[a[k] for k in order], None) == status


def test_cross_entropy_workspaces(L):
    """Pure host functions: 0 where nothing runs, bounded by what they hold."""
    for f in (L.fp8_cross_entropy_workspace_bytes, L.fp8_cross_entropy_grad_workspace_bytes):
        assert f(0, 100, 64) == 0 and f(-1, 100, 64) == 0 and f(8, 0, 64) == 0 and f(8, 100, 24) == 0
        assert 0 < f(1, 1, 16) < 1 << 20
        for M, N, K in ((1, 32768, 1536), (4096, 65536, 1536), (8192, 131072, 4096), (100000, 1000, 64)):
            assert f(M, N, K) < 3 << 30
    assert L.fp8_cross_entropy_workspace_bytes(1, 32768, 1536) < 1 << 20  # a token's score needs no 16-bit operands


def test_binding_refuses_cross_entropy():
    a, b, t = torch.zeros(4, 32, dtype=torch.uint8), torch.zeros(9, 32, dtype=torch.uint8), torch.zeros(4, dtype=torch.int64)
    one = torch.ones(1)
    for args, kw, text in [
        ((a.float(), b, t), {}, "1-byte"), ((a, b[:, :16], t), {}, "K mismatch"), ((a, b, t[:3]), {}, "targets must be"),
        ((a, b, t.float()), {}, "targets must be"), ((a, b, t), dict(a_scale_inv=torch.ones(3)), "a_scale_inv"),
        ((a, b, t), dict(b_scale_inv=torch.ones(4)), "b_scale_inv"), ((a, b, t), dict(loss=torch.zeros(3)), "loss must be"),
        ((a, b, t), dict(lse=torch.zeros(4, dtype=torch.float64)), "lse must be"), ((a, b, t), dict(mean_out=one), "mean_out"),
        ((a.t(), b, t), {}, "unit column stride"),
    ]:
        with pytest.raises(ValueError, match=text):
            fp8mi.fp8_cross_entropy(*args, **kw)
    lse = torch.zeros(4)
    for kw, text in [
        (dict(a_scale_inv=torch.ones(4)), "no row scales"), (dict(b_scale_inv=torch.ones(9)), "no row scales"),
        (dict(da=torch.zeros(4, 32)), "da must be"), (dict(db=torch.zeros(9, 16, dtype=torch.bfloat16)), "db has shape"),
        (dict(dloss=torch.ones(3)), "dloss must be"), (dict(lse=torch.zeros(5)), "lse must be"),
    ]:
        args = dict(lse=lse, dloss=one)
        args.update(kw)
        with pytest.raises(ValueError, match=text):
            fp8mi.fp8_cross_entropy_grad(a, b, t, **args)
