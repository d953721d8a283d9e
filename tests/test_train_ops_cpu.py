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


def test_binding_refuses_lists():
    f32 = lambda n=4: torch.zeros(n)  # noqa: E731

    def step(p=None, g=None, m=None, v=None, t=1, **kw):
        fp8mi.fp8_adamw_step(p or [f32()], g or [f32()], m or [f32()], v or [f32()], t, **kw)

    for kw, text in [
        (dict(g=[f32(5)]), "elements"), (dict(g=[f32(), f32()]), "grads for"), (dict(m=[f32(3)]), "elements"),
        (dict(p=[torch.zeros(4, 4).t()], g=[f32(16)], m=[f32(16)], v=[f32(16)]), "contiguous"),
        (dict(p=[torch.zeros(4, dtype=torch.int32)]), "params must be"), (dict(g=[torch.zeros(4, dtype=torch.uint8)]), "grads must be"),
        (dict(m=[torch.zeros(4, dtype=torch.bfloat16)]), "float32, or codes"), (dict(masters=[]), "one entry per"),
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
