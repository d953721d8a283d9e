"""Fp8Mlp: the feed-forward block that the norm, the fused-epilogue products
and their gradients make together -- training through autograd, HIP graph
replays, and serving -- against the block in fp64.

Bounds: one E4M3 rounding is off by at most 2^-4 of a value, 0.026 of it in the
2-norm, one E5M2 rounding twice that; errors of independent tensors add in
squares.  u carries n's and W_up's (0.037), y - h those of u, W_down and of u's
own error (0.052, times the activation's slope near 1): 0.08.  Gradients add
E5M2 roundings of dY and dZ (0.053 each) to three or four of E4M3's: 0.16."""
import pytest
import torch

from tests import block_ref as R
from tests.gpu_util import DEV

pytestmark = pytest.mark.gpu
fp8mi = pytest.importorskip("fp8_tensor_scaled_quantize_amd")
from fp8_tensor_scaled_quantize_amd.mlp import Fp8Mlp, fp8_mlp  # noqa: E402

BF = torch.bfloat16
Y_BOUND, G_BOUND = 0.08, 0.16


def make(d, f, act, gated, bias):
    n = 2 * f if gated else f
    nw = (1 + R.rand((d,), 0.1, torch.float32, 1)).to(BF)
    wu, wd = R.rand((n, d), d ** -0.5, BF, 2), R.rand((d, f), f ** -0.5, BF, 3)
    bu = R.rand((n,), 0.1, BF, 4) if bias else None
    bd = R.rand((d,), 0.1, BF, 5) if bias else None
    cpu = [nw, wu, wd, bu, bd]
    dev = [None if t is None else t.to(DEV) for t in cpu]
    return cpu, dev, Fp8Mlp(dev[0], dev[1], dev[2], dev[3], dev[4], act, gated, 1e-6, 4)


def reference(cpu, x, res, act, gated):
    nw, wu, wd, bu, bd = (None if t is None else t.double().requires_grad_() for t in cpu)
    x = x.double().requires_grad_()
    h = x if res is None else x + res.double()
    n = h / torch.sqrt((h * h).mean(-1, keepdim=True) + 1e-6) * nw
    t = n @ wu.t() + (0 if bu is None else bu)
    u = R.act(t[..., 0::2], act)[0] * t[..., 1::2] if gated else R.act(t, act)[0]
    return u @ wd.t() + (0 if bd is None else bd) + h, h, (x, nw, wu, wd, bu, bd)


def off(a, b):
    a, b = a.detach().cpu().double(), b.detach().double()
    return float((a - b).norm() / b.norm())


@pytest.mark.parametrize("d,f,act,gated,bias", [(256, 512, "gelu", False, True), (512, 688, "silu", True, False),
                                                (1536, 6912, "silu", False, True), (128, 320, "relu", True, True)])
def test_training_step(d, f, act, gated, bias):
    """Values and gradients after the rings have seen the data once."""
    print(f"mlp {d}x{f} {act} gated={gated}", flush=True)
    cpu, dev, block = make(d, f, act, gated, bias)
    x, res, dy = R.rand((3, 48, d), 1.0, BF, 6), R.rand((3, 48, d), 1.0, BF, 7), R.rand((3, 48, d), 1e-2, BF, 8)
    xd, rd, dyd = x.to(DEV).requires_grad_(), res.to(DEV).requires_grad_(), dy.to(DEV)
    for t in dev:
        if t is not None:
            t.requires_grad_()
    for step in range(2):  # the first step runs at scale 1 and fills the rings
        for t in (xd, rd, *dev):
            if t is not None:
                t.grad = None
        y = fp8_mlp(xd, block, rd)
        y.backward(dyd)
    torch.cuda.synchronize()
    want, h, leaves = reference(cpu, x, res, act, gated)
    want.backward(dy.double())
    assert off(y - (xd + rd), want - h) < Y_BOUND
    assert off(xd.grad, leaves[0].grad) < G_BOUND and torch.equal(xd.grad, rd.grad)
    for got, ref in zip(dev, leaves[1:]):
        if got is not None:
            assert off(got.grad, ref.grad) < G_BOUND, tuple(got.shape)


def test_backward_needs_the_latest_forward():
    _, _, block = make(128, 256, "gelu", False, False)
    with pytest.raises(RuntimeError, match="needs a forward"):
        block.backward(torch.zeros(16, 128, dtype=BF, device=DEV))
    x = R.rand((16, 128), 1.0, BF, 9).to(DEV).requires_grad_()
    y = fp8_mlp(x, block)
    block.forward(x.detach())
    with pytest.raises(RuntimeError, match="another forward"):
        y.backward(torch.ones_like(y))


def test_weights_must_fit():
    w = torch.zeros
    with pytest.raises(ValueError):
        Fp8Mlp(w(16, device=DEV), w(32, 16, device=DEV), w(16, 31, device=DEV))
    with pytest.raises(ValueError):
        Fp8Mlp(w(16, device=DEV), w(32, 16, device=DEV), w(16, 32, device=DEV), gated=True)


@pytest.mark.parametrize("tokens", [1, 7, 40])
def test_decode(tokens):
    """Serving steps, eager and from a graph, on a residual stream in place."""
    d, f = 512, 1376
    cpu, dev, block = make(d, f, "silu", True, False)
    with pytest.raises(RuntimeError, match="freeze"):
        block.decode(torch.zeros(1, d, dtype=BF, device=DEV), torch.zeros(1, d, dtype=BF, device=DEV))
    block.freeze()
    for k in range(2):
        block.calibrate(R.rand((64, d), 1.0, BF, 20 + k).to(DEV), R.rand((64, d), 1.0, BF, 30 + k).to(DEV))
    x, res = torch.empty(tokens, d, dtype=BF, device=DEV), torch.empty(tokens, d, dtype=BF, device=DEV)
    x0, r0 = R.rand((tokens, d), 1.0, BF, 40), R.rand((tokens, d), 1.0, BF, 41)
    graph = torch.cuda.CUDAGraph()
    x.copy_(x0), res.copy_(r0)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        block.decode(x, res)
    torch.cuda.synchronize()
    want, h, _ = reference(cpu, x0, r0, "silu", True)
    assert off(res - (x0.to(DEV) + r0.to(DEV)), want - h) < Y_BOUND
    with torch.cuda.graph(graph):
        block.decode(x, res)
    for k in range(3):
        a, b = R.rand((tokens, d), 1.0, BF, 50 + k).to(DEV), R.rand((tokens, d), 1.0, BF, 60 + k).to(DEV)
        x.copy_(a), res.copy_(b)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        eager = b.clone()
        block.decode(a, eager)
        torch.cuda.synchronize()
        assert torch.equal(res, eager), f"replay {k}"


def test_training_step_in_a_graph():
    """A whole step captured; replays equal eager steps of a second block."""
    d, f, rows = 256, 512, 160
    _, _, a = make(d, f, "gelu", False, True)
    _, _, b = make(d, f, "gelu", False, True)
    x, dy = torch.empty(rows, d, dtype=BF, device=DEV), torch.empty(rows, d, dtype=BF, device=DEV)
    x.copy_(R.rand((rows, d), 1.0, BF, 70)), dy.copy_(R.rand((rows, d), 1e-2, BF, 71))

    def step(block):
        y = block.forward(x)
        return [y, *(t for t in block.backward(dy).values() if t is not None)]

    step(a), step(b)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step(a)
    for k in range(3):
        x.copy_(R.rand((rows, d), 1.0 + k, BF, 72 + k)), dy.copy_(R.rand((rows, d), 1e-2, BF, 80 + k))
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        want = step(b)
        torch.cuda.synchronize()
        for u, v in zip(out, want):
            assert torch.equal(u, v), f"replay {k}"
        for name in a.rings:
            assert torch.equal(a.rings[name], b.rings[name]), (k, name)
