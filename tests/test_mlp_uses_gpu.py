"""Fp8Mlp in the orders and shapes that a program uses it in: serving between a
forward and its backward, tensors changed under a pending backward, any token
count, weights frozen again under a captured decode, first steps of a fresh
block.

Bounds as in test_mlp_gpu.py: 0.08 of a value's 2-norm for outputs, 0.16 for
gradients; equal call sequences have to give equal bits."""
import pytest
import torch

from tests import block_ref as R
from tests.gpu_util import DEV
from tests.test_mlp_gpu import BF, G_BOUND, Y_BOUND, make, off, reference

pytestmark = pytest.mark.gpu
fp8mi = pytest.importorskip("fp8_tensor_scaled_quantize_amd")
from fp8_tensor_scaled_quantize_amd.mlp import Fp8Mlp, fp8_mlp  # noqa: E402


def batch(rows, d, seed, sigma=1.0):
    return R.rand((rows, d), sigma, BF, seed).to(DEV)


def same(got, want):
    torch.cuda.synchronize()
    for name, g in got.items():
        assert (g is None) == (want[name] is None), name
        assert g is None or torch.equal(g, want[name]), name


@pytest.mark.parametrize("act,gated", [("gelu", False), ("silu", True)])
def test_decode_between_forward_and_backward(act, gated):
    """Serving steps leave a pending backward as it was."""
    d, f = 256, 512
    _, _, a = make(d, f, act, gated, True)
    _, _, b = make(d, f, act, gated, True)
    x, dy, tok = batch(48, d, 1), batch(48, d, 2, 1e-2), batch(3, d, 3)
    a.freeze()
    for step in range(2):  # a fresh block's scales are far from each other, later ones nearly equal
        a.forward(x), b.forward(x)
        a.decode(tok, tok.clone())
        same(a.backward(dy), b.backward(dy))


@pytest.mark.parametrize("what", ["x", "norm_weight"])
@pytest.mark.parametrize("tape", [False, True])
def test_in_place_change_before_backward(what, tape):
    """What backward reads again must be as forward saw it."""
    _, dev, block = make(128, 256, "gelu", False, False)
    x, dy = batch(32, 128, 4), batch(32, 128, 5)
    if tape:
        leaf = x.clone().requires_grad_()
        x = leaf * 1  # a stream that its owner may update
        y = fp8_mlp(x, block)
    else:
        y = block.forward(x)
    with torch.no_grad():
        (x if what == "x" else dev[0]).add_(0.25)
    with pytest.raises(RuntimeError, match="changed in place"):
        y.backward(dy) if tape else block.backward(dy)


@pytest.mark.parametrize("how", ["decode", "rmsnorm", "mm_act", "rmsnorm_grad"])
def test_in_place_change_by_the_library(how):
    """The library's own in-place forms count as changes too."""
    d = 128
    _, dev, block = make(d, 256, "gelu", False, False)
    x, other, dy = batch(32, d, 6), batch(32, d, 7), batch(32, d, 8)
    block.freeze()
    block.forward(x)
    one = torch.ones(1, device=DEV)
    if how == "decode":
        block.decode(other, x)
    elif how == "rmsnorm":
        fp8mi.fp8_rmsnorm(other, None, residual=x, scale=one, sum_out=x.view(32, d))
    elif how == "mm_act":
        a, b = torch.zeros(32, 64, dtype=torch.uint8, device=DEV), torch.zeros(d, 64, dtype=torch.uint8, device=DEV)
        fp8mi.fp8_mm_act(a, b, residual=x, out=x)
    else:
        fp8mi.fp8_rmsnorm_grad(other, dy, None, torch.ones(32, device=DEV), dsum=x, dx=x, need_dweight=False)
    torch.cuda.synchronize()
    with pytest.raises(RuntimeError, match="changed in place"):
        block.backward(dy)


def test_residual_sum_is_the_blocks_own():
    """With a residual the saved sum is the block's: x and residual may go."""
    _, _, a = make(128, 256, "gelu", False, False)
    _, _, b = make(128, 256, "gelu", False, False)
    x, r, dy = batch(32, 128, 9), batch(32, 128, 10), batch(32, 128, 11, 1e-2)
    a.forward(x.clone(), r.clone())
    b.forward(x, r)
    x.zero_(), r.zero_()
    same(b.backward(dy), a.backward(dy))


@pytest.mark.parametrize("tokens", [0, 1, 7, 40, 250])
@pytest.mark.parametrize("act,gated,bias", [("gelu", False, True), ("silu", True, False)])
def test_any_token_count(tokens, act, gated, bias):
    d, f = 256, 512
    cpu, dev, block = make(d, f, act, gated, bias)
    x, res, dy = R.rand((tokens, d), 1.0, BF, 12), R.rand((tokens, d), 1.0, BF, 13), R.rand((tokens, d), 1e-2, BF, 14)
    xd, rd = x.to(DEV).requires_grad_(), res.to(DEV).requires_grad_()
    for t in dev:
        if t is not None:
            t.requires_grad_()
    print(f"mlp tokens {tokens} {act} gated={gated}", flush=True)
    for step in range(2):  # the first step fills the rings
        for t in (xd, rd, *dev):
            if t is not None:
                t.grad = None
        y = fp8_mlp(xd, block, rd)
        y.backward(dy.to(DEV))
    torch.cuda.synchronize()
    want, h, leaves = reference(cpu, x, res, act, gated)
    want.backward(dy.double())
    if tokens == 0:
        assert xd.grad.shape == (0, d) and all(t is None or not t.grad.any() for t in dev)
        return
    assert off(y - (xd + rd), want - h) < Y_BOUND
    assert off(xd.grad, leaves[0].grad) < G_BOUND and torch.equal(xd.grad, rd.grad)
    for got, ref in zip(dev, leaves[1:]):
        if got is not None:
            assert off(got.grad, ref.grad) < G_BOUND, tuple(got.shape)


def test_training_refusals_come_first():
    """What a backward cannot take is refused before a ring has moved."""
    d = 128
    _, _, block = make(d, 256, "gelu", False, True)
    x, dy = batch(16, d, 15), batch(16, d, 16)
    block.forward(x)
    rings = {k: r.clone() for k, r in block.rings.items()}
    for t in (dy.float(), dy.half(), dy[:8], dy.reshape(32, 64)):
        with pytest.raises(ValueError, match="dy"):
            block.backward(t)
    for k, r in block.rings.items():
        assert torch.equal(r, rings[k]), k


@pytest.mark.parametrize("dt", [torch.float16, torch.float32])
@pytest.mark.parametrize("with_res", [False, True])
@pytest.mark.parametrize("tokens", [40, 48])
def test_streams_of_other_types(dt, with_res, tokens):
    """fp16 and fp32 x (and residual): the output is bf16, dx has x's type.
    Gradients of 1e-6, where fp16 has steps of 2^-24: dx's own rounding, half a
    step an element, is in its bound."""
    d, f, sigma = 256, 512, 1e-6
    cpu, dev, block = make(d, f, "gelu", False, True)
    x, dy = R.rand((tokens, d), 1.0, dt, 59), R.rand((tokens, d), sigma, BF, 61)
    res = R.rand((tokens, d), 1.0, dt, 60) if with_res else None
    xd, rd = x.to(DEV).requires_grad_(), None if res is None else res.to(DEV)
    for t in dev:
        t.requires_grad_()
    block.seed(xd.detach(), rd)
    y = fp8_mlp(xd, block, rd)
    y.backward(dy.to(DEV))
    torch.cuda.synchronize()
    want, h, leaves = reference(cpu, x, res, "gelu", False)
    want.backward(dy.double())
    assert y.dtype == BF and xd.grad.dtype == dt
    assert off(y.double().cpu() - h, want - h) < Y_BOUND + 2.0 ** -9 * float((want.norm() / (want - h).norm()).detach())
    half = 2.0 ** -25 if dt is torch.float16 else 0.0
    assert off(xd.grad, leaves[0].grad) < G_BOUND + half * (tokens * d) ** 0.5 / float(leaves[0].grad.norm())
    for got, ref in zip(dev, leaves[1:]):
        assert off(got.grad, ref.grad) < G_BOUND, tuple(got.shape)


@pytest.mark.parametrize("bias", [False, True])
def test_linear_pair_without_activation(bias):
    """act="none" without gating trains as well: dz is dy."""
    d, f = 256, 512
    cpu, dev, block = make(d, f, "none", False, bias)
    x, dy = R.rand((48, d), 1.0, BF, 17), R.rand((48, d), 1e-2, BF, 18)
    for step in range(2):
        y = block.forward(x.to(DEV))
        got = block.backward(dy.to(DEV))
    torch.cuda.synchronize()
    want, h, leaves = reference(cpu, x, None, "none", False)
    want.backward(dy.double())
    assert off(y - x.to(DEV), want - h) < Y_BOUND
    for name, leaf in zip(("x", "norm_weight", "w_up", "w_down", "b_up", "b_down"), leaves):
        if leaf is not None:
            assert off(got[name], leaf.grad) < G_BOUND, name


def test_freeze_again_under_a_captured_decode():
    """New weights, frozen again, reach a decode captured before."""
    d, f, tokens = 256, 704, 5
    _, dev, block = make(d, f, "silu", True, False)
    block.freeze()
    block.calibrate(batch(64, d, 19))
    at = [t.data_ptr() for pair in block._frozen for t in pair]
    x, res = batch(tokens, d, 20), batch(tokens, d, 21)
    block.decode(x, res)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        block.decode(x, res)
    for k in range(3):
        dev[1].copy_(R.rand(dev[1].shape, (1 + k) * d ** -0.5, BF, 22 + k))
        dev[2].copy_(R.rand(dev[2].shape, f ** -0.5, BF, 25 + k))
        block.freeze()
        assert at == [t.data_ptr() for pair in block._frozen for t in pair]
        a, b = batch(tokens, d, 28 + k), batch(tokens, d, 31 + k)
        x.copy_(a), res.copy_(b)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        block.decode(a, b)
        torch.cuda.synchronize()
        assert torch.equal(res, b), k


@pytest.mark.parametrize("frozen", [False, True])
def test_one_calibration_of_small_weights(frozen):
    """One calibrate call on weights far below E4M3's range at scale 1, taken
    back by the down-projection's."""
    d, f = 512, 1376
    cpu, dev, block = make(d, f, "silu", True, False)
    cpu[1], cpu[2] = R.rand((2 * f, d), 1e-4, BF, 34), R.rand((d, f), 1e4, BF, 35)
    block = Fp8Mlp(dev[0], cpu[1].to(DEV), cpu[2].to(DEV), None, None, "silu", True, 1e-6, 4)
    if frozen:
        block.freeze()
    block.calibrate(batch(64, d, 36), batch(64, d, 37))
    block.freeze()
    x, res = R.rand((7, d), 1.0, BF, 38), R.rand((7, d), 1.0, BF, 39)
    got = block.decode(x.to(DEV), res.to(DEV))
    torch.cuda.synchronize()
    want, h, _ = reference(cpu, x, res, "silu", True)
    # the residual stream's one bf16 rounding (2^-9 of |y|) is in the bound too
    assert off(got - (x.to(DEV) + res.to(DEV)), want - h) < Y_BOUND + 2.0 ** -9 * float((want.norm() / (want - h).norm()).detach())


def test_calibrate_leaves_training_alone():
    d = 128
    _, _, block = make(d, 256, "gelu", False, False)
    _, _, twin = make(d, 256, "gelu", False, False)
    x, dy = batch(32, d, 40), batch(32, d, 41, 1e-2)
    block.forward(x), twin.forward(x)
    before = {k: r.clone() for k, r in block.rings.items()}
    block.calibrate(batch(16, d, 42))
    for k, r in block.rings.items():
        assert torch.equal(r, before[k]) == (k != "u"), k
    same(block.backward(dy), twin.backward(dy))


@pytest.mark.parametrize("act,gated,bias", [("gelu", False, True), ("silu", True, False), ("none", False, False)])
def test_seeded_first_step(act, gated, bias):
    """After seed() the first step has its values and its gradients, dy far
    below what E5M2 holds at scale 1 (2^-17) included, and the next one too."""
    d, f = 256, 512
    cpu, dev, block = make(d, f, act, gated, bias)
    x, res, dy = R.rand((48, d), 1.0, BF, 43), R.rand((48, d), 1.0, BF, 44), R.rand((48, d), 1e-6, BF, 45)
    want, h, leaves = reference(cpu, x, res, act, gated)
    want.backward(dy.double())
    block.seed(x.to(DEV), res.to(DEV))
    for step in range(2):
        y = block.forward(x.to(DEV), res.to(DEV))
        got = block.backward(dy.to(DEV))
        torch.cuda.synchronize()
        assert off(y - (x.to(DEV) + res.to(DEV)), want - h) < Y_BOUND
        # x's gradient holds dy itself: the block's own share of it, and one bf16 rounding
        share = leaves[0].grad - dy.double()
        assert off(got["x"] - dy.to(DEV), share) < G_BOUND + 2.0 ** -8 * float(leaves[0].grad.norm() / share.norm())
        for name, leaf in zip(("norm_weight", "w_up", "w_down", "b_up", "b_down"), leaves[1:]):
            if leaf is not None:
                assert off(got[name], leaf.grad) < G_BOUND, (step, name)


def test_forward_without_backward_equals_the_saved_one():
    _, _, a = make(256, 512, "silu", True, True)
    _, _, b = make(256, 512, "silu", True, True)
    for k in range(3):
        x = batch(40, 256, 46 + k)
        assert torch.equal(a.forward(x, save_for_backward=False), b.forward(x)), k
        for name in a.rings:
            assert torch.equal(a.rings[name], b.rings[name]), (k, name)


def test_widths_and_types_are_checked_first():
    d = 128
    _, _, block = make(d, 256, "gelu", False, False)
    block.freeze()
    x = batch(8, 2 * d, 50)
    for call in (lambda: block.forward(x), lambda: block.calibrate(x), lambda: fp8_mlp(x, block),
                 lambda: block.forward(batch(8, d, 51), batch(8, 2 * d, 52)), lambda: block.seed(x),
                 lambda: block.decode(x, x.clone())):
        with pytest.raises(ValueError):
            call()
    h = batch(8, d, 62)  # a width given as several dimensions is one
    assert torch.equal(block.forward(h.view(2, 4, 8, d // 8)).view(8, d), make(d, 256, "gelu", False, False)[2].forward(h))
    assert block.backward(h)["x"].shape == (2, 4, 8, d // 8)
    for dt in (torch.float16, torch.float32):
        a, r = batch(3, d, 53).to(dt), batch(3, d, 54).to(dt)
        keep = r.clone()
        with pytest.raises(ValueError, match="bfloat16"):
            block.decode(a, r)
        torch.cuda.synchronize()
        assert torch.equal(r, keep)


def test_a_freeze_that_fails_leaves_no_weights():
    d = 128
    _, dev, block = make(d, 256, "gelu", False, False)
    block.w_down = dev[2].double()
    with pytest.raises(ValueError):
        block.freeze()
    with pytest.raises(RuntimeError, match="freeze"):
        block.decode(batch(3, d, 55), batch(3, d, 56))


def test_a_forward_that_fails_ends_the_pending_backward():
    """It has replaced some of the multipliers that the backward would read."""
    d = 128
    _, dev, block = make(d, 256, "gelu", False, False)
    x, dy = batch(16, d, 57), batch(16, d, 58)
    block.forward(x)
    block.w_down = dev[2].double()
    with pytest.raises(ValueError):
        block.forward(4 * x)
    with pytest.raises(RuntimeError, match="needs a forward"):
        block.backward(dy)


def test_residual_of_another_leading_shape():
    d = 128
    _, _, block = make(d, 256, "gelu", False, False)
    x, r = batch(32, d, 63).view(2, 16, d).requires_grad_(), batch(32, d, 64).requires_grad_()
    fp8_mlp(x, block, r).backward(batch(32, d, 65).view(2, 16, d))
    torch.cuda.synchronize()
    assert r.grad.shape == (32, d) and torch.equal(x.grad.view(32, d), r.grad)
