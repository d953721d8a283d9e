"""Fp8Head, AdamW and a training step that runs them behind Fp8Mlp."""
import numpy as np
import pytest
import torch

import fp8_tensor_scaled_quantize_amd as fp8mi
import train_ref as R
from fp8_tensor_scaled_quantize_amd import interleave_gated
from fp8_tensor_scaled_quantize_amd.head import Fp8Head, fp8_head_loss
from fp8_tensor_scaled_quantize_amd.mlp import Fp8Mlp, fp8_mlp
from fp8_tensor_scaled_quantize_amd.optim import AdamW

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
HALF = 2.0 ** -8


def rand(*shape, sigma=1.0, dtype=torch.bfloat16, seed=0):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return (torch.randn(*shape, generator=g, device=DEV) * sigma).to(dtype)


def f64(t):
    return t.detach().cpu().double().numpy()


def head(d=64, vocab=300, dtype=torch.bfloat16, seed=0):
    return Fp8Head(1 + 0.1 * rand(d, dtype=torch.float32, seed=seed).to(dtype), rand(vocab, d, sigma=2 / d ** 0.5, dtype=dtype, seed=seed + 1))


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32, torch.float16])
@pytest.mark.parametrize("residual", [False, True])
def test_head_against_the_formulas(dtype, residual):
    """Loss and gradients from the codes that the norm and the quantize give
    (tested on their own), in 64 bits from there."""
    d, T = 64, 77
    hd = head(d, dtype=dtype)
    x = rand(T, d, dtype=dtype, seed=5)
    res = rand(T, d, dtype=dtype, seed=6) if residual else None
    t = torch.randint(-1, 300, (T,), device=DEV)
    hd.seed(x, res)
    rings = {k: r.clone() for k, r in hd.rings.items()}
    loss = hd.forward(x, t, res)
    g = hd.backward(torch.full((), 2.0, device=DEV))
    inv = [torch.empty(1, device=DEV) for _ in range(2)]
    rstd, h = torch.empty(T, device=DEV), torch.empty_like(x)
    nq = fp8mi.fp8_rmsnorm(x, hd.norm_weight, "e4m3", residual=res, ring=rings["n"], scale_inv_out=inv[0], rstd_out=rstd,
                           sum_out=h)
    wq = fp8mi.fp8_quantize(hd.weight, "e4m3", ring=rings["w"], scale_inv_out=inv[1])
    codes = nq.cpu().numpy(), wq.cpu().numpy()
    l = R.logits(*codes, float(inv[0]), float(inv[1]))
    _, _, mean = R.cross_entropy(l, t.cpu().numpy())
    # logits below 2^4 with 64-term sums: errors of 2^-24 * 2^7 each, a mean of them
    assert abs(float(loss) - mean[0]) <= 2.0 ** -16
    G = R.cross_entropy_grad(l, t.cpu().numpy(), 2.0 * mean[1])
    dn = G @ (R.decode_e4m3(codes[1]) * float(inv[1]))
    dw = G.T @ (R.decode_e4m3(codes[0]) * float(inv[0]))
    hh, r, w = f64(h) if residual else f64(x), f64(rstd)[:, None], f64(hd.norm_weight)
    gw = dn * w
    dx = r * gw - r ** 3 * (gw * hh).mean(1, keepdims=True) * hh
    dnw = (dn * hh * r).sum(0)
    # G and dn round to bf16 once each, dx and dw once more: independent half steps, in norm
    for got, want, roundings in ((g["x"], dx, 3), (g["weight"], dw, 2), (g["norm_weight"], dnw, 2)):
        assert np.linalg.norm(f64(got) - want) <= roundings * HALF * np.linalg.norm(want)


def test_head_on_the_tape_and_in_several_dimensions():
    hd = head()
    x, res = rand(2, 9, 64, seed=3).requires_grad_(), rand(18, 64, seed=4).requires_grad_()
    hd.norm_weight.requires_grad_()
    hd.weight.requires_grad_()
    t = torch.randint(0, 300, (2, 9), device=DEV)
    with torch.no_grad():
        hd.seed(x, res)
    kept = {k: r.clone() for k, r in hd.rings.items()}
    loss = fp8_head_loss(x, t, hd, res)
    (3 * loss).backward()
    for k, r in hd.rings.items():
        r.copy_(kept[k])
    with torch.no_grad():
        assert torch.equal(hd.forward(x, t, res), loss.detach())
        g = hd.backward(torch.full((), 3.0, device=DEV))
    assert torch.equal(x.grad, g["x"]) and torch.equal(res.grad, g["x"].reshape(18, 64))
    assert torch.equal(hd.weight.grad, g["weight"]) and torch.equal(hd.norm_weight.grad, g["norm_weight"].to(torch.bfloat16))


def test_head_refuses():
    hd = head()
    x, t = rand(4, 64), torch.zeros(4, dtype=torch.int64, device=DEV)
    with pytest.raises(RuntimeError, match="save_for_backward"):
        hd.backward(torch.ones((), device=DEV))
    with pytest.raises(RuntimeError, match="freeze"):
        hd.score(x, t)
    for bad in (rand(8, 32), rand(64)[:, None]):
        with pytest.raises(ValueError, match="must be"):
            hd.forward(bad, t)
    with pytest.raises(ValueError, match="targets for"):
        hd.forward(x, t[:3])
    rings = [r.clone() for r in hd.rings.values()]
    with pytest.raises(ValueError, match="targets must be"):
        hd.forward(x, t.float())
    assert all(torch.equal(a, b) for a, b in zip(rings, hd.rings.values()))  # refused before a ring has moved
    with pytest.raises(ValueError, match="multiple of 16"):
        Fp8Head(rand(40), rand(10, 40))
    with pytest.raises(ValueError, match="does not fit"):
        Fp8Head(hd.norm_weight, rand(10, 32))
    for change in (lambda: x.add_(1), lambda: t.add_(1), lambda: hd.norm_weight.add_(1)):
        hd.forward(x, t)
        change()
        with pytest.raises(RuntimeError, match="changed in place"):
            hd.backward(torch.ones((), device=DEV))
    a = fp8_head_loss(x.clone().requires_grad_(), t, hd)
    hd.forward(x, t)
    with pytest.raises(RuntimeError, match="another forward"):
        a.backward()


def test_targets_elsewhere_are_refused_before_a_ring_moves():
    hd = head()
    rings = [r.clone() for r in hd.rings.values()]
    with pytest.raises(ValueError, match="targets are on"):
        hd.forward(rand(4, 64), torch.zeros(4, dtype=torch.int64))
    assert all(torch.equal(a, b) for a, b in zip(rings, hd.rings.values()))


def test_no_rows_strided_targets_and_one_token():
    hd = head()
    hd.freeze()
    loss = hd.forward(rand(0, 64), torch.zeros(0, dtype=torch.int64, device=DEV))
    g = hd.backward(torch.ones((), device=DEV))
    assert float(loss) == 0 and g["x"].shape == (0, 64) and not g["weight"].any() and not g["norm_weight"].any()
    x, t = rand(6, 64, seed=3), torch.arange(12, device=DEV)
    assert torch.equal(hd.score(x, t[::2]), hd.score(x, t[::2].contiguous()))
    one = hd.score(x[0], t[4])
    assert one.shape == () and torch.equal(one, hd.score(x[:1], t[4:5])[0])


def test_score_in_a_graph_and_after_a_new_freeze():
    hd = head(vocab=1000)
    hd.freeze()
    x, t = rand(3, 64, seed=8), torch.tensor([5, -1, 999], device=DEV)
    want = hd.score(x, t)
    assert want.shape == (3,) and want[1] == 0
    # against the formula: the norm's codes and W's carry half a step of E4M3 each (2^-4 of a value), independent over
    # 64 terms: a logit of about 2 units is off by 2 * 2^-4 * a few
    h = f64(x)
    n = h / np.sqrt((h ** 2).mean(1, keepdims=True) + 1e-6) * f64(hd.norm_weight)
    exact, _, _ = R.cross_entropy(n @ f64(hd.weight).T, t.cpu().numpy())
    assert np.abs(f64(want) - exact).max() <= 0.5
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = hd.score(x, t)
    for k in range(3):
        x.copy_(rand(3, 64, seed=20 + k))
        hd.weight.mul_(1.1)
        hd.freeze()
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(got, hd.score(x, t))


def model(seed=0, vocab=500):
    d, f = 64, 96
    nw = 1 + 0.1 * rand(d, dtype=torch.float32, seed=seed)
    w = [rand(f, d, sigma=d ** -0.5, seed=seed + k) for k in (1, 2)]
    block = Fp8Mlp(nw, interleave_gated(*w), rand(d, f, sigma=f ** -0.5, seed=seed + 3), b_down=rand(d, sigma=0.1, seed=seed + 4),
                   act="silu", gated=True)
    hd = head(d, vocab, seed=seed + 5)
    params = [block.norm_weight, block.w_up, block.w_down, block.b_down, hd.norm_weight, hd.weight]
    for p in params:
        p.requires_grad_()
    return block, hd, params


@pytest.mark.parametrize("bits", [32, 8])
def test_training_steps(bits):
    """Block, head and optimizer together: each step's gradients are those of the
    parts called by hand, and its weights those of fp8_adamw_step on them."""
    (block, hd, params), (block2, hd2, params2) = model(), model()
    x, t = rand(37, 64, seed=30), torch.randint(-1, 500, (37,), device=DEV)
    decay = [0.0, 0.1, 0.1, 0.0, 0.0, 0.1]
    opt = AdamW(params, lr=1e-2, betas=(0.9, 0.95), weight_decay=decay, state_bits=bits, max_norm=0.5, seed=3)
    with torch.no_grad():
        for b, h in ((block, hd), (block2, hd2)):
            b.seed(x)
            h.seed(x)
    masters = [p.detach().float() if p.dtype != torch.float32 else None for p in params2]
    kind = torch.float32 if bits == 32 else torch.uint8
    m, v = ([torch.zeros(p.numel(), dtype=kind, device=DEV) for p in params2] for _ in range(2))
    ms, vs = ([torch.zeros(-(-p.numel() // 256), device=DEV) if bits == 8 else None for p in params2] for _ in range(2))
    for step in range(1, 4):
        loss = fp8_head_loss(fp8_mlp(x, block), t, hd)
        loss.backward()
        opt.step()
        with torch.no_grad():
            y = block2.forward(x)
            loss2 = hd2.forward(y, t)
            gh = hd2.backward(torch.ones((), device=DEV))
            gb = block2.backward(gh["x"])
            grads = [gb["norm_weight"], gb["w_up"], gb["w_down"], gb["b_down"], gh["norm_weight"].to(torch.bfloat16), gh["weight"]]
            clip = torch.empty(1, device=DEV)
            norm = fp8mi.fp8_grad_norm(grads, 0.5, clip_out=clip)
            fp8mi.fp8_adamw_step([p.detach() for p in params2], grads, m, v, step, lr=1e-2, betas=(0.9, 0.95),
                                 weight_decay=decay, masters=masters, exp_avg_scales=ms, exp_avg_sq_scales=vs,
                                 grad_scale=clip, seed=3)
        assert torch.equal(loss.detach(), loss2) and torch.equal(opt.norm, norm) and torch.isfinite(loss2)
        for p, q, g in zip(params, params2, grads):
            assert torch.equal(p.grad, g) and torch.equal(p.detach(), q.detach())
            assert g.abs().max() > 0
        opt.zero_grad()
        assert all(p.grad is None for p in params)


def test_a_whole_step_captured():
    """Forward, backward and optimizer in one graph: replays go on as eager steps do."""
    (block, hd, params), (block2, hd2, params2) = model(2), model(2)
    x, t = rand(32, 64, seed=31), torch.randint(0, 500, (32,), device=DEV)
    opts = [AdamW(p, lr=1e-2, max_norm=1.0, capturable=True) for p in (params, params2)]

    def step(b, h, o):
        loss = h.forward(b.forward(x), t)
        gh = h.backward(torch.ones((), device=DEV))
        gb = b.backward(gh["x"])
        o.step([gb["norm_weight"], gb["w_up"], gb["w_down"], gb["b_down"], gh["norm_weight"], gh["weight"]])
        return loss

    with torch.no_grad():
        for b, h, o in ((block, hd, opts[0]), (block2, hd2, opts[1])):
            b.seed(x)
            h.seed(x)
            step(b, h, o)  # the seeded first backward synchronises nothing, but runs once outside the graph
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            loss = step(block, hd, opts[0])
        for k in range(3):
            x.copy_(rand(32, 64, seed=40 + k))
            torch.cuda.synchronize()
            graph.replay()
            torch.cuda.synchronize()
            assert torch.equal(loss, step(block2, hd2, opts[1]))
            torch.cuda.synchronize()
            assert all(torch.equal(p, q) for p, q in zip(params, params2))
    assert int(opts[0].step_words[0]) == 4


def test_optimizer_state_goes_on_elsewhere():
    g = [rand(300, seed=k) for k in range(4)]
    for bits in (32, 8):
        a, b, c = (rand(300, seed=9) for _ in range(3))
        whole, first, second = (AdamW([p], state_bits=bits) for p in (a, b, c))
        for k in range(4):
            whole.step([g[k]])
        for k in range(2):
            first.step([g[k]])
        c.copy_(b)
        second.load_state_dict(first.state_dict())
        for k in range(2, 4):
            second.step([g[k]])
        assert torch.equal(a, c)
    with pytest.raises(ValueError, match="do not fit"):
        AdamW([a], state_bits=32).load_state_dict(whole.state_dict())


def test_optimizer_refuses_and_skips():
    with pytest.raises(ValueError, match="no params"):
        AdamW([])
    p = [rand(10, seed=1), rand(20, seed=2)]
    with pytest.raises(ValueError, match="state_bits"):
        AdamW(p, state_bits=16)
    with pytest.raises(ValueError, match="weight decays"):
        AdamW(p, weight_decay=[0.1])
    opt = AdamW(p, max_norm=1.0)
    with pytest.raises(ValueError, match="gradients for"):
        opt.step([p[0]])
    kept = [q.clone() for q in p]
    opt.step([None, None])
    assert opt.steps == 0
    bad = rand(20)
    bad[3] = float("inf")
    opt.step([rand(10), bad])
    assert all(torch.equal(a, b) for a, b in zip(p, kept))  # a gradient that is not finite: skipped
    opt.step([None, rand(20)])
    assert torch.equal(p[0], kept[0]) and not torch.equal(p[1], kept[1])
    with pytest.raises(ValueError, match="twice"):
        AdamW([p[0], p[0]]).step([rand(10), rand(10)])
    p[1].zero_()
    opt.sync_masters()
    assert not opt.masters[1].any()
