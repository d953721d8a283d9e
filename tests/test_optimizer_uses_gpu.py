"""AdamW over params whose gradients are not always there, and a captured step's
8-bit states."""
import pytest
import torch

import fp8_tensor_scaled_quantize_amd as fp8mi
from fp8_tensor_scaled_quantize_amd.optim import AdamW

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


def rand(n, seed, dtype=torch.float32):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return torch.randn(n, generator=g, device=DEV).to(dtype)


@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("capturable", [False, True])
def test_a_late_param_counts_its_own_steps(bits, capturable):
    """A first update is lr times the gradient's sign, whatever the others' count: m /
    (1 - b1) and the root of v / (1 - b2) are g and |g|, each off by its few
    roundings (of 8-bit states the update takes the values before they are rounded)."""
    lr = 1e-3
    p = [rand(300, 1), torch.zeros(300, device=DEV), torch.zeros(300, device=DEV)]
    opt = AdamW(p, lr=lr, weight_decay=0.0, state_bits=bits, capturable=capturable)
    g = rand(300, 2) + 0.01
    for k in range(200):
        opt.step([rand(300, 10 + k), None, None])
    assert not p[1].any() and not p[2].any()
    opt.step([g, g, None])
    assert (p[1] + lr * torch.sign(g)).abs().max() <= 1e-4 * lr and not p[2].any()
    opt.step([None, None, g])
    assert (p[2] + lr * torch.sign(g)).abs().max() <= 1e-4 * lr
    # and so it is after the states went elsewhere
    q = [t.clone() for t in p]
    other = AdamW(q, lr=lr, weight_decay=0.0, state_bits=bits, capturable=capturable)
    other.load_state_dict(opt.state_dict())
    for k in range(3):
        grads = [rand(300, 50 + k), rand(300, 60 + k) if k else None, rand(300, 70 + k)]
        opt.step(grads)
        other.step(grads)
    assert all(torch.equal(x, y) for x, y in zip(p, q))
    assert opt.state_dict()["param_steps"] == [204, 3, 4] and other.state_dict()["param_steps"] == [204, 3, 4]


@pytest.mark.parametrize("bits", [32, 8])
def test_each_param_as_if_it_were_alone(bits):
    """Whether the others have gradients changes nothing in a param's own steps, the
    8-bit states' random numbers among them."""
    pattern = [(0, 1, 2), (1, 2), (0, 2), (2,), (1,), (0, 1, 2), (0, 1)]
    p = [rand(700 + i, i, torch.bfloat16) for i in range(3)]
    opt = AdamW(p, lr=1e-2, state_bits=bits, seed=5)
    alone = [[t.clone() for t in p] for _ in range(3)]
    opts = [AdamW(a, lr=1e-2, state_bits=bits, seed=5) for a in alone]
    for k, at in enumerate(pattern):
        grads = [rand(700 + i, 100 * k + i, torch.bfloat16) for i in range(3)]
        opt.step([g if i in at else None for i, g in enumerate(grads)])
        for i in at:
            opts[i].step(grads)  # all have gradients: only the i-th param is looked at
    for i in range(3):
        assert torch.equal(p[i], alone[i][i]) and torch.equal(opt.exp_avg[i], opts[i].exp_avg[i])
        assert torch.equal(opt.exp_avg_sq[i], opts[i].exp_avg_sq[i]) and torch.equal(opt.masters[i], opts[i].masters[i])


def test_a_state_of_one_count():
    """A state that holds one count for all, and a count that is set, reach every param."""
    p = [rand(300, 1), rand(20, 2)]
    opt = AdamW(p)
    opt.step([rand(300, 3), rand(20, 4)])
    state = {k: v for k, v in opt.state_dict().items() if k != "param_steps"}
    other = AdamW([t.clone() for t in p])
    other.load_state_dict(state)
    for o in (opt, other):
        o.step([rand(300, 5), None])
        assert o.steps == 2
    assert torch.equal(opt.params[0], other.params[0]) and opt.state_dict()["param_steps"] == [2, 1]
    opt.steps = 7
    assert opt.state_dict()["param_steps"] == [7, 7]


def test_a_captured_step_keeps_its_params():
    """Params that leave a captured step's rhythm are refused, before anything is
    written; a first step may be captured with some gradients missing."""
    p = [rand(300, 1), rand(300, 2)]
    twin = [t.clone() for t in p]
    opt, eager = AdamW(p, capturable=True), AdamW(twin, capturable=True)
    g = rand(300, 3)
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        opt.step([g, None])
    for _ in range(3):
        graph.replay()
        torch.cuda.synchronize()
        eager.step([g, None])
        assert all(torch.equal(x, y) for x, y in zip(p, twin))
    opt.step([None, g])  # its own count: untouched by the graph
    eager.step([None, g])
    assert torch.equal(p[1], twin[1]) and opt.state_dict()["param_steps"] == [3, 1]
    more = AdamW([rand(30, k) for k in range(3)], capturable=True)  # the rest may part at any time
    gs = [rand(30, 10 + k) for k in range(3)]
    more.step([None, *gs[1:]])
    torch.cuda.synchronize()
    with torch.cuda.graph(torch.cuda.CUDAGraph()):
        more.step([gs[0], None, None])
    more.step([None, None, gs[2]])
    assert more.state_dict()["param_steps"] == [0, 1, 2]
    more.load_state_dict(dict(more.state_dict(), param_steps=[5, 6, 6]))
    more.step(gs)
    assert more.state_dict()["param_steps"] == [6, 7, 7]
    both = AdamW([t.clone() for t in twin], capturable=True)
    both.step([g, g])
    torch.cuda.synchronize()
    with torch.cuda.graph(torch.cuda.CUDAGraph()):
        both.step([g, g])
    kept = [t.clone() for t in both.params]
    with pytest.raises(RuntimeError, match="captured"):
        both.step([g, None])
    with pytest.raises(ValueError, match="captured"):
        both.load_state_dict(opt.state_dict())
    with torch.cuda.graph(torch.cuda.CUDAGraph()):
        with pytest.raises(RuntimeError, match="captured"):
            both.step([None, g])
        g.clone()  # (an empty graph warns)
    assert all(torch.equal(x, y) for x, y in zip(kept, both.params)) and both.state_dict()["param_steps"] == [1, 1]


def test_a_bad_gradient_of_one_group_stops_all():
    p = [rand(300, 1), rand(20, 2)]
    opt = AdamW(p)
    opt.step([rand(300, 3), None])
    kept = [t.clone() for t in p]
    for bad in (rand(21, 4), rand(20, 4).double(), rand(20, 4).cpu()):
        with pytest.raises(ValueError):
            opt.step([rand(300, 3), bad])
        assert torch.equal(p[0], kept[0]) and opt.state_dict()["param_steps"] == [1, 0]


def test_captured_8_bit_states_are_the_eager_ones():
    """Codes and scales go by the gradients, the seed, the step and the clip alone: a
    replayed step's are an eager one's, bit for bit.  Weights: lr's quotient
    and the corrections in fp32 from the device's or the host's fp64, a rounding or
    two of the update apart."""
    def make():
        w = [rand(n, 7 + n) * 0.05 for n in (5000, 77)]
        return dict(w=w, p=[t.to(torch.bfloat16) for t in w], g=[rand(t.numel(), 9, torch.bfloat16) for t in w],
                    m=[torch.zeros(t.numel(), dtype=torch.uint8, device=DEV) for t in w],
                    v=[torch.zeros(t.numel(), dtype=torch.uint8, device=DEV) for t in w],
                    ms=[torch.zeros(-(-t.numel() // 256), device=DEV) for t in w],
                    vs=[torch.zeros(-(-t.numel() // 256), device=DEV) for t in w])

    def run(s, step, lr, clip):
        fp8mi.fp8_adamw_step(s["p"], s["g"], s["m"], s["v"], step, lr=lr, betas=(0.9, 0.95), weight_decay=0.1,
                             masters=s["w"], exp_avg_scales=s["ms"], exp_avg_sq_scales=s["vs"], grad_scale=clip, seed=3)

    a, b = make(), make()
    words = torch.zeros(fp8mi.ADAMW_STEP_WORDS, dtype=torch.int32, device=DEV)
    lr, clip = torch.empty(1, device=DEV), torch.empty(1, device=DEV)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        run(a, words, lr, clip)
    for t in range(1, 5):
        lr.fill_(3e-3 * t)
        clip.fill_(0.5 if t % 2 else 2.0)
        before = [w.clone() for w in b["w"]]
        graph.replay()
        torch.cuda.synchronize()
        run(b, t, float(lr), clip)
        assert int(words[0]) == t
        for name in ("m", "v", "ms", "vs"):
            assert all(torch.equal(x, y) for x, y in zip(a[name], b[name])), name
        for x, y, w, px, py in zip(a["w"], b["w"], before, a["p"], b["p"]):
            assert not torch.equal(y, w)  # there was a step
            # the step's factors differ by a half step each on either side, its update by 4 with the product's and the sum's
            assert ((x - y).abs() <= t * (4 * 2.0 ** -24 * (3 * float(lr) + w.abs()) + 2.0 ** -24 * w.abs())).all()
            assert torch.equal(px, x.to(torch.bfloat16)) and torch.equal(py, y.to(torch.bfloat16))
