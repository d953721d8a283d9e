"""Cases of what a training step of the fp8 layers ends with: the softmax cross
entropy over a vocabulary from the head's E4M3 operands, its gradient, the
norm of all gradients and the AdamW step over many tensors, with states in 32
or in 8 bits.  Sizes follow the 1.2B-model linears of this repository's
configurations (hidden 1536, feed-forward 6912) and generic vocabularies, from
the scoring of a single token to training steps.

`run` computes a case in plain torch operations in 32 bits, or, where `own` is
true, by the framework's operators.  8-bit states are returned as float8
tensors next to their blocks' multipliers."""
from __future__ import annotations

import math

import torch

own = False

DT = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
EB = {"bf16": 2, "f16": 2, "f32": 4}
E4M3 = torch.float8_e4m3fn
E4M3_MAX = 448.0
BLOCK = 256  # elements of an 8-bit state that share a scale
LR, BETA1, BETA2, EPS, DECAY = 3e-4, 0.9, 0.95, 1e-8, 0.1
SEED = 20240229  # of the 8-bit states' rounding
MAX_NORM = 1.0
HIDDEN, FFN = 1536, 6912


def listed():
    ce = dict(op="ce", K=HIDDEN, ignored=0.0, row_scales=False)
    grad = dict(op="ce_grad", K=HIDDEN, ignored=0.0, weights=False)
    opt = dict(op="adamw", grad="bf16", shapes="block", clip=False)
    return [
        # scoring of one new token while serving, codes as a row-scaled norm gives them
        dict(ce, name="ce 1x32768x1536 score", M=1, N=32768, row_scales=True),
        # a ragged batch of prompts, odd vocabulary, a third of the positions masked out of the loss
        dict(ce, name="ce 333x50001x1536 masked", M=333, N=50001, ignored=0.34),
        # the training step's loss
        dict(ce, name="ce 4096x65536x1536 train", M=4096, N=65536),
        # a small classifier's or a toy model's gradient: launch latency counts
        dict(grad, name="ce grad 64x1000x512", M=64, N=1000, K=512),
        # a ragged batch with weighted, partly masked tokens and an odd vocabulary
        dict(grad, name="ce grad 1111x50001x1536 weighted", M=1111, N=50001, ignored=0.2, weights=True),
        # the training step's gradient
        dict(grad, name="ce grad 4096x65536x1536 train", M=4096, N=65536),
        # norm weights and biases of a few blocks in fp32: small tensors, launch latency counts
        dict(opt, name="adamw 24 vectors f32", param="f32", grad="f32", master=False, bits=32, shapes="vectors", count=24),
        # one feed-forward block, bf16 weights with fp32 masters, clipped
        dict(opt, name="adamw 1 block master", param="bf16", master=True, bits=32, count=1, clip=True),
        # ragged tensors in fp16 with 8-bit states
        dict(opt, name="adamw 9 ragged f16 8-bit", param="f16", grad="f16", master=False, bits=8, shapes="ragged", count=9),
        # eight blocks with 8-bit states and fp32 masters
        dict(opt, name="adamw 8 blocks 8-bit", param="bf16", master=True, bits=8, count=8),
        # the norm of a few small gradients
        dict(op="grad_norm", name="grad norm 24 vectors f32", grad="f32", shapes="vectors", count=24),
        # the norm of eight blocks' gradients
        dict(op="grad_norm", name="grad norm 8 blocks", grad="bf16", shapes="block", count=8),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["ce", "ce", "ce_grad", "ce_grad", "adamw", "adamw", "grad_norm"])
    if op in ("ce", "ce_grad"):
        K = 16 * _log(rng, 4, 256)
        N = _log(rng, 2, 65536)
        M = _log(rng, 1, max(2, min(8192, 4096 * 65536 * 1536 // (N * K))))
        case = dict(op=op, M=M, N=N, K=K, ignored=rng.choice([0.0, 0.0, 0.3]))
        if op == "ce":
            case["row_scales"] = rng.random() < 0.4
        else:
            case["weights"] = rng.random() < 0.4
        return case
    shapes = rng.choice(["vectors", "ragged", "block"])
    count = rng.randint(1, 8) if shapes == "block" else _log(rng, 1, 100)
    case = dict(op=op, grad=rng.choice(["bf16", "bf16", "f16", "f32"]), shapes=shapes, count=count)
    if op == "adamw":
        case.update(param=rng.choice(["bf16", "f16", "f32"]), bits=rng.choice([8, 32]), clip=rng.random() < 0.4)
        case["master"] = case["param"] != "f32" and rng.random() < 0.7
    return case


def _sizes(case):
    """The tensors' element counts."""
    n = case["count"]
    if case["shapes"] == "vectors":
        return [(HIDDEN, FFN, HIDDEN + 1, 1)[i % 4] for i in range(n)]
    if case["shapes"] == "ragged":  # from tiny to a few millions, no two alike
        return [1 + (i * i * 7919 + 17 * i + 3) * (1 + 200 * (i % 3)) % 3000017 for i in range(n)]
    return [s for _ in range(n) for s in (HIDDEN, FFN * HIDDEN, FFN, HIDDEN * FFN, HIDDEN)]


# ------------------------------------------------------------------ inputs
def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    return g


def _randn(g, *shape, sigma=1.0):
    return torch.randn(*shape, generator=g, device="cuda") * sigma


def _codes(v):
    """E4M3 codes of a matrix at its own scale, and 1 / scale."""
    s = E4M3_MAX / v.abs().amax()
    return (v * s).clamp(-E4M3_MAX, E4M3_MAX).to(E4M3).view(torch.uint8), (1 / s).reshape(1)


def _views(flat, sizes):
    return list(flat.split(sizes))


def prepare(case, seed):
    g = _gen(seed)
    s = {"case": case}
    if case["op"] in ("ce", "ce_grad"):
        M, N, K = case["M"], case["N"], case["K"]
        # a head part-way through training: hidden rows lean towards their target's weights
        w = _randn(g, N, K, sigma=2.0 / math.sqrt(K))
        t = torch.randint(0, N, (M,), generator=g, device="cuda")
        x = _randn(g, M, K) + 4 * torch.nn.functional.normalize(w[t], dim=1) * torch.rand(M, 1, generator=g, device="cuda")
        s["a"], s["sa"] = _codes(x)
        s["b"], s["sb"] = _codes(w)
        if case.get("row_scales"):
            s["sa"] = s["sa"] * torch.exp(_randn(g, M, sigma=0.2))
            s["sb"] = s["sb"] * torch.exp(_randn(g, N, sigma=0.1))
        s["targets"] = torch.where(torch.rand(M, generator=g, device="cuda") < case["ignored"], -100, t)
        if case["op"] == "ce":
            s["loss"], s["lse"] = torch.empty(M, device="cuda"), torch.empty(M, device="cuda")
            s["mean"] = torch.empty(2, device="cuda")
        else:
            s["lse"] = _logits(s).logsumexp(1)
            count = (s["targets"] >= 0).sum().clamp(min=1).float()
            s["dloss"] = (torch.rand(M, generator=g, device="cuda") + 0.5) / count if case["weights"] else (1 / count).reshape(1)
            s["da"] = torch.empty(M, K, dtype=torch.bfloat16, device="cuda")
            s["db"] = torch.empty(N, K, dtype=torch.bfloat16, device="cuda")
        return s
    sizes = _sizes(case)
    total = sum(sizes)
    # every tensor's gradients at its own size, as layers' are
    size = torch.repeat_interleave(torch.exp(_randn(g, len(sizes))), torch.tensor(sizes, device="cuda"), output_size=total)
    s["flat_grad"] = (_randn(g, total, sigma=2e-3) * size).to(DT[case["grad"]])
    s["grads"] = _views(s["flat_grad"], sizes)
    s["norm"], s["clip"] = torch.empty(1, device="cuda"), torch.empty(1, device="cuda")
    if case["op"] == "grad_norm":
        return s
    w = _randn(g, total, sigma=0.02)
    s["flat_param"] = w.to(DT[case["param"]])
    s["params"] = _views(s["flat_param"], sizes)
    s["flat_master"] = w if case["master"] else None
    s["masters"] = _views(w, sizes) if case["master"] else None
    # states of a run that is some hundred steps old
    m, v = _randn(g, total, sigma=5e-4) * size, (_randn(g, total, sigma=2e-3) * size).square() + (1e-3 * size).square()
    s["steps"] = 300
    if case["bits"] == 32:
        s["flat_m"], s["flat_v"] = m, v
        s["m"], s["v"] = _views(m, sizes), _views(v, sizes)
        s["m_scales"] = s["v_scales"] = None
    else:
        blocks = [-(-n // BLOCK) for n in sizes]
        # an element's block, its place among whole blocks, its place in its tensor and that tensor's number (by the
        # last two go the rounding's random numbers)
        of = torch.tensor(sizes, device="cuda")
        s["tensor"] = torch.repeat_interleave(torch.arange(len(sizes), device="cuda"), of, output_size=total)
        s["index"] = torch.arange(total, device="cuda") - (of.cumsum(0) - of)[s["tensor"]]
        of = torch.tensor(blocks, device="cuda")
        s["block_of"] = (of.cumsum(0) - of)[s["tensor"]] + s["index"] // BLOCK
        s["place"] = s["block_of"] * BLOCK + s["index"] % BLOCK
        s["padded"] = sum(blocks) * BLOCK
        s["flat_ms"], s["flat_vs"] = (_block_max(x, s) / E4M3_MAX for x in (m.abs(), v.sqrt()))
        s["flat_m"], s["flat_v"] = ((x / sc[s["block_of"]]).clamp(-E4M3_MAX, E4M3_MAX).to(E4M3).view(torch.uint8)
                                    for x, sc in ((m, s["flat_ms"]), (v.sqrt(), s["flat_vs"])))
        s["m"], s["v"] = _views(s["flat_m"], sizes), _views(s["flat_v"], sizes)
        s["m_scales"], s["v_scales"] = _views(s["flat_ms"], blocks), _views(s["flat_vs"], blocks)
    s["scale"] = torch.full((1,), 0.73, device="cuda") if case["clip"] else None
    return s


def _block_max(x, s):
    whole = torch.zeros(s["padded"], device="cuda", dtype=x.dtype)
    whole[s["place"]] = x
    return whole.view(-1, BLOCK).amax(1)


# ------------------------------------------------------------------ plain forms
def _logits(s):
    t = torch.matmul(s["a"].view(E4M3).float(), s["b"].view(E4M3).float().t())
    return t * (s["sa"].reshape(-1, 1) * s["sb"].reshape(1, -1))


def _plain_ce(s):
    t, l = s["targets"], _logits(s)
    top = l.amax(1)
    lse = top + torch.log(torch.exp(l - top[:, None]).sum(1))
    counted = t >= 0
    loss = (lse - l.gather(1, t.clamp(min=0)[:, None])[:, 0]) * counted
    count = counted.sum()
    inv = torch.where(count > 0, 1 / count.double(), 0.0)
    return {"loss": loss, "lse": lse, "mean": torch.stack([loss.double().sum() * inv, inv]).float()}


def _plain_ce_grad(s):
    t = s["targets"]
    p = torch.exp(_logits(s) - s["lse"][:, None])
    counted = (t >= 0).float()
    at = t.clamp(min=0)[:, None]
    p.scatter_add_(1, at, -torch.ones_like(at, dtype=torch.float32))
    p *= (s["dloss"] * counted)[:, None]
    da = torch.matmul(p, s["b"].view(E4M3).float()) * s["sb"]
    db = torch.matmul(p.t(), s["a"].view(E4M3).float()) * s["sa"]
    return {"da": da.to(torch.bfloat16), "db": db.to(torch.bfloat16)}


def _mix(h):
    """A 32-bit integer hash (two multiplications between shifts), on 64-bit
    integers that hold 32 bits."""
    h = ((h ^ (h >> 16)) * 0x85EBCA6B) & 0xFFFFFFFF
    h = ((h ^ (h >> 13)) * 0xC2B2AE35) & 0xFFFFFFFF
    return h ^ (h >> 16)


def _uniforms(s):
    """Two numbers in (0, 1) per element, from the seed, the step, the tensor's
    number and the element's place: a hash for each four elements, whose words
    follow one another by shifts and exclusive ors."""
    key = _mix(_mix(_mix(torch.tensor(SEED, device="cuda")) ^ s["steps"]) ^ s["tensor"])
    group = s["index"] >> 2
    h = _mix((group & 0xFFFFFFFF) ^ key ^ _mix(group >> 32)) | 1
    for k in range(1, 4):
        x = h ^ ((h << 13) & 0xFFFFFFFF)
        x = x ^ (x >> 17)
        x = x ^ ((x << 5) & 0xFFFFFFFF)
        h = torch.where((s["index"] & 3) >= k, x, h)
    return ((h & 0xFFFF).float() + 0.5) / 65536, ((h >> 16).float() + 0.5) / 65536


def _steps_of(y):
    """|y| in steps of the E4M3 grid below it (at least the subnormals' 2^-9),
    and that step."""
    step = torch.exp2((torch.frexp(y)[1] - 1).clamp(min=-6).to(y.dtype) - 3)
    return y / step, step


def _encode_m(m, s, u):
    scale = _block_max(m.abs(), s) / E4M3_MAX
    scale = torch.where(scale >= 2.0 ** -100, scale, 0.0)
    of = scale[s["block_of"]]
    y, step = _steps_of((m.abs() / torch.where(of > 0, of, math.inf)).clamp(max=E4M3_MAX))
    k = torch.floor(y)
    return (torch.sign(m) * (k + (u < y - k)) * step).to(E4M3), scale


def _encode_v(v, s, u):
    """The root of v in 8 bits, rounded so that v itself is met on average;
    never from above zero to zero."""
    r = torch.sqrt(v)
    scale = _block_max(r, s) / E4M3_MAX
    of = scale[s["block_of"]]
    y, step = _steps_of((r / torch.where(of > 0, of, math.inf)).clamp(max=E4M3_MAX))
    k = torch.floor(y)
    f = y - k
    up = (u * (2 * k + 1) < f * (2 * k + f)) | ((k == 0) & (f > 0))
    return ((k + up) * step).to(E4M3), scale


def _plain_adamw(s):
    case = s["case"]
    s["steps"] += 1
    t = s["steps"]
    g = s["flat_grad"].float()
    if s["scale"] is not None:
        g = g * s["scale"]
    w = (s["flat_param"] if s["flat_master"] is None else s["flat_master"]).float()
    if case["bits"] == 32:
        m, v = s["flat_m"], s["flat_v"]
    else:
        m = s["flat_m"].view(E4M3).float() * s["flat_ms"][s["block_of"]]
        v = (s["flat_v"].view(E4M3).float() * s["flat_vs"][s["block_of"]]).square()
    m = BETA1 * m + (1 - BETA1) * g
    v = BETA2 * v + (1 - BETA2) * g * g
    w = w * (1 - LR * DECAY) - LR / (1 - BETA1 ** t) * m / (torch.sqrt(v) / math.sqrt(1 - BETA2 ** t) + EPS)
    out = {}
    if case["bits"] == 32:
        s["flat_m"].copy_(m)
        s["flat_v"].copy_(v)
    else:
        um, uv = _uniforms(s)
        codes, scale = _encode_m(m, s, um)
        s["flat_m"].copy_(codes.view(torch.uint8))
        s["flat_ms"].copy_(scale)
        codes, scale = _encode_v(v, s, uv)
        s["flat_v"].copy_(codes.view(torch.uint8))
        s["flat_vs"].copy_(scale)
    s["flat_param"].copy_(w)
    if s["flat_master"] is not None:
        s["flat_master"].copy_(w)
    return _adamw_outputs(s)


def _adamw_outputs(s):
    out = {"param": s["flat_param"]}
    if s["flat_master"] is not None:
        out["master"] = s["flat_master"]
    if s["case"]["bits"] == 32:
        out.update(m=s["flat_m"], v=s["flat_v"])
    else:
        out.update(m=s["flat_m"].view(E4M3), v=s["flat_v"].view(E4M3), m_scale=s["flat_ms"], v_scale=s["flat_vs"])
    return out


def _plain_grad_norm(s):
    norm = torch.sqrt(s["flat_grad"].double().square().sum()).float().reshape(1)
    return {"norm": norm, "clip": (MAX_NORM / (norm + 1e-6)).clamp(max=1.0)}


# ------------------------------------------------------------------ the framework's operators
def _own_ce(s):
    import fp8_tensor_scaled_quantize_amd as fp8mi
    fp8mi.fp8_cross_entropy(s["a"], s["b"], s["targets"], s["sa"], s["sb"], loss=s["loss"], lse=s["lse"],
                            mean_out=s["mean"])
    return {"loss": s["loss"], "lse": s["lse"], "mean": s["mean"]}


def _own_ce_grad(s):
    import fp8_tensor_scaled_quantize_amd as fp8mi
    fp8mi.fp8_cross_entropy_grad(s["a"], s["b"], s["targets"], s["lse"], s["dloss"], s["sa"], s["sb"], da=s["da"],
                                 db=s["db"])
    return {"da": s["da"], "db": s["db"]}


def _own_adamw(s):
    import fp8_tensor_scaled_quantize_amd as fp8mi
    s["steps"] += 1
    fp8mi.adamw_step(s["params"], s["grads"], s["m"], s["v"], s["steps"], lr=LR, betas=(BETA1, BETA2), eps=EPS,
                     weight_decay=DECAY, masters=s["masters"], exp_avg_scales=s["m_scales"],
                     exp_avg_sq_scales=s["v_scales"], grad_scale=s["scale"], seed=SEED)
    return _adamw_outputs(s)


def _own_grad_norm(s):
    import fp8_tensor_scaled_quantize_amd as fp8mi
    fp8mi.grad_norm(s["grads"], max_norm=MAX_NORM, out=s["norm"], clip_out=s["clip"])
    return {"norm": s["norm"], "clip": s["clip"]}


_PLAIN = {"ce": _plain_ce, "ce_grad": _plain_ce_grad, "adamw": _plain_adamw, "grad_norm": _plain_grad_norm}
_OWN = {"ce": _own_ce, "ce_grad": _own_ce_grad, "adamw": _own_adamw, "grad_norm": _own_grad_norm}


def run(state):
    return (_OWN if own else _PLAIN)[state["case"]["op"]](state)


def work(case):
    op = case["op"]
    if op in ("ce", "ce_grad"):
        M, N, K = case["M"], case["N"], case["K"]
        if op == "ce":
            return {"bytes": (M + N) * K + 16 * M, "flops": 2 * M * N * K}
        return {"bytes": 3 * (M + N) * K + 16 * M, "flops": 6 * M * N * K}
    n = sum(_sizes(case))
    if op == "grad_norm":
        return {"bytes": n * EB[case["grad"]] + 8, "flops": 2 * n}
    state = 16 if case["bits"] == 32 else 4 + 16 / BLOCK
    # a master is read in the parameter's place, which is then written alone
    per = EB[case["grad"]] + state + (8 + EB[case["param"]] if case["master"] else 2 * EB[case["param"]])
    return {"bytes": n * per, "flops": (20 if case["bits"] == 32 else 60) * n}


# ------------------------------------------------------------------ 64 bits
def _exact_logits(s, rows):
    a, b = (s[k].view(E4M3).double() for k in ("a", "b"))
    return torch.mm(a[rows] * s["sa"].double().expand(a.shape[0])[rows, None],
                    (b * s["sb"].double().expand(b.shape[0])[:, None]).t().contiguous())


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op in ("ce", "ce_grad"):
        M, t = case["M"], s["targets"]
        parts = [slice(i, min(i + 1024, M)) for i in range(0, M, 1024)]
        if op == "ce":
            lse, at = torch.empty(M, dtype=torch.float64, device="cuda"), torch.zeros(M, dtype=torch.float64, device="cuda")
            for p in parts:
                l = _exact_logits(s, p)
                lse[p] = torch.logsumexp(l, 1)
                at[p] = l[torch.arange(l.shape[0], device="cuda"), t[p].clamp(min=0)]
            loss = torch.where(t < 0, 0.0, lse - at)
            count = int((t >= 0).sum())
            mean = torch.tensor([float(loss.sum()) / count, 1 / count] if count else [0.0, 0.0], dtype=torch.float64)
            return {"loss": loss, "lse": lse, "mean": mean}
        a, b = s["a"].view(E4M3).double() * s["sa"].double(), s["b"].view(E4M3).double() * s["sb"].double()
        da, db = torch.empty_like(a), torch.zeros_like(b)
        d = s["dloss"].double().expand(M)
        for p in parts:
            # the saved lse is an input like the others
            g = torch.exp(_exact_logits(s, p) - s["lse"][p].double()[:, None])
            rows = torch.arange(g.shape[0], device="cuda")
            g[rows, t[p].clamp(min=0)] -= 1
            g *= torch.where(t[p] < 0, 0.0, d[p])[:, None]
            da[p] = torch.mm(g, b)
            db += torch.mm(g.t().contiguous(), a[p])
        return {"da": da, "db": db}
    g = s["flat_grad"].double()
    if op == "grad_norm":
        norm = torch.linalg.vector_norm(g)
        return {"norm": norm.reshape(1), "clip": torch.clamp(MAX_NORM / (norm + 1e-6), max=1.0).reshape(1)}
    if s["scale"] is not None:
        g = g * s["scale"].double()
    t = s["steps"] + 1
    w = (s["flat_param"] if s["flat_master"] is None else s["flat_master"]).double()
    m, v = s["flat_m"], s["flat_v"]
    if case["bits"] == 8:
        m = m.view(E4M3).double() * s["flat_ms"].double()[s["block_of"]]
        v = (v.view(E4M3).double() * s["flat_vs"].double()[s["block_of"]]) ** 2
    m = torch.lerp(g, m.double(), BETA1)
    v = torch.lerp(g ** 2, v.double(), BETA2)
    mhat, vhat = m / (1 - BETA1 ** t), v / (1 - BETA2 ** t)
    w = w - LR * DECAY * w - LR * mhat / (vhat ** 0.5 + EPS)
    out = {"param": w}
    if case["master"]:
        out["master"] = w
    if case["bits"] == 32:
        out.update(m=m, v=v)
    else:  # the values that the codes round, before the rounding
        ms, vs = _block_max(m.abs(), s) / E4M3_MAX, _block_max(v.sqrt(), s) / E4M3_MAX
        out.update(m=m / ms[s["block_of"]], v=v.sqrt() / vs[s["block_of"]], m_scale=ms, v_scale=vs)
    return out
