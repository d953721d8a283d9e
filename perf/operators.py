"""Cases of the operators around an fp8 linear layer: the root-mean-square norm
that makes its fp8 input (with the residual's addition, forward and backward),
and the fp8 product with bias, activation and residual in its epilogue with
the activation's gradient.  Sizes follow the 1.2B-model linears of this
repository's configurations (hidden 1536, feed-forward 6912), single tokens to
8192-token training steps, plus generic widths.

`run` computes a case in plain torch operations in 32 bits, or, where `own` is
true, by the framework's operators.  fp8 codes are returned as float8 tensors
next to their dequantisation multipliers."""
from __future__ import annotations

import math

import torch

own = False

H = 16  # ring history length
RING_WORDS = H + 4 + 1024
DT = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
F8 = {"e4m3": torch.float8_e4m3fn, "e5m2": torch.float8_e5m2}
FMAX = {"e4m3": 448.0, "e5m2": 57344.0}
EPS = 1e-6
GELU_C, GELU_A = math.sqrt(2.0 / math.pi), 0.044715


def listed():
    norm = dict(op="norm", weight="bf16", fmt="e4m3")
    mm = dict(op="mm", bias="bf16", gated=False, residual="none", out="bf16", keep_z=False, row_scales=False)
    return [
        # one new token through a block's norm while serving: launch latency counts
        dict(norm, name="norm 1x4096 serve", rows=1, cols=4096, dtype="bf16", residual=True, scaling="row",
             save=False),
        # an odd width and a ragged token count, fp16, a calibrated scale
        dict(norm, name="norm 1000x1535 f16", rows=1000, cols=1535, dtype="f16", residual=False, scaling="tensor",
             save=False),
        # the training step's norm: delayed scaling, h and 1/rms kept for the backward pass
        dict(norm, name="norm 8192x1536 train", rows=8192, cols=1536, dtype="bf16", residual=True, scaling="ring",
             save=True),
        # backward of a small fp32 norm of odd width
        dict(op="norm_grad", name="norm grad 250x1535 f32", rows=250, cols=1535, dtype="f32", weight="f32",
             residual=False),
        # the training step's backward, with the gradient of the residual path
        dict(op="norm_grad", name="norm grad 8192x1536", rows=8192, cols=1536, dtype="bf16", weight="bf16",
             residual=True),
        # one new token, gated up-projection, fp8 output for the down-projection
        dict(mm, name="mm 1x13824x1536 gated", M=1, N=13824, K=1536, act="silu", gated=True, out="e4m3",
             row_scales=True, bias="none"),
        # a serving batch's down-projection with the residual stream
        dict(mm, name="mm 32x1536x6912 residual", M=32, N=1536, K=6912, act="none", residual="bf16"),
        # an odd number of tokens and columns (N tail), plain activation
        dict(mm, name="mm 1000x1537x2048 gelu", M=1000, N=1537, K=2048, act="gelu", residual="f32", bias="f32"),
        # training, up-projection: pre-activations kept, fp8 output
        dict(mm, name="mm 8192x6912x1536 gelu", M=8192, N=6912, K=1536, act="gelu", out="e4m3", keep_z=True),
        # training, down-projection with the residual stream
        dict(mm, name="mm 8192x1536x6912 residual", M=8192, N=1536, K=6912, act="none", residual="bf16"),
        # activation gradient of a ragged batch of odd width
        dict(op="act_grad", name="act grad 250x1537 relu", rows=250, cols=1537, dtype="f16", act="relu", gated=False,
             fmt="e5m2", scaling="tensor", bias=False),
        # the training step's activation gradient with the bias gradient, delayed scaling
        dict(op="act_grad", name="act grad 8192x6912 gelu", rows=8192, cols=6912, dtype="bf16", act="gelu",
             gated=False, fmt="e5m2", scaling="ring", bias=True),
    ]


def _log(rng, lo, hi):
    v = int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))
    return v + 1 if v == 3072 else v


def draw(rng):
    op = rng.choice(["norm", "norm", "norm_grad", "mm", "mm", "act_grad"])
    if op in ("norm", "norm_grad"):
        cols = _log(rng, 64, 16384)
        rows = _log(rng, 1, max(2, min(32768, (1 << 25) // cols)))
        case = dict(op=op, rows=rows, cols=cols, dtype=rng.choice(["bf16", "bf16", "f16", "f32"]),
                    weight=rng.choice(["bf16", "f32"]), residual=rng.random() < 0.6)
        if op == "norm":
            case.update(fmt=rng.choice(["e4m3", "e4m3", "e5m2"]), scaling=rng.choice(["row", "ring", "tensor"]),
                        save=rng.random() < 0.5)
        return case
    if op == "mm":
        gated = rng.random() < 0.4
        K = 16 * _log(rng, 4, 512)
        K = K + 16 if K == 3072 else K
        N = _log(rng, 32, 13824)
        N += N % 2 if gated else 0
        N = N + 2 if N == 3072 else N
        most = 8192 * 6912 * 1536
        M = _log(rng, 1, max(2, min(8192, most // (N * K))))
        return dict(op=op, M=M, N=N, K=K, act=rng.choice(["silu", "gelu", "relu"] if gated else
                                                         ["none", "silu", "gelu", "relu"]),
                    gated=gated, bias=rng.choice(["none", "bf16", "f32"]),
                    residual=rng.choice(["none", "none", "bf16", "f32"]), out=rng.choice(["bf16", "bf16", "e4m3"]),
                    keep_z=rng.random() < 0.4, row_scales=rng.random() < 0.5)
    gated = rng.random() < 0.4
    cols = _log(rng, 16, 6912)
    rows = _log(rng, 1, max(2, min(16384, (8192 * 6912) // (cols * (2 if gated else 1)))))
    return dict(op=op, rows=rows, cols=cols, dtype=rng.choice(["bf16", "bf16", "f16"]),
                act=rng.choice(["silu", "gelu", "relu"]), gated=gated, fmt=rng.choice(["e5m2", "e5m2", "e4m3"]),
                scaling=rng.choice(["ring", "tensor"]), bias=rng.random() < 0.5)


# ------------------------------------------------------------------ inputs
def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    return g


def _randn(g, *shape, sigma=1.0):
    return torch.randn(*shape, generator=g, device="cuda") * sigma


def _codes(g, rows, cols, sigma):
    """fp8 codes of N(0, sigma^2) values at a per-tensor scale, and 1 / scale."""
    v = _randn(g, rows, cols, sigma=sigma)
    s = FMAX["e4m3"] / v.abs().amax()
    return (v * s).clamp(-448, 448).to(F8["e4m3"]).view(torch.uint8), (1 / s).reshape(1)


def _ring(fmt, amax):
    """A ring part-way through training: a few amaxes in its history, the
    scale that they give, the next slot."""
    words = torch.zeros(RING_WORDS, dtype=torch.int32)
    f = words.view(torch.float32)
    f[:3] = torch.tensor([0.7, 1.0, 0.8]) * amax
    f[H] = FMAX[fmt] / amax
    words[H + 1] = 3
    return words.cuda()


def prepare(case, seed):
    g = _gen(seed)
    s = {"case": case}
    op = case["op"]
    if op in ("norm", "norm_grad"):
        rows, cols, dt = case["rows"], case["cols"], DT[case["dtype"]]
        # activations of a residual stream: unequal rows, a few large channels
        row = torch.exp(_randn(g, rows, 1, sigma=0.5))
        col = 1 + 6 * (torch.rand(1, cols, generator=g, device="cuda") < 0.01)
        s["x"] = (_randn(g, rows, cols) * row * col).to(dt)
        s["w"] = (1 + 0.1 * _randn(g, cols)).to(DT[case["weight"]])
        s["res"] = (_randn(g, rows, cols) * row).to(dt) if case["residual"] else None
    if op == "norm":
        s["eps"] = EPS
        s["codes"] = torch.empty(rows, cols, dtype=torch.uint8, device="cuda")
        s["scale_inv"] = torch.empty(rows if case["scaling"] == "row" else 1, device="cuda")
        s["amax"] = torch.empty_like(s["scale_inv"]) if case["scaling"] != "row" else None
        s["h"] = torch.empty_like(s["x"]) if case["residual"] else None
        s["rstd"] = torch.empty(rows, device="cuda") if case["save"] else None
        s["ring"] = _ring(case["fmt"], 30.0) if case["scaling"] == "ring" else None
        s["scale"] = (torch.full((1,), FMAX[case["fmt"]] / 30.0, device="cuda") if case["scaling"] == "tensor"
                      else None)
    elif op == "norm_grad":
        s["dy"] = _randn(g, rows, cols, sigma=1e-2).to(dt)
        s["rstd"] = torch.rsqrt(s["x"].float().square().mean(1) + EPS)
        s["dx"] = torch.empty_like(s["x"])
        s["dw"] = torch.empty(cols, device="cuda")
        if s["res"] is not None:
            s["res"] = _randn(g, rows, cols, sigma=1e-2).to(dt)  # here: the gradient of the residual path
        # scratch that a training loop keeps: the partial sums of the weight's gradient
        s["ws"] = torch.empty(1024 * cols, device="cuda")
    elif op == "mm":
        M, N, K = case["M"], case["N"], case["K"]
        No = N // 2 if case["gated"] else N
        s["a"], s["sa"] = _codes(g, M, K, 1.0)
        s["b"], s["sb"] = _codes(g, N, K, 1.0 / math.sqrt(K))  # gated: rows 2j gate, 2j + 1 value
        if case["row_scales"]:
            s["sa"] = s["sa"] * torch.exp(_randn(g, M, sigma=0.3))
            s["sb"] = s["sb"] * torch.exp(_randn(g, N, sigma=0.1))
        s["bias"] = None if case["bias"] == "none" else _randn(g, N, sigma=0.1).to(DT[case["bias"]])
        s["res"] = None if case["residual"] == "none" else _randn(g, M, No).to(DT[case["residual"]])
        s["z"] = torch.empty(M, N, dtype=torch.bfloat16, device="cuda") if case["keep_z"] else None
        s["out"] = torch.empty(M, No, dtype=torch.bfloat16 if case["out"] == "bf16" else torch.uint8, device="cuda")
        s["out_scale"] = None if case["out"] == "bf16" else torch.full((1,), FMAX[case["out"]] / 24.0, device="cuda")
    else:
        rows, cols, mul = case["rows"], case["cols"], 2 if case["gated"] else 1
        s["dy"] = (_randn(g, rows, cols, sigma=1e-3) * torch.exp(_randn(g, rows, 1, sigma=0.5))).to(DT[case["dtype"]])
        s["z"] = _randn(g, rows, cols * mul, sigma=1.5).to(torch.bfloat16)
        s["codes"] = torch.empty(rows, cols * mul, dtype=torch.uint8, device="cuda")
        s["codes_t"] = torch.empty(cols * mul, rows, dtype=torch.uint8, device="cuda")
        s["scale_inv"] = torch.empty(1, device="cuda")
        s["db"] = torch.empty(cols * mul, dtype=torch.bfloat16, device="cuda") if case["bias"] else None
        # scratch that a training loop keeps: the partial sums of the bias gradient
        s["ws"] = (torch.empty(-(-rows // 128) * cols * mul, dtype=torch.float64, device="cuda") if case["bias"]
                   else None)
        s["ring"] = _ring(case["fmt"], 0.03) if case["scaling"] == "ring" else None
        s["scale"] = (torch.full((1,), FMAX[case["fmt"]] / 0.03, device="cuda") if case["scaling"] == "tensor"
                      else None)
    return s


# ------------------------------------------------------------------ plain forms
def _scale_of(m, fmax):
    return torch.where((m > 0) & torch.isfinite(m), fmax / m, torch.ones_like(m))


def _encode(y, s, fmt):
    return (y * s).clamp(-FMAX[fmt], FMAX[fmt]).to(F8[fmt])


def _ring_used(ring):
    return ring.view(torch.float32)[H:H + 1].clone()


def _ring_fold(ring, amax, fmax):
    f = ring.view(torch.float32)
    f.index_copy_(0, ring[H + 1:H + 2].long(), amax.reshape(1))
    f[H:H + 1] = _scale_of(f[:H].amax().reshape(1), fmax)
    ring[H + 1] = (ring[H + 1] + 1) % H


def _ring_state(ring):
    f = ring.view(torch.float32)
    return {"hist": f[:H], "scale": f[H:H + 1], "slot": ring[H + 1:H + 2]}


def _act(t, act):
    if act == "relu":
        return t * (t > 0)
    if act == "silu":
        return t / (1 + torch.exp(-t))
    if act == "gelu":
        return t / (1 + torch.exp(-2 * GELU_C * (t + GELU_A * t * t * t)))
    return t


def _act_slope(t, act):
    if act == "relu":
        return (t > 0).float()
    if act == "silu":
        p = 1 / (1 + torch.exp(-t))
        return p * (1 + t * (1 - p))
    p = 1 / (1 + torch.exp(-2 * GELU_C * (t + GELU_A * t * t * t)))
    return p * (1 + t * (1 - p) * 2 * GELU_C * (1 + 3 * GELU_A * t * t))


def _plain_norm(s):
    case = s["case"]
    fmax, dt = FMAX[case["fmt"]], s["x"].dtype
    h = s["x"].float()
    if s["res"] is not None:
        h = h + s["res"].float()
    rstd = 1 / torch.sqrt(h.square().mean(1) + s["eps"])
    y = h * rstd[:, None] * s["w"].float()
    out = {}
    if case["scaling"] == "row":
        amax = y.abs().amax(1)
        q = _scale_of(amax, fmax)
        codes = _encode(y, q[:, None], case["fmt"])
    else:
        amax = y.abs().amax().reshape(1)
        q = _ring_used(s["ring"]) if case["scaling"] == "ring" else s["scale"]
        codes = _encode(y, q, case["fmt"])
        out["amax"] = amax
        if case["scaling"] == "ring":
            _ring_fold(s["ring"], amax, fmax)
            out["ring"] = _ring_state(s["ring"])
    out.update(codes=codes, scale_inv=1 / q)
    if s["h"] is not None:
        out["h"] = h.to(dt)
    if case["save"]:
        out["rstd"] = rstd
    return out


def _plain_norm_grad(s):
    h, dy, r = s["x"].float(), s["dy"].float(), s["rstd"][:, None]
    g = dy * s["w"].float()
    dx = r * g - r * r * r * (g * h).mean(1, keepdim=True) * h
    if s["res"] is not None:
        dx = dx + s["res"].float()
    return {"dx": dx.to(s["x"].dtype), "dw": (dy * (h * r)).sum(0)}


def _plain_mm(s):
    case = s["case"]
    t = torch.matmul(s["a"].view(F8["e4m3"]).float(), s["b"].view(F8["e4m3"]).float().t())
    t = t * (s["sa"].reshape(-1, 1) * s["sb"].reshape(1, -1))
    if s["bias"] is not None:
        t = t + s["bias"].float()
    y = _act(t[:, 0::2], case["act"]) * t[:, 1::2] if case["gated"] else _act(t, case["act"])
    if s["res"] is not None:
        y = y + s["res"].float()
    out = {"y": y.to(torch.bfloat16) if case["out"] == "bf16" else _encode(y, s["out_scale"], case["out"])}
    if case["keep_z"]:
        out["z"] = t.to(torch.bfloat16)
    return out


def _plain_act_grad(s):
    case = s["case"]
    fmt = case["fmt"]
    dy, z = s["dy"].float(), s["z"].float()
    if case["gated"]:
        t, v = z[:, 0::2], z[:, 1::2]
        dz = torch.stack([dy * v * _act_slope(t, case["act"]), dy * _act(t, case["act"])], dim=2).flatten(1)
    else:
        dz = dy * _act_slope(z, case["act"])
    q = _ring_used(s["ring"]) if case["scaling"] == "ring" else s["scale"]
    codes = _encode(dz, q, fmt)
    out = {"codes": codes, "codes_t": codes.view(torch.uint8).t().contiguous().view(F8[fmt]), "scale_inv": 1 / q}
    if case["scaling"] == "ring":
        _ring_fold(s["ring"], dz.abs().amax(), FMAX[fmt])
        out["ring"] = _ring_state(s["ring"])
    if case["bias"]:
        out["db"] = dz.sum(0).to(torch.bfloat16)
    return out


# ------------------------------------------------------------------ the framework's operators
def _own_norm(s):
    import fp8_tensor_scaled_quantize_amd as fp8mi
    case = s["case"]
    fp8mi.fp8_rmsnorm(s["x"], s["w"], case["fmt"], eps=s["eps"], residual=s["res"], out=s["codes"],
                      row_scaled=case["scaling"] == "row", scale=s["scale"], ring=s["ring"],
                      scale_inv_out=s["scale_inv"], amax_out=s["amax"], sum_out=s["h"], rstd_out=s["rstd"])
    out = {"codes": s["codes"].view(F8[case["fmt"]]), "scale_inv": s["scale_inv"]}
    if case["scaling"] != "row":
        out["amax"] = s["amax"]
    if case["scaling"] == "ring":
        out["ring"] = _ring_state(s["ring"])
    if s["h"] is not None:
        out["h"] = s["h"]
    if case["save"]:
        out["rstd"] = s["rstd"]
    return out


def _own_norm_grad(s):
    import fp8_tensor_scaled_quantize_amd as fp8mi
    fp8mi.fp8_rmsnorm_grad(s["dy"], s["x"], s["w"], s["rstd"], dsum=s["res"], dx=s["dx"], dweight=s["dw"],
                           workspace=s["ws"])
    return {"dx": s["dx"], "dw": s["dw"]}


def _own_mm(s):
    import fp8_tensor_scaled_quantize_amd as fp8mi
    case = s["case"]
    fp8mi.fp8_mm_act(s["a"], s["b"], s["sa"], s["sb"], bias=s["bias"], act=case["act"], gated=case["gated"],
                     residual=s["res"], z_out=s["z"], out=s["out"], out_fmt=None if case["out"] == "bf16" else case["out"],
                     out_scale=s["out_scale"])
    out = {"y": s["out"] if case["out"] == "bf16" else s["out"].view(F8[case["out"]])}
    if case["keep_z"]:
        out["z"] = s["z"]
    return out


def _own_act_grad(s):
    import fp8_tensor_scaled_quantize_amd as fp8mi
    case = s["case"]
    fp8mi.fp8_act_grad(s["dy"], s["z"], case["act"], gated=case["gated"], fmt=case["fmt"], out_row=s["codes"],
                       out_t=s["codes_t"], scale=s["scale"], ring=s["ring"], scale_inv_out=s["scale_inv"],
                       bias_grad_out=s["db"], workspace=s["ws"])
    out = {"codes": s["codes"].view(F8[case["fmt"]]), "codes_t": s["codes_t"].view(F8[case["fmt"]]),
           "scale_inv": s["scale_inv"]}
    if case["scaling"] == "ring":
        out["ring"] = _ring_state(s["ring"])
    if case["bias"]:
        out["db"] = s["db"]
    return out


_PLAIN = {"norm": _plain_norm, "norm_grad": _plain_norm_grad, "mm": _plain_mm, "act_grad": _plain_act_grad}
_OWN = {"norm": _own_norm, "norm_grad": _own_norm_grad, "mm": _own_mm, "act_grad": _own_act_grad}


def run(state):
    return (_OWN if own else _PLAIN)[state["case"]["op"]](state)


def work(case):
    eb = {"bf16": 2, "f16": 2, "f32": 4, "none": 0}
    op = case["op"]
    if op == "norm":
        n, e = case["rows"] * case["cols"], eb[case["dtype"]]
        per = 1 + e * (3 if case["residual"] else 1)  # codes; x, and the residual read and the sum written
        rows = case["rows"] * 4 * (int(case["save"]) + int(case["scaling"] == "row"))
        return {"bytes": n * per + rows + case["cols"] * eb[case["weight"]], "flops": 8 * n}
    if op == "norm_grad":
        n, e = case["rows"] * case["cols"], eb[case["dtype"]]
        return {"bytes": n * e * (4 if case["residual"] else 3) + 4 * case["rows"] +
                case["cols"] * (4 + eb[case["weight"]]), "flops": 12 * n}
    if op == "mm":
        M, N, K = case["M"], case["N"], case["K"]
        No = N // 2 if case["gated"] else N
        nbytes = M * K + N * K + N * eb[case["bias"]] + M * No * (eb[case["residual"]] +
                                                                  (2 if case["out"] == "bf16" else 1))
        return {"bytes": nbytes + (2 * M * N if case["keep_z"] else 0), "flops": 2 * M * N * K}
    mul = 2 if case["gated"] else 1
    n = case["rows"] * case["cols"]
    return {"bytes": n * (2 + 4 * mul) + (2 * case["cols"] * mul if case["bias"] else 0), "flops": 20 * n}


# ------------------------------------------------------------------ 64 bits
def _exact_codes(v, q, fmt):
    """The values that codes round, before the rounding to 8 bits."""
    return torch.clamp(v * q, min=-FMAX[fmt], max=FMAX[fmt])


def _exact_ring(ring, amax, fmt):
    hist = ring.view(torch.float32)[:H].double()
    slot = int(ring[H + 1])
    hist[slot] = amax
    return {"hist": hist, "scale": (FMAX[fmt] / hist.max()).reshape(1), "slot": None}


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    d = {k: v.double() for k, v in s.items() if isinstance(v, torch.Tensor) and v.is_floating_point()}
    if op == "norm":
        h = d["x"] + d["res"] if case["residual"] else d["x"]
        rms = torch.sqrt((h * h).sum(1) / case["cols"] + EPS)
        y = h / rms[:, None] * d["w"]
        out = {}
        if case["scaling"] == "row":
            q = FMAX[case["fmt"]] / y.abs().max(1).values
            out.update(codes=_exact_codes(y, q[:, None], case["fmt"]), scale_inv=1 / q)
        else:
            q = s["ring"].view(torch.float32)[H].double() if case["scaling"] == "ring" else d["scale"]
            out.update(codes=_exact_codes(y, q, case["fmt"]), scale_inv=(1 / q).reshape(1),
                       amax=y.abs().max().reshape(1))
            if case["scaling"] == "ring":
                out["ring"] = _exact_ring(s["ring"], y.abs().max(), case["fmt"])
        if case["residual"]:
            out["h"] = h
        if case["save"]:
            out["rstd"] = 1 / rms
        return out
    if op == "norm_grad":
        xhat = d["x"] * d["rstd"].reshape(-1, 1)
        dxhat = d["dy"] * d["w"]
        proj = (dxhat * xhat).sum(1, keepdim=True) / case["cols"]
        dx = (dxhat - xhat * proj) * d["rstd"].reshape(-1, 1)
        return {"dx": dx + d["res"] if case["residual"] else dx, "dw": torch.einsum("ij,ij->j", d["dy"], xhat)}
    if op == "mm":
        A, B = (s[k].view(F8["e4m3"]).double() for k in ("a", "b"))
        t = torch.mm(A * d["sa"].reshape(-1, 1), (B * d["sb"].reshape(-1, 1)).t().contiguous())
        if s["bias"] is not None:
            t += d["bias"]
        u = t[:, ::2] if case["gated"] else t
        if case["act"] == "relu":
            y = torch.clamp(u, min=0)
        elif case["act"] == "silu":
            y = u * torch.sigmoid(u)
        elif case["act"] == "gelu":
            y = 0.5 * u * (1 + torch.tanh(GELU_C * (u + GELU_A * u ** 3)))
        else:
            y = u
        if case["gated"]:
            y = y * t[:, 1::2]
        if s["res"] is not None:
            y = y + d["res"]
        out = {"y": y if case["out"] == "bf16" else _exact_codes(y, d["out_scale"], case["out"])}
        if case["keep_z"]:
            out["z"] = t
        return out
    dy, z = d["dy"], d["z"]
    u = z[:, ::2] if case["gated"] else z
    if case["act"] == "relu":
        a, slope = torch.clamp(u, min=0), (u > 0).double()
    elif case["act"] == "silu":
        p = torch.sigmoid(u)
        a, slope = u * p, p + u * p * (1 - p)
    else:
        th = torch.tanh(GELU_C * (u + GELU_A * u ** 3))
        a, slope = 0.5 * u * (1 + th), 0.5 * (1 + th) + 0.5 * u * (1 - th * th) * GELU_C * (1 + 3 * GELU_A * u * u)
    dz = dy * slope
    if case["gated"]:
        both = torch.empty_like(z)
        both[:, ::2], both[:, 1::2] = dz * z[:, 1::2], dy * a
        dz = both
    q = s["ring"].view(torch.float32)[H].double() if case["scaling"] == "ring" else d["scale"]
    codes = _exact_codes(dz, q, case["fmt"])
    out = {"codes": codes, "codes_t": codes.t().contiguous(), "scale_inv": (1 / q).reshape(1)}
    if case["scaling"] == "ring":
        out["ring"] = _exact_ring(s["ring"], dz.abs().max(), case["fmt"])
    if case["bias"]:
        out["db"] = dz.sum(0)
    return out
