"""64-bit forms of the operators that end a training step, for the tests:
AdamW (and the rounding of its 8-bit states) and the softmax cross entropy
with its gradient.  Plain numpy, written from the formulas."""
import numpy as np

U32 = 2.0 ** -24  # half a step of fp32, relative


def decode_e4m3(codes):
    c = np.asarray(codes).astype(np.int64)
    e, m = (c >> 3) & 15, c & 7
    v = np.where(e == 0, m * 2.0 ** -9, (8 + m) * 2.0 ** (e - 10.0))
    v = np.where((e == 15) & (m == 7), np.nan, v)
    return np.where(c & 128, -v, v)


# ------------------------------------------------------------------ AdamW
def adamw(w, g, m, v, t, lr, b1, b2, eps, wd, c=1.0):
    """(w, m, v) after step t, in 64 bits."""
    w, g, m, v = (np.asarray(x, np.float64) for x in (w, g, m, v))
    g = g * c
    m = b1 * m + (1 - b1) * g
    v = b2 * v + (1 - b2) * g ** 2
    return w - lr * (wd * w + (m / (1 - b1 ** t)) / (np.sqrt(v / (1 - b2 ** t)) + eps)), m, v


def adamw_bounds(w, g, m, v, t, lr, b1, b2, eps, wd, c=1.0):
    """How far fp32 arithmetic may be from adamw(): each of an expression's
    roundings is at most U32 of a term's magnitude.  m and v: c g, the two
    coefficients, two products (g squared: two more) and the sum, at most 6 and
    8 roundings of each term.  The update: its m and v (v's halved by the root),
    root, root_scale, product, sum, lr's quotient, product and division, 8 more.
    w: the decay (lr, wd, product, difference, product) and the difference."""
    w, g, m, v = (np.abs(np.asarray(x, np.float64)) for x in (w, g, m, v))
    g = g * abs(c)
    tm, tv = b1 * m + (1 - b1) * g, b2 * v + (1 - b2) * g ** 2
    em, ev = 6 * U32 * tm, 8 * U32 * tv
    step = lr / (1 - b1 ** t) / (np.sqrt(tv / (1 - b2 ** t)) + eps + 1e-300)
    return step * tm * (6 + 4 + 8 + 1) * U32 + 6 * U32 * w, em, ev


def mix32(h):
    h = np.asarray(h, np.uint64) & np.uint64(0xFFFFFFFF)
    m = np.uint64(0xFFFFFFFF)
    h = ((h ^ (h >> np.uint64(16))) * np.uint64(0x85EBCA6B)) & m
    h = ((h ^ (h >> np.uint64(13))) * np.uint64(0xC2B2AE35)) & m
    return h ^ (h >> np.uint64(16))


def uniforms(n, seed, step, tensor):
    """The rounding's random numbers of a tensor's n elements: (for m, for v)."""
    key = mix32(mix32(mix32(seed) ^ np.uint64(step)) ^ np.uint64(tensor))
    x = mix32(np.arange(-(-n // 4), dtype=np.uint64) ^ key ^ mix32(0)) | np.uint64(1)
    words = []
    for _ in range(4):
        words.append(x)
        x = x ^ ((x << np.uint64(13)) & np.uint64(0xFFFFFFFF))
        x = x ^ (x >> np.uint64(17))
        x = x ^ ((x << np.uint64(5)) & np.uint64(0xFFFFFFFF))
    h = np.stack(words, 1).reshape(-1)[:n]
    return ((h & np.uint64(0xFFFF)).astype(np.float64) + 0.5) / 65536, ((h >> np.uint64(16)).astype(np.float64) + 0.5) / 65536


def block_scales(x, block=256):
    """max |x| / 448 of each block of a flat array, and that of each element."""
    n = x.size
    pad = np.zeros(-(-n // block) * block)
    pad[:n] = np.abs(x)
    s = pad.reshape(-1, block).max(1) / 448
    return s, np.repeat(s, block)[:n]


def grid(y):
    """y >= 0 in steps of the E4M3 grid: whole steps, the rest, the step."""
    e = np.floor(np.log2(np.maximum(y, 2.0 ** -6)))
    e = np.where(2.0 ** e > np.maximum(y, 2.0 ** -6), e - 1, e)
    step = 2.0 ** (e - 3)
    k = np.floor(y / step)
    return k, y / step - k, step


def adamw8_fp32(codes_m, scales_m, codes_v, scales_v, g, seed, step, tensor, b1, b2, c=None):
    """The new codes and scales of an 8-bit step, operation by operation in IEEE
    fp32: (codes of |m| with its sign, scales, codes of sqrt(v), scales)."""
    f = np.float32
    n = len(g)
    ms, vs = (np.repeat(x.astype(f), 256)[:n] for x in (scales_m, scales_v))
    g = g.astype(f) if c is None else g.astype(f) * f(c)
    m = f(b1) * (decode_e4m3(codes_m).astype(f) * ms) + f(1 - b1) * g
    q = decode_e4m3(codes_v).astype(f) * vs
    r = np.sqrt(f(b2) * (q * q) + f(1 - b2) * g * g)
    out = []
    for x, u, root in ((m, uniforms(n, seed, step, tensor)[0].astype(f), False),
                       (r, uniforms(n, seed, step, tensor)[1].astype(f), True)):
        pad = np.zeros(-(-n // 256) * 256, f)
        pad[:n] = np.abs(x)
        s = pad.reshape(-1, 256).max(1) * (f(1) / f(448))
        s = np.where(s < f(2.0 ** -100), f(0), s)
        per = np.repeat(s, 256)[:n]
        y = np.minimum(np.abs(x) / np.where(per > 0, per, f(np.inf)), f(448))
        e = np.maximum(np.frexp(y)[1] - 1, -6)
        unit = np.exp2((e - 3).astype(f))
        k = np.floor(y / unit)
        t = y / unit - k
        up = (u * (2 * k + 1) < t * (2 * k + t)) | ((k == 0) & (t > 0)) if root else u < t
        out += [np.copysign((k + up) * unit, x), s]
    return out


# ------------------------------------------------------------------ cross entropy
def logits(a_codes, b_codes, sa, sb):
    a, b = decode_e4m3(a_codes) * np.reshape(sa, (-1, 1)), decode_e4m3(b_codes) * np.reshape(sb, (-1, 1))
    return a @ b.T


def cross_entropy(l, targets):
    """(loss per row, log of the sum of exponentials, [mean, 1 / count])."""
    top = l.max(1)
    lse = top + np.log(np.exp(l - top[:, None]).sum(1))
    counted = targets >= 0
    loss = np.where(counted, lse - l[np.arange(len(l)), np.maximum(targets, 0)], 0.0)
    n = counted.sum()
    return loss, lse, np.array([loss.sum() / n, 1 / n]) if n else np.zeros(2)


def cross_entropy_grad(l, targets, dloss):
    """Gradient of sum dloss loss with respect to the logits."""
    top = l.max(1, keepdims=True)
    p = np.exp(l - top)
    p /= p.sum(1, keepdims=True)
    p[np.arange(len(l)), np.maximum(targets, 0)] -= 1
    return p * np.where(targets >= 0, np.broadcast_to(dloss, targets.shape), 0.0)[:, None]
