"""Plain 64-bit forms of the gated block, the linear layer, AdamW and the linear layer in 8-bit floating point, and the
error bounds that the tests allow.

A bound counts roundings: ``half(dtype)`` relative for the one rounding of a 16-bit number, U = 2^-24 for an fp32
operation, and 2 K U of the terms' magnitudes for a sum of K products on the tensor cores (each step of an fp32
sum off by 2^-23 at most).  The activations take their exponentials from the hardware's 2^x and reciprocal:
with |x| below 32 where they matter, an exponent off by 32 U ln 2 and two approximations of 2^-22 make SLOPE = 1e-5 a
generous bound, relative for act(g) and absolute for act'(g) (which is below 1.2 and passes zero).  The reciprocal and
2^x flush what is below 2^-126 to zero: a sigmoid s (or a normal distribution's tail) is off by 2^-126 more, and
so are act = g s by |g| of that and act' = s + g s (1 - s) c' by 1 + |g| c', where c' <= 1.6 + 0.22 g^2."""
import math

import torch

from ops_reference import U, floor, half

SLOPE = 1e-5


def flushed(g):
    g = g.abs()
    return 2.0 ** -126 * (2.0 + 2.0 * g + g ** 3)


def act(g, name):
    """act(g) and act'(g)."""
    if name == "gelu_erf":
        cdf = 0.5 * torch.special.erfc(-g / math.sqrt(2.0))
        return g * cdf, cdf + g * torch.exp(-0.5 * g * g) / math.sqrt(2.0 * math.pi)
    if name == "gelu_tanh":
        c = 2.0 * math.sqrt(2.0 / math.pi)
        s = torch.sigmoid(c * (g + 0.044715 * g ** 3))
        return g * s, s + g * s * (1.0 - s) * c * (1.0 + 3 * 0.044715 * g * g)
    if name == "none":
        return g, torch.ones_like(g)
    a = 1.702 if name == "gelu_sigmoid" else 1.0
    s = torch.sigmoid(a * g)
    return g * s, s + a * g * s * (1.0 - s)


def product(a, b, bias=None):
    """(a b^T (+ bias), bound before the rounding) for 64-bit a [M][K], b [N][K]."""
    y = a @ b.t()
    tol = (2 * a.shape[1] + 4) * U * (a.abs() @ b.abs().t())
    if bias is not None:
        y = y + bias.double()
        tol = tol + 2 * U * y.abs()
    return y, tol


def rounded(y, tol, dtype):
    return tol * 1.01 + half(dtype) * y.abs() + floor(dtype)


def glu(x, w, bias, name, dtype):
    """(h, bound, p, bound)."""
    p, tol = product(x.double(), w.double(), bias)
    value, gate = p.chunk(2, 1)
    dv, dg = tol.chunk(2, 1)
    a, _ = act(gate, name)
    h = value * a
    da = 1.2 * dg + SLOPE * a.abs() + flushed(gate)
    return h, rounded(h, dv * a.abs() + value.abs() * da + dv * da, dtype), p, rounded(p, tol, dtype)


def glu_backward(dh, p, x, w, name, dtype):
    """(dx, bound, dw, bound, db, bound) from the kept p: dp is rounded once, then two products."""
    dh, x, w = dh.double(), x.double(), w.double()
    value, gate = p.double().chunk(2, 1)
    a, da = act(gate, name)
    dp = torch.cat([dh * a, dh * value * da], 1)
    flush = flushed(gate)
    exact = torch.cat([dh.abs() * (SLOPE * a.abs() + flush), (dh * value).abs() * (SLOPE + flush)], 1) + 8 * U * dp.abs()  # before dp's rounding
    off = exact + half(dtype) * dp.abs() + floor(dtype)
    dx, tx = product(dp, w.t())
    dw, tw = product(dp.t(), x.t())
    chain = (dp.shape[0] / 8 + 160) * U  # a warp's rows, eight warps, up to 128 blocks
    db, tb = dp.sum(0), exact.sum(0) + chain * dp.abs().sum(0)
    return (dx, rounded(dx, tx + 1.01 * off @ w.abs(), dtype), dw, rounded(dw, tw + 1.01 * off.t() @ x.abs(), dtype), db, tb + 1e-30)


def linear_backward(dy, x, w, dtype):
    """(dx, bound, dw, bound, db, bound)."""
    dy, x, w = dy.double(), x.double(), w.double()
    dx, tx = product(dy, w.t())
    dw, tw = product(dy.t(), x.t())
    chain = (dy.shape[0] / 8 + 160) * U
    return dx, rounded(dx, tx, dtype), dw, rounded(dw, tw, dtype), dy.sum(0), chain * dy.abs().sum(0) + 1e-30


def e4m3(v, size, root=False):
    """(q, scale) of the last dimension of v (fp32) in runs of ``size``."""
    K = v.shape[-1]
    runs = torch.nn.functional.pad(v.float(), (0, -K % size)).view(*v.shape[:-1], -1, size)
    most = runs.abs().amax(-1)
    top = torch.full_like(most, 448.0)
    zero = most < 2.0 ** -100
    scale = torch.where(zero, 0.0, most / top)
    q = runs * torch.where(zero, 0.0, top / most)[..., None]
    q = torch.where(zero[..., None], 0.0, q)
    if root:
        q = torch.where(q > 0, q.clamp_min(2.0 ** -9), q)
    return q.to(torch.float8_e4m3fn).flatten(-2)[..., :K], scale


def widen(q, scale, size):
    """The values that e4m3 numbers with a scale for each run of the last dimension stand for, in fp32."""
    return q.float() * scale.repeat_interleave(size, -1)[..., :q.shape[-1]]


def linear_fp8(q, sx, w, sw, bias):
    """(y, bound without the output's rounding): the runs' sums on the tensor cores, then a product of scales, an fp32 sum
    over the runs and the bias."""
    N, K = w.shape
    x = q.double() * sx.double().repeat_interleave(128, 1)[:, :K]
    v = w.double() * sw.double().repeat_interleave(128, 0)[:N].repeat_interleave(128, 1)[:, :K]
    y = x @ v.t()
    tol = (2 * 128 + 2 * sx.shape[1] + 8) * U * (x.abs() @ v.abs().t())
    if bias is not None:
        y = y + bias.double()
        tol = tol + 2 * U * bias.double().abs()
    return y, tol


def adamw(p, g, m, v, step, lr, beta1, beta2, eps, decay, grad_scale=None):
    """(p, m, v, r) in fp32, each operation rounded on its own."""
    f = torch.float32
    p, g = p.to(f), g.to(f)
    if grad_scale is not None:
        g = g * grad_scale
    m = m * beta1 + g * (1.0 - beta1)
    v = v * beta2 + (g * (1.0 - beta2)) * g
    r = torch.sqrt(v)
    p = p * (1.0 - lr * decay) - (m * (lr / (1.0 - beta1 ** step))) / (r * (1.0 / math.sqrt(1.0 - beta2 ** step)) + eps)
    return p, m, v, r
