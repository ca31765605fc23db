"""Plain 64-bit forms of the operators around the MLP, and the error bounds that the tests allow.

A bound counts roundings: ``half(dtype)`` relative for the one rounding of an output, and
U = 2^-24 relative for each fp32 operation, times the length of the longest chain of additions in
a sum (``CHAIN``: 40 terms in a lane, 5 shuffles, 16 warps, and a few operations around them)."""
import math

import torch

U = 2.0 ** -24
CHAIN = 96


def half(dtype):
    return torch.finfo(dtype).eps / 2


def floor(dtype):
    """Half the spacing of the subnormal numbers."""
    return torch.finfo(dtype).smallest_normal * torch.finfo(dtype).eps / 2


def layernorm(x, gamma, beta, eps):
    """(y, mean, rstd) in 64 bits."""
    x = x.double()
    mean = x.mean(1)
    d = x - mean[:, None]
    rstd = 1.0 / torch.sqrt((d * d).mean(1) + eps)
    y = d * rstd[:, None]
    if gamma is not None:
        y = y * gamma.double() + beta.double()
    return y, mean, rstd


def layernorm_bounds(x, gamma, beta, y, rstd, dtype):
    """How far (y, mean, rstd) may be off.  The kernel takes deviations from the row's first
    element: its mean is off by CHAIN roundings of their average magnitude A, and so is every
    deviation; the variance's error is of second order in that, and CHAIN / 2 of its roundings
    reach rstd."""
    x = x.double()
    A = (x - x[:, :1]).abs().mean(1)
    off = CHAIN * U * A
    r = CHAIN * U + (off * rstd) ** 2
    mean_tol = off + 2 * U * (x[:, 0].abs() + A)
    g = gamma.double().abs() if gamma is not None else torch.ones_like(x[0])
    b = beta.double().abs() if beta is not None else torch.zeros_like(x[0])
    xhat = (x - x.mean(1, keepdim=True)).abs() * rstd[:, None]
    y_tol = half(dtype) * y.abs() + floor(dtype) + g * ((off * rstd)[:, None] + xhat * (r[:, None] + 4 * U)) * 1.01 + 4 * U * b
    return y_tol, mean_tol, rstd * r


def layernorm_bounds_about_the_mean(x, gamma, beta, y, mean, rstd, dtype):
    """As layernorm_bounds, for rows whose first element may be anything.  The kernel's deviations
    are those from an origin o, the number of the row's type nearest to a first mean that is off by
    CHAIN roundings of avg|x|; the mean is o plus the deviations' average, which is off by CHAIN
    roundings of B = avg|x - o|, the variance their squares' average less that average's square,
    and so no worse than CHAIN roundings of 1 + (the average over the spread)^2.  (The bounds of
    layernorm_bounds hold too: o is at most as far from the mean as the first element is.)"""
    x = x.double()
    apart = half(dtype) * mean.abs() + floor(dtype) + CHAIN * U * x.abs().mean(1)  # |mean - o|
    off = CHAIN * U * ((x - mean[:, None]).abs().mean(1) + apart)
    r = CHAIN * U * (1.0 + (apart * rstd) ** 2) + (off * rstd) ** 2
    g = gamma.double().abs() if gamma is not None else torch.ones_like(x[0])
    b = beta.double().abs() if beta is not None else torch.zeros_like(x[0])
    xhat = (x - mean[:, None]).abs() * rstd[:, None]
    y_tol = half(dtype) * y.abs() + floor(dtype) + g * ((off * rstd)[:, None] + xhat * (r[:, None] + 4 * U)) * 1.01 + 4 * U * b
    return y_tol, off + 2 * U * mean.abs(), rstd * r


def layernorm_backward(dy, x, gamma, mean, rstd):
    """(dx, dgamma, dbeta) in 64 bits."""
    dy, x, r = dy.double(), x.double(), rstd.double()[:, None]
    xhat = (x - mean.double()[:, None]) * r
    g = dy * gamma.double() if gamma is not None else dy
    dx = r * (g - g.mean(1, keepdim=True) - xhat * (g * xhat).mean(1, keepdim=True))
    return dx, (dy * xhat).sum(0), dy.sum(0)


def layernorm_backward_bounds(dy, x, gamma, mean, rstd, dx, dtype):
    dy, x, r = dy.double(), x.double(), rstd.double()[:, None]
    xhat = ((x - mean.double()[:, None]) * r).abs()
    g = (dy * gamma.double() if gamma is not None else dy).abs()
    dx_tol = half(dtype) * dx.abs() + floor(dtype) + \
        CHAIN * U * r * (g + g.mean(1, keepdim=True) + xhat * (g * xhat).mean(1, keepdim=True))
    # a column's sum: the rows of one team in turn, 8 teams, up to 160 blocks in runs of 20
    chain = (x.shape[0] / 152 + 48) * U
    return dx_tol, chain * (dy.abs() * xhat).sum(0) + 1e-30, chain * dy.abs().sum(0) + 1e-30


def quantize(v):
    """(q, scale) of the rows of v (exact fp32 values): the definition, ties to even."""
    v = v.float()
    bad = ~torch.isfinite(v).all(1)
    most = torch.where(bad[:, None], 0.0, v).abs().amax(1)
    scale = most / torch.full_like(most, 127.0)
    q = torch.round(v.double() / torch.where(scale > 0, scale, 1.0).double()[:, None]).clamp(-127, 127)
    q = torch.where((bad | (scale == 0))[:, None], 0.0, q)
    return q.to(torch.int8), torch.where(bad, float("nan"), scale)


def linear_i8(q, sx, w, sw, bias):
    """(y, bound without the output's rounding): exact integer sums, then three fp32 roundings."""
    s = torch.matmul(q.double(), w.double().t())
    y = s * sx.double()[:, None] * sw.double()
    tol = 4 * U * y.abs()
    if bias is not None:
        tol = tol + 2 * U * bias.double().abs()
        y = y + bias.double()
    return y, tol


def act(p, name):
    if name == "geglu":
        value, gate = p.chunk(2, -1)
        return value * act(gate, "gelu_erf")
    if name == "gelu_erf":
        return 0.5 * p * torch.special.erfc(p * -math.sqrt(0.5))
    if name == "gelu_tanh":
        return 0.5 * p * (1.0 + torch.tanh(math.sqrt(2.0 / math.pi) * (p + 0.044715 * p ** 3)))
    if name == "gelu_sigmoid":
        return p * torch.sigmoid(1.702 * p)
    if name == "silu":
        return p * torch.sigmoid(p)
    return p


def route(x, w_router, top_k, normalize):
    logits = x.double() @ w_router.double().t()
    order = torch.sort(logits, dim=1, descending=True, stable=True)[1][:, :top_k]
    prob = torch.softmax(logits, 1)
    w = prob.gather(1, order)
    return order, w / w.sum(1, keepdim=True) if normalize else w


def moe(x, w_router, w_up, w_down, b_up, b_down, R, top_k, name, normalize, dtype):
    """(y, ids, weights, bound of y) in 64 bits.  The bound follows the kernel's steps: a sum of K
    products in the tensor cores is off by at most K 2^-23 of its terms' magnitudes; the
    activation by 2e-5 of its value beyond that, passed on with a slope of at most 1.15; the
    hidden layer's two parts keep it to half(dtype)^2; a weight is off by a few roundings."""
    ids, weights = route(x, w_router, top_k, normalize)
    y, tol = torch.zeros_like(x, dtype=torch.float64), torch.zeros_like(x, dtype=torch.float64)
    X = x.double()
    D, F = x.shape[1], w_down.shape[2]
    for e in range(w_router.shape[0]):
        t, j = torch.nonzero(ids == e, as_tuple=True)
        if not t.numel():
            continue
        wu, wd = w_up[e].double(), w_down[e].double()
        p = X[t] @ wu.t()
        dp = (D * 2 + 4) * U * (X[t].abs() @ wu.abs().t())
        if b_up is not None:
            p = p + b_up[e].double()
            dp = dp + 2 * U * p.abs()
        h = act(p, name)
        if name == "geglu":
            value, gate = p.chunk(2, -1)
            dv, dg = dp.chunk(2, -1)
            dh = dv * act(gate, "gelu_erf").abs() + value.abs() * 1.15 * dg + dv * 1.15 * dg
        else:
            dh = 1.15 * dp
        dh = dh + (2e-5 + half(dtype) ** 2) * h.abs() + floor(dtype)
        z = h @ wd.t()
        dz = dh @ wd.abs().t() + (F * 4 + 16) * U * (h.abs() @ wd.abs().t())
        if b_down is not None:
            z = z + b_down[e].double()
            dz = dz + 2 * U * z.abs()
        w = weights[t, j].unsqueeze(1)
        y.index_add_(0, t, z * w)
        tol.index_add_(0, t, dz * w + 64 * U * w * z.abs())
    if R is not None:
        y = y + R.double()
    return y, ids, weights, tol + (half(dtype) + 4 * U) * y.abs() + floor(dtype)
