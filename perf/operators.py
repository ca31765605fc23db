"""The operators around a feed-forward block: their cases, inputs and plain forms.

Four operators, in the forms in which a transformer's feed-forward sublayer uses them:

* ``ln_fwd``  layer norm of the rows of X[M][D], with the row statistics that a backward
  pass needs:  y = (x - mean) * rstd * gamma + beta,  rstd = 1 / sqrt(var + eps);
* ``ln_bwd``  its backward pass:  g = dy * gamma,  xhat = (x - mean) * rstd,
  dx = rstd * (g - avg(g) - xhat * avg(g * xhat)),  dgamma = sum_rows dy * xhat,
  dbeta = sum_rows dy;
* ``w8a8``    a linear layer in 8-bit integers: each token (row of X) is quantised by its
  largest magnitude, s = max|x| / 127, q = round(x / s) to the nearest integer (ties to
  even), and y[m][n] = s[m] * t[n] * sum_k q[m][k] * w[n][k] + b[n], where the int8 weight
  w[n][:] has the scale t[n];
* ``moe``     a mixture-of-experts feed-forward layer for a few tokens: logits of the router,
  the top_k experts of each token (a tie goes to the lower index), their softmax weights,
  act(x W_up[e]^T + b_up[e]) W_down[e]^T + b_down[e] for each of them, summed by weight.

``run`` computes a plain form from elementary torch operations where ``own`` is false, and
calls the package's operators where it is true.
"""
import math

import torch

own = False

DTYPES = {"f16": torch.float16, "bf16": torch.bfloat16}
EPS = 1e-5


# ---------------------------------------------------------------------------
# Cases
# ---------------------------------------------------------------------------

def _ln(op, M, D, dtype, affine=True, pad=0):
    return {"op": op, "M": M, "D": D, "dtype": dtype, "affine": affine, "pad": pad}


def _w8a8(M, N, K, dtype, bias=False, pad=0):
    return {"op": "w8a8", "M": M, "N": N, "K": K, "dtype": dtype, "bias": bias, "pad": pad}


def _moe(T, D, F, E, k, act, dtype, bias=False, normalize=True):
    return {"op": "moe", "T": T, "D": D, "F": F, "E": E, "top_k": k, "act": act, "dtype": dtype, "bias": bias,
            "normalize": normalize}


def listed():
    return [
        # a decoding step of eight sequences: the latency of the call
        {"name": "ln_fwd_decode_8x1280_bf16", **_ln("ln_fwd", 8, 1280, "bf16")},
        # the pre-norm of the SigLIP MLP: 729 image patches, rows of 4.5 warps of 16-byte vectors
        {"name": "ln_fwd_siglip_729x1152_f16", **_ln("ln_fwd", 729, 1152, "f16")},
        # a training batch of SDXL level-1 tokens (larger than the L2 cache)
        {"name": "ln_fwd_batch_65536x640_bf16", **_ln("ln_fwd", 65536, 640, "bf16")},
        # the backward pass of the SigLIP pre-norm for one image
        {"name": "ln_bwd_siglip_729x1152_f16", **_ln("ln_bwd", 729, 1152, "f16")},
        # odd rows of a slice of a wider tensor (pitch 649): almost no row starts on a 16-byte boundary
        {"name": "ln_bwd_odd_1000x643_bf16", **_ln("ln_bwd", 1000, 643, "bf16", True, 6)},
        # a training batch of SDXL level-2 tokens (larger than the L2 cache)
        {"name": "ln_bwd_batch_32768x1280_bf16", **_ln("ln_bwd", 32768, 1280, "bf16")},
        # a decoding step of four sequences through the SDXL level-2 projection: the weight's bytes count
        {"name": "w8a8_decode_4x10240x1280_bf16", **_w8a8(4, 10240, 1280, "bf16", True)},
        # the SigLIP up projection: a ragged last row block
        {"name": "w8a8_siglip_729x4304x1152_f16", **_w8a8(729, 4304, 1152, "f16")},
        # the same projection for a batch of 16384 tokens: matrix-product bound
        {"name": "w8a8_batch_16384x4304x1152_f16", **_w8a8(16384, 4304, 1152, "f16")},
        # one token of a decoding step, two of eight GEGLU experts of the SDXL level-2 size
        {"name": "moe_token_1of8x1280x5120_bf16", **_moe(1, 1280, 5120, 8, 2, "geglu", "bf16")},
        # nine tokens over sixteen biased tanh-GELU experts of the SigLIP size: most experts have a token or two
        {"name": "moe_ragged_9of16x1152x4304_f16", **_moe(9, 1152, 4304, 16, 2, "gelu_tanh", "f16", True)},
        # sixty-four tokens over thirty-two GEGLU experts, four each: every expert's weights are read
        {"name": "moe_batch_64of32x1280x5120_bf16", **_moe(64, 1280, 5120, 32, 4, "geglu", "bf16")},
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["ln_fwd", "ln_bwd", "w8a8", "moe"])
    dtype = rng.choice(["f16", "bf16"])
    if op in ("ln_fwd", "ln_bwd"):
        while True:
            M, D = _log(rng, 1, 65536), _log(rng, 8, 16384)
            if M * D <= 65536 * 640:
                break
        if rng.random() < 0.6:
            D = max(8, D // 8 * 8)
        return _ln(op, M, D, dtype, rng.random() < 0.8, rng.choice([0, 0, 8, 3]))
    if op == "w8a8":
        while True:
            M, N, K = _log(rng, 1, 16384), _log(rng, 8, 16384), max(16, _log(rng, 64, 8192) // 16 * 16)
            if M * N * K <= 16384 * 4304 * 1152 and M * K <= 1 << 25 and N * K <= 1 << 26 and M * N <= 16384 * 4304:
                break
        return _w8a8(M, N, K, dtype, rng.random() < 0.5, rng.choice([0, 0, 16]))
    act = rng.choice(["geglu", "gelu_erf", "gelu_tanh", "silu"])
    while True:
        T, E = _log(rng, 1, 64), _log(rng, 2, 64)
        D, F = max(64, _log(rng, 64, 2560) // 8 * 8), max(64, _log(rng, 64, 8192) // 8 * 8)
        if E * D * F * (3 if act == "geglu" else 2) <= 32 * 1280 * 5120 * 3:
            break
    return _moe(T, D, F, E, rng.randint(1, min(E, 8)), act, dtype, rng.random() < 0.5, rng.random() < 0.5)


def work(case):
    """What one pass cannot do without: inputs read once, outputs written once."""
    if case["op"] == "ln_fwd":
        M, D = case["M"], case["D"]
        return {"bytes": 4 * M * D + 8 * M + (4 * D if case["affine"] else 0), "flops": 8 * M * D}
    if case["op"] == "ln_bwd":
        M, D = case["M"], case["D"]
        return {"bytes": 6 * M * D + 8 * M + (10 * D if case["affine"] else 8 * D), "flops": 14 * M * D}
    if case["op"] == "w8a8":
        M, N, K = case["M"], case["N"], case["K"]
        return {"bytes": 2 * M * K + N * K + 4 * N + 4 * M + 2 * M * N + (2 * N if case["bias"] else 0),
                "flops": 2 * M * N * K}
    T, D, F, E, k = (case[n] for n in ("T", "D", "F", "E", "top_k"))
    rows = (2 if case["act"] == "geglu" else 1) * F
    touched = int(E * (1.0 - (1.0 - k / E) ** T))  # experts that T tokens reach, on average
    touched = max(k, min(touched, E))
    per = (rows + F) * D
    return {"bytes": 2 * touched * (per + (rows + D if case["bias"] else 0)) + 2 * E * D + 4 * T * D + 8 * T * k,
            "flops": 2 * T * k * per + 2 * T * E * D}


# ---------------------------------------------------------------------------
# Inputs
# ---------------------------------------------------------------------------

def _rows(gen, M, D, pad, dtype, scale=1.0):
    """Rows as a residual stream has them: each with a scale and an offset of its own; the row pitch is D + pad."""
    x = torch.randn(M, D + pad, generator=gen, device="cuda")
    x *= scale * (0.25 + 2.0 * torch.rand(M, 1, generator=gen, device="cuda"))
    x += torch.randn(M, 1, generator=gen, device="cuda")
    return x.to(dtype)[:, :D]


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    dt = DTYPES[case["dtype"]]
    st = {"case": dict(case), "dtype": dt}

    def randn(*shape, std=1.0):
        return (torch.randn(*shape, generator=gen, device="cuda") * std).to(dt)

    if case["op"] in ("ln_fwd", "ln_bwd"):
        M, D = case["M"], case["D"]
        st["X"] = _rows(gen, M, D, case["pad"], dt)
        st["gamma"] = (1.0 + 0.2 * torch.randn(D, generator=gen, device="cuda")).to(dt) if case["affine"] else None
        st["beta"] = randn(D, std=0.1) if case["affine"] else None
        if case["op"] == "ln_fwd":
            st["Y"] = torch.empty(M, D, dtype=dt, device="cuda")
            st["mean"], st["rstd"] = torch.empty(M, device="cuda"), torch.empty(M, device="cuda")
        else:
            st["dY"] = randn(M, D + case["pad"], std=0.5)[:, :D]
            x = st["X"].double()  # the forward pass's statistics
            mean = x.mean(1)
            st["mean"] = mean.float()
            st["rstd"] = (1.0 / torch.sqrt((x - mean[:, None]).square_().mean(1) + EPS)).float()
            st["dX"] = torch.empty(M, D, dtype=dt, device="cuda")
            st["dgamma"], st["dbeta"] = torch.empty(D, device="cuda"), torch.empty(D, device="cuda")
            if own:
                from transformer_mlp_gemms_gb300 import kt_ops
                st["workspace"] = kt_ops.layernorm_backward_workspace(M, D)
    elif case["op"] == "w8a8":
        M, N, K = case["M"], case["N"], case["K"]
        st["X"] = _rows(gen, M, K, case["pad"], dt, 0.5)
        st["X"][:, 3::97] *= 8.0  # a few channels carry far larger values, as activations' do
        w = torch.randn(N, K, generator=gen, device="cuda") / math.sqrt(K)
        st["wscale"] = w.abs().amax(1) / 127.0
        st["W"] = torch.round(w / st["wscale"][:, None]).clamp_(-127, 127).to(torch.int8)
        st["bias"] = randn(N, std=math.sqrt(0.02)) if case["bias"] else None
        st["Q"] = torch.empty(M, K, dtype=torch.int8, device="cuda")
        st["scale"] = torch.empty(M, device="cuda")
        st["Y"] = torch.empty(M, N, dtype=dt, device="cuda")
    else:
        T, D, F, E, k = (case[n] for n in ("T", "D", "F", "E", "top_k"))
        rows = (2 if case["act"] == "geglu" else 1) * F
        st["X"] = randn(T, D)
        st["W_router"] = randn(E, D, std=1.0 / math.sqrt(D))
        st["W_up"] = randn(E, rows, D, std=1.0 / math.sqrt(D))
        st["W_down"] = randn(E, D, F, std=1.0 / math.sqrt(F))
        st["b_up"] = randn(E, rows, std=math.sqrt(0.02)) if case["bias"] else None
        st["b_down"] = randn(E, D, std=math.sqrt(0.02)) if case["bias"] else None
        st["Y"] = torch.empty(T, D, dtype=dt, device="cuda")
        st["ids"] = torch.empty(T, k, dtype=torch.int32, device="cuda")
        st["weights"] = torch.empty(T, k, device="cuda")
        if own:
            from transformer_mlp_gemms_gb300 import kt_mlp, kt_ops
            act = {"geglu": kt_mlp.KT_ACT_GEGLU, "gelu_erf": kt_mlp.KT_ACT_GELU_ERF,
                   "gelu_tanh": kt_mlp.KT_ACT_GELU_TANH, "silu": kt_mlp.KT_ACT_SILU}[case["act"]]
            st["plan"] = kt_ops.MoePlan(T, D, F, E, k, act, kt_mlp.KT_F16 if case["dtype"] == "f16" else kt_mlp.KT_BF16,
                                        bias=case["bias"], normalize=case["normalize"])
    return st


# ---------------------------------------------------------------------------
# One pass
# ---------------------------------------------------------------------------

def run(st):
    op = st["case"]["op"]
    if own:
        return _OWN[op](st)
    return _PLAIN[op](st)


def _own_ln_fwd(st):
    from transformer_mlp_gemms_gb300 import kt_ops
    kt_ops.kt_layernorm_forward(st["X"], st["gamma"], st["beta"], EPS, st["Y"], st["mean"], st["rstd"])
    return {"y": st["Y"], "mean": st["mean"], "rstd": st["rstd"]}


def _own_ln_bwd(st):
    from transformer_mlp_gemms_gb300 import kt_ops
    kt_ops.kt_layernorm_backward(st["dY"], st["X"], st["gamma"], st["mean"], st["rstd"], st["dX"], st["dgamma"],
                                 st["dbeta"], st["workspace"])
    return {"dx": st["dX"], "dgamma": st["dgamma"], "dbeta": st["dbeta"]}


def _own_w8a8(st):
    from transformer_mlp_gemms_gb300 import kt_ops
    kt_ops.kt_quantize_rows(st["X"], st["Q"], st["scale"])
    kt_ops.kt_linear_i8(st["Q"], st["scale"], st["W"], st["wscale"], st["bias"], st["Y"])
    return {"y": st["Y"], "scale": st["scale"]}


def _own_moe(st):
    st["plan"].run(st["X"], st["W_router"], st["W_up"], st["W_down"], st["Y"], st["b_up"], st["b_down"],
                   ids=st["ids"], weights=st["weights"])
    return {"y": st["Y"], "ids": st["ids"], "weights": st["weights"]}


def _plain_ln_fwd(st):
    x = st["X"].float()
    mean = x.mean(1)
    xc = x - mean[:, None]
    rstd = 1.0 / torch.sqrt((xc * xc).mean(1) + EPS)
    y = xc * rstd[:, None]
    if st["gamma"] is not None:
        y = y * st["gamma"].float() + st["beta"].float()
    return {"y": y.to(st["dtype"]), "mean": mean, "rstd": rstd}


def _plain_ln_bwd(st):
    dy, x = st["dY"].float(), st["X"].float()
    rstd = st["rstd"][:, None]
    xhat = (x - st["mean"][:, None]) * rstd
    g = dy * st["gamma"].float() if st["gamma"] is not None else dy
    dx = rstd * (g - g.mean(1, keepdim=True) - xhat * (g * xhat).mean(1, keepdim=True))
    return {"dx": dx.to(st["dtype"]), "dgamma": (dy * xhat).sum(0), "dbeta": dy.sum(0)}


def _plain_w8a8(st):
    x = st["X"].float()
    most = x.abs().amax(1)
    scale = most / torch.full_like(most, 127.0)  # a division by a plain number is a product with its rounded inverse
    # the quotient in 64 bits: rounded to 32 it could land on a tie that it does not have
    q = torch.round(x.double() / torch.where(scale > 0, scale, 1.0).double()[:, None]).clamp_(-127, 127).float()
    y = torch.matmul(q, st["W"].float().t()) * (scale[:, None] * st["wscale"])
    if st["bias"] is not None:
        y = y + st["bias"].float()
    return {"y": y.to(st["dtype"]), "scale": scale}


def _act(p, act):
    if act == "geglu":
        value, gate = p.chunk(2, -1)
        return value * _act(gate, "gelu_erf")
    if act == "gelu_erf":
        return 0.5 * p * torch.special.erfc(p * -math.sqrt(0.5))
    if act == "gelu_tanh":
        return p / (1.0 + torch.exp(-2.0 * math.sqrt(2.0 / math.pi) * (p + 0.044715 * p * p * p)))
    return p / (1.0 + torch.exp(-p))


def _route(case, x, w_router, dtype):
    """ids and weights of each token's experts; the logits in 64 bits, because an order hangs on them."""
    logits = torch.matmul(x.double(), w_router.double().t())
    top, ids = (v[:, :case["top_k"]] for v in torch.sort(logits, dim=1, descending=True, stable=True))
    p = torch.exp((top - logits.amax(1, keepdim=True)).to(dtype))
    if case["normalize"]:
        return ids, p / p.sum(1, keepdim=True)
    return ids, p / torch.exp((logits - logits.amax(1, keepdim=True)).to(dtype)).sum(1, keepdim=True)


def _plain_moe(st):
    case, x = st["case"], st["X"].float()
    T, E, k = case["T"], case["E"], case["top_k"]
    ids, weights = _route(case, st["X"], st["W_router"], torch.float32)
    token = torch.arange(T, device=x.device)[:, None].expand(T, k)
    if T * k < E:  # fewer pairs of a token and an expert than experts: each pair takes its expert's weights
        pick = ids.reshape(-1)
        x = x[token.reshape(-1)][:, None]
        place = (torch.arange(T * k, device=x.device).view(T, k), 0)
    else:  # else every expert sees every token
        pick = slice(None)
        place = (ids, token)
    p = torch.matmul(x, st["W_up"][pick].float().transpose(1, 2))
    if st["b_up"] is not None:
        p = p + st["b_up"][pick].float()[:, None]
    z = torch.matmul(_act(p, case["act"]), st["W_down"][pick].float().transpose(1, 2))
    if st["b_down"] is not None:
        z = z + st["b_down"][pick].float()[:, None]
    y = (z[place] * weights[:, :, None]).sum(1)
    return {"y": y.to(st["dtype"]), "ids": ids.int(), "weights": weights}


_OWN = {"ln_fwd": _own_ln_fwd, "ln_bwd": _own_ln_bwd, "w8a8": _own_w8a8, "moe": _own_moe}
_PLAIN = {"ln_fwd": _plain_ln_fwd, "ln_bwd": _plain_ln_bwd, "w8a8": _plain_w8a8, "moe": _plain_moe}


# ---------------------------------------------------------------------------
# The definitions in 64 bits
# ---------------------------------------------------------------------------

def exact(case, seed):
    st = prepare(case, seed)
    return {"ln_fwd": _exact_ln_fwd, "ln_bwd": _exact_ln_bwd, "w8a8": _exact_w8a8, "moe": _exact_moe}[case["op"]](st)


def _exact_ln_fwd(st):
    x = st["X"].to(torch.float64)
    n = x.shape[1]
    mean = x.sum(1) / n
    var = ((x - mean.unsqueeze(1)) ** 2).sum(1) / n
    rstd = (var + EPS) ** -0.5
    y = (x - mean.unsqueeze(1)) * rstd.unsqueeze(1)
    if st["gamma"] is not None:
        y = st["gamma"].double() * y + st["beta"].double()
    return {"y": y, "mean": mean, "rstd": rstd}


def _exact_ln_bwd(st):
    dy, x = st["dY"].to(torch.float64), st["X"].to(torch.float64)
    n = x.shape[1]
    r = st["rstd"].double().unsqueeze(1)
    xhat = (x - st["mean"].double().unsqueeze(1)) * r
    g = dy if st["gamma"] is None else dy * st["gamma"].double()
    a, b = g.sum(1, keepdim=True), (g * xhat).sum(1, keepdim=True)
    return {"dx": (n * g - a - xhat * b) * (r / n), "dgamma": torch.einsum("md,md->d", dy, xhat),
            "dbeta": torch.ones(x.shape[0], dtype=torch.float64, device=x.device) @ dy}


def _exact_w8a8(st):
    x = st["X"].to(torch.float64)
    scale = (x.abs().max(1).values / 127).float().double()  # the definition's scale is a 32-bit number
    q = (x / scale.clamp_min(1e-300).unsqueeze(1)).round().clamp(-127, 127)
    y = (q @ st["W"].double().t()) * scale.unsqueeze(1) * st["wscale"].double()
    return {"y": y if st["bias"] is None else y + st["bias"].double(), "scale": scale}


def _exact_moe(st):
    case, x = st["case"], st["X"].double()
    logits = x @ st["W_router"].double().t()
    prob = torch.softmax(logits, 1)
    order = torch.argsort(logits, dim=1, descending=True, stable=True)[:, :case["top_k"]]
    weights = prob.gather(1, order)
    if case["normalize"]:
        weights = weights / weights.sum(1, keepdim=True)
    y = torch.zeros_like(x)
    for e in range(case["E"]):
        t, j = torch.nonzero(order == e, as_tuple=True)
        if not t.numel():
            continue
        p = x[t] @ st["W_up"][e].double().t()
        if st["b_up"] is not None:
            p = p + st["b_up"][e].double()
        if case["act"] == "geglu":
            gate = p[:, case["F"]:]
            h = p[:, :case["F"]] * gate * 0.5 * (1.0 + torch.erf(gate / math.sqrt(2.0)))
        elif case["act"] == "gelu_erf":
            h = p * 0.5 * (1.0 + torch.erf(p / math.sqrt(2.0)))
        elif case["act"] == "gelu_tanh":
            h = 0.5 * p * (1.0 + torch.tanh(math.sqrt(2.0 / math.pi) * (p + 0.044715 * p ** 3)))
        else:
            h = p * torch.sigmoid(p)
        z = h @ st["W_down"][e].double().t()
        if st["b_down"] is not None:
            z = z + st["b_down"][e].double()
        y.index_add_(0, t, z * weights[t, j].unsqueeze(1))
    return {"y": y, "ids": None, "weights": weights}
