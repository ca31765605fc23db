"""Training and serving of a gated feed-forward block: the operators' cases, inputs and plain forms.

Five operators, in the forms in which a training step and a server use them.  Weights are [out][in].

* ``glu_fwd``  the gated up projection:  [value | gate] = X W^T + b,  h = value * act(gate); a training
  step keeps p = [value | gate] for the backward pass, a server does not;
* ``glu_bwd``  its gradients from dh and the kept p:  dvalue = dh * act(gate),
  dgate = dh * value * act'(gate),  dx = [dvalue | dgate] W,  dW = [dvalue | dgate]^T X,  db = the sums
  of [dvalue | dgate] over the tokens (fp32);
* ``linear``   a linear layer (the down projection) forward and backward, as one training step takes it:
  y = X W^T + b,  dx = dy W,  dW = dy^T X,  db = sum of dy over the tokens (fp32);
* ``fp8``      a linear layer in 8-bit floating point (e4m3) with a scale for each block of 128: each
  token's activations are quantised in runs of 128 columns,  s = max|x| / 448,  q = e4m3(x * (448 / max|x|))
  (both quotients in fp32), and  y[m][n] = sum over runs j of s[m][j] t[n / 128][j] sum_k q[m][k] w[n][k] + b[n]
  with a weight scale t for each 128 x 128 block;
* ``adamw``    one AdamW step over many tensors at once, in fp32 with every operation rounded on its own:
  m = b1 m + (1 - b1) g,  v = b2 v + ((1 - b2) g) g,  r = sqrt(v),
  p = p (1 - lr wd) - (m (lr / (1 - b1^t))) / (r / sqrt(1 - b2^t) + eps);  the moments are held in fp32, or in
  e4m3 with a scale for each 256 values of a tensor: m itself, and r in the place of v (r > 0 as 2^-9 at
  least, so that no step divides by a root that was rounded away).

``run`` computes a plain form from elementary torch operations where ``own`` is false, and calls the
package's operators where it is true.
"""
import math

import torch

own = False

DTYPES = {"f16": torch.float16, "bf16": torch.bfloat16, "f32": torch.float32}
STATE_BLOCK = 256      # values of a tensor that share an 8-bit state's scale
E4M3_MAX = 448.0
LEAST = 2.0 ** -100    # a block with no larger magnitude is held as zeros
BETA1, BETA2, ADAM_EPS, LR, STEP, DECAY = 0.9, 0.999, 1e-8, 1e-3, 7, 0.1


# ---------------------------------------------------------------------------
# Cases
# ---------------------------------------------------------------------------

def _glu(op, M, D, F, act, dtype, bias=False, pad=0, keep=True):
    return {"op": op, "M": M, "D": D, "F": F, "act": act, "dtype": dtype, "bias": bias, "pad": pad, "keep": keep}


def _linear(M, N, K, dtype, bias=False, pad=0):
    return {"op": "linear", "M": M, "N": N, "K": K, "dtype": dtype, "bias": bias, "pad": pad}


def _fp8(M, N, K, dtype, bias=False, pad=0):
    return {"op": "fp8", "M": M, "N": N, "K": K, "dtype": dtype, "bias": bias, "pad": pad}


def _adamw(layers, D, F, odd, bits, param, grad, copy):
    """``layers`` gated feed-forward blocks' tensors: up [2F][D], its bias, down [D][F], its bias, a norm's gamma
    and beta, each ``odd`` elements longer than that.  ``copy``: the 16-bit copy of fp32 parameters, or ''."""
    return {"op": "adamw", "layers": layers, "D": D, "F": F, "odd": odd, "bits": bits, "param": param, "grad": grad, "copy": copy}


def listed():
    return [
        # a decoding step of four sequences through the SDXL level-2 up projection: the weight's bytes count
        {"name": "glu_fwd_decode_4x1280x5120_bf16", **_glu("glu_fwd", 4, 1280, 5120, "silu", "bf16", keep=False)},
        # training on one SigLIP image of 729 patches: a ragged last row block, a hidden size that is no multiple of 32
        {"name": "glu_fwd_siglip_729x1152x4304_f16", **_glu("glu_fwd", 729, 1152, 4304, "gelu_tanh", "f16", True)},
        # training on a batch of 16384 SDXL level-2 tokens: bound by the matrix product
        {"name": "glu_fwd_batch_16384x1280x5120_bf16", **_glu("glu_fwd", 16384, 1280, 5120, "gelu_erf", "bf16", True)},
        # the gradients for one SigLIP image: two products with few tiles, one of them over 729 tokens alone
        {"name": "glu_bwd_siglip_729x1152x4304_f16", **_glu("glu_bwd", 729, 1152, 4304, "gelu_tanh", "f16", True)},
        # the gradients for the batch of 16384 tokens
        {"name": "glu_bwd_batch_16384x1280x5120_bf16", **_glu("glu_bwd", 16384, 1280, 5120, "gelu_erf", "bf16", True)},
        # the down projection of a small model's training step: odd tokens, rows of a wider tensor
        {"name": "linear_small_331x640x2560_f16", **_linear(331, 640, 2560, "f16", True, 8)},
        # the down projection of the batch of 16384 tokens
        {"name": "linear_batch_16384x1280x5120_bf16", **_linear(16384, 1280, 5120, "bf16", True)},
        # a decoding step of four sequences in 8-bit floating point: the weight's bytes count
        {"name": "fp8_decode_4x10240x1280_bf16", **_fp8(4, 10240, 1280, "bf16", True)},
        # the SigLIP up projection: ragged blocks of tokens, channels and columns
        {"name": "fp8_siglip_729x4304x1152_f16", **_fp8(729, 4304, 1152, "f16")},
        # a large square product: bound by the 8-bit tensor rate
        {"name": "fp8_batch_8192x8192x8192_bf16", **_fp8(8192, 8192, 8192, "bf16")},
        # one small block's six tensors, fp32 parameters with their bf16 copies: the latency of the call
        {"name": "adamw_one_640x640_f32", **_adamw(1, 640, 640, 0, 32, "f32", "bf16", "bf16")},
        # eight SDXL level-2 blocks (157 million parameters) in bf16 with 8-bit moments: bound by memory
        {"name": "adamw_eight_1280x5120_8bit", **_adamw(8, 1280, 5120, 3, 8, "bf16", "bf16", "")},
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["glu_fwd", "glu_bwd", "linear", "fp8", "adamw"])
    dtype = rng.choice(["f16", "bf16"])
    if op in ("glu_fwd", "glu_bwd"):
        while True:
            M, D, F = _log(rng, 1, 16384), max(64, _log(rng, 64, 4096) // 8 * 8), max(64, _log(rng, 64, 8192) // 8 * 8)
            if M * D * F <= 16384 * 1280 * 5120:
                break
        act = rng.choice(["gelu_erf", "gelu_tanh", "gelu_sigmoid", "silu"])
        return _glu(op, M, D, F, act, dtype, rng.random() < 0.5, rng.choice([0, 0, 8, 24]), op == "glu_bwd" or rng.random() < 0.7)
    if op == "linear":
        while True:
            M, N, K = _log(rng, 1, 16384), max(64, _log(rng, 64, 8192) // 8 * 8), max(64, _log(rng, 64, 8192) // 8 * 8)
            if M * N * K <= 16384 * 1280 * 5120:
                break
        return _linear(M, N, K, dtype, rng.random() < 0.5, rng.choice([0, 0, 8, 24]))
    if op == "fp8":
        while True:
            M, N, K = _log(rng, 1, 16384), max(8, _log(rng, 64, 16384) // 8 * 8), max(64, _log(rng, 64, 16384) // 16 * 16)
            if M * N * K <= 8192 * 8192 * 8192 and M * K <= 1 << 27 and N * K <= 1 << 27 and M * N <= 1 << 27:
                break
        return _fp8(M, N, K, dtype, rng.random() < 0.5, rng.choice([0, 0, 16]))
    while True:
        layers, D, F = _log(rng, 1, 40), _log(rng, 16, 2560), _log(rng, 16, 8192)
        if layers * 3 * D * F <= 8 * 3 * 1280 * 5120:
            break
    param, copy = rng.choice([("f32", ""), ("f32", "bf16"), ("f32", "f16"), (dtype, "")])
    return _adamw(layers, D, F, rng.choice([0, 0, 1, 5]), rng.choice([8, 32]), param, rng.choice([dtype, "f32"]), copy)


def _adamw_sizes(case):
    D, F = case["D"], case["F"]
    return [n + case["odd"] for n in (2 * F * D, 2 * F, D * F, D, D, D)] * case["layers"]


def work(case):
    """What one pass cannot do without: inputs read once, outputs written once."""
    op = case["op"]
    if op == "glu_fwd":
        M, D, F = case["M"], case["D"], case["F"]
        return {"bytes": 2 * M * D + 4 * F * D + 2 * M * F + (4 * M * F if case["keep"] else 0) + (4 * F if case["bias"] else 0),
                "flops": 4 * M * D * F}
    if op == "glu_bwd":
        M, D, F = case["M"], case["D"], case["F"]
        return {"bytes": 6 * M * F + 4 * M * D + 8 * F * D + (8 * F if case["bias"] else 0), "flops": 8 * M * D * F}
    if op == "linear":
        M, N, K = case["M"], case["N"], case["K"]
        return {"bytes": 4 * M * N + 4 * M * K + 4 * N * K + (6 * N if case["bias"] else 0), "flops": 6 * M * N * K}
    if op == "fp8":
        M, N, K = case["M"], case["N"], case["K"]
        runs = -(-K // 128)
        return {"bytes": 2 * M * K + 4 * M * runs + N * K + 4 * runs * -(-N // 128) + 2 * M * N + (2 * N if case["bias"] else 0),
                "flops": 2 * M * N * K}
    n = sum(_adamw_sizes(case))
    size = {"f32": 4, "f16": 2, "bf16": 2, "": 0}
    state = 8 if case["bits"] == 32 else 2 + 8 / STATE_BLOCK
    return {"bytes": int(n * (2 * size[case["param"]] + size[case["grad"]] + size[case["copy"]] + 2 * state)), "flops": 14 * n}


# ---------------------------------------------------------------------------
# Inputs
# ---------------------------------------------------------------------------

def _rows(gen, M, D, pad, dtype, scale=1.0):
    """Rows as a residual stream has them after a norm: each with a scale of its own; the row pitch is D + pad."""
    x = torch.randn(M, D + pad, generator=gen, device="cuda")
    x *= scale * (0.5 + torch.rand(M, 1, generator=gen, device="cuda"))
    return x.to(dtype)[:, :D]


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    op = case["op"]
    st = {"case": dict(case)}
    if op == "adamw":
        return _prepare_adamw(st, gen)
    dt = st["dtype"] = DTYPES[case["dtype"]]

    def randn(*shape, std=1.0):
        return (torch.randn(*shape, generator=gen, device="cuda") * std).to(dt)

    def empty(*shape, dtype=dt):
        return torch.empty(*shape, dtype=dtype, device="cuda")

    if op in ("glu_fwd", "glu_bwd"):
        M, D, F, pad = (case[n] for n in ("M", "D", "F", "pad"))
        st["X"] = _rows(gen, M, D, pad, dt)
        st["W"] = randn(2 * F, D, std=1.0 / math.sqrt(D))
        st["b"] = randn(2 * F, std=math.sqrt(0.02)) if case["bias"] else None
        if op == "glu_fwd":
            st["H"], st["P"] = empty(M, F), empty(M, 2 * F) if case["keep"] else None
        else:
            p = torch.matmul(st["X"].float(), st["W"].float().t())  # what the forward pass kept
            st["P"] = (p if st["b"] is None else p + st["b"].float()).to(dt)
            st["dH"] = _rows(gen, M, F, pad, dt, 0.25)
            st["dX"], st["dW"] = empty(M, D), empty(2 * F, D)
            st["db"] = empty(2 * F, dtype=torch.float32) if case["bias"] else None
            if own:
                from transformer_mlp_gemms_gb300 import kt_ops
                st["workspace"] = kt_ops.glu_backward_workspace(M, D, F)
    elif op == "linear":
        M, N, K, pad = (case[n] for n in ("M", "N", "K", "pad"))
        st["X"] = _rows(gen, M, K, pad, dt)
        st["W"] = randn(N, K, std=1.0 / math.sqrt(K))
        st["b"] = randn(N, std=math.sqrt(0.02)) if case["bias"] else None
        st["dY"] = _rows(gen, M, N, pad, dt, 0.25)
        st["Y"], st["dX"], st["dW"] = empty(M, N), empty(M, K), empty(N, K)
        st["db"] = empty(N, dtype=torch.float32) if case["bias"] else None
        if own:
            from transformer_mlp_gemms_gb300 import kt_ops
            st["workspace"] = kt_ops.linear_backward_workspace(M, N, K)
    else:
        M, N, K = case["M"], case["N"], case["K"]
        st["X"] = _rows(gen, M, K, case["pad"], dt, 0.5)
        st["X"][:, 3::97] *= 8.0  # a few channels carry far larger values, as activations' do
        w = torch.randn(N, K, generator=gen, device="cuda") / math.sqrt(K)
        w *= 0.5 + torch.rand(N, 1, generator=gen, device="cuda")
        nb, kb = -(-N // 128), -(-K // 128)
        most = torch.zeros(nb * 128, kb * 128, device="cuda")
        most[:N, :K] = w.abs()
        st["wscale"] = (most.view(nb, 128, kb, 128).amax((1, 3)) / E4M3_MAX).contiguous()
        each = st["wscale"].repeat_interleave(128, 0)[:N].repeat_interleave(128, 1)[:, :K]
        st["W"] = (w / each).clamp_(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn)
        st["bias"] = randn(N, std=math.sqrt(0.02)) if case["bias"] else None
        st["Q"] = empty(M, K, dtype=torch.float8_e4m3fn)
        st["scale"] = empty(M, kb, dtype=torch.float32)
        st["Y"] = empty(M, N)
    return st


def _prepare_adamw(st, gen):
    """The tensors lie in one buffer each for parameters, gradients and moments, every one from a multiple of 256
    elements on; what is between them is zero."""
    case = st["case"]
    st["sizes"] = _adamw_sizes(case)
    st["room"] = [-(-n // STATE_BLOCK) * STATE_BLOCK for n in st["sizes"]]
    st["decay"] = [DECAY if k % 6 in (0, 2) else 0.0 for k in range(len(st["sizes"]))]
    total, dev = sum(st["room"]), "cuda"
    inside = torch.zeros(total, dtype=torch.bool, device=dev)
    offset = 0
    for n, room in zip(st["sizes"], st["room"]):
        inside[offset:offset + n] = True
        offset += room

    def values(std):  # magnitudes over several orders, as gradients of many layers have them
        v = torch.randn(total, generator=gen, device=dev)
        v *= std * torch.exp2(-6.0 * torch.rand(total // STATE_BLOCK, 1, generator=gen, device=dev)).expand(-1, STATE_BLOCK).reshape(-1)
        return v.mul_(inside)

    st["P"] = values(0.1).to(DTYPES[case["param"]])
    st["G"] = values(1e-2).to(DTYPES[case["grad"]])
    m, r = values(5e-3), values(1e-2).abs_()
    if case["bits"] == 32:
        st["m"], st["v"] = m, r.square_()
    else:
        st["m"], st["m_scale"] = _to_blocks(m, False)
        st["v"], st["v_scale"] = _to_blocks(r, True)
    st["copy"] = torch.zeros(total, dtype=DTYPES[case["copy"]], device=dev) if case["copy"] else None

    def parts(flat, unit=1):
        got, o = [], 0
        for n, room in zip(st["sizes"], st["room"]):
            got.append(flat[o // unit:(o + n + unit - 1) // unit])
            o += room
        return got

    # a program's own lists of tensors
    st["params"], st["grads"], st["ms"], st["vs"] = (parts(st[k]) for k in ("P", "G", "m", "v"))
    st["m_scales"], st["v_scales"] = (parts(st[k], STATE_BLOCK) if case["bits"] == 8 else None for k in ("m_scale", "v_scale"))
    st["copies"] = parts(st["copy"]) if case["copy"] else None
    return st


# ---------------------------------------------------------------------------
# One pass
# ---------------------------------------------------------------------------

def run(st):
    op = st["case"]["op"]
    if own:
        return _OWN[op](st)
    return _PLAIN[op](st)


def _act_code(name):
    from transformer_mlp_gemms_gb300 import kt_mlp
    return {"gelu_erf": kt_mlp.KT_ACT_GELU_ERF, "gelu_tanh": kt_mlp.KT_ACT_GELU_TANH,
            "gelu_sigmoid": kt_mlp.KT_ACT_GELU_SIGMOID, "silu": kt_mlp.KT_ACT_SILU}[name]


def _own_glu_fwd(st):
    from transformer_mlp_gemms_gb300 import kt_ops
    kt_ops.kt_glu_forward(st["X"], st["W"], st["b"], st["H"], st["P"], _act_code(st["case"]["act"]))
    return {"h": st["H"], "p": st["P"]} if st["P"] is not None else {"h": st["H"]}


def _own_glu_bwd(st):
    from transformer_mlp_gemms_gb300 import kt_ops
    kt_ops.kt_glu_backward(st["dH"], st["P"], st["X"], st["W"], st["dX"], st["dW"], st["db"], _act_code(st["case"]["act"]),
                           st["workspace"])
    return _some(dx=st["dX"], dw=st["dW"], db=st["db"])


def _own_linear(st):
    from transformer_mlp_gemms_gb300 import kt_ops
    kt_ops.kt_linear_forward(st["X"], st["W"], st["b"], st["Y"])
    kt_ops.kt_linear_backward(st["dY"], st["X"], st["W"], st["dX"], st["dW"], st["db"], st["workspace"])
    return _some(y=st["Y"], dx=st["dX"], dw=st["dW"], db=st["db"])


def _own_fp8(st):
    from transformer_mlp_gemms_gb300 import kt_ops
    kt_ops.kt_quantize_fp8(st["X"], st["Q"], st["scale"])
    kt_ops.kt_linear_fp8(st["Q"], st["scale"], st["W"], st["wscale"], st["bias"], st["Y"])
    return {"y": st["Y"], "q": st["Q"], "scale": st["scale"]}


def _own_adamw(st):
    from transformer_mlp_gemms_gb300 import kt_ops
    kt_ops.kt_adamw(st["params"], st["grads"], st["ms"], st["vs"], STEP, LR, BETA1, BETA2, ADAM_EPS, st["decay"],
                    m_scales=st["m_scales"], v_scales=st["v_scales"], copies=st["copies"])
    return _adamw_outputs(st)


def _some(**outputs):
    return {k: v for k, v in outputs.items() if v is not None}


def _adamw_outputs(st):
    return _some(p=st["P"], m=st["m"], v=st["v"], m_scale=st.get("m_scale"), v_scale=st.get("v_scale"), copy=st["copy"])


def _act(g, act):
    """act(g) and its derivative."""
    if act == "gelu_erf":
        phi = 0.5 * torch.special.erfc(g * -math.sqrt(0.5))
        return g * phi, phi + g * torch.exp(-0.5 * g * g) * (1.0 / math.sqrt(2.0 * math.pi))
    if act == "gelu_tanh":
        c = 2.0 * math.sqrt(2.0 / math.pi)
        s = 1.0 / (1.0 + torch.exp(-c * (g + 0.044715 * g * g * g)))
        return g * s, s + g * s * (1.0 - s) * c * (1.0 + 3.0 * 0.044715 * g * g)
    a = 1.702 if act == "gelu_sigmoid" else 1.0
    s = 1.0 / (1.0 + torch.exp(-a * g))
    return g * s, s + a * g * s * (1.0 - s)


def _plain_glu_fwd(st):
    F = st["case"]["F"]
    p = torch.matmul(st["X"].float(), st["W"].float().t())
    if st["b"] is not None:
        p = p + st["b"].float()
    h = (p[:, :F] * _act(p[:, F:], st["case"]["act"])[0]).to(st["dtype"])
    return {"h": h, "p": p.to(st["dtype"])} if st["P"] is not None else {"h": h}


def _plain_glu_bwd(st):
    F = st["case"]["F"]
    p, dh, x = st["P"].float(), st["dH"].float(), st["X"].float()
    a, da = _act(p[:, F:], st["case"]["act"])
    dp = torch.cat([dh * a, dh * p[:, :F] * da], 1)
    return _some(dx=torch.matmul(dp, st["W"].float()).to(st["dtype"]), dw=torch.matmul(dp.t(), x).to(st["dtype"]),
                 db=dp.sum(0) if st["db"] is not None else None)


def _plain_linear(st):
    x, w, dy = st["X"].float(), st["W"].float(), st["dY"].float()
    y = torch.matmul(x, w.t())
    if st["b"] is not None:
        y = y + st["b"].float()
    return _some(y=y.to(st["dtype"]), dx=torch.matmul(dy, w).to(st["dtype"]), dw=torch.matmul(dy.t(), x).to(st["dtype"]),
                 db=dy.sum(0) if st["db"] is not None else None)


def _runs(x, size):
    """The last dimension in runs of ``size``, the last one filled up with zeros."""
    short = -x.shape[-1] % size
    if short:
        x = torch.cat([x, x.new_zeros(*x.shape[:-1], short)], -1)
    return x.view(*x.shape[:-1], -1, size)


def _to_runs(x, size):
    """x in runs of ``size``: their scales, and the quotients that e4m3 rounds."""
    runs = _runs(x, size)
    most = runs.abs().amax(-1)
    top = torch.full_like(most, E4M3_MAX)  # a quotient with a plain number is a product with its rounded inverse
    zero = most < LEAST
    scale = torch.where(zero, 0.0, most / top)
    q = runs * torch.where(zero, 0.0, top / torch.where(zero, 1.0, most))[..., None]
    return scale, q


def _to_blocks(x, root):
    """A moment in e4m3 with a scale for each 256 values; ``root``: what is above zero stays so."""
    scale, q = _to_runs(x, STATE_BLOCK)
    if root:
        q = torch.where(q > 0, q.clamp_min(2.0 ** -9), q)
    return q.to(torch.float8_e4m3fn).view(-1), scale


def _plain_fp8(st):
    M, K = st["X"].shape
    N = st["W"].shape[0]
    scale, q = _to_runs(st["X"].float(), 128)
    q = q.to(torch.float8_e4m3fn)
    kb = scale.shape[1]
    x = (q.float() * scale[..., None]).view(M, -1)[:, :K]
    w = st["W"].float() * st["wscale"].repeat_interleave(128, 0)[:N].repeat_interleave(128, 1)[:, :K]
    y = torch.matmul(x, w.t())
    if st["bias"] is not None:
        y = y + st["bias"].float()
    return {"y": y.to(st["dtype"]), "q": q.view(M, kb * 128)[:, :K], "scale": scale}


def _plain_adamw(st):
    case = st["case"]
    p, g = st["P"].float(), st["G"].float()
    wide = torch.tensor(st["room"], device=p.device)
    keep = torch.tensor([1.0 - LR * d for d in st["decay"]], dtype=torch.float64).float().to(p.device).repeat_interleave(wide, output_size=p.numel())
    if case["bits"] == 32:
        m, v = st["m"], st["v"]
    else:
        m = (st["m"].float().view(-1, STATE_BLOCK) * st["m_scale"][:, None]).view(-1)
        r = (st["v"].float().view(-1, STATE_BLOCK) * st["v_scale"][:, None]).view(-1)
        v = r * r
    m = m * BETA1 + g * (1.0 - BETA1)
    v = v * BETA2 + (g * (1.0 - BETA2)) * g
    r = torch.sqrt(v)
    p = p * keep - (m * (LR / (1.0 - BETA1 ** STEP))) / (r * (1.0 / math.sqrt(1.0 - BETA2 ** STEP)) + ADAM_EPS)
    st["P"].copy_(p)
    if st["copy"] is not None:
        st["copy"].copy_(p)
    if case["bits"] == 32:
        st["m"].copy_(m)
        st["v"].copy_(v)
    else:
        for name, x in (("m", m), ("v", r)):
            q, scale = _to_blocks(x, name == "v")
            st[name].copy_(q)
            st[name + "_scale"].copy_(scale)
    return _adamw_outputs(st)


_OWN = {"glu_fwd": _own_glu_fwd, "glu_bwd": _own_glu_bwd, "linear": _own_linear, "fp8": _own_fp8, "adamw": _own_adamw}
_PLAIN = {"glu_fwd": _plain_glu_fwd, "glu_bwd": _plain_glu_bwd, "linear": _plain_linear, "fp8": _plain_fp8, "adamw": _plain_adamw}


# ---------------------------------------------------------------------------
# The definitions in 64 bits
# ---------------------------------------------------------------------------

def exact(case, seed):
    st = prepare(case, seed)
    return {"glu_fwd": _exact_glu_fwd, "glu_bwd": _exact_glu_bwd, "linear": _exact_linear, "fp8": _exact_fp8,
            "adamw": _exact_adamw}[case["op"]](st)


def _gate64(g, act):
    """act(g) and act'(g)."""
    if act == "gelu_erf":
        cdf = 0.5 * (1.0 + torch.erf(g / math.sqrt(2.0)))
        return g * cdf, cdf + g * torch.exp(-g ** 2 / 2.0) / math.sqrt(2.0 * math.pi)
    if act == "gelu_tanh":
        k = math.sqrt(2.0 / math.pi)
        t = torch.tanh(k * (g + 0.044715 * g ** 3))
        return 0.5 * g * (1.0 + t), 0.5 * (1.0 + t) + 0.5 * g * (1.0 - t ** 2) * k * (1.0 + 0.134145 * g ** 2)
    a = {"gelu_sigmoid": 1.702, "silu": 1.0}[act]
    s = torch.sigmoid(a * g)
    return g * s, s * (1.0 + a * g * torch.sigmoid(-a * g))


def _exact_glu_fwd(st):
    p = torch.einsum("md,fd->mf", st["X"].double(), st["W"].double())
    if st["b"] is not None:
        p += st["b"].double()
    value, gate = p.chunk(2, 1)
    h = value * _gate64(gate, st["case"]["act"])[0]
    return {"h": h, "p": p} if st["case"]["keep"] else {"h": h}


def _exact_glu_bwd(st):
    value, gate = st["P"].double().chunk(2, 1)
    a, slope = _gate64(gate, st["case"]["act"])
    dh = st["dH"].double()
    dp = torch.hstack([dh * a, dh * value * slope])
    out = {"dx": dp @ st["W"].double(), "dw": torch.einsum("mf,md->fd", dp, st["X"].double())}
    if st["case"]["bias"]:
        out["db"] = torch.ones(dp.shape[0], dtype=torch.float64, device=dp.device) @ dp
    return out


def _exact_linear(st):
    x, w, dy = (st[k].double() for k in ("X", "W", "dY"))
    y = torch.einsum("mk,nk->mn", x, w)
    out = {"y": y if st["b"] is None else y + st["b"].double(), "dx": dy @ w, "dw": torch.einsum("mn,mk->nk", dy, x)}
    if st["b"] is not None:
        out["db"] = torch.ones(x.shape[0], dtype=torch.float64, device=x.device) @ dy
    return out


def _exact_fp8(st):
    """The product of the quantised operands in 64 bits; the definition's quotients are 32-bit numbers."""
    x, w = st["X"], st["W"].double()
    M, K = x.shape
    N = w.shape[0]
    y = torch.zeros(M, N, dtype=torch.float64, device=x.device)
    scales, quotients = [], []
    for j, k in enumerate(range(0, K, 128)):
        run = x[:, k:k + 128].to(torch.float64)
        most = run.abs().max(1).values
        inverse = (448.0 / most).float().double()
        quotient = torch.nan_to_num(run * inverse[:, None])
        q = quotient.float().to(torch.float8_e4m3fn).double()
        s = most / 448.0
        t = st["wscale"][:, j].double().repeat_interleave(128)[:N]
        y += s[:, None] * ((q @ w[:, k:k + 128].t()) * t)
        scales.append(s)
        quotients.append(quotient)
    if st["bias"] is not None:
        y += st["bias"].double()
    return {"y": y, "q": torch.cat(quotients, 1), "scale": torch.stack(scales, 1)}


def _exact_adamw(st):
    case = st["case"]
    g, p = st["G"].double(), st["P"].double()
    decay = torch.cat([torch.full((n,), d, dtype=torch.float64, device=g.device) for n, d in zip(st["room"], st["decay"])])
    m, v = st["m"].double(), st["v"].double()
    if case["bits"] == 8:
        m = m * st["m_scale"].double().repeat_interleave(STATE_BLOCK)
        v = (v * st["v_scale"].double().repeat_interleave(STATE_BLOCK)) ** 2
    m = BETA1 * m + (1.0 - BETA1) * g
    v = BETA2 * v + (1.0 - BETA2) * g ** 2
    p = p - LR * ((m / (1.0 - BETA1 ** STEP)) / ((v / (1.0 - BETA2 ** STEP)).sqrt() + ADAM_EPS) + decay * p)
    out = {"p": p}
    if case["bits"] == 32:
        out.update(m=m, v=v)
    else:
        for name, x in (("m", m), ("v", v.sqrt())):
            x = x.view(-1, STATE_BLOCK)
            s = x.abs().max(1).values / 448.0
            out[name], out[name + "_scale"] = torch.nan_to_num(x / s[:, None]).view(-1), s
    if case["copy"]:
        out["copy"] = p
    return out
