"""The operators of include/kt_ops.h as a feed-forward sublayer uses them, on one GB300:

    python -m transformer_mlp_gemms_gb300.example_block

1. Decoding with a mixture of experts: x = x + moe(layer_norm(x)) for a few tokens, captured once
   into a CUDA graph and replayed on a residual stream that is updated in place.
2. A quantised MLP: layer norm, 8-bit rows, the 8-bit up projection, the activation as its output
   is quantised again, the 8-bit down projection; beside the same MLP in fp16 (``kt_mlp.Plan``).
3. Training a layer norm's gamma and beta by gradient descent with the backward pass.
"""
from __future__ import annotations

import torch

from . import kt_mlp, kt_ops

EPS = 1e-5


def decode(tokens=4, D=640, F=1280, experts=8, top_k=2, steps=8, seed=0):
    """Runs ``steps`` blocks on a residual stream by replaying one graph; returns the stream and the
    experts of the last step."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    dt = torch.bfloat16

    def randn(*shape, std=1.0):
        return (torch.randn(*shape, generator=g, device="cuda") * std).to(dt)

    x = randn(tokens, D)
    gamma, beta = torch.ones(D, dtype=dt, device="cuda"), torch.zeros(D, dtype=dt, device="cuda")
    router, up, down = randn(experts, D, std=D ** -0.5), randn(experts, 2 * F, D, std=D ** -0.5), randn(experts, D, F, std=F ** -0.5)
    normed = torch.empty_like(x)
    ids = torch.empty(tokens, top_k, dtype=torch.int32, device="cuda")
    plan = kt_ops.MoePlan(tokens, D, F, experts, top_k, kt_mlp.KT_ACT_GEGLU, kt_mlp.KT_BF16)

    def block():
        kt_ops.kt_layernorm_forward(x, gamma, beta, EPS, normed)
        plan.run(normed, router, up, down, x, R=x, ids=ids)

    block()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        block()
    for _ in range(steps - 1):
        graph.replay()
    if plan.status() != kt_mlp.KT_OK:
        raise RuntimeError("the mixture-of-experts layer reported " + kt_mlp.kt_last_error())
    return x, ids


def quantise_weight(w):
    """An [out][in] weight as int8 with a scale for each output channel."""
    scale = w.float().abs().amax(1) / 127.0
    return torch.round(w.float() / scale[:, None]).clamp_(-127, 127).to(torch.int8), scale


def quantised_mlp(M=729, D=1152, F=4304, seed=0):
    """Returns the 8-bit MLP's output, and the fp16 MLP's on the same weights."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    dt = torch.float16

    def randn(*shape, std=1.0):
        return (torch.randn(*shape, generator=g, device="cuda") * std).to(dt)

    x, gamma, beta = randn(M, D), (1 + 0.1 * torch.randn(D, generator=g, device="cuda")).to(dt), randn(D, std=0.1)
    w_up, w_down = randn(F, D, std=D ** -0.5), randn(D, F, std=F ** -0.5)
    (up, up_scale), (down, down_scale) = quantise_weight(w_up), quantise_weight(w_down)

    normed, hidden, y = torch.empty_like(x), torch.empty(M, F, dtype=dt, device="cuda"), torch.empty_like(x)
    q, qh = torch.empty(M, D, dtype=torch.int8, device="cuda"), torch.empty(M, F, dtype=torch.int8, device="cuda")
    s, sh = torch.empty(M, device="cuda"), torch.empty(M, device="cuda")
    kt_ops.kt_layernorm_forward(x, gamma, beta, EPS, normed)
    kt_ops.kt_quantize_rows(normed, q, s)
    kt_ops.kt_linear_i8(q, s, up, up_scale, None, hidden)
    kt_ops.kt_quantize_rows(hidden, qh, sh, kt_mlp.KT_ACT_GELU_TANH)
    kt_ops.kt_linear_i8(qh, sh, down, down_scale, None, y)

    exact = torch.empty_like(x)
    plan = kt_mlp.Plan(M, D, F, kt_mlp.KT_ACT_GELU_TANH, kt_mlp.KT_F16, False, layernorm=True, ln_eps=EPS,
                       weight_layout=kt_mlp.KT_W_OUT_IN)
    plan.run_ex(x, w_up, w_down, exact, ln_gamma=gamma, ln_beta=beta)
    if kt_ops.kt_linear_i8_status() != kt_mlp.KT_OK or plan.status() != kt_mlp.KT_OK:  # both wait for the stream
        raise RuntimeError("an MLP reported " + kt_mlp.kt_last_error())
    return y, exact


def train_norm(M=512, D=640, steps=60, lr=0.5, seed=0):
    """Fits gamma and beta to a layer norm with other ones; returns the losses (mean squares)."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    dt = torch.bfloat16
    x = torch.randn(M, D, generator=g, device="cuda").to(dt)
    want_gamma, want_beta = (1 + 0.3 * torch.randn(2, D, generator=g, device="cuda")).to(dt)
    target, y, dx = torch.empty_like(x), torch.empty_like(x), torch.empty_like(x)
    kt_ops.kt_layernorm_forward(x, want_gamma, want_beta, EPS, target)
    gamma, beta = torch.ones(D, device="cuda"), torch.zeros(D, device="cuda")  # the optimiser's, in fp32
    mean, rstd = torch.empty(M, device="cuda"), torch.empty(M, device="cuda")
    dgamma, dbeta = torch.empty(D, device="cuda"), torch.empty(D, device="cuda")
    workspace = kt_ops.layernorm_backward_workspace(M, D)
    losses = []
    for _ in range(steps):
        gamma16, beta16 = gamma.to(dt), beta.to(dt)
        kt_ops.kt_layernorm_forward(x, gamma16, beta16, EPS, y, mean, rstd)
        error = y.float() - target.float()
        losses.append(error.square().mean())
        kt_ops.kt_layernorm_backward(error.to(dt), x, gamma16, mean, rstd, dx, dgamma, dbeta, workspace)
        gamma -= lr / M * dgamma
        beta -= lr / M * dbeta
    return torch.stack(losses).tolist()


def main():
    x, ids = decode()
    print(f"decoding: 8 blocks on a stream of {list(x.shape)}, finite {bool(x.isfinite().all())}, last experts {ids.tolist()}")
    y, exact = quantised_mlp()
    off = ((y.float() - exact.float()).norm() / exact.float().norm()).item()
    print(f"8-bit MLP {list(y.shape)}: {off:.4f} of the fp16 MLP's norm away from it")
    losses = train_norm()
    print(f"training a layer norm: loss {losses[0]:.4f} -> {losses[-1]:.2e} in {len(losses)} steps")


if __name__ == "__main__":
    main()
