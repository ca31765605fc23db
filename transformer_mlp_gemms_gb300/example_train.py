"""A gated feed-forward sublayer trained, then served in 8-bit floating point, on one GB300:

    python -m transformer_mlp_gemms_gb300.example_train

    y = x + down(value * gelu(gate)),  [value | gate] = up(layer_norm(x))

1. Training: forward, backward and AdamW from the operators of include/kt_ops.h.  The optimiser
   keeps the parameters in fp32 and hands their bf16 rounding to the next step; the matrices'
   moments are 8-bit, the vectors' fp32.  The first step runs as it is, the others replay it as a
   CUDA graph (the step's number lives on the device).
2. Serving: the trained matrices in e4m3 with a scale for each block of 128 x 128, the tokens in
   e4m3 with a scale for each run of 128; the gate is applied as the hidden layer is quantised.
"""
from __future__ import annotations

import torch

from . import kt_mlp, kt_ops

EPS = 1e-5
ACT = kt_mlp.KT_ACT_GELU_ERF
MATRICES, VECTORS = ("up", "down"), ("gamma", "beta", "b_up", "b_down")


def init(D, F, seed=0):
    """The parameters in fp32."""
    g = torch.Generator(device="cuda").manual_seed(seed)

    def randn(*shape, std):
        return torch.randn(*shape, generator=g, device="cuda") * std

    return {"gamma": 1 + randn(D, std=0.1), "beta": randn(D, std=0.1), "up": randn(2 * F, D, std=D ** -0.5),
            "b_up": randn(2 * F, std=0.1), "down": randn(D, F, std=F ** -0.5), "b_down": randn(D, std=0.1)}


class Sublayer:
    """The sublayer's 16-bit parameters ``w``, its gradients ``grad`` (matrices in bf16, vectors in fp32) and what its
    backward pass wants kept, for M tokens."""

    def __init__(self, M, D, F, params):
        bf16 = dict(dtype=torch.bfloat16, device="cuda")
        self.w = {k: t.bfloat16() for k, t in params.items()}
        self.grad = {k: torch.empty_like(self.w[k] if k in MATRICES else t) for k, t in params.items()}
        self.mean, self.rstd = torch.empty(2, M, device="cuda").unbind()
        self.normed, self.d_normed, self.dx = torch.empty(3, M, D, **bf16).unbind()
        self.h, self.dh = torch.empty(2, M, F, **bf16).unbind()
        self.p, self.y = torch.empty(M, 2 * F, **bf16), torch.empty(M, D, **bf16)
        self.workspaces = (kt_ops.linear_backward_workspace(M, D, F), kt_ops.glu_backward_workspace(M, D, F),
                           kt_ops.layernorm_backward_workspace(M, D))

    def forward(self, x):
        """y, without the residual stream that it is added to."""
        w = self.w
        kt_ops.kt_layernorm_forward(x, w["gamma"], w["beta"], EPS, self.normed, self.mean, self.rstd)
        kt_ops.kt_glu_forward(self.normed, w["up"], w["b_up"], self.h, self.p, ACT)
        kt_ops.kt_linear_forward(self.h, w["down"], w["b_down"], self.y)
        return self.y

    def backward(self, dy, x):
        """The gradients of the parameters into ``grad``; returns x's through the sublayer (the residual stream adds dy)."""
        w, d = self.w, self.grad
        kt_ops.kt_linear_backward(dy, self.h, w["down"], self.dh, d["down"], d["b_down"], self.workspaces[0])
        kt_ops.kt_glu_backward(self.dh, self.p, self.normed, w["up"], self.d_normed, d["up"], d["b_up"], ACT, self.workspaces[1])
        kt_ops.kt_layernorm_backward(self.d_normed, x, w["gamma"], self.mean, self.rstd, self.dx, d["gamma"], d["beta"],
                                     self.workspaces[2])
        return self.dx


class Optimiser:
    """AdamW for ``params`` (fp32, in place), whose roundings go to ``layer.w``."""

    def __init__(self, params, layer, lr, weight_decay):
        self.lr, self.step = lr, torch.zeros((), dtype=torch.int64, device="cuda")
        self.groups = []
        for names, dtype, decay in ((MATRICES, torch.float8_e4m3fn, weight_decay), (VECTORS, torch.float32, 0.0)):
            p = [params[k] for k in names]
            group = dict(params=p, grads=[layer.grad[k] for k in names], copies=[layer.w[k] for k in names], weight_decay=decay,
                         m=[torch.zeros_like(t, dtype=dtype) for t in p], v=[torch.zeros_like(t, dtype=dtype) for t in p])
            if dtype != torch.float32:
                for key in ("m_scales", "v_scales"):
                    group[key] = [torch.zeros(-(-t.numel() // kt_ops.KT_ADAMW_BLOCK), device="cuda") for t in p]
            self.groups.append(group)

    def update(self):
        self.step += 1
        for group in self.groups:
            kt_ops.kt_adamw(step=self.step, lr=self.lr, beta2=0.99, **group)


def train(M=4096, D=640, F=2560, steps=50, lr=1e-3, seed=0, replay=True):
    """Fits a sublayer to another one's outputs; returns it, its parameters and the losses (mean squares)."""
    x = torch.randn(M, D, generator=torch.Generator(device="cuda").manual_seed(seed), device="cuda").bfloat16()
    target = Sublayer(M, D, F, init(D, F, seed + 1)).forward(x)
    params = init(D, F, seed + 2)
    layer = Sublayer(M, D, F, params)
    optimiser = Optimiser(params, layer, lr, 0.01)
    losses, loss = torch.empty(steps, device="cuda"), torch.empty((), device="cuda")

    def step():
        error = layer.forward(x).float() - target.float()
        loss.copy_(error.square().mean())
        layer.backward(error.mul_(1.0 / M).bfloat16(), x)
        optimiser.update()

    step()
    losses[0] = loss
    if replay and steps > 1:
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            step()
    for i in range(1, steps):
        if replay:
            graph.replay()
        else:
            step()
        losses[i] = loss
    if kt_ops.kt_matmul_status() != kt_mlp.KT_OK:  # waits for the stream
        raise RuntimeError("a product reported " + kt_mlp.kt_last_error())
    return layer, params, losses.tolist()


def quantise_matrix(w):
    """An [out][in] matrix in e4m3 with a scale for each block of 128 x 128."""
    N, K = w.shape
    blocks = torch.nn.functional.pad(w.float(), (0, -K % 128, 0, -N % 128)).unflatten(0, (-1, 128)).unflatten(2, (-1, 128))
    scale = (blocks.abs().amax((1, 3)) / 448.0).clamp_min(2.0 ** -100)
    q = (blocks / scale[:, None, :, None]).to(torch.float8_e4m3fn)
    return q.flatten(2, 3).flatten(0, 1)[:N, :K].contiguous(), scale


def serve(x, w):
    """y of the sublayer for the tokens x, in 8-bit floating point, from its 16-bit parameters."""
    M, D = x.shape
    F = w["down"].shape[1]
    (up, up_scale), (down, down_scale) = quantise_matrix(w["up"]), quantise_matrix(w["down"])  # once, as a model is loaded
    e4m3 = dict(dtype=torch.float8_e4m3fn, device="cuda")
    normed, p, y = torch.empty_like(x), torch.empty(M, 2 * F, dtype=x.dtype, device="cuda"), torch.empty_like(x)
    q, s = torch.empty(M, D, **e4m3), torch.empty(M, -(-D // 128), device="cuda")
    qh, sh = torch.empty(M, F, **e4m3), torch.empty(M, -(-F // 128), device="cuda")
    kt_ops.kt_layernorm_forward(x, w["gamma"], w["beta"], EPS, normed)
    kt_ops.kt_quantize_fp8(normed, q, s)
    kt_ops.kt_linear_fp8(q, s, up, up_scale, w["b_up"], p)
    kt_ops.kt_quantize_fp8(p, qh, sh, kt_mlp.KT_ACT_GEGLU)
    kt_ops.kt_linear_fp8(qh, sh, down, down_scale, w["b_down"], y)
    if kt_ops.kt_matmul_status() != kt_mlp.KT_OK:  # waits for the stream
        raise RuntimeError("a product reported " + kt_mlp.kt_last_error())
    return y


def main():
    layer, _, losses = train()
    print(f"training a gated sublayer: loss {losses[0]:.4f} -> {losses[-1]:.4f} in {len(losses)} steps")
    x = torch.randn(8, layer.normed.shape[1], device="cuda").bfloat16()
    y = serve(x, layer.w)
    exact = Sublayer(8, x.shape[1], layer.h.shape[1], layer.w).forward(x)
    off = ((y.float() - exact.float()).norm() / exact.float().norm()).item()
    print(f"served in e4m3 {list(y.shape)}: {off:.4f} of the bf16 sublayer's norm away from it")


if __name__ == "__main__":
    main()
