"""AdamW over many tensors on the GPU: the definition's operations one by one, bit for bit."""
import pytest
import torch

from transformer_mlp_gemms_gb300 import kt_mlp, kt_ops

import train_reference as ref

pytestmark = pytest.mark.gpu
DT = {"f16": torch.float16, "bf16": torch.bfloat16, "f32": torch.float32}
HYPER = dict(lr=2e-3, beta1=0.9, beta2=0.99, eps=1e-8)
BLOCK = kt_ops.KT_ADAMW_BLOCK


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from transformer_mlp_gemms_gb300 import build
    build.build()
    kt_ops.load()


class Tensors:
    """Parameters, moments and what the definition makes of them; ``shift``: elements by which each tensor starts off an
    allocation's beginning."""

    def __init__(self, g, sizes, param, grad, bits, copy, shift=0):
        def make(n, dtype, std):
            t = torch.zeros(n + shift, dtype=dtype, device="cuda")[shift:]
            t.copy_((std * torch.randn(n, generator=g) * torch.exp(torch.randn(n, generator=g))).to(DT.get(dtype, dtype)))
            return t

        self.bits, self.sizes = bits, sizes
        self.g, self.grad, self.make = g, DT[grad], make
        self.p = [make(n, DT[param], 0.1) for n in sizes]
        state = torch.float32 if bits == 32 else torch.float8_e4m3fn
        self.m, self.v = ([torch.zeros(n + shift, dtype=state, device="cuda")[shift:] for n in sizes] for _ in range(2))
        blocks = [-(-n // BLOCK) for n in sizes]
        self.ms, self.vs = ([torch.zeros(n, device="cuda") for n in blocks] if bits == 8 else None for _ in range(2))
        self.copies = [make(n, DT[copy], 1.0) for n in sizes] if copy else None
        self.decay = [0.1 if i % 3 == 0 else 0.0 for i in range(len(sizes))]
        self.expect = [dict(p=p.clone(), m=torch.zeros(p.numel(), device="cuda"), v=torch.zeros(p.numel(), device="cuda")) for p in self.p]

    def grads(self):
        return [self.make(n, self.grad, 1e-2) for n in self.sizes]

    def step(self, grads, step, **kw):
        kt_ops.kt_adamw(self.p, grads, self.m, self.v, step, **HYPER, weight_decay=self.decay, m_scales=self.ms, v_scales=self.vs,
                        copies=self.copies, **kw)

    def follow(self, grads, step, scale=None):
        """The same step by the definition."""
        for e, g, d, n in zip(self.expect, grads, self.decay, self.sizes):
            p, m, v, r = ref.adamw(e["p"], g, e["m"], e["v"], step, *HYPER.values(), d, scale)
            e["full"], e["p"] = p, p.to(e["p"].dtype)
            if self.bits == 32:
                e["m"], e["v"] = m, v
                continue
            for name, x in (("m", m), ("v", r)):
                q, s = ref.e4m3(x, BLOCK, root=name == "v")
                e[name + "q"], e[name + "s"] = q, s
                wide = ref.widen(q, s, BLOCK)
                e[name] = wide if name == "m" else wide * wide

    def check(self):
        for i, e in enumerate(self.expect):
            assert torch.equal(self.p[i], e["p"]), (i, "p")
            if self.copies:
                assert torch.equal(self.copies[i], e["full"].to(self.copies[i].dtype)), (i, "copy")
            if self.bits == 32:
                assert torch.equal(self.m[i], e["m"]) and torch.equal(self.v[i], e["v"]), i
            else:
                for name, got, scales in (("m", self.m, self.ms), ("v", self.v, self.vs)):
                    assert torch.equal(scales[i], e[name + "s"]), (i, name + " scale")
                    assert torch.equal(got[i].view(torch.uint8), e[name + "q"].view(torch.uint8)), (i, name)


SIZES = [1, 7, 255, 256, 257, 2048, 2049, 5000, 40003]


@pytest.mark.parametrize("bits", [8, 32])
@pytest.mark.parametrize("param,grad,copy", [("f32", "f32", ""), ("f32", "bf16", "bf16"), ("f32", "f16", "f16"), ("bf16", "bf16", ""),
                                             ("f16", "f16", ""), ("bf16", "f32", ""), ("f16", "f32", ""), ("f16", "bf16", ""), ("bf16", "f16", "")])
@pytest.mark.parametrize("shift", [0, 1])
def test_steps(param, grad, copy, bits, shift):
    t = Tensors(torch.Generator().manual_seed(bits), SIZES, param, grad, bits, copy, shift)
    for step in range(1, 5):
        grads = t.grads()
        t.step(grads, step)
        t.follow(grads, step)
        t.check()


@pytest.mark.parametrize("bits", [8, 32])
@pytest.mark.parametrize("count", [1, 24, 25, 360, 361, 800])
def test_many_tensors(count, bits):
    """On both sides of each number of tensors that a launch's parameters hold; some of no length."""
    g = torch.Generator().manual_seed(count)
    sizes = [int(n) for n in torch.randint(0, 3000, (count,), generator=g)]
    t = Tensors(g, sizes, "f32", "bf16", bits, "bf16")
    grads = t.grads()
    t.step(grads, 1)
    t.follow(grads, 1)
    t.check()


@pytest.mark.parametrize("bits", [8, 32])
def test_a_large_tensor_among_small_ones(bits):
    t = Tensors(torch.Generator().manual_seed(5), [300, 3_000_017, 10, 1_000_000], "bf16", "bf16", bits, "")
    for step in (1, 2):
        grads = t.grads()
        t.step(grads, step)
        t.follow(grads, step)
    t.check()


def test_moments_of_any_magnitude():
    """Blocks of zeros, of values below what a scale can divide, of one value among zeros, of magnitudes far apart (a root
    that is not zero stays so), and infinities and NaN, which stay within their block."""
    n = 8 * BLOCK
    t = Tensors(torch.Generator().manual_seed(5), [n], "f32", "f32", 8, "")
    g = torch.zeros(8, BLOCK)
    g[1] = 1e-30  # m is below 2^-100
    g[2, 17] = 3.0
    g[3] = torch.exp2(torch.linspace(-60, 10, BLOCK))
    g[4] = -1e10
    g[5] = torch.linspace(-1, 1, BLOCK)
    g[5, 9] = float("nan")
    g[6] = 1.0
    g[6, 200] = float("inf")
    g[7] = 1e-3
    grads = [g.view(-1).cuda()]
    before = t.p[0].clone()
    t.step(grads, 1)
    t.follow(grads, 1)
    bad = slice(5 * BLOCK, 7 * BLOCK)
    for got, want in ((t.p[0], t.expect[0]["p"]), (t.ms[0], t.expect[0]["ms"]), (t.vs[0], t.expect[0]["vs"])):
        assert torch.equal(got.nan_to_num(-7.0), want.nan_to_num(-7.0))
    good = torch.ones(n, dtype=torch.bool)
    good[bad] = False
    for got, want in ((t.m[0], t.expect[0]["mq"]), (t.v[0], t.expect[0]["vq"])):
        assert torch.equal(got.view(torch.uint8)[good.cuda()], want.view(torch.uint8)[good.cuda()])
    assert (t.v[0][3 * BLOCK:4 * BLOCK].float() > 0).all()
    assert t.ms[0][5].isnan() and t.vs[0][5].isnan() and not t.ms[0][6].isfinite()
    assert t.p[0][good.cuda()].isfinite().all()
    assert torch.equal(t.p[0][:BLOCK], before[:BLOCK] * (1.0 - HYPER["lr"] * 0.1))


@pytest.mark.parametrize("bits", [8, 32])
def test_a_captured_step_counts_on(bits):
    """The step's number on the device, raised in the graph; the gradients' scale likewise."""
    t = Tensors(torch.Generator().manual_seed(6), [300, 5000], "f32", "bf16", bits, "bf16")
    grads = t.grads()
    step = torch.zeros(1, dtype=torch.int64, device="cuda")
    scale = torch.tensor(0.5, device="cuda")
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step.add_(1)
        t.step(grads, step, grad_scale=scale)
    for i in range(1, 6):
        for g, new in zip(grads, t.grads()):
            g.copy_(new)
        scale.fill_(1.0 / i)
        graph.replay()
        torch.cuda.synchronize()
        t.follow(grads, i, scale)
        t.check()


def test_the_definition_is_the_usual_one():
    """Against AdamW in 64 bits: p is off by a few fp32 roundings of itself and of the step."""
    g = torch.Generator().manual_seed(9)
    p = torch.randn(5000, generator=g, dtype=torch.float64)
    t = [torch.empty(5000, device="cuda")]
    t[0].copy_(p)
    p = t[0].double()
    m, v = [torch.zeros(5000, device="cuda")], [torch.zeros(5000, device="cuda")]
    mx, vx = torch.zeros_like(p), torch.zeros_like(p)
    tol = torch.zeros_like(p)
    for step in range(1, 6):
        grad = torch.randn(5000, generator=g).cuda()
        kt_ops.kt_adamw(t, [grad], m, v, step, 1e-2, 0.9, 0.999, 1e-8, 0.05)
        mx, vx = 0.9 * mx + 0.1 * grad.double(), 0.999 * vx + 0.001 * grad.double() ** 2
        update = (mx / (1 - 0.9 ** step)) / ((vx / (1 - 0.999 ** step)).sqrt() + 1e-8)
        p = p * (1 - 1e-2 * 0.05) - 1e-2 * update
        # m: a sum of up to 5 terms that may cancel; v: none do; the quotient's and the difference's roundings
        terms = sum(0.9 ** k for k in range(step)) * 0.1 * 4.5
        tol = tol + 2.0 ** -24 * (3 * p.abs() + 1e-2 * (16 * update.abs() + 16 * terms / (vx / (1 - 0.999 ** step)).sqrt()))
    assert ((t[0].double() - p).abs() <= tol).all()


@pytest.mark.parametrize("kind", ["any", "near powers", "few bits", "wide"])
def test_roots_and_quotients_are_correctly_rounded(kind):
    """p = -(m / (sqrt(v) + 1)) bit for bit (halved moments, no gradient, lr 1, a correction of 1 / sqrt(1 - 1/4)): random
    significands, ones next to powers of two, ones of few bits, and magnitudes past those that the quick way takes."""
    n = 1 << 23
    g = torch.Generator(device="cuda").manual_seed(len(kind))
    bits = lambda lo, hi: torch.randint(lo, hi, (n,), generator=g, device="cuda", dtype=torch.int64)  # noqa: E731

    def values(span):
        significand = {"near powers": (bits(-40, 40) + (1 << 23)) % (1 << 23), "few bits": bits(0, 1 << 12) << 11}.get(kind, bits(0, 1 << 23))
        return (((127 + bits(-span, span + 1)) << 23) | significand).to(torch.int32).view(torch.float32)

    span = 126 if kind == "wide" else 20
    m, v = values(span) * torch.where(bits(0, 2) == 0, 1.0, -1.0), values(span)
    m[:1000], v[:2000:2] = 0.0, 0.0
    p, zero = torch.zeros(n, device="cuda"), torch.zeros(n, device="cuda")
    a, r = m * 0.5 * (1.0 / (1.0 - 0.5 ** 2)), torch.sqrt(v * 0.5)
    want = 0.0 - a / (r * (1.0 / (1.0 - 0.5 ** 2) ** 0.5) + 1e-6)
    kt_ops.kt_adamw([p], [zero], [m.clone()], [v.clone()], 2, 1.0, 0.5, 0.5, 1e-6)
    assert torch.equal(p, want)


def test_on_another_stream_and_without_tensors():
    t = Tensors(torch.Generator().manual_seed(6), [300, 5000], "f32", "bf16", 32, "")
    grads = t.grads()
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    t.step(grads, 1, stream=side)
    side.synchronize()
    t.follow(grads, 1)
    t.check()
    kt_ops.kt_adamw([], [], [], [], 1, 1e-3)


def exact_quotients(a, b):
    """AdamW as a division: p = -(a / |b|), for a next to b in magnitude.  Moments that hardly move (beta1 = 1 - 2^-30 is 1 in
    fp32, and a gradient times 2^-30 is lost beside a), a second moment of the gradient's square alone (whose root is the
    gradient), no eps, and a rate of 2^-30 / (1 - beta1) = 1."""
    p = torch.zeros_like(a)
    kt_ops.kt_adamw([p], [b.clone()], [a.clone()], [torch.zeros_like(a)], 1, 2.0 ** -30, 1 - 2.0 ** -30, 0.0, 0.0)
    return -p


@pytest.mark.parametrize("exponent", [0, -38, 29])
def test_quotients_of_every_divisor_are_correctly_rounded(exponent):
    """Every significand as the divisor, for numerators at and next to powers of two, where a divisor next to the next
    power leaves the quotient next to the middle of two numbers (1.0 / 0x1.fffffep+0, 0x1.aaaaa6p+0 / 0x1.fffffap+0).
    The once refined reciprocal has to be the nearest number for that, which hangs on the hardware's approximation."""
    b = (torch.arange(1 << 23, device="cuda", dtype=torch.int32) + 0x3F800000).view(torch.float32)
    g = torch.Generator(device="cuda").manual_seed(1)
    some = (torch.randint(0, 1 << 23, b.shape, generator=g, device="cuda", dtype=torch.int32) + 0x3F800000).view(torch.float32)
    up = 2.0 ** -23
    numerators = [1.0, 1 + up, 1 + 2 * up, 1 + 3 * up, 2 - up, 2 - 2 * up, 2 - 3 * up, 1.5, float.fromhex("0x1.aaaaa6p+0"), 4 / 3, 1.75]
    for a in [torch.full_like(b, n) for n in numerators] + [some, b.flip(0), b]:
        want = (a.double() / b.double()).float()  # (of 24-bit numbers: the 53-bit quotient's rounding does not decide)
        assert torch.equal(exact_quotients(a * 2.0 ** exponent, b * 2.0 ** exponent), want)


def test_roots_of_every_number_are_correctly_rounded():
    """Both parities of the exponent: p = -(m 2^15 / (sqrt(v) 2^15)) with m the exact root, so that any other root than that
    leaves something else than -1."""
    v = (torch.arange(1 << 24, device="cuda", dtype=torch.int32) + 0x3F800000).view(torch.float32)
    m = v.double().sqrt().float()
    p, zero, beta = torch.zeros_like(v), torch.zeros_like(v), 1 - 2.0 ** -30
    kt_ops.kt_adamw([p], [zero], [m.clone()], [v.clone()], 1, 2.0 ** -15, beta, beta, 0.0)
    assert (p == -1).all()
    p.zero_()
    off = torch.nextafter(m, torch.full_like(m, float("inf")))  # another root would show
    kt_ops.kt_adamw([p], [zero], [off], [v.clone()], 1, 2.0 ** -15, beta, beta, 0.0)
    assert (p != -1).all()
