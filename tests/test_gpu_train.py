"""GPU checks of the operators that train through packed weights and score a vocabulary, against
their formulas in 64 bits: awq_gated_w4a16, awq_gated_w4a16_grad, awq_linear_w4a16_grad,
awq_cross_entropy and awq_cross_entropy_grad.

Tolerances are worked out per element from the roundings the header names, u16 = 2^-11 (fp16) and
ubf = 2^-8 (bf16), relative to the value rounded:
  * a product of rounded operands is off by at most (2 u16 + acc) * sum |a| |b|, where acc =
    (K / 16 + 16) * 2^-23 covers the fp32 accumulation (one truncation per 16-deep step, bounded by
    the sum of magnitudes);
  * act has |act'| <= 1.2 and |act''| <= 1;
  * a result is rounded once to bf16.
"""
import math

import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu

U16, UBF = 2.0 ** -11, 2.0 ** -8
F8 = torch.float64


@pytest.fixture(scope="module")
def awq():
    import weight_only_quantization_awq_b200 as m
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    return m


def acc(K):
    return (K / 16 + 16) * 2.0 ** -23


def packed(O, I, gs, zeros, s16, seed, scale=0.01):
    """A packed layer of random codes and its 64-bit weights."""
    rng = np.random.default_rng([20261202, 31, seed])
    nG = I // gs
    code = rng.integers(0, 16, (O, I))
    z = rng.integers(0, 16, (O, nG)) if zeros else np.full((O, nG), 8)
    delta = (scale * np.exp(0.5 * rng.standard_normal((O, nG)))).astype(np.float16)
    nib = np.zeros((O, I // 8), np.uint32)
    for k in range(8):
        nib |= code[:, k::8].astype(np.uint32) << np.uint32(4 * k)
    zw = None
    if zeros:
        zp = np.zeros((O, (nG + 7) // 8 * 8), np.int64)
        zp[:, :nG] = z
        zw = np.zeros((O, zp.shape[1] // 8), np.uint32)
        for k in range(8):
            zw |= zp[:, k::8].astype(np.uint32) << np.uint32(4 * k)
    s = np.exp(-2.0 * rng.random(I)).astype(np.float16) if s16 else None
    D = (code - np.repeat(z, gs, 1)) * np.repeat(delta.astype(np.float64), gs, 1)
    dev = lambda a: torch.from_numpy(a.view(np.int32) if a.dtype == np.uint32 else a).cuda()  # noqa: E731
    w = (dev(nib), dev(delta), dev(zw) if zeros else None, dev(s) if s16 else None)
    return w, dev(D), dev(s).to(F8) if s16 else torch.ones(I, dtype=F8, device="cuda")


def rand(M, cols, seed, scale=1.0):
    rng = np.random.default_rng([20261202, 32, seed])
    x = rng.standard_normal((M, cols)) * scale
    x[:, rng.choice(cols, max(1, cols // 64))] *= 30.0
    return torch.from_numpy(x.astype(np.float32)).cuda().to(torch.bfloat16)


def act64(g, act):
    """act(g) and act'(g) in 64 bits."""
    g = g.detach().requires_grad_(True)
    f = {"silu": torch.nn.functional.silu, "gelu": torch.nn.functional.gelu,
         "gelu_tanh": lambda t: torch.nn.functional.gelu(t, approximate="tanh")}[act]
    a = f(g)
    (d,) = torch.autograd.grad(a.sum(), g)
    return a.detach(), d


def within(got, ref, tol, what):
    got = got.to(F8)
    assert torch.isfinite(got).all(), what
    over = (got - ref).abs() - tol
    assert (over <= 0).all(), (what, float(((got - ref).abs() / tol.clamp(min=1e-300)).max()))


def gated_ref(x, D, s, act):
    """h, its tolerance, and what the gradient needs."""
    F = D.shape[0] // 2
    xs = x.to(F8) / s
    gu = xs @ D.T
    e = (2 * U16 + acc(D.shape[1])) * (xs.abs() @ D.abs().T) * 1.01 + 1e-30
    g, u, eg, eu = gu[:, :F], gu[:, F:], e[:, :F], e[:, F:]
    a, da = act64(g, act)
    # fp32 evaluation of the activation: a few units of 2^-22 of |g|
    ea = 1.2 * eg + 2.0 ** -20 * g.abs()
    h = a * u
    eh = u.abs() * ea + a.abs() * eu + ea * eu
    return h, eh + UBF * (h.abs() + eh) + 1e-38, (a, da, g, u, ea, eu, eg)


SHAPES = [  # M, in, F, gs, zeros, s16, act
    (1, 64, 1, 64, False, True, "silu"),
    (1, 128, 7, 128, True, True, "silu"),
    (2, 64, 33, 32, True, False, "gelu"),
    (3, 192, 130, 64, False, True, "gelu_tanh"),
    (5, 512, 688, 128, True, True, "silu"),
    (8, 1024, 96, 32, False, True, "silu"),
    (16, 256, 129, 128, True, False, "gelu_tanh"),
    (17, 320, 64, 64, True, True, "silu"),
    (33, 640, 257, 128, False, True, "gelu"),
    (64, 128, 1000, 128, True, True, "silu"),
    (100, 896, 511, 64, True, False, "silu"),
    (128, 512, 128, 32, False, True, "gelu_tanh"),
    (255, 256, 300, 32, True, True, "silu"),
    (257, 384, 1031, 128, True, True, "gelu"),
    (513, 2048, 704, 128, False, False, "silu"),
    (600, 128, 2051, 64, True, True, "gelu"),
]


@pytest.mark.parametrize("M,I,F,gs,zeros,s16,act", SHAPES)
def test_gated(awq, M, I, F, gs, zeros, s16, act):
    w, D, s = packed(2 * F, I, gs, zeros, s16, M + F)
    x = rand(M, I, M + 1)
    out = torch.full((M, F), float("nan"), dtype=torch.bfloat16, device="cuda")
    h = awq.awq_gated_w4a16(x, *w, group_size=gs, act=act, out=out)
    assert h is out
    ref, tol, _ = gated_ref(x, D, s, act)
    within(h, ref, tol, "h")


def dx_ref(d, ed, D, s, K):
    """dx of operand gradients d (each off by at most ed) and its tolerance."""
    dx = (d @ D) / s
    e = ((ed @ D.abs()) * (1 + 2 * U16) + (2 * U16 + acc(K)) * (d.abs() @ D.abs())) / s * 1.01
    return dx, e + UBF * (dx.abs() + e) + 1e-38


@pytest.mark.parametrize("M,I,F,gs,zeros,s16,act", SHAPES)
def test_gated_grad(awq, M, I, F, gs, zeros, s16, act):
    w, D, s = packed(2 * F, I, gs, zeros, s16, M + F)
    x, dh = rand(M, I, M + 1), rand(M, F, M + 2, 1e-3)
    if M > 2:
        dh[1] = 0                                    # a row of padding
    out = torch.full((M, I), float("nan"), dtype=torch.bfloat16, device="cuda")
    dx = awq.awq_gated_w4a16_grad(dh, x, *w, group_size=gs, act=act, out=out)
    assert dx is out
    _, _, (a, da, g, u, ea, eu, eg) = gated_ref(x, D, s, act)
    d = dh.to(F8)
    dg, du = d * u * da, d * a
    eda = eg + 2.0 ** -20 * (1 + g.abs())            # |act''| <= 1; fp32 evaluation of act'
    # fp16's subnormal step below the scaled row: 2^-25 of 2^15 / 2^12 (the bound's slack)
    floor = 2.0 ** -26 * torch.cat((dg, du), 1).abs().amax(1, keepdim=True)
    edg = d.abs() * (eu * 1.2 + u.abs() * eda + eu * eda)
    edu = d.abs() * ea
    dd = torch.cat((dg, du), 1)
    ref, tol = dx_ref(dd, torch.cat((edg, edu), 1) + floor, D, s, 2 * F)
    within(dx, ref, tol, "dx")
    if M > 2:
        assert (dx[1] == 0).all()


@pytest.mark.parametrize("M,O,I,gs,zeros,s16", [
    (1, 1, 64, 64, False, True), (1, 9, 128, 128, True, True), (2, 130, 64, 32, True, False),
    (7, 64, 1024, 128, False, True), (16, 1000, 192, 64, True, True), (19, 512, 1376 // 32 * 64, 64, False, True),
    (65, 2048, 256, 32, True, False), (130, 77, 640, 128, True, True), (256, 1031, 384, 128, False, True),
    (300, 4096, 512, 64, True, True), (700, 333, 2304, 128, True, False),
    (600, 6001, 128, 64, True, True), (515, 1200, 4096, 128, False, True),
])
def test_linear_grad(awq, M, O, I, gs, zeros, s16):
    w, D, s = packed(O, I, gs, zeros, s16, M + O)
    dy = rand(M, O, M + 3, 1e-4)
    out = torch.full((M, I), float("nan"), dtype=torch.bfloat16, device="cuda")
    dx = awq.awq_linear_w4a16_grad(dy, *w, group_size=gs, out=out)
    assert dx is out
    ref, tol = dx_ref(dy.to(F8), torch.zeros_like(dy, dtype=F8), D, s, O)
    within(dx, ref, tol, "dx")


def ce_case(M, V, I, seed, scale=0.05):
    rng = np.random.default_rng([20261202, 33, seed])
    x = torch.from_numpy(rng.standard_normal((M, I)).astype(np.float32)).cuda().to(torch.bfloat16)
    W = torch.from_numpy((scale * rng.standard_normal((V, I))).astype(np.float32)).cuda().to(torch.bfloat16)
    labels = torch.from_numpy(rng.integers(0, V, M)).cuda()
    if M > 2:
        labels[::3] = -100
        labels[1] = V - 1
        labels[2] = 0
    return x, W, labels


CE_SHAPES = [(1, 1, 64), (1, 100, 128), (2, 257, 64), (3, 4096, 192), (13, 9973, 512), (128, 64, 1024),
             (129, 1000, 320), (255, 5003, 64), (256, 256, 512), (300, 12345, 128), (511, 33, 2048), (70, 20011, 256),
             (2100, 16500, 64)]


@pytest.mark.parametrize("M,V,I", CE_SHAPES)
def test_cross_entropy(awq, M, V, I):
    x, W, labels = ce_case(M, V, I, M + V)
    loss, lse = awq.awq_cross_entropy(x, W, labels)
    l = x.to(F8) @ W.to(F8).T
    el = acc(I) * (x.to(F8).abs() @ W.to(F8).abs().T)
    ref = torch.logsumexp(l, 1)
    # exponentials, their sum and the logarithm in fp32: (32 + V / 32) additions of 2^-24 at most,
    # a few units for each exponential (whose argument is rounded at |l - max|), one for the value
    spread = (l.amax(1) - l.amin(1))
    tol = el.amax(1) + (64 + V / 32) * 2.0 ** -24 + 2.0 ** -22 * spread + 2.0 ** -22 * (ref.abs() + l.abs().amax(1) + 1)
    within(lse, ref, tol, "lse")
    scored = (labels >= 0) & (labels < V)
    at = labels.clamp(0, V - 1)[:, None]
    want = torch.where(scored, ref - l.gather(1, at)[:, 0], 0.0)
    within(loss, want, tol + el.gather(1, at)[:, 0] + 2.0 ** -23 * l.abs().amax(1), "loss")
    assert (loss[~scored] == 0).all()


@pytest.mark.parametrize("want_dw", [True, False])
@pytest.mark.parametrize("M,V,I", CE_SHAPES)
def test_cross_entropy_grad(awq, M, V, I, want_dw):
    x, W, labels = ce_case(M, V, I, M + V)
    _, lse = awq.awq_cross_entropy(x, W, labels)
    rng = np.random.default_rng([20261202, 34, M])
    dloss = torch.from_numpy((rng.random(M) / M).astype(np.float32)).cuda()
    nan = dict(dtype=torch.bfloat16, device="cuda")
    dx0 = torch.full((M, I), float("nan"), **nan)
    dW0 = torch.full((V, I), float("nan"), **nan) if want_dw else None
    dx, dW = awq.awq_cross_entropy_grad(x, W, labels, lse, dloss, want_dw=want_dw, dx=dx0, dW=dW0)
    assert dx is dx0 and dW is dW0
    x8, W8 = x.to(F8), W.to(F8)
    l = x8 @ W8.T
    el = acc(I) * (x8.abs() @ W8.abs().T) + 2.0 ** -21 * (1 + l.abs() + lse.to(F8).abs()[:, None])
    p = torch.exp(l - lse.to(F8)[:, None])
    scored = (labels >= 0) & (labels < V)
    wgt = torch.where(scored, dloss.to(F8), 0.0)[:, None]
    ep = p * el * 1.01
    p[torch.arange(M, device="cuda"), labels.clamp(0, V - 1)] -= 1.0
    d, ed = p * wgt, ep * wgt.abs()
    ed = ed + UBF * (d.abs() + ed) + 1e-38
    dx_r = d @ W8
    e = ed @ W8.abs() + acc(V + 4096) * (d.abs() @ W8.abs())
    within(dx, dx_r, e + UBF * (dx_r.abs() + e) + 1e-38, "dx")
    if want_dw:
        dW_r = d.T @ x8
        e = ed.T @ x8.abs() + acc(M) * (d.abs().T @ x8.abs())
        within(dW, dW_r, e + UBF * (dW_r.abs() + e) + 1e-38, "dW")
