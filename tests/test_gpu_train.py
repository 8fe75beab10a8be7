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


@pytest.mark.parametrize("M", [1, 3, 64, 100, 130])
def test_cross_entropy_grad_of_a_label_is_not_rounded(awq, M):
    """The label's term makes up most of a row of dx (and, for few tokens, of dW).  With a gradient half way
    between two bf16 numbers its rounding alone would be off by 2^-8 of it, as much as the result's own."""
    V, I = 3000, 256
    x, W, labels = ce_case(M, V, I, M)
    labels[:] = torch.arange(M, device="cuda") * 7
    x *= 2.0 ** -10
    W[labels] *= 64
    _, lse = awq.awq_cross_entropy(x, W, labels)
    x8, W8, rows = x.to(F8), W.to(F8), torch.arange(M, device="cuda")
    l = x8 @ W8.T
    el = acc(I) * (x8.abs() @ W8.abs().T) + 2.0 ** -21 * (1 + l.abs() + lse.to(F8).abs()[:, None])
    p = torch.exp(l - lse.to(F8)[:, None])
    dloss = ((1 + 2.0 ** -8) / (1 - p[rows, labels])).float()
    dx, dW = awq.awq_cross_entropy_grad(x, W, labels, lse, dloss)
    wgt = dloss.to(F8)[:, None]
    ep = p * el * 1.01
    p[rows, labels] -= 1.0
    d, ed = p * wgt, ep * wgt.abs() + 2.0 ** -23 * (p * wgt).abs()     # before any rounding to 16 bits
    off = torch.ones_like(d)
    off[rows, labels] = 0.0
    dx_r = d @ W8
    e = (ed + UBF * off * d.abs()) @ W8.abs() + acc(V + 4096) * (d.abs() @ W8.abs())
    within(dx, dx_r, e + UBF * (dx_r.abs() + e) + 1e-38, "dx")
    dW_r = d.T @ x8
    u = UBF * UBF if M <= 128 else UBF                 # two bf16 numbers, or one
    e = (ed + u * d.abs()).T @ x8.abs() + acc(2 * M) * 2 * (d.abs().T @ x8.abs())
    within(dW, dW_r, e + UBF * (dW_r.abs() + e) + 1e-38, "dW")


# ------------------------------------------------------------------ what the formulas leave open
def ffn(seed, M=40, I=256, F=320, gs=64):
    w, D, s = packed(2 * F, I, gs, True, True, seed)
    return w, D, s, rand(M, I, seed + 1), rand(M, F, seed + 2, 1e-3)


def every_call(awq, M, seed=7):
    """One call of each operator on its own inputs, as functions that return their outputs."""
    w, D, s, x, dh = ffn(seed, M=M)
    wl, _, _ = packed(192, 256, 64, False, True, seed + 3)
    dy = rand(M, 192, seed + 4, 1e-4)
    xc, W, labels = ce_case(M, 5003, 128, seed + 5)
    _, lse = awq.awq_cross_entropy(xc, W, labels)
    dloss = torch.full((M,), 1.0 / M, device="cuda")
    return {
        "gated": lambda: (awq.awq_gated_w4a16(x, *w, group_size=64),),
        "gated_grad": lambda: (awq.awq_gated_w4a16_grad(dh, x, *w, group_size=64),),
        "linear_grad": lambda: (awq.awq_linear_w4a16_grad(dy, *wl, group_size=64),),
        "ce": lambda: awq.awq_cross_entropy(xc, W, labels),
        "ce_grad": lambda: awq.awq_cross_entropy_grad(xc, W, labels, lse, dloss),
    }


# tokens of every path: decode, dequantised on the way (one and several token tiles), dense
PATHS = [1, 11, 40, 130, 200, 400]


@pytest.mark.parametrize("M", PATHS)
def test_same_bits_again_and_on_another_stream(awq, M):
    for name, call in every_call(awq, M).items():
        first = [t.clone() for t in call()]
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            other = call()
        torch.cuda.current_stream().wait_stream(side)
        for a, b, c in zip(first, call(), other):
            assert torch.equal(a, b) and torch.equal(a, c), name


@pytest.mark.parametrize("M", PATHS)
def test_captured_and_replayed(awq, M):
    calls = every_call(awq, M)
    want = {n: [t.clone() for t in c()] for n, c in calls.items()}
    torch.cuda.synchronize()
    graphs = {}
    for n, c in calls.items():                       # two graphs of each call, replayed in turn
        pair = []
        for _ in range(2):
            g = torch.cuda.CUDAGraph()
            with torch.cuda.graph(g):
                outs = c()
            pair.append((g, outs))
        graphs[n] = pair
    for _ in range(2):
        for n, pair in graphs.items():
            for g, outs in pair:
                for t in outs:
                    t.fill_(float("nan"))
                g.replay()
    torch.cuda.synchronize()
    for n, pair in graphs.items():
        for _, outs in pair:
            for a, b in zip(want[n], outs):
                assert torch.equal(a, b), n


def test_calls_on_two_streams_at_once(awq):
    a, b = every_call(awq, 40, seed=7), every_call(awq, 40, seed=50)
    want = {n: ([t.clone() for t in a[n]()], [t.clone() for t in b[n]()]) for n in a}
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    got = []
    for _ in range(3):
        for n in a:
            with torch.cuda.stream(s1):
                x = a[n]()
            with torch.cuda.stream(s2):
                y = b[n]()
            got.append((n, x, y))
    torch.cuda.synchronize()
    for n, x, y in got:
        for t, w in zip(x, want[n][0]):
            assert torch.equal(t, w), n
        for t, w in zip(y, want[n][1]):
            assert torch.equal(t, w), n


def test_calls_back_to_back(awq):
    """Calls of every path in mixed order with nothing between them, each reading what the one before it
    wrote where it can: kernels start while their predecessors end, and workspaces are used again at once."""
    calls = {(n, M): c for M in PATHS for n, c in every_call(awq, M, seed=60 + M).items()}
    chains = {}
    for M in (1, 20, 130, 300):
        w, _, _ = packed(2 * 2816, 1024, 128, True, True, 70 + M)
        wd, _, _ = packed(2816, 1024, 128, False, True, 71 + M)
        x = rand(M, 1024, 72 + M)

        def chain(x=x, w=w, wd=wd):
            h = awq.awq_gated_w4a16(x, *w)
            y = awq.awq_linear_w4a16_grad(h, *wd)     # [M, 1024] again
            z = awq.awq_gated_w4a16(y, *w)
            return h, y, z, awq.awq_gated_w4a16_grad(z, y, *w)
        chains[("chain", M)] = chain
    calls.update(chains)
    want = {}
    for n, c in calls.items():
        want[n] = [t.clone() for t in c()]
        torch.cuda.synchronize()
    order = np.random.default_rng(20261208).permutation(np.repeat(np.arange(len(calls)), 8))
    names = list(calls)
    for part in np.array_split(order, 4):
        got = [(names[k], calls[names[k]]()) for k in part]
        torch.cuda.synchronize()
        for n, outs in got:
            for a, b in zip(outs, want[n]):
                assert torch.equal(a, b), n


@pytest.mark.parametrize("M", PATHS[1:])
def test_a_bad_token_stays_alone(awq, M):
    """NaN and infinities of one token reach that token's results only."""
    w, _, _, x, dh = ffn(9, M=M)
    good_h = awq.awq_gated_w4a16(x, *w, group_size=64)
    good_dx = awq.awq_gated_w4a16_grad(dh, x, *w, group_size=64)
    bad = x.clone()
    bad[1, 3], bad[1, 200] = float("nan"), float("inf")
    bad[M - 1] = float("-inf")
    h = awq.awq_gated_w4a16(bad, *w, group_size=64)
    dx = awq.awq_gated_w4a16_grad(dh, bad, *w, group_size=64)
    keep = torch.ones(M, dtype=torch.bool, device="cuda")
    keep[1] = keep[M - 1] = False
    assert torch.equal(h[keep], good_h[keep]) and torch.equal(dx[keep], good_dx[keep])
    assert not torch.isfinite(h[1].float()).all()
    wl, _, _ = packed(192, 256, 64, False, True, 12)
    dy = rand(M, 192, 13, 1e-4)
    good = awq.awq_linear_w4a16_grad(dy, *wl, group_size=64)
    dy[1, 5] = float("nan")
    got = awq.awq_linear_w4a16_grad(dy, *wl, group_size=64)
    keep[M - 1] = True
    assert torch.equal(got[keep], good[keep]) and torch.isnan(got[1].float()).any()


@pytest.mark.parametrize("M", [5, 64, 300])
def test_unscored_tokens_may_hold_anything(awq, M):
    x, W, labels = ce_case(M, 1000, 192, 21)
    labels[:] = torch.arange(M, device="cuda")
    labels[1], labels[2], labels[3], labels[4] = -100, 1000, -(2 ** 62), 2 ** 62
    off = [1, 2, 3, 4]
    _, lse = awq.awq_cross_entropy(x, W, labels)
    dloss = torch.full((M,), 0.25, device="cuda")
    want = awq.awq_cross_entropy_grad(x, W, labels, lse, dloss)
    bad, bad_d = x.clone(), dloss.clone()
    bad[1], bad[2], bad[3] = float("nan"), float("inf"), 3e38
    bad_d[1], bad_d[4] = float("nan"), float("inf")
    loss, bad_lse = awq.awq_cross_entropy(bad, W, labels)
    assert (loss[off] == 0).all() and torch.isfinite(loss).all()
    got = awq.awq_cross_entropy_grad(bad, W, labels, bad_lse, bad_d)
    assert (got[0][off] == 0).all()
    keep = torch.ones(M, dtype=torch.bool, device="cuda")
    keep[off] = False
    assert torch.equal(got[0][keep], want[0][keep]) and torch.equal(got[1], want[1])


def test_all_tokens_unscored(awq):
    x, W, labels = ce_case(33, 1000, 128, 22)
    labels[:] = -100
    loss, lse = awq.awq_cross_entropy(x, W, labels)
    dx, dW = awq.awq_cross_entropy_grad(x, W, labels, lse, torch.ones(33, device="cuda"))
    assert (loss == 0).all() and (dx == 0).all() and (dW == 0).all() and torch.isfinite(lse).all()


def test_certain_and_hopeless_labels(awq):
    """A label far above its rivals keeps the digits of its small loss, one far below keeps its large one,
    and a token with the same label as another adds to the same row of dW."""
    I, V = 128, 300
    W = torch.zeros(V, I, device="cuda", dtype=torch.bfloat16)
    W[7, 0] = 1.0
    x = torch.zeros(4, I, device="cuda", dtype=torch.bfloat16)
    x[0, 0], x[1, 0], x[2, 0], x[3, 0] = 20.0, -20.0, 200.0, -200.0
    labels = torch.full((4,), 7, device="cuda")
    loss, lse = awq.awq_cross_entropy(x, W, labels)
    l = x.to(F8) @ W.to(F8).T
    want = torch.logsumexp(l, 1) - l[:, 7]
    want[0] = math.log1p((V - 1) * math.exp(-20.0))
    want[2] = math.log1p((V - 1) * math.exp(-200.0))   # 0 in fp32
    # exp and log1p to a few units of fp32; 2 ulp of ex2 and its argument
    assert ((loss.to(F8) - want).abs() <= 2.0 ** -20 * want + 1e-38).all()
    dx, dW = awq.awq_cross_entropy_grad(x, W, labels, lse, torch.ones(4, device="cuda"))
    # row 7 of dW: sum over tokens of (p - 1) x, p = 2^-...: tokens 1 and 3 dominate
    p = torch.exp(l - torch.logsumexp(l, 1, keepdim=True))[:, 7] - 1
    ref = (p[:, None] * x.to(F8)).sum(0)
    assert abs(float(dW[7, 0]) - float(ref[0])) <= 2 * UBF * float((p.abs() * x[:, 0].to(F8).abs()).sum())


@pytest.mark.parametrize("M", PATHS)
@pytest.mark.parametrize("wscale,xscale,dscale", [(2.0 ** -12, 2.0 ** -40, 2.0 ** -60), (8.0, 2.0 ** 20, 2.0 ** 30),
                                                  (0.01, 2.0 ** -100, 1.0)])
def test_extreme_magnitudes(awq, M, wscale, xscale, dscale):
    """Powers of two far from 1 in weights, activations and gradients: nothing overflows or is flushed on
    the way (linear in each factor where the activation is linear: GELU of a large or tiny gate)."""
    O, I = 160, 256
    w, D, s = packed(O, I, 128, True, True, 33, scale=wscale)
    dy = (rand(M, O, 34).float() * dscale).to(torch.bfloat16)
    ref, tol = dx_ref(dy.to(F8), torch.zeros_like(dy, dtype=F8), D, s, O)
    within(awq.awq_linear_w4a16_grad(dy, *w), ref, tol, "dx")
    x = (rand(M, I, 35).float() * xscale).to(torch.bfloat16)
    ref, tol, _ = gated_ref(x, D, s, "silu")
    inside = ref.abs() < 1e37
    h = awq.awq_gated_w4a16(x, *w).to(F8)
    tol = tol + 2.0 ** -133                          # bf16 subnormals
    assert ((h - ref).abs()[inside] <= tol[inside]).all()


@pytest.mark.parametrize("M,rows", [(1, 8), (11, 16), (40, 64), (400, 512)])
def test_memory_behind_the_results_is_left_alone(awq, M, rows):
    w, _, _, x, dh = ffn(41, M=M)
    for call, cols in ((lambda out: awq.awq_gated_w4a16(x, *w, group_size=64, out=out), 320),
                       (lambda out: awq.awq_gated_w4a16_grad(dh, x, *w, group_size=64, out=out), 256)):
        buf = torch.full((rows, cols), 7.0, dtype=torch.bfloat16, device="cuda")
        call(buf[:M])
        assert (buf[M:] == 7.0).all() and not (buf[:M] == 7.0).all()


def test_gradients_against_differences(awq):
    """<dx, v> against central differences of the 64-bit forward along v."""
    M, I, F = 6, 128, 96
    for act in ("silu", "gelu", "gelu_tanh"):
        w, D, s = packed(2 * F, I, 64, True, True, 61)
        x, dh = rand(M, I, 62), rand(M, F, 63)
        dx = awq.awq_gated_w4a16_grad(dh, x, *w, group_size=64, act=act).to(F8)
        v = rand(M, I, 64).to(F8)

        def f(t):
            gu = ((x.to(F8) + t * v) / s) @ D.T
            return (act64(gu[:, :F], act)[0] * gu[:, F:] * dh.to(F8)).sum()
        e = 1e-6
        num = float((f(e) - f(-e)) / (2 * e))
        # elementwise bound of test_gated_grad, summed over |v| in the root-mean-square sense
        assert abs(float((dx * v).sum()) - num) <= 2.0 ** -7 * float(((dx * v) ** 2).sum().sqrt()) * 4
    x, W, labels = ce_case(6, 257, 64, 65)
    loss, lse = awq.awq_cross_entropy(x, W, labels)
    dloss = torch.ones(6, device="cuda")
    dx, dW = awq.awq_cross_entropy_grad(x, W, labels, lse, dloss)
    scored = labels >= 0

    def g(xx, WW):
        l = xx @ WW.T
        return (torch.logsumexp(l, 1) - l.gather(1, labels.clamp(min=0)[:, None])[:, 0])[scored].sum()
    e = 1e-6
    vx, vW = rand(6, 64, 66).to(F8), rand(257, 64, 67).to(F8)
    num = float((g(x.to(F8) + e * vx, W.to(F8)) - g(x.to(F8) - e * vx, W.to(F8))) / (2 * e))
    assert abs(float((dx.to(F8) * vx).sum()) - num) <= 2.0 ** -7 * float(((dx.to(F8) * vx) ** 2).sum().sqrt()) * 4
    num = float((g(x.to(F8), W.to(F8) + e * vW) - g(x.to(F8), W.to(F8) - e * vW)) / (2 * e))
    assert abs(float((dW.to(F8) * vW).sum()) - num) <= 2.0 ** -7 * float(((dW.to(F8) * vW) ** 2).sum().sqrt()) * 4


@pytest.mark.parametrize("M", [3, 60, 300])
def test_block_and_head_together(awq, M):
    """x -> gated -> down projection -> head -> loss and all the way back through packed layers, against
    64-bit autograd on the weights that the packed storage stands for."""
    I, F, V = 256, 448, 1500
    w, D, s = packed(2 * F, I, 128, True, True, 71)
    wd, Dd, sd = packed(I, F, 64, False, True, 72)
    x = rand(M, I, 73)
    _, W, labels = ce_case(M, V, I, 74)
    h = awq.awq_gated_w4a16(x, *w)
    y = awq.awq_linear_w4a16(h, *wd, group_size=64)
    y = (y.float() / y.float().norm(dim=1, keepdim=True) * 16).to(torch.bfloat16)
    loss, lse = awq.awq_cross_entropy(y, W, labels)
    n = int((labels >= 0).sum())
    dy, _ = awq.awq_cross_entropy_grad(y, W, labels, lse, torch.full((M,), 1.0 / max(n, 1), device="cuda"), want_dw=False)
    dh = awq.awq_linear_w4a16_grad(dy, *wd, group_size=64)
    dx = awq.awq_gated_w4a16_grad(dh, x, *w)
    # 64 bits, the rounded activations between the calls taken as they are
    y8 = y.to(F8).requires_grad_(True)
    lg = y8 @ W.to(F8).T
    scored = labels >= 0
    ref = (torch.logsumexp(lg, 1) - lg.gather(1, labels.clamp(min=0)[:, None])[:, 0])[scored].sum() / max(n, 1)
    assert abs(float(loss.sum()) / max(n, 1) - float(ref.detach())) <= 1e-5 * abs(float(ref.detach())) + 1e-6
    dy8 = torch.autograd.grad(ref, y8)[0]
    dh8 = (dy8 @ Dd) / sd
    x8 = x.to(F8).requires_grad_(True)
    gu = (x8 / s) @ D.T
    hh = torch.nn.functional.silu(gu[:, :F]) * gu[:, F:]
    dx8 = torch.autograd.grad((hh * dh8).sum(), x8)[0]
    for got, want in ((dy, dy8), (dh, dh8), (dx, dx8)):
        # three calls in a row, each rounding its result to bf16 (2^-8) and its operands to fp16 or bf16:
        # relative error in the 2-norm below 2^-8 a call and operand
        assert float((got.to(F8) - want).norm()) <= 6 * UBF * float(want.norm())
