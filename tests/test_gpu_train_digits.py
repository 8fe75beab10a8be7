"""GPU checks of the digits that the gated, gradient and cross-entropy calls keep: the label's gradient of
confident tokens, and magnitudes at the ends of the formats.  Tolerances as in test_gpu_train and
test_gpu_train_paths."""
import numpy as np
import pytest
import torch

from test_gpu_train import F8, PATHS, UBF, awq, ce_case, dx_ref, gated_ref, packed, rand, within  # noqa: F401
from test_gpu_train_paths import BF16_NORM, normwise

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("want_dw", [False, True])
@pytest.mark.parametrize("M", [1, 13, 64, 65, 130, 300])
def test_label_gradient_of_confident_tokens(awq, M, want_dw):  # noqa: F811
    """d[label] = exp(t - lse) - 1 where t is nearly lse: what is left is as exact as t and lse are.

    Dense positive rows of 4096 columns, t from 13 to 21, 1 - p from 1e-2 to 1e-4.  Column 0 is 1 in the label's row
    of W and 0 elsewhere, so dx[:, 0] is d[label] itself, rounded to bf16.  t in fp32 is 64 chains (32 lanes of two)
    of 64 FMAs and a tree: each rounding of a chain is at most 2^-24 of at most t / 64, those of a level of the tree
    2^-24 t in all; as independent and uniform errors their standard deviations are sqrt(64 x 64 / 3) / 64 = 0.6 and
    below sqrt(2 / 3) = 0.8 of 2^-24 t, together one: the bound is eight of those, 2^-21 t.  (lse is an input.)"""
    I, V, L = 4096, 301, 77
    rng = np.random.default_rng([20261209, 41, M])
    x = np.abs(rng.standard_normal((M, I))) + 0.2
    x[:, 0] = 0.0
    W = np.abs(rng.standard_normal((V, I))) * 0.3 + 1.0
    W *= 0.29 / W.mean()
    W[L] *= 1.0 / 0.29
    gap = np.log((V - 1) / 10.0 ** -(2 + 2 * rng.random(M)))   # t minus the other logits
    x *= (gap / (0.71 * I * x.mean(1)))[:, None] * 64           # rows of W carry 1 / 64
    W /= 64
    W[:, 0] = 0.0
    W[L, 0] = 1.0
    dev = lambda a: torch.from_numpy(a.astype(np.float32)).cuda().to(torch.bfloat16)  # noqa: E731
    x, W = dev(x), dev(W)
    labels = torch.full((M,), L, device="cuda")
    _, lse = awq.awq_cross_entropy(x, W, labels)
    t = (x.to(F8) * W[L].to(F8)).sum(1)
    d = torch.expm1(t - lse.to(F8))
    assert ((-d > 3e-5) & (-d < 5e-2)).all() and (t > 10).all()
    dx, dW = awq.awq_cross_entropy_grad(x, W, labels, lse, torch.ones(M, device="cuda"), want_dw=want_dw)
    et = 2.0 ** -21 * t + 2.0 ** -22 * d.abs()       # and the rounding of expm1
    within(dx[:, 0], d, et + UBF * (d.abs() + et), "d[label]")
    if want_dw:
        ref = (d[:, None] * x.to(F8)).sum(0)
        u = UBF * UBF if M <= 128 else UBF
        e = ((et + u * d.abs())[:, None] * x.to(F8)).sum(0) + 2.0 ** -16 * ref.abs()
        within(dW[L], ref, e + UBF * (ref.abs() + e) + 1e-30, "dW[label]")


def signed_gates(F, I, scale, seed):
    """A packed layer (group 128) whose gate rows are positive (even f) or negative throughout."""
    rng = np.random.default_rng([20261209, 42, seed])
    code = rng.integers(0, 16, (2 * F, I))
    code[:F] = np.where(np.arange(F)[:, None] % 2 == 0, 12, 4)
    nib = np.zeros((2 * F, I // 8), np.uint32)
    for k in range(8):
        nib |= code[:, k::8].astype(np.uint32) << np.uint32(4 * k)
    delta = (scale * np.exp(0.3 * rng.standard_normal((2 * F, I // 128)))).astype(np.float16)
    D = (code - 8) * np.repeat(delta.astype(np.float64), 128, 1)
    dev = lambda a: torch.from_numpy(a).cuda()  # noqa: E731
    return (dev(nib.view(np.int32)), dev(delta), None, None), dev(D)


@pytest.mark.parametrize("M", PATHS)
@pytest.mark.parametrize("act", ["silu", "gelu", "gelu_tanh"])
def test_gates_far_from_zero(awq, M, act):  # noqa: F811
    """Gates of +-2^70: the derivative is 1 or 0 (gelu_tanh's polynomial in g^2 leaves fp32's range on the way)."""
    F, I = 72, 256
    w, D = signed_gates(F, I, 0.01, M)
    x = (rand(M, I, 43).float().abs() * 2.0 ** 68).to(torch.bfloat16)
    dh = (rand(M, F, 44).float() * 2.0 ** -90).to(torch.bfloat16)
    gu = x.to(F8) @ D.T
    g, u, d = gu[:, :F], gu[:, F:], dh.to(F8)
    assert (g.abs() > 2.0 ** 66).all()
    on = (g > 0).to(F8)
    dx = awq.awq_gated_w4a16_grad(dh, x, *w, act=act)
    assert torch.isfinite(dx.float()).all()
    normwise(dx, torch.cat((d * u * on, d * g * on), 1) @ D, BF16_NORM, "dx")
    h = awq.awq_gated_w4a16(x, *w, act=act)
    off = (g < 0)
    assert (h[off] == 0).all()


@pytest.mark.parametrize("M", PATHS)
def test_rows_near_the_end_of_the_range(awq, M):  # noqa: F811
    """Rows of 2^112 through weights of 2^-12: results of 2^105, whatever the order of the power-of-two factors."""
    O, I = 160, 256
    w, D, s = packed(O, I, 128, True, True, 45, scale=2.0 ** -12)
    dy = (rand(M, O, 46).float() * 2.0 ** 110).to(torch.bfloat16)
    ref, tol = dx_ref(dy.to(F8), torch.zeros_like(dy, dtype=F8), D, s, O)
    assert ref.abs().max() < 2.0 ** 126
    dx = awq.awq_linear_w4a16_grad(dy, *w)
    within(dx, ref, tol, "dx")
    normwise(dx, ref, BF16_NORM, "dx")
    F = 72
    w, D = signed_gates(F, I, 2.0 ** -12, M)
    x = (rand(M, I, 47).float().abs() * 2.0 ** 112).to(torch.bfloat16)
    dh = (rand(M, F, 48).float() * 2.0 ** -100).to(torch.bfloat16)
    gu = x.to(F8) @ D.T
    g, u, d = gu[:, :F], gu[:, F:], dh.to(F8)
    assert (g.abs() > 2.0 ** 100).all() and gu.abs().max() < 2.0 ** 126
    on = (g > 0).to(F8)
    dx = awq.awq_gated_w4a16_grad(dh, x, *w)
    normwise(dx, torch.cat((d * u * on, d * g * on), 1) @ D, BF16_NORM, "gated dx")
    h = awq.awq_gated_w4a16(x, *w)
    assert (h[g < 0] == 0).all()


@pytest.mark.parametrize("M", PATHS)
@pytest.mark.parametrize("wscale,xscale,dscale", [(2.0 ** -12, 2.0 ** -40, 2.0 ** -60), (8.0, 2.0 ** 20, 2.0 ** 30),
                                                  (0.01, 2.0 ** -100, 2.0 ** 60), (2.0 ** -12, 1.0, 2.0 ** -100)])
def test_gated_grad_of_extreme_magnitudes(awq, M, wscale, xscale, dscale):  # noqa: F811
    F, I = 160, 256
    w, D, s = packed(2 * F, I, 128, True, True, 49, scale=wscale)
    x = (rand(M, I, 50).float() * xscale).to(torch.bfloat16)
    dh = (rand(M, F, 51).float() * dscale).to(torch.bfloat16)
    _, _, (a, da, g, u, _, _, eg) = gated_ref(x, D, s, "silu")
    d = dh.to(F8)
    ref = (torch.cat((d * u * da, d * a), 1) @ D) / s
    assert 2.0 ** -120 < float(ref.abs().amax()) < 2.0 ** 120
    # g is off by at most eg and act' is between -0.1 and 1.1 with |act''| <= 1: act' is off by min(eg, 1.2), and only
    # where |g| < eg + 40 (beyond, exp(-40) of a step).  Of large gates that is the whole step of the few near zero.
    unsure = torch.where(g.abs() < eg + 40, eg.clamp(max=1.2), 0.0)
    step = ((d * u).abs() * unsure) @ D[:F].abs() / s
    normwise(awq.awq_gated_w4a16_grad(dh, x, *w), ref, BF16_NORM + float(step.norm() / ref.norm()), "dx")


@pytest.mark.parametrize("M", PATHS)
def test_gated_grad_beside_an_outlying_scale(awq, M):  # noqa: F811
    """One group scale 2^12 above the others sets the exponents of the layer and of the token's gradients.  Its
    row has no gradient here, so dx is made of the others alone, 2^12 further down in fp16's range."""
    F, I = 160, 256
    w, D, s = packed(2 * F, I, 128, True, True, 52)
    w[1][7, 1] *= 2.0 ** 12
    D[7, 128:] *= 2.0 ** 12
    x, dh = rand(M, I, 53), rand(M, F, 54, 1e-3)
    dh[:, 7] = 0
    _, _, (a, da, _, u, _, _, _) = gated_ref(x, D, s, "silu")
    d = dh.to(F8)
    normwise(awq.awq_gated_w4a16_grad(dh, x, *w), (torch.cat((d * u * da, d * a), 1) @ D) / s, BF16_NORM, "dx")


@pytest.mark.parametrize("M,V,I", [(129, 20001, 256), (700, 33000, 512), (2048, 40000, 128), (5000, 9001, 64)])
def test_head_gradient_of_single_labels(awq, M, V, I):  # noqa: F811
    """A row of dW that one token labels is that token's x times (p - 1) dloss, and little else: with the 16-bit rounding
    of that factor beside its own it is off by sqrt(2) x 1.7e-3 in the root mean square, with the factor exact by
    1.7e-3 (test_gpu_train_paths).  Half of the tokens are alone with their label here, the other half share 7 labels."""
    x, W, labels = ce_case(M, V, I, M + I)
    order = torch.from_numpy(np.random.default_rng([20261209, 55, M]).permutation(V)[:M]).cuda()
    labels[:] = order
    labels[1::2] = torch.arange(M // 2, device="cuda") % 7
    single = order[::2][order[::2] >= 7]
    labels[0] = -100
    single = single[single != order[0]]
    _, lse = awq.awq_cross_entropy(x, W, labels)
    dloss = torch.from_numpy((np.random.default_rng([20261209, 56, M]).random(M) + 0.5).astype(np.float32)).cuda()
    dx, dW = awq.awq_cross_entropy_grad(x, W, labels, lse, dloss)
    x8 = x.to(F8)
    d = torch.exp(x8 @ W.to(F8).T - lse.to(F8)[:, None])
    scored = labels >= 0
    d[scored, labels[scored]] -= 1.0
    d *= torch.where(scored, dloss.to(F8), 0.0)[:, None]
    dW_r = d.T @ x8
    normwise(dW[single], dW_r[single], 2e-3, "rows of one token")
    normwise(dW, dW_r, BF16_NORM, "dW")
    normwise(dx, d @ W.to(F8), BF16_NORM, "dx")


@pytest.mark.parametrize("M", [5, 100, 300])
def test_infinite_gradients_stay_infinite(awq, M):  # noqa: F811
    """dloss of one token infinite: the row of its label is -inf as the formula's is, not NaN from the remainder of a
    rounding, and no other token has a part in it."""
    x, W, labels = ce_case(M, 500, 64, M)
    labels[:] = torch.arange(M, device="cuda")
    x[2], W[2] = 0.125, 0.125                        # a logit of 1
    W[3:] = 0.0
    W[:2] = 0.0
    _, lse = awq.awq_cross_entropy(x, W, labels)
    dloss = torch.zeros(M, device="cuda")
    dloss[2] = float("inf")
    dx, dW = awq.awq_cross_entropy_grad(x, W, labels, lse, dloss)
    assert (dW[2].float() == float("-inf")).all()
    keep = torch.arange(M, device="cuda") != 2
    assert (dx[keep] == 0).all()
