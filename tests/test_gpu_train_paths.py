"""GPU checks of the gated, gradient and cross-entropy calls where a CTA has several tiles: ranges that cross
tiles, several passes over a CTA's tiles, several accumulations in turn, several pieces of the vocabulary, and
chains of calls.  Formulas in 64 bits and elementwise tolerances as in test_gpu_train; beside them
norm-wise bounds, which a lost digit in one operand does not pass.

bf16 results: the rounding of the result is at most 2^-8 of a value, 2^-8 / sqrt(3) x 0.72 = 1.7e-3 in the
root mean square over mantissas (0.72: the mean square of 1 / mantissa over [1, 2)), and each operand
rounded to fp16 adds 2^-11 / sqrt(3) x 0.72 = 2e-4 to it, in squares: below 1.8e-3 for up to six operands.
"""
import pytest
import torch

import test_gpu_train as base
from test_gpu_train import F8, awq, ce_case, dx_ref, gated_ref, packed, rand, within  # noqa: F401
from test_train_indexing import SMS, first, gd_plan, skinny_plan

pytestmark = pytest.mark.gpu

BF16_NORM = 2.5e-3


def normwise(got, ref, bound, what):
    ref = ref.to(F8)
    err = float((got.to(F8) - ref).norm() / ref.norm())
    assert err <= bound, (what, err)


def segments(M, tiles, k):
    """Most tiles that a CTA's range touches, and how many ranges cross from one tile into another."""
    _, _, ks, grid, units = skinny_plan(M, tiles, k)
    spans = [(first(units, grid, c + 1) - 1) // ks - first(units, grid, c) // ks + 1 for c in range(grid)]
    return max(spans), sum(s > 1 for s in spans)


DECODE = [  # M, in, F, gs, zeros, s16, act, passes over a CTA's tiles
    (1, 512, 5000, 128, True, True, "silu", 1),
    (8, 512, 5003, 64, False, True, "gelu", 1),
    (9, 2048, 11000, 32, True, True, "silu", 1),
    (16, 1024, 14001, 32, False, False, "gelu_tanh", 1),
    (7, 4096, 9500, 32, True, True, "silu", 2),
    (12, 4096, 9511, 64, True, True, "silu", 2),
]


@pytest.mark.parametrize("M,I,F,gs,zeros,s16,act,passes", DECODE)
def test_decode_of_several_tiles(awq, M, I, F, gs, zeros, s16, act, passes):  # noqa: F811
    tiles = -(-F // 16)
    own = -(-tiles // SMS)
    fit = max(n for n in range(1, 33) if gd_plan(M, I, gs, 1 if M <= 8 else 2, n)[3] <= 224 * 1024)
    assert own >= 2 and fit >= min(own, 4) and -(-own // fit) == passes
    w, D, s = packed(2 * F, I, gs, zeros, s16, M + F)
    x = rand(M, I, M + 1)
    out = torch.full((M, F), float("nan"), dtype=torch.bfloat16, device="cuda")
    awq.awq_gated_w4a16(x, *w, group_size=gs, act=act, out=out)
    ref, tol, _ = gated_ref(x, D, s, act)
    within(out, ref, tol, "h")
    normwise(out, ref, BF16_NORM, "h")


STAGED = [  # M, in, F, gs, zeros, s16, act: products dequantised on the way
    (77, 512, 11008, 64, True, True, "silu"),
    (144, 320, 11001, 64, False, True, "gelu"),
    (20, 640, 19200, 128, True, False, "silu"),
    (64, 128, 20000, 64, True, True, "gelu_tanh"),    # K of one stage: several whole tiles a CTA
    (200, 640, 6400, 64, True, True, "silu"),         # two token tiles
    (280, 1024, 5760, 128, False, True, "gelu_tanh"),
    (100, 4096, 3001, 128, True, True, "silu"),
    (50, 2048, 3001, 32, True, True, "silu"),
]


@pytest.mark.parametrize("M,I,F,gs,zeros,s16,act", STAGED)
def test_gated_of_several_tiles(awq, M, I, F, gs, zeros, s16, act):  # noqa: F811
    if I <= 1024:
        most, cross = segments(M, -(-F // 64), I)
        assert most >= 2 and cross > 50
    w, D, s = packed(2 * F, I, gs, zeros, s16, M + F)
    x = rand(M, I, M + 1)
    out = torch.full((M, F), float("nan"), dtype=torch.bfloat16, device="cuda")
    awq.awq_gated_w4a16(x, *w, group_size=gs, act=act, out=out)
    ref, tol, _ = gated_ref(x, D, s, act)
    within(out, ref, tol, "h")
    normwise(out, ref, BF16_NORM, "h")


@pytest.mark.parametrize("M,I,F,gs,zeros,s16,act", [c for c in STAGED if c[0] <= 144] + [
    (144, 4096, 1003, 128, False, True, "silu"), (33, 11008, 700, 128, True, True, "gelu"),
    (600, 512, 4109, 64, True, True, "silu"), (1500, 256, 2051, 32, False, True, "gelu_tanh")])
def test_gated_grad_of_several_tiles(awq, M, I, F, gs, zeros, s16, act):  # noqa: F811
    w, D, s = packed(2 * F, I, gs, zeros, s16, M + F)
    x, dh = rand(M, I, M + 1), rand(M, F, M + 2, 1e-3)
    out = torch.full((M, I), float("nan"), dtype=torch.bfloat16, device="cuda")
    awq.awq_gated_w4a16_grad(dh, x, *w, group_size=gs, act=act, out=out)
    _, _, (a, da, _, u, _, _, _) = gated_ref(x, D, s, act)
    d = dh.to(F8)
    normwise(out, (torch.cat((d * u * da, d * a), 1) @ D) / s, BF16_NORM, "dx")
    base.test_gated_grad(awq, M, I, F, gs, zeros, s16, act)


@pytest.mark.parametrize("M,O,I,gs,zeros,s16", [
    (200, 11008, 2560, 128, True, True), (250, 1000, 11008, 64, False, True), (130, 2000, 11008, 128, True, True),
    (40, 1111, 25600, 64, True, False), (288, 3300, 5120, 32, True, True), (19, 4096, 11008, 128, False, True),
    (10, 100, 24576, 128, True, True),               # K of one stage
    (1, 5000, 19008, 64, True, True),                # a tile of half its columns
    (700, 1003, 8192, 64, True, True), (1300, 333, 4096, 32, False, True)])
def test_linear_grad_of_several_tiles(awq, M, O, I, gs, zeros, s16):  # noqa: F811
    if M <= 288:
        assert segments(M, -(-I // 128), O)[0] >= 2
    w, D, s = packed(O, I, gs, zeros, s16, M + O)
    dy = rand(M, O, M + 3, 1e-4)
    out = torch.full((M, I), float("nan"), dtype=torch.bfloat16, device="cuda")
    awq.awq_linear_w4a16_grad(dy, *w, group_size=gs, out=out)
    ref, tol = dx_ref(dy.to(F8), torch.zeros_like(dy, dtype=F8), D, s, O)
    within(out, ref, tol, "dx")
    normwise(out, ref, BF16_NORM, "dx")


# several tiles a pair, and accumulations of 1024 columns: 2 (the last of one slab), 3 and 4 to a tile
CE_WIDE = [(13, 40000, 1088), (128, 20001, 2112), (13, 40000, 4096), (64, 20000, 3136), (129, 20001, 1088),
           (300, 20000, 2112), (129, 33000, 4096)]


@pytest.mark.parametrize("M,V,I", CE_WIDE)
def test_cross_entropy_of_several_accumulations(awq, M, V, I):  # noqa: F811
    base.test_cross_entropy(awq, M, V, I)
    x, W, labels = ce_case(M, V, I, M + V)
    loss, _ = awq.awq_cross_entropy(x, W, labels)
    l = x.to(F8) @ W.to(F8).T
    scored = labels >= 0
    want = (torch.logsumexp(l, 1) - l.gather(1, labels.clamp(min=0)[:, None])[:, 0])[scored]
    # A step of the tensor cores drops at most 2^-23 of a partial sum.  Of a logit of 4096 columns in one go that is
    # 256 steps, 1e-6 of the losses and more; in runs of 64 steps a quarter of the steps on a quarter of the
    # sum.  The label's own logit, which weighs most, is rounded to fp32 a few times.
    normwise(loss[scored], want, 1e-6, "loss")


@pytest.mark.parametrize("want_dw", [True, False])
@pytest.mark.parametrize("M,V,I", [(13, 40000, 1088), (64, 20001, 2112), (100, 33000, 1088), (300, 20001, 2112),
                                   (8200, 13000, 64), (20000, 9001, 64)])
def test_cross_entropy_grad_of_several_tiles_and_pieces(awq, M, V, I, want_dw):  # noqa: F811
    vc = max((64 << 20) // (2 * M), 4096)
    assert M < 8000 or -(-V // vc) >= 3               # a first, a middle and a last piece
    base.test_cross_entropy_grad(awq, M, V, I, want_dw)


@pytest.mark.parametrize("M", [1, 2, 4, 5, 8, 16, 20])
def test_gated_then_linear(awq, M):  # noqa: F811
    """A block of every decoded token: the linear starts while the gated product ends and reads its result.  New
    values in the same buffers each time, so that a stale line of the call before would show."""
    w, _, _ = packed(2 * 2816, 1024, 128, True, True, 90)
    wd, _, _ = packed(1024, 2816, 128, False, True, 91)
    xs = [rand(M, 1024, 100 + k) for k in range(4)]
    h = torch.empty(M, 2816, dtype=torch.bfloat16, device="cuda")
    y = torch.empty(M, 1024, dtype=torch.bfloat16, device="cuda")
    ref = []
    for x in xs:
        awq.awq_gated_w4a16(x, *w, out=h)
        torch.cuda.synchronize()
        ref.append((h.clone(), awq.awq_linear_w4a16(h, *wd).clone()))
        torch.cuda.synchronize()
    assert all(torch.isfinite(b.float()).all() for _, b in ref)
    got = []
    for k in range(60):
        awq.awq_gated_w4a16(xs[k % 4], *w, out=h)
        awq.awq_linear_w4a16(h, *wd, out=y)
        got.append((h.clone(), y.clone()))
    # the same without copies in between: nothing but the two kernels on the stream
    outs = [torch.empty_like(y) for _ in range(60)]
    for k in range(60):
        awq.awq_gated_w4a16(xs[k % 4], *w, out=h)
        awq.awq_linear_w4a16(h, *wd, out=outs[k])
    for k in range(60):
        assert torch.equal(got[k][0], ref[k % 4][0]), k
        for t in (got[k][1], outs[k]):
            if M <= 16:
                assert torch.equal(t, ref[k % 4][1]), k
            else:       # from 17 tokens on the linear adds its K splits in any order: one step of bf16 apart
                a, b = t.to(F8), ref[k % 4][1].to(F8)
                assert ((a - b).abs() <= 2.0 ** -7 * b.abs() + 2.0 ** -16 * b.abs().amax()).all(), k
