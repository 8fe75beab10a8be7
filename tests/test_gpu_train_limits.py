"""GPU checks of the gated, gradient and cross-entropy calls at the ends of the sizes they admit: the widest
inputs, many tokens, large vocabularies, matrices of more than 2^32 elements; and graphs that run at once.
Formulas in 64 bits and tolerances as in test_gpu_train; of the largest matrices, a sample of the results."""
import pytest
import torch

import test_gpu_train as base
from test_gpu_train import F8, awq, ce_case, every_call, gated_ref, packed, rand, within  # noqa: F401
from test_gpu_train_paths import BF16_NORM, normwise

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("M", [1, 2, 3, 16, 20, 150, 300])
def test_widest_input(awq, M):  # noqa: F811
    base.test_gated(awq, M, 49152, 37, 128, True, True, "silu")
    base.test_gated_grad(awq, M, 49152, 37, 128, False, True, "silu")
    base.test_linear_grad(awq, M, 75, 49152, 64, True, True)


@pytest.mark.parametrize("M", [3, 100, 200])
def test_widest_head(awq, M):  # noqa: F811
    base.test_cross_entropy(awq, M, 701, 49152)
    base.test_cross_entropy_grad(awq, M, 701, 49152, True)


def test_many_tokens(awq):  # noqa: F811
    M = 1 << 20
    w, D, s = packed(2 * 24, 64, 64, True, True, 5)
    x, dh = rand(M, 64, 6), rand(M, 24, 7, 1e-3)
    h = awq.awq_gated_w4a16(x, *w, group_size=64)
    dx = awq.awq_gated_w4a16_grad(dh, x, *w, group_size=64)
    wl, Dl, sl = packed(40, 64, 64, False, True, 8)
    dy = rand(M, 40, 9)
    dl = awq.awq_linear_w4a16_grad(dy, *wl, group_size=64)
    for k in range(0, M, 1 << 17):
        r = slice(k, k + (1 << 17))
        ref, tol, (a, da, _, u, _, _, _) = gated_ref(x[r], D, s, "silu")
        within(h[r], ref, tol, "h")
        d = dh[r].to(F8)
        normwise(dx[r], (torch.cat((d * u * da, d * a), 1) @ D) / s, BF16_NORM, "dx")
        normwise(dl[r], (dy[r].to(F8) @ Dl) / sl, BF16_NORM, "linear dx")
    xc, W, labels = ce_case(M, 70, 64, 10)
    loss, lse = awq.awq_cross_entropy(xc, W, labels)
    dloss = torch.full((M,), 1.0, device="cuda")
    dxc, dW = awq.awq_cross_entropy_grad(xc, W, labels, lse, dloss)
    l = xc.to(F8) @ W.to(F8).T
    ref = torch.logsumexp(l, 1)
    scored = labels >= 0
    at = labels.clamp(min=0)
    assert float((lse.to(F8) - ref).norm() / ref.norm()) < 1e-6
    want = torch.where(scored, ref - l[torch.arange(M, device="cuda"), at], 0.0)
    assert float((loss.to(F8) - want).norm() / want.norm()) < 1e-6
    p = torch.exp(l - ref[:, None])
    p[torch.arange(M, device="cuda"), at] -= 1.0
    p[~scored] = 0.0
    normwise(dxc, p @ W.to(F8), BF16_NORM, "dx")
    normwise(dW, p.T @ xc.to(F8), BF16_NORM * 2 ** 0.5, "dW")


@pytest.mark.parametrize("M", [3, 150])
def test_largest_vocabulary(awq, M):  # noqa: F811
    """2^24 entries: the gradients of 150 tokens take 75 pieces."""
    V, I = 1 << 24, 64
    g = torch.Generator(device="cuda").manual_seed(11)
    W = (torch.randn(V, I, device="cuda", generator=g) * 0.2).to(torch.bfloat16)
    x = torch.randn(M, I, device="cuda", generator=g).to(torch.bfloat16)
    labels = torch.randint(0, V, (M,), device="cuda", generator=g)
    labels[0], labels[1], labels[2] = V - 1, V, 0
    loss, lse = awq.awq_cross_entropy(x, W, labels)
    dloss = torch.rand(M, device="cuda", generator=g)
    dx, dW = awq.awq_cross_entropy_grad(x, W, labels, lse, dloss)
    x8, parts = x.to(F8), []
    for k in range(0, V, 1 << 20):
        parts.append(torch.logsumexp(x8 @ W[k:k + (1 << 20)].to(F8).T, 1))
    ref = torch.logsumexp(torch.stack(parts), 0)
    scored = labels < V
    t = (x8 * W[labels.clamp(max=V - 1)].to(F8)).sum(1)
    assert float((lse.to(F8) - ref).norm() / ref.norm()) < 1e-6
    within(loss, torch.where(scored, ref - t, 0.0), 2.0 ** -19 * ref, "loss")
    wgt = torch.where(scored, dloss.to(F8), 0.0)[:, None]
    dxr = torch.zeros(M, I, dtype=F8, device="cuda")
    num = den = 0.0
    for k in range(0, V, 1 << 20):
        Wk = W[k:k + (1 << 20)].to(F8)
        d = torch.exp(x8 @ Wk.T - ref[:, None])
        here = scored & (labels >= k) & (labels < k + (1 << 20))
        d[here, labels[here] - k] -= 1.0
        d *= wgt
        dxr += d @ Wk
        dWk = d.T @ x8
        num += float((dW[k:k + (1 << 20)].to(F8) - dWk).square().sum())
        den += float(dWk.square().sum())
    normwise(dx, dxr, BF16_NORM, "dx")
    assert (num / den) ** 0.5 <= BF16_NORM * 2 ** 0.5


def test_matrices_beyond_32_bits(awq):  # noqa: F811
    """2 x 524293 rows of 4096: 2^32 codes and more, 8.6 GB of dequantised weights."""
    F, I, gs = (1 << 19) + 5, 4096, 128
    g = torch.Generator(device="cuda").manual_seed(12)
    q = torch.randint(-2 ** 31, 2 ** 31, (2 * F, I // 8), device="cuda", generator=g, dtype=torch.int64).to(torch.int32)
    sc = (torch.rand(2 * F, I // gs, device="cuda", generator=g) * 0.01 + 0.002).half()
    zeros = torch.randint(-2 ** 31, 2 ** 31, (2 * F, I // gs // 8), device="cuda", generator=g, dtype=torch.int64).to(torch.int32)
    s = (torch.rand(I, device="cuda", generator=g) * 0.5 + 0.5).half()

    def rows(idx):                                    # 64-bit weights of some rows
        sh = 4 * torch.arange(8, device="cuda")
        code = (q[idx].to(torch.int64)[:, :, None] >> sh & 15).reshape(len(idx), I)
        z = (zeros[idx].to(torch.int64)[:, :, None] >> sh & 15).reshape(len(idx), I // gs)
        return (code - z.repeat_interleave(gs, 1)) * sc[idx].to(F8).repeat_interleave(gs, 1)
    f = torch.cat((torch.arange(40, device="cuda"), torch.randint(0, F, (500,), device="cuda", generator=g),
                   torch.arange(F - 40, F, device="cuda")))
    D = torch.cat((rows(f), rows(F + f)))
    for M in (1, 9, 20):
        x = rand(M, I, 13 + M)
        h = awq.awq_gated_w4a16(x, q, sc, zeros, s, group_size=gs)
        ref, tol, _ = gated_ref(x, D, s.to(F8), "silu")
        within(h[:, f], ref, tol, "h")
        normwise(h[:, f], ref, BF16_NORM, "h")
    M = 2
    dy, dh, x = rand(M, 2 * F, 14), rand(M, F, 15, 1e-3), rand(M, I, 16)
    dl = awq.awq_linear_w4a16_grad(dy, q, sc, zeros, s, group_size=gs)
    dx = awq.awq_gated_w4a16_grad(dh, x, q, sc, zeros, s, group_size=gs)
    want_l, want = torch.zeros(M, I, dtype=F8, device="cuda"), torch.zeros(M, I, dtype=F8, device="cuda")
    xs = x.to(F8) / s.to(F8)
    for k in range(0, F, 1 << 16):
        idx = torch.arange(k, min(k + (1 << 16), F), device="cuda")
        G, U = rows(idx), rows(F + idx)
        want_l += dy[:, idx].to(F8) @ G + dy[:, F + idx].to(F8) @ U
        a, da = base.act64(xs @ G.T, "silu")
        d = dh[:, idx].to(F8)
        want += (d * (xs @ U.T) * da) @ G + (d * a) @ U
    normwise(dl, want_l / s.to(F8), BF16_NORM, "linear dx")
    normwise(dx, want / s.to(F8), BF16_NORM, "dx")


def test_head_beyond_32_bits(awq):  # noqa: F811
    """1.1 million entries of 4096: 4.5e9 elements of W and of dW."""
    V, I = 1100003, 4096
    g = torch.Generator(device="cuda").manual_seed(17)
    W = torch.empty(V, I, dtype=torch.bfloat16, device="cuda")
    for k in range(0, V, 1 << 17):
        W[k:k + (1 << 17)] = torch.randn(min(1 << 17, V - k), I, device="cuda", generator=g) * 0.03
    for M in (5, 130):
        x = torch.randn(M, I, device="cuda", generator=g).to(torch.bfloat16)
        labels = torch.randint(V - 1000, V, (M,), device="cuda", generator=g)
        labels[0], labels[1] = V - 1, -1
        loss, lse = awq.awq_cross_entropy(x, W, labels)
        dloss = torch.ones(M, device="cuda")
        dx, dW = awq.awq_cross_entropy_grad(x, W, labels, lse, dloss)
        x8 = x.to(F8)
        scored = labels >= 0
        dxr, top = torch.zeros(M, I, dtype=F8, device="cuda"), []
        for k in range(0, V, 1 << 17):
            top.append(torch.logsumexp(x8 @ W[k:k + (1 << 17)].to(F8).T, 1))
        ref = torch.logsumexp(torch.stack(top), 0)
        assert float((lse.to(F8) - ref).norm() / ref.norm()) < 1e-6
        t = (x8 * W[labels.clamp(min=0)].to(F8)).sum(1)
        within(loss, torch.where(scored, ref - t, 0.0), 2.0 ** -19 * ref, "loss")
        for k in range(0, V, 1 << 17):
            Wk = W[k:k + (1 << 17)].to(F8)
            d = torch.exp(x8 @ Wk.T - ref[:, None])
            here = scored & (labels >= k) & (labels < k + (1 << 17))
            d[here, labels[here] - k] -= 1.0
            d[~scored] = 0.0
            dxr += d @ Wk
            if k == 0 or k + (1 << 17) >= V:
                normwise(dW[k:k + (1 << 17)], d.T @ x8, BF16_NORM * 2 ** 0.5, "dW")
        normwise(dx, dxr, BF16_NORM, "dx")
        del dW


@pytest.mark.parametrize("M", [11, 130, 400])
def test_graphs_at_once(awq, M):  # noqa: F811
    """Two graphs of each call, each with its own workspace, replayed on two streams at the same time."""
    calls = (every_call(awq, M, seed=7), every_call(awq, M, seed=90))
    want = [{n: [t.clone() for t in c()] for n, c in cs.items()} for cs in calls]
    torch.cuda.synchronize()
    graphs = []
    for cs in calls:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs = {n: c() for n, c in cs.items()}
        graphs.append((g, outs))
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    for _ in range(10):
        for (g, _), st in zip(graphs, streams):
            with torch.cuda.stream(st):
                g.replay()
    torch.cuda.synchronize()
    for (_, outs), w in zip(graphs, want):
        for n, ts in outs.items():
            for a, b in zip(ts, w[n]):
                assert torch.equal(a, b), n
