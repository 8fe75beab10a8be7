"""What the training and scoring operators on packed weights are measured on.

The operators:
  gated        h = act(g) * u with (g | u) = (x / s) dequant(W)^T, W the joint gate and up matrix
               [2 F, in] in packed 4-bit storage;
  gated_grad   the gradient of h with respect to x, g and u computed again from x;
  linear_grad  the gradient of a packed linear with respect to its input, (dy dequant(W)) / s;
  ce           softmax cross entropy of x W^T (a dense 16-bit output head) per token, with the log
               of each row's sum of exponentials;
  ce_grad      its gradient with respect to x and to W.

A case is measured as listed() gives it, draw() gives more of the same ranges.  Sizes are those of
the benchmark's block (in 4096, F 11008), of its up_proj workload (13824 x 5120), of the smallest
workload (512), and odd ones between.
"""
import math
import random

import torch

own = False

ACTS = ("silu", "gelu", "gelu_tanh")


def listed():
    return [
        # one sequence being decoded: a single token through the gate and up projections of a 7B block
        {"name": "gated_decode_m1", "op": "gated", "M": 1, "in": 4096, "F": 11008, "gs": 128, "zeros": False,
         "s16": True, "act": "silu"},
        # a small serving batch, zero points, the 13B block's widths
        {"name": "gated_decode_m8", "op": "gated", "M": 8, "in": 5120, "F": 13824, "gs": 128, "zeros": True,
         "s16": True, "act": "silu"},
        # a short prompt of odd length, 1/s folded into the norm before, fine groups, another activation
        {"name": "gated_prompt_m77", "op": "gated", "M": 77, "in": 4096, "F": 11008, "gs": 64, "zeros": True,
         "s16": False, "act": "gelu_tanh"},
        # prefill of a long prompt, or a training batch
        {"name": "gated_prefill_m2048", "op": "gated", "M": 2048, "in": 4096, "F": 11008, "gs": 128, "zeros": True,
         "s16": True, "act": "silu"},
        # tuning a small model on short batches: ragged tokens and an odd inner width
        {"name": "gated_grad_m50_small", "op": "gated_grad", "M": 50, "in": 512, "F": 1371, "gs": 32, "zeros": True,
         "s16": True, "act": "gelu"},
        # a training batch through the 7B block's gated projections
        {"name": "gated_grad_m2048", "op": "gated_grad", "M": 2048, "in": 4096, "F": 11008, "gs": 128,
         "zeros": True, "s16": True, "act": "silu"},
        # a few soft-prompt tokens tuned through the wide down projection
        {"name": "linear_grad_m19_down", "op": "linear_grad", "M": 19, "in": 11008, "out": 4096, "gs": 128,
         "zeros": False, "s16": True},
        # a training batch through the 13B up projection
        {"name": "linear_grad_m2048", "op": "linear_grad", "M": 2048, "in": 5120, "out": 13824, "gs": 128,
         "zeros": True, "s16": True},
        # scoring the answer tokens of a few multiple-choice prompts
        {"name": "ce_score_m13", "op": "ce", "M": 13, "in": 4096, "V": 32000, "dw": False},
        # the perplexity of a context window: all its positions but the last
        {"name": "ce_window_m2047", "op": "ce", "M": 2047, "in": 4096, "V": 32000, "dw": False},
        # tuning a small model whose vocabulary has an odd size, head frozen
        {"name": "ce_grad_m129_small", "op": "ce_grad", "M": 129, "in": 512, "V": 9973, "dw": False},
        # a training batch with a trained head
        {"name": "ce_grad_m2048", "op": "ce_grad", "M": 2048, "in": 4096, "V": 32000, "dw": True},
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(("gated", "gated_grad", "linear_grad", "ce", "ce_grad"))
    top = 1.6e12                                       # flops of the largest listed case
    while True:
        M = _log_int(rng, 1, 2048)
        if op in ("ce", "ce_grad"):
            case = {"op": op, "M": M, "in": 64 * _log_int(rng, 4, 80), "V": _log_int(rng, 1000, 50000),
                    "dw": op == "ce_grad" and rng.random() < 0.5}
        else:
            gs = rng.choice((32, 64, 128))
            step = max(64, gs)
            case = {"op": op, "M": M, "in": step * _log_int(rng, 256 // step, 8192 // step), "gs": gs,
                    "zeros": rng.random() < 0.5, "s16": rng.random() < 0.7}
            if op == "linear_grad":
                case["out"] = _log_int(rng, 300, 14000)
            else:
                case["F"] = _log_int(rng, 300, 14000)
                case["act"] = rng.choice(ACTS)
        if work(case)["flops"] <= top:
            return case


def work(case):
    M, I = case["M"], case["in"]
    if case["op"] in ("ce", "ce_grad"):
        V = case["V"]
        by, fl = 2 * M * I + 2 * V * I + 8 * M, 2.0 * M * V * I
        if case["op"] == "ce":
            return {"bytes": by + 8 * M, "flops": fl}
        return {"bytes": by + 8 * M + 2 * M * I + (2 * V * I if case["dw"] else 0), "flops": fl * (3 if case["dw"] else 2)}
    O = case["out"] if case["op"] == "linear_grad" else 2 * case["F"]
    nG = I // case["gs"]
    by = O * I / 2 + 2 * O * nG + (4 * O * ((nG + 7) // 8) if case["zeros"] else 0) + (2 * I if case["s16"] else 0)
    fl = 2.0 * M * O * I
    if case["op"] == "gated":
        return {"bytes": by + 2 * M * I + M * O, "flops": fl}
    if case["op"] == "gated_grad":
        return {"bytes": by + 4 * M * I + M * O, "flops": 2 * fl}
    return {"bytes": by + 2 * M * O + 2 * M * I, "flops": fl}


# ------------------------------------------------------------------ inputs
def _packed(case, O, gen):
    """A packed layer as the packing calls leave it: group-wise 4-bit codes of W * s with s from the
    activations' statistic at alpha = 0.5, fp16 scales, zero points, fp16 s."""
    I, gs = case["in"], case["gs"]
    nG = I // gs
    dev = "cuda"
    chan = torch.ones(I, device=dev)
    hot = torch.randperm(I, generator=gen, device=dev)[: max(1, I // 100)]
    chan[hot] = torch.exp(torch.empty(hot.numel(), device=dev).uniform_(math.log(10.0), math.log(100.0), generator=gen))
    s = torch.sqrt(chan / chan.max()) if case["s16"] else torch.ones(I, device=dev)
    W = torch.randn(O, I, generator=gen, device=dev)
    W *= 0.02 * torch.exp(0.3 * torch.randn(O, 1, generator=gen, device=dev)) * s
    Wg = W.view(O, nG, gs)
    if case["zeros"]:
        lo, hi = Wg.amin(2, keepdim=True), Wg.amax(2, keepdim=True)
        delta = (hi - lo) / 15
        z = torch.clamp(torch.round(-lo / delta), 0, 15)
        q = torch.clamp(torch.round(Wg / delta) + z, 0, 15)
        zi = torch.zeros(O, (nG + 7) // 8 * 8, dtype=torch.int32, device=dev)
        zi[:, :nG] = z.squeeze(2).to(torch.int32)
        zeros = _nibbles(zi)
    else:
        delta = Wg.abs().amax(2, keepdim=True) / 7
        q = torch.clamp(torch.round(Wg / delta), -8, 7) + 8
        zeros = None
    del W, Wg
    return {"qweight": _nibbles(q.to(torch.int32).view(O, I)), "scales": delta.squeeze(2).to(torch.float16),
            "zeros": zeros, "s16": s.to(torch.float16) if case["s16"] else None, "group_size": gs}, chan


def _nibbles(c):
    """[rows, n] codes of 4 bits as [rows, n / 8] int32 words, column 8 w + k in bits 4 k .. 4 k + 3."""
    words = c[:, 0::8].clone()
    for k in range(1, 8):
        words |= c[:, k::8] << (4 * k)
    return words.contiguous()


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    M, I, dev = case["M"], case["in"], "cuda"
    if case["op"] in ("ce", "ce_grad"):
        V = case["V"]
        W = (0.02 * torch.randn(V, I, generator=gen, device=dev)).to(torch.bfloat16)
        labels = torch.randint(0, V, (M,), generator=gen, device=dev)
        x = torch.randn(M, I, generator=gen, device=dev)
        # a trained model's rows lean towards the label, some strongly
        pull = 8.0 * torch.rand(M, 1, generator=gen, device=dev)
        picked = W[labels].float()
        x = (x + pull * picked / picked.norm(dim=1, keepdim=True)).to(torch.bfloat16)
        # every tenth position is not scored (prompt or padding)
        labels = torch.where(torch.rand(M, generator=gen, device=dev) < 0.1, -100, labels)
        state = {"op": case["op"], "x": x, "W": W, "labels": labels}
        if case["op"] == "ce_grad":
            state["lse"] = torch.logsumexp(x.float() @ W.float().t(), dim=1)
            n = max(1, int((labels >= 0).sum()))
            state["dloss"] = (0.5 + torch.rand(M, generator=gen, device=dev)) / n
            state["dw"] = case["dw"]
        return state
    O = case["out"] if case["op"] == "linear_grad" else 2 * case["F"]
    packed, chan = _packed(case, O, gen)
    state = {"op": case["op"], "packed": packed, "act": case.get("act")}
    if case["op"] != "linear_grad":
        x = torch.randn(M, I, generator=gen, device=dev)
        if case["s16"]:
            x = x * chan
        state["x"] = x.to(torch.bfloat16)
    if case["op"] != "gated":
        width = O if case["op"] == "linear_grad" else case["F"]
        d = 1e-3 * torch.randn(M, width, generator=gen, device=dev)
        if M > 1:                                     # rows of padding carry no gradient
            d[torch.rand(M, generator=gen, device=dev) < 0.05] = 0.0
        state["d"] = d.to(torch.bfloat16)
    return state


# ------------------------------------------------------------------ the plain forms
def _dense(p):
    """The weights that the packed storage stands for, (code - z) * scale, in 32 bits."""
    O = p["qweight"].shape[0]
    at = torch.arange(0, 32, 4, dtype=torch.int32, device=p["qweight"].device)
    codes = ((p["qweight"].unsqueeze(2) >> at) & 15).view(O, -1, p["group_size"]).float()
    scales = p["scales"].float()
    if p["zeros"] is None:
        codes -= 8.0
    else:
        codes -= ((p["zeros"].unsqueeze(2) >> at) & 15).view(O, -1)[:, : scales.shape[1]].float().unsqueeze(2)
    return (codes * scales.unsqueeze(2)).view(O, -1)


def _act(g, act):
    """act(g) and its derivative."""
    if act == "silu":
        sig = 1.0 / (1.0 + torch.exp(-g))
        return g * sig, sig * (1.0 + g * (1.0 - sig))
    if act == "gelu":
        cdf = 0.5 * (1.0 + torch.erf(g * math.sqrt(0.5)))
        return g * cdf, cdf + g * torch.exp(-0.5 * g * g) / math.sqrt(2.0 * math.pi)
    c = math.sqrt(2.0 / math.pi)
    t = torch.tanh(c * (g + 0.044715 * g * g * g))
    return 0.5 * g * (1.0 + t), 0.5 * (1.0 + t) + 0.5 * g * (1.0 - t * t) * c * (1.0 + 3 * 0.044715 * g * g)


def _plain(st):
    if st["op"] in ("ce", "ce_grad"):
        x, W, labels = st["x"].float(), st["W"].float(), st["labels"]
        logits = x @ W.t()
        scored = labels >= 0
        at = torch.where(scored, labels, 0).unsqueeze(1)
        if st["op"] == "ce":
            top = logits.amax(1, keepdim=True)
            lse = (top + torch.log(torch.exp(logits - top).sum(1, keepdim=True))).squeeze(1)
            return {"loss": torch.where(scored, lse - logits.gather(1, at).squeeze(1), 0.0), "lse": lse}
        d = torch.exp(logits - st["lse"].unsqueeze(1))
        d.scatter_add_(1, at, torch.full_like(at, -1, dtype=torch.float32))
        d *= torch.where(scored, st["dloss"], 0.0).unsqueeze(1)
        out = {"dx": (d @ W).to(torch.bfloat16)}
        if st["dw"]:
            out["dW"] = (d.t() @ x).to(torch.bfloat16)
        return out
    p = st["packed"]
    Wd = _dense(p)
    s = 1.0 if p["s16"] is None else p["s16"].float()
    if st["op"] == "linear_grad":
        return {"dx": ((st["d"].float() @ Wd) / s).to(torch.bfloat16)}
    gu = (st["x"].float() / s) @ Wd.t()
    F = gu.shape[1] // 2
    a, da = _act(gu[:, :F], st["act"])
    if st["op"] == "gated":
        return {"h": (a * gu[:, F:]).to(torch.bfloat16)}
    d = st["d"].float()
    dgu = torch.cat((d * gu[:, F:] * da, d * a), 1)
    return {"dx": ((dgu @ Wd) / s).to(torch.bfloat16)}


def run(st):
    if not own:
        return _plain(st)
    import weight_only_quantization_awq_b200 as awq
    if st["op"] == "ce":
        loss, lse = awq.awq_cross_entropy(st["x"], st["W"], st["labels"])
        return {"loss": loss, "lse": lse}
    if st["op"] == "ce_grad":
        dx, dW = awq.awq_cross_entropy_grad(st["x"], st["W"], st["labels"], st["lse"], st["dloss"], want_dw=st["dw"])
        return {"dx": dx, "dW": dW} if st["dw"] else {"dx": dx}
    p = st["packed"]
    w = (p["qweight"], p["scales"], p["zeros"], p["s16"])
    if st["op"] == "gated":
        return {"h": awq.awq_gated_w4a16(st["x"], *w, group_size=p["group_size"], act=st["act"])}
    if st["op"] == "gated_grad":
        return {"dx": awq.awq_gated_w4a16_grad(st["d"], st["x"], *w, group_size=p["group_size"], act=st["act"])}
    return {"dx": awq.awq_linear_w4a16_grad(st["d"], *w, group_size=p["group_size"])}


# ------------------------------------------------------------------ 64 bits
def exact(case, seed):
    """The definitions, in 64 bits, column by column of the storage."""
    st = prepare(case, seed)
    f8 = torch.float64
    if st["op"] in ("ce", "ce_grad"):
        x, W, labels = st["x"].to(f8), st["W"].to(f8), st["labels"]
        M = x.shape[0]
        logits = torch.einsum("mi,vi->mv", x, W)
        rows = torch.arange(M, device=x.device)
        scored = (labels >= 0).to(f8)
        safe = labels.clamp(min=0)
        if st["op"] == "ce":
            lse = torch.logsumexp(logits, 1)
            return {"loss": (lse - logits[rows, safe]) * scored, "lse": lse}
        prob = torch.softmax(logits, 1)               # lse is the same logits' log-sum
        prob[rows, safe] -= 1.0
        prob *= (scored * st["dloss"].to(f8))[:, None]
        out = {"dx": torch.einsum("mv,vi->mi", prob, W)}
        if st["dw"]:
            out["dW"] = torch.einsum("mv,mi->vi", prob, x)
        return out
    p = st["packed"]
    O, words = p["qweight"].shape
    I, gs = 8 * words, p["group_size"]
    Wd = torch.empty(O, I, dtype=f8, device="cuda")
    group = torch.arange(I, device="cuda") // gs
    for k in range(8):                                # nibble k of every word: columns k, k + 8, ...
        g = group[k::8]
        code = torch.bitwise_and(torch.bitwise_right_shift(p["qweight"], 4 * k), 15).to(f8)
        if p["zeros"] is None:
            z = 8.0
        else:
            z = torch.bitwise_and(torch.bitwise_right_shift(p["zeros"][:, g // 8], (4 * (g % 8)).to(torch.int32)), 15).to(f8)
        Wd[:, k::8] = (code - z) * p["scales"][:, g].to(f8)
    s = torch.ones(I, dtype=f8, device="cuda") if p["s16"] is None else p["s16"].to(f8)
    if st["op"] == "linear_grad":
        return {"dx": torch.einsum("mo,oi->mi", st["d"].to(f8), Wd) / s}
    F = O // 2
    xs = st["x"].to(f8) / s
    g, u = torch.einsum("mi,fi->mf", xs, Wd[:F]), torch.einsum("mi,fi->mf", xs, Wd[F:])
    g.requires_grad_(True)
    a = {"silu": torch.nn.functional.silu, "gelu": torch.nn.functional.gelu,
         "gelu_tanh": lambda t: torch.nn.functional.gelu(t, approximate="tanh")}[st["act"]](g)
    if st["op"] == "gated":
        return {"h": (a * u).detach()}
    d = st["d"].to(f8)
    (dg,) = torch.autograd.grad((a * u * d).sum(), g)
    du = (d * a).detach()
    return {"dx": (torch.einsum("mf,fi->mi", dg, Wd[:F]) + torch.einsum("mf,fi->mi", du, Wd[F:])) / s}
