"""Host-side refusals of the gated, gradient and cross-entropy calls: the C entry points return the
documented status before any CUDA work, and the binding refuses operands that do not fit the packed
layout before a pointer reaches the library (no GPU needed)."""
import ctypes

import pytest
import torch

awq = pytest.importorskip("weight_only_quantization_awq_b200")
lib = awq.lib

ARG, ALIGN, UNSUP = 1, 2, 3
FAKE = 0x10000          # a 16-byte aligned address that is never dereferenced
NULL = None

GATED = [FAKE, 4, 512, 688, FAKE, FAKE, FAKE, FAKE, 128, 0, FAKE, NULL]
GATED_GRAD = [FAKE] + GATED
LINEAR_GRAD = [FAKE, 4, 512, 688, FAKE, FAKE, NULL, FAKE, 128, FAKE, NULL]
CE = [FAKE, 4, 512, FAKE, 1000, FAKE, FAKE, FAKE, NULL]
CE_GRAD = [FAKE, 4, 512, FAKE, 1000, FAKE, FAKE, FAKE, FAKE, FAKE, NULL]


def call(f, base, kw):
    a = list(base)
    for k, v in kw.items():
        a[k] = v
    return f(*a)


@pytest.mark.parametrize("kw,status", [
    ({0: NULL}, ARG), ({4: NULL}, ARG), ({5: NULL}, ARG), ({10: NULL}, ARG), ({1: 0}, ARG), ({2: 0}, ARG),
    ({3: 0}, ARG), ({3: -1}, ARG), ({3: 1 << 40}, ARG), ({9: 3}, ARG), ({9: -1}, ARG), ({8: 96}, UNSUP),
    ({2: 520}, UNSUP), ({2: 576}, UNSUP), ({2: 49152 + 128}, UNSUP), ({1: (1 << 20) + 1}, UNSUP),
    ({0: FAKE + 2}, ALIGN), ({4: FAKE + 4}, ALIGN), ({5: FAKE + 1}, ALIGN), ({6: FAKE + 2}, ALIGN),
    ({7: FAKE + 2}, ALIGN), ({10: FAKE + 8}, ALIGN)])
def test_gated_rejects_on_host(kw, status):
    assert call(lib.awq_gated_w4a16, GATED, kw) == status
    assert lib.awq_last_error().decode() != ""
    assert call(lib.awq_gated_w4a16_grad, GATED_GRAD, {k + 1: v for k, v in kw.items()}) == status
    assert call(lib.awq_gated_w4a16_grad, GATED_GRAD, {0: NULL}) == ARG
    assert call(lib.awq_gated_w4a16_grad, GATED_GRAD, {0: FAKE + 2}) == ALIGN


@pytest.mark.parametrize("kw,status", [
    ({0: NULL}, ARG), ({4: NULL}, ARG), ({9: NULL}, ARG), ({1: 0}, ARG), ({3: 0}, ARG), ({8: 16}, UNSUP),
    ({2: 100}, UNSUP), ({2: 576}, UNSUP), ({3: (1 << 24) + 1}, UNSUP), ({0: FAKE + 2}, ALIGN),
    ({9: FAKE + 8}, ALIGN), ({7: FAKE + 8}, ALIGN)])
def test_linear_grad_rejects_on_host(kw, status):
    assert call(lib.awq_linear_w4a16_grad, LINEAR_GRAD, kw) == status
    assert lib.awq_last_error().decode() != ""


@pytest.mark.parametrize("kw,status", [
    ({0: NULL}, ARG), ({3: NULL}, ARG), ({5: NULL}, ARG), ({6: NULL}, ARG), ({7: NULL}, ARG), ({1: 0}, ARG),
    ({4: 0}, ARG), ({2: 100}, UNSUP), ({4: (1 << 24) + 1}, UNSUP), ({1: (1 << 20) + 1}, UNSUP),
    ({0: FAKE + 2}, ALIGN), ({3: FAKE + 8}, ALIGN), ({5: FAKE + 4}, ALIGN), ({6: FAKE + 2}, ALIGN)])
def test_cross_entropy_rejects_on_host(kw, status):
    assert call(lib.awq_cross_entropy, CE, kw) == status
    assert lib.awq_last_error().decode() != ""
    assert call(lib.awq_cross_entropy_grad, CE_GRAD, kw) == status


def test_cross_entropy_grad_rejects_on_host():
    assert call(lib.awq_cross_entropy_grad, CE_GRAD, {8: NULL}) == ARG
    assert call(lib.awq_cross_entropy_grad, CE_GRAD, {8: FAKE + 8}) == ALIGN
    assert call(lib.awq_cross_entropy_grad, CE_GRAD, {9: FAKE + 8}) == ALIGN


def cpu_layer(out=64, inp=256, gs=128):
    return [torch.zeros(out, inp // 8, dtype=torch.int32), torch.zeros(out, inp // gs, dtype=torch.float16), None,
            torch.ones(inp, dtype=torch.float16)]


def bf(*shape):
    return torch.zeros(*shape, dtype=torch.bfloat16)


@pytest.mark.parametrize("bad,match", [
    (dict(w0=torch.zeros(63, 32, dtype=torch.int32), w1=torch.zeros(63, 2, dtype=torch.float16)), "even"),
    (dict(x=bf(3, 255)), "multiple"), (dict(x=torch.zeros(3, 256)), "bfloat16"),
    (dict(w1=torch.zeros(64, 1, dtype=torch.float16)), "scales"), (dict(w3=torch.ones(128, dtype=torch.float16)), "s16"),
    (dict(), "CUDA")])
def test_binding_refuses_gated(bad, match):
    w = cpu_layer()
    x = bad.get("x", bf(3, 256))
    for k in range(4):
        w[k] = bad.get(f"w{k}", w[k])
    with pytest.raises(ValueError, match=match):
        awq.awq_gated_w4a16(x, *w)
    with pytest.raises(ValueError, match=match):
        awq.awq_gated_w4a16_grad(bf(3, w[0].shape[0] // 2), x, *w)


def test_binding_refuses_linear_grad_and_act():
    w = cpu_layer()
    with pytest.raises(ValueError, match="CUDA"):
        awq.awq_linear_w4a16_grad(bf(3, 64), *w)
    with pytest.raises(ValueError, match="multiple"):
        awq.awq_linear_w4a16_grad(bf(3, 64), *w, group_size=96)
    assert awq._act_code("silu") == 0 and awq._act_code("gelu_tanh") == 2
    with pytest.raises(ValueError, match="act"):
        awq._act_code("relu")


@pytest.mark.parametrize("x,W,labels,match", [
    (torch.zeros(3, 64), bf(10, 64), torch.zeros(3, dtype=torch.int64), "bfloat16"),
    (bf(3, 64), bf(10, 128), torch.zeros(3, dtype=torch.int64), "width"),
    (bf(3, 64), bf(10, 64), torch.zeros(3, dtype=torch.int32), "int64"),
    (bf(3, 64), bf(10, 64), torch.zeros(4, dtype=torch.int64), "labels"),
    (bf(3, 64), bf(10, 64), torch.zeros(3, dtype=torch.int64), "CUDA")])
def test_binding_refuses_cross_entropy(x, W, labels, match):
    with pytest.raises(ValueError, match=match):
        awq.awq_cross_entropy(x, W, labels)
    f = torch.zeros(3)
    with pytest.raises(ValueError, match=match):
        awq.awq_cross_entropy_grad(x, W, labels, f, f)


def test_results_must_not_overlap_inputs():
    buf = bf(8, 64)
    with pytest.raises(ValueError, match="overlaps"):
        awq._apart(buf[2:4], "out", buf[3:5])
    awq._apart(buf[2:4], "out", buf[4:5], buf[:2], None)
