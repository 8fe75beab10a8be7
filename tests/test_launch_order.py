"""Kernels that start while the kernel before them on the stream still runs (programmatic launches): how
their sources read what that kernel may have written.  No GPU needed.

A load by __ldg, or one through a `const T *__restrict__` pointer, which the compiler may turn into the
same, is for memory that nobody writes while the kernel runs.  Activations, gradients, labels and workspaces
may be results of the kernel before, which is still running when such a kernel starts."""
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))),
                    "weight_only_quantization_awq_b200", "csrc")

# every kernel that waits for its predecessor itself: source, name, what it reads that may be a result
KERNELS = [
    ("k_w4a16_stream.cu", "w4a16_gemv_kernel", ["a.x"]),
    ("k_w4a16_mma.cu", "xs_prep_kernel", ["x"]),
    ("k_w4a16_mma.cu", "w4a16_mma_kernel", ["xsp", "src", "xsm"]),
    ("k_w4a16_dec.cu", "w4a16_dec_kernel", ["L.x", "xg"]),
    ("k_gated_dec.cu", "gated_dec_kernel", ["a.x"]),
    ("k_dequant.cu", "rows16_kernel", ["x", "r", "dh", "dr"]),
    ("k_dequant.cu", "dequant_kernel", ["dmax"]),
    ("k_dequant.cu", "scored_rows_kernel", ["x", "labels", "res"]),
    ("k_dense.cu", "gemm16_kernel", ["a.sx", "a.dmax", "a.grow", "a.dh", "a.labels", "a.lse", "a.dloss", "a.x", "a.res", "a.owner"]),
    ("k_dense.cu", "gemm_finish_kernel", ["a.part4", "a.sx", "a.dmax", "a.grow", "a.res", "p"]),
    ("k_dense.cu", "ce_final_kernel", ["part", "labels", "tgt"]),
    ("k_skinny.cu", "skinny_kernel", ["a.sx", "a.dmax", "a.grow", "a.dh"]),
    ("k_skinny.cu", "skinny_finish_kernel", ["a.part", "a.sx", "a.dmax", "a.grow", "a.dh", "p"]),
]


def source(name):
    with open(os.path.join(CSRC, name)) as f:
        return re.sub(r"//[^\n]*", "", f.read())


def test_the_list_is_complete():
    found = set()
    for name in sorted(os.listdir(CSRC)):
        if name.endswith(".cu"):
            s = source(name)
            for m in re.finditer(r"__global__[^;{]*?\b(\w+_kernel)\s*\(", s):
                body = s[m.end():s.find("__global__", m.end()) if "__global__" in s[m.end():] else len(s)]
                if "griddep_wait()" in body:
                    found.add((name, m.group(1)))
    assert found == {(f, k) for f, k, _ in KERNELS}


@pytest.mark.parametrize("name,kernel,results", KERNELS)
def test_results_are_not_read_as_constants(name, kernel, results):
    s = source(name)
    for r in results:
        # anywhere in the file, the device functions of the kernel among them
        bad = re.findall(r"__ldg\((?:reinterpret_cast<[^>]*>\()?\s*\(?" + re.escape(r) + r"\b(?!\s*->)[^;]*;", s)
        assert not bad, (kernel, r, bad)
    args = re.search(kernel + r"\s*\(([^{]*)\)\s*\{", s).group(1)
    body = s[s.index(kernel):]
    for r in results:
        if re.search(r"const \w+ \*\s*__restrict__ " + re.escape(r) + r"\b", args):
            # a promise to the compiler: then every read of it names its instruction
            plain = re.findall(r"(?<![\w.*>])" + re.escape(r) + r"\s*\[", body)
            assert not plain, (kernel, r, "read by a plain load")
