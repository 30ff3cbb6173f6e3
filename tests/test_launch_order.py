"""Kernels launched with programmatic serialisation may start while the kernel ahead of them runs. Each of the
full-precision operators' kernels waits for it (griddepcontrol.wait) on every path, before it ends at the latest: a
CTA that left without waiting could let the grid be complete before the one ahead is. Checked in the sources, CPU."""
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "bit_linear_layers_b200", "csrc")
HEADERS = ["bl_layernorm.cuh", "bl_layernorm_grad.cuh", "bl_embedding.cuh", "bl_gradclip.cuh"]
WAIT = re.compile(r"\bgrid_(begin|dependency_wait)\(\)")


def kernels(text):
    """(name, body) of every kernel of a source text."""
    text = re.sub(r"//[^\n]*", "", text)
    for m in re.finditer(r"__global__", text):
        head = text.index("{", m.end())
        name = re.findall(r"(\w+_kernel)\s*\(", text[m.end():head])[-1]
        depth, at = 1, head + 1
        while depth:
            depth += {"{": 1, "}": -1}.get(text[at], 0)
            at += 1
        yield name, text[head:at]


@pytest.mark.parametrize("header", HEADERS)
def test_every_kernel_waits_on_every_path(header):
    with open(os.path.join(CSRC, header)) as f:
        found = dict(kernels(f.read()))
    assert found
    for name, body in found.items():
        wait = WAIT.search(body)
        assert wait, f"{name} does not wait for the kernel ahead"
        for r in re.finditer(r"\breturn\b", body):
            assert wait.start() < r.start(), f"{name} may return without waiting"


def test_the_check_sees_a_kernel_that_leaves_early():
    body = """__global__ void __launch_bounds__(32) early_kernel(int n) { if (n) { return; } grid_begin(); }
              __global__ void late_kernel(int n) { grid_begin(); if (n) { return; } }"""
    found = dict(kernels(body))
    assert list(found) == ["early_kernel", "late_kernel"]
    early = found["early_kernel"]
    assert WAIT.search(early).start() > early.index("return") and WAIT.search(found["late_kernel"])


def test_programmatic_launches_are_of_these_kernels():
    names = {n for h in HEADERS for n, _ in kernels(open(os.path.join(CSRC, h)).read())}
    for f in ("bl_api.cu", "bl_norm.cu", "bl_norm_grad.cu"):
        with open(os.path.join(CSRC, f)) as src:
            for k in re.findall(r"\b(\w+_kernel)\b", " ".join(re.findall(r"launch_after\(([^,]*),", src.read()))):
                assert k in names, k
