"""Serving operators without a GPU, beyond test_serving_host.py: rules that the
sources keep, and what the Python side and the build refuse or report."""
import os
import re

import pytest
import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
SERVE = os.path.join(ROOT, "rank_biased_window_b200", "csrc", "serve")


def _functions(text):
    """(head, body) of every function of a source laid out with its braces in the first column."""
    for m in re.finditer(r"^((?:template|__global__|__device__|struct)[^;{}]*?\([^{};]*\)[^{};]*)\{\n(.*?)^\}",
                         text, re.M | re.S):
        yield m.group(1), m.group(2)


@pytest.mark.parametrize("name", ["rotary.cuh", "cache_append.cuh", "cache_attn.cuh", "cache_evict.cuh"])
def test_kernels_wait_before_they_read(name):
    """A kernel may start while the one before it runs, and only its wait makes
    earlier writes visible: it stands in the kernel itself, in front of whatever
    reads global memory, and on every way through it."""
    with open(os.path.join(SERVE, name)) as f:
        text = f.read()
    kernels = [(h, b) for h, b in _functions(text) if "__global__" in h]
    assert len(kernels) == text.count("__global__ ")
    for head, body in _functions(text):
        if "__global__" not in head:
            assert "grid_dep_wait" not in body, head
            continue
        assert body.count("grid_dep_wait()") == 1, head
        before = re.sub(r"//.*", "", body.split("grid_dep_wait()")[0])
        assert "return" not in before, head
        for read in ("__ld", "parts_of", "place_of", "segment_of", "select_begin", "a.lengths", "a.mass",
                     "a.kept", "a.pos[", "a.start[", "_mass<", "fetch", "bulk_load"):
            assert read not in before, (head, read)
