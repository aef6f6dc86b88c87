"""Which kernels of the paged cache the bounds-checked build covers: their sources, without a GPU."""
import os
import re

import pytest

import block_diffusion_speculative_dfl_gb300 as dfl

CSRC = os.path.join(os.path.dirname(os.path.abspath(dfl.__file__)), "csrc")


def functions(path):
    """Name -> body of every function of a file that starts a line."""
    src, out = re.sub(r"__launch_bounds__\((?:[^()]|\([^()]*\))*\)", "", open(path).read()), {}
    for m in re.finditer(r"^(?:__global__|__device__)[^;{]*?(\w+)\s*\([^;{]*\)\s*\{", src, re.M):
        depth, i = 1, m.end()
        while depth:
            depth += {"{": 1, "}": -1}.get(src[i], 0)
            i += 1
        out[m.group(1)] = src[m.start():i]
    return out


# what writes its own thread's place only: n < N, i < total
PLAIN = {"pages_save_kernel"}


@pytest.mark.parametrize("name", ["pages.cu", "kv4_cache.cu", "kv4_attn.cu", "kv4_attn_tc.cu", "kv4_attn.cuh"])
def test_every_kernel_checks_the_places_it_computes(name):
    fs = functions(os.path.join(CSRC, name))
    kernels = [n for n, body in fs.items() if body.startswith(("__global__", "template")) and "__global__" in body]
    assert len(kernels) == open(os.path.join(CSRC, name)).read().count("__global__ void")
    for k in set(kernels) - PLAIN:
        called = [k] + [n for n in fs if n != k and re.search(rf"\b{n}\(", fs[k])]
        assert any("DFL_IN_BOUNDS" in fs[n] for n in called), k
