"""Orders inside the kernels that no run can show to be right, checked in their
source: what would go wrong without them waits for a coincidence on the GPU."""
import glob
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))),
                    "sparse_mixture_experts_gemm_gb300", "csrc")


def kernels():
    """(file, name, body) of every kernel; a body ends where the next one starts."""
    for path in sorted(glob.glob(os.path.join(CSRC, "*.cu"))):
        with open(path) as f:
            text = re.sub(r"//[^\n]*", "", f.read())
        for part in text.split("__global__")[1:]:
            name = re.search(r"(\w+)\s*\(\s*(?:const\b|int\b|[A-Z])", re.sub(r"__launch_bounds__\([^{]*?\)\s*(?=\w+\()", "", part, count=1))
            yield os.path.basename(path), name.group(1) if name else "?", part


TMEM_KERNELS = [(f, n, b) for f, n, b in kernels() if "tmem_alloc" in b]


def test_kernels_are_found():
    assert {"decay_chunk.cu", "matmul_fp8.cu", "gemm.cu", "gemm2sm.cu", "gemm_q4.cu", "router.cu"} <= {f for f, _, _ in TMEM_KERNELS}


@pytest.mark.parametrize("file,name,body", TMEM_KERNELS, ids=[f"{f}:{n}" for f, n, _ in TMEM_KERNELS])
def test_tmem_is_taken_before_dependents_start(file, name, body):
    """The warp that takes a CTA's TMEM columns has them before it lets the next
    kernel start, and in the mixer's kernels every warp of the CTA: one of that
    kernel's CTAs that takes columns and then waits for this grid would
    otherwise hold what this CTA waits for."""
    trigger = body.find("pdl_launch_dependents()")
    if trigger < 0:
        return
    alloc = body.find("tmem_alloc")
    assert 0 <= alloc < trigger
    if file in ("decay_chunk.cu", "matmul_fp8.cu"):
        assert "__syncthreads()" in body[alloc:trigger]


def test_state_rows_are_fenced_before_copies_reuse_their_stages():
    """The initial state's rows pass through the last TMA stages by ordinary
    stores; copies of the asynchronous proxy into the same stages wait for the
    barrier s_ready, and a proxy fence has to come before its first arrival."""
    body = next(b for f, n, b in TMEM_KERNELS if f == "decay_chunk.cu" and "load_rows<" in b)
    stores = body.index("load_rows<")
    first_arrival = body.index("warp_arrive(s_ready)")
    assert "fence_proxy_async_smem()" in body[stores:body.index("__syncthreads()", stores)]
    assert stores < first_arrival
