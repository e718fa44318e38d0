"""The attention kernels where a call goes wrong or its inputs leave the ordinary
range, on the GPU: waits that run out, scores and weights at the ends of float32."""
import numpy as np
import pytest
import torch

import sparse_mixture_experts_gemm_gb300 as moe
from oracle import attention as oracle
from test_gpu_attention import BF16, I32, check_attend, check_decode, ends, f64, gen, make_table, normal, \
    prefill_inputs, random_cache

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def dev():
    moe.build()
    moe.lib()
    yield torch.device("cuda", 0)
    assert moe.moe_noalloc_status()[0] == moe.MOE_OK


@pytest.fixture
def stall():
    """Waits that run out after 2 ms, as copies stop; calls are as ever afterwards."""
    yield lambda loads: moe.moe_debug_attention_stall(loads, 2000)
    moe.moe_debug_attention_stall(-1)


# ------------------------------------------------- waits that run out
@pytest.mark.parametrize("loads", [0, 1, 2, 3, 5])
@pytest.mark.parametrize("D", [128, 256])
def test_decode_ends_when_a_wait_runs_out(dev, stall, D, loads):
    """Copies that stop after some pages: the call ends and says so, and the next
    one has the results of the one before."""
    g = gen(D + loads)
    lens = [9000, 70, 1, 40000]  # more pages than shares: some of a team's rows end, some do not
    table, P = make_table(g, lens)
    cache = random_cache(g, P, 2, D, dev)
    args = (normal(g, 4, 16, D).to(dev), cache, table.to(dev), torch.tensor(lens, dtype=I32, device=dev))
    ref = moe.attention_decode(*args)
    assert moe.moe_noalloc_status()[0] == moe.MOE_OK
    stall(loads)
    moe.attention_decode(*args)
    code, detail = moe.moe_noalloc_status()
    assert code == (moe.MOE_ERR_DEVICE_TIMEOUT if loads < 4 else moe.MOE_OK) and (loads > 3 or detail // 100 == 12)
    moe.moe_debug_attention_stall(-1)
    assert torch.equal(moe.attention_decode(*args), ref)
    assert moe.moe_noalloc_status()[0] == moe.MOE_OK
