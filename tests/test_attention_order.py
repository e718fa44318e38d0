"""Orders inside the attention kernels that no run can show to be right, checked in
their source (as in test_kernel_order.py), and the test hook's arguments."""
import os
import re

import numpy as np
import pytest

import sparse_mixture_experts_gemm_gb300 as moe
from sparse_mixture_experts_gemm_gb300 import buildlib as moe_build

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))),
                    "sparse_mixture_experts_gemm_gb300", "csrc")


def source(name):
    with open(os.path.join(CSRC, name)) as f:
        return re.sub(r"//[^\n]*", "", f.read())


def block(text, start):
    """The braces' body that opens first behind `start`."""
    at = depth = text.index("{", text.index(start))
    depth = 0
    for i in range(at, len(text)):
        depth += {"{": 1, "}": -1}.get(text[i], 0)
        if depth == 0:
            return text[at + 1:i]
    raise AssertionError(start)


def outer_exits(body):
    """Positions of the breaks that leave the loop whose body this is: those in no
    loop further in."""
    inner = re.sub(r"for \([^{;]*;[^{;]*;[^{]*\) \{", lambda m: "\x01" * len(m.group(0)), body)
    exits, depth, loops = [], 0, []
    for i, c in enumerate(inner):
        if c == "\x01" and (i + 1 == len(inner) or inner[i + 1] != "\x01"):
            depth += 1
            loops.append(depth)
        elif c == "{":
            depth += 1
        elif c == "}":
            if loops and loops[-1] == depth:
                loops.pop()
            depth -= 1
        elif inner.startswith("break;", i) and not loops:
            exits.append(i)
    return exits


def test_exits_are_found():
    assert outer_exits("if (a) break; for (int i = 0; i < 3; ++i) { if (b) { break; } } { break; }") == [7, 66]


def test_a_team_of_decode_leaves_its_rows_by_a_vote():
    """The four warps of a team meet at named barriers in every row.  A warp that
    left, or stayed, on what it saw of an abort itself could leave the others
    waiting: after the wait for a row they vote, and what comes before the vote
    leaves no loop."""
    rows = block(source("attn_decode.cu"), "for (int nr = 0;; ++nr)")
    vote = rows.index("named_bar_any(kVote + team, 32 * kTeamWarps, !ok)")
    exits = outer_exits(rows)
    assert len(exits) == 2 and vote < exits[0] < exits[1]
    assert rows.index("poll_d(") < vote < rows.index("todo.n") < rows.index("make_queries<D>")
    assert "named_bar" not in rows[:vote] and "return" not in rows


def test_a_cta_of_decode_waits_for_copies_after_an_abort():
    """Whichever role aborted: the consumers may do so when the copies' warps have ended."""
    body = source("attn_decode.cu").split("__global__")[1]
    end = body.rindex("__syncthreads()")
    assert end < body.index("__nanosleep", end) and "if (*abort_flag)" in body[end:]
    assert "poll_d(" not in body[end:]


def test_softmax_warps_of_prefill_leave_their_items_by_a_vote():
    """With heads of 128 two warps meet at a named barrier in every item, so whether
    they take the next is decided by both; with an item both meet once more,
    whatever they see of an abort meanwhile."""
    body = source("attn_prefill.cu").split("__global__")[1]
    items = block(body, "for (int k = 0;; ++k) {\n      const bool more")
    vote = items.index("if (D == 128 ? named_bar_any(1 + wq, 64, !more) : !more) break;")
    assert items.index("next_item(k, it)") < vote < items.index("Tile<kCut>")
    assert [items.startswith("break;", e) for e in outer_exits(items)] == [True] and outer_exits(items)[0] < items.index("Tile<kCut>")
    meets = [m.start() for m in re.finditer(r"named_bar_sync\(1 \+ wq, 64\)", items)]
    assert len(meets) == 1 and "return" not in re.sub(r"auto \w+ = \[&\]\([^)]*\) \{.*?\n      \};", "", items, flags=re.S)
    # not within a loop or a branch on what a warp saw: the last brace before it opens the case of 128 columns
    assert items.rindex("if constexpr (D == 128) {", 0, meets[0]) > items.rindex("}", 0, meets[0])


def test_what_a_signal_of_prefill_tells_of_is_done_before_it():
    """The signal to the other CTA that P is there is an asynchronous store, whose
    release need not cover the warp's earlier stores: those have to be done, in every
    lane, when it is issued."""
    text = source("attn_prefill.cu")
    cleaned = block(text, "static __device__ __noinline__ void take_out")
    last = max(cleaned.rindex("st.shared"), cleaned.rindex("atom.shared"))
    assert last < cleaned.index('"fence.acq_rel.cluster;"') < cleaned.index("fence_proxy_async_smem()")
    made = block(text, "auto made = [&](int n)")
    assert made.index("tc_fence_before()") < made.index("__syncwarp()") < made.index("st_async_tx4")
    body = text.split("__global__")[1]
    for at in (m.start() for m in re.finditer(r"\bmade\(n\);", body)):
        before = body[:at]
        stored = max(before.rindex("st_pairs_16x32("), before.rfind("st_32x16("))
        assert stored < before.rindex("wait_st()") < before.rindex("clean(j)")


def test_rows_of_queries_that_no_copy_writes_are_zeros():
    """Where a group of heads does not divide 128 the last rows of a tile of queries
    belong to no token; they are written once, before the first copy and product."""
    body = source("attn_prefill.cu").split("__global__")[1]
    at = body.index("const int rows = a.tokens * a.group;")
    fence = body.index("fence_proxy_async_smem();", at)
    assert at < body.index("st.shared.v4.u32", at) < fence < body.index("__syncthreads()") < body.index("tma_load_3d_pair")
    for D in (128, 256):  # the same arithmetic: each 16-byte piece of those rows once, and no other
        for group in range(1, 65):
            rows = 128 // group * group
            n = 128 - rows
            pieces = [i // (n * 8) * 16384 + rows * 128 + i % (n * 8) * 16 for i in range(n * (D // 8))]
            want = [b * 16384 + r * 128 + 16 * p for b in range(D // 64) for r in range(rows, 128) for p in range(8)]
            assert pieces == want


def test_products_of_prefill_end_before_their_memory_goes():
    """The warp of the MMAs waits for them whether or not it saw an abort, by a limit
    that no hook shortens; both CTAs of a pair wait for what is in flight."""
    body = source("attn_prefill.cu").split("__global__")[1]
    drain = body.index("tc_commit2(smem_u32(&ctl.drain))")
    before = body[:drain].rstrip()
    assert before.endswith("if (one)") and before[:-len("if (one)")].rstrip().endswith("}")
    assert "poll(smem_u32(&ctl.drain), 0, nullptr, 1 << 21)" in body[drain:]
    told, met = body.index("cluster_map(smem_u32(&ctl.abort_flag), rank ^ 1)"), body.rindex("cluster_sync_all()")
    assert "__syncwarp();" in body[told:met]  # (the pair's barrier wants whole warps)
    assert drain < told < met < body.index("tmem_dealloc2") < body.index("__nanosleep")


@pytest.fixture(scope="module")
def lib():
    moe_build.build()
    return moe.lib()


@pytest.mark.parametrize("args,code", [((0, 0), moe.MOE_ERR_INVALID_ARG), ((5, 2000001), moe.MOE_ERR_INVALID_ARG),
                                       ((0, -1), moe.MOE_ERR_INVALID_ARG), ((5, 2000000), moe.MOE_OK),
                                       ((-1, 0), moe.MOE_OK)])
def test_stall_hook_arguments(lib, args, code):
    assert lib.moe_debug_attention_stall(*args) == code
    assert lib.moe_debug_attention_stall(-1, 0) == moe.MOE_OK


def test_scales_whose_exponents_of_two_are_infinite_are_refused(lib):
    """Scores are multiplied by scale times log2(e): that is finite up to 2.35e38."""
    P = 0x10000  # never dereferenced
    prefill = lambda s: lib.moe_attention_prefill(P, P, P, None, None, 0, 8, 2, 4, 2, 128, 512, 256, 256, s, P, None, 0, None)  # noqa: E731
    decode = lambda s: lib.moe_attention_decode(P, 512, P, P, 8, P, 4, P, 0, 4, 2, 128, s, P, P, 0, None)  # noqa: E731
    for call in (prefill, decode):
        assert call(2.35e38) == moe.MOE_OK and call(1e-45) == moe.MOE_OK
        assert call(2.4e38) == moe.MOE_ERR_INVALID_ARG and call(3e38) == moe.MOE_ERR_INVALID_ARG
    assert np.isfinite(np.float32(2.35e38) * np.float32(np.log2(np.e)))
