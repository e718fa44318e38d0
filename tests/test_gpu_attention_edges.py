"""The attention kernels where a call goes wrong or its inputs leave the ordinary
range, on the GPU: waits that run out, scores and weights at the ends of float32."""
import numpy as np
import pytest
import torch

import sparse_mixture_experts_gemm_gb300 as moe
from oracle import attention as oracle
from test_gpu_attention import BF16, I32, check_attend, check_decode, check_rope, ends, f64, gen, \
    make_table, normal, prefill_inputs, random_cache, rope_freq, rows_of

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


@pytest.mark.parametrize("loads", [0, 1, 2, 3, 4, 7, 12, 23, 1000])
@pytest.mark.parametrize("D,Hq,Hk,ql,kl", [(128, 8, 2, [700, 90], [700, 90]), (256, 16, 2, [700, 90], [700, 90]),
                                           (128, 8, 2, [60], [9000]), (256, 16, 2, [60], [9000])])
def test_prefill_ends_when_a_wait_runs_out(dev, stall, D, Hq, Hk, ql, kl, loads):
    """Copies that stop anywhere in a tile of rows, of one or of several a cluster, with
    keys whole and in parts."""
    q, k, v = (x.to(dev) for x in prefill_inputs(D + loads, sum(ql), sum(kl), Hq, Hk, D))
    args = (q, k, v, ends(ql, dev), ends(kl, dev))
    ref = moe.attention_prefill(*args)
    assert moe.moe_noalloc_status()[0] == moe.MOE_OK
    stall(loads)
    moe.attention_prefill(*args)
    code, detail = moe.moe_noalloc_status()
    # (a tile of rows at the least has its first keys and values to copy)
    assert code == moe.MOE_ERR_DEVICE_TIMEOUT if loads < 2 else code in (moe.MOE_ERR_DEVICE_TIMEOUT, moe.MOE_OK)
    assert detail // 100 == (11 if code else 0) and (code == moe.MOE_OK or loads < 1000)
    moe.moe_debug_attention_stall(-1)
    assert torch.equal(moe.attention_prefill(*args), ref)
    assert moe.moe_noalloc_status()[0] == moe.MOE_OK


def test_prefill_of_many_tiles_ends_when_a_wait_runs_out(dev, stall):
    """Clusters with several tiles of rows each: aborts in a later one."""
    q, k, v = (x.to(dev) for x in prefill_inputs(3, 3000, 3000, 32, 8, 128))
    ref = moe.attention_prefill(q, k, v)
    for loads in (30, 61, 90):
        stall(loads)
        moe.attention_prefill(q, k, v)
        assert moe.moe_noalloc_status()[0] == moe.MOE_ERR_DEVICE_TIMEOUT
        moe.moe_debug_attention_stall(-1)
        assert torch.equal(moe.attention_prefill(q, k, v), ref)


def test_prefill_tiles_of_rows_may_outlast_a_wait(dev, stall):
    """The schedule is two tiles of rows ahead and waits for one to be done, which
    over the longest keys takes longer than any other wait: here up to 650 us, with
    200 us for the others."""
    q, k, v = (x.to(dev) for x in prefill_inputs(4, 65536, 65536, 4, 4, 128))
    ref = moe.attention_prefill(q, k, v)
    moe.moe_debug_attention_stall(2 ** 31 - 1, 200)
    got = moe.attention_prefill(q, k, v)
    assert moe.moe_noalloc_status()[0] == moe.MOE_OK
    assert torch.equal(got, ref)


# ------------------------------------- scores and weights at the ends of float32
@pytest.mark.parametrize("Hq,Hk,D", [(16, 2, 256), (8, 4, 128)])
def test_prefill_scores_of_minus_infinity(dev, Hq, Hk, D):
    """Keys whose score is minus infinity weigh nothing; a row of no others is 0 / 0,
    whether its keys are cut into parts or not; rows that see no key are zeros."""
    for T, M in ((4, 4000), (100, 300)):  # in parts, and not
        q, k, v = prefill_inputs(T, T, M, Hq, Hk, D)
        q[..., 5] = q[..., 5].abs() + 1
        hidden = k.clone()
        hidden[:M // 2, :, 5] = float("-inf")
        got = moe.attention_prefill(q.to(dev), hidden.to(dev), v.to(dev))
        check_attend(got, q, k[M // 2:], v[M // 2:], D ** -0.5, [0, T], [0, M - M // 2])
        hidden[:, :, 5] = float("-inf")
        assert torch.isnan(moe.attention_prefill(q.to(dev), hidden.to(dev), v.to(dev))).all()
    q, k, v = prefill_inputs(9, 40, 9000, Hq, Hk, D)
    off, koff = ends([3, 37], dev), ends([8999, 1], dev)
    got = moe.attention_prefill(q.to(dev), k.to(dev), v.to(dev), off, koff)
    assert not got[3:39].any() and got[:3].any() and got[39].any()


@pytest.mark.parametrize("L", [40, 64, 900, 30000])
@pytest.mark.parametrize("D", [128, 256])
def test_decode_scores_of_minus_infinity(dev, D, L):
    """Tokens whose score is below what float32 holds weigh nothing next to others; a
    row of no others is not a number, as 0 / 0 is, and not that of an empty sequence."""
    g = gen(L + D)
    table, P = make_table(g, [L])
    codes, affine = random_cache(g, P, 1, D, dev)
    q = (normal(g, 1, 4, D).abs() + 1) * 2.0 ** 20
    hidden = affine.clone()
    at = torch.arange(L // 2)
    hidden[table[0].long()[at // 64].to(dev), 0, :, (at % 64).to(dev), 0] = torch.tensor([0.0, -2.0 ** 127], dtype=BF16, device=dev)
    n = torch.tensor([L], dtype=I32, device=dev)
    got = moe.attention_decode(q.to(dev), (codes, hidden), table.to(dev), n, scale=2.0 ** -24)
    # the same as over the other tokens, in a cache of their own
    m = L - L // 2
    rest = [torch.zeros(-(-m // 64), *t.shape[1:], dtype=t.dtype) for t in (codes, affine)]
    to = torch.arange(m)
    for t, x in zip(rest, rows_of((codes, affine), table, 0, L // 2, L)):
        t[to // 64, :, :, to % 64] = x
    check_decode(got, q, rest, torch.arange(len(rest[0]))[None], [m], 2.0 ** -24)
    hidden[:, 0, :, :, 0] = torch.tensor([0.0, -2.0 ** 127], dtype=BF16, device=dev)
    got = moe.attention_decode(q.to(dev), (codes, hidden), table.to(dev), n, scale=2.0 ** -24)
    assert torch.isnan(got).all()
    assert not moe.attention_decode(q.to(dev), (codes, hidden), table.to(dev), n * 0, scale=2.0 ** -24).any()


FAR = [([300], [300], 16, 2, 256), ([300], [300], 8, 2, 128), ([5], [6000], 16, 2, 256), ([5], [6000], 8, 2, 128)]


@pytest.mark.parametrize("ql,kl,Hq,Hk,D", FAR)
@pytest.mark.parametrize("e", [12, 20, 30, 40, 60, 100])
def test_prefill_large_scores(dev, ql, kl, Hq, Hk, D, e):
    """Scores of small whole numbers times 2^e, exact in fp32: each query has the mean
    of the values of its largest.  (Half a step of bf16 for each weight, and one for
    the result.)"""
    g = gen(e + D + sum(kl))
    T, M = sum(ql), sum(kl)
    q = torch.zeros(T, Hq, D)
    q.scatter_(2, torch.randint(0, D, (T, Hq, 1), generator=g), 2.0 ** (e // 2))
    k = torch.randint(-3, 4, (M, Hk, D), generator=g) * 2.0 ** (e - e // 2)
    v = normal(g, M, Hk, D)
    q, k = q.to(BF16), k.to(BF16)
    got = f64(moe.attention_prefill(q.to(dev), k.to(dev), v.to(dev), ends(ql, dev), ends(kl, dev)))
    for h in range(Hq):
        s = f64(q[:, h]) @ f64(k[:, h // (Hq // Hk)]).T
        s[np.arange(M)[None] > np.arange(T)[:, None] + M - T] = -np.inf
        p = (s == s.max(1, keepdims=True)) / 1.0
        p /= p.sum(1, keepdims=True)
        x = f64(v[:, h // (Hq // Hk)])
        ref, mag = p @ x, p @ np.abs(x)
        assert (np.abs(got[:, h] - ref) <= 2.0 ** -8 * (np.abs(ref) + mag) * (1 + 2.0 ** -6) + mag * (M / 16 + 64) * 2.0 ** -23).all()


@pytest.mark.parametrize("ql,kl,Hq,Hk,D", FAR)
@pytest.mark.parametrize("e", [8, 14, 18])
def test_prefill_scores_far_from_zero(dev, ql, kl, Hq, Hk, D, e):
    """Scores that differ by a few units next to a common part of up to 2^18, exact in
    fp32: the weights are those of the differences (scale and log2(e) rounded to
    fp32 and the exponential's last bits leave 2^-19 of a weight)."""
    g = gen(e + D + sum(kl))
    T, M = sum(ql), sum(kl)
    q, k, v = torch.zeros(T, Hq, D), torch.zeros(M, Hk, D), normal(g, M, Hk, D)
    q[..., 0], k[..., 0] = 2.0 ** (e // 2), 2.0 ** (e - e // 2)
    q[..., 1] = 1
    k[..., 1] = torch.arange(M)[:, None] % 89 * 2.0 ** -4  # the largest in each tile or part another
    q, k = q.to(BF16), k.to(BF16)
    got = moe.attention_prefill(q.to(dev), k.to(dev), v.to(dev), ends(ql, dev), ends(kl, dev), scale=1.0)
    k[..., 0] = 0
    ref, mag, _ = oracle.attend(f64(q), f64(k), f64(v), 1.0, ends(ql), ends(kl))
    tol = 2.0 ** -8 * (np.abs(ref) + mag) * (1 + 2.0 ** -6) + mag * ((M / 16 + 64) * 2.0 ** -23 + 2.0 ** -18)
    assert (np.abs(f64(got) - ref) <= tol).all()


@pytest.mark.parametrize("T,M", [(150, 150), (3, 5000)])
@pytest.mark.parametrize("D", [128, 256])
def test_scales_near_the_ends_of_float32(dev, D, T, M):
    """Scores that a scale brings into range, and scales of which nothing but means are left."""
    q, k, v = prefill_inputs(D + T, T, M, 4, 2, D)
    table, P = make_table(gen(T), [M])
    codes, affine = random_cache(gen(D), P, 2, D, dev)
    n = torch.tensor([M], dtype=I32, device=dev)
    for scale, e in ((2.0 ** 100 * D ** -0.5, -50), (1e-44, 0), (1e-38, 0)):
        qs, ks, a = q * 2.0 ** e, k * 2.0 ** e, affine.clone()
        a[:, 0] *= 2.0 ** e
        check_attend(moe.attention_prefill(qs.to(dev), ks.to(dev), v.to(dev), scale=scale), qs, ks, v, scale)
        got = moe.attention_decode(qs[:1].to(dev), (codes, a), table.to(dev), n, scale=scale)
        check_decode(got, qs[:1], (codes, a), table, [M], scale)


@pytest.mark.parametrize("T,M,Hq,Hk,D", [(600, 600, 8, 2, 128), (600, 600, 16, 2, 256), (300, 300, 1, 1, 256), (40, 3000, 8, 2, 128),
                                         (40, 3000, 16, 2, 256)])
def test_prefill_infinite_values(dev, T, M, Hq, Hk, D):
    """A query that sees an infinity in v has it, one that sees both or a NaN has NaN,
    wherever their tokens fall among the tiles and parts; other columns, heads and
    earlier queries are as they were."""
    q, k, v = prefill_inputs(T + M + D, T, M, Hq, Hk, D)
    ref = moe.attention_prefill(q.to(dev), k.to(dev), v.to(dev)).cpu()
    inf, nan, h = float("inf"), float("nan"), Hk - 1
    rng = np.random.default_rng(T + D)
    what = {}  # column -> [(token, value)]
    for c in range(0, D, 3):
        places = [0, M // 3, M - 1, M - 2, M - T, M - T // 2, *rng.integers(M - T, M, 8), *rng.integers(0, M, 4)]
        what[c] = [(int(x), rng.choice([inf, -inf, inf, -inf, nan])) for x in rng.permutation(places)[:rng.integers(1, 3)]]
    for c, marks in what.items():
        for at, x in marks:
            v[at, h, c] = x
    got = moe.attention_prefill(q.to(dev), k.to(dev), v.to(dev)).cpu()
    want = ref.clone().float()
    group = slice(h * (Hq // Hk), (h + 1) * (Hq // Hk))
    for c, marks in what.items():
        for at in {at for at, _ in marks}:
            x = v[at, h, c].float()  # (of two at one place the last)
            want[max(0, at - (M - T)):, group, c] += x
    assert torch.equal(torch.isnan(got), torch.isnan(want))
    assert torch.equal(torch.nan_to_num(got.float(), nan=0.0), torch.nan_to_num(want, nan=0.0))


# --------------------------------------------------- the largest and the widest
def test_cache_past_32_bits(dev):
    """Pages whose codes lie more than 2^32 bytes into the cache, written, read back and
    attended to."""
    g = gen(31)
    H, D, P, L = 2, 256, 140000, 300
    cache = (torch.zeros(P, 2, H, 64, D // 2, dtype=torch.uint8, device=dev),
             torch.zeros(P, 2, H, 64, D // 64, 2, dtype=BF16, device=dev))
    assert cache[0].numel() > 1 << 32
    table = torch.tensor([[P - 1, 0, P - 2, 131072, 70000]], dtype=I32)
    k, v, q = normal(g, L, H, D), normal(g, L, H, D), normal(g, 1, 16, D)
    moe.kv_cache_write(cache, k.to(dev), v.to(dev), table.to(dev))
    ko, vo = moe.kv_cache_read(cache, table.to(dev), ends([L], dev), L)
    for got, x in ((ko, k), (vo, v)):
        ref = oracle.values(*oracle.quantise(f64(x)))
        assert (np.abs(f64(got) - ref) <= np.abs(ref) * 2.0 ** -8 * (1 + 2.0 ** -14)).all()
    pages = table[0].long()
    small = tuple(t[pages.to(dev)] for t in cache)
    got = moe.attention_decode(q.to(dev), cache, table.to(dev), torch.tensor([L], dtype=I32, device=dev))
    check_decode(got, q, small, torch.arange(5)[None], [L], D ** -0.5)


def test_prefill_past_32_bits(dev):
    """Keys, values and outputs more than 2^31 elements into their tensors."""
    g = gen(32)
    Hk, D, M = 8, 256, (1 << 20) + 1000
    k = torch.zeros(M, Hk, D, dtype=BF16, device=dev)
    v = torch.zeros(M, Hk, D, dtype=BF16, device=dev)
    assert k.numel() > 1 << 31
    a, b, c = normal(g, 3, 16, D), normal(g, 900, Hk, D), normal(g, 900, Hk, D)
    k[-900:], v[-900:] = b.to(dev), c.to(dev)
    got = moe.attention_prefill(a.to(dev), k, v, ends([1, 2], dev), ends([M - 900, 900], dev))
    assert not got[0].any()  # (zero values)
    check_attend(got[1:], a[1:], b, c, D ** -0.5)
    del v
    # as queries: those of the last sequence, far into q and out
    out = torch.full_like(k, 7.0)
    off = torch.tensor([M - 900, M], dtype=I32, device=dev)
    moe.attention_prefill(k, b.to(dev), c.to(dev), off, ends([900], dev), out=out)
    check_attend(out[-900:], b, b, c, D ** -0.5)
    assert (out[:100] == 7).all() and (out[M - 1000:M - 900] == 7).all()


@pytest.mark.parametrize("Hq,Hk,D", [(4096, 4096, 128), (4096, 1, 128), (4096, 64, 256), (2047, 89, 256)])
def test_many_heads(dev, Hq, Hk, D):
    g = gen(Hk)
    q, k, v = (normal(g, 3, h, D) for h in (Hq, Hk, Hk))
    w, f, pos = torch.ones(D, dtype=BF16), rope_freq(64), torch.tensor([0, 5, 77], dtype=I32)
    qo, ko = moe.qk_norm_rope(*(x.to(dev) for x in (q, k, w, w, pos, f)))
    check_rope(qo, q, w, pos, f, 1e-6)
    check_rope(ko, k, w, pos, f, 1e-6)
    if Hq // Hk <= 64:
        check_attend(moe.attention_prefill(q.to(dev), k.to(dev), v.to(dev)), q, k, v, D ** -0.5)
    cache = moe.kv_cache(2, Hk, D, dev)
    table, n = torch.tensor([[1, 0]], dtype=I32), torch.tensor([3], dtype=I32, device=dev)
    moe.kv_cache_write(cache, k.to(dev), v.to(dev), table.to(dev))
    kr, vr = moe.kv_cache_read(cache, table.to(dev), ends([3], dev), 3)
    for got, x in ((kr, k), (vr, v)):
        ref = oracle.values(*oracle.quantise(f64(x)))
        assert (np.abs(f64(got) - ref) <= np.abs(ref) * 2.0 ** -8 * (1 + 2.0 ** -14)).all()
    check_decode(moe.attention_decode(q[:1].to(dev), cache, table.to(dev), n), q[:1], cache, table, [3], D ** -0.5)


@pytest.mark.parametrize("e", [0, -60, 100])
def test_cache_codes_next_to_borders(dev, e):
    """Values that are next to the middle between two codes by less than float32 holds
    beside the bias: the code is that of the definition, on either side of it."""
    odd = torch.arange(1, 16, 2)  # bias -1, -3, ..: next to zero (x - bias) / 2 is 0.5, 1.5, ..
    rows = []
    for b in odd.tolist():
        for lo, hi in ((-b, 30 - b), (-b * 5, 150 - b * 5)):  # scale 2, 10
            near = torch.tensor([s * m for m in (2.0 ** -24, 2.0 ** -30, 2.0 ** -45) for s in (1, -1)] + [0.0])
            row = torch.zeros(64, dtype=torch.float64)
            row[0], row[1], row[2:9] = lo, hi, near
            row[9:16] = torch.tensor([lo + (hi - lo) / 30 * i for i in (1, 3, 5, 7, 9, 11, 13)], dtype=torch.float64)
            rows.append(row)
    x = (torch.stack(rows) * 2.0 ** e).to(BF16).view(8, 1, 128)
    cache = moe.kv_cache(1, 1, 128, dev)
    table = torch.zeros(1, 1, dtype=I32)
    moe.kv_cache_write(cache, x.to(dev), -x.to(dev), table.to(dev))
    codes, affine = rows_of(cache, table, 0, 0, 8)
    for w, y in enumerate((x, -x)):
        c, s, b = oracle.quantise(f64(y))
        assert np.array_equal(f64(affine[:, w, ..., 0]), s) and np.array_equal(f64(affine[:, w, ..., 1]), b)
        assert np.array_equal(oracle.unpack(codes[:, w].numpy()), c)


@pytest.mark.parametrize("T,M,Hq,Hk,D", [(300, 300, 8, 2, 128), (300, 300, 16, 2, 256), (40, 3000, 8, 2, 128), (40, 3000, 16, 2, 256)])
@pytest.mark.parametrize("x", [float("inf"), -float("inf")])
def test_prefill_infinite_keys(dev, T, M, Hq, Hk, D, x):
    """An infinity in a key: for queries whose score it makes minus infinity the key
    weighs nothing, for the others that see it the row is NaN."""
    q, k, v = prefill_inputs(T + M + D + 1, T, M, Hq, Hk, D)
    h, group = Hk - 1, slice((Hk - 1) * (Hq // Hk), Hq)
    clean = moe.attention_prefill(q.to(dev), k.to(dev), v.to(dev)).cpu()
    for at in (0, M // 3, M - T, M - T // 2, M - 1):
        k2 = k.clone()
        k2[at, h, 9] = x
        got = moe.attention_prefill(q.to(dev), k2.to(dev), v.to(dev)).cpu()
        sees = (torch.arange(T) + M - T >= at)[:, None].expand(T, Hq).clone()
        sees[:, :group.start] = False
        gone = sees & (q[..., 9].float() * x < 0)
        if at == 0 and T == M:
            gone[0] = False  # (no other key)
        assert torch.equal(torch.isnan(got).all(-1), sees & ~gone) and torch.equal(torch.isnan(got).any(-1), sees & ~gone)
        assert torch.equal(got[~sees], clean[~sees])
        keep = np.arange(M) != at
        for i in np.flatnonzero(gone.any(1).numpy())[::7]:
            n = M - T + i + 1
            rows = np.flatnonzero(gone[i].numpy())
            a, b = f64(k[:n, h])[keep[:n]], f64(v[:n, h])[keep[:n]]
            s = f64(q[i, rows]) @ a.T * D ** -0.5
            p = np.exp(s - s.max(1, keepdims=True))
            p /= p.sum(1, keepdims=True)
            ref, mag = p @ b, p @ np.abs(b)
            reach = (np.abs(f64(q[i, rows])) @ np.abs(a).T).max(1, keepdims=True)
            tol = 2.0 ** -8 * (np.abs(ref) + mag) * (1 + 2.0 ** -6) + \
                mag * ((n / 16 + 64) * 2.0 ** -23 + 2 * D ** -0.5 * reach * (D / 8 + 8) * 2.0 ** -23)
            assert (np.abs(f64(got[i, rows]) - ref) <= tol).all()
