"""The full-attention layer's operators on the GPU against the float64 oracle.

Tolerances, from the arithmetic (half a step of bf16 is 2^-8 of a value):
  * rope: the norm in fp32 under 2^-18 of a value, sine and cosine and the two
    products as much again, then one rounding;
  * attention: weights rounded to bf16 before they multiply the values (2^-8 of
    the sum of magnitudes A = sum_j p_j |v_j|), the result rounded once; a score
    summed in fp32 is off by (D / 8 + 8) 2^-23 of its magnitudes, which changes
    its weight by scale times that, in the numerator and in the sum; sums over L
    keys on hardware that truncates: (L / 16 + 64) 2^-23 of A;
  * decode: the same, but what is rounded is weight times scale, which multiplies
    codes less 8: at most 8 p_t scale_t each; the weights that multiply biases
    are two bf16 parts (the second rounds what the first, off by 2^-8, leaves: 2^-16
    of the weight); the rest is fp32 of magnitudes at most 15 scale + |bias|;
  * the cache: codes, scales and biases exactly those of the definition, values
    within half a step.
"""
import numpy as np
import pytest
import torch

import sparse_mixture_experts_gemm_gb300 as moe
from oracle import attention as oracle

pytestmark = pytest.mark.gpu

BF16, I32 = torch.bfloat16, torch.int32


@pytest.fixture(scope="module")
def dev():
    moe.build()
    moe.lib()
    yield torch.device("cuda", 0)
    assert moe.moe_noalloc_status()[0] == moe.MOE_OK


def f64(t):
    return t.detach().cpu().to(torch.float64).numpy()


def gen(seed):
    g = torch.Generator()
    g.manual_seed(seed)
    return g


def normal(g, *shape, std=1.0):
    return (torch.randn(shape, generator=g) * std).to(BF16)


def ends(lens, device="cpu"):
    return torch.tensor([0, *lens], device=device).cumsum(0).to(I32)


# ------------------------------------------------------------------ rope
def check_rope(got, x, w, positions, freq, eps):
    ref, y = oracle.norm_rope(f64(x), f64(w), f64(positions), None if freq is None else f64(freq), eps)
    unit = np.abs(y)
    if freq is not None and len(freq):
        half = len(freq)
        pair = np.abs(y[..., :half]) + np.abs(y[..., half:2 * half])
        unit = np.concatenate([pair, pair, unit[..., 2 * half:]], -1)
    assert (np.abs(f64(got) - ref) <= np.abs(ref) * 2.0 ** -8 + unit * 2.0 ** -17 + 1e-30).all()


def rope_freq(rot, theta=1e7):
    return theta ** (-torch.arange(0, rot, 2, dtype=torch.float64) / rot) if rot else torch.zeros(0, dtype=torch.float64)


@pytest.mark.parametrize("N,Hq,Hk,D,rot", [
    (1, 16, 2, 256, 64), (1, 1, 1, 128, 128), (3, 5, 3, 128, 16), (7, 3, 1, 256, 256), (64, 16, 2, 256, 64),
    (130, 6, 2, 128, 96), (33, 64, 8, 128, 0), (2500, 4, 1, 256, 32), (5, 17, 1, 128, 48), (2433, 1, 1, 128, 128),
])
def test_rope(dev, N, Hq, Hk, D, rot):
    g = gen(N + Hq + D + rot)
    q, k = normal(g, N, Hq, D, std=2.0), normal(g, N, Hk, D, std=0.1)
    qw, kw = (1 + normal(g, D, std=0.2)).to(BF16), (1 + normal(g, D, std=0.2)).to(BF16)
    pos = torch.randint(0, 1 << 20, (N,), generator=g).to(I32)
    f = rope_freq(rot)
    qo, ko = moe.qk_norm_rope(*(x.to(dev) for x in (q, k, qw, kw, pos, f)), eps=1e-5)
    check_rope(qo, q, qw, pos, f, 1e-5)
    check_rope(ko, k, kw, pos, f, 1e-5)


def test_rope_far_and_negative_positions(dev):
    """Angles of up to 2^31 radians; positions below zero turn the other way."""
    g = gen(1)
    pos = torch.tensor([0, 1, -1, 2 ** 31 - 1, -2 ** 31, 123456789, 131071], dtype=I32)
    q, w, f = normal(g, 7, 2, 128), torch.ones(128, dtype=BF16), rope_freq(128)
    a, b = moe.qk_norm_rope(*(x.to(dev) for x in (q, q, w, w, pos, f)))
    check_rope(a, q, w, pos, f, 1e-6)
    assert torch.equal(a, b)


def test_rope_strided_in_place_and_none(dev):
    """Slices of a fused projection, over themselves; no rotation; single
    [heads][D] rows; batches of tokens."""
    g = gen(2)
    N, Hq, Hk, D = 21, 4, 2, 128
    qkv = normal(g, N, (Hq + 2 * Hk) * D + 8).to(dev)
    w, f = (1 + normal(g, D, std=0.1)).to(BF16).to(dev), rope_freq(64).to(dev)
    pos = torch.arange(N, dtype=I32, device=dev)
    q = qkv[:, 8:8 + Hq * D].unflatten(1, (Hq, D))
    k = qkv[:, 8 + Hq * D:8 + (Hq + Hk) * D].unflatten(1, (Hk, D))
    rest = qkv[:, 8 + (Hq + Hk) * D:].clone()
    ref = moe.qk_norm_rope(q.contiguous(), k.contiguous(), w, w, pos, f)
    plain = moe.qk_norm_rope(q, k, w, w, None, None)
    check_rope(plain[0], q.cpu(), w.cpu(), pos.cpu(), None, 1e-6)
    batch = moe.qk_norm_rope(q.unflatten(0, (3, 7)), k.unflatten(0, (3, 7)), w, w, pos.view(3, 7), f)
    assert torch.equal(batch[0].flatten(0, 1), ref[0]) and torch.equal(batch[1].flatten(0, 1), ref[1])
    one = moe.qk_norm_rope(q[5], k[5], w, w, pos[5], f)
    assert torch.equal(one[0], ref[0][5]) and torch.equal(one[1], ref[1][5])
    got = moe.qk_norm_rope(q, k, w, w, pos, f, q_out=q, k_out=k)
    assert got[0] is q and torch.equal(q, ref[0]) and torch.equal(k, ref[1])
    assert torch.equal(qkv[:, 8 + (Hq + Hk) * D:], rest)
    empty = moe.qk_norm_rope(q[:0], k[:0], w, w, pos[:0], f)
    assert empty[0].shape == (0, Hq, D)


@pytest.mark.parametrize("D", [128, 256])
@pytest.mark.parametrize("eps", [1e-6, 0.0])
def test_rope_special_rows(dev, D, eps):
    """Zeros, squares past float32's range and below it, NaN and infinity: their
    neighbours are untouched."""
    g = gen(D)
    x = torch.randn(8, 3, D, generator=g).clamp(-4, 4)
    for i, size in enumerate([0, 1e20, 5e37, 1e-20, 1e-36]):
        x[i, 1] *= size
    x[5, 1, 7], x[6, 1, D - 1] = float("nan"), float("inf")
    x = x.to(BF16)
    w, f, pos = torch.ones(D, dtype=BF16), rope_freq(64), torch.arange(8, dtype=I32)
    got, _ = moe.qk_norm_rope(*(t.to(dev) for t in (x, x, w, w, pos, f)), eps=eps)
    bad = np.isnan(f64(got)).any(-1)
    want = np.zeros((8, 3), bool)
    want[5, 1] = want[6, 1] = True
    assert np.array_equal(bad, want)
    ok = [0, 1, 2, 3, 4, 7]
    check_rope(got.cpu()[ok], x[ok], w, pos[ok], f, eps)
    assert not f64(got)[0, 1].any()


# --------------------------------------------------------------- prefill
def check_attend(got, q, k, v, scale, offsets=None, k_offsets=None):
    ref, mag, reach = oracle.attend(f64(q), f64(k), f64(v), scale, offsets, k_offsets)
    D, L = q.shape[-1], k.shape[0]
    score = 2 * scale * reach * (D / 8 + 8) * 2.0 ** -23
    tol = 2.0 ** -8 * (np.abs(ref) + mag) * (1 + 2.0 ** -6) + mag * ((L / 16 + 64) * 2.0 ** -23 + score[..., None])
    err = np.abs(f64(got) - ref)
    assert (err <= tol + 1e-30).all(), (err / np.maximum(tol, 1e-30)).max()


def prefill_inputs(seed, N, M, Hq, Hk, D, std=1.5):
    g = gen(seed)
    return normal(g, N, Hq, D, std=std), normal(g, M, Hk, D), normal(g, M, Hk, D)


PREFILL_LENS = [[1], [2], [17], [63], [64], [127], [128], [129], [255], [257], [700], [1, 1, 1], [0, 5, 0], [0, 0],
                [130, 0, 1, 64, 257, 31], [300, 200], [16, 15, 17, 128], [1] * 70]


@pytest.mark.parametrize("lens", PREFILL_LENS, ids=lambda x: "-".join(map(str, x[:8])))
@pytest.mark.parametrize("Hq,Hk,D", [(8, 1, 256), (6, 2, 128)])
def test_prefill(dev, lens, Hq, Hk, D):
    N = sum(lens)
    q, k, v = prefill_inputs(N + len(lens), N, N, Hq, Hk, D)
    off = ends(lens)
    got = moe.attention_prefill(q.to(dev), k.to(dev), v.to(dev), offsets=off.to(dev))
    check_attend(got, q, k, v, D ** -0.5, off)
    if len(set(lens)) == 1 and N:  # the same as a dense batch
        a = [x.to(dev).unflatten(0, (len(lens), lens[0])) for x in (q, k, v)]
        assert torch.equal(moe.attention_prefill(*a).flatten(0, 1), got)
    if len(lens) == 1:
        assert torch.equal(moe.attention_prefill(q.to(dev), k.to(dev), v.to(dev)), got)


@pytest.mark.parametrize("Hq,Hk,D", [(1, 1, 256), (16, 2, 256), (3, 1, 256), (5, 5, 128), (32, 8, 128), (24, 2, 128),
                                     (40, 1, 256), (64, 1, 128), (14, 2, 256)])
@pytest.mark.parametrize("N", [1, 45, 150])
def test_prefill_heads(dev, Hq, Hk, D, N):
    q, k, v = prefill_inputs(N + Hq, N, N, Hq, Hk, D)
    check_attend(moe.attention_prefill(q.to(dev), k.to(dev), v.to(dev), scale=0.11), q, k, v, 0.11)


@pytest.mark.parametrize("ql,kl", [([1], [1000]), ([5], [128]), ([100], [613]), ([256], [256 + 4096]), ([3, 40, 1], [3, 200, 129]),
                                   ([10, 0, 7, 300], [4, 9, 0, 299]), ([2, 2], [0, 0]), ([200], [30]), ([33, 1], [33, 2500]),
                                   ([1] * 20, [17 * i for i in range(20)])])
@pytest.mark.parametrize("Hq,Hk,D", [(8, 1, 256), (8, 4, 128)])
def test_prefill_behind_a_prefix(dev, ql, kl, Hq, Hk, D):
    """Queries that are the last of longer keys, also of fewer keys than queries
    (the first queries see nothing: zeros)."""
    q, k, v = prefill_inputs(sum(ql) + 3, sum(ql), sum(kl), Hq, Hk, D)
    oq, ok = ends(ql), ends(kl)
    got = moe.attention_prefill(q.to(dev), k.to(dev), v.to(dev), oq.to(dev), ok.to(dev))
    check_attend(got, q, k, v, D ** -0.5, oq, ok)
    for i, (a, b) in enumerate(zip(ql, kl)):
        assert not got[oq[i]:oq[i] + max(0, min(a, a - b))].any()


@pytest.mark.parametrize("D,Hq,Hk", [(256, 16, 2), (128, 8, 2)])
def test_prefill_long(dev, D, Hq, Hk):
    """A prompt of 2,900 tokens (every output), several rounds of key tiles."""
    q, k, v = prefill_inputs(D, 2900, 2900, Hq, Hk, D)
    check_attend(moe.attention_prefill(q.to(dev), k.to(dev), v.to(dev)), q, k, v, D ** -0.5)


@pytest.mark.parametrize("D", [128, 256])
def test_prefill_growing_scores(dev, D):
    """Scores that grow along the keys by hundreds, so that the running maximum
    moves in every tile; and ones that fall."""
    q, k, v = prefill_inputs(7, 900, 900, 2, 1, D)
    for sign in (1, -1):
        ramp = (torch.arange(900.0)[:, None, None] * sign * 0.05 + 1).to(BF16)
        q1 = torch.ones_like(q)
        k1 = (k * 0.01 + ramp).to(BF16)
        check_attend(moe.attention_prefill(q1.to(dev), k1.to(dev), v.to(dev)), q1, k1, v, D ** -0.5)


def test_prefill_slices_of_a_fused_projection(dev):
    g = gen(3)
    n, T, Hq, Hk, D = 3, 70, 8, 2, 128
    w = (Hq + 2 * Hk) * D
    qkv = normal(g, n, T, w + 16).to(dev)
    q, k, v = (qkv[..., a:b].unflatten(-1, (-1, D)) for a, b in
               ((0, Hq * D), (Hq * D, (Hq + Hk) * D), ((Hq + Hk) * D, w)))
    assert torch.equal(moe.attention_prefill(q, k, v),
                       moe.attention_prefill(q.contiguous(), k.contiguous(), v.contiguous()))


@pytest.mark.parametrize("D", [128, 256])
@pytest.mark.parametrize("what", ["nan", "inf", "lowest"])
def test_prefill_hidden_tokens_reach_nobody(dev, D, what):
    """NaN, infinities and the lowest value in keys and values reach only the
    queries that see their token: neither the earlier ones, nor the next packed
    sequence's, nor those of the sequence before."""
    lens = [150, 90, 201]
    q, k, v = prefill_inputs(11, sum(lens), sum(lens), 4, 2, D)
    off = ends(lens)
    ref = moe.attention_prefill(q.to(dev), k.to(dev), v.to(dev), off.to(dev))
    x = {"nan": float("nan"), "inf": float("inf"), "lowest": torch.finfo(BF16).min}[what]
    for at in (150 + 40, 150, 239):  # inside the second sequence
        for side in ("k", "v"):
            k2, v2 = k.clone(), v.clone()
            (k2 if side == "k" else v2)[at, 1, 5] = x
            got = moe.attention_prefill(q.to(dev), k2.to(dev), v2.to(dev), off.to(dev))
            keep = torch.ones(sum(lens), 4, dtype=torch.bool)
            keep[at:240, 2:] = False
            assert torch.equal(got.cpu()[keep], ref.cpu()[keep])
            if what != "lowest":
                hit = got.cpu()[at:240, 2:].float()
                col = ~torch.isfinite(hit[..., 5]) if side == "v" else ~torch.isfinite(hit).all(-1)
                if side == "v" or what == "nan":
                    assert col.all()


def test_prefill_bad_offsets_stay_in_bounds(dev):
    """Offsets past the end or running backwards are clamped; rows of one sequence
    have its results (rows 50 .. of these offsets lie in the third sequence, 50 ..
    200, too), and rows of no sequence what out held."""
    q, k, v = (x.to(dev) for x in prefill_inputs(12, 200, 200, 4, 1, 128))
    off = torch.tensor([0, 90, 50, 1 << 30, -5], dtype=I32, device=dev)
    out = torch.full_like(q, 7.0)
    moe.attention_prefill(q, k, v, off, out=out)
    torch.cuda.synchronize()
    assert torch.equal(out[:50], moe.attention_prefill(q[:90], k[:90], v[:90])[:50])
    off = torch.tensor([10, 90, 120], dtype=I32, device=dev)
    out = torch.full_like(q, 7.0)
    moe.attention_prefill(q, k, v, off, out=out)
    assert (out[:10] == 7).all() and (out[120:] == 7).all()
    assert torch.equal(out[10:90], moe.attention_prefill(q[10:90], k[10:90], v[10:90]))


SPLIT = [([5], [5000], 16, 2, 256), ([1], [9001], 16, 2, 256), ([1], [700], 1, 1, 128), ([3, 40], [3000, 6000], 8, 2, 128),
         ([200], [4000], 8, 4, 128), ([0, 17, 0, 300], [9, 20, 0, 6000], 8, 1, 256), ([60, 2], [2500, 1], 5, 5, 128),
         ([2, 2, 2, 2], [4000, 100, 0, 3000], 12, 2, 256), ([500], [1900], 8, 2, 256), ([33], [2048], 64, 1, 128),
         ([1] * 40, [(37 * i) % 300 for i in range(39)] + [9000], 8, 1, 128),
         ([1500, 130], [1510, 7000], 4, 1, 256), ([900, 0, 70, 40, 300], [900, 5, 4000, 6000, 310], 8, 2, 128)]


@pytest.mark.parametrize("ql,kl,Hq,Hk,D", SPLIT)
def test_prefill_few_queries_over_many_keys(dev, ql, kl, Hq, Hk, D):
    """The keys are cut into parts: sequences with fewer tiles than parts, with
    queries that see nothing, and rows of no sequence, which stay."""
    from sparse_mixture_experts_gemm_gb300 import attention
    N, M, front = sum(ql), sum(kl), 3
    if M >= 2000:  # (700 keys, and 500 queries over 1,900, are not worth a second kernel)
        assert attention._prefill_workspace(N + 2 * front, M, len(ql), Hq, Hk, D) > 0
    q, k, v = prefill_inputs(N + M, N + 2 * front, M, Hq, Hk, D)
    oq, ok = ends(ql) + front, ends(kl)
    out = torch.full((N + 2 * front, Hq, D), 7.0, dtype=BF16, device=dev)
    moe.attention_prefill(q.to(dev), k.to(dev), v.to(dev), oq.to(dev), ok.to(dev), out=out)
    check_attend(out[front:-front], q[front:-front], k, v, D ** -0.5, oq - front, ok)
    assert (out[:front] == 7).all() and (out[-front:] == 7).all()
    again = torch.full_like(out, 7.0)
    moe.attention_prefill(q.to(dev), k.to(dev), v.to(dev), oq.to(dev), ok.to(dev), out=again)
    assert torch.equal(again, out)


def test_prefill_bad_offsets_in_parts(dev):
    """Offsets that run to and fro, so that there are more tiles than the sizes alone
    allow: a row of one sequence has its results, the others lie in several."""
    q, k, v = prefill_inputs(78, 42, 9000, 16, 1, 128)
    oq = torch.tensor([0, 40] + [1, 40] * 6, dtype=I32, device=dev)
    ok = torch.tensor([0, 9000] * 7, dtype=I32, device=dev)
    from sparse_mixture_experts_gemm_gb300 import attention
    assert attention._prefill_workspace(42, 9000, 13, 16, 1, 128) > 0
    out = torch.full((42, 16, 128), 7.0, dtype=BF16, device=dev)
    moe.attention_prefill(q.to(dev), k.to(dev), v.to(dev), oq, ok, out=out)
    check_attend(out[:1], q[:1], k[:8961], v[:8961], 128 ** -0.5, [0, 1], [0, 8961])
    assert (out[40:] == 7).all()


def test_prefill_few_queries_dense(dev):
    """[n][T] queries over [n][M] keys in parts."""
    q, k, v = prefill_inputs(77, 4 * 3, 4 * 3000, 8, 2, 256)
    got = moe.attention_prefill(*(x.to(dev).unflatten(0, (4, -1)) for x in (q, k, v)))
    check_attend(got.flatten(0, 1), q, k, v, 256 ** -0.5, ends([3] * 4), ends([3000] * 4))


@pytest.mark.parametrize("bad", ["nan", "inf"])
@pytest.mark.parametrize("D", [128, 256])
def test_queries_that_are_not_finite_keep_to_themselves(dev, D, bad):
    for T, M in ((150, 150), (3, 3000)):
        q, k, v = (x.to(dev) for x in prefill_inputs(T + D, T, M, 8, 2, D))
        ref = moe.attention_prefill(q, k, v)
        q[1, 5, 7] = float(bad)
        got = moe.attention_prefill(q, k, v)
        keep = torch.ones(T, 8, dtype=torch.bool, device=dev)
        keep[1, 5] = False
        assert torch.equal(got[keep], ref[keep]) and not torch.isfinite(got[1, 5]).all()
    g = gen(D)
    table, P = make_table(g, [70, 900])
    cache, L = random_cache(g, P, 2, D, dev), torch.tensor([70, 900], dtype=I32, device=dev)
    q = normal(g, 2, 8, D).to(dev)
    ref = moe.attention_decode(q, cache, table.to(dev), L)
    q[1, 5, 7] = float(bad)
    got = moe.attention_decode(q, cache, table.to(dev), L)
    keep = torch.ones(2, 8, dtype=torch.bool, device=dev)
    keep[1, 5] = False
    assert torch.equal(got[keep], ref[keep]) and not torch.isfinite(got[1, 5]).all()


@pytest.mark.parametrize("D", [128, 256])
@pytest.mark.parametrize("what", ["nan", "inf"])
def test_prefill_hidden_tokens_of_parts(dev, D, what):
    """As above, where the keys are cut: a token among the last, which some queries
    see, and one that all of them see."""
    T, M = 40, 3000
    q, k, v = prefill_inputs(D, T, M + 70, 8, 2, D)
    oq, ok = torch.tensor([0, T], dtype=I32, device=dev), torch.tensor([0, M], dtype=I32, device=dev)
    ref = moe.attention_prefill(q.to(dev), k.to(dev), v.to(dev), oq, ok).cpu()
    x = float(what)
    for at in (M - 1, M - 20, M - T, 1500, M, M + 69):  # the last two: behind the sequence
        for side in ("k", "v"):
            k2, v2 = k.clone(), v.clone()
            (k2 if side == "k" else v2)[at, 1, 5] = x
            got = moe.attention_prefill(q.to(dev), k2.to(dev), v2.to(dev), oq, ok).cpu()
            keep = torch.ones(T, 8, dtype=torch.bool)
            if at < M:
                keep[max(0, at - (M - T)):, 4:] = False
            assert torch.equal(got[keep], ref[keep])
            if at < M and (side == "v" or what == "nan"):
                hit = got[max(0, at - (M - T)):, 4:].float()
                assert (~torch.isfinite(hit[..., 5]) if side == "v" else ~torch.isfinite(hit).all(-1)).all()


def test_prefill_is_repeatable(dev):
    q, k, v = (x.to(dev) for x in prefill_inputs(5, 1500, 1500, 16, 2, 256))
    first = moe.attention_prefill(q, k, v)
    for _ in range(4):
        assert torch.equal(moe.attention_prefill(q, k, v), first)


# ----------------------------------------------------------------- cache
def make_table(g, reach, extra=2):
    """Pages in random order for sequences of these lengths: (table, pages)"""
    need = [-(-r // 64) for r in reach]
    P = sum(need) + extra
    order = torch.randperm(P, generator=g).to(I32)
    table = torch.zeros(len(reach), max(max(need), 1), dtype=I32)
    at = 0
    for i, n in enumerate(need):
        table[i, :n] = order[at:at + n]
        at += n
    return table, P


def rows_of(cache, table, i, a, b):
    """codes [b - a][2][H][D / 2] and affine of sequence i's positions a .. b"""
    at = torch.arange(a, b)
    page = table[i].long()[at // 64]
    return tuple(x.cpu()[page, :, :, at % 64] for x in cache)


@pytest.mark.parametrize("H,D", [(2, 256), (1, 128), (3, 128), (5, 256)])
@pytest.mark.parametrize("starts,lens", [([0], [1]), ([0], [200]), ([63, 64, 0, 5], [1, 1, 1, 1]),
                                         ([100, 0, 7, 0], [30, 0, 129, 64]), ([3] * 40, [2] * 40)])
def test_cache_write_and_read(dev, H, D, starts, lens):
    g = gen(sum(lens) + H)
    N = sum(lens)
    k, v = normal(g, N, H, D), normal(g, N, H, D, std=3.0)
    table, P = make_table(g, [a + b for a, b in zip(starts, lens)])
    cache = moe.kv_cache(P, H, D, dev)
    for t in cache:
        t.view(torch.uint8).fill_(0x5a)
    st, off = torch.tensor(starts, dtype=I32), ends(lens)
    moe.kv_cache_write(cache, k.to(dev), v.to(dev), table.to(dev), st.to(dev), off.to(dev))
    touched = torch.zeros(P, 64, dtype=torch.bool)
    for i, (a, n) in enumerate(zip(starts, lens)):
        codes, affine = rows_of(cache, table, i, a, a + n)
        for w, x in enumerate((k, v)):
            c, s, b = oracle.quantise(f64(x[off[i]:off[i + 1]]))
            assert np.array_equal(oracle.unpack(codes[:, w].numpy()), c)
            assert np.array_equal(f64(affine[:, w, ..., 0]), s) and np.array_equal(f64(affine[:, w, ..., 1]), b)
        at = torch.arange(a, a + n)
        touched[table[i].long()[at // 64], at % 64] = True
    rest = cache[0].cpu().permute(0, 3, 1, 2, 4)[~touched]
    assert (rest == 0x5a).all()
    out = [torch.full((N + 3, H, D), 7.0, dtype=BF16, device=dev) for _ in range(2)]
    moe.kv_cache_read(cache, table.to(dev), off.to(dev), N + 3, st.to(dev), *out)
    for x, got in zip((k, v), out):
        ref = oracle.values(*oracle.quantise(f64(x)))
        assert (np.abs(f64(got[:N]) - ref) <= np.abs(ref) * 2.0 ** -8 * (1 + 2.0 ** -14)).all() and (got[N:] == 7).all()


def test_cache_dense_and_strided(dev):
    """[n][T][H][D] slices of a fused projection give what packed tokens give."""
    g = gen(4)
    n, T, H, D = 3, 5, 2, 128
    kv = normal(g, n, T, 2 * H * D + 8).to(dev)
    k, v = kv[..., :H * D].unflatten(-1, (H, D)), kv[..., H * D:2 * H * D].unflatten(-1, (H, D))
    table, P = make_table(g, [70] * n)
    table = table.to(dev)
    st = torch.tensor([0, 60, 64], dtype=I32, device=dev)
    a, b = moe.kv_cache(P, H, D, dev), moe.kv_cache(P, H, D, dev)
    moe.kv_cache_write(a, k, v, table, st)
    off = ends([T] * n, dev)
    moe.kv_cache_write(b, k.flatten(0, 1).contiguous(), v.flatten(0, 1).contiguous(), table, st, off)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1].view(torch.int16), b[1].view(torch.int16))
    one = moe.kv_cache(P, H, D, dev)
    moe.kv_cache_write(one, k[0], v[0], table[:1])
    got, _ = moe.kv_cache_read(one, table[:1], ends([T], dev), T)
    want, _ = moe.kv_cache_read(a, table[:1], ends([T], dev), T)
    assert torch.equal(got, want)


def test_cache_special_groups(dev):
    """Constant groups, zeros, tiny and full ranges, NaN and infinity."""
    big = torch.finfo(BF16).max
    x = torch.zeros(8, 1, 128, dtype=BF16)
    x[1, 0, :64] = 3.25
    x[2, 0, 0], x[2, 0, 1] = big, -big
    x[3, 0, 5] = 2.0 ** -133
    x[4, 0, 70] = float("nan")
    x[5, 0, 3] = float("-inf")
    x[6, 0, :64] = torch.linspace(-1e-39, 1e-39, 64).to(BF16)
    x[7, 0, :64] = (torch.arange(64) / 63 * big).to(BF16)
    cache = moe.kv_cache(1, 1, 128, dev)
    table, off = torch.zeros(1, 1, dtype=I32, device=dev), ends([8], dev)
    moe.kv_cache_write(cache, x.to(dev), x.to(dev), table)
    k, v = moe.kv_cache_read(cache, table, off, 8)
    assert torch.equal(k.view(torch.int16), v.view(torch.int16))
    got, want = f64(k)[:, 0], f64(x)[:, 0]
    assert not got[0].any() and (got[1] == want[1]).all()
    assert np.isnan(got[4, 64:]).all() and (got[4, :64] == 0).all() and np.isnan(got[5, :64]).all()
    for i in (2, 3, 6, 7):
        span = want[i, :64].max() - want[i, :64].min()
        # half a code's step, bias and scale a half step of bf16 off, also below the normal range
        assert (np.abs(got[i, :64] - want[i, :64]) <= span / 30 + span * 2.0 ** -8 * 2 + 16 * 2.0 ** -134 +
                np.abs(want[i, :64].min()) * 2.0 ** -8 + np.abs(want[i, :64]) * 2.0 ** -8).all()
        assert np.isfinite(got[i]).all()


def test_cache_bad_pages_are_skipped(dev):
    """Pages outside the cache and positions past the table are written nowhere,
    read as zeros, not attended to, and reported."""
    g = gen(6)
    H, D, N = 1, 128, 200
    k, v = normal(g, N, H, D).to(dev), normal(g, N, H, D).to(dev)
    cache = moe.kv_cache(4, H, D, dev)
    good = torch.tensor([[2, 0, 1, 3]], dtype=I32, device=dev)
    moe.kv_cache_write(cache, k, v, good)
    assert moe.moe_noalloc_status()[0] == moe.MOE_OK
    kept = [t.clone() for t in cache]
    bad = torch.tensor([[2, 4, -1]], dtype=I32, device=dev)  # the fourth page is past the table
    off = ends([N], dev)
    ref, _ = moe.kv_cache_read(cache, good, off, N)
    for call in (lambda: moe.kv_cache_write(cache, k, v, bad), lambda: moe.kv_cache_read(cache, bad, off, N)):
        got = call()
        assert moe.moe_noalloc_status()[0] == moe.MOE_ERR_DEVICE_BOUNDS
        assert moe.moe_noalloc_status()[0] == moe.MOE_OK
    assert torch.equal(got[0][:64], ref[:64]) and not got[0][64:].any()
    assert torch.equal(cache[0], kept[0]) and torch.equal(cache[1], kept[1])
    q = normal(g, 1, 4, D).to(dev)
    got = moe.attention_decode(q, cache, bad, torch.tensor([150], dtype=I32, device=dev))
    assert moe.moe_noalloc_status()[0] == moe.MOE_ERR_DEVICE_BOUNDS
    assert torch.equal(got, moe.attention_decode(q, cache, good, torch.tensor([64], dtype=I32, device=dev)))
    st = torch.tensor([-3], dtype=I32, device=dev)
    moe.kv_cache_write(cache, k[:3], v[:3], good, st)
    assert moe.moe_noalloc_status()[0] == moe.MOE_ERR_DEVICE_BOUNDS and torch.equal(cache[0], kept[0])


# ---------------------------------------------------------------- decode
def random_cache(g, P, H, D, dev):
    codes = torch.randint(0, 256, (P, 2, H, 64, D // 2), generator=g, dtype=torch.int64).to(torch.uint8)
    affine = torch.stack([torch.rand(P, 2, H, 64, D // 64, generator=g) * 0.4 + 0.05,
                          torch.randn(P, 2, H, 64, D // 64, generator=g) * 0.3 - 1.7], -1).to(BF16)
    return codes.to(dev), affine.to(dev)


def check_decode(got, q, cache, table, lens, scale):
    D, H = q.shape[-1], cache[0].shape[2]
    for i, L in enumerate(lens):
        if L == 0:
            assert not got[i].any()
            continue
        codes, affine = rows_of(cache, table, i, 0, L)
        c = [oracle.unpack(codes[:, w].numpy()) for w in (0, 1)]
        s, b = (f64(affine[..., j]) for j in (0, 1))
        k, v = (oracle.values(c[w], s[:, w], b[:, w]) for w in (0, 1))
        x = f64(q[i:i + 1])
        ref, _, reach = oracle.attend(x, k, v, scale, [0, 1], [0, L])
        step = np.repeat(s[:, 1], 64, -1)
        _, rounded, _ = oracle.attend(x, k, step * np.abs(c[1] - 8.0), scale, [0, 1], [0, L])
        _, mag, _ = oracle.attend(x, k, step * 15 + np.abs(np.repeat(b[:, 1], 64, -1)), scale, [0, 1], [0, L])
        _, _, reach = oracle.attend(x, np.repeat(s[:, 0], 64, -1) * 136 + np.abs(np.repeat(b[:, 0], 64, -1)), v, scale,
                                    [0, 1], [0, L])
        score = 2 * scale * reach * (D / 8 + 8) * 2.0 ** -23
        tol = 2.0 ** -8 * (np.abs(ref) + rounded) * (1 + 2.0 ** -6) + \
            mag * (2.0 ** -16 + (L / 16 + 64) * 2.0 ** -23 + score[..., None])
        err = np.abs(f64(got[i:i + 1]) - ref)
        assert (err <= tol).all(), (i, L, (err / tol).max())


DECODE_LENS = [[1], [2], [15], [16], [17], [63], [64], [65], [200], [1000], [0], [0, 1, 64, 0, 65, 500], [128] * 5,
               [3000], list(range(1, 60, 3)), [0, 0, 2500, 1, 1]]


@pytest.mark.parametrize("lens", DECODE_LENS, ids=lambda x: "-".join(map(str, x[:6])))
@pytest.mark.parametrize("Hq,H,D", [(16, 2, 256), (6, 2, 128)])
def test_decode(dev, lens, Hq, H, D):
    g = gen(sum(lens) + D)
    table, P = make_table(g, lens)
    cache = random_cache(g, P, H, D, dev)
    q = normal(g, len(lens), Hq, D)
    got = moe.attention_decode(q.to(dev), cache, table.to(dev), torch.tensor(lens, dtype=I32, device=dev))
    check_decode(got, q, cache, table, lens, D ** -0.5)


@pytest.mark.parametrize("Hq,H,D", [(1, 1, 256), (8, 8, 128), (3, 1, 256), (9, 1, 128), (16, 1, 256), (40, 2, 128),
                                    (10, 5, 256), (71, 1, 128)])
@pytest.mark.parametrize("lens", [[1, 130], [700]])
def test_decode_heads(dev, Hq, H, D, lens):
    g = gen(Hq + D)
    table, P = make_table(g, lens)
    cache = random_cache(g, P, H, D, dev)
    q = normal(g, len(lens), Hq, D)
    got = moe.attention_decode(q.to(dev), cache, table.to(dev), torch.tensor(lens, dtype=I32, device=dev), scale=0.1)
    check_decode(got, q, cache, table, lens, 0.1)


def test_decode_many_short_and_one_long(dev):
    g = gen(8)
    lens = [20000] + [i % 7 for i in range(300)]
    table, P = make_table(g, lens)
    cache = random_cache(g, P, 1, 128, dev)
    q = normal(g, len(lens), 8, 128)
    got = moe.attention_decode(q.to(dev), cache, table.to(dev), torch.tensor(lens, dtype=I32, device=dev))
    check_decode(got, q, cache, table, lens, 128 ** -0.5)


def test_decode_strided_queries_and_clamped_lengths(dev):
    """Queries as slices of a fused projection; lengths below zero count as 0, past
    the table as its end (reported)."""
    g = gen(9)
    lens = [100, 64, 3]
    table, P = make_table(g, lens)
    table = table.to(dev)
    cache = random_cache(g, P, 2, 128, dev)
    wide = normal(g, 3, 4 * 128 + 24).to(dev)
    q = wide[:, 16:16 + 512].unflatten(1, (4, 128))
    L = torch.tensor(lens, dtype=I32, device=dev)
    ref = moe.attention_decode(q.contiguous(), cache, table, L)
    assert torch.equal(moe.attention_decode(q, cache, table, L), ref)
    out = torch.full_like(ref, 7.0)
    assert moe.attention_decode(q, cache, table, torch.tensor([-1, 1000, 3], dtype=I32, device=dev), out=out) is out
    assert moe.moe_noalloc_status()[0] == moe.MOE_ERR_DEVICE_BOUNDS
    assert not out[0].any() and torch.equal(out[2], ref[2])
    assert torch.equal(out[1], moe.attention_decode(q, cache, table, torch.tensor([0, 128, 0], dtype=I32, device=dev))[1])


@pytest.mark.parametrize("D", [128, 256])
def test_decode_hidden_tokens_reach_nobody(dev, D):
    """NaN and infinite scales behind a sequence's end, in its last page and in
    others', change nothing; inside they reach their own heads only."""
    g = gen(D)
    lens = [70, 130]
    table, P = make_table(g, lens)
    cache = random_cache(g, P, 2, D, dev)
    q, td, L = normal(g, 2, 8, D).to(dev), table.to(dev), torch.tensor(lens, dtype=I32, device=dev)
    ref = moe.attention_decode(q, cache, td, L)
    used = torch.zeros(P, 64, dtype=torch.bool, device=dev)
    for i, n in enumerate(lens):
        at = torch.arange(n, device=dev)
        used[td[i].long()[at // 64], at % 64] = True
    for bad in (float("nan"), float("inf"), -float("inf"), torch.finfo(BF16).min):
        codes, affine = cache[0].clone(), cache[1].clone()
        affine.permute(0, 3, 1, 2, 4, 5)[~used] = bad
        assert torch.equal(moe.attention_decode(q, (codes, affine), td, L), ref)
    affine = cache[1].clone()
    affine[table[0, 0].item(), 1, 0, 9, 1, 1] = float("nan")  # values, head 0, columns 64 .. 127
    got = moe.attention_decode(q, (cache[0], affine), td, L)
    bad = torch.isnan(got)
    want = torch.zeros_like(bad)
    want[0, :4, 64:128] = True
    assert torch.equal(bad, want) and torch.equal(got[~want], ref[~want])
    affine = cache[1].clone()
    affine[table[0, 1].item(), 0, 1, 5, 0, 0] = float("nan")  # keys, head 1
    got = moe.attention_decode(q, (cache[0], affine), td, L)
    assert torch.isnan(got[0, 4:]).all() and torch.equal(got[0, :4], ref[0, :4]) and torch.equal(got[1], ref[1])


# ------------------------------------------------- a layer, streams, graphs
def test_a_layer_in_turn(dev):
    """Prompts in two pieces and new tokens through all four operators against one
    float64 pass over the quantised keys and values."""
    g = gen(21)
    Hq, Hk, D, lens, new = 8, 2, 128, [90, 1, 200], 3
    n, total = len(lens), [x + new for x in lens]
    w, f = (1 + normal(g, D, std=0.1)).to(BF16).to(dev), rope_freq(64).to(dev)
    x = [normal(g, t, (Hq + 2 * Hk), D).to(dev) for t in total]
    table, P = make_table(g, total)
    table = table.to(dev)
    cache = moe.kv_cache(P, Hk, D, dev)

    def roped(i, a, b):
        qkv = x[i][a:b]
        pos = torch.arange(a, b, dtype=I32, device=dev)
        return (*moe.qk_norm_rope(qkv[:, :Hq], qkv[:, Hq:Hq + Hk], w, w, pos, f), qkv[:, Hq + Hk:])

    outs = [[] for _ in lens]
    cuts = [x // 2 for x in lens]
    for piece in range(2):
        parts = [roped(i, 0, cuts[i]) if piece == 0 else roped(i, cuts[i], lens[i]) for i in range(n)]
        q, k, v = (torch.cat([p[j] for p in parts]) for j in range(3))
        got = [len(p[0]) for p in parts]
        st = torch.tensor([0 if piece == 0 else c for c in cuts], dtype=I32, device=dev)
        moe.kv_cache_write(cache, k, v, table, st, ends(got, dev))
        reach = cuts if piece == 0 else lens
        ke, ve = moe.kv_cache_read(cache, table, ends(reach, dev), sum(reach))
        o = moe.attention_prefill(q, ke, ve, ends(got, dev), ends(reach, dev))
        for i, p in enumerate(o.split(got)):
            outs[i].append(p)
    for t in range(new):
        parts = [roped(i, lens[i] + t, lens[i] + t + 1) for i in range(n)]
        q, k, v = (torch.stack([p[j] for p in parts]) for j in range(3))
        st = torch.tensor([x + t for x in lens], dtype=I32, device=dev)
        moe.kv_cache_write(cache, k, v, table, st)
        o = moe.attention_decode(q[:, 0], cache, table, st + 1)
        for i in range(n):
            outs[i].append(o[i:i + 1])
    for i in range(n):
        q, k, v = roped(i, 0, total[i])
        kq, vq = (oracle.values(*oracle.quantise(f64(t))) for t in (k, v))
        ref, mag, _ = oracle.attend(f64(q), kq, vq, D ** -0.5)
        # keys and values a half step of bf16 off, weights, values and result rounded
        big = np.abs(vq).max()
        score = D ** -0.5 * np.abs(f64(q)).sum(-1).max() * np.abs(kq).max() * 2.0 ** -8
        assert (np.abs(f64(torch.cat(outs[i])) - ref) <= 2.0 ** -8 * (np.abs(ref) + 3 * big) + 2 * score * big).all()
        assert np.linalg.norm(f64(torch.cat(outs[i])) - ref) <= 2.0 ** -6 * np.linalg.norm(ref)


def test_streams_and_graphs(dev):
    """The operators on another stream, and captured with new inputs at replay."""
    g = gen(22)
    Hq, Hk, D, lens = 16, 2, 256, [100, 300]
    table, P = make_table(g, [x + 1 for x in lens])
    table = table.to(dev)
    w, f = torch.ones(D, dtype=BF16, device=dev), rope_freq(64).to(dev)
    data = [normal(g, 2, Hq + 2 * Hk, D).to(dev) for _ in range(3)]
    prompt = normal(g, sum(lens), Hq + 2 * Hk, D).to(dev)
    pos = torch.tensor(lens, dtype=I32, device=dev)

    def step(x, cache, p, stream=None):
        q, k = moe.qk_norm_rope(x[:, :Hq], x[:, Hq:Hq + Hk], w, w, p, f, stream=stream)
        moe.kv_cache_write(cache, k[:, None], x[:, None, Hq + Hk:], table, p, stream=stream)
        o = moe.attention_prefill(prompt[:, :Hq], prompt[:, Hq:Hq + Hk], prompt[:, Hq + Hk:], ends(lens, dev),
                                  stream=stream)
        return q, moe.attention_decode(q, cache, table, p + 1, stream=stream), o

    cache = moe.kv_cache(P, Hk, D, dev)
    moe.kv_cache_write(cache, prompt[:, Hq:Hq + Hk], prompt[:, Hq + Hk:], table, None, ends(lens, dev))
    base = [t.clone() for t in cache]
    want = [step(x, [t.clone() for t in base], pos) for x in data]
    side = torch.cuda.Stream(dev)
    side.wait_stream(torch.cuda.current_stream(dev))
    torch.cuda.synchronize()
    p1 = pos.clone()
    with torch.cuda.stream(side):
        got = step(data[0], [t.clone() for t in base], p1)
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want[0]))
    static, e, p2 = data[0].clone(), ends(lens, dev), pos + 1

    def captured():
        q, k = moe.qk_norm_rope(static[:, :Hq], static[:, Hq:Hq + Hk], w, w, pos, f)
        moe.kv_cache_write(cache, k[:, None], static[:, None, Hq + Hk:], table, pos)
        o = moe.attention_prefill(prompt[:, :Hq], prompt[:, Hq:Hq + Hk], prompt[:, Hq + Hk:], e)
        return q, moe.attention_decode(q, cache, table, p2), o

    graphs = []
    for _ in range(2):
        side.wait_stream(torch.cuda.current_stream(dev))
        with torch.cuda.stream(side):
            captured()
        torch.cuda.current_stream(dev).wait_stream(side)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            outs = captured()
        graphs.append((graph, outs))
    for x, ref in list(zip(data, want)) * 2:
        for t, b in zip(cache, base):
            t.copy_(b)
        static.copy_(x)
        for graph, outs in graphs:
            graph.replay()
            assert all(torch.equal(a, b) for a, b in zip(outs, ref))


def test_refuses_tensors_of_other_types(dev):
    q = torch.zeros(2, 4, 128, device=dev, dtype=BF16)
    k = torch.zeros(2, 2, 128, device=dev, dtype=BF16)
    cache, pages = moe.kv_cache(2, 2, 128, dev), torch.zeros(1, 2, dtype=I32, device=dev)
    for call in (lambda: moe.attention_prefill(q.float(), k, k), lambda: moe.attention_prefill(q, k, k.half()),
                 lambda: moe.attention_prefill(q, k, k, torch.zeros(2, device=dev)),
                 lambda: moe.attention_prefill(q, k, k, out=torch.zeros(2, 4, 128, device=dev)),
                 lambda: moe.attention_decode(q, cache, pages, torch.zeros(1, dtype=I32, device=dev)),
                 lambda: moe.attention_decode(q[:1], cache, pages, torch.zeros(1, device=dev)),
                 lambda: moe.kv_cache_write(cache, k, k, pages.long()),
                 lambda: moe.kv_cache_write(cache, k[:, :1], k[:, :1], pages),
                 lambda: moe.attention_prefill(q.transpose(1, 2), k.transpose(1, 2), k.transpose(1, 2))):
        with pytest.raises(ValueError):
            call()
    with pytest.raises(moe.MoeError):
        moe.attention_prefill(q[..., :64].contiguous(), k[..., :64].contiguous(), k[..., :64].contiguous())


# ------------------------------------------------------------ further cases
@pytest.mark.parametrize("H,D,starts,lens", [(1, 128, [5, 0, 40], [9000, 1, 4000]), (3, 256, [0], [7000]),
                                             (5, 128, [0, 64], [2500, 700]), (40, 256, [3], [130])])
def test_cache_long(dev, H, D, starts, lens):
    """Blocks of several tokens, of one sequence and across the end of one."""
    test_cache_write_and_read(dev, H, D, starts, lens)


@pytest.mark.parametrize("e", [-120, -60, -9, 0, 60, 119])
def test_cache_codes_on_borders(dev, e):
    """Multiples of 2^e, many of which lie exactly between two codes (those round to
    the even one): differences, scales and those borders are exact in fp32."""
    g = gen(e + 200)
    span = torch.randint(1, 8, (300, 2, 2, 1), generator=g) * 30  # scale 2, 4, .. times 2^e
    x = (torch.rand(300, 2, 2, 64, generator=g) * (span + 1)).floor().clamp(max=span)
    x[..., :1], x[..., 1:2] = torch.zeros_like(span, dtype=x.dtype), span.to(x.dtype)
    x = ((x - (span // 2)).double() * 2.0 ** e).to(BF16).flatten(2)
    cache = moe.kv_cache(5, 2, 128, dev)
    table = torch.tensor([[4, 1, 0, 2, 3]], dtype=I32)
    moe.kv_cache_write(cache, x.to(dev), -x.to(dev), table.to(dev))
    codes, affine = rows_of(cache, table, 0, 0, 300)
    for w, y in enumerate((x, -x)):
        c, s, b = oracle.quantise(f64(y))
        assert np.array_equal(oracle.unpack(codes[:, w].numpy()), c)
        assert np.array_equal(f64(affine[:, w, ..., 0]), s) and np.array_equal(f64(affine[:, w, ..., 1]), b)


@pytest.mark.parametrize("D", [128, 256])
def test_powers_of_two_pass_through(dev, D):
    """Values times 2^j give results times 2^j; queries times 2^j with keys by 2^-j
    change nothing: no sum or part of it has a range of its own."""
    g = gen(D + 1)
    q, k, v = (x.to(dev) for x in prefill_inputs(D + 2, 200, 200, 4, 2, D))
    ref = moe.attention_prefill(q, k, v)
    lens = [150, 700]
    table, P = make_table(g, lens)
    codes, affine = random_cache(g, P, 2, D, dev)
    qd, td, L = normal(g, 2, 8, D).to(dev), table.to(dev), torch.tensor(lens, dtype=I32, device=dev)
    want = moe.attention_decode(qd, (codes, affine), td, L)
    for j in (-80, -30, 30, 80):
        f = 2.0 ** j
        assert torch.equal(moe.attention_prefill(q, k, v * f), ref * f)
        assert torch.equal(moe.attention_prefill(q * f, k / f, v), ref)
        a = affine.clone()
        a[:, 1] *= f
        assert torch.equal(moe.attention_decode(qd, (codes, a), td, L), want * f)
        a = affine.clone()
        a[:, 0] /= f
        assert torch.equal(moe.attention_decode(qd * f, (codes, a), td, L), want)


def test_prefill_dense_behind_a_prefix(dev):
    """[n][T] queries over [n][M] keys: what packed ones give; also T > M."""
    for T, M in ((33, 170), (1, 90), (90, 40)):
        q, _, _ = prefill_inputs(T, 3 * T, 1, 8, 2, 128)
        _, k, v = prefill_inputs(M, 1, 3 * M, 8, 2, 128)
        a, b, c = q.to(dev), k.to(dev), v.to(dev)
        got = moe.attention_prefill(*(x.unflatten(0, (3, -1)) for x in (a, b, c)))
        assert torch.equal(got.flatten(0, 1), moe.attention_prefill(a, b, c, ends([T] * 3, dev), ends([M] * 3, dev)))


@pytest.mark.parametrize("D,Hq", [(128, 8), (256, 16)])
def test_prefill_leaves_rows_of_no_sequence(dev, D, Hq):
    """Rows before the first and behind the last sequence, next to tiles that are not full."""
    q, k, v = (x.to(dev) for x in prefill_inputs(D, 300, 400, Hq, 2, D))
    oq = torch.tensor([7, 50, 50, 203], dtype=I32, device=dev)
    ok = torch.tensor([3, 100, 101, 390], dtype=I32, device=dev)
    out = torch.full_like(q, 7.0)
    moe.attention_prefill(q, k, v, oq, ok, out=out)
    assert (out[:7] == 7).all() and (out[203:] == 7).all()
    assert torch.equal(out[7:50], moe.attention_prefill(q[7:50], k[3:100], v[3:100]))
    assert torch.equal(out[50:203], moe.attention_prefill(q[50:203], k[101:390], v[101:390]))


def test_decode_shared_pages(dev):
    """Sequences whose first pages are the same ones, and one in the table twice."""
    g = gen(21)
    cache = random_cache(g, 9, 2, 256, dev)
    table = torch.tensor([[3, 1, 7, 0], [3, 1, 8, 2], [3, 1, 7, 0], [4, 4, 4, 4]], dtype=I32)
    lens = [250, 190, 130, 200]
    q = normal(g, 4, 16, 256)
    got = moe.attention_decode(q.to(dev), cache, table.to(dev), torch.tensor(lens, dtype=I32, device=dev))
    check_decode(got, q, cache, table, lens, 256 ** -0.5)


def test_decode_more_rows_than_shares(dev):
    g = gen(22)
    lens = torch.randint(1, 140, (700,), generator=g).tolist()
    table, P = make_table(g, lens)
    cache = random_cache(g, P, 2, 128, dev)
    q = normal(g, len(lens), 20, 128)  # 10 query heads a key/value head: rows of 8 and of 2
    got = moe.attention_decode(q.to(dev), cache, table.to(dev), torch.tensor(lens, dtype=I32, device=dev))
    check_decode(got, q, cache, table, lens, 128 ** -0.5)


def test_nothing_to_do(dev):
    e = lambda *shape: torch.zeros(*shape, dtype=BF16, device=dev)  # noqa: E731
    i = lambda *shape: torch.zeros(*shape, dtype=I32, device=dev)  # noqa: E731
    cache = moe.kv_cache(2, 2, 128, dev)
    assert moe.attention_prefill(e(0, 4, 128), e(0, 2, 128), e(0, 2, 128), i(3)).shape == (0, 4, 128)
    assert not moe.attention_prefill(e(5, 4, 128) + 1, e(0, 2, 128), e(0, 2, 128)).any()
    assert moe.attention_decode(e(0, 4, 128), cache, i(0, 3), i(0)).shape == (0, 4, 128)
    assert not moe.attention_decode(e(3, 4, 128) + 1, cache, i(3, 0), i(3)).any()
    assert moe.kv_cache_read(cache, i(0, 1), i(1), 0)[0].shape == (0, 2, 128)
    moe.kv_cache_write(cache, e(0, 2, 128), e(0, 2, 128), i(1, 2))
    assert moe.qk_norm_rope(e(0, 4, 128), e(0, 2, 128), e(128), e(128), None, None)[1].shape == (0, 2, 128)


def test_calls_at_once_on_two_streams(dev):
    """Both operators on two streams at a time: each call has its own workspace."""
    g = gen(23)
    work = []
    for i in range(2):
        lens = [3000 + 500 * i, 70, 1, 900]
        table, P = make_table(g, lens)
        cache = random_cache(g, P, 2, 256, dev)
        q, k, v = (x.to(dev) for x in prefill_inputs(30 + i, 900, 900, 16, 2, 256))
        qd = normal(g, 4, 16, 256).to(dev)
        args = (qd, cache, table.to(dev), torch.tensor(lens, dtype=I32, device=dev))
        work.append((args, (q, k, v), moe.attention_decode(*args), moe.attention_prefill(q, k, v), torch.cuda.Stream(dev)))
    torch.cuda.synchronize()
    got = [[], []]
    for _ in range(20):
        for (args, qkv, _, _, s), to in zip(work, got):
            to.append((moe.attention_decode(*args, stream=s), moe.attention_prefill(*qkv, stream=s)))
    torch.cuda.synchronize()
    for (_, _, a, b, _), to in zip(work, got):
        assert all(torch.equal(x, a) and torch.equal(y, b) for x, y in to)


@pytest.mark.parametrize("lens", [(37, 0, 130, 5), (1,), (200, 64, 63)])
def test_example_layer(dev, lens):
    """The example's decoding in a graph against attention over the cache's values
    read back: those are rounded to bf16, as are the weights of both ways and both
    results, each by 2^-8 at most (a key's roundings move a score of its size by as
    much): eight of them at most, 2^-5."""
    from examples import attention_layer
    diff, last = attention_layer.run(lens, new=4, device=dev)
    assert diff <= 2.0 ** -5
    assert last.shape == (len(lens), 512) and torch.isfinite(last).all()
