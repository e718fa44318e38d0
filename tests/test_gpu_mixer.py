"""The mixer's operators on the GPU against the float64 oracle.

Tolerances, from the arithmetic:
  * one rounding to bf16 (8 significant bits) is at most 2^-8 of the value;
  * the norm in fp32: at most ~40 sequential additions of a thread and its
    reduction, half of whose relative error reaches the norm, the reciprocal
    square root (2 ulp) and three products: under 2^-18;
  * an e4m3 code is within 2^-4 of its value relatively, or 2^-10 absolutely
    below the smallest normal, times (1 + 2^-10) for values at a tie;
  * a product summed in fp32 in pieces of 32: (K / 32 + 32) 2^-23 of the sum
    of magnitudes (a factor 2 over rounding for hardware that truncates);
  * the scan's state: fp32 sums, 1e-5 of the head's largest entry; its
    outputs 1e-2 of the row's largest value, the bar of the block's outputs.
"""
import numpy as np
import pytest
import torch

import sparse_mixture_experts_gemm_gb300 as moe
import sparse_mixture_experts_gemm_gb300.mixer as mixer_binding
from oracle import mixer

pytestmark = pytest.mark.gpu

BF16, F32, F8 = torch.bfloat16, torch.float32, torch.float8_e4m3fn
VALUES = mixer.e4m3_values()


@pytest.fixture(scope="module")
def dev():
    moe.build()
    return torch.device("cuda", 0)


def f64(t):
    return t.detach().cpu().to(torch.float64).numpy()


def codes_of(t):
    return VALUES[t.detach().cpu().view(torch.uint8).numpy()]


def gen(seed):
    g = torch.Generator()
    g.manual_seed(seed)
    return g


def normal(g, *shape, dtype=F32, std=1.0):
    return (torch.randn(shape, generator=g) * std).to(dtype)


# ------------------------------------------------------------------ norm
NORM_SHAPES = [(1, 1), (1, 8), (3, 7), (1, 2048), (5, 64), (37, 512), (4, 1001), (9, 1000), (130, 2048),
               (2, 2056), (3, 4104), (7, 8192), (2, 8200), (2, 16384), (2, 16383), (301, 264)]


def check_codes(codes, scales, y):
    """codes and scales of the float64 rows y"""
    top = np.abs(y).max(1)
    assert np.allclose(f64(scales), top / 448, rtol=2.0 ** -18, atol=0)
    r = y * np.where(top == 0, 0, 448 / np.where(top == 0, 1, top))[:, None]
    err = np.abs(codes_of(codes) - r)
    assert (err <= np.maximum(np.abs(r) * 2.0 ** -4, 2.0 ** -10) * (1 + 2.0 ** -10)).all()


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("rows,d", NORM_SHAPES)
@pytest.mark.parametrize("residual", [False, True])
def test_norm(dev, rows, d, dtype, residual):
    g = gen(rows * 10007 + d)
    x, w = normal(g, rows, d, dtype=dtype), (1 + normal(g, d, std=0.2)).to(dtype)
    r = normal(g, rows, d, dtype=dtype, std=3.0) if residual else None
    xd, wd, rd = x.to(dev), w.to(dev), None if r is None else r.to(dev)
    out, s = moe.add_rmsnorm(xd, wd, rd, eps=1e-5)
    codes, scales, s8 = moe.add_rmsnorm_fp8(xd, wd, rd, eps=1e-5)
    y, _ = mixer.rmsnorm(f64(x), f64(w), 1e-5, None if r is None else f64(r))
    unit = 2.0 ** -18 + (2.0 ** -8 if dtype == BF16 else 0)
    assert (np.abs(f64(out) - y) <= np.abs(y) * unit + 1e-30).all()
    check_codes(codes, scales, y)
    if residual:
        want = (x.float() + r.float()).to(dtype)
        assert torch.equal(s.cpu(), want) and torch.equal(s8.cpu(), want)
    else:
        assert s is None and s8 is None


def test_norm_strided_rows_and_in_place(dev):
    """Rows of a wider tensor, also at an offset off the 16-byte boundary; the
    sum over the residual, the output over x."""
    g = gen(5)
    wide, w = normal(g, 33, 700, dtype=BF16).to(dev), normal(g, 256, dtype=BF16).to(dev)
    r = normal(g, 33, 256, dtype=BF16).to(dev)
    for at in (0, 8, 3):
        x = wide[:, at:at + 256]
        ref, ref_s = moe.add_rmsnorm(x.contiguous(), w, r)
        out, s = moe.add_rmsnorm(x, w, r)
        assert torch.equal(out, ref) and torch.equal(s, ref_s)
        c = moe.add_rmsnorm_fp8(x, w, r)
        c_ref = moe.add_rmsnorm_fp8(x.contiguous(), w, r)
        assert torch.equal(c[0].view(torch.uint8), c_ref[0].view(torch.uint8)) and torch.equal(c[1], c_ref[1])
        # the residual itself as a slice, and both in place
        r2, x2 = r.clone(), x.contiguous()
        out, s = moe.add_rmsnorm(x2, w, r2, sum_out=r2, out=x2)
        assert s is r2 and torch.equal(r2, ref_s) and torch.equal(x2, ref)


def test_norm_special_rows(dev):
    """Zeros, one huge value, tiny values, NaN, infinity; their neighbours
    are untouched."""
    d = 256
    x = torch.ones(7, d)
    x[0] = 0
    x[1] = 0
    x[1, 7] = 1e18
    x[2] *= 1e-30
    x[3, 5] = float("nan")
    x[4, 200] = float("inf")
    x[5] *= 1e-38
    w = torch.ones(d)
    codes, scales, _ = moe.add_rmsnorm_fp8(x.to(dev), w.to(dev), eps=1e-6)
    c, s = codes_of(codes), f64(scales)
    assert s[0] == 0 and not c[0].any()
    assert c[1, 7] == 448 and not np.delete(c[1], 7).any()
    for i in (3, 4):
        assert np.isnan(s[i]) and np.isnan(c[i]).all()
    for i in (2, 6):
        assert (c[i] == 448).all() and s[i] > 0
    y, _ = mixer.rmsnorm(x.numpy()[[2, 6]], w.numpy(), 1e-6)
    assert np.allclose(s[[2, 6]], y.max(1) / 448, rtol=1e-5)
    assert not np.isnan(c[5]).any() and (c[5] == c[5][0]).all()
    q, qs = moe.quantize_fp8(x.to(dev))
    c, s = codes_of(q), f64(qs)
    assert s[0] == 0 and not c[0].any() and (c[6] == 448).all() and abs(s[6] - 1 / 448) < 1e-9
    assert (c[2] == 448).all() and np.isnan(s[3]) and np.isnan(s[4]) and np.isnan(c[4]).all()


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("d", [7, 256, 2048, 16384])
def test_norm_zero_rows_without_eps(dev, d, dtype):
    """eps may be 0: a row of zeros gives zeros, scale 0 and zero codes, by
    itself and as the sum of two rows that cancel."""
    g = gen(d)
    x, w = normal(g, 3, d, dtype=dtype), (1 + normal(g, d, std=0.2)).to(dtype)
    x[1] = 0
    r = torch.zeros_like(x)
    r[2] = -x[2]
    out, s = moe.add_rmsnorm(x.to(dev), w.to(dev), r.to(dev), eps=0.0)
    codes, scales, _ = moe.add_rmsnorm_fp8(x.to(dev), w.to(dev), r.to(dev), eps=0.0)
    assert not out[1:].any() and not s[1:].any() and not scales[1:].any() and not codes[1:].float().any()
    y, _ = mixer.rmsnorm(f64(x[:1]), f64(w), 0.0)
    unit = 2.0 ** -18 + (2.0 ** -8 if dtype == BF16 else 0)
    assert (np.abs(f64(out[:1]) - y) <= np.abs(y) * unit + 1e-30).all()
    check_codes(codes[:1], scales[:1], y)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("d", [7, 256, 1001, 2048, 16384])
@pytest.mark.parametrize("eps", [1e-6, 0.0])
def test_norm_rows_whose_squares_leave_the_range(dev, d, dtype, eps):
    """Finite rows of 1e18 to 1e38 have their norm, with one large element or
    with all of them; without eps so have rows of 1e-18 to 1e-36, where a product
    s w below 2^-126 is off by up to 2^-150.  Weights of 1/2 to 1, so that none
    exceeds the range."""
    g = gen(d + 1)
    sizes = [1e18, 2e19, 1e20, 1e30, 5e37] + ([1e-18, 1e-20, 1e-30, 1e-36] if eps == 0 else [])
    x = normal(g, 2 * len(sizes), d).clamp(-5, 5)
    for i, size in enumerate(sizes):
        x[2 * i] *= size
        x[2 * i + 1, 1:] *= size * 1e-3
        x[2 * i + 1, 0] = 3 * size
    x, w = x.to(dtype), (1 - torch.rand(d, generator=g) / 2).to(dtype)
    assert torch.isfinite(x).all()
    y, _ = mixer.rmsnorm(f64(x), f64(w), eps)
    out, _ = moe.add_rmsnorm(x.to(dev), w.to(dev), eps=eps)
    codes, scales, _ = moe.add_rmsnorm_fp8(x.to(dev), w.to(dev), eps=eps)
    unit = 2.0 ** -18 + (2.0 ** -8 if dtype == BF16 else 0)
    under = 2.0 ** -149 / np.sqrt((f64(x) ** 2).mean(1, keepdims=True) + eps)
    assert (np.abs(f64(out) - y) <= np.abs(y) * unit + under + 1e-30).all()
    check_codes(codes, scales, y)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("d", [7, 264, 2048])
def test_codes_go_by_the_scale_that_is_returned(dev, d, dtype):
    """Rows so small that their scale is one of float32's last values, which
    round max / 448 by up to half: scale * code is still y (the code within 2^-4
    of y / scale, or 2^-10 below the smallest normal code; past 448, where the
    scale was rounded down, 448)."""
    g = gen(d)
    x = normal(g, 12, d).clamp(-3, 3)
    for i in range(12):
        x[i] *= 3e-37 * 4.0 ** -i
    x = x.to(dtype)
    codes, scales = moe.quantize_fp8(x.to(dev))
    c, s, y = codes_of(codes), f64(scales), f64(x)
    top = np.abs(y).max(1)
    assert (np.abs(s - top / 448) <= np.maximum(top / 448 * 2.0 ** -23, 2.0 ** -150)).all()
    live = s > 0
    assert live.sum() >= 8 and not c[~live].any()
    r = np.clip(y[live] / s[live, None], -448, 448)
    assert (np.abs(c[live] - r) <= np.maximum(np.abs(r) * 2.0 ** -4, 2.0 ** -10) * (1 + 2.0 ** -10)).all()


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("rows,d", [(1, 16), (5, 33), (200, 2048), (3, 16384)])
def test_quantize(dev, rows, d, dtype):
    w = normal(gen(d), rows, d, dtype=dtype, std=0.02)
    codes, scales = moe.quantize_fp8(w.to(dev))
    check_codes(codes, scales, f64(w))
    # rows of every other stride
    wide = normal(gen(d), rows, 2 * d, dtype=dtype).to(dev)
    a, b = moe.quantize_fp8(wide[:, d:]), moe.quantize_fp8(wide[:, d:].contiguous())
    assert torch.equal(a[0].view(torch.uint8), b[0].view(torch.uint8)) and torch.equal(a[1], b[1])


# ---------------------------------------------------------------- matmul
def make_matmul(seed, T, N, K, dev):
    g = gen(seed)
    x, xs = moe.quantize_fp8(normal(g, T, K).to(dev)) if T else (torch.empty(0, K, dtype=F8, device=dev),
                                                                 torch.empty(0, device=dev))
    w, ws = moe.quantize_fp8(normal(g, N, K, std=K ** -0.5).to(dev))
    return x, xs, w, ws


def check_matmul(out, x, xs, w, ws):
    X, W = codes_of(x), codes_of(w)
    ref = mixer.matmul(X, f64(xs), W, f64(ws))
    mag = mixer.matmul(np.abs(X), f64(xs), np.abs(W), f64(ws))
    K = X.shape[1]
    assert (np.abs(f64(out) - ref) <= np.abs(ref) * 2.0 ** -8 + mag * (K / 32 + 32) * 2.0 ** -23).all()


@pytest.mark.parametrize("T,N,K", [
    (1, 1, 16), (1, 8192, 2048), (2, 130, 48), (3, 2048, 4096), (8, 64, 128), (15, 127, 272),
    (16, 2048, 4096), (17, 513, 512), (31, 256, 2064), (33, 1000, 1040), (64, 129, 256), (65, 2500, 2048),
    (100, 16, 4096), (128, 128, 128), (129, 255, 144), (250, 777, 2000), (301, 2500, 2048),
    (512, 1024, 16), (513, 4100, 640), (1100, 2300, 1024), (2500, 511, 272), (2048, 2048, 2048),
])
def test_matmul(dev, T, N, K):
    a = make_matmul(T + N + K, T, N, K, dev)
    check_matmul(moe.matmul_fp8(*a), *a)


def test_matmul_wide_k(dev):
    """K past what moe_quantize_fp8 takes: the codes are drawn directly."""
    T, N, K = 40, 96, 131072
    g = gen(3)

    def drawn(rows, std):
        c = (normal(g, rows, K) * 100).clamp(-448, 448).to(F8)
        return c.to(dev), (torch.rand(rows, generator=g) * std).to(dev)

    a = (*drawn(T, 1.0), *drawn(N, K ** -0.5))
    check_matmul(moe.matmul_fp8(*a), *a)


@pytest.mark.parametrize("T", [1, 5, 40, 200, 700])
def test_matmul_strides_and_guards(dev, T):
    """Strided x, w and out; what lies between out's rows stays as it was."""
    N, K = 333, 208
    x, xs, w, ws = make_matmul(T, T, N, K, dev)
    ref = moe.matmul_fp8(x, xs, w, ws)
    X = torch.zeros(T, 512, dtype=torch.uint8, device=dev).fill_(0x7f).view(F8)
    W = torch.zeros(N, 304, dtype=torch.uint8, device=dev).fill_(0x7f).view(F8)
    X[:, 16:16 + K], W[:, 32:32 + K] = x, w
    out = torch.full((T + 2, 401), 7.0, dtype=BF16, device=dev)
    got = moe.matmul_fp8(X[:, 16:16 + K], xs, W[:, 32:32 + K], ws, out=out[1:T + 1, 5:5 + N])
    assert torch.equal(got, ref)
    out[1:T + 1, 5:5 + N] = 7.0
    assert (out == 7.0).all()


def test_matmul_is_repeatable_and_empty(dev):
    for T in (1, 16, 300, 2000):
        a = make_matmul(9, T, 1030, 2048, dev)
        first = moe.matmul_fp8(*a)
        for _ in range(5):
            assert torch.equal(moe.matmul_fp8(*a), first)
    a = make_matmul(9, 0, 64, 64, dev)
    assert moe.matmul_fp8(*a).shape == (0, 64)


def test_matmul_nan_stays_in_its_row(dev):
    x, xs, w, ws = make_matmul(4, 20, 300, 256, dev)
    x.view(torch.uint8)[3, 17] = 0x7f
    w.view(torch.uint8)[200, 5] = 0xff
    out = f64(moe.matmul_fp8(x, xs, w, ws))
    bad = np.isnan(out)
    want = np.zeros_like(bad)
    want[3], want[:, 200] = True, True
    assert np.array_equal(bad, want)


# ------------------------------------------------------------------ scan
O_TOL, S_TOL = 1e-2, 1e-5


def scan_inputs(seed, N, n, Hk, Hv, dk, dv, state=True):
    g = gen(seed)
    q = normal(g, N, Hk, dk, std=1 / dk)
    k = normal(g, N, Hk, dk, std=dk ** -0.5)
    v = normal(g, N, Hv, dv)
    decay = 1 - torch.exp(-torch.rand(Hv, generator=g) * 7)
    s = normal(g, n, Hv, dv, dk, std=0.1) if state else None
    return q.to(BF16), k.to(BF16), v.to(BF16), decay, s


def check_scan(o, S, q, k, v, decay, s, offsets):
    ro, rs = mixer.decay_scan(f64(q), f64(k), f64(v), f64(decay), None if s is None else f64(s), offsets)
    o, S = f64(o), f64(S).reshape(rs.shape)
    assert np.isfinite(o).all() and np.isfinite(S).all()
    if o.size:
        oe = np.abs(o - ro).max(2) / np.maximum(np.abs(ro).max(2), 1e-30)
        assert oe.max() <= O_TOL, oe.max()
    if S.size:
        se = np.abs(S - rs).max((2, 3)) / np.maximum(np.abs(rs).max((2, 3)), 1e-30)
        assert se.max() <= S_TOL, se.max()


SCAN_LENS = [[1], [2], [7], [63], [64], [65], [128], [129], [300], [1000], [1] * 9, [2] * 5, [17] * 3,
             [200] * 2, [1, 0, 5], [0, 0], [0, 130, 1, 64, 0, 257], [700, 3], [9, 8, 7, 6, 5, 4]]


@pytest.mark.parametrize("lens", SCAN_LENS, ids=lambda x: "-".join(map(str, x)))
@pytest.mark.parametrize("Hk,Hv,dk,dv", [(2, 4, 128, 128), (1, 3, 64, 80)])
def test_scan(dev, lens, Hk, Hv, dk, dv):
    n, N = len(lens), sum(lens)
    q, k, v, decay, s = scan_inputs(N + n, N, n, Hk, Hv, dk, dv)
    off = torch.tensor([0] + lens).cumsum(0).to(torch.int32)
    o, S = moe.gdn_decay_scan(q.to(dev), k.to(dev), v.to(dev), decay.to(dev), s.to(dev), off.to(dev))
    check_scan(o, S, q, k, v, decay, s, off)
    if len(set(lens)) == 1 and N:  # the same as a dense batch, from zero states
        d4 = [x.to(dev).unflatten(0, (n, lens[0])) for x in (q, k, v)]
        o, S = moe.gdn_decay_scan(*d4, decay.to(dev))
        check_scan(o.flatten(0, 1), S, q, k, v, decay, None, off)


@pytest.mark.parametrize("Hk,Hv,dk,dv", [(1, 1, 64, 16), (1, 8, 128, 32), (4, 4, 64, 256), (2, 2, 128, 144),
                                         (16, 32, 128, 128), (1, 1, 128, 1024)])
@pytest.mark.parametrize("N", [1, 3, 150])
def test_scan_heads(dev, Hk, Hv, dk, dv, N):
    q, k, v, decay, s = scan_inputs(N, N, 1, Hk, Hv, dk, dv)
    o, S = moe.gdn_decay_scan(q.to(dev), k.to(dev), v.to(dev), decay.to(dev), s[0].to(dev))
    check_scan(o, S, q, k, v, decay, s, [0, N])


@pytest.mark.parametrize("N", [1, 5, 400])
def test_scan_extreme_decays(dev, N):
    """Decays of 0 (the state holds one token), 1 (a plain sum), tiny and
    nearly 1."""
    q, k, v, _, s = scan_inputs(N, N, 1, 1, 6, 128, 64)
    decay = torch.tensor([0.0, 1.0, 1e-20, 0.5, 1 - 2.0 ** -24, 1e-42])
    o, S = moe.gdn_decay_scan(q.to(dev), k.to(dev), v.to(dev), decay.to(dev), s[0].to(dev))
    check_scan(o, S, q, k, v, decay, s, [0, N])


def test_scan_full_size(dev):
    """2,048 tokens, 16 key heads, 32 value heads of 128 (every output)."""
    q, k, v, decay, s = scan_inputs(7, 2048, 1, 16, 32, 128, 128)
    o, S = moe.gdn_decay_scan(q.to(dev), k.to(dev), v.to(dev), decay.to(dev), s[0].to(dev))
    check_scan(o, S, q, k, v, decay, s, [0, 2048])


def test_scan_long(dev):
    """20,000 tokens through one head with a long memory."""
    q, k, v, _, s = scan_inputs(8, 20000, 1, 1, 2, 64, 16)
    decay = torch.tensor([0.9999, 0.99])
    o, S = moe.gdn_decay_scan(q.to(dev), k.to(dev), v.to(dev), decay.to(dev), s[0].to(dev))
    check_scan(o, S, q, k, v, decay, s, [0, 20000])


@pytest.mark.parametrize("cut", [1, 64, 100, 256, 399])
def test_scan_in_pieces(dev, cut):
    q, k, v, decay, s = scan_inputs(9, 400, 1, 2, 4, 128, 128)
    q, k, v, decay, s = (x.to(dev) for x in (q, k, v, decay, s))
    st = s[0].clone()
    o1, _ = moe.gdn_decay_scan(q[:cut], k[:cut], v[:cut], decay, st, state_out=st)
    o2, _ = moe.gdn_decay_scan(q[cut:], k[cut:], v[cut:], decay, st, state_out=st)
    check_scan(torch.cat([o1, o2]), st, q, k, v, decay, s, [0, 400])


@pytest.mark.parametrize("n,T", [(6, 1), (1, 6), (2, 300)])
def test_scan_slices_of_a_fused_projection(dev, n, T):
    Hk, Hv, dk, dv = 2, 4, 128, 64
    q, k, v, decay, s = scan_inputs(11, n * T, n, Hk, Hv, dk, dv)
    a, b = Hk * dk, 2 * Hk * dk
    qkv = torch.cat([x.flatten(1) for x in (q, k, v)], 1).to(dev).unflatten(0, (n, T))
    o, S = moe.gdn_decay_scan(qkv[..., :a].unflatten(-1, (Hk, dk)), qkv[..., a:b].unflatten(-1, (Hk, dk)),
                              qkv[..., b:].unflatten(-1, (Hv, dv)), decay.to(dev), s.to(dev))
    check_scan(o.flatten(0, 1), S, q, k, v, decay, s, [T * i for i in range(n + 1)])


def test_scan_bad_offsets_stay_in_bounds(dev):
    """Offsets past the end or running backwards are clamped: nothing is
    read or written outside, and well-formed sequences keep their results."""
    q, k, v, decay, s = (x.to(dev) for x in scan_inputs(12, 200, 4, 1, 2, 128, 64))
    off = torch.tensor([0, 90, 50, 1 << 30, -5], dtype=torch.int32, device=dev)
    o, S = moe.gdn_decay_scan(q, k, v, decay, s, off)
    torch.cuda.synchronize()
    ref, Sr = moe.gdn_decay_scan(q[:90], k[:90], v[:90], decay, s[0])
    check_scan(ref, S[0], q[:90], k[:90], v[:90], decay, s[:1], [0, 90])
    assert torch.isfinite(S).all() and torch.equal(S[1], s[1])


# ------------------------------------------------------------- streams
def test_scan_packed_long_sequence_is_cut(dev):
    """One sequence outlasts its batch and is scanned in segments, between
    empty and short ones; also with the state updated in place."""
    lens = [5, 9000, 0, 130]
    q, k, v, decay, s = scan_inputs(13, sum(lens), 4, 1, 2, 128, 80)
    decay[1] = 0.999
    off = torch.tensor([0] + lens).cumsum(0).to(torch.int32)
    qd, kd, vd, dd, sd = (x.to(dev) for x in (q, k, v, decay, s))
    o, S = moe.gdn_decay_scan(qd, kd, vd, dd, sd, off.to(dev))
    check_scan(o, S, q, k, v, decay, s, off)
    o2, _ = moe.gdn_decay_scan(qd, kd, vd, dd, sd, off.to(dev), state_out=sd)
    assert torch.equal(o, o2) and torch.equal(S, sd)


def test_scan_shares(dev):
    """Heads that are cut into one share per SM, whichever head ends inside it:
    every output, and the state in place or not.  An output's three roundings to
    bf16 (state, scores, result) are each within 2^-8 of their terms, whose
    magnitudes the scan of the magnitudes adds up."""
    q, k, v, decay, s = scan_inputs(18, 3001, 1, 13, 52, 128, 64)
    qd, kd, vd, dd, sd = (x.to(dev) for x in (q, k, v, decay, s[0]))
    o, S = moe.gdn_decay_scan(qd, kd, vd, dd, sd)
    ro, rs = mixer.decay_scan(f64(q), f64(k), f64(v), f64(decay), f64(s))
    terms, _ = mixer.decay_scan(*(np.abs(f64(x)) for x in (q, k, v)), f64(decay), np.abs(f64(s)))
    assert (np.abs(f64(o) - ro) <= 2.0 ** -8 * (np.abs(ro) + terms) * (1 + 2.0 ** -6)).all()
    assert np.linalg.norm(f64(o) - ro) <= 2.0 ** -8 * np.linalg.norm(ro)
    assert (np.abs(f64(S) - rs[0]).max((1, 2)) <= S_TOL * np.abs(rs[0]).max((1, 2))).all()
    o2, _ = moe.gdn_decay_scan(qd, kd, vd, dd, sd, state_out=sd)
    assert torch.equal(o, o2) and torch.equal(S, sd)


@pytest.mark.parametrize("lens", [[1, 700, 0, 2049, 37, 1311, 64, 300, 999], [2900], [17, 2100, 16, 1800, 1700]])
def test_scan_packed_and_cut_within_the_bound(dev, lens):
    """Packed sequences of few heads, cut where SMs are idle: every output within
    the bound of test_scan_shares."""
    q, k, v, decay, s = scan_inputs(23, sum(lens), len(lens), 2, 4, 128, 128)
    off = torch.tensor([0] + lens).cumsum(0).to(torch.int32)
    assert mixer_binding._decay_workspace(sum(lens), len(lens), True, 4, 128, 128) >= 4 * 128 * 128 * 4
    o, S = moe.gdn_decay_scan(*(x.to(dev) for x in (q, k, v, decay, s, off)))
    ro, rs = mixer.decay_scan(f64(q), f64(k), f64(v), f64(decay), f64(s), off)
    terms, _ = mixer.decay_scan(*(np.abs(f64(x)) for x in (q, k, v)), f64(decay), np.abs(f64(s)), off)
    assert (np.abs(f64(o) - ro) <= 2.0 ** -8 * (np.abs(ro) + terms) * (1 + 2.0 ** -6)).all()
    assert np.linalg.norm(f64(o) - ro) <= 2.0 ** -8 * np.linalg.norm(ro)
    assert (np.abs(f64(S) - rs).max((2, 3)) <= S_TOL * np.abs(rs).max((2, 3))).all()


@pytest.mark.parametrize("T,Hk,Hv,dv", [(4800, 10, 30, 256), (6401, 6, 60, 80), (10001, 16, 32, 128)])
def test_scan_shares_in_pieces(dev, T, Hk, Hv, dv):
    """One call against short ones that pass the state along."""
    q, k, v, decay, s = (x.to(dev) for x in scan_inputs(19, T, 1, Hk, Hv, 128, dv))
    o, S = moe.gdn_decay_scan(q, k, v, decay, s[0])
    st, parts = s[0].clone(), []
    for a in range(0, T, 600):
        parts.append(moe.gdn_decay_scan(q[a:a + 600], k[a:a + 600], v[a:a + 600], decay, st, state_out=st)[0])
    both = torch.cat(parts).float()
    # both are within the bound of test_scan_shares; without cancellation the
    # kernel gives the terms' magnitudes to 3 x 2^-8
    terms, _ = moe.gdn_decay_scan(q.abs(), k.abs(), v.abs(), decay, s[0].abs())
    bound = 2.0 ** -8 * (both.abs() + terms.float()) * (1 + 2.0 ** -5)
    assert ((o.float() - both).abs() <= 2 * bound).all()
    assert (o.float() - both).norm() <= 2 * 2.0 ** -8 * both.norm()
    assert ((S - st).abs().amax((1, 2)) <= 2 * S_TOL * st.abs().amax((1, 2))).all()


@pytest.mark.parametrize("n,T", [(1, 1), (3, 8), (1, 2000), (3, 700)])
def test_scan_in_place(dev, n, T):
    """Writing the state over the initial one changes no bit."""
    q, k, v, decay, s = (x.to(dev) for x in scan_inputs(14, n * T, n, 1, 2, 128, 144))
    q, k, v = (x.unflatten(0, (n, T)) for x in (q, k, v))
    o, S = moe.gdn_decay_scan(q, k, v, decay, s)
    o2, _ = moe.gdn_decay_scan(q, k, v, decay, s, state_out=s)
    assert torch.equal(o, o2) and torch.equal(S, s)


def test_scan_many_packed_sequences(dev):
    """More sequences than a block has threads, of every kind."""
    lens = [(7 * i) % 23 if i % 3 else 64 * (i % 5) + i % 2 for i in range(700)]
    q, k, v, decay, s = scan_inputs(15, sum(lens), 700, 1, 1, 64, 16)
    off = torch.tensor([0] + lens).cumsum(0).to(torch.int32)
    o, S = moe.gdn_decay_scan(*(x.to(dev) for x in (q, k, v, decay, s, off)))
    check_scan(o, S, q, k, v, decay, s, off)


def test_scan_several_cut_among_many(dev):
    """Decode tokens, short and long prompts in one call: only the longest are
    cut, and their segments stand apart from the others in the call's table."""
    lens = [1] * 50 + [5000] + [3] * 30 + [40] * 200 + [9000, 0, 17, 4097] + [16, 18] * 20
    q, k, v, decay, s = scan_inputs(20, sum(lens), len(lens), 1, 2, 64, 32)
    decay[1] = 0.9995
    off = torch.tensor([0] + lens).cumsum(0).to(torch.int32)
    qd, kd, vd, dd, sd, od = (x.to(dev) for x in (q, k, v, decay, s, off))
    o, S = moe.gdn_decay_scan(qd, kd, vd, dd, sd, od)
    check_scan(o, S, q, k, v, decay, s, off)
    o2, _ = moe.gdn_decay_scan(qd, kd, vd, dd, sd, od, state_out=sd)
    assert torch.equal(o, o2) and torch.equal(S, sd)


@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
def test_scan_nan_stays_in_its_sequence(dev, bad):
    """Sequences around one of NaN or infinite q, k, v and state: no bit of
    theirs changes."""
    lens = [70, 3, 100, 130, 2, 64]
    q, k, v, decay, s = (x.to(dev) for x in scan_inputs(16, sum(lens), len(lens), 1, 2, 128, 64))
    off = torch.tensor([0] + lens).cumsum(0).to(torch.int32).to(dev)
    o, S = moe.gdn_decay_scan(q, k, v, decay, s, off)
    for i in (1, 2, 4):
        lo, hi = int(off[i]), int(off[i + 1])
        x = [t.clone() for t in (q, k, v, s)]
        for t in x[:3]:
            t[lo:hi] = bad
        x[3][i] = bad
        o2, S2 = moe.gdn_decay_scan(x[0], x[1], x[2], decay, x[3], off)
        keep = [j for j in range(len(lens)) if j != i]
        assert torch.equal(S2[keep], S[keep])
        assert torch.equal(o2[:lo], o[:lo]) and torch.equal(o2[hi:], o[hi:])
        assert not torch.isfinite(S2[i]).any()


@pytest.mark.parametrize("bad", [float("nan"), float("-inf")])
@pytest.mark.parametrize("T,at", [(8, 3), (300, 0), (300, 100), (300, 128), (300, 299), (3000, 2000)])
def test_scan_nan_reaches_no_earlier_token(dev, T, at, bad):
    """A value that is not finite in one column of one token: the tokens
    before it and the other columns keep the oracle's results; from it on the
    column has none."""
    q, k, v, decay, s = scan_inputs(17, T, 1, 1, 2, 128, 80)
    decay[0] = 0.0
    clean = mixer.decay_scan(f64(q), f64(k), f64(v), f64(decay), f64(s))
    vb = v.clone()
    vb[at, :, 37] = bad
    vb[at + (T - at) // 2, 0, 41] = bad
    o, S = moe.gdn_decay_scan(q.to(dev), k.to(dev), vb.to(dev), decay.to(dev), s[0].to(dev))
    o, S = f64(o), f64(S)
    hidden = np.zeros(o.shape, bool)
    hidden[at:, :, 37] = True
    hidden[at + (T - at) // 2:, 0, 41] = True
    assert not np.isfinite(o[hidden]).any() and np.isfinite(o[~hidden]).all()
    top = np.maximum(np.abs(clean[0]).max(2, keepdims=True), 1e-30)
    assert (np.where(hidden, 0, np.abs(o - clean[0])) / top).max() <= O_TOL
    rows = np.ones(S.shape[:2], bool)
    rows[:, 37] = False
    rows[0, 41] = False
    assert not np.isfinite(S[~rows]).any()
    err = np.abs(S - clean[1].reshape(S.shape))[rows]
    assert err.max() <= S_TOL * np.abs(clean[1]).max()


@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
@pytest.mark.parametrize("T,at", [(8, 3), (300, 100), (300, 130), (3000, 2000)])
def test_scan_nan_in_k_or_q_reaches_no_earlier_token(dev, T, at, bad):
    """No bit of the outputs before the token changes; one in q changes no other
    token's outputs and no state either."""
    q, k, v, decay, s = (x.to(dev) for x in scan_inputs(22, T, 1, 1, 2, 128, 80))
    o, S = moe.gdn_decay_scan(q, k, v, decay, s[0])
    kb, qb = k.clone(), q.clone()
    kb[at, 0, 5], qb[at, 0, 5] = bad, bad
    o2, S2 = moe.gdn_decay_scan(q, kb, v, decay, s[0])
    assert torch.equal(o2[:at], o[:at]) and not torch.isfinite(S2[..., 5]).any()
    o3, S3 = moe.gdn_decay_scan(qb, k, v, decay, s[0])
    rest = [t for t in range(T) if t != at]
    assert torch.equal(o3[rest], o[rest]) and torch.equal(S3, S) and not torch.isfinite(o3[at]).any()


def test_other_stream(dev):
    """Each operator on a stream that is not the current one, results read
    there; and captured in a CUDA graph on it."""
    side = torch.cuda.Stream()
    x = normal(gen(1), 50, 256, dtype=BF16).to(dev)
    wn = torch.ones(256, dtype=BF16, device=dev)
    w, ws = moe.quantize_fp8(normal(gen(2), 512, 256).to(dev))
    decay = torch.tensor([0.9], device=dev)
    torch.cuda.synchronize()

    def layer(stream=None):
        c, sc, _ = moe.add_rmsnorm_fp8(x, wn, stream=stream)
        y = moe.matmul_fp8(c, sc, w, ws, stream=stream)
        q, k, v = (y[:, 128 * i:128 * (i + 1)].unflatten(1, (1, 128)) for i in range(3))
        return moe.gdn_decay_scan(q, k, v, decay, stream=stream)

    ref = layer()
    got = layer(side)
    got2 = layer(side.cuda_stream)
    side.synchronize()
    for a, b in ((got, ref), (got2, ref)):
        assert all(torch.equal(u, v) for u, v in zip(a, b))
    with torch.cuda.stream(side):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=side):
            cap = layer()
    cap[0].zero_()
    x_old = x.clone()
    x.copy_(x_old)
    g.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(u, v) for u, v in zip(cap, ref))


@pytest.mark.parametrize("packed", [False, True])
def test_segmented_scan_on_another_stream_and_in_a_graph(dev, packed):
    """A scan with a workspace and three or four launches, on a stream that is
    not the current one (given as an object and as a handle) and captured; the
    workspace's memory is handed on to other tensors of that stream meanwhile."""
    lens = [5, 2900, 0, 130, 1] if packed else [1500, 1500]
    q, k, v, decay, s = (x.to(dev) for x in scan_inputs(21, sum(lens), len(lens), 2, 4, 128, 128))
    off = torch.tensor([0] + lens).cumsum(0).to(torch.int32).to(dev) if packed else None
    if not packed:
        q, k, v = (x.unflatten(0, (2, 1500)) for x in (q, k, v))
    need = mixer_binding._decay_workspace(sum(lens), len(lens), packed, 4, 128, 128)
    assert need >= 4 * 128 * 128 * 4  # (it is cut)
    ref = moe.gdn_decay_scan(q, k, v, decay, s, off)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    got = []
    for stream in (side, side.cuda_stream):
        got.append(moe.gdn_decay_scan(q, k, v, decay, s, off, stream=stream))
        with torch.cuda.stream(side):
            torch.empty(need, dtype=torch.uint8, device=dev).fill_(0xff)
    side.synchronize()
    with torch.cuda.stream(side):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=side):
            cap = moe.gdn_decay_scan(q, k, v, decay, s, off)
    for _ in range(3):
        cap[0].zero_()
        cap[1].zero_()
        g.replay()
        torch.cuda.synchronize()
        got.append(tuple(x.clone() for x in cap))
    for o, S in got:
        assert torch.equal(o, ref[0]) and torch.equal(S, ref[1])


@pytest.mark.parametrize("lens", [(37, 0, 130, 5), (1,), (200, 64, 63)])
def test_example_layer(dev, lens):
    """The example's decoding in a graph against one pass.  Codes of nearly
    equal rows differ by at most the rounding of both: rms 2^-4 / sqrt(3)
    each, 5e-2 together; the states see bf16 roundings of k and v, 2^-8 each."""
    from examples import hybrid_layer
    diff, sdiff, last = hybrid_layer.run(lens, new=4, device=dev)
    assert diff <= 5e-2 and sdiff <= 2.0 ** -7
    assert last.shape == (len(lens), 512) and torch.isfinite(last).all()


def test_binding_refusals(dev):
    x = torch.zeros(4, 64, dtype=BF16, device=dev)
    w = torch.ones(64, dtype=BF16, device=dev)
    with pytest.raises(ValueError):
        moe.add_rmsnorm(x, w[:32])
    with pytest.raises(ValueError):
        moe.add_rmsnorm(x.half(), w.half())
    with pytest.raises(ValueError):
        moe.add_rmsnorm(x, w, residual=x[:2])
    with pytest.raises(ValueError):
        moe.add_rmsnorm(x.t(), torch.ones(4, dtype=BF16, device=dev))
    with pytest.raises(ValueError):
        moe.add_rmsnorm(x.cpu(), w)
    with pytest.raises(ValueError):
        moe.add_rmsnorm_fp8(x, w, codes=torch.empty(4, 64, device=dev))
    c, s = moe.quantize_fp8(x)
    with pytest.raises(ValueError):
        moe.matmul_fp8(c, s, c[:, :32], s)
    with pytest.raises(ValueError):
        moe.matmul_fp8(c, s[:2], c, s)
    with pytest.raises(ValueError):
        moe.matmul_fp8(x, s, c, s)
    with pytest.raises(moe.MoeError):
        moe.matmul_fp8(c[:, :24], s, c[:, :24], s)
    q = torch.zeros(4, 2, 64, dtype=BF16, device=dev)
    d = torch.ones(2, device=dev)
    with pytest.raises(ValueError):
        moe.gdn_decay_scan(q, q[:3], q, d)
    with pytest.raises(ValueError):
        moe.gdn_decay_scan(q, q, q, d[:1])
    with pytest.raises(ValueError):
        moe.gdn_decay_scan(q, q, q, d, state=torch.zeros(2, 64, 64, dtype=BF16, device=dev))
    with pytest.raises(ValueError):
        moe.gdn_decay_scan(q, q, q, d, offsets=torch.zeros(2, dtype=torch.int64, device=dev))
    with pytest.raises(ValueError):
        moe.gdn_decay_scan(q[None], q[None], q[None], d, offsets=torch.zeros(2, dtype=torch.int32, device=dev))
    with pytest.raises(moe.MoeError):
        z = torch.zeros(4, 2, 32, dtype=BF16, device=dev)
        moe.gdn_decay_scan(z, z, z, d)
