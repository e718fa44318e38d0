"""The mixer's operators without a GPU: the oracle against closed forms (and
its planted mistakes against them), and every refusal of the C entry points,
which answer on the host before anything is launched."""
import ctypes

import numpy as np
import pytest
import torch

import sparse_mixture_experts_gemm_gb300 as moe
import sparse_mixture_experts_gemm_gb300.mixer as binding
from oracle import mixer
from sparse_mixture_experts_gemm_gb300 import buildlib as moe_build


@pytest.fixture(scope="module")
def lib():
    moe_build.build()
    return moe.lib()


# ------------------------------------------------------------- the oracle
def test_e4m3_values():
    v = mixer.e4m3_values()
    assert v[0] == 0 and v[1] == 2.0 ** -9 and v[8] == 2.0 ** -6 and v[0x38] == 1.0
    assert v[0x7e] == 448.0 and v[0xfe] == -448.0 and np.isnan(v[0x7f]) and np.isnan(v[0xff])
    assert (np.diff(v[:0x7f]) > 0).all()


def test_norm_closed_form():
    """Rows of +-c have mean square c^2: the norm of c (1, -1, ..) is +-weight."""
    w = np.linspace(0.5, 2, 8)
    x = np.array([[3.0, -3.0] * 4, [0.25] * 8])
    y, s = mixer.rmsnorm(x - 1, w, 0.0, residual=np.ones((2, 8)))
    assert np.allclose(y, np.sign(x) * w, rtol=1e-14) and np.array_equal(s, x)
    y, _ = mixer.rmsnorm(np.zeros((1, 4)), np.ones(4), 1e-6)
    assert not y.any()


@pytest.mark.parametrize("mutation", [1, 2])
def test_norm_mistakes_are_seen(mutation):
    rng = np.random.default_rng(1)
    x, r, w = rng.normal(size=(3, 16)), rng.normal(size=(3, 16)), np.ones(16)
    y, _ = mixer.rmsnorm(x, w, 0.0, r)
    assert np.allclose((y * y).mean(1), 1.0)
    bad, _ = mixer.rmsnorm(x, w, 0.0, r, mutation=mutation)
    assert not np.allclose(bad, y, rtol=1e-3)


def test_matmul_closed_form():
    x, w = np.eye(3, 4), np.arange(12.0).reshape(3, 4)
    out = mixer.matmul(x, [1, 2, 3], w, [1, 10, 100])
    want = w[:, :3].T * np.array([[1], [2], [3]]) * np.array([[1, 10, 100]])
    assert np.array_equal(out, want)
    assert not np.array_equal(mixer.matmul(x, [1, 2, 3], w, [1, 10, 100], mutation=3), want)


def test_scan_closed_form():
    """o_t = sum_{j <= t} lambda^(t - j) (q_t . k_j) v_j + lambda^(t + 1) S_0 q_t."""
    rng = np.random.default_rng(2)
    N, Hk, Hv, dk, dv = 9, 2, 4, 8, 6
    q, k, v = rng.normal(size=(N, Hk, dk)), rng.normal(size=(N, Hk, dk)), rng.normal(size=(N, Hv, dv))
    lam, S0 = np.array([0.9, 0.5, 0.0, 1.0]), rng.normal(size=(2, Hv, dv, dk))
    off = [0, 4, 9]
    o, S = mixer.decay_scan(q, k, v, lam, S0, off)
    for i, (a, b) in enumerate(zip(off, off[1:])):
        for h in range(Hv):
            for t in range(a, b):
                ref = lam[h] ** (t - a + 1) * S0[i, h] @ q[t, h // 2]
                for j in range(a, t + 1):
                    ref = ref + lam[h] ** (t - j) * (q[t, h // 2] @ k[j, h // 2]) * v[j, h]
                assert np.allclose(o[t, h], ref, rtol=1e-10, atol=1e-12)
            ref = lam[h] ** (b - a) * S0[i, h]
            for j in range(a, b):
                ref = ref + lam[h] ** (b - 1 - j) * np.outer(v[j, h], k[j, h // 2])
            assert np.allclose(S[i, h], ref, rtol=1e-10, atol=1e-12)


@pytest.mark.parametrize("mutation", [4, 5, 6, 7])
def test_scan_mistakes_are_seen(mutation):
    rng = np.random.default_rng(3)
    q, k, v = rng.normal(size=(5, 2, 8)), rng.normal(size=(5, 2, 8)), rng.normal(size=(5, 4, 8))
    lam = np.array([0.9, 0.8, 0.7, 0.6])
    good = mixer.decay_scan(q, k, v, lam)
    bad = mixer.decay_scan(q, k, v, lam, mutation=mutation)
    assert not np.allclose(good[0], bad[0], rtol=1e-3)


# -------------------------------------------------------------- refusals
P = 0x10000  # never dereferenced: each call below answers on the host


def _norm(lib, fp8=False, **kw):
    a = dict(x=P, r=None, w=P, dt=moe.MOE_BF16, rows=4, d=64, xs=64, rs=64, eps=1e-6, s=None, out=P,
             scales=P)
    a.update(kw)
    head = (a["x"], a["r"], a["w"], a["dt"], a["rows"], a["d"], a["xs"], a["rs"], a["eps"], a["s"],
            a["out"])
    return lib.moe_add_rmsnorm_fp8(*head, a["scales"], None) if fp8 else lib.moe_add_rmsnorm(*head, None)


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("kw,code", [
    (dict(x=None), moe.MOE_ERR_INVALID_ARG),
    (dict(w=None), moe.MOE_ERR_INVALID_ARG),
    (dict(out=None), moe.MOE_ERR_INVALID_ARG),
    (dict(dt=5), moe.MOE_ERR_INVALID_ARG),
    (dict(rows=-1), moe.MOE_ERR_INVALID_ARG),
    (dict(d=0, xs=0), moe.MOE_ERR_INVALID_ARG),
    (dict(xs=63), moe.MOE_ERR_INVALID_ARG),
    (dict(r=P, rs=63), moe.MOE_ERR_INVALID_ARG),
    (dict(eps=-1.0), moe.MOE_ERR_INVALID_ARG),
    (dict(eps=float("nan")), moe.MOE_ERR_INVALID_ARG),
    (dict(d=16385, xs=16385), moe.MOE_ERR_UNSUPPORTED),
    (dict(rows=1 << 31), moe.MOE_ERR_UNSUPPORTED),
    (dict(x=P + 1), moe.MOE_ERR_ALIGNMENT),
    (dict(w=P + 2, dt=moe.MOE_F32), moe.MOE_ERR_ALIGNMENT),
    (dict(s=P + 1), moe.MOE_ERR_ALIGNMENT),
    (dict(r=P + 1), moe.MOE_ERR_ALIGNMENT),
    (dict(x=None, w=None, rows=0), moe.MOE_OK),
])
def test_norm_refusals(lib, fp8, kw, code):
    assert _norm(lib, fp8, **kw) == code


def test_norm_fp8_scales_refusals(lib):
    assert _norm(lib, True, scales=None) == moe.MOE_ERR_INVALID_ARG
    assert _norm(lib, True, scales=P + 2) == moe.MOE_ERR_ALIGNMENT


@pytest.mark.parametrize("args,code", [
    ((P, 9, 4, 64, 64, P, P), moe.MOE_ERR_INVALID_ARG),
    ((None, moe.MOE_BF16, 4, 64, 64, P, P), moe.MOE_ERR_INVALID_ARG),
    ((P, moe.MOE_BF16, 4, 64, 60, P, P), moe.MOE_ERR_INVALID_ARG),
    ((P, moe.MOE_BF16, 4, 64, 64, None, P), moe.MOE_ERR_INVALID_ARG),
    ((P, moe.MOE_BF16, 4, 20000, 20000, P, P), moe.MOE_ERR_UNSUPPORTED),
    ((P + 2, moe.MOE_F32, 4, 64, 64, P, P), moe.MOE_ERR_ALIGNMENT),
    ((None, moe.MOE_BF16, 0, 64, 64, None, None), moe.MOE_OK),
])
def test_quantize_refusals(lib, args, code):
    assert lib.moe_quantize_fp8(*args, None) == code


@pytest.mark.parametrize("kw,code", [
    (dict(T=-1), moe.MOE_ERR_INVALID_ARG),
    (dict(N=0), moe.MOE_ERR_INVALID_ARG),
    (dict(K=0), moe.MOE_ERR_INVALID_ARG),
    (dict(x=None), moe.MOE_ERR_INVALID_ARG),
    (dict(ws=None), moe.MOE_ERR_INVALID_ARG),
    (dict(out=None), moe.MOE_ERR_INVALID_ARG),
    (dict(x_stride=32), moe.MOE_ERR_INVALID_ARG),
    (dict(w_stride=48), moe.MOE_ERR_INVALID_ARG),
    (dict(out_stride=9), moe.MOE_ERR_INVALID_ARG),
    (dict(K=72, x_stride=80, w_stride=80), moe.MOE_ERR_UNSUPPORTED),
    (dict(K=1 << 18, x_stride=1 << 18, w_stride=1 << 18), moe.MOE_ERR_UNSUPPORTED),
    (dict(T=(1 << 22) + 1), moe.MOE_ERR_UNSUPPORTED),
    (dict(N=(1 << 20) + 1, out_stride=1 << 21), moe.MOE_ERR_UNSUPPORTED),
    (dict(x=P + 8), moe.MOE_ERR_ALIGNMENT),
    (dict(w=P + 1), moe.MOE_ERR_ALIGNMENT),
    (dict(x_stride=72), moe.MOE_ERR_ALIGNMENT),
    (dict(xs=P + 2), moe.MOE_ERR_ALIGNMENT),
    (dict(out=P + 1), moe.MOE_ERR_ALIGNMENT),
    (dict(T=0, x=None, xs=None, out=None), moe.MOE_OK),
])
def test_matmul_refusals(lib, kw, code):
    a = dict(x=P, xs=P, T=3, x_stride=64, w=P, ws=P, N=10, K=64, w_stride=64, out=P, out_stride=10)
    a.update(kw)
    assert lib.moe_matmul_fp8(a["x"], a["xs"], a["T"], a["x_stride"], a["w"], a["ws"], a["N"], a["K"],
                              a["w_stride"], a["out"], a["out_stride"], None) == code


@pytest.mark.parametrize("kw,code", [
    (dict(N=-1), moe.MOE_ERR_INVALID_ARG),
    (dict(n=-1), moe.MOE_ERR_INVALID_ARG),
    (dict(n=0), moe.MOE_ERR_INVALID_ARG),            # tokens of no sequence
    (dict(n=3), moe.MOE_ERR_INVALID_ARG),            # 16 tokens in 3 equal sequences
    (dict(Hk=3), moe.MOE_ERR_INVALID_ARG),
    (dict(q=None), moe.MOE_ERR_INVALID_ARG),
    (dict(o=None), moe.MOE_ERR_INVALID_ARG),
    (dict(decay=None), moe.MOE_ERR_INVALID_ARG),
    (dict(qs=255), moe.MOE_ERR_INVALID_ARG),
    (dict(vs=100), moe.MOE_ERR_INVALID_ARG),
    (dict(dk=96, qs=512, ks=512), moe.MOE_ERR_UNSUPPORTED),
    (dict(dv=24), moe.MOE_ERR_UNSUPPORTED),
    (dict(dv=1040, vs=8192), moe.MOE_ERR_UNSUPPORTED),
    (dict(N=1 << 31, n=1), moe.MOE_ERR_UNSUPPORTED),
    (dict(qs=260), moe.MOE_ERR_ALIGNMENT),
    (dict(k=P + 8), moe.MOE_ERR_ALIGNMENT),
    (dict(s_out=P + 4), moe.MOE_ERR_ALIGNMENT),
    (dict(off=P + 2), moe.MOE_ERR_ALIGNMENT),
    (dict(N=0, n=0, q=None, k=None, v=None, o=None), moe.MOE_OK),
])
def test_decay_scan_refusals(lib, kw, code):
    a = dict(q=P, k=P, v=P, decay=P, s_in=None, s_out=P, o=P, off=None, N=16, n=2, Hk=2, Hv=4, dk=128,
             dv=64, qs=256, ks=256, vs=256)
    a.update(kw)
    assert lib.gdn_decay_scan(a["q"], a["k"], a["v"], a["decay"], a["s_in"], a["s_out"], a["o"],
                              a["off"], a["N"], a["n"], a["Hk"], a["Hv"], a["dk"], a["dv"], a["qs"],
                              a["ks"], a["vs"], None, 0, None) == code


def test_decay_workspace_is_asked_for(lib):
    """A call that needs a workspace is refused without one."""
    need = ctypes.c_size_t(0)
    assert lib.gdn_decay_workspace(16, 2, 0, 4, 128, 64, None) == moe.MOE_ERR_INVALID_ARG
    assert lib.gdn_decay_workspace(-1, 2, 0, 4, 128, 64, ctypes.byref(need)) == moe.MOE_ERR_INVALID_ARG
    assert lib.gdn_decay_workspace(65536, 1, 0, 4, 128, 128, ctypes.byref(need)) == moe.MOE_OK
    assert need.value % (4 * 4 * 128 * 128) == 0  # whole states
    if need.value:
        for ws, n in ((None, need.value), (P, need.value - 1)):
            assert lib.gdn_decay_scan(P, P, P, P, None, P, P, None, 65536, 1, 4, 4, 128, 128, 512, 512,
                                      512, ws, n, None) == moe.MOE_ERR_INVALID_ARG


@pytest.mark.parametrize("n,N", [(64, 16384), (192, 32768), (256, 65536), (1024, 131072), (257, 16640), (3000, 65536)])
def test_decay_workspace_of_many_packed_sequences(lib, n, N):
    """States in the workspace go by the sequences that can be cut, not by all
    that are packed: at most two per whole segment of the tokens (16 key and 32
    value heads of 128 x 128, a state of 2 MB)."""
    need = ctypes.c_size_t(0)
    assert lib.gdn_decay_workspace(N, n, 1, 32, 128, 128, ctypes.byref(need)) == moe.MOE_OK
    assert need.value <= 30 << 20


@pytest.mark.parametrize("n,N,heads,cut", [(1, 2900, 1, True), (1, 2900, 32, True), (9, 5461, 4, True), (6, 3400, 8, True),
                                           (9, 5461, 32, False), (65, 4160, 32, False), (1, 200, 1, False)])
def test_decay_packed_cut_goes_by_idle_sms(lib, n, N, heads, cut):
    """Whether the longest sequence of a packed batch may be cut depends on the
    SMs that its heads leave idle: without a cut the workspace has no state."""
    need = ctypes.c_size_t(0)
    assert lib.gdn_decay_workspace(N, n, 1, heads, 128, 128, ctypes.byref(need)) == moe.MOE_OK
    assert (need.value >= 128 * 128 * 4) == cut


@pytest.mark.parametrize("which", ["qs", "ks", "vs"])
@pytest.mark.parametrize("off", [None, P])
def test_decay_scan_refuses_strides_that_no_tensor_map_takes(lib, which, off):
    """A tensor map's strides end at 2^40 bytes.  With offsets the recurrent
    kernel is launched before the chunked ones, so the call has to be refused
    before either."""
    a = dict(qs=256, ks=256, vs=256)
    a[which] = 1 << 39
    assert lib.gdn_decay_scan(P, P, P, P, None, P, P, off, 64, 2, 2, 4, 128, 64, a["qs"], a["ks"], a["vs"],
                              P, 1 << 30, None) == moe.MOE_ERR_UNSUPPORTED


# ------------------------------------------------------------- the binding
class OnGpu(torch.Tensor):
    """A CPU tensor that says it is on GPU `dev`, for checks that come before
    any launch."""
    dev = 0
    is_cuda = True

    def get_device(self):
        return self.dev


def on_gpu(*shape, dtype=torch.bfloat16):
    return torch.zeros(*shape, dtype=dtype).as_subclass(OnGpu)


CALLS = {
    "add_rmsnorm": lambda t: binding.add_rmsnorm(t["x"], t["weight"], t["residual"], out=t["out"], sum_out=t["sum"]),
    "add_rmsnorm_fp8": lambda t: binding.add_rmsnorm_fp8(t["x"], t["weight"], t["residual"], codes=t["codes"],
                                                         scales=t["scales"], sum_out=t["sum"]),
    "quantize_fp8": lambda t: binding.quantize_fp8(t["x"], codes=t["codes"], scales=t["scales"]),
    "matmul_fp8": lambda t: binding.matmul_fp8(t["codes"], t["scales"], t["w"], t["w_scales"], out=t["out"]),
    "gdn_decay_scan": lambda t: binding.gdn_decay_scan(t["q"], t["k"], t["v"], t["decay"], state=t["state"],
                                                       offsets=t["offsets"], out=t["o"], state_out=t["state_out"]),
}
USES = {
    "add_rmsnorm": ["x", "weight", "residual", "out", "sum"],
    "add_rmsnorm_fp8": ["x", "weight", "residual", "codes", "scales", "sum"],
    "quantize_fp8": ["x", "codes", "scales"],
    "matmul_fp8": ["codes", "scales", "w", "w_scales", "out"],
    "gdn_decay_scan": ["q", "k", "v", "decay", "state", "offsets", "o", "state_out"],
}


def operands():
    f8, f32 = torch.float8_e4m3fn, torch.float32
    t = {"x": on_gpu(4, 64), "weight": on_gpu(64), "residual": on_gpu(4, 64), "out": on_gpu(4, 64), "sum": on_gpu(4, 64),
         "codes": on_gpu(4, 64, dtype=f8), "scales": on_gpu(4, dtype=f32), "w": on_gpu(64, 64, dtype=f8),
         "w_scales": on_gpu(64, dtype=f32), "decay": on_gpu(2, dtype=f32), "offsets": on_gpu(3, dtype=torch.int32),
         "state": on_gpu(2, 2, 64, 64, dtype=f32), "state_out": on_gpu(2, 2, 64, 64, dtype=f32)}
    for name in ("q", "k", "v", "o"):
        t[name] = on_gpu(4, 2, 64)
    return t


@pytest.fixture
def launches(monkeypatch):
    """The library replaced by a recorder of its calls, on GPU 0 as the current one."""
    seen = []

    class Recorder:
        def __getattr__(self, name):
            return lambda *a: seen.append(name) or 0

    monkeypatch.setattr(binding, "_lib", lambda: Recorder())
    monkeypatch.setattr(binding, "_raw_stream", lambda dev: 0)
    monkeypatch.setattr(binding, "_decay_workspace", lambda *a: 0)
    monkeypatch.setattr(binding, "_current_device", lambda: 0, raising=False)
    monkeypatch.setattr(binding, "_gpus", 2, raising=False)
    return seen


@pytest.mark.parametrize("name", CALLS)
def test_one_device_per_call(launches, name):
    """The kernels run on the current device: a tensor of another one, or all of
    them, is refused before the library is called."""
    CALLS[name](operands())
    assert launches == ["moe_" + name if name != "gdn_decay_scan" else name]
    for elsewhere in [[n] for n in USES[name]] + [USES[name]]:
        t = operands()
        for n in elsewhere:
            t[n].dev = 1
        with pytest.raises(ValueError, match="device"):
            CALLS[name](t)
    assert len(launches) == 1


def test_stream_of_another_device_is_refused(launches):
    class Stream:
        device_index, cuda_stream = 1, 5

    t = operands()
    with pytest.raises(ValueError, match="device"):
        binding.quantize_fp8(t["x"], codes=t["codes"], scales=t["scales"], stream=Stream())
    assert launches == []
