"""The full-attention layer's operators without a GPU: the oracle against closed
forms (and its planted mistakes against them), and every refusal of the C entry
points and the binding, which answer on the host before anything is launched."""
import ctypes

import numpy as np
import pytest
import torch

import sparse_mixture_experts_gemm_gb300 as moe
from oracle import attention
from sparse_mixture_experts_gemm_gb300 import buildlib as moe_build


@pytest.fixture(scope="module")
def lib():
    moe_build.build()
    return moe.lib()


# ------------------------------------------------------------- the oracle
def test_rope_closed_form():
    """Quarter turns swap the pair; two turns of a add up to one of 2 a; the
    norm of a pair stays."""
    w = np.ones(8)
    x = np.arange(1.0, 9.0).reshape(1, 1, 8)
    y, n = attention.norm_rope(x, w, [1], [np.pi / 2, 0.0], 0.0)
    assert np.allclose((n * n).mean(), 1.0)
    assert np.allclose(y[0, 0, [0, 2]], [-n[0, 0, 2], n[0, 0, 0]]) and np.allclose(y[0, 0, [1, 3, 4, 5, 6, 7]],
                                                                                  n[0, 0, [1, 3, 4, 5, 6, 7]])
    once, _ = attention.norm_rope(x, w, [3], [0.3, 0.1], 0.0)
    far, _ = attention.norm_rope(x, w, [6], [0.3, 0.1], 0.0)
    twice, _ = attention.norm_rope(once, w, [3], [0.3, 0.1], 0.0)
    assert np.allclose(twice, far)


@pytest.mark.parametrize("mutation", [1, 2])
def test_rope_mistakes_are_seen(mutation):
    x = np.random.default_rng(1).normal(size=(3, 2, 8))
    a = (np.ones(8), [0, 5, 9], [0.5, 0.2], 1e-6)
    assert not np.allclose(attention.norm_rope(x, *a)[0], attention.norm_rope(x, *a, mutation=mutation)[0], rtol=1e-3)


def test_attend_closed_form():
    """Equal scores average the visible values; a large one picks its key."""
    v = np.arange(12.0).reshape(4, 1, 3)
    q, k = np.zeros((2, 1, 3)), np.ones((4, 1, 3))
    o, mag, _ = attention.attend(q, k, v, 1.0)
    assert np.allclose(o[0, 0], v[:3, 0].mean(0)) and np.allclose(o[1, 0], v[:, 0].mean(0)) and np.allclose(o, mag)
    k = np.eye(4, 3)[:, None] * 1e3
    o, _, _ = attention.attend(np.eye(3)[1:2, None], k, v, 1.0)
    assert np.allclose(o[0, 0], v[1, 0])
    # a query before the first key sees nothing
    o, _, _ = attention.attend(np.ones((3, 1, 3)), np.ones((1, 1, 3)), np.ones((1, 1, 3)), 1.0)
    assert not o[:2].any() and np.allclose(o[2], 1)


@pytest.mark.parametrize("mutation", [3, 4, 5])
def test_attend_mistakes_are_seen(mutation):
    rng = np.random.default_rng(2)
    q, k, v = rng.normal(size=(3, 4, 8)), rng.normal(size=(7, 2, 8)), rng.normal(size=(7, 2, 8))
    assert not np.allclose(attention.attend(q, k, v, 0.3)[0], attention.attend(q, k, v, 0.3, mutation=mutation)[0],
                           rtol=1e-3)


def test_quantise_closed_form():
    x = np.arange(64.0)[None] * 0.25  # 0 .. 15.75: scale 1.05, rounded to bf16
    c, s, b = attention.quantise(x)
    assert b[0, 0] == 0 and s[0, 0] == attention.bf16(1.05) and c[0, 0] == 0 and c[0, 63] == 15
    assert (np.abs(attention.values(c, s, b) - x) <= s[0, 0] * 0.51).all()
    c, s, b = attention.quantise(np.full((1, 128), 3.25))
    assert not s.any() and not c.any() and (b == 3.25).all()
    assert attention.bf16(1 + 2.0 ** -8) == 1 and attention.bf16(1 + 3 * 2.0 ** -8) == 1 + 2.0 ** -6


def test_unpack_mistake_is_seen():
    c = np.array([[0x21, 0x43]], np.uint8)
    assert attention.unpack(c).tolist() == [[1, 2, 3, 4]]
    assert attention.unpack(c, mutation=6).tolist() == [[2, 1, 4, 3]]


# -------------------------------------------------------------- refusals
P = 0x10000  # never dereferenced: each call below answers on the host
BAD, ALIGN, UNSUP, OK = (moe.MOE_ERR_INVALID_ARG, moe.MOE_ERR_ALIGNMENT, moe.MOE_ERR_UNSUPPORTED, moe.MOE_OK)


def _rope(lib, **kw):
    a = dict(q=P, k=P, qw=P, kw=P, pos=P, f=P, N=4, Hq=4, Hk=2, D=128, rot=64, qs=512, ks=256, eps=1e-6, qo=P,
             qos=512, ko=P, kos=256)
    a.update(kw)
    return lib.moe_qk_norm_rope(*a.values(), None)


@pytest.mark.parametrize("kw,code", [
    (dict(q=None), BAD), (dict(k=None), BAD), (dict(qw=None), BAD), (dict(kw=None), BAD), (dict(pos=None), BAD),
    (dict(f=None), BAD), (dict(qo=None), BAD), (dict(ko=None), BAD), (dict(N=-1), BAD), (dict(Hq=0), BAD),
    (dict(Hk=0), BAD), (dict(rot=-16), BAD), (dict(rot=144), BAD), (dict(qs=504), BAD), (dict(kos=248), BAD),
    (dict(eps=-1.0), BAD), (dict(eps=float("nan")), BAD),
    (dict(D=64, rot=16), UNSUP), (dict(D=192), UNSUP), (dict(rot=24), UNSUP), (dict(N=1 << 31), UNSUP),
    (dict(qs=1 << 39), UNSUP), (dict(Hq=4097, qs=4097 * 128, qos=4097 * 128), UNSUP),
    (dict(q=P + 8), ALIGN), (dict(ko=P + 2), ALIGN), (dict(qw=P + 4), ALIGN), (dict(pos=P + 2), ALIGN),
    (dict(f=P + 4), ALIGN), (dict(qs=516), ALIGN),
    (dict(N=0, q=None, k=None, pos=None), OK),
])
def test_rope_refusals(lib, kw, code):
    assert _rope(lib, **kw) == code


def _prefill(lib, **kw):
    a = dict(q=P, k=P, v=P, off=P, koff=P, nq=4, nk=8, n=2, Hq=4, Hk=2, D=128, qs=512, ks=256, vs=256, scale=0.1, out=P,
             ws=None, bytes=0)
    a.update(kw)
    return lib.moe_attention_prefill(*a.values(), None)


@pytest.mark.parametrize("kw,code", [
    (dict(q=None), BAD), (dict(k=None), BAD), (dict(v=None), BAD), (dict(out=None), BAD), (dict(nq=-1), BAD),
    (dict(nk=-1), BAD), (dict(n=-1), BAD), (dict(Hq=3), BAD), (dict(Hk=0), BAD), (dict(Hq=0), BAD),
    (dict(scale=0.0), BAD), (dict(scale=-1.0), BAD), (dict(scale=float("nan")), BAD), (dict(scale=float("inf")), BAD),
    (dict(off=None), BAD), (dict(koff=None), BAD), (dict(off=None, koff=None, n=3), BAD), (dict(qs=256), BAD),
    (dict(vs=128), BAD),
    (dict(D=64), UNSUP), (dict(Hq=130, qs=130 * 128), UNSUP), (dict(nq=1 << 31), UNSUP), (dict(ks=1 << 38), UNSUP),
    (dict(q=P + 8), ALIGN), (dict(out=P + 8), ALIGN), (dict(off=P + 2), ALIGN), (dict(koff=P + 1), ALIGN),
    (dict(vs=260), ALIGN),
    (dict(nk=1 << 20), BAD), (dict(nk=1 << 20, ws=P, bytes=1 << 10), BAD), (dict(nk=1 << 20, bytes=1 << 30), BAD),
    (dict(nk=1 << 20, ws=P + 8, bytes=1 << 30), ALIGN),
    (dict(nq=0, q=None, out=None), OK), (dict(n=0), OK),
])
def test_prefill_refusals(lib, kw, code):
    assert _prefill(lib, **kw) == code


def test_prefill_workspace(lib):
    """None where the tiles fill the GPU or keys are few, else room for the parts:
    a row of outputs, a maximum and a sum per query, head and part."""
    need = ctypes.c_size_t(0)

    def size(*a):
        assert lib.moe_attention_prefill_workspace(*a, ctypes.byref(need)) == OK
        return need.value

    assert size(4096, 4096, 1, 16, 2, 256) == 0 and size(17, 17, 1, 16, 2, 256) == 0 and size(64, 256, 2, 8, 2, 128) == 0
    for a in ((1, 4096, 1, 16, 2, 256), (40, 20000, 1, 32, 8, 128), (8, 65536, 4, 4, 4, 256), (1, 1 << 29, 1, 64, 1, 128),
              (4781, 20254, 2, 4, 1, 256), (2000, 50000, 8, 8, 2, 256)):
        row = a[0] * a[3] * (a[5] * 4 + 8)
        parts = size(*a) // row
        assert 2 <= parts <= 32 and need.value == parts * row
    assert size(0, 100, 1, 16, 2, 256) == 0 and size(5, 0, 1, 16, 2, 256) == 0 and size(5, 5000, 0, 16, 2, 256) == 0
    for a, code in (((-1, 4, 1, 4, 2, 128), BAD), ((1, -4, 1, 4, 2, 128), BAD), ((1, 4, -1, 4, 2, 128), BAD),
                    ((1, 4, 1, 3, 2, 128), BAD), ((1, 4, 1, 4, 2, 64), UNSUP), ((1 << 30, 4, 1, 4, 2, 128), UNSUP)):
        assert lib.moe_attention_prefill_workspace(*a, ctypes.byref(need)) == code
    assert lib.moe_attention_prefill_workspace(4, 4, 1, 4, 2, 128, None) == BAD


def _write(lib, **kw):
    a = dict(codes=P, affine=P, pages=8, k=P, v=P, table=P, width=4, starts=P, off=P, N=4, n=2, H=2, D=128, ks=256,
             vs=256)
    a.update(kw)
    return lib.moe_kv_write(*a.values(), None)


def _read(lib, **kw):
    a = dict(codes=P, affine=P, pages=8, table=P, width=4, starts=P, off=P, N=4, n=2, H=2, D=128, k=P, v=P)
    a.update(kw)
    return lib.moe_kv_read(*a.values(), None)


@pytest.mark.parametrize("call", [_write, _read])
@pytest.mark.parametrize("kw,code", [
    (dict(codes=None), BAD), (dict(affine=None), BAD), (dict(k=None), BAD), (dict(v=None), BAD),
    (dict(table=None), BAD), (dict(pages=-1), BAD), (dict(width=-1), BAD), (dict(N=-1), BAD), (dict(n=-1), BAD),
    (dict(H=0), BAD), (dict(off=None, n=3), BAD),
    (dict(D=64), UNSUP), (dict(D=512), UNSUP), (dict(pages=1 << 24), UNSUP), (dict(N=1 << 31), UNSUP),
    (dict(width=1 << 26), UNSUP),
    (dict(codes=P + 8), ALIGN), (dict(affine=P + 4), ALIGN), (dict(k=P + 2), ALIGN), (dict(table=P + 2), ALIGN),
    (dict(starts=P + 1), ALIGN), (dict(off=P + 2), ALIGN),
    (dict(N=0, k=None, v=None, codes=None), OK), (dict(n=0), OK),
])
def test_cache_refusals(lib, call, kw, code):
    assert call(lib, **kw) == code


def test_cache_write_stride_refusals(lib):
    assert _write(lib, ks=128) == BAD and _write(lib, vs=1 << 39) == UNSUP and _write(lib, ks=260) == ALIGN


def _decode(lib, **kw):
    need = ctypes.c_size_t(0)
    assert lib.moe_attention_decode_workspace(2, 4, 4, 2, 128, ctypes.byref(need)) == OK
    a = dict(q=P, qs=512, codes=P, affine=P, pages=8, table=P, width=4, lens=P, n=2, Hq=4, Hk=2, D=128, scale=0.1,
             out=P, ws=P, bytes=need.value)
    a.update(kw)
    return lib.moe_attention_decode(*a.values(), None)


@pytest.mark.parametrize("kw,code", [
    (dict(q=None), BAD), (dict(codes=None), BAD), (dict(affine=None), BAD), (dict(table=None), BAD),
    (dict(lens=None), BAD), (dict(out=None), BAD), (dict(pages=-1), BAD), (dict(width=-1), BAD), (dict(n=-1), BAD),
    (dict(Hq=3), BAD), (dict(Hk=0), BAD), (dict(scale=0.0), BAD), (dict(scale=float("inf")), BAD), (dict(qs=256), BAD),
    (dict(D=64), UNSUP), (dict(pages=1 << 24), UNSUP), (dict(qs=1 << 39), UNSUP), (dict(width=1 << 26), UNSUP),
    (dict(q=P + 8), ALIGN), (dict(out=P + 2), ALIGN), (dict(codes=P + 1), ALIGN), (dict(affine=P + 2), ALIGN),
    (dict(table=P + 2), ALIGN), (dict(lens=P + 1), ALIGN), (dict(ws=P + 4), ALIGN), (dict(qs=516), ALIGN),
    (dict(n=0, q=None), OK),
])
def test_decode_refusals(lib, kw, code):
    assert _decode(lib, **kw) == code


def test_decode_workspace_refusals(lib):
    need = ctypes.c_size_t(0)
    for a, code in (((-1, 4, 4, 2, 128), BAD), ((1, -1, 4, 2, 128), BAD), ((1, 4, 3, 2, 128), BAD),
                    ((1, 4, 4, 2, 64), UNSUP), ((1, 1 << 26, 4, 2, 128), UNSUP)):
        assert lib.moe_attention_decode_workspace(*a, ctypes.byref(need)) == code
    assert lib.moe_attention_decode_workspace(1, 4, 4, 2, 128, None) == BAD


def test_binding_refuses_what_it_cannot_take(lib):
    """CPU tensors, other types and shapes that do not agree."""
    bf = torch.bfloat16
    q, k, w = torch.zeros(3, 4, 128, dtype=bf), torch.zeros(3, 2, 128, dtype=bf), torch.zeros(128, dtype=bf)
    pos, f = torch.zeros(3, dtype=torch.int32), torch.zeros(32, dtype=torch.float64)
    with pytest.raises(ValueError, match="CUDA"):
        moe.qk_norm_rope(q, k, w, w, pos, f)
    with pytest.raises(ValueError, match="agree"):
        moe.qk_norm_rope(q, k[:2], w, w, pos, f)
    with pytest.raises(ValueError, match="CUDA"):
        moe.attention_prefill(q, k, k)
    with pytest.raises(ValueError, match="agree"):
        moe.attention_prefill(q, k, k[:2])
    with pytest.raises(ValueError, match="agree"):
        moe.attention_prefill(q[None], k, k)
    cache = moe.kv_cache(4, 2, 128, device="cpu")
    assert cache[0].shape == (4, 2, 2, 64, 64) and cache[1].shape == (4, 2, 2, 64, 2, 2)
    pages = torch.zeros(1, 4, dtype=torch.int32)
    for call in (lambda: moe.kv_cache_write(cache, k, k, pages), lambda: moe.kv_cache_read(cache, pages, pos, 3),
                 lambda: moe.attention_decode(q[:1], cache, pages, pos[:1])):
        with pytest.raises(ValueError, match="CUDA"):
            call()
