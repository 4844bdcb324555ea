"""CPU tests of softmax attention and rotary positions: the oracles against closed
forms and differences, the frequencies, the library's refusals (no call here
launches a kernel: each is refused before), the Python checks."""
import ctypes
import math

import numpy as np
import pytest
import torch

import kimi_delta_attention_bwd_gb300 as kda
from kimi_delta_attention_bwd_gb300 import _lib
from oracle import rotary as orot
from oracle import softmax_attention as osm

FAKE = 1 << 20  # 256-byte aligned non-null fake address; never dereferenced


# ---------------------------------------------------------------- oracle pins
def _draw(seed, Nq, Nk, Hq, Hkv, D):
    r = np.random.RandomState(seed)
    return r.randn(Nq, Hq, D), r.randn(Nk, Hkv, D), r.randn(Nk, Hkv, D), r.randn(Nq, Hq, D)


def test_oracle_equal_keys_average_the_values():
    q, _, v, _ = _draw(0, 5, 5, 2, 1, 4)
    ref, _, _ = osm.attend(q, np.ones((5, 1, 4)), v, [0, 5], [0, 5], 0.5, True)
    for i in range(5):
        assert np.allclose(ref["o"][i], v[:i + 1, 0].mean(0)[None])
        assert np.allclose(ref["lse"][i], 0.5 * q[i].sum(-1) + math.log(i + 1))


def test_oracle_one_large_logit_selects_its_value():
    q, k, v, _ = _draw(1, 3, 6, 1, 1, 4)
    k[4] = 1e4 * q[2]
    ref, _, _ = osm.attend(q, k, v, [0, 3], [0, 6], 1.0, True)
    assert np.allclose(ref["o"][2], v[4])


def test_oracle_offsets_and_empty_rows():
    # three queries over two keys: the first sees none; five keys: the first sees three
    q, k, v, g = _draw(2, 6, 7, 1, 1, 4)
    ref, _, _ = osm.attend(q, k, v, [0, 3, 6], [0, 2, 7], 1.0, True, g)
    assert np.all(ref["o"][0] == 0) and ref["lse"][0, 0] == -np.inf and np.all(ref["dq"][0] == 0)
    assert np.allclose(ref["o"][1], v[0])
    s = q[3, 0] @ k[2:5, 0].T
    assert np.allclose(ref["lse"][3, 0], np.log(np.exp(s).sum()))
    # a document of no keys, and one of no queries
    ref, _, _ = osm.attend(q, k, v, [0, 6, 6], [0, 0, 7], 1.0, False, g)
    assert np.all(ref["o"] == 0) and np.all(ref["dk"] == 0)


@pytest.mark.parametrize("causal", [True, False])
def test_oracle_gradients_are_differences(causal):
    q, k, v, g = _draw(3, 7, 9, 4, 2, 3)
    cu, cuk = [0, 4, 7], [0, 3, 9]
    f = lambda q, k, v: (osm.attend(q, k, v, cu, cuk, 0.7, causal)[0]["o"] * g).sum()  # noqa: E731
    ref, _, _ = osm.attend(q, k, v, cu, cuk, 0.7, causal, g)
    h = 1e-5
    for n, x in (("dq", q), ("dk", k), ("dv", v)):
        num = np.zeros(x.shape)
        for i in np.ndindex(x.shape):
            old = x[i]
            x[i] = old + h
            up = f(q, k, v)
            x[i] = old - h
            num[i] = (up - f(q, k, v)) / (2 * h)
            x[i] = old
        assert np.allclose(ref[n], num, atol=2e-8), n


def test_oracle_rotary_is_a_rotation():
    r = np.random.RandomState(4)
    x, y = r.randn(3, 2, 10), r.randn(3, 2, 10)
    f = 10.0 ** -np.arange(3)
    for inter in (False, True):
        pos = np.array([0, 5, 100])
        a = orot.turn(x, pos, f, inter)
        assert np.allclose(a[0], x[0]) and np.allclose(a[..., 6:], x[..., 6:])
        assert np.allclose((a ** 2).sum(-1), (x ** 2).sum(-1))
        assert np.allclose(orot.turn(a, pos, f, inter, inverse=True), x)
        # products depend on the difference of positions alone
        b = orot.turn(y, pos + 7, f, inter)
        a2, b2 = orot.turn(x, pos + 30, f, inter), orot.turn(y, pos + 37, f, inter)
        assert np.allclose((a * b).sum(-1), (a2 * b2).sum(-1))
        # the gradient's map is the transpose
        assert np.allclose((orot.turn(x, pos, f, inter, 1.5) * y).sum(),
                           (x * orot.turn(y, pos, f, inter, 1.5, True)).sum())
    assert np.allclose(orot.turn(np.eye(2)[:1][None], [1], [0.3])[0, 0], [math.cos(0.3), math.sin(0.3)])
    assert np.allclose(orot.turn(np.array([[[1.0, 2.0, 3.0, 4.0]]]), [1], [0.3, 0.0], True)[0, 0, 2:], [3, 4])


# ---------------------------------------------------------------- frequencies
def test_rotary_frequencies():
    f, s = kda.rotary_frequencies(8, base=100.0, device="cpu")
    assert s == 1.0 and f.dtype == torch.float32
    assert np.allclose(f.numpy(), 100.0 ** (-np.arange(4) / 4), rtol=1e-7)
    lin, s = kda.rotary_frequencies(8, base=100.0, factor=4.0, scaling="linear", device="cpu")
    assert s == 1.0 and torch.allclose(lin * 4, f)
    ntk, s = kda.rotary_frequencies(8, base=100.0, factor=4.0, scaling="ntk", device="cpu")
    assert s == 1.0 and ntk[0] == 1.0 and abs(float(ntk[-1] / f[-1]) - 0.25) < 1e-6
    kw = dict(base=10000.0, factor=8.0, scaling="yarn", original_length=4096, device="cpu")
    y, s = kda.rotary_frequencies(128, **kw)
    f, _ = kda.rotary_frequencies(128, device="cpu")
    turns = 4096 * f.double() / (2 * math.pi)
    assert abs(s - (0.1 * math.log(8.0) + 1)) < 1e-12
    # (the ramp's ends are rounded outwards to whole pairs)
    assert torch.equal(y[turns > 32 * 1.2], f[turns > 32 * 1.2])
    assert torch.allclose(y[turns < 1 / 1.2], f[turns < 1 / 1.2] / 8)
    mid = (turns < 20) & (turns > 2)
    assert mid.any() and bool(((y < f) & (y > f / 8))[mid].all())
    for bad in (dict(rot=0), dict(rot=7), dict(rot=8, base=1.0), dict(rot=8, factor=0.5), dict(rot=8, scaling="x"),
                dict(rot=8, scaling="yarn"), dict(rot=2, scaling="ntk", factor=2.0)):
        with pytest.raises(ValueError):
            kda.rotary_frequencies(device="cpu", **bad)


# ---------------------------------------------------------------- refusals of the C entries
def _prob(B=2, T=100, Tk=100, Hq=4, Hkv=2, D=64, dtype=torch.bfloat16, causal=1, cu=None, cuk=None, n_docs=2,
          host=None, khost=None):
    p = _lib.kda_softmax_problem(B, T, Tk, Hq, Hkv, D, _lib._dt(dtype), 0.0, causal, n_docs if cu else 0, cu, cuk,
                                 None if host is None else host.ctypes.data,
                                 None if khost is None else khost.ctypes.data)
    p.keep = (host, khost)
    return p


def _fwd(p, q=FAKE, o=FAKE, lse=FAKE, ws=FAKE, n=1 << 40, save=1):
    P = ctypes.c_void_p
    return _lib.load().kda_softmax_fwd(ctypes.byref(p), P(q), P(FAKE), P(FAKE), P(o), P(lse), save, P(ws), n, None)


def _bwd(p, dO=FAKE, dv=FAKE, ws=FAKE, n=1 << 40):
    P = ctypes.c_void_p
    return _lib.load().kda_softmax_bwd(ctypes.byref(p), P(FAKE), P(FAKE), P(FAKE), P(FAKE), P(dO), P(FAKE), P(FAKE),
                                       P(dv), P(ws), n, None)


def test_softmax_refusals():
    for call in (_fwd, _bwd):
        for bad in (dict(B=0), dict(T=0), dict(Tk=0), dict(Hq=0), dict(Hkv=0), dict(Hq=3), dict(Hq=8192), dict(causal=2),
                    dict(dtype=torch.float16), dict(B=1 << 16, T=1 << 16), dict(cu=FAKE, n_docs=0),
                    dict(cuk=FAKE), dict(cu=FAKE, Tk=101),
                    dict(B=1, T=1 << 23, Tk=1 << 23, Hq=4096, Hkv=1, cu=FAKE, n_docs=1 << 23)):
            assert call(_prob(**bad)) == -1, bad
        assert call(_prob(D=96)) == -2 and call(_prob(D=32)) == -2
        assert call(_prob(cu=FAKE + 2)) == -3
        for off in ([1, 100, 200], [0, 120, 100], [0, 100, 199], [0, -1, 200]):
            assert call(_prob(cu=FAKE, host=np.array(off, np.int32))) == -4, off
            assert call(_prob(cu=FAKE, cuk=FAKE, khost=np.array(off, np.int32))) == -4, off
        assert call(_prob(), ws=0) == -5 and call(_prob(), n=255) == -5 and call(_prob(), ws=FAKE + 16) == -3
    assert _fwd(_prob(), q=0) == -1 and _fwd(_prob(), o=0) == -1 and _fwd(_prob(), lse=0) == -1
    assert _fwd(_prob(), q=FAKE + 8) == -3
    assert _bwd(_prob(), dO=0) == -1 and _bwd(_prob(), dv=0) == -1 and _bwd(_prob(), dO=FAKE + 8) == -3


def test_softmax_workspace_size():
    lib = _lib.load()
    size = lambda b, **kw: lib.kda_softmax_workspace_size(ctypes.byref(_prob(**kw)), b)  # noqa: E731
    assert 0 < size(0) <= size(0, cu=FAKE) < size(1, cu=FAKE)
    assert size(0) % 256 == 0 and size(0) < size(1)
    assert size(0, D=96) == 0 and size(1, T=0) == 0 and lib.kda_softmax_workspace_size(None, 0) == 0


def test_softmax_decode_refusals():
    lib = _lib.load()
    P = ctypes.c_void_p

    def call(n=2, cap=8, Hq=4, Hkv=2, D=64, dt=0, q=FAKE, kc=FAKE, ln=FAKE, ws=FAKE, nb=1 << 40):
        return lib.kda_softmax_decode(n, cap, Hq, Hkv, D, dt, 0.0, P(q), P(FAKE), P(FAKE), P(kc), P(FAKE), P(ln),
                                      P(FAKE), P(ws), nb, None)
    for bad in (dict(n=0), dict(cap=0), dict(Hq=0), dict(Hkv=0), dict(Hq=5), dict(Hq=5000), dict(dt=2), dict(q=0),
                dict(kc=0), dict(ln=0)):
        assert call(**bad) == -1, bad
    assert call(D=48) == -2 and call(q=FAKE + 4) == -3 and call(ln=FAKE + 2) == -3 and call(ws=FAKE + 64) == -3
    assert call(ws=0) == -5 and call(nb=128) == -5
    size = lib.kda_softmax_decode_workspace_size
    assert size(0, 8, 4, 2, 64) == 0 and size(1, 8, 4, 2, 96) == 0
    assert 0 < size(1, 8, 4, 2, 64) < size(1, 1 << 17, 4, 2, 64)


def test_rotary_refusals():
    lib = _lib.load()
    P = ctypes.c_void_p

    def call(n=4, T=4, Hq=2, Hkv=1, D=64, rot=64, dt=0, inter=0, inv=0, f=FAKE, pos=None, cu=None, nd=0, q=FAKE, k=FAKE,
             oq=2 * FAKE, ok=2 * FAKE):
        return lib.kda_rotary(n, T, Hq, Hkv, D, rot, dt, inter, inv, 0.0, P(f), P(pos), P(cu), nd, P(q), P(k), P(oq),
                              P(ok), None)
    for bad in (dict(n=0), dict(n=1 << 31), dict(T=0), dict(Hq=0), dict(Hkv=-1), dict(D=0), dict(D=1026), dict(rot=0),
                dict(rot=63), dict(rot=66), dict(dt=2), dict(inter=2), dict(inv=-1), dict(f=0), dict(q=0), dict(k=0),
                dict(oq=0), dict(ok=0), dict(pos=FAKE, cu=FAKE, nd=1), dict(cu=FAKE, nd=0), dict(oq=FAKE),
                dict(ok=FAKE)):
        assert call(**bad) == -1, bad
    assert call(q=FAKE + 8) == -3 and call(f=FAKE + 2) == -3 and call(pos=FAKE + 1) == -3


# ---------------------------------------------------------------- refusals of the Python entries
def test_python_softmax_refusals():
    q, k = torch.zeros(1, 4, 4, 64), torch.zeros(1, 4, 2, 64)
    cu = torch.tensor([0, 4], dtype=torch.int32)
    with pytest.raises(ValueError, match="CUDA"):
        kda.kda_softmax_forward(q, k, k)
    with pytest.raises(ValueError, match="multiple"):
        kda.kda_softmax_forward(q[:, :, :3], k, k)
    with pytest.raises(ValueError, match="v must have shape"):
        kda.kda_softmax_forward(q, k, k[:, :3])
    with pytest.raises(ValueError, match="need cu_seqlens_k"):
        kda.kda_softmax_forward(q, k[:, :3], k[:, :3], cu_seqlens=cu)
    with pytest.raises(ValueError, match="comes with cu_seqlens"):
        kda.kda_softmax_forward(q, k, k, cu_seqlens_k=cu)
    with pytest.raises(ValueError, match="comes with cu_seqlens_k"):
        kda.kda_softmax_forward(q, k, k, cu_seqlens=cu, cu_seqlens_k_host=cu)
    with pytest.raises(ValueError, match="cu_seqlens_k must have shape"):
        kda.kda_softmax_forward(q, k, k, cu_seqlens=cu, cu_seqlens_k=torch.zeros(3, dtype=torch.int32))
    with pytest.raises(ValueError, match="two offsets"):
        kda.kda_softmax_forward(q, k, k, cu_seqlens=cu[:1])
    with pytest.raises(ValueError, match="4 dimensions"):
        kda.kda_softmax_forward(q[0], k, k)
    ctx = kda.SoftmaxContext(None, q, k, k, q, None, None, (None, None), None, False)
    with pytest.raises(ValueError, match="saved nothing"):
        kda.kda_softmax_backward(ctx, q)
    ctx.saved = True
    with pytest.raises(ValueError, match="q must be a CUDA tensor"):
        kda.kda_softmax_backward(ctx, q)
    n = torch.zeros(1, dtype=torch.int32)
    with pytest.raises(ValueError, match="CUDA"):
        kda.kda_softmax_decode_step(q[:, 0], k[:, 0], k[:, 0], k, k.clone(), n)
    with pytest.raises(ValueError, match="v_cache must have shape"):
        kda.kda_softmax_decode_step(q[:, 0], k[:, 0], k[:, 0], k, k[:, :3], n)
    with pytest.raises(ValueError, match="multiple"):
        kda.kda_softmax_decode_step(q[:, 0, :3], k[:, 0], k[:, 0], k, k.clone(), n)


def test_python_rotary_refusals():
    q, k, f = torch.zeros(1, 4, 4, 64), torch.zeros(1, 4, 2, 64), torch.zeros(32)
    with pytest.raises(ValueError, match="CUDA"):
        kda.kda_rotary(q, k, f)
    with pytest.raises(ValueError, match="pairs"):
        kda.kda_rotary(q, k, torch.zeros(33))
    with pytest.raises(ValueError, match="positive"):
        kda.kda_rotary(q, k, f, scale=0.0)
    with pytest.raises(ValueError, match="need positions"):
        kda.kda_rotary(q[0], k[0], f)
    with pytest.raises(ValueError, match="not both"):
        kda.kda_rotary(q, k, f, positions=torch.zeros(1, 4, dtype=torch.int32),
                       cu_seqlens=torch.tensor([0, 4], dtype=torch.int32))
    with pytest.raises(ValueError, match="positions must have shape"):
        kda.kda_rotary(q, k, f, positions=torch.zeros(4, dtype=torch.int32))
    with pytest.raises(ValueError, match="k must have shape"):
        kda.kda_rotary(q, k[:, :3], f)
    with pytest.raises(ValueError, match="out_k without k"):
        kda.kda_rotary(q, None, f, out_k=k)


@pytest.mark.parametrize("scale", [1e-46, 1e-300, 0.0, -1.0, 1e39, math.inf, math.nan])
def test_scales_that_are_not_positive_fp32_numbers_are_refused(scale):
    """Positive in 64 bits is not enough: what vanishes in fp32 would select the default."""
    q, k, f = torch.zeros(1, 4, 4, 64, device="meta"), torch.zeros(1, 4, 2, 64, device="meta"), torch.zeros(32)
    with pytest.raises(ValueError, match="scale must be positive"):
        kda._positive(scale)
    with pytest.raises(ValueError, match="scale must be positive"):
        kda.kda_rotary(q, k, f, scale=scale)
    for s in (1e-38, 1e-45, 0.125, 3e38):
        kda._positive(s)


def test_scales_that_are_not_finite_are_refused_by_the_c_entries():
    lib = _lib.load()
    P = ctypes.c_void_p
    for scale in (math.inf, -math.inf, math.nan):
        p = _prob()
        p.scale = scale
        assert _fwd(p) == -1 and _bwd(p) == -1
        assert lib.kda_softmax_decode(2, 8, 4, 2, 64, 0, scale, *[P(FAKE)] * 8, 1 << 40, None) == -1
        assert lib.kda_rotary(4, 4, 2, 1, 64, 64, 0, 0, 0, scale, P(FAKE), None, None, 0, *[P(FAKE)] * 2,
                              *[P(2 * FAKE)] * 2, None) == -1


def test_softmax_scales_are_checked(monkeypatch):
    """The calls refuse before anything is launched (tensors on the host that the device checks let pass)."""
    from kimi_delta_attention_bwd_gb300 import softmax
    monkeypatch.setattr(softmax, "_all_well", lambda *a: True)
    q, k = torch.zeros(1, 4, 4, 64), torch.zeros(1, 4, 2, 64)
    for scale in (1e-46, math.inf, -1.0):
        with pytest.raises(ValueError, match="scale must be positive"):
            kda.kda_softmax_forward(q, k, k, scale=scale)
        with pytest.raises(ValueError, match="scale must be positive"):
            kda.kda_softmax_decode_step(q[0], k[0], k[0], torch.zeros(4, 9, 2, 64), torch.zeros(4, 9, 2, 64),
                                        torch.zeros(4, dtype=torch.int32), scale=scale)
