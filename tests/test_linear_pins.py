"""CPU pins of the linear-attention and layer-norm oracles (closed forms,
finite differences) and the host-side refusals of their entry points (every
call below fails validation, so no kernel is ever launched)."""
import ctypes

import numpy as np
import pytest
import torch

import kimi_delta_attention_bwd_gb300 as kda
from kimi_delta_attention_bwd_gb300 import _lib
from oracle import layer_norm as oln
from oracle import linear_attention as ola

FAKE = 1 << 20  # 256-byte aligned non-null fake address; never dereferenced


def _inputs(seed, N, H, dk, dv, docs):
    r = np.random.default_rng(seed)
    cu = [0] + list(np.cumsum(docs))
    assert cu[-1] == N
    return dict(q=r.normal(size=(N, H, dk)), k=r.normal(size=(N, H, dk)), v=r.normal(size=(N, H, dv)),
                A_log=r.normal(size=H) - 1.0, cu=cu, scale=0.3, h0=r.normal(size=(len(docs), H, dk, dv)))


def test_two_tokens_by_hand():
    # e^-a = 1/2: S1 = h/2 + k1 v1, S2 = S1/2 + k2 v2 (all scalars)
    x = dict(q=np.array([3.0, 5.0]).reshape(2, 1, 1), k=np.array([2.0, -1.0]).reshape(2, 1, 1),
             v=np.array([4.0, 6.0]).reshape(2, 1, 1), A_log=np.array([np.log(np.log(2.0))]), cu=[0, 2], scale=0.5,
             h0=np.array(8.0).reshape(1, 1, 1, 1))
    o, hf = ola.forward(**x)
    s1, s2 = 4.0 + 8.0, 6.0 - 6.0
    np.testing.assert_allclose(o.ravel(), [0.5 * 3.0 * s1, 0.5 * 5.0 * s2], atol=1e-14)
    np.testing.assert_allclose(hf.ravel(), [s2], atol=1e-14)


def test_masked_product_form():
    x = _inputs(2, 40, 2, 5, 3, [13, 0, 1, 26])
    o, _ = ola.forward(**x)
    a = np.exp(x["A_log"])
    for d in range(4):
        s = slice(x["cu"][d], x["cu"][d + 1])
        n = s.stop - s.start
        i = np.arange(n)
        for h in range(2):
            w = np.where(i[:, None] >= i, np.exp(-a[h] * np.clip(i[:, None] - i, 0, None)), 0.0)
            ref = (x["q"][s, h] @ x["k"][s, h].T * w) @ x["v"][s, h]
            ref += np.exp(-a[h] * (i + 1))[:, None] * (x["q"][s, h] @ x["h0"][d, h])
            np.testing.assert_allclose(o[s, h], 0.3 * ref, rtol=1e-11, atol=1e-12)


@pytest.mark.parametrize("name", ["q", "k", "v", "A_log", "h0"])
def test_linear_finite_differences(name):
    x = _inputs(3, 9, 2, 4, 3, [5, 0, 4])
    r = np.random.default_rng(4)
    dO, dh = r.normal(size=(9, 2, 3)), r.normal(size=(3, 2, 4, 3))
    g = ola.backward(**x, dO=dO, dh_final=dh)["d" + name]

    def loss(arr):
        o, hf = ola.forward(**{**x, name: arr})
        return (o * dO).sum() + (hf * dh).sum()

    e = 1e-5
    for idx in [tuple(r.integers(0, s) for s in x[name].shape) for _ in range(6)]:
        p, m = x[name].copy(), x[name].copy()
        p[idx] += e
        m[idx] -= e
        fd = (loss(p) - loss(m)) / (2 * e)
        assert abs(fd - g[idx]) <= 1e-7 * max(1.0, abs(fd)), (idx, fd, g[idx])


def test_layer_norm_by_hand():
    # (1, 2, 6): mean 3, variance 14/3
    y = oln.forward(np.array([[1.0, 2.0, 6.0]]), np.array([1.0, 2.0, 1.0]), np.array([0.0, 0.0, 5.0]), eps=0.0)
    s = np.sqrt(14.0 / 3.0)
    np.testing.assert_allclose(y, [[-2.0 / s, -2.0 / s, 3.0 / s + 5.0]], rtol=1e-14)


def test_layer_norm_finite_differences():
    r = np.random.default_rng(5)
    x, w, dy = r.normal(size=(3, 7)), r.normal(size=7), r.normal(size=(3, 7))
    dx, dw, db = oln.backward(x, w, dy)
    e = 1e-6
    for arr, g, idx in ((x, dx, (1, 4)), (x, dx, (2, 0)), (w, dw, (3,))):
        p, m = arr.copy(), arr.copy()
        p[idx] += e
        m[idx] -= e
        f = lambda t: (oln.forward(t if arr is x else x, t if arr is w else w) * dy).sum()  # noqa: E731
        fd = (f(p) - f(m)) / (2 * e)
        assert abs(fd - g[idx]) <= 1e-7 * max(1.0, abs(fd))
    np.testing.assert_allclose(db, dy.sum(0))


# ---------------------------------------------------------------- refusals on the host
def _prob(**kw):
    a = dict(B=2, T=100, H=4, dk=32, dv=64, dtype=torch.bfloat16)
    a.update({k: v for k, v in kw.items() if k in a})
    p = _lib.make_problem(a["B"], a["T"], a["H"], a["dk"], a["dv"], a["dtype"])
    if "cu_host" in kw:
        p.cu_seqlens, p.n_docs, p.cu_seqlens_host = FAKE, len(kw["cu_host"]) - 1, kw["cu_host"].ctypes.data
    return p


def _fwd(p, q=FAKE, o=FAKE, ws=FAKE, ws_bytes=1 << 40, h0=None):
    P = ctypes.c_void_p
    return _lib.load().kda_linear_fwd(ctypes.byref(p), P(q), P(FAKE), P(FAKE), P(FAKE), P(h0), P(o), None, 1, P(ws),
                                      ws_bytes, None)


def _bwd(p, dO=FAKE, dv=FAKE, ws=FAKE, ws_bytes=1 << 40):
    P = ctypes.c_void_p
    return _lib.load().kda_linear_bwd(ctypes.byref(p), P(FAKE), P(FAKE), P(FAKE), P(FAKE), None, P(dO), None, P(FAKE),
                                      P(FAKE), P(dv), None, None, P(ws), ws_bytes, None)


def test_linear_refusals():
    assert _fwd(_prob(dk=48)) == -2
    assert _fwd(_prob(T=0)) == -1
    assert _fwd(_prob(dtype=torch.float16)) == -1
    assert _fwd(_prob(), q=0) == -1
    assert _fwd(_prob(), o=0) == -1
    assert _fwd(_prob(), q=FAKE + 4) == -3
    assert _fwd(_prob(), h0=FAKE + 8) == -3
    assert _fwd(_prob(), ws=FAKE + 16) == -3
    assert _fwd(_prob(), ws=0) == -5
    assert _fwd(_prob(), ws_bytes=255) == -5
    for bad in ([0, 100], [0, 120, 100, 200], [1, 200], [0, -1, 200]):
        assert _fwd(_prob(cu_host=np.array(bad, np.int32))) == -4
    assert _bwd(_prob(), dO=0) == -1
    assert _bwd(_prob(), dv=0) == -1
    assert _bwd(_prob(), ws_bytes=300) == -5
    assert _bwd(_prob(dv=96)) == -2


def test_linear_workspace_size():
    lib = _lib.load()
    size = lambda fb, **kw: lib.kda_linear_workspace_size(ctypes.byref(_prob(**kw)), fb)  # noqa: E731
    assert 0 < size(0) <= size(1)
    assert size(0) % 256 == 0
    assert size(0, dk=48) == 0 and size(1, T=0) == 0
    assert lib.kda_linear_workspace_size(None, 0) == 0
    # a short batch keeps no segment states; one long row does
    assert size(0, T=200) < 4096 < size(0, B=1, T=65536)


def test_decode_refusals():
    lib = _lib.load()
    P = ctypes.c_void_p

    def call(n=2, H=4, dk=32, dv=64, dt=0, ptr=FAKE, st=FAKE):
        return lib.kda_linear_decode(n, H, dk, dv, dt, 0.0, P(ptr), P(FAKE), P(FAKE), P(FAKE), P(st), P(FAKE), None)
    assert call(n=0) == -1 and call(H=0) == -1 and call(H=5000) == -1 and call(dt=2) == -1
    assert call(ptr=0) == -1 and call(st=0) == -1
    assert call(st=FAKE + 4) == -3
    assert call(dk=16) == -2 and call(dv=32) == -2


def test_layer_norm_refusals():
    lib = _lib.load()
    P = ctypes.c_void_p

    def fwd(n=4, D=8, dt=0, x=FAKE, w=FAKE, mean=None, rstd=None):
        return lib.kda_layer_norm_fwd(n, D, dt, 0.0, P(x), P(w), None, P(FAKE), P(mean), P(rstd), None)

    def bwd(n=4, D=8, dt=0, dy=FAKE, mean=FAKE, ws=FAKE, ws_bytes=1 << 40):
        return lib.kda_layer_norm_bwd(n, D, dt, P(FAKE), P(FAKE), P(dy), P(mean), P(FAKE), P(FAKE), P(FAKE), None, P(ws),
                                      ws_bytes, None)
    assert fwd(n=0) == -1 and fwd(n=-1) == -1 and fwd(D=0) == -1 and fwd(dt=3) == -1 and fwd(D=(1 << 24) + 1) == -2
    assert fwd(x=0) == -1 and fwd(w=0) == -1 and fwd(mean=FAKE) == -1 and fwd(rstd=FAKE) == -1
    assert fwd(x=FAKE + 2) == -3
    assert bwd(dy=0) == -1 and bwd(mean=0) == -1 and bwd(ws=0) == -5 and bwd(ws_bytes=16) == -5
    assert bwd(ws=FAKE + 8) == -3 and bwd(dy=FAKE + 2) == -3
    assert lib.kda_layer_norm_workspace_size(0, 8, 0) == 0
    assert lib.kda_layer_norm_workspace_size(4, 8, 0) >= 2 * 8 * 4


def test_python_entry_points_refuse_host_tensors_and_bad_shapes():
    q = torch.zeros(1, 4, 2, 32)
    v = torch.zeros(1, 4, 2, 64)
    A = torch.zeros(2)
    with pytest.raises(ValueError, match="CUDA"):
        kda.kda_linear_forward(q, q, v, A)
    with pytest.raises(ValueError, match="k must have shape"):
        kda.kda_linear_forward(q, q[:, :3], v, A)
    with pytest.raises(ValueError, match="A_log must have shape"):
        kda.kda_linear_forward(q, q, v, torch.zeros(3))
    with pytest.raises(ValueError, match="two offsets"):
        kda.kda_linear_forward(q, q, v, A, cu_seqlens=torch.zeros(1, dtype=torch.int32))
    cu = torch.tensor([0, 4], dtype=torch.int32)
    with pytest.raises(ValueError, match="cu_seqlens_host has 3"):
        kda.kda_linear_forward(q, q, v, A, cu_seqlens=cu, cu_seqlens_host=torch.tensor([0, 2, 4], dtype=torch.int32))
    with pytest.raises(ValueError, match="int32"):
        kda.kda_linear_forward(q, q, v, A, cu_seqlens=cu, cu_seqlens_host=torch.tensor([0, 4]))
    with pytest.raises(ValueError, match="comes with"):
        kda.kda_linear_forward(q, q, v, A, cu_seqlens_host=cu)
    with pytest.raises(ValueError, match="3 dimensions"):
        kda.kda_linear_decode_step(q, q, v, A, torch.zeros(1, 2, 32, 64))
    with pytest.raises(ValueError, match="CUDA"):
        kda.kda_layer_norm(torch.zeros(2, 8), torch.ones(8))
    with pytest.raises(ValueError, match="last axis"):
        kda.kda_layer_norm(torch.zeros(2, 0), torch.ones(0))


def test_linear_refuses_a_final_state_over_a_saved_h0():
    # every other argument is valid but the workspace, which is checked last: nothing is launched
    P = ctypes.c_void_p
    call = lambda save, h_final: _lib.load().kda_linear_fwd(  # noqa: E731
        ctypes.byref(_prob()), P(FAKE), P(FAKE), P(FAKE), P(FAKE), P(FAKE), P(FAKE), P(h_final), save, None, 0, None)
    assert call(1, FAKE) == -1
    assert call(0, FAKE) == -5 and call(1, 2 * FAKE) == -5


def test_linear_backward_looks_at_the_forward_s_device():
    # tensors of the forward that are not on the current device are refused like any other argument
    q, v = torch.zeros(1, 4, 2, 32), torch.zeros(1, 4, 2, 64)
    ctx = kda.LinearContext(None, q, q, v, torch.zeros(2), None, None, None, None, 1, True)
    with pytest.raises(ValueError, match="q must be a CUDA tensor"):
        kda.kda_linear_backward(ctx, v)
