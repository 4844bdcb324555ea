"""Rotary positions (kda_rotary) against its oracle.

Tolerances: the cosine and sine are off by 2^-21 (the angle by 2^-32 of a turn
and fp32's rounding of it and of the function), the two products and their
sum by 3 * 2^-24 of their magnitudes, at most (|a| + |b|) scale, and the output is rounded
once: 2^-8 (bf16) or 2^-24 (fp32) of the value."""
import numpy as np
import pytest
import torch

import kimi_delta_attention_bwd_gb300 as kda
from oracle import rotary as orot

pytestmark = pytest.mark.gpu
DT = {"bf16": torch.bfloat16, "f32": torch.float32}
ROUND = {"bf16": 2.0 ** -8, "f32": 2.0 ** -24}


def check(y, x, pos, f, dt, interleaved=False, scale=1.0, inverse=False):
    x, y = (t.double().cpu().numpy().reshape(-1, *t.shape[-2:]) for t in (x, y))
    pos, f = np.asarray(pos).reshape(-1), f.double().cpu().numpy()
    r = orot.turn(x, pos, f, interleaved, scale, inverse)
    rot = 2 * f.size
    lim = np.zeros(r.shape)
    a = np.abs(x)
    if interleaved:
        both = np.repeat(a[..., 0:rot:2] + a[..., 1:rot:2], 2, -1)
    else:
        both = np.concatenate([a[..., :rot // 2] + a[..., rot // 2:rot]] * 2, -1)
    lim[..., :rot] = (2.0 ** -21 + 3 * 2.0 ** -24) * scale * both * (1 + ROUND[dt]) + ROUND[dt] * np.abs(r[..., :rot])
    bad = ~(np.abs(y - r) <= lim)
    assert not bad.any(), (int(bad.sum()), np.argwhere(bad)[:4].tolist(), y[bad][:4], r[bad][:4])


def draw(seed, *s, dt):
    return torch.randn(*s, generator=torch.Generator().manual_seed(seed)).to(DT[dt]).cuda()


@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("D,rot", [(64, 64), (128, 128), (128, 64), (128, 16), (64, 2), (64, 30), (6, 4), (10, 10), (192, 64)])
def test_rotary(dt, interleaved, D, rot):
    f, _ = kda.rotary_frequencies(rot, base=500000.0)
    q, k = draw(1, 2, 33, 3, D, dt=dt), draw(2, 2, 33, 1, D, dt=dt)
    pos = np.tile(np.arange(33), 2)
    a, b = kda.kda_rotary(q, k, f, interleaved=interleaved, scale=1.25)
    check(a, q, pos, f, dt, interleaved, 1.25)
    check(b, k, pos, f, dt, interleaved, 1.25)
    a, b = kda.kda_rotary_backward(q, k, f, interleaved=interleaved, scale=1.25)
    check(a, q, pos, f, dt, interleaved, 1.25, True)
    check(b, k, pos, f, dt, interleaved, 1.25, True)


@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("n", [1, 7, 1215, 1216, 5001])
def test_given_positions_far_and_negative(dt, n):
    f, _ = kda.rotary_frequencies(64)
    f[3], f[4] = 2.75, -0.3  # (any finite frequency)
    q, k = draw(3, n, 4, 64, dt=dt), draw(4, n, 2, 64, dt=dt)
    pos = torch.randint(-2 ** 31, 2 ** 31 - 1, (n,), generator=torch.Generator().manual_seed(5)).to(torch.int32)
    pos[0] = 2 ** 31 - 1
    a, b = kda.kda_rotary(q, k, f, positions=pos.cuda())
    check(a, q, pos.numpy(), f, dt)
    check(b, k, pos.numpy(), f, dt)


def test_documents_and_rows():
    f, _ = kda.rotary_frequencies(64)
    lens = [5, 0, 1, 1300, 40, 0]
    cu = torch.tensor([0] + list(np.cumsum(lens)), dtype=torch.int32)
    pos = np.concatenate([np.arange(n) for n in lens])
    q, k = draw(6, 1, sum(lens), 2, 64, dt="bf16"), draw(7, 1, sum(lens), 1, 64, dt="bf16")
    a, b = kda.kda_rotary(q, k, f, cu_seqlens=cu.cuda())
    check(a, q, pos, f, "bf16")
    check(b, k, pos, f, "bf16")
    # the same positions, given
    c, d = kda.kda_rotary(q, k, f, positions=torch.from_numpy(pos).to(torch.int32)[None].cuda())
    assert torch.equal(a, c) and torch.equal(b, d)


@pytest.mark.parametrize("rot", [64, 32, 12])
def test_in_place_and_queries_alone(rot):
    f, _ = kda.rotary_frequencies(rot)
    q, k = draw(8, 3, 50, 2, 64, dt="bf16"), draw(9, 3, 50, 1, 64, dt="bf16")
    a, b = kda.kda_rotary(q, k, f)
    c, none = kda.kda_rotary(q, None, f)
    assert none is None and torch.equal(a, c)
    q2, k2 = q.clone(), k.clone()
    x, y = kda.kda_rotary(q2, k2, f, out_q=q2, out_k=k2)
    assert x is q2 and y is k2 and torch.equal(a, q2) and torch.equal(b, k2)
    with pytest.raises(ValueError, match="together"):
        kda.kda_rotary(q, k, f, out_q=q)
    both = torch.empty(2 * q.numel(), dtype=q.dtype, device="cuda")
    near = both[:q.numel()].view_as(q)
    with pytest.raises(ValueError, match="out_q overlaps q"):
        kda.kda_rotary(near, None, f, out_q=both[64:64 + q.numel()].view_as(q))


def test_a_frequency_that_is_not_finite_shows():
    f, _ = kda.rotary_frequencies(8)
    f[1] = float("inf")
    q = draw(10, 1, 3, 1, 8, dt="f32")
    a, _ = kda.kda_rotary(q, None, f)
    assert torch.isnan(a[..., 1]).all() and torch.isnan(a[..., 5]).all()
    assert torch.isfinite(a[..., [0, 2, 3, 4, 6, 7]]).all()


def test_autograd():
    f, s = kda.rotary_frequencies(32, factor=8.0, scaling="yarn", original_length=128)
    q, k = (draw(i, 2, 20, h, 64, dt="f32").requires_grad_() for i, h in ((11, 4), (12, 2)))
    dq, dk = draw(13, 2, 20, 4, 64, dt="f32"), draw(14, 2, 20, 2, 64, dt="f32")
    a, b = kda.rotary(q, k, f, interleaved=True, scale=s)
    want = kda.kda_rotary_backward(dq, dk, f, interleaved=True, scale=s)
    got = torch.autograd.grad([a, b], [q, k], [dq, dk], retain_graph=True)
    assert all(torch.equal(x, y) for x, y in zip(got, want))
    # one gradient alone, and an inner product with the outputs: the map is linear
    assert torch.equal(torch.autograd.grad(b, k, dk, retain_graph=True)[0], want[1])
    assert torch.equal(torch.autograd.grad(a, q, dq, retain_graph=True)[0], want[0])
    lhs, rhs = float((a.detach().double() * dq).sum()), float((q.detach().double() * want[0]).sum())
    assert abs(lhs - rhs) <= 1e-5 * float(a.detach().norm() * dq.norm())


def test_graph_replay():
    f, _ = kda.rotary_frequencies(64)
    q, k = draw(15, 9, 4, 64, dt="bf16"), draw(16, 9, 2, 64, dt="bf16")
    pos = torch.arange(9, dtype=torch.int32, device="cuda")
    kda.kda_rotary(q, k, f, positions=pos)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        a, b = kda.kda_rotary(q, k, f, positions=pos)
    pos.add_(1000)
    graph.replay()
    c, d = kda.kda_rotary(q, k, f, positions=pos)
    assert torch.equal(a, c) and torch.equal(b, d)


@pytest.mark.parametrize("off", [[0, 80, 70], [1, 30, 70], [0, 30, 71], [0, 30, 69], [0, -5, 70], [0, 71, 70], [70, 0]])
def test_wrong_offsets_show(off):
    f, _ = kda.rotary_frequencies(32)
    q, k = draw(17, 1, 70, 2, 64, dt="bf16"), draw(18, 1, 70, 1, 64, dt="bf16")
    cu = torch.tensor(off, dtype=torch.int32, device="cuda")
    for call in (kda.kda_rotary, kda.kda_rotary_backward):
        a, b = call(q, k, f, cu_seqlens=cu)
        nan = torch.isnan(a[:, :, 0, :32])
        assert nan.any() and torch.equal(nan, torch.isnan(b[:, :, 0, :32]))
        assert torch.equal(a[..., 32:], q[..., 32:]) and torch.equal(b[..., 32:], k[..., 32:])


@pytest.mark.parametrize("n_docs,tokens", [(5000, 5000), (5000, 40), (40, 5000), (3, 1)])
def test_one_wrong_offset_among_many_shows(n_docs, tokens):
    """Wherever it stands: between documents that no token's own search comes to."""
    f, _ = kda.rotary_frequencies(8)
    q = draw(19, 1, tokens, 1, 8, dt="f32")
    r = np.random.RandomState(20)
    good = np.sort(r.randint(0, tokens + 1, n_docs + 1)).astype(np.int32)
    good[0], good[-1] = 0, tokens
    assert torch.isfinite(kda.kda_rotary(q, None, f, cu_seqlens=torch.from_numpy(good).cuda())[0]).all()
    for at in {1, n_docs // 2, n_docs - 1}:
        for wrong in (tokens + 1, -1):
            cu = good.copy()
            cu[at] = wrong
            assert torch.isnan(kda.kda_rotary(q, None, f, cu_seqlens=torch.from_numpy(cu).cuda())[0]).any(), (at, wrong)
