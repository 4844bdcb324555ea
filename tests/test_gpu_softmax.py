"""Softmax attention (kda_softmax_*) against its oracle.

Tolerances, per element, from M, the sum of the magnitudes of an output's terms
(the oracle's second answer), A the largest sum of magnitudes of a logit's
terms, L the longest sum, D the head's width:
 - a logit is a sum of D products in fp32, off by (D + 8) 2^-23 A (2^-23: the
   tensor pipe's sums may truncate); weights are exponentials of differences of
   two of them, by a function good to 2^-22: each is off by
   E = 2 ((D + 8) 2^-23 A) + 2^-20 of itself, and quotients of them by 2 E;
 - the sums over rows or keys add (L + D) 2^-23 M;
 - bf16 io: weights (dv, o) and their gradients (dq, dk) are rounded to bf16
   once, half a step is 2^-8 of each; delta is a sum over o, whose weights were
   rounded too: 2 * 2^-8 M in dq and dk, whose M counts both;
 - the output's own rounding, 2^-8 or 2^-24 of the value.
"""
import numpy as np
import pytest
import torch

import kimi_delta_attention_bwd_gb300 as kda
from oracle import softmax_attention as osm

pytestmark = pytest.mark.gpu

DT = {"bf16": torch.bfloat16, "f32": torch.float32}
ROUND = {"bf16": 2.0 ** -8, "f32": 2.0 ** -24}


def make(seed, lq, lk, Hq, Hkv, D, dt, rows=False, std=1.5):
    g = torch.Generator().manual_seed(seed)
    B = len(lq) if rows else 1
    nq, nk = sum(lq) // B, sum(lk) // B
    r = lambda *s: torch.randn(*s, generator=g)  # noqa: E731
    x = dict(q=(std * r(B, nq, Hq, D)).to(DT[dt]), k=r(B, nk, Hkv, D).to(DT[dt]), v=r(B, nk, Hkv, D).to(DT[dt]),
             dO=r(B, nq, Hq, D).to(DT[dt]))
    off = lambda n: torch.tensor([0] + list(np.cumsum(n)), dtype=torch.int32)  # noqa: E731
    x["cu"], x["cu_k"] = off(lq), off(lk)
    x["rows"], x["same"] = rows, list(lq) == list(lk)
    return x


def flat(t):
    return t.double().numpy().reshape(-1, *t.shape[2:])


def oracle(x, causal=True, backward=True, scale=None):
    D = x["q"].shape[-1]
    return osm.attend(flat(x["q"]), flat(x["k"]), flat(x["v"]), x["cu"].tolist(), x["cu_k"].tolist(),
                      scale or D ** -0.5, causal, flat(x["dO"]) if backward else None)


def run(x, causal=True, backward=True, host=False, scale=None):
    d = {n: t.cuda() if isinstance(t, torch.Tensor) else t for n, t in x.items()}
    kw = {}
    if not x["rows"]:
        kw = dict(cu_seqlens=d["cu"], cu_seqlens_k=None if x["same"] else d["cu_k"])
        if host:
            kw.update(cu_seqlens_host=x["cu"], cu_seqlens_k_host=None if x["same"] else x["cu_k"])
    o, lse, ctx = kda.kda_softmax_forward(d["q"], d["k"], d["v"], scale=scale, causal=causal,
                                          save_for_backward=backward, **kw)
    got = dict(o=o, lse=lse)
    if backward:
        got.update(kda.kda_softmax_backward(ctx, d["dO"]))
    assert kda.kda_device_status(ctx.workspace) == 0
    return got


def limits(ans, dt, D, x, op=None):
    ref, mag, A = ans
    L = max(x["q"].shape[0] * x["q"].shape[1], x["k"].shape[0] * x["k"].shape[1]) + D
    if "dk" in ref:
        L *= x["q"].shape[2] // x["k"].shape[2]
    E = 2 * (D + 8) * 2.0 ** -23 * A + 2.0 ** -20
    R = ROUND[dt]
    op = {"bf16": 2.0 ** -8, "f32": 0.0}[dt] if op is None else op
    lim = {}
    for n, r in ref.items():
        if n == "lse":
            lim[n] = 2 * E + L * 2.0 ** -23 + 2.0 ** -22 * mag[n]
        else:
            lim[n] = (2 * E + L * 2.0 ** -23 + op * (1 if n in ("o", "dv") else 2)) * mag[n] * (1 + R) + R * np.abs(r)
    return lim


def check(got, ans, dt, D, x, op=None):
    for n, lim in limits(ans, dt, D, x, op).items():
        r = ans[0][n]
        g = got[n].detach().double().cpu().numpy().reshape(r.shape)
        same = (g == r) & np.isinf(r)
        bad = ~((np.abs(np.where(same, 0.0, g) - np.where(same, 0.0, r)) <= lim + 1e-30) | same)
        assert not bad.any(), (n, int(bad.sum()), np.argwhere(bad)[:4].tolist(), g[bad][:4], r[bad][:4])


# (query lengths, key lengths): one token to several tiles, tile borders, pieces over prefixes, rows without keys
ROWS = [([1], [1]), ([2], [2]), ([63, 63], [63, 63]), ([64], [64]), ([65], [65]), ([127], [127]), ([128], [128]),
        ([129], [129]), ([255], [255]), ([256], [256]), ([257] * 2, [257] * 2), ([300], [300]), ([515], [515]),
        ([1], [700]), ([130], [389]), ([200], [70]), ([384], [129]), ([5], [1])]
PACKED = [([5], [5]), ([1] * 9, [1] * 9), ([100, 0, 1, 27, 300, 128, 1], None), ([0, 0, 40], None), ([256, 1, 255], None),
          ([7, 130, 0, 64], [200, 130, 33, 5]), ([60, 70], [0, 400]), ([300, 3], [1, 300])]


@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("case", range(len(ROWS)))
def test_rows(dt, D, causal, case):
    lq, lk = ROWS[case]
    Hq, Hkv = [(2, 2), (4, 2), (3, 1)][case % 3]
    x = make(case, lq, lk, Hq, Hkv, D, dt, rows=True)
    check(run(x, causal), oracle(x, causal), dt, D, x)


@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("case", range(len(PACKED)))
def test_packed(dt, D, causal, case):
    lq, lk = PACKED[case]
    Hq, Hkv = [(2, 1), (3, 3), (6, 2)][case % 3]
    x = make(50 + case, lq, lk or lq, Hq, Hkv, D, dt)
    check(run(x, causal, host=case % 2 == 0), oracle(x, causal), dt, D, x)


@pytest.mark.parametrize("dt", ["f32", "bf16"])
def test_many_documents(dt):
    r = np.random.RandomState(5)
    lq = r.randint(0, 7, 3000).tolist()
    lk = [a + int(b) for a, b in zip(lq, r.randint(0, 4, 3000))]
    x = make(6, lq, lk, 2, 1, 64, dt)
    check(run(x), oracle(x), dt, 64, x)


@pytest.mark.parametrize("D", [64, 128])
def test_long_rows(D):
    x = make(7, [2100], [2100], 2, 1, D, "bf16", rows=True)
    check(run(x), oracle(x), "bf16", D, x)


@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("D", [64, 128])
def test_sharp_and_shifted_logits(dt, D):
    """Logits far from zero: a running maximum that grows along the keys, and rows where one key takes all."""
    x = make(8, [400], [400], 2, 2, D, dt, rows=True, std=1.0)
    ramp = torch.linspace(0.0, 40.0, 400)[None, :, None]
    x["q"][..., 0] = (D ** 0.5 * torch.ones(1, 400, 2)).to(DT[dt])
    x["k"][..., 0] = ramp.expand(1, 400, 2).to(DT[dt])
    check(run(x), oracle(x), dt, D, x)
    x["k"][..., 0] = -x["k"][..., 0] * 4  # the largest logits come first, the rest vanish
    check(run(x, causal=False), oracle(x, causal=False), dt, D, x)


@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("lq,lk,rows,causal", [
    ([1], [5000], True, True), ([300], [3001], True, True), ([300], [3001], True, False), ([40] * 3, [1500] * 3, True, True),
    ([130, 0, 9, 1, 300, 60], [4000, 10, 9, 2500, 150, 0], False, True), ([3000, 1], [3000, 1], False, True),
    ([2, 500], [3500, 520], False, False)])
def test_few_queries_on_many_keys(dt, D, lq, lk, rows, causal):
    """Tiles whose keys are cut into pieces and joined, whole ones beside them, and the backward after them."""
    x = make(40, lq, lk, 2, 1, D, dt, rows=rows)
    check(run(x, causal), oracle(x, causal), dt, D, x)


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("lq,lk", [([31], [31]), ([32, 33, 96], [32, 33, 96]), ([97, 1], [63, 65]), ([160], [33]),
                                   ([224, 31], [320, 1])])
@pytest.mark.parametrize("causal", [True, False])
def test_fp32_blocks(D, lq, lk, causal):
    """Borders of the fp32 kernels' smaller blocks."""
    x = make(43, lq, lk, 4, 2, D, "f32")
    check(run(x, causal), oracle(x, causal), "f32", D, x)


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("lq,lk", [([50], [50]), ([1, 2, 40, 64], [1, 2, 40, 64]), ([200, 129, 256], [256, 130, 255])])
@pytest.mark.parametrize("causal", [True, False])
def test_short_documents_take_operands_of_two_parts(D, lq, lk, causal):
    """Few bf16 roundings do not average out: weights and their gradients are off by 2^-16 (two parts), and so is the o
    of delta (its value and what rounding left); the outputs' own rounding remains."""
    x = make(44, lq, lk, 4, 2, D, "bf16")
    check(run(x, causal), oracle(x, causal), "bf16", D, x, op=2.0 ** -16)


@pytest.mark.parametrize("n", [1023, 1024, 1025])
def test_both_sides_of_the_small_problems_border(n):
    x = make(45, [40, n - 40], [40, n - 40], 2, 1, 64, "bf16")
    check(run(x), oracle(x), "bf16", 64, x)


def test_pieces_with_values_that_are_not_finite():
    x = make(41, [3, 200], [4000, 200], 2, 1, 64, "bf16")
    want = run(x, backward=False)
    x["q"][0, 1, 0, 5] = float("nan")
    got = run(x, backward=False)
    assert torch.isnan(got["o"][0, 1, 0]).all() and torch.isnan(got["lse"][0, 1, 0])
    got["o"][0, 1, 0], got["lse"][0, 1, 0] = want["o"][0, 1, 0], want["lse"][0, 1, 0]
    assert torch.equal(got["o"], want["o"]) and torch.equal(got["lse"], want["lse"])


def test_scale_is_used():
    x = make(9, [70], [70], 2, 2, 64, "bf16", rows=True)
    check(run(x, scale=0.4), oracle(x, scale=0.4), "bf16", 64, x)


@pytest.mark.parametrize("T", [2, 8, 40, 200, 700])
@pytest.mark.parametrize("D", [64, 128])
def test_bf16_outputs_are_near_their_rounding(T, D):
    """In the 2-norm the outputs are off by at most 1.5 times what rounding the exact ones to bf16 gives: the
    roundings of the weights (or their gradients) and of the output are independent, sqrt(2), and delta adds little."""
    x = make(10, [T] * max(1, 400 // T), [T] * max(1, 400 // T), 8, 4, D, "bf16")
    got, (ref, _, _) = run(x), oracle(x)
    for n in ("o", "dq", "dk", "dv"):
        r = ref[n]
        rounded = torch.from_numpy(r).to(torch.bfloat16).double().numpy()
        off = np.linalg.norm(got[n].double().cpu().numpy().reshape(r.shape) - r)
        assert off <= 1.5 * np.linalg.norm(rounded - r), (n, off / np.linalg.norm(rounded - r))


@pytest.mark.parametrize("dt", ["f32", "bf16"])
def test_neighbours_do_not_reach(dt):
    """Infinities and NaN in one document leave the others' results as they were, bit for bit."""
    lq, lk = [70, 130, 40], [90, 130, 300]
    x = make(11, lq, lk, 4, 2, 64, dt)
    want = run(x)
    for n, cu in (("q", x["cu"]), ("k", x["cu_k"]), ("v", x["cu_k"]), ("dO", x["cu"])):
        x[n][0, int(cu[1]):int(cu[2])] = float("nan") if n in ("q", "v") else float("inf")
    got = run(x)
    for n in want:
        cu = x["cu_k"] if n in ("dk", "dv") else x["cu"]
        for part in (slice(0, int(cu[1])), slice(int(cu[2]), None)):
            assert torch.equal(got[n][0, part], want[n][0, part]), n
        assert not torch.isfinite(got[n][0, int(cu[1]):int(cu[2])]).all() or n == "lse"


def test_nan_reaches_its_own_row():
    x = make(12, [40], [40], 1, 1, 64, "bf16", rows=True)
    x["q"][0, 17, 0, 3] = float("nan")
    got = run(x, backward=False)
    assert torch.isnan(got["o"][0, 17]).all() and torch.isnan(got["lse"][0, 17]).all()
    rest = [i for i in range(40) if i != 17]
    assert torch.isfinite(got["o"][0, rest]).all()


@pytest.mark.parametrize("dt", ["f32", "bf16"])
def test_two_runs_give_the_same_bits(dt):
    x = make(13, [300, 1, 200], [300, 1, 200], 8, 2, 128, dt)
    a, b = run(x), run(x)
    for n in a:
        assert torch.equal(a[n], b[n]), n


@pytest.mark.parametrize("rows", [True, False])
def test_graph_replay_on_other_values_and_offsets(rows):
    x = make(14, [150, 150], [150, 150], 4, 2, 64, "bf16", rows=rows)
    y = make(15, [150, 150] if rows else [20, 280], [150, 150] if rows else [20, 280], 4, 2, 64, "bf16", rows=rows)
    d = {n: x[n].cuda() for n in ("q", "k", "v", "dO", "cu")}
    cu = None if rows else d["cu"]

    def step():
        o, lse, ctx = kda.kda_softmax_forward(d["q"], d["k"], d["v"], cu_seqlens=cu)
        return dict(o=o, lse=lse, **kda.kda_softmax_backward(ctx, d["dO"]))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step()
    for z in (x, y):
        for n in d:
            d[n].copy_(z[n])
        graph.replay()
        torch.cuda.synchronize()
        want = run(z)
        for n in got:
            assert torch.equal(got[n], want[n]), n


def test_backward_on_another_stream_and_twice():
    x = make(16, [200], [200], 4, 4, 64, "bf16", rows=True)
    want = run(x)
    d = {n: x[n].cuda() for n in ("q", "k", "v", "dO")}
    o, _, ctx = kda.kda_softmax_forward(d["q"], d["k"], d["v"])
    first = kda.kda_softmax_backward(ctx, d["dO"])
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        second = kda.kda_softmax_backward(ctx, d["dO"])
    del ctx
    torch.cuda.synchronize()
    for g in (first, second):
        for n in g:
            assert torch.equal(g[n], want[n]), n


@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_two_streams_at_once(dt):
    """Two problems' steps in flight at once, each on a stream of its own, again and again."""
    xs = [make(46, [700, 0, 300], [700, 0, 300], 4, 2, 128, dt), make(47, [900], [900], 8, 8, 64, dt, rows=True)]
    want = [run(x) for x in xs]
    d = [{n: x[n].cuda() for n in ("q", "k", "v", "dO", "cu")} for x in xs]
    streams = [torch.cuda.Stream() for _ in xs]
    torch.cuda.synchronize()
    got = []
    for _ in range(5):
        for i, s in enumerate(streams):
            with torch.cuda.stream(s):
                o, lse, ctx = kda.kda_softmax_forward(d[i]["q"], d[i]["k"], d[i]["v"],
                                                      cu_seqlens=None if xs[i]["rows"] else d[i]["cu"])
                got.append((i, dict(o=o, lse=lse, **kda.kda_softmax_backward(ctx, d[i]["dO"]))))
                del ctx
    torch.cuda.synchronize()
    for i, g in got:
        for n in g:
            assert torch.equal(g[n], want[i][n]), n


@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_two_graphs_share_a_workspace(dt):
    """A step of each of two problems, captured over one workspace and replayed in turn."""
    xs = [make(48, [200, 100], [200, 100], 4, 2, 128, dt), make(49, [150], [150], 4, 4, 128, dt, rows=True)]
    want = [run(x) for x in xs]
    d = [{n: x[n].cuda() for n in ("q", "k", "v", "dO", "cu")} for x in xs]
    kw = [dict(cu_seqlens=None if x["rows"] else y["cu"]) for x, y in zip(xs, d)]
    size = max(kda.kda_softmax_forward(y["q"], y["k"], y["v"], **k)[2].workspace.numel() for y, k in zip(d, kw))
    shared = torch.empty(size, dtype=torch.uint8, device="cuda")

    def step(i):
        o, lse, ctx = kda.kda_softmax_forward(d[i]["q"], d[i]["k"], d[i]["v"], workspace=shared, **kw[i])
        return dict(o=o, lse=lse, **kda.kda_softmax_backward(ctx, d[i]["dO"]))
    graphs, outs = [], []
    for i in range(2):
        step(i)
        torch.cuda.synchronize()
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1]):
            outs.append(step(i))
    for i in (0, 1, 1, 0):
        graphs[i].replay()
    torch.cuda.synchronize()
    for i in range(2):
        for n in outs[i]:
            assert torch.equal(outs[i][n], want[i][n]), n


def test_a_thread_s_first_call():
    """Threads that have made no CUDA call yet: a forward in one, a backward in another."""
    import threading
    x = make(42, [200], [200], 4, 4, 64, "bf16", rows=True)
    want = run(x)
    d = {n: x[n].cuda() for n in ("q", "k", "v", "dO")}
    torch.cuda.synchronize()
    out = {}

    def forward():
        out["o"], _, out["ctx"] = kda.kda_softmax_forward(d["q"], d["k"], d["v"])

    def backward():
        out.update(kda.kda_softmax_backward(out["ctx"], d["dO"]))
    for f in (forward, backward):
        t = threading.Thread(target=f)
        t.start()
        t.join()
    torch.cuda.synchronize()
    for n in ("o", "dq", "dk", "dv"):
        assert torch.equal(out[n], want[n]), n


def test_more_than_2_31_values():
    """Offsets past 31 bits: the last documents of a long axis give the bits that they give alone (as many of them as
    have too many tiles for any to be cut, which would change the order of sums)."""
    docs, last, L, Hq, D = 3000, 700, 90, 64, 128
    g = torch.Generator(device="cuda").manual_seed(43)
    r = lambda *s: torch.randn(*s, generator=g, device="cuda", dtype=torch.bfloat16)  # noqa: E731
    q, k, v, dO = r(1, docs * L, Hq, D), r(1, docs * L, 1, D), r(1, docs * L, 1, D), r(1, docs * L, Hq, D)
    assert q.numel() > 2 ** 31

    def step(part, n):
        cu = torch.arange(n + 1, dtype=torch.int32, device="cuda") * L
        o, lse, ctx = kda.kda_softmax_forward(*(t[:, part] for t in (q, k, v)), cu_seqlens=cu)
        res = dict(o=o, lse=lse, **kda.kda_softmax_backward(ctx, dO[:, part]))
        assert kda.kda_device_status(ctx.workspace) == 0
        return res
    whole, tail = step(slice(0, None), docs), step(slice((docs - last) * L, None), last)
    for n in tail:
        assert torch.equal(whole[n][:, -last * L:], tail[n]), n
    f, _ = kda.rotary_frequencies(D)
    pos = torch.arange(docs * L, dtype=torch.int32, device="cuda")[None]
    a, _ = kda.kda_rotary(q, None, f, positions=pos)
    b, _ = kda.kda_rotary(q[:, -50:], None, f, positions=pos[:, -50:].contiguous())
    assert torch.equal(a[:, -50:], b)


def test_bad_offsets_and_foreign_workspaces_are_reported():
    x = make(17, [30, 40], [30, 40], 2, 2, 64, "bf16")
    d = {n: x[n].cuda() for n in ("q", "k", "v", "dO")}
    for off in ([0, 80, 70], [1, 30, 70], [0, 30, 71], [0, -5, 70]):
        out = torch.full_like(d["q"], 7.0)
        bad = torch.tensor(off, dtype=torch.int32, device="cuda")
        _, _, ctx = kda.kda_softmax_forward(d["q"], d["k"], d["v"], cu_seqlens=bad, out=out)
        assert kda.kda_device_status(ctx.workspace) == -4
        assert (out == 7.0).all()
        kda.kda_softmax_backward(ctx, d["dO"])
        assert kda.kda_device_status(ctx.workspace) != 0
    # a workspace that another problem's forward saved
    _, _, one = kda.kda_softmax_forward(d["q"], d["k"], d["v"], causal=False)
    _, _, two = kda.kda_softmax_forward(d["q"], d["k"], d["v"], causal=True)
    two.workspace = one.workspace
    kda.kda_softmax_backward(two, d["dO"])
    assert kda.kda_device_status(two.workspace) == -5


def test_autograd_matches_the_calls_and_differences():
    x = make(18, [33, 50], [33, 50], 4, 2, 64, "f32")
    want = run(x)
    d = {n: x[n].cuda() for n in ("q", "k", "v", "dO", "cu")}
    leaves = [d[n].requires_grad_() for n in ("q", "k", "v")]
    o = kda.softmax_attention(*leaves, cu_seqlens=d["cu"])
    g = torch.autograd.grad(o, leaves, d["dO"])
    assert torch.equal(o, want["o"])
    for n, t in zip(("dq", "dk", "dv"), g):
        assert torch.equal(t, want[n]), n
    # without recording nothing is saved, and the bits are the same
    with torch.no_grad():
        assert torch.equal(kda.softmax_attention(*leaves, cu_seqlens=d["cu"]), o)
    # an incoming gradient that is a strided view
    wide = torch.zeros(*o.shape[:-1], 65, device="cuda")
    wide[..., 1:] = d["dO"]
    for t, u in zip(torch.autograd.grad(kda.softmax_attention(*leaves, cu_seqlens=d["cu"]), leaves, wide[..., 1:]), g):
        assert torch.equal(t, u)


def test_a_training_step_captured_into_a_graph():
    """Positions, attention and their gradients through autograd, captured once and replayed on other values."""
    xs = [make(50, [70, 1, 229], [70, 1, 229], 4, 2, 64, "bf16"), make(51, [100, 200, 0], [100, 200, 0], 4, 2, 64, "bf16")]
    d = {n: xs[0][n].cuda() for n in ("q", "k", "v", "dO", "cu")}
    freq = kda.rotary_frequencies(64)[0]

    def step():
        leaves = [d[n].detach().requires_grad_() for n in ("q", "k", "v")]
        q, k = kda.rotary(leaves[0], leaves[1], freq, cu_seqlens=d["cu"])
        o = kda.softmax_attention(q, k, leaves[2], cu_seqlens=d["cu"])
        return [o.detach(), *torch.autograd.grad(o, leaves, d["dO"])]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step()
    for x in xs[::-1]:
        for n in d:
            d[n].copy_(x[n])
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(got, step()):
            assert torch.equal(a, b)


# ---------------------------------------------------------------- single tokens
def decode_case(seed, lens, cap, Hq, Hkv, D, dt):
    g = torch.Generator().manual_seed(seed)
    n = len(lens)
    r = lambda *s: torch.randn(*s, generator=g).to(DT[dt])  # noqa: E731
    return dict(q=(1.5 * torch.randn(n, Hq, D, generator=g)).to(DT[dt]), k=r(n, Hkv, D), v=r(n, Hkv, D),
                k_cache=r(n, cap, Hkv, D), v_cache=r(n, cap, Hkv, D), lengths=torch.tensor(lens, dtype=torch.int32))


def check_decode(x, dt, **kw):
    d = {n: t.cuda() for n, t in x.items()}
    cap, D = x["k_cache"].shape[1], x["q"].shape[-1]
    # places behind the new token hold anything
    for i, n in enumerate(x["lengths"].tolist()):
        if 0 <= n < cap:
            d["k_cache"][i, n + 1:] = float("nan")
            d["v_cache"][i, n + 1:] = float("inf")
    before = {n: d[n].clone() for n in ("k_cache", "v_cache")}
    o = kda.kda_softmax_decode_step(d["q"], d["k"], d["v"], d["k_cache"], d["v_cache"], d["lengths"], **kw)
    for i, n in enumerate(x["lengths"].tolist()):
        if not 0 <= n < cap:
            assert (o[i] == 0).all()
            continue
        for a in ("k", "v"):
            before[a + "_cache"][i, n] = d[a][i]
        K = torch.cat([x["k_cache"][i, :n], x["k"][i:i + 1]])[None]
        V = torch.cat([x["v_cache"][i, :n], x["v"][i:i + 1]])[None]
        one = dict(q=x["q"][i][None, None], k=K, v=V)
        ans = osm.attend(flat(one["q"]), flat(K), flat(V), [0, 1], [0, n + 1], kw.get("scale") or D ** -0.5, True)
        check(dict(o=o[i], lse=torch.from_numpy(ans[0]["lse"])), ans, dt, D, one)
    for n, t in before.items():
        assert torch.equal(d[n].nan_to_num(3.0, 4.0), t.nan_to_num(3.0, 4.0)), n
    return o


@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("heads", [(1, 1), (8, 8), (6, 2), (16, 1), (17, 1), (40, 2)])
def test_decode(dt, D, heads):
    check_decode(decode_case(20, [0, 1, 15, 16, 63, 64, 100, 128, 199], 200, *heads, D, dt), dt)


@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("lens,cap", [([5000], 5001), ([0], 1), ([130], 4096), ([1000, 1, 4095], 4096), ([255] * 70, 256)])
def test_decode_lengths(dt, lens, cap):
    check_decode(decode_case(21, lens, cap, 8, 2, 64, dt), dt)


def test_decode_idle_and_full_sequences():
    x = decode_case(22, [3, -1, 50, 7, 49], 50, 4, 2, 64, "bf16")
    d = {n: t.cuda() for n, t in x.items()}
    from kimi_delta_attention_bwd_gb300 import _lib
    ws = torch.empty(_lib.kda_softmax_decode_workspace_size(5, 50, 4, 2, 64), dtype=torch.uint8, device="cuda")
    check_decode(x, "bf16", workspace=ws)
    assert kda.kda_device_status(ws) == -4  # (a sequence has no room)
    d["lengths"][2] = 9
    kda.kda_softmax_decode_step(*(d[n] for n in ("q", "k", "v", "k_cache", "v_cache", "lengths")), workspace=ws)
    assert kda.kda_device_status(ws) == 0


def test_decode_pieces_agree_with_one_piece():
    """A long cache read in pieces by one sequence, and whole where the sequences fill the GPU."""
    x = decode_case(23, [3000], 3001, 4, 4, 128, "f32")
    a = check_decode(x, "f32")
    many = {n: t.expand(200, *t.shape[1:]).contiguous() for n, t in x.items()}
    d = {n: t.cuda() for n, t in many.items()}
    b = kda.kda_softmax_decode_step(*(d[n] for n in ("q", "k", "v", "k_cache", "v_cache", "lengths")))
    assert torch.allclose(a.expand_as(b), b, rtol=0, atol=2e-6)


def test_decode_in_a_cache_of_more_than_2_31_values():
    g = torch.Generator(device="cuda").manual_seed(44)
    n, cap, H, D = 2, 180000, 48, 128
    kc, vc = (torch.randn(n, cap, H, D, generator=g, device="cuda", dtype=torch.bfloat16) for _ in range(2))
    assert kc.numel() > 2 ** 31
    q, k, v = (torch.randn(n, H, D, generator=g, device="cuda", dtype=torch.bfloat16) for _ in range(3))
    lengths = torch.tensor([5, cap - 1], dtype=torch.int32, device="cuda")
    o = kda.kda_softmax_decode_step(q, k, v, kc, vc, lengths)
    assert torch.equal(kc[1, cap - 1], k[1]) and torch.equal(vc[1, cap - 1], v[1])
    for h in (0, 47):
        p = torch.softmax((q[1, h].double() @ kc[1, :, h].double().T) * D ** -0.5, -1)
        V = vc[1, :, h].double()
        want, mag = p @ V, p @ V.abs()
        # two-part weights (2^-16), fp32 sums over 180000 keys in pieces of below 2^13 (2^-10), the output's rounding
        assert ((o[1, h].double() - want).abs() <= 2.0 ** -10 * mag + 2.0 ** -8 * want.abs()).all()


def test_prompt_then_tokens_is_the_longer_prompt():
    """A prompt through norm, rotary positions and attention into a cache, then tokens one by one, as a captured
    graph that is replayed: the rows of the whole prompt."""
    torch.manual_seed(24)
    B, T, n, Hq, Hkv, D = 2, 37, 5, 4, 2, 64
    f, s = kda.rotary_frequencies(32, base=500000.0, factor=2.0, scaling="yarn", original_length=64)
    x = torch.randn(B, T + n, (Hq + 2 * Hkv) * D, device="cuda")
    w = 1 + 0.1 * torch.randn(D, device="cuda")

    def project(x):
        q, k, v = x.to(torch.bfloat16).split([Hq * D, Hkv * D, Hkv * D], -1)
        q, k, v = (t.unflatten(-1, (-1, D)).contiguous() for t in (q, k, v))
        return kda.kda_layer_norm(q, w), kda.kda_layer_norm(k, w), v
    q, k, v = project(x)
    q, k = kda.kda_rotary(q, k, f, scale=s)
    want, _, _ = kda.kda_softmax_forward(q, k, v, save_for_backward=False)
    kc, vc = (torch.full((B, T + n, Hkv, D), float("nan"), device="cuda", dtype=torch.bfloat16) for _ in range(2))
    kc[:, :T], vc[:, :T] = k[:, :T], v[:, :T]
    lengths = torch.full((B,), T, dtype=torch.int32, device="cuda")
    token = x[:, T].clone()

    def step():
        q, k, v = project(token)
        q, k = kda.kda_rotary(q, k, f, positions=lengths, scale=s)
        o = kda.kda_softmax_decode_step(q, k, v, kc, vc, lengths)
        lengths.add_(1)
        return o
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    lengths.fill_(T)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        o = step()
    lengths.fill_(T)
    for i in range(n):
        token.copy_(x[:, T + i])
        graph.replay()
        # two roundings of each side's weights and two of its outputs, of values below the largest |v|
        assert float((o.float() - want[:, T + i].float()).abs().max()) <= 4 * 2.0 ** -8 * float(v.abs().max())
    assert torch.equal(kc, k) and torch.equal(vc, v) and int(lengths[0]) == T + n


def test_a_hybrid_block_trains():
    """Norm, a linear-attention layer and a softmax-attention layer with rotary positions on packed documents: the
    gradients of all leaves against differences along a random direction."""
    torch.manual_seed(25)
    B, T, Hq, Hkv, D = 1, 150, 4, 2, 64
    cu = torch.tensor([0, 60, 61, 150], dtype=torch.int32, device="cuda")
    f, _ = kda.rotary_frequencies(D)
    x = torch.randn(B, T, Hq * D, device="cuda")
    shapes = dict(w=(Hq * D,), wq=(Hq * D, Hq * D), wk=(Hq * D, Hkv * D), wv=(Hq * D, Hkv * D))
    leaves = {n: (torch.randn(*s, device="cuda") / (Hq * D) ** 0.5).requires_grad_() for n, s in shapes.items()}
    A = torch.linspace(-4.0, -1.0, Hq, device="cuda").requires_grad_()
    leaves["A"] = A
    up = torch.randn(B, T, Hq, D, device="cuda")

    def block(p):
        y = kda.layer_norm(x, 1 + p["w"])
        h = y.view(B, T, Hq, D)
        y = y + kda.linear_attention(h, h, h, p["A"], cu_seqlens=cu).reshape(B, T, Hq * D) * 0.1
        q, k, v = ((y @ p[n]).view(B, T, -1, D) for n in ("wq", "wk", "wv"))
        q, k = kda.rotary(q, k, f, cu_seqlens=cu)
        return (kda.softmax_attention(q, k, v, cu_seqlens=cu) * up).sum()
    names = list(leaves)
    grads = torch.autograd.grad(block(leaves), [leaves[n] for n in names])
    for n, g in zip(names, grads):
        with torch.no_grad():
            step = torch.randn_like(leaves[n])
            h = 2e-3 * float(leaves[n].norm() / step.norm())
            p, m = dict(leaves), dict(leaves)
            p[n], m[n] = leaves[n] + h * step, leaves[n] - h * step
            num = float(block(p).double() - block(m).double()) / (2 * h)
        want = float((g.double() * step.double()).sum())
        # the differences' own error: fp32 noise of a sum of B T Hq D terms over 2 h, and a third derivative's h^2
        scale = float(g.norm() * step.norm())
        assert abs(num - want) <= 2e-2 * scale, (n, num, want, scale)


# ---------------------------------------------------------------- what a backward takes from its forward
def _offsets_of(n):
    return torch.tensor([0] + list(np.cumsum(n)), dtype=torch.int32)


# (whole tiles; tiles that the forward, or both passes, cut into pieces)
BETWEEN = [([100, 0, 1, 199], [100, 0, 1, 199], [1, 198, 100, 1]), ([130, 0, 9, 161], [4000, 10, 9, 1150], [3, 200, 90, 7]),
           ([3000, 1], [3000, 1], [1, 3000])]


@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("case", range(len(BETWEEN)))
def test_offsets_overwritten_between_the_passes(dt, D, case):
    """One buffer of offsets for every batch, the next batch's in it before this one's backward."""
    lq, lk, after = BETWEEN[case]
    x = make(60 + case, lq, lk, 2, 1, D, dt)
    want = run(x)
    d = {n: x[n].cuda() for n in ("q", "k", "v", "dO", "cu", "cu_k")}
    kw = dict(cu_seqlens=d["cu"], cu_seqlens_k=None if x["same"] else d["cu_k"])
    o, lse, ctx = kda.kda_softmax_forward(d["q"], d["k"], d["v"], **kw)
    d["cu"].copy_(_offsets_of(after))
    if not x["same"]:
        d["cu_k"].copy_(d["cu_k"].flip(0).sub(d["cu_k"][-1]).neg())
    got = dict(o=o, lse=lse, **kda.kda_softmax_backward(ctx, d["dO"]))
    assert kda.kda_device_status(ctx.workspace) == 0
    for n in got:
        assert torch.equal(got[n], want[n]), n


@pytest.mark.parametrize("how", ["moved", "recomputed"])
@pytest.mark.parametrize("own_keys", [False, True])
def test_offsets_that_live_in_the_step_alone(how, own_keys):
    """Saved tensors moved to the host, or formed again by a checkpoint, and offsets that the step made and dropped:
    their memory holds others before the backward."""
    from torch.utils.checkpoint import checkpoint
    lq, lk = [100, 0, 1, 199], [100, 20, 31, 349] if own_keys else [100, 0, 1, 199]
    x = make(64, lq, lk, 4, 2, 64, "bf16")
    want = run(x)
    d = {n: x[n].cuda() for n in ("q", "k", "v", "dO")}
    leaves = [d[n].requires_grad_() for n in ("q", "k", "v")]

    def step(q, k, v):
        cu, cu_k = x["cu"].cuda(), x["cu_k"].cuda()
        return kda.softmax_attention(q, k, v, cu_seqlens=cu, cu_seqlens_k=cu_k if own_keys else None)
    if how == "moved":
        with torch.autograd.graph.save_on_cpu():
            o = step(*leaves)
    else:
        o = checkpoint(step, *leaves, use_reentrant=False)
    others = [torch.tensor([0, 300, 300, 300, 300], dtype=torch.int32, device="cuda") for _ in range(64)]
    for n, g in zip(("dq", "dk", "dv"), torch.autograd.grad(o, leaves, d["dO"])):
        assert torch.equal(g, want[n]), n
    assert torch.equal(o, want["o"]) and len(others) == 64


@pytest.mark.parametrize("wanted", [0, 1, 2])
def test_one_gradient_alone(wanted):
    x = make(65, [70, 130], [70, 130], 4, 2, 64, "bf16")
    want = run(x)
    d = {n: x[n].cuda() for n in ("q", "k", "v", "dO", "cu")}
    args = [d[n] for n in ("q", "k", "v")]
    args[wanted].requires_grad_()
    o = kda.softmax_attention(*args, cu_seqlens=d["cu"])
    assert torch.equal(torch.autograd.grad(o, args[wanted], d["dO"])[0], want[("dq", "dk", "dv")[wanted]])


def test_a_graph_s_backward_follows_its_own_forward_s_offsets():
    """The two passes captured apart; the forward replayed on other offsets, the buffer overwritten, the backward
    replayed."""
    xs = [make(66, [150, 150], [150, 150], 4, 2, 64, "bf16"), make(67, [20, 280], [20, 280], 4, 2, 64, "bf16")]
    want = [run(x) for x in xs]
    d = {n: xs[0][n].cuda() for n in ("q", "k", "v", "dO", "cu")}
    kda.kda_softmax_backward(kda.kda_softmax_forward(d["q"], d["k"], d["v"], cu_seqlens=d["cu"])[2], d["dO"])
    torch.cuda.synchronize()
    graphs = [torch.cuda.CUDAGraph(), torch.cuda.CUDAGraph()]
    with torch.cuda.graph(graphs[0]):
        o, lse, ctx = kda.kda_softmax_forward(d["q"], d["k"], d["v"], cu_seqlens=d["cu"])
    with torch.cuda.graph(graphs[1]):
        got = dict(o=o, lse=lse, **kda.kda_softmax_backward(ctx, d["dO"]))
    for x, w in zip(xs, want):
        for n in d:
            d[n].copy_(x[n])
        graphs[0].replay()
        d["cu"].copy_(torch.tensor([0, 77, 300], dtype=torch.int32))
        graphs[1].replay()
        for n in got:
            assert torch.equal(got[n], w[n]), n


@pytest.mark.parametrize("given", [False, True])
def test_a_context_dropped_while_another_stream_s_backward_runs(given):
    """What the forward allocated and the backward reads (workspace and o, or o alone) is not handed out on the forward's
    stream before that backward has ended (only addresses are compared: nothing is written over it)."""
    x = make(68, [300, 200], [300, 200], 4, 2, 64, "bf16")
    want = run(x)
    d = {n: x[n].cuda() for n in ("q", "k", "v", "dO", "cu")}
    ws = kda.kda_softmax_forward(d["q"], d["k"], d["v"], cu_seqlens=d["cu"])[2].workspace if given else None
    other = torch.cuda.Stream()
    o, _, ctx = kda.kda_softmax_forward(d["q"], d["k"], d["v"], cu_seqlens=d["cu"], workspace=ws)
    kept = [(t.data_ptr(), t.numel() * t.element_size()) for t in ((o,) if given else (o, ctx.workspace))]
    other.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(other):
        torch.cuda._sleep(100_000_000)  # about 50 ms: the backward waits behind it
        got = kda.kda_softmax_backward(ctx, d["dO"])
    del ctx, o, _
    for at, size in kept:
        blocks = [torch.empty(size, dtype=torch.uint8, device="cuda") for _ in range(4)]
        assert all(not at - size < b.data_ptr() < at + size for b in blocks)
    other.synchronize()
    for n in got:
        assert torch.equal(got[n], want[n]), n


@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("D", [64, 128])
def test_a_refused_backward_s_gradients_are_not_numbers(dt, D):
    """Offsets that the device refused, and workspaces that other problems' forwards saved: rows and packed, more and
    fewer documents, with cut tiles and without."""
    x = make(69, [30, 40], [30, 40], 4, 2, D, dt)
    d = {n: x[n].cuda() for n in ("q", "k", "v", "dO", "cu")}
    bad = torch.tensor([0, 80, 70], dtype=torch.int32, device="cuda")
    leaves = [d[n].detach().requires_grad_() for n in ("q", "k", "v")]
    o = kda.softmax_attention(*leaves, cu_seqlens=bad)
    for g in torch.autograd.grad(o, leaves, d["dO"]):
        assert torch.isnan(g).all()
    y = make(70, [1] * 9 + [700, 1500], [1] * 9 + [700, 1500], 4, 2, D, dt)
    e = {n: y[n].cuda() for n in ("q", "k", "v", "dO", "cu")}
    short, long = (lambda: kda.kda_softmax_forward(d["q"], d["k"], d["v"], cu_seqlens=d["cu"])[2],
                   lambda **kw: kda.kda_softmax_forward(e["q"], e["k"], e["v"], **kw)[2])
    for ctx, other, dO in ((short(), long(cu_seqlens=e["cu"]), d["dO"]), (short(), long(), d["dO"]),
                           (long(), long(cu_seqlens=e["cu"]), e["dO"]), (long(cu_seqlens=e["cu"]), long(), e["dO"]),
                           (long(cu_seqlens=e["cu"]), long(cu_seqlens=e["cu"], causal=False), e["dO"])):
        ws = torch.zeros(max(ctx.workspace.numel(), other.workspace.numel()), dtype=torch.uint8, device="cuda")
        ws[:other.workspace.numel()] = other.workspace
        ctx.workspace = ws
        for n, g in kda.kda_softmax_backward(ctx, dO).items():
            assert torch.isnan(g).all(), n
        assert kda.kda_device_status(ws) == -5


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("lens,rows", [([50, 1, 64, 256, 200, 2, 40, 255] * 3, False), ([64] * 20, True), ([256] * 5, True)])
@pytest.mark.parametrize("causal", [True, False])
def test_short_documents_of_large_problems_take_two_parts_too(D, lens, rows, causal):
    """The operands' parts follow the document, not the batch that it stands in."""
    assert sum(lens) > 1024
    x = make(71, lens, lens, 4, 2, D, "bf16", rows=rows)
    check(run(x, causal), oracle(x, causal), "bf16", D, x, op=2.0 ** -16)


@pytest.mark.parametrize("D", [64, 128])
def test_each_document_of_a_large_problem_is_near_its_rounding(D):
    """The bound of test_bf16_outputs_are_near_their_rounding, for every document (of two tokens at least: one alone has
    o = v and no gradients of q and k) by itself."""
    lens = [2, 8, 33, 64, 65, 129, 200, 256, 257, 300, 700, 16, 100]
    x = make(72, lens, lens, 8, 4, D, "bf16")
    got, (ref, _, _) = run(x), oracle(x)
    at = np.cumsum([0] + lens)
    for n in ("o", "dq", "dk", "dv"):
        g = got[n].double().cpu().numpy().reshape(ref[n].shape)
        for a, b in zip(at[:-1], at[1:]):
            r = ref[n][a:b]
            rounded = torch.from_numpy(r).to(torch.bfloat16).double().numpy()
            off = np.linalg.norm(g[a:b] - r) / np.linalg.norm(rounded - r)
            assert off <= 1.5, (n, b - a, off)


def test_outputs_and_workspaces_that_overlap_are_refused():
    from kimi_delta_attention_bwd_gb300 import _lib
    x = make(73, [30, 40], [30, 40], 2, 2, 64, "f32")
    d = {n: x[n].cuda() for n in ("q", "k", "v", "dO")}
    n = d["q"].numel()
    both = torch.zeros(2 * n, dtype=torch.int32, device="cuda")
    out = both[:n].view(torch.float32).view_as(d["q"])
    for i in (0, n - 3):
        both[i:i + 3] = x["cu"]
        with pytest.raises(ValueError, match="out overlaps cu_seqlens"):
            kda.kda_softmax_forward(d["q"], d["k"], d["v"], cu_seqlens=both[i:i + 3], out=out)
    cu = both[n:n + 3]  # (right behind it: taken)
    cu.copy_(x["cu"])
    with pytest.raises(ValueError, match="out overlaps cu_seqlens_k"):
        kda.kda_softmax_forward(d["q"], d["k"], d["v"], cu_seqlens=cu, cu_seqlens_k=both[:3], out=out)
    o, _, ctx = kda.kda_softmax_forward(d["q"], d["k"], d["v"], cu_seqlens=cu, out=out)
    assert o is out
    size = ctx.workspace.numel()
    ws = torch.zeros(size + 4 * n, dtype=torch.uint8, device="cuda")
    inside = ws[size:].view(torch.float32).view_as(d["q"])
    for name, kw in (("q", dict(q=inside)), ("k", dict(k=inside)), ("v", dict(v=inside)), ("out", dict(out=inside)),
                     ("cu_seqlens", dict(cu_seqlens=ws[size - 12:size].view(torch.int32)))):
        a = dict(q=d["q"], k=d["k"], v=d["v"], cu_seqlens=cu)
        a.update(kw)
        with pytest.raises(ValueError, match=f"workspace overlaps {name}"):
            kda.kda_softmax_forward(**a, workspace=ws[:size + 256])
    kda.kda_softmax_forward(inside, d["k"], d["v"], cu_seqlens=cu, workspace=ws[:size])

    t = {m: u.cuda() for m, u in decode_case(74, [3, 7], 16, 2, 2, 64, "f32").items()}
    step = lambda **kw: kda.kda_softmax_decode_step(*({**t, **kw}[m] for m in ("q", "k", "v", "k_cache", "v_cache", "lengths")),  # noqa: E731
                                                    **{m: u for m, u in kw.items() if m in ("out", "workspace")})
    size = _lib.kda_softmax_decode_workspace_size(2, 16, 2, 2, 64)
    ws = torch.zeros(size + 4 * t["k_cache"].numel(), dtype=torch.uint8, device="cuda")
    wide, small = ws[size:].view(torch.float32), t["k_cache"].view(-1)
    for match, kw in (("workspace overlaps k_cache", dict(k_cache=wide.view_as(t["k_cache"]), workspace=ws[:size + 256])),
                      ("workspace overlaps q", dict(q=wide[:256].view_as(t["q"]), workspace=ws[:size + 256])),
                      ("workspace overlaps out", dict(out=wide[:256].view_as(t["q"]), workspace=ws[:size + 256])),
                      ("workspace overlaps lengths", dict(lengths=wide[:2].view(torch.int32), workspace=ws[:size + 256])),
                      ("out overlaps lengths", dict(out=wide[:256].view_as(t["q"]), lengths=wide[254:256].view(torch.int32))),
                      ("k_cache overlaps lengths", dict(lengths=small[-2:].view(torch.int32))),
                      ("v_cache overlaps lengths", dict(lengths=t["v_cache"].view(-1)[:2].view(torch.int32)))):
        with pytest.raises(ValueError, match=match):
            step(**kw)
    step(q=wide[:256].view_as(t["q"]), workspace=ws[:size])


def test_a_hybrid_block_s_gradients_are_its_slopes():
    """Norm, a linear-attention layer and a softmax-attention layer with rotary positions on packed documents: the
    difference along each leaf's own gradient is the gradient's norm.  (The loss is a sum in 64 bits of 38400 terms of about
    1 that are off by a few 2^-21 each, about 1e-4 together; h |g| is above 0.02 for every leaf, so that noise is below 0.5%
    of the difference, and the h^2 of a third derivative, with h 0.2% of the leaf, smaller: 2% allows for both.  A gradient
    of the wrong sign is off by 200%, one of another direction by 100%.)"""
    torch.manual_seed(26)
    B, T, Hq, Hkv, D = 1, 150, 4, 2, 64
    cu = torch.tensor([0, 60, 61, 150], dtype=torch.int32, device="cuda")
    f, _ = kda.rotary_frequencies(D)
    x = torch.randn(B, T, Hq * D, device="cuda")
    shapes = dict(w=(Hq * D,), wq=(Hq * D, Hq * D), wk=(Hq * D, Hkv * D), wv=(Hq * D, Hkv * D))
    leaves = {n: (torch.randn(*s, device="cuda") / (Hq * D) ** 0.5).requires_grad_() for n, s in shapes.items()}
    leaves["A"] = torch.linspace(-4.0, -1.0, Hq, device="cuda").requires_grad_()
    up = torch.randn(B, T, Hq, D, device="cuda")

    def block(p):
        y = kda.layer_norm(x, 1 + p["w"])
        h = y.view(B, T, Hq, D)
        y = y + kda.linear_attention(h, h, h, p["A"], cu_seqlens=cu).reshape(B, T, Hq * D) * 0.1
        q, k, v = ((y @ p[n]).view(B, T, -1, D) for n in ("wq", "wk", "wv"))
        q, k = kda.rotary(q, k, f, cu_seqlens=cu)
        return (kda.softmax_attention(q, k, v, cu_seqlens=cu).double() * up).sum()
    names = list(leaves)
    for n, g in zip(names, torch.autograd.grad(block(leaves), [leaves[n] for n in names])):
        with torch.no_grad():
            size = float(g.double().norm())
            h = 2e-3 * float(leaves[n].norm())
            assert h * size > 0.02, (n, h, size)
            p, m = ({**leaves, n: leaves[n] + s * h / size * g} for s in (1, -1))
            num = float(block(p) - block(m)) / (2 * h)
        assert abs(num - size) <= 2e-2 * size, (n, num, size)


@pytest.mark.parametrize("dt", ["f32", "bf16"])
def test_linear_attention_s_backward_reads_no_offsets_either(dt):
    """The forward's table holds its documents: offsets overwritten, or made and dropped by a checkpointed step."""
    from torch.utils.checkpoint import checkpoint
    g = torch.Generator().manual_seed(75)
    off = torch.tensor([0, 700, 701, 1001], dtype=torch.int32)
    q, k, v, dO = (torch.randn(1, 1001, 2, 64, generator=g).to(DT[dt]).cuda() for _ in range(4))
    A = torch.tensor([-3.0, -1.0], device="cuda")
    args = [t.requires_grad_() for t in (q, k, v, A)]
    cu = off.cuda()
    want = torch.autograd.grad(kda.linear_attention(*args, cu_seqlens=cu), args, dO)
    _, _, ctx = kda.kda_linear_forward(*(t.detach() for t in args), cu_seqlens=cu)
    cu.copy_(torch.tensor([0, 3, 500, 1001], dtype=torch.int32))
    for a, b in zip(kda.kda_linear_backward(ctx, dO, want_dh0=False).values(), want):
        assert torch.equal(a, b)
    o = checkpoint(lambda *a: kda.linear_attention(*a, cu_seqlens=off.cuda()), *args, use_reentrant=False)
    others = [torch.tensor([0, 3, 500, 1001], dtype=torch.int32, device="cuda") for _ in range(64)]
    for a, b in zip(torch.autograd.grad(o, args, dO), want):
        assert torch.equal(a, b)
    assert len(others) == 64


@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("lq,lk,rows,causal", [([3000], [40], True, False), ([2500], [100], True, True), ([1500] * 2, [130] * 2, True, False),
                                               ([2000, 0, 700], [64, 5, 129], False, False), ([4000, 3], [1, 5], False, True)])
def test_many_queries_on_few_keys(dt, D, lq, lk, rows, causal):
    """Only the keys' tiles are cut: the forward's table launch has lists of the backward alone.  Two backwards of one
    forward give the same bits."""
    x = make(76, lq, lk, 4, 1, D, dt, rows=rows)
    check(run(x, causal), oracle(x, causal), dt, D, x)
    d = {n: x[n].cuda() for n in ("q", "k", "v", "dO", "cu", "cu_k")}
    kw = {} if rows else dict(cu_seqlens=d["cu"], cu_seqlens_k=d["cu_k"])
    ctx = kda.kda_softmax_forward(d["q"], d["k"], d["v"], causal=causal, **kw)[2]
    one, two = kda.kda_softmax_backward(ctx, d["dO"]), kda.kda_softmax_backward(ctx, d["dO"])
    for n in one:
        assert torch.equal(one[n], two[n]), n


@pytest.mark.parametrize("rows", [False, True])
def test_a_forward_that_saves_nothing_takes_the_workspace(rows):
    """A saving forward's workspace, used by one that does not save: the first one's backward is refused."""
    x = make(77, [600, 600], [600, 600], 4, 2, 64, "bf16", rows=rows)
    d = {n: x[n].cuda() for n in ("q", "k", "v", "dO", "cu")}
    kw = {} if rows else dict(cu_seqlens=d["cu"])
    ctx = kda.kda_softmax_forward(d["q"], d["k"], d["v"], **kw)[2]
    kda.kda_softmax_forward(d["q"], d["k"], d["v"], save_for_backward=False, workspace=ctx.workspace, **kw)
    for n, g in kda.kda_softmax_backward(ctx, d["dO"]).items():
        assert torch.isnan(g).all(), n
    assert kda.kda_device_status(ctx.workspace) == -5
    # and a saving one serves again
    _, _, ctx = kda.kda_softmax_forward(d["q"], d["k"], d["v"], workspace=ctx.workspace, **kw)
    want = run(x)
    for n, g in kda.kda_softmax_backward(ctx, d["dO"]).items():
        assert torch.equal(g, want[n]), n
    assert kda.kda_device_status(ctx.workspace) == 0
