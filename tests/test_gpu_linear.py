"""Linear attention with one decay per head (kda_linear_*) against its oracle.

Tolerances, per element, from M, the oracle on the absolute values of the
inputs (the sum of the magnitudes of the terms of each output):
 - bf16 io.  What enters the fp32 results (states, decay gradient) is split
   into three bf16 parts, 2^-24 of a term; the fp32 sums of at most 64 + 16
   products per chunk add 80 * 2^-23 < 2^-16, over a document's chunks below
   2^-14 M in all.  A bf16 output's terms each pass one computed operand (a
   weighted pair, or the state) that is rounded to bf16 once, half a step is
   2^-8 of it: 2^-8 M more; and the output's own rounding, 2^-8 of the value.
 - fp32 io.  Three parts (2^-24) per operand, six products: below 100 sums per
   chunk and product, 100 * 2^-23 < 2^-16, M; plus 2^-24 of the value.
The decays add a few 2^-23 of a term times a m e^-am <= 1/e, well inside both.
The bound on bf16 outputs above is wider than the kernels need: they keep every
computed operand in two bf16 parts, off by 2^-16 of itself, and
test_outputs_are_rounded_once holds them to that.
"""
import numpy as np
import pytest
import torch

import kimi_delta_attention_bwd_gb300 as kda
from kimi_delta_attention_bwd_gb300 import _lib
from oracle import linear_attention as ola

pytestmark = pytest.mark.gpu

DT = {"bf16": torch.bfloat16, "f32": torch.float32}
REL = {"bf16": 2.0 ** -14, "f32": 2.0 ** -16}
OPERAND = {"bf16": 2.0 ** -8, "f32": 0.0}  # rounding of the operands of the io outputs
ROUND = {"bf16": 2.0 ** -8, "f32": 2.0 ** -24}
SHAPES = [(32, 64), (64, 64), (64, 128), (128, 128)]


def make(seed, docs, H, dk, dv, dt, rows=False, A=None):
    g = torch.Generator().manual_seed(seed)
    N = sum(docs)
    r = lambda *s: torch.randn(*s, generator=g)  # noqa: E731
    B = len(docs) if rows else 1
    x = dict(q=r(B, N // B, H, dk).to(DT[dt]), k=r(B, N // B, H, dk).to(DT[dt]), v=r(B, N // B, H, dv).to(DT[dt]),
             A_log=(torch.linspace(-6.0, 1.0, H) if A is None else torch.tensor(A)).float(),
             h0=r(len(docs), H, dk, dv), dO=r(B, N // B, H, dv).to(DT[dt]), dh=r(len(docs), H, dk, dv))
    x["cu"] = None if rows else torch.tensor([0] + list(np.cumsum(docs)), dtype=torch.int32)
    x["docs"] = docs
    return x


def oracle(x, backward=True, h0=True, dh=True, scale=None):
    H, dk = x["q"].shape[2:]
    cu = [0] + list(np.cumsum(x["docs"]))
    scale = scale or dk ** -0.5
    f = lambda t: t.double().numpy().reshape(-1, *t.shape[2:])  # noqa: E731
    res = {}
    for key, fn in (("ref", lambda t: t), ("mag", np.abs)):
        q, k, v, dO = (fn(f(x[n])) for n in ("q", "k", "v", "dO"))
        a = dict(q=q, k=k, v=v, A_log=x["A_log"].double().numpy(), cu=cu, scale=scale,
                 h0=fn(x["h0"].double().numpy()) if h0 else None)
        o, hf = ola.forward(**a)
        out = dict(o=o, h_final=hf)
        if backward:
            out.update(ola.backward(**a, dO=dO, dh_final=fn(x["dh"].double().numpy()) if dh else None))
        res[key] = out
    return res


def check(got, res, dt, names=None):
    for n, r in res["ref"].items():
        if names is not None and n not in names:
            continue
        g = got[n].detach().double().cpu().numpy().reshape(r.shape)
        lim = REL[dt] * np.abs(res["mag"][n])
        if n in ("o", "dq", "dk", "dv"):
            lim = lim + OPERAND[dt] * np.abs(res["mag"][n]) + ROUND[dt] * np.abs(r)
            lim = lim * (1 + ROUND[dt])  # (the last rounding is of the computed value)
        bad = ~(np.abs(g - r) <= lim + 1e-30)
        assert not bad.any(), (n, int(bad.sum()), g[bad][:4], r[bad][:4], lim[bad][:4])


def run(x, backward=True, h0=True, dh=True, host=True, **kw):
    d = {k: v.cuda() if isinstance(v, torch.Tensor) else v for k, v in x.items()}
    o, hf, ctx = kda.kda_linear_forward(d["q"], d["k"], d["v"], d["A_log"], h0=d["h0"] if h0 else None,
                                        cu_seqlens=d["cu"], cu_seqlens_host=x["cu"] if host else None,
                                        save_for_backward=backward, **kw)
    got = dict(o=o, h_final=hf)
    if backward:
        got.update(kda.kda_linear_backward(ctx, d["dO"], d["dh"] if dh else None))
    torch.cuda.synchronize()
    assert kda.kda_device_status(ctx.workspace) == 0
    return got


@pytest.mark.parametrize("T", [1, 2, 63, 64, 65, 130])
def test_rows(T):
    x = make(T, [T, T], 3, 32, 64, "bf16", rows=True)
    check(run(x), oracle(x), "bf16")


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("dk,dv", SHAPES)
def test_packed_documents(dk, dv, dt):
    # an empty document, single tokens, chunk borders; 300 and 700 tokens are cut into segments of 256
    x = make(dk + dv, [5, 0, 300, 1, 64, 1, 700, 0], 2, dk, dv, dt)
    check(run(x), oracle(x), dt)


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("dk,dv", SHAPES)
def test_rows_cut_into_segments(dk, dv, dt):
    x = make(7 + dk, [577, 577], 2, dk, dv, dt, rows=True)
    check(run(x), oracle(x), dt)


def test_without_states_and_with_a_scale():
    x = make(11, [90, 0, 333], 2, 64, 64, "bf16")
    res = oracle(x, h0=False, dh=False, scale=0.75)
    check(run(x, h0=False, dh=False, scale=0.75), res, "bf16")


def test_offsets_known_on_the_device_alone():
    x = make(12, [10, 500, 0, 33], 2, 32, 64, "bf16")
    a, b = run(x, host=True), run(x, host=False)
    for n in a:
        assert torch.equal(a[n], b[n]), n


@pytest.mark.parametrize("A", [[-np.inf, -30.0], [3.0, 60.0]])
def test_no_decay_and_total_decay(A):
    # no decay: a running sum; a = e^3, e^60: nothing of the token before is left
    x = make(13, [200, 1, 270], 2, 32, 64, "bf16", A=A)
    res = oracle(x)
    if np.isinf(A[0]):  # 0 times the (finite) derivative
        for r in res.values():
            r["dA_log"][0] = 0.0
    check(run(x), res, "bf16")


def test_a_document_does_not_see_its_neighbours():
    docs = [70, 129, 1, 300]
    x = make(14, docs, 2, 64, 128, "bf16")
    y = dict(x)
    for n in ("q", "k", "v", "dO"):  # the neighbours of document 1 hold infinities and NaN
        t = x[n].clone()
        t[:, :70] = float("inf")
        t[:, 199:] = float("nan")
        y[n] = t
    a, b = run(x), run(y)
    for n in ("o", "dq", "dk", "dv"):
        assert torch.equal(a[n][:, 70:199], b[n][:, 70:199]), n
    for n in ("h_final", "dh0"):
        assert torch.equal(a[n][1], b[n][1]), n


def test_gradients_that_are_not_wanted():
    x = make(15, [400, 3], 2, 128, 128, "bf16")
    d = {k: v.cuda() if isinstance(v, torch.Tensor) else v for k, v in x.items()}
    _, _, ctx = kda.kda_linear_forward(d["q"], d["k"], d["v"], d["A_log"], h0=d["h0"], cu_seqlens=d["cu"])
    a = kda.kda_linear_backward(ctx, d["dO"], d["dh"])
    b = kda.kda_linear_backward(ctx, d["dO"], d["dh"], want_dA_log=False, want_dh0=False)
    c = kda.kda_linear_backward(ctx, d["dO"], d["dh"])  # the workspace serves again
    assert b["dA_log"] is None and b["dh0"] is None
    # (with the decay gradient the state enters its products in one more part: the last bits differ)
    check(b, oracle(x), "bf16", names=("dq", "dk", "dv"))
    for n in a:
        assert torch.equal(a[n], c[n]), n


def test_given_outputs_and_states_left_alone():
    x = make(16, [100, 20], 2, 32, 64, "bf16")
    d = {k: v.cuda() if isinstance(v, torch.Tensor) else v for k, v in x.items()}
    out, fin = torch.empty_like(d["v"]), torch.empty_like(d["h0"])
    ref = run(x, backward=False)
    o, hf, ctx = kda.kda_linear_forward(d["q"], d["k"], d["v"], d["A_log"], h0=d["h0"], cu_seqlens=d["cu"], out=out,
                                        final_state=fin, save_for_backward=False)
    assert o is out and hf is fin and torch.equal(o, ref["o"]) and torch.equal(hf, ref["h_final"])
    assert torch.equal(d["h0"].cpu(), x["h0"])
    with pytest.raises(ValueError, match="saved nothing"):
        kda.kda_linear_backward(ctx, d["dO"])
    _, none, _ = kda.kda_linear_forward(d["q"], d["k"], d["v"], d["A_log"], cu_seqlens=d["cu"],
                                        want_final_state=False)
    assert none is None


def test_bad_offsets_on_the_device_do_no_work():
    x = make(17, [60, 60], 2, 32, 64, "bf16")
    d = {k: v.cuda() if isinstance(v, torch.Tensor) else v for k, v in x.items()}
    for bad in ([0, 130, 120], [0, 60, 119], [3, 60, 120]):
        out = torch.full_like(d["v"], 7.0)
        cu = torch.tensor(bad, dtype=torch.int32, device="cuda")
        _, _, ctx = kda.kda_linear_forward(d["q"], d["k"], d["v"], d["A_log"], cu_seqlens=cu, out=out)
        assert kda.kda_device_status(ctx.workspace) == -4
        assert bool((out == 7.0).all())
        kda.kda_linear_backward(ctx, d["dO"])
        assert kda.kda_device_status(ctx.workspace) in (-4, -5)


def test_a_workspace_that_nothing_saved_is_refused():
    x = make(18, [60, 60], 2, 32, 64, "bf16")
    d = {k: v.cuda() if isinstance(v, torch.Tensor) else v for k, v in x.items()}
    _, _, ctx = kda.kda_linear_forward(d["q"], d["k"], d["v"], d["A_log"], cu_seqlens=d["cu"])
    ctx.workspace.zero_()
    kda.kda_linear_backward(ctx, d["dO"])
    assert kda.kda_device_status(ctx.workspace) == -5


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("dk,dv", SHAPES)
def test_decode_continues_a_prompt(dk, dv, dt):
    # the prompt's state, then four single tokens, against one document of all of them
    n, T, H = 3, 70, 2
    x = make(19 + dk, [T + 4] * n, H, dk, dv, dt, rows=True)
    res = oracle(x, backward=False)
    d = {k: v.cuda() if isinstance(v, torch.Tensor) else v for k, v in x.items()}
    cut = lambda t, s: t[:, s].contiguous()  # noqa: E731
    _, state, _ = kda.kda_linear_forward(cut(d["q"], slice(0, T)), cut(d["k"], slice(0, T)),
                                         cut(d["v"], slice(0, T)), d["A_log"], h0=d["h0"], save_for_backward=False)
    outs = [kda.kda_linear_decode_step(cut(d["q"], T + i), cut(d["k"], T + i), cut(d["v"], T + i), d["A_log"], state)
            for i in range(4)]
    o = torch.stack(outs, 1)
    sel = {k: {"o": r["o"].reshape(n, T + 4, H, dv)[:, T:], "h_final": r["h_final"]} for k, r in res.items()}
    check(dict(o=o, h_final=state), sel, dt)


def test_on_another_stream_and_as_a_graph():
    x = make(20, [300, 0, 45], 2, 32, 64, "bf16")
    ref = run(x)
    d = {k: v.cuda() if isinstance(v, torch.Tensor) else v for k, v in x.items()}
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())

    def step():
        o, hf, ctx = kda.kda_linear_forward(d["q"], d["k"], d["v"], d["A_log"], h0=d["h0"], cu_seqlens=d["cu"],
                                            cu_seqlens_host=x["cu"])
        return dict(o=o, h_final=hf, **kda.kda_linear_backward(ctx, d["dO"], d["dh"]))

    with torch.cuda.stream(s):
        a = step()
    s.synchronize()
    for n in ref:
        assert torch.equal(ref[n], a[n]), n
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        b = step()
    keep = d["q"].clone()
    d["q"].zero_()
    g.replay()
    torch.cuda.synchronize()
    assert not bool(b["o"].any())
    d["q"].copy_(keep)
    g.replay()
    torch.cuda.synchronize()
    for n in ref:
        assert torch.equal(ref[n], b[n]), n


def test_autograd_matches_the_direct_calls():
    x = make(21, [130, 1, 300], 2, 64, 64, "bf16")
    ref = run(x)
    d = {k: v.cuda() if isinstance(v, torch.Tensor) else v for k, v in x.items()}
    leaves = [d[n].clone().requires_grad_() for n in ("q", "k", "v", "A_log", "h0")]
    o, hf = kda.linear_attention(*leaves[:4], h0=leaves[4], cu_seqlens=d["cu"], output_final_state=True)
    torch.autograd.backward([o, hf], [d["dO"], d["dh"]])
    assert torch.equal(o, ref["o"]) and torch.equal(hf, ref["h_final"])
    for t, n in zip(leaves, ("dq", "dk", "dv", "dA_log", "dh0")):
        assert torch.equal(t.grad, ref[n]), n
    # the state alone: dO is zero
    fixed = kda.linear_attention(leaves[0].detach(), leaves[1], leaves[2].detach(), d["A_log"], cu_seqlens=d["cu"],
                                 output_final_state=True)[1]
    gk, = torch.autograd.grad(fixed.sum(), [leaves[1]])
    assert bool(torch.isfinite(gk).all()) and bool(gk.any())
    with torch.no_grad():
        assert torch.equal(kda.linear_attention(*leaves[:4], h0=leaves[4], cu_seqlens=d["cu"]), ref["o"])


def test_gradients_against_differences():
    # fp32, a direction per leaf: (L(x + e u) - L(x - e u)) / 2e for the loss in 64 bits
    x = make(22, [100, 30], 2, 32, 64, "f32")
    got = run(x)
    g = torch.Generator().manual_seed(5)

    def loss(**kw):
        y = {**x, **kw}
        r = run(y, backward=False)
        return float((r["o"].double().cpu() * x["dO"].double()).sum() + (r["h_final"].double().cpu() * x["dh"].double()).sum())

    # the loss's own error: 2^-16 of the sum of magnitudes over 2e; both are far below the directional derivative
    mag = oracle(x, backward=False)["mag"]
    noise = 2.0 ** -16 * float((mag["o"] * np.abs(x["dO"].double().numpy().reshape(mag["o"].shape))).sum()
                               + (mag["h_final"] * np.abs(x["dh"].double().numpy())).sum())
    for leaf, grad in (("q", "dq"), ("k", "dk"), ("v", "dv"), ("A_log", "dA_log"), ("h0", "dh0")):
        ref = got[grad].double().cpu().reshape(x[leaf].shape)
        u = ref / ref.norm() + 0.1 * torch.randn(x[leaf].shape, generator=g, dtype=torch.float64) / ref.numel() ** 0.5
        e = 0.25 if leaf != "A_log" else 0.01
        p, m = (x[leaf].double() + s * e * u for s in (1, -1))
        fd = (loss(**{leaf: p.float()}) - loss(**{leaf: m.float()})) / (2 * e)
        want = float((ref * u).sum())
        # the loss is linear in q, v, h0 and k; in A_log the third derivative leaves e^2 / 6 of its size
        lim = noise / e + (2e-3 * abs(want) if leaf == "A_log" else 1e-4 * abs(want))
        assert abs(fd - want) <= lim, (leaf, fd, want, lim)


def test_layer_norm_linear_attention_layer_norm():
    # a block as it would be used: norm of the hidden states, heads, per-head norm of the output
    B, T, H, dk, dv = 2, 90, 2, 32, 64
    g = torch.Generator().manual_seed(23)
    r = lambda *s: torch.randn(*s, generator=g)  # noqa: E731
    hid = r(B, T, H * (2 * dk + dv)).to(torch.bfloat16)
    w1, b1, w2, dy = 1 + 0.1 * r(hid.shape[-1]), 0.1 * r(hid.shape[-1]), 1 + 0.1 * r(dv), r(B, T, H, dv)
    A = torch.tensor([-3.0, -0.5])

    def block(hid, w1, b1, A, w2, ln, attn):
        y = ln(hid, w1, b1)
        q, k, v = (t.reshape(B, T, H, -1).contiguous() for t in y.split([H * dk, H * dk, H * dv], -1))
        return ln(attn(q, k, v, A), w2, None)

    own = [t.cuda().requires_grad_() for t in (hid, w1, b1, A, w2)]
    out = block(*own, kda.layer_norm, kda.linear_attention)
    got = torch.autograd.grad(out, own, dy.cuda().to(torch.bfloat16))

    def ln64(x, w, b):
        z = (x - x.mean(-1, keepdim=True)) / (x.var(-1, unbiased=False, keepdim=True) + 1e-6).sqrt() * w
        return z if b is None else z + b

    def attn64(q, k, v, A):
        i = torch.arange(T)
        w = torch.exp(-torch.exp(A)[:, None, None] * (i[:, None] - i).clamp(min=0)) * (i[:, None] >= i)
        return torch.einsum("bthd,bshd,hts,bshe->bthe", q, k, w, v) * dk ** -0.5

    leaves = [t.double().requires_grad_() for t in (hid, w1, b1, A, w2)]
    ref = block(*leaves, ln64, attn64)
    want = torch.autograd.grad(ref, leaves, dy.to(torch.bfloat16).double())
    # three bf16 roundings lie between the input and an output, six to a gradient, each 2^-8 of its tensor at most
    # and independent from value to value; in the 2-norm: 6 * 2^-8, doubled for the norms' Jacobians
    for a, b in zip([out, *got], [ref, *want]):
        e = (a.double().cpu() - b).norm() / b.norm()
        assert e <= 12 * 2.0 ** -8, float(e)


@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_states_updated_in_place(dt):
    # h_final in h0's place, the long document in pieces that may end in any order
    x = make(30, [1500, 20, 0], 2, 64, 64, dt)
    ref = run(x, backward=False)
    d = {k: v.cuda() if isinstance(v, torch.Tensor) else v for k, v in x.items()}
    for _ in range(5):
        st = d["h0"].clone()
        o, hf, _ = kda.kda_linear_forward(d["q"], d["k"], d["v"], d["A_log"], h0=st, final_state=st,
                                          cu_seqlens=d["cu"], save_for_backward=False)
        assert hf is st and torch.equal(o, ref["o"]) and torch.equal(st, ref["h_final"])
    with pytest.raises(ValueError, match="final_state"):
        kda.kda_linear_forward(d["q"], d["k"], d["v"], d["A_log"], h0=st, final_state=st, cu_seqlens=d["cu"])


@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_a_graph_replayed_on_other_offsets(dt):
    # captured with documents that need no cut, replayed with one that elsewhere would be cut
    x, y = make(31, [200] * 5, 2, 32, 64, dt), make(31, [0, 960, 10, 30, 0], 2, 32, 64, dt)
    d = {k: v.cuda() if isinstance(v, torch.Tensor) else v for k, v in x.items()}
    run(x)

    def step():
        o, hf, ctx = kda.kda_linear_forward(d["q"], d["k"], d["v"], d["A_log"], h0=d["h0"], cu_seqlens=d["cu"],
                                            cu_seqlens_host=x["cu"])
        return dict(o=o, h_final=hf, **kda.kda_linear_backward(ctx, d["dO"], d["dh"]))

    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        got = step()
    for z in (y, x):
        for n in ("q", "k", "v", "A_log", "h0", "cu", "dO", "dh"):
            d[n].copy_(z[n])
        g.replay()
        torch.cuda.synchronize()
        check(got, oracle(z), dt)


@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_more_documents_than_the_table_has_threads(dt):
    docs = [int(n) for n in np.random.default_rng(35).integers(0, 4, 2500)]
    docs[1200] = 600
    x = make(35, docs, 1, 32, 64, dt)
    check(run(x, host=False), oracle(x), dt)


def test_two_calls_at_once():
    # one problem, two streams, a workspace each
    x = make(32, [700, 1, 64, 0, 35], 2, 128, 128, "bf16")
    ref = run(x)
    d = {k: v.cuda() if isinstance(v, torch.Tensor) else v for k, v in x.items()}
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    got = []
    for i in range(6):
        with torch.cuda.stream(streams[i % 2]):
            o, hf, ctx = kda.kda_linear_forward(d["q"], d["k"], d["v"], d["A_log"], h0=d["h0"], cu_seqlens=d["cu"])
            got.append(dict(o=o, h_final=hf, **kda.kda_linear_backward(ctx, d["dO"], d["dh"])))
    torch.cuda.synchronize()
    for a in got:
        for n in ref:
            assert torch.equal(a[n], ref[n]), n


def test_a_training_step_captured_into_a_graph():
    x = make(33, [90, 300], 2, 64, 64, "bf16")
    d = {k: v.cuda() if isinstance(v, torch.Tensor) else v for k, v in x.items()}
    w = torch.linspace(0.5, 1.5, 64, device="cuda")

    def step():
        leaves = [d[n].detach().requires_grad_() for n in ("q", "k", "v", "A_log", "h0")] + [w.detach().requires_grad_()]
        o, hf = kda.linear_attention(*leaves[:4], h0=leaves[4], cu_seqlens=d["cu"], cu_seqlens_host=x["cu"],
                                     output_final_state=True)
        y = kda.layer_norm(o, leaves[5])
        return torch.autograd.grad([y, hf], leaves, [d["dO"], d["dh"]])

    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        ref = [t.clone() for t in step()]
    torch.cuda.current_stream().wait_stream(s)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        got = step()
    for _ in range(2):
        g.replay()
    torch.cuda.synchronize()
    for a, b in zip(ref, got):
        assert torch.equal(a, b)


def test_gradients_that_arrive_unaligned():
    # slices of a larger gradient, and nothing saved where nothing is recorded
    x = make(34, [70], 1, 32, 64, "bf16", rows=True)
    d = {k: v.cuda() if isinstance(v, torch.Tensor) else v for k, v in x.items()}
    ctx = kda.kda_linear_forward(d["q"], d["k"], d["v"], d["A_log"])[2]
    ref = kda.kda_linear_backward(ctx, d["dO"], d["dh"], want_dA_log=False)
    q = d["q"].clone().requires_grad_()
    o, hf = kda.linear_attention(q, d["k"], d["v"], d["A_log"], output_final_state=True)
    buf, hbuf = torch.empty(1 + o.numel(), dtype=o.dtype, device="cuda"), torch.empty(1 + hf.numel(), device="cuda")
    dO, dh = buf[1:].view_as(o).copy_(d["dO"]), hbuf[1:].view_as(hf).copy_(d["dh"])
    gq, = torch.autograd.grad([o, hf], [q], [dO, dh])
    assert torch.equal(gq, ref["dq"])
    y = kda.layer_norm(q, torch.ones(32, device="cuda"))
    gy = torch.empty(1 + y.numel(), dtype=y.dtype, device="cuda")[1:].view_as(y).copy_(d["k"])
    assert bool(torch.isfinite(torch.autograd.grad(y, [q], gy)[0]).all())
    with torch.no_grad():
        before = torch.cuda.memory_allocated()
        torch.cuda.reset_peak_memory_stats()
        kda.linear_attention(q, d["k"], d["v"], d["A_log"])
        ws = torch.cuda.max_memory_allocated() - before - 2 * d["v"].numel()
    prob = _lib.make_problem(1, 70, 1, 32, 64, torch.bfloat16, None, None, None)
    assert ws < _lib.kda_linear_workspace_size(prob, True)


def test_python_refusals_on_the_device():
    x = make(24, [40], 2, 32, 64, "bf16", rows=True)
    d = {k: v.cuda() if isinstance(v, torch.Tensor) else v for k, v in x.items()}
    f = kda.kda_linear_forward
    with pytest.raises(ValueError, match="contiguous"):
        f(d["q"].transpose(1, 2).contiguous().transpose(1, 2), d["k"], d["v"], d["A_log"])
    with pytest.raises(ValueError, match="v must be torch.bfloat16"):
        f(d["q"], d["k"], d["v"].float(), d["A_log"])
    with pytest.raises(kda.KdaError, match="INVALID_ARG"):
        f(d["q"].half(), d["k"].half(), d["v"].half(), d["A_log"])
    with pytest.raises(kda.KdaError, match="UNSUPPORTED"):
        f(d["q"], d["k"], torch.zeros(1, 40, 2, 32, dtype=torch.bfloat16, device="cuda"), d["A_log"])
    with pytest.raises(kda.KdaError, match="WORKSPACE"):
        f(d["q"], d["k"], d["v"], d["A_log"], workspace=torch.empty(64, dtype=torch.uint8, device="cuda"))
    with pytest.raises(kda.KdaError, match="BAD_SEQLENS"):
        bad = torch.tensor([0, 50], dtype=torch.int32)
        f(d["q"], d["k"], d["v"], d["A_log"], cu_seqlens=bad.cuda(), cu_seqlens_host=bad)
    with pytest.raises(kda.KdaError, match="INVALID_ARG"):
        z = torch.zeros(0, 2, 32, dtype=torch.bfloat16, device="cuda")
        kda.kda_linear_decode_step(z, z, torch.zeros(0, 2, 64, dtype=torch.bfloat16, device="cuda"), d["A_log"],
                                   torch.zeros(0, 2, 32, 64, device="cuda"))
    assert _lib.load() is not None


def check_rounded_once(got, res):
    """bf16 outputs y of a value r are its rounding, but where the computed value
    c lies across a border: |y - r| <= |y - c| + d <= |bf16(r) - c| + d <=
    |bf16(r) - r| + 2 d with d = |c - r|.  A term passes at most two computed
    operands, each off by 2^-16, and the fp32 sums of at most 64 + 16 products a
    chunk add as much again (80 * 2^-23): d <= 2^-14 M per element.  In the 2-norm
    the terms' errors are as independent as the terms themselves, whose sum r is:
    d <= (2 * 2^-16 + 2^-16) |r|, below 2^-14 |r|."""
    for n in ("o", "dq", "dk", "dv"):
        r = res["ref"][n]
        g = got[n].double().cpu().numpy().reshape(r.shape)
        once = np.abs(torch.from_numpy(r).to(torch.bfloat16).double().numpy() - r)
        bad = ~(np.abs(g - r) <= once + 2 * 2.0 ** -14 * np.abs(res["mag"][n]) + 1e-30)
        assert not bad.any(), (n, int(bad.sum()))
        e, lim = np.linalg.norm(g - r), np.linalg.norm(once) + 2 * 2.0 ** -14 * np.linalg.norm(r)
        assert e <= lim, (n, e / np.linalg.norm(r), lim / np.linalg.norm(r))


@pytest.mark.parametrize("rows", [False, True])
@pytest.mark.parametrize("dk,dv", SHAPES)
def test_outputs_are_rounded_once(dk, dv, rows):
    docs = [301, 301] if rows else [5, 0, 300, 1, 64, 700]
    x = make(40 + dk + dv, docs, 2, dk, dv, "bf16", rows=rows)
    check_rounded_once(run(x), oracle(x))


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("dk,dv", SHAPES)
def test_unwanted_gradients_leave_the_others_bits(dk, dv, dt):
    # a frozen A_log or an h0 that needs no gradient: dq, dk and dv are what they are with them
    x = make(50 + dk + dv, [70, 400, 3], 2, dk, dv, dt)
    d = {k: v.cuda() if isinstance(v, torch.Tensor) else v for k, v in x.items()}
    _, _, ctx = kda.kda_linear_forward(d["q"], d["k"], d["v"], d["A_log"], h0=d["h0"], cu_seqlens=d["cu"])
    a = kda.kda_linear_backward(ctx, d["dO"], d["dh"])
    b = kda.kda_linear_backward(ctx, d["dO"], d["dh"], want_dA_log=False, want_dh0=False)
    for n in ("dq", "dk", "dv"):
        assert torch.equal(a[n], b[n]), n


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("saved", ["rows", "offsets"])
def test_a_workspace_saved_for_rows_does_not_serve_offsets(saved, dt):
    # the same sizes and as many documents, but another layout of the workspace
    x = make(60, [320, 320], 2, 32, 64, dt, rows=True)
    d = {k: v.cuda() if isinstance(v, torch.Tensor) else v for k, v in x.items()}
    cu = torch.tensor([0, 320, 640], dtype=torch.int32, device="cuda")
    size = max(_lib.kda_linear_workspace_size(_lib.make_problem(2, 320, 2, 32, 64, d["q"].dtype, None, c), True)
               for c in (None, cu))
    _, _, ctx = kda.kda_linear_forward(d["q"], d["k"], d["v"], d["A_log"], cu_seqlens=None if saved == "rows" else cu,
                                       workspace=torch.empty(size, dtype=torch.uint8, device="cuda"))
    assert kda.kda_device_status(ctx.workspace) == 0
    ctx.problem = _lib.make_problem(2, 320, 2, 32, 64, d["q"].dtype, None, cu if saved == "rows" else None)
    kda.kda_linear_backward(ctx, d["dO"])
    assert kda.kda_device_status(ctx.workspace) == -5


@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_a_decay_that_is_not_a_number_shows(dt):
    # a diverged A_log of one head reaches that head's outputs, and no other head's
    x = make(61, [90, 400, 1], 3, 32, 64, dt, A=[-2.0, -1.0, 0.0])
    y = dict(x, A_log=torch.tensor([-2.0, float("nan"), 0.0]))
    a, b = run(x), run(y)
    for n in ("o", "dq", "dv", "h_final", "dh0", "dA_log"):
        g = b[n][:, 1] if n in ("h_final", "dh0") else b[n][1] if n == "dA_log" else b[n][:, :, 1]
        assert bool(torch.isnan(g).all() if n != "dv" else torch.isnan(g[:, :89]).all()), n
    for h in (0, 2):
        for n in ("o", "dq", "dk", "dv"):
            assert torch.equal(a[n][:, :, h], b[n][:, :, h]), n
        for n in ("h_final", "dh0"):
            assert torch.equal(a[n][:, h], b[n][:, h]), n
        assert torch.equal(a["dA_log"][h], b["dA_log"][h])
    d = {k: v.cuda() if isinstance(v, torch.Tensor) else v for k, v in y.items()}
    state = d["h0"].clone()
    o = kda.kda_linear_decode_step(*(d[n][0, :3].contiguous() for n in ("q", "k", "v")), d["A_log"], state)
    assert bool(torch.isnan(o[:, 1]).all()) and bool(torch.isnan(state[:, 1]).all())
    assert bool(torch.isfinite(o[:, ::2]).all()) and bool(torch.isfinite(state[:, ::2]).all())


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("rows", [False, True])
def test_a_document_of_many_pieces(rows, dt):
    # about twenty pieces of 256 tokens and a shorter last one: the fold takes them eight at a time, in place
    docs = [5001] if rows else [40, 5001, 1, 70]
    x = make(70, docs, 1, 32, 64, dt, rows=rows)
    prob = _lib.make_problem(1, sum(docs), 1, 32, 64, x["q"].dtype, None, None if rows else x["cu"])
    prob.cu_seqlens_host = None if rows else x["cu"].data_ptr()
    states = 4 * 32 * 64
    assert _lib.kda_linear_workspace_size(prob, False) > 18 * states  # (a state a piece)
    check(run(x), oracle(x), dt)
    if dt == "bf16":
        check_rounded_once(run(x), oracle(x))


def test_the_workspace_is_a_saved_tensor():
    # freed by the backward while an output lives, and moved by the hooks that move saved tensors
    x = make(71, [700, 1, 300], 2, 64, 64, "bf16")
    d = {k: v.cuda() if isinstance(v, torch.Tensor) else v for k, v in x.items()}
    ref = run(x)
    size = _lib.kda_linear_workspace_size(_lib.make_problem(1, 1001, 2, 64, 64, torch.bfloat16, None, d["cu"]), True)

    def step():
        leaves = [d[n].clone().requires_grad_() for n in ("q", "k", "v", "A_log", "h0")]
        out = kda.linear_attention(*leaves[:4], h0=leaves[4], cu_seqlens=d["cu"], cu_seqlens_host=x["cu"],
                                   output_final_state=True)
        return leaves, out

    leaves, out = step()
    grads = [torch.empty_like(t) for t in leaves]
    before = torch.cuda.memory_allocated()
    for g, t in zip(grads, torch.autograd.grad(out, leaves, [d["dO"], d["dh"]])):
        g.copy_(t)
    del t
    assert before - torch.cuda.memory_allocated() >= size
    with torch.autograd.graph.save_on_cpu():
        leaves, out = step()
    moved = torch.autograd.grad(out, leaves, [d["dO"], d["dh"]])
    for a, b, n in zip(grads, moved, ("dq", "dk", "dv", "dA_log", "dh0")):
        assert torch.equal(a, ref[n]) and torch.equal(b, ref[n]), n


@pytest.mark.parametrize("kind", ["tensor", "array"])
@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_host_offsets_overwritten_between_the_passes(dt, kind):
    # one host buffer for every batch's offsets, the next batch's (nothing to cut) in it before this one's backward
    x = make(72, [600, 0, 100], 2, 32, 64, dt)
    ref = run(x)
    d = {k: v.cuda() if isinstance(v, torch.Tensor) else v for k, v in x.items()}
    host = x["cu"].clone() if kind == "tensor" else x["cu"].numpy().copy()
    _, _, ctx = kda.kda_linear_forward(d["q"], d["k"], d["v"], d["A_log"], h0=d["h0"], cu_seqlens=d["cu"],
                                       cu_seqlens_host=host)
    for i, n in enumerate((0, 240, 480, 700)):
        host[i] = n
    got = kda.kda_linear_backward(ctx, d["dO"], d["dh"])
    assert kda.kda_device_status(ctx.workspace) == 0
    for n in got:
        assert torch.equal(got[n], ref[n]), n


def test_outputs_that_overlap_inputs_are_refused():
    x = make(73, [70, 20], 2, 64, 64, "bf16")
    d = {k: v.cuda() if isinstance(v, torch.Tensor) else v for k, v in x.items()}
    f, size = kda.kda_linear_forward, d["v"].numel()
    for n in ("q", "k", "v"):
        with pytest.raises(ValueError, match=f"out overlaps {n}"):
            f(d["q"], d["k"], d["v"], d["A_log"], cu_seqlens=d["cu"], out=d[n])
    buf = torch.cat([d["v"].flatten(), d["v"].flatten()])
    v = buf[:size].view_as(d["v"]).copy_(d["v"])
    with pytest.raises(ValueError, match="out overlaps v"):
        f(d["q"], d["k"], v, d["A_log"], cu_seqlens=d["cu"], out=buf[size - 64:2 * size - 64].view_as(v))
    ref = f(d["q"], d["k"], d["v"], d["A_log"], cu_seqlens=d["cu"])[0]
    assert torch.equal(ref, f(d["q"], d["k"], v, d["A_log"], cu_seqlens=d["cu"], out=buf[size:].view_as(v))[0])
    states = torch.cat([d["h0"], d["h0"]])
    with pytest.raises(ValueError, match="final_state overlaps h0"):
        f(d["q"], d["k"], d["v"], d["A_log"], h0=states[:2], cu_seqlens=d["cu"], final_state=states[1:3],
          save_for_backward=False)
    # a token's step reads its q, k and v before it writes
    q, k, v = (d[n][0, :3].contiguous() for n in ("q", "k", "v"))
    a, b = d["h0"][:1].repeat(3, 1, 1, 1), d["h0"][:1].repeat(3, 1, 1, 1)
    ref = kda.kda_linear_decode_step(q, k, v, d["A_log"], a)
    for t in (q, k, v):
        b.copy_(d["h0"][:1])
        args = [t if t is u else u.clone() for u in (q, k, v)]
        keep = t.clone()
        assert torch.equal(kda.kda_linear_decode_step(*args, d["A_log"], b, out=t), ref) and torch.equal(a, b)
        t.copy_(keep)
    two = torch.cat([v, v])
    with pytest.raises(ValueError, match="out overlaps v"):
        kda.kda_linear_decode_step(q, k, two[:3], d["A_log"], a, out=two[1:4])
    rows = torch.zeros(9, 64, device="cuda")
    with pytest.raises(ValueError, match="out overlaps x"):
        kda.kda_layer_norm(rows[:8], torch.ones(64, device="cuda"), out=rows[1:])


def test_a_context_dropped_while_another_stream_s_backward_runs():
    # its workspace is not handed out on the forward's stream before that backward has ended (only addresses are
    # compared: nothing is written over it)
    x = make(74, [300, 200], 2, 64, 64, "bf16")
    ref = run(x)
    d = {k: v.cuda() if isinstance(v, torch.Tensor) else v for k, v in x.items()}
    other = torch.cuda.Stream()
    _, _, ctx = kda.kda_linear_forward(d["q"], d["k"], d["v"], d["A_log"], h0=d["h0"], cu_seqlens=d["cu"])
    size, at = ctx.workspace.numel(), ctx.workspace.data_ptr()
    other.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(other):
        torch.cuda._sleep(100_000_000)  # about 50 ms: the backward waits behind it
        got = kda.kda_linear_backward(ctx, d["dO"], d["dh"])
    del ctx
    blocks = [torch.empty(size, dtype=torch.uint8, device="cuda") for _ in range(4)]
    assert all(not at - size < b.data_ptr() < at + size for b in blocks)
    other.synchronize()
    for n in got:
        assert torch.equal(got[n], ref[n]), n
