"""Layer norm (kda_layer_norm and its backward) against its oracle.

Tolerances.  The mean of D values is off by at most D-independent tree sums
of 16 serial values and log2 levels, below 32 * 2^-24 of mean |x|; that moves
xh by 2^-19 mean|x| r, and r by as much relatively.  Every output is then a
handful of fp32 operations: 2^-18 (1 + mean|x| r) of its terms' magnitudes,
plus the output type's rounding (bf16 2^-8, fp32 2^-24 of the value).  dw and
db sum n rows in a tree of at most n / blocks + 64 serial values: 2^-16 of the
sum of magnitudes.
"""
import numpy as np
import pytest
import torch

import kimi_delta_attention_bwd_gb300 as kda
from oracle import layer_norm as oln

pytestmark = pytest.mark.gpu

DT = {"bf16": torch.bfloat16, "f32": torch.float32}
ROUND = {"bf16": 2.0 ** -8, "f32": 2.0 ** -24}


def make(seed, n, D, dt, mean=1.0, std=1.5):
    g = torch.Generator().manual_seed(seed)
    r = lambda *s: torch.randn(*s, generator=g)  # noqa: E731
    return dict(x=(std * r(n, D) + mean * r(n, 1)).to(DT[dt]), w=1 + 0.1 * r(D), b=0.1 * r(D), dy=r(n, D).to(DT[dt]))


def limits(x, w, b, dy, dt):
    """(reference, limit) of y, dx, dw, db."""
    f = {k: v.double().numpy() for k, v in dict(x=x, w=w, b=b, dy=dy).items()}
    y = oln.forward(f["x"], f["w"], f["b"])
    dx, dw, db = oln.backward(f["x"], f["w"], f["dy"])
    mu = f["x"].mean(-1, keepdims=True)
    r = 1 / np.sqrt(((f["x"] - mu) ** 2).mean(-1, keepdims=True) + 1e-6)
    xh = np.abs(f["x"] - mu) * r
    e = 2.0 ** -18 * (1 + np.abs(f["x"]).mean(-1, keepdims=True) * r)
    gw = np.abs(f["dy"] * f["w"])
    my = xh * np.abs(f["w"]) + np.abs(f["b"]) + np.abs(f["w"])
    mdx = r * (gw + gw.mean(-1, keepdims=True) + (1 + xh) * (gw * (1 + xh)).mean(-1, keepdims=True))
    return {"y": (y, e * my + ROUND[dt] * np.abs(y)), "dx": (dx, e * mdx + ROUND[dt] * np.abs(dx)),
            "dw": (dw, (np.abs(f["dy"]) * (1 + xh) * (2.0 ** -16 + e)).sum(0)),
            "db": (db, 2.0 ** -16 * np.abs(f["dy"]).sum(0))}


def check(got, lim):
    for n, (ref, tol) in lim.items():
        g = got[n].double().cpu().numpy().reshape(ref.shape)
        bad = ~(np.abs(g - ref) <= tol + 1e-30)
        assert not bad.any(), (n, int(bad.sum()), g[bad][:4], ref[bad][:4], tol[np.broadcast_to(bad, tol.shape)][:4])


def run(t):
    d = {k: v.cuda() for k, v in t.items()}
    y, mean, rstd = kda.kda_layer_norm(d["x"], d["w"], d["b"], return_stats=True)
    dx, dw, db = kda.kda_layer_norm_backward(d["x"], d["w"], d["dy"], mean, rstd)
    torch.cuda.synchronize()
    return dict(y=y, dx=dx, dw=dw, db=db)


# one value, widths around the lane groups, the warp and the CTA, every vector width, both wide paths
@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("n,D", [(5, 1), (3, 2), (130, 3), (1, 16), (1001, 17), (77, 64), (300, 100), (9, 512),
                                 (9, 513), (33, 520), (50, 1000), (700, 1024), (21, 2050), (640, 4096), (7, 5003),
                                 (5, 8192), (6, 8200), (3, 12001), (5, 16384), (3, 16386), (2, 40000)])
def test_matches_oracle(n, D, dt):
    t = make(n + D, n, D, dt)
    check(run(t), limits(**t, dt=dt))


@pytest.mark.parametrize("n,D,dt", [(9, 6001, "bf16"), (9, 6016, "bf16"), (9, 2999, "f32"), (9, 3008, "f32")])
def test_rows_whose_slots_fill_48_kilobytes(n, D, dt):
    t = make(D, n, D, dt)
    check(run(t), limits(t["x"], t["w"], t["b"], t["dy"], dt))


def test_many_short_rows():
    t = make(1, 40003, 64, "f32")
    check(run(t), limits(**t, dt="f32"))


def test_a_mean_far_above_the_spread():
    # 16 bits of the fp32 values hold the mean: the centred second moment keeps what is left
    t = make(2, 64, 1024, "f32", mean=300.0, std=1.0)
    check(run(t), limits(**t, dt="f32"))


def test_constant_rows():
    # no spread: xh = 0, y = bias, dx = (g - mean g) / sqrt(eps)
    t = make(3, 6, 256, "f32")
    t["x"] = torch.full((6, 256), 0.5)
    got = run(t)
    assert torch.equal(got["y"].cpu(), t["b"].expand(6, 256))
    assert not bool(got["dw"].any())
    ref = oln.backward(*(t[k].double().numpy() for k in ("x", "w", "dy")))[0]
    lim = 2.0 ** -18 * 1e3 * np.abs(t["dy"].double().numpy() * t["w"].double().numpy()).max()
    assert np.abs(got["dx"].double().cpu().numpy() - ref).max() <= lim


def test_a_bad_row_stays_alone():
    t = make(4, 40, 300, "bf16")
    u = dict(t, x=t["x"].clone())
    u["x"][7] = float("nan")
    u["x"][8, 3] = float("inf")
    a, b = run(t), run(u)
    keep = [i for i in range(40) if i not in (7, 8)]
    for n in ("y", "dx"):
        assert torch.equal(a[n][keep], b[n][keep]), n


def test_without_bias_shapes_and_outputs():
    t = make(5, 24, 96, "bf16")
    d = {k: v.cuda() for k, v in t.items()}
    x4 = d["x"].view(2, 3, 4, 96)
    y = kda.kda_layer_norm(x4, d["w"])
    assert y.shape == x4.shape
    out = torch.empty_like(x4)
    y2, mean, rstd = kda.kda_layer_norm(x4, d["w"], torch.zeros(96, device="cuda"), out=out, return_stats=True)
    assert y2 is out and torch.equal(y, y2) and mean.shape == (2, 3, 4) and mean.dtype == torch.float32
    dx, dw, db = kda.kda_layer_norm_backward(x4, d["w"], d["dy"].view(x4.shape), mean, rstd, want_dbias=False)
    assert dx.shape == x4.shape and dw.shape == (96,) and db is None
    ref = limits(t["x"], t["w"], torch.zeros(96), t["dy"], "bf16")
    check(dict(y=y, dx=dx, dw=dw), {k: ref[k] for k in ("y", "dx", "dw")})
    # eps large against the variance
    big = kda.kda_layer_norm(x4, d["w"], eps=4.0).double().cpu().numpy().reshape(24, 96)
    r = oln.forward(t["x"].double().numpy(), t["w"].double().numpy(), eps=4.0)
    assert (np.abs(big - r) <= 2.0 ** -8 * np.abs(r) + 2.0 ** -16).all()


@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("n,D", [(700, 64), (37, 1001), (400, 10001), (5, 40003)])
def test_in_place(n, D, dt):
    g = torch.Generator().manual_seed(D)
    x = torch.randn(n, D, generator=g).to(dt).cuda()
    w, b = (torch.randn(D, generator=g).cuda() for _ in range(2))
    y = kda.kda_layer_norm(x, w, b)
    assert kda.kda_layer_norm(x, w, b, out=x) is x and torch.equal(x, y)


def test_deterministic_on_another_stream_and_as_a_graph():
    t = make(6, 3001, 640, "bf16")
    ref = run(t)
    d = {k: v.cuda() for k, v in t.items()}

    def step():
        y, mean, rstd = kda.kda_layer_norm(d["x"], d["w"], d["b"], return_stats=True)
        dx, dw, db = kda.kda_layer_norm_backward(d["x"], d["w"], d["dy"], mean, rstd)
        return dict(y=y, dx=dx, dw=dw, db=db)

    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        a = step()
    s.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        b = step()
    for _ in range(2):
        g.replay()
    torch.cuda.synchronize()
    for n in ref:
        assert torch.equal(ref[n], a[n]) and torch.equal(ref[n], b[n]), n


def test_autograd_matches_the_direct_calls():
    t = make(7, 65, 200, "f32")
    ref = run(t)
    leaves = [t[k].cuda().requires_grad_() for k in ("x", "w", "b")]
    y = kda.layer_norm(*leaves)
    g = torch.autograd.grad(y, leaves, t["dy"].cuda())
    for a, n in zip((y, *g), ("y", "dx", "dw", "db")):
        assert torch.equal(a, ref[n]), n
    kda.layer_norm(*leaves).sum().backward()  # an expanded gradient
    z = kda.layer_norm(leaves[0], leaves[1])
    assert len(torch.autograd.grad(z.sum(), leaves[:2])) == 2


def test_gradient_against_differences():
    t = make(8, 12, 128, "f32")
    got = run(t)
    d = {k: v.cuda() for k, v in t.items()}

    def loss(**kw):
        y = kda.kda_layer_norm(*({**d, **kw}[k] for k in ("x", "w", "b")))
        return float((y.double() * d["dy"].double()).sum())

    for leaf, grad in (("x", "dx"), ("w", "dw"), ("b", "db")):
        u = got[grad] / got[grad].norm()
        e = 1e-2
        fd = (loss(**{leaf: d[leaf] + e * u}) - loss(**{leaf: d[leaf] - e * u})) / (2 * e)
        want = float((got[grad].double() * u.double()).sum())
        # fp32 noise of the loss, 2^-20 of 12 * 128 terms of about 1, over e; e^2 of the third derivative
        assert abs(fd - want) <= 1536 * 2.0 ** -20 / e + 1e-3 * abs(want), (leaf, fd, want)


def test_refusals_on_the_device():
    x = torch.zeros(4, 6, device="cuda")
    w = torch.ones(6, device="cuda")
    f = kda.kda_layer_norm
    with pytest.raises(ValueError, match="contiguous"):
        f(torch.zeros(6, 4, device="cuda").t(), w)
    with pytest.raises(ValueError, match="w must have shape"):
        f(x, torch.ones(5, device="cuda"))
    with pytest.raises(ValueError, match="w must be torch.float32"):
        f(x, w.double())
    with pytest.raises(kda.KdaError, match="INVALID_ARG"):
        f(x.half(), w)
    with pytest.raises(kda.KdaError, match="INVALID_ARG"):
        f(x[:0], w)
    with pytest.raises(kda.KdaError, match="ALIGNMENT"):
        f(torch.zeros(5, 6, device="cuda")[1:], w)
    with pytest.raises(kda.KdaError, match="WORKSPACE"):
        s = torch.zeros(4, device="cuda")
        kda.kda_layer_norm_backward(x, w, x, s, s, workspace=torch.empty(16, dtype=torch.uint8, device="cuda"))


def flat(seed, n, D, dt, spread):
    """Rows around 0.3, which no sum of copies represents exactly."""
    t = make(seed, n, D, dt)
    return dict(t, x=(0.3 + spread * torch.randn(n, D, generator=torch.Generator().manual_seed(D))).to(DT[dt]))


# the bound by path.  Rows in registers: 16 (32 above 8192 columns) serial values and log2 levels per sum, the
# 2^-18 (1 + mean |x| r) of above.  Rows above 16384 columns: compensated sums, and a mean that is corrected by its
# own residual: 2^-24 |mu| r of its last rounding, 2^-24 each of x - mu, r's three operations (half of the
# variance's 2^-22), xh and the product with w, below 2^-21 (1 + mean |x| r) in all.
@pytest.mark.parametrize("spread", [0.0, 1e-4])
@pytest.mark.parametrize("n,D", [(5, 300), (3, 5003), (3, 12001), (3, 40000), (2, 1 << 20)])
@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_rows_of_little_spread(n, D, dt, spread):
    t = flat(n, n, D, dt, spread)
    lim = limits(**t, dt=dt)
    if D > 16384:
        for k, rnd in (("y", ROUND[dt]), ("dx", ROUND[dt])):
            ref, tol = lim[k]
            lim[k] = (ref, (tol - rnd * np.abs(ref)) / 8 + rnd * np.abs(ref))
    check(run(t), lim)


def test_the_widest_rows():
    t = flat(9, 2, 1 << 24, "f32", 1e-4)
    check(run(t), limits(**t, dt="f32"))


# At least three rows to a group of threads, of a number that leaves the last ones ragged: the groups' rows keep
# their columns, the next rows come while one is summed, dw and db are carried over the rows.  Widths with and
# without edges of: lane groups, one-row CTAs, two CTAs per SM (5003, 5120 in bf16), sums in shared memory (8200 to
# 16384, in fp32 with and without room for the next row), rows read in passes.
MANY = [(120001, 17), (40003, 100), (20011, 256), (6007, 513), (4001, 1001), (2503, 2050), (1013, 5003), (1013, 5120),
        (509, 6144), (501, 8200), (501, 10001), (480, 13001), (470, 14400), (470, 16384), (470, 16386), (461, 20001)]


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("n,D", MANY)
def test_many_rows_to_a_group(n, D, dt):
    t = make(n + D, n, D, dt)
    lim = limits(**t, dt=dt)
    check(run(t), lim)
    x = t["x"].cuda()
    kda.kda_layer_norm(x, t["w"].cuda(), t["b"].cuda(), out=x)
    check(dict(y=x), {"y": lim["y"]})
