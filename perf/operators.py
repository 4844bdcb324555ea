"""Performance cases of the linear-attention and layer-norm operators.

Linear attention with one decay per head (A_log [H], decay a = exp(A_log) per token, state dk x dv):
    S_t = exp(-a) S_{t-1} + k_t v_t^T,    o_t = scale S_t^T q_t
as a prompt pass, as a training step and as the single-token step of serving; and layer norm over the last
axis, forward and backward.  `run` computes each case either in plain torch operations (fp32, rounded once at
the end) or, with `own` set, through this package's entry points.  `exact` is the definition in 64 bits.
"""
import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
SIZE = {"bf16": 2, "f32": 4}


def listed():
    return [
        # a chat turn's first token on a small model: one short prompt, where the launches are the time
        dict(name="prompt short", op="linear", step="forward", dtype="bf16", B=1, T=77, H=8, dk=32, dv=64, docs=0),
        # the 300M layer's batch as an inference pass
        dict(name="prompt 300M layer", op="linear", step="forward", dtype="bf16", B=16, T=2048, H=8, dk=32, dv=64,
             docs=0),
        # one long document read into a state: few heads and no batch, so only its length can be shared out
        dict(name="prompt long document", op="linear", step="forward", dtype="bf16", B=1, T=65501, H=8, dk=64, dv=128,
             docs=0),
        # the 300M layer's training step on packed documents (some of length 0 and 1)
        dict(name="train 300M packed", op="linear", step="train", dtype="bf16", B=1, T=32768, H=8, dk=32, dv=64,
             docs=45),
        # the large heads' training step, packed rows
        dict(name="train 128x128 packed", op="linear", step="train", dtype="bf16", B=4, T=8192, H=16, dk=128, dv=128,
             docs=14),
        # a reference run in fp32 with odd row lengths
        dict(name="train f32", op="linear", step="train", dtype="f32", B=4, T=1001, H=8, dk=64, dv=64, docs=0),
        # one user's next token
        dict(name="token one sequence", op="token", dtype="bf16", n=1, H=8, dk=32, dv=64),
        # a full serving batch's next tokens, large heads
        dict(name="token serving batch", op="token", dtype="bf16", n=256, H=16, dk=128, dv=128),
        # the norm in front of a decoded token's layer
        dict(name="norm decode", op="norm", step="forward", dtype="bf16", rows=8, D=1024),
        # the norm of a training batch, both passes
        dict(name="norm train", op="norm", step="train", dtype="bf16", rows=32768, D=2048),
        # the norm over each head's output in fp32: very many short rows
        dict(name="norm per head f32", op="norm", step="train", dtype="f32", rows=262144, D=64),
        # a width that no vector load divides
        dict(name="norm odd width", op="norm", step="train", dtype="bf16", rows=4099, D=5003),
    ]


def _spread(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["linear", "linear", "linear", "token", "norm", "norm"])
    dtype = rng.choice(["bf16", "bf16", "f32"])
    if op == "norm":
        D = _spread(rng, 32, 12000)
        if rng.random() < 0.5:
            D = max(8, D // 8 * 8)
        return dict(op="norm", step=rng.choice(["forward", "train"]), dtype=dtype,
                    rows=_spread(rng, 1, max(1, (1 << 26) // D)), D=D)
    dk, dv = rng.choice([(32, 64), (64, 64), (64, 128), (128, 128)])
    H = rng.randint(1, 16)
    if op == "token":
        return dict(op="token", dtype=dtype, n=_spread(rng, 1, 256), H=H, dk=dk, dv=dv)
    step = rng.choice(["forward", "train"])
    T = _spread(rng, 1, 32768)
    if rng.random() < 0.5:
        B, docs = 1, min(T, _spread(rng, 1, 64))
    else:
        B, docs = rng.randint(1, max(1, min(16, 32768 // T))), 0
    return dict(op="linear", step=step, dtype=dtype, B=B, T=T, H=H, dk=dk, dv=dv, docs=docs)


def _lengths(case, seed):
    """Document lengths over the flattened tokens: the rows, or `docs` pieces of uneven lengths, among them (from
    eight documents on) an empty one and one of a single token."""
    if not case["docs"]:
        return [case["T"]] * case["B"]
    n, d = case["B"] * case["T"], case["docs"]
    g = torch.Generator().manual_seed(seed)
    w = torch.exp(torch.randn(d, generator=g, dtype=torch.float64))
    if d >= 8:
        w[2] = 0.0
        w[5] = 0.0
    cut = torch.floor(torch.cumsum(w, 0) / w.sum() * n).to(torch.int64)
    cut[-1] = n
    lens = torch.diff(cut, prepend=torch.zeros(1, dtype=torch.int64)).tolist()
    if d >= 8:
        big = max(range(d), key=lambda i: lens[i])
        if lens[big] > 1:
            lens[big] -= 1
            lens[5] += 1
    return lens


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    dt = DTYPES[case["dtype"]]

    def normal(*shape, dtype=dt, std=1.0):
        return (torch.randn(*shape, generator=g, device="cuda") * std).to(dtype)

    s = dict(case=case)
    if case["op"] == "norm":
        n, D = case["rows"], case["D"]
        s["x"] = (torch.randn(n, D, generator=g, device="cuda") * 1.5
                  + torch.randn(n, 1, generator=g, device="cuda")).to(dt)
        s["w"] = 1.0 + normal(D, dtype=torch.float32, std=0.1)
        s["bias"] = normal(D, dtype=torch.float32, std=0.1)
        if case["step"] == "train":
            s["dy"] = normal(n, D)
        return s
    H, dk, dv = case["H"], case["dk"], case["dv"]
    # slopes 2^-1 .. 2^-8 over the heads, each off by a learned few percent
    s["A_log"] = (-math.log(2.0) * torch.linspace(1.0, 8.0, H, device="cuda")
                  + 0.05 * torch.randn(H, generator=g, device="cuda")).float()
    if case["op"] == "token":
        n = case["n"]
        s["q"], s["k"], s["v"] = normal(n, H, dk), normal(n, H, dk), normal(n, H, dv)
        s["state"] = normal(n, H, dk, dv, dtype=torch.float32, std=2.0)
        return s
    B, T = case["B"], case["T"]
    s["q"], s["k"], s["v"] = normal(B, T, H, dk), normal(B, T, H, dk), normal(B, T, H, dv)
    lens = _lengths(case, seed)
    s["cu"] = s["cu_host"] = None
    if case["docs"]:
        cu = torch.zeros(len(lens) + 1, dtype=torch.int32)
        cu[1:] = torch.cumsum(torch.tensor(lens), 0)
        s["cu"], s["cu_host"] = cu.cuda(), cu
    s["h0"] = normal(len(lens), H, dk, dv, dtype=torch.float32, std=0.5)
    if case["step"] == "train":
        s["dO"] = normal(B, T, H, dv)
        s["dh"] = normal(len(lens), H, dk, dv, dtype=torch.float32)
    return s


# ---------------------------------------------------------------- plain forms
def _plain_linear(q, k, v, A_log, h0, cu, chunk=64):
    """o, h_final of the flattened tokens [N, H, d] with documents cu, in chunks of the token axis: the pairs of
    a chunk directly, the earlier chunks through a matrix of decays between chunks.  The decays are exponentials
    of token distances, formed in 64 bits."""
    N, H, dk = q.shape
    dv = v.shape[-1]
    pad = (-N) % chunk
    nc = (N + pad) // chunk
    dev = q.device
    a = torch.exp(A_log.double())
    pos = torch.arange(N + pad, device=dev)
    cu = cu.to(device=dev, dtype=torch.int64)
    nd = cu.numel() - 1
    doc = torch.searchsorted(cu[1:].contiguous(), pos, right=True)  # the padding belongs to no document
    if pad:
        q, k, v = (torch.nn.functional.pad(t, (0, 0, 0, 0, 0, pad)) for t in (q, k, v))
    docs_q = doc.clamp(max=nd - 1)
    q, k, v = (t.view(nc, chunk, H, -1).transpose(1, 2) for t in (q, k, v))  # [nc, H, C, d]
    doc, pos = doc.view(nc, chunk), pos.view(nc, chunk)

    def decay(dist, keep):  # exp(-a dist) where keep, else 0, for every head: [H, ...]
        e = torch.exp(-a.view(-1, *[1] * dist.dim()) * dist.clamp(min=0).double())
        return torch.where(keep, e, torch.zeros_like(e)).float()

    d_in = pos[:, :, None] - pos[:, None, :]
    w_in = decay(d_in, (d_in >= 0) & (doc[:, :, None] == doc[:, None, :])).transpose(0, 1)
    o = ((q @ k.transpose(-1, -2)) * w_in) @ v
    # what each chunk adds to the state of the document that runs at its end
    last = pos[:, -1]
    w_out = decay(last[:, None] - pos, doc == doc[:, -1:]).transpose(0, 1)
    kv = (k * w_out[..., None]).transpose(-1, -2) @ v  # [nc, H, dk, dv]
    # the state entering a chunk, for the document that runs at its start
    gap = pos[:, 0][:, None] - 1 - last[None, :]
    w_c = decay(gap, (gap >= 0) & (doc[:, 0][:, None] == doc[:, -1][None, :]))  # [H, nc, nc]
    start = cu[docs_q.view(nc, chunk)]
    ent = (w_c @ kv.transpose(0, 1).reshape(H, nc, dk * dv)).view(H, nc, dk, dv).transpose(0, 1)
    w_row = decay(pos - pos[:, :1] + 1, (doc == doc[:, :1])).transpose(0, 1)
    o = o + (q * w_row[..., None]) @ ent
    # the documents' initial states
    w_h = decay(pos - start + 1, doc < nd).transpose(0, 1)
    rows = q.transpose(1, 2).reshape(N + pad, H, dk) * w_h.transpose(1, 2).reshape(N + pad, H, 1)
    order = torch.arange(N + pad, device=dev)
    slot = order - cu[docs_q]
    longest = int((cu[1:] - cu[:-1]).max())
    wide = torch.zeros(nd, longest, H, dk, device=dev).index_put((docs_q[:N], slot[:N]), rows[:N])
    from_h0 = torch.einsum("nlhi,nhij->nlhj", wide, h0)[docs_q[:N], slot[:N]]
    o = o.transpose(1, 2).reshape(N + pad, H, dv)[:N] + from_h0
    # final states: the initial one decayed, plus the chunks and the tokens of a document's last chunk
    lens = cu[1:] - cu[:-1]
    hf = decay(lens, lens >= 0).transpose(0, 1)[..., None, None] * h0
    end = (cu[1:] - 1).clamp(min=0)
    ce = end // chunk
    gap = end[:, None] - last[None, :]
    own_chunk = (gap >= 0) & (doc[:, -1][None, :] == torch.arange(nd, device=dev)[:, None])
    own_chunk &= (torch.arange(nc, device=dev)[None, :] < ce[:, None]) & (lens > 0)[:, None]
    hf = hf + (decay(gap, own_chunk) @ kv.transpose(0, 1).reshape(H, nc, dk * dv)).view(H, nd, dk, dv).transpose(0, 1)
    gap = end[:, None] - pos[ce]
    w_e = decay(gap, (gap >= 0) & (doc[ce] == torch.arange(nd, device=dev)[:, None])).transpose(0, 1)
    return o, hf + (k[ce] * w_e[..., None]).transpose(-1, -2) @ v[ce]


def _plain_cu(s):
    c = s["case"]
    if s["cu"] is not None:
        return s["cu"]
    return torch.arange(c["B"] + 1, device="cuda") * c["T"]


def _run_plain(s):
    c = s["case"]
    if c["op"] == "norm":
        x, w, D = s["x"].float(), s["w"], c["D"]
        mean = x.mean(-1, keepdim=True)
        xc = x - mean
        r = 1.0 / torch.sqrt((xc * xc).mean(-1, keepdim=True) + 1e-6)
        xh = xc * r
        y = (xh * w + s["bias"]).to(s["x"].dtype)
        if c["step"] == "forward":
            return dict(y=y)
        dy = s["dy"].float()
        g = dy * w
        dx = r * (g - g.mean(-1, keepdim=True) - xh * (g * xh).mean(-1, keepdim=True))
        return dict(y=y, dx=dx.to(s["x"].dtype), dw=(dy * xh).sum(0), dbias=dy.sum(0))
    scale = 1.0 / math.sqrt(c["dk"])
    dt = DTYPES[c["dtype"]]
    if c["op"] == "token":
        q, k, v = (s[n].float() for n in ("q", "k", "v"))
        keep = torch.exp(-torch.exp(s["A_log"].double())).float()[None, :, None, None]
        new = keep * s["state"] + k[..., None] * v[..., None, :]
        s["state"].copy_(new)
        return dict(o=(scale * (q[..., None] * new).sum(-2)).to(dt), state=s["state"])
    H, B, T = c["H"], c["B"], c["T"]
    q, k, v = (s[n].float().view(B * T, H, -1) for n in ("q", "k", "v"))
    if c["step"] == "forward":
        o, hf = _plain_linear(q * scale, k, v, s["A_log"], s["h0"], _plain_cu(s))
        return dict(o=o.to(dt).view(B, T, H, -1), h_final=hf)
    ins = [t.detach().clone().requires_grad_() for t in (q, k, v, s["A_log"], s["h0"])]
    o, hf = _plain_linear(ins[0] * scale, ins[1], ins[2], ins[3], ins[4], _plain_cu(s))
    g = torch.autograd.grad([o, hf], ins, [s["dO"].float().view(B * T, H, -1), s["dh"]])
    return dict(o=o.detach().to(dt).view(B, T, H, -1), h_final=hf.detach(),
                dq=g[0].to(dt).view(B, T, H, -1), dk=g[1].to(dt).view(B, T, H, -1), dv=g[2].to(dt).view(B, T, H, -1),
                dA_log=g[3], dh0=g[4])


# ---------------------------------------------------------------- this package's entry points
def _run_own(s):
    import kimi_delta_attention_bwd_gb300 as kda
    c = s["case"]
    if c["op"] == "norm":
        if c["step"] == "forward":
            return dict(y=kda.kda_layer_norm(s["x"], s["w"], s["bias"]))
        y, mean, rstd = kda.kda_layer_norm(s["x"], s["w"], s["bias"], return_stats=True)
        dx, dw, db = kda.kda_layer_norm_backward(s["x"], s["w"], s["dy"], mean, rstd)
        return dict(y=y, dx=dx, dw=dw, dbias=db)
    if c["op"] == "token":
        o = kda.kda_linear_decode_step(s["q"], s["k"], s["v"], s["A_log"], s["state"])
        return dict(o=o, state=s["state"])
    train = c["step"] == "train"
    o, hf, ctx = kda.kda_linear_forward(s["q"], s["k"], s["v"], s["A_log"], h0=s["h0"], cu_seqlens=s["cu"],
                                        cu_seqlens_host=s["cu_host"], save_for_backward=train)
    if not train:
        return dict(o=o, h_final=hf)
    g = kda.kda_linear_backward(ctx, s["dO"], s["dh"])
    return dict(o=o, h_final=hf, dq=g["dq"], dk=g["dk"], dv=g["dv"], dA_log=g["dA_log"], dh0=g["dh0"])


def run(s):
    return _run_own(s) if own else _run_plain(s)


# ---------------------------------------------------------------- what a pass cannot do without
def work(case):
    e = SIZE[case["dtype"]]
    if case["op"] == "norm":
        n, D = case["rows"], case["D"]
        if case["step"] == "forward":
            return dict(bytes=2 * n * D * e + 8 * D, flops=7 * n * D)
        return dict(bytes=4 * n * D * e + 16 * D, flops=20 * n * D)
    H, dk, dv = case["H"], case["dk"], case["dv"]
    if case["op"] == "token":
        n = case["n"]
        return dict(bytes=n * H * (8 * dk * dv + 2 * (dk + dv) * e) + 4 * H, flops=5 * n * H * dk * dv)
    n = case["B"] * case["T"]
    docs = case["docs"] or case["B"]
    per, st = (2 * dk + 2 * dv) * e, 4 * docs * H * dk * dv
    if case["step"] == "forward":
        return dict(bytes=n * H * per + 2 * st, flops=4 * n * H * dk * dv)
    return dict(bytes=n * H * (per + dv * e + (2 * dk + dv) * e) + 4 * st, flops=16 * n * H * dk * dv)


# ---------------------------------------------------------------- the definition in 64 bits
def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "norm":
        return _exact_norm(s)
    scale = 1.0 / math.sqrt(case["dk"])
    a = torch.exp(s["A_log"].double())
    if case["op"] == "token":
        st = torch.exp(-a)[:, None, None] * s["state"].double()
        st = st + torch.einsum("nhi,nhj->nhij", s["k"].double(), s["v"].double())
        return dict(o=scale * torch.einsum("nhi,nhij->nhj", s["q"].double(), st), state=st)
    return _exact_linear(s, scale, a)


def _exact_norm(s):
    """Row by row in blocks: the mean, the centred second moment, and the derivative of the quotient."""
    x, w = s["x"].double(), s["w"].double()
    n, D = x.shape
    mu = x.sum(1) / D
    var = ((x - mu[:, None]) ** 2).sum(1) / D
    sd = (var + 1e-6).sqrt()
    z = (x - mu[:, None]) / sd[:, None]
    y = z * w + s["bias"].double()
    if s["case"]["step"] == "forward":
        return dict(y=y)
    dy = s["dy"].double()
    dz = dy * w
    dvar = -0.5 * (dz * (x - mu[:, None])).sum(1) / sd ** 3
    dmu = -(dz.sum(1) / sd)
    dx = dz / sd[:, None] + (2.0 / D) * dvar[:, None] * (x - mu[:, None]) + dmu[:, None] / D
    return dict(y=y, dx=dx, dw=torch.einsum("nd,nd->d", dy, z), dbias=dy.sum(0))


def _exact_linear(s, scale, a, block=64):
    """Document after document, block after block: the state carried forward, its gradient carried back."""
    c = s["case"]
    H, dk, dv = c["H"], c["dk"], c["dv"]
    N = c["B"] * c["T"]
    q, k, v = (s[n].double().reshape(N, H, -1).transpose(0, 1) for n in ("q", "k", "v"))  # [H, N, d]
    cu = s["cu_host"].tolist() if s["cu"] is not None else [i * c["T"] for i in range(c["B"] + 1)]
    train = c["step"] == "train"
    o = torch.empty(H, N, dv, dtype=torch.float64, device="cuda")
    hf = torch.empty(len(cu) - 1, H, dk, dv, dtype=torch.float64, device="cuda")
    if train:
        dO = s["dO"].double().reshape(N, H, dv).transpose(0, 1)
        dq, dkk, dvv = torch.empty_like(q), torch.empty_like(k), torch.empty_like(v)
        dh0, dA = torch.empty_like(hf), torch.zeros(H, dtype=torch.float64, device="cuda")
    i = torch.arange(block, device="cuda")
    lower = torch.exp(-a[:, None, None] * (i[:, None] - i[None, :]).clamp(min=0)) * (i[:, None] >= i[None, :])
    for d in range(len(cu) - 1):
        S = s["h0"][d].double()
        cuts = list(range(cu[d], cu[d + 1], block))
        for b in cuts:
            n = min(block, cu[d + 1] - b)
            Q, K, V = q[:, b:b + n], k[:, b:b + n], v[:, b:b + n]
            up = torch.exp(-a[:, None] * (i[:n] + 1))[..., None]
            dn = torch.exp(-a[:, None] * (n - 1 - i[:n]))[..., None]
            L = lower[:, :n, :n]
            o[:, b:b + n] = scale * ((L * (Q @ K.transpose(1, 2))) @ V + up * (Q @ S))
            if train:
                G = dO[:, b:b + n]
                dq[:, b:b + n] = scale * ((L * (G @ V.transpose(1, 2))) @ K + up * (G @ S.transpose(1, 2)))
            S = torch.exp(-a * n)[:, None, None] * S + (dn * K).transpose(1, 2) @ V
        hf[d] = S
        if not train:
            continue
        R = s["dh"][d].double()
        flow = (R * S).sum((1, 2))  # <dS_t, S_t> after the last token, walked back over the document below
        for b in reversed(cuts):
            n = min(block, cu[d + 1] - b)
            Q, K, V, G = q[:, b:b + n], k[:, b:b + n], v[:, b:b + n], dO[:, b:b + n]
            up = torch.exp(-a[:, None] * (i[:n] + 1))[..., None]
            dn = torch.exp(-a[:, None] * (n - 1 - i[:n]))[..., None]
            U = lower[:, :n, :n].transpose(1, 2)
            dkk[:, b:b + n] = scale * ((U * (V @ G.transpose(1, 2))) @ Q) + dn * (V @ R.transpose(1, 2))
            dvv[:, b:b + n] = scale * ((U * (K @ Q.transpose(1, 2))) @ G) + dn * (K @ R)
            R = torch.exp(-a * n)[:, None, None] * R + scale * (up * Q).transpose(1, 2) @ G
            turn = (Q * dq[:, b:b + n]).sum(-1) - (K * dkk[:, b:b + n]).sum(-1)  # [H, n]
            later = torch.flip(torch.cumsum(torch.flip(turn, [1]), 1), [1])
            dA -= (flow[:, None] + later).sum(1)
            flow = flow + turn.sum(1)
        dh0[d] = R
    out = dict(o=o.transpose(0, 1).reshape(c["B"], c["T"], H, dv), h_final=hf)
    if train:
        back = lambda t: t.transpose(0, 1).reshape(c["B"], c["T"], H, -1)  # noqa: E731
        out.update(dq=back(dq), dk=back(dkk), dv=back(dvv), dA_log=a * dA, dh0=dh0)
    return out
