"""Performance cases of the softmax-attention and rotary-position operators.

Softmax attention with grouped heads (Hq query heads share Hkv key heads), per document with Lq queries and Lk keys:
    o_i = sum_j p_ij v_j,   p_ij = exp(scale q_i k_j - lse_i),   lse_i = log sum_j exp(scale q_i k_j),
over the keys j <= i + Lk - Lq where it is causal, over all keys else; as a prompt pass, as a training step and as
the single-token step over a cache; and rotary positions of queries and keys, both ways.  `run` computes each case
either in plain torch operations (fp32, rounded once at the end) or, with `own` set, through this package's entry
points.  `exact` is the definition in 64 bits.
"""
import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
SIZE = {"bf16": 2, "f32": 4}


def listed():
    return [
        # a chat turn's first token on a small model: one short prompt, where the launches are the time
        dict(name="prompt short", op="attention", step="forward", dtype="bf16", B=1, T=77, Tk=77, Hq=8, Hkv=8, D=64,
             causal=True, docs=0),
        # the 300M layer's batch as an inference pass
        dict(name="prompt 300M batch", op="attention", step="forward", dtype="bf16", B=16, T=2048, Tk=2048, Hq=8, Hkv=8,
             D=64, causal=True, docs=0),
        # one long document with grouped heads
        dict(name="prompt long document", op="attention", step="forward", dtype="bf16", B=1, T=16381, Tk=16381, Hq=16,
             Hkv=4, D=128, causal=True, docs=0),
        # a serving batch that mixes the next pieces of several prompts: every request's queries see its keys so far
        # (one with fewer keys than queries, whose first rows see none; one without queries)
        dict(name="prompt pieces", op="attention", step="forward", dtype="bf16", B=1, T=4096, Tk=30011, Hq=16, Hkv=2,
             D=128, causal=True, docs=11),
        # the 300M layer's training step on packed documents (some of length 0 and 1)
        dict(name="train 300M packed", op="attention", step="train", dtype="bf16", B=1, T=16384, Tk=16384, Hq=8, Hkv=8,
             D=64, causal=True, docs=23),
        # the large heads' training step, grouped
        dict(name="train large heads", op="attention", step="train", dtype="bf16", B=4, T=8192, Tk=8192, Hq=16, Hkv=4,
             D=128, causal=True, docs=0),
        # a reference run in fp32 with odd row lengths, every key seen
        dict(name="train f32", op="attention", step="train", dtype="f32", B=4, T=1001, Tk=1001, Hq=8, Hkv=8, D=64,
             causal=False, docs=0),
        # one user's next token over a short cache
        dict(name="token one sequence", op="token", dtype="bf16", n=1, cap=1024, Hq=8, Hkv=8, D=64),
        # one user's next token at the end of a long document: only the cache's length can be shared out
        dict(name="token long cache", op="token", dtype="bf16", n=1, cap=131072, Hq=16, Hkv=4, D=128),
        # a full serving batch's next tokens, caches of uneven lengths
        dict(name="token serving batch", op="token", dtype="bf16", n=64, cap=8192, Hq=16, Hkv=4, D=128),
        # the positions of a decoded batch: part of each head, interleaved pairs, far positions
        dict(name="rotary decode", op="rotary", step="forward", dtype="bf16", N=64, Hq=16, Hkv=4, D=128, rot=64,
             interleaved=True, docs=0),
        # the positions of a training batch, both ways
        dict(name="rotary train", op="rotary", step="train", dtype="bf16", N=32768, Hq=16, Hkv=4, D=128, rot=128,
             interleaved=False, docs=4),
    ]


def _spread(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["attention", "attention", "attention", "token", "token", "rotary"])
    dtype = rng.choice(["bf16", "bf16", "bf16", "f32"])
    D = rng.choice([64, 128])
    Hkv = rng.choice([1, 2, 3, 4, 8])
    Hq = Hkv * rng.choice([1, 2, 3, 4, 8])
    if op == "rotary":
        rot = rng.choice([D, D, D // 2, D // 4, 2 * rng.randint(1, D // 2)])
        N = _spread(rng, 1, max(1, 4_000_000 // (D * (Hq + Hkv))))
        return dict(op="rotary", step=rng.choice(["forward", "train"]), dtype=dtype, N=N, Hq=Hq, Hkv=Hkv, D=D, rot=rot,
                    interleaved=rng.random() < 0.5, docs=rng.choice([0, min(N, _spread(rng, 1, 32))]))
    if op == "token":
        n = _spread(rng, 1, 64)
        cap = _spread(rng, 1, max(1, min(131072, 120_000_000 // (n * Hkv * D))))
        return dict(op="token", dtype=dtype, n=n, cap=cap, Hq=Hq, Hkv=Hkv, D=D)
    step = rng.choice(["forward", "train"])
    # (fp32 and drawn cases stay well below the listed ones' work)
    T = _spread(rng, 1, 8192 if dtype == "bf16" else 2048)
    causal = rng.random() < 0.75
    if rng.random() < 0.5:
        B, docs = 1, min(T, _spread(rng, 1, 32))
        Tk = T if rng.random() < 0.6 else T + _spread(rng, 1, 4096)
    else:
        B, docs = rng.randint(1, max(1, min(8, 8192 // T))), 0
        Tk = T if rng.random() < 0.6 else _spread(rng, 1, 8192 if dtype == "bf16" else 2048)
    return dict(op="attention", step=step, dtype=dtype, B=B, T=T, Tk=Tk, Hq=Hq, Hkv=Hkv, D=D, causal=causal, docs=docs)


def _pieces(n, d, salt):
    """d uneven lengths that sum to n (from eight on, among them an empty one and one of a single token)."""
    g = torch.Generator().manual_seed(1000 * n + 10 * d + salt)
    w = torch.exp(torch.randn(d, generator=g, dtype=torch.float64))
    if d >= 8:
        w[2] = w[5] = 0.0
    cut = torch.floor(torch.cumsum(w, 0) / w.sum() * n).to(torch.int64)
    cut[-1] = n
    lens = torch.diff(cut, prepend=torch.zeros(1, dtype=torch.int64)).tolist()
    if d >= 8:
        big = max(range(d), key=lambda i: lens[i])
        if lens[big] > 1:
            lens[big] -= 1
            lens[5] += 1
    return lens


def _lengths(case):
    """(query lengths, key lengths) of the case's documents: its plan, the same for every seed.  With keys of their
    own, each document's keys are its queries and a prefix, but for one that has fewer keys than queries."""
    if not case["docs"]:
        return [case["T"]] * case["B"], [case["Tk"]] * case["B"]
    lq = _pieces(case["T"], case["docs"], 1)
    if case["Tk"] == case["T"]:
        return lq, list(lq)
    lk = [a + b for a, b in zip(lq, _pieces(case["Tk"] - case["T"], case["docs"], 2))]
    if len(lk) >= 2:
        few, many = (max(range(len(lq)), key=lambda i: lq[i]), min(range(len(lq)), key=lambda i: lk[i]))
        if few != many:
            lk[many] += lk[few] - lq[few] // 2
            lk[few] = lq[few] // 2
    return lq, lk


def _cache_lengths(case):
    """Tokens in each sequence's cache before the step: half full to full, the first one full, the second empty."""
    g = torch.Generator().manual_seed(31 * case["n"] + case["cap"])
    u = torch.rand(case["n"], generator=g, dtype=torch.float64) * 0.5 + 0.5
    n = torch.floor(u * case["cap"]).to(torch.int32).clamp(max=case["cap"] - 1)
    n[0] = case["cap"] - 1
    if case["n"] > 1:
        n[1] = 0
    return n


def _offsets(lens):
    cu = torch.zeros(len(lens) + 1, dtype=torch.int32)
    cu[1:] = torch.cumsum(torch.tensor(lens), 0)
    return cu


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    dt = DTYPES[case["dtype"]]

    def normal(*shape, std=1.0):
        return (torch.randn(*shape, generator=g, device="cuda") * std).to(dt)

    s = dict(case=case)
    Hq, Hkv, D = case["Hq"], case["Hkv"], case["D"]
    if case["op"] == "rotary":
        N, rot = case["N"], case["rot"]
        s["q"], s["k"] = normal(1, N, Hq, D), normal(1, N, Hkv, D)
        # a base of 500000 for long contexts, its frequencies held in fp32 as a model's buffer holds them
        s["inv_freq"] = (500000.0 ** (-torch.arange(0, rot, 2, dtype=torch.float64) / rot)).float().cuda()
        s["cu"] = s["pos"] = None
        if case["docs"]:
            s["cu"] = _offsets(_pieces(N, case["docs"], 3)).cuda()
        else:  # a decoded batch: every token somewhere in its own context, up to a million tokens in
            s["pos"] = torch.randint(0, 1 << 20, (1, N), generator=g, device="cuda", dtype=torch.int32)
        if case["step"] == "train":
            s["dq"], s["dk"] = normal(1, N, Hq, D), normal(1, N, Hkv, D)
        return s
    if case["op"] == "token":
        n, cap = case["n"], case["cap"]
        s["q"], s["k"], s["v"] = normal(n, Hq, D, std=1.5), normal(n, Hkv, D), normal(n, Hkv, D)
        s["k_cache"], s["v_cache"] = normal(n, cap, Hkv, D), normal(n, cap, Hkv, D)
        s["lengths"] = _cache_lengths(case).cuda()
        return s
    B, T, Tk = case["B"], case["T"], case["Tk"]
    # logits of a standard deviation of 1.5: some keys matter much more than others
    s["q"], s["k"], s["v"] = normal(B, T, Hq, D, std=1.5), normal(B, Tk, Hkv, D), normal(B, Tk, Hkv, D)
    s["cu"] = s["cu_k"] = None
    if case["docs"]:
        lq, lk = _lengths(case)
        s["cu"] = _offsets(lq).cuda()
        s["cu_k"] = _offsets(lk).cuda() if Tk != T else None
    if case["step"] == "train":
        s["dO"] = normal(B, T, Hq, D)
    return s


# ---------------------------------------------------------------- plain forms
def _plain_seen(s):
    """[1 or B, T, Tk]: which keys each query sees."""
    c = s["case"]
    i, j = torch.arange(c["T"], device="cuda"), torch.arange(c["Tk"], device="cuda")
    if not c["docs"]:
        seen = j[None, :] <= i[:, None] + (c["Tk"] - c["T"])
        return (seen if c["causal"] else torch.ones_like(seen))[None]
    cu = s["cu"].long()
    cu_k = cu if s["cu_k"] is None else s["cu_k"].long()
    dq = torch.searchsorted(cu[1:].contiguous(), i, right=True)
    dk = torch.searchsorted(cu_k[1:].contiguous(), j, right=True)
    seen = dq[:, None] == dk[None, :]
    if c["causal"]:
        ends = i - cu[1:][dq] + cu_k[1:][dq]  # the last key that a query sees, in the packed axis
        seen &= j[None, :] <= ends[:, None]
    return seen[None]


def _plain_attention(s):
    c = s["case"]
    B, T, Tk, Hkv, D, G = c["B"], c["T"], c["Tk"], c["Hkv"], c["D"], c["Hq"] // c["Hkv"]
    dt, scale = DTYPES[c["dtype"]], 1.0 / math.sqrt(c["D"])

    def heads(x, L):  # [B, L, Hkv g, D] -> [B, Hkv, g L, D]: a group's rows share one key head's product
        return x.float().view(B, L, Hkv, -1, D).permute(0, 2, 3, 1, 4).reshape(B, Hkv, -1, D)

    def back(x, L):
        return x.view(B, Hkv, -1, L, D).permute(0, 3, 1, 2, 4).reshape(B, L, -1, D).to(dt)

    q, k, v = heads(s["q"], T) * scale, heads(s["k"], Tk), heads(s["v"], Tk)
    p = q @ k.transpose(-1, -2)
    wide = p.view(B, Hkv, G, T, Tk)
    wide.masked_fill_(~_plain_seen(s)[:, None, None], -math.inf)
    m = p.amax(-1, keepdim=True)
    m = torch.where(m == -math.inf, torch.zeros_like(m), m)
    p.sub_(m).exp_()
    total = p.sum(-1, keepdim=True)
    lse = (total.log() + m).view(B, Hkv * G, T).transpose(1, 2).contiguous()
    p.div_(torch.where(total == 0, torch.ones_like(total), total))
    o = p @ v
    out = dict(o=back(o, T), lse=lse)
    if c["step"] == "train":
        dO = heads(s["dO"], T)
        out["dv"] = back(p.transpose(-1, -2) @ dO, Tk)
        dp = dO @ v.transpose(-1, -2)
        dp.sub_((dO * o).sum(-1, keepdim=True))
        p.mul_(dp)
        del dp
        out["dq"] = back((p @ k) * scale, T)
        out["dk"] = back(p.transpose(-1, -2) @ q, Tk)
    return out


def _plain_token(s):
    c = s["case"]
    n, cap, Hkv, D, G = c["n"], c["cap"], c["Hkv"], c["D"], c["Hq"] // c["Hkv"]
    row, at = torch.arange(n, device="cuda"), s["lengths"].long()
    s["k_cache"][row, at] = s["k"]
    s["v_cache"][row, at] = s["v"]
    q = s["q"].float().view(n, Hkv, G, D) * (1.0 / math.sqrt(D))
    k, v = s["k_cache"].float().transpose(1, 2), s["v_cache"].float().transpose(1, 2)
    x = q @ k.transpose(-1, -2)  # [n, Hkv, G, cap]
    x = x.masked_fill(torch.arange(cap, device="cuda")[None, None, None, :] > at[:, None, None, None], -math.inf)
    p = torch.exp(x - x.amax(-1, keepdim=True))
    o = (p @ v) / p.sum(-1, keepdim=True)
    return dict(o=o.reshape(n, Hkv * G, D).to(DTYPES[c["dtype"]]), k_cache=s["k_cache"], v_cache=s["v_cache"])


def _plain_rotary(s):
    c = s["case"]
    rot, dt = c["rot"], DTYPES[c["dtype"]]
    pos = s["pos"]
    if s["cu"] is not None:
        cu = s["cu"].long()
        t = torch.arange(c["N"], device="cuda")
        pos = (t - cu[torch.searchsorted(cu[1:].contiguous(), t, right=True)])[None]
    ang = pos.double()[..., None] * s["inv_freq"].double()  # [1, N, rot / 2]: far positions need 64 bits
    cos, sin = torch.cos(ang).float()[:, :, None], torch.sin(ang).float()[:, :, None]

    def turn(x, sin):
        x = x.float()
        head, rest = x[..., :rot], x[..., rot:]
        if c["interleaved"]:
            a, b = head[..., 0::2], head[..., 1::2]
            y = torch.stack([a * cos - b * sin, b * cos + a * sin], -1).flatten(-2)
        else:
            a, b = head[..., :rot // 2], head[..., rot // 2:]
            y = torch.cat([a * cos - b * sin, b * cos + a * sin], -1)
        return torch.cat([y, rest], -1).to(dt)

    out = dict(q=turn(s["q"], sin), k=turn(s["k"], sin))
    if c["step"] == "train":
        out.update(dq=turn(s["dq"], -sin), dk=turn(s["dk"], -sin))
    return out


def _run_plain(s):
    return {"attention": _plain_attention, "token": _plain_token, "rotary": _plain_rotary}[s["case"]["op"]](s)


# ---------------------------------------------------------------- this package's entry points
def _run_own(s):
    import kimi_delta_attention_bwd_gb300 as kda
    c = s["case"]
    if c["op"] == "rotary":
        at = dict(positions=s["pos"], cu_seqlens=s["cu"], interleaved=c["interleaved"])
        q, k = kda.kda_rotary(s["q"], s["k"], s["inv_freq"], **at)
        if c["step"] == "forward":
            return dict(q=q, k=k)
        dq, dk = kda.kda_rotary_backward(s["dq"], s["dk"], s["inv_freq"], **at)
        return dict(q=q, k=k, dq=dq, dk=dk)
    if c["op"] == "token":
        o = kda.kda_softmax_decode_step(s["q"], s["k"], s["v"], s["k_cache"], s["v_cache"], s["lengths"])
        return dict(o=o, k_cache=s["k_cache"], v_cache=s["v_cache"])
    train = c["step"] == "train"
    o, lse, ctx = kda.kda_softmax_forward(s["q"], s["k"], s["v"], causal=c["causal"], cu_seqlens=s["cu"],
                                          cu_seqlens_k=s["cu_k"], save_for_backward=train)
    if not train:
        return dict(o=o, lse=lse)
    g = kda.kda_softmax_backward(ctx, s["dO"])
    return dict(o=o, lse=lse, dq=g["dq"], dk=g["dk"], dv=g["dv"])


def run(s):
    return _run_own(s) if own else _run_plain(s)


# ---------------------------------------------------------------- what a pass cannot do without
def work(case):
    e = SIZE[case["dtype"]]
    Hq, Hkv, D = case["Hq"], case["Hkv"], case["D"]
    if case["op"] == "rotary":
        n = case["N"] * (Hq + Hkv)
        ways = 2 if case["step"] == "train" else 1
        return dict(bytes=ways * 2 * n * D * e + 4 * case["N"], flops=ways * 3 * n * case["rot"])
    if case["op"] == "token":
        seen = int(_cache_lengths(case).sum()) + case["n"]
        return dict(bytes=2 * seen * Hkv * D * e + case["n"] * (2 * Hq + 2 * Hkv) * D * e, flops=4 * seen * Hq * D)
    pairs = 0
    for a, b in zip(*_lengths(case)):
        if not case["causal"]:
            pairs += a * b
        else:  # query i sees max(0, min(b, i + 1 + b - a)) keys
            rows = min(a, b)
            pairs += rows * b - rows * (rows - 1) // 2
    nq, nk = case["B"] * case["T"] * Hq, case["B"] * case["Tk"] * Hkv
    if case["step"] == "forward":
        return dict(bytes=2 * (nq + nk) * D * e + 4 * nq, flops=4 * pairs * Hq * D)
    return dict(bytes=(4 * nq + 4 * nk) * D * e + 4 * nq, flops=14 * pairs * Hq * D)


# ---------------------------------------------------------------- the definition in 64 bits
def exact(case, seed):
    s = prepare(case, seed)
    return {"attention": _exact_attention, "token": _exact_token, "rotary": _exact_rotary}[case["op"]](s)


def _exact_attention(s, block=2048):
    """Document after document, head after head, in blocks of queries over the keys that the block's last one sees."""
    c = s["case"]
    Hq, D, G = c["Hq"], c["D"], c["Hq"] // c["Hkv"]
    train = c["step"] == "train"
    q, k, v = (s[n].reshape(-1, s[n].shape[2], D).transpose(0, 1) for n in ("q", "k", "v"))  # [H, N, D]
    dev = dict(dtype=torch.float64, device="cuda")
    o, lse = torch.zeros(q.shape, **dev), torch.full(q.shape[:2], -math.inf, **dev)
    if train:
        dO = s["dO"].reshape(-1, Hq, D).transpose(0, 1)
        dq, dk, dv = torch.zeros(q.shape, **dev), torch.zeros(k.shape, **dev), torch.zeros(v.shape, **dev)
    a0 = b0 = 0
    for a, b in zip(*_lengths(c)):
        for h in range(Hq):
            K, V = k[h // G, b0:b0 + b].double(), v[h // G, b0:b0 + b].double()
            for x in range(0, a, block):
                n = min(block, a - x)
                last = min(b, x + n + b - a) if c["causal"] else b
                if last <= 0:
                    continue
                at = slice(a0 + x, a0 + x + n)
                Q = q[h, at].double()
                S = (Q @ K[:last].T) / math.sqrt(D)
                if c["causal"]:
                    i = torch.arange(x, x + n, device="cuda")[:, None] + (b - a)
                    S[torch.arange(last, device="cuda")[None, :] > i] = -math.inf
                L = torch.logsumexp(S, 1)
                P = torch.exp(S - torch.where(L == -math.inf, torch.zeros_like(L), L)[:, None])
                lse[h, at] = L
                o[h, at] = P @ V[:last]
                if train:
                    R = dO[h, at].double()
                    dv[h // G, b0:b0 + last] += P.T @ R
                    M = R @ V[:last].T
                    dS = P * (M - (P * M).sum(1, keepdim=True)) / math.sqrt(D)
                    dq[h, at] = dS @ K[:last]
                    dk[h // G, b0:b0 + last] += dS.T @ Q
        a0, b0 = a0 + a, b0 + b
    out = dict(o=o.transpose(0, 1).reshape(s["q"].shape), lse=lse.T.reshape(s["q"].shape[:3]))
    if train:
        out.update(dq=dq.transpose(0, 1).reshape(s["q"].shape), dk=dk.transpose(0, 1).reshape(s["k"].shape),
                   dv=dv.transpose(0, 1).reshape(s["v"].shape))
    return out


def _exact_token(s):
    """Sequence after sequence, the new token behind its cache."""
    c = s["case"]
    G, D = c["Hq"] // c["Hkv"], c["D"]
    kc, vc = s["k_cache"].clone(), s["v_cache"].clone()
    o = torch.empty(c["n"], c["Hq"], D, dtype=torch.float64, device="cuda")
    for i, n in enumerate(s["lengths"].tolist()):
        kc[i, n], vc[i, n] = s["k"][i], s["v"][i]
        for h in range(c["Hkv"]):
            K, V = kc[i, :n + 1, h].double(), vc[i, :n + 1, h].double()
            w = torch.softmax(s["q"][i, h * G:(h + 1) * G].double() @ K.T / math.sqrt(D), -1)
            o[i, h * G:(h + 1) * G] = w @ V
    return dict(o=o, k_cache=kc.double(), v_cache=vc.double())


def _exact_rotary(s):
    """Each pair as a complex number times exp(i angle); the way back times its conjugate."""
    c = s["case"]
    rot, N = c["rot"], c["N"]
    pos = s["pos"]
    if s["cu"] is not None:
        pos = torch.cat([torch.arange(n, device="cuda") for n in _pieces(N, c["docs"], 3)])[None]
    w = torch.polar(torch.ones(1, N, rot // 2, dtype=torch.float64, device="cuda"),
                    pos.double()[..., None] * s["inv_freq"].double())[:, :, None]

    def turn(x, w):
        x = x.double()
        pairs = x[..., :rot].reshape(*x.shape[:-1], rot // 2, 2) if c["interleaved"] else \
            x[..., :rot].reshape(*x.shape[:-1], 2, rot // 2).transpose(-1, -2)
        y = torch.view_as_real(torch.view_as_complex(pairs.contiguous()) * w)
        y = (y if c["interleaved"] else y.transpose(-1, -2)).reshape(*x.shape[:-1], rot)
        return torch.cat([y, x[..., rot:]], -1)

    out = dict(q=turn(s["q"], w), k=turn(s["k"], w))
    if c["step"] == "train":
        out.update(dq=turn(s["dq"], w.conj()), dk=turn(s["dk"], w.conj()))
    return out
