"""Cases, plain forms and calls of the linear-attention operators.

Three operators of one layer, as a serving program runs them:

* ``norm_rope``: per-head RMSNorm of q and k and the rotation by position, in one pass
  (one or three position axes, q and k as slices of a packed projection or on their own);
* ``chunk``: the prompt pass of linear attention with a decay for each head,
  ``S_t = e^{g_t} S_{t-1} + k_t v_t^T``, ``o_t = scale S_t^T q_t``, packed sequences;
* ``step``: one or a few new tokens for every sequence, the state updated in place.

``run`` computes the plain form (elementary fp32 torch operations) while ``own`` is false
and calls the package where it is true.  ``exact`` evaluates the definitions in fp64.
"""

import math

import torch

own = False

D = 128  # channels of a head
DEV = "cuda"
CHUNK = 128  # tokens of a chunk of the plain prompt form


# ------------------------------------------------------------------------- the cases
def listed():
    return [
        # one new token of one conversation: nothing but latency
        dict(name="norm_rope 1 token", op="norm_rope", tokens=1, hq=16, hk=16, freqs=64, axes=1,
             interleaved=False, packed=True, norm=True, dtype="bf16", start=40000),
        # one layer's prompt at this repository's prefill size
        dict(name="norm_rope prompt", op="norm_rope", tokens=8192, hq=96, hk=96, freqs=64, axes=1,
             interleaved=False, packed=False, norm=True, dtype="bf16", start=0),
        # image and video tokens (time, height, width), shared key heads, half of each head rotated
        dict(name="norm_rope video", op="norm_rope", tokens=10007, hq=32, hk=8, freqs=32, axes=3,
             interleaved=True, packed=True, norm=True, dtype="bf16", start=1 << 20),
        # the smallest prompt of the workloads, in fp32
        dict(name="chunk tiny fp32", op="chunk", lens="256", h=2, hk=2, decay="token", h0=False,
             dtype="fp32"),
        # an fp32 layer over a ragged batch
        dict(name="chunk ragged fp32", op="chunk", lens="700,1,0,1337,64", h=16, hk=8,
             decay="head", h0=True, dtype="fp32"),
        # one layer's prompt at this repository's prefill size, per-token decays
        dict(name="chunk prompt", op="chunk", lens="8192", h=96, hk=96, decay="token", h0=True,
             dtype="bf16"),
        # a packed batch of prompts of very different lengths
        dict(name="chunk ragged", op="chunk",
             lens="4096,17,2500,129,1,3001,700,64,1999,333,2048,1500,90,1111", h=48, hk=48,
             decay="token", h0=True, dtype="bf16"),
        # a long document with few heads, constant decays
        dict(name="chunk long", op="chunk", lens="131072", h=16, hk=16, decay="head", h0=False,
             dtype="bf16"),
        # key heads shared by groups of value heads, several prompts of one odd length
        dict(name="chunk shared keys", op="chunk", lens="1501,1501,1501,1501", h=32, hk=16,
             decay="token", h0=False, dtype="bf16"),
        # one token of one conversation
        dict(name="step 1 sequence", op="step", n=1, t=1, h=16, hk=16, decay="token",
             dtype="bf16"),
        # this repository's decode size
        dict(name="step 512 sequences", op="step", n=512, t=1, h=96, hk=96, decay="token",
             dtype="bf16"),
        # a verify pass over drafted tokens, part of them accepted
        dict(name="step 5 drafted tokens", op="step", n=96, t=5, h=48, hk=48, decay="head",
             dtype="bf16"),
    ]


def _log_int(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 1)))))))


def draw(rng):
    op = rng.choice(["norm_rope", "chunk", "chunk", "step"])
    dtype = rng.choice(["bf16", "bf16", "fp32"])
    h = rng.choice([1, 2, 4, 6, 8, 12, 16, 32, 48, 64, 96])
    hk = rng.choice([x for x in range(1, h + 1) if h % x == 0 and h // x <= 8])
    if op == "norm_rope":
        most = (8192 * 192 // (2 if dtype == "fp32" else 1)) // (h + hk)
        axes = rng.choice([1, 1, 3])
        return dict(op=op, tokens=_log_int(rng, 1, min(65536, most)), hq=h, hk=hk,
                    freqs=rng.choice([8, 16, 24, 32, 48, 64, 64]), axes=axes,
                    interleaved=rng.random() < 0.4, packed=rng.random() < 0.5,
                    norm=rng.random() < 0.85, dtype=dtype, start=_log_int(rng, 1, 1 << 20))
    if op == "step":
        t = rng.choice([1, 1, 1, 2, 3, 5, 8, 16])
        return dict(op=op, n=_log_int(rng, 1, max(1, min(512, 512 * 96 // (h * t)))), t=t, h=h,
                    hk=hk, decay=rng.choice(["token", "head"]), dtype=dtype)
    # tokens x heads of the padded batch stay below the largest listed prompt's
    most = (1 << 21 if dtype == "bf16" else 1 << 16) // h
    n = _log_int(rng, 1, 24)
    longest = _log_int(rng, 1, max(1, min(65536, most // n)))
    lens = [longest] + [rng.randint(0, longest) for _ in range(n - 1)]
    rng.shuffle(lens)
    return dict(op=op, lens=",".join(map(str, lens)), h=h, hk=hk,
                decay=rng.choice(["token", "token", "head"]), h0=rng.random() < 0.5, dtype=dtype)


def _dtype(case):
    return torch.bfloat16 if case["dtype"] == "bf16" else torch.float32


def _lens(case):
    return [int(x) for x in case["lens"].split(",")]


# ------------------------------------------------------------------------- the inputs
def _decays(case, shape, gen):
    """Log-decays: per token -e^A Softplus(z), A one log-scale a head (a trained gate's
    spread: half-lives from about one token to hundreds); per head the geometric ladder
    -2^(-8 (h + 1) / H)."""
    h = case["h"]
    if case["decay"] == "head":
        i = torch.arange(1, h + 1, device=DEV, dtype=torch.float32)
        jitter = 1 + 0.1 * torch.rand(h, generator=gen, device=DEV)
        return -torch.exp2(-8 * i / h) * jitter
    a = torch.rand(h, generator=gen, device=DEV) * 6 - 5
    z = torch.randn(*shape, h, generator=gen, device=DEV)
    return -torch.exp(a) * torch.nn.functional.softplus(z)


def prepare(case, seed):
    gen = torch.Generator(device=DEV)
    gen.manual_seed(seed)
    dt = _dtype(case)

    def normal(*shape):
        return torch.randn(*shape, generator=gen, device=DEV)

    if case["op"] == "norm_rope":
        nt, hq, hk, f = case["tokens"], case["hq"], case["hk"], case["freqs"]
        if case["packed"]:  # q, k and v as one projection's rows
            qkv = (normal(nt, hq + 2 * hk, D) * 2).to(dt)
            q, k = qkv[:, :hq], qkv[:, hq:hq + hk]
        else:
            q, k = (normal(nt, hq, D) * 2).to(dt), (normal(nt, hk, D) * 2).to(dt)
        inv = (10000.0 ** (-torch.arange(f, dtype=torch.float64) / f)).to(torch.float32).to(DEV)
        s = dict(case=case, q=q, k=k, inv_freq=inv, axis=None)
        t = torch.arange(nt, device=DEV, dtype=torch.int32)
        shift = int(torch.randint(0, 1000, (1,), generator=gen, device=DEV))
        if case["axes"] == 1:
            s["pos"] = t + case["start"] + shift
        else:  # frames of 24 x 40 patches
            s["pos"] = torch.stack([t // 960 + case["start"] + shift, (t // 40) % 24, t % 40])
            s["axis"] = (torch.arange(f, device=DEV) % 3).to(torch.int32)
        s["wq"] = s["wk"] = s["eps"] = None
        if case["norm"]:
            s["wq"], s["wk"], s["eps"] = 1 + 0.2 * normal(D), 1 + 0.2 * normal(D), 1e-6
        return s
    if case["op"] == "chunk":
        lens = _lens(case)
        nt, n = sum(lens), len(lens)
        unit = lambda x: x / x.norm(dim=-1, keepdim=True)  # noqa: E731
        s = dict(case=case, lens=lens, scale=1.0,
                 q=unit(normal(nt, case["hk"], D)).to(dt), k=unit(normal(nt, case["hk"], D)).to(dt),
                 v=normal(nt, case["h"], D).to(dt), g=_decays(case, (nt,), gen), h0=None)
        if case["h0"]:
            s["h0"] = normal(n, case["h"], D, D) * 0.1
        cu = torch.zeros(n + 1, dtype=torch.int64)
        cu[1:] = torch.cumsum(torch.tensor(lens), 0)
        s["cu"] = cu.to(torch.int32).to(DEV)
        return s
    n, t, h, hk = case["n"], case["t"], case["h"], case["hk"]
    tok = (n,) if t == 1 else (n, t)
    s = dict(case=case, scale=D ** -0.5, q=normal(*tok, hk, D).to(dt), k=normal(*tok, hk, D).to(dt),
             v=normal(*tok, h, D).to(dt), g=_decays(case, tok, gen), advance=None)
    s["S"] = normal(n, h, D, D) * 0.1
    if t > 1:
        s["advance"] = torch.randint(0, t + 1, (n,), generator=gen, device=DEV).to(torch.int32)
    return s


# ------------------------------------------------------------------------- plain forms
def _plain_norm_rope(s):
    case = s["case"]
    f, nt = case["freqs"], case["tokens"]
    pos = s["pos"].double()
    pos = pos.unsqueeze(1) if s["axis"] is None else pos[s["axis"].long()].transpose(0, 1)
    ang = pos * s["inv_freq"].double()  # [tokens, freqs]: far positions need 64 bits
    cos, sin = torch.cos(ang).float().view(nt, 1, f), torch.sin(ang).float().view(nt, 1, f)

    def one(x, w):
        y = x.float()
        if s["eps"] is not None:
            y = y * torch.rsqrt((y * y).mean(-1, keepdim=True) + s["eps"]) * w
        out = y.clone()
        if case["interleaved"]:
            a, b = y[..., 0:2 * f:2], y[..., 1:2 * f:2]
            out[..., 0:2 * f:2], out[..., 1:2 * f:2] = a * cos - b * sin, a * sin + b * cos
        else:
            a, b = y[..., :f], y[..., f:2 * f]
            out[..., :f], out[..., f:2 * f] = a * cos - b * sin, a * sin + b * cos
        return out.to(x.dtype)

    return one(s["q"], s["wq"]), one(s["k"], s["wk"])


def _plain_chunk(s):
    case, lens, c = s["case"], s["lens"], CHUNK
    h, hk, n = case["h"], case["hk"], len(s["lens"])
    nc = max(1, -(-max(lens) // c))
    start = s["cu"][:-1].long().unsqueeze(1)
    size = s["cu"][1:].long().unsqueeze(1) - start
    at = torch.arange(nc * c, device=DEV).unsqueeze(0)
    real = at < size  # [n, nc c]: the sequences padded to one length
    idx = torch.where(real, start + at, 0)

    def lay(x, heads):  # [tokens, heads, ...] -> [n, h, nc, c, ...]
        y = x[idx.view(-1)].view(n, nc, c, *x.shape[1:])
        y = y.repeat_interleave(h // heads, dim=3)
        return y.permute(0, 3, 1, 2, *range(4, y.dim()))

    mask = real.view(n, 1, nc, c)
    q, k, v = lay(s["q"], hk).float(), lay(s["k"], hk).float(), lay(s["v"], h).float()
    k = torch.where(mask.unsqueeze(-1), k, 0.0)
    g = s["g"].double()
    g = lay(g, h) if g.dim() == 2 else g.view(1, h, 1, 1).expand(n, h, nc, c)
    G = torch.cumsum(torch.where(mask, g, 0.0), dim=3)
    total = G[..., -1]
    lower = torch.ones(c, c, device=DEV, dtype=torch.bool).tril()
    decay = torch.exp(torch.where(lower, G.unsqueeze(4) - G.unsqueeze(3), -math.inf)).float()
    o = ((q @ k.transpose(3, 4)) * decay) @ v
    local = (k * torch.exp(total.unsqueeze(3) - G).float().unsqueeze(4)).transpose(3, 4) @ v
    # states entering chunk 0 .. nc (the last is the final state)
    E = torch.cumsum(total, dim=2)
    into = torch.cat([torch.zeros_like(E[..., :1]), E], dim=2)
    before = torch.ones(nc + 1, nc, device=DEV, dtype=torch.bool).tril(-1)
    carry = torch.exp(torch.where(before, into.unsqueeze(3) - E.unsqueeze(2), -math.inf)).float()
    S = (carry @ local.reshape(n, h, nc, D * D)).view(n, h, nc + 1, D, D)
    if s["h0"] is not None:
        S = S + torch.exp(into).float().view(n, h, nc + 1, 1, 1) * s["h0"].transpose(2, 3).unsqueeze(2)
    o = o + torch.exp(G).float().unsqueeze(4) * (q @ S[:, :, :nc])
    o = (s["scale"] * o).permute(0, 2, 3, 1, 4).reshape(n * nc * c, h, D)
    return o[real.view(-1)].to(s["v"].dtype), S[:, :, nc].transpose(2, 3).contiguous()


def _plain_step(s):
    case = s["case"]
    n, t, h, rep = case["n"], case["t"], case["h"], case["h"] // case["hk"]

    def lay(x, r):  # [n(, t), heads, ...] -> [n, h, t, ...]
        return x.view(n, t, *x.shape[-2:]).repeat_interleave(r, dim=2).float().transpose(1, 2)

    q, k, v = lay(s["q"], rep), lay(s["k"], rep), lay(s["v"], 1)
    g = s["g"].double()
    g = g.view(1, h, 1).expand(n, h, t) if case["decay"] == "head" else g.view(n, t, h).transpose(1, 2)
    G = torch.cumsum(g, dim=2)
    lower = torch.ones(t, t, device=DEV, dtype=torch.bool).tril()
    decay = torch.exp(torch.where(lower, G.unsqueeze(3) - G.unsqueeze(2), -math.inf)).float()
    St = s["S"].transpose(2, 3)
    o = ((q @ k.transpose(2, 3)) * decay) @ v + torch.exp(G).float().unsqueeze(3) * (q @ St)
    o = (s["scale"] * o).transpose(1, 2).to(s["v"].dtype).reshape(s["v"].shape)
    if s["advance"] is None:
        end, kept = G[..., -1], torch.ones(n, 1, t, device=DEV, dtype=torch.bool)
    else:
        adv = s["advance"].long().view(n, 1, 1)
        end = torch.where(adv > 0, G, 0.0).gather(2, (adv - 1).clamp(min=0).expand(n, h, 1)).squeeze(2)
        kept = torch.arange(t, device=DEV).view(1, 1, t) < adv
    w = torch.exp(torch.where(kept, end.unsqueeze(2) - G, -math.inf)).float()
    s["S"].mul_(torch.exp(end).float().view(n, h, 1, 1)).add_(v.transpose(2, 3) @ (k * w.unsqueeze(3)))
    return o, s["S"]


# ------------------------------------------------------------------------- one pass
def run(s):
    case = s["case"]
    if not own:
        return {"norm_rope": _plain_norm_rope, "chunk": _plain_chunk, "step": _plain_step}[case["op"]](s)
    import chunked_gated_delta_fwd_gb300 as kda

    if case["op"] == "norm_rope":
        return kda.qk_norm_rope(s["q"], s["k"], s["pos"], s["inv_freq"], q_weight=s["wq"],
                                k_weight=s["wk"], eps=s["eps"], freq_axis=s["axis"],
                                interleaved=case["interleaved"])
    if case["op"] == "chunk":
        return kda.linear_chunk_fwd(s["q"], s["k"], s["v"], s["g"], s["h0"], s["cu"],
                                    scale=s["scale"])
    if case["t"] == 1:
        o = kda.linear_recurrent_step(s["q"], s["k"], s["v"], s["g"], s["S"], scale=s["scale"])
    else:
        o = kda.linear_recurrent_multi_step(s["q"], s["k"], s["v"], s["g"], s["S"], s["advance"],
                                            scale=s["scale"])
    return o, s["S"]


# ------------------------------------------------------------------------- the work
def work(case):
    e = 2 if case["dtype"] == "bf16" else 4
    if case["op"] == "norm_rope":
        rows = case["tokens"] * (case["hq"] + case["hk"])
        return {"bytes": 2 * rows * D * e + 4 * case["axes"] * case["tokens"] + 4 * case["freqs"] +
                (8 * D if case["norm"] else 0), "flops": 10 * rows * D}
    h, hk = case["h"], case["hk"]
    if case["op"] == "chunk":
        lens = _lens(case)
        nt, n = sum(lens), len(lens)
        g = 4 * nt * h if case["decay"] == "token" else 4 * h
        states = n * h * D * D * 4 * (2 if case["h0"] else 1)
        # q.k and p.v over the causal half of a 128-token chunk, q S and k^T v whole
        return {"bytes": nt * D * e * 2 * (h + hk) + g + states + 4 * (n + 1),
                "flops": nt * h * (2 * D * CHUNK + 4 * D * D)}
    n, t = case["n"], case["t"]
    g = 4 * n * t * h if case["decay"] == "token" else 4 * h
    return {"bytes": 2 * n * h * D * D * 4 + n * t * D * e * 2 * (h + hk) + g,
            "flops": n * t * h * 4 * D * D}


# ------------------------------------------------------------------------- in 64 bits
def _exact_norm_rope(s):
    """The rotation as a product of complex numbers."""
    case = s["case"]
    f, nt = case["freqs"], case["tokens"]
    pos = s["pos"].double().reshape(case["axes"], nt)
    of = torch.zeros(f, dtype=torch.long, device=DEV) if s["axis"] is None else s["axis"].long()
    turn = torch.polar(torch.ones(f, nt, dtype=torch.float64, device=DEV),
                       pos.index_select(0, of) * s["inv_freq"].double().view(f, 1))
    turn = turn.t().view(nt, 1, f)
    got = []
    for x, w in ((s["q"], s["wq"]), (s["k"], s["wk"])):
        y = x.double()
        if s["eps"] is not None:
            y = y / (y.square().sum(-1, keepdim=True) / D + s["eps"]).sqrt() * w.double()
        y = y.contiguous()
        part = y[..., :2 * f]
        if case["interleaved"]:
            pairs = part.reshape(nt, -1, f, 2)
        else:
            pairs = part.reshape(nt, -1, 2, f).transpose(2, 3)
        z = torch.view_as_real(torch.view_as_complex(pairs.contiguous()) * turn)
        z = z if case["interleaved"] else z.transpose(2, 3)
        got.append(torch.cat([z.reshape(nt, -1, 2 * f), y[..., 2 * f:]], dim=-1))
    return got


def _recurrence(q, k, v, a, S, scale):
    """Token by token: q, k, v [units, t, D], a [units, t], S [units, D(k), D(v)]."""
    o = torch.empty_like(v)
    for i in range(v.shape[1]):
        S.mul_(a[:, i].view(-1, 1, 1)).baddbmm_(k[:, i].unsqueeze(2), v[:, i].unsqueeze(1))
        o[:, i] = torch.bmm(q[:, i].unsqueeze(1), S).squeeze(1)
    return scale * o, S


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "norm_rope":
        return _exact_norm_rope(s)
    h, rep = case["h"], case["h"] // case["hk"]
    q = s["q"].double().repeat_interleave(rep, dim=-2)
    k = s["k"].double().repeat_interleave(rep, dim=-2)
    v, g = s["v"].double(), s["g"].double()
    if g.dim() == 1:
        g = g.expand(v.shape[:-1])
    if case["op"] == "chunk":
        o = torch.empty_like(v)
        n, longest = len(s["lens"]), max(s["lens"])
        pad = [torch.zeros(n, longest, h, D, dtype=torch.float64, device=DEV) for _ in range(3)]
        a = torch.ones(n, longest, h, dtype=torch.float64, device=DEV)  # past the end: nothing changes
        cu = s["cu"].tolist()
        for i in range(n):
            for x, y in zip(pad, (q, k, v)):
                x[i, :s["lens"][i]] = y[cu[i]:cu[i + 1]]
            a[i, :s["lens"][i]] = torch.exp(g[cu[i]:cu[i + 1]])
        units = lambda x: x.transpose(1, 2).reshape(n * h, longest, *x.shape[3:])  # noqa: E731
        S = torch.zeros(n, h, D, D, dtype=torch.float64, device=DEV)
        if s["h0"] is not None:
            S = S + s["h0"].double().transpose(2, 3)
        po, S = _recurrence(*(units(x) for x in pad), units(a), S.reshape(n * h, D, D), s["scale"])
        po = po.view(n, h, longest, D).transpose(1, 2)
        for i in range(n):
            o[cu[i]:cu[i + 1]] = po[i, :s["lens"][i]]
        return o, S.view(n, h, D, D).transpose(2, 3).contiguous()
    n, t = case["n"], case["t"]
    lay = lambda x: x.reshape(n, t, h, -1).transpose(1, 2).reshape(n * h, t, -1)  # noqa: E731
    a = torch.exp(lay(g)).squeeze(2)
    S0 = s["S"].double().transpose(2, 3).reshape(n * h, D, D).contiguous()
    o, S = _recurrence(lay(q), lay(k), lay(v), a, S0.clone(), s["scale"])
    if s["advance"] is not None:  # the state again, over the accepted tokens alone
        on = (torch.arange(t, device=DEV) < s["advance"].long().view(n, 1, 1)).expand(n, h, t)
        on = on.reshape(n * h, t)
        _, S = _recurrence(lay(q), torch.where(on.unsqueeze(2), lay(k), 0.0), lay(v),
                           torch.where(on, a, 1.0), S0, s["scale"])
    return (o.view(n, h, t, D).transpose(1, 2).reshape(s["v"].shape),
            S.view(n, h, D, D).transpose(2, 3).contiguous())
