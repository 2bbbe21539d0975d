"""Cases, plain forms and calls of the operators around a recurrent-state layer.

Three operators of one serving step, as a hybrid model's program runs them:

* ``conv``: the short causal depthwise convolution in front of a recurrent layer, over packed
  prompts (``conv``) or one or a few new tokens with the last inputs kept (``conv_step``);
* ``scan``: the selective state space scan,
  ``h_t = exp(delta_t A) h_{t-1} + delta_t x_t B_t``, ``y_t = (C_t . h_t + D x_t) SiLU(z_t)``,
  over packed prompts (``scan``) or new tokens with the state in place (``scan_step``);
* ``verify``: drafted tokens against the target's probabilities from given random numbers; its
  counts are what the two states are advanced by.

``run`` computes the plain form (elementary torch operations) while ``own`` is false and calls
the package where it is true.  ``exact`` evaluates the definitions in fp64.
"""

import math

import torch

own = False

DEV = "cuda"


# ------------------------------------------------------------------------- the cases
def listed():
    return [
        # q (or k, or v) of one layer's prompt at this repository's prefill size, 96 heads of 128
        dict(name="conv prompt", op="conv", lens="8192", c=12288, w=4, bias=False, silu=True,
             state=False, packed=False, dtype="bf16"),
        # a ragged batch that goes on from kept inputs, a slice of a packed projection
        dict(name="conv ragged fp32", op="conv", lens="700,1,0,1337,64,2,3001", c=2056, w=3,
             bias=True, silu=False, state=True, packed=True, dtype="fp32"),
        # one new token of one conversation: nothing but latency
        dict(name="conv 1 token", op="conv_step", n=1, t=1, c=12288, w=4, bias=False, silu=True,
             packed=False, dtype="bf16"),
        # drafted tokens of a batch, part of them kept
        dict(name="conv 5 drafted tokens", op="conv_step", n=96, t=5, c=6144, w=4, bias=True,
             silu=True, packed=True, dtype="bf16"),
        # a small layer in fp32 over a short prompt
        dict(name="scan tiny fp32", op="scan", lens="256", c=512, s=16, groups=1, gate=False,
             h0=False, dtype="fp32"),
        # one prompt at this repository's prefill length
        dict(name="scan prompt", op="scan", lens="8192", c=8192, s=16, groups=1, gate=True,
             h0=False, dtype="bf16"),
        # a packed batch of prompts of very different lengths that go on from kept states
        dict(name="scan ragged", op="scan",
             lens="4096,17,2500,129,1,3001,700,64,1999,333,2048,0,1500,90,1111", c=4096, s=16,
             groups=2, gate=True, h0=True, dtype="bf16"),
        # a long document in a layer with few channels
        dict(name="scan long", op="scan", lens="65536", c=2048, s=16, groups=1, gate=True, h0=False,
             dtype="bf16"),
        # one new token of many conversations: the states' traffic
        dict(name="scan step 512 sequences", op="scan_step", n=512, t=1, c=8192, s=16, groups=1,
             gate=True, dtype="bf16"),
        # drafted tokens of a batch, part of them kept
        dict(name="scan step 5 drafted tokens", op="scan_step", n=96, t=5, c=4096, s=16, groups=1,
             gate=True, dtype="bf16"),
        # one conversation, a small vocabulary
        dict(name="verify 1 sequence", op="verify", n=1, t=4, vocab=32000, keep=0.7, dtype="fp32"),
        # a batch with long drafts and a large vocabulary
        dict(name="verify 128 sequences", op="verify", n=128, t=7, vocab=163840, keep=0.8,
             dtype="fp32"),
    ]


def _log_int(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 1)))))))


def _lens_of(rng, most):
    """Lengths of a packed batch whose padded token count stays within ``most``."""
    n = _log_int(rng, 1, 24)
    longest = _log_int(rng, 1, max(1, min(65536, most // n)))
    lens = [longest] + [rng.randint(0, longest) for _ in range(n - 1)]
    rng.shuffle(lens)
    return ",".join(map(str, lens))


def draw(rng):
    op = rng.choice(["conv", "conv_step", "scan", "scan", "scan_step", "verify"])
    dtype = rng.choice(["bf16", "bf16", "fp32"])
    if op == "verify":
        vocab, t = _log_int(rng, 1000, 200000), rng.choice([0, 1, 2, 3, 4, 5, 7, 8, 11, 15])
        most = 128 * 8 * 163840 // ((t + 1) * vocab)
        return dict(op=op, n=_log_int(rng, 1, max(1, min(256, most))), t=t, vocab=vocab,
                    keep=rng.choice([0.2, 0.5, 0.7, 0.9]), dtype=dtype)
    tok = rng.choice([1, 1, 1, 2, 3, 5, 8, 16])
    if op in ("conv", "conv_step"):
        c = 8 * _log_int(rng, 1, 1536)
        case = dict(op=op, c=c, w=rng.choice([2, 3, 4, 4]), bias=rng.random() < 0.5,
                    silu=rng.random() < 0.7, packed=rng.random() < 0.5, dtype=dtype)
        if op == "conv":
            most = (1 << 26) // c // (2 if dtype == "fp32" else 1)
            return dict(case, lens=_lens_of(rng, most), state=rng.random() < 0.5)
        return dict(case, n=_log_int(rng, 1, max(1, min(512, (1 << 22) // (c * tok)))), t=tok)
    s, groups = rng.choice([8, 16, 16, 16, 32]), rng.choice([1, 1, 2, 4])
    c = 8 * groups * _log_int(rng, 1, 1024 // groups)
    case = dict(op=op, c=c, s=s, groups=groups, gate=rng.random() < 0.6, dtype=dtype)
    if op == "scan":
        most = (1 << 30) // (c * s) // (2 if dtype == "fp32" else 1)
        return dict(case, lens=_lens_of(rng, most), h0=rng.random() < 0.5)
    return dict(case, n=_log_int(rng, 1, max(1, min(512, (1 << 26) // (c * s * tok)))), t=tok)


def _dtype(case):
    return torch.bfloat16 if case["dtype"] == "bf16" else torch.float32


def _lens(case):
    return [int(x) for x in case["lens"].split(",")]


# ------------------------------------------------------------------------- the inputs
def prepare(case, seed):
    gen = torch.Generator(device=DEV)
    gen.manual_seed(seed)
    dt, op = _dtype(case), case["op"]

    def normal(*shape):
        return torch.randn(*shape, generator=gen, device=DEV)

    def uniform(*shape):
        return torch.rand(*shape, generator=gen, device=DEV)

    s = dict(case=case)
    if op == "verify":
        n, t, v = case["n"], case["t"], case["vocab"]
        p = torch.softmax(3.0 * normal(n, t + 1, v), dim=-1)
        # a draft that is the target's own distribution a share `keep` of the time
        q = torch.softmax(3.0 * normal(n, t, v), dim=-1)
        q.mul_(1 - case["keep"]).add_(p[:, :t], alpha=case["keep"])
        race = torch.empty_like(q).exponential_(generator=gen)
        s["tokens"] = (q / race).argmax(dim=-1).to(torch.int32)  # drawn from q
        s["p"], s["q"] = p.to(dt), q.to(dt)
        s["u_accept"], s["u_sample"] = uniform(n, t), uniform(n)
        return s
    c = case["c"]
    if op in ("conv", "scan"):
        lens = s["lens"] = _lens(case)
        n, lead = len(lens), (sum(lens),)
        cu = torch.zeros(n + 1, dtype=torch.int64)
        cu[1:] = torch.cumsum(torch.tensor(lens), 0)
        s["cu"] = cu.to(torch.int32).to(DEV)
    else:
        n = case["n"]
        lead = (n,) if case["t"] == 1 else (n, case["t"])
        s["advance"] = None
        if case["t"] > 1:
            s["advance"] = torch.randint(0, case["t"] + 1, (n,), generator=gen,
                                         device=DEV).to(torch.int32)
    if op in ("conv", "conv_step"):
        w = case["w"]
        s["x"] = normal(*lead, c + 512).to(dt)[..., 256:256 + c] if case["packed"] else \
            normal(*lead, c).to(dt)
        s["w"] = normal(c, w) / math.sqrt(w)
        s["bias"] = 0.1 * normal(c) if case["bias"] else None
        s["state"] = normal(n, w - 1, c).to(dt) if op == "conv_step" or case["state"] else None
        return s
    ns, g = case["s"], case["groups"]
    # x and the gate as one projection's rows, B and C as another's next to delta's low-rank part
    s["x"], s["z"] = normal(*lead, c).to(dt), None
    if case["gate"]:
        xz = normal(*lead, 2 * c).to(dt)
        s["x"], s["z"] = xz[..., :c], xz[..., c:]
    low = normal(*lead, 64 + 2 * g * ns).to(dt)
    s["B"] = low[..., 64:64 + g * ns].unflatten(-1, (g, ns))
    s["C"] = low[..., 64 + g * ns:].unflatten(-1, (g, ns))
    s["dt"] = (0.5 * normal(*lead, c)).to(dt)
    # steps of 1e-3 to 1e-1 before training, a ladder of decays 1 .. S a channel
    step = torch.exp(uniform(c) * math.log(100.0) + math.log(1e-3))
    s["dt_bias"] = step + torch.log(-torch.expm1(-step))
    s["A"] = -torch.arange(1, ns + 1, device=DEV) * torch.exp(0.1 * normal(c, ns))
    s["D"] = 1 + 0.1 * normal(c)
    s["h"] = 0.3 * normal(n, c, ns) if op == "scan_step" or case["h0"] else None
    return s


# ------------------------------------------------------------------------- plain forms
def _silu(y):
    return y / (1 + torch.exp(-y))


def _plain_conv(s):
    case, x, st, cu = s["case"], s["x"], s["state"], s["cu"].long()
    w, k, nt, n = case["w"], case["w"] - 1, s["x"].shape[0], len(s["lens"])
    at = torch.arange(nt, device=DEV)
    seq = torch.searchsorted(cu[1:], at, right=True)
    first = cu[seq]
    y = torch.zeros(nt, case["c"], device=DEV) if s["bias"] is None else \
        s["bias"].expand(nt, case["c"]).clone()
    for j in range(w):
        src = at - (k - j)
        inside = (src >= first).unsqueeze(1)
        tap = torch.where(inside, x[src.clamp(min=0)].float(), 0.0)
        if st is not None:
            row = (src - first + k).clamp(0, k - 1)
            tap = torch.where(inside, tap, st[seq, row].float())
        y += s["w"][:, j] * tap
    if case["silu"]:
        y = _silu(y)
    end = cu[1:].unsqueeze(1) - k + torch.arange(k, device=DEV)  # [n, k]: rows of the last inputs
    inside = (end >= cu[:-1].unsqueeze(1)).unsqueeze(2)
    kept = torch.zeros(n, k, case["c"], dtype=x.dtype, device=DEV)
    if st is not None:
        row = (end - cu[:-1].unsqueeze(1) + k).clamp(0, k - 1)
        kept = st[torch.arange(n, device=DEV).unsqueeze(1), row]
    if nt > 0:
        kept = torch.where(inside, x[end.clamp(min=0)], kept)
    return y.to(x.dtype), kept


def _plain_conv_step(s):
    case, x, st = s["case"], s["x"], s["state"]
    n, t, w, c = case["n"], case["t"], case["w"], case["c"]
    rows = torch.cat([st, x.reshape(n, t, c)], dim=1)
    y = 0.0 if s["bias"] is None else s["bias"]
    for j in range(w):
        y = y + s["w"][:, j] * rows[:, j:j + t].float()
    if case["silu"]:
        y = _silu(y)
    adv = torch.full((n,), t, device=DEV) if s["advance"] is None else s["advance"].long()
    keep = adv.unsqueeze(1) + torch.arange(w - 1, device=DEV)
    st.copy_(rows[torch.arange(n, device=DEV).unsqueeze(1), keep])
    return y.to(x.dtype).view(x.shape), st


def _delta(s):
    """The step of every token and channel in fp32, log(1 + e^v) without loss at either end."""
    v = s["dt"].float() + s["dt_bias"]
    return torch.clamp(v, min=0) + torch.log1p(torch.exp(-v.abs()))


def _finish(s, y, x):
    y = y + s["D"] * x.float()
    if s["z"] is not None:
        y = y * _silu(s["z"].float())
    return y.to(x.dtype)


def _plain_scan(s):
    """Every sequence cut into segments that are walked side by side, twice: from a zero state
    for what a segment adds, then from the state it enters with."""
    case, lens = s["case"], s["lens"]
    n, c, ns, g = len(lens), case["c"], case["s"], case["groups"]
    longest = max(1, max(lens))
    seg = 1 << max(4, (longest.bit_length() + 1) // 2)
    m = -(-longest // seg)
    start = s["cu"][:-1].long().unsqueeze(1)
    size = s["cu"][1:].long().unsqueeze(1) - start
    at = torch.arange(m * seg, device=DEV).unsqueeze(0)
    real = at < size
    idx = torch.where(real, start + at, 0).view(-1)
    mask = real.view(n, m, seg, 1)
    if sum(lens) == 0:
        h = torch.zeros(n, c, ns, device=DEV) if s["h"] is None else s["h"]
        return s["x"].clone(), h

    def lay(t, *tail):
        return t[idx].view(n, m, seg, *tail)

    delta = torch.where(mask, lay(_delta(s), c), 0.0)
    dx = torch.where(mask, delta * lay(s["x"].float(), c), 0.0)
    B, C = lay(s["B"].float(), g, ns), lay(s["C"].float(), g, ns)
    A = s["A"].view(g, c // g, ns)

    def walk(h, y):
        for j in range(seg):
            a = torch.exp(delta[:, :, j].view(n, m, g, c // g, 1) * A)
            h = a * h + dx[:, :, j].view(n, m, g, c // g, 1) * B[:, :, j].unsqueeze(3)
            if y is not None:
                y[:, :, j] = (h * C[:, :, j].unsqueeze(3)).sum(-1).view(n, m, c)
        return h

    zero = torch.zeros(n, m, g, c // g, ns, device=DEV)
    local = walk(zero, None)
    total = torch.exp(delta.double().sum(2).view(n, m, g, c // g, 1) * A.double()).float()
    into = [torch.zeros_like(zero[:, 0]) if s["h"] is None else s["h"].view(n, g, c // g, ns)]
    for i in range(m):
        into.append(total[:, i] * into[i] + local[:, i])
    y = torch.empty(n, m, seg, c, device=DEV)
    walk(torch.stack(into[:-1], dim=1), y)
    y = y.view(n * m * seg, c)[real.view(-1)]
    return _finish(s, y, s["x"]), into[-1].reshape(n, c, ns)


def _plain_scan_step(s):
    case = s["case"]
    n, t, c, ns, g = case["n"], case["t"], case["c"], case["s"], case["groups"]
    delta = _delta(s).view(n, t, g, c // g, 1)
    dx = delta * s["x"].float().reshape(n, t, g, c // g, 1)
    B, C = (s[i].float().reshape(n, t, g, 1, ns) for i in "BC")
    A, h = s["A"].view(g, c // g, ns), s["h"].view(n, g, c // g, ns)
    kept, y = h, torch.empty(n, t, c, device=DEV)
    for j in range(t):
        h = torch.exp(delta[:, j] * A) * h + dx[:, j] * B[:, j]
        y[:, j] = (h * C[:, j]).sum(-1).view(n, c)
        if s["advance"] is not None:
            kept = torch.where((s["advance"] > j).view(n, 1, 1, 1), h, kept)
    s["h"].copy_((h if s["advance"] is None else kept).view(n, c, ns))
    return _finish(s, y.view(s["x"].shape), s["x"]), s["h"]


def _plain_verify(s):
    case, p, q = s["case"], s["p"], s["q"]
    n, t, v = case["n"], case["t"], case["vocab"]
    rows = torch.arange(n, device=DEV)
    ids = s["tokens"].long()
    at = ids.unsqueeze(2)
    # products of two fp32 numbers are exact in 64 bits: no border is decided by a rounding
    ok = s["u_accept"].double() * q.gather(2, at).squeeze(2).double() < \
        p[:, :t].gather(2, at).squeeze(2).double()
    kept = torch.cumprod(ok.long(), dim=1).sum(dim=1)  # drafted tokens accepted
    w = p[rows, kept].float()
    rest = w
    if t > 0:
        rest = w - torch.where((kept < t).unsqueeze(1), q[rows, kept.clamp(max=t - 1)].float(), 0.0)

    def units(x):  # weights as whole numbers of 2^-56: their sums do not depend on the order
        return (torch.where(x > 0, x, 0.0).clamp(max=1.0).double() * 2.0 ** 56).long()

    run = torch.cumsum(units(rest), dim=1)
    run = torch.where(run[:, -1:] > 0, run, torch.cumsum(units(w), dim=1))
    total = run[:, -1]
    u = (s["u_sample"].double() * 2.0 ** 24).long()
    limit = (total >> 32) * u * 256 + (((total & 0xffffffff) * u) >> 24)  # floor(total u)
    new = (run <= limit.unsqueeze(1)).sum(dim=1)
    place = torch.arange(t + 1, device=DEV).unsqueeze(0)
    out = torch.cat([ids, ids.new_zeros(n, 1)], dim=1)
    out = torch.where(place < kept.unsqueeze(1), out, -1)
    out[rows, kept] = new
    return out.to(torch.int32), (kept + 1).to(torch.int32)


# ------------------------------------------------------------------------- one pass
def run(s):
    case, op = s["case"], s["case"]["op"]
    if not own:
        return {"conv": _plain_conv, "conv_step": _plain_conv_step, "scan": _plain_scan,
                "scan_step": _plain_scan_step, "verify": _plain_verify}[op](s)
    import chunked_gated_delta_fwd_gb300 as kda

    if op == "verify":
        return kda.verify_draft(s["tokens"], s["q"], s["p"], s["u_accept"], s["u_sample"])
    if op == "conv":
        return kda.causal_conv_fwd(s["x"], s["w"], s["bias"], s["state"], s["cu"],
                                   silu=case["silu"])
    if op == "conv_step":
        if case["t"] == 1:
            y = kda.causal_conv_step(s["x"], s["w"], s["state"], s["bias"], silu=case["silu"])
        else:
            y = kda.causal_conv_multi_step(s["x"], s["w"], s["state"], s["advance"], s["bias"],
                                           silu=case["silu"])
        return y, s["state"]
    more = dict(D=s["D"], z=s["z"], dt_bias=s["dt_bias"])
    if op == "scan":
        return kda.selective_scan_fwd(s["x"], s["dt"], s["A"], s["B"], s["C"], s["h"], s["cu"],
                                      **more)
    if case["t"] == 1:
        y = kda.selective_step(s["x"], s["dt"], s["A"], s["B"], s["C"], s["h"], **more)
    else:
        y = kda.selective_multi_step(s["x"], s["dt"], s["A"], s["B"], s["C"], s["h"], s["advance"],
                                     **more)
    return y, s["h"]


# ------------------------------------------------------------------------- the work
def work(case):
    e, op = 2 if case["dtype"] == "bf16" else 4, case["op"]
    if op == "verify":
        n, t, v = case["n"], case["t"], case["vocab"]
        rejected = 1 - case["keep"] ** t  # such a sequence needs a row of q too
        return {"bytes": int(n * (v * e * (1 + rejected) + t * (2 * e + 8) + 4 * t + 12)),
                "flops": int(n * v * (1 + rejected))}
    c = case["c"]
    if op in ("conv", "scan"):
        n, nt = len(_lens(case)), sum(_lens(case))
    else:
        n, nt = case["n"], case["n"] * case["t"]
    if op in ("conv", "conv_step"):
        w = case["w"]
        states = 2 if op == "conv_step" or case["state"] else 1
        return {"bytes": 2 * nt * c * e + states * n * (w - 1) * c * e + 4 * c * (w + case["bias"]),
                "flops": nt * c * (2 * w + (4 if case["silu"] else 0))}
    ns = case["s"]
    states = 2 if op == "scan_step" or case["h0"] else 1
    return {"bytes": nt * e * (c * (4 if case["gate"] else 3) + 2 * case["groups"] * ns) +
            states * 4 * n * c * ns + 4 * c * (ns + 2),
            "flops": nt * c * (7 * ns + 12)}


# ------------------------------------------------------------------------- in 64 bits
def _exact_conv(s):
    """Sequence by sequence: kept inputs and tokens as one row, every window of it times w."""
    case, x = s["case"], s["x"]
    k = case["w"] - 1
    outs, kept, first = [], [], 0
    for i, size in enumerate(s["lens"]):
        old = torch.zeros(k, case["c"], dtype=x.dtype, device=DEV) if s["state"] is None \
            else s["state"][i]
        row = torch.cat([old, x[first:first + size]])
        kept.append(row[size:].double())
        first += size
        if size > 0:
            outs.append(torch.einsum("tcw,cw->tc", row.double().unfold(0, k + 1, 1), s["w"].double()))
    y = torch.cat(outs) if outs else x.double()
    if s["bias"] is not None:
        y = y + s["bias"].double()
    return (y * torch.sigmoid(y) if case["silu"] else y), torch.stack(kept)


def _exact_conv_step(s):
    case = s["case"]
    n, t, k, c = case["n"], case["t"], case["w"] - 1, case["c"]
    row = torch.cat([s["state"], s["x"].reshape(n, t, c)], dim=1).double()
    y = torch.einsum("ntcw,cw->ntc", row.unfold(1, k + 1, 1), s["w"].double())
    if s["bias"] is not None:
        y = y + s["bias"].double()
    if case["silu"]:
        y = y * torch.sigmoid(y)
    adv = [t] * n if s["advance"] is None else s["advance"].tolist()
    return y.reshape(s["x"].shape), torch.stack([row[i, a:a + k] for i, a in enumerate(adv)])


def _exact_scan(s, lens, advance=None):
    """Token by token over all sequences; a sequence that has ended keeps its state."""
    case = s["case"]
    n, c, ns, g = len(lens), case["c"], case["s"], case["groups"]
    first = torch.tensor([0] + lens[:-1]).cumsum(0).to(DEV)
    size = torch.tensor(lens, device=DEV)
    flat = {i: s[i].reshape(-1, *s[i].shape[-tail:]) for i, tail in
            (("x", 1), ("dt", 1), ("B", 2), ("C", 2))}
    h = torch.zeros(n, c, ns, dtype=torch.float64, device=DEV) if s["h"] is None else s["h"].double()
    h, kept = h.clone(), h.clone()
    y = torch.zeros(flat["x"].shape, dtype=torch.float64, device=DEV)
    A, bias = s["A"].double(), s["dt_bias"].double()
    most, even = max(lens), min(lens) == max(lens)
    for t in range(most):
        live = torch.arange(n, device=DEV) if even else (size > t).nonzero().squeeze(1)
        rows = first[live] + t
        delta = torch.nn.functional.softplus(flat["dt"][rows].double() + bias, threshold=700.0)
        wide = [flat[i][rows].double().repeat_interleave(c // g, dim=1) for i in "BC"]
        old = h if even else h[live]
        new = old * torch.exp(delta.unsqueeze(2) * A)
        new += (delta * flat["x"][rows].double()).unsqueeze(2) * wide[0]
        y[rows] = torch.einsum("ncs,ncs->nc", new, wide[1])
        if even:
            h = new
        else:
            h[live] = new
        if advance is not None:
            kept = torch.where((advance > t).view(n, 1, 1), h, kept)
    y = y + s["D"].double() * flat["x"].double()
    if s["z"] is not None:
        z = s["z"].reshape(-1, c).double()
        y = y * z * torch.sigmoid(z)
    return y.view(s["x"].shape), (h if advance is None else kept)


def _exact_verify(s):
    case = s["case"]
    n, t = case["n"], case["t"]
    tokens, u = s["tokens"].tolist(), s["u_accept"].double().tolist()
    draw = s["u_sample"].double().tolist()
    out, count = [], []
    for i in range(n):
        k = 0
        while k < t:
            p, q = (float(s[x][i, k, tokens[i][k]]) for x in "pq")
            if not u[i][k] * q < p:
                break
            k += 1
        w = s["p"][i, k].double()
        rest = w if k == t else torch.clamp(w - s["q"][i, k].double(), min=0)
        rest = rest if float(rest.sum()) > 0 else w
        run = torch.cumsum(rest, dim=0)
        new = int((run > draw[i] * run[-1]).long().argmax())
        out.append(tokens[i][:k] + [new] + [-1] * (t - k))
        count.append(k + 1)
    return (torch.tensor(out, dtype=torch.int32, device=DEV),
            torch.tensor(count, dtype=torch.int32, device=DEV))


def exact(case, seed):
    s, op = prepare(case, seed), case["op"]
    if op == "verify":
        return _exact_verify(s)
    if op == "conv":
        return _exact_conv(s)
    if op == "conv_step":
        return _exact_conv_step(s)
    if op == "scan":
        return _exact_scan(s, s["lens"])
    return _exact_scan(s, [case["t"]] * case["n"], s["advance"])
