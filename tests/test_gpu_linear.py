"""GPU parity of linear attention with a decay for each head against the fp64 oracle.

Bounds, elementwise.  M is the result of the same recurrence on |q|, |k|, |v|, |h0|: the sum
of the magnitudes of every term of a result.  u = 2^-24.
* fp32 arithmetic: a result meets at most 128 (channels) + 64 (keys of a chunk) + 128 (state
  row) + 64 (local state) additions, two a chunk in the scan (lengths here stay below 40
  chunks), and decays whose exponentials are off by |x| u + 4 u on terms that weigh e^x: all
  in all below 512 u M.
* bf16: tensor-core operands are rounded to bf16 twice on the way to o, the scores and the
  state copy, half a step (2^-8) each and each on a part of the terms; o is rounded once:
  2^-8 |o| + 2^-8 (1 + 2^-6) M.  The weighted keys of the state update are kept as two bf16
  parts (2^-16), so the fp32 states stay within (2^-16 + 512 u) M.
The relative L2 bounds of the package are checked as well.
"""

import numpy as np
import pytest
import torch

import oracle
from tests.gpu_helpers import F32_REL_L2, assert_close, errors, to64

pytestmark = pytest.mark.gpu

DT = [torch.bfloat16, torch.float32]
IDS = ["bf16", "f32"]
U = 2.0 ** -24


@pytest.fixture(scope="module")
def kda():
    import chunked_gated_delta_fwd_gb300 as m

    return m


def make(lens, H, Hk, dtype, seed, decay="token", h0=True, strong=False):
    gen = torch.Generator().manual_seed(seed)
    nt = sum(lens)
    unit = lambda x: x / x.norm(dim=-1, keepdim=True).clamp_min(1e-6)  # noqa: E731
    q = unit(torch.randn(nt, Hk, 128, generator=gen)).to(dtype)
    k = unit(torch.randn(nt, Hk, 128, generator=gen)).to(dtype)
    v = torch.randn(nt, H, 128, generator=gen).to(dtype)
    if decay == "head":
        g = -torch.rand(H, generator=gen) * 0.5
    else:
        a = torch.rand(H, generator=gen) * 6 - 5
        g = -torch.exp(a) * torch.nn.functional.softplus(torch.randn(nt, H, generator=gen))
    if strong:
        g = g * 40
    s0 = torch.randn(len(lens), H, 128, 128, generator=gen) * 0.1 if h0 else None
    cu = torch.tensor([0] + list(np.cumsum(lens)), dtype=torch.int32)
    return dict(q=q, k=k, v=v, g=g, h0=s0, cu=cu)


def magnitudes(d, scale, n_advance=None):
    a = lambda t: None if t is None else np.abs(to64(t))  # noqa: E731
    return oracle.linear_recurrence(a(d["q"]), a(d["k"]), a(d["v"]), d["g"], a(d["h0"]), d["cu"],
                                    abs(scale), n_advance)


def check(o, hT, d, scale=1.0, dtype=None, n_advance=None, fp32_cores=False):
    """o and hT against the oracle; bf16 `dtype` with `fp32_cores` still rounds o."""
    dtype = dtype or d["q"].dtype
    ro, rh = oracle.linear_recurrence(d["q"], d["k"], d["v"], d["g"], d["h0"], d["cu"], scale,
                                      n_advance)
    mo, mh = magnitudes(d, scale, n_advance)
    bo, bh = 512 * U * mo, 512 * U * mh
    if dtype == torch.bfloat16:
        bo = bo + 2.0 ** -8 * np.abs(ro)
        if not fp32_cores:
            bo, bh = bo + 2.0 ** -8 * (1 + 2.0 ** -6) * mo, bh + 2.0 ** -16 * mh
    if o is not None and ro.size:
        err = np.abs(to64(o) - ro)
        assert np.all(err <= bo + 1e-30), float(np.max(err / (bo + 1e-30)))
        assert_close(o, ro, dtype, "o")
    if hT is not None:
        err = np.abs(to64(hT) - rh)
        assert np.all(err <= bh + 1e-30), float(np.max(err / (bh + 1e-30)))
        assert errors(hT, rh)[0] <= F32_REL_L2
    return ro, rh


def cuda(d):
    return {k: (v.cuda() if isinstance(v, torch.Tensor) else v) for k, v in d.items()}


def chunk(kda, d, **kw):
    c = cuda(d)
    return kda.linear_chunk_fwd(c["q"], c["k"], c["v"], c["g"], c["h0"], c["cu"], **kw)


# ------------------------------------------------------------------- the prompt pass
@pytest.mark.parametrize("dtype", DT, ids=IDS)
@pytest.mark.parametrize("T", [1, 2, 15, 31, 32, 33, 63, 64, 65, 127, 128, 129, 191, 255, 256, 257,
                               385])
def test_lengths(kda, dtype, T):
    d = make([T], 2, 2, dtype, seed=T, h0=T % 2 == 1)
    check(*chunk(kda, d, scale=0.7), d, 0.7)
    kda.get_device_error()


@pytest.mark.parametrize("dtype", DT, ids=IDS)
@pytest.mark.parametrize("decay", ["token", "head"])
@pytest.mark.parametrize("h0", [False, True], ids=["zero", "h0"])
def test_ragged_batch_and_shared_keys(kda, dtype, decay, h0):
    d = make([130, 0, 1, 64, 0, 300, 127, 129, 3], 6, 2, dtype, seed=5, decay=decay, h0=h0)
    check(*chunk(kda, d), d)


@pytest.mark.parametrize("H,Hk", [(1, 1), (5, 5), (8, 1), (12, 4)])
def test_bf16_head_layouts(kda, H, Hk):
    d = make([200, 77], H, Hk, torch.bfloat16, seed=H)
    check(*chunk(kda, d), d)


def test_bf16_on_fp32_cores(kda):
    d = make([150, 0, 65], 4, 2, torch.bfloat16, seed=8)
    check(*chunk(kda, d, flags=kda.FP32_CORES), d, fp32_cores=True)


@pytest.mark.parametrize("dtype", DT, ids=IDS)
def test_batched_without_cu_seqlens(kda, dtype):
    d = make([150, 150, 150], 3, 3, dtype, seed=12)
    c = cuda(d)
    sh = lambda t: t.view(3, 150, *t.shape[1:])  # noqa: E731
    o, hT = kda.linear_chunk_fwd(sh(c["q"]), sh(c["k"]), sh(c["v"]), sh(c["g"]), c["h0"])
    check(o.view(450, 3, 128), hT, d)
    one, none = kda.linear_chunk_fwd(c["q"].unsqueeze(0), c["k"].unsqueeze(0), c["v"].unsqueeze(0),
                                     c["g"].unsqueeze(0), c["h0"], c["cu"],
                                     output_final_state=False)
    assert none is None and torch.equal(one.view(450, 3, 128), o.view(450, 3, 128))


@pytest.mark.parametrize("dtype", DT, ids=IDS)
def test_strong_decays_and_dropped_states(kda, dtype):
    """g down to several hundred below zero, to the lowest fp32 value and to -inf: the
    state is dropped there and what follows is exact to the same bound."""
    d = make([300, 140], 3, 3, dtype, seed=21, strong=True)
    d["g"][17, 0] = d["g"][100:103, 1] = -float("inf")
    d["g"][128, 0] = d["g"][0, 2] = d["g"][310, 1] = -float("inf")
    d["g"][200, 0] = -3.4e38
    d["g"][40:60, 2] = -1e4
    d["g"][256:300] = -0.01
    check(*chunk(kda, d), d)


@pytest.mark.parametrize("dtype", DT, ids=IDS)
def test_no_decay(kda, dtype):
    d = make([260], 2, 2, dtype, seed=23)
    d["g"].zero_()
    check(*chunk(kda, d), d)


@pytest.mark.parametrize("dtype", DT, ids=IDS)
def test_neighbours_with_nan_and_inf_stay_by_themselves(kda, dtype):
    """Sequences and heads next to non-finite inputs get the results that they get alone."""
    lens, H = [70, 50, 130, 90], 3
    d = make(lens, H, H, dtype, seed=31)
    ro, rh = check(*chunk(kda, d), d)
    bad = {k: (v.clone() if isinstance(v, torch.Tensor) else v) for k, v in d.items()}
    a, b = int(d["cu"][1]), int(d["cu"][2])
    bad["q"][a:b] = float("nan")
    bad["k"][a:b] = float("inf")
    bad["v"][a:b] = float("nan")
    bad["g"][a:b] = float("nan")
    bad["h0"][1] = float("nan")
    bad["v"][b:, 1] = float("nan")       # and one head of the sequences behind
    bad["k"][b:, 1] = float("inf")
    o, hT = chunk(kda, bad)
    g, gh = chunk(kda, d)
    keep = [h for h in range(H) if h != 1]
    assert torch.equal(o[:a], g[:a]) and torch.equal(hT[0], gh[0])
    assert torch.equal(o[b:][:, keep], g[b:][:, keep])
    assert torch.equal(hT[2:][:, keep], gh[2:][:, keep])


@pytest.mark.parametrize("dtype", DT, ids=IDS)
def test_state_in_place_and_split_prompt(kda, dtype):
    """Two calls over the halves of a prompt, the state handed on in place, equal one."""
    d = make([333], 4, 4, dtype, seed=41)
    c = cuda(d)
    S = c["h0"].clone()
    outs = []
    for a, b in ((0, 140), (140, 333)):
        cut = lambda t: t[a:b].unsqueeze(0).contiguous()  # noqa: E731
        o, hT = kda.linear_chunk_fwd(cut(c["q"]), cut(c["k"]), cut(c["v"]), cut(c["g"]), S,
                                     final_state_out=S)
        assert hT is S
        outs.append(o[0])
    check(torch.cat(outs), S, d)


@pytest.mark.parametrize("dtype", DT, ids=IDS)
def test_empty_batches(kda, dtype):
    d = make([0, 0, 0], 2, 2, dtype, seed=43)
    o, hT = chunk(kda, d)
    assert o.shape == (0, 2, 128) and torch.equal(hT.cpu(), d["h0"])
    d["h0"] = None
    assert torch.count_nonzero(chunk(kda, d)[1]) == 0


@pytest.mark.parametrize("dtype", DT, ids=IDS)
def test_malformed_cu_seqlens_is_reported(kda, dtype):
    d = make([100, 60], 2, 2, dtype, seed=45)
    kda.get_device_error()
    for cu in ([0, 100, 150], [5, 100, 160], [0, 120, 90], [0, -7, 160], [0, 100, 1 << 30]):
        d["cu"] = torch.tensor(cu, dtype=torch.int32)
        chunk(kda, d)
        with pytest.raises(kda.KdaError, match="cu_seqlens"):
            kda.get_device_error()
    d["cu"] = torch.tensor([0, 100, 150], dtype=torch.int32)  # rows behind the last sequence
    out = torch.full((160, 2, 128), 7.0, dtype=dtype, device="cuda")
    chunk(kda, d, out=out)
    assert bool((out[150:] == 7).all()) and not bool((out[:150] == 7).any())
    with pytest.raises(kda.KdaError):
        kda.get_device_error()


@pytest.mark.parametrize("dtype", DT, ids=IDS)
def test_many_sequences_and_repeatable_bits(kda, dtype):
    """More (sequence, head) pairs than the GPU has SMs, run twice: the same bits."""
    lens = [int(x) for x in np.random.default_rng(3).integers(0, 200, 90)]
    d = make(lens, 4, 2, dtype, seed=47)
    o, hT = chunk(kda, d)
    o2, hT2 = chunk(kda, d)
    assert torch.equal(o, o2) and torch.equal(hT, hT2)
    check(o, hT, d)


def test_two_streams_and_a_captured_graph(kda):
    a, b = make([300, 40], 4, 2, torch.bfloat16, seed=51), make([129], 4, 2, torch.bfloat16, seed=52)
    ra, rb = chunk(kda, a), chunk(kda, b)
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    ca, cb = cuda(a), cuda(b)
    torch.cuda.synchronize()
    call = lambda c, **kw: kda.linear_chunk_fwd(c["q"], c["k"], c["v"], c["g"], c["h0"], c["cu"],  # noqa: E731
                                                **kw)
    with torch.cuda.stream(s1):
        oa = call(ca)
    with torch.cuda.stream(s2):
        ob = call(cb)
    torch.cuda.synchronize()
    assert torch.equal(oa[0], ra[0]) and torch.equal(oa[1], ra[1])
    assert torch.equal(ob[0], rb[0]) and torch.equal(ob[1], rb[1])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        go, gh = call(ca)
    ca["v"].mul_(2)
    ca["h0"].mul_(2)
    for _ in range(2):
        graph.replay()
    want = call(ca)
    assert torch.equal(go, want[0]) and torch.equal(gh, want[1])


def test_chunk_refusals(kda):
    d = cuda(make([64], 4, 2, torch.bfloat16, seed=61))
    base = dict(q=d["q"], k=d["k"], v=d["v"], g=d["g"], h0=d["h0"], cu=d["cu"])
    bad = [
        dict(k=d["k"].float()), dict(k=d["k"][:, :1].contiguous()), dict(v=d["v"][:63]),
        dict(v=d["v"][:, :3].contiguous()), dict(g=d["g"][:63]), dict(g=d["g"].double()),
        dict(g=d["g"][0, :3].contiguous()), dict(h0=d["h0"][:, :2].contiguous()),
        dict(cu=d["cu"].long()), dict(cu=None), dict(cu=d["cu"][:1]), dict(v=d["v"].transpose(0, 1)),
        dict(q=d["q"].half(), k=d["k"].half(), v=d["v"].half()), dict(scale=float("nan")),
        dict(q=d["q"][0], k=d["k"][0]), dict(v=d["v"][0]),
        dict(out=d["v"][:63]), dict(final_state_out=d["h0"][:, :2].contiguous()),
        dict(flags=1 << 12),
    ]
    for x in bad:
        a = dict(base)
        a.update(x)
        args = [a.pop(n) for n in ("q", "k", "v", "g", "h0", "cu")]
        with pytest.raises((TypeError, ValueError, kda.KdaError)):
            kda.linear_chunk_fwd(*args, **a)


# --------------------------------------------------------------------- single tokens
@pytest.mark.parametrize("dtype", DT, ids=IDS)
@pytest.mark.parametrize("N,H,Hk,decay", [(1, 1, 1, "token"), (5, 6, 2, "token"), (90, 4, 4, "head"),
                                          (3, 8, 1, "head")])
def test_single_steps(kda, dtype, N, H, Hk, decay):
    """Four tokens in a row, one call each, against the oracle's four."""
    d = make([4] * N, H, Hk, dtype, seed=N, decay=decay)
    if decay == "token":
        d["g"][1] = -float("inf")
    c = cuda(d)
    S, outs = c["h0"].clone(), []
    for t in range(4):
        at = lambda x: x.view(N, 4, *x.shape[1:])[:, t].contiguous()  # noqa: E731
        g = c["g"] if decay == "head" else at(c["g"])
        outs.append(kda.linear_recurrent_step(at(c["q"]), at(c["k"]), at(c["v"]), g, S, scale=0.3))
    check(torch.stack(outs, 1).view(4 * N, H, 128), S, d, 0.3, fp32_cores=True)


@pytest.mark.parametrize("dtype", DT, ids=IDS)
@pytest.mark.parametrize("T", [1, 3, 16])
def test_multi_steps_with_partial_advance(kda, dtype, T):
    N, H = 6, 4
    d = make([T] * N, H, 2, dtype, seed=T)
    adv = [0, 1, T, max(0, T - 1), T, min(2, T)]
    c = cuda(d)
    sh = lambda t: t.view(N, T, *t.shape[1:])  # noqa: E731
    S = c["h0"].clone()
    n = torch.tensor(adv, dtype=torch.int32, device="cuda")
    o = kda.linear_recurrent_multi_step(sh(c["q"]), sh(c["k"]), sh(c["v"]), sh(c["g"]), S, n)
    check(o.view(N * T, H, 128), S, d, n_advance=adv, fp32_cores=True)
    assert torch.equal(S[0], c["h0"][0])
    S2, S3 = c["h0"].clone(), c["h0"].clone()
    n[1], n[2] = -5, 99  # clamped to [0, T]
    none = kda.linear_recurrent_multi_step(sh(c["q"]), sh(c["k"]), sh(c["v"]), sh(c["g"]), S2, n,
                                           return_outputs=False)
    assert none is None and torch.equal(S2[1], c["h0"][1]) and torch.equal(S2[2], S[2])
    kda.linear_recurrent_multi_step(sh(c["q"]), sh(c["k"]), sh(c["v"]), sh(c["g"]), S3)
    check(None, S3, d)


def test_step_refusals_and_no_sequences(kda):
    d = cuda(make([1] * 3, 4, 2, torch.float32, seed=71))
    S = d["h0"]
    ok = dict(q=d["q"], k=d["k"], v=d["v"], g=d["g"], S=S)
    for x in (dict(S=None), dict(q=d["q"][:2]), dict(k=d["k"].bfloat16()), dict(v=d["v"][:2]), dict(S=S[:2]),
              dict(S=S.bfloat16()), dict(S=S.transpose(2, 3)), dict(g=d["g"][:2]),
              dict(g=d["g"].bfloat16()), dict(out=d["v"][:2]), dict(scale=float("inf")),
              dict(q=d["q"].unsqueeze(1), k=d["k"].unsqueeze(1))):
        a = dict(ok)
        a.update(x)
        with pytest.raises((TypeError, ValueError, kda.KdaError)):
            kda.linear_recurrent_step(**a)
    m = {n: (t if n == "S" else t.unsqueeze(1)) for n, t in ok.items()}
    long = {n: (t if n == "S" else t.expand(3, 17, *t.shape[2:]).contiguous()) for n, t in m.items()}
    for a in (long, dict(m, n_advance=torch.zeros(2, dtype=torch.int32, device="cuda")),
              dict(m, n_advance=torch.zeros(3, device="cuda"))):
        with pytest.raises((TypeError, ValueError, kda.KdaError)):
            kda.linear_recurrent_multi_step(**a)
    e = {n: t[:0].contiguous() for n, t in ok.items()}
    assert kda.linear_recurrent_step(**e).shape == (0, 4, 128)


def test_step_captured_and_replayed(kda):
    d = cuda(make([1] * 40, 8, 8, torch.bfloat16, seed=73))
    S, ref = d["h0"].clone(), d["h0"].clone()
    out = torch.empty_like(d["v"])
    args = (d["q"], d["k"], d["v"], d["g"])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        kda.linear_recurrent_step(*args, S, out=out)
    for _ in range(3):
        graph.replay()
        want = kda.linear_recurrent_step(*args, ref)
    assert torch.equal(S, ref) and torch.equal(out, want)


# ---------------------------------------------------------------------- as one layer
@pytest.mark.parametrize("dtype", DT, ids=IDS)
def test_layer_prompt_then_tokens(kda, dtype):
    """Norm and rotation, prompt pass, output gate, then single tokens and a drafted run with
    the same operators: against the oracle's chain over the whole sequences."""
    lens, extra, H, Hk = [150, 37], 4, 4, 2
    gen = torch.Generator().manual_seed(81)
    full = [n + extra for n in lens]
    nt = sum(full)
    qkv = torch.randn(nt, H + Hk + Hk, 128, generator=gen).to(dtype)
    x = torch.randn(nt, H, 128, generator=gen).to(dtype)
    g = -torch.rand(nt, H, generator=gen)
    wq, wk = torch.rand(128, generator=gen) + 0.5, torch.rand(128, generator=gen) + 0.5
    f = (10000.0 ** (-torch.arange(32, dtype=torch.float64) / 32)).float()
    pos = torch.cat([torch.arange(n) for n in full]).to(torch.int32)
    scale = 128 ** -0.5
    q_in, k_in, v_in = qkv[:, :Hk], qkv[:, Hk:2 * Hk], qkv[:, 2 * Hk:].contiguous()
    dev = {n: t.cuda() for n, t in dict(qkv=qkv, x=x, g=g, wq=wq, wk=wk, f=f, pos=pos, v=v_in).items()}
    qn, kn = kda.qk_norm_rope(dev["qkv"][:, :Hk], dev["qkv"][:, Hk:2 * Hk], dev["pos"], dev["f"],
                              q_weight=dev["wq"], k_weight=dev["wk"])
    starts = np.cumsum([0] + full)
    prompt = torch.cat([torch.arange(s, s + n) for s, n in zip(starts, lens)]).cuda()
    cu = torch.tensor([0] + list(np.cumsum(lens)), dtype=torch.int32).cuda()
    o, S = kda.linear_chunk_fwd(qn[prompt], kn[prompt], dev["v"][prompt], dev["g"][prompt], None, cu,
                                scale=scale)
    got = torch.empty(nt, H, 128, dtype=dtype, device="cuda")
    got[prompt] = kda.output_gate(o, dev["x"][prompt])
    one = torch.tensor([s + n for s, n in zip(starts, lens)]).cuda()  # one token each
    got[one] = kda.output_gate(kda.linear_recurrent_step(qn[one], kn[one], dev["v"][one],
                                                         dev["g"][one], S, scale=scale), dev["x"][one])
    draft = torch.stack([torch.arange(s + n + 1, s + n + extra) for s, n in zip(starts, lens)]).cuda()
    got[draft] = kda.output_gate(
        kda.linear_recurrent_multi_step(qn[draft], kn[draft], dev["v"][draft], dev["g"][draft], S,
                                        scale=scale), dev["x"][draft])
    # the oracle takes the operators' own normed q and k: their parity is tested by itself
    full_cu = torch.tensor(starts, dtype=torch.int32)
    d = dict(q=qn.cpu(), k=kn.cpu(), v=v_in, g=g, h0=None, cu=full_cu)
    ro, rh = oracle.linear_recurrence(d["q"], d["k"], d["v"], d["g"], None, full_cu, scale)
    ref = oracle.output_gate(ro, x)
    rel, _ = errors(got, ref)
    assert rel <= (1e-2 if dtype == torch.bfloat16 else 1e-5), rel
    assert errors(S, rh)[0] <= F32_REL_L2
    qr = oracle.norm_rope(q_in, pos, f, wq)
    assert errors(qn, qr)[0] <= (2.0 ** -8 if dtype == torch.bfloat16 else 1e-6)


# -------------------------------------------------------------------------- segments
@pytest.mark.parametrize("decay", ["token", "head"])
@pytest.mark.parametrize("n", [1, 2, 5])
def test_segments_match_the_oracle(kda, n, decay):
    """Sequences cut into segments of n chunks: empty, one-token, exact and ragged lengths."""
    d = make([700, 0, 1, 128 * n, 128 * n + 1, 127], 3, 3, torch.bfloat16, seed=90 + n, decay=decay)
    check(*chunk(kda, d, flags=kda.segment_chunks(n), scale=0.5), d, 0.5)
    kda.get_device_error()


def test_segments_with_the_state_in_place_and_dropped(kda):
    d = make([1500], 2, 1, torch.bfloat16, seed=95)
    d["g"][600:603] = -float("inf")
    S = d["h0"].cuda()
    c = cuda(d)
    o, hT = kda.linear_chunk_fwd(c["q"], c["k"], c["v"], c["g"], S, c["cu"], final_state_out=S,
                                 flags=kda.segment_chunks(3))
    assert hT is S
    check(o, S, d)


def test_segments_chosen_for_a_long_sequence(kda):
    """One long sequence with few heads is cut by default (the kernels that ran say so) and
    agrees with the uncut run and, on its first head, with the oracle."""
    d = make([8192 + 77], 2, 2, torch.bfloat16, seed=97, decay="head")
    kda.profile_enable(True)
    o, hT = chunk(kda, d)
    ran = kda.profile_collect()
    kda.profile_enable(False)
    assert ran["kda_linear_tc"][0] == 1 and "kda_linear_tc_state" in ran
    o1, h1 = chunk(kda, d, flags=kda.SEQUENTIAL)
    assert errors(o, to64(o1))[0] <= 2.0 ** -8 and errors(hT, to64(h1))[0] <= F32_REL_L2
    one = dict(d, q=d["q"][:, :1], k=d["k"][:, :1], v=d["v"][:, :1], g=d["g"][:1], h0=d["h0"][:, :1])
    check(o[:, :1], hT[:, :1], one)


def test_segments_with_malformed_cu_seqlens(kda):
    d = make([400, 300], 2, 2, torch.bfloat16, seed=99)
    kda.get_device_error()
    for cu in ([0, 700, 500], [300, 700, 700], [0, -3, 900]):
        d["cu"] = torch.tensor(cu, dtype=torch.int32)
        chunk(kda, d, flags=kda.segment_chunks(1))
        with pytest.raises(kda.KdaError, match="cu_seqlens"):
            kda.get_device_error()


# ---------------------------------------------------------------- how chains are drawn
@pytest.mark.parametrize("n", [7, 40, 1100])
def test_long_ragged_batches_against_the_fp32_cores(kda, n):
    """More chains than SMs, four chunks each on average: drawn by ticket, the longest first
    (1100 sequences: as they come).  Against the fp32-core path on the same inputs, itself
    held to the oracle above."""
    gen = torch.Generator(device="cuda").manual_seed(n)
    lens = np.random.default_rng(n).integers(0, 1300, n)
    lens[0], lens[-1] = 0, 2500
    H = 160 // n + 1 if n < 160 else 1
    nt = int(lens.sum())
    assert n * H > 152 and nt >= n * 512
    unit = lambda x: x / x.norm(dim=-1, keepdim=True)  # noqa: E731
    r = lambda *s: torch.randn(*s, generator=gen, device="cuda")  # noqa: E731
    q, k = unit(r(nt, H, 128)).bfloat16(), unit(r(nt, H, 128)).bfloat16()
    v, g, h0 = r(nt, H, 128).bfloat16(), -0.2 * r(nt, H).abs(), 0.1 * r(n, H, 128, 128)
    cu = torch.tensor([0] + list(np.cumsum(lens)), dtype=torch.int32, device="cuda")
    kda.get_device_error()
    o, hT = kda.linear_chunk_fwd(q, k, v, g, h0, cu)
    ro, rh = kda.linear_chunk_fwd(q, k, v, g, h0, cu, flags=kda.FP32_CORES)
    kda.get_device_error()
    for x, y, tol in ((o, ro, 2.0 ** -8), (hT, rh, F32_REL_L2)):
        rel = float((x.double() - y.double()).norm() / y.double().norm())
        assert rel <= tol, rel
        big = (x.double() - y.double()).abs().max() / y.double().square().mean().sqrt()
        assert float(big) <= 40 * tol, float(big)


def test_a_workspace_is_reused_from_call_to_call(kda):
    """One workspace, full of garbage at first, for calls of all kinds in a row."""
    ds = [make([700, 90, 1, 0, 512], 48, 48, torch.bfloat16, seed=101, h0=False),
          make([4100], 2, 2, torch.bfloat16, seed=102), make([130, 70], 3, 3, torch.float32, seed=103)]
    want = [chunk(kda, d) for d in ds]
    need = max(kda.linear_chunk_fwd_workspace_size(int(d["cu"][-1]), len(d["cu"]) - 1,
                                                   d["v"].shape[1], d["v"].dtype) for d in ds)
    ws = torch.randint(0, 256, (need,), dtype=torch.uint8, device="cuda")
    for _ in range(2):
        for d, (o, hT) in zip(ds, want):
            o2, h2 = chunk(kda, d, workspace=ws)
            assert torch.equal(o, o2) and torch.equal(hT, h2)
    with pytest.raises(kda.KdaError, match="WORKSPACE"):
        chunk(kda, ds[1], workspace=ws[:256])


def test_every_path_captured_and_replayed_back_to_back(kda):
    """Uncut, drawn by ticket, cut into segments and fp32 cores, one after another in one graph
    on one workspace, replayed without a pause: a kernel that begins while the one before it
    ends sees all that its call wrote, and leaves the next call's part alone."""
    ds = [make([700, 90, 1, 0, 1300], 40, 40, torch.bfloat16, seed=111),
          make([1300, 90, 1, 0, 1300], 40, 40, torch.bfloat16, seed=116),
          make([3000], 2, 1, torch.bfloat16, seed=112), make([200], 3, 3, torch.bfloat16, seed=113),
          make([130, 70], 3, 3, torch.float32, seed=114), make([900], 8, 8, torch.float32, seed=115)]
    kda.profile_enable(True)
    want = [chunk(kda, d) for d in ds]
    ran = kda.profile_collect()
    kda.profile_enable(False)
    assert {"kda_linear_order", "kda_linear_tc_state", "kda_linear_out"} <= set(ran)
    cs = [cuda(d) for d in ds]
    need = max(kda.linear_chunk_fwd_workspace_size(int(d["cu"][-1]), len(d["cu"]) - 1,
                                                   d["v"].shape[1], d["v"].dtype) for d in ds)
    ws = torch.randint(0, 256, (need,), dtype=torch.uint8, device="cuda")
    call = lambda c: kda.linear_chunk_fwd(c["q"], c["k"], c["v"], c["g"], c["h0"], c["cu"],  # noqa: E731
                                          workspace=ws)
    kda.get_device_error()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = [call(c) for c in cs + cs[::-1]]
    for _ in range(20):
        graph.replay()
    for (o, hT), (ro, rh) in zip(got, want + want[::-1]):
        assert torch.equal(o, ro) and torch.equal(hT, rh)
    for o, hT in got:
        o.fill_(float("nan"))
        hT.fill_(float("nan"))
    graph.replay()
    for (o, hT), (ro, rh) in zip(got, want + want[::-1]):
        assert torch.equal(o, ro) and torch.equal(hT, rh)
    kda.get_device_error()


@pytest.mark.parametrize("T,H,cut", [(1024, 1, True), (1100, 19, False), (1500, 38, True),
                                     (2300, 50, True), (8300, 51, True)])
def test_lengths_around_the_cut(kda, T, H, cut):
    """Prompts about as long as it takes to be cut (segments of one chunk and more), against the
    uncut run."""
    gen = torch.Generator(device="cuda").manual_seed(T)
    unit = lambda x: x / x.norm(dim=-1, keepdim=True)  # noqa: E731
    r = lambda *s: torch.randn(*s, generator=gen, device="cuda")  # noqa: E731
    q, k, v = unit(r(1, T, H, 128)).bfloat16(), unit(r(1, T, H, 128)).bfloat16(), r(1, T, H, 128).bfloat16()
    g, h0 = -0.05 * r(1, T, H).abs(), 0.1 * r(1, H, 128, 128)
    kda.profile_enable(True)
    o, hT = kda.linear_chunk_fwd(q, k, v, g, h0)
    ran = kda.profile_collect()
    kda.profile_enable(False)
    assert ("kda_linear_tc_state" in ran) == cut
    ro, rh = kda.linear_chunk_fwd(q, k, v, g, h0, flags=kda.SEQUENTIAL)
    kda.get_device_error()
    assert errors(o, to64(ro))[0] <= 2.0 ** -8 and errors(hT, to64(rh))[0] <= F32_REL_L2


# ------------------------------------------------------------------- offsets past 32 bits
@pytest.mark.parametrize("flags", ["tensor cores", "fp32 cores"])
def test_a_prompt_whose_offsets_pass_32_bits(kda, flags):
    """The last sequence of a batch with over 2^31 elements equals the same sequence by itself."""
    fl = kda.FP32_CORES if flags == "fp32 cores" else 0
    H, lens = 96, [180000, 300]
    nt = sum(lens)
    assert nt * H * 128 > 2 ** 31
    gen = torch.Generator(device="cuda").manual_seed(7)
    r = lambda *s: torch.randn(*s, generator=gen, device="cuda", dtype=torch.bfloat16)  # noqa: E731
    q, k, v = 0.1 * r(nt, H, 128), 0.1 * r(nt, H, 128), r(nt, H, 128)
    g = -0.1 * torch.rand(nt, H, generator=gen, device="cuda")
    h0 = 0.1 * torch.randn(2, H, 128, 128, generator=gen, device="cuda")
    cu = torch.tensor([0, lens[0], nt], dtype=torch.int32, device="cuda")
    o, hT = kda.linear_chunk_fwd(q, k, v, g, h0, cu, flags=fl)
    tail = lambda x: x[lens[0]:].clone()  # noqa: E731
    ro, rh = kda.linear_chunk_fwd(tail(q), tail(k), tail(v), tail(g), h0[1:].clone(), cu[1:] - lens[0],
                                  flags=fl | kda.SEQUENTIAL)
    kda.get_device_error()
    assert torch.equal(o[lens[0]:], ro) and torch.equal(hT[1:], rh)
    del q, k, v, o
    torch.cuda.empty_cache()


def test_steps_whose_states_pass_32_bits(kda):
    N, H = 1400, 96
    assert N * H * 128 * 128 > 2 ** 31
    gen = torch.Generator(device="cuda").manual_seed(8)
    r = lambda *s: torch.randn(*s, generator=gen, device="cuda", dtype=torch.bfloat16)  # noqa: E731
    S = torch.zeros(N, H, 128, 128, device="cuda")
    S[-1] = torch.randn(H, 128, 128, generator=gen, device="cuda")
    one = S[-1:].clone()
    for T in (1, 3):
        q, k, v = r(N, T, H, 128), r(N, T, H, 128), r(N, T, H, 128)
        g = -torch.rand(N, T, H, generator=gen, device="cuda")
        last = [x[-1:].clone() for x in (q, k, v, g)]
        if T == 1:
            o = kda.linear_recurrent_step(*(x[:, 0] for x in (q, k, v, g)), S)
            ro = kda.linear_recurrent_step(*(x[:, 0] for x in last), one)
        else:
            o = kda.linear_recurrent_multi_step(q, k, v, g, S)
            ro = kda.linear_recurrent_multi_step(*last, one)
        assert torch.equal(o[-1:], ro) and torch.equal(S[-1:], one)
    del S
    torch.cuda.empty_cache()
