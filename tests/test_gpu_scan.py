"""GPU parity of the selective state space scan against the fp64 oracle.

Bounds, elementwise.  u = 2^-24, Mh and My the results of the same recurrence on |x|, |B|, |C|,
|h0| (delta >= 0).  |dt + bias| stays below 10 here.
* delta: the exponent's argument is off by 2 |v| u, the exponential by 4 u, quotient, series and
  sum by 6 u: 30 u of itself.
* a term of a state has met up to T decays.  Each is off by 4 u (exponential) and by the error of
  its argument x = delta A log2(e), 33 u |x|; over all of them the arguments add up to the
  log of the term's weight, and a weight below e^-60 counts for nothing: 60 * 33 u + 4 T u.  Each
  token's product and sum add 2 u: Th = (1980 + 6 T + 64) u Mh.
* y: a sum over S <= 32 states and D x: Ty = (1980 + 6 T + 64 + S + 4) u My; the gate passes it on
  and adds (10 + 3 |z|) u |y| of its own; bf16 rounds once, 2^-8 |y|.
The package's relative L2 bound, 1e-5 in fp32, is checked as well.
"""

import numpy as np
import pytest
import torch

import oracle
from tests.gpu_helpers import F32_REL_L2, errors, to64

pytestmark = pytest.mark.gpu

DT = [torch.bfloat16, torch.float32]
IDS = ["bf16", "f32"]
U = 2.0 ** -24


@pytest.fixture(scope="module")
def kda():
    import chunked_gated_delta_fwd_gb300 as m

    return m


def make(lens, ch, S, G, dtype, seed, h0=True, gate=True, skip=True, bias=True, strong=1.0):
    gen = torch.Generator().manual_seed(seed)
    nt = sum(lens)
    r = lambda *s: torch.randn(*s, generator=gen)  # noqa: E731
    xz = r(nt, 2 * ch).to(dtype)
    low = r(nt, 16 + 2 * G * S).to(dtype)
    d = dict(x=xz[:, :ch], z=xz[:, ch:] if gate else None, xz=xz, low=low, S=S, G=G, ch=ch,
             dt=(0.5 * r(nt, ch)).to(dtype), A=-(torch.rand(ch, S, generator=gen) * 8 + 0.1) * strong,
             D=r(ch) if skip else None, bias=r(ch) - 3.0 if bias else None,
             h0=r(len(lens), ch, S) if h0 else None)
    d["B"] = low[:, 16:16 + G * S].unflatten(1, (G, S))
    d["C"] = low[:, 16 + G * S:].unflatten(1, (G, S))
    d["cu"] = torch.tensor([0] + list(np.cumsum(lens)), dtype=torch.int32)
    return d


def on_gpu(d):
    """The inputs as a program holds them: x and z, and B and C, slices of packed projections."""
    c = lambda t: None if t is None else t.cuda()  # noqa: E731
    g = {k: c(d[k]) for k in ("dt", "A", "D", "bias", "h0", "cu")}
    xz, low, ch, n = d["xz"].cuda(), d["low"].cuda(), d["ch"], d["G"] * d["S"]
    g["x"], g["z"] = xz[:, :ch], None if d["z"] is None else xz[:, ch:]
    g["B"] = low[:, 16:16 + n].unflatten(1, (d["G"], d["S"]))
    g["C"] = low[:, 16 + n:].unflatten(1, (d["G"], d["S"]))
    return g


def scan(kda, d, **kw):
    g = on_gpu(d)
    return kda.selective_scan_fwd(g["x"], g["dt"], g["A"], g["B"], g["C"], g["h0"], g["cu"],
                                  D=g["D"], z=g["z"], dt_bias=g["bias"], **kw)


def check(y, hT, d, softplus=True, n_advance=None):
    args = (d["A"], d["B"].float(), d["C"].float(), d["h0"], d["cu"])
    more = dict(dt_bias=d["bias"], softplus=softplus, n_advance=n_advance)
    f = lambda t: None if t is None else t.float()  # noqa: E731
    ry, rh = oracle.selective_scan(f(d["x"]), f(d["dt"]), *args, D=d["D"], z=f(d["z"]), **more)
    a = lambda t: None if t is None else np.abs(to64(t))  # noqa: E731
    My, Mh = oracle.selective_scan(a(d["x"]), f(d["dt"]), d["A"], a(d["B"]), a(d["C"]), a(d["h0"]),
                                   d["cu"], D=a(d["D"]), **more)
    T = int(np.max(np.diff(d["cu"].numpy())))
    grow = 1980 + 6 * T + 64
    by = (grow + d["S"] + 4) * U * My
    if d["z"] is not None:
        z = to64(d["z"])
        by = by * np.abs(z / (1 + np.exp(-z))) + (10 + 3 * np.abs(z)) * U * np.abs(ry)
    if d["x"].dtype == torch.bfloat16:
        by = by * (1 + 2.0 ** -8) + 2.0 ** -8 * np.abs(ry)
    if y is not None and ry.size:
        err = np.abs(to64(y).reshape(ry.shape) - ry)
        assert np.all(err <= by + 1e-30), float(np.max(err / (by + 1e-30)))
        if y.dtype == torch.float32:
            assert errors(y.reshape(ry.shape), ry)[0] <= F32_REL_L2
    if hT is not None:
        err = np.abs(to64(hT) - rh)
        bh = grow * U * Mh
        assert np.all(err <= bh + 1e-30), float(np.max(err / (bh + 1e-30)))
        assert errors(hT, rh)[0] <= F32_REL_L2


LENS = [[1], [7], [8], [9], [16], [17], [63, 1], [0, 5, 0, 33, 2, 0], [64, 65, 127], [300], [0, 0]]


@pytest.mark.parametrize("dtype", DT, ids=IDS)
@pytest.mark.parametrize("S", [8, 16, 32])
@pytest.mark.parametrize("lens", LENS)
def test_prompts(kda, dtype, S, lens):
    d = make(lens, 48, S, 2, dtype, seed=sum(lens) + S)
    y, hT = scan(kda, d)
    check(y, hT, d)
    kda.get_device_error()


@pytest.mark.parametrize("dtype", DT, ids=IDS)
@pytest.mark.parametrize("ch,G", [(8, 1), (16, 2), (24, 1), (40, 1), (72, 3), (1000, 5), (2048, 1)])
def test_channels_and_groups(kda, dtype, ch, G):
    for S in (8, 16, 32):
        d = make([33, 20], ch, S, G, dtype, seed=ch + S)
        check(*scan(kda, d), d)


@pytest.mark.parametrize("dtype", DT, ids=IDS)
@pytest.mark.parametrize("h0,gate,skip,bias", [(False, False, False, False), (True, False, True, False),
                                               (False, True, False, True)])
def test_optional_inputs(kda, dtype, h0, gate, skip, bias):
    d = make([40, 3, 90], 24, 16, 1, dtype, seed=4, h0=h0, gate=gate, skip=skip, bias=bias)
    check(*scan(kda, d), d)


def test_steps_used_as_given(kda):
    d = make([50, 31], 24, 16, 1, torch.float32, seed=6)
    d["dt"], d["bias"] = d["dt"].abs() * 0.2, d["bias"].abs() * 0.05
    y, hT = scan(kda, d, softplus=False)
    check(y, hT, d, softplus=False)


@pytest.mark.parametrize("dtype", DT, ids=IDS)
def test_strong_and_absent_decays(kda, dtype):
    d = make([70], 24, 16, 1, dtype, seed=7, strong=400.0)  # decays that underflow at once
    check(*scan(kda, d), d)
    d = make([2000], 8, 8, 1, dtype, seed=8)
    d["A"][:] = 0.0
    check(*scan(kda, d), d)
    d = make([3000], 8, 16, 1, dtype, seed=9, strong=0.01)  # slow decays over many tokens
    check(*scan(kda, d), d)


@pytest.mark.parametrize("v", [-60.0, -30.0, -9.0, -1e-3, 0.0, 1e-3, 9.0, 30.0, 60.0])
def test_softplus_over_its_range(kda, v):
    """hT of one token from a zero state is delta x B: delta itself, to (2 |v| + 10) u."""
    n, dev = 64, "cuda"
    dt = torch.linspace(v - 0.5, v + 0.5, n, device=dev).view(1, n)
    one = torch.ones(1, n, device=dev)
    _, h = kda.selective_scan_fwd(one.unsqueeze(0), dt.unsqueeze(0), torch.zeros(n, 8, device=dev),
                                  torch.ones(1, 1, 1, 8, device=dev), torch.ones(1, 1, 1, 8, device=dev))
    ref = np.logaddexp(0.0, to64(dt[0]))
    assert np.all(np.abs(to64(h)[0, :, 0] - ref) <= (2 * abs(v) + 10) * U * ref)


@pytest.mark.parametrize("dtype", DT, ids=IDS)
def test_batches_in_place_and_outputs_of_the_caller(kda, dtype):
    d = make([40] * 3, 40, 16, 1, dtype, seed=12)
    g = on_gpu(d)
    v = lambda t: t.unflatten(0, (3, 40))  # noqa: E731
    h = g["h0"].clone()
    out = torch.full((120, 64), 7.0, dtype=dtype, device="cuda")
    y, hT = kda.selective_scan_fwd(v(g["x"]), v(g["dt"]), g["A"], v(g["B"]), v(g["C"]), h, D=g["D"],
                                   z=v(g["z"]), dt_bias=g["bias"], out=v(out[:, 16:56]),
                                   final_state_out=h)
    check(y, hT, d)
    assert hT.data_ptr() == h.data_ptr()
    assert torch.all(out[:, :16] == 7) and torch.all(out[:, 56:] == 7)
    y2, none = scan(kda, d, output_final_state=False)
    assert none is None and torch.equal(y2, y.reshape(120, 40))


@pytest.mark.parametrize("dtype", DT, ids=IDS)
def test_long_prompts_continue_from_their_states(kda, dtype):
    d = make([1500], 40, 16, 1, dtype, seed=13)
    y, hT = scan(kda, d)
    check(y, hT, d)
    for cut in (1, 700, 1024):
        a, b = dict(d), dict(d)
        for k in ("x", "z", "dt", "B", "C", "xz", "low"):
            a[k], b[k] = d[k][:cut], d[k][cut:]
        a["cu"], b["cu"] = (torch.tensor([0, n], dtype=torch.int32) for n in (cut, 1500 - cut))
        ya, ha = scan(kda, a)
        b["h0"] = ha.cpu()
        yb, hb = scan(kda, b)
        check(torch.cat([ya, yb]), hb, d)


@pytest.mark.parametrize("dtype", DT, ids=IDS)
@pytest.mark.parametrize("S", [8, 16, 32])
@pytest.mark.parametrize("lens", [[4097], [5000, 0, 1, 4100], [2600, 2048, 33, 3500], [9000]])
def test_few_channels_of_long_sequences(kda, dtype, S, lens):
    """Few enough (sequence, channels) for sequences to be cut, among them some shorter than a
    segment; in place, and twice the same bits."""
    d = make(lens, 24, S, 1, dtype, seed=sum(lens) + S, strong=0.05)
    y, hT = scan(kda, d)
    check(y, hT, d)
    g = on_gpu(d)
    h = g["h0"].clone()
    y2, _ = kda.selective_scan_fwd(g["x"], g["dt"], g["A"], g["B"], g["C"], h, g["cu"], D=g["D"],
                                   z=g["z"], dt_bias=g["bias"], final_state_out=h)
    assert torch.equal(y, y2) and torch.equal(h, hT)
    y3, none = scan(kda, d, output_final_state=False)
    assert none is None and torch.equal(y3, y)


def test_cut_sequences_malformed_captured_and_with_non_finite_inputs(kda):
    d = make([4500, 4700], 40, 16, 1, torch.bfloat16, seed=21, strong=0.05)
    g = on_gpu(d)
    args = (g["x"], g["dt"], g["A"], g["B"], g["C"], g["h0"])
    more = dict(D=g["D"], z=g["z"], dt_bias=g["bias"])
    y0, h0 = kda.selective_scan_fwd(*args, g["cu"], **more)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y1, h1 = kda.selective_scan_fwd(*args, g["cu"], **more)
        y2, h2 = kda.selective_scan_fwd(*args[:5], h1, g["cu"], **more)
    graph.replay()
    y3, h3 = kda.selective_scan_fwd(*args[:5], h0, g["cu"], **more)
    assert torch.equal(y0, y1) and torch.equal(h0, h1)
    assert torch.equal(y2, y3) and torch.equal(h2, h3)
    for cu in ([0, 9000, 4000], [7, 4500, 9200], [0, -5, 9200], [0, 2 ** 31 - 1, 9200]):
        buf = torch.full((9200 + 64, 40), 7.0, dtype=torch.bfloat16, device="cuda")
        kept = torch.full((4, 40, 16), 7.0, device="cuda")
        kda.selective_scan_fwd(*args, torch.tensor(cu, dtype=torch.int32, device="cuda"),
                               out=buf[32:-32], final_state_out=kept[1:3], **more)
        with pytest.raises(kda.KdaError):
            kda.get_device_error()
        assert torch.all(buf[:32] == 7) and torch.all(buf[-32:] == 7)
        assert torch.all(kept[0] == 7) and torch.all(kept[3] == 7)
    bad = dict(d)
    bad["xz"] = d["xz"].clone()
    bad["xz"][1000, 5] = float("nan")
    bad["xz"][6000, 7] = float("inf")
    y4, h4 = scan(kda, bad)
    same = torch.ones(9200, 40, dtype=torch.bool)
    same[1000:4500, 5] = same[6000:, 7] = False
    assert torch.equal(y4.cpu()[same], y0.cpu()[same]) and torch.isnan(h4[0, 5]).all()
    keep = torch.ones(2, 40, dtype=torch.bool)
    keep[0, 5] = keep[1, 7] = False
    assert torch.equal(h4.cpu()[keep], h0.cpu()[keep])


@pytest.mark.parametrize("dtype", DT, ids=IDS)
@pytest.mark.parametrize("S,N,ch,G,T", [(16, 1, 2560, 1, 401), (16, 5, 512, 2, 400), (8, 1, 4872, 1, 392),
                                        (32, 1, 1280, 1, 399), (16, 1, 4960, 1, 1600)])
def test_more_channels_than_run_at_once(kda, dtype, S, N, ch, G, T):
    """Channels for more than one and less than two (or more than two and less than three) rounds
    over the SMs, whose last ones are shared by two CTAs: odd and even tiles, in place, captured,
    and the same bits as a part of the channels alone."""
    d = make([T] * N, ch, S, G, dtype, seed=ch + T, strong=0.05)
    if N == 1:
        y, hT = scan(kda, d)  # packed, one sequence
    g = on_gpu(d)
    v = lambda t: t.unflatten(0, (N, T))  # noqa: E731
    h = g["h0"].clone()
    args = (v(g["x"]), v(g["dt"]), g["A"], v(g["B"]), v(g["C"]))
    more = dict(D=g["D"], z=v(g["z"]), dt_bias=g["bias"])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y2, _ = kda.selective_scan_fwd(*args, h, final_state_out=h, **more)
        y3, h3 = kda.selective_scan_fwd(*args, h, **more)
    graph.replay()
    check(y2, h, d)
    y4, h4 = kda.selective_scan_fwd(*args, h, **more)
    assert torch.equal(y3, y4) and torch.equal(h3, h4)
    if N == 1:
        assert torch.equal(y, y2[0]) and torch.equal(hT, h)
        part = ch // 16 * 8
        some = [t[..., :part] for t in args[:2]] + [g["A"][:part]] + list(args[3:])
        y5, h5 = kda.selective_scan_fwd(*some, g["h0"][:, :part].contiguous(), D=g["D"][:part],
                                        z=more["z"][..., :part], dt_bias=g["bias"][:part])
        assert torch.equal(y5, y2[..., :part]) and torch.equal(h5, h[:, :part])


def test_shared_channels_malformed_and_with_non_finite_inputs(kda):
    d = make([400], 2560, 16, 1, torch.bfloat16, seed=23, strong=0.05)
    g = on_gpu(d)
    args = (g["x"], g["dt"], g["A"], g["B"], g["C"], g["h0"])
    more = dict(D=g["D"], z=g["z"], dt_bias=g["bias"])
    y0, h0 = scan(kda, d)
    for cu in ([0, 399], [7, 400], [400, 400], [0, 7], [0, 2 ** 31 - 1], [300, -1]):
        buf = torch.full((400 + 64, 2560), 7.0, dtype=torch.bfloat16, device="cuda")
        kept = torch.full((3, 2560, 16), 7.0, device="cuda")
        kda.selective_scan_fwd(*args, torch.tensor(cu, dtype=torch.int32, device="cuda"),
                               out=buf[32:-32], final_state_out=kept[1:2], **more)
        with pytest.raises(kda.KdaError):
            kda.get_device_error()
        assert torch.all(buf[:32] == 7) and torch.all(buf[-32:] == 7)
        assert torch.all(kept[0] == 7) and torch.all(kept[2] == 7)
        if cu in ([400, 400], [300, -1]):  # no tokens: the state as it came
            assert torch.equal(kept[1:2], g["h0"])
    bad = dict(d)
    bad["xz"] = d["xz"].clone()
    bad["xz"][100, 5::160] = float("nan")  # of one unit in ten
    y1, h1 = scan(kda, bad)
    same = torch.ones(400, 2560, dtype=torch.bool)
    same[100:, 5::160] = False
    assert torch.equal(y1.cpu()[same], y0.cpu()[same]) and torch.isnan(h1[0, 5::160]).all()
    keep = torch.ones(2560, dtype=torch.bool)
    keep[5::160] = False
    assert torch.equal(h1[0].cpu()[keep], h0[0].cpu()[keep])


def test_results_do_not_depend_on_the_batch(kda):
    """A sequence alone, among others and twice: the same bits."""
    lens = [130, 0, 64, 777, 9]
    d = make(lens, 40, 16, 1, torch.bfloat16, seed=14)
    y, hT = scan(kda, d)
    y2, hT2 = scan(kda, d)
    assert torch.equal(y, y2) and torch.equal(hT, hT2)
    for n, (b, e) in enumerate(zip(d["cu"][:-1], d["cu"][1:])):
        one = dict(d)
        for k in ("x", "z", "dt", "B", "C", "xz", "low"):
            one[k] = d[k][b:e]
        one["cu"], one["h0"] = torch.tensor([0, e - b], dtype=torch.int32), d["h0"][n:n + 1]
        y1, h1 = scan(kda, one)
        assert torch.equal(y1, y[b:e]) and torch.equal(h1[0], hT[n])


def test_many_sequences(kda):
    gen = torch.Generator().manual_seed(3)
    lens = torch.randint(0, 12, (300,), generator=gen).tolist()
    d = make(lens, 24, 8, 1, torch.float32, seed=15)
    check(*scan(kda, d), d)


def test_non_finite_inputs_stay_in_their_channel_and_sequence(kda):
    d = make([30, 30], 48, 16, 1, torch.float32, seed=16)
    y, hT = scan(kda, d)
    bad = dict(d)
    bad["xz"] = d["xz"].clone()
    bad["xz"][10, 5] = float("nan")
    bad["xz"][40, 7] = float("inf")
    bad["xz"][59, 48 + 9] = float("nan")  # the gate of the last token
    y2, hT2 = scan(kda, bad)
    same = torch.ones(60, 48, dtype=torch.bool)
    same[10:30, 5] = same[40:, 7] = same[59, 9] = False
    assert torch.equal(y.cpu()[same], y2.cpu()[same])
    assert torch.isnan(y2[10:30, 5]).all() and torch.isnan(y2[59, 9])
    keep = torch.ones(2, 48, dtype=torch.bool)
    keep[0, 5] = keep[1, 7] = False
    assert torch.equal(hT.cpu()[keep], hT2.cpu()[keep])
    bad = dict(d, dt=d["dt"].clone())  # steps that are not numbers, or endless
    bad["dt"][13, 3], bad["dt"][37, 4] = float("nan"), float("inf")
    y3, hT3 = scan(kda, bad)
    same = torch.ones(60, 48, dtype=torch.bool)
    same[13:30, 3] = same[37:, 4] = False
    assert torch.equal(y.cpu()[same], y3.cpu()[same]) and torch.isnan(y3[13:30, 3]).all()
    keep = torch.ones(2, 48, dtype=torch.bool)
    keep[0, 3] = keep[1, 4] = False
    assert torch.equal(hT.cpu()[keep], hT3.cpu()[keep])


def test_growing_states(kda):
    """A above 0: the same bounds hold, the weights of old terms above 1."""
    d = make([90, 33], 24, 16, 1, torch.float32, seed=22)
    d["A"] = d["A"].abs() * 0.05
    y, hT = scan(kda, d)
    check(y, hT, d)


def test_malformed_offsets_are_reported_and_stay_inside(kda):
    d = make([40, 30, 30], 40, 16, 1, torch.float32, seed=17)
    g = on_gpu(d)
    for cu in ([0, 60, 40, 100], [5, 60, 100, 100], [0, 60, 90, 99], [0, -7, 300, 100],
               [0, 100, 100, 2 ** 31 - 1], [-2 ** 31, 3, 2, 1], [90, 1, 0, 100]):
        buf = torch.full((164, 40), 7.0, device="cuda")
        kept = torch.full((5, 40, 16), 7.0, device="cuda")
        kda.selective_scan_fwd(g["x"], g["dt"], g["A"], g["B"], g["C"], g["h0"],
                               torch.tensor(cu, dtype=torch.int32, device="cuda"), D=g["D"],
                               z=g["z"], dt_bias=g["bias"], out=buf[32:132],
                               final_state_out=kept[1:4])
        with pytest.raises(kda.KdaError):
            kda.get_device_error()
        assert torch.all(buf[:32] == 7) and torch.all(buf[132:] == 7)
        assert torch.all(kept[0] == 7) and torch.all(kept[4] == 7)
    kda.get_device_error()


@pytest.mark.parametrize("dtype", DT, ids=IDS)
@pytest.mark.parametrize("S", [8, 16, 32])
@pytest.mark.parametrize("N,ch,G", [(1, 8, 1), (5, 24, 1), (33, 48, 2), (3, 2048, 1)])
def test_one_token(kda, dtype, S, N, ch, G):
    d = make([1] * N, ch, S, G, dtype, seed=N + S)
    g = on_gpu(d)
    h = g["h0"].clone()
    y = kda.selective_step(g["x"], g["dt"], g["A"], g["B"], g["C"], h, D=g["D"], z=g["z"],
                           dt_bias=g["bias"])
    check(y, h, d)
    h = g["h0"].clone()
    d["z"] = d["D"] = d["bias"] = None
    y = kda.selective_step(g["x"], g["dt"], g["A"], g["B"], g["C"], h)
    check(y, h, d)


@pytest.mark.parametrize("dtype", DT, ids=IDS)
@pytest.mark.parametrize("S", [8, 16, 32])
@pytest.mark.parametrize("T", [1, 2, 5, 16])
def test_drafted_tokens(kda, dtype, S, T):
    N = 7
    d = make([T] * N, 40, S, 1, dtype, seed=10 * T + S)
    adv = torch.tensor([0, T, 1, T // 2, T - 1, -3, 99], dtype=torch.int32)
    g = on_gpu(d)
    v = lambda t: t.unflatten(0, (N, T))  # noqa: E731
    tok = [v(g["x"]), v(g["dt"]), g["A"], v(g["B"]), v(g["C"])]
    more = dict(D=g["D"], z=v(g["z"]), dt_bias=g["bias"])
    h = g["h0"].clone()
    y = kda.selective_multi_step(*tok, h, adv.cuda(), **more)
    check(y, h, d, n_advance=adv)
    assert torch.equal(h[0], g["h0"][0]) and torch.equal(h[5], g["h0"][5])
    h2 = g["h0"].clone()
    assert kda.selective_multi_step(*tok, h2, adv.cuda(), return_outputs=False, **more) is None
    assert torch.equal(h, h2)
    h3 = g["h0"].clone()
    y3 = kda.selective_multi_step(*tok, h3, **more)
    assert torch.equal(y3, y)
    check(None, h3, d)


def test_offsets_past_32_bits(kda):
    """Rows behind element 2^31, and states behind it: the last ones against a short call."""
    ch, nt = 8192, 2 ** 18 + 64
    gen = torch.Generator(device="cuda").manual_seed(1)
    r = lambda *s: torch.randn(*s, generator=gen, device="cuda")  # noqa: E731
    x = torch.randn(nt, ch, generator=gen, device="cuda", dtype=torch.bfloat16)
    B, C = r(nt, 1, 8).bfloat16(), r(nt, 1, 8).bfloat16()
    A = -torch.ones(ch, 8, device="cuda")
    cu = torch.tensor([0, nt - 64, nt], dtype=torch.int32, device="cuda")
    y, hT = kda.selective_scan_fwd(x, x, A, B, C, cu_seqlens=cu)
    tail = [t[-64:].clone().unsqueeze(0) for t in (x, B, C)]
    y2, h2 = kda.selective_scan_fwd(tail[0], tail[0], A, tail[1], tail[2])
    assert torch.equal(y[-64:], y2[0]) and torch.equal(hT[1], h2[0])
    del x, y
    N = 2 ** 14 + 3  # x 8192 x 16 states
    h = torch.zeros(N, ch, 16, device="cuda")
    h[-3:] = r(3, ch, 16)
    want = h[-3:].clone()
    x = r(N, ch).bfloat16()
    B, C = r(N, 1, 16).bfloat16(), r(N, 1, 16).bfloat16()
    A = -torch.ones(ch, 16, device="cuda")
    y = kda.selective_step(x, x, A, B, C, h)
    y2 = kda.selective_step(x[-3:], x[-3:], A, B[-3:], C[-3:], want)
    assert torch.equal(y[-3:], y2) and torch.equal(h[-3:], want)


def test_captured_and_on_another_stream(kda):
    d = make([70, 9], 40, 16, 1, torch.bfloat16, seed=18)
    g = on_gpu(d)
    args = (g["x"], g["dt"], g["A"], g["B"], g["C"], g["h0"], g["cu"])
    more = dict(D=g["D"], z=g["z"], dt_bias=g["bias"])
    y0, h0 = kda.selective_scan_fwd(*args, **more)
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    step = (g["x"][:2], g["dt"][:2], g["A"], g["B"][:2], g["C"][:2])
    with torch.cuda.stream(st):
        y1, h1 = kda.selective_scan_fwd(*args, **more)
        with torch.cuda.graph(graph, stream=st):
            y2, h2 = kda.selective_scan_fwd(*args, **more)
            y3 = kda.selective_step(*step, h2)
    torch.cuda.current_stream().wait_stream(st)
    for _ in range(2):
        graph.replay()
    ref = h0.clone()
    y4 = kda.selective_step(*step, ref)
    torch.cuda.synchronize()
    assert torch.equal(y0, y1) and torch.equal(y0, y2) and torch.equal(h0, h1)
    assert torch.equal(h2, ref) and torch.equal(y3, y4)


def test_binding_checks(kda):
    z = lambda *s: torch.zeros(*s, device="cuda")  # noqa: E731
    x, A, b, h = z(6, 16), z(16, 8), z(6, 1, 8), z(6, 16, 8)
    for call in (lambda: kda.selective_step(x, x[:, :8], A, b, b, h),
                 lambda: kda.selective_step(x, x[:5], A, b, b, h),
                 lambda: kda.selective_step(x, x.bfloat16(), A, b, b, h),
                 lambda: kda.selective_step(x, x, A[:8], b, b, h),
                 lambda: kda.selective_step(x, x, A.bfloat16(), b, b, h),
                 lambda: kda.selective_step(x, x, A, b[:, 0], b, h),
                 lambda: kda.selective_step(x, x, A, b, b[:5], h),
                 lambda: kda.selective_step(x, x, A, b, b, h[:5]),
                 lambda: kda.selective_step(x, x, A, b, b, None),
                 lambda: kda.selective_step(x, x, A, b, b, h.bfloat16()),
                 lambda: kda.selective_step(x, x, A, b, b, h, z=x[:, :8]),
                 lambda: kda.selective_step(x, x, A, b, b, h, D=z(8)),
                 lambda: kda.selective_step(x, x, A, b, b, h, dt_bias=z(17)),
                 lambda: kda.selective_step(x, x, A, b, b, h, out=z(6, 8)),
                 lambda: kda.selective_step(x, x.cpu(), A, b, b, h),
                 lambda: kda.selective_scan_fwd(x, x, A, b, b),
                 lambda: kda.selective_scan_fwd(x.unsqueeze(0), x.unsqueeze(0), A, b.unsqueeze(0),
                                                b.unsqueeze(0), h),
                 lambda: kda.selective_multi_step(x, x, A, b, b, h)):
        with pytest.raises((ValueError, TypeError)):
            call()
    with pytest.raises(kda.KdaError):
        kda.selective_step(x, x, z(16, 24), z(6, 1, 24), z(6, 1, 24), z(6, 16, 24))
    with pytest.raises(kda.KdaError):  # broadcast rows
        kda.selective_step(x[:1].expand(6, 16), x, A, b, b, h)
