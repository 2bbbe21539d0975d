"""GPU parity of the short causal convolution against the fp64 oracle.

Bounds, elementwise, u = 2^-24, M = |bias| + sum |w| |x| of a result: a sum of W + 1 <= 5 terms in
fp32 is within 6 u M.  SiLU passes an error on with a factor of at most 1.1 and adds its own: the
exponent's argument is off by 2 |y| u, the exponential by 4 u, the sum and the quotient by 4 u, so
(8 + 2 |y|) u of itself; below |y| = 88 nothing is smaller than 1e-36.  bf16 rounds once: 2^-8 of the
result.  Kept inputs are copies and have to be equal.
"""

import numpy as np
import pytest
import torch

import oracle
from tests.gpu_helpers import to64

pytestmark = pytest.mark.gpu

DT = [torch.bfloat16, torch.float32]
IDS = ["bf16", "f32"]
U = 2.0 ** -24


@pytest.fixture(scope="module")
def kda():
    import chunked_gated_delta_fwd_gb300 as m

    return m


def make(lens, C, W, dtype, seed, bias=True, state=True, extra=0):
    gen = torch.Generator().manual_seed(seed)
    nt = sum(lens)
    full = torch.randn(nt, C + 2 * extra, generator=gen).to(dtype)
    d = dict(x=full[:, extra:extra + C], full=full, extra=extra,
             w=torch.randn(C, W, generator=gen),
             b=torch.randn(C, generator=gen) if bias else None,
             s=torch.randn(len(lens), W - 1, C, generator=gen).to(dtype) if state else None)
    d["cu"] = torch.tensor([0] + list(np.cumsum(lens)), dtype=torch.int32)
    return d


def cuda(t):
    return None if t is None else t.cuda()


def check_y(y, d, silu, n_advance=None):
    """y against the oracle; returns the oracle's kept inputs."""
    ref, last = oracle.causal_conv(d["x"].float(), d["w"], d["b"], None if d["s"] is None else
                                   d["s"].float(), d["cu"], silu, n_advance)
    a = lambda t: None if t is None else np.abs(to64(t))  # noqa: E731
    M, _ = oracle.causal_conv(a(d["x"]), a(d["w"]), a(d["b"]), a(d["s"]), d["cu"], False)
    bound = 6 * U * M
    if silu:
        bound = 1.1 * bound + (8 + 2 * M) * U * np.abs(ref)
    if d["x"].dtype == torch.bfloat16:
        bound = bound * (1 + 2.0 ** -8) + 2.0 ** -8 * np.abs(ref)
    err = np.abs(to64(y).reshape(ref.shape) - ref)
    assert np.all(err <= bound + 1e-30), float(np.max(err / (bound + 1e-30)))
    return last


@pytest.mark.parametrize("dtype", DT, ids=IDS)
@pytest.mark.parametrize("W", [2, 3, 4])
@pytest.mark.parametrize("lens", [[1], [2], [3], [16], [17], [40], [0, 1, 0, 2, 3, 0], [15, 1, 18, 2],
                                  [1] * 40, [13, 3, 2, 1, 14, 200], [0, 0]])
def test_prompts(kda, dtype, W, lens):
    d = make(lens, 24, W, dtype, seed=sum(lens) + W)
    y, last = kda.causal_conv_fwd(cuda(d["x"]), cuda(d["w"]), cuda(d["b"]), cuda(d["s"]),
                                  cuda(d["cu"]))
    assert np.array_equal(to64(last), check_y(y, d, True))
    kda.get_device_error()


@pytest.mark.parametrize("dtype", DT, ids=IDS)
@pytest.mark.parametrize("C", [8, 16, 72, 1000, 2056])
def test_channels_no_state_no_bias(kda, dtype, C):
    d = make([70, 1, 35], C, 4, dtype, seed=C, bias=False, state=False)
    y, last = kda.causal_conv_fwd(cuda(d["x"]), cuda(d["w"]), None, None, cuda(d["cu"]), silu=False)
    assert np.array_equal(to64(last), check_y(y, d, False))


@pytest.mark.parametrize("dtype", DT, ids=IDS)
def test_slices_batches_and_no_final_state(kda, dtype):
    d = make([50, 50, 50], 40, 3, dtype, seed=3, extra=16)
    full = cuda(d["full"])
    x = full[:, 16:56].view(3, 50, 40)
    out = torch.full((150, 64), 7.0, dtype=dtype, device="cuda")
    y, last = kda.causal_conv_fwd(x, cuda(d["w"]), cuda(d["b"]), cuda(d["s"]), out=out[:, 8:48].view(3, 50, 40),
                                  output_final_state=False)
    assert last is None and y.data_ptr() == out[:, 8:48].data_ptr()
    check_y(y, d, True)
    assert torch.all(out[:, :8] == 7) and torch.all(out[:, 48:] == 7)


@pytest.mark.parametrize("dtype", DT, ids=IDS)
@pytest.mark.parametrize("lens", [[16, 16, 16], [15, 17, 1, 2, 33, 0, 14, 16], [1] * 33, [5000]])
def test_state_in_place(kda, dtype, lens):
    """Many channels and starts next to the borders of the runs: what one thread overwrites no
    other one still reads."""
    d = make(lens, 1024, 4, dtype, seed=11)
    s = cuda(d["s"])
    y, last = kda.causal_conv_fwd(cuda(d["x"]), cuda(d["w"]), cuda(d["b"]), s, cuda(d["cu"]),
                                  final_state_out=s)
    assert last.data_ptr() == s.data_ptr()
    y2, last2 = kda.causal_conv_fwd(cuda(d["x"]), cuda(d["w"]), cuda(d["b"]), cuda(d["s"]),
                                    cuda(d["cu"]))
    assert torch.equal(y, y2) and torch.equal(s, last2)


def test_every_border_of_a_run(kda):
    for first in range(1, 40):
        d = make([first, 40 - first, 5], 8, 4, torch.float32, seed=first)
        y, last = kda.causal_conv_fwd(cuda(d["x"]), cuda(d["w"]), cuda(d["b"]), cuda(d["s"]),
                                      cuda(d["cu"]), silu=False)
        assert np.array_equal(to64(last), check_y(y, d, False))


@pytest.mark.parametrize("dtype", DT, ids=IDS)
@pytest.mark.parametrize("W,N,C,silu", [(4, 1, 8, True), (2, 5, 136, False), (3, 33, 64, True)])
def test_one_token(kda, dtype, W, N, C, silu):
    d = make([1] * N, C, W, dtype, seed=N)
    s = cuda(d["s"])
    y = kda.causal_conv_step(cuda(d["x"]), cuda(d["w"]), s, cuda(d["b"]), silu=silu)
    assert np.array_equal(to64(s), check_y(y, d, silu))


@pytest.mark.parametrize("dtype", DT, ids=IDS)
@pytest.mark.parametrize("W", [2, 3, 4])
@pytest.mark.parametrize("T", [1, 2, 4, 5, 16])
def test_drafted_tokens(kda, dtype, W, T):
    N, C = 7, 48
    d = make([T] * N, C, W, dtype, seed=10 * T + W, extra=8)
    adv = torch.tensor([0, T, 1, T // 2, T - 1, -3, 99], dtype=torch.int32)
    x = cuda(d["full"])[:, 8:8 + C].view(N, T, C)
    s = cuda(d["s"])
    y = kda.causal_conv_multi_step(x, cuda(d["w"]), s, cuda(adv), cuda(d["b"]))
    assert np.array_equal(to64(s), check_y(y, d, True, adv))
    s2 = cuda(d["s"])  # the state alone, and all T
    assert kda.causal_conv_multi_step(x, cuda(d["w"]), s2, cuda(adv), return_outputs=False) is None
    assert torch.equal(s, s2)
    s3 = cuda(d["s"])
    kda.causal_conv_multi_step(x, cuda(d["w"]), s3)
    assert np.array_equal(to64(s3), oracle.causal_conv(d["x"].float(), d["w"], None, d["s"].float(),
                                                       d["cu"])[1])


def test_non_finite_inputs_reach_their_own_channels_and_tokens(kda):
    d = make([20, 20], 16, 4, torch.float32, seed=5)
    clean, _ = kda.causal_conv_fwd(cuda(d["x"]), cuda(d["w"]), cuda(d["b"]), None, cuda(d["cu"]))
    x = d["x"].clone()
    x[18, 3], x[19, 4] = float("nan"), float("inf")
    y, last = kda.causal_conv_fwd(cuda(x), cuda(d["w"]), cuda(d["b"]), None, cuda(d["cu"]))
    same = torch.ones(40, 16, dtype=torch.bool)
    same[18:20, 3] = same[19, 4] = False
    assert torch.equal(y.cpu()[same], clean.cpu()[same])
    assert torch.isnan(y[18:20, 3]).all() and torch.isnan(last[0, 1, 3])
    big = torch.full((1, 8), 1e30, device="cuda")
    taps = torch.tensor([[0.0, 1.0]] * 4 + [[0.0, -1.0]] * 4, device="cuda")
    y = kda.causal_conv_step(big, taps, torch.zeros(1, 1, 8, device="cuda"))
    assert torch.all(y[0, :4] == 1e30) and torch.all(y[0, 4:] == 0)  # SiLU at both ends


def test_malformed_offsets_are_reported_and_stay_inside(kda):
    C, nt = 64, 100
    for cu in ([0, 60, 40, 100], [5, 60, 100, 100], [0, 60, 90, 99], [0, -7, 300, 100],
               [0, 100, 100, 2 ** 31 - 1], [-2 ** 31, 3, 2, 1], [90, 1, 0, 100]):
        buf = torch.full((nt + 64, C), 7.0, device="cuda")
        kept = torch.full((3 + 2, 3, C), 7.0, device="cuda")
        x = torch.randn(nt, C, device="cuda")
        kda.causal_conv_fwd(x, torch.randn(C, 4, device="cuda"), None, None,
                            torch.tensor(cu, dtype=torch.int32, device="cuda"), out=buf[32:32 + nt],
                            final_state_out=kept[1:4])
        with pytest.raises(kda.KdaError):
            kda.get_device_error()
        assert torch.all(buf[:32] == 7) and torch.all(buf[32 + nt:] == 7)
        assert torch.all(kept[0] == 7) and torch.all(kept[4] == 7)
    kda.get_device_error()


def test_offsets_past_32_bits(kda):
    C, nt = 8192, 2 ** 18 + 100  # the last rows begin behind element 2^31
    x = torch.randn(nt, C, device="cuda", dtype=torch.bfloat16)
    w = torch.randn(C, 4, device="cuda")
    y, last = kda.causal_conv_fwd(x.unsqueeze(0), w, silu=False)
    part, last2 = kda.causal_conv_fwd(x[-40:].clone().unsqueeze(0), w, silu=False)
    assert torch.equal(y[0, -30:], part[0, -30:]) and torch.equal(last, last2)
    del x, y


def test_captured_and_on_another_stream(kda):
    d = make([30, 9], 256, 4, torch.bfloat16, seed=2)
    x, w, b, s, cu = (cuda(d[k]) for k in ("x", "w", "b", "s", "cu"))
    y0, last0 = kda.causal_conv_fwd(x, w, b, s, cu)
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.stream(st):
        y1, last1 = kda.causal_conv_fwd(x, w, b, s, cu)
        with torch.cuda.graph(graph, stream=st):
            y2, last2 = kda.causal_conv_fwd(x, w, b, s, cu)
            y3 = kda.causal_conv_step(x[:2], w, last2, b)
    torch.cuda.current_stream().wait_stream(st)
    for _ in range(2):
        graph.replay()
    ref = last0.clone()
    y4 = kda.causal_conv_step(x[:2], w, ref, b)
    torch.cuda.synchronize()
    assert torch.equal(y0, y1) and torch.equal(y0, y2) and torch.equal(last0, last1)
    assert torch.equal(last2, ref) and torch.equal(y3, y4)


def test_binding_checks(kda):
    x, w = torch.zeros(6, 16, device="cuda"), torch.zeros(16, 4, device="cuda")
    s = torch.zeros(6, 3, 16, device="cuda")
    for call in (lambda: kda.causal_conv_step(x, w[:8], s),
                 lambda: kda.causal_conv_step(x, w.double(), s),
                 lambda: kda.causal_conv_step(x, w, s[:5]),
                 lambda: kda.causal_conv_step(x, w, s.bfloat16()),
                 lambda: kda.causal_conv_step(x, w, s, torch.zeros(8, device="cuda")),
                 lambda: kda.causal_conv_step(x, w, s, out=torch.zeros(5, 16, device="cuda")),
                 lambda: kda.causal_conv_step(x.half(), w, s.half()),
                 lambda: kda.causal_conv_step(x.t(), w, s),
                 lambda: kda.causal_conv_step(x[:, ::2], w[:8], s),
                 lambda: kda.causal_conv_step(x.unsqueeze(0), w, s),
                 lambda: kda.causal_conv_fwd(x, w),
                 lambda: kda.causal_conv_fwd(x, w, cu_seqlens=torch.zeros(2, device="cuda")),
                 lambda: kda.causal_conv_fwd(x.unsqueeze(0), w, state=s),
                 lambda: kda.causal_conv_multi_step(x.view(2, 3, 16), w, s[:2],
                                                    torch.zeros(3, dtype=torch.int32, device="cuda"))):
        with pytest.raises((ValueError, TypeError)):
            call()
    with pytest.raises(kda.KdaError):  # broadcast rows
        kda.causal_conv_step(x[:1].expand(6, 16), w, s)
    with pytest.raises(kda.KdaError):
        kda.causal_conv_step(torch.zeros(6, 20, device="cuda")[:, 1:17], w, s)
