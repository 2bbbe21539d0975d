"""GPU parity of the per-head norm with rotation against the fp64 oracle.

Bound, elementwise.  With u = 2^-24 and r the length of the rotated pair (its value before
the rotation, so |y| <= r): the sum of squares is 8 products and 4 + 7 additions deep (its
relative error halves under the root), rsqrtf 2 u, the two products 2 u, sine and cosine 2 ulp
of a turn fraction rounded to fp32 (pi u as an angle), two products and a sum: below 32 u r.
bf16 adds half a step of the value, 2^-8 |y|.
"""

import numpy as np
import pytest
import torch

import oracle
from tests.gpu_helpers import to64

pytestmark = pytest.mark.gpu

DT = [torch.bfloat16, torch.float32]
IDS = ["bf16", "f32"]


@pytest.fixture(scope="module")
def kda():
    import chunked_gated_delta_fwd_gb300 as m

    return m


def _inv_freq(F):
    return (10000.0 ** (-torch.arange(F, dtype=torch.float64) / F)).float()


def _check(got, x, positions, f, w, eps, axis=None, interleaved=False):
    ref = oracle.norm_rope(x, positions, f, w, eps, axis, interleaved)
    still = oracle.norm_rope(x, positions * 0, f, w, eps, axis, interleaved)  # not turned
    F = len(f)
    r = np.abs(still)
    lo, hi = (slice(0, 2 * F, 2), slice(1, 2 * F, 2)) if interleaved else (slice(0, F),
                                                                          slice(F, 2 * F))
    r[..., lo] = r[..., hi] = np.hypot(still[..., lo], still[..., hi])
    bound = 32 * 2.0 ** -24 * r + (2.0 ** -8 * np.abs(ref) if got.dtype == torch.bfloat16 else 0.0)
    err = np.abs(to64(got) - ref)
    assert np.all(err <= bound + 1e-37), float(np.max(err / (bound + 1e-37)))


def _case(kda, nt, Hq, Hk, dtype, F=64, interleaved=False, eps=1e-6, weights=True, axes=1,
          start=0, packed=False, seed=0):
    gen = torch.Generator().manual_seed(seed)
    if packed:
        qkv = torch.randn(nt, Hq + 2 * Hk, 128, generator=gen).to(dtype)
        q, k = qkv[:, :Hq], qkv[:, Hq:Hq + Hk]
        dev = qkv.cuda()
        dq, dk = dev[:, :Hq], dev[:, Hq:Hq + Hk]
    else:
        q = torch.randn(nt, Hq, 128, generator=gen).to(dtype)
        k = torch.randn(nt, Hk, 128, generator=gen).to(dtype)
        dq, dk = q.cuda(), k.cuda()
    wq = wk = None
    if weights and eps is not None:
        wq, wk = torch.rand(128, generator=gen) + 0.5, torch.rand(128, generator=gen) + 0.5
    if axes == 1:
        pos, axis = (torch.arange(nt) + start).to(torch.int32), None
    else:
        pos = torch.randint(-50, 1 << 20, (axes, nt), generator=gen).to(torch.int32)
        axis = torch.randint(0, axes, (F,), generator=gen).to(torch.int32)
    f = _inv_freq(F)
    cu = lambda t: None if t is None else t.cuda()  # noqa: E731
    qo, ko = kda.qk_norm_rope(dq, dk, pos.cuda(), f.cuda(), q_weight=cu(wq), k_weight=cu(wk),
                              eps=eps, freq_axis=cu(axis), interleaved=interleaved)
    assert qo.shape == q.shape and ko.shape == k.shape and qo.is_contiguous()
    _check(qo, q, pos, f, wq, eps, axis, interleaved)
    _check(ko, k, pos, f, wk, eps, axis, interleaved)
    assert torch.equal(dq.cpu(), q) and torch.equal(dk.cpu(), k)  # the inputs stay as they were


@pytest.mark.parametrize("dtype", DT, ids=IDS)
@pytest.mark.parametrize("interleaved", [False, True], ids=["half", "pairs"])
@pytest.mark.parametrize("F", [8, 24, 32, 64])
def test_frequencies_and_pairings(kda, dtype, interleaved, F):
    _case(kda, 37, 3, 2, dtype, F=F, interleaved=interleaved, seed=F)


@pytest.mark.parametrize("dtype", DT, ids=IDS)
@pytest.mark.parametrize("nt,Hq,Hk,F,interleaved,packed", [
    (3701, 2, 1, 64, False, False), (3655, 1, 1, 24, True, True), (5003, 4, 2, 32, True, True),
    (7301, 1, 1, 64, False, False), (1001, 8, 1, 64, False, True), (1537, 6, 3, 40, True, False),
    (1825, 24, 4, 64, False, False), (3649, 3, 3, 8, False, True)])
def test_few_heads_of_many_tokens(kda, dtype, nt, Hq, Hk, F, interleaved, packed):
    """The units that hold rows of several tokens, with token counts that end inside one."""
    _case(kda, nt, Hq, Hk, dtype, F=F, interleaved=interleaved, packed=packed, start=1000, seed=nt)


@pytest.mark.parametrize("dtype", DT, ids=IDS)
def test_any_finite_frequency(kda, dtype):
    """Frequencies below 0, above a turn a token, near 0 and 0; positions of both signs."""
    gen = torch.Generator().manual_seed(21)
    q = torch.randn(33, 2, 128, generator=gen).to(dtype)
    k = torch.randn(33, 1, 128, generator=gen).to(dtype)
    f = torch.tensor([-0.7, 40.5, 1e-7, 0.0, -1e-30, 6.2831855, 1e5, 1.0])
    pos = torch.randint(-100000, 100000, (33,), generator=gen).to(torch.int32)
    pos[:3] = torch.tensor([0, -(1 << 31), (1 << 31) - 1], dtype=torch.int64).to(torch.int32)
    # at 2^31 x 1e5 rad the oracle's own fp64 angle is off by 2^-6: that frequency stays small there
    f_far = f.clone()
    f_far[6] = 0.5
    for rows, freq in ((slice(0, 3), f_far), (slice(3, 33), f)):
        qo, ko = kda.qk_norm_rope(q[rows].cuda(), k[rows].cuda(), pos[rows].cuda(), freq.cuda())
        _check(qo, q[rows], pos[rows], freq, None, 1e-6, None, False)
        _check(ko, k[rows], pos[rows], freq, None, 1e-6, None, False)


@pytest.mark.parametrize("dtype", DT, ids=IDS)
def test_a_frequency_that_is_not_finite_shows(kda, dtype):
    q = torch.ones(5, 1, 128, dtype=dtype, device="cuda")
    f = torch.ones(8, device="cuda")
    f[3] = float("nan")
    f[5] = float("inf")
    qo, _ = kda.qk_norm_rope(q, q.clone(), torch.arange(5, dtype=torch.int32, device="cuda"), f)
    bad = torch.isnan(qo).any(0).any(0).cpu()
    assert bad.nonzero().flatten().tolist() == [3, 5, 11, 13]


@pytest.mark.parametrize("nt,Hq,Hk", [(1, 1, 1), (1, 96, 96), (17, 2, 1), (5, 33, 11), (3, 64, 1)])
@pytest.mark.parametrize("dtype", DT, ids=IDS)
def test_token_and_head_counts(kda, nt, Hq, Hk, dtype):
    _case(kda, nt, Hq, Hk, dtype, seed=nt + Hq)


@pytest.mark.parametrize("dtype", DT, ids=IDS)
@pytest.mark.parametrize("axes,start", [(1, (1 << 31) - 41), (3, 0)], ids=["far", "axes"])
def test_far_positions_and_axes(kda, dtype, axes, start):
    _case(kda, 40, 4, 2, dtype, F=48, axes=axes, start=start, seed=7)


@pytest.mark.parametrize("dtype", DT, ids=IDS)
@pytest.mark.parametrize("eps,weights", [(None, False), (1e-6, False), (0.0, True), (0.5, True)])
def test_norm_settings(kda, dtype, eps, weights):
    _case(kda, 11, 2, 2, dtype, eps=eps, weights=weights, seed=3)


@pytest.mark.parametrize("dtype", DT, ids=IDS)
def test_slices_of_a_packed_projection(kda, dtype):
    _case(kda, 70, 8, 2, dtype, F=32, packed=True, interleaved=True, seed=9)


def test_in_place_on_a_packed_projection(kda):
    gen = torch.Generator().manual_seed(1)
    qkv = torch.randn(2, 19, 10, 128, generator=gen).bfloat16().cuda()  # [B, T, heads, 128]
    before = qkv.clone()
    q, k = qkv[:, :, :6], qkv[:, :, 6:8]
    pos = torch.arange(19, dtype=torch.int32, device="cuda").repeat(2, 1)
    f = _inv_freq(64).cuda()
    ref = kda.qk_norm_rope(before[:, :, :6], before[:, :, 6:8], pos, f)
    kda.qk_norm_rope(q, k, pos, f, q_out=q, k_out=k)
    assert torch.equal(q, ref[0]) and torch.equal(k, ref[1])
    assert torch.equal(qkv[:, :, 8:], before[:, :, 8:])  # the rest of the rows is not touched


def test_zero_rows_large_values_and_non_finite_rows(kda):
    x = torch.randn(6, 2, 128, generator=torch.Generator().manual_seed(2))
    x[1] = 0.0
    x[2] *= 1e15          # squares near 1e30 still sum in fp32
    x[4, 1, 5] = float("inf")
    x[5, 0, 7] = float("nan")
    pos = torch.arange(6, dtype=torch.int32)
    f = _inv_freq(64)
    y, _ = kda.qk_norm_rope(x.cuda(), x.cuda(), pos.cuda(), f.cuda())
    clean = [(t, h) for t in range(6) for h in range(2) if (t, h) not in ((4, 1), (5, 0))]
    for t, h in clean:  # a non-finite row stays by itself
        _check(y[t:t + 1, h:h + 1], x[t:t + 1, h:h + 1], pos[t:t + 1], f, None, 1e-6)
    assert not torch.isfinite(y[5, 0]).any()


def test_no_tokens_and_axis_out_of_range(kda):
    e = torch.zeros(0, 2, 128, device="cuda")
    f = _inv_freq(8).cuda()
    q, k = kda.qk_norm_rope(e, e, torch.zeros(0, dtype=torch.int32, device="cuda"), f)
    assert q.shape == (0, 2, 128) and k.shape == (0, 2, 128)
    kda.get_device_error()
    x = torch.randn(3, 2, 128, device="cuda")
    pos = torch.zeros(2, 3, dtype=torch.int32, device="cuda")
    axis = torch.tensor([0, 1, 0, 2, 0, 0, -1, 0], dtype=torch.int32, device="cuda")
    kda.qk_norm_rope(x, x, pos, f, freq_axis=axis)
    with pytest.raises(kda.KdaError, match="freq_axis"):
        kda.get_device_error()
    kda.get_device_error()


def test_refusals(kda):
    x = torch.randn(3, 2, 128, device="cuda")
    pos, f = torch.zeros(3, dtype=torch.int32, device="cuda"), _inv_freq(64).cuda()
    bad = [
        dict(q=x.half(), k=x.half()), dict(k=x.bfloat16()), dict(k=x[:2]), dict(pos=pos[:2]),
        dict(pos=pos.long()), dict(f=f.double()), dict(q=x[..., ::2], k=x[..., ::2]),
        dict(q=x.transpose(0, 1), k=x.transpose(0, 1)), dict(f=f[:12].contiguous()),
        dict(q_weight=torch.ones(64, device="cuda")), dict(pos=torch.stack([pos, pos])),
        dict(eps=None, q_weight=torch.ones(128, device="cuda")), dict(q_out=x[:2]),
        dict(freq_axis=torch.zeros(3, dtype=torch.int32, device="cuda")),
        dict(q=x[:, :, :64].contiguous(), k=x[:, :, :64].contiguous()),
        dict(q=x[:1].expand(3, 2, 128)),
    ]
    for b in bad:
        a = dict(q=x, k=x, pos=pos, f=f)
        a.update(b)
        args = [a.pop(n) for n in ("q", "k", "pos", "f")]
        with pytest.raises((TypeError, ValueError, kda.KdaError)):
            kda.qk_norm_rope(*args, **a)


def test_captured_and_replayed_on_another_stream(kda):
    f = _inv_freq(64).cuda()
    q, k = torch.randn(9, 4, 128, device="cuda"), torch.randn(9, 2, 128, device="cuda")
    pos = torch.arange(9, dtype=torch.int32, device="cuda")
    qo, ko = torch.empty_like(q), torch.empty_like(k)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        kda.qk_norm_rope(q, k, pos, f, q_out=qo, k_out=ko)
    s.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        kda.qk_norm_rope(q, k, pos, f, q_out=qo, k_out=ko)
    q.copy_(torch.randn_like(q))
    pos += 100
    graph.replay()
    rq, rk = kda.qk_norm_rope(q, k, pos, f)
    assert torch.equal(qo, rq) and torch.equal(ko, rk)


@pytest.mark.parametrize("Hq,Hk,nt", [(4, 2, 600), (2, 1, 4000)])
def test_offsets_past_32_bits(kda, Hq, Hk, nt):
    """Tokens far apart in one large buffer, in place, against the same rows side by side."""
    step = -(-(2 ** 31 + 2 ** 28) // nt // 8) * 8
    base = torch.zeros(nt * step, dtype=torch.bfloat16, device="cuda")
    assert base.numel() > 2 ** 31
    q = base.as_strided((nt, Hq, 128), (step, 128, 1))
    k = base.as_strided((nt, Hk, 128), (step, 128, 1), Hq * 128)
    gen = torch.Generator(device="cuda").manual_seed(nt)
    q.copy_(torch.randn(nt, Hq, 128, generator=gen, device="cuda"))
    k.copy_(torch.randn(nt, Hk, 128, generator=gen, device="cuda"))
    pos, f = torch.arange(nt, dtype=torch.int32, device="cuda"), _inv_freq(64).cuda()
    rq, rk = kda.qk_norm_rope(q.contiguous(), k.contiguous(), pos, f)
    kda.qk_norm_rope(q, k, pos, f, q_out=q, k_out=k)
    assert torch.equal(q, rq) and torch.equal(k, rk)
    assert not base[-(step - (Hq + Hk) * 128):].any()  # behind the last row
    del base, q, k
    torch.cuda.empty_cache()
