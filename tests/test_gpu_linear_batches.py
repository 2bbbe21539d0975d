"""Linear attention on batches that meet each way of drawing the work (as they come, by ticket,
cut into segments, fp32 cores): neighbours of non-finite inputs, offsets that are malformed, and
one long prompt packed with many short ones.  What is compared with the fp32 cores is compared
within the bf16 and fp32 bounds of the other tests; neighbours are compared bit by bit."""

import numpy as np
import pytest
import torch

from tests.gpu_helpers import F32_REL_L2

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def kda():
    import chunked_gated_delta_fwd_gb300 as m

    return m


def make(lens, H, dtype, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    nt = sum(lens)
    unit = lambda x: x / x.norm(dim=-1, keepdim=True)  # noqa: E731
    r = lambda *s: torch.randn(*s, generator=gen, device="cuda")  # noqa: E731
    return dict(q=unit(r(nt, H, 128)).to(dtype), k=unit(r(nt, H, 128)).to(dtype),
                v=r(nt, H, 128).to(dtype), g=-0.1 * r(nt, H).abs(),
                h0=0.1 * r(len(lens), H, 128, 128),
                cu=torch.tensor([0] + list(np.cumsum(lens)), dtype=torch.int32, device="cuda"))


def run(kda, d, flags=0):
    return kda.linear_chunk_fwd(d["q"], d["k"], d["v"], d["g"], d["h0"], d["cu"], flags=flags)


def kernels(kda, call):
    kda.profile_enable(True)
    got = call()
    ran = set(kda.profile_collect())
    kda.profile_enable(False)
    return got, ran


WAYS = {  # way: (lengths, heads, type, flags, a kernel that shows it)
    "tickets": ([900, 700, 130, 1300, 5], 40, torch.bfloat16, "", "kda_linear_order"),
    "forced segments": ([300, 130, 400, 90], 3, torch.bfloat16, "cut", "kda_linear_tc_state"),
    "segments": ([3000, 2900, 3100], 2, torch.bfloat16, "", "kda_linear_tc_state"),
    "fp32 cores": ([130, 70, 200, 90], 3, torch.bfloat16, "fp32", "kda_linear_out"),
    "fp32": ([130, 70, 200, 90], 3, torch.float32, "", "kda_linear_out"),
}


@pytest.mark.parametrize("way", sorted(WAYS))
@pytest.mark.parametrize("which", ["q", "k", "v", "g", "h0"])
@pytest.mark.parametrize("value", [float("nan"), float("inf")], ids=["nan", "inf"])
def test_non_finite_inputs_stay_in_their_sequence_and_head(kda, way, which, value):
    lens, H, dtype, how, shows = WAYS[way]
    flags = {"cut": kda.segment_chunks(1), "fp32": kda.FP32_CORES}.get(how, 0)
    d = make(lens, H, dtype, seed=len(way))
    (o, hT), ran = kernels(kda, lambda: run(kda, d, flags))
    assert shows in ran
    bad = {n: t.clone() for n, t in d.items()}
    a, b = int(d["cu"][1]), int(d["cu"][2])
    # all of sequence 1, and head 1 of the last one
    last = int(d["cu"][-2])
    for where in ((slice(a, b), slice(None)), (slice(last, None), slice(1, 2))):
        if which == "h0":
            where = (slice(1, 2) if where[0].start == a else slice(-1, None), where[1])
        bad[which][where] = -value if which == "g" else value
    x, xT = run(kda, bad, flags)
    keep = [h for h in range(H) if h != 1]
    assert torch.equal(x[:a], o[:a]) and torch.equal(xT[0], hT[0])
    assert torch.equal(x[b:last], o[b:last]) and torch.equal(xT[2:-1], hT[2:-1])
    assert torch.equal(x[last:][:, keep], o[last:][:, keep]) and torch.equal(xT[-1, keep], hT[-1, keep])
    kda.get_device_error()


@pytest.mark.parametrize("n,H", [(8, 40), (1100, 1)])
def test_malformed_offsets_drawn_by_ticket(kda, n, H):
    """With an order (up to 1024 sequences) and without one: reported, and the next call on good
    offsets is as it was."""
    d = make([520] * n, H, torch.bfloat16, seed=n)
    good = d["cu"]
    (o, hT), ran = kernels(kda, lambda: run(kda, d))
    assert ("kda_linear_order" in ran) == (n <= 1024)
    kda.get_device_error()
    nt = int(good[-1])
    for change in ({1: nt, 2: 0, 3: nt, 4: 0}, {0: 9}, {n: nt + 7}, {n: nt - 7}, {5: -3}, {n // 2: 1 << 30}):
        d["cu"] = good.clone()
        for i, x in change.items():
            d["cu"][i] = x
        run(kda, d)
        with pytest.raises(kda.KdaError, match="cu_seqlens"):
            kda.get_device_error()
    d["cu"] = good
    x, xT = run(kda, d)
    kda.get_device_error()
    assert torch.equal(x, o) and torch.equal(xT, hT)


@pytest.mark.parametrize("long,short,H", [(9000, [1] * 4, 16), (9000, [1] * 100, 16), (20000, [1, 0, 130] * 30, 2),
                                          (9000, [600] * 12, 16)])
@pytest.mark.parametrize("at", ["first", "last"])
def test_one_long_prompt_among_short_ones(kda, long, short, H, at):
    lens = [long] + short if at == "first" else short + [long]
    d = make(lens, H, torch.bfloat16, seed=long + len(short))
    o, hT = run(kda, d)
    ro, rh = run(kda, d, kda.FP32_CORES)
    kda.get_device_error()
    for x, y, tol in ((o, ro, 2.0 ** -8), (hT, rh, F32_REL_L2)):
        assert float((x.double() - y.double()).norm() / y.double().norm()) <= tol


@pytest.mark.parametrize("flags,most", [("", 4.7e-6), ("fp32", 1e-6)])
def test_the_stated_accuracy_of_the_final_state(kda, flags, most):
    """Against 64 bits, in the 2-norm: the 16 bits of each weighted value (4.4e-6 rms over all
    values and weights, less where the last tokens weigh 1, and 2e-7 of fp32) and the fp32 sums."""
    d = make([1000, 300], 8, torch.bfloat16, seed=77)
    _, hT = run(kda, d, kda.FP32_CORES if flags else 0)
    ref = d["h0"].double()
    cu = d["cu"].tolist()
    for n in range(2):
        s = slice(cu[n], cu[n + 1])
        G = d["g"][s].double().cumsum(0)
        w = torch.exp(G[-1] - G)
        ref[n] = torch.exp(G[-1])[:, None, None] * ref[n] + torch.einsum(
            "th,thv,thk->hvk", w, d["v"][s].double(), d["k"][s].double())
    off = float((hT.double() - ref).norm() / ref.norm())
    assert off <= most, off
