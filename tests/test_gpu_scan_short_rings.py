"""The selective scan on batches of many (sequence, channels) of a few hundred tokens, which rings of
four warps take: up to 63 tiles, so that a warp takes many in turn and copies two ahead, with lengths
at and beside whole tiles and rounds.  Bounds as in the other tests of the scan."""

import pytest
import torch

from tests.test_gpu_scan import DT, IDS, check, make, on_gpu, scan

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def kda():
    import chunked_gated_delta_fwd_gb300 as m

    return m


def lengths(seed):
    """40 lengths of 0 to 500 tokens; among them 9 to 60 tiles of 8, rounds of four tiles (32 tokens)
    and one token more or less."""
    gen = torch.Generator().manual_seed(seed)
    fixed = [0, 1, 31, 32, 33, 63, 64, 65, 72, 95, 96, 97, 128, 479, 480, 481, 500]
    rest = torch.randint(66, 480, (40 - len(fixed),), generator=gen).tolist()
    lens = fixed + rest
    return [lens[i] for i in torch.randperm(40, generator=gen).tolist()]


@pytest.mark.parametrize("dtype", DT, ids=IDS)
@pytest.mark.parametrize("S,G", [(8, 1), (16, 2), (32, 1)])
def test_ragged_batches(kda, dtype, S, G):
    """From kept states, in place, and twice the same bits."""
    d = make(lengths(S), 256, S, G, dtype, seed=S, strong=0.05)
    y, hT = scan(kda, d)
    check(y, hT, d)
    g = on_gpu(d)
    h = g["h0"].clone()
    y2, _ = kda.selective_scan_fwd(g["x"], g["dt"], g["A"], g["B"], g["C"], h, g["cu"], D=g["D"],
                                   z=g["z"], dt_bias=g["bias"], final_state_out=h)
    assert torch.equal(y, y2) and torch.equal(h, hT)
    kda.get_device_error()


@pytest.mark.parametrize("dtype", DT, ids=IDS)
def test_the_same_bits_as_a_sequence_alone(kda, dtype):
    """Alone, its channels do not fill the SMs and take rings of twelve: the same tiles."""
    d = make(lengths(1), 256, 16, 1, dtype, seed=1)
    y, hT = scan(kda, d)
    g = on_gpu(d)
    cu = d["cu"].tolist()
    for n in range(0, 40, 3):
        b, e = cu[n], cu[n + 1]
        row = lambda t: t[b:e].unsqueeze(0)  # noqa: E731
        y1, h1 = kda.selective_scan_fwd(row(g["x"]), row(g["dt"]), g["A"], row(g["B"]), row(g["C"]),
                                        g["h0"][n:n + 1], D=g["D"], z=row(g["z"]), dt_bias=g["bias"])
        assert torch.equal(y1[0], y[b:e]) and torch.equal(h1[0], hT[n])


def test_malformed_offsets_and_non_finite_inputs(kda):
    lens = lengths(2)
    d = make(lens, 256, 16, 1, torch.bfloat16, seed=2)
    g, nt = on_gpu(d), sum(lens)
    args = (g["x"], g["dt"], g["A"], g["B"], g["C"], g["h0"])
    more = dict(D=g["D"], z=g["z"], dt_bias=g["bias"])
    y0, h0 = scan(kda, d)
    good = d["cu"].tolist()
    for at, v in ((7, 0), (7, nt), (0, 5), (40, nt - 1), (20, -3), (20, 2 ** 31 - 1), (40, nt + 900)):
        cu = list(good)
        cu[at] = v
        buf = torch.full((nt + 64, 256), 7.0, dtype=torch.bfloat16, device="cuda")
        kept = torch.full((42, 256, 16), 7.0, device="cuda")
        kda.selective_scan_fwd(*args, torch.tensor(cu, dtype=torch.int32, device="cuda"),
                               out=buf[32:-32], final_state_out=kept[1:41], **more)
        with pytest.raises(kda.KdaError):
            kda.get_device_error()
        assert torch.all(buf[:32] == 7) and torch.all(buf[-32:] == 7)
        assert torch.all(kept[0] == 7) and torch.all(kept[41] == 7)
    long = [n for n in range(40) if lens[n] > 200][:2]
    bad = dict(d, xz=d["xz"].clone())
    same, keep = torch.ones(nt, 256, dtype=torch.bool), torch.ones(40, 256, dtype=torch.bool)
    for n, c, v in ((long[0], 5, float("nan")), (long[1], 70, float("inf"))):
        first = good[n] + 150
        bad["xz"][first, c] = v
        same[first:good[n + 1], c] = keep[n, c] = False
    y1, h1 = scan(kda, bad)
    assert torch.equal(y1.cpu()[same], y0.cpu()[same]) and torch.equal(h1.cpu()[keep], h0.cpu()[keep])
    assert not torch.isfinite(y1.cpu()[~same]).any() and not torch.isfinite(h1.cpu()[~keep]).any()
