"""The causal convolution on prompts large enough for runs of 32 and 64 tokens, with sequences that
begin at and beside the borders of the runs, without tokens and of one to three, and with kept inputs
read and written in place.  Bounds as in the other tests of the convolution."""

import numpy as np
import pytest
import torch

from tests.gpu_helpers import to64
from tests.test_gpu_conv import DT, IDS, check_y, cuda, make

pytestmark = pytest.mark.gpu

C = 4096


@pytest.fixture(scope="module")
def kda():
    import chunked_gated_delta_fwd_gb300 as m

    return m


def lengths(run, most):
    """Sequences that begin run - 3 .. run + 3 and 2 run - 1 .. 2 run + 3 tokens behind a border of
    the runs, short and empty ones among them, `most` tokens in all."""
    lens, at = [], 0

    def begin(t):  # the next sequence begins at token t
        nonlocal at
        lens.append(t - at)
        at = t

    base = 0
    for off in list(range(run - 3, run + 4)) + list(range(2 * run - 1, 2 * run + 4)):
        begin(base + off)
        base += 3 * run
    for short in (0, 1, 0, 2, 3, 0, 0, 1, 1, 2, 3, 3):
        begin(at + short)
    begin(base)              # at a border, then one to three tokens before and behind it
    for n in (1, 2, 3):
        begin(base + n * 2 * run - n)
        begin(base + n * 2 * run)
        begin(base + n * 2 * run + n)
    begin(most)
    return lens + [0]


@pytest.mark.parametrize("dtype", DT, ids=IDS)
@pytest.mark.parametrize("W,run,most", [(2, 64, 4900), (3, 64, 5001), (4, 64, 5107), (4, 32, 2600)])
def test_borders_of_long_runs(kda, dtype, W, run, most):
    d = make(lengths(run, most), C, W, dtype, seed=most)
    s = cuda(d["s"])
    x, w, b, cu = (cuda(d[k]) for k in ("x", "w", "b", "cu"))
    y, last = kda.causal_conv_fwd(x, w, b, s, cu, final_state_out=s)
    assert last.data_ptr() == s.data_ptr()
    assert np.array_equal(to64(last), check_y(y, d, True))
    y2, last2 = kda.causal_conv_fwd(x, w, b, cuda(d["s"]), cu)
    assert torch.equal(y, y2) and torch.equal(last, last2)
    kda.get_device_error()
