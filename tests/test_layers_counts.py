"""Counts of the convolution, the scan and the verification that no kernel's 32-bit indices hold are
refused on the host."""

import pytest
import torch

import __graft_entry__

FAKE = 0x10000  # 16-byte aligned, never dereferenced: nothing here reaches a device
MOST = 1 << 30


@pytest.fixture(scope="module")
def kda():
    __graft_entry__._build_module().build()
    import chunked_gated_delta_fwd_gb300 as m

    return m


def _conv(L, cu=None, n_seqs=0, B=1, T=64, last=FAKE):
    return L.kda_causal_conv_fwd(FAKE, 1, FAKE, None, None, cu, n_seqs, B, T, 64, 4, 64, FAKE, 64, last,
                                 None, 1)


@pytest.mark.parametrize("n", [MOST + 1, 2 ** 31 - 1])
def test_conv_sequences_past_the_search(kda, n):
    """n_seqs beyond 2^30: the middle of two indices would pass 2^31."""
    assert _conv(kda.lib, cu=FAKE, n_seqs=n) == 1
    assert b"sequences" in kda.lib.kda_last_error_string()
    assert _conv(kda.lib, B=n, T=0) == 1   # the walk over sequences without tokens
    assert b"sequences" in kda.lib.kda_last_error_string()


@pytest.mark.skipif(torch.cuda.is_available(), reason="pointers are made up: only without a device")
def test_conv_counts_up_to_the_limit_pass_the_checks(kda):
    for kw in (dict(cu=FAKE, n_seqs=MOST), dict(B=MOST, T=0), dict(B=MOST + 1, T=1)):
        assert _conv(kda.lib, **kw) in (6, 8)
