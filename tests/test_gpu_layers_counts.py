"""Sizes past 2^31 of the convolution, the scan and the verification are refused by the binding: as
32-bit arguments they would be cut off to small ones.  The tensors hold little or no memory."""

import pytest
import torch

pytestmark = pytest.mark.gpu

PAST = 2 ** 32 + 8


@pytest.fixture(scope="module")
def kda():
    import chunked_gated_delta_fwd_gb300 as m

    return m


def test_token_rows(kda):
    x, w = torch.zeros(1, 16, device="cuda").expand(PAST, 16), torch.zeros(16, 4, device="cuda")
    with pytest.raises(ValueError, match="2\\^31"):
        kda.causal_conv_step(x, w, torch.zeros(8, 3, 16, device="cuda"))
    with pytest.raises(ValueError, match="2\\^31"):
        kda.causal_conv_fwd(x.unsqueeze(1), w)
    b = torch.zeros(1, 1, 8, device="cuda").expand(PAST, 1, 8)
    with pytest.raises(ValueError, match="2\\^31"):
        kda.selective_step(x, x, torch.zeros(16, 8, device="cuda"), b, b, torch.zeros(8, 16, 8, device="cuda"))
    with pytest.raises(ValueError, match="2\\^31"):
        kda.selective_multi_step(x.unsqueeze(1), x.unsqueeze(1), torch.zeros(16, 8, device="cuda"),
                                 b.unsqueeze(1), b.unsqueeze(1), torch.zeros(8, 16, 8, device="cuda"))


def test_offsets(kda):
    x, w = torch.zeros(6, 16, device="cuda"), torch.zeros(16, 4, device="cuda")
    cu = torch.empty(2 ** 32 + 2, dtype=torch.int32, device="cuda")  # 17 GB, never touched
    with pytest.raises(ValueError, match="2\\^31"):
        kda.causal_conv_fwd(x, w, cu_seqlens=cu, output_final_state=False)
    b = torch.zeros(6, 1, 8, device="cuda")
    with pytest.raises(ValueError, match="2\\^31"):
        kda.selective_scan_fwd(x, x, torch.zeros(16, 8, device="cuda"), b, b, cu_seqlens=cu,
                               output_final_state=False)


def test_vocabulary(kda):
    e = lambda *s, dtype=torch.float32: torch.empty(*s, dtype=dtype, device="cuda")  # noqa: E731
    with pytest.raises(ValueError, match="2\\^31"):
        kda.verify_draft(e(0, 1, dtype=torch.int32), e(0, 1, PAST), e(0, 2, PAST), e(0, 1), e(0))
