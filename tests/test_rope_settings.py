"""Settings of the norm with rotation that the binding refuses before it looks at a tensor."""

import pytest
import torch

import __graft_entry__


@pytest.fixture(scope="module")
def kda():
    __graft_entry__._build_module().build()
    import chunked_gated_delta_fwd_gb300 as m

    return m


@pytest.mark.parametrize("eps", [-1.0, -1e-6, -float("inf"), float("nan")])
def test_a_negative_eps_does_not_turn_the_norm_off(kda, eps):
    x = torch.zeros(4, 2, 128)
    with pytest.raises(ValueError, match="eps"):
        kda.qk_norm_rope(x, x, torch.zeros(4, dtype=torch.int32), torch.zeros(64), eps=eps)


@pytest.mark.parametrize("eps", [None, 0, 0.0, 1e-6])
def test_the_settings_that_are_allowed_pass(kda, eps):
    x = torch.zeros(4, 2, 128)
    with pytest.raises(ValueError, match="CUDA"):  # the next check: no CUDA tensors
        kda.qk_norm_rope(x, x, torch.zeros(4, dtype=torch.int32), torch.zeros(64), eps=eps)
