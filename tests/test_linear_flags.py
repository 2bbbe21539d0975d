"""Flags of the KDA calls that linear attention does not know are refused, by the binding and by
the C calls; none of them may stand for something else there."""

import pytest
import torch

import __graft_entry__

FAKE = 0x10000  # 16-byte aligned, never dereferenced: every call below fails on the host


@pytest.fixture(scope="module")
def kda():
    __graft_entry__._build_module().build()
    import chunked_gated_delta_fwd_gb300 as m

    return m


FOREIGN = ["UNBOUNDED_GATE", "SCALAR_GATE", "CHECK_INPUTS", "PRECISE", "_HEAD_DECAY"]


@pytest.mark.parametrize("name", FOREIGN)
@pytest.mark.parametrize("more", [0, 1, 2, 5 << 16])
def test_the_binding_refuses_flags_of_other_calls(kda, name, more):
    x, g = torch.zeros(1, 4, 2, 128), torch.zeros(1, 4, 2)
    with pytest.raises(ValueError, match="flags"):
        kda.linear_chunk_fwd(x, x, x, g, flags=getattr(kda, name) | more)


@pytest.mark.parametrize("name", FOREIGN[:-1])
def test_the_c_calls_refuse_flags_of_other_calls(kda, name):
    flag, L = getattr(kda, name), kda.lib
    assert L.kda_linear_chunk_fwd(FAKE, FAKE, FAKE, 1, FAKE, 1.0, None, None, 0, 1, 64, 4, 2, 128, 128,
                                  FAKE, FAKE, FAKE, 1 << 40, None, flag) == 1
    assert L.kda_linear_recurrent_step(FAKE, FAKE, FAKE, 1, FAKE, 1.0, FAKE, FAKE, 4, 4, 2, 128, 128,
                                       None, flag) == 1
    assert L.kda_linear_recurrent_multi_step(FAKE, FAKE, FAKE, 1, FAKE, 1.0, FAKE, FAKE, None, 4, 4, 4,
                                             2, 128, 128, None, flag) == 1
    assert b"flags" in L.kda_last_error_string()


def test_every_other_bit_is_refused(kda):
    x, g = torch.zeros(1, 4, 2, 128), torch.zeros(1, 4, 2)
    for bit in list(range(2, 16)) + [32, 40]:
        with pytest.raises(ValueError, match="flags"):
            kda.linear_chunk_fwd(x, x, x, g, flags=1 << bit)
    with pytest.raises(ValueError, match="flags"):
        kda.linear_chunk_fwd(x, x, x, g, flags=-1)


def test_the_flags_that_are_known_pass_the_check(kda):
    x, g = torch.zeros(1, 4, 2, 128), torch.zeros(1, 4, 2)
    for flags in (0, kda.FP32_CORES, kda.SEQUENTIAL, kda.segment_chunks(3),
                  kda.SEQUENTIAL | kda.segment_chunks(65535)):
        with pytest.raises(ValueError, match="CUDA"):  # the next check: no CUDA tensors
            kda.linear_chunk_fwd(x, x, x, g, flags=flags)
