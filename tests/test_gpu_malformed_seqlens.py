"""cu_seqlens that is not what it should be: reported, and nothing behind a workspace, an output
or a final state is written.  Every buffer lies inside a larger one whose other bytes are
watched; the offsets go up and down inside [0, NT], so that their rising parts alone add up to
several times the tokens that the workspaces are sized for."""

import pytest
import torch

pytestmark = pytest.mark.gpu

GUARD = 1 << 24  # watched bytes on either side (more than 64 chunks' states)
MARK = 0xA5


@pytest.fixture(scope="module")
def kda():
    import chunked_gated_delta_fwd_gb300 as m

    return m


class Watched:
    """`n` bytes between two watched stretches."""

    def __init__(self, n):
        n = -(-n // 256) * 256
        self.n, self.all = n, torch.full((n + 2 * GUARD,), MARK, dtype=torch.uint8, device="cuda")

    def view(self, shape, dtype):
        size = torch.Size(shape).numel() * dtype.itemsize
        return self.all[GUARD:GUARD + size].view(dtype).view(shape)

    def untouched(self):
        return bool((self.all[:GUARD] == MARK).all()) and bool((self.all[GUARD + self.n:] == MARK).all())


def sawtooth(nt, n):
    return torch.tensor([0] + [nt if i % 2 == 0 else 0 for i in range(n)], dtype=torch.int32)


def run(kda, call, sizes, nt, H, n, cu, dtype):
    """The call on watched buffers; the error must be reported and the marks be whole."""
    gen = torch.Generator(device="cuda").manual_seed(nt + n)
    r = lambda *s: torch.randn(*s, generator=gen, device="cuda")  # noqa: E731
    q, k, v = (0.1 * r(nt, H, 128)).to(dtype), (0.1 * r(nt, H, 128)).to(dtype), r(nt, H, 128).to(dtype)
    ws, o, hT = Watched(sizes), Watched(v.numel() * dtype.itemsize), Watched(n * H * 65536)
    kda.get_device_error()
    call(q, k, v, cu.cuda(), workspace=ws.view((ws.n,), torch.uint8), out=o.view(v.shape, dtype),
         final_state_out=hT.view((n, H, 128, 128), torch.float32))
    with pytest.raises(kda.KdaError, match="cu_seqlens"):
        kda.get_device_error()
    assert ws.untouched() and o.untouched() and hT.untouched()


@pytest.mark.parametrize("nt,n,H", [(640, 3, 2), (640, 9, 2), (1000, 41, 3), (130, 2500, 1)])
@pytest.mark.parametrize("path", ["f32", "bf16 on fp32 cores", "bf16", "bf16 segments"])
def test_linear_prompts_whose_offsets_go_up_and_down(kda, path, nt, n, H):
    dtype = torch.float32 if path == "f32" else torch.bfloat16
    flags = {"bf16 on fp32 cores": kda.FP32_CORES, "bf16 segments": kda.segment_chunks(1)}.get(path, 0)
    g = -0.1 * torch.ones(nt, H, device="cuda")
    run(kda, lambda q, k, v, cu, **kw: kda.linear_chunk_fwd(q, k, v, g, None, cu, flags=flags, **kw),
        kda.linear_chunk_fwd_workspace_size(nt, n, H, dtype, flags), nt, H, n, sawtooth(nt, n), dtype)


@pytest.mark.parametrize("nt,n,H", [(640, 9, 2), (130, 2500, 1)])
@pytest.mark.parametrize("path", ["f32", "bf16", "bf16 segments"])
def test_kda_prompts_whose_offsets_go_up_and_down(kda, path, nt, n, H):
    dtype = torch.float32 if path == "f32" else torch.bfloat16
    flags = kda.segment_chunks(1) if path == "bf16 segments" else 0
    g = -0.1 * torch.ones(nt, H, 128, device="cuda")
    beta = torch.full((nt, H), 0.5, device="cuda", dtype=dtype)
    run(kda, lambda q, k, v, cu, **kw: kda.chunk_fwd(q, k, v, g, beta, None, cu, flags=flags, **kw),
        kda.chunk_fwd_workspace_size(nt, n, H, dtype, flags), nt, H, n, sawtooth(nt, n), dtype)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=["bf16", "f32"])
def test_a_good_batch_of_many_sequences_after_a_bad_one(kda, dtype):
    """Over 1024 offsets in several rounds of the plan: right before and behind a malformed call
    on the same workspace."""
    gen = torch.Generator(device="cuda").manual_seed(5)
    n = 2300
    lens = torch.randint(0, 5, (n,), generator=gen, device="cuda")
    cu = torch.cat([lens.new_zeros(1), lens.cumsum(0)]).to(torch.int32)
    nt = int(cu[-1])
    r = lambda *s: torch.randn(*s, generator=gen, device="cuda")  # noqa: E731
    q, k, v = r(nt, 1, 128).to(dtype), r(nt, 1, 128).to(dtype), r(nt, 1, 128).to(dtype)
    g = -0.1 * torch.ones(nt, 1, device="cuda")
    flags = kda.FP32_CORES
    ws = torch.empty(kda.linear_chunk_fwd_workspace_size(nt, n, 1, dtype, flags), dtype=torch.uint8,
                     device="cuda")
    kda.get_device_error()
    call = lambda cu: kda.linear_chunk_fwd(q, k, v, g, None, cu, flags=flags, workspace=ws)  # noqa: E731
    o, hT = call(cu)
    kda.get_device_error()
    bad = cu.clone()
    bad[1500] = 0
    call(bad)
    with pytest.raises(kda.KdaError, match="cu_seqlens"):
        kda.get_device_error()
    o2, hT2 = call(cu)
    kda.get_device_error()
    assert torch.equal(o, o2) and torch.equal(hT, hT2)
    x = torch.arange(nt, device="cuda")
    seq = torch.searchsorted(cu[1:].long(), x, right=True)
    same = (seq.view(-1, 1) == seq.view(1, -1)) & (x.view(-1, 1) >= x.view(1, -1))
    w = torch.exp(-0.1 * (x.view(-1, 1) - x.view(1, -1)).double()) * same
    ref = ((q[:, 0].double() @ k[:, 0].double().T) * w) @ v[:, 0].double()
    # at most five terms of 128 products each: 512 u of the sum of magnitudes, o rounded once
    big = ((q[:, 0].double().abs() @ k[:, 0].double().abs().T) * w) @ v[:, 0].double().abs()
    half = 2.0 ** -8 * ref.abs() if dtype == torch.bfloat16 else 0.0
    assert bool(((o[:, 0].double() - ref).abs() <= 512 * 2.0 ** -24 * big + half + 1e-30).all())


def test_segments_whose_count_passes_32_bits(kda):
    """Overlapping sequences that ask for over 2^31 segments between them."""
    nt, n = 5932032, 92700
    flags = kda.segment_chunks(1)
    assert (n // 2) * (nt // 128) > 2 ** 31
    q = torch.zeros(nt, 1, 128, dtype=torch.bfloat16, device="cuda")
    g = torch.zeros(1, device="cuda")
    need = kda.linear_chunk_fwd_workspace_size(nt, n, 1, torch.bfloat16, flags)
    ws, o = Watched(need), Watched(2 * q.numel())
    kda.get_device_error()
    kda.linear_chunk_fwd(q, q, q, g, None, sawtooth(nt, n).cuda(), flags=flags,
                         workspace=ws.view((ws.n,), torch.uint8), output_final_state=False,
                         out=o.view(q.shape, torch.bfloat16))
    with pytest.raises(kda.KdaError, match="cu_seqlens"):
        kda.get_device_error()
    assert ws.untouched() and o.untouched()
    assert not bool(o.view(q.shape, torch.bfloat16).any())
    del q, ws, o
    torch.cuda.empty_cache()
