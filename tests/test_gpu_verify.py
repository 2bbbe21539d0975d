"""The verification of drafted tokens against an oracle in exact fractions: results are whole
numbers and have to be equal, whatever the row's length, split and type."""

import numpy as np
import pytest
import torch

import oracle

pytestmark = pytest.mark.gpu

DT = [torch.bfloat16, torch.float32]
IDS = ["bf16", "f32"]


@pytest.fixture(scope="module")
def kda():
    import chunked_gated_delta_fwd_gb300 as m

    return m


def make(N, T, V, dtype, seed, keep=0.6, sharp=2.0):
    gen = torch.Generator().manual_seed(seed)
    r = lambda *s: torch.randn(*s, generator=gen)  # noqa: E731
    p = torch.softmax(sharp * r(N, T + 1, V), -1)
    q = keep * p[:, :T] + (1 - keep) * torch.softmax(sharp * r(N, T, V), -1)
    draft = torch.multinomial(q.reshape(-1, V), 1, generator=gen).view(N, T) if T else \
        torch.zeros(N, 0)
    return [draft.to(torch.int32), q.to(dtype), p.to(dtype), torch.rand(N, T, generator=gen),
            torch.rand(N, generator=gen)]


def check(kda, args):
    got = [t.cpu().numpy() for t in kda.verify_draft(*(a.cuda() for a in args))]
    want = oracle.verify_draft(args[0].tolist(), args[1].float(), args[2].float(), args[3].tolist(),
                               args[4].tolist())
    assert np.array_equal(got[1], want[1])
    assert np.array_equal(got[0], want[0])
    return got


@pytest.mark.parametrize("dtype", DT, ids=IDS)
@pytest.mark.parametrize("T", [0, 1, 4, 15])
@pytest.mark.parametrize("V", [1, 2, 31, 32, 33, 127, 1000, 4096, 5003])
def test_against_the_oracle(kda, dtype, T, V):
    check(kda, make(5, T, V, dtype, seed=V + T))


@pytest.mark.parametrize("dtype", DT, ids=IDS)
@pytest.mark.parametrize("N,V", [(1, 50001), (3, 32768), (150, 700), (400, 64), (2, 200000)])
def test_batches_and_vocabularies(kda, dtype, N, V):
    check(kda, make(N, 2, V, dtype, seed=N, keep=0.3))


def test_every_count_of_accepted_tokens(kda):
    draft, q, p, ua, us = make(16, 15, 257, torch.float32, seed=1)
    at = draft.long().unsqueeze(2)
    ratio = (p[:, :15].gather(2, at) / q.gather(2, at)).squeeze(2)
    for n in range(16):  # the first n accepted, the next one not
        ua[n] = (0.5 * ratio[n]).clamp(max=0.9)
        if n < 15:
            q[n, n] = 0.0
            q[n, n, draft[n, n]] = 1.0
            ua[n, n] = 0.999999
            p[n, n, draft[n, n]] = 0.01
    _, count = check(kda, [draft, q, p, ua, us])
    assert count.tolist() == list(range(1, 17))


def test_borders_and_equality(kda):
    p = torch.zeros(6, 2, 8)
    q = torch.zeros(6, 1, 8)
    p[:, 0, :4], q[:, 0, 0] = 0.25, 0.5
    p[:, 1, 7] = 1.0
    draft = torch.zeros(6, 1, dtype=torch.int32)
    ua = torch.tensor([0.5, 0.5 - 2.0 ** -25, 0.0, 0.75, 0.75, 0.75]).view(6, 1)
    us = torch.tensor([0.0, 0.9, 0.9, 1 / 3, 2 / 3, 1 - 2.0 ** -24])
    tokens, count = check(kda, [draft, q, p, ua, us])
    assert count.tolist() == [1, 2, 2, 1, 1, 1] and tokens[0].tolist() == [1, -1]
    assert tokens[1].tolist() == [0, 7] and tokens[5].tolist() == [3, -1]


def test_short_drafts_and_tokens_outside(kda):
    args = make(8, 4, 100, torch.float32, seed=2)
    args[3][:] = 0.0  # whatever is drafted is accepted
    for n, v in enumerate([-1, 100, 2 ** 31 - 1, -2 ** 31, 5, 99, -1, 0]):
        args[0][n, n % 5 if n % 5 < 4 else 0] = v
    _, count = check(kda, args)
    assert count[0] == 1 and count[1] == 2 and count[2] == 3 and count[3] == 4


def test_weights_that_are_not_probabilities(kda):
    draft, q, p, ua, us = make(9, 1, 70, torch.float32, seed=3)
    ua[:] = 0.999
    at = torch.arange(9)
    p[at, 0, draft[:, 0].long()] = 0.0              # rejected throughout
    p[0, 0, 3] = float("nan")
    p[1, 0, 4] = float("inf")
    p[2, 0] = -1.0
    p[3, 0] = 0.0                                   # nothing to draw from
    q[4, 0] = 2.0                                   # nothing is left of p
    q[5, 0, 8] = float("nan")
    p[6, 0, 9:] = 1e-30                             # below a weight's last bit
    p[7, 0] = 1.0
    q[8, 0, 0] = float("inf")
    tokens, _ = check(kda, [draft, q, p, ua, us])
    assert tokens[3, 0] == 0 and tokens[2, 0] == 0
    # sums beyond 256 stop there: some token of the row
    p, q = torch.ones(4, 2, 3000), torch.zeros(4, 1, 3000)
    t, c = kda.verify_draft(torch.full((4, 1), -1, dtype=torch.int32).cuda(), q.cuda(), p.cuda(),
                            torch.zeros(4, 1).cuda(), torch.tensor([0.0, 0.3, 0.9, 0.999]).cuda())
    assert torch.all((t[:, 0] >= 0) & (t[:, 0] < 3000)) and torch.all(c == 1)


def test_rows_past_32_bits(kda):
    N, T, V = 9, 15, 1 << 24
    p = torch.zeros(N, T + 1, V, dtype=torch.bfloat16, device="cuda")
    q = torch.zeros(N, T, V, dtype=torch.bfloat16, device="cuda")
    q[:, :, 7] = 1.0
    p[:, :, 7] = 1.0
    p[:, T, 7] = 0.0
    p[:, T, V - 1] = 1.0
    t, c = kda.verify_draft(torch.full((N, T), 7, dtype=torch.int32, device="cuda"), q, p,
                            torch.full((N, T), 0.5, device="cuda"), torch.full((N,), 0.5, device="cuda"))
    assert torch.all(t[:, :T] == 7) and torch.all(t[:, T] == V - 1) and torch.all(c == T + 1)


def test_captured_given_outputs_and_no_sequences(kda):
    args = [a.cuda() for a in make(6, 3, 999, torch.float32, seed=4)]
    t0, c0 = kda.verify_draft(*args)
    buf = torch.full((8, 4), 77, dtype=torch.int32, device="cuda")
    cnt = torch.full((8,), 77, dtype=torch.int32, device="cuda")
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.stream(st):
        with torch.cuda.graph(graph, stream=st):
            kda.verify_draft(*args, tokens_out=buf[1:7], n_advance_out=cnt[1:7])
    torch.cuda.current_stream().wait_stream(st)
    graph.replay()
    assert torch.equal(buf[1:7], t0) and torch.equal(cnt[1:7], c0)
    assert torch.all(buf[0] == 77) and torch.all(buf[7] == 77) and cnt[0] == 77 and cnt[7] == 77
    args[4].uniform_()
    graph.replay()
    assert torch.equal(buf[1:7], kda.verify_draft(*args)[0])
    t, c = kda.verify_draft(*(a[:0] for a in args))
    assert t.shape == (0, 4) and c.shape == (0,)


def test_binding_checks(kda):
    d, q, p, ua, us = (a.cuda() for a in make(2, 3, 50, torch.float32, seed=5))
    for bad in ((d.long(), q, p, ua, us), (d[:, :2], q, p, ua, us), (d, q[:, :2], p, ua, us),
                (d, q.bfloat16(), p, ua, us), (d, q.half(), p.half(), ua, us), (d, q, p, ua.double(), us),
                (d, q, p, ua, us[:1]), (d, q, p.cpu(), ua, us), (d, q, p[..., ::2], ua, us)):
        with pytest.raises((ValueError, TypeError)):
            kda.verify_draft(*bad)
    p = torch.zeros(2, 17, 50, device="cuda")
    with pytest.raises(kda.KdaError):
        kda.verify_draft(torch.zeros(2, 16, dtype=torch.int32, device="cuda"), p[:, :16].contiguous(), p,
                         torch.zeros(2, 16, device="cuda"), us)
