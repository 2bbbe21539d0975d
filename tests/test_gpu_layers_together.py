"""The convolution, the scan, the KDA step and the verification as a serving program runs them:
prompts, then drafted tokens of which a part is kept, then the same again -- against the kept
tokens run in one go."""

import pytest
import torch

pytestmark = pytest.mark.gpu

C, S, W, T, V = 128, 16, 4, 4, 600


@pytest.fixture(scope="module")
def kda():
    import chunked_gated_delta_fwd_gb300 as m

    return m


class Layer:
    """One recurrent layer of each kind over the same inputs; float32, so that only the order of
    sums differs between the forms."""

    def __init__(self, kda, N, gen):
        r = lambda *s: torch.randn(*s, generator=gen, device="cuda")  # noqa: E731
        self.kda, self.N = kda, N
        self.w, self.A, self.D = r(C, W) / 2, -r(C, S).abs() - 0.1, r(C)
        self.table = r(V, C)              # embeddings
        self.mix = r(C, C + 2 * S) * C ** -0.5

    def around(self, u):
        low = u @ self.mix
        return (u, low[..., :C].contiguous(), self.A, low[..., C:C + S].unsqueeze(-2),
                low[..., C + S:].unsqueeze(-2))

    def gates(self, u):
        g = -torch.sigmoid(u).unsqueeze(-2).contiguous()
        return g, torch.sigmoid(u[..., :1]).contiguous()

    def prompt(self, ids, cu):
        x = self.table[ids]
        u, self.conv = self.kda.causal_conv_fwd(x, self.w, cu_seqlens=cu)
        y, self.h = self.kda.selective_scan_fwd(*self.around(u), cu_seqlens=cu, D=self.D, z=x)
        k = torch.nn.functional.normalize(u, dim=-1).unsqueeze(-2)
        g, beta = self.gates(u)
        o, self.S = self.kda.chunk_fwd(k, k, u.unsqueeze(-2), g, beta, cu_seqlens=cu)
        return y, o.squeeze(-2)

    def verify(self, ids, n_advance):
        x = self.table[ids]
        u = self.kda.causal_conv_multi_step(x, self.w, self.conv, n_advance)
        y = self.kda.selective_multi_step(*self.around(u), self.h, n_advance, D=self.D, z=x)
        k = torch.nn.functional.normalize(u, dim=-1).unsqueeze(-2)
        g, beta = self.gates(u)
        o = self.kda.recurrent_multi_step(k, k, u.unsqueeze(-2), g, beta, self.S, n_advance)
        return y, o.squeeze(-2)


def close(a, b):
    """Sums in another order over at most 200 tokens: the package's fp32 bound."""
    assert (a - b).norm() <= 1e-5 * b.norm(), float((a - b).norm() / b.norm())


def test_prompt_draft_verify_replay(kda):
    gen = torch.Generator(device="cuda").manual_seed(0)
    lens = [70, 3, 121, 1, 64]
    N = len(lens)
    layer = Layer(kda, N, gen)
    ids = [torch.randint(0, V, (n,), generator=gen, device="cuda") for n in lens]
    cu = torch.tensor([0] + lens, device="cuda").cumsum(0).to(torch.int32)
    layer.prompt(torch.cat(ids), cu)
    last = torch.randint(0, V, (N, 1), generator=gen, device="cuda")
    zeros = torch.zeros(N, dtype=torch.int32, device="cuda")
    heard = [[] for _ in range(N)]
    counts = []
    for _ in range(4):
        p = torch.softmax(2 * torch.randn(N, T + 1, V, generator=gen, device="cuda"), -1)
        q = 0.7 * p[:, :T] + 0.3 / V
        draft = torch.multinomial(q.view(-1, V), 1, generator=gen).view(N, T)
        block = torch.cat([last, draft], dim=1)
        before = layer.h.clone()
        layer.verify(block, zeros)                       # the verify pass: states stay
        assert torch.equal(layer.h, before)
        tokens, adv = kda.verify_draft(draft.to(torch.int32), q, p,
                                       torch.rand(N, T, generator=gen, device="cuda"),
                                       torch.rand(N, generator=gen, device="cuda"))
        y, o = layer.verify(block, adv)                  # the replay: states move on
        for n in range(N):
            a = int(adv[n])
            assert torch.equal(tokens[n, :a - 1].long(), draft[n, :a - 1])
            assert torch.all(tokens[n, a:] == -1) and 0 <= int(tokens[n, a - 1]) < V
            heard[n].append((block[n, :a], y[n, :a], o[n, :a]))
        counts += adv.tolist()
        last = tokens.long().gather(1, adv.long().unsqueeze(1) - 1)
    assert 1 < sum(counts) / len(counts) < T + 1         # some kept, some not
    conv, h, state = layer.conv, layer.h, layer.S
    whole = [torch.cat([ids[n]] + [b for b, _, _ in heard[n]]) for n in range(N)]
    cu2 = torch.tensor([0] + [len(w) for w in whole], device="cuda").cumsum(0).to(torch.int32)
    y, o = layer.prompt(torch.cat(whole), cu2)
    assert torch.equal(layer.conv, conv)
    close(h, layer.h)
    close(state, layer.S)
    for n in range(N):
        b = int(cu2[n]) + lens[n]
        close(torch.cat([v for _, v, _ in heard[n]]), y[b:int(cu2[n + 1])])
        close(torch.cat([v for _, _, v in heard[n]]), o[b:int(cu2[n + 1])])
