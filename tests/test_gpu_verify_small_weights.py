"""The verification where small weights decide.  Weights are whole numbers of 2^-56, so a row of
weights of 2^-56 to 2^-24 is drawn from as exactly as one of large ones; results are whole numbers and
have to equal the oracle's exact fractions."""

import numpy as np
import pytest
import torch

from tests.test_gpu_verify import DT, IDS, check

pytestmark = pytest.mark.gpu

# Lengths that one, two, four and eight CTAs share, whole 16-byte pieces and not.
SIZES = [8, 31, 700, 5000, 5003, 32768, 50001, 200000]


@pytest.fixture(scope="module")
def kda():
    import chunked_gated_delta_fwd_gb300 as m

    return m


def spread(gen, lo, hi, *shape):
    """Weights whose logarithms are uniform between lo and hi (to base 2)."""
    return torch.exp2(lo + (hi - lo) * torch.rand(*shape, generator=gen, dtype=torch.float64)).float()


def units(w):
    return int(float(w) * 2.0 ** 56)


@pytest.mark.parametrize("dtype", DT, ids=IDS)
@pytest.mark.parametrize("V", [2, 16, 4099])
def test_single_weights_of_every_exponent(kda, dtype, V):
    """One weight against another, the random number on either side of the border between them."""
    gen = torch.Generator().manual_seed(V)
    exps = torch.arange(0, -57, -1, dtype=torch.float64).repeat(2 if V > 16 else 6)
    N = len(exps)
    rand = lambda: torch.rand(N, generator=gen, dtype=torch.float64)  # noqa: E731
    first = torch.exp2(exps - rand()).to(dtype)
    second = (first.double() * torch.exp2(4 * rand() - 2)).clamp(2.0 ** -56, 1.0).to(dtype)
    p = torch.zeros(2 * N, 1, V, dtype=dtype)
    us, want = torch.zeros(2 * N), []
    for n in range(N):
        a, b = units(first[n]), units(second[n])
        at = n * 7 % (V - 1)
        p[2 * n:2 * n + 2, 0, at], p[2 * n:2 * n + 2, 0, V - 1] = first[n], second[n]
        border = -(-(a << 24) // (a + b))  # of the random number, in units of 2^-24
        us[2 * n], us[2 * n + 1] = (border - 1) / 2 ** 24, border / 2 ** 24
        want += [at if a else V - 1, V - 1]
    none = torch.zeros(2 * N, 0, dtype=torch.int32)
    us = us.clamp(min=0.0)
    tokens, _ = check(kda, [none, torch.zeros(2 * N, 0, V, dtype=dtype), p, torch.zeros(2 * N, 0), us])
    assert tokens[:, 0].tolist() == want


@pytest.mark.parametrize("dtype", DT, ids=IDS)
@pytest.mark.parametrize("V", SIZES)
@pytest.mark.parametrize("lo,hi", [(-60, -40), (-56, -24)])
def test_rows_of_small_weights(kda, dtype, V, lo, hi):
    """Whole rows, of p behind an accepted token and of max(p - q, 0) behind a rejected one."""
    N = 8 if V < 50000 else 2
    gen = torch.Generator().manual_seed(V - lo)
    p = spread(gen, lo, hi, N, 2, V)
    q = p[:, :1] * torch.tensor([0.25, 0.75, 1.0, 2.0])[torch.randint(0, 4, (N, 1, V), generator=gen)]
    draft = torch.randint(0, V, (N, 1), generator=gen)
    at = torch.arange(N)
    q[at, 0, draft[:, 0]] = 1.0
    p[at[::2], 0, draft[::2, 0]] = 1.0  # every other one is accepted
    _, count = check(kda, [draft.to(torch.int32), q.to(dtype), p.to(dtype), torch.full((N, 1), 0.5),
                           torch.rand(N, generator=gen)])
    assert count.tolist() == [2, 1] * (N // 2)


@pytest.mark.parametrize("dtype", DT, ids=IDS)
@pytest.mark.parametrize("V", SIZES)
def test_a_few_small_weights_in_a_row_of_zeros(kda, dtype, V):
    where = [V // 5, V // 2, V - 1]
    weights = [2.0 ** -48, 2.0 ** -47, 2.0 ** -50]     # 256, 512 and 64 units
    us = [0.0, 255 / 832, 257 / 832, 767 / 832, 769 / 832, 1 - 2.0 ** -24]
    want = [where[i] for i in (0, 0, 1, 1, 2, 2)] + where
    N = len(want)
    p = torch.zeros(N, 1, V, dtype=dtype)
    for v, w in zip(where, weights):
        p[:6, 0, v] = w
    for i, v in enumerate(where):  # the smallest weight of all, alone
        p[6 + i, 0, v] = 2.0 ** -56
    none = torch.zeros(N, 0, dtype=torch.int32)
    tokens, _ = check(kda, [none, torch.zeros(N, 0, V, dtype=dtype), p, torch.zeros(N, 0),
                            torch.tensor(us + [0.0, 0.5, 1 - 2.0 ** -24])])
    assert tokens[:, 0].tolist() == want


@pytest.mark.parametrize("dtype", DT, ids=IDS)
@pytest.mark.parametrize("V", SIZES)
def test_a_small_rest_behind_a_rejected_token(kda, dtype, V):
    """2^-48 is left of p behind q at one token, and 0 at all others: that one is drawn, not one
    of p's."""
    places = [0, V // 3, V - 2]
    N = len(places)
    p = torch.full((N, 2, V), 2.0 ** -9, dtype=dtype)
    q = torch.full((N, 1, V), 2.0 ** -9, dtype=dtype)
    for n, v in enumerate(places):
        p[n, 0, v], q[n, 0, v] = 2.0 ** -45 + 2.0 ** -48, 2.0 ** -45
    q[:, 0, V - 1] = 0.5
    draft = torch.full((N, 1), V - 1, dtype=torch.int32)
    tokens, count = check(kda, [draft, q, p, torch.full((N, 1), 0.5), torch.tensor([0.0, 0.5, 0.999])])
    assert tokens[:, 0].tolist() == places and np.all(count == 1)


@pytest.mark.parametrize("dtype", DT, ids=IDS)
def test_zero_draws_the_first_token_that_weighs_anything(kda, dtype):
    N, V = 57, 1003
    p = torch.zeros(N, 1, V, dtype=dtype)
    for n in range(N):
        p[n, 0, 3 + n] = 2.0 ** -n
        p[n, 0, 500:] = 0.001
    none = torch.zeros(N, 0, dtype=torch.int32)
    tokens, _ = check(kda, [none, torch.zeros(N, 0, V, dtype=dtype), p, torch.zeros(N, 0), torch.zeros(N)])
    assert tokens[:, 0].tolist() == [3 + n for n in range(N)]
