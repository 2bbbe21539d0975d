"""The convolution, scan and verification entries without a GPU: bad arguments are refused on
the host, in the C calls and in the binding."""

import ctypes

import pytest
import torch

import __graft_entry__

FAKE = 0x10000  # 16-byte aligned, never dereferenced: every case below fails on the host


@pytest.fixture(scope="module")
def kda():
    __graft_entry__._build_module().build()
    import chunked_gated_delta_fwd_gb300 as m

    return m


def _conv(L, x=FAKE, dtype=1, w=FAKE, b=None, state=None, cu=None, n_seqs=0, B=1, T=64, C=64, W=4,
          sx=64, y=FAKE, sy=64, last=FAKE, flags=1):
    return L.kda_causal_conv_fwd(x, dtype, w, b, state, cu, n_seqs, B, T, C, W, sx, y, sy, last,
                                 None, flags)


def test_conv_rejects_bad_arguments(kda):
    f = lambda **kw: _conv(kda.lib, **kw)  # noqa: E731
    assert f(dtype=2) == 3
    assert f(C=0) == 2 and f(C=4) == 2 and f(C=68, sx=72, sy=72) == 2 and f(C=1 << 25) == 2
    assert f(W=1) == 2 and f(W=5) == 2
    assert f(flags=2) == 1
    assert f(cu=FAKE, n_seqs=0) == 1 and f(cu=FAKE, n_seqs=2, B=2) == 1
    assert f(B=0) == 1 and f(T=-1) == 1 and f(T=1 << 31) == 1
    assert f(B=4, T=(1 << 31) - 65536) == 1
    assert f(x=None) == 1 and f(w=None) == 1 and f(y=None) == 1
    assert f(sx=56) == 1 and f(sy=0) == 1                 # a stride below the row
    assert f(sx=1 << 32) == 1
    assert f(sx=68) == 4 and f(dtype=0, sy=66) == 4
    assert f(x=FAKE + 8) == 4 and f(w=FAKE + 4) == 4 and f(b=FAKE + 8) == 4
    assert f(state=FAKE + 2) == 4 and f(last=FAKE + 8) == 4
    assert f(T=0, last=None) == 0                         # nothing to do, no device needed
    assert b"kda_causal_conv_fwd" in kda.lib.kda_last_error_string()


def test_conv_steps_reject_bad_arguments(kda):
    L = kda.lib

    def one(x=FAKE, dtype=1, w=FAKE, state=FAKE, y=FAKE, N=4, C=64, W=4, sx=64, sy=64, flags=0):
        return L.kda_causal_conv_step(x, dtype, w, None, state, y, N, C, W, sx, sy, None, flags)

    def multi(y=FAKE, N=4, T=4, sx=64):
        return L.kda_causal_conv_multi_step(FAKE, 1, FAKE, None, FAKE, y, None, N, T, 64, 4, sx, 64,
                                            None, 0)

    assert one(dtype=9) == 3 and one(C=12) == 2 and one(W=6) == 2 and one(N=-1) == 2
    assert one(x=None) == 1 and one(w=None) == 1 and one(state=None) == 1 and one(y=None) == 1
    assert one(sx=63) == 1 and one(sx=65) == 4 and one(state=FAKE + 4) == 4 and one(flags=4) == 1
    assert one(N=0) == 0
    assert multi(T=0) == 2 and multi(T=17) == 2 and multi(N=1 << 30, T=4) == 1 and multi(sx=8) == 1
    assert multi(N=0) == 0


def _scan(L, x=FAKE, dt=FAKE, A=FAKE, B=FAKE, C=FAKE, dtype=1, D=None, z=None, h0=None, cu=None,
          n_seqs=0, batch=1, T=64, ch=64, S=16, G=1, sx=64, sdt=64, sB=16, sC=16, sz=64, y=FAKE,
          sy=64, hT=FAKE, flags=1):
    return L.kda_selective_scan_fwd(x, dt, A, B, C, dtype, D, z, None, h0, cu, n_seqs, batch, T, ch,
                                    S, G, sx, sdt, sB, sC, sz, y, sy, hT, None, flags)


def test_scan_rejects_bad_arguments(kda):
    f = lambda **kw: _scan(kda.lib, **kw)  # noqa: E731
    assert f(dtype=2) == 3
    assert f(S=0) == 2 and f(S=4) == 2 and f(S=12) == 2 and f(S=64) == 2
    assert f(ch=0) == 2 and f(G=0) == 2 and f(G=3) == 2 and f(ch=24, G=2) == 2
    assert f(flags=2) == 1
    assert f(cu=FAKE, n_seqs=0) == 1 and f(cu=FAKE, n_seqs=2, batch=2) == 1
    assert f(batch=0) == 1 and f(T=-1) == 1 and f(T=1 << 31) == 1 and f(batch=1 << 16, T=1 << 16) == 1
    for name in ("x", "dt", "A", "B", "C", "y"):
        assert f(**{name: None}) == 1, name
    for name in ("x", "dt", "A", "B", "C", "y", "D", "z", "h0", "hT"):
        assert f(**{name: FAKE + 8}) == 4, name
    assert f(sx=32) == 1 and f(sdt=0) == 1 and f(sB=8) == 1 and f(sC=8) == 1 and f(z=FAKE, sz=8) == 1
    assert f(sB=20) == 4 and f(sy=68) == 4 and f(dtype=0, sC=18) == 4
    assert f(G=2, sB=16, sC=32) == 1                      # a row of B is groups x states
    assert f(T=0, hT=None) == 0
    assert b"kda_selective_scan_fwd" in kda.lib.kda_last_error_string()


def test_scan_steps_reject_bad_arguments(kda):
    L = kda.lib

    def one(x=FAKE, h=FAKE, y=FAKE, dtype=1, N=4, S=16, ch=64, G=1, sx=64, flags=1):
        return L.kda_selective_step(x, FAKE, FAKE, FAKE, FAKE, dtype, None, None, None, h, y, N, ch,
                                    S, G, sx, 64, 16, 16, 64, 64, None, flags)

    def multi(T=4, N=4, y=FAKE, h=FAKE):
        return L.kda_selective_multi_step(FAKE, FAKE, FAKE, FAKE, FAKE, 1, None, None, None, h, y,
                                          None, N, T, 64, 16, 1, 64, 64, 16, 16, 64, 64, None, 1)

    assert one(dtype=5) == 3 and one(S=24) == 2 and one(ch=20) == 2 and one(N=-2) == 2
    assert one(x=None) == 1 and one(h=None) == 1 and one(y=None) == 1 and one(flags=8) == 1
    assert one(h=FAKE + 4) == 4 and one(sx=60) == 1 and one(sx=68) == 4
    assert one(N=0) == 0
    assert multi(T=0) == 2 and multi(T=17) == 2 and multi(N=1 << 30) == 1 and multi(h=None) == 1
    assert multi(N=0) == 0


def _verify(L, draft=FAKE, q=FAKE, p=FAKE, dtype=0, ua=FAKE, us=FAKE, tokens=FAKE, adv=FAKE, N=2,
            T=4, V=100):
    return L.kda_verify_draft(draft, q, p, dtype, ua, us, tokens, adv, N, T, V, None)


def test_verify_rejects_bad_arguments(kda):
    f = lambda **kw: _verify(kda.lib, **kw)  # noqa: E731
    assert f(dtype=2) == 3
    assert f(N=-1) == 2 and f(T=-1) == 2 and f(T=16) == 2 and f(V=0) == 2 and f(N=1 << 25) == 2
    for name in ("draft", "q", "p", "ua", "us", "tokens", "adv"):
        assert f(**{name: None}) == 1, name
    assert f(p=FAKE + 4) == 4 and f(q=FAKE + 8) == 4 and f(us=FAKE + 2) == 4
    assert f(N=0) == 0
    assert b"kda_verify_draft" in kda.lib.kda_last_error_string()


def test_binding_refuses_cpu_tensors(kda):
    x, w = torch.zeros(4, 64), torch.zeros(64, 4)
    with pytest.raises(ValueError):
        kda.causal_conv_fwd(x.unsqueeze(0), w)
    with pytest.raises(ValueError):
        kda.causal_conv_step(x, w, torch.zeros(4, 3, 64))
    with pytest.raises(ValueError):
        kda.causal_conv_multi_step(x.unsqueeze(0), w, torch.zeros(1, 3, 64))
    A, b = torch.zeros(64, 16), torch.zeros(4, 1, 16)
    with pytest.raises(ValueError):
        kda.selective_scan_fwd(x.unsqueeze(0), x.unsqueeze(0), A, b.unsqueeze(0), b.unsqueeze(0))
    with pytest.raises(ValueError):
        kda.selective_step(x, x, A, b, b, torch.zeros(4, 64, 16))
    with pytest.raises(ValueError):
        kda.verify_draft(torch.zeros(1, 2, dtype=torch.int32), torch.zeros(1, 2, 9),
                         torch.zeros(1, 3, 9), torch.zeros(1, 2), torch.zeros(1))


@pytest.mark.skipif(torch.cuda.is_available(), reason="checks the no-GPU error path")
def test_valid_calls_without_gpu_fail_cleanly(kda):
    assert _conv(kda.lib) in (6, 8)
    assert _scan(kda.lib) in (6, 8)
    assert _verify(kda.lib) in (6, 8)
    assert _verify(kda.lib, T=0, draft=None, q=None, ua=None) in (6, 8)
    assert ctypes.c_char_p(kda.lib.kda_last_error_string()).value
