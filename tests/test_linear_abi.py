"""The linear-attention and norm-rotation entries without a GPU: bad arguments are refused
on the host, in the C calls and in the binding."""

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


def _rope(L, dtype=1, eps=1e-6, n_axes=1, axis=None, F=64, nt=10, Hq=4, Hk=2, d=128, q=FAKE,
          w=None, pos=FAKE, sq=512, sk=256, sqo=512, sko=256):
    return L.kda_qk_norm_rope(q, FAKE, dtype, w, None, eps, pos, n_axes, axis, FAKE, F, 0, FAKE,
                              FAKE, nt, Hq, Hk, d, sq, sk, sqo, sko, None)


def test_norm_rope_rejects_bad_arguments(kda):
    f = lambda **kw: _rope(kda.lib, **kw)  # noqa: E731
    assert f(dtype=2) == 3
    assert f(d=64) == 2
    assert f(Hq=0) == 2 and f(Hk=0) == 2
    assert f(F=0) == 2 and f(F=12) == 2 and f(F=72) == 2
    assert f(n_axes=0) == 1
    assert f(n_axes=3) == 1                      # several axes without freq_axis
    assert f(nt=-1) == 1
    assert f(eps=float("nan")) == 1 and f(eps=float("inf")) == 1
    assert f(eps=-1.0, w=FAKE) == 1              # a weight without the norm
    assert f(q=None) == 1 and f(pos=None) == 1
    assert f(q=FAKE + 8) == 4 and f(w=FAKE + 4) == 4
    assert f(sq=511) == 1 and f(sko=0) == 1      # a stride below the row
    assert f(sq=513) == 4 and f(dtype=0, sk=258) == 4
    assert f(nt=0) == 0                          # nothing to do, no device needed
    assert b"kda_qk_norm_rope" in kda.lib.kda_last_error_string()


def _chunk(L, dtype=1, scale=1.0, h0=None, cu=None, n_seqs=0, B=1, T=64, H=4, Hk=2, dk=128,
           dv=128, q=FAKE, g=FAKE, o=FAKE, hT=FAKE, ws=FAKE, ws_bytes=1 << 40, flags=0):
    return L.kda_linear_chunk_fwd(q, FAKE, FAKE, dtype, g, scale, h0, cu, n_seqs, B, T, H, Hk, dk,
                                  dv, o, hT, ws, ws_bytes, None, flags)


def test_linear_chunk_rejects_bad_arguments(kda):
    f = lambda **kw: _chunk(kda.lib, **kw)  # noqa: E731
    assert f(dtype=2) == 3
    assert f(dk=64) == 2 and f(dv=64) == 2
    assert f(H=0) == 2 and f(Hk=0) == 2 and f(H=5) == 2 and f(Hk=8) == 2
    assert f(scale=float("nan")) == 1 and f(scale=float("inf")) == 1
    assert f(cu=FAKE, n_seqs=0) == 1 and f(cu=FAKE, n_seqs=2, B=2) == 1
    assert f(B=0) == 1 and f(T=-1) == 1 and f(T=1 << 31) == 1
    assert f(B=4, T=1 << 62) == 1  # (their product is 0 in 64 bits)
    assert f(q=None) == 1 and f(g=None) == 1 and f(o=None) == 1 and f(ws=None) == 1
    assert f(q=FAKE + 8) == 4 and f(h0=FAKE + 4) == 4 and f(ws=FAKE + 16) == 4
    assert f(dtype=0, ws_bytes=16) == 5
    assert f(flags=1 << 10) == 1
    assert b"kda_linear_chunk_fwd" in kda.lib.kda_last_error_string()


def test_linear_workspace_size(kda):
    f = kda.linear_chunk_fwd_workspace_size
    assert f(-1, 1, 2) == 0 and f(10, 0, 2) == 0 and f(10, 1, 0) == 0
    assert kda.lib.kda_linear_chunk_fwd_workspace_size(10, 1, 2, 5, 0) == 0
    # the fp32-core path keeps a state a 64-token chunk and head
    a, b = f(4096, 1, 4, torch.float32), f(8192, 1, 4, torch.float32)
    assert b - a >= 64 * 4 * 128 * 128 * 4
    assert f(4096, 1, 4, torch.bfloat16, kda.FP32_CORES) == a
    assert f(0, 3, 4) > 0


def test_linear_steps_reject_bad_arguments(kda):
    L = kda.lib

    def one(dtype=1, g=FAKE, scale=1.0, S=FAKE, o=FAKE, N=4, H=4, Hk=2, dk=128, flags=0):
        return L.kda_linear_recurrent_step(FAKE, FAKE, FAKE, dtype, g, scale, S, o, N, H, Hk, dk,
                                           128, None, flags)

    def multi(T=4, N=4, o=FAKE, q=FAKE, flags=0):
        return L.kda_linear_recurrent_multi_step(q, FAKE, FAKE, 1, FAKE, 1.0, FAKE, o, None, N, T,
                                                 4, 2, 128, 128, None, flags)

    assert one(dtype=7) == 3 and one(dk=64) == 2 and one(Hk=3) == 2 and one(N=-1) == 2
    assert one(scale=float("inf")) == 1 and one(g=None) == 1 and one(o=None) == 1
    assert one(S=FAKE + 4) == 4 and one(flags=1) == 1
    assert one(N=1 << 30, H=1 << 15, Hk=1) == 1
    assert one(N=0) == 0
    assert multi(T=0) == 2 and multi(T=17) == 2 and multi(q=None) == 1 and multi(o=FAKE + 2) == 4
    assert multi(N=0) == 0


def test_binding_refuses_cpu_tensors(kda):
    x = torch.zeros(4, 2, 128)
    with pytest.raises(ValueError):
        kda.qk_norm_rope(x, x, torch.zeros(4, dtype=torch.int32), torch.zeros(64))
    with pytest.raises(ValueError):
        kda.linear_chunk_fwd(x.unsqueeze(0), x.unsqueeze(0), x.unsqueeze(0), torch.zeros(1, 4, 2))
    with pytest.raises(ValueError):
        kda.linear_recurrent_step(x, x, x, torch.zeros(4, 2), torch.zeros(4, 2, 128, 128))


@pytest.mark.skipif(torch.cuda.is_available(), reason="checks the no-GPU error path")
def test_valid_calls_without_gpu_fail_cleanly(kda):
    assert _chunk(kda.lib) in (6, 8)
    assert _rope(kda.lib) in (6, 8)
    assert ctypes.c_char_p(kda.lib.kda_last_error_string()).value
