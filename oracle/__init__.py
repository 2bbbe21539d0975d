"""fp64 CPU oracle for the KDA forward -- TEST INFRASTRUCTURE ONLY.

Only ``tests/``, ``__graft_entry__.smoke()`` and the ``cpu_baseline`` /
``--impl reference`` legs of ``bench.py`` may import this package.  The CUDA
library never links, loads or calls it, and the two share no code.

Functions and the passages they follow:

* :func:`gate` -- bounded log-decay ``g = g_min * Sigmoid(exp(A_h) z)``
  ("Kimi K3 technical report review" (devpress/CSDN), section 3.2, Eq. 5).
* :func:`recurrence` -- the token-by-token KDA recurrence
  ``S_t = (I - b k k^T) Diag(alpha) S_{t-1} + b k v^T``, ``o_t = S_t^T q_t``
  (same review, section 3.1, Eq. 1; "Kimi K3: architecture, training and
  inference systems" (weigao.cc), section 3.1, product and delta forms).
  Implemented in C (``kda_oracle.c``), double precision, threads over
  (sequence, head) units.
* :func:`explicit_product_form` -- the same recurrence with the transition
  matrix ``(I - b k k^T) Diag(alpha)`` formed explicitly (numpy, tiny sizes).
* :func:`chunked` -- the chunkwise WY/UT form for a chunk size ``C``
  ("Kimi K3 notes" (s1mplewind blog), section "Chunkwise form": M, W, U, the
  state update and the inter/intra-chunk output split), evaluated with explicit
  cumulative decays in fp64 and a library linear solve; tiny sizes only.
* :func:`decode_step` -- one token of the recurrence for many independent
  (sequence, head) states, the decode form.
* :func:`l2_normalize` -- ``x / sqrt(|x|^2 + eps)`` per token and head, the
  L2Norm applied to q and k before the recurrence ("Kimi K3: architecture,
  training and inference systems", section 3.2, the q / k branches; done inside
  the FlashKDA prepare kernel, "Kimi K3 notes", section "FlashKDA", K1).
* :func:`gate_softplus` -- the unbounded gate ``g = -exp(A_h) Softplus(z)`` that
  the bounded one replaced ("Kimi K3 technical report review", section 3.2).
* :func:`output_gate` -- the head-wise RMSNorm of the KDA output times the
  full-rank Sigmoid gate ("Kimi K3 technical report review", section 3.3, Eq. 6;
  the same systems page, section 3.3), without the W_o / W_g projections.
* :func:`causal_conv`, :func:`selective_scan`, :func:`verify_draft` -- the short causal
  convolution, the selective state space scan and the verification of drafted tokens.

Pins: ``tests/test_oracle.py`` checks these against closed forms, special
cases and invariants the pages fix (see that file's docstring).
"""

from __future__ import annotations

import ctypes
import os
import subprocess
from typing import Optional

import numpy as np

_HERE = os.path.dirname(os.path.abspath(__file__))
_SRC = os.path.join(_HERE, "kda_oracle.c")
_BUILD = os.path.join(_HERE, "_build")
_LIB_PATH = os.path.join(_BUILD, "libkda_oracle.so")

_lib_cache: dict = {}


def compile_oracle(src: str = _SRC, out: str = _LIB_PATH) -> str:
    """Compile the C oracle into a shared library (plain gcc, -O2, IEEE fp)."""
    os.makedirs(os.path.dirname(out), exist_ok=True)
    if os.path.exists(out) and os.path.getmtime(out) >= os.path.getmtime(src):
        return out
    tmp = out + f".tmp{os.getpid()}"
    subprocess.check_call(["gcc", "-O2", "-std=c11", "-shared", "-fPIC", "-pthread", src,
                           "-o", tmp, "-lm"])
    os.replace(tmp, out)
    return out


def load(path: Optional[str] = None):
    """Load (building first if needed) the oracle library at ``path``."""
    path = path or compile_oracle()
    if path in _lib_cache:
        return _lib_cache[path]
    lib = ctypes.CDLL(path)
    dp = ctypes.POINTER(ctypes.c_double)
    lib.kda_oracle_gate.argtypes = [dp, dp, ctypes.c_double, ctypes.c_int64, ctypes.c_int,
                                    ctypes.c_int, dp]
    lib.kda_oracle_gate.restype = None
    lib.kda_oracle_recurrence.argtypes = [dp, dp, dp, dp, dp, dp,
                                          ctypes.POINTER(ctypes.c_int64), ctypes.c_int,
                                          ctypes.c_int, ctypes.c_int, ctypes.c_int,
                                          ctypes.c_int, dp, dp, ctypes.c_int]
    lib.kda_oracle_recurrence.restype = ctypes.c_int
    _lib_cache[path] = lib
    return lib


def _f64(x) -> np.ndarray:
    if x is None:
        return None
    if hasattr(x, "detach"):  # torch tensor: exact widening to fp64 on the host
        x = x.detach().to("cpu").double().numpy()
    return np.ascontiguousarray(np.asarray(x, dtype=np.float64))


def _ptr(a):
    if a is None:
        return None
    return a.ctypes.data_as(ctypes.POINTER(ctypes.c_double))


def gate(z, A, g_min: float = -5.0, lib=None) -> np.ndarray:
    """g[t, h, c] = g_min * Sigmoid(exp(A[h]) * z[t, h, c]) in fp64."""
    lib = lib or load()
    z = _f64(z)
    A = _f64(A)
    NT, H, dk = z.shape
    g = np.empty_like(z)
    lib.kda_oracle_gate(_ptr(z), _ptr(A), float(g_min), NT, H, dk, _ptr(g))
    return g


def recurrence(q, k, v, g, beta, h0=None, cu_seqlens=None, form: int = 0,
               n_threads: Optional[int] = None, lib=None):
    """Token-by-token KDA forward.  Returns ``(o, hT)`` as fp64 arrays.

    q, k, g: [NT, H, dk]; v: [NT, H, dv]; beta: [NT, H]; h0: [N, H, dv, dk] or
    None; cu_seqlens: [N+1] (default: one sequence of NT tokens).
    ``form`` 0 = product form, 1 = delta form.
    """
    lib = lib or load()
    q, k, v, g, beta, h0 = (_f64(x) for x in (q, k, v, g, beta, h0))
    NT, H, dk = q.shape
    dv = v.shape[2]
    if cu_seqlens is None:
        cu = np.array([0, NT], dtype=np.int64)
    else:
        if hasattr(cu_seqlens, "detach"):
            cu_seqlens = cu_seqlens.detach().cpu().numpy()
        cu = np.ascontiguousarray(np.asarray(cu_seqlens, dtype=np.int64))
    N = len(cu) - 1
    if h0 is not None:
        assert h0.shape == (N, H, dv, dk), h0.shape
    o = np.zeros((NT, H, dv), dtype=np.float64)
    hT = np.zeros((N, H, dv, dk), dtype=np.float64)
    if n_threads is None:
        n_threads = os.cpu_count() or 1
    rc = lib.kda_oracle_recurrence(_ptr(q), _ptr(k), _ptr(v), _ptr(g), _ptr(beta), _ptr(h0),
                                   cu.ctypes.data_as(ctypes.POINTER(ctypes.c_int64)), N, H, dk,
                                   dv, int(form), _ptr(o), _ptr(hT), int(n_threads))
    if rc != 0:
        raise ValueError("oracle rejected its arguments")
    return o, hT


def decode_step(q, k, v, g, beta, S, n_threads: Optional[int] = None, lib=None):
    """One decode token for N independent sequences.

    q, k, g: [N, H, dk]; v: [N, H, dv]; beta: [N, H]; S: [N, H, dv, dk].
    Returns ``(o [N, H, dv], S_new [N, H, dv, dk])``.
    """
    q = _f64(q)
    N = q.shape[0]
    cu = np.arange(N + 1, dtype=np.int64)
    return recurrence(q, k, v, g, beta, h0=S, cu_seqlens=cu, n_threads=n_threads, lib=lib)


def explicit_product_form(q, k, v, g, beta, h0=None):
    """KDA with the transition matrix formed explicitly (one sequence).

    For each token: ``M_t = (I - b k k^T) @ Diag(exp(g))`` (a dk x dk matrix),
    ``S = M_t @ S + b * outer(k, v)``, ``o_t = S^T q``.  Tiny sizes only.
    Returns ``(o [T, H, dv], hT [H, dv, dk])``.
    """
    q, k, v, g, beta, h0 = (_f64(x) for x in (q, k, v, g, beta, h0))
    T, H, dk = q.shape
    dv = v.shape[2]
    o = np.zeros((T, H, dv))
    hT = np.zeros((H, dv, dk))
    eye = np.eye(dk)
    for h in range(H):
        S = np.zeros((dk, dv)) if h0 is None else h0[h].T.copy()
        for t in range(T):
            kt = k[t, h]
            M = (eye - beta[t, h] * np.outer(kt, kt)) @ np.diag(np.exp(g[t, h]))
            S = M @ S + beta[t, h] * np.outer(kt, v[t, h])
            o[t, h] = S.T @ q[t, h]
        hT[h] = S.T
    return o, hT


def chunked(q, k, v, g, beta, h0=None, cu_seqlens=None, C: int = 64):
    """Chunkwise WY/UT evaluation of KDA in fp64 (brute force, tiny sizes).

    Per chunk [t] of length L <= C, with G the inclusive cumulative sum of g
    inside the chunk and Gamma = exp(G) (row r holds gamma_r = prod_{j<=r} alpha_j):
        A   = StrictTril(Diag(beta) (Gamma*K) (K/Gamma)^T)
        M   = (I + A)^{-1} Diag(beta)
        W   = M (Gamma*K),   U = M V
        Vt  = U - W S                       (the "pseudo-value" term)
        O   = (Gamma*Q) S + Tril((Gamma*Q) (K/Gamma)^T) Vt
        S'  = Diag(gamma_C) S + ((gamma_C/Gamma)*K)^T Vt
    following "Kimi K3 notes" (s1mplewind blog), section "Chunkwise form".
    fp64 holds exp(+-5C) for C <= 64, so no tile references are needed here.
    """
    q, k, v, g, beta, h0 = (_f64(x) for x in (q, k, v, g, beta, h0))
    NT, H, dk = q.shape
    dv = v.shape[2]
    if cu_seqlens is None:
        cu = [0, NT]
    else:
        if hasattr(cu_seqlens, "detach"):
            cu_seqlens = cu_seqlens.detach().cpu().numpy()
        cu = [int(x) for x in cu_seqlens]
    N = len(cu) - 1
    o = np.zeros((NT, H, dv))
    hT = np.zeros((N, H, dv, dk))
    for n in range(N):
        for h in range(H):
            S = np.zeros((dk, dv)) if h0 is None else h0[n, h].T.copy()
            for s in range(cu[n], cu[n + 1], C):
                e = min(s + C, cu[n + 1])
                L = e - s
                K = k[s:e, h]
                Q = q[s:e, h]
                V = v[s:e, h]
                b = beta[s:e, h]
                G = np.cumsum(g[s:e, h], axis=0)
                Gam = np.exp(G)
                Kg, Kn, Qg = Gam * K, K / Gam, Gam * Q
                A = np.tril(np.diag(b) @ Kg @ Kn.T, -1)
                M = np.linalg.solve(np.eye(L) + A, np.diag(b))
                W, U = M @ Kg, M @ V
                Vt = U - W @ S
                o[s:e, h] = Qg @ S + np.tril(Qg @ Kn.T) @ Vt
                gC = Gam[-1]
                S = gC[:, None] * S + (np.exp(G[-1][None, :] - G) * K).T @ Vt
            hT[n, h] = S.T
    return o, hT


def chunk_cumsum(g, cu_seqlens=None, C: int = 64) -> np.ndarray:
    """Running sum of g inside each C-token chunk of each sequence (chunks start
    at cu[n] + C m): the log of the in-chunk cumulative decay Gamma of the
    chunkwise form ("Kimi K3 notes", section "Chunkwise form")."""
    g = _f64(g)
    NT = g.shape[0]
    if cu_seqlens is None:
        cu = [0, NT]
    else:
        if hasattr(cu_seqlens, "detach"):
            cu_seqlens = cu_seqlens.detach().cpu().numpy()
        cu = [int(x) for x in cu_seqlens]
    out = np.zeros_like(g)
    for n in range(len(cu) - 1):
        for s in range(cu[n], cu[n + 1], C):
            e = min(s + C, cu[n + 1])
            out[s:e] = np.cumsum(g[s:e], axis=0)
    return out


def l2_normalize(x, eps: float) -> np.ndarray:
    """``x / sqrt(sum_c x_c^2 + eps)`` over the last axis (one head's channels) in
    fp64.  The pages name the L2Norm without an epsilon; ``eps`` is the caller's."""
    x = _f64(x)
    return x / np.sqrt(np.sum(x * x, axis=-1, keepdims=True) + eps)


def output_gate(o, x, w=None, eps: float = 1e-6) -> np.ndarray:
    """``Sigmoid(x) * w * o / sqrt(mean_c(o_c^2) + eps)`` over the last axis (the dv
    channels of one head) in fp64: the head-wise RMSNorm of the recurrent output
    and the input-dependent full-rank gate, ``x`` being the gate logits W_g x_t.
    ``w`` is the RMSNorm weight over the channels (None: ones)."""
    o, x = _f64(o), _f64(x)
    rms = np.sqrt(np.mean(o * o, axis=-1, keepdims=True) + eps)
    y = o / rms / (1.0 + np.exp(-x))
    if w is not None:
        y = y * _f64(w)
    return y


def gate_softplus(z, A) -> np.ndarray:
    """``g[t, h, c] = -exp(A[h]) * log(1 + exp(z[t, h, c]))`` in fp64 (Softplus as
    ``logaddexp(0, z)``, exact for large |z|)."""
    z, A = _f64(z), _f64(A)
    return -np.exp(A)[None, :, None] * np.logaddexp(0.0, z)


def linear_recurrence(q, k, v, g, h0=None, cu_seqlens=None, scale: float = 1.0, n_advance=None):
    """Linear attention with a decay for each head, token by token in fp64:
    ``S_t = e^{g_t} S_{t-1} + k_t v_t^T``, ``o_t = scale S_t^T q_t`` (KDA without the
    erase and with one decay a head).  q, k [NT, Hk, dk], v [NT, H, dv] (value head h uses
    key head h // (H // Hk)), g [NT, H] or [H], h0 [N, H, dv, dk] or None.  ``n_advance``
    [N]: the returned state is the one after that many tokens of each sequence (None: all;
    the outputs are always of every token).  Returns ``(o, hT)``."""
    q, k, v, g, h0 = (_f64(x) for x in (q, k, v, g, h0))
    NT, H, dv = v.shape
    rep = H // q.shape[1]
    q, k = np.repeat(q, rep, axis=1), np.repeat(k, rep, axis=1)
    g = np.broadcast_to(g, (NT, H))
    if cu_seqlens is None:
        cu = [0, NT]
    else:
        if hasattr(cu_seqlens, "detach"):
            cu_seqlens = cu_seqlens.detach().cpu().numpy()
        cu = [int(x) for x in cu_seqlens]
    N, dk = len(cu) - 1, k.shape[2]
    o, hT = np.zeros((NT, H, dv)), np.zeros((N, H, dv, dk))
    for n in range(N):
        S = np.zeros((H, dv, dk)) if h0 is None else h0[n].copy()
        last = cu[n + 1] - cu[n] if n_advance is None else int(n_advance[n])
        if last == 0:
            hT[n] = S
        for i, t in enumerate(range(cu[n], cu[n + 1])):
            S = np.exp(g[t])[:, None, None] * S + v[t][:, :, None] * k[t][:, None, :]
            o[t] = scale * np.einsum("hvk,hk->hv", S, q[t])
            if i + 1 == last:
                hT[n] = S
    return o, hT


def norm_rope(x, positions, inv_freq, weight=None, eps=1e-6, freq_axis=None, interleaved=False):
    """``x / rms(x) * weight`` over the channels of each head (eps None: x as it is), then
    the rotation of the pairs (i, i + F), or (2i, 2i + 1), by ``positions[axis_i] *
    inv_freq[i]``, as a complex product, fp64.  x [NT, H, D], positions [NT] or
    [n_axes, NT]; channels from 2F on are not rotated."""
    x, inv_freq = _f64(x), _f64(inv_freq)
    pos = _f64(positions)
    F = len(inv_freq)
    axis = np.zeros(F, dtype=int) if freq_axis is None else np.asarray(
        freq_axis.cpu() if hasattr(freq_axis, "cpu") else freq_axis, dtype=int)
    pos = pos.reshape(-1, x.shape[0])
    y = x
    if eps is not None:
        y = y / np.sqrt(np.mean(y * y, axis=-1, keepdims=True) + eps)
        if weight is not None:
            y = y * _f64(weight)
    turn = np.exp(1j * pos[axis].T * inv_freq)[:, None, :]
    out = y.copy()
    lo, hi = (slice(0, 2 * F, 2), slice(1, 2 * F, 2)) if interleaved else (slice(0, F),
                                                                          slice(F, 2 * F))
    z = (y[..., lo] + 1j * y[..., hi]) * turn
    out[..., lo], out[..., hi] = z.real, z.imag
    return out


def _silu(x):
    with np.errstate(over="ignore"):
        return x / (1.0 + np.exp(-x))


def _softplus(x):
    return np.maximum(x, 0.0) + np.log1p(np.exp(-np.abs(x)))


def causal_conv(x, weight, bias=None, state=None, cu_seqlens=None, silu=True, n_advance=None):
    """Short causal depthwise convolution, y_t = act(bias + sum_j w[:, j] x_{t-W+1+j}); the inputs
    before a sequence are state[n] [W-1, C] or zeros.  Returns (y, final state), the latter behind
    the first n_advance[n] tokens of a sequence (None: all)."""
    x, w = _f64(x), _f64(weight)
    W, C = w.shape[1], x.shape[-1]
    cu = [0, x.shape[0]] if cu_seqlens is None else [int(c) for c in cu_seqlens]
    N = len(cu) - 1
    old = np.zeros((N, W - 1, C)) if state is None else _f64(state)
    y, last = np.zeros_like(x), np.zeros((N, W - 1, C))
    for n in range(N):
        rows = np.concatenate([old[n], x[cu[n]:cu[n + 1]]])
        size = cu[n + 1] - cu[n]
        for t in range(size):
            y[cu[n] + t] = np.einsum("wc,cw->c", rows[t:t + W], w)
        adv = size if n_advance is None else min(max(int(n_advance[n]), 0), size)
        last[n] = rows[adv:adv + W - 1]
    if bias is not None:
        y = y + _f64(bias)
    return (_silu(y) if silu else y), last


def selective_scan(x, dt, A, B, C, h0=None, cu_seqlens=None, D=None, z=None, dt_bias=None,
                   softplus=True, n_advance=None):
    """h_t = exp(delta_t A) h_{t-1} + delta_t x_t B_t, y_t = (C_t . h_t + D x_t) SiLU(z_t) token by
    token: x, dt, z [NT, channels], A [channels, S], B, C [NT, G, S], h0 [N, channels, S].
    Returns (y, hT), the latter behind the first n_advance[n] tokens (None: all)."""
    x, dt, A, B, C = _f64(x), _f64(dt), _f64(A), _f64(B), _f64(C)
    nt, ch = x.shape
    per = ch // B.shape[1]
    delta = dt + (0.0 if dt_bias is None else _f64(dt_bias))
    if softplus:
        delta = _softplus(delta)
    cu = [0, nt] if cu_seqlens is None else [int(c) for c in cu_seqlens]
    N = len(cu) - 1
    y, hT = np.zeros_like(x), np.zeros((N,) + A.shape)
    for n in range(N):
        h = np.zeros_like(A) if h0 is None else _f64(h0)[n].copy()
        adv = cu[n + 1] - cu[n] if n_advance is None else int(n_advance[n])
        hT[n] = h
        for t in range(cu[n], cu[n + 1]):
            b, c = np.repeat(B[t], per, axis=0), np.repeat(C[t], per, axis=0)
            h = np.exp(delta[t][:, None] * A) * h + (delta[t] * x[t])[:, None] * b
            y[t] = (c * h).sum(axis=1)
            if t - cu[n] < adv:
                hT[n] = h
    if D is not None:
        y = y + _f64(D) * x
    if z is not None:
        y = y * _silu(_f64(z))
    return y, hT


def verify_draft(draft, q, p, u_accept, u_sample):
    """Accepted drafted tokens and the token behind them, in exact fractions: draft [N][T], q
    [N][T][V], p [N][T+1][V].  Returns (tokens [N][T+1], n_advance [N])."""
    from fractions import Fraction

    p, q = _f64(p), _f64(q)
    N, T1, V = p.shape
    tokens, count = np.full((N, T1), -1, dtype=np.int64), np.zeros(N, dtype=np.int64)

    def whole(w):
        return [int(min(max(float(v), 0.0), 1.0) * 2.0 ** 56) if v > 0 else 0 for v in w]

    for n in range(N):
        k, rejected = 0, False
        while k < T1 - 1 and 0 <= int(draft[n][k]) < V:
            d = int(draft[n][k])
            a, b = float(q[n, k, d]), float(p[n, k, d])
            u = float(u_accept[n][k])
            good = np.isfinite(a) and np.isfinite(b)
            if not (Fraction(u) * Fraction(a) < Fraction(b) if good else u * a < b):
                rejected = True
                break
            k += 1
        w = p[n, k].astype(np.float32)
        with np.errstate(invalid="ignore"):
            rest = whole(w - q[n, k].astype(np.float32)) if rejected else whole(w)
        if sum(rest) == 0:
            rest = whole(w)
        limit = sum(rest) * int(float(u_sample[n]) * 2 ** 24) >> 24
        run, new = 0, 0
        for v, r in enumerate(rest):
            run += r
            if run > limit:
                new = v
                break
        tokens[n, :k] = draft[n][:k]
        tokens[n, k] = new
        count[n] = k + 1
    return tokens, count
