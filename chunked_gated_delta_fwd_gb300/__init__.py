"""GB300 Kimi Delta Attention (KDA) forward -- Python binding of libkda.

A thin ctypes layer over the C ABI in ``include/kda.h``: it checks tensor
dtypes, devices and contiguity, passes ``data_ptr()`` values and the current
CUDA stream, and raises :class:`KdaError` on a non-OK status.  Every step of
the computation runs in the library's CUDA kernels; there is no CPU or
PyTorch fallback, and importing this package fails if ``libkda.so`` has not
been built (``python chunked_gated_delta_fwd_gb300/_build.py``).

Entry points (same names as the C calls, without the ``kda_`` prefix):

* :func:`gate` -- ``g = g_min * Sigmoid(exp(A_h) z)`` (optionally the in-chunk
  running sum),
* :func:`chunk_fwd` -- prefill over whole (packed, variable-length) sequences,
* :func:`recurrent_step` -- one decode token per sequence, state in place,
* :func:`qk_norm_rope` -- per-head RMSNorm of q and k with the rotation by position,
* :func:`linear_chunk_fwd`, :func:`linear_recurrent_step`,
  :func:`linear_recurrent_multi_step` -- linear attention with a decay for each head,
* :func:`causal_conv_fwd`, :func:`causal_conv_step`, :func:`causal_conv_multi_step` -- the short
  causal convolution in front of a recurrent layer,
* :func:`selective_scan_fwd`, :func:`selective_step`, :func:`selective_multi_step` -- the
  selective state space scan,
* :func:`verify_draft` -- how many drafted tokens are kept, the ``n_advance`` of the multi-step
  calls.
"""

from __future__ import annotations

import ctypes
import os
from typing import Optional

import torch

from . import _build

__all__ = ["KdaError", "gate", "chunk_fwd", "chunk_fwd_gated", "chunk_fwd_workspace_size", "recurrent_step",
           "library_path", "lib", "get_device_error", "profile_enable", "profile_collect", "G_MIN", "F32", "BF16", "FP32_CORES", "SEQUENTIAL",
           "segment_chunks", "recurrent_multi_step", "chunk_fwd_checkpointed",
           "chunk_fwd_fused", "gate_softplus", "UNBOUNDED_GATE",
           "output_gate", "SCALAR_GATE", "CHECK_INPUTS", "PRECISE", "selftest_wait_timeout",
           "qk_norm_rope", "linear_chunk_fwd", "linear_chunk_fwd_workspace_size",
           "linear_recurrent_step", "linear_recurrent_multi_step",
           "causal_conv_fwd", "causal_conv_step", "causal_conv_multi_step",
           "selective_scan_fwd", "selective_step", "selective_multi_step", "verify_draft"]

G_MIN = -5.0
F32, BF16 = 0, 1
FP32_CORES = 1  # flag of chunk_fwd: evaluate bf16 inputs on fp32 CUDA cores
SEQUENTIAL = 2  # flag of chunk_fwd: never split a sequence's chain into segments
UNBOUNDED_GATE = 4  # flag of chunk_fwd: any g <= 0 (range-robust fp32-core evaluation)
SCALAR_GATE = 8  # flag of chunk_fwd: g is [..., H], one log-decay per token and head
CHECK_INPUTS = 16  # flag of chunk_fwd: check g and beta against their ranges on the device
PRECISE = 32  # flag of chunk_fwd (bf16 tensor cores): the state update at tf32 precision
_HEAD_DECAY = 64  # flag of the linear-attention calls, set from g's shape
_LINEAR_FLAGS = FP32_CORES | SEQUENTIAL | 0xffff0000  # what a user may give linear_chunk_fwd

_STATUS = {
    0: "KDA_OK", 1: "KDA_ERR_INVALID_ARG", 2: "KDA_ERR_UNSUPPORTED_SHAPE",
    3: "KDA_ERR_UNSUPPORTED_DTYPE", 4: "KDA_ERR_MISALIGNED", 5: "KDA_ERR_WORKSPACE_TOO_SMALL",
    6: "KDA_ERR_CUDA", 7: "KDA_ERR_DEVICE_TIMEOUT", 8: "KDA_ERR_NO_DEVICE",
}


class KdaError(RuntimeError):
    def __init__(self, status: int, message: str):
        super().__init__(f"{_STATUS.get(status, status)}: {message}")
        self.status = status


def library_path() -> str:
    return os.environ.get("KDA_LIBRARY", _build.LIB)


def _load() -> ctypes.CDLL:
    path = library_path()
    if not os.path.exists(path):
        raise ImportError(f"libkda.so not found at {path}; build it with "
                          f"`python chunked_gated_delta_fwd_gb300/_build.py`")
    L = ctypes.CDLL(path)
    vp, i32, i64, f32, sz, u32 = (ctypes.c_void_p, ctypes.c_int, ctypes.c_int64, ctypes.c_float,
                                  ctypes.c_size_t, ctypes.c_uint)
    L.kda_gate.argtypes = [vp, i32, vp, f32, vp, i64, i32, i32, vp, vp, i32, vp]
    L.kda_gate_softplus.argtypes = [vp, i32, vp, vp, i64, i32, i32, vp]
    L.kda_output_gate.argtypes = [vp, i32, vp, vp, f32, vp, i64, i32, i32, vp]
    L.kda_chunk_fwd_workspace_size.argtypes = [i64, i32, i32, i32]
    L.kda_chunk_fwd_workspace_size.restype = sz
    L.kda_chunk_fwd_workspace_size_ex.argtypes = [i64, i32, i32, i32, u32]
    L.kda_chunk_fwd_workspace_size_ex.restype = sz
    L.kda_chunk_fwd.argtypes = [vp, vp, vp, i32, vp, vp, vp, vp, i32, i32, i64, i32, i32, i32, vp,
                                vp, vp, sz, vp]
    L.kda_chunk_fwd_ex.argtypes = L.kda_chunk_fwd.argtypes + [u32]
    L.kda_chunk_fwd_checkpointed.argtypes = (L.kda_chunk_fwd.argtypes[:16] + [vp, i32, i64]
                                             + L.kda_chunk_fwd.argtypes[16:] + [u32])
    L.kda_chunk_fwd_fused.argtypes = [vp, vp, vp, i32, vp, vp, vp, f32, vp, vp, vp, i32, i32, i64,
                                      i32, i32, i32, f32, vp, vp, f32, vp, vp, vp, sz, vp, u32]
    L.kda_chunk_fwd_gated.argtypes = [vp, vp, vp, i32, vp, vp, f32, vp, vp, vp, i32, i32, i64,
                                      i32, i32, i32, vp, vp, vp, sz, vp]
    L.kda_recurrent_step.argtypes = [vp, vp, vp, i32, vp, vp, vp, vp, i32, i32, i32, i32, vp]
    L.kda_recurrent_multi_step.argtypes = [vp, vp, vp, i32, vp, vp, vp, vp, vp, i32, i32, i32,
                                           i32, i32, vp]
    L.kda_qk_norm_rope.argtypes = [vp, vp, i32, vp, vp, f32, vp, i32, vp, vp, i32, i32, vp, vp,
                                   i64, i32, i32, i32, i64, i64, i64, i64, vp]
    L.kda_linear_chunk_fwd_workspace_size.argtypes = [i64, i32, i32, i32, u32]
    L.kda_linear_chunk_fwd_workspace_size.restype = sz
    L.kda_linear_chunk_fwd.argtypes = [vp, vp, vp, i32, vp, f32, vp, vp, i32, i32, i64, i32, i32,
                                       i32, i32, vp, vp, vp, sz, vp, u32]
    L.kda_linear_recurrent_step.argtypes = [vp, vp, vp, i32, vp, f32, vp, vp, i32, i32, i32, i32,
                                            i32, vp, u32]
    L.kda_linear_recurrent_multi_step.argtypes = [vp, vp, vp, i32, vp, f32, vp, vp, vp, i32, i32,
                                                  i32, i32, i32, i32, vp, u32]
    conv = [vp, i32, vp, vp, vp]
    L.kda_causal_conv_fwd.argtypes = conv + [vp, i32, i32, i64, i32, i32, i64, vp, i64, vp, vp, u32]
    L.kda_causal_conv_step.argtypes = conv + [vp, i32, i32, i32, i64, i64, vp, u32]
    L.kda_causal_conv_multi_step.argtypes = conv + [vp, vp, i32, i32, i32, i32, i64, i64, vp, u32]
    scan = [vp, vp, vp, vp, vp, i32, vp, vp, vp]
    L.kda_selective_scan_fwd.argtypes = scan + [vp, vp, i32, i32, i64, i32, i32, i32, i64, i64, i64,
                                                i64, i64, vp, i64, vp, vp, u32]
    L.kda_selective_step.argtypes = scan + [vp, vp, i32, i32, i32, i32, i64, i64, i64, i64, i64,
                                            i64, vp, u32]
    L.kda_selective_multi_step.argtypes = scan + [vp, vp, vp, i32, i32, i32, i32, i32, i64, i64,
                                                  i64, i64, i64, i64, vp, u32]
    L.kda_verify_draft.argtypes = [vp, vp, vp, i32, vp, vp, vp, vp, i32, i32, i32, vp]
    L.kda_selftest_wait_timeout.argtypes = [u32, ctypes.POINTER(i32), vp]
    L.kda_selftest_wait_timeout.restype = ctypes.c_int
    L.kda_last_error_string.restype = ctypes.c_char_p
    L.kda_get_device_error.argtypes = [vp]
    L.kda_version.restype = ctypes.c_char_p
    L.kda_profile_enable.argtypes = [i32]
    L.kda_profile_get.argtypes = [i32, ctypes.POINTER(ctypes.c_char_p), ctypes.POINTER(i32),
                                  ctypes.POINTER(ctypes.c_double)]
    for fn in (L.kda_gate, L.kda_chunk_fwd, L.kda_chunk_fwd_ex, L.kda_chunk_fwd_gated,
               L.kda_recurrent_step, L.kda_recurrent_multi_step, L.kda_get_device_error):
        fn.restype = ctypes.c_int
    return L


lib = _load()


def _check(status: int):
    if status != 0:
        raise KdaError(status, lib.kda_last_error_string().decode())


def _ptr(t: Optional[torch.Tensor]):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream(device) -> ctypes.c_void_p:
    return ctypes.c_void_p(torch.cuda.current_stream(device).cuda_stream)


def _dtype_code(t: torch.Tensor) -> int:
    if t.dtype == torch.bfloat16:
        return BF16
    if t.dtype == torch.float32:
        return F32
    raise TypeError(f"unsupported dtype {t.dtype} (bfloat16 or float32)")


def _need(t: torch.Tensor, name: str, dtype=None, device=None):
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if dtype is not None and t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if device is not None and t.device != device:
        raise ValueError(f"{name} is on {t.device}, expected {device}")


def gate(z: torch.Tensor, A: torch.Tensor, g_min: float = G_MIN, *, out=None,
         with_cumsum: bool = False, cu_seqlens: Optional[torch.Tensor] = None):
    """g = g_min * Sigmoid(exp(A[h]) * z) for z of shape [..., H, 128] (bf16/fp32).

    Returns g (fp32, z's shape), or (g, gcum) with ``with_cumsum`` where gcum is the
    running sum of g inside each 64-token chunk of each sequence.
    """
    _need(z, "z")
    _need(A, "A", torch.float32, z.device)
    H, dk = z.shape[-2], z.shape[-1]
    NT = z.numel() // (H * dk) if z.numel() else 0
    g = out if out is not None else torch.empty(z.shape, dtype=torch.float32, device=z.device)
    _need(g, "out", torch.float32, z.device)
    gcum = torch.empty_like(g) if with_cumsum else None
    if cu_seqlens is not None:
        _need(cu_seqlens, "cu_seqlens", torch.int32, z.device)
    n_seqs = cu_seqlens.numel() - 1 if cu_seqlens is not None else 1
    with torch.cuda.device(z.device):
        _check(lib.kda_gate(_ptr(z), _dtype_code(z), _ptr(A), float(g_min), _ptr(g), NT, H, dk,
                            _ptr(gcum), _ptr(cu_seqlens), n_seqs, _stream(z.device)))
    return (g, gcum) if with_cumsum else g


def output_gate(o: torch.Tensor, gate: torch.Tensor, weight=None, eps: float = 1e-6, *,
                out=None):
    """y = Sigmoid(gate) * weight * o / sqrt(mean(o^2) + eps) over the 128 channels of
    each (token, head); o, gate [..., H, 128] (bf16/fp32, same dtype), weight fp32
    [128] or None.  ``out=o`` works in place."""
    _need(o, "o")
    _need(gate, "gate", o.dtype, o.device)
    if tuple(gate.shape) != tuple(o.shape):
        raise ValueError("gate must have the shape of o")
    if weight is not None:
        _need(weight, "weight", torch.float32, o.device)
    H, dv = o.shape[-2], o.shape[-1]
    NT = o.numel() // (H * dv) if o.numel() else 0
    y = out if out is not None else torch.empty_like(o)
    _need(y, "out", o.dtype, o.device)
    with torch.cuda.device(o.device):
        _check(lib.kda_output_gate(_ptr(o), _dtype_code(o), _ptr(gate), _ptr(weight), float(eps),
                                   _ptr(y), NT, H, dv, _stream(o.device)))
    return y


def gate_softplus(z: torch.Tensor, A: torch.Tensor, *, out=None):
    """The unbounded gate g = -exp(A[h]) * Softplus(z), z [..., H, 128] (bf16/fp32);
    a prefill on it needs the ``UNBOUNDED_GATE`` flag.  Returns g (fp32)."""
    _need(z, "z")
    _need(A, "A", torch.float32, z.device)
    H, dk = z.shape[-2], z.shape[-1]
    NT = z.numel() // (H * dk) if z.numel() else 0
    g = out if out is not None else torch.empty(z.shape, dtype=torch.float32, device=z.device)
    _need(g, "out", torch.float32, z.device)
    with torch.cuda.device(z.device):
        _check(lib.kda_gate_softplus(_ptr(z), _dtype_code(z), _ptr(A), _ptr(g), NT, H, dk,
                                     _stream(z.device)))
    return g


def chunk_fwd_workspace_size(n_tokens: int, n_seqs: int, H: int, dtype=torch.bfloat16,
                             flags: int = 0) -> int:
    code = BF16 if dtype == torch.bfloat16 else F32
    return int(lib.kda_chunk_fwd_workspace_size_ex(int(n_tokens), int(n_seqs), int(H), code,
                                                   int(flags)))


def segment_chunks(n: int) -> int:
    """Flag bits forcing chain segments of n chunks (KDA_CHUNK_SEGMENT_CHUNKS)."""
    return (int(n) & 0xFFFF) << 16


def chunk_fwd(q, k, v, g, beta, h0=None, cu_seqlens=None, *, output_final_state=True,
              workspace=None, flags: int = 0, out=None, final_state_out=None):
    """KDA prefill over whole sequences.

    q, k: [B, T, H, 128] or packed [T, H, 128] (with ``cu_seqlens``), bf16 or fp32;
    v like q; g: same shape, fp32 log-decays in [-5, 0] (with ``flags`` holding
    ``SCALAR_GATE``: [..., H], one per token and head); beta: [..., H] (dtype of q);
    h0: [N, H, 128, 128] fp32 (the state stored transposed, [dv][dk]) or None;
    cu_seqlens: int32 [N+1] on the device, or None for B sequences of length T.
    Returns ``(o, hT)`` with o like v and hT [N, H, 128, 128] fp32 (None if not asked).
    """
    _need(g, "g", torch.float32, q.device)
    c = _chunk_setup(q, k, v, beta, h0, cu_seqlens, output_final_state, workspace, flags, out,
                     final_state_out)
    with torch.cuda.device(q.device):
        _check(lib.kda_chunk_fwd_ex(_ptr(q), _ptr(k), _ptr(v), c["dt"], _ptr(g), _ptr(beta),
                                    _ptr(h0), _ptr(cu_seqlens), c["N"], c["B"], c["T"], c["H"],
                                    c["dk"], c["dv"], _ptr(c["o"]), _ptr(c["hT"]),
                                    _ptr(c["ws"]), c["ws"].numel(), _stream(q.device),
                                    int(flags)))
    return c["o"], c["hT"]


def chunk_fwd_checkpointed(q, k, v, g, beta, h0=None, cu_seqlens=None, *,
                           ckpt_tokens: int = 512, ckpt_capacity=None, ckpt_out=None,
                           output_final_state=True, workspace=None, flags: int = 0, out=None,
                           final_state_out=None):
    """``chunk_fwd`` that also returns the state after every ``ckpt_tokens`` tokens of
    each sequence (bf16, tensor-core path).  Sequence n contributes
    floor(len_n / ckpt_tokens) checkpoints, stacked in sequence order into
    ``ckpt`` [n_ckpt, H, 128, 128] fp32 (layout of hT).  ``ckpt_capacity`` (slots to
    allocate) defaults to the exact count, read from ``cu_seqlens`` on the host.
    Returns ``(o, hT, ckpt)``."""
    _need(g, "g", torch.float32, q.device)
    c = _chunk_setup(q, k, v, beta, h0, cu_seqlens, output_final_state, workspace, flags, out,
                     final_state_out)
    if ckpt_capacity is None:
        if ckpt_out is not None:
            ckpt_capacity = ckpt_out.shape[0]
        elif cu_seqlens is None:
            ckpt_capacity = c["B"] * (c["T"] // int(ckpt_tokens))
        else:
            lens = torch.diff(cu_seqlens.to("cpu", torch.int64))
            ckpt_capacity = int((lens.clamp(min=0) // int(ckpt_tokens)).sum())
    ck = ckpt_out if ckpt_out is not None else torch.empty(
        (int(ckpt_capacity), c["H"], c["dv"], c["dk"]), dtype=torch.float32, device=q.device)
    _need(ck, "ckpt_out", torch.float32, q.device)
    if ck.shape[0] < int(ckpt_capacity):
        raise ValueError(f"ckpt_out holds {ck.shape[0]} < {ckpt_capacity} checkpoints")
    with torch.cuda.device(q.device):
        _check(lib.kda_chunk_fwd_checkpointed(
            _ptr(q), _ptr(k), _ptr(v), c["dt"], _ptr(g), _ptr(beta), _ptr(h0),
            _ptr(cu_seqlens), c["N"], c["B"], c["T"], c["H"], c["dk"], c["dv"], _ptr(c["o"]),
            _ptr(c["hT"]), _ptr(ck) if int(ckpt_capacity) > 0 else None, int(ckpt_tokens),
            int(ckpt_capacity), _ptr(c["ws"]), c["ws"].numel(), _stream(q.device), int(flags)))
    return c["o"], c["hT"], ck


def chunk_fwd_fused(q, k, v, beta, h0=None, cu_seqlens=None, *, g=None, z=None, A=None,
                    g_min: float = -5.0, qk_l2_eps=None, out_gate=None, out_norm_weight=None,
                    out_norm_eps: float = 1e-6, output_final_state=True, workspace=None,
                    flags: int = 0, out=None, final_state_out=None):
    """bf16 prefill with the prologue and epilogue fused: exactly one of ``g`` (fp32
    log-decays) and ``z`` + ``A`` (gate computed in-kernel); ``qk_l2_eps`` (None: q, k
    used as given) L2-normalises q and k per token and head; ``out_gate`` [..., H,
    128] (dtype of q) applies o <- Sigmoid(out_gate) * w * o / rms(o) per head, with
    ``out_norm_weight`` fp32 [128] (None: ones).  Returns ``(o, hT)``."""
    if (g is None) == (z is None):
        raise ValueError("give exactly one of g and z")
    if g is not None:
        _need(g, "g", torch.float32, q.device)
    else:
        _need(z, "z", q.dtype, q.device)
        _need(A, "A", torch.float32, q.device)
    if out_gate is not None:
        _need(out_gate, "out_gate", q.dtype, q.device)
        if tuple(out_gate.shape) != tuple(v.shape):
            raise ValueError(f"out_gate must have the shape of v {tuple(v.shape)}")
    if out_norm_weight is not None:
        _need(out_norm_weight, "out_norm_weight", torch.float32, q.device)
    c = _chunk_setup(q, k, v, beta, h0, cu_seqlens, output_final_state, workspace, flags, out,
                     final_state_out)
    with torch.cuda.device(q.device):
        _check(lib.kda_chunk_fwd_fused(
            _ptr(q), _ptr(k), _ptr(v), c["dt"], _ptr(g), _ptr(z), _ptr(A), float(g_min),
            _ptr(beta), _ptr(h0), _ptr(cu_seqlens), c["N"], c["B"], c["T"], c["H"], c["dk"],
            c["dv"], -1.0 if qk_l2_eps is None else float(qk_l2_eps), _ptr(out_gate),
            _ptr(out_norm_weight), float(out_norm_eps), _ptr(c["o"]), _ptr(c["hT"]),
            _ptr(c["ws"]), c["ws"].numel(), _stream(q.device), int(flags)))
    return c["o"], c["hT"]


def chunk_fwd_gated(q, k, v, z, A, beta, h0=None, cu_seqlens=None, *, g_min: float = -5.0,
                    output_final_state=True, workspace=None, out=None, final_state_out=None):
    """KDA prefill with the bounded gate g = g_min * Sigmoid(exp(A_h) z) evaluated
    inside the chunk kernels (g is never materialised).  bf16 only; z like k,
    A fp32 [H].  Everything else as ``chunk_fwd``."""
    _need(z, "z", q.dtype, q.device)
    _need(A, "A", torch.float32, q.device)
    c = _chunk_setup(q, k, v, beta, h0, cu_seqlens, output_final_state, workspace, 0, out,
                     final_state_out)
    with torch.cuda.device(q.device):
        _check(lib.kda_chunk_fwd_gated(_ptr(q), _ptr(k), _ptr(v), c["dt"], _ptr(z), _ptr(A),
                                       float(g_min), _ptr(beta), _ptr(h0), _ptr(cu_seqlens),
                                       c["N"], c["B"], c["T"], c["H"], c["dk"], c["dv"],
                                       _ptr(c["o"]), _ptr(c["hT"]), _ptr(c["ws"]),
                                       c["ws"].numel(), _stream(q.device)))
    return c["o"], c["hT"]


def _chunk_setup(q, k, v, beta, h0, cu_seqlens, output_final_state, workspace, flags, out,
                 final_state_out):
    """Checks the chunk inputs and allocates the outputs and the workspace."""
    dev = q.device
    for name, t in (("q", q), ("k", k), ("v", v), ("beta", beta)):
        _need(t, name, q.dtype, dev)
    dt = _dtype_code(q)
    H, dk, dv = q.shape[-2], q.shape[-1], v.shape[-1]
    if cu_seqlens is not None:
        _need(cu_seqlens, "cu_seqlens", torch.int32, dev)
        N = cu_seqlens.numel() - 1
        B, T = 1, q.numel() // (H * dk)
        if q.dim() == 4 and q.shape[0] != 1:
            raise ValueError("with cu_seqlens, q must be packed as [1, NT, H, D] or [NT, H, D]")
    else:
        if q.dim() != 4:
            raise ValueError("q must be [B, T, H, D] without cu_seqlens")
        B, T = q.shape[0], q.shape[1]
        N = B
    NT = B * T if cu_seqlens is None else T
    if h0 is not None:
        _need(h0, "h0", torch.float32, dev)
        if tuple(h0.shape) != (N, H, dv, dk):
            raise ValueError(f"h0 must be [{N}, {H}, {dv}, {dk}], got {tuple(h0.shape)}")
    o = out if out is not None else torch.empty(v.shape, dtype=v.dtype, device=dev)
    _need(o, "out", v.dtype, dev)
    hT = None
    if output_final_state:
        hT = final_state_out if final_state_out is not None else torch.empty(
            (N, H, dv, dk), dtype=torch.float32, device=dev)
        _need(hT, "final_state_out", torch.float32, dev)
    need = chunk_fwd_workspace_size(NT, N, H, q.dtype, flags)
    if workspace is None:
        workspace = torch.empty(max(need, 1), dtype=torch.uint8, device=dev)
    _need(workspace, "workspace", torch.uint8, dev)
    return dict(dt=dt, N=N, B=B, T=T, H=H, dk=dk, dv=dv, o=o, hT=hT, ws=workspace)


def recurrent_step(q, k, v, g, beta, S, *, out=None):
    """One decode token: q, k, v [N, H, 128] (bf16/fp32), g [N, H, 128] fp32,
    beta [N, H], S [N, H, 128, 128] fp32 updated in place.  Returns o [N, H, 128]."""
    dev = q.device
    for name, t in (("q", q), ("k", k), ("v", v), ("beta", beta)):
        _need(t, name, q.dtype, dev)
    _need(g, "g", torch.float32, dev)
    _need(S, "S", torch.float32, dev)
    N, H, dk = q.shape
    dv = v.shape[-1]
    o = out if out is not None else torch.empty(v.shape, dtype=v.dtype, device=dev)
    _need(o, "out", v.dtype, dev)
    with torch.cuda.device(dev):
        _check(lib.kda_recurrent_step(_ptr(q), _ptr(k), _ptr(v), _dtype_code(q), _ptr(g),
                                      _ptr(beta), _ptr(S), _ptr(o), N, H, dk, dv, _stream(dev)))
    return o


def recurrent_multi_step(q, k, v, g, beta, S, n_advance=None, *, out=None,
                         return_outputs=True):
    """T tokens per sequence: q, k, v [N, T, H, 128] (bf16/fp32), g [N, T, H, 128]
    fp32, beta [N, T, H], S [N, H, 128, 128] fp32 advanced in place by n_advance[n]
    tokens (int32 [N] on the device; None = all T).  Returns o [N, T, H, 128] (the
    outputs of all T tokens), or None when return_outputs is False."""
    dev = q.device
    for name, t in (("q", q), ("k", k), ("v", v), ("beta", beta)):
        _need(t, name, q.dtype, dev)
    _need(g, "g", torch.float32, dev)
    _need(S, "S", torch.float32, dev)
    if n_advance is not None:
        _need(n_advance, "n_advance", torch.int32, dev)
    N, T, H, dk = q.shape
    dv = v.shape[-1]
    o = None
    if return_outputs:
        o = out if out is not None else torch.empty(v.shape, dtype=v.dtype, device=dev)
        _need(o, "out", v.dtype, dev)
    with torch.cuda.device(dev):
        _check(lib.kda_recurrent_multi_step(_ptr(q), _ptr(k), _ptr(v), _dtype_code(q), _ptr(g),
                                            _ptr(beta), _ptr(S), _ptr(o), _ptr(n_advance), N, T,
                                            H, dk, dv, _stream(dev)))
    return o


def _call(fn, dev, *args, tail=()):
    """``fn(*args, stream, *tail)`` with ``dev`` current, on its current stream; raises on an
    error.  (Small calls are bound by what happens here: the device is switched only if it
    has to be, pointers and the stream go over as plain integers.)"""
    index = dev.index
    if index == torch._C._cuda_getDevice():
        status = fn(*args, torch._C._cuda_getCurrentRawStream(index), *tail)
    else:
        with torch.cuda.device(dev):
            status = fn(*args, torch._C._cuda_getCurrentRawStream(index), *tail)
    if status != 0:
        raise KdaError(status, lib.kda_last_error_string().decode())


def _addr(t):
    return None if t is None else t.data_ptr()


def _token_stride(t: torch.Tensor, name: str) -> int:
    """Elements between the tokens of a [..., H, 128] tensor whose heads are contiguous
    and whose leading dimensions step as one (a slice of a packed projection has more
    elements a token than its own)."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    shape = t.shape
    if len(shape) < 3:
        raise ValueError(f"{name} must be [..., H, 128]")
    H, d = shape[-2:]
    if t.is_contiguous():
        return H * d
    step = expect = None
    for size, stride in zip(reversed(shape[:-2]), reversed(t.stride()[:-2])):
        if size == 1:
            continue
        if step is None:
            step = stride
        elif stride != expect:
            raise ValueError(f"{name}: the tokens must be one stride apart")
        expect = stride * size
    if (d > 1 and t.stride(-1) != 1) or (H > 1 and t.stride(-2) != d):
        raise ValueError(f"{name}: the heads of a token must be contiguous")
    return H * d if step is None else step


def qk_norm_rope(q, k, positions, inv_freq, *, q_weight=None, k_weight=None, eps=1e-6,
                 freq_axis=None, interleaved: bool = False, q_out=None, k_out=None):
    """Per-head RMSNorm of q and k and the rotation by position, in one pass.

    q [..., Hq, 128], k [..., Hk, 128] (bf16/fp32, the same leading dimensions); both may be
    slices of a packed projection (heads contiguous, tokens one stride apart).  ``eps`` >= 0, or
    None to turn the norm off; ``q_weight``/``k_weight`` fp32 [128] or None.  ``positions`` int32
    [...] (the leading dimensions of q), or [n_axes, ...] with ``freq_axis`` int32 [n_freq],
    the axis of every frequency.  ``inv_freq`` fp32 [n_freq], n_freq a multiple of 8 up to 64:
    the first 2 n_freq channels turn, as pairs (i, i + n_freq) or, ``interleaved``, (2i, 2i+1).
    Returns ``(q_out, k_out)``; ``q_out=q, k_out=k`` works in place.
    """
    if eps is None:
        eps = -1.0  # the library's sign for no norm, which is not taken from a caller
    elif not eps >= 0:
        raise ValueError(f"eps must be 0 or above, or None for no norm; got {eps}")
    sq, sk = _token_stride(q, "q"), _token_stride(k, "k")
    dev, shape, shape_k = q.device, q.shape, k.shape
    lead = tuple(shape[:-2])
    H, d = shape[-2:]
    Hk, dk = shape_k[-2:]
    if k.device != dev or k.dtype != q.dtype:
        raise ValueError("q and k must have one dtype and device")
    if shape_k[:-2] != lead or dk != d:
        raise ValueError(f"k must be {lead} + (Hk, {d}), got {tuple(shape_k)}")
    dt = _dtype_code(q)
    _need(positions, "positions", torch.int32, dev)
    _need(inv_freq, "inv_freq", torch.float32, dev)
    n_axes, n_freq, at = 1, inv_freq.numel(), positions.shape
    if at != lead:
        if len(at) < 1 or at[1:] != lead:
            raise ValueError(f"positions must be {lead} or (n_axes,) + {lead}, got {tuple(at)}")
        n_axes = at[0]
    if freq_axis is not None:
        _need(freq_axis, "freq_axis", torch.int32, dev)
        if freq_axis.numel() != n_freq:
            raise ValueError("freq_axis must have one entry a frequency")
    for name, w in (("q_weight", q_weight), ("k_weight", k_weight)):
        if w is not None:
            _need(w, name, torch.float32, dev)
            if w.numel() != d:
                raise ValueError(f"{name} must have {d} entries")
    soq, sok = H * d, Hk * d
    if q_out is None:
        q_out = torch.empty_like(q, memory_format=torch.contiguous_format)
    else:
        soq = _rope_out(q_out, q, "q_out")
    if k_out is None:
        k_out = torch.empty_like(k, memory_format=torch.contiguous_format)
    else:
        sok = _rope_out(k_out, k, "k_out")
    nt = 1
    for x in lead:
        nt *= x
    _call(lib.kda_qk_norm_rope, dev, q.data_ptr(), k.data_ptr(), dt, _addr(q_weight),
          _addr(k_weight), float(eps), positions.data_ptr(), n_axes,
          _addr(freq_axis), inv_freq.data_ptr(), n_freq, 1 if interleaved else 0,
          q_out.data_ptr(), k_out.data_ptr(), nt, H, Hk, d, sq, sk, soq, sok)
    return q_out, k_out


def _rope_out(y, x, name):
    if not isinstance(y, torch.Tensor) or y.shape != x.shape or y.dtype != x.dtype \
            or y.device != x.device:
        raise ValueError(f"{name} must have the shape, dtype and device of its input")
    return _token_stride(y, name)


def _linear_inputs(q, k, v, g, lead):
    """Checks what the linear-attention calls share: q, k ``lead`` + [Hk, dk], v ``lead``
    + [H, dv], g ``lead`` + [H] or [H].  Returns (dtype code, H, Hk, dk, dv, flag of g)."""
    dev, dtype = q.device, q.dtype
    _need(q, "q", dtype, dev)
    _need(k, "k", dtype, dev)
    _need(v, "v", dtype, dev)
    _need(g, "g", torch.float32, dev)
    dt = _dtype_code(q)
    qs, vs, gs = q.shape, v.shape, g.shape
    if not lead or len(vs) != len(lead) + 2:
        raise ValueError(f"q and v must be [..., heads, 128], got {tuple(qs)} and {tuple(vs)}")
    Hk, dk = qs[-2:]
    H, dv = vs[-2:]
    if k.shape != qs:
        raise ValueError(f"k must have the shape of q {tuple(qs)}, got {tuple(k.shape)}")
    if vs[:-2] != lead:
        raise ValueError(f"v must be {lead} + (H, dv), got {tuple(vs)}")
    if gs == lead + (H,):
        return dt, H, Hk, dk, dv, 0
    if gs == (H,):
        return dt, H, Hk, dk, dv, _HEAD_DECAY
    raise ValueError(f"g must be {lead + (H,)} or ({H},), got {tuple(gs)}")


def _like(t, name, shape, dtype, device, given=False):
    """``t`` checked against what a result needs, or (unless it has to be ``given``) a new
    tensor."""
    if t is None and not given:
        return torch.empty(shape, dtype=dtype, device=device)
    _need(t, name, dtype, device)
    if t.shape != shape:
        raise ValueError(f"{name} must be {tuple(shape)}, got {tuple(t.shape)}")
    return t


def linear_chunk_fwd_workspace_size(n_tokens: int, n_seqs: int, H: int, dtype=torch.bfloat16,
                                    flags: int = 0) -> int:
    code = BF16 if dtype == torch.bfloat16 else F32
    return int(lib.kda_linear_chunk_fwd_workspace_size(int(n_tokens), int(n_seqs), int(H), code,
                                                       int(flags)))


def linear_chunk_fwd(q, k, v, g, h0=None, cu_seqlens=None, *, scale: float = 1.0,
                     output_final_state=True, workspace=None, flags: int = 0, out=None,
                     final_state_out=None):
    """Prompt pass of linear attention with a decay for each head,
    ``S_t = e^{g_t} S_{t-1} + k_t v_t^T``, ``o_t = scale S_t^T q_t``.

    q, k [B, T, Hk, 128] or packed [NT, Hk, 128] (with ``cu_seqlens``), v [..., H, 128], H a
    multiple of Hk (value head h uses key head h // (H // Hk)); bf16 or fp32.  g fp32
    log-decays <= 0, [..., H] (one a token and head) or [H].  h0, cu_seqlens, outputs and
    ``workspace`` as :func:`chunk_fwd`; ``flags``: ``FP32_CORES``, ``SEQUENTIAL`` and
    ``segment_chunks(n)`` (segments of n 128-token chunks).  ``out`` must not overlap an input;
    ``final_state_out`` may be h0.  bf16 inputs run on the tensor cores, where scores and the
    state that q meets are rounded to bf16 and what a token adds to the state keeps 16 bits
    (hT 4e-6 off); ``FP32_CORES`` keeps fp32 sums throughout (2e-7) at some ten times the time.
    Returns ``(o, hT)``; hT is the S of :func:`linear_recurrent_step`.
    """
    if int(flags) & ~_LINEAR_FLAGS:
        raise ValueError(f"flags 0x{int(flags):x}: only FP32_CORES, SEQUENTIAL and segment_chunks(n)")
    lead = tuple(q.shape[:-2])
    dt, H, Hk, dk, dv, fl = _linear_inputs(q, k, v, g, lead)
    dev = q.device
    if cu_seqlens is not None:
        _need(cu_seqlens, "cu_seqlens", torch.int32, dev)
        if len(lead) not in (1, 2) or (len(lead) == 2 and lead[0] != 1):
            raise ValueError("with cu_seqlens, q must be packed as [1, NT, Hk, D] or [NT, Hk, D]")
        N, B, T = cu_seqlens.numel() - 1, 1, lead[-1]
        NT = T
    else:
        if len(lead) != 2:
            raise ValueError("q must be [B, T, Hk, D] without cu_seqlens")
        B, T = lead
        N, NT = B, B * T
    if h0 is not None:
        _need(h0, "h0", torch.float32, dev)
        if tuple(h0.shape) != (N, H, dv, dk):
            raise ValueError(f"h0 must be [{N}, {H}, {dv}, {dk}], got {tuple(h0.shape)}")
    o = torch.empty_like(v) if out is None else _like(out, "out", v.shape, v.dtype, dev)
    hT = None
    if output_final_state:
        hT = _like(final_state_out, "final_state_out", (N, H, dv, dk), torch.float32, dev)
    fl |= int(flags)
    if workspace is None:
        if dev.index == torch._C._cuda_getDevice():  # (the size depends on the SM count)
            need = lib.kda_linear_chunk_fwd_workspace_size(NT, N, H, dt, fl)
        else:
            with torch.cuda.device(dev):
                need = lib.kda_linear_chunk_fwd_workspace_size(NT, N, H, dt, fl)
        workspace = torch.empty(max(need, 1), dtype=torch.uint8, device=dev)
    else:
        _need(workspace, "workspace", torch.uint8, dev)
    _call(lib.kda_linear_chunk_fwd, dev, q.data_ptr(), k.data_ptr(), v.data_ptr(), dt,
          g.data_ptr(), float(scale), _addr(h0), _addr(cu_seqlens), N, B, T, H, Hk, dk, dv,
          o.data_ptr(), _addr(hT), workspace.data_ptr(), workspace.numel(), tail=(fl,))
    return o, hT


def linear_recurrent_step(q, k, v, g, S, *, scale: float = 1.0, out=None):
    """One token of :func:`linear_chunk_fwd`'s recurrence: q, k [N, Hk, 128], v [N, H, 128]
    (bf16/fp32), g fp32 [N, H] or [H], S [N, H, 128, 128] fp32 updated in place.
    Returns o [N, H, 128]."""
    if q.dim() != 3:
        raise ValueError(f"q must be [N, Hk, D], got {tuple(q.shape)}")
    N, dev = q.shape[0], q.device
    dt, H, Hk, dk, dv, fl = _linear_inputs(q, k, v, g, (N,))
    _like(S, "S", (N, H, dv, dk), torch.float32, dev, given=True)
    o = torch.empty_like(v) if out is None else _like(out, "out", v.shape, v.dtype, dev)
    _call(lib.kda_linear_recurrent_step, dev, q.data_ptr(), k.data_ptr(), v.data_ptr(), dt,
          g.data_ptr(), float(scale), S.data_ptr(), o.data_ptr(), N, H, Hk, dk, dv, tail=(fl,))
    return o


def linear_recurrent_multi_step(q, k, v, g, S, n_advance=None, *, scale: float = 1.0, out=None,
                                return_outputs=True):
    """T <= 16 tokens per sequence: q, k [N, T, Hk, 128], v [N, T, H, 128] (bf16/fp32), g fp32
    [N, T, H] or [H], S [N, H, 128, 128] fp32 advanced in place by n_advance[n] tokens
    (int32 [N] on the device; None = all T).  Returns o [N, T, H, 128] (the outputs of all T
    tokens), or None when return_outputs is False."""
    if q.dim() != 4:
        raise ValueError(f"q must be [N, T, Hk, D], got {tuple(q.shape)}")
    N, T, dev = q.shape[0], q.shape[1], q.device
    dt, H, Hk, dk, dv, fl = _linear_inputs(q, k, v, g, (N, T))
    _like(S, "S", (N, H, dv, dk), torch.float32, dev, given=True)
    if n_advance is not None:
        _need(n_advance, "n_advance", torch.int32, dev)
        if n_advance.numel() != N:
            raise ValueError(f"n_advance must have {N} entries")
    o = _like(out, "out", v.shape, v.dtype, dev) if return_outputs else None
    _call(lib.kda_linear_recurrent_multi_step, dev, q.data_ptr(), k.data_ptr(), v.data_ptr(), dt,
          g.data_ptr(), float(scale), S.data_ptr(), _addr(o), _addr(n_advance), N, T, H, Hk, dk,
          dv, tail=(fl,))
    return o


def _row_stride(t: torch.Tensor, name: str, tail: tuple, dtype, device) -> int:
    """Elements between the tokens of a [..., *tail] tensor whose tokens are contiguous in
    themselves and one stride apart (a slice of a packed projection has more elements a token
    than its own); ``t`` is checked on the way."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.device != device:
        raise ValueError(f"{name} is on {t.device}, expected {device}")
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    shape, k = t.shape, len(tail)
    dims = len(shape)
    if dims <= k or shape[dims - k:] != tail:
        raise ValueError(f"{name} must be [..., {', '.join(map(str, tail))}], got {tuple(shape)}")
    row = tail[0] if k == 1 else tail[0] * tail[1]
    stride = t.stride()
    if dims == k + 1 and stride[-1] == 1 and (k == 1 or tail[0] == 1 or stride[1] == tail[1]):
        return row if shape[0] == 1 else stride[0]  # (one leading dimension, most calls)
    if t.is_contiguous():
        return row
    inner = 1
    for i in range(dims - 1, dims - 1 - k, -1):
        if stride[i] != inner and shape[i] > 1:
            raise ValueError(f"{name}: the elements of a token must be contiguous")
        inner *= shape[i]
    step = expect = None
    for i in range(dims - 1 - k, -1, -1):
        if shape[i] == 1:
            continue
        if step is None:
            step = stride[i]
        elif stride[i] != expect:
            raise ValueError(f"{name}: the tokens must be one stride apart")
        expect = stride[i] * shape[i]
    return row if step is None else step


def _count(n, name):
    """``n``, which goes over as a 32-bit integer (ctypes would cut it off)."""
    if n > 0x7fffffff:
        raise ValueError(f"{name}: {n} is more than 2^31 - 1")
    return n


def _tokens(x, name):
    """(shape, dtype, device, dtype code) of a call's first tensor, tokens of channels."""
    if not isinstance(x, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if not x.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    shape, dtype = x.shape, x.dtype
    if len(shape) < 2:
        raise ValueError(f"{name} must be [..., channels], got {tuple(shape)}")
    _count(max(shape), name)
    return shape, dtype, x.device, _dtype_code(x)


def _packed(lead, cu_seqlens, dev, name):
    """(N, B, T) of a prompt call whose tokens have the leading dimensions ``lead``."""
    if cu_seqlens is not None:
        _need(cu_seqlens, "cu_seqlens", torch.int32, dev)
        if len(lead) not in (1, 2) or (len(lead) == 2 and lead[0] != 1):
            raise ValueError(f"with cu_seqlens, {name} must be packed as [1, NT, C] or [NT, C]")
        return _count(cu_seqlens.numel() - 1, "cu_seqlens"), 1, lead[-1]
    if len(lead) != 2:
        raise ValueError(f"{name} must be [B, T, C] without cu_seqlens")
    return lead[0], lead[0], lead[1]


def _conv_inputs(x, weight, bias):
    """(row stride, shape, dtype, device, C, W, dtype code) of a convolution's checked inputs."""
    shape, dtype, dev, code = _tokens(x, "x")
    C = shape[-1]
    sx = _row_stride(x, "x", (C,), dtype, dev)
    _need(weight, "weight", torch.float32, dev)
    ws = weight.shape
    if len(ws) != 2 or ws[0] != C:
        raise ValueError(f"weight must be [{C}, W], got {tuple(ws)}")
    if bias is not None:
        _need(bias, "bias", torch.float32, dev)
        if bias.shape != (C,):
            raise ValueError(f"bias must be [{C}], got {tuple(bias.shape)}")
    return sx, shape, dtype, dev, C, _count(ws[1], "weight"), code


def _rows_out(out, x, C):
    """``out`` (or a new contiguous tensor) of x's shape, and its token stride."""
    if out is None:
        return torch.empty_like(x, memory_format=torch.contiguous_format), C
    s = _row_stride(out, "out", (C,), x.dtype, x.device)
    if out.shape != x.shape:
        raise ValueError(f"out must be {tuple(x.shape)}, got {tuple(out.shape)}")
    return out, s


def causal_conv_fwd(x, weight, bias=None, state=None, cu_seqlens=None, *, silu: bool = True,
                    output_final_state=True, out=None, final_state_out=None):
    """Short causal depthwise convolution over whole sequences,
    ``y_t[c] = act(bias[c] + sum_j weight[c, j] x_{t-W+1+j}[c])``, act SiLU or (``silu=False``)
    the identity.

    x [B, T, C] or packed [NT, C] (with ``cu_seqlens``), bf16 or fp32, C a multiple of 8; its
    tokens may be slices of a packed projection.  weight fp32 [C, W], W 2 to 4, bias fp32 [C].
    state [N, W-1, C] (dtype of x): the inputs before each sequence, oldest first, or None.
    ``out`` must not overlap x; ``final_state_out`` may be ``state``.
    Returns ``(y, final_state)``; final_state (None if not asked) is the state of
    :func:`causal_conv_step`.
    """
    sx, shape, dtype, dev, C, W, dt = _conv_inputs(x, weight, bias)
    N, B, T = _packed(shape[:-1], cu_seqlens, dev, "x")
    kept = (N, W - 1, C)
    if state is not None:
        _like(state, "state", kept, dtype, dev)
    last = _like(final_state_out, "final_state_out", kept, dtype, dev) \
        if output_final_state else None
    y, sy = _rows_out(out, x, C)
    _call(lib.kda_causal_conv_fwd, dev, x.data_ptr(), dt, weight.data_ptr(), _addr(bias),
          _addr(state), _addr(cu_seqlens), N, B, T, C, W, sx, y.data_ptr(), sy, _addr(last),
          tail=(1 if silu else 0,))
    return y, last


def causal_conv_step(x, weight, state, bias=None, *, silu: bool = True, out=None):
    """One new token of :func:`causal_conv_fwd` for N sequences: x [N, C], state [N, W-1, C]
    updated in place.  Returns y [N, C]."""
    sx, shape, dtype, dev, C, W, dt = _conv_inputs(x, weight, bias)
    if len(shape) != 2:
        raise ValueError(f"x must be [N, C], got {tuple(shape)}")
    N = shape[0]
    _like(state, "state", (N, W - 1, C), dtype, dev, given=True)
    y, sy = _rows_out(out, x, C)
    _call(lib.kda_causal_conv_step, dev, x.data_ptr(), dt, weight.data_ptr(), _addr(bias),
          state.data_ptr(), y.data_ptr(), N, C, W, sx, sy, tail=(1 if silu else 0,))
    return y


def _advance(n_advance, N, dev):
    if n_advance is not None:
        _need(n_advance, "n_advance", torch.int32, dev)
        if n_advance.numel() != N:
            raise ValueError(f"n_advance must have {N} entries")
    return _addr(n_advance)


def causal_conv_multi_step(x, weight, state, n_advance=None, bias=None, *, silu: bool = True,
                           out=None, return_outputs=True):
    """T <= 16 new tokens a sequence: x [N, T, C], state [N, W-1, C] left as it is behind the
    first n_advance[n] tokens (int32 [N] on the device; None = all T).  Returns y [N, T, C] (of
    all T tokens), or None when return_outputs is False."""
    sx, shape, dtype, dev, C, W, dt = _conv_inputs(x, weight, bias)
    if len(shape) != 3:
        raise ValueError(f"x must be [N, T, C], got {tuple(shape)}")
    N, T, _ = shape
    _like(state, "state", (N, W - 1, C), dtype, dev, given=True)
    adv = _advance(n_advance, N, dev)
    y, sy = _rows_out(out, x, C) if return_outputs else (None, C)
    _call(lib.kda_causal_conv_multi_step, dev, x.data_ptr(), dt, weight.data_ptr(), _addr(bias),
          state.data_ptr(), _addr(y), adv, N, T, C, W, sx, sy, tail=(1 if silu else 0,))
    return y


def _scan_inputs(x, dt, A, B, C, D, z, dt_bias):
    """(shape of x, device, channels, states, groups, dtype code, strides of x, dt, B, C, z) of a
    scan's checked inputs."""
    shape, dtype, dev, code = _tokens(x, "x")
    n, lead = shape[-1], shape[:-1]
    _need(A, "A", torch.float32, dev)
    As = A.shape
    if len(As) != 2 or As[0] != n:
        raise ValueError(f"A must be [{n}, states], got {tuple(As)}")
    S = _count(As[1], "A")
    G = B.shape[-2] if isinstance(B, torch.Tensor) and B.dim() > 2 else 1
    row, bc = (n,), (G, S)
    sx = _row_stride(x, "x", row, dtype, dev)
    sdt = _row_stride(dt, "dt", row, dtype, dev)
    sB = _row_stride(B, "B", bc, dtype, dev)
    sC = _row_stride(C, "C", bc, dtype, dev)
    if dt.shape != shape:
        raise ValueError(f"dt must be {tuple(shape)}, got {tuple(dt.shape)}")
    whole = B.shape
    if whole != lead + bc:
        raise ValueError(f"B must be {tuple(lead + bc)}, got {tuple(whole)}")
    if C.shape != whole:
        raise ValueError(f"C must be {tuple(whole)}, got {tuple(C.shape)}")
    sz = n
    if z is not None:
        sz = _row_stride(z, "z", row, dtype, dev)
        if z.shape != shape:
            raise ValueError(f"z must be {tuple(shape)}, got {tuple(z.shape)}")
    if D is not None:
        _need(D, "D", torch.float32, dev)
        if D.shape != row:
            raise ValueError(f"D must be [{n}], got {tuple(D.shape)}")
    if dt_bias is not None:
        _need(dt_bias, "dt_bias", torch.float32, dev)
        if dt_bias.shape != row:
            raise ValueError(f"dt_bias must be [{n}], got {tuple(dt_bias.shape)}")
    return shape, dev, n, S, G, code, sx, sdt, sB, sC, sz


def selective_scan_fwd(x, dt, A, B, C, h0=None, cu_seqlens=None, *, D=None, z=None, dt_bias=None,
                       softplus: bool = True, output_final_state=True, out=None,
                       final_state_out=None):
    """Prompt pass of the selective state space scan: with delta_t = softplus(dt_t + dt_bias)
    (``softplus=False``: dt_t + dt_bias),
    ``h_t = exp(delta_t A) h_{t-1} + delta_t x_t B_t``, ``y_t = (C_t . h_t + D x_t) SiLU(z_t)``.

    x, dt, z [B, T, channels] or packed [NT, channels] (with ``cu_seqlens``), B, C
    [..., groups, states] (states 8, 16 or 32; a group's channels, a multiple of 8, are
    neighbours), bf16 or fp32; their tokens may be slices of packed projections.  A fp32
    [channels, states], D and dt_bias fp32 [channels] or None, z None for no gate.  h0 fp32
    [N, channels, states] or None.  ``out`` must not overlap an input; ``final_state_out`` may be
    h0.  Long sequences of few channels are cut into segments that run at once (the same result up
    to rounding).  Returns ``(y, hT)``; hT (None if not asked) is the h of :func:`selective_step`.
    """
    shape, dev, n, S, G, code, sx, sdt, sB, sC, sz = _scan_inputs(x, dt, A, B, C, D, z, dt_bias)
    N, batch, T = _packed(shape[:-1], cu_seqlens, dev, "x")
    if h0 is not None:
        _like(h0, "h0", (N, n, S), torch.float32, dev)
    hT = _like(final_state_out, "final_state_out", (N, n, S), torch.float32, dev) \
        if output_final_state else None
    y, sy = _rows_out(out, x, n)
    _call(lib.kda_selective_scan_fwd, dev, x.data_ptr(), dt.data_ptr(), A.data_ptr(), B.data_ptr(),
          C.data_ptr(), code, _addr(D), _addr(z), _addr(dt_bias), _addr(h0), _addr(cu_seqlens), N,
          batch, T, n, S, G, sx, sdt, sB, sC, sz, y.data_ptr(), sy, _addr(hT),
          tail=(1 if softplus else 0,))
    return y, hT


def selective_step(x, dt, A, B, C, h, *, D=None, z=None, dt_bias=None, softplus: bool = True,
                   out=None):
    """One new token of :func:`selective_scan_fwd` for N sequences: x, dt, z [N, channels], B, C
    [N, groups, states], h fp32 [N, channels, states] updated in place.  Returns y [N, channels]."""
    shape, dev, n, S, G, code, sx, sdt, sB, sC, sz = _scan_inputs(x, dt, A, B, C, D, z, dt_bias)
    if len(shape) != 2:
        raise ValueError(f"x must be [N, channels], got {tuple(shape)}")
    N = shape[0]
    _like(h, "h", (N, n, S), torch.float32, dev, given=True)
    y, sy = _rows_out(out, x, n)
    _call(lib.kda_selective_step, dev, x.data_ptr(), dt.data_ptr(), A.data_ptr(), B.data_ptr(),
          C.data_ptr(), code, _addr(D), _addr(z), _addr(dt_bias), h.data_ptr(), y.data_ptr(), N, n, S,
          G, sx, sdt, sB, sC, sz, sy, tail=(1 if softplus else 0,))
    return y


def selective_multi_step(x, dt, A, B, C, h, n_advance=None, *, D=None, z=None, dt_bias=None,
                         softplus: bool = True, out=None, return_outputs=True):
    """T <= 16 new tokens a sequence: x, dt, z [N, T, channels], B, C [N, T, groups, states], h fp32
    [N, channels, states] advanced in place by n_advance[n] tokens (int32 [N] on the device;
    None = all T).  Returns y [N, T, channels] (of all T tokens), or None when return_outputs is
    False."""
    shape, dev, n, S, G, code, sx, sdt, sB, sC, sz = _scan_inputs(x, dt, A, B, C, D, z, dt_bias)
    if len(shape) != 3:
        raise ValueError(f"x must be [N, T, channels], got {tuple(shape)}")
    N, T, _ = shape
    _like(h, "h", (N, n, S), torch.float32, dev, given=True)
    adv = _advance(n_advance, N, dev)
    y, sy = _rows_out(out, x, n) if return_outputs else (None, n)
    _call(lib.kda_selective_multi_step, dev, x.data_ptr(), dt.data_ptr(), A.data_ptr(),
          B.data_ptr(), C.data_ptr(), code, _addr(D), _addr(z), _addr(dt_bias), h.data_ptr(),
          _addr(y), adv, N, T, n, S, G, sx, sdt, sB, sC, sz, sy, tail=(1 if softplus else 0,))
    return y


def verify_draft(draft_tokens, draft_probs, target_probs, accept_uniforms, sample_uniforms, *,
                 tokens_out=None, n_advance_out=None):
    """Decides how many drafted tokens every sequence keeps and draws the token behind them.

    draft_tokens int32 [N, T] (T <= 15; an entry outside the vocabulary ends a draft), the
    distributions they were drawn from draft_probs [N, T, V], the target's target_probs
    [N, T+1, V] (bf16 or fp32), accept_uniforms fp32 [N, T] and sample_uniforms fp32 [N] in [0, 1).
    Token i is accepted while ``accept_uniforms[i] * q_i(d_i) < p_i(d_i)``; the next one is drawn
    from max(p - q, 0) where one was rejected, else from p.  Returns ``(tokens, n_advance)``: int32
    [N, T+1], the accepted tokens, the drawn one, then -1, and int32 [N], how many they are: the
    n_advance of the multi-step calls over the last token before the draft and the draft.
    """
    dev = target_probs.device if isinstance(target_probs, torch.Tensor) else None
    _need(target_probs, "target_probs")
    if target_probs.dim() != 3 or target_probs.shape[1] < 1:
        raise ValueError(f"target_probs must be [N, T+1, V], got {tuple(target_probs.shape)}")
    N, T, V = target_probs.shape
    _count(max(N, T, V), "target_probs")
    T -= 1
    dt = _dtype_code(target_probs)
    _like(draft_tokens, "draft_tokens", (N, T), torch.int32, dev, given=True)
    _like(draft_probs, "draft_probs", (N, T, V), target_probs.dtype, dev, given=True)
    _like(accept_uniforms, "accept_uniforms", (N, T), torch.float32, dev, given=True)
    _like(sample_uniforms, "sample_uniforms", (N,), torch.float32, dev, given=True)
    tokens = _like(tokens_out, "tokens_out", (N, T + 1), torch.int32, dev)
    count = _like(n_advance_out, "n_advance_out", (N,), torch.int32, dev)
    _call(lib.kda_verify_draft, dev, draft_tokens.data_ptr(), draft_probs.data_ptr(),
          target_probs.data_ptr(), dt, accept_uniforms.data_ptr(), sample_uniforms.data_ptr(),
          tokens.data_ptr(), count.data_ptr(), N, T, V)
    return tokens, count


def profile_enable(on: bool = True):
    """Start (clearing earlier records) or stop per-kernel CUDA-event timing."""
    lib.kda_profile_enable(1 if on else 0)


def profile_collect() -> dict:
    """Waits for the recorded events; returns {kernel: (launches, total_ms)}."""
    n = lib.kda_profile_collect()
    if n < 0:
        raise KdaError(6, "profile collection failed")
    out = {}
    for i in range(n):
        name = ctypes.c_char_p()
        launches = ctypes.c_int()
        total = ctypes.c_double()
        lib.kda_profile_get(i, ctypes.byref(name), ctypes.byref(launches), ctypes.byref(total))
        out[name.value.decode()] = (launches.value, total.value)
    return out


def selftest_wait_timeout(timeout_us: int = 1000, device=None) -> int:
    """Runs the library's bounded-wait self-test (a kernel whose waits nothing
    signals gives up after ``timeout_us``); synchronizes and returns how many of
    its four waiting warps saw the wait end unsatisfied.  The device error flag is
    left set to KDA_ERR_DEVICE_TIMEOUT for :func:`get_device_error`."""
    device = device or torch.device("cuda", torch.cuda.current_device())
    n = ctypes.c_int(-1)
    with torch.cuda.device(device):
        _check(lib.kda_selftest_wait_timeout(int(timeout_us), ctypes.byref(n), _stream(device)))
    return n.value


def get_device_error(device=None):
    """Raise KdaError if a kernel recorded a device-side error (syncs the stream)."""
    device = device or torch.device("cuda", torch.cuda.current_device())
    with torch.cuda.device(device):
        _check(lib.kda_get_device_error(_stream(device)))
