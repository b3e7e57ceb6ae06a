"""Gated-delta-rule decode for AMD MI355X (gfx950): Python binding of ``include/rgdr.h``.

Argument marshalling only: every step of the computation runs in the HIP kernels of
``librgdr.so``; PyTorch supplies device memory and the current stream. There is no CPU
fallback: if the library is missing, the first call of any binding function raises
``ImportError``. The ``rgdr_`` calls and ``la_gate`` go through ctypes, the linear-attention calls
through the CPython module ``_la_binding`` (``csrc/la_binding.cpp``), which checks and calls; where
it finds that a call does not fit, the checks here say why. It is loaded by the first of those calls.

* ``rgdr_decode``  -- the recurrent gated-delta-rule decode step (MindSpore Lite API page
  "lite_boost.ops.recurrent_gated_delta_rule"), in place on a bf16 state pool.
* ``recurrent_gated_delta_rule`` -- the page's functional form: returns ``(out, state_out)``
  and leaves ``state`` untouched.
* ``rgdr_decode_snapshots`` -- ``rgdr_decode`` that also returns the state after every
  token (speculative decoding: the state of each candidate accepted prefix).
* ``rgdr_decode_gated`` -- the decode step with the gate front end fused in: takes the raw
  gate projections instead of g and beta.
* ``rgdr_prefill`` / ``rgdr_prefill_gated`` -- the same recurrence over long sequences
  (T up to 65536; the page's notes hand prefill to a chunk-level operator), same arguments.
* ``la_gate`` -- the gate front end (README "com.microsoft.LinearAttentionGate").
* ``la_decode`` / ``la_prefill`` -- linear attention with a decay for each head (no delta
  correction), for a few tokens and for prompts, on pools of fp32, bf16 or 8-bit states.
* ``la_state_quantize`` / ``la_state_dequantize`` -- states into and out of 8-bit pools.
* ``la_norm_gate`` -- the per-head norm of the outputs times the output gate.
* ``la_conv`` -- the short causal convolution in front of a recurrence, on a pool of last inputs.
* ``la_rope`` -- rotary positions of queries and keys; ``la_rope_frequencies`` -- their frequencies.
* ``ssm_decode`` / ``ssm_prefill`` -- the selective state space scan (a decay for each channel and
  state), for a few tokens and for prompts, on pools of fp32 or bf16 states.
* ``rgdr_validate`` -- synchronous check of the index arrays.

A non-OK status from the library raises ``RuntimeError`` (the page's error behaviour).

Calls run on the current stream, or on the one given as ``stream``: what they read has to be ready
there, and what they write is ready there behind them. Tensors may be dropped when a call returns.

With ``RGDR_VALIDATE=1`` in the environment (read at import; ``VALIDATE`` holds it), every
call that takes lengths, accepted counts or slots of entries first checks them with
``rgdr_validate``: a synchronous copy to the host, for debugging only (it cannot run under graph
capture). A bad length, count or slot then raises ``RuntimeError`` instead of being clamped or
skipped by the kernel. (``la_state_quantize`` and ``la_state_dequantize``, whose slots may be out
of range, check nothing.)
"""
import ctypes as C
import math
import os

import torch

__all__ = ["rgdr_decode", "rgdr_decode_snapshots", "rgdr_decode_gated",
           "rgdr_decode_gated_snapshots", "rgdr_prefill", "rgdr_prefill_gated",
           "rgdr_prefill_ws", "rgdr_prefill_gated_ws", "rgdr_prefill_workspace_size",
           "rgdr_prefill_noalloc",
           "recurrent_gated_delta_rule", "la_gate", "la_decode", "la_prefill",
           "la_prefill_workspace_size", "la_state_quantize", "la_state_dequantize",
           "la_norm_gate", "la_conv", "la_rope", "la_rope_frequencies", "ssm_decode", "ssm_prefill",
           "ssm_prefill_workspace_size",
           "rgdr_validate", "VALIDATE",
           "rgdr_validate_host", "status_string", "library", "LIB_PATH", "RGDR_F32",
           "RGDR_F16", "RGDR_BF16", "RGDR_MXI8"]

LIB_PATH = os.path.join(os.path.dirname(os.path.abspath(__file__)), "librgdr.so")

RGDR_F32, RGDR_F16, RGDR_BF16, RGDR_MXI8 = 0, 1, 2, 3
RGDR_NORMALIZE_QK = 1  # option bit of rgdr_decode_gated
NORMALIZE_QK = RGDR_NORMALIZE_QK
LA_GATE_SIGMOID = 1    # option bit of la_norm_gate
LA_CONV_SILU = 1       # option bit of la_conv
LA_ROPE_INTERLEAVED = 1  # option bit of la_rope
SSM_DT_SOFTPLUS = 1    # option bit of ssm_decode and ssm_prefill
LA_BLOCK = 32          # columns of a state row that share a scale byte in an 8-bit pool
_DTYPE_CODE = {torch.float32: RGDR_F32, torch.float16: RGDR_F16, torch.bfloat16: RGDR_BF16}


class _Strides(C.Structure):  # la_strides of include/rgdr.h
    _fields_ = [("b", C.c_int64), ("h", C.c_int64), ("t", C.c_int64)]


_lib = None
_quick = None  # the CPython module
VALIDATE = os.environ.get("RGDR_VALIDATE", "") == "1"


def library():
    """Load ``librgdr.so`` (built by ``gated_delta_rule_rgdr_amd/build.py``)."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(LIB_PATH):
        raise ImportError(
            f"{LIB_PATH} is missing: build it with `python -m gated_delta_rule_rgdr_amd.build` "
            "(there is no fallback path)")
    lib = C.CDLL(LIB_PATH)
    vp, i32, i64, f32 = C.c_void_p, C.c_int32, C.c_int64, C.c_float
    lib.rgdr_decode.restype = C.c_int
    lib.rgdr_decode.argtypes = [vp] * 10 + [f32] + [i32] * 7 + [vp, vp, vp]
    lib.rgdr_decode_snapshots.restype = C.c_int
    lib.rgdr_decode_snapshots.argtypes = [vp] * 10 + [f32] + [i32] * 7 + [vp, vp, vp, vp]
    lib.rgdr_decode_gated.restype = C.c_int
    lib.rgdr_decode_gated.argtypes = ([vp] * 7 + [C.c_int] + [vp] * 5 + [f32] + [i32] * 7
                                      + [vp] * 2 + [C.c_uint32, vp])
    lib.rgdr_decode_gated_snapshots.restype = C.c_int
    lib.rgdr_decode_gated_snapshots.argtypes = ([vp] * 7 + [C.c_int] + [vp] * 5 + [f32]
                                                + [i32] * 7 + [vp] * 3 + [C.c_uint32, vp])
    lib.rgdr_prefill.restype = C.c_int
    lib.rgdr_prefill.argtypes = lib.rgdr_decode.argtypes
    lib.rgdr_prefill_gated.restype = C.c_int
    lib.rgdr_prefill_gated.argtypes = lib.rgdr_decode_gated.argtypes
    lib.rgdr_prefill_noalloc.restype = C.c_int
    lib.rgdr_prefill_noalloc.argtypes = lib.rgdr_decode.argtypes
    lib.rgdr_prefill_workspace_size.restype = C.c_int
    lib.rgdr_prefill_workspace_size.argtypes = [i32] * 5 + [C.POINTER(C.c_size_t)]
    lib.rgdr_prefill_ws.restype = C.c_int
    lib.rgdr_prefill_ws.argtypes = [vp] * 10 + [f32] + [i32] * 7 + [vp, vp, vp, C.c_size_t, vp]
    lib.rgdr_prefill_gated_ws.restype = C.c_int
    lib.rgdr_prefill_gated_ws.argtypes = ([vp] * 7 + [C.c_int] + [vp] * 5 + [f32] + [i32] * 7
                                          + [vp] * 2 + [C.c_uint32, vp, C.c_size_t, vp])
    lib.la_gate.restype = C.c_int
    lib.la_gate.argtypes = [vp, vp, vp, vp, C.c_int, i64, i32, vp, C.c_int, vp, C.c_int, vp]
    st = C.POINTER(_Strides)
    lib.la_decode.restype = C.c_int
    lib.la_decode.argtypes = ([vp, st] * 4 + [vp, vp, C.c_int] + [vp] * 3 + [f32] + [i32] * 7
                              + [vp, st, vp, vp, vp])
    lib.la_prefill.restype = C.c_int
    lib.la_prefill.argtypes = lib.la_decode.argtypes[:-1] + [vp, C.c_size_t, vp]
    lib.la_prefill_workspace_size.restype = C.c_int
    lib.la_prefill_workspace_size.argtypes = [i32] * 5 + [C.POINTER(C.c_size_t)]
    lib.la_state_quantize.restype = C.c_int
    lib.la_state_quantize.argtypes = [vp, C.c_int, i32, vp, vp, vp, i32, vp] + [i32] * 4 + [vp]
    lib.la_state_dequantize.restype = C.c_int
    lib.la_state_dequantize.argtypes = [vp, vp, i32, vp, vp, C.c_int, i32, vp] + [i32] * 4 + [vp]
    lib.la_norm_gate.restype = C.c_int
    lib.la_norm_gate.argtypes = ([vp, st, vp, st, vp, i64, C.c_int, vp, f32, C.c_uint32]
                                 + [i32] * 4 + [vp, st, vp])
    lib.la_conv.restype = C.c_int
    lib.la_conv.argtypes = ([vp, st, vp, vp, C.c_int] + [vp] * 4 + [C.c_uint32] + [i32] * 5
                            + [vp, st, vp, vp])
    lib.la_rope.restype = C.c_int
    lib.la_rope.argtypes = ([vp, st, vp, st, vp, vp, C.c_int, vp, f32, C.c_uint32] + [i32] * 6
                            + [vp, st, vp, st, vp])
    lib.ssm_decode.restype = C.c_int
    lib.ssm_decode.argtypes = ([vp, st, vp, st, vp, vp, st, vp, st, vp, vp, st, vp, C.c_int, vp,
                                C.c_int] + [vp] * 3 + [C.c_uint32] + [i32] * 6 + [vp, st, vp, vp])
    lib.ssm_prefill.restype = C.c_int
    lib.ssm_prefill.argtypes = lib.ssm_decode.argtypes[:-1] + [vp, C.c_size_t, vp]
    lib.ssm_prefill_workspace_size.restype = C.c_int
    lib.ssm_prefill_workspace_size.argtypes = [i32] * 5 + [C.POINTER(C.c_size_t)]
    lib.rgdr_validate.restype = C.c_int
    lib.rgdr_validate.argtypes = [vp, vp, vp, i32, i32, i32, vp]
    lib.rgdr_validate_host.restype = C.c_int
    lib.rgdr_validate_host.argtypes = [vp, vp, vp, i32, i32, i32]
    lib.rgdr_status_string.restype = C.c_char_p
    lib.rgdr_status_string.argtypes = [C.c_int]
    _lib = lib
    return lib


def _load_quick():
    """Load the CPython module of the linear-attention calls; the others do without it."""
    global _quick
    library()
    from . import _la_binding
    _quick = _la_binding


def status_string(code: int) -> str:
    return library().rgdr_status_string(code).decode()


def _check(code: int, what: str):
    if code != 0:
        raise RuntimeError(f"{what}: {status_string(code)}")


def _stream_handle(stream, device):
    s = stream if stream is not None else torch.cuda.current_stream(device)
    return s.cuda_stream


def _same_device(ref, **tensors):
    """Every tensor on ref's GPU: the library launches on the current device and takes the
    pointers as that device's addresses."""
    for name, t in tensors.items():
        if t is not None and t.device != ref.device:
            raise RuntimeError(f"{name} is on {t.device}, expected {ref.device}")


def _validate_indices(lens, idx, nacc, T, N, stream):
    code = rgdr_validate(lens, idx, nacc, T, N, stream)
    _check(code, "index arrays (RGDR_VALIDATE)")


def _dtype_code(dtype, name):
    if dtype not in _DTYPE_CODE:
        raise RuntimeError(f"{name}: unsupported dtype {dtype}")
    return _DTYPE_CODE[dtype]


def _dev(t, name, dtype, ndim=None):
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if not t.is_cuda:
        raise RuntimeError(f"{name} must be on the GPU")
    if t.dtype != dtype:
        raise RuntimeError(f"{name} must be {dtype}, got {t.dtype}")
    if ndim is not None and t.dim() != ndim:
        raise RuntimeError(f"{name} must have {ndim} dimensions, got {t.dim()}")
    if not t.is_contiguous():
        raise RuntimeError(f"{name} must be contiguous")
    return t


def rgdr_decode(query, key, value, beta, state_pool, actual_seq_lengths, ssm_state_indices,
                g, gk, num_accepted_tokens, scale=1.0, *, out=None, state_out=None,
                stream=None):
    """One decode step (T <= 8); returns ``(out, state_out)``.

    Shapes (page parameter list; the state is a slot pool): query/key bf16
    ``[B,H_q,T,D_k]``, value bf16 ``[B,H_v,T,D_v]``, beta bf16 ``[B,H_v,T]``, state_pool bf16
    ``[N_slots,H_v,D_k,D_v]``, g fp32 ``[B,H_v,T]``, gk fp32 ``[B,H_v,T,D_k]``, the three index
    arrays int32 ``[B]``. ``state_out`` defaults to ``state_pool`` (in-place update of the
    named slots); ``out`` is allocated if not given.
    """
    return _plain_call("rgdr_decode", query, key, value, beta, state_pool, actual_seq_lengths,
                       ssm_state_indices, g, gk, num_accepted_tokens, scale, out, state_out,
                       stream)


def rgdr_decode_snapshots(query, key, value, beta, state_pool, actual_seq_lengths,
                          ssm_state_indices, g, gk, num_accepted_tokens, scale=1.0, *,
                          out=None, state_out=None, state_snapshots=None, stream=None):
    """``rgdr_decode`` that also stores the state after every token; returns
    ``(out, state_out, state_snapshots)``.

    ``state_snapshots``: bf16 ``[B, T, H_v, D_k, D_v]``, allocated (uninitialised) if not
    given. Entry ``[b, t]`` is written for ``t`` below the clamped length of entry ``b`` when
    its slot is valid, and holds the state after its first ``t + 1`` tokens; other entries
    keep what the buffer held.
    """
    state_snapshots = _snapshot_buffer(query, value, state_pool, state_snapshots, stream)
    out, state_out = _plain_call("rgdr_decode_snapshots", query, key, value, beta, state_pool,
                                 actual_seq_lengths, ssm_state_indices, g, gk,
                                 num_accepted_tokens, scale, out, state_out, stream,
                                 extra={"state_snapshots": state_snapshots})
    return out, state_out, state_snapshots


def _snapshot_buffer(query, value, state_pool, state_snapshots, stream):
    """The per-token state buffer of a snapshot call: checked, or allocated uninitialised."""
    if not isinstance(query, torch.Tensor) or not isinstance(value, torch.Tensor) \
            or not isinstance(state_pool, torch.Tensor):
        raise TypeError("query, value and state_pool must be torch.Tensor")
    if query.dim() != 4 or value.dim() != 4 or state_pool.dim() != 4:
        raise RuntimeError("query, value and state_pool must have 4 dimensions")
    B, _, T, Dk = query.shape
    Hv, Dv = value.shape[1], value.shape[3]
    if state_snapshots is None:
        return _empty((B, T, Hv, Dk, Dv), torch.bfloat16, query.device, stream)
    _dev(state_snapshots, "state_snapshots", torch.bfloat16, 5)
    if tuple(state_snapshots.shape) != (B, T, Hv, Dk, Dv):
        raise RuntimeError("state_snapshots must be [B, T, H_v, D_k, D_v]")
    return state_snapshots


def rgdr_prefill(query, key, value, beta, state_pool, actual_seq_lengths, ssm_state_indices,
                 g, gk, num_accepted_tokens, scale=1.0, *, out=None, state_out=None,
                 stream=None):
    """The same recurrence over long sequences (T up to 65536, the prefill counterpart the
    page's notes name); arguments and results as ``rgdr_decode``."""
    return _plain_call("rgdr_prefill", query, key, value, beta, state_pool, actual_seq_lengths,
                       ssm_state_indices, g, gk, num_accepted_tokens, scale, out, state_out,
                       stream)


def rgdr_prefill_workspace_size(B, H_v, T, D_k, D_v, device=None):
    """Bytes of workspace ``rgdr_prefill_ws`` uses for a call of these sizes on ``device``
    (0: such a call runs in one pass and needs none)."""
    lib = library()
    n = C.c_size_t(0)
    with torch.cuda.device(device if device is not None else torch.cuda.current_device()):
        rc = lib.rgdr_prefill_workspace_size(B, H_v, T, D_k, D_v, C.byref(n))
    _check(rc, "rgdr_prefill_workspace_size")
    return n.value


def _workspace(query, value, state_pool, workspace, stream):
    """The caller's workspace (a uint8 CUDA tensor), or one allocated for the call."""
    if workspace is None:
        B, _, T, Dk = query.shape
        Hv, Dv = value.shape[1], value.shape[3]
        nbytes = rgdr_prefill_workspace_size(B, Hv, T, Dk, Dv, query.device)
        workspace = _empty(max(nbytes, 1), torch.uint8, query.device, stream)
    if workspace.dtype != torch.uint8 or not workspace.is_cuda or not workspace.is_contiguous():
        raise RuntimeError("workspace must be a contiguous uint8 CUDA tensor")
    return workspace


def rgdr_prefill_ws(query, key, value, beta, state_pool, actual_seq_lengths, ssm_state_indices,
                    g, gk, num_accepted_tokens, scale=1.0, *, workspace=None, out=None,
                    state_out=None, stream=None):
    """``rgdr_prefill`` with a workspace (a uint8 CUDA tensor of at least
    ``rgdr_prefill_workspace_size`` bytes; allocated for the call when None). Calls of few
    sequences then evaluate all segments of a sequence at once."""
    workspace = _workspace(query, value, state_pool, workspace, stream)
    return _plain_call("rgdr_prefill_ws", query, key, value, beta, state_pool,
                       actual_seq_lengths, ssm_state_indices, g, gk, num_accepted_tokens, scale,
                       out, state_out, stream, workspace=workspace)


def rgdr_prefill_noalloc(query, key, value, beta, state_pool, actual_seq_lengths,
                         ssm_state_indices, g, gk, num_accepted_tokens, scale=1.0, *, out=None,
                         state_out=None, stream=None):
    """``rgdr_prefill_ws`` whose workspace is the library's fixed 128 MiB device array: the
    call allocates no device memory itself (``out`` and ``state_out`` are still allocated
    here when not given). Calls that overlap on one device race on that array."""
    return _plain_call("rgdr_prefill_noalloc", query, key, value, beta, state_pool,
                       actual_seq_lengths, ssm_state_indices, g, gk, num_accepted_tokens, scale,
                       out, state_out, stream)


def _plain_call(fn, query, key, value, beta, state_pool, actual_seq_lengths, ssm_state_indices,
                g, gk, num_accepted_tokens, scale, out, state_out, stream, extra=None,
                workspace=None):
    extra = extra or {}  # further output buffers, passed after state_out in this order
    lib = library()
    _dev(query, "query", torch.bfloat16, 4)
    B, Hq, T, Dk = query.shape
    _dev(key, "key", torch.bfloat16, 4)
    _dev(value, "value", torch.bfloat16, 4)
    _dev(beta, "beta", torch.bfloat16, 3)
    _dev(state_pool, "state_pool", torch.bfloat16, 4)
    _dev(g, "g", torch.float32, 3)
    _dev(gk, "gk", torch.float32, 4)
    for nm, t in (("actual_seq_lengths", actual_seq_lengths),
                  ("ssm_state_indices", ssm_state_indices),
                  ("num_accepted_tokens", num_accepted_tokens)):
        _dev(t, nm, torch.int32, 1)
        if t.shape[0] != B:
            raise RuntimeError(f"{nm} must have shape [{B}]")
    Hv, Dv = value.shape[1], value.shape[3]
    N = state_pool.shape[0]
    if tuple(key.shape) != (B, Hq, T, Dk) or tuple(value.shape) != (B, Hv, T, Dv) \
            or tuple(beta.shape) != (B, Hv, T) or tuple(g.shape) != (B, Hv, T) \
            or tuple(gk.shape) != (B, Hv, T, Dk) or tuple(state_pool.shape) != (N, Hv, Dk, Dv):
        raise RuntimeError(f"{fn}: inconsistent shapes")
    if out is None:
        out = _empty((B, Hv, T, Dv), torch.bfloat16, query.device, stream)
    else:
        _dev(out, "out", torch.bfloat16, 4)
        if tuple(out.shape) != (B, Hv, T, Dv):
            raise RuntimeError("out must be [B, H_v, T, D_v]")
    if state_out is None:
        state_out = state_pool
    else:
        _dev(state_out, "state_out", torch.bfloat16, 4)
        if state_out.shape != state_pool.shape:
            raise RuntimeError("state_out must have the pool's shape")
    _same_device(query, key=key, value=value, beta=beta, state_pool=state_pool,
                 actual_seq_lengths=actual_seq_lengths, ssm_state_indices=ssm_state_indices,
                 g=g, gk=gk, num_accepted_tokens=num_accepted_tokens, out=out,
                 state_out=state_out, **extra)
    if VALIDATE:
        _validate_indices(actual_seq_lengths, ssm_state_indices, num_accepted_tokens, T, N,
                          stream)
    with torch.cuda.device(query.device):
        rc = getattr(lib, fn)(query.data_ptr(), key.data_ptr(), value.data_ptr(),
                              beta.data_ptr(), state_pool.data_ptr(),
                              actual_seq_lengths.data_ptr(), ssm_state_indices.data_ptr(),
                              g.data_ptr(), gk.data_ptr(), num_accepted_tokens.data_ptr(),
                              float(scale), B, Hq, Hv, T, Dk, Dv, N, out.data_ptr(),
                              state_out.data_ptr(), *[t.data_ptr() for t in extra.values()],
                              *_ws_args(workspace, query), _stream_handle(stream, query.device))
    _check(rc, fn)
    _hold(stream, query, key, value, beta, state_pool, actual_seq_lengths, ssm_state_indices, g, gk,
          num_accepted_tokens, out, state_out, workspace, *extra.values())
    return out, state_out


def _ws_args(workspace, ref):
    if workspace is None:
        return ()
    _same_device(ref, workspace=workspace)
    return (workspace.data_ptr(), workspace.numel())


def rgdr_decode_gated(query, key, value, a, b, dt_bias, decay_scale, state_pool,
                      actual_seq_lengths, ssm_state_indices, gk, num_accepted_tokens, scale=1.0,
                      *, normalize_qk=False, out=None, state_out=None, stream=None):
    """One decode step with the gate fused in; returns ``(out, state_out)``.

    ``a``, ``b``: raw gate projections ``[B, T, H_v]`` (float32 or float16, head axis last);
    ``dt_bias``, ``decay_scale``: float32 ``[H_v]``. ``g = decay_scale * softplus(a + dt_bias)``
    and ``beta = sigmoid(b)`` are computed in the kernel in fp32. With ``normalize_qk`` the
    kernel also divides each token's query and key head vector by its L2 norm (the
    operator's unit-norm precondition), so raw projections may be passed. Other arguments as
    ``rgdr_decode`` (which takes g and beta instead).
    """
    return _gated_call("rgdr_decode_gated", query, key, value, a, b, dt_bias, decay_scale,
                       state_pool, actual_seq_lengths, ssm_state_indices, gk,
                       num_accepted_tokens, scale, normalize_qk, out, state_out, stream)


def rgdr_decode_gated_snapshots(query, key, value, a, b, dt_bias, decay_scale, state_pool,
                                actual_seq_lengths, ssm_state_indices, gk, num_accepted_tokens,
                                scale=1.0, *, normalize_qk=False, out=None, state_out=None,
                                state_snapshots=None, stream=None):
    """``rgdr_decode_gated`` that also stores the state after every token, as
    ``rgdr_decode_snapshots`` extends ``rgdr_decode``; returns
    ``(out, state_out, state_snapshots)`` with the buffer as described there."""
    state_snapshots = _snapshot_buffer(query, value, state_pool, state_snapshots, stream)
    out, state_out = _gated_call("rgdr_decode_gated_snapshots", query, key, value, a, b,
                                 dt_bias, decay_scale, state_pool, actual_seq_lengths,
                                 ssm_state_indices, gk, num_accepted_tokens, scale,
                                 normalize_qk, out, state_out, stream,
                                 extra={"state_snapshots": state_snapshots})
    return out, state_out, state_snapshots


def rgdr_prefill_gated(query, key, value, a, b, dt_bias, decay_scale, state_pool,
                       actual_seq_lengths, ssm_state_indices, gk, num_accepted_tokens,
                       scale=1.0, *, normalize_qk=False, out=None, state_out=None,
                       stream=None):
    """``rgdr_prefill`` with the gate fused in, as ``rgdr_decode_gated`` extends
    ``rgdr_decode``."""
    return _gated_call("rgdr_prefill_gated", query, key, value, a, b, dt_bias, decay_scale,
                       state_pool, actual_seq_lengths, ssm_state_indices, gk,
                       num_accepted_tokens, scale, normalize_qk, out, state_out, stream)


def rgdr_prefill_gated_ws(query, key, value, a, b, dt_bias, decay_scale, state_pool,
                          actual_seq_lengths, ssm_state_indices, gk, num_accepted_tokens,
                          scale=1.0, *, normalize_qk=False, workspace=None, out=None,
                          state_out=None, stream=None):
    """``rgdr_prefill_gated`` with a workspace, as ``rgdr_prefill_ws`` extends
    ``rgdr_prefill``."""
    workspace = _workspace(query, value, state_pool, workspace, stream)
    return _gated_call("rgdr_prefill_gated_ws", query, key, value, a, b, dt_bias, decay_scale,
                       state_pool, actual_seq_lengths, ssm_state_indices, gk,
                       num_accepted_tokens, scale, normalize_qk, out, state_out, stream,
                       workspace=workspace)


def _gated_call(fn, query, key, value, a, b, dt_bias, decay_scale, state_pool,
                actual_seq_lengths, ssm_state_indices, gk, num_accepted_tokens, scale,
                normalize_qk, out, state_out, stream, extra=None, workspace=None):
    extra = extra or {}  # further output buffers, passed after state_out in this order
    lib = library()
    _dev(query, "query", torch.bfloat16, 4)
    B, Hq, T, Dk = query.shape
    _dev(key, "key", torch.bfloat16, 4)
    _dev(value, "value", torch.bfloat16, 4)
    _dev(state_pool, "state_pool", torch.bfloat16, 4)
    _dev(gk, "gk", torch.float32, 4)
    if a.dtype not in (torch.float32, torch.float16):
        raise RuntimeError("gate projections must be float32 or float16")
    _dev(a, "a", a.dtype, 3)
    _dev(b, "b", a.dtype, 3)
    _dev(dt_bias, "dt_bias", torch.float32, 1)
    _dev(decay_scale, "decay_scale", torch.float32, 1)
    for nm, t in (("actual_seq_lengths", actual_seq_lengths),
                  ("ssm_state_indices", ssm_state_indices),
                  ("num_accepted_tokens", num_accepted_tokens)):
        _dev(t, nm, torch.int32, 1)
        if t.shape[0] != B:
            raise RuntimeError(f"{nm} must have shape [{B}]")
    Hv, Dv = value.shape[1], value.shape[3]
    N = state_pool.shape[0]
    if tuple(key.shape) != (B, Hq, T, Dk) or tuple(value.shape) != (B, Hv, T, Dv) \
            or tuple(a.shape) != (B, T, Hv) or tuple(b.shape) != (B, T, Hv) \
            or tuple(gk.shape) != (B, Hv, T, Dk) or tuple(state_pool.shape) != (N, Hv, Dk, Dv) \
            or dt_bias.shape[0] != Hv or decay_scale.shape[0] != Hv:
        raise RuntimeError(f"{fn}: inconsistent shapes")
    if out is None:
        out = _empty((B, Hv, T, Dv), torch.bfloat16, query.device, stream)
    else:
        _dev(out, "out", torch.bfloat16, 4)
        if tuple(out.shape) != (B, Hv, T, Dv):
            raise RuntimeError("out must be [B, H_v, T, D_v]")
    if state_out is None:
        state_out = state_pool
    else:
        _dev(state_out, "state_out", torch.bfloat16, 4)
        if state_out.shape != state_pool.shape:
            raise RuntimeError("state_out must have the pool's shape")
    _same_device(query, key=key, value=value, a=a, b=b, dt_bias=dt_bias,
                 decay_scale=decay_scale, state_pool=state_pool,
                 actual_seq_lengths=actual_seq_lengths, ssm_state_indices=ssm_state_indices,
                 gk=gk, num_accepted_tokens=num_accepted_tokens, out=out, state_out=state_out,
                 **extra)
    if VALIDATE:
        _validate_indices(actual_seq_lengths, ssm_state_indices, num_accepted_tokens, T, N,
                          stream)
    with torch.cuda.device(query.device):
        rc = getattr(lib, fn)(query.data_ptr(), key.data_ptr(), value.data_ptr(),
                              a.data_ptr(), b.data_ptr(), dt_bias.data_ptr(),
                              decay_scale.data_ptr(), _DTYPE_CODE[a.dtype],
                              state_pool.data_ptr(), actual_seq_lengths.data_ptr(),
                              ssm_state_indices.data_ptr(), gk.data_ptr(),
                              num_accepted_tokens.data_ptr(), float(scale), B, Hq, Hv, T,
                              Dk, Dv, N, out.data_ptr(), state_out.data_ptr(),
                              *[t.data_ptr() for t in extra.values()],
                              NORMALIZE_QK if normalize_qk else 0,
                              *_ws_args(workspace, query), _stream_handle(stream, query.device))
    _check(rc, fn)
    _hold(stream, query, key, value, a, b, dt_bias, decay_scale, state_pool, actual_seq_lengths,
          ssm_state_indices, gk, num_accepted_tokens, out, state_out, workspace, *extra.values())
    return out, state_out


def recurrent_gated_delta_rule(query, key, value, beta, state, actual_seq_lengths,
                               ssm_state_indices, g, gk, num_accepted_tokens, scale_value=1.0):
    """The page's functional signature: ``(out, state_out)`` with ``state`` left unchanged.

    ``state_out`` starts as a device copy of ``state``; the kernel then writes every slot a
    batch entry names. Feed it back as ``state`` for the next step.
    """
    state_out = torch.empty_like(state)
    state_out.copy_(state)
    return rgdr_decode(query, key, value, beta, state_out, actual_seq_lengths,
                       ssm_state_indices, g, gk, num_accepted_tokens, scale_value)


def la_gate(a, dt_bias, decay_scale, b=None, *, want_beta=None, decay_dtype=None,
            beta_dtype=None, decay_out=None, beta_out=None, stream=None):
    """``decay = decay_scale * softplus(a + dt_bias)``, ``beta = sigmoid(b)`` (fp32 math).

    ``a``/``b``: float32 or float16, any rank >= 1, head axis last. ``dt_bias`` and
    ``decay_scale``: float32 ``[H]``. ``decay`` has ``decay_dtype`` (default: a's dtype);
    ``beta`` (computed when ``want_beta``, default ``b is not None``) has ``beta_dtype``
    (default a's dtype; ``torch.bfloat16`` feeds ``rgdr_decode`` directly).
    """
    lib = library()
    if a.dtype not in (torch.float32, torch.float16):
        raise RuntimeError("a must be float32 or float16")
    _dev(a, "a", a.dtype)
    if a.dim() < 1:
        raise RuntimeError("a must have rank >= 1")
    H = a.shape[-1]
    _dev(dt_bias, "dt_bias", torch.float32, 1)
    _dev(decay_scale, "decay_scale", torch.float32, 1)
    if dt_bias.shape[0] != H or decay_scale.shape[0] != H:
        raise RuntimeError("dt_bias and decay_scale must be [H]")
    if want_beta is None:
        want_beta = b is not None
    if b is not None:
        _dev(b, "b", a.dtype)
        if b.shape != a.shape:
            raise RuntimeError("b must have a's shape")
    decay_dtype = decay_dtype or a.dtype
    if decay_out is None:
        decay_out = _empty(a.shape, decay_dtype, a.device, stream)
    _dev(decay_out, "decay_out", decay_dtype)
    beta_t = None
    if want_beta:
        beta_dtype = beta_dtype or a.dtype
        beta_t = beta_out if beta_out is not None else _empty(a.shape, beta_dtype, a.device, stream)
        _dev(beta_t, "beta_out", beta_dtype)
    n_rows = a.numel() // H if H else 0
    _same_device(a, dt_bias=dt_bias, decay_scale=decay_scale, b=b, decay_out=decay_out,
                 beta_out=beta_t)
    with torch.cuda.device(a.device):
        rc = lib.la_gate(a.data_ptr(), dt_bias.data_ptr(), decay_scale.data_ptr(),
                         b.data_ptr() if b is not None else None, _DTYPE_CODE[a.dtype], n_rows,
                         H, decay_out.data_ptr(), _dtype_code(decay_dtype, "decay_out"),
                         beta_t.data_ptr() if beta_t is not None else None,
                         _dtype_code(beta_dtype, "beta_out") if beta_t is not None else 0,
                         _stream_handle(stream, a.device))
    _check(rc, "la_gate")
    _hold(stream, a, dt_bias, decay_scale, b, decay_out, beta_t)
    return decay_out, beta_t


def _rows(t, name, dtypes, ndim=4):
    """A [B, H, T, D] operand whose D elements are contiguous; the other axes may have any
    strides."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if not t.is_cuda:
        raise RuntimeError(f"{name} must be on the GPU")
    if t.dtype not in dtypes:
        raise RuntimeError(f"{name} must be {' or '.join(map(str, dtypes))}, got {t.dtype}")
    if t.dim() != ndim:
        raise RuntimeError(f"{name} must have {ndim} dimensions, got {t.dim()}")
    if ndim == 4 and t.shape[3] > 1 and t.stride(3) != 1:
        raise RuntimeError(f"{name}: the last axis must be contiguous")
    return t


def _index(t, name, n):
    if t is None:
        return None
    _dev(t, name, torch.int32, 1)
    if t.shape[0] != n:
        raise RuntimeError(f"{name} must have shape [{n}]")
    return t.data_ptr()


def _torch_stream(stream, device):
    if isinstance(stream, torch.cuda.Stream):
        return stream
    return torch.cuda.ExternalStream(stream.cuda_stream, device=device)


def _empty(shape, dtype, device, stream):
    """A new tensor for a kernel on `stream`. The allocator hands out memory whose earlier use is
    over on the stream it allocates for, so it is asked with that stream current; what the caller
    does with the tensor on the stream that is current now also ends before its memory is handed
    out again."""
    if stream is None:
        return torch.empty(shape, dtype=dtype, device=device)
    with torch.cuda.stream(_torch_stream(stream, device)):
        t = torch.empty(shape, dtype=dtype, device=device)
    t.record_stream(torch.cuda.current_stream(device))
    return t


def _hold(stream, *tensors):
    """A call on a stream of its own: the caller may drop the tensors once it returns (a slot array
    made for the call), so their memory is not handed out again before the kernels are over."""
    if stream is None:
        return
    for t in tensors:
        if t is not None:
            t.record_stream(_torch_stream(stream, t.device))


_STATE_TYPES = (torch.float32, torch.bfloat16, torch.int8)


def _scales(state, scales, name):
    """The scale bytes of an 8-bit pool, checked against its codes; None for other pools."""
    if state.dtype != torch.int8:
        if scales is not None:
            raise RuntimeError(f"{name}: only an int8 pool has scales")
        return None
    if scales is None:
        raise RuntimeError(f"an int8 pool needs {name}")
    _dev(scales, name, torch.uint8, 4)
    if state.shape[3] % LA_BLOCK or \
            tuple(scales.shape) != (*state.shape[:3], state.shape[3] // LA_BLOCK):
        raise RuntimeError(f"{name} must be [N_slots, H_v, D_k, D_v / {LA_BLOCK}]")
    return scales


def _la_refuse(fn, query, key, value, g, state_pool, lens, idx, nacc, state_scales, out,
               state_out, state_scales_out, workspace, final=True):
    """The checks of a linear-attention call one by one, each with its message."""
    _rows(query, "query", (torch.bfloat16,))
    _rows(key, "key", (torch.bfloat16,))
    _rows(value, "value", (torch.bfloat16,))
    B, Hq, T, Dk = query.shape
    Hv, Dv = value.shape[1], value.shape[3]
    if isinstance(g, torch.Tensor) and g.dim() == 1:
        _dev(g, "g", torch.float32, 1)
    else:
        _rows(g, "g", (torch.float32,), 3)
    if not isinstance(state_pool, torch.Tensor) or state_pool.dtype not in _STATE_TYPES:
        raise RuntimeError("state_pool must be a float32, bfloat16 or int8 tensor")
    _dev(state_pool, "state_pool", state_pool.dtype, 4)
    N = state_pool.shape[0]
    if tuple(key.shape) != (B, Hq, T, Dk) or tuple(value.shape) != (B, Hv, T, Dv) \
            or tuple(g.shape) not in ((B, Hv, T), (Hv,)) \
            or tuple(state_pool.shape) != (N, Hv, Dk, Dv):
        raise RuntimeError(f"{fn}: inconsistent shapes")
    _scales(state_pool, state_scales, "state_scales")
    if state_out is not state_pool:
        _dev(state_out, "state_out", state_pool.dtype, 4)
        if state_out.shape != state_pool.shape:
            raise RuntimeError("state_out must have the pool's shape")
    _scales(state_out, state_scales_out, "state_scales_out")
    index = {"actual_seq_lengths": lens, "ssm_state_indices": idx, "num_accepted_tokens": nacc}
    for nm, t in index.items():
        _index(t, nm, B)
    if out is not None:
        _rows(out, "out", (torch.bfloat16,))
        if tuple(out.shape) != (B, Hv, T, Dv):
            raise RuntimeError("out must be [B, H_v, T, D_v]")
    if workspace is not None and (not isinstance(workspace, torch.Tensor)
                                  or workspace.dtype != torch.uint8 or not workspace.is_cuda
                                  or not workspace.is_contiguous()):
        raise RuntimeError("workspace must be a contiguous uint8 CUDA tensor")
    _same_device(query, key=key, value=value, g=g, state_pool=state_pool, out=out,
                 state_scales=state_scales, state_out=state_out,
                 state_scales_out=state_scales_out, workspace=workspace, **index)
    if final:
        raise RuntimeError(f"{fn}: unsupported arguments")


def _raw_stream(t, stream):
    """The stream's handle; by default the current one of t's device."""
    if stream is not None:
        return stream.cuda_stream
    dev = t.get_device() if isinstance(t, torch.Tensor) else -1
    return torch._C._cuda_getCurrentRawStream(dev) if dev >= 0 else 0


def _la_call(fn, query, key, value, g, state_pool, lens, idx, nacc, scale, state_scales, out,
             state_out, state_scales_out, stream, workspace=None):
    if _quick is None:
        _load_quick()
    if state_out is None:
        if state_scales_out is not None:
            raise RuntimeError("state_scales_out goes with state_out")
        state_out, state_scales_out = state_pool, state_scales
    if stream is not None or VALIDATE:
        out, workspace = _la_prepare(fn, query, key, value, g, state_pool, lens, idx, nacc,
                                     state_scales, out, state_out, state_scales_out, stream,
                                     workspace)
    done = _quick.attention(fn == "la_prefill", query, key, value, g, state_pool, state_scales,
                            lens, idx, nacc, scale, out, state_out, state_scales_out, workspace,
                            _raw_stream(query, stream))
    if done is None:
        _la_refuse(fn, query, key, value, g, state_pool, lens, idx, nacc, state_scales, out,
                   state_out, state_scales_out, workspace)
    rc, out = done
    if rc:
        _check(rc, fn)
    if stream is not None:
        _hold(stream, query, key, value, g, state_pool, state_scales, lens, idx, nacc, out, state_out,
              state_scales_out, workspace)
    return (out, state_out) if state_scales is None else (out, state_out, state_scales_out)


def _la_prepare(fn, query, key, value, g, state_pool, lens, idx, nacc, state_scales, out,
                state_out, state_scales_out, stream, workspace):
    """What a call needs before it when it has a stream of its own (its new tensors belong to that
    stream) or when the index arrays are to be checked."""
    _la_refuse(fn, query, key, value, g, state_pool, lens, idx, nacc, state_scales, out,
               state_out, state_scales_out, workspace, final=False)
    B, Hq, T, Dk = query.shape
    Hv, Dv = value.shape[1], value.shape[3]
    if VALIDATE and B:
        _validate_given(lens, idx, nacc, B, T, state_pool.shape[0], query.device, stream)
    if stream is not None:
        if out is None:
            out = _empty((B, Hv, T, Dv), torch.bfloat16, query.device, stream)
        if fn == "la_prefill" and workspace is None:
            size = la_prefill_workspace_size(B, Hv, T, Dk, Dv, query.device)
            if size:
                workspace = _empty(size, torch.uint8, query.device, stream)
    return out, workspace


def la_decode(query, key, value, g, state_pool, actual_seq_lengths=None, ssm_state_indices=None,
              num_accepted_tokens=None, scale=1.0, *, state_scales=None, out=None,
              state_out=None, state_scales_out=None, stream=None):
    """Linear attention with a decay for each head, T <= 8 tokens per entry:
    ``S = exp(g) S + k v^T``, ``o = S^T (scale q)``; returns ``(out, state_out)``, for an int8
    pool ``(out, state_out, state_scales_out)``.

    query/key bf16 ``[B,H_q,T,D_k]``, value bf16 ``[B,H_v,T,D_v]``: any strides, the last axis
    contiguous, rows at multiples of 8 elements (``x.transpose(1, 2)`` of a ``[B,T,H,D]``
    projection is fine). g fp32 ``[B,H_v,T]`` of any strides (``la_gate``'s decay with its last
    axes transposed), or ``[H_v]``: one decay for each head. state_pool float32, bfloat16 or int8
    ``[N_slots,H_v,D_k,D_v]``; an int8 pool comes with ``state_scales``, uint8
    ``[N_slots,H_v,D_k,D_v/32]``. The index arrays are int32 ``[B]`` as in ``rgdr_decode``; left
    out, every token is valid, entry b is in slot b and every valid token is accepted. The state
    is updated in place unless ``state_out`` is given.
    """
    return _la_call("la_decode", query, key, value, g, state_pool, actual_seq_lengths,
                    ssm_state_indices, num_accepted_tokens, scale, state_scales, out, state_out,
                    state_scales_out, stream)


def la_prefill(query, key, value, g, state_pool, actual_seq_lengths=None, ssm_state_indices=None,
               num_accepted_tokens=None, scale=1.0, *, state_scales=None, workspace=None,
               out=None, state_out=None, state_scales_out=None, stream=None):
    """``la_decode`` over whole prompts (T up to 65536); arguments and results as there.

    ``workspace``: a uint8 CUDA tensor of ``la_prefill_workspace_size`` bytes for calls of few
    entries, which then work on parts of a prompt at once; allocated for the call when None."""
    return _la_call("la_prefill", query, key, value, g, state_pool, actual_seq_lengths,
                    ssm_state_indices, num_accepted_tokens, scale, state_scales, out, state_out,
                    state_scales_out, stream, workspace)


def la_prefill_workspace_size(B, H_v, T, D_k, D_v, device=None):
    """Bytes of workspace that ``la_prefill`` uses for a call of these sizes on ``device`` (0:
    it needs none)."""
    lib = library()
    n = C.c_size_t(0)
    with torch.cuda.device(device if device is not None else torch.cuda.current_device()):
        rc = lib.la_prefill_workspace_size(B, H_v, T, D_k, D_v, C.byref(n))
    _check(rc, "la_prefill_workspace_size")
    return n.value


def _slots(src_slots, dst_slots, n_src):
    """The number of entries of a state move: the index arrays' length, or every source."""
    for name, t in (("src_slots", src_slots), ("dst_slots", dst_slots)):
        if t is not None:
            if not isinstance(t, torch.Tensor) or t.dim() != 1:
                raise TypeError(f"{name} must be a torch.Tensor of one dimension")
            return t.shape[0]
    return n_src


def la_state_quantize(state, codes=None, scales=None, *, src_slots=None, dst_slots=None,
                      stream=None):
    """Slots ``src_slots`` of ``state`` (float32 or bfloat16 ``[N,H_v,D_k,D_v]``) into slots
    ``dst_slots`` of an 8-bit pool; returns ``(codes, scales)``, int8 ``[M,H_v,D_k,D_v]`` and
    uint8 ``[M,H_v,D_k,D_v/32]`` (value = code * 2^(scale - 127)).

    The slot arrays are int32 ``[n]`` (None: entry i is slot i). Without ``codes`` and
    ``scales``, a pool of n slots is allocated, in entry order. A source slot out of range counts
    as a zero state, an entry whose destination is out of range is skipped."""
    if not isinstance(state, torch.Tensor) or state.dtype not in (torch.float32, torch.bfloat16):
        raise RuntimeError("state must be a float32 or bfloat16 tensor")
    _dev(state, "state", state.dtype, 4)
    N, H, Dk, Dv = state.shape
    n = _slots(src_slots, dst_slots, N)
    if Dv % LA_BLOCK:
        raise RuntimeError(f"D_v must be a multiple of {LA_BLOCK}")
    if (codes is None) != (scales is None):
        raise RuntimeError("codes and scales go together")
    if codes is None:
        if dst_slots is not None:
            raise RuntimeError("dst_slots names slots of given codes and scales")
        codes = _empty((n, H, Dk, Dv), torch.int8, state.device, stream)
        scales = _empty((n, H, Dk, Dv // LA_BLOCK), torch.uint8, state.device, stream)
    return _move("la_state_quantize", state, codes, scales, src_slots, dst_slots, n, stream)


def la_state_dequantize(codes, scales, state=None, *, dtype=torch.bfloat16, src_slots=None,
                        dst_slots=None, stream=None):
    """The way back: slots ``src_slots`` of the 8-bit pool into slots ``dst_slots`` of ``state``
    (float32 or bfloat16; allocated with ``dtype``, in entry order, when None). Returns
    ``state``. Both types hold the 8-bit values exactly. Slots as in ``la_state_quantize``."""
    _dev(codes, "codes", torch.int8, 4)
    n = _slots(src_slots, dst_slots, codes.shape[0])
    if state is None:
        if dst_slots is not None:
            raise RuntimeError("dst_slots names slots of a given state")
        if dtype not in (torch.float32, torch.bfloat16):
            raise RuntimeError("dtype must be float32 or bfloat16")
        state = _empty((n, *codes.shape[1:]), dtype, codes.device, stream)
    elif not isinstance(state, torch.Tensor) or \
            state.dtype not in (torch.float32, torch.bfloat16):
        raise RuntimeError("state must be a float32 or bfloat16 tensor")
    _move("la_state_dequantize", state, codes, scales, src_slots, dst_slots, n, stream)
    return state


def _move(fn, state, codes, scales, src_slots, dst_slots, n, stream):
    if _quick is None:
        _load_quick()
    rc = _quick.move(fn == "la_state_dequantize", state, codes, scales, src_slots, dst_slots, n,
                     _raw_stream(state, stream))
    if rc is None:
        _dev(state, "state", state.dtype, 4)
        _dev(codes, "codes", torch.int8, 4)
        if codes.shape[1:] != state.shape[1:]:
            raise RuntimeError(f"{fn}: codes and state must have the same [H_v, D_k, D_v]")
        _scales(codes, scales, "scales")
        _index(src_slots, "src_slots", n)
        _index(dst_slots, "dst_slots", n)
        _same_device(state, codes=codes, scales=scales, src_slots=src_slots, dst_slots=dst_slots)
        raise RuntimeError(f"{fn}: unsupported arguments")
    if rc:
        _check(rc, fn)
    _hold(stream, state, codes, scales, src_slots, dst_slots)
    return codes, scales


def _norm_refuse(x, weight, gate, lens, out):
    _rows(x, "x", tuple(_DTYPE_CODE))
    B, H, T, D = x.shape
    for nm, t in (("gate", gate), ("out", out)):
        if t is not None:
            _rows(t, nm, (x.dtype,))
            if tuple(t.shape) != (B, T, H, D):
                raise RuntimeError(f"{nm} must be [B, T, H, D]")
    if not isinstance(weight, torch.Tensor) or tuple(weight.shape) not in ((D,), (H, D)):
        raise RuntimeError("weight must be a [D] or [H, D] tensor")
    _dev(weight, "weight", torch.float32)
    _index(lens, "actual_seq_lengths", B)
    _same_device(x, weight=weight, gate=gate, out=out, actual_seq_lengths=lens)


def la_norm_gate(x, weight, gate=None, *, eps=1e-6, sigmoid=False, actual_seq_lengths=None,
                 out=None, stream=None):
    """The norm and gate behind the attention: ``weight * x / sqrt(mean(x^2) + eps) *
    silu(gate)`` over rows of D values (``sigmoid``: sigmoid(gate) instead; no gate: the norm).

    ``x`` ``[B,H,T,D]`` as ``la_decode`` and ``rgdr_decode`` return it, ``gate`` ``[B,T,H,D]``
    as a projection gives it; float32, float16 or bfloat16, any strides with the last axis
    contiguous and rows at multiples of 8 elements, D a multiple of 8 up to 8192. ``weight``
    float32 ``[D]`` or ``[H,D]``. Returns ``out``, ``[B,T,H,D]`` of x's type; rows of tokens past
    ``actual_seq_lengths`` (int32 ``[B]``) are zero."""
    if _quick is None:
        _load_quick()
    if stream is not None or VALIDATE:
        _norm_refuse(x, weight, gate, actual_seq_lengths, out)
        B, H, T, D = x.shape
        if VALIDATE:
            _validate_lengths(actual_seq_lengths, T, stream)
        if out is None and stream is not None:
            out = _empty((B, T, H, D), x.dtype, x.device, stream)
    done = _quick.norm_gate(x, weight, gate, eps, LA_GATE_SIGMOID if sigmoid else 0,
                            actual_seq_lengths, out, _raw_stream(x, stream))
    if done is None:
        _norm_refuse(x, weight, gate, actual_seq_lengths, out)
        raise RuntimeError("la_norm_gate: unsupported arguments")
    rc, out = done
    if rc:
        _check(rc, "la_norm_gate")
    if stream is not None:
        _hold(stream, x, weight, gate, actual_seq_lengths, out)
    return out


def _validate_given(lens, idx, nacc, B, T, N, device, stream):
    """rgdr_validate of a call's index arrays, any of which may be left out."""
    def given(t, other):
        return t if t is not None else torch.as_tensor(other, dtype=torch.int32, device=device)
    n = given(lens, [T] * B)
    _validate_indices(n, given(idx, range(B)), nacc if nacc is not None else n, T, N, stream)


def _validate_lengths(lens, T, stream):
    """The same of a call whose only index array is its lengths."""
    if lens is not None and lens.shape[0] and T:
        _validate_given(lens, None, None, lens.shape[0], T, lens.shape[0], lens.device,
                        stream)


def _tokens(t, name, dtypes, shape):
    """A [B, T, ..] operand whose last axis is contiguous; the other axes may have any strides."""
    _rows(t, name, dtypes, len(shape))
    if t.shape[-1] > 1 and t.stride(-1) != 1:
        raise RuntimeError(f"{name}: the last axis must be contiguous")
    if tuple(t.shape) != tuple(shape):
        raise RuntimeError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")


def _vector(t, name, shape):
    """An optional fp32 parameter."""
    if t is not None:
        _dev(t, name, torch.float32)
        if tuple(t.shape) != tuple(shape):
            raise RuntimeError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")


def _pool(t, name, dtypes, shape):
    if not isinstance(t, torch.Tensor) or t.dtype not in dtypes:
        raise RuntimeError(f"{name} must be a tensor of {' or '.join(map(str, dtypes))}")
    _dev(t, name, t.dtype, len(shape) + 1)
    if tuple(t.shape[1:]) != tuple(shape):
        raise RuntimeError(f"{name} must be [N_slots, {', '.join(map(str, shape))}]")


def _conv_refuse(x, weight, bias, state_pool, lens, idx, nacc, out, state_out):
    _rows(x, "x", tuple(_DTYPE_CODE), 3)
    B, T, Ch = x.shape
    _tokens(x, "x", (x.dtype,), x.shape)
    if not isinstance(weight, torch.Tensor) or weight.dim() != 2:
        raise RuntimeError("weight must be a [C, W] tensor")
    W = weight.shape[1]
    _vector(weight, "weight", (Ch, W))
    _vector(bias, "bias", (Ch,))
    _pool(state_pool, "state_pool", (x.dtype,), (W - 1, Ch))
    if state_out is not state_pool:
        _pool(state_out, "state_out", (x.dtype,), (W - 1, Ch))
        if state_out.shape != state_pool.shape:
            raise RuntimeError("state_out must have the pool's shape")
    index = {"actual_seq_lengths": lens, "ssm_state_indices": idx, "num_accepted_tokens": nacc}
    for nm, t in index.items():
        _index(t, nm, B)
    if out is not None:
        _tokens(out, "out", (x.dtype,), x.shape)
    _same_device(x, weight=weight, bias=bias, state_pool=state_pool, out=out, state_out=state_out,
                 **index)


def la_conv(x, weight, state_pool, actual_seq_lengths=None, ssm_state_indices=None,
            num_accepted_tokens=None, *, bias=None, silu=True, out=None, state_out=None,
            stream=None):
    """The short causal convolution between an input projection and a recurrence:
    ``y[t] = silu(bias + sum_j weight[:, j] line[t - (W - 1) + j])`` (``silu=False``: without silu)
    for each channel, on the line of the slot's W - 1 inputs and the call's; returns
    ``(out, state_out)``.

    x ``[B,T,C]`` float32, float16 or bfloat16, any strides with the last axis contiguous and rows
    at multiples of 8 elements (columns of a wider projection are fine), T up to 65536, C a multiple
    of 8. weight float32 ``[C,W]`` with W 2, 3 or 4 (a depthwise convolution's ``[C,1,W]`` weight
    without its middle axis), bias float32 ``[C]``. state_pool ``[N_slots,W-1,C]`` of x's type: the
    inputs before the call, the latest last; it receives those of the accepted tokens, in place
    unless ``state_out`` is given. A new sequence's slot is zeros. The index arrays are int32
    ``[B]``, each may be left out, as in ``la_decode``."""
    if _quick is None:
        _load_quick()
    if state_out is None:
        state_out = state_pool
    if stream is not None or VALIDATE:
        _conv_refuse(x, weight, bias, state_pool, actual_seq_lengths, ssm_state_indices,
                     num_accepted_tokens, out, state_out)
        if VALIDATE and x.shape[0]:
            _validate_given(actual_seq_lengths, ssm_state_indices, num_accepted_tokens,
                            x.shape[0], x.shape[1], state_pool.shape[0], x.device, stream)
        if out is None and stream is not None:
            out = _empty(x.shape, x.dtype, x.device, stream)
    done = _quick.conv(x, weight, bias, state_pool, actual_seq_lengths, ssm_state_indices,
                       num_accepted_tokens, LA_CONV_SILU if silu else 0, out, state_out,
                       _raw_stream(x, stream))
    if done is None:
        _conv_refuse(x, weight, bias, state_pool, actual_seq_lengths, ssm_state_indices,
                     num_accepted_tokens, out, state_out)
        raise RuntimeError("la_conv: unsupported arguments")
    rc, out = done
    if rc:
        _check(rc, "la_conv")
    if stream is not None:
        _hold(stream, x, weight, bias, state_pool, actual_seq_lengths, ssm_state_indices,
              num_accepted_tokens, out, state_out)
    return out, state_out


def _rope_refuse(query, key, inv_freq, positions, lens, query_out, key_out):
    _rows(query, "query", tuple(_DTYPE_CODE))
    B, Hq, T, D = query.shape
    if key is not None:
        _rows(key, "key", (query.dtype,))
        if (key.shape[0], key.shape[2], key.shape[3]) != (B, T, D):
            raise RuntimeError("key must be [B, H_k, T, D] with query's B, T and D")
    elif key_out is not None:
        raise RuntimeError("key_out goes with key")
    _dev(inv_freq, "inv_freq", torch.float32, 1)
    if 2 * inv_freq.shape[0] > D:
        raise RuntimeError(f"inv_freq turns {2 * inv_freq.shape[0]} columns of {D}")
    if positions is not None:
        _dev(positions, "positions", torch.int32)
        if tuple(positions.shape) not in ((B,), (B, T)):
            raise RuntimeError("positions must be [B] or [B, T]")
    _index(lens, "actual_seq_lengths", B)
    for nm, t, x in (("query_out", query_out, query), ("key_out", key_out, key)):
        if t is not None:
            _rows(t, nm, (query.dtype,))
            if t.shape != x.shape:
                raise RuntimeError(f"{nm} must have the shape of what it receives")
    _same_device(query, key=key, inv_freq=inv_freq, positions=positions, query_out=query_out,
                 key_out=key_out, actual_seq_lengths=lens)


def la_rope(query, key, inv_freq, positions=None, *, interleaved=False, factor=1.0,
            actual_seq_lengths=None, query_out=None, key_out=None, stream=None):
    """Rotary positions: pair i of each row's first ``2 len(inv_freq)`` columns (columns i and
    ``len(inv_freq) + i``, or 2i and 2i + 1 when ``interleaved``) is turned by ``position *
    inv_freq[i]`` and multiplied by ``factor``; the other columns are copied. Returns
    ``(query_out, key_out)``, contiguous when allocated.

    query ``[B,H_q,T,D]``, key ``[B,H_k,T,D]`` (or None) float32, float16 or bfloat16, any strides
    with the last axis contiguous and rows at multiples of 8 elements, D a multiple of 8 up to 1024.
    inv_freq float32, as from ``la_rope_frequencies``. positions int32 ``[B]``: the position of each
    entry's first token (the tokens that came before it), or ``[B,T]``: each token's own; None: all
    start at 0. ``query_out=query, key_out=key`` turns them in place. Rows of tokens past
    ``actual_seq_lengths`` (int32 ``[B]``) are zero."""
    if _quick is None:
        _load_quick()
    if stream is not None or VALIDATE:
        _rope_refuse(query, key, inv_freq, positions, actual_seq_lengths, query_out, key_out)
        if VALIDATE:
            _validate_lengths(actual_seq_lengths, query.shape[2], stream)
        if query_out is None and stream is not None:
            query_out = _empty(query.shape, query.dtype, query.device, stream)
        if key_out is None and key is not None and stream is not None:
            key_out = _empty(key.shape, key.dtype, key.device, stream)
    done = _quick.rope(query, key, inv_freq, positions, actual_seq_lengths, factor,
                       LA_ROPE_INTERLEAVED if interleaved else 0, query_out, key_out,
                       _raw_stream(query, stream))
    if done is None:
        _rope_refuse(query, key, inv_freq, positions, actual_seq_lengths, query_out, key_out)
        raise RuntimeError("la_rope: unsupported arguments")
    rc, query_out, key_out = done
    if rc:
        _check(rc, "la_rope")
    if stream is not None:
        _hold(stream, query, key, inv_freq, positions, actual_seq_lengths, query_out, key_out)
    return query_out, key_out


def la_rope_frequencies(rotary_dim, base=10000.0, *, scaling=None, scale=1.0, original_length=None,
                        fast_turns=32.0, slow_turns=1.0, device="cuda"):
    """The frequencies ``base ** (-2 i / rotary_dim)`` that ``la_rope`` takes, computed in 64 bits;
    returns ``(inv_freq, factor)``, float32 ``[rotary_dim / 2]`` and la_rope's factor.

    For texts ``scale`` times as long as those that a model was trained on, ``scaling`` is
    ``"linear"`` (every frequency divided by ``scale``), ``"base"`` (a larger base, so that the
    slowest pair is divided by ``scale`` and the fastest stays) or ``"blend"``: pairs that turn at
    least ``fast_turns`` times within ``original_length`` tokens stay, those that turn at most
    ``slow_turns`` times are divided by ``scale``, those between go over linearly in their index,
    and the factor is ``0.1 ln(scale) + 1``."""
    if rotary_dim < 2 or rotary_dim % 2:
        raise RuntimeError("rotary_dim must be even and at least 2")
    if not base > 1.0:
        raise RuntimeError("base must be above 1")
    if scaling not in (None, "linear", "base", "blend"):
        raise RuntimeError("scaling must be None, 'linear', 'base' or 'blend'")
    if not scale >= 1.0:
        raise RuntimeError("scale must be at least 1")
    half, factor = rotary_dim // 2, 1.0
    i = torch.arange(half, dtype=torch.float64)
    if scaling == "base" and rotary_dim > 2:
        base = base * scale ** (rotary_dim / (rotary_dim - 2))
    freq = base ** (-2.0 * i / rotary_dim)
    if scaling == "linear":
        freq = freq / scale
    elif scaling == "blend":
        if not original_length or original_length <= 0 or not fast_turns > slow_turns > 0:
            raise RuntimeError("'blend' needs original_length and fast_turns > slow_turns > 0")

        def index(turns):  # of the pair that turns this often within original_length tokens
            return rotary_dim * math.log(original_length / (turns * 2 * math.pi)) / (2 * math.log(base))
        low = max(math.floor(index(fast_turns)), 0)
        high = min(math.ceil(index(slow_turns)), rotary_dim - 1)
        divided = ((i - low) / max(high - low, 1e-3)).clamp(0.0, 1.0) if high > 0 else torch.ones_like(i)
        freq = freq * (1 - divided) + freq / scale * divided
        factor = 0.1 * math.log(scale) + 1.0
    return freq.to(torch.float32).to(device), factor


def _ssm_refuse(fn, x, dt, A, Bm, Cm, state_pool, lens, idx, nacc, D, z, dt_bias, out, state_out,
                workspace):
    _rows(x, "x", tuple(_DTYPE_CODE), 3)
    B, T, Ch = x.shape
    for nm, t in (("x", x), ("dt", dt), ("z", z), ("out", out)):
        if t is not None or nm == "dt":
            _tokens(t, nm, (x.dtype,), x.shape)
    _dev(A, "A", torch.float32, 2)
    N = A.shape[1]
    _vector(A, "A", (Ch, N))
    _rows(Bm, "B", (x.dtype,))
    for nm, t in (("B", Bm), ("C", Cm)):
        _tokens(t, nm, (x.dtype,), (B, T, Bm.shape[2], N))
    _vector(D, "D", (Ch,))
    _vector(dt_bias, "dt_bias", (Ch,))
    _pool(state_pool, "state_pool", (torch.float32, torch.bfloat16), (Ch, N))
    if state_out is not state_pool:
        _pool(state_out, "state_out", (state_pool.dtype,), (Ch, N))
        if state_out.shape != state_pool.shape:
            raise RuntimeError("state_out must have the pool's shape")
    index = {"actual_seq_lengths": lens, "ssm_state_indices": idx, "num_accepted_tokens": nacc}
    for nm, t in index.items():
        _index(t, nm, B)
    if workspace is not None and (not isinstance(workspace, torch.Tensor)
                                  or workspace.dtype != torch.uint8 or not workspace.is_cuda
                                  or not workspace.is_contiguous()):
        raise RuntimeError("workspace must be a contiguous uint8 CUDA tensor")
    _same_device(x, dt=dt, A=A, B=Bm, C=Cm, state_pool=state_pool, D=D, z=z, dt_bias=dt_bias,
                 out=out, state_out=state_out, workspace=workspace, **index)


def _ssm_call(fn, x, dt, A, Bm, Cm, state_pool, lens, idx, nacc, D, z, dt_bias, dt_softplus, out,
              state_out, stream, workspace=None):
    if _quick is None:
        _load_quick()
    if state_out is None:
        state_out = state_pool
    if stream is not None or VALIDATE:
        _ssm_refuse(fn, x, dt, A, Bm, Cm, state_pool, lens, idx, nacc, D, z, dt_bias, out,
                    state_out, workspace)
        B, T, Ch = x.shape
        if VALIDATE and B:
            _validate_given(lens, idx, nacc, B, T, state_pool.shape[0], x.device, stream)
        if stream is not None:
            if out is None:
                out = _empty(x.shape, x.dtype, x.device, stream)
            if fn == "ssm_prefill" and workspace is None:
                size = ssm_prefill_workspace_size(B, T, Ch, A.shape[1], Bm.shape[2], x.device)
                if size:
                    workspace = _empty(size, torch.uint8, x.device, stream)
    done = _quick.scan(fn == "ssm_prefill", x, dt, A, Bm, Cm, state_pool, lens, idx, nacc, D, z,
                       dt_bias, SSM_DT_SOFTPLUS if dt_softplus else 0, out, state_out, workspace,
                       _raw_stream(x, stream))
    if done is None:
        _ssm_refuse(fn, x, dt, A, Bm, Cm, state_pool, lens, idx, nacc, D, z, dt_bias, out,
                    state_out, workspace)
        raise RuntimeError(f"{fn}: unsupported arguments")
    rc, out = done
    if rc:
        _check(rc, fn)
    if stream is not None:
        _hold(stream, x, dt, A, Bm, Cm, state_pool, lens, idx, nacc, D, z, dt_bias, out, state_out,
              workspace)
    return out, state_out


def ssm_decode(x, dt, A, B, C, state_pool, actual_seq_lengths=None, ssm_state_indices=None,
               num_accepted_tokens=None, *, D=None, z=None, dt_bias=None, dt_softplus=True,
               out=None, state_out=None, stream=None):
    """The selective state space scan, T <= 8 tokens per entry: for each channel, on its N states,
    ``d = softplus(dt + dt_bias)``, ``h = exp(d A) h + d x B``, ``y = (C . h + D x) silu(z)``;
    returns ``(out, state_out)``.

    x, dt, z ``[B,T,C]`` and B, C ``[B,T,G,N]`` (group g serves channels g C/G on) of one type,
    float32, float16 or bfloat16, any strides with the last axis contiguous and rows at multiples of
    8 elements (columns of a wider projection are fine); C/G a multiple of 8, N 8, 16 or 32. A
    float32 ``[C,N]``, D and dt_bias float32 ``[C]``; D, z and dt_bias may be left out.
    ``dt_softplus=False`` takes ``d = dt + dt_bias``. state_pool float32 or bfloat16
    ``[N_slots,C,N]``, updated in place unless ``state_out`` is given; a new sequence's slot is
    zeros. The index arrays are int32 ``[B]``, each may be left out, as in ``la_decode``."""
    return _ssm_call("ssm_decode", x, dt, A, B, C, state_pool, actual_seq_lengths,
                     ssm_state_indices, num_accepted_tokens, D, z, dt_bias, dt_softplus, out,
                     state_out, stream)


def ssm_prefill(x, dt, A, B, C, state_pool, actual_seq_lengths=None, ssm_state_indices=None,
                num_accepted_tokens=None, *, D=None, z=None, dt_bias=None, dt_softplus=True,
                workspace=None, out=None, state_out=None, stream=None):
    """``ssm_decode`` over whole prompts (T up to 65536); arguments and results as there.

    ``workspace``: a uint8 CUDA tensor of ``ssm_prefill_workspace_size`` bytes for calls of few
    channels, which then work on parts of a prompt at once; allocated for the call when None."""
    return _ssm_call("ssm_prefill", x, dt, A, B, C, state_pool, actual_seq_lengths,
                     ssm_state_indices, num_accepted_tokens, D, z, dt_bias, dt_softplus, out,
                     state_out, stream, workspace)


def ssm_prefill_workspace_size(B, T, channels, N, groups=1, device=None):
    """Bytes of workspace that ``ssm_prefill`` uses for a call of B entries, T tokens and so many
    channels of N states in so many groups on ``device`` (0: it needs none)."""
    lib = library()
    n = C.c_size_t(0)
    with torch.cuda.device(device if device is not None else torch.cuda.current_device()):
        rc = lib.ssm_prefill_workspace_size(B, T, channels, N, groups, C.byref(n))
    _check(rc, "ssm_prefill_workspace_size")
    return n.value


def rgdr_validate(actual_seq_lengths, ssm_state_indices, num_accepted_tokens, T, N_slots,
                  stream=None):
    """Synchronous check of device index arrays; returns the status code (0 = valid)."""
    lib = library()
    B = actual_seq_lengths.shape[0]
    for nm, t in (("actual_seq_lengths", actual_seq_lengths),
                  ("ssm_state_indices", ssm_state_indices),
                  ("num_accepted_tokens", num_accepted_tokens)):
        _dev(t, nm, torch.int32, 1)
        if t.shape[0] != B:
            raise RuntimeError(f"{nm} must have shape [{B}]")
    _same_device(actual_seq_lengths, ssm_state_indices=ssm_state_indices,
                 num_accepted_tokens=num_accepted_tokens)
    with torch.cuda.device(actual_seq_lengths.device):
        return lib.rgdr_validate(actual_seq_lengths.data_ptr(), ssm_state_indices.data_ptr(),
                                 num_accepted_tokens.data_ptr(), B, T, N_slots,
                                 _stream_handle(stream, actual_seq_lengths.device))


def rgdr_validate_host(actual_seq_lengths, ssm_state_indices, num_accepted_tokens, T, N_slots):
    """The same checks on host (CPU) int32 tensors; returns the status code."""
    lib = library()
    ts = [torch.as_tensor(x, dtype=torch.int32).contiguous()
          for x in (actual_seq_lengths, ssm_state_indices, num_accepted_tokens)]
    B = ts[0].shape[0]
    return lib.rgdr_validate_host(ts[0].data_ptr(), ts[1].data_ptr(), ts[2].data_ptr(),
                                  B, T, N_slots)
