"""GB300 (sm_103a) normalised causal linear attention with a recurrent S/z state.

    phi(x) = ELU(x) + 1
    S_t = alpha_t S_{t-1} + phi(k_t) v_t^T,   z_t = alpha_t z_{t-1} + phi(k_t)
    y_t = phi(q_t)^T S_t / (phi(q_t)^T z_t + eps)

and its relatives on the same states: the delta rule (delta_rule*), linear attention with a
constant decay per head (decay_*), and what a beam search does with states between
decode steps (beam_select, state_reorder).

Every step runs in the CUDA kernels of liblinattn.so, reached through its C ABI
(include/linattn.h).  The functions below only check tensor metadata, allocate
outputs with torch, and pass raw device pointers and the current CUDA stream;
PyTorch supplies device memory and streams, nothing else.
"""
from __future__ import annotations

import torch

from . import _native
from ._native import LinAttnError  # noqa: F401

_DTYPES = {torch.bfloat16: _native.LA_DTYPE_BF16, torch.float32: _native.LA_DTYPE_FP32}


def _ptr(t):
    return None if t is None else t.data_ptr()


def _stream(device):
    return torch.cuda.current_stream(device).cuda_stream


def _device_guard(device):
    """Makes `device` current for the duration of a library call.  The library
    launches on the current device (the default stream's handle 0 names that
    device's stream) and keeps its per-device state (status word, scratch, SM
    count) for the current device, so the tensors' device must be current."""
    return torch.cuda.device(device)


def _require(t, name, shape, dtype, device):
    if t is None:
        return
    if not t.is_cuda or t.device != device:
        raise ValueError(f"{name} must be on {device}")
    if tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {tuple(shape)}")
    if t.dtype != dtype:
        raise ValueError(f"{name} has dtype {t.dtype}, expected {dtype}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")


def state_init(B, H, r, dv, device="cuda", S=None, z=None):
    """Zero state: returns (S [B,H,r,dv], z [B,H,r]) in FP32."""
    device = torch.device(device)
    if S is None:
        S = torch.empty((B, H, r, dv), device=device, dtype=torch.float32)
    if z is None:
        z = torch.empty((B, H, r), device=device, dtype=torch.float32)
    _require(S, "S", (B, H, r, dv), torch.float32, S.device)
    _require(z, "z", (B, H, r), torch.float32, S.device)
    with _device_guard(S.device):
        st = _native.lib().la_state_init(_ptr(S), _ptr(z), B, H, r, dv, _stream(S.device))
    _native.check(st, "la_state_init")
    return S, z


def prefill_workspace_bytes(B, H, T, r, dv, chunk=64, device=None) -> int:
    """Scratch bytes of prefill_chunked for these sizes on `device` (default: the
    current device); the plan depends on the device's SM count."""
    if device is None:
        return int(_native.lib().la_prefill_workspace_bytes(B, H, T, r, dv, chunk))
    with _device_guard(torch.device(device)):
        return int(_native.lib().la_prefill_workspace_bytes(B, H, T, r, dv, chunk))


def prefill_chunked(q, k, v, alpha=None, S0=None, z0=None, chunk=64, eps=1e-6, y=None, S_out=None, z_out=None,
                    workspace=None):
    """Chunkwise prefill.  q, k [B,H,T,r], v [B,H,T,dv] (bf16 or fp32, same dtype);
    alpha [B,H,T] fp32 or None; S0 [B,H,r,dv], z0 [B,H,r] fp32 or None.
    Returns (y [B,H,T,dv] in the input dtype, S_T, z_T)."""
    return _prefill(q, k, v, alpha, S0, z0, chunk, eps, y, S_out, z_out, workspace, None)


def backward_states_bytes(B, H, T, device=None) -> int:
    """Bytes of the states a training forward can keep for the backward's sequence
    segments on `device` (0: the backward would not split the sequence)."""
    if device is None:
        return int(_native.lib().la_backward_states_bytes(B, H, T))
    with _device_guard(torch.device(device)):
        return int(_native.lib().la_backward_states_bytes(B, H, T))


def prefill_chunked_save(q, k, v, alpha=None, S0=None, z0=None, chunk=64, eps=1e-6, y=None, S_out=None, z_out=None,
                         d_out=None, workspace=None, keep_states=True):
    """prefill_chunked that also returns what the backward can reuse: d [B,H,T]
    fp32, the denominator of every output row (phi(q_t) . z_t + eps), and the
    states entering the backward's sequence segments (a flat fp32 tensor, or None
    when there are none or keep_states is False), for
    prefill_backward(..., d=d, states=states).  Returns (y, S_T, z_T, d, states)."""
    B, H, T, _ = q.shape
    if d_out is None:
        d_out = torch.empty((B, H, T), device=q.device, dtype=torch.float32)
    _require(d_out, "d_out", (B, H, T), torch.float32, q.device)
    states = None
    if keep_states and q.dtype == torch.bfloat16:
        nbytes = backward_states_bytes(B, H, T, device=q.device)
        if nbytes:
            states = torch.empty(nbytes // 4, device=q.device, dtype=torch.float32)
    return _prefill(q, k, v, alpha, S0, z0, chunk, eps, y, S_out, z_out, workspace, d_out, states) + (d_out, states)


def _prefill(q, k, v, alpha, S0, z0, chunk, eps, y, S_out, z_out, workspace, d_out, states=None):
    if q.dtype not in _DTYPES:
        raise ValueError(f"unsupported dtype {q.dtype}")
    B, H, T, r = q.shape
    dv = v.shape[3]
    dev = q.device
    _require(q, "q", (B, H, T, r), q.dtype, dev)
    _require(k, "k", (B, H, T, r), q.dtype, dev)
    _require(v, "v", (B, H, T, dv), q.dtype, dev)
    _require(alpha, "alpha", (B, H, T), torch.float32, dev)
    _require(S0, "S0", (B, H, r, dv), torch.float32, dev)
    _require(z0, "z0", (B, H, r), torch.float32, dev)
    if y is None:
        y = torch.empty((B, H, T, dv), device=dev, dtype=q.dtype)
    if S_out is None:
        S_out = torch.empty((B, H, r, dv), device=dev, dtype=torch.float32)
    if z_out is None:
        z_out = torch.empty((B, H, r), device=dev, dtype=torch.float32)
    _require(y, "y", (B, H, T, dv), q.dtype, dev)
    _require(S_out, "S_out", (B, H, r, dv), torch.float32, dev)
    _require(z_out, "z_out", (B, H, r), torch.float32, dev)
    need = prefill_workspace_bytes(B, H, T, r, dv, chunk, device=dev)
    if need and workspace is None:
        workspace = torch.empty(need, device=dev, dtype=torch.uint8)
    ws_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    with _device_guard(dev):
        if d_out is None:
            st = _native.lib().la_prefill_chunked(
                _ptr(q), _ptr(k), _ptr(v), _DTYPES[q.dtype], _ptr(alpha), _ptr(S0), _ptr(z0), B, H, T, r, dv, chunk,
                float(eps), _ptr(y), _ptr(S_out), _ptr(z_out), _ptr(workspace), ws_bytes, _stream(dev))
            _native.check(st, "la_prefill_chunked")
        else:
            st = _native.lib().la_prefill_chunked_save(
                _ptr(q), _ptr(k), _ptr(v), _DTYPES[q.dtype], _ptr(alpha), _ptr(S0), _ptr(z0), B, H, T, r, dv, chunk,
                float(eps), _ptr(y), _ptr(S_out), _ptr(z_out), _ptr(d_out), _ptr(states), _ptr(workspace), ws_bytes,
                _stream(dev))
            _native.check(st, "la_prefill_chunked_save")
    return y, S_out, z_out


def varlen_workspace_bytes(B, H, total_T, r, dv, device=None) -> int:
    """Scratch bytes of prefill_varlen for these sizes on `device` (default: the
    current device); it depends on the device's SM count, not on the lengths."""
    if device is None:
        return int(_native.lib().la_prefill_varlen_workspace_bytes(B, H, total_T, r, dv))
    with _device_guard(torch.device(device)):
        return int(_native.lib().la_prefill_varlen_workspace_bytes(B, H, total_T, r, dv))


def prefill_varlen(q, k, v, cu_seqlens, alpha=None, S0=None, z0=None, chunk=64, eps=1e-6, y=None, S_out=None,
                   z_out=None, workspace=None):
    """Packed sequences of different lengths: q, k [total_T, H, r], v [total_T, H, dv]
    (bf16, token-major); cu_seqlens int32 [B+1] on the device (sequence b is tokens
    cu_seqlens[b] .. cu_seqlens[b+1]-1); alpha [total_T, H] fp32 or None; S0
    [B,H,r,dv], z0 [B,H,r] fp32 or None; workspace uint8 of varlen_workspace_bytes
    (allocated here when None).  Returns (y [total_T, H, dv], S_T, z_T)."""
    if q.dtype not in _DTYPES:
        raise ValueError(f"unsupported dtype {q.dtype}")
    total_T, H, r = q.shape
    dv = v.shape[2]
    dev = q.device
    if cu_seqlens.dtype != torch.int32 or cu_seqlens.dim() != 1 or cu_seqlens.device != dev:
        raise ValueError("cu_seqlens must be a 1-D int32 tensor on the device of q")
    B = cu_seqlens.numel() - 1
    _require(q, "q", (total_T, H, r), q.dtype, dev)
    _require(k, "k", (total_T, H, r), q.dtype, dev)
    _require(v, "v", (total_T, H, dv), q.dtype, dev)
    _require(cu_seqlens, "cu_seqlens", (B + 1,), torch.int32, dev)
    _require(alpha, "alpha", (total_T, H), torch.float32, dev)
    _require(S0, "S0", (B, H, r, dv), torch.float32, dev)
    _require(z0, "z0", (B, H, r), torch.float32, dev)
    if y is None:
        y = torch.empty((total_T, H, dv), device=dev, dtype=q.dtype)
    if S_out is None:
        S_out = torch.empty((B, H, r, dv), device=dev, dtype=torch.float32)
    if z_out is None:
        z_out = torch.empty((B, H, r), device=dev, dtype=torch.float32)
    _require(y, "y", (total_T, H, dv), q.dtype, dev)
    _require(S_out, "S_out", (B, H, r, dv), torch.float32, dev)
    _require(z_out, "z_out", (B, H, r), torch.float32, dev)
    need = varlen_workspace_bytes(B, H, total_T, r, dv, device=dev)
    if need and workspace is None:
        workspace = torch.empty(need, device=dev, dtype=torch.uint8)
    ws_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    with _device_guard(dev):
        st = _native.lib().la_prefill_varlen(
            _ptr(q), _ptr(k), _ptr(v), _DTYPES[q.dtype], _ptr(alpha), _ptr(S0), _ptr(z0), _ptr(cu_seqlens), B, H,
            total_T, r, dv, chunk, float(eps), _ptr(y), _ptr(S_out), _ptr(z_out), _ptr(workspace), ws_bytes,
            _stream(dev))
    _native.check(st, "la_prefill_varlen")
    return y, S_out, z_out


def prefill_chunked_noalloc(q, k, v, y, S_out, z_out, alpha=None, S0=None, z0=None, chunk=64, eps=1e-6):
    """As prefill_chunked, with the library's built-in scratch instead of a
    workspace; nothing is allocated here either, so y [B,H,T,dv] (input dtype),
    S_out [B,H,r,dv] and z_out [B,H,r] (fp32) must be given.  Calls that may
    overlap in time share one buffer per device and must be serialised."""
    if q.dtype not in _DTYPES:
        raise ValueError(f"unsupported dtype {q.dtype}")
    B, H, T, r = q.shape
    dv = v.shape[3]
    dev = q.device
    _require(q, "q", (B, H, T, r), q.dtype, dev)
    _require(k, "k", (B, H, T, r), q.dtype, dev)
    _require(v, "v", (B, H, T, dv), q.dtype, dev)
    _require(alpha, "alpha", (B, H, T), torch.float32, dev)
    _require(S0, "S0", (B, H, r, dv), torch.float32, dev)
    _require(z0, "z0", (B, H, r), torch.float32, dev)
    if y is None or S_out is None or z_out is None:
        raise ValueError("y, S_out and z_out must be given (this entry point allocates nothing)")
    _require(y, "y", (B, H, T, dv), q.dtype, dev)
    _require(S_out, "S_out", (B, H, r, dv), torch.float32, dev)
    _require(z_out, "z_out", (B, H, r), torch.float32, dev)
    with _device_guard(dev):
        st = _native.lib().la_prefill_chunked_noalloc(
            _ptr(q), _ptr(k), _ptr(v), _DTYPES[q.dtype], _ptr(alpha), _ptr(S0), _ptr(z0), B, H, T, r, dv, chunk,
            float(eps), _ptr(y), _ptr(S_out), _ptr(z_out), _stream(dev))
    _native.check(st, "la_prefill_chunked_noalloc")
    return y, S_out, z_out


def decode_step(q, k, v, S, z, alpha=None, eps=1e-6, y=None):
    """One token per request, state updated in place.  q, k [B,H,1,r], v [B,H,1,dv];
    S [B,H,r,dv], z [B,H,r] fp32 (overwritten); alpha [B,H] fp32 or None.  Returns y [B,H,1,dv]."""
    if q.dtype not in _DTYPES:
        raise ValueError(f"unsupported dtype {q.dtype}")
    B, H, one, r = q.shape
    dv = v.shape[3]
    dev = q.device
    if one != 1:
        raise ValueError("decode takes one token per request")
    _require(k, "k", (B, H, 1, r), q.dtype, dev)
    _require(v, "v", (B, H, 1, dv), q.dtype, dev)
    _require(S, "S", (B, H, r, dv), torch.float32, dev)
    _require(z, "z", (B, H, r), torch.float32, dev)
    _require(alpha, "alpha", (B, H), torch.float32, dev)
    if y is None:
        y = torch.empty((B, H, 1, dv), device=dev, dtype=q.dtype)
    _require(y, "y", (B, H, 1, dv), q.dtype, dev)
    with _device_guard(dev):
        st = _native.lib().la_decode_step(_ptr(q), _ptr(k), _ptr(v), _DTYPES[q.dtype], _ptr(alpha), _ptr(S), _ptr(z),
                                          B, H, r, dv, float(eps), _ptr(y), _stream(dev))
    _native.check(st, "la_decode_step")
    return y


def prefill_backward(q, k, v, y, dy, alpha=None, S0=None, z0=None, dS_T=None, dz_T=None, eps=1e-6, workspace=None,
                     d=None, states=None):
    """Gradients of prefill_chunked: given the forward inputs, its output y and
    dy [B,H,T,dv] (and optionally dS_T [B,H,r,dv], dz_T [B,H,r] in fp32), returns
    (dq, dk, dv, dalpha or None, dS0, dz0); dq, dk, dv in the input dtype.
    d: the [B,H,T] fp32 denominators from prefill_chunked_save (eps is then not
    used), or None to recompute them; states: the segment states from the same
    call (with d only), or None."""
    if states is not None and d is None:
        raise ValueError("states are taken only together with d")
    if q.dtype not in _DTYPES:
        raise ValueError(f"unsupported dtype {q.dtype}")
    B, H, T, r = q.shape
    dvd = v.shape[3]
    dev = q.device
    for t, name, shape in ((q, "q", (B, H, T, r)), (k, "k", (B, H, T, r)), (v, "v", (B, H, T, dvd)),
                           (y, "y", (B, H, T, dvd)), (dy, "dy", (B, H, T, dvd))):
        _require(t, name, shape, q.dtype, dev)
    _require(alpha, "alpha", (B, H, T), torch.float32, dev)
    _require(S0, "S0", (B, H, r, dvd), torch.float32, dev)
    _require(z0, "z0", (B, H, r), torch.float32, dev)
    _require(dS_T, "dS_T", (B, H, r, dvd), torch.float32, dev)
    _require(dz_T, "dz_T", (B, H, r), torch.float32, dev)
    _require(d, "d", (B, H, T), torch.float32, dev)
    dq, dk, dv_out = torch.empty_like(q), torch.empty_like(k), torch.empty_like(v)
    dalpha = torch.empty((B, H, T), device=dev, dtype=torch.float32) if alpha is not None else None
    dS0 = torch.empty((B, H, r, dvd), device=dev, dtype=torch.float32)
    dz0 = torch.empty((B, H, r), device=dev, dtype=torch.float32)
    need = int(_native.lib().la_backward_workspace_bytes(B, H, T))
    if workspace is None:
        workspace = torch.empty(need, device=dev, dtype=torch.uint8)
    ws_bytes = workspace.numel() * workspace.element_size()
    with _device_guard(dev):
        if d is None:
            st = _native.lib().la_prefill_backward(
                _ptr(q), _ptr(k), _ptr(v), _DTYPES[q.dtype], _ptr(alpha), _ptr(S0), _ptr(z0), B, H, T, r, dvd,
                float(eps), _ptr(y), _ptr(dy), _ptr(dS_T), _ptr(dz_T), _ptr(dq), _ptr(dk), _ptr(dv_out), _ptr(dalpha),
                _ptr(dS0), _ptr(dz0), _ptr(workspace), ws_bytes, _stream(dev))
            _native.check(st, "la_prefill_backward")
        else:
            st = _native.lib().la_prefill_backward_saved(
                _ptr(q), _ptr(k), _ptr(v), _DTYPES[q.dtype], _ptr(alpha), _ptr(S0), _ptr(z0), B, H, T, r, dvd,
                _ptr(y), _ptr(dy), _ptr(d), _ptr(states), _ptr(dS_T), _ptr(dz_T), _ptr(dq), _ptr(dk), _ptr(dv_out),
                _ptr(dalpha), _ptr(dS0), _ptr(dz0), _ptr(workspace), ws_bytes, _stream(dev))
            _native.check(st, "la_prefill_backward_saved")
    return dq, dk, dv_out, dalpha, dS0, dz0


def delta_rule(q, k, v, beta=None, S0=None, y=None, S_out=None):
    """Delta-rule memory: p = S^T k, S += beta k (v - p)^T, y = S^T q (after the write).
    q, k [B,H,T,r], v [B,H,T,dv] (bf16 or fp32, same dtype); beta [B,H,T] fp32 or
    None (1); S0 [B,H,r,dv] fp32 or None (zero).  Returns (y [B,H,T,dv], S_T).
    The token recurrence in FP32 (la_delta_rule)."""
    return _delta("la_delta_rule", q, k, v, beta, S0, y, S_out, None)


def delta_chunked_workspace_bytes(B, H, T) -> int:
    return int(_native.lib().la_delta_chunked_workspace_bytes(B, H, T))


def delta_rule_chunked(q, k, v, beta=None, S0=None, y=None, S_out=None, workspace=None):
    """The same memory in chunks of 64 tokens on the tensor cores (la_delta_rule_chunked):
    bf16 q, k [B,H,T,128], v [B,H,T,dv] with dv a multiple of 64; BF16 operands,
    FP32 state.  workspace: a device buffer of delta_chunked_workspace_bytes bytes
    (allocated here when None).  Returns (y [B,H,T,dv], S_T)."""
    B, H, T = q.shape[:3]
    if workspace is None and T > 0:
        workspace = torch.empty(delta_chunked_workspace_bytes(B, H, T), device=q.device, dtype=torch.uint8)
    return _delta("la_delta_rule_chunked", q, k, v, beta, S0, y, S_out, workspace)


def _delta(entry, q, k, v, beta, S0, y, S_out, workspace):
    if q.dtype not in _DTYPES:
        raise ValueError(f"unsupported dtype {q.dtype}")
    B, H, T, r = q.shape
    dv = v.shape[3]
    dev = q.device
    _require(q, "q", (B, H, T, r), q.dtype, dev)
    _require(k, "k", (B, H, T, r), q.dtype, dev)
    _require(v, "v", (B, H, T, dv), q.dtype, dev)
    _require(beta, "beta", (B, H, T), torch.float32, dev)
    _require(S0, "S0", (B, H, r, dv), torch.float32, dev)
    if y is None:
        y = torch.empty((B, H, T, dv), device=dev, dtype=q.dtype)
    if S_out is None:
        S_out = torch.empty((B, H, r, dv), device=dev, dtype=torch.float32)
    _require(y, "y", (B, H, T, dv), q.dtype, dev)
    _require(S_out, "S_out", (B, H, r, dv), torch.float32, dev)
    args = [_ptr(q), _ptr(k), _ptr(v), _DTYPES[q.dtype], _ptr(beta), _ptr(S0), B, H, T, r, dv, _ptr(y), _ptr(S_out)]
    if entry == "la_delta_rule_chunked":
        args += [_ptr(workspace), 0 if workspace is None else workspace.numel() * workspace.element_size()]
    with _device_guard(dev):
        st = getattr(_native.lib(), entry)(*args, _stream(dev))
    _native.check(st, entry)
    return y, S_out


def _workspace(workspace, need, device):
    """The caller's workspace, or one of `need` bytes (None when there is no need for one), and its size."""
    if workspace is None:
        return (torch.empty(need, device=device, dtype=torch.uint8), need) if need else (None, 0)
    if not workspace.is_cuda or workspace.device != device or not workspace.is_contiguous():
        raise ValueError(f"workspace must be contiguous and on {device}")
    return workspace, workspace.numel() * workspace.element_size()


def _call(entry, device, *args):
    """One library call on `device` and its current stream (appended to args)."""
    fn = getattr(_native.lib(), entry)
    index = device.index
    if index == torch.cuda.current_device():
        st = fn(*args, torch._C._cuda_getCurrentRawStream(index))
    else:
        with _device_guard(device):
            st = fn(*args, _stream(device))
    if st:
        _native.check(st, entry)


def _want(t, name, shape, dtype, device):
    """_require for a tensor that must be given: one pass over what it compares, as these calls may be
    a few microseconds long."""
    if t.shape != shape or t.dtype != dtype or t.device != device or not t.is_contiguous() or not t.is_cuda:
        _require(t, name, shape, dtype, device)


def _out(t, name, shape, dtype, device):
    """The caller's output tensor, or a new one."""
    if t is None:
        return torch.empty(shape, dtype=dtype, device=device)
    _want(t, name, shape, dtype, device)
    return t


def _decay_inputs(q, k, v, decay, shape_qk, shape_v, H):
    dt = q.dtype
    if dt not in _DTYPES:
        raise ValueError(f"unsupported dtype {dt}")
    dev = q.device
    _want(q, "q", shape_qk, dt, dev)
    _want(k, "k", shape_qk, dt, dev)
    _want(v, "v", shape_v, dt, dev)
    if decay is None:
        raise ValueError("decay must be given (ones for no decay)")
    _want(decay, "decay", (H,), torch.float32, dev)
    return dt, dev


def _bytes(entry, device, *args):
    if device is None or device.index == torch.cuda.current_device():
        return int(getattr(_native.lib(), entry)(*args))
    with _device_guard(device):
        return int(getattr(_native.lib(), entry)(*args))


def decay_prefill_workspace_bytes(B, H, T, r, dv, dtype=torch.bfloat16, device=None) -> int:
    """Scratch bytes of decay_prefill for these sizes on `device` (default: the current one)."""
    return _bytes("la_decay_prefill_workspace_bytes", None if device is None else torch.device(device), B, H, T, r, dv,
                  _DTYPES[dtype])


def decay_prefill(q, k, v, decay, S0=None, scale=1.0, y=None, S_out=None, workspace=None):
    """Linear attention with a constant decay per head: S <- decay S + k v^T, y = scale S^T q.
    q, k [B,H,T,r], v [B,H,T,dv] (bf16 or fp32, same dtype); decay [H] fp32 in 0..1; S0
    [B,H,r,dv] fp32 or None (zero).  Returns (y [B,H,T,dv] in the input dtype, S_T).
    Prompts run on the tensor cores when they are bf16, r is 64 or 128, dv a multiple of 64 and
    q, k, v, y start on 16-byte boundaries (a slice at an odd offset may not); everything else, and
    fp32 for a state to fp32's own rounding, takes the token recurrence, several times slower."""
    B, H, T, r = q.shape
    dv = v.shape[3]
    dt, dev = _decay_inputs(q, k, v, decay, (B, H, T, r), (B, H, T, dv), H)
    if S0 is not None:
        _want(S0, "S0", (B, H, r, dv), torch.float32, dev)
    y = _out(y, "y", (B, H, T, dv), dt, dev)
    S_out = _out(S_out, "S_out", (B, H, r, dv), torch.float32, dev)
    dt = _DTYPES[dt]
    workspace, ws_bytes = _workspace(workspace, _bytes("la_decay_prefill_workspace_bytes", dev, B, H, T, r, dv, dt), dev)
    _call("la_decay_prefill", dev, q.data_ptr(), k.data_ptr(), v.data_ptr(), dt, decay.data_ptr(), _ptr(S0), B, H, T, r,
          dv, scale, y.data_ptr(), S_out.data_ptr(), _ptr(workspace), ws_bytes)
    return y, S_out


def decay_prefill_varlen(q, k, v, decay, cu_seqlens, S0=None, scale=1.0, y=None, S_out=None):
    """decay_prefill for packed sequences: q, k [total_T, H, r], v [total_T, H, dv]
    (token-major); cu_seqlens int32 [B+1] on the device (sequence b is tokens
    cu_seqlens[b] .. cu_seqlens[b+1]-1); S0 [B,H,r,dv] fp32 or None.  Returns
    (y [total_T, H, dv], S_T [B,H,r,dv])."""
    total_T, H, r = q.shape
    dv = v.shape[2]
    dt, dev = _decay_inputs(q, k, v, decay, (total_T, H, r), (total_T, H, dv), H)
    if cu_seqlens.dtype != torch.int32 or cu_seqlens.dim() != 1 or cu_seqlens.device != dev:
        raise ValueError("cu_seqlens must be a 1-D int32 tensor on the device of q")
    B = cu_seqlens.numel() - 1
    _want(cu_seqlens, "cu_seqlens", (B + 1,), torch.int32, dev)
    if S0 is not None:
        _want(S0, "S0", (B, H, r, dv), torch.float32, dev)
    y = _out(y, "y", (total_T, H, dv), dt, dev)
    S_out = _out(S_out, "S_out", (B, H, r, dv), torch.float32, dev)
    _call("la_decay_prefill_varlen", dev, q.data_ptr(), k.data_ptr(), v.data_ptr(), _DTYPES[dt], decay.data_ptr(),
          _ptr(S0), cu_seqlens.data_ptr(), B, H, total_T, r, dv, scale, y.data_ptr(), S_out.data_ptr())
    return y, S_out


def decay_decode_step(q, k, v, decay, S, scale=1.0, y=None):
    """One token per request of decay_prefill, S [B,H,r,dv] fp32 updated in place.
    q, k [B,H,1,r], v [B,H,1,dv]; decay [H] fp32.  Returns y [B,H,1,dv]."""
    B, H, one, r = q.shape
    dv = v.shape[3]
    if one != 1:
        raise ValueError("decode takes one token per request")
    dt, dev = _decay_inputs(q, k, v, decay, (B, H, 1, r), (B, H, 1, dv), H)
    _want(S, "S", (B, H, r, dv), torch.float32, dev)
    y = _out(y, "y", (B, H, 1, dv), dt, dev)
    _call("la_decay_decode_step", dev, q.data_ptr(), k.data_ptr(), v.data_ptr(), _DTYPES[dt], decay.data_ptr(),
          S.data_ptr(), B, H, r, dv, scale, y.data_ptr())
    return y


def decay_backward_workspace_bytes(B, H, T, r, dv, dtype=torch.bfloat16, device=None) -> int:
    """Scratch bytes of decay_backward for these sizes on `device` (default: the current one)."""
    return _bytes("la_decay_backward_workspace_bytes", None if device is None else torch.device(device), B, H, T, r, dv,
                  _DTYPES[dtype])


def decay_backward(q, k, v, dy, decay, S0=None, dS_T=None, scale=1.0, workspace=None):
    """Gradients of decay_prefill: from its inputs, dy [B,H,T,dv] and optionally dS_T
    [B,H,r,dv] fp32, returns (dq, dk, dv, dS0); dq, dk, dv in the input dtype, dS0 in
    fp32.  The decay is a constant of the head and gets no gradient."""
    B, H, T, r = q.shape
    dvd = v.shape[3]
    dt, dev = _decay_inputs(q, k, v, decay, (B, H, T, r), (B, H, T, dvd), H)
    _want(dy, "dy", (B, H, T, dvd), dt, dev)
    if S0 is not None:
        _want(S0, "S0", (B, H, r, dvd), torch.float32, dev)
    if dS_T is not None:
        _want(dS_T, "dS_T", (B, H, r, dvd), torch.float32, dev)
    dq, dk, dv_out = torch.empty_like(q), torch.empty_like(k), torch.empty_like(v)
    dS0 = torch.empty((B, H, r, dvd), device=dev, dtype=torch.float32)
    dt = _DTYPES[dt]
    workspace, ws_bytes = _workspace(workspace, _bytes("la_decay_backward_workspace_bytes", dev, B, H, T, r, dvd, dt), dev)
    _call("la_decay_backward", dev, q.data_ptr(), k.data_ptr(), v.data_ptr(), dt, decay.data_ptr(), _ptr(S0), B, H, T, r,
          dvd, scale, dy.data_ptr(), _ptr(dS_T), dq.data_ptr(), dk.data_ptr(), dv_out.data_ptr(), dS0.data_ptr(),
          _ptr(workspace), ws_bytes)
    return dq, dk, dv_out, dS0


def beam_select(logits, scores, done=None, eos=-1, next_scores=None, parents=None, tokens=None, done_out=None):
    """A beam search's choice: the best K of K beams x V tokens of every request, by
    scores + log_softmax(logits), best first, ties to the lower k V + v.
    logits [B,K,V] (bf16 or fp32; rows may be padded: any stride between them, one for
    all); scores [B,K] fp32; done [B,K] uint8 or None: beams that have ended (their one
    candidate is the token eos, the score unchanged); eos the token that ends a beam, -1 none.
    Returns (next_scores [B,K] fp32, parents [B,K] int32, tokens [B,K] int32, done_out
    [B,K] uint8).  A slot without a candidate has score -inf, itself as parent and token 0."""
    dt = logits.dtype
    if dt not in _DTYPES:
        raise ValueError(f"unsupported dtype {dt}")
    if not logits.is_cuda:
        raise ValueError("logits must be on a CUDA device")
    B, K, V = logits.shape
    dev = logits.device
    if logits.is_contiguous():
        stride = V
    else:
        stride = logits.stride(1) if K > 1 else logits.stride(0) if B > 1 else V
        if (V > 1 and logits.stride(2) != 1) or (B > 1 and K > 1 and logits.stride(0) != K * stride):
            raise ValueError("logits must have contiguous rows at one stride")
    bk = (B, K)
    _want(scores, "scores", bk, torch.float32, dev)
    if done is not None:
        _want(done, "done", bk, torch.uint8, dev)
    next_scores = _out(next_scores, "next_scores", bk, torch.float32, dev)
    parents = _out(parents, "parents", bk, torch.int32, dev)
    tokens = _out(tokens, "tokens", bk, torch.int32, dev)
    done_out = _out(done_out, "done_out", bk, torch.uint8, dev)
    _call("la_beam_select", dev, logits.data_ptr(), _DTYPES[dt], stride, scores.data_ptr(), _ptr(done), B, K, V, eos,
          next_scores.data_ptr(), parents.data_ptr(), tokens.data_ptr(), done_out.data_ptr())
    return next_scores, parents, tokens, done_out


def state_reorder(S, parents, z=None, S_out=None, z_out=None):
    """Moves recurrent states after a beam search's choice: slot j of request b receives
    the state of its slot parents[b, j].  S [B*K,H,r,dv], z [B*K,H,r] fp32 (or None);
    parents [B,K] int32 on the device.  In place unless S_out (and z_out) are given.
    Returns (S_out, z_out)."""
    if parents.dim() != 2:
        raise ValueError("parents must be [B, K]")
    B, K = parents.shape
    n, H, r, dv = S.shape
    dev = S.device
    _want(parents, "parents", (B, K), torch.int32, dev)
    _want(S, "S", (B * K, H, r, dv), torch.float32, dev)
    if z is not None:
        _want(z, "z", (B * K, H, r), torch.float32, dev)
    elif z_out is not None:
        raise ValueError("z_out is taken only together with z")
    if S_out is None:
        if z_out is not None:
            raise ValueError("z_out is taken only together with S_out")
        S_out, z_out = S, z
    else:
        _want(S_out, "S_out", (B * K, H, r, dv), torch.float32, dev)
        if z is not None:
            if z_out is None:
                z_out = z if S_out.data_ptr() == S.data_ptr() else torch.empty_like(z)
            _want(z_out, "z_out", (B * K, H, r), torch.float32, dev)
    _call("la_state_reorder", dev, S.data_ptr(), _ptr(z), parents.data_ptr(), B, K, H, r, dv, S_out.data_ptr(), _ptr(z_out))
    return S_out, z_out


def last_device_status(device="cuda") -> int:
    """Synchronises the current stream and returns (and clears) the device status word."""
    dev = torch.device(device)
    with _device_guard(dev):
        return int(_native.lib().la_last_device_status(_stream(dev)))
