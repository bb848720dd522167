"""Binding of the selective state space scan, its single-token step and the norms
around a block (C ABI in ``include/gdn.h``; argument marshalling only)."""
from __future__ import annotations

import contextlib

import torch

from .gdn import CONV_SILU, GDN_BF16, GDN_F32, GDN_OK, GDNError, load_library

SSM_SOFTPLUS = 32      # GDN_SSM_SOFTPLUS
GATE_SILU, NORM_GATE_FIRST, NORM_UNIT_OFFSET = 64, 128, 256

_CODES = {torch.bfloat16: GDN_BF16, torch.float32: GDN_F32}


def _code(t, name):
    code = _CODES.get(t.dtype)
    if code is None:
        raise TypeError(f"{name} must be bfloat16 or float32, got {t.dtype}")
    return code


def _check(t, name, shape, dtype, dev, strided=False):
    """Address of a CUDA tensor of this shape, dtype and device, contiguous unless `strided`."""
    if isinstance(t, torch.Tensor) and t.get_device() == dev.index and t.dtype is dtype and \
            t.shape == shape and (strided or t.is_contiguous()):
        return t.data_ptr()
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.device != dev:
        raise ValueError(f"{name} is on {t.device}, expected {dev}")
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if t.shape != shape:
        raise ValueError(f"{name} must be {tuple(shape)}, got {tuple(t.shape)}")
    raise ValueError(f"{name} must be contiguous")


def _opt(t, name, shape, dtype, dev):
    return None if t is None else _check(t, name, shape, dtype, dev)


def _rows(t, name, inner):
    """Elements between the rows of `t`, whose last `inner` dimensions are one dense row
    and whose leading dimensions are evenly spaced."""
    if t.is_contiguous():
        return 0
    size, stride = t.shape, t.stride()
    want = 1
    for i in range(t.dim() - 1, t.dim() - 1 - inner, -1):
        if size[i] != 1 and stride[i] != want:
            raise ValueError(f"the rows of {name} must be contiguous")
        want *= size[i]
    row = step = None
    for i in range(t.dim() - 1 - inner, -1, -1):
        if size[i] == 1:
            continue
        if row is None:
            row = step = stride[i]
            if row < want:
                raise ValueError(f"the rows of {name} overlap")
        elif stride[i] != step:
            raise ValueError(f"the rows of {name} must be evenly spaced")
        step *= size[i]
    return row or 0


def _cuda(t, name):
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.device.type != "cuda":
        raise ValueError(f"{name} must be a CUDA tensor (got {t.device})")
    return t.device


def _elsewhere(dev, stream):
    """Whether a call has to run on another stream or device than the current ones."""
    return stream is not None or dev.index != torch.cuda.current_device()


@contextlib.contextmanager
def _on(dev, stream):
    """The tensors' device and the caller's stream as the current ones, so that what is
    allocated here belongs to the stream that uses it."""
    with torch.cuda.device(dev):
        with torch.cuda.stream(stream if stream is not None else torch.cuda.current_stream(dev)):
            yield


def _raw_stream(dev):
    return torch._C._cuda_getCurrentRawStream(dev.index)


def gdn_ssm_prefill_workspace_size(N, T, HK, HV, dk, dv, dtype, varlen) -> int:
    """Bytes of workspace for ``gdn_ssm_prefill`` with at most N sequences and T tokens (0: none)."""
    code = dtype if isinstance(dtype, int) else _code(torch.empty(0, dtype=dtype), "dtype")
    return int(load_library().gdn_ssm_prefill_workspace_size(
        int(N), int(T), int(HK), int(HV), int(dk), int(dv), code, int(bool(varlen))))


def gdn_ssm_prefill(x, b, c, dt, a, d=None, dt_bias=None, h0=None, cu_seqlens=None,
                    softplus: bool = False, y=None, hT=None, workspace=None, stream=None,
                    output_final_state: bool = True):
    """Selective state space scan over prompts through ``gdn_ssm_prefill``.

    x [B,T,HV,dv]; b, c [B,T,HK,dk] (bf16 or fp32; each may be a part of a wider row, as
    the short convolution over x | b | c leaves them); dt [B,T,HV] fp32; a, d, dt_bias
    [HV] fp32 (d, dt_bias optional); h0 [N,HV,dv,dk] fp32 or None; cu_seqlens int32 [N+1]
    (then B == 1) or None.  ``softplus``: the step sizes are softplus(dt + dt_bias).
    Returns (y [B,T,HV,dv], hT [N,HV,dv,dk] or None).
    """
    lib = load_library()
    dev = _cuda(x, "x")
    if _elsewhere(dev, stream):
        with _on(dev, stream):
            return gdn_ssm_prefill(x, b, c, dt, a, d, dt_bias, h0, cu_seqlens, softplus, y, hT,
                                   workspace, None, output_final_state)
    code = _code(x, "x")
    if x.dim() != 4 or not isinstance(b, torch.Tensor) or b.dim() != 4:
        raise ValueError("expected x [B,T,HV,dv] and b, c [B,T,HK,dk]")
    B, T, HV, dv = x.shape
    HK, dk = b.shape[2], b.shape[3]
    _check(b, "b", (B, T, HK, dk), x.dtype, dev, True)
    _check(c, "c", (B, T, HK, dk), x.dtype, dev, True)
    f32 = torch.float32
    dt_p = _check(dt, "dt", (B, T, HV), f32, dev)
    a_p = _check(a, "a", (HV,), f32, dev)
    d_p = _opt(d, "d", (HV,), f32, dev)
    bias_p = _opt(dt_bias, "dt_bias", (HV,), f32, dev)
    N, cu_p = B, None
    if cu_seqlens is not None:
        if B != 1:
            raise ValueError("with cu_seqlens the batch dimension must be 1 (packed)")
        if cu_seqlens.dim() != 1 or cu_seqlens.numel() < 1:
            raise ValueError("cu_seqlens must be [N+1]")
        N = cu_seqlens.numel() - 1
        cu_p = _check(cu_seqlens, "cu_seqlens", (N + 1,), torch.int32, dev)
    h0_p = _opt(h0, "h0", (N, HV, dv, dk), f32, dev)
    x_row, b_row, c_row = _rows(x, "x", 2), _rows(b, "b", 2), _rows(c, "c", 2)
    y_p = None if y is None else _check(y, "y", (B, T, HV, dv), x.dtype, dev)
    if y is None:
        y = x.new_empty((B, T, HV, dv))
        y_p = y.data_ptr()
    hT_p = _opt(hT, "hT", (N, HV, dv, dk), f32, dev)
    if hT is None and output_final_state:
        hT = dt.new_empty((N, HV, dv, dk))
        hT_p = hT.data_ptr()
    ws_p, ws_bytes = None, 0
    if workspace is None:
        ws_bytes = lib.gdn_ssm_prefill_workspace_size(N, T, HK, HV, dk, dv, code, cu_p is not None)
        if ws_bytes:
            workspace = dt.new_empty((ws_bytes + 3) // 4)
            ws_p = workspace.data_ptr()
    else:
        ws_p = _check(workspace, "workspace", workspace.shape, workspace.dtype, dev)
        ws_bytes = workspace.numel() * workspace.element_size()
    st = lib.gdn_ssm_prefill(x.data_ptr(), b.data_ptr(), c.data_ptr(), dt_p, a_p, d_p, bias_p, h0_p,
                             cu_p, N, T, HK, HV, dk, dv, x_row, b_row, c_row,
                             SSM_SOFTPLUS if softplus else 0, code, y_p, hT_p, ws_p, ws_bytes,
                             _raw_stream(dev))
    if st != GDN_OK:
        raise GDNError(st, "gdn_ssm_prefill")
    return y, hT


def gdn_ssm_step_workspace_size(N, HK, HV, dk, dv) -> int:
    """Bytes of workspace ``gdn_ssm_step`` needs."""
    return int(load_library().gdn_ssm_step_workspace_size(int(N), int(HK), int(HV), int(dk), int(dv)))


def gdn_ssm_step(xbc, dt, a, state, d=None, dt_bias=None, conv_weight=None, conv_bias=None,
                 conv_state=None, silu: bool = False, softplus: bool = False, state_out=None,
                 conv_state_out=None, y=None, workspace=None, stream=None):
    """One token of the scan for N sequences through ``gdn_ssm_step``.

    xbc [N, HV*dv + 2*HK*dk] (a row x | b | c; may be a part of a wider row); dt [N,HV]
    fp32; state [N,HV,dv,dk] fp32.  With conv_weight [C,W] fp32 (conv_bias [C]) the row is
    convolved first, over the carried inputs conv_state [N,W-1,C].  The states move in
    place unless ``state_out`` / ``conv_state_out`` are given.  Returns y [N,HV,dv].
    """
    lib = load_library()
    dev = _cuda(xbc, "xbc")
    if _elsewhere(dev, stream):
        with _on(dev, stream):
            return gdn_ssm_step(xbc, dt, a, state, d, dt_bias, conv_weight, conv_bias, conv_state,
                                silu, softplus, state_out, conv_state_out, y, workspace)
    code = _code(xbc, "xbc")
    if xbc.dim() != 2 or not isinstance(state, torch.Tensor) or state.dim() != 4:
        raise ValueError("expected xbc [N, HV*dv + 2*HK*dk] and state [N,HV,dv,dk]")
    N, C = xbc.shape
    HV, dv, dk = state.shape[1:]
    HK = (C - HV * dv) // (2 * dk) if dk else 0
    if HK < 1 or HV * dv + 2 * HK * dk != C:
        raise ValueError(f"xbc rows of {C} are not HV*dv + 2*HK*dk for state {tuple(state.shape)}")
    f32 = torch.float32
    state_p = _check(state, "state", (N, HV, dv, dk), f32, dev)
    out_p = state_p if state_out is None else _check(state_out, "state_out", (N, HV, dv, dk), f32, dev)
    dt_p = _check(dt, "dt", (N, HV), f32, dev)
    a_p = _check(a, "a", (HV,), f32, dev)
    d_p = _opt(d, "d", (HV,), f32, dev)
    bias_p = _opt(dt_bias, "dt_bias", (HV,), f32, dev)
    W, w_p, cb_p, cs_p, co_p = 0, None, None, None, None
    if conv_weight is not None:
        if conv_weight.dim() != 2:
            raise ValueError("conv_weight must be [C, width]")
        W = conv_weight.shape[1]
        if conv_state is None:
            raise ValueError("a convolution needs its conv_state")
        w_p = _check(conv_weight, "conv_weight", (C, W), f32, dev)
        cb_p = _opt(conv_bias, "conv_bias", (C,), f32, dev)
        cs_p = co_p = _check(conv_state, "conv_state", (N, W - 1, C), xbc.dtype, dev)
        if conv_state_out is not None:
            co_p = _check(conv_state_out, "conv_state_out", (N, W - 1, C), xbc.dtype, dev)
    row = _rows(xbc, "xbc", 1)
    y_p = None if y is None else _check(y, "y", (N, HV, dv), xbc.dtype, dev)
    if y is None:
        y = xbc.new_empty((N, HV, dv))
        y_p = y.data_ptr()
    if workspace is None:
        ws_bytes = lib.gdn_ssm_step_workspace_size(N, HK, HV, dk, dv)
        workspace = dt.new_empty((ws_bytes + 3) // 4)
        ws_p = workspace.data_ptr()
    else:
        ws_p = _check(workspace, "workspace", workspace.shape, workspace.dtype, dev)
        ws_bytes = workspace.numel() * workspace.element_size()
    st = lib.gdn_ssm_step(xbc.data_ptr(), dt_p, a_p, d_p, bias_p, w_p, cb_p, cs_p, co_p, W, state_p,
                          out_p, N, HK, HV, dk, dv, row,
                          (SSM_SOFTPLUS if softplus else 0) | (CONV_SILU if silu else 0), code, y_p,
                          ws_p, ws_bytes, _raw_stream(dev))
    if st != GDN_OK:
        raise GDNError(st, "gdn_ssm_step")
    return y


_GATES = {"sigmoid": 0, "silu": GATE_SILU}


def _gate_flag(gate):
    if gate not in _GATES:
        raise ValueError("gate must be 'sigmoid' or 'silu'")
    return _GATES[gate]


def gdn_gated_norm(o, z=None, weight=None, eps: float = 1e-6, gate: str = "sigmoid",
                   gate_first: bool = False, unit_offset: bool = False, y=None, stream=None):
    """Norm of the read-out with its gate through ``gdn_gated_norm``.

    o, z [..., G, D] (bf16 or fp32; z may be a part of a wider row): every group of D is
    normalised on its own.  weight [D] or [G, D] fp32.  y = rms(o) w f(z), or
    rms(o f(z)) w with ``gate_first``.  Returns y like o (dense).
    """
    lib = load_library()
    dev = _cuda(o, "o")
    if _elsewhere(dev, stream):
        with _on(dev, stream):
            return gdn_gated_norm(o, z, weight, eps, gate, gate_first, unit_offset, y)
    code = _code(o, "o")
    if o.dim() < 2:
        raise ValueError("expected o [..., G, D]")
    G, D = o.shape[-2:]
    flags = _gate_flag(gate) | (NORM_GATE_FIRST if gate_first else 0) | \
        (NORM_UNIT_OFFSET if unit_offset else 0)
    z_p, z_row, w_p, wg = None, 0, None, 1
    if z is not None:
        z_p = _check(z, "z", o.shape, o.dtype, dev, True)
        z_row = _rows(z, "z", 2)
    if weight is not None:
        if weight.dim() == 2:
            wg = G
        w_p = _check(weight, "weight", (G, D) if weight.dim() == 2 else (D,), torch.float32, dev)
    o_row = _rows(o, "o", 2)
    y_p = None if y is None else _check(y, "y", o.shape, o.dtype, dev)
    if y is None:
        y = torch.empty_like(o) if o_row == 0 else o.new_empty(o.shape)
        y_p = y.data_ptr()
    n = o.numel()
    if n == 0:
        return y
    st = lib.gdn_gated_norm(o.data_ptr(), z_p, w_p, n // (G * D), G, D, o_row, z_row, wg, eps, flags,
                            code, y_p, _raw_stream(dev))
    if st != GDN_OK:
        raise GDNError(st, "gdn_gated_norm")
    return y


def gdn_residual_norm(x, residual=None, weight=None, post_weight=None, z=None, scale: float = 1.0,
                      eps: float = 1e-6, gate: str = "sigmoid", unit_offset: bool = False,
                      residual_out=None, y=None, stream=None):
    """What lies between two blocks, in one pass, through ``gdn_residual_norm``.

    x [..., C] the block's output, z like it (gate logits) or None, residual [..., C] in
    x's type or fp32 or None; weight, post_weight [C] fp32 or None.  With
    t = rms(x) post_weight f(z) (norm and gate where given): h = residual + scale t and
    y = rms(h) weight.  Returns (y, h), h in the residual's type (x's without one); pass
    ``residual_out=residual`` to add in place.
    """
    lib = load_library()
    dev = _cuda(x, "x")
    if _elsewhere(dev, stream):
        with _on(dev, stream):
            return gdn_residual_norm(x, residual, weight, post_weight, z, scale, eps, gate,
                                     unit_offset, residual_out, y)
    code = _code(x, "x")
    if x.dim() < 1:
        raise ValueError("expected x [..., C]")
    C = x.shape[-1]
    shape, f32 = x.shape, torch.float32
    flags = _gate_flag(gate) | (NORM_UNIT_OFFSET if unit_offset else 0)
    x_p = _check(x, "x", shape, x.dtype, dev)
    kept = residual if residual is not None else residual_out if residual_out is not None else x
    rdtype = kept.dtype
    if rdtype not in (x.dtype, f32):
        raise TypeError(f"residual must be {x.dtype} or float32, got {rdtype}")
    r_p = _opt(residual, "residual", shape, rdtype, dev)
    z_p = _opt(z, "z", shape, x.dtype, dev)
    w_p = _opt(weight, "weight", (C,), f32, dev)
    pw_p = _opt(post_weight, "post_weight", (C,), f32, dev)
    ro_p = _opt(residual_out, "residual_out", shape, rdtype, dev)
    if residual_out is None:
        residual_out = torch.empty_like(kept)
        ro_p = residual_out.data_ptr()
    y_p = None if y is None else _check(y, "y", shape, x.dtype, dev)
    if y is None:
        y = torch.empty_like(x)
        y_p = y.data_ptr()
    n = x.numel()
    if n == 0:
        return y, residual_out
    st = lib.gdn_residual_norm(x_p, r_p, w_p, pw_p, z_p, n // C, C, scale, eps, flags, code,
                               _CODES[rdtype], ro_p, y_p, _raw_stream(dev))
    if st != GDN_OK:
        raise GDNError(st, "gdn_residual_norm")
    return y, residual_out
