"""Inputs and tolerances shared by the tests of the state space scan and the norms."""
from __future__ import annotations

import numpy as np
import torch

from oracle import ssm_oracle as S

U = {torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}   # half a step, relative
U32 = 2.0 ** -24


def make_scan(lengths, HK, HV, dk, dv, dtype, seed, packed=True, h0=True, pad=0, row_extra=0,
              step_mean=-2.0):
    """One problem on the CPU; x, b, c are parts of one row [.., HV*dv + 2*HK*dk + row_extra]
    and `pad` rows follow the last sequence."""
    gen = torch.Generator().manual_seed(seed)
    B, T = (1, sum(lengths) + pad) if packed else (len(lengths), lengths[0])
    row = torch.randn(B, T, HV * dv + 2 * HK * dk + row_extra, generator=gen).to(dtype)
    p = dict(row=row, dt=torch.randn(B, T, HV, generator=gen),
             dt_bias=step_mean + 0.5 * torch.randn(HV, generator=gen),
             a=-(0.2 + 3 * torch.rand(HV, generator=gen)), d=torch.randn(HV, generator=gen),
             h0=torch.randn(len(lengths), HV, dv, dk, generator=gen) if h0 else None,
             cu_seqlens=None)
    if packed:
        p["cu_seqlens"] = torch.tensor(np.concatenate([[0], np.cumsum(lengths)]), dtype=torch.int32)
    return p


def split_row(row, HK, HV, dk, dv):
    x = row[..., :HV * dv].unflatten(-1, (HV, dv))
    b = row[..., HV * dv:HV * dv + HK * dk].unflatten(-1, (HK, dk))
    c = row[..., HV * dv + HK * dk:HV * dv + 2 * HK * dk].unflatten(-1, (HK, dk))
    return x, b, c


def to_cuda(p):
    return {k: v.cuda() if isinstance(v, torch.Tensor) else v for k, v in p.items()}


def within(out, ref, allow, what):
    out = S.f64(out)
    assert out.shape == ref.shape, (what, out.shape, ref.shape)
    assert np.all(np.isfinite(out)), f"{what}: non-finite values"
    over = np.abs(out - ref) - allow
    assert not out.size or over.max() <= 0, \
        f"{what}: {np.abs(out - ref).flat[over.argmax()]:.3e} off where {np.broadcast_to(allow, ref.shape).flat[over.argmax()]:.3e} is allowed"


def check_scan(y, hT, ref, dtype, tensor_cores, what=""):
    """Bounds: the result's own rounding, the fp32 roundings on the way (doubled, for sums
    in another order and the hardware exponential), and on the tensor-core path three bf16
    roundings of each term of y, more than any has (term_bounds counts them term by term):
    with u = 2^-8, (1 + u)^3 - 1 = 3 u (1 + u + u^2 / 3) <= 3 u (1 + 2^-6)."""
    r_y, r_h, y_abs, y_units, h_units = ref
    u = U[dtype]
    allow = u * np.abs(r_y) + 2 * U32 * (1 + u) * y_units
    if tensor_cores:
        allow = allow + 3 * U[torch.bfloat16] * (1 + 2.0 ** -6) * y_abs
    within(y, r_y, allow + 1e-37, what + "y")
    if hT is not None:
        within(hT, r_h, 2 * U32 * h_units + 1e-37, what + "hT")


def term_bounds(p, HK, HV, dk, dv, rate=1.0):
    """Exact y and hT, the bound of each y and of each norm of y over a sequence and head.

    A term of y inside its chunk of 128 tokens is rounded to bf16 once, one from before it twice
    (its weighted value, the state), d x not at all; fp32 roundings as the oracle counts them,
    doubled.  In norm a rounding of a value m 2^e, 1 <= m < 2, is uniform within 2^(e-8): its mean
    square is at most (2^-8)^2 / 3 of the value's square, and the roundings are independent."""
    x, b, c = split_row(p["row"], HK, HV, dk, dv)
    y, h, _, y_units, h_units = S.scan(x, b, c, p["dt"], rate * S.f64(p["a"]), p["d"], p["dt_bias"], p["h0"],
                                       p["cu_seqlens"], True)
    near, far, squares = S.chunk_terms(x, b, c, p["dt"], rate * S.f64(p["a"]), p["dt_bias"], p["h0"], p["cu_seqlens"], True)
    u = U[torch.bfloat16]
    allow = u * np.abs(y) + 2 * U32 * (1 + u) * y_units + u * near + 2 * u * (1 + u) * far
    norm = u / np.sqrt(3) * np.sqrt(y * y + squares) + 2 * U32 * y_units
    return y, h, allow, norm, h_units


def sequences(p):
    if p["cu_seqlens"] is None:
        B, T = p["dt"].shape[:2]
        return [(n, slice(0, T)) for n in range(B)]
    cu = [int(v) for v in p["cu_seqlens"]]
    return [(0, slice(s, e)) for s, e in zip(cu, cu[1:]) if e > s]


def in_norm(out, y, norm, where, least=2000):
    """Whether every (sequence, head) of at least `least` outputs is within its norm's bound."""
    err = S.f64(out) - y
    ok = True
    for n, t in where:
        for h in range(y.shape[2]):
            e, lim = err[n, t, h], norm[n, t, h]
            if e.size >= least:
                ok = ok and np.linalg.norm(e) <= np.linalg.norm(lim)
    return ok
