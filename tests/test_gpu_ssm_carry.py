"""States and carried inputs from the prompt form to the token form, against the exact
continuation in float64."""
import numpy as np
import pytest
import torch

import linear_attention_recurrence_rule_b200 as gdn
from oracle import ssm_oracle as S
from ssm_util import U, U32, in_norm, sequences, split_row, term_bounds, within

pytestmark = pytest.mark.gpu

BF16, F32 = torch.bfloat16, torch.float32


@pytest.mark.parametrize("dtype,dk,dv", [(F32, 32, 32), (F32, 128, 64), (BF16, 64, 64), (BF16, 128, 64), (BF16, 128, 128)])
def test_states_from_prompt_to_tokens(dtype, dk, dv):
    """The prompt's outputs and states on the row the convolution stored; then token by token
    against the exact continuation from the prompt's exact state, whose errors add up: the
    prompt's, and each token's (decays are at most 1, so none grows)."""
    HK, HV, W, steps, lengths = 1, 2, 4, 4, [37, 1, 150]
    N, C = len(lengths), HV * dv + 2 * HK * dk
    gen = torch.Generator().manual_seed(dk + dv)
    r = lambda *s: torch.randn(*s, generator=gen)   # noqa: E731
    proj, dt = r(1, sum(lengths), C).to(dtype), r(1, sum(lengths), HV)
    toks, tdt = r(steps, N, C).to(dtype), r(steps, N, HV)
    dt_bias, a, d, cw, cb = -2 + r(HV), -3 * torch.rand(HV, generator=gen), r(HV), r(C, W) / 2, 0.1 * r(C)
    w1, w2 = 1 + 0.1 * r(HV, dv), 1 + 0.1 * r(HV * dv)
    cu = torch.tensor(np.concatenate([[0], np.cumsum(lengths)]), dtype=torch.int32)
    conv = torch.zeros(N, W - 1, C, dtype=dtype, device="cuda")
    xbc = gdn.gdn_short_conv(proj.cuda(), cw.cuda(), cb.cuda(), conv, cu.cuda(), silu=True)
    p = dict(row=xbc.cpu(), dt=dt, a=a, d=d, dt_bias=dt_bias, h0=None, cu_seqlens=cu)
    y, h = gdn.gdn_ssm_prefill(*split_row(xbc, HK, HV, dk, dv), dt.cuda(), a.cuda(), d=d.cuda(), dt_bias=dt_bias.cuda(),
                               cu_seqlens=cu.cuda(), softplus=True)
    if dtype == BF16 and dk == 128:
        ref, state, allow, norm, units = term_bounds(p, HK, HV, dk, dv)
        assert in_norm(y, ref, norm, sequences(p))
    else:
        ref, state, _, y_units, units = S.scan(*split_row(p["row"], HK, HV, dk, dv), dt, a, d, dt_bias, None, cu, True)
        allow = U[dtype] * np.abs(ref) + 2 * U32 * (1 + U[dtype]) * y_units
    within(y, ref, allow + 1e-37, "prompt y")
    within(h, state, 2 * U32 * units + 1e-37, "prompt state")
    # the carried inputs are the prompt's last rows (zeros before its first)
    start = [int(v) for v in cu]
    want = torch.stack([torch.cat([torch.zeros(W - 1, C, dtype=dtype), proj[0, s:e]])[-(W - 1):]
                        for s, e in zip(start, start[1:])])
    assert torch.equal(conv.cpu(), want)
    carried = S.f64(want)
    group = np.arange(HV) // (HV // HK)
    for i in range(steps):
        yt = gdn.gdn_ssm_step(toks[i].cuda(), tdt[i].cuda(), a.cuda(), h, d=d.cuda(), dt_bias=dt_bias.cuda(),
                              conv_weight=cw.cuda(), conv_bias=cb.cuda(), conv_state=conv, silu=True, softplus=True)
        row, after = S.conv_token(toks[i], cw, cb, carried, True)
        # the convolved row in fp32: W + 1 terms and a SiLU, at most (W + 8) units of sum |terms|
        # (its slope of up to 1.1 is inside the 8, and once more for what it enters)
        size, _ = S.conv_token(toks[i].double().abs(), cw.abs(), cb.abs(), np.abs(carried), False)
        row_units = 1.1 * (W + 8) * np.maximum(size, np.abs(row))
        parts = [[np.abs(v[:, :HV * dv]).reshape(N, HV, dv), np.abs(v[:, HV * dv:HV * dv + HK * dk]).reshape(N, HK, dk)[:, group],
                  np.abs(v[:, HV * dv + HK * dk:]).reshape(N, HK, dk)[:, group]] for v in (row, row_units)]
        (x, b, c), (ex, eb, ec) = parts
        delta = S.softplus(S.f64(tdt[i]) + S.f64(dt_bias))[..., None]
        ref, state, _, y_units, step_units = S.step(row, tdt[i], a, state, d, dt_bias, True)
        before = units
        units = units + step_units + (delta * ex)[..., None] * b[:, :, None] + (delta * x)[..., None] * eb[:, :, None]
        y_units = y_units + np.einsum("nhvk,nhk->nhv", units - step_units, c) + np.einsum("nhvk,nhk->nhv", np.abs(state), ec) \
            + np.abs(S.f64(d))[:, None] * ex
        within(yt, ref, U[dtype] * np.abs(ref) + 2 * U32 * (1 + U[dtype]) * y_units + 1e-37, f"token {i} y")
        within(h, state, 2 * U32 * units + 1e-37, f"token {i} state")
        assert torch.equal(conv.cpu().double(), torch.from_numpy(after)) and (units >= before).all()
        # the norms behind it, against the oracle's on the library's own values
        z, res = r(N, HV, dv).to(dtype), r(N, HV * dv)
        n = gdn.gdn_gated_norm(yt, z.cuda(), w1.cuda(), gate="silu", gate_first=True)
        n_ref = S.gated_norm(yt, z, w1, 1e-6, "silu", True, False)
        within(n, n_ref, (U[dtype] + 128 * U32) * np.abs(n_ref) + (2e-6 if dtype == BF16 else 0) * np.abs(n_ref), "norm")
        out, kept = gdn.gdn_residual_norm(n.view(N, -1), res.cuda(), w2.cuda(), scale=0.5)
        o_ref, k_ref, t_ref = S.residual_norm(n.view(N, -1), res, w2, None, None, 0.5, 1e-6, "sigmoid", False)
        k_err = 2 * U32 * (np.abs(k_ref) + np.abs(t_ref))
        within(kept, k_ref, k_err, "residual")
        within(out, o_ref, (U[dtype] + 128 * U32) * np.abs(o_ref) + np.abs(S.f64(w2)) * k_err
               / np.sqrt(np.mean(k_ref ** 2, -1, keepdims=True)), "out")
        carried = after
