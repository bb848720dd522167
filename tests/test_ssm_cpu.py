"""Host-side checks of the state space scan, its step and the norms (no call here
reaches a GPU), and the oracle's own pins."""
import ctypes

import numpy as np
import pytest
import torch

from linear_attention_recurrence_rule_b200 import _build, gdn, ssm
from oracle import ssm_oracle as S
from ssm_util import in_norm, make_scan, sequences, split_row, term_bounds

OK, INVALID, UNSUPPORTED, ALIGNMENT, WORKSPACE = (gdn.GDN_OK, gdn.GDN_ERR_INVALID_ARG, gdn.GDN_ERR_UNSUPPORTED,
                                                  gdn.GDN_ERR_ALIGNMENT, gdn.GDN_ERR_WORKSPACE)
P = ctypes.c_void_p


@pytest.fixture(scope="module")
def lib():
    _build.build()
    return gdn.load_library()


def prefill(lib, **kw):
    a = dict(x=P(0x1000), b=P(0x2000), c=P(0x3000), dt=P(0x4000), a=P(0x5000), d=None, bias=None, h0=None, cu=None,
             N=1, T=64, HK=1, HV=2, dk=128, dv=64, xr=0, br=0, cr=0, flags=0, dtype=gdn.GDN_BF16, y=P(0x6000),
             hT=None, ws=None, wsb=0)
    assert not set(kw) - set(a)
    a.update(kw)
    return lib.gdn_ssm_prefill(*a.values(), None)


def test_prefill_refusals(lib):
    for name in ("x", "b", "c", "dt", "a", "y"):
        assert prefill(lib, **{name: None}) == INVALID
    assert prefill(lib, HV=3, HK=2) == INVALID
    assert prefill(lib, N=-1) == INVALID
    assert prefill(lib, T=-1) == INVALID
    assert prefill(lib, dtype=9) == INVALID
    assert prefill(lib, flags=16) == INVALID
    assert prefill(lib, dk=48) == UNSUPPORTED
    assert prefill(lib, dv=256) == UNSUPPORTED
    assert prefill(lib, N=1 << 20, T=1 << 20) == UNSUPPORTED
    assert prefill(lib, N=2, T=(1 << 62) + 1) == UNSUPPORTED
    assert prefill(lib, N=1 << 27, T=1, HV=2) == UNSUPPORTED    # 2^28 states
    assert prefill(lib, N=1 << 27, T=1, HV=2, dtype=gdn.GDN_F32, dk=32, dv=32) == UNSUPPORTED
    assert prefill(lib, xr=120) == INVALID          # rows would overlap
    assert prefill(lib, br=64) == INVALID
    for name in ("x", "b", "c", "y", "h0", "hT"):
        assert prefill(lib, **{name: P(0x7008)}) == ALIGNMENT
    assert prefill(lib, xr=132) == ALIGNMENT        # not a multiple of 16 bytes
    assert prefill(lib, dt=P(0x4002)) == ALIGNMENT
    assert prefill(lib, cu=P(0x4002)) == ALIGNMENT
    assert prefill(lib, N=0, x=None, y=None, a=None) == OK
    need = lib.gdn_ssm_prefill_workspace_size(3, 5000, 1, 2, 128, 64, gdn.GDN_BF16, 1)
    assert need > 0
    cu = dict(cu=P(0x8000), N=3, T=5000)
    assert prefill(lib, **cu) == WORKSPACE
    assert prefill(lib, ws=P(0x9000), wsb=need - 1, **cu) == WORKSPACE
    assert prefill(lib, ws=P(0x9008), wsb=need, **cu) == ALIGNMENT


def test_workspace_size_of_rejected_sizes(lib):
    f = lib.gdn_ssm_prefill_workspace_size
    assert f(1, 64, 2, 3, 128, 128, gdn.GDN_BF16, 0) == 0
    assert f(1, 64, 1, 2, 100, 128, gdn.GDN_BF16, 0) == 0
    assert f(-1, 64, 1, 2, 128, 128, gdn.GDN_BF16, 0) == 0
    assert f(0, 64, 1, 2, 128, 128, gdn.GDN_BF16, 1) == 0


@pytest.mark.parametrize("dtype,dk,dv", [(gdn.GDN_BF16, 128, 128), (gdn.GDN_BF16, 128, 64), (gdn.GDN_BF16, 64, 64),
                                         (gdn.GDN_F32, 32, 32), (gdn.GDN_F32, 128, 128)])
@pytest.mark.parametrize("varlen", [0, 1])
def test_workspace_of_a_larger_call_serves_smaller_ones(lib, dtype, dk, dv, varlen):
    # the number of segments goes up and down with the sizes; the workspace must not
    size = lib.gdn_ssm_prefill_workspace_size
    for HK, HV in ((1, 1), (1, 3), (8, 32), (16, 32), (1, 24), (4, 128), (1, 300)):
        for N in (1, 2, 7, 8, 64):
            sizes = [size(N, T, HK, HV, dk, dv, dtype, varlen)
                     for T in [*range(1, 3000, 31), *range(3000, 70000, 997), 1 << 20, 1 << 24]]
            assert sizes == sorted(sizes), (HK, HV, N)
        for T in (1, 129, 1152, 4096, 10368, 16384, 65536):
            sizes = [size(N, T, HK, HV, dk, dv, dtype, varlen) for N in [*range(1, 130), 1000, 1023, 1024, 1025, 1100, 5000]]
            assert sizes == sorted(sizes), (HK, HV, T)
    # and no call is given less than its own segments need: a state each, one a sequence at least
    assert size(7, 100, 1, 3, dk, dv, dtype, 1) >= 7 * 3 * dk * dv * 4


def step(lib, **kw):
    a = dict(xbc=P(0x1000), dt=P(0x2000), a=P(0x3000), d=None, bias=None, w=P(0x4000), cb=None, cs=P(0x5000),
             co=P(0x5000), W=4, state=P(0x6000), out=P(0x6000), N=2, HK=1, HV=2, dk=128, dv=64, row=0, flags=0,
             dtype=gdn.GDN_BF16, y=P(0x7000), ws=P(0x8000), wsb=1 << 30)
    assert not set(kw) - set(a)
    a.update(kw)
    return lib.gdn_ssm_step(*a.values(), None)


def test_step_refusals(lib):
    for name in ("xbc", "dt", "a", "state", "out", "y", "cs", "co"):
        assert step(lib, **{name: None}) == INVALID
    assert step(lib, HK=3) == INVALID
    assert step(lib, flags=1) == INVALID
    assert step(lib, dtype=5) == INVALID
    assert step(lib, row=100) == INVALID
    assert step(lib, W=1) == UNSUPPORTED
    assert step(lib, W=9) == UNSUPPORTED
    assert step(lib, dk=96) == UNSUPPORTED
    assert step(lib, dv=257) == UNSUPPORTED
    assert step(lib, N=1 << 30, HV=4) == UNSUPPORTED
    assert step(lib, state=P(0x6008)) == ALIGNMENT
    assert step(lib, out=P(0x6008)) == ALIGNMENT
    assert step(lib, xbc=P(0x1001)) == ALIGNMENT
    assert step(lib, w=P(0x4002)) == ALIGNMENT
    assert step(lib, N=0, xbc=None) == OK
    assert step(lib, N=262141) == UNSUPPORTED
    need = lib.gdn_ssm_step_workspace_size(2, 1, 2, 128, 64)
    assert need == 2 * (2 * 8 + (2 * 64 + 2 * 128) * 4)
    assert step(lib, ws=None) == WORKSPACE and step(lib, wsb=need - 1) == WORKSPACE
    assert step(lib, ws=P(0x8008)) == ALIGNMENT
    assert lib.gdn_ssm_step_workspace_size(2, 3, 2, 128, 64) == 0


def test_step_refuses_rows_past_32_bits(lib):
    # a row is rounded up to blocks of 256 channels in 32 bits
    rows = dict(N=1, HK=1, dk=32, dv=1)
    assert step(lib, HV=(1 << 31) - 256 - 64, ws=None, **rows) == WORKSPACE
    assert step(lib, HV=(1 << 31) - 255 - 64, **rows) == UNSUPPORTED
    assert step(lib, HV=(1 << 31) - 1 - 64, **rows) == UNSUPPORTED
    assert lib.gdn_ssm_step_workspace_size(1, 1, (1 << 31) - 1 - 64, 32, 1) == 0


def gated(lib, **kw):
    a = dict(o=P(0x1000), z=P(0x2000), w=P(0x3000), rows=4, G=2, D=64, o_row=0, z_row=0, wg=1, eps=1e-6, flags=0,
             dtype=gdn.GDN_BF16, y=P(0x4000))
    assert not set(kw) - set(a)
    a.update(kw)
    return lib.gdn_gated_norm(*a.values(), None)


def residual(lib, **kw):
    a = dict(x=P(0x1000), r=P(0x2000), w=P(0x3000), pw=None, z=None, rows=4, C=64, scale=1.0, eps=1e-6, flags=0,
             dtype=gdn.GDN_BF16, rd=gdn.GDN_F32, ro=P(0x4000), y=P(0x5000))
    assert not set(kw) - set(a)
    a.update(kw)
    return lib.gdn_residual_norm(*a.values(), None)


def test_norm_refusals(lib):
    assert gated(lib, o=None) == INVALID and gated(lib, y=None) == INVALID
    assert gated(lib, rows=-1) == INVALID and gated(lib, D=0) == INVALID and gated(lib, G=0) == INVALID
    assert gated(lib, wg=3) == INVALID and gated(lib, flags=1) == INVALID and gated(lib, dtype=3) == INVALID
    assert gated(lib, eps=-1.0) == INVALID and gated(lib, eps=float("nan")) == INVALID
    assert gated(lib, o_row=127) == INVALID and gated(lib, z_row=127) == INVALID
    assert gated(lib, D=65537) == UNSUPPORTED and gated(lib, rows=1 << 31) == UNSUPPORTED
    assert gated(lib, o=P(0x1001)) == ALIGNMENT and gated(lib, w=P(0x3002)) == ALIGNMENT
    assert gated(lib, rows=0, o=None) == OK
    assert residual(lib, x=None) == INVALID and residual(lib, y=None, ro=None) == INVALID
    assert residual(lib, C=0) == INVALID and residual(lib, flags=128) == INVALID
    assert residual(lib, eps=float("inf")) == INVALID
    assert residual(lib, dtype=gdn.GDN_F32, rd=gdn.GDN_BF16) == UNSUPPORTED
    assert residual(lib, C=65537) == UNSUPPORTED and residual(lib, rows=1 << 31) == UNSUPPORTED
    assert residual(lib, ro=P(0x4002)) == ALIGNMENT and residual(lib, x=P(0x1001)) == ALIGNMENT
    assert residual(lib, rows=0, x=None) == OK


def test_binding_refuses_host_tensors_and_bad_layouts(lib):
    x = torch.zeros(1, 4, 2, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="CUDA tensor"):
        ssm.gdn_ssm_prefill(x, x, x, x, x)
    with pytest.raises(ValueError, match="CUDA tensor"):
        ssm.gdn_ssm_step(x, x, x, x)
    with pytest.raises(ValueError, match="CUDA tensor"):
        ssm.gdn_gated_norm(x)
    with pytest.raises(ValueError, match="CUDA tensor"):
        ssm.gdn_residual_norm(x)
    with pytest.raises(TypeError):
        ssm.gdn_gated_norm([1.0])
    with pytest.raises(ValueError, match="gate must be"):
        ssm._gate_flag("tanh")
    # row distances
    row = torch.zeros(2, 5, 300)
    part = row[..., 10:10 + 128].unflatten(-1, (2, 64))
    assert ssm._rows(part, "x", 2) == 300
    assert ssm._rows(torch.zeros(2, 5, 2, 64), "x", 2) == 0
    assert ssm._rows(row[:, :1, :128].unflatten(-1, (2, 64)), "x", 2) == 1500   # one token each
    assert ssm._rows(row[:1, :1, :128].unflatten(-1, (2, 64)), "x", 2) == 0
    with pytest.raises(ValueError, match="evenly spaced"):
        ssm._rows(row[:, :4, :128].unflatten(-1, (2, 64)), "x", 2)
    with pytest.raises(ValueError, match="contiguous"):
        ssm._rows(torch.zeros(2, 5, 64, 2).transpose(2, 3), "x", 2)
    with pytest.raises(ValueError, match="overlap"):
        ssm._rows(torch.zeros(1, 1, 2, 64).expand(1, 5, 2, 64), "x", 2)


# ---------------------------------------------------------------- the oracle's pins
def rand(*s, seed=0):
    return np.random.RandomState(seed).randn(*s)


def test_oracle_closed_forms():
    # no decay and unit steps: the state is the running sum of x b^T
    x, b, c = rand(1, 6, 2, 3), rand(1, 6, 1, 4, seed=1), rand(1, 6, 1, 4, seed=2)
    y, h, *_ = S.scan(x, b, c, np.ones((1, 6, 2)), np.zeros(2))
    want = np.einsum("thv,tk->hvk", x[0], b[0, :, 0])
    assert np.allclose(h[0], want)
    assert np.allclose(y[0, -1], np.einsum("hvk,k->hv", want, c[0, -1, 0]))
    # halving: 8 -> 4 + 1 -> 2.5 + 1 with x = b = c = 1
    one = np.ones((1, 2, 1, 1))
    y, h, *_ = S.scan(one, one, one, np.ones((1, 2, 1)), np.array([-np.log(2)]), None, None, np.full((1, 1, 1, 1), 8.0))
    assert np.allclose(y.ravel(), [5.0, 3.5]) and np.allclose(h, 3.5)
    # d adds the value itself; a step of zero leaves the state
    y2, h2, *_ = S.scan(one, one, one, np.zeros((1, 2, 1)), np.array([-1.0]), np.array([3.0]), None,
                        np.full((1, 1, 1, 1), 8.0))
    assert np.allclose(y2.ravel(), 11.0) and np.allclose(h2, 8.0)


def test_oracle_packing_groups_and_split():
    lengths = [3, 0, 5]
    cu = np.concatenate([[0], np.cumsum(lengths)])
    x, b, c = rand(1, 8, 4, 3), rand(1, 8, 2, 5, seed=1), rand(1, 8, 2, 5, seed=2)
    dt, a, h0 = rand(1, 8, 4, seed=3), -np.abs(rand(4, seed=4)), rand(3, 4, 3, 5, seed=5)
    y, h, *_ = S.scan(x, b, c, dt, a, None, None, h0, cu, True)
    for n in range(3):
        s = slice(cu[n], cu[n + 1])
        yn, hn, *_ = S.scan(x[:, s], b[:, s], c[:, s], dt[:, s], a, None, None, h0[n:n + 1], None, True)
        assert np.allclose(y[:, s], yn) and np.allclose(h[n], hn[0])
    # head 3 reads group 1
    yh, _, *_ = S.scan(x[:, :, 3:], b[:, :, 1:], c[:, :, 1:], dt[:, :, 3:], a[3:], None, None, h0[:, 3:], cu, True)
    assert np.allclose(y[:, :, 3:], yh)
    # one token at a time
    state = h0[2:3]
    for t in range(3, 8):
        row = np.concatenate([x[0, t].ravel(), b[0, t].ravel(), c[0, t].ravel()])[None]
        yt, state, *_ = S.step(row, dt[:, t], a, state, None, None, True)
        assert np.allclose(yt[0], y[0, t])
    assert np.allclose(state[0], h[2])


def test_oracle_error_units_cover_fp32():
    # the bounds hold for a plain fp32 evaluation, and are not idle
    rs = np.random.RandomState(0)
    T, HV, dv, dk = 60, 2, 4, 8
    x, b, c = (rs.randn(1, T, 2, n).astype(np.float32) for n in (dv, dk, dk))
    dt, a = rs.rand(1, T, HV).astype(np.float32), -np.array([0.1, 2.0], np.float32)
    y, h, ya, yu, hu = S.scan(x, b, c, dt, a)
    s = np.zeros((HV, dv, dk), np.float32)
    worst = 0
    for t in range(T):
        al = np.exp(dt[0, t] * a)[:, None, None]
        s = al * s + (dt[0, t][:, None] * x[0, t])[:, :, None] * b[0, t][:, None]
        out = (s * c[0, t][:, None]).sum(-1)
        err = np.abs(out - y[0, t]) / (yu[0, t] * 2.0 ** -24)
        worst = max(worst, err.max())
    assert worst <= 1 and worst > 1e-3
    assert (np.abs(s - h[0]) <= hu[0] * 2.0 ** -24).all()


def test_oracle_chunk_terms():
    # the two sums are the scan's sum of |terms| (without d x), whatever the chunk
    p = make_scan([1, 70, 0, 45], 2, 4, 8, 6, torch.float32, seed=3)
    parts = split_row(p["row"], 2, 4, 8, 6)
    y, _, total, _, _ = S.scan(*parts, p["dt"], p["a"], None, p["dt_bias"], p["h0"], p["cu_seqlens"], True)
    for chunk in (1, 32, 128):
        near, far, squares = S.chunk_terms(*parts, p["dt"], p["a"], p["dt_bias"], p["h0"], p["cu_seqlens"], True, chunk)
        assert np.allclose(near + far, total)
        assert (squares <= 2 * (near ** 2 + far ** 2) * (1 + 1e-9)).all()
    # roundings drawn at random leave errors of that mean square
    rs, T, dv, dk = np.random.RandomState(0), 8, 4, 3
    x, b, c, dt = rs.randn(1, T, 1, dv), rs.randn(1, T, 1, dk), rs.randn(1, T, 1, dk), rs.rand(1, T, 1)
    a, h0 = np.array([-0.3]), rs.randn(1, 1, dv, dk)
    exact = S.scan(x, b, c, dt, a, None, None, h0)[0][0, :, 0]
    *_, squares = S.chunk_terms(x, b, c, dt, a, None, h0, chunk=4)
    total, draws = np.zeros((T, dv)), 4000
    eps = lambda *s: 1 + 1e-6 * rs.randn(draws, *s)   # noqa: E731
    St, out = np.broadcast_to(h0[0, 0], (draws, dv, dk)), []
    for s in (0, 4):
        X, Bm, Cm, dl = x[0, s:s + 4, 0], b[0, s:s + 4, 0], c[0, s:s + 4, 0], dt[0, s:s + 4, 0]
        g = np.cumsum(dl) * a[0]
        P = np.tril(np.exp(g[:, None] - g[None]) * dl * (Cm @ Bm.T)) * eps(4, 4)
        out.append(P @ X + np.exp(g)[:, None] * np.einsum("tk,nvk->ntv", Cm, St * eps(dv, dk)))
        wx = (dl * np.exp(g[-1] - g))[:, None] * X * eps(4, dv)
        St = np.exp(g[-1]) * St + np.einsum("ntv,tk->nvk", wx, Bm)
    seen = ((np.concatenate(out, 1) - exact) ** 2).mean(0) / 1e-12
    assert np.allclose(seen, squares[0, :, 0], rtol=0.15)     # 4000 draws: 2.2% standard error


def test_bound_in_norm_is_not_idle():
    # an exact result, rounded, is inside it; one with decay rates off by 2% is not
    p = make_scan([1411], 1, 2, 128, 64, torch.bfloat16, seed=1, packed=False, step_mean=-4.0)
    ref, _, _, norm, _ = term_bounds(p, 1, 2, 128, 64)
    off, *_ = term_bounds(p, 1, 2, 128, 64, rate=1.02)
    assert in_norm(torch.from_numpy(ref).to(torch.bfloat16), ref, norm, sequences(p))
    assert not in_norm(torch.from_numpy(off).to(torch.bfloat16), ref, norm, sequences(p))


def test_oracle_norms():
    o, z, w = rand(3, 2, 8), rand(3, 2, 8, seed=1), rand(8, seed=2)
    y = S.gated_norm(o, z, w, 0.0, "sigmoid", False, False)
    assert np.allclose(y / w / (1 / (1 + np.exp(-z))), o / np.sqrt((o ** 2).mean(-1, keepdims=True)))
    # gate first: a gate that is the same everywhere cancels
    assert np.allclose(S.gated_norm(o, np.full_like(z, 0.7), None, 0.0, "silu", True, False), S.rms(o, 0.0))
    y, h, t = S.residual_norm(o, z, w, None, None, 0.5, 0.0, "sigmoid", True)
    assert np.allclose(h, z + 0.5 * o) and np.allclose(y, S.rms(h, 0.0) * (1 + w)) and np.allclose(t, 0.5 * o)
    y, h, t = S.residual_norm(7 * o, None, None, np.ones(8), None, 1.0, 0.0, "sigmoid", False)
    assert np.allclose(h, S.rms(o, 0.0)) and np.allclose(y, S.rms(o, 0.0))
