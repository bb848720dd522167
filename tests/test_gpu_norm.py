"""The norms around a block through the C ABI against the float64 oracle."""
import numpy as np
import pytest
import torch

import linear_attention_recurrence_rule_b200 as gdn
from oracle import ssm_oracle as S
from ssm_util import U, U32, within

pytestmark = pytest.mark.gpu

BF16, F32 = torch.bfloat16, torch.float32


def units(D):
    # a thread sums at most 32 squares (or D / 256 in the element-wise kernel), then a tree
    # of at most 5 + 32 sums; products, square root and exponential: 16 more; twice for
    # sums in another order
    return 2 * (max(32, D / 256) + 37 + 16)


def gate_rel(dtype):
    return 4e-6 if dtype == BF16 else 8 * U32   # the bf16 path's fast sigmoid


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("G,D", [(1, 1), (3, 8), (32, 128), (5, 100), (2, 333), (1, 1536), (4, 512), (1, 4096), (1, 5000),
                                 (1, 16384), (1, 65536)])
@pytest.mark.parametrize("gate_first", [False, True])
def test_gated_norm(dtype, G, D, gate_first):
    gen = torch.Generator().manual_seed(G + D)
    rows = 1 if D > 10000 else 7
    o = torch.randn(rows, G, D, generator=gen).to(dtype)
    wide = 3 * torch.randn(rows, G * D + 24, generator=gen).to(dtype)
    z = wide[:, 8:8 + G * D].unflatten(-1, (G, D))
    per_group = G > 1 and D % 2 == 0
    w = torch.randn(*((G, D) if per_group else (D,)), generator=gen)
    for act in ("silu", "sigmoid"):
        y = gdn.gdn_gated_norm(o.cuda(), wide.cuda()[:, 8:8 + G * D].unflatten(-1, (G, D)), w.cuda(), gate=act,
                               gate_first=gate_first, unit_offset=act == "silu")
        ref = S.gated_norm(o, z, w, 1e-6, act, gate_first, act == "silu")
        within(y, ref, np.abs(ref) * (U[dtype] + 2 * units(D) * U32 + 2 * gate_rel(dtype)) + 1e-37, f"y {act}")


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_gated_norm_without_gate_weight_and_in_place(dtype):
    gen = torch.Generator().manual_seed(0)
    o = torch.randn(2, 9, 4, 64, generator=gen).to(dtype)
    g = o.cuda()
    y = gdn.gdn_gated_norm(g, eps=1e-3, y=g)
    assert y.data_ptr() == g.data_ptr()
    ref = S.gated_norm(o, None, None, 1e-3, "silu", False, False)
    within(y, ref, np.abs(ref) * (U[dtype] + units(64) * U32), "y")
    # a misaligned view takes the element-wise kernel
    base = torch.randn(9 * 128 + 1, generator=gen).to(dtype)
    m = base[1:].view(9, 1, 128)
    y = gdn.gdn_gated_norm(base.cuda()[1:].view(9, 1, 128))
    ref = S.gated_norm(m, None, None, 1e-6, "silu", False, False)
    within(y, ref, np.abs(ref) * (U[dtype] + units(128) * U32), "misaligned")
    # zero rows normalise to zero
    y = gdn.gdn_gated_norm(torch.zeros(3, 2, 96, dtype=dtype, device="cuda"))
    assert not y.any()
    assert gdn.gdn_gated_norm(torch.empty(0, 2, 96, dtype=dtype, device="cuda")).shape == (0, 2, 96)


@pytest.mark.parametrize("dtype,rdtype", [(F32, F32), (BF16, BF16), (BF16, F32)])
@pytest.mark.parametrize("rows,C", [(1, 1), (5, 64), (3, 777), (130, 256), (33, 512), (2, 2048), (3, 4096), (2, 8192), (1, 20000),
                                    (1, 65536)])
@pytest.mark.parametrize("post,gated", [(False, False), (True, False), (True, True), (False, True)])
def test_residual_norm(dtype, rdtype, rows, C, post, gated):
    gen = torch.Generator().manual_seed(rows + C)
    x = torch.randn(rows, C, generator=gen).to(dtype)
    res = (2 * torch.randn(rows, C, generator=gen)).to(rdtype)
    z = torch.randn(rows, C, generator=gen).to(dtype) if gated else None
    w = torch.randn(C, generator=gen)
    pw = torch.randn(C, generator=gen) if post else None
    cu = lambda t: None if t is None else t.cuda()   # noqa: E731
    for offset, act in ((False, "sigmoid"), (True, "silu")):
        g = res.cuda()
        y, h = gdn.gdn_residual_norm(x.cuda(), g, w.cuda(), post_weight=cu(pw), z=cu(z), scale=0.7, gate=act,
                                     unit_offset=offset, residual_out=g if offset else None)
        ry, rh, rt = S.residual_norm(x, res, w, pw, z, 0.7, 1e-6, act, offset)
        k = units(C) * U32 + (2 * gate_rel(dtype) if gated else 0)
        h_err = k * np.abs(rt) + 4 * U32 * (np.abs(rh) + np.abs(rt))
        within(h, rh, U[rdtype] * np.abs(rh) + h_err * (1 + U[rdtype]) + 1e-37, "h")
        if offset:
            assert h.data_ptr() == g.data_ptr()
        # y = h w / rms(h): h's own error and that of the sum of squares (relative to the
        # row's rms, at most the largest relative error in the row's norm)
        inv = 1 / np.sqrt(np.mean(rh * rh, -1, keepdims=True) + 1e-6)
        norm_rel = np.linalg.norm(h_err, axis=-1, keepdims=True) / np.maximum(np.linalg.norm(rh, axis=-1, keepdims=True), 1e-30)
        wv = np.abs(S.f64(w) + (1 if offset else 0))
        allow = U[dtype] * np.abs(ry) + (h_err * inv * wv + np.abs(ry) * (norm_rel + units(C) * U32)) * (1 + U[dtype])
        within(y, ry, allow + 1e-37, "y")


def test_residual_norm_optional_parts_streams_and_graph():
    gen = torch.Generator().manual_seed(3)
    x = torch.randn(4, 9, 256, generator=gen).to(BF16).cuda()
    y, h = gdn.gdn_residual_norm(x)
    ref = S.rms(S.f64(x), 1e-6)
    within(y, ref, np.abs(ref) * (U[BF16] + units(256) * U32), "y")
    assert torch.equal(h, x)
    # y may be x, on another stream, and the same when captured
    want, wh = gdn.gdn_residual_norm(x, x, scale=0.25)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    again = x.clone()
    torch.cuda.synchronize()
    gdn.gdn_residual_norm(again, x, scale=0.25, y=again, stream=side)
    side.synchronize()
    assert torch.equal(again, want)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y, h = gdn.gdn_residual_norm(x, x, scale=0.25)
        n = gdn.gdn_gated_norm(y, x)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(y, want) and torch.equal(h, wh) and torch.equal(n, gdn.gdn_gated_norm(want, x))
    assert gdn.gdn_residual_norm(x[:0])[0].shape == (0, 9, 256)


def test_offsets_past_32_bits():
    rows, C = 530_000, 4096                                   # 2.2e9 elements
    gen = torch.Generator(device="cuda").manual_seed(2)
    x = torch.empty(rows, C, dtype=BF16, device="cuda").normal_(generator=gen)
    w = torch.empty(128, device="cuda").normal_(generator=gen)
    assert x.numel() > 2 ** 31
    y = gdn.gdn_gated_norm(x.view(rows, 32, 128), x.view(rows, 32, 128), w)
    assert torch.equal(y[-5:], gdn.gdn_gated_norm(x[-5:].view(5, 32, 128), x[-5:].view(5, 32, 128), w))
    del y
    y, h = gdn.gdn_residual_norm(x, x, scale=0.5)
    y2, h2 = gdn.gdn_residual_norm(x[-5:], x[-5:], scale=0.5)
    assert torch.equal(y[-5:], y2) and torch.equal(h[-5:], h2)
