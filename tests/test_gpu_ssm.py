"""The selective state space scan over prompts and for single tokens, through the C
ABI, against the float64 oracle."""
import numpy as np
import pytest
import torch

import linear_attention_recurrence_rule_b200 as gdn
from oracle import ssm_oracle as S
from ssm_util import U, U32, check_scan, make_scan, split_row, to_cuda, within

pytestmark = pytest.mark.gpu

BF16, F32 = torch.bfloat16, torch.float32


def on_tensor_cores(dk, dv, dtype):
    return dtype == BF16 and dk == 128 and dv in (64, 128)


def run(p, HK, HV, dk, dv, **kw):
    g = to_cuda(p)
    x, b, c = split_row(g["row"], HK, HV, dk, dv)
    return gdn.gdn_ssm_prefill(x, b, c, g["dt"], g["a"], d=g["d"], dt_bias=g["dt_bias"], h0=g["h0"],
                               cu_seqlens=g["cu_seqlens"], **kw)


def oracle(p, HK, HV, dk, dv, soft):
    x, b, c = split_row(p["row"], HK, HV, dk, dv)
    return S.scan(x, b, c, p["dt"], p["a"], p["d"], p["dt_bias"], p["h0"], p["cu_seqlens"], soft)


DIMS = [(32, 32), (64, 64), (128, 64), (128, 128), (64, 128), (128, 32), (32, 128)]


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("dk,dv", DIMS)
@pytest.mark.parametrize("HK,HV", [(1, 2), (2, 2), (1, 3)])
def test_packed_ragged(dtype, dk, dv, HK, HV):
    # an empty sequence, one token, lengths around the tiles of 32 and 128 tokens
    lengths = [1, 0, 127, 128, 129, 33, 2, 260]
    p = make_scan(lengths, HK, HV, dk, dv, dtype, seed=dk + dv + HV, row_extra=8)
    y, hT = run(p, HK, HV, dk, dv, softplus=True)
    check_scan(y, hT, oracle(p, HK, HV, dk, dv, True), dtype, on_tensor_cores(dk, dv, dtype))


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("T", [1, 2, 31, 128, 300])
@pytest.mark.parametrize("h0", [False, True])
def test_batched(dtype, T, h0):
    HK, HV, dk, dv = 1, 2, 128, 64
    p = make_scan([T] * 3, HK, HV, dk, dv, dtype, seed=T, packed=False, h0=h0)
    y, hT = run(p, HK, HV, dk, dv, softplus=True)
    check_scan(y, hT, oracle(p, HK, HV, dk, dv, True), dtype, on_tensor_cores(dk, dv, dtype))


@pytest.mark.parametrize("dtype,dk,dv", [(F32, 32, 32), (F32, 128, 128), (BF16, 128, 128), (BF16, 128, 64),
                                         (BF16, 64, 64)])
@pytest.mark.parametrize("packed", [False, True])
def test_long_sequences_are_cut(dtype, dk, dv, packed):
    # long enough that a sequence is cut into several segments; mild decays carry the
    # state across them
    HK, HV = 1, 2
    lengths = [1500, 1, 1301] if packed else [1411] * 2
    p = make_scan(lengths, HK, HV, dk, dv, dtype, seed=5 + dk, packed=packed, step_mean=-6.0)
    y, hT = run(p, HK, HV, dk, dv, softplus=True)
    check_scan(y, hT, oracle(p, HK, HV, dk, dv, True), dtype, on_tensor_cores(dk, dv, dtype))


@pytest.mark.parametrize("dtype,dk,dv", [(F32, 64, 64), (BF16, 128, 128), (BF16, 128, 64)])
def test_state_in_place_and_split_prompt(dtype, dk, dv):
    # hT may be h0, and a prompt in two calls equals one call
    HK, HV, T, cut = 2, 4, 900, 389
    p = make_scan([T] * 2, HK, HV, dk, dv, dtype, seed=11, packed=False, step_mean=-4.0)
    ref = oracle(p, HK, HV, dk, dv, True)
    g = to_cuda(p)
    state = g["h0"].clone()
    ys = []
    for t0, t1 in ((0, cut), (cut, T)):
        x, b, c = split_row(g["row"][:, t0:t1].contiguous(), HK, HV, dk, dv)
        y, h = gdn.gdn_ssm_prefill(x, b, c, g["dt"][:, t0:t1].contiguous(), g["a"], d=g["d"],
                                   dt_bias=g["dt_bias"], h0=state, hT=state, softplus=True)
        assert h.data_ptr() == state.data_ptr()
        ys.append(y)
    check_scan(torch.cat(ys, 1), state, ref, dtype, on_tensor_cores(dk, dv, dtype))


@pytest.mark.parametrize("dtype,dk,dv", [(F32, 32, 64), (BF16, 128, 128), (BF16, 128, 64)])
def test_rows_behind_the_last_sequence(dtype, dk, dv):
    # NaN inputs there reach nothing, and y is left as it was
    HK, HV, lengths, pad = 1, 2, [70, 200, 3], 150
    p = make_scan(lengths, HK, HV, dk, dv, dtype, seed=3, pad=pad)
    p["row"][:, sum(lengths):] = float("nan")
    p["dt"][:, sum(lengths):] = float("nan")
    y0 = torch.full((1, sum(lengths) + pad, HV, dv), 7.0, dtype=dtype, device="cuda")
    y, hT = run(p, HK, HV, dk, dv, softplus=True, y=y0)
    assert y.data_ptr() == y0.data_ptr() and bool((y[:, sum(lengths):] == 7).all())
    n = sum(lengths)
    q = dict(p, row=p["row"][:, :n], dt=p["dt"][:, :n])
    check_scan(y[:, :n], hT, oracle(q, HK, HV, dk, dv, True), dtype, on_tensor_cores(dk, dv, dtype))


@pytest.mark.parametrize("dtype,dk,dv", [(F32, 64, 32), (BF16, 128, 128), (BF16, 128, 64)])
def test_a_nan_stays_in_its_sequence(dtype, dk, dv):
    HK, HV, lengths = 1, 2, [130, 50, 77]
    p = make_scan(lengths, HK, HV, dk, dv, dtype, seed=4)
    want = oracle(p, HK, HV, dk, dv, True)
    p["row"][:, 130:180] = float("nan")
    y, hT = run(p, HK, HV, dk, dv, softplus=True)
    keep = list(range(130)) + list(range(180, 257))
    check_scan(y[:, keep], hT[[0, 2]], (want[0][:, keep], want[1][[0, 2]], want[2][:, keep],
                                        want[3][:, keep], want[4][[0, 2]]), dtype,
               on_tensor_cores(dk, dv, dtype))


@pytest.mark.parametrize("dtype,dk,dv", [(F32, 32, 32), (F32, 128, 128), (BF16, 128, 128), (BF16, 128, 64),
                                         (BF16, 64, 128)])
def test_extreme_steps(dtype, dk, dv):
    # step sizes of zero (a padded token changes nothing), of -inf under softplus, and so
    # large that the state is forgotten at once; decay rate zero
    HK, HV, T = 1, 3, 200
    p = make_scan([T], HK, HV, dk, dv, dtype, seed=6, packed=False)
    p["a"] = torch.tensor([-1.0, -200.0, 0.0])
    p["dt_bias"] = None
    p["dt"][:, 10:40] = -float("inf")
    p["dt"][:, 50] = 300.0
    p["dt"][:, 100:104] = -100.0
    y, hT = run(p, HK, HV, dk, dv, softplus=True)
    check_scan(y, hT, oracle(p, HK, HV, dk, dv, True), dtype, on_tensor_cores(dk, dv, dtype))
    p["dt"] = torch.rand(1, T, HV)
    p["dt"][:, 20:60] = 0.0
    p["dt"][:, 60] = 50.0
    y, hT = run(p, HK, HV, dk, dv)
    check_scan(y, hT, oracle(p, HK, HV, dk, dv, False), dtype, on_tensor_cores(dk, dv, dtype))


def test_empty_calls():
    p = make_scan([0, 0], 1, 2, 128, 64, BF16, seed=1)
    y, hT = run(p, 1, 2, 128, 64, softplus=True)
    assert y.shape == (1, 0, 2, 64) and torch.equal(hT.cpu(), p["h0"])
    p = make_scan([0, 0], 1, 2, 32, 32, F32, seed=1, packed=False, h0=False)
    y, hT = run(p, 1, 2, 32, 32)
    assert hT.shape == (2, 2, 32, 32) and not hT.any()
    e = torch.empty(0, 5, 2, 64, dtype=BF16, device="cuda")
    y, hT = gdn.gdn_ssm_prefill(e, e[:, :, :1], e[:, :, :1], torch.empty(0, 5, 2, device="cuda"),
                                torch.zeros(2, device="cuda"))
    assert y.numel() == 0 and hT.shape == (0, 2, 64, 64)


@pytest.mark.parametrize("dtype,dk,dv", [(F32, 32, 32), (F32, 128, 128), (BF16, 64, 64), (BF16, 128, 64),
                                         (BF16, 128, 128)])
@pytest.mark.parametrize("N", [1, 200, 1500])
def test_batches_of_empty_sequences_with_rows_behind_them(dtype, dk, dv, N):
    # no CTA of the scan has a token: what is launched behind the call must still find hT
    # written and the workspace free (the next call rewrites both at once)
    HK, HV, T, rounds = 1, 2, 300, 20
    p = make_scan([0] * N, HK, HV, dk, dv, dtype, seed=N, pad=T)
    p["row"].fill_(float("nan"))
    g = to_cuda(p)
    x, b, c = split_row(g["row"], HK, HV, dk, dv)
    n = gdn.gdn_ssm_prefill_workspace_size(N, T, HK, HV, dk, dv, dtype, True)
    ws = torch.zeros(max(n, 16), dtype=torch.uint8, device="cuda")
    y = torch.full((1, T, HV, dv), 7.0, dtype=dtype, device="cuda")
    h0 = [torch.randn(N, HV, dv, dk, device="cuda") for _ in range(rounds)]
    hT = torch.zeros_like(h0[0])
    copies = []
    for h in h0:
        gdn.gdn_ssm_prefill(x, b, c, g["dt"], g["a"], d=g["d"], dt_bias=g["dt_bias"], h0=h,
                            cu_seqlens=g["cu_seqlens"], softplus=True, y=y, hT=hT, workspace=ws)
        copies.append(hT.clone())
    torch.cuda.synchronize()
    assert bool((y == 7).all())
    for h, got in zip(h0, copies):
        assert torch.equal(h, got)
    assert gdn.gdn_read_status(ws) == 0


@pytest.mark.parametrize("dk,dv", [(32, 32), (128, 128)])
@pytest.mark.parametrize("HV,T", [(8, 8192), (300, 1024)])
def test_decays_near_one_do_not_drift(dk, dv, HV, T):
    """Equal step sizes, so that every rounding of a decay points the same way, and no inputs:
    the state is h0 times one decay.  Allowed, in units of 2^-24 relative: one for each tile of
    16 tokens (the states' product), one for each of at most T / 128 segments (their chaining), 8
    for the last tile's decay and the product of all tiles' against its exponential, and 10 |log
    decay| (a product, four sums and an exponential behind each log, doubled for expm1f's slope).
    One rounding of each token's decay would be up to T / 2."""
    gen = torch.Generator().manual_seed(dk)
    a = -torch.linspace(0.5, 1.5, HV) / T
    h0 = 1 + torch.rand(1, HV, dv, dk, generator=gen)
    x, k = torch.zeros(1, T, HV, dv), torch.zeros(1, T, 1, dk)
    k[0, :, 0, 3] = 1.0
    y, hT = gdn.gdn_ssm_prefill(x.cuda(), k.cuda(), k.cuda(), torch.ones(1, T, HV).cuda(), a.cuda(), h0=h0.cuda())
    log = np.arange(1, T + 1)[:, None] * S.f64(a)
    units = T / 16 + T / 128 + 8 + 10 * np.abs(log[-1])
    ref = np.exp(log[-1])[None, :, None, None] * S.f64(h0)
    within(hT, ref, U32 * units[:, None, None] * ref, "hT")
    # the read-out multiplies once more, by the decays inside its tile
    ref = np.exp(log)[None, :, :, None] * S.f64(h0)[:, None, :, :, 3]
    within(y, ref, U32 * (units[:, None] + 8) * ref, "y")


@pytest.mark.parametrize("HV,dv", [(1, 128), (2, 64), (3, 64)])
@pytest.mark.parametrize("resets", [0, 1, 12, 31])
def test_each_score_is_rounded_once(HV, dv, resets):
    """x is the identity and b = c a unit vector, so y[i, j] is the score of tokens i and j alone,
    delta_j e^(decays behind j, up to i): exact but for its own rounding to bf16 (half a step of
    the value's binade) and fp32 errors: 40 roundings of its log2 decay, 16 for the rest.  In
    every 32 tokens the first `resets` of them forget everything, which must cost the scores of
    the tokens behind them no digits (nothing but a factor with one of them in it is 0)."""
    gen = torch.Generator().manual_seed(resets)
    dt = 0.02 + 0.3 * torch.rand(1, dv, HV, generator=gen)
    dt[:, torch.arange(dv) % 32 < resets] = 300.0
    a = -(0.3 + torch.rand(HV, generator=gen))
    x = torch.eye(dv).view(1, dv, 1, dv).expand(1, dv, HV, dv).to(BF16).contiguous()
    k = torch.zeros(1, dv, 1, 128, dtype=BF16)
    k[..., 5] = 1
    y, _ = gdn.gdn_ssm_prefill(x.cuda(), k.cuda(), k.cuda(), dt.cuda(), a.cuda())
    y, delta = S.f64(y)[0], S.f64(dt)[0]
    run = np.cumsum(delta * S.f64(a), axis=0)
    log = np.where(np.tri(dv, dtype=bool)[:, None], run[:, :, None] - run.T[None], -np.inf)     # [i, h, j]
    ref = np.exp(log) * delta.T[None]
    top = np.maximum(np.abs(y), ref)
    half = 2.0 ** (np.floor(np.log2(np.maximum(top, 1e-37))) - 8)
    units = 40 * np.abs(np.where(ref > 0, log, 0)) / np.log(2) + 16
    within(torch.from_numpy(y), ref, half + U32 * units * ref + 1e-37, "scores")


@pytest.mark.parametrize("HV,dv", [(148, 128), (296, 64), (147, 64)])
def test_each_carried_value_is_rounded_once(HV, dv):
    """One token's value in every column and b = c a unit vector: behind the first chunk of 128
    tokens y[i, j] is the value of token j alone, weighted to the chunk's end (rounded to bf16:
    half a step of its binade), decayed on, and rounded for the output.  fp32 on the way: 40
    roundings of the log2 decay, 24 for the rest.  (Heads enough that no sequence is cut.)"""
    gen = torch.Generator().manual_seed(HV)
    T, L = 200, 128
    dt = 0.01 + 0.1 * torch.rand(1, T, HV, generator=gen)
    a = -(0.2 + 0.8 * torch.rand(HV, generator=gen))
    value = (1 + torch.rand(HV, dv, generator=gen)).to(BF16)
    x = torch.zeros(1, T, HV, dv, dtype=BF16)
    j = torch.arange(dv)
    x[0, j, :, j] = value.t()
    k = torch.zeros(1, T, 1, 128, dtype=BF16)
    k[..., 9] = 1
    y, _ = gdn.gdn_ssm_prefill(x.cuda(), k.cuda(), k.cuda(), dt.cuda(), a.cuda())
    y, delta = S.f64(y)[0, L:], S.f64(dt)[0]
    run = np.cumsum(delta * S.f64(a), axis=0)                                       # [t, h]
    end = run[L - 1]
    weighted = delta[:dv].T * np.exp(end[:, None] - run[:dv].T) * S.f64(value)       # [h, j]
    on = np.exp(run[L:] - end)[:, :, None]
    ref = on * weighted

    def half(v):
        return 2.0 ** (np.floor(np.log2(v)) - 8)
    log = np.abs(run[L:, :, None] - run[:dv].T) / np.log(2)
    allow = half(np.maximum(np.abs(y), ref)) + on * half(weighted) + U32 * (40 * log + 24) * ref
    within(torch.from_numpy(y), ref, allow, "carried")


@pytest.mark.parametrize("dtype,dk,dv", [(F32, 32, 32), (BF16, 128, 128)])
def test_many_sequences(dtype, dk, dv):
    # more sequences than one block of the segment table takes at a time
    gen = np.random.RandomState(0)
    lengths = [int(v) for v in gen.randint(0, 3, 1500)]
    p = make_scan(lengths, 1, 1, dk, dv, dtype, seed=2)
    if dk == 128:
        p["h0"] = 0.1 * p["h0"]
    y, hT = run(p, 1, 1, dk, dv, softplus=True)
    check_scan(y, hT, oracle(p, 1, 1, dk, dv, True), dtype, on_tensor_cores(dk, dv, dtype))


@pytest.mark.parametrize("dtype,dk,dv", [(F32, 32, 32), (BF16, 128, 64)])
def test_long_sequences_between_many_short_ones(dtype, dk, dv):
    # nearly as many segments as are put in order: the long ones come last in the batch
    gen = np.random.RandomState(1)
    lengths = [int(v) for v in gen.randint(0, 3, 980)] + [700, 0, 1500, 129]
    p = make_scan(lengths, 1, 2, dk, dv, dtype, seed=3)
    if dk == 128:
        p["h0"] = 0.1 * p["h0"]
    y, hT = run(p, 1, 2, dk, dv, softplus=True)
    check_scan(y, hT, oracle(p, 1, 2, dk, dv, True), dtype, on_tensor_cores(dk, dv, dtype))


def test_without_final_state_and_optional_vectors():
    for dtype, dk, dv in ((F32, 64, 64), (BF16, 128, 128)):
        p = make_scan([700], 1, 2, dk, dv, dtype, seed=9, packed=False, h0=False)
        p["d"] = p["dt_bias"] = None
        y, hT = run(p, 1, 2, dk, dv, softplus=True, output_final_state=False)
        assert hT is None
        check_scan(y, None, oracle(p, 1, 2, dk, dv, True), dtype, on_tensor_cores(dk, dv, dtype))


def test_results_repeat_bit_for_bit_and_streams():
    HK, HV, dk, dv = 2, 4, 128, 64
    p = make_scan([600, 77, 1000], HK, HV, dk, dv, BF16, seed=8)
    y, hT = run(p, HK, HV, dk, dv, softplus=True)
    side = torch.cuda.Stream()
    g = to_cuda(p)
    x, b, c = split_row(g["row"], HK, HV, dk, dv)
    torch.cuda.synchronize()
    for _ in range(3):
        y2, h2 = gdn.gdn_ssm_prefill(x, b, c, g["dt"], g["a"], d=g["d"], dt_bias=g["dt_bias"],
                                     h0=g["h0"], cu_seqlens=g["cu_seqlens"], softplus=True, stream=side)
        side.synchronize()
        assert torch.equal(y, y2) and torch.equal(hT, h2)


@pytest.mark.parametrize("dtype,dk,dv,HK,HV", [(BF16, 128, 128, 1, 4), (BF16, 128, 64, 4, 16), (BF16, 64, 64, 1, 2),
                                               (F32, 128, 128, 1, 4), (F32, 32, 32, 1, 300)])
def test_one_workspace_for_calls_of_many_sizes(dtype, dk, dv, HK, HV):
    # sized for the largest: 5 sequences of 1200 tokens; smaller calls are cut otherwise, some finer
    for packed in (False, True):
        n = gdn.gdn_ssm_prefill_workspace_size(5, 6000 if packed else 1200, HK, HV, dk, dv, dtype, packed)
        ws = torch.full((max(n, 16) + 64,), 255, dtype=torch.uint8, device="cuda")
        behind = ws[max(n, 16):].clone()
        for lengths in ([1200] * 5, [1152], [1037] * 2, [640] * 3, [130], [1], [384] * 5):
            if packed and len(lengths) == 5:
                lengths = [v + w for v, w in zip(lengths, (0, -5, 0, 5, 0))]
            p = make_scan(lengths, HK, HV, dk, dv, dtype, seed=sum(lengths), packed=packed, step_mean=-4.0)
            y, hT = run(p, HK, HV, dk, dv, softplus=True)
            y2, h2 = run(p, HK, HV, dk, dv, softplus=True, workspace=ws[:n] if n else None)
            assert torch.equal(y, y2) and torch.equal(hT, h2), lengths
            assert not n or gdn.gdn_read_status(ws) == 0
        assert torch.equal(ws[max(n, 16):], behind)


def test_two_captured_graphs_with_their_own_workspaces():
    HK, HV, dk, dv = 1, 2, 128, 128
    n = gdn.gdn_ssm_prefill_workspace_size(2, 900, HK, HV, dk, dv, BF16, False)
    states, graphs, outs, want = [], [], [], []
    for seed in (21, 22):
        p = make_scan([900] * 2, HK, HV, dk, dv, BF16, seed=seed, packed=False)
        g = to_cuda(p)
        x, b, c = split_row(g["row"], HK, HV, dk, dv)
        ws = torch.empty(max(n, 16), dtype=torch.uint8, device="cuda")

        def call():
            return gdn.gdn_ssm_prefill(x, b, c, g["dt"], g["a"], d=g["d"], dt_bias=g["dt_bias"],
                                       h0=g["h0"], softplus=True, workspace=ws)
        want.append(tuple(t.clone() for t in call()))
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            outs.append(call())
        graphs.append(graph)
        states.append((g, x, b, c, ws))
    for _ in range(2):
        for graph in graphs:
            graph.replay()
    torch.cuda.synchronize()
    for got, ref in zip(outs, want):
        assert torch.equal(got[0], ref[0]) and torch.equal(got[1], ref[1])
    for s in states:
        assert gdn.gdn_read_status(s[-1]) == 0


@pytest.mark.parametrize("HK,HV,dv", [(1, 2, 128), (1, 2, 64), (1, 3, 64)])
def test_timeout_path_then_normal_call(HK, HV, dv):
    """Waits that give up (no hang: the test-only call has one role stopped from the start,
    and the flag set that the others' waits look at) leave the status word, free everything
    and return; the next call is exact again."""
    import ctypes
    from linear_attention_recurrence_rule_b200 import gdn as binding
    P, i32 = ctypes.c_void_p, ctypes.c_int
    f = binding.load_library().gdn_selftest_ssm_timeout
    f.restype, f.argtypes = i32, [P] * 5 + [i32, ctypes.c_int64, i32, i32, i32, P, P, P, ctypes.c_size_t, P]
    T = 1500
    p = make_scan([T], HK, HV, 128, dv, BF16, seed=41, packed=False, h0=False)
    p["d"] = p["dt_bias"] = None
    g = to_cuda(p)
    x, b, c = (t.contiguous() for t in split_row(g["row"], HK, HV, 128, dv))
    n = gdn.gdn_ssm_prefill_workspace_size(1, T, HK, HV, 128, dv, BF16, False)
    ws = torch.zeros(n, dtype=torch.uint8, device="cuda")
    y, hT = torch.empty_like(x), torch.empty(1, HV, dv, 128, device="cuda")
    rc = f(*(t.data_ptr() for t in (x, b, c, g["dt"], g["a"])), 1, T, HK, HV, dv, y.data_ptr(), hT.data_ptr(),
           ws.data_ptr(), n, torch.cuda.current_stream().cuda_stream)
    assert rc == 0
    torch.cuda.synchronize()
    assert gdn.gdn_read_status(ws) == binding.GDN_ERR_TIMEOUT
    y, hT = gdn.gdn_ssm_prefill(x, b, c, g["dt"], g["a"], softplus=True, workspace=ws)
    assert gdn.gdn_read_status(ws) == 0
    check_scan(y, hT, oracle(p, HK, HV, 128, dv, True), BF16, True)


# ---------------------------------------------------------------- one token
def make_step(N, HK, HV, dk, dv, W, dtype, seed, row_extra=0):
    gen = torch.Generator().manual_seed(seed)
    C = HV * dv + 2 * HK * dk
    r = lambda *s: torch.randn(*s, generator=gen)   # noqa: E731
    return dict(xbc=r(N, C + row_extra).to(dtype)[:, :C], conv_weight=r(C, W) / W ** 0.5, conv_bias=0.1 * r(C),
                conv_state=r(N, W - 1, C).to(dtype), dt=r(N, HV), dt_bias=-1 + r(HV), a=-torch.rand(HV, generator=gen) * 4,
                d=r(HV), state=r(N, HV, dv, dk))


def check_step(p, y, state, conv_state, dtype, silu, soft):
    row, cs = S.conv_token(p["xbc"], p["conv_weight"], p["conv_bias"], p["conv_state"], silu)
    ry, rs, ya, yu, hu = S.step(row, p["dt"], p["a"], p["state"], p["d"], p["dt_bias"], soft)
    # the convolved row itself is an fp32 sum of W + 1 terms and a SiLU: error at most
    # (W + 8) units of the sum of |terms|, entering y and the state as a change of x, b, c
    W = p["conv_weight"].shape[1]
    ra, _ = S.conv_token(p["xbc"].double().abs(), p["conv_weight"].abs(), p["conv_bias"].abs(),
                         p["conv_state"].double().abs(), False)
    over = (W + 8) * np.maximum(ra, np.abs(row))   # units; |silu'| <= 1.1 is inside the 8
    N, HV, dv, dk = p["state"].shape
    HK = (row.shape[1] - HV * dv) // (2 * dk)
    grp = np.arange(HV) // (HV // HK)

    def parts(v):
        v = np.abs(v)
        return (v[:, :HV * dv].reshape(N, HV, dv), v[:, HV * dv:HV * dv + HK * dk].reshape(N, HK, dk)[:, grp],
                v[:, HV * dv + HK * dk:].reshape(N, HK, dk)[:, grp])
    x, b, c = parts(row)
    ex, eb, ec = parts(1.1 * over)
    delta = S.f64(p["dt"]) + S.f64(p["dt_bias"])
    delta = np.abs(S.softplus(delta) if soft else delta)[..., None]
    hu = hu + (delta * ex)[..., None] * b[:, :, None] + (delta * x)[..., None] * eb[:, :, None]
    yu = yu + np.einsum("nhvk,nhk->nhv", hu, c) + np.einsum("nhvk,nhk->nhv", np.abs(rs), ec) \
        + np.abs(S.f64(p["d"]))[:, None] * ex
    within(y, ry, U[dtype] * np.abs(ry) + 2 * U32 * yu + 1e-37, "y")
    within(state, rs, 2 * U32 * hu + 1e-37, "state")
    assert torch.equal(conv_state.cpu().double(), torch.from_numpy(cs)), "carried inputs"


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("N,HK,HV,dk,dv,W", [(1, 1, 1, 32, 32, 2), (3, 2, 4, 128, 128, 4), (5, 1, 6, 128, 64, 4),
                                             (2, 4, 4, 64, 100, 8), (1, 1, 2, 128, 256, 3), (7, 2, 6, 32, 1, 5)])
@pytest.mark.parametrize("in_place", [False, True])
def test_step(dtype, N, HK, HV, dk, dv, W, in_place):
    p = make_step(N, HK, HV, dk, dv, W, dtype, seed=N + dv, row_extra=3)
    g = to_cuda(p)
    args = dict(d=g["d"], dt_bias=g["dt_bias"], conv_weight=g["conv_weight"], conv_bias=g["conv_bias"],
                conv_state=g["conv_state"], silu=True, softplus=True)
    if in_place:
        y = gdn.gdn_ssm_step(g["xbc"], g["dt"], g["a"], g["state"], **args)
        check_step(p, y, g["state"], g["conv_state"], dtype, True, True)
    else:
        so, co = torch.empty_like(g["state"]), torch.empty_like(g["conv_state"])
        y = gdn.gdn_ssm_step(g["xbc"], g["dt"], g["a"], g["state"], state_out=so, conv_state_out=co, **args)
        check_step(p, y, so, co, dtype, True, True)
        assert torch.equal(g["state"].cpu(), p["state"]) and torch.equal(g["conv_state"].cpu(), p["conv_state"])


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_step_without_convolution_or_softplus(dtype):
    N, HK, HV, dk, dv = 4, 2, 4, 64, 64
    p = make_step(N, HK, HV, dk, dv, 2, dtype, seed=31)
    p["dt"] = p["dt"].abs()
    g = to_cuda(p)
    y = gdn.gdn_ssm_step(g["xbc"], g["dt"], g["a"], g["state"])
    ry, rs, _, yu, hu = S.step(p["xbc"], p["dt"], p["a"], p["state"])
    within(y, ry, U[dtype] * np.abs(ry) + 2 * U32 * yu, "y")
    within(g["state"], rs, 2 * U32 * hu, "state")
    # activation off, no bias
    p["conv_bias"] = torch.zeros_like(p["conv_bias"])
    g = to_cuda(p)
    y = gdn.gdn_ssm_step(g["xbc"], g["dt"], g["a"], g["state"], d=g["d"], dt_bias=g["dt_bias"],
                         conv_weight=g["conv_weight"], conv_state=g["conv_state"], softplus=True)
    check_step(p, y, g["state"], g["conv_state"], dtype, False, True)


def test_step_of_no_sequences_and_captured():
    p = make_step(0, 1, 2, 64, 64, 4, BF16, seed=1)
    g = to_cuda(p)
    assert gdn.gdn_ssm_step(g["xbc"], g["dt"], g["a"], g["state"]).shape == (0, 2, 64)
    # a captured step moves the states in place once per replay
    p = make_step(3, 1, 2, 128, 64, 4, BF16, seed=2)
    g = to_cuda(p)
    h = {k: v.clone() for k, v in g.items()}

    def call(q):
        return gdn.gdn_ssm_step(q["xbc"], q["dt"], q["a"], q["state"], d=q["d"], dt_bias=q["dt_bias"],
                                conv_weight=q["conv_weight"], conv_bias=q["conv_bias"],
                                conv_state=q["conv_state"], silu=True, softplus=True)
    call(h)
    h = {k: v.clone() for k, v in g.items()}
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y = call(h)
    for _ in range(3):
        graph.replay()
    for _ in range(3):
        want = call(g)
    assert torch.equal(y, want) and torch.equal(h["state"], g["state"])
    assert torch.equal(h["conv_state"], g["conv_state"])


# ---------------------------------------------------------------- the run of them
@pytest.mark.parametrize("dtype,dk,dv", [(F32, 32, 32), (F32, 128, 64), (BF16, 128, 64), (BF16, 128, 128)])
def test_block_over_prompt_then_tokens(dtype, dk, dv):
    """Convolution, scan, gated norm and residual norm over a ragged prompt, then token by
    token with the carried states: the same as the prompt form over the longer prompt, and
    as the oracle's composition."""
    HK, HV, W, steps = 1, 2, 4, 3
    lengths = [37, 1, 150]
    C, width = HV * dv + 2 * HK * dk, HV * dv
    full = [n + steps for n in lengths]
    gen = torch.Generator().manual_seed(77)
    r = lambda *s: torch.randn(*s, generator=gen)   # noqa: E731
    proj, z, res = r(1, sum(full), C).to(dtype), r(1, sum(full), width).to(dtype), r(1, sum(full), width)
    dt, dt_bias, a, d = r(1, sum(full), HV), -2 + r(HV), -torch.rand(HV, generator=gen) * 3, r(HV)
    cw, cb, w1, w2, w3 = r(C, W) / 2, 0.1 * r(C), 1 + 0.1 * r(HV, dv), 1 + 0.1 * r(width), 1 + 0.1 * r(width)
    dev = {k: v.cuda() for k, v in dict(proj=proj, z=z, res=res, dt=dt, dt_bias=dt_bias, a=a, d=d, cw=cw, cb=cb,
                                        w1=w1, w2=w2, w3=w3).items()}

    def tail(y, z, res):
        n = gdn.gdn_gated_norm(y, z.view(y.shape), dev["w1"], gate="silu", gate_first=True)
        return gdn.gdn_residual_norm(n.view(z.shape), res, dev["w3"], post_weight=dev["w2"], scale=0.5)

    def prompt(rows, lens):
        cu = torch.tensor(np.concatenate([[0], np.cumsum(lens)]), dtype=torch.int32).cuda()
        q = {k: dev[k][:, rows].contiguous() for k in ("proj", "z", "res", "dt")}
        conv = torch.zeros(len(lens), W - 1, C, dtype=dtype, device="cuda")
        xbc = gdn.gdn_short_conv(q["proj"], dev["cw"], dev["cb"], conv, cu, silu=True)
        y, h = gdn.gdn_ssm_prefill(*split_row(xbc, HK, HV, dk, dv), q["dt"], dev["a"], d=dev["d"],
                                   dt_bias=dev["dt_bias"], cu_seqlens=cu, softplus=True)
        return (y, h, conv, xbc) + tail(y, q["z"], q["res"])

    starts = np.concatenate([[0], np.cumsum(full)])
    head = [t for n, s in zip(lengths, starts) for t in range(s, s + n)]
    every = list(range(sum(full)))
    y1, h, conv, _, out1, _ = prompt(head, lengths)
    yf, hf, convf, xbc, outf, resf = prompt(every, full)
    # prompts against the oracle on the convolved values the library stored
    cu = torch.tensor(starts, dtype=torch.int32)
    ref = S.scan(*split_row(xbc.cpu(), HK, HV, dk, dv), dt, a, d, dt_bias, None, cu, True)
    tc = on_tensor_cores(dk, dv, dtype)
    check_scan(yf, hf, ref, dtype, tc)
    assert torch.equal(y1, yf[:, head]) or tc or dtype == F32
    # the norms against the oracle on the library's own y
    n_ref = S.gated_norm(yf, z.reshape(yf.shape), w1, 1e-6, "silu", True, False)
    n_lib = gdn.gdn_gated_norm(yf, dev["z"].view(yf.shape), dev["w1"], gate="silu", gate_first=True)
    within(n_lib, n_ref, (U[dtype] + 128 * U32) * np.abs(n_ref) + (2e-6 if dtype == BF16 else 0) * np.abs(n_ref), "norm")
    o_ref, h_ref, t_ref = S.residual_norm(n_lib.reshape(z.shape), res, w3, w2, None, 0.5, 1e-6, "sigmoid", False)
    h_err = 128 * U32 * (np.abs(h_ref) + np.abs(t_ref))
    within(resf, h_ref, h_err, "residual")
    scale = np.abs(o_ref) / np.maximum(np.abs(h_ref), 1e-30)
    within(outf, o_ref, U[dtype] * np.abs(o_ref) + scale * h_err + 128 * U32 * np.abs(o_ref), "out")
    # token by token: states against the prompt form's, both within their bounds of the
    # exact ones; the token form keeps the convolved row in fp32, the prompt form rounds it
    for i in range(steps):
        rows = [int(s) + n + i for n, s in zip(lengths, starts)]
        q = {k: dev[k][0, rows].contiguous() for k in ("proj", "z", "res", "dt")}
        y = gdn.gdn_ssm_step(q["proj"], q["dt"], dev["a"], h, d=dev["d"], dt_bias=dev["dt_bias"],
                             conv_weight=dev["cw"], conv_bias=dev["cb"], conv_state=conv, silu=True, softplus=True)
        out, _ = tail(y, q["z"], q["res"])
        # one rounding of each of x, b, c, then the outputs' own and the tensor-core terms
        lim = 5 * U[dtype] * ref[2][0, rows] + 8 * U32 * ref[3][0, rows]
        within(y, S.f64(yf)[0, rows], lim, "token y")
        assert bool(torch.isfinite(out).all())
    assert torch.equal(conv, convf)


# ---------------------------------------------------------------- offsets past 32 bits
def test_prefill_offsets_past_32_bits():
    # 2.2e9 elements of x and y: the last heads of the last tokens against a call on those
    # heads alone (other cuts, so within the bounds of two results: the output's rounding
    # each, and twice the terms' -- taken relative to the rows' norms)
    HK, HV, dk, dv, T = 1, 64, 128, 128, 270_000
    gen = torch.Generator(device="cuda").manual_seed(0)
    x = torch.empty(1, T, HV, dv, dtype=BF16, device="cuda").normal_(generator=gen)
    b, c = (torch.empty(1, T, HK, dk, dtype=BF16, device="cuda").normal_(generator=gen) for _ in range(2))
    dt = torch.empty(1, T, HV, device="cuda").normal_(generator=gen)
    a, bias = -torch.linspace(0.5, 4, HV, device="cuda"), torch.full((HV,), -2.0, device="cuda")
    y, hT = gdn.gdn_ssm_prefill(x, b, c, dt, a, dt_bias=bias, softplus=True)
    assert y.numel() > 2 ** 31
    few = slice(HV - 2, HV)
    y2, h2 = gdn.gdn_ssm_prefill(x[:, :, few], b, c, dt[:, :, few].contiguous(), a[few].contiguous(),
                                 dt_bias=bias[few].contiguous(), softplus=True)
    u, v = y[0, -4096:, few].double(), y2[0, -4096:].double()
    assert float((u - v).norm() / v.norm()) < 6 * U[BF16]
    assert float((hT[:, few] - h2).double().norm() / h2.double().norm()) < 2e-6
    # and of the first tokens, so that no offset wraps onto them
    u, v = y[0, :4096, few].double(), y2[0, :4096].double()
    assert float((u - v).norm() / v.norm()) < 6 * U[BF16]


def test_step_offsets_past_32_bits():
    N, HK, HV, dk, dv, W = 4200, 1, 32, 128, 128, 4          # 2.2e9 state elements
    C = HV * dv + 2 * HK * dk
    gen = torch.Generator(device="cuda").manual_seed(1)
    r = lambda *s: torch.empty(*s, device="cuda").normal_(generator=gen)   # noqa: E731
    state, xbc, dt = r(N, HV, dv, dk), r(N, C).to(BF16), r(N, HV)
    assert state.numel() > 2 ** 31
    cw, cs, a = r(C, W), r(N, W - 1, C).to(BF16), -torch.rand(HV, generator=gen, device="cuda")
    last = slice(N - 3, N)
    s2, c2 = state[last].clone(), cs[last].clone()
    y2 = gdn.gdn_ssm_step(xbc[last].contiguous(), dt[last].contiguous(), a, s2, conv_weight=cw, conv_state=c2, silu=True,
                          softplus=True)
    y = gdn.gdn_ssm_step(xbc, dt, a, state, conv_weight=cw, conv_state=cs, silu=True, softplus=True)
    assert torch.equal(y[last], y2) and torch.equal(state[last], s2) and torch.equal(cs[last], c2)
