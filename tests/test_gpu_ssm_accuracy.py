"""How far the scan's outputs may be off on the tensor cores, counted term by term and in
norm, against the float64 oracle."""
import pytest
import torch

import linear_attention_recurrence_rule_b200 as gdn
from ssm_util import U32, in_norm, make_scan, sequences, split_row, term_bounds, to_cuda, within

pytestmark = pytest.mark.gpu

BF16 = torch.bfloat16


def run(p, HK, HV, dk, dv):
    g = to_cuda(p)
    return gdn.gdn_ssm_prefill(*split_row(g["row"], HK, HV, dk, dv), g["dt"], g["a"], d=g["d"], dt_bias=g["dt_bias"],
                               h0=g["h0"], cu_seqlens=g["cu_seqlens"], softplus=True)


CASES = [(1, 2, 128), (1, 2, 64), (1, 3, 64), (2, 4, 64)]


@pytest.mark.parametrize("HK,HV,dv", CASES)
@pytest.mark.parametrize("lengths,packed,step_mean", [([128], False, -2.0), ([260] * 2, False, -2.0),
                                                      ([1, 700, 33, 390], True, -4.0), ([1411], False, -6.0)])
@pytest.mark.parametrize("skip", [True, False])
def test_terms_on_tensor_cores(HK, HV, dv, lengths, packed, step_mean, skip):
    dk = 128
    p = make_scan(lengths, HK, HV, dk, dv, BF16, seed=sum(lengths) + dv, packed=packed, step_mean=step_mean)
    if not skip:
        p["d"] = p["h0"] = None
    y, hT = run(p, HK, HV, dk, dv)
    ref, h, allow, norm, h_units = term_bounds(p, HK, HV, dk, dv)
    within(y, ref, allow + 1e-37, "y")
    within(hT, h, 2 * U32 * h_units + 1e-37, "hT")
    assert in_norm(y, ref, norm, sequences(p)), "y in norm"
