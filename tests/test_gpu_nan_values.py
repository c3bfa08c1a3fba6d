"""NaN that a call is given reaches its results: a broken gate or value shows instead of turning into a number."""
import pytest
import torch

import linear_testlib as lib
from gated_delta_rule_148_b200 import kda

pytestmark = pytest.mark.gpu
NAN = float("nan")


def _all_nan(x):
    return bool(torch.isnan(x).all())


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_values_in_decode(dtype):
    c = lib.to_cuda(lib.case(90, [1] * 5, 4, 2, 64, 128, dtype))
    want_state = c["init_state"].clone()
    want = kda.linear_decode(c["q"], c["k"], c["v"], c["log_alpha"], want_state)
    state = c["init_state"].clone()
    c["v"][3, 2, 7] = NAN
    o = kda.linear_decode(c["q"], c["k"], c["v"], c["log_alpha"], state)
    hit = torch.zeros_like(o, dtype=torch.bool)
    hit[3, 2, 7] = True
    assert _all_nan(o[hit]) and torch.equal(o[~hit], want[~hit])
    assert _all_nan(state[3, 2, :, 7]) and torch.equal(state[:3], want_state[:3])
    c = lib.to_cuda(lib.case(91, [1] * 5, 4, 2, 64, 128, dtype))
    c["log_alpha"][1, 3] = NAN
    o = kda.linear_decode(c["q"], c["k"], c["v"], c["log_alpha"], c["init_state"])
    assert _all_nan(o[1, 3]) and torch.isfinite(o[[0, 2, 3, 4]]).all() and torch.isfinite(o[1, :3]).all()
    assert kda.get_device_status() == kda.KDA_OK


def test_values_in_the_delta_rule_s_decode_and_prompt():
    g = torch.Generator().manual_seed(92)
    H, d = 2, 64
    q, k, v = (torch.nn.functional.normalize(torch.randn(3, H, d, generator=g), dim=-1).bfloat16().cuda() for _ in range(3))
    la, beta = -torch.rand(3, H, d, generator=g).cuda(), torch.rand(3, H, generator=g).cuda()
    v[1, 0, 5] = NAN
    o = kda.decode(q, k, v, la, beta, torch.zeros(3, H, d, d, device="cuda"))
    assert torch.isnan(o[1, 0, 5]) and torch.isfinite(o[[0, 2]]).all()
    o, s = kda.prefill(q, k, v, la, beta, torch.tensor([0, 3], dtype=torch.int32, device="cuda"), chunk=16)
    assert torch.isnan(o[1, 0, 5]) and torch.isnan(o[2, 0, 5]) and torch.isnan(s[0, 0, :, 5]).all()
    assert kda.get_device_status() == kda.KDA_OK


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_gradients_of_shared_heads(dtype):
    """dq of a key head is the sum over its value heads: one of them NaN, the sum NaN."""
    c = lib.to_cuda(lib.case(93, [40], 4, 2, 64, 64, dtype))
    c["grad_o"][11, 1, 3] = NAN
    g = kda.linear_prefill_backward(c["q"], c["k"], c["v"], c["log_alpha"], c["cu_seqlens"], c["grad_o"], init_state=c["init_state"])
    assert _all_nan(g["dq"][11, 0]) and torch.isfinite(g["dq"][:, 1]).all()
    assert kda.get_device_status() == kda.KDA_OK
