"""A decay that is NaN reaches the results: a broken gate shows instead of passing for a decay of 0."""
import pytest
import torch

import linear_testlib as lib
from gated_delta_rule_148_b200 import kda

pytestmark = pytest.mark.gpu
NAN = float("nan")


def _all_nan(x):
    return bool(torch.isnan(x).all())


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("dk,dv,at", [(64, 64, 70), (128, 128, 71), (64, 64, 129), (128, 128, 0)])
def test_a_decay_that_is_nan(dtype, dk, dv, at):
    """From its token on o is NaN, and so are the state, its gradient before the token and all decays' gradients of
    that sequence and head; nothing else changes."""
    clean = lib.case(94, [200, 90], 2, 2, dk, dv, dtype)
    c = {n: x.clone() if isinstance(x, torch.Tensor) else x for n, x in clean.items()}
    c["log_alpha"][at, 1] = NAN
    clean, c = lib.to_cuda(clean), lib.to_cuda(c)

    def run(c):
        o, s = kda.linear_prefill(c["q"], c["k"], c["v"], c["log_alpha"], c["cu_seqlens"], init_state=c["init_state"])
        g = kda.linear_prefill_backward(c["q"], c["k"], c["v"], c["log_alpha"], c["cu_seqlens"], c["grad_o"],
                                        grad_final_state=c["grad_final_state"], init_state=c["init_state"])
        assert kda.get_device_status() == kda.KDA_OK
        return o, s, g

    (wo, ws, wg), (o, s, g) = run(clean), run(c)
    assert _all_nan(o[at:200, 1]) and _all_nan(s[0, 1])
    assert torch.equal(o[:at], wo[:at]) and torch.equal(o[:, 0], wo[:, 0]) and torch.equal(o[200:], wo[200:])
    assert torch.equal(s[:, 0], ws[:, 0]) and torch.equal(s[1], ws[1])
    assert _all_nan(g["dq"][at:200, 1]) and _all_nan(g["dk"][:at, 1]) and _all_nan(g["dv"][:at, 1])
    assert _all_nan(g["dlog_alpha"][:200, 1]) and _all_nan(g["dS0"][0, 1])
    assert torch.equal(g["dq"][:at], wg["dq"][:at])
    for name in ("dq", "dk", "dv", "dlog_alpha"):
        assert torch.equal(g[name][:, 0], wg[name][:, 0]) and torch.equal(g[name][200:], wg[name][200:]), name
    assert torch.equal(g["dS0"][1], wg["dS0"][1]) and torch.equal(g["dS0"][:, 0], wg["dS0"][:, 0])


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_a_head_s_constant_decay_that_is_nan(dtype):
    c = lib.to_cuda(lib.case(95, [150, 3], 3, 1, 64, 64, dtype, decay="head"))
    c["log_alpha"][2] = NAN
    o, s = kda.linear_prefill(c["q"], c["k"], c["v"], c["log_alpha"], c["cu_seqlens"], init_state=c["init_state"])
    assert _all_nan(o[:, 2]) and _all_nan(s[:, 2]) and torch.isfinite(o[:, :2]).all() and torch.isfinite(s[:, :2]).all()
    g = kda.linear_prefill_backward(c["q"], c["k"], c["v"], c["log_alpha"], c["cu_seqlens"], c["grad_o"], init_state=c["init_state"])
    assert torch.isnan(g["dlog_alpha"][2]) and torch.isfinite(g["dlog_alpha"][:2]).all() and _all_nan(g["dq"])
    assert kda.get_device_status() == kda.KDA_OK


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_a_decay_that_is_nan_at_a_pad_has_no_effect(dtype):
    c = lib.case(96, [100], 2, 2, 64, 64, dtype, pads=0.3)
    want = kda.linear_prefill(*(lib.to_cuda(c)[n] for n in ("q", "k", "v", "log_alpha", "cu_seqlens", "pad_mask", "init_state")))
    c["log_alpha"][c["pad_mask"] == 0] = NAN
    got = kda.linear_prefill(*(lib.to_cuda(c)[n] for n in ("q", "k", "v", "log_alpha", "cu_seqlens", "pad_mask", "init_state")))
    assert all(torch.equal(a, b) for a, b in zip(want, got))
    assert kda.get_device_status() == kda.KDA_OK
