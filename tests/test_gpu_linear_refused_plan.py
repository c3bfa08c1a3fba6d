"""A linear-attention call whose cu_seqlens are invalid leaves its own mark in its workspace, which its later kernels go by."""
import pytest
import torch

import linear_testlib as lib
from gated_delta_rule_148_b200 import kda

pytestmark = pytest.mark.gpu
REFUSED = -1


def _marks(ws, B):
    return ws[: 4 * (B + 1)].view(torch.int32)[B].item()


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("lengths,H", [([30, 40], 2), ([4096], 1)], ids=["short", "few_long_heads"])
def test_refused_calls_are_marked_and_the_next_are_whole(dtype, lengths, H):
    c = lib.case(80, lengths, H, 1, 64, 64, dtype, decay="head")
    d = lib.to_cuda(c)
    N, B = sum(lengths), len(lengths)
    ws = torch.zeros(kda.linear_prefill_workspace(N, B, H, 1, 64, 64, dtype=c["dtype"]).numel(), dtype=torch.uint8, device="cuda")
    a = kda.LinearBackwardArgs()
    a.dtype, a.num_seqs, a.total_tokens, a.H, a.Hk, a.dk, a.dv = kda.KDA_BF16 if dtype == "bf16" else kda.KDA_F32, B, N, H, 1, 64, 64
    a.decay = kda.KDA_DECAY_HEAD
    back = torch.zeros(kda.load().kda_linear_prefill_backward_workspace_size(a), dtype=torch.uint8, device="cuda")
    bad = torch.tensor([0, N + 1] if B == 1 else [0, 40, 30], dtype=torch.int32, device="cuda")
    o, s = torch.full_like(d["v"], 7.0), torch.full_like(d["init_state"], 7.0)

    def prefill(cu):
        return kda.linear_prefill(d["q"], d["k"], d["v"], d["log_alpha"], cu, init_state=d["init_state"], o=o, final_state=s,
                                  workspace=ws)

    def backward(cu):
        return kda.linear_prefill_backward(d["q"], d["k"], d["v"], d["log_alpha"], cu, d["grad_o"],
                                           grad_final_state=d["grad_final_state"], init_state=d["init_state"], workspace=back)

    prefill(bad)
    assert kda.get_device_status() == kda.KDA_ERR_DEVICE_CHECK and _marks(ws, B) == REFUSED
    assert torch.all(o == 7) and torch.all(s == 7)
    backward(bad)
    backward(d["cu_seqlens"])      # an error is latched: refused too
    assert kda.get_device_status() == kda.KDA_ERR_DEVICE_CHECK and _marks(back, B) == REFUSED
    prefill(d["cu_seqlens"])
    g = backward(d["cu_seqlens"])
    assert kda.get_device_status() == kda.KDA_OK and _marks(ws, B) > 0 and _marks(back, B) > 0
    ref, mag = lib.backward(c), lib.backward(c, mag=True)
    for name in ("dq", "dk", "dv"):
        lib.check(name, g[name], ref[name], mag[name], 1 if dtype == "bf16" else 0, dtype == "bf16")
    for name in ("dlog_alpha", "dS0"):
        lib.check(name, g[name], ref[name], mag[name], 0, False)
