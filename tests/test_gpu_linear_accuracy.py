"""Relative 2-norms of whole outputs against the 64-bit recurrence: the accuracy that the header states, near enough that a
part left out of a product shows (bounds derived in linear_accuracy_lib)."""
import pytest
import torch

import linear_accuracy_lib as bounds
import linear_testlib as lib
from gated_delta_rule_148_b200 import kda

pytestmark = pytest.mark.gpu


def _check(c):
    d = lib.to_cuda(c)
    bf16 = c["dtype"] == torch.bfloat16
    o, s = kda.linear_prefill(d["q"], d["k"], d["v"], d["log_alpha"], d["cu_seqlens"], pad_mask=d["pad_mask"],
                              init_state=d["init_state"])
    g = kda.linear_prefill_backward(d["q"], d["k"], d["v"], d["log_alpha"], d["cu_seqlens"], d["grad_o"],
                                    grad_final_state=d["grad_final_state"], pad_mask=d["pad_mask"], init_state=d["init_state"])
    assert kda.get_device_status() == kda.KDA_OK
    (ro, rs), rg = lib.prefill(c), lib.backward(c)
    wide = bounds.BF16_NORM if bf16 else bounds.FP32_NORM
    off = {"o": (bounds.relative(o, ro), wide), "final_state": (bounds.relative(s, rs), bounds.FP32_NORM),
           "dS0": (bounds.relative(g["dS0"], rg["dS0"]), bounds.FP32_NORM),
           "dlog_alpha": (bounds.relative(g["dlog_alpha"], rg["dlog_alpha"]), bounds.TWO_PART_NORM if bf16 else bounds.FP32_NORM)}
    off.update({n: (bounds.relative(g[n], rg[n]), wide) for n in ("dq", "dk", "dv")})
    print({n: f"{x:.2e}" for n, (x, _) in off.items()})
    assert all(x <= bound for x, bound in off.values()), off


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("dk,dv", [(64, 64), (64, 128), (128, 64), (128, 128)])
def test_ragged_batch(dtype, dk, dv):
    _check(lib.case(110, [700, 129, 1, 260], 4, 2, dk, dv, dtype, pads=0.03))


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_constant_decays_of_a_head(dtype):
    _check(lib.case(111, [400, 90], 2, 1, 128, 128, dtype, decay="head"))


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_few_long_heads(dtype):
    """bf16: the sweeps start from segments' states."""
    _check(lib.case(112, [4096], 1, 1, 64, 64, dtype))


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("rows", [1, 40])
def test_decode(dtype, rows):
    c = lib.case(113, [1] * rows, 8, 2, 128, 128, dtype)
    d = lib.to_cuda(c)
    o = kda.linear_decode(d["q"], d["k"], d["v"], d["log_alpha"], d["init_state"])
    ro, rs = lib.prefill(c)
    assert bounds.relative(d["init_state"], rs) <= bounds.FP32_NORM
    # no operand is rounded: the output alone
    assert bounds.relative(o, ro) <= (3.0 ** -0.5 * lib.HALF_BF16 if dtype == "bf16" else bounds.FP32_NORM)


def test_captured_calls_write_every_output_on_every_replay():
    """Two captured prefills and backwards with workspaces of their own, replayed on two streams at once; every output is
    overwritten before each replay."""
    cs = [lib.case(120 + i, [300, 40], 2, 1, 128, 128, "bf16", pads=0.1) for i in range(2)]
    graphs = []
    for c in cs:
        d = lib.to_cuda(c)

        def call(o=None, s=None, ws=None):
            o, s = kda.linear_prefill(d["q"], d["k"], d["v"], d["log_alpha"], d["cu_seqlens"], pad_mask=d["pad_mask"],
                                      init_state=d["init_state"], o=o, final_state=s, workspace=ws)
            g = kda.linear_prefill_backward(d["q"], d["k"], d["v"], d["log_alpha"], d["cu_seqlens"], d["grad_o"],
                                            grad_final_state=d["grad_final_state"], pad_mask=d["pad_mask"], init_state=d["init_state"])
            return [o, s] + [g[n] for n in sorted(g)]

        want = [x.clone() for x in call()]
        ws = kda.linear_prefill_workspace(340, 2, 2, 1, 128, 128)
        o, s = torch.empty_like(want[0]), torch.empty_like(want[1])
        stream, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
        stream.wait_stream(torch.cuda.current_stream())
        with torch.cuda.graph(graph, stream=stream):
            got = call(o, s, ws)
        graphs.append((graph, stream, got, want, d, ws))
    for _ in range(3):
        for graph, stream, got, *_ in graphs:
            for x in got:
                x.fill_(7.0)
        for graph, stream, *_ in graphs:
            stream.wait_stream(torch.cuda.current_stream())
            with torch.cuda.stream(stream):
                graph.replay()
        for graph, stream, *_ in graphs:
            torch.cuda.current_stream().wait_stream(stream)
        torch.cuda.synchronize()
        for _, _, got, want, *_ in graphs:
            assert all(torch.equal(a, b) for a, b in zip(got, want))
    assert kda.get_device_status() == kda.KDA_OK


@pytest.mark.parametrize("dtype,rows,D", [("bf16", 6000, 8192), ("f32", 6000, 2056), ("f32", 3000, 16384)])
def test_norm_weight_gradient_of_many_wide_rows(dtype, rows, D):
    """Rows this wide have a block each, 148 blocks at least: a thread adds rows / 148 of them one by one, then up to 296
    blocks' sums are added in 32 shares and the shares together: fp32 steps of 2^-24 of the sum of absolute terms."""
    g = torch.Generator(device="cuda").manual_seed(130)
    dt = torch.bfloat16 if dtype == "bf16" else torch.float32
    x, dy = (torch.randn(rows, D, generator=g, device="cuda").to(dt) for _ in range(2))
    _, dw = kda.rms_norm_backward(x, None, dy, eps=1e-5)
    c = 1 / (x.double().square().mean(1, keepdim=True) + 1e-5).sqrt()
    terms = dy.double() * x.double() * c
    steps = rows / 148 + 1 + 296 / 32 + 32
    assert ((dw.double() - terms.sum(0)).abs() <= (2.0 ** -19 + steps * 2.0 ** -24) * terms.abs().sum(0)).all()
    # in the 2-norm the steps' errors are independent, half a step at most each, of sums that grow with the root of the rows
    assert bounds.relative(dw, terms.sum(0).cpu()) <= steps ** 0.5 * 2.0 ** -24 + 2.0 ** -22
