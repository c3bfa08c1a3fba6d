"""CPU: the bounds of the accuracy tests lie between what the linear-attention kernels' splits into bf16 parts leave and what
one part fewer would: the mistake is planted in the oracle."""
import pytest
import torch

import linear_accuracy_lib as bounds
import linear_testlib as lib


def _parts(x, n):
    """Sum of the first n bf16 parts of x (in 64 bits; the parts are taken in fp32, as the kernels do)."""
    rest, out = x.float(), torch.zeros_like(x)
    for _ in range(n):
        p = rest.bfloat16().float()
        out += p.double()
        rest = rest - p
    return out


def _state(c, parts):
    """A chunk's share of the state, K^T (w V), with w V in so many parts."""
    b = c["log_alpha"].double().cumsum(0)
    w = (b[-1] - b).exp()
    wv = w[:, :, None] * c["v"].double()
    return torch.einsum("nhk,nhv->hkv", c["k"].double(), wv if parts is None else _parts(wv, parts))


@pytest.mark.parametrize("la_scale", [1.0, 0.01])
def test_states_need_three_parts(la_scale):
    c = lib.case(100, [128], 4, 4, 128, 128, "bf16", la_scale=la_scale)
    ref = _state(c, None)
    assert bounds.relative(_state(c, 3), ref) < bounds.FP32_NORM / 8
    assert bounds.relative(_state(c, 2), ref) > 2 * bounds.FP32_NORM


def test_decay_gradients_need_two_parts():
    """<S, D>, with both as so many parts; one value per chunk and head."""
    g = torch.Generator().manual_seed(101)
    S, D = (torch.randn(64, 128, 128, generator=g, dtype=torch.float64) for _ in range(2))
    ref = (S * D).sum((1, 2))
    assert bounds.relative((_parts(S, 2) * _parts(D, 2)).sum((1, 2)), ref) < bounds.TWO_PART_NORM
    assert bounds.relative((_parts(S, 1) * _parts(D, 2)).sum((1, 2)), ref) > 8 * bounds.TWO_PART_NORM


def test_bf16_outputs_allow_one_rounded_operand():
    """o = P V rounded to bf16: with P rounded to bf16 within the bound, with v rounded once more to half its bits not."""
    g = torch.Generator().manual_seed(102)
    P, V = (torch.randn(64, 128, 128, generator=g, dtype=torch.float64) for _ in range(2))
    V = V.bfloat16().double()
    ref = P @ V
    assert bounds.relative((_parts(P, 1) @ V).bfloat16(), ref) < bounds.BF16_NORM
    assert bounds.relative((_parts(P, 1) @ V.to(torch.float8_e4m3fn).double()).bfloat16(), ref) > 4 * bounds.BF16_NORM
