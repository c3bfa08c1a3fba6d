"""Plain 64-bit linear attention (token by token, on the CPU) and inputs for its tests.

Bounds: every test compares element by element with ``rel * mag``, where mag is the same
recurrence on the absolute values of all inputs, i.e. the sum of the absolute values of the
terms that make up the element.  A path of n roundings to fp32 (half a step is 2^-24 of the
value; a tensor core's fp32 sums may truncate, 2^-23) is off by at most n 2^-23 of its term:
ROUNDINGS counts the longest path (sums over d <= 128 columns and <= 128 rows of a chunk,
states chained over segments, the three products of a split operand), so
F32 = 512 * 2^-23 = 2^-14.  A bf16 operand or output adds half a bf16 step, 2^-8, each.
"""
from __future__ import annotations

import torch

F32 = 2.0 ** -14
HALF_BF16 = 2.0 ** -8


def case(seed, lengths, H, Hk, dk, dv, dtype, decay="token", pads=0.0, state=True, la_scale=1.0):
    g = torch.Generator().manual_seed(seed)

    def normal(*shape):
        return torch.randn(shape, generator=g)

    dt = torch.bfloat16 if dtype == "bf16" else torch.float32
    N, B = sum(lengths), len(lengths)
    c = dict(lengths=list(lengths), H=H, Hk=Hk, dk=dk, dv=dv, dtype=dt)
    for name in ("q", "k"):
        x = normal(N, Hk, dk)
        c[name] = (x / x.norm(dim=-1, keepdim=True).clamp_min(1e-30)).to(dt)
    c["v"] = normal(N, H, dv).to(dt)
    c["log_alpha"] = -la_scale * torch.nn.functional.softplus(normal(*((H,) if decay == "head" else (N, H))) - 2.0)
    cu = [0]
    for n in lengths:
        cu.append(cu[-1] + n)
    c["cu_seqlens"] = torch.tensor(cu, dtype=torch.int32)
    c["pad_mask"] = (torch.rand(N, generator=g) >= pads).to(torch.uint8) if pads else None
    c["init_state"] = 0.1 * normal(B, H, dk, dv) if state else None
    c["grad_o"] = normal(N, H, dv).to(dt)
    c["grad_final_state"] = normal(B, H, dk, dv) if state else None
    return c


def spoil_pads(c, value=float("nan")):
    """Puts ``value`` into everything at the pads: nothing there may be read."""
    pad = c["pad_mask"] == 0
    for name in ("q", "k", "v", "grad_o"):
        c[name][pad] = value
    if c["log_alpha"].dim() == 2:
        c["log_alpha"][pad] = value
    return c


def to_cuda(c):
    return {k: v.cuda() if isinstance(v, torch.Tensor) else v for k, v in c.items()}


def _rows(c, mag):
    G = c["H"] // c["Hk"]
    real = torch.ones(c["q"].shape[0], dtype=torch.bool) if c["pad_mask"] is None else c["pad_mask"] != 0
    f = (lambda x: None if x is None else x.double().abs()) if mag else (lambda x: None if x is None else x.double())
    x = {}
    for name in ("q", "k", "v", "grad_o"):
        y = torch.where(real[:, None, None], f(c[name]), torch.zeros((), dtype=torch.float64))
        x[name] = y.repeat_interleave(G, dim=1) if name in ("q", "k") else y
    la = c["log_alpha"].double()
    la = la if la.dim() == 2 else la.expand(len(real), c["H"])
    x["a"] = torch.where(real[:, None], la, torch.zeros((), dtype=torch.float64)).exp()
    x["init"], x["final_grad"] = f(c["init_state"]), f(c["grad_final_state"])
    return x, real, G


def prefill(c, mag=False):
    """(o, final_state) in 64 bits; mag: of the absolute values."""
    x, _, _ = _rows(c, mag)
    o = torch.zeros(c["v"].shape, dtype=torch.float64)
    final = torch.zeros(len(c["lengths"]), c["H"], c["dk"], c["dv"], dtype=torch.float64)
    cu = c["cu_seqlens"].tolist()
    for b in range(len(c["lengths"])):
        S = final[b] if x["init"] is None else x["init"][b].clone()
        for t in range(cu[b], cu[b + 1]):
            S = x["a"][t][:, None, None] * S + x["k"][t][:, :, None] * x["v"][t][:, None, :]
            o[t] = torch.einsum("hk,hkv->hv", x["q"][t], S)
        final[b] = S
    return o, final


def backward(c, mag=False):
    """dict of 64-bit gradients; mag: the sums of the absolute values of their terms."""
    x, real, G = _rows(c, mag)
    N, H, Hk = c["q"].shape[0], c["H"], c["Hk"]
    out = dict(dq=torch.zeros(N, H, c["dk"], dtype=torch.float64), dk=torch.zeros(N, H, c["dk"], dtype=torch.float64),
               dv=torch.zeros(N, H, c["dv"], dtype=torch.float64), dlog_alpha=torch.zeros(N, H, dtype=torch.float64),
               dS0=torch.zeros(len(c["lengths"]), H, c["dk"], c["dv"], dtype=torch.float64))
    cu = c["cu_seqlens"].tolist()
    for b in range(len(c["lengths"])):
        S = out["dS0"][b].clone() if x["init"] is None else x["init"][b]
        states = [S]
        for t in range(cu[b], cu[b + 1]):
            S = x["a"][t][:, None, None] * S + x["k"][t][:, :, None] * x["v"][t][:, None, :]
            states.append(S)
        D = torch.zeros_like(S) if x["final_grad"] is None else x["final_grad"][b].clone()
        for t in reversed(range(cu[b], cu[b + 1])):
            S, before, a = states.pop(), states[-1], x["a"][t][:, None, None]
            D = D + x["q"][t][:, :, None] * x["grad_o"][t][:, None, :]
            out["dq"][t] = torch.einsum("hkv,hv->hk", S, x["grad_o"][t])
            out["dk"][t] = torch.einsum("hkv,hv->hk", D, x["v"][t])
            out["dv"][t] = torch.einsum("hkv,hk->hv", D, x["k"][t])
            out["dlog_alpha"][t] = (a * before * D).sum((1, 2))
            D = a * D
        out["dS0"][b] = D
    for name in ("dq", "dk", "dv", "dlog_alpha"):
        out[name][~real] = 0.0
    for name in ("dq", "dk"):
        out[name] = out[name].reshape(N, Hk, G, -1).sum(2)
    if c["log_alpha"].dim() == 1:
        out["dlog_alpha"] = out["dlog_alpha"].sum(0)
    return out


def check(name, got, ref, mag, bf16_roundings, out_bf16):
    """|got - ref| <= F32 mag + bf16_roundings 2^-8 mag (+ 2^-8 |ref| for a bf16 output)."""
    got = got.detach().cpu().double()
    bound = (F32 + bf16_roundings * HALF_BF16) * mag + 1e-30
    if out_bf16:
        bound = bound + HALF_BF16 * (ref.abs() + bound)
    off = (got - ref).abs()
    assert torch.isfinite(got).all(), name
    assert (off <= bound).all(), f"{name}: {(off / bound).max().item():.3g} of the bound"
