"""CPU checks of the linear-attention and RMS-norm entry points: struct layouts, workspace sizes and
host-side refusals (every refused call returns before the first CUDA call; addresses are never used)."""
import ctypes
import os
import subprocess

import pytest
import torch

from gated_delta_rule_148_b200 import kda

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
BASE = 0x7F0000000000
STRUCTS = {"kda_linear_args": kda.LinearArgs, "kda_linear_decode_args": kda.LinearDecodeArgs,
           "kda_linear_backward_args": kda.LinearBackwardArgs, "kda_rms_norm_args": kda.RmsNormArgs,
           "kda_rms_norm_backward_args": kda.RmsNormBackwardArgs}


def test_struct_layouts_match_the_header(tmp_path):
    lines = ['#include <stdio.h>', '#include <stddef.h>', '#include "kda.h"', 'int main(void){']
    for name, cls in STRUCTS.items():
        lines.append(f'printf("{name} %zu\\n", sizeof({name}));')
        lines += [f'printf("{name}.{f} %zu\\n", offsetof({name}, {f}));' for f, _ in cls._fields_]
    (tmp_path / "layout.c").write_text("\n".join(lines + ["return 0;}"]))
    exe = tmp_path / "layout"
    subprocess.check_call(["gcc", "-std=c99", "-I", os.path.join(ROOT, "include"), str(tmp_path / "layout.c"), "-o", str(exe)])
    got = dict(line.split() for line in subprocess.check_output([str(exe)], text=True).splitlines())
    for name, cls in STRUCTS.items():
        assert int(got[name]) == ctypes.sizeof(cls)
        for f, _ in cls._fields_:
            assert int(got[f"{name}.{f}"]) == getattr(cls, f).offset, (name, f)


def _spread(a, names, at=BASE):
    for i, name in enumerate(names):
        setattr(a, name, at + i * 0x10000000)
    return a


def _prefill():
    a = kda.LinearArgs()
    a.dtype, a.num_seqs, a.total_tokens, a.H, a.Hk, a.dk, a.dv = kda.KDA_BF16, 2, 256, 4, 2, 64, 128
    _spread(a, ("q", "k", "v", "log_alpha", "cu_seqlens", "init_state", "o", "final_state", "workspace"))
    a.workspace_bytes = kda.load().kda_linear_prefill_workspace_size(ctypes.byref(a))
    return a


def _backward():
    a = kda.LinearBackwardArgs()
    a.dtype, a.num_seqs, a.total_tokens, a.H, a.Hk, a.dk, a.dv = kda.KDA_BF16, 2, 256, 4, 2, 64, 128
    _spread(a, ("q", "k", "v", "log_alpha", "cu_seqlens", "init_state", "grad_o", "grad_final_state", "grad_q", "grad_k",
                "grad_v", "grad_log_alpha", "grad_init_state", "workspace"))
    a.workspace_bytes = kda.load().kda_linear_prefill_backward_workspace_size(ctypes.byref(a))
    return a


def _decode():
    a = kda.LinearDecodeArgs()
    a.dtype, a.B, a.H, a.Hk, a.dk, a.dv = kda.KDA_BF16, 8, 4, 2, 64, 128
    return _spread(a, ("q", "k", "v", "log_alpha", "mask", "state", "o"))


def _norm():
    a = kda.RmsNormArgs()
    a.dtype, a.out_dtype, a.rows, a.D, a.eps, a.group = kda.KDA_BF16, kda.KDA_E4M3, 16, 256, 1e-6, 128
    return _spread(a, ("x", "residual", "weight", "y", "scale", "residual_out"))


def _norm_backward():
    a = kda.RmsNormBackwardArgs()
    a.dtype, a.rows, a.D, a.eps = kda.KDA_BF16, 16, 256, 1e-6
    _spread(a, ("x", "weight", "grad_y", "grad_residual", "grad_x", "grad_weight", "workspace"))
    a.workspace_bytes = kda.load().kda_rms_norm_backward_workspace_size(ctypes.byref(a))
    return a


CALLS = {"kda_linear_prefill": _prefill, "kda_linear_prefill_backward": _backward, "kda_linear_decode": _decode,
         "kda_rms_norm": _norm, "kda_rms_norm_backward": _norm_backward}
INVALID, UNSUPPORTED = kda.KDA_ERR_INVALID_ARG, kda.KDA_ERR_UNSUPPORTED
LINEAR = ("kda_linear_prefill", "kda_linear_prefill_backward", "kda_linear_decode")
REFUSED = [(f, {"dtype": kda.KDA_E4M3}, INVALID) for f in CALLS]
REFUSED += [(f, m, s) for f in LINEAR for m, s in (
    ({"H": 0}, INVALID), ({"Hk": 0}, INVALID), ({"Hk": 3}, INVALID), ({"Hk": 8}, INVALID), ({"dk": 96}, UNSUPPORTED),
    ({"dv": 256}, UNSUPPORTED), ({"dv": 0}, INVALID), ({"decay": 2}, INVALID), ({"q": None}, INVALID), ({"v": None}, INVALID),
    ({"log_alpha": None}, INVALID), ({"log_alpha": BASE + 0x30000002}, INVALID))]
REFUSED += [(f, m, INVALID) for f in LINEAR[:2] for m in (
    {"num_seqs": -1}, {"total_tokens": -1}, {"num_seqs": 0}, {"cu_seqlens": None}, {"cu_seqlens": BASE + 0x40000002},
    {"k": BASE + 0x10000008}, {"v": BASE + 0x20000002}, {"workspace": None}, {"workspace": BASE + 0x80000010}, {"workspace_bytes": 8},
    {"init_state": BASE + 0x50000004})]
REFUSED += [("kda_linear_prefill", m, INVALID) for m in (
    {"o": None}, {"o": BASE + 16}, {"o": BASE + 0x20000000}, {"o": BASE + 0x30000000}, {"final_state": BASE + 0x50000010},
    {"final_state": BASE + 0x60000000}, {"workspace": BASE + 0x60000000}, {"pad_mask": BASE + 0x60000010})]
REFUSED += [("kda_linear_prefill_backward", m, INVALID) for m in (
    {"grad_o": None}, {"grad_q": None}, {"grad_k": None}, {"grad_v": None}, {"grad_log_alpha": None}, {"grad_o": BASE + 0x60000008},
    {"grad_q": BASE}, {"grad_k": BASE + 0x80000000}, {"grad_v": BASE + 0x60000000}, {"grad_log_alpha": BASE + 0x30000000},
    {"grad_init_state": BASE + 0x70000000}, {"grad_init_state": BASE + 0x50000000})]
REFUSED += [("kda_linear_decode", m, INVALID) for m in (
    {"B": -1}, {"state": None}, {"state": BASE + 0x50000004}, {"o": None}, {"o": BASE + 0x50000000}, {"o": BASE + 2}, {"state": BASE},
    {"mask": BASE + 0x50000000})]
REFUSED += [("kda_rms_norm", m, s) for m, s in (
    ({"rows": -1}, INVALID), ({"rows": 1 << 31}, UNSUPPORTED), ({"D": 12}, INVALID), ({"D": 0}, INVALID), ({"D": 16392}, UNSUPPORTED),
    ({"eps": -1.0}, INVALID), ({"eps": float("nan")}, INVALID), ({"eps": float("inf")}, INVALID), ({"out_dtype": kda.KDA_F32}, INVALID),
    ({"out_dtype": 9}, INVALID), ({"group": 48}, UNSUPPORTED), ({"group": -32}, UNSUPPORTED), ({"scale": None}, INVALID),
    ({"out_dtype": kda.KDA_BF16}, INVALID), ({"out_dtype": kda.KDA_BF16, "group": 0}, INVALID), ({"residual": None}, INVALID),
    ({"x": None}, INVALID), ({"y": None}, INVALID), ({"x": BASE + 8}, INVALID), ({"weight": BASE + 0x20000004}, INVALID),
    ({"y": BASE}, INVALID), ({"scale": BASE + 0x30000000}, INVALID), ({"residual_out": BASE}, INVALID),
    ({"residual_out": BASE + 0x10000010}, INVALID), ({"scale": BASE + 0x20000000}, INVALID))]
REFUSED += [("kda_rms_norm_backward", m, s) for m, s in (
    ({"rows": -1}, INVALID), ({"D": 4}, INVALID), ({"D": 20000}, UNSUPPORTED), ({"x": None}, INVALID), ({"grad_y": None}, INVALID),
    ({"grad_x": None}, INVALID), ({"workspace": None}, INVALID), ({"workspace_bytes": 100}, INVALID),
    ({"workspace": BASE + 0x60000040}, INVALID), ({"grad_x": BASE}, INVALID), ({"grad_x": BASE + 0x30000010}, INVALID),
    ({"grad_weight": BASE + 0x10000000}, INVALID), ({"grad_y": BASE + 0x20000008}, INVALID))]


@pytest.mark.parametrize("call,change,status", REFUSED, ids=lambda x: str(x) if not callable(x) else "")
def test_refusals(call, change, status):
    a = CALLS[call]()
    for name, value in change.items():
        setattr(a, name, value)
    assert getattr(kda.load(), call)(ctypes.byref(a), None) == status


def test_null_and_empty_calls():
    lib = kda.load()
    for call in CALLS:
        assert getattr(lib, call)(None, None) == INVALID
    a = _prefill()
    a.num_seqs = a.total_tokens = 0
    assert lib.kda_linear_prefill(ctypes.byref(a), None) == kda.KDA_OK
    a = _backward()
    a.num_seqs = a.total_tokens = 0
    assert lib.kda_linear_prefill_backward(ctypes.byref(a), None) == kda.KDA_OK
    a = _decode()
    a.B = 0
    assert lib.kda_linear_decode(ctypes.byref(a), None) == kda.KDA_OK
    a = _norm()
    a.rows = 0
    assert lib.kda_rms_norm(ctypes.byref(a), None) == kda.KDA_OK


def test_workspace_sizes():
    lib = kda.load()
    for size, make in (("kda_linear_prefill_workspace_size", _prefill), ("kda_linear_prefill_backward_workspace_size", _backward),
                       ("kda_rms_norm_backward_workspace_size", _norm_backward)):
        assert getattr(lib, size)(None) == 0
        a = make()
        assert getattr(lib, size)(ctypes.byref(a)) > 0
        a.dtype = 9
        assert getattr(lib, size)(ctypes.byref(a)) == 0
    # the states are few: below a fifth of the inputs' bytes for a long prompt
    a = _prefill()
    a.num_seqs, a.total_tokens, a.H, a.Hk, a.dk, a.dv = 1, 131072, 32, 32, 128, 128
    assert lib.kda_linear_prefill_workspace_size(ctypes.byref(a)) < 131072 * 32 * 128 * 2 * 3 // 5


def test_binding_refuses_what_it_cannot_take():
    x = torch.zeros(4, 2, 64)
    cu = torch.tensor([0, 4], dtype=torch.int32)
    with pytest.raises(TypeError):
        kda.linear_prefill(x, x, x, torch.zeros(4, 2), cu)
    with pytest.raises(TypeError):
        kda.linear_decode(x, x, x, torch.zeros(4, 2), torch.zeros(4, 2, 64, 64))
    with pytest.raises(TypeError):
        kda.linear_prefill_backward(x, x, x, torch.zeros(4, 2), cu, x)
    with pytest.raises(ValueError):
        kda.linear_prefill(x, x, torch.zeros(4, 3, 64), torch.zeros(4, 3), cu)       # 3 value heads on 2
    with pytest.raises(ValueError):
        kda.linear_prefill(x[0], x[0], x[0], torch.zeros(2), cu)
    with pytest.raises(TypeError):
        kda.rms_norm(torch.zeros(4, 64))
    with pytest.raises(TypeError):
        kda.rms_norm_quant(torch.zeros(4, 64))
    with pytest.raises(ValueError):
        kda.rms_norm_quant(torch.zeros(4, 64), quant="e5m2")
    with pytest.raises(TypeError):
        kda.rms_norm_backward(torch.zeros(4, 64), None, torch.zeros(4, 64))
