"""CPU checks of the workspaces that the binding makes or takes for the linear-attention and norm calls."""
import pytest
import torch

from gated_delta_rule_148_b200 import kda


def _norm_backward(rows, D, eps):
    a = kda.RmsNormBackwardArgs()
    a.dtype, a.rows, a.D, a.eps = kda.KDA_BF16, rows, D, eps
    return a


def test_a_refused_call_leaves_no_workspace_size_behind():
    """eps is no size, so a call with a bad one shares its sizes with the good ones that follow."""
    sizes, like = (kda.KDA_BF16, 37, 264), torch.zeros(1)
    kda._workspace(_norm_backward(37, 264, -1.0), "kda_rms_norm_backward", sizes, None, like)
    a = _norm_backward(37, 264, 1e-6)
    ws = kda._workspace(a, "kda_rms_norm_backward", sizes, None, like)
    assert ws.numel() == a.workspace_bytes == 37 * 264 * 4


def test_workspace_size_does_not_depend_on_eps():
    lib = kda.load()
    assert lib.kda_rms_norm_backward_workspace_size(_norm_backward(37, 264, float("nan"))) == 37 * 264 * 4
    assert lib.kda_rms_norm_backward_workspace_size(_norm_backward(-1, 264, 1e-6)) == 0
    assert lib.kda_rms_norm_backward_workspace_size(_norm_backward(37, 12, 1e-6)) == 0


@pytest.mark.parametrize("workspace", [torch.zeros(4096, dtype=torch.uint8)[::2], torch.zeros(1, dtype=torch.uint8).expand(1 << 20),
                                       torch.zeros(64, 64, dtype=torch.uint8).t()], ids=["strided", "expanded", "transposed"])
def test_a_workspace_must_be_contiguous(workspace):
    """Its elements' count is taken for the bytes behind its address: an expanded one has fewer, a strided one other owners."""
    with pytest.raises(ValueError):
        kda._workspace(_norm_backward(4, 64, 1e-6), "kda_rms_norm_backward", (kda.KDA_BF16, 4, 64), workspace, torch.zeros(1))


def test_a_workspace_of_another_type_counts_its_bytes():
    a = _norm_backward(4, 64, 1e-6)
    assert kda._workspace(a, "kda_rms_norm_backward", (kda.KDA_BF16, 4, 64), torch.zeros(256), torch.zeros(1)).numel() == 256
    assert a.workspace_bytes == 1024
