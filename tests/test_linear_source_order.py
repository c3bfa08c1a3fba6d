"""CPU checks of the order in which the linear-attention kernels touch what their warps share, read off the
source: orders that hold by timing alone never show in a result."""
import os
import re

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "gated_delta_rule_148_b200", "csrc")


def _source(name):
    with open(os.path.join(CSRC, name)) as f:
        return re.sub(r"//[^\n]*", "", f.read())


def _in_order(text, *what):
    """Every one of ``what`` is in ``text``, each (its first occurrence from there) behind the one before."""
    at = 0
    for w in what:
        i = text.find(w, at)
        if i < 0:
            return False
        at = i + len(w)
    return True


def test_a_next_items_product_waits_for_the_row_sums_in_its_place():
    """Gradients in bf16: the row sums q.E and k.F pass through columns of A's accumulator.  Stored, read by the third
    warpgroup, told by tab_free, which the next item's A = K Q^T waits for."""
    src = _source("kda_linear_backward_tc.cu")
    grad = src[src.index("grad_kernel(LinearParams p"):]
    products = grad[grad.index("if (warp == 16) {", grad.index("if (warp == 17) {")):grad.index("if (warp == 18) {")]
    groups = grad[grad.index("if (warp == 18) {"):grad.index("// ======") if "// ======" in grad else len(grad)]
    assert _in_order(groups, "tmem_st1(tm + lanes + T_A + 16 + y", "tmem_st_wait();", "fence_before_sync();", "mbar_arrive(summed);")
    assert _in_order(groups, "wait.warp(summed, it", "fence_after_sync();", "tmem_ld2(tm + lanes + T_A + 16", "fence_before_sync();",
                     "mbar_arrive(tab_free);")
    assert groups.count("mbar_arrive(tab_free);") == 1 and groups.count("tmem_ld2(") == 1
    before = products[:products.index("mma_bf16(tm + T_A,")]
    assert _in_order(before, "if (it > 0) ok = wait(tab_free, it - 1", "if (!ok) break;", "fence_after_sync();")


KERNELS = ("kda_linear.cu", "kda_linear_tc.cu", "kda_linear_backward_tc.cu", "kda_linear_decode.cu", "kda_norm.cu")


def _kernel_starts(src):
    """(name, body up to the first return) of each kernel."""
    for m in re.finditer(r"__global__ void(?:\s+__launch_bounds__\((?:[^()]|\([^()]*\))*\))?\s+(\w+)\(", src):
        body = src[src.index("{", m.end()) + 1:]
        yield m.group(1), body[:body.index("return;")]


def test_a_block_leaves_with_all_its_threads_or_none():
    """On a latched error a kernel's threads leave together: the word may change between two warps' looks at it."""
    assert "return __syncthreads_or(device_error_latched(err));" in _source("kda_internal.cuh")
    assert "return __syncthreads_or(device_error_latched(p.err) | " in _source("kda_linear.cuh")
    for name in KERNELS:
        src = _source(name)
        assert src.count("device_error_latched(") == src.count("__syncthreads_or(stop || device_error_latched("), name
        kernels = list(_kernel_starts(src))
        assert len(kernels) == src.count("__global__"), name
        for kernel, start in kernels:
            # its first return, before any of its threads goes a way of its own
            assert re.search(r"if \((block_leaves\((p\.)?err\)|(lin::)?call_ended\(p, sbase\))\) $", start) or \
                re.search(r"if \(__syncthreads_or\(\w+ \|\| device_error_latched\(p\.err\)\)\) \{[^}]*\}\s*$", start), (name, kernel)
            assert not re.search(r"if \((warp|w|lane)\b", start), (name, kernel)


def test_the_delta_rule_s_kernels_leave_in_whole_blocks_too():
    for name in sorted(os.listdir(CSRC)):
        if name.endswith(".cu") and name not in KERNELS:
            assert "device_error_latched(" not in _source(name), name
    # after the state's loads, before any store
    src = _source("kda_decode.cu")
    assert _in_order(src, "__ldcs(", "if (block_leaves(p.err)) return;", "__stcs(", "store_elem")


def test_kernels_behind_a_plan_look_at_the_call_s_own_word():
    """cu_seqlens that a plan refuses: its tables are not to be read, whoever clears the library's error word meanwhile."""
    for name in KERNELS[:3]:
        src = _source(name)
        for kernel, start in _kernel_starts(src):
            if kernel == "plan_kernel":
                plan = src[src.index("plan_kernel(LinearParams p"):]
                assert _in_order(plan, "device_error_latched(", "sbase[p.num_seqs] = kRefused;", "return;", "if (bad) {",
                                 "sbase[p.num_seqs] = kRefused;", "return;")
            else:
                assert "call_ended(p, sbase)) " in start, (name, kernel)
