"""GPU parity of linear attention (prefill, decode, backward) against the plain 64-bit
recurrence; bounds by counted roundings (linear_testlib)."""
import pytest
import torch

import linear_testlib as lib
from gated_delta_rule_148_b200 import kda

pytestmark = pytest.mark.gpu

# roundings of operands to bf16 on the longest path of a bf16 call (o and gradients: the pair
# weight or the state; fp32 outputs of a bf16 call: none)
BF16_OPERANDS = 1


def _prefill(c, **kw):
    d = lib.to_cuda(c)
    o, s = kda.linear_prefill(d["q"], d["k"], d["v"], d["log_alpha"], d["cu_seqlens"], pad_mask=d["pad_mask"],
                              init_state=d["init_state"], **kw)
    assert kda.get_device_status() == kda.KDA_OK
    return o, s


def _check_prefill(c):
    o, s = _prefill(c)
    (ro, rs), (mo, ms) = lib.prefill(c), lib.prefill(c, mag=True)
    bf16 = c["dtype"] == torch.bfloat16
    lib.check("o", o, ro, mo, BF16_OPERANDS if bf16 else 0, bf16)
    lib.check("final_state", s, rs, ms, 0, False)
    return o, s


def _backward(c, **kw):
    d = lib.to_cuda(c)
    g = kda.linear_prefill_backward(d["q"], d["k"], d["v"], d["log_alpha"], d["cu_seqlens"], d["grad_o"],
                                    grad_final_state=d["grad_final_state"], pad_mask=d["pad_mask"],
                                    init_state=d["init_state"], **kw)
    assert kda.get_device_status() == kda.KDA_OK
    return g


def _check_backward(c):
    g, ref, mag = _backward(c), lib.backward(c), lib.backward(c, mag=True)
    bf16 = c["dtype"] == torch.bfloat16
    for name in ("dq", "dk", "dv"):
        lib.check(name, g[name], ref[name], mag[name], BF16_OPERANDS if bf16 else 0, bf16)
    for name in ("dlog_alpha", "dS0"):
        lib.check(name, g[name], ref[name], mag[name], 0, False)
    return g


LENGTHS = [[1], [63, 64, 65], [0, 1, 129, 0, 255, 2]]


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("dk,dv", [(64, 64), (64, 128), (128, 64), (128, 128)])
@pytest.mark.parametrize("lengths", LENGTHS, ids=str)
def test_prefill_and_backward_shapes(dtype, dk, dv, lengths):
    c = lib.case(1, lengths, 2, 2, dk, dv, dtype)
    _check_prefill(c)
    _check_backward(c)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("decay", ["token", "head"])
@pytest.mark.parametrize("H,Hk", [(1, 1), (6, 2), (4, 1)])
def test_shared_heads_pads_and_decay_layouts(dtype, decay, H, Hk):
    c = lib.spoil_pads(lib.case(2, [70, 200], H, Hk, 128, 64, dtype, decay=decay, pads=0.2))
    o, _ = _check_prefill(c)
    g = _check_backward(c)
    pad = (c["pad_mask"] == 0).cuda()
    assert torch.all(o[pad] == 0)
    for name in ("dq", "dk", "dv") + (("dlog_alpha",) if decay == "token" else ()):
        assert torch.all(g[name][pad] == 0), name


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_without_states(dtype):
    c = lib.case(3, [50, 300], 2, 1, 64, 128, dtype, state=False)
    _check_prefill(c)
    _check_backward(c)
    o, s = _prefill(c, want_final_state=False)
    assert s is None
    assert torch.equal(o, _prefill(c)[0])
    assert _backward(c, want_grad_init_state=False)["dS0"] is None


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_all_pads_and_only_empty_sequences(dtype):
    c = lib.case(4, [5, 130, 0], 2, 2, 64, 64, dtype, pads=0.5)
    c["pad_mask"].zero_()
    lib.spoil_pads(c)
    o, s = _prefill(c)
    assert torch.all(o == 0) and torch.equal(s.cpu(), c["init_state"])
    g = _backward(c)
    assert all(torch.all(g[n] == 0) for n in ("dq", "dk", "dv", "dlog_alpha"))
    assert torch.equal(g["dS0"].cpu(), c["grad_final_state"])
    c = lib.case(5, [0, 0], 2, 2, 64, 64, dtype)
    o, s = _prefill(c)
    assert o.shape == (0, 2, 64) and torch.equal(s.cpu(), c["init_state"])
    c = lib.case(5, [0, 0], 2, 2, 64, 64, dtype, decay="head")
    g = _backward(c)
    assert torch.equal(g["dS0"].cpu(), c["grad_final_state"]) and torch.all(g["dlog_alpha"] == 0)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_strong_and_absent_decays(dtype):
    """Resets (a = 0 in fp32) between weak decays: the digits of the weak ones must survive."""
    c = lib.case(6, [300, 90], 2, 2, 128, 128, dtype)
    for t, x in ((10, -1e30), (11, -200.0), (75, -3e38), (200, -104.0), (310, -1000.0)):
        c["log_alpha"][t] = x
    c["log_alpha"][100:120] = 0.0
    _check_prefill(c)
    _check_backward(c)
    c = lib.case(7, [400], 2, 2, 64, 64, dtype, la_scale=100.0)
    _check_prefill(c)
    _check_backward(c)
    c = lib.case(8, [400], 2, 2, 64, 64, dtype)
    c["log_alpha"].zero_()
    _check_prefill(c)
    _check_backward(c)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("H,lengths", [(2, [2500, 3, 1700]), (32, [1100, 517])], ids=["few_heads", "many_heads"])
def test_longer_sequences(dtype, H, lengths):
    c = lib.case(9, lengths, H, max(1, H // 4), 128, 128, dtype, pads=0.02)
    _check_prefill(c)
    c = lib.case(9, [x // 2 for x in lengths], H, max(1, H // 4), 128, 128, dtype, pads=0.02)
    _check_backward(c)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_state_in_place_same_bits_and_split_continuation(dtype):
    """final_state over init_state; the same call twice; a prompt in two calls."""
    c = lib.case(10, [333], 3, 3, 128, 128, dtype)
    o, s = _prefill(c)
    d = lib.to_cuda(c)
    o2, s2 = kda.linear_prefill(d["q"], d["k"], d["v"], d["log_alpha"], d["cu_seqlens"], init_state=d["init_state"],
                                final_state=d["init_state"])
    assert s2 is d["init_state"] and torch.equal(o, o2) and torch.equal(s, s2)
    g1, g2 = _backward(c), _backward(c)
    assert all(torch.equal(g1[n], g2[n]) for n in g1)
    state, parts = lib.to_cuda(c)["init_state"], []
    for a, b in ((0, 150), (150, 333)):
        cu = torch.tensor([0, b - a], dtype=torch.int32, device="cuda")
        y, state = kda.linear_prefill(*(d[n][a:b] for n in ("q", "k", "v", "log_alpha")), cu, init_state=state)
        parts.append(y)
    (ro, rs), (mo, ms) = lib.prefill(c), lib.prefill(c, mag=True)
    bf16 = dtype == "bf16"
    lib.check("o", torch.cat(parts), ro, mo, BF16_OPERANDS if bf16 else 0, bf16)
    lib.check("state", state, rs, ms, 0, False)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("dk,dv", [(64, 64), (64, 128), (128, 64), (128, 128)])
@pytest.mark.parametrize("rows,H,Hk", [(1, 3, 1), (2, 40, 8), (70, 6, 6)])
def test_decode(dtype, dk, dv, rows, H, Hk):
    state = None
    for step, decay in enumerate(("token", "head", "token")):
        c = lib.case(20 + step, [1] * rows, H, Hk, dk, dv, dtype, decay=decay, pads=0.3)
        if state is None:
            state = c["init_state"].cuda()
        c["init_state"] = state.cpu()
        mask = c["pad_mask"]
        lib.spoil_pads(c)
        d, before = lib.to_cuda(c), state.clone()
        o = kda.linear_decode(d["q"], d["k"], d["v"], d["log_alpha"], state, mask=d["pad_mask"])
        assert kda.get_device_status() == kda.KDA_OK
        (ro, rs), (mo, ms) = lib.prefill(c), lib.prefill(c, mag=True)
        lib.check("o", o, ro, mo, 0, dtype == "bf16")
        lib.check("state", state, rs, ms, 0, False)
        off = (mask == 0).cuda()
        assert torch.equal(state[off], before[off]) and torch.all(o[off] == 0)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_prompt_then_steps_between_norms(dtype):
    """The operators as a block uses them: residual and norm, prompt, norm per head, then single tokens."""
    H, d, T, steps, D = 4, 64, 150, 4, 256
    c = lib.case(30, [T + steps] * 2, H, 2, d, d, dtype, state=False)
    dev = lib.to_cuda(c)
    g = torch.Generator().manual_seed(31)
    x, res = (torch.randn(2 * (T + steps), D, generator=g).to(c["dtype"]).cuda() for _ in range(2))
    w = (1 + 0.1 * torch.randn(D, generator=g)).cuda()
    y, r = kda.rms_norm(x, w, residual=res)
    rr = (x.double() + res.double()).to(c["dtype"])
    ref = rr.double() * torch.rsqrt(rr.double().square().mean(1, keepdim=True) + 1e-6) * w.double()
    step = lib.HALF_BF16 if dtype == "bf16" else 0.0
    assert torch.equal(r, rr) and ((y.double() - ref).abs() <= (step + 2.0 ** -18) * ref.abs() + 1e-30).all()
    c["v"] = y.reshape(-1, H, d).cpu()          # the block's values come from the normed input
    v = y.reshape(-1, H, d)
    first = torch.cat([torch.arange(T), torch.arange(T + steps, 2 * T + steps)]).cuda()
    cu = torch.tensor([0, T, 2 * T], dtype=torch.int32, device="cuda")
    o, state = kda.linear_prefill(*(a[first].contiguous() for a in (dev["q"], dev["k"], v, dev["log_alpha"])), cu)
    outs = torch.zeros(2 * (T + steps), H, d, dtype=c["dtype"], device="cuda")
    outs[first] = o
    for s in range(steps):
        rows = torch.tensor([T + s, 2 * T + steps + s], device="cuda")
        outs[rows] = kda.linear_decode(*(a[rows].contiguous() for a in (dev["q"], dev["k"], v, dev["log_alpha"])), state)
    (ro, rs), (mo, ms) = lib.prefill(c), lib.prefill(c, mag=True)
    lib.check("o", outs, ro, mo, BF16_OPERANDS if dtype == "bf16" else 0, dtype == "bf16")
    lib.check("state", state, rs, ms, 0, False)
    y8, scale, none = kda.rms_norm_quant(outs, torch.ones(d, device="cuda"), group=64)
    f = outs.double()
    n = f * torch.rsqrt(f.square().mean(-1, keepdim=True) + 1e-6)
    assert none is None and y8.shape == outs.shape and scale.shape == (2 * (T + steps), H, 1)
    top = n.abs().amax(-1, keepdim=True)
    # e4m3: half a step of 2^-3 (values down to 2^-6 of 448 ulps of the scale), fp32 arithmetic before it
    assert ((y8.double() * scale.double() - n).abs() <= 2.0 ** -4 * n.abs() + 2.0 ** -9 * top / 448 + 2.0 ** -18 * top).all()
    assert kda.get_device_status() == kda.KDA_OK


def test_gradient_against_differences():
    """fp32: o and the state are linear in q (at fixed k, v), in k and in v, so central differences are
    exact up to rounding; in log_alpha they are off by h^2/6 of the third derivative, which is at
    most the sum over pairs of (distance)^3-weighted terms: with h = 2^-8 along a unit-size
    direction over <= 40 tokens, (40 h)^2 / 6 of the sum of absolute terms."""
    for decay in ("token", "head"):
        c = lib.case(40, [40, 23], 2, 1, 64, 64, "f32", decay=decay)
        g = lib.to_cuda(_to_cpu(_backward(c)))
        mag = lib.backward(c, mag=True)

        def loss(c):
            o, s = _prefill(c)
            return (o.double().cpu() * c["grad_o"].double()).sum() + (s.double().cpu() * c["grad_final_state"].double()).sum()

        mo, ms = lib.prefill(c, mag=True)
        total = (mo * c["grad_o"].abs()).sum() + (ms * c["grad_final_state"].abs()).sum()
        for name, key, h in (("q", "dq", 1.0), ("k", "dk", 1.0), ("v", "dv", 1.0), ("log_alpha", "dlog_alpha", 2.0 ** -8),
                             ("init_state", "dS0", 1.0)):
            gen = torch.Generator().manual_seed(41)
            u = torch.rand(c[name].shape, generator=gen) - 0.5
            if name == "log_alpha":
                u = u * 2
            lo, hi = dict(c), dict(c)
            lo[name], hi[name] = c[name] - h * u, c[name] + h * u
            diff = (loss(hi) - loss(lo)) / (2 * h)
            have = (g[key].cpu().double() * u.double()).sum()
            size = (mag[key] * u.double().abs()).sum()
            bound = lib.F32 * size + lib.F32 * (total + h * size) / h
            if name == "log_alpha":
                bound = bound + (40 * h) ** 2 / 6 * 40 * size
            assert abs(diff - have) <= bound, (decay, name, abs(diff - have) / bound)


def _to_cpu(g):
    return {k: None if v is None else v.cpu() for k, v in g.items()}


def test_captured_calls_on_two_streams():
    """Two captured prefills and backwards with workspaces of their own, replayed at the same time on two
    streams, and an eager call between: the bits of the eager calls."""
    cs = [lib.case(50 + i, [300, 40], 2, 1, 128, 128, "bf16", pads=0.1) for i in range(2)]
    want = [(_prefill(c), _backward(c)) for c in cs]
    graphs = []
    for c in cs:
        d = lib.to_cuda(c)
        o, s = torch.empty_like(d["v"]), torch.empty_like(d["init_state"])
        ws = kda.linear_prefill_workspace(340, 2, 2, 1, 128, 128)
        stream, graph, hold = torch.cuda.Stream(), torch.cuda.CUDAGraph(), {}
        stream.wait_stream(torch.cuda.current_stream())
        with torch.cuda.graph(graph, stream=stream):
            kda.linear_prefill(d["q"], d["k"], d["v"], d["log_alpha"], d["cu_seqlens"], pad_mask=d["pad_mask"],
                               init_state=d["init_state"], o=o, final_state=s, workspace=ws)
            hold = kda.linear_prefill_backward(d["q"], d["k"], d["v"], d["log_alpha"], d["cu_seqlens"], d["grad_o"],
                                               grad_final_state=d["grad_final_state"], pad_mask=d["pad_mask"],
                                               init_state=d["init_state"])
        graphs.append((graph, stream, o, s, hold, d, ws))
    for _ in range(3):
        for graph, stream, *_ in graphs:
            stream.wait_stream(torch.cuda.current_stream())
            with torch.cuda.stream(stream):
                graph.replay()
        eager = _prefill(cs[0])
        for graph, stream, *_ in graphs:
            torch.cuda.current_stream().wait_stream(stream)
        torch.cuda.synchronize()
        assert torch.equal(eager[0], want[0][0][0])
        for ((o, s), g), (_, _, go, gs, hold, *_) in zip(want, graphs):
            assert torch.equal(o, go) and torch.equal(s, gs)
            assert all(torch.equal(g[n], hold[n]) for n in g)
            go.zero_()
    assert kda.get_device_status() == kda.KDA_OK


def test_invalid_cu_seqlens_is_latched_and_writes_nothing():
    c = lib.to_cuda(lib.case(60, [30, 40], 2, 2, 64, 64, "bf16"))
    o, s = torch.full_like(c["v"], 7.0), torch.full_like(c["init_state"], 7.0)
    for bad in ([0, 30, 71], [1, 30, 70], [0, 40, 30], [0, -1, 70]):
        cu = torch.tensor(bad, dtype=torch.int32, device="cuda")
        kda.linear_prefill(c["q"], c["k"], c["v"], c["log_alpha"], cu, o=o, final_state=s)
        assert kda.get_device_status() == kda.KDA_ERR_DEVICE_CHECK
        assert torch.all(o == 7) and torch.all(s == 7)
        kda.linear_prefill_backward(c["q"], c["k"], c["v"], c["log_alpha"], cu, c["grad_o"])
        assert kda.get_device_status() == kda.KDA_ERR_DEVICE_CHECK
    assert kda.get_device_status() == kda.KDA_OK


def test_offsets_past_31_bits():
    """136 value heads on one query/key head, 131072 + 77 tokens: 2.3e9 elements of v and o.  A reset 150 tokens before
    the end cuts the past off, so the end equals a call on those tokens alone."""
    N, H, d, tail = 131072 + 77, 136, 128, 150
    g = torch.Generator(device="cuda").manual_seed(70)
    q, k = (torch.nn.functional.normalize(torch.randn(N, 1, d, generator=g, device="cuda"), dim=-1).bfloat16() for _ in range(2))
    v = torch.randn(1024, H, d, generator=g, device="cuda").bfloat16().repeat(N // 1024 + 1, 1, 1)[:N].contiguous()
    la = -torch.rand(N, H, generator=g, device="cuda") * 0.2
    la[N - tail] = -1000.0
    o, s = kda.linear_prefill(q, k, v, la, torch.tensor([0, N], dtype=torch.int32, device="cuda"))
    last = [x[N - tail:].contiguous() for x in (q, k, v, la)]
    o2, s2 = kda.linear_prefill(*last, torch.tensor([0, tail], dtype=torch.int32, device="cuda"))
    assert kda.get_device_status() == kda.KDA_OK
    # both are within the bound of the same exact values
    mo, ms = kda.linear_prefill(*(x.float().abs() for x in last[:3]), last[3],
                                torch.tensor([0, tail], dtype=torch.int32, device="cuda"))
    assert ((s - s2).abs() <= 2 * lib.F32 * ms + 1e-30).all()
    step = 2 * (lib.F32 + 2 * lib.HALF_BF16)
    assert ((o[N - tail:].float() - o2.float()).abs() <= step * mo + 1e-30).all()
    assert torch.isfinite(o).all()


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_many_short_sequences_and_a_long_one(dtype):
    """More sequences than the plan keeps in shared memory, most of them empty or a few tokens long."""
    lengths = [i % 4 for i in range(1100)] + [900]
    c = lib.case(12, lengths, 1, 1, 64, 64, dtype)
    _check_prefill(c)
    _check_backward(c)


@pytest.mark.parametrize("lengths", [[3300, 260, 2000, 129, 1, 0, 700], [128 * 9, 128 * 9 + 1, 128 * 8 - 1]], ids=["mixed", "near"])
def test_segments_of_mixed_lengths(lengths):
    """Segments of several chunks, taken longest first: each state lands where it belongs, and twice the same bits."""
    c = lib.case(13, lengths, 16, 4, 128, 64, "bf16", pads=0.05)
    o, s = _check_prefill(lib.spoil_pads(c))
    o2, s2 = _prefill(c)
    assert torch.equal(o, o2) and torch.equal(s, s2)


@pytest.mark.parametrize("lengths,H,Hk,dk,dv,kw", [
    ([3600], 1, 1, 128, 128, dict(state=False)),
    ([9000, 1, 0, 5000], 2, 1, 64, 128, dict(pads=0.05)),
    ([14 * 256 + 1], 2, 2, 128, 64, dict(decay="head")),
    ([4300], 1, 1, 64, 64, dict(la_scale=20.0, pads=0.3)),
], ids=["no_states", "mixed", "one_row_over", "strong_decays"])
def test_backward_of_few_long_heads(lengths, H, Hk, dk, dv, kw):
    """Few heads of long sequences: parts of them are swept from states of their own, twice with the same bits."""
    c = lib.case(15, lengths, H, Hk, dk, dv, "bf16", **kw)
    if c["pad_mask"] is not None:
        lib.spoil_pads(c)
    g = _check_backward(c)
    again = _backward(c)
    assert all(torch.equal(g[n], again[n]) for n in g)
    less = _backward(c, want_grad_init_state=False)
    assert less["dS0"] is None
    assert all(torch.equal(g[n], less[n]) for n in ("dq", "dk", "dv", "dlog_alpha"))


def test_backward_of_few_long_heads_with_waits_that_run_out():
    c = lib.case(16, [4096], 1, 1, 128, 128, "bf16")
    d = lib.to_cuda(c)
    kda.debug_set_fault(0, 50)
    try:
        kda.linear_prefill_backward(d["q"], d["k"], d["v"], d["log_alpha"], d["cu_seqlens"], d["grad_o"],
                                    init_state=d["init_state"])
        assert kda.get_device_status() == kda.KDA_ERR_DEVICE_TIMEOUT
        assert 41 <= kda.debug_timeout_site() <= 117
    finally:
        kda.debug_set_fault(0, 0)
    _check_backward(c)


def test_calls_on_another_stream(monkeypatch):
    """With a stream given, a call's outputs and workspace are made on it, so that nobody else gets their memory while
    it runs; the results are those of the current stream."""
    c = lib.case(17, [300, 70], 4, 2, 128, 64, "bf16")
    d = lib.to_cuda(c)
    x = torch.randn(70, 256, generator=torch.Generator().manual_seed(17)).cuda()
    w = torch.ones(256).cuda()
    other, made = torch.cuda.Stream(), []

    def noted(fn):
        def call(*args, **kw):
            made.append(torch.cuda.current_stream())
            return fn(*args, **kw)
        return call

    def step(stream):
        state = d["init_state"].clone()
        if stream is not None:
            stream.wait_stream(torch.cuda.current_stream())
        out = [*kda.linear_prefill(d["q"], d["k"], d["v"], d["log_alpha"], d["cu_seqlens"],
                                   init_state=d["init_state"], stream=stream)]
        g = kda.linear_prefill_backward(d["q"], d["k"], d["v"], d["log_alpha"], d["cu_seqlens"], d["grad_o"],
                                        grad_final_state=d["grad_final_state"], init_state=d["init_state"], stream=stream)
        out += [g[n] for n in sorted(g)]
        rows = [d[n][:2].contiguous() for n in ("q", "k", "v", "log_alpha")]
        if stream is not None:
            stream.wait_stream(torch.cuda.current_stream())
        out += [kda.linear_decode(*rows, state, stream=stream), state]
        out += [kda.rms_norm(x, w, stream=stream)[0]]
        y, scale, _ = kda.rms_norm_quant(x, w, quant="int8", group=64, stream=stream)
        out += [y, scale, *kda.rms_norm_backward(x, w, x, stream=stream)]
        torch.cuda.synchronize()
        return out

    want = step(None)
    monkeypatch.setattr(kda, "_workspace", noted(kda._workspace))
    monkeypatch.setattr(kda, "_check_device", noted(kda._check_device))
    got = step(other)
    assert len(made) == 9 and all(s == other for s in made)
    assert torch.cuda.current_stream() != other
    assert all(torch.equal(a, b) for a, b in zip(want, got))
    assert kda.get_device_status() == kda.KDA_OK


def test_waits_that_run_out_are_reported():
    """A limit shorter than any load: the call returns, its status says so, and the next calls are whole."""
    c = lib.case(14, [500, 300], 4, 2, 128, 128, "bf16")
    d = lib.to_cuda(c)
    kda.debug_set_fault(0, 50)
    try:
        kda.linear_prefill(d["q"], d["k"], d["v"], d["log_alpha"], d["cu_seqlens"], init_state=d["init_state"])
        assert kda.get_device_status() == kda.KDA_ERR_DEVICE_TIMEOUT
        assert 41 <= kda.debug_timeout_site() <= 69
        kda.linear_prefill_backward(d["q"], d["k"], d["v"], d["log_alpha"], d["cu_seqlens"], d["grad_o"],
                                    init_state=d["init_state"])
        assert kda.get_device_status() == kda.KDA_ERR_DEVICE_TIMEOUT
        assert 71 <= kda.debug_timeout_site() <= 117
    finally:
        kda.debug_set_fault(0, 0)
    _check_prefill(c)
    _check_backward(c)
