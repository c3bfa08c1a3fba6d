"""Cases of the linear-attention and RMS-norm operators: inputs, plain forms and exact values.

The operators (value head h reads key head h // (H / Hk); pads are identity steps with o = 0):
  linear_prefill   S_t = a_t S_{t-1} + k_t v_t^T, o_t = S_t^T q_t over a packed batch, a_t = exp(log_alpha)
  linear_decode    one such step for each row, the state updated in place
  linear_backward  gradients of <o, grad_o> + <final_state, grad_final_state>
  rms_norm         r = x + residual, y = r rsqrt(mean(r^2) + eps) w, as is or in 8 bits with scales
  rms_backward     gradients of the norm, the gradient that reaches r along the residual added

``run`` computes them in elementary torch operations, or with the library's calls where ``own`` is
true; ``exact`` computes them in 64 bits, token by token or row by row.
"""
import math

import torch

own = False

EPS = 1e-6
CHUNK = 128                      # of the plain chunked form
F8_MAX, I8_MAX = 448.0, 127.0
TINY = 2.0 ** -100               # an all-zero group's scale is TINY / F8_MAX (or I8_MAX)


# ------------------------------------------------------------------------------------ cases
def listed():
    return [
        # a long prompt of one user: the benchmark's own prefill shape
        dict(name="prefill_long", op="prefill", lengths="131072", H=32, Hk=32, dk=128, dv=128, dtype="bf16",
             decay="token", pads=0.0, state=False),
        # a batch of prompts continued from cached states, ragged, some padded, one empty, shared key heads
        dict(name="prefill_ragged", op="prefill", lengths="4099,1,0,1537,777,63,2048,300", H=32, Hk=8, dk=128,
             dv=64, dtype="bf16", decay="token", pads=0.02, state=True),
        # a short fp32 prompt with a constant decay for each head: latency, and the fp32 form
        dict(name="prefill_f32", op="prefill", lengths="128,517", H=2, Hk=2, dk=64, dv=64, dtype="f32",
             decay="head", pads=0.0, state=True),
        # a serving step of a full batch: the benchmark's own decode shape
        dict(name="decode_batch", op="decode", rows=256, masked=26, H=32, Hk=32, dk=128, dv=128, dtype="bf16",
             decay="token"),
        # a serving step of a single user: latency
        dict(name="decode_one", op="decode", rows=1, masked=0, H=32, Hk=8, dk=128, dv=128, dtype="bf16",
             decay="head"),
        # a training step's backward over one long sequence
        dict(name="backward_long", op="backward", lengths="16384", H=32, Hk=32, dk=128, dv=128, dtype="bf16",
             decay="token", pads=0.0, state=False),
        # a training step over packed documents, shared key heads, a learnt decay for each head, fp32
        dict(name="backward_packed_f32", op="backward", lengths="700,1,129,0,1031,64", H=8, Hk=4, dk=64, dv=128,
             dtype="f32", decay="head", pads=0.03, state=True),
        # the block's input: residual added, normalised, e4m3 with a scale for 128 columns
        dict(name="norm_prompt_e4m3", op="norm", rows=16384, D=4096, dtype="bf16", residual=True, quant="e4m3",
             group=128),
        # the same in a serving step of a few users, a scale for each row: latency
        dict(name="norm_decode_e4m3", op="norm", rows=4, D=4096, dtype="bf16", residual=True, quant="e4m3", group=0),
        # linear attention's output, normalised for each head (rows of d_v)
        dict(name="norm_heads", op="norm", rows=131072 * 8, D=128, dtype="bf16", residual=False, quant="", group=0),
        # a training step's backward of the block's norm
        dict(name="norm_backward", op="norm_backward", rows=16384, D=4096, dtype="bf16", residual=True),
        # the same at an odd size in fp32, without a residual
        dict(name="norm_backward_odd_f32", op="norm_backward", rows=1003, D=2056, dtype="f32", residual=False),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["prefill", "prefill", "backward", "backward", "decode", "norm", "norm_backward"])
    dtype = rng.choice(["bf16", "bf16", "bf16", "f32"])
    if op in ("norm", "norm_backward"):
        D = 8 * _log_int(rng, 4, 1024)                       # 32 .. 8192 columns, multiples of 8
        rows = _log_int(rng, 1, 16384 * 4096 // D // (2 if dtype == "f32" else 1))
        case = dict(op=op, rows=rows, D=D, dtype=dtype, residual=rng.random() < 0.6)
        if op == "norm":
            quant = rng.choice(["", "e4m3", "int8"]) if dtype == "bf16" else ""
            case.update(quant=quant, group=rng.choice([0, 64, 128]) if quant else 0)
        return case
    H = rng.choice([1, 2, 3, 4, 6, 8, 16, 24, 32])
    Hk = H // rng.choice([g for g in (1, 2, 3, 4, 8) if H % g == 0])
    case = dict(op=op, H=H, Hk=Hk, dk=rng.choice([64, 128]), dv=rng.choice([64, 128]), dtype=dtype,
                decay=rng.choice(["token", "token", "head"]))
    if op == "decode":
        rows = _log_int(rng, 1, 256)
        return dict(case, rows=rows, masked=rng.randint(0, rows // 8))
    most = (32768 if op == "prefill" else 8192) // (8 if dtype == "f32" else 1)
    total = _log_int(rng, 1, most)
    n = rng.randint(1, 8)
    cuts = sorted(rng.randint(0, total) for _ in range(n - 1))
    lengths = [b - a for a, b in zip([0] + cuts, cuts + [total])]
    return dict(case, lengths=",".join(map(str, lengths)), pads=rng.choice([0.0, 0.0, 0.05]), state=rng.random() < 0.5)


def _lengths(case):
    return [int(x) for x in case["lengths"].split(",")]


# ------------------------------------------------------------------------------------ inputs
def _dtype(case):
    return torch.bfloat16 if case["dtype"] == "bf16" else torch.float32


def _token_inputs(case, rows, g):
    """q, k: unit rows; v ~ N(0, 1); gates -softplus(N(-2, 1)), or slopes from 2^-1 down to 2^-8 over the heads."""
    def normal(*shape):
        return torch.randn(shape, generator=g, device="cuda")

    H, Hk, dk, dv, dt = case["H"], case["Hk"], case["dk"], case["dv"], _dtype(case)
    s = {}
    for name in ("q", "k"):
        x = normal(rows, Hk, dk)
        s[name] = (x / x.norm(dim=-1, keepdim=True)).to(dt)
    s["v"] = normal(rows, H, dv).to(dt)
    if case["decay"] == "token":
        s["log_alpha"] = -torch.nn.functional.softplus(normal(rows, H) - 2.0)
    else:
        i = torch.arange(H, device="cuda", dtype=torch.float32)
        s["log_alpha"] = -torch.exp2(-1.0 - 7.0 * i / max(H - 1, 1)) * (1.0 + 0.1 * torch.rand(H, generator=g, device="cuda"))
    return s


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    op, dt = case["op"], _dtype(case)

    def normal(*shape):
        return torch.randn(shape, generator=g, device="cuda")

    if op in ("norm", "norm_backward"):
        rows, D = case["rows"], case["D"]
        s = dict(case=case, x=normal(rows, D).to(dt), weight=1.0 + 0.1 * normal(D))
        if op == "norm":
            s["residual"] = (2.0 * normal(rows, D)).to(dt) if case["residual"] else None
        else:
            s["grad_y"] = normal(rows, D).to(dt)
            s["grad_residual"] = normal(rows, D).to(dt) if case["residual"] else None
        return s
    if op == "decode":
        rows = case["rows"]
        s = dict(case=case, **_token_inputs(case, rows, g))
        s["state"] = 0.1 * normal(rows, case["H"], case["dk"], case["dv"])
        mask = torch.ones(rows, dtype=torch.uint8, device="cuda")
        mask[torch.randperm(rows, generator=g, device="cuda")[:case["masked"]]] = 0
        s["mask"] = mask if case["masked"] else None
        return s
    lengths = _lengths(case)
    N, B = sum(lengths), len(lengths)
    s = dict(case=case, lengths=lengths, **_token_inputs(case, N, g))
    cu = [0]
    for n in lengths:
        cu.append(cu[-1] + n)
    s["cu_seqlens"] = torch.tensor(cu, dtype=torch.int32, device="cuda")
    s["pad_mask"] = (torch.rand(N, generator=g, device="cuda") >= case["pads"]).to(torch.uint8) if case["pads"] else None
    shape = (B, case["H"], case["dk"], case["dv"])
    s["init_state"] = 0.1 * normal(*shape) if case["state"] else None
    if op == "backward":
        s["grad_o"] = normal(N, case["H"], case["dv"]).to(dt)
        s["grad_final_state"] = normal(*shape) if case["state"] else None
    return s


# ------------------------------------------------------------------------------------ one pass
def run(s):
    if own:
        return _run_own(s)
    op = s["case"]["op"]
    if op == "prefill":
        return _plain_prefill(s)
    if op == "decode":
        return _plain_decode(s)
    if op == "backward":
        return _plain_backward(s)
    return _plain_norm(s) if op == "norm" else _plain_norm_backward(s)


def _run_own(s):
    from gated_delta_rule_148_b200 import kda

    case = s["case"]
    if case["op"] == "prefill":
        o, state = kda.linear_prefill(s["q"], s["k"], s["v"], s["log_alpha"], s["cu_seqlens"], pad_mask=s["pad_mask"],
                                      init_state=s["init_state"])
        return {"o": o, "state": state}
    if case["op"] == "decode":
        o = kda.linear_decode(s["q"], s["k"], s["v"], s["log_alpha"], s["state"], mask=s["mask"])
        return {"o": o, "state": s["state"]}
    if case["op"] == "backward":
        return kda.linear_prefill_backward(s["q"], s["k"], s["v"], s["log_alpha"], s["cu_seqlens"], s["grad_o"],
                                           grad_final_state=s["grad_final_state"], pad_mask=s["pad_mask"],
                                           init_state=s["init_state"])
    if case["op"] == "norm":
        if not case["quant"]:
            y, r = kda.rms_norm(s["x"], s["weight"], residual=s["residual"], eps=EPS)
            return {"y": y, "r": r}
        y8, scale, r = kda.rms_norm_quant(s["x"], s["weight"], residual=s["residual"], eps=EPS, quant=case["quant"],
                                          group=case["group"])
        return {"y": _values(y8), "scale": scale, "r": r}
    dx, dw = kda.rms_norm_backward(s["x"], s["weight"], s["grad_y"], grad_residual=s["grad_residual"], eps=EPS)
    return {"dx": dx, "dw": dw}


def _values(y8):
    """8-bit values as floating numbers (in units of their scales): e4m3 is that already, int8 fits bf16 exactly."""
    return y8 if y8.is_floating_point() else y8.to(torch.bfloat16)


# ------------------------------------------------------------------------------------ plain linear attention
def _chunked(s):
    """The batch in chunks of CHUNK rows [n, C], none across two sequences: packed row of each, which are real
    tokens, the sequence of each chunk; fp32 operands [n, H, C, d] with zero rows for the rest; 64-bit decays."""
    case, dev = s["case"], s["q"].device
    C, H, G = CHUNK, case["H"], case["H"] // case["Hk"]
    lens = torch.tensor(s["lengths"])
    per = (lens + C - 1) // C
    seq = torch.repeat_interleave(torch.arange(len(lens)), per)
    first = torch.cumsum(lens, 0) - lens
    c0 = first[seq] + C * (torch.arange(len(seq)) - (torch.cumsum(per, 0) - per)[seq])
    rows = c0[:, None] + torch.arange(C)
    inside = rows < (first + lens)[seq][:, None]
    rows = torch.where(inside, rows, torch.zeros_like(rows)).to(dev)
    real = inside.to(dev)
    if s["pad_mask"] is not None:
        real = real & (s["pad_mask"][rows] != 0)

    def operand(x, group):
        x = torch.where(real[:, :, None, None], x[rows].float(), torch.zeros((), device=dev))
        return x.repeat_interleave(group, dim=2).transpose(1, 2).contiguous()

    la = s["log_alpha"].double()
    la = la[rows] if la.dim() == 2 else la.expand(len(seq), C, H)
    b = torch.cumsum(torch.where(real[:, :, None], la, torch.zeros((), dtype=la.dtype, device=dev)), 1).transpose(1, 2)
    seq = seq.to(dev)
    ends = torch.cumsum(b[:, :, -1], 0)                               # [n, H], over the whole batch
    return dict(rows=rows, inside=inside.to(dev), real=real, seq=seq, b=b, ends=ends, starts=ends - b[:, :, -1],
                q=operand(s["q"], G), k=operand(s["k"], G), v=operand(s["v"], 1),
                decay=_masked_exp(b[:, :, :, None] - b[:, :, None, :], _lower(C, dev)))


def _lower(C, dev):
    return torch.ones(C, C, dtype=torch.bool, device=dev).tril()


def _masked_exp(x, keep):
    return torch.where(keep, x, torch.full((), -math.inf, dtype=x.dtype, device=x.device)).exp().float()


def _mix(weights, parts):
    """[H, i, j] x [j, H, a, b] -> [i, H, a, b]: decayed sums of the chunks' parts."""
    n, H, a, b = parts.shape
    return torch.bmm(weights, parts.transpose(0, 1).reshape(H, n, a * b)).reshape(H, -1, a, b).transpose(0, 1)


def _spread(seq, c, B):
    """Decays between the batch's chunks and each sequence's two ends, [H, ..]: 64-bit exponents."""
    n, dev = len(seq), seq.device
    order = torch.arange(n, device=dev)
    of = seq[None, :] == torch.arange(B, device=dev)[:, None]          # [B, n]
    E, S0 = c["ends"].t(), c["starts"].t()                             # [H, n]
    before = (seq[:, None] == seq[None, :]) & (order[None, :] < order[:, None])
    any_of = of.any(1)
    first = torch.argmax(of.int(), 1) if n else torch.zeros(B, dtype=torch.long, device=dev)
    last = n - 1 - torch.argmax(of.flip(1).int(), 1) if n else first
    pick = lambda x, i: torch.where(any_of, x[:, i], torch.zeros((), dtype=x.dtype, device=dev)) if n else x.new_zeros(x.shape[0], B)  # noqa: E731
    begin, end = pick(S0, first), pick(E, last)                        # [H, B]
    return dict(
        start_from=_masked_exp(S0[:, :, None] - E[:, None, :], before),                       # chunk i's start <- chunk j
        start_init=_masked_exp(S0[:, :, None] - begin[:, None, :], of.t()),                   # chunk i's start <- initial state
        end_from=_masked_exp(end[:, :, None] - E[:, None, :], of),                            # final state <- chunk j
        end_init=(end - begin).exp().float().t())                                             # [B, H]


def _chunk_starts(s, c, w, local):
    S = _mix(w["start_from"], local)
    return S if s["init_state"] is None else S + _mix(w["start_init"], s["init_state"])


def _scatter(x, c, N):
    """[n, H, C, d] -> [N, H, d], zeros at pads."""
    out = x.new_zeros(N, x.shape[1], x.shape[3])
    out[c["rows"][c["inside"]]] = torch.where(c["real"][:, :, None, None], x.transpose(1, 2), x.new_zeros(()))[c["inside"]]
    return out


def _plain_prefill(s):
    c = _chunked(s)
    B = len(s["lengths"])
    w = _spread(c["seq"], c, B)
    to_end = (c["b"][:, :, -1:] - c["b"]).exp().float()[..., None]
    local = (c["k"] * to_end).transpose(2, 3) @ c["v"]
    S = _chunk_starts(s, c, w, local)
    o = (c["q"] @ c["k"].transpose(2, 3) * c["decay"]) @ c["v"] + c["b"].exp().float()[..., None] * (c["q"] @ S)
    final = _mix(w["end_from"], local)
    if s["init_state"] is not None:
        final = final + w["end_init"][:, :, None, None] * s["init_state"]
    return {"o": _scatter(o, c, s["q"].shape[0]).to(s["q"].dtype), "state": final.contiguous()}


def _plain_decode(s):
    case, S = s["case"], s["state"]
    G = case["H"] // case["Hk"]
    on = torch.ones(S.shape[0], dtype=torch.bool, device=S.device) if s["mask"] is None else s["mask"] != 0
    q, k = (s[x].float().repeat_interleave(G, dim=1) for x in ("q", "k"))
    a = torch.where(on[:, None], s["log_alpha"].exp(), torch.ones((), device=S.device))
    k = torch.where(on[:, None, None], k, torch.zeros((), device=S.device))
    S.mul_(a[:, :, None, None]).add_(k[..., None] * s["v"].float()[:, :, None, :])
    o = (q[:, :, None, :] @ S)[:, :, 0]
    return {"o": torch.where(on[:, None, None], o, torch.zeros((), device=S.device)).to(s["q"].dtype), "state": S}


def _plain_backward(s):
    case = s["case"]
    N, B, G = s["q"].shape[0], len(s["lengths"]), case["H"] // case["Hk"]
    c = _chunked(s)
    w = _spread(c["seq"], c, B)
    q, k, v, b = c["q"], c["k"], c["v"], c["b"]
    do = torch.where(c["real"][:, :, None, None], s["grad_o"][c["rows"]].float(), torch.zeros((), device=q.device))
    do = do.transpose(1, 2).contiguous()
    eb, to_end = b.exp().float()[..., None], (b[:, :, -1:] - b).exp().float()[..., None]
    whole = b[:, :, -1].exp().float()
    local = (k * to_end).transpose(2, 3) @ v
    S = _chunk_starts(s, c, w, local)
    back = (q * eb).transpose(2, 3) @ do                               # share of each chunk in its start's gradient
    # gradient of chunk j's end: the later chunks' shares and the final state's, decayed
    D = _mix(w["start_from"].transpose(1, 2), back)
    dS0 = _mix(w["start_init"].transpose(1, 2), back)
    if s["grad_final_state"] is not None:
        D = D + _mix(w["end_from"].transpose(1, 2), s["grad_final_state"])
        dS0 = dS0 + w["end_init"][:, :, None, None] * s["grad_final_state"]
    qk = q @ k.transpose(2, 3)
    M = do @ v.transpose(2, 3) * c["decay"]
    doS, vD = eb * (do @ S.transpose(2, 3)), to_end * (v @ D.transpose(2, 3))
    dq, dk = M @ k + doS, M.transpose(2, 3) @ q + vD
    dv = (qk * c["decay"]).transpose(2, 3) @ do + to_end * (k @ D)
    # decays: what passes over row u from rows s < u to rows t >= u, to the chunk's end, from its start, and through it
    pairs = (qk * M).double().flip(2).cumsum(2).flip(2).tril(-1).sum(3)
    to_rows = (q * doS).sum(3, dtype=torch.float64).flip(2).cumsum(2).flip(2)
    rows_on = (k * vD).sum(3, dtype=torch.float64)
    from_rows = rows_on.cumsum(2) - rows_on
    through = (whole[:, :, None, None] * S * D).sum((2, 3), dtype=torch.float64)
    dla = _scatter((pairs + to_rows + from_rows + through[..., None])[..., None], c, N)[..., 0]
    if s["log_alpha"].dim() == 1:
        dla = dla.sum(0)
    dt = s["q"].dtype
    group = lambda x: _scatter(x, c, N).reshape(N, case["Hk"], G, -1).sum(2).to(dt)  # noqa: E731
    return {"dq": group(dq), "dk": group(dk), "dv": _scatter(dv, c, N).to(dt), "dlog_alpha": dla.float(), "dS0": dS0.contiguous()}


# ------------------------------------------------------------------------------------ plain norm
def _plain_norm(s):
    case, x = s["case"], s["x"]
    if s["residual"] is not None:
        r = (x.float() + s["residual"].float()).to(x.dtype)
    else:
        r = None
    f = (x if r is None else r).float()
    y = f * torch.rsqrt((f * f).mean(1, keepdim=True) + EPS) * s["weight"]
    if not case["quant"]:
        return {"y": y.to(x.dtype), "r": r}
    rows, D = x.shape
    group = case["group"] or D
    most = F8_MAX if case["quant"] == "e4m3" else I8_MAX
    padded = torch.nn.functional.pad(y.abs(), (0, -D % group)).reshape(rows, -1, group)
    scale = padded.amax(2).clamp_min(TINY) / most
    z = y / scale.repeat_interleave(group, dim=1)[:, :D]
    y8 = z.to(torch.float8_e4m3fn) if case["quant"] == "e4m3" else z.round().clamp(-I8_MAX, I8_MAX).to(torch.int8)
    return {"y": _values(y8), "scale": scale, "r": r}


def _plain_norm_backward(s):
    x, dy = s["x"].float(), s["grad_y"].float()
    rstd = torch.rsqrt((x * x).mean(1, keepdim=True) + EPS)
    g = dy * s["weight"]
    dx = rstd * (g - x * (rstd * rstd * (x * g).mean(1, keepdim=True)))
    if s["grad_residual"] is not None:
        dx = dx + s["grad_residual"].float()
    return {"dx": dx.to(s["x"].dtype), "dw": (dy * x * rstd).sum(0, dtype=torch.float64).float()}


# ------------------------------------------------------------------------------------ what a pass cannot do without
def work(case):
    e = 2 if case["dtype"] == "bf16" else 4
    op = case["op"]
    if op in ("norm", "norm_backward"):
        n, D = case["rows"] * case["D"], case["D"]
        if op == "norm_backward":
            return {"bytes": n * e * (3 + case["residual"]) + 8 * D, "flops": 12 * n}
        out = n * (1 if case["quant"] else e)
        if case["quant"]:
            out += 4 * case["rows"] * (-(-D // case["group"]) if case["group"] else 1)
        return {"bytes": n * e * (3 if case["residual"] else 1) + out + 4 * D, "flops": (6 if case["quant"] else 4) * n}
    H, Hk, dk, dv = case["H"], case["Hk"], case["dk"], case["dv"]
    state = 4 * H * dk * dv
    if op == "decode":
        on, rows = case["rows"] - case["masked"], case["rows"]
        decay = 4 * H * (on if case["decay"] == "token" else 1)
        moved = on * (2 * state + e * (2 * Hk * dk + H * dv)) + rows * (e * H * dv + (1 if case["masked"] else 0)) + decay
        return {"bytes": moved, "flops": 5 * on * H * dk * dv}
    lengths = _lengths(case)
    N, B = sum(lengths), len(lengths)
    decay = 4 * H * (N if case["decay"] == "token" else 1)
    other = 4 * (B + 1) + (N if case["pads"] else 0)
    if op == "prefill":
        moved = N * e * (2 * Hk * dk + 2 * H * dv) + decay + other + B * state * (2 if case["state"] else 1)
        return {"bytes": moved, "flops": 4 * N * H * dk * dv}
    moved = N * e * (4 * Hk * dk + 3 * H * dv) + 2 * decay + other + B * state * (3 if case["state"] else 1)
    return {"bytes": moved, "flops": 10 * N * H * dk * dv}


# ------------------------------------------------------------------------------------ exact values
def exact(case, seed):
    op = case["op"]
    s = prepare(case, seed)
    if op in ("norm", "norm_backward"):
        return _exact_norm(s) if op == "norm" else _exact_norm_backward(s)
    if op == "decode":
        return _exact_decode(s)
    longest = max(_lengths(case))
    if longest > (140000 if op == "prefill" else 20000):
        return None
    return _exact_prefill(s) if op == "prefill" else _exact_backward(s)


class _Steps:
    """The batch's tokens in step order, 64 bits, SPAN steps at a time: what each sequence has at each step
    (a sequence that has no such token, or a pad there, gets a decay of 1 and zero vectors)."""

    SPAN = 128

    def __init__(self, s):
        case, dev = s["case"], s["q"].device
        self.s, self.case, self.G = s, case, case["H"] // case["Hk"]
        self.B, self.T = len(s["lengths"]), max(s["lengths"])
        self.lens, self.first = torch.tensor(s["lengths"], device=dev), s["cu_seqlens"][:-1].long()
        la = s["log_alpha"].double()
        self.la = la if la.dim() == 2 else la.expand(max(s["q"].shape[0], 1), case["H"])

    def block(self, t0, names):
        t = torch.arange(t0, min(t0 + self.SPAN, self.T), device=self.lens.device)[:, None]
        on = t < self.lens
        rows = torch.where(on, self.first + t, torch.zeros_like(t))
        if self.s["pad_mask"] is not None:
            on = on & (self.s["pad_mask"][rows] != 0)
        got = {"n": len(t), "rows": rows, "on": on, "a": torch.where(on[..., None], self.la[rows], 0.0).exp()[..., None, None]}
        for name in names:
            x = torch.where(on[..., None, None], self.s[name][rows].double(), 0.0)
            got[name] = x.repeat_interleave(self.G, dim=2) if name in ("q", "k") else x
        return got

    def zeros(self):
        c = self.case
        return torch.zeros(self.B, c["H"], c["dk"], c["dv"], dtype=torch.float64, device=self.lens.device)

    def put(self, out, got, steps):
        """Rows of `out` from the real tokens' entries of the block's `steps`."""
        out[got["rows"][got["on"]]] = torch.stack(steps)[got["on"]]


def _advance(S, got, i):
    return torch.addcmul(S * got["a"][i], got["k"][i][..., :, None], got["v"][i][..., None, :])


def _exact_prefill(s):
    st = _Steps(s)
    S = st.zeros() if s["init_state"] is None else s["init_state"].double()
    o = torch.zeros(s["v"].shape, dtype=torch.float64, device="cuda")
    for t0 in range(0, st.T, st.SPAN):
        got, steps = st.block(t0, ("q", "k", "v")), []
        for i in range(got["n"]):
            S = _advance(S, got, i)
            steps.append((got["q"][i][..., None, :] @ S)[..., 0, :])
        st.put(o, got, steps)
    return {"o": o, "state": S}


def _exact_backward(s):
    st, case = _Steps(s), s["case"]
    new = lambda like: torch.zeros(like.shape, dtype=torch.float64, device="cuda")  # noqa: E731
    dq, dk, dv, dla = new(s["q"]), new(s["k"]), new(s["v"]), new(st.la[:s["q"].shape[0]])
    S = st.zeros() if s["init_state"] is None else s["init_state"].double()
    dS = st.zeros() if s["grad_final_state"] is None else s["grad_final_state"].double()
    kept = []
    for t0 in range(0, st.T, st.SPAN):
        kept.append(S)
        got = st.block(t0, ("k", "v"))
        for i in range(got["n"]):
            S = _advance(S, got, i)
    share = lambda x: x.reshape(x.shape[0], case["Hk"], st.G, -1).sum(2)  # noqa: E731
    for t0 in reversed(range(0, st.T, st.SPAN)):
        got, states, steps = st.block(t0, ("q", "k", "v", "grad_o")), [kept.pop()], []
        for i in range(got["n"]):
            states.append(_advance(states[-1], got, i))
        for i in reversed(range(got["n"])):
            dS = torch.addcmul(dS, got["q"][i][..., :, None], got["grad_o"][i][..., None, :])
            steps.append((share((states[i + 1] @ got["grad_o"][i][..., None])[..., 0]), share((dS @ got["v"][i][..., None])[..., 0]),
                          (got["k"][i][..., None, :] @ dS)[..., 0, :], (got["a"][i] * states[i] * dS).sum((2, 3))))
            dS = got["a"][i] * dS
        for out, parts in zip((dq, dk, dv, dla), zip(*reversed(steps))):
            st.put(out, got, parts)
    return {"dq": dq, "dk": dk, "dv": dv, "dlog_alpha": dla if s["log_alpha"].dim() == 2 else dla.sum(0), "dS0": dS}


def _exact_decode(s):
    st = dict(s, lengths=[1] * s["case"]["rows"], pad_mask=s["mask"], init_state=s["state"],
              cu_seqlens=torch.arange(s["case"]["rows"] + 1, device="cuda"))
    return _exact_prefill(st)


def _exact_norm(s):
    case, x = s["case"], s["x"].double()
    r = None if s["residual"] is None else (x + s["residual"].double()).to(s["x"].dtype)
    f = x if r is None else r.double()
    y = f / (f.square().sum(1, keepdim=True) / case["D"] + EPS).sqrt() * s["weight"].double()
    if not case["quant"]:
        return {"y": y, "r": r}
    group, D = case["group"] or case["D"], case["D"]
    e4m3 = case["quant"] == "e4m3"
    scale, out = [], torch.empty_like(y)
    for c0 in range(0, D, group):
        part = y[:, c0:c0 + group]
        sc = part.abs().max(1).values.clamp(min=TINY) / (F8_MAX if e4m3 else I8_MAX)
        z = part / sc[:, None]
        if e4m3:        # steps of 2^(e-3), e >= -6: ties to the even multiple
            step = torch.exp2(torch.floor(torch.log2(z.abs().clamp(min=2.0 ** -6))) - 3.0)
            z = torch.clamp(torch.round(z / step) * step, -F8_MAX, F8_MAX)
        else:
            z = torch.clamp(torch.round(z), -I8_MAX, I8_MAX)
        out[:, c0:c0 + group] = z
        scale.append(sc)
    return {"y": out, "scale": torch.stack(scale, 1), "r": r}


def _exact_norm_backward(s):
    x, dy, w = s["x"].double(), s["grad_y"].double(), s["weight"].double()
    D = s["case"]["D"]
    rstd = 1.0 / (x.square().sum(1, keepdim=True) / D + EPS).sqrt()
    xhat = x * rstd
    g = dy * w
    dx = (g - xhat * (g * xhat).sum(1, keepdim=True) / D) * rstd
    if s["grad_residual"] is not None:
        dx = dx + s["grad_residual"].double()
    return {"dx": dx, "dw": (dy * xhat).sum(0)}
