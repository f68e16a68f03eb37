"""Cases and plain forms of the quantised decode layer's operators.

    recurrent   the gated delta rule token by token, on a pool of states, for a ragged batch
    norm        residual addition, root-mean-square norm and rows in 8 bits
    gated       norm per head, times weight and silu(gate), and rows in 8 bits
    quantize    rows in 8 bits as they are
    matmul      product of rows and weights in 8 bits, with a scale for each row and channel

``listed()`` and ``draw()`` give cases, ``prepare()`` what a program holds before the call,
``run()`` one pass: in elementary torch operations, or through the package where ``own`` is true.

Rows in 8 bits come back as the values they stand for, in bf16, the type of the layer's
activations: two correct sums that differ in their last bit may round one value of many
thousands to the neighbouring step, and a step is 1/127 of the row's largest value.
"""
import math
import random

import torch

own = False

TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
EPS = 1e-6
NORMAL = 2.0 ** -126          # a row whose scale would be smaller stands for zeros


def listed():
    return [
        # one sequence's decode step: nothing but latency
        dict(name="recurrent_step_1", op="recurrent", seqs=1, longest=1, key_heads=16, heads=16, dk=128, dv=128,
             io="bf16", out="bf16", packed=True, padded=False, unit=False),
        # the decode benchmark's batch, a full pool of states
        dict(name="recurrent_step_256", op="recurrent", seqs=256, longest=1, key_heads=16, heads=16, dk=128, dv=128,
             io="bf16", out="bf16", packed=False, padded=False, unit=False),
        # mixed batch: prompts of up to 600 tokens beside decode steps, shared key heads, idle entries
        dict(name="recurrent_ragged_48", op="recurrent", seqs=48, longest=600, key_heads=8, heads=32, dk=128, dv=128,
             io="bf16", out="f32", packed=True, padded=True, unit=True),
        # a decode step's norm at the layer's width (16 heads of 128)
        dict(name="norm_decode_16", op="norm", rows=16, width=2048, io="bf16", residual="bf16", weight="f32"),
        # a prompt's norm, residual stream in 32 bits
        dict(name="norm_prompt_8192", op="norm", rows=8192, width=4096, io="bf16", residual="f32", weight="bf16"),
        # the heads' outputs of a decode step, the gate a part of a wider projection's rows
        dict(name="gated_decode_61", op="gated", rows=61, heads=16, dv=128, io="bf16", weight="f32", packed=True),
        # the heads' outputs of the benchmark's 4 x 4096 tokens
        dict(name="gated_prompt_16384", op="gated", rows=16384, heads=16, dv=128, io="bf16", weight="f32", packed=False),
        # activations of an odd width
        dict(name="quantize_odd_37", op="quantize", rows=37, width=1001, io="f32"),
        # the weights of the layer's input projection (q, k, v, gate, and a decay and a strength for each of 16 heads)
        dict(name="quantize_weight_8224", op="quantize", rows=8224, width=2048, io="bf16"),
        # that projection in a decode step of 16 sequences: bound by the weights' bytes
        dict(name="matmul_decode_16", op="matmul", m=16, n=8224, k=2048, out="bf16", bias=False, padded=True),
        # odd sizes, rows that are not padded, a bias and an output in 32 bits
        dict(name="matmul_odd_333", op="matmul", m=333, n=1001, k=1537, out="f32", bias=True, padded=False),
        # a prompt's projection at a large width
        dict(name="matmul_prompt_8192", op="matmul", m=8192, n=8192, k=8192, out="bf16", bias=False, padded=True),
    ]


def _log(rng, lo, hi):
    """A whole number between lo and hi, spread evenly over its logarithm."""
    return min(hi, max(lo, round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49))))))


def draw(rng):
    op = rng.choice(["recurrent", "norm", "gated", "quantize", "matmul"])
    io = rng.choice(["bf16", "bf16", "f32"])
    flip = lambda: rng.random() < 0.5  # noqa: E731
    if op == "recurrent":
        key_heads = rng.choice([1, 2, 4, 8, 16])
        heads = key_heads * rng.choice([1, 1, 2, 4])
        dk, dv = rng.choice([16, 32, 64, 128, 128, 128]), rng.choice([32, 64, 96, 128, 128, 128])
        longest = rng.choice([1, 1, _log(rng, 2, 8), _log(rng, 2, 600)])
        most = min(256, 4096 * 128 * 128 // (heads * dk * dv), max(1, 48 * 32 * 600 // (heads * longest)))
        return dict(op=op, seqs=_log(rng, 1, max(1, most)), longest=longest, key_heads=key_heads, heads=heads, dk=dk,
                    dv=dv, io=io, out=rng.choice([io, "f32"]), packed=flip(), padded=flip(), unit=flip())
    if op == "norm":
        width = _log(rng, 64, 16384) if flip() else 8 * _log(rng, 8, 2048)
        return dict(op=op, rows=_log(rng, 1, max(1, min(8192, 8192 * 2048 // width))), width=width, io=io,
                    residual=rng.choice(["bf16", "f32", "none"]), weight=rng.choice(["bf16", "f32"]))
    if op == "gated":
        heads, dv = rng.choice([1, 3, 8, 16, 32, 64]), rng.choice([32, 64, 96, 128, 128])
        return dict(op=op, rows=_log(rng, 1, 8192 * 16 * 128 // (heads * dv * 2)), heads=heads, dv=dv, io=io,
                    weight=rng.choice(["bf16", "f32"]), packed=flip())
    if op == "quantize":
        width = _log(rng, 16, 16384)
        return dict(op=op, rows=_log(rng, 1, max(1, min(8192, 8224 * 1024 // width))), width=width, io=io)
    n, k = (16 * _log(rng, 1, 512), 16 * _log(rng, 4, 512)) if flip() else (_log(rng, 16, 8192), _log(rng, 64, 8192))
    out = rng.choice(["bf16", "f32"])
    return dict(op=op, m=_log(rng, 1, 8192 if out == "bf16" else 4096), n=n, k=k, out=out, bias=flip(), padded=flip())


def _lengths(case):
    """Tokens of each sequence: the longest first, one of none, the others spread over the logarithm."""
    r = random.Random(case["seqs"] * 1009 + case["longest"])
    if case["longest"] == 1:
        return [1] * case["seqs"]
    some = [_log(r, 1, case["longest"]) for _ in range(case["seqs"])]
    some[0] = case["longest"]
    if case["seqs"] > 2:
        some[1] = 0
    return some


def _idle(case):
    """Entries of a padded batch that hold no sequence (slot -1)."""
    return [case["padded"] and i % 7 == 3 for i in range(case["seqs"])]


def _pad16(width):
    return (width + 15) // 16 * 16


def prepare(case, seed):
    g = torch.Generator("cuda").manual_seed(seed)
    normal = lambda *s: torch.randn(*s, device="cuda", generator=g)  # noqa: E731
    state = dict(case=case)
    if case["op"] == "recurrent":
        lens, idle = _lengths(case), _idle(case)
        S, N, H, Hk, dk, dv = case["seqs"], sum(lens), case["heads"], case["key_heads"], case["dk"], case["dv"]
        rows = N + (5 if case["padded"] else 0)      # rows behind the last sequence: left as they are
        io = TYPES[case["io"]]
        if case["packed"]:                           # parts of one projection's rows
            row = normal(rows, (2 * Hk * dk + H * dv)).to(io)
            q, k, v = row.split([Hk * dk, Hk * dk, H * dv], dim=1)
        else:
            q, k, v = normal(rows, Hk * dk).to(io), normal(rows, Hk * dk).to(io), normal(rows, H * dv).to(io)
        q, k, v = q.unflatten(1, (Hk, dk)), k.unflatten(1, (Hk, dk)), v.unflatten(1, (H, dv))
        if not case["unit"]:                         # normalised already
            for x in (q, k):
                x.copy_((x.float() / x.float().norm(dim=-1, keepdim=True)).to(io))
        # trained layers' decay sits close to 1
        alpha = 0.9 + 0.1 * torch.rand(rows, H, device="cuda", generator=g)
        beta = torch.sigmoid(normal(rows, H))
        pool = S + S // 4 + 1
        slots = torch.randperm(pool, device="cuda", generator=g)[:S].to(torch.int32)
        slots[torch.tensor(idle, device="cuda")] = -1
        starts = [0]
        for n in lens:
            starts.append(starts[-1] + n)
        state.update(q=q, k=k, v=v, alpha=alpha, beta=beta, slots=slots, lens=lens, starts=starts,
                     cu=None if case["longest"] == 1 and not case["padded"] else torch.tensor(starts, dtype=torch.int32, device="cuda"),
                     state=0.02 * normal(pool, H, dk, dv), out=torch.full((rows, H, dv), 7.0, device="cuda", dtype=TYPES[case["out"]]))
    elif case["op"] in ("norm", "quantize"):
        R, D = case["rows"], case["width"]
        loud = torch.where(torch.rand(D, device="cuda", generator=g) < 0.01, 20.0, 1.0)   # a few channels stand out
        x = (normal(R, D) * loud).to(TYPES[case["io"]])
        state.update(x=x)
        if R > 3:
            x[R // 2] = 0                            # a row of padding
        if case["op"] == "norm":
            state.update(weight=(1 + 0.1 * normal(D)).to(TYPES[case["weight"]]), residual=None)
            if case["residual"] != "none":
                state["residual"] = (3 * normal(R, D)).to(TYPES[case["residual"]])
                if R > 3:
                    state["residual"][R // 2] = 0
    elif case["op"] == "gated":
        R, H, dv, io = case["rows"], case["heads"], case["dv"], TYPES[case["io"]]
        x = (0.1 * normal(R, H, dv)).to(io)
        if R > 3:
            x[R // 2] = 0
        gate = normal(R, (3 if case["packed"] else 1) * H * dv).to(io)
        state.update(x=x, gate=gate[:, -H * dv:].unflatten(1, (H, dv)), weight=(1 + 0.1 * normal(dv)).to(TYPES[case["weight"]]))
    else:
        m, n, k = case["m"], case["n"], case["k"]
        width = _pad16(k) if case["padded"] else k
        whole = lambda r: torch.zeros(r, width, dtype=torch.int8, device="cuda")[:, :k].copy_(  # noqa: E731
            (40 * normal(r, k)).round().clamp(-127, 127))
        state.update(x=whole(m), w=whole(n), xs=0.01 + 0.02 * torch.rand(m, device="cuda", generator=g),
                     ws=0.0005 + 0.001 * torch.rand(n, device="cuda", generator=g), bias=normal(n) if case["bias"] else None)
    return state


def _values(q, scale):
    """What rows in 8 bits stand for."""
    return torch.mul(q, scale.unsqueeze(-1), out=torch.empty(q.shape, device=q.device, dtype=torch.bfloat16))


def _rows8(y):
    """Rows in 8 bits and their scales: the row's largest absolute value is 127 steps."""
    scale = y.abs().amax(-1) / 127
    scale = torch.where(scale < NORMAL, 0.0, scale)
    q = (y / torch.where(scale == 0, 1.0, scale).unsqueeze(-1)).round() * (scale != 0).unsqueeze(-1)
    return q.to(torch.int8), scale


def _recurrent(s):
    c = s["case"]
    group = c["heads"] // c["key_heads"]
    q, k, v = s["q"].float(), s["k"].float(), s["v"].float()
    if c["unit"]:
        q, k = (x / (x.square().sum(-1, keepdim=True) + EPS).sqrt() for x in (q, k))
    q, k = q.repeat_interleave(group, 1), k.repeat_interleave(group, 1)
    first = torch.tensor(s["starts"][:-1], device=q.device)
    lens = torch.tensor(s["lens"], device=q.device)
    live = s["slots"] >= 0
    at = s["slots"].long().clamp(min=0)
    h = s["state"][at]                                                  # [S, H, dk, dv]
    for t in range(c["longest"]):                                       # token t of every sequence that has one
        on = (lens > t)
        row = torch.where(on, first + t, 0)
        kt, qt, a, b = k[row], q[row], s["alpha"][row], s["beta"][row]
        p = (h * kt.unsqueeze(-1)).sum(-2)
        u = b.unsqueeze(-1) * (v[row] - a.unsqueeze(-1) * p)
        new = a[..., None, None] * h + kt.unsqueeze(-1) * u.unsqueeze(-2)
        o = (new * qt.unsqueeze(-1)).sum(-2) * live[:, None, None]
        h = torch.where(on[:, None, None, None], new, h)
        s["out"][row[on]] = o[on].to(s["out"].dtype)
    s["state"][at[live]] = h[live]
    return dict(o=s["out"], state=s["state"])


def _plain(s):
    c = s["case"]
    if c["op"] == "recurrent":
        return _recurrent(s)
    if c["op"] == "norm":
        h = s["x"].float() if s["residual"] is None else s["x"].float() + s["residual"].float()
        q, scale = _rows8(h / (h.square().mean(-1, keepdim=True) + EPS).sqrt() * s["weight"].float())
        out = dict(values=_values(q, scale), scale=scale)
        return out if s["residual"] is None else dict(out, residual=h.to(s["residual"].dtype))
    if c["op"] == "gated":
        x, gate = s["x"].float(), s["gate"].float()
        y = x / (x.square().mean(-1, keepdim=True) + EPS).sqrt() * s["weight"].float() * gate / (1 + (-gate).exp())
        q, scale = _rows8(y.flatten(1))
        return dict(values=_values(q, scale), scale=scale)
    if c["op"] == "quantize":
        q, scale = _rows8(s["x"].float())
        return dict(values=_values(q, scale), scale=scale)
    y = (s["x"].float() @ s["w"].float().t()) * s["xs"].unsqueeze(1) * s["ws"]
    return (y if s["bias"] is None else y + s["bias"]).to(TYPES[c["out"]])


def _own(s):
    import chunked_gated_delta_14_b200 as gdn
    c = s["case"]
    if c["op"] == "recurrent":
        o = gdn.recurrent_fwd(s["q"], s["k"], s["v"], s["alpha"], s["beta"], s["state"], s["slots"], s["cu"],
                              qk_norm_eps=EPS if c["unit"] else None, out=s["out"])
        return dict(o=o, state=s["state"])
    if c["op"] == "norm":
        q, scale, residual = gdn.add_rms_norm_int8(s["x"], s["weight"], s["residual"], eps=EPS)
        out = dict(values=_values(q, scale), scale=scale)
        return out if residual is None else dict(out, residual=residual)
    if c["op"] == "gated":
        q, scale = gdn.gated_rms_norm_int8(s["x"], s["gate"], s["weight"], eps=EPS)
        return dict(values=_values(q, scale), scale=scale)
    if c["op"] == "quantize":
        q, scale = gdn.quantize_int8(s["x"])
        return dict(values=_values(q, scale), scale=scale)
    return gdn.int8_matmul(s["x"], s["xs"], s["w"], s["ws"], s["bias"], out_dtype=TYPES[c["out"]])


def run(state):
    return _own(state) if own else _plain(state)


def work(case):
    size = lambda t: 2 if case[t] == "bf16" else 4  # noqa: E731
    if case["op"] == "recurrent":
        lens = [0 if off else n for n, off in zip(_lengths(case), _idle(case))]
        n, live, cells = sum(lens), sum(x > 0 for x in lens), case["heads"] * case["dk"] * case["dv"]
        row = (2 * case["key_heads"] * case["dk"] + case["heads"] * case["dv"]) * size("io") + case["heads"] * (8 + case["dv"] * size("out"))
        return {"bytes": 8 * live * cells + n * row, "flops": 7 * n * cells}
    if case["op"] == "norm":
        cells = case["rows"] * case["width"]
        both = 0 if case["residual"] == "none" else 2 * size("residual")
        return {"bytes": cells * (size("io") + both + 1) + 4 * case["rows"] + case["width"] * size("weight"), "flops": 6 * cells}
    if case["op"] == "gated":
        cells = case["rows"] * case["heads"] * case["dv"]
        return {"bytes": cells * (2 * size("io") + 1) + 4 * case["rows"], "flops": 12 * cells}
    if case["op"] == "quantize":
        cells = case["rows"] * case["width"]
        return {"bytes": cells * (size("io") + 1) + 4 * case["rows"], "flops": 3 * cells}
    m, n, k = case["m"], case["n"], case["k"]
    return {"bytes": (m + n) * (k + 4) + m * n * size("out") + (4 * n if case["bias"] else 0), "flops": 2 * m * n * k}


def exact(case, seed):
    """The definitions, sequence by sequence and row by row, in 64 bits."""
    s = prepare(case, seed)
    if case["op"] == "recurrent":
        group, norm = case["heads"] // case["key_heads"], case["unit"]
        o, pool = s["out"].double(), s["state"].double()
        eye = torch.eye(case["dk"], dtype=torch.float64, device=o.device)
        for i, slot in enumerate(s["slots"].tolist()):
            a, e = s["starts"][i], s["starts"][i + 1]
            if slot < 0:
                o[a:e] = 0
                continue
            S = pool[slot].transpose(1, 2).clone()                      # d_v x d_k for each head
            for t in range(a, e):
                q, k = (torch.stack([s[x][t, j // group].double() for j in range(case["heads"])]) for x in ("q", "k"))
                if norm:
                    q, k = q / (q.pow(2).sum(1, True) + EPS).sqrt(), k / (k.pow(2).sum(1, True) + EPS).sqrt()
                v, al, be = s["v"][t].double(), s["alpha"][t].double(), s["beta"][t].double()
                S = al[:, None, None] * (S @ (eye - be[:, None, None] * k[:, :, None] * k[:, None, :])) + be[:, None, None] * v[:, :, None] * k[:, None, :]
                o[t] = (S @ q[:, :, None])[:, :, 0]
            pool[slot] = S.transpose(1, 2)
        return dict(o=o, state=pool)
    if case["op"] == "matmul":
        y = torch.einsum("mk,nk->mn", s["x"].double() * s["xs"].double()[:, None], s["w"].double() * s["ws"].double()[:, None])
        return y + s["bias"].double() if case["bias"] else y
    x = s["x"].double()
    out = {}
    if case["op"] == "norm":
        if s["residual"] is not None:
            x = x + s["residual"].double()
            out["residual"] = x
        x = x * torch.rsqrt(x.pow(2).mean(1, True) + EPS) * s["weight"].double()
    elif case["op"] == "gated":
        x = x * torch.rsqrt(x.pow(2).mean(2, True) + EPS) * s["weight"].double() * torch.nn.functional.silu(s["gate"].double())
        x = x.reshape(x.shape[0], -1)
    top = x.abs().max(1).values
    steps = torch.where(top[:, None] > 0, torch.round(127 * x / top.clamp(min=1e-300)[:, None]), 0.0)
    return dict(out, values=steps * (top / 127)[:, None], scale=top / 127)
