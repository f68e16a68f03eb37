"""Decode-layer operators on the GPU against plain implementations in 64 bits.

Tolerances count roundings: u = 2^-24 is half a step of fp32 relative to the
value, 2^-8 of bf16.  They were derived before the first run, beside each check.
"""
import math

import pytest
import torch

import bench
import chunked_gated_delta_14_b200 as gdn

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
HALF = {torch.bfloat16: 2.0 ** -8, torch.float32: U}
BF, F = torch.bfloat16, torch.float32


def rng(seed):
    return torch.Generator("cuda").manual_seed(seed)


def randn(g, *s):
    return torch.randn(*s, device="cuda", generator=g)


# ------------------------------------------------------------------ recurrent_fwd

def rule64(q, k, v, alpha, beta, state, slots, starts, o, eps=None):
    """The recurrence in 64 bits, one sequence at a time.  Also the largest ||h column|| + |v|
    each slot's columns saw, which scales the error bound."""
    Hk, H = q.shape[1], v.shape[1]
    o, pool = o.double().clone(), state.double().clone()
    big = torch.zeros(pool.shape[0], H, pool.shape[3], dtype=torch.float64, device=q.device)
    for i, slot in enumerate(slots):
        a, e = starts[i], starts[i + 1]
        if slot < 0:
            o[a:e] = 0
            continue
        h = pool[slot]
        for t in range(a, e):
            qt, kt = (x[t].double().repeat_interleave(H // Hk, 0) for x in (q, k))
            if eps is not None:
                qt, kt = (x / (x.pow(2).sum(-1, keepdim=True) + eps).sqrt() for x in (qt, kt))
            al = 1.0 if alpha is None else alpha[t].double()[:, None]
            be = 1.0 if beta is None else beta[t].double()[:, None]
            p = torch.einsum("hij,hi->hj", h, kt)
            uu = be * (v[t].double() - al * p)
            big[slot] = torch.maximum(big[slot], h.norm(dim=1) + v[t].double().abs() + uu.abs())
            h = (al[..., None] if alpha is not None else 1.0) * h + kt[:, :, None] * uu[:, None, :]
            big[slot] = torch.maximum(big[slot], h.norm(dim=1))
            o[t] = torch.einsum("hij,hi->hj", h, qt)
        pool[slot] = h
    return o, pool, big


def check_rule(got_o, got_state, want, slots, starts, q, dk, longest, eps=None):
    """||k|| <= 1 and alpha, beta in [0, 1] make every transition a contraction, so the
    errors of the tokens add.  A token's: the sum of p in runs of dk / 8 and 3 exchanges,
    and at most 12 more roundings (v - alpha p, beta, alpha h, k u, their sum; 4 more for
    normalised k and q), each relative to at most ||h|| + |v| + |u| of the column."""
    o, pool, big = want
    one = (dk / 8 + 3 + 12 + (dk / 8 if eps is not None else 0)) * U * 1.1
    err = (got_state.double() - pool).norm(dim=2)              # by column
    assert (err <= longest * one * big + 1e-30).all(), float((err / (longest * one * big + 1e-30)).max())
    for i, slot in enumerate(slots):
        a, e = starts[i], starts[i + 1]
        if slot < 0 or a == e:
            continue
        qn = q[a:e].double().norm(dim=-1).amax().clamp(min=1.0) if eps is None else 1.0
        tol = (longest + 1) * one * qn * big[slot] + HALF[got_o.dtype] * o[a:e].abs() * (1 + 2 ** -7)
        assert ((got_o[a:e].double() - o[a:e]).abs() <= tol + 1e-30).all(), i


def make_rule(seed, lens, Hk, H, dk, dv, io=BF, pool=None, packed=False, gates=True, tail=0, unit=False):
    g = rng(seed)
    N = sum(lens) + tail
    if packed:
        row = randn(g, N, 2 * Hk * dk + H * dv + 8).to(io)
        q, k, v = row[:, :Hk * dk], row[:, Hk * dk:2 * Hk * dk], row[:, 2 * Hk * dk:2 * Hk * dk + H * dv]
    else:
        q, k, v = randn(g, N, Hk * dk).to(io), randn(g, N, Hk * dk).to(io), randn(g, N, H * dv).to(io)
    q, k, v = q.unflatten(1, (Hk, dk)), k.unflatten(1, (Hk, dk)), v.unflatten(1, (H, dv))
    if not unit:
        for x in (q, k):     # 0.99: bf16 may round a unit vector to a longer one
            x.copy_((0.99 * x.float() / x.float().norm(dim=-1, keepdim=True)).to(io))
    alpha = 0.8 + 0.2 * torch.rand(N, H, device="cuda", generator=g) if gates else None
    beta = torch.rand(N, H, device="cuda", generator=g) if gates else None
    state = 0.1 * randn(g, pool or len(lens), H, dk, dv)
    starts = [0]
    for n in lens:
        starts.append(starts[-1] + n)
    return q, k, v, alpha, beta, state, starts


@pytest.mark.parametrize("io", [BF, F])
@pytest.mark.parametrize("dk,dv,Hk,H", [(128, 128, 2, 4), (16, 32, 1, 1), (32, 96, 3, 3), (64, 64, 1, 8), (128, 32, 5, 5)])
def test_recurrent_one_token_each(io, dk, dv, Hk, H):
    S = 5
    q, k, v, al, be, state, starts = make_rule(1, [1] * S, Hk, H, dk, dv, io)
    want = rule64(q, k, v, al, be, state, range(S), starts, torch.zeros(S, H, dv, device="cuda"))
    o = gdn.recurrent_fwd(q, k, v, al, be, state)
    gdn.device_check()
    assert o.dtype == io and o.shape == (S, H, dv)
    check_rule(o, state, want, range(S), starts, q, dk, 1)


@pytest.mark.parametrize("io", [BF, F])
@pytest.mark.parametrize("dk,dv,Hk,H", [(128, 128, 4, 8), (64, 96, 2, 4), (16, 64, 3, 9), (32, 32, 4, 4)])
def test_recurrent_one_token_each_of_many_heads(io, dk, dv, Hk, H):
    """Two blocks a SM and more, where a block takes more columns; some entries idle."""
    S = 320 // H + 1
    q, k, v, al, be, state, starts = make_rule(41, [1] * S, Hk, H, dk, dv, io, pool=S + 3, packed=True)
    slots = torch.randperm(S + 3, generator=torch.Generator().manual_seed(1))[:S].tolist()
    slots[5] = slots[S - 1] = -1
    want = rule64(q, k, v, al, be, state, slots, starts, torch.zeros(S, H, dv, device="cuda"), 1e-6)
    o = gdn.recurrent_fwd(q, k, v, al, be, state, torch.tensor(slots, dtype=torch.int32, device="cuda"), qk_norm_eps=1e-6, o_dtype=F)
    gdn.device_check()
    check_rule(o, state, want, slots, starts, q, dk, 1, 1e-6)
    assert (o[5] == 0).all() and (o[S - 1] == 0).all()


@pytest.mark.parametrize("lens", [[3, 2, 0, 1], [40, 30, 0, 20]])
def test_recurrent_reads_nothing_of_idle_entries_and_rows_of_no_sequence(lens):
    """NaN in the tokens and states that belong to no sequence."""
    q, k, v, al, be, state, starts = make_rule(42, lens, 1, 2, 64, 64, BF, pool=6, tail=3)
    slots = [4, -1, 0, 2]
    cu = torch.tensor(starts, dtype=torch.int32, device="cuda")
    want = rule64(q, k, v, al, be, state, slots, starts, torch.zeros(v.shape, device="cuda"))
    for t in (q, k, v, al, be):
        t[starts[1]:starts[2]] = math.nan
        t[starts[4]:] = math.inf
    for i in (1, 3, 5):
        state[i] = math.nan
    o = gdn.recurrent_fwd(q, k, v, al, be, state, torch.tensor(slots, dtype=torch.int32, device="cuda"), cu, o_dtype=F)
    live = torch.tensor([0, 2, 4], device="cuda")
    q[starts[1]:starts[2]] = 0
    check_rule(o, state[live], (want[0], want[1][live], want[2][live]), [2, -1, 0, 1], starts, q, 64, max(lens))
    assert (o[starts[1]:starts[2]] == 0).all() and (o[starts[4]:] == 0).all()
    assert state[[1, 3, 5]].isnan().all()


@pytest.mark.parametrize("io,packed,unit,o_dtype", [(BF, True, True, F), (BF, False, False, BF), (F, True, False, BF), (F, False, True, F)])
@pytest.mark.parametrize("dk,dv,Hk,H", [(128, 128, 1, 4), (16, 96, 2, 2), (64, 32, 2, 6)])
def test_recurrent_ragged_pool(io, packed, unit, o_dtype, dk, dv, Hk, H):
    lens, slots = [7, 0, 1, 33, 2, 3], [4, 0, -1, 7, 2, 1]
    q, k, v, al, be, state, starts = make_rule(2, lens, Hk, H, dk, dv, io, pool=9, packed=packed, tail=3, unit=unit)
    cu = torch.tensor(starts, dtype=torch.int32, device="cuda")
    out = torch.full((q.shape[0], H, dv), 5.0, device="cuda", dtype=o_dtype)
    eps = 1e-6 if unit else None
    before = state.clone()
    want = rule64(q, k, v, al, be, state, slots, starts, out, eps)
    o = gdn.recurrent_fwd(q, k, v, al, be, state, torch.tensor(slots, dtype=torch.int32, device="cuda"), cu,
                          qk_norm_eps=eps, out=out)
    gdn.device_check()
    assert o is out
    check_rule(o, state, want, slots, starts, q, dk, max(lens), eps)
    assert (o[starts[-1]:] == 5).all()                       # rows of no sequence
    assert (o[starts[2]:starts[3]] == 0).all()               # an idle entry
    for i in (0, 3, 5, 6, 8):                                # states of no sequence, and of one with no tokens
        assert torch.equal(state[i], before[i])


def test_recurrent_of_nothing():
    none = torch.zeros(0, 2, 64, device="cuda")
    state = randn(rng(45), 3, 2, 64, 64)
    before = state.clone()
    cu = lambda *n: torch.tensor(n, dtype=torch.int32, device="cuda")  # noqa: E731
    assert gdn.recurrent_fwd(none, none, none, None, None, state).shape == (0, 2, 64)
    gdn.recurrent_fwd(none, none, none, None, None, state, None, cu(0, 0, 0))
    x = randn(rng(46), 4, 2, 64)
    o = gdn.recurrent_fwd(x, x, x, None, None, state, None, cu(0))
    o2 = gdn.recurrent_fwd(x, x, x, None, None, state, cu(2, 1), cu(3, 3, 3))
    assert not o.any() and not o2.any() and torch.equal(state, before)


def test_recurrent_made_output_is_zero_behind_the_last_sequence():
    q, k, v, al, be, state, starts = make_rule(3, [2, 1], 1, 1, 64, 64, tail=4)
    cu = torch.tensor(starts, dtype=torch.int32, device="cuda")
    o = gdn.recurrent_fwd(q, k, v, al, be, state, None, cu, o_dtype=F)
    assert (o[3:] == 0).all() and o.dtype == F


def test_recurrent_without_gates_and_with_unaligned_rows():
    lens = [4, 5]
    q, k, v, _, _, state, starts = make_rule(4, lens, 2, 2, 128, 64, BF, gates=False)
    odd = lambda x: torch.empty(x.shape[0], x.shape[1], x.shape[2] + 1, device="cuda", dtype=x.dtype)[..., 1:].copy_(x)  # noqa: E731
    cu = torch.tensor(starts, dtype=torch.int32, device="cuda")
    want = rule64(q, k, v, None, None, state, range(2), starts, torch.zeros_like(v))
    o = gdn.recurrent_fwd(odd(q), odd(k), odd(v), None, None, state, None, cu)
    check_rule(o, state, want, range(2), starts, q, 128, 5)


@pytest.mark.parametrize("dk,dv,Hk,H,io", [(128, 128, 1, 1, F), (32, 96, 1, 1, F), (128, 128, 1, 3, BF), (128, 128, 3, 3, F),
                                           (16, 128, 1, 4, BF), (64, 128, 1, 3, F)])
def test_recurrent_long_sequences_of_many_lengths(dk, dv, Hk, H, io):
    """Lengths whose mean is over 16, where the blocks take the longest sequences first, and from
    296 sequences and heads on two column quads a lane."""
    g = torch.Generator().manual_seed(8)
    lens = [1, 0, 200, 63, 64, 65, 2] + torch.randint(0, 60, (140,), generator=g).tolist()
    slots = torch.randperm(160, generator=g)[:len(lens)].tolist()
    slots[3] = slots[40] = -1
    q, k, v, al, be, state, starts = make_rule(8, lens, Hk, H, dk, dv, io, pool=160, tail=4)
    assert starts[-1] >= 16 * len(lens)
    out = torch.full(v.shape, 5.0, device="cuda", dtype=io)
    want = rule64(q, k, v, al, be, state, slots, starts, out)
    gdn.recurrent_fwd(q, k, v, al, be, state, torch.tensor(slots, dtype=torch.int32, device="cuda"),
                      torch.tensor(starts, dtype=torch.int32, device="cuda"), out=out)
    gdn.device_check()
    check_rule(out, state, want, slots, starts, q, dk, max(lens))
    assert (out[starts[-1]:] == 5).all() and (out[starts[3]:starts[4]] == 0).all()


def test_recurrent_many_long_sequences():
    """More than 512 sequences of 16 tokens and more on average."""
    lens = [20, 0, 33] + [17] * 540
    slots = list(range(len(lens)))[::-1]
    q, k, v, al, be, state, starts = make_rule(47, lens, 1, 1, 16, 32, F)
    want = rule64(q, k, v, al, be, state, slots, starts, torch.zeros_like(v))
    o = gdn.recurrent_fwd(q, k, v, al, be, state, torch.tensor(slots, dtype=torch.int32, device="cuda"),
                          torch.tensor(starts, dtype=torch.int32, device="cuda"))
    gdn.device_check()
    check_rule(o, state, want, slots, starts, q, 16, max(lens))


@pytest.mark.parametrize("dk,dv,H", [(128, 128, 2), (16, 32, 2), (128, 128, 60)])
def test_recurrent_decays_of_any_size(dk, dv, H):
    """Decays of 0 and near it, and long runs of small ones: no product of theirs is divided by."""
    lens = [67, 13, 1, 1, 4]
    q, k, v, al, be, state, starts = make_rule(9, lens, 1, H, dk, dv, F)
    g = rng(10)
    pick = torch.tensor([0.0, 1e-38, 1e-30, 1e-12, 1e-6, 0.01, 0.5, 1.0], device="cuda")
    al = pick[torch.randint(0, 8, al.shape, device="cuda", generator=g)]
    al[starts[2]:starts[4]] = 0
    want = rule64(q, k, v, al, be, state, range(5), starts, torch.zeros_like(v))
    o = gdn.recurrent_fwd(q, k, v, al, be, state, None, torch.tensor(starts, dtype=torch.int32, device="cuda"))
    check_rule(o, state, want, range(5), starts, q, dk, max(lens))


def test_recurrent_equals_the_chunked_pass_and_takes_its_state():
    """A prompt through chunk_fwd, its final state written into the pool, then single tokens."""
    g, T, H = rng(5), 70, 2
    q, k, v, al, be, state, starts = make_rule(5, [T], H, H, 128, 128, F, pool=3)
    o_all, s_all = gdn.chunk_fwd(q[None].contiguous(), k[None].contiguous(), v[None].contiguous(), al[None], be[None], kernel="simt")
    n = T - 6
    part = lambda x: x[None, :n].contiguous()  # noqa: E731
    gdn.chunk_fwd(part(q), part(k), part(v), part(al), part(be), kernel="simt", S_T=state[1:2])
    slot = torch.tensor([1], dtype=torch.int32, device="cuda")
    for t in range(n, T):
        o = gdn.recurrent_fwd(q[t:t + 1], k[t:t + 1], v[t:t + 1], al[t:t + 1], be[t:t + 1], state, slot)
        assert (o[0] - o_all[0, t]).abs().max() <= 1e-4      # the fp32 kernels' own bar
    assert (state[1] - s_all[0]).abs().max() <= 1e-4


def test_recurrent_bad_slots_and_ranges_touch_nothing_and_are_reported():
    # the kernel compares every entry with the pool and the rows before it uses it
    q, k, v, al, be, state, _ = make_rule(6, [1, 1, 1, 1], 1, 2, 128, 128, pool=4)
    before = state.clone()
    for slots, cu, rows in (([3, 4, -2, 0], [0, 1, 2, 3, 4], (0, 3)), ([0, 1, 2, 3], [0, 1, 0, 5, 6], (0,)), ([0, 1, 2, 3], [-1, 1, 2, 2, 4], (1, 3))):
        state.copy_(before)
        out = torch.full((4, 2, 128), 5.0, device="cuda", dtype=BF)
        gdn.recurrent_fwd(q, k, v, al, be, state, torch.tensor(slots, dtype=torch.int32, device="cuda"),
                          torch.tensor(cu, dtype=torch.int32, device="cuda"), out=out)
        with pytest.raises(gdn.GDNError, match="out of bounds"):
            gdn.device_check()
        gdn.device_check()                                   # cleared
        live = [slots[i] for i in rows]
        for i in range(4):
            assert torch.equal(state[i], before[i]) == (i not in live), (slots, cu, i)


def test_recurrent_state_offsets_past_32_bits():
    """A pool of 8.6 GB whose last state lies past 2^31 elements."""
    H, P = 16, 8200
    q, k, v, al, be, small, starts = make_rule(7, [1, 2], H, H, 128, 128, pool=2)
    state = torch.zeros(P, H, 128, 128, device="cuda")
    state[P - 1], state[0] = small[0], small[1]
    want = rule64(q, k, v, al, be, small, [0, 1], starts, torch.zeros_like(v))
    o = gdn.recurrent_fwd(q, k, v, al, be, state, torch.tensor([P - 1, 0], dtype=torch.int32, device="cuda"),
                          torch.tensor(starts, dtype=torch.int32, device="cuda"))
    check_rule(o, torch.stack([state[P - 1], state[0]]), want, [0, 1], starts, q, 128, 2)
    assert not state[1:P - 1].any()


# ------------------------------------------------------------------ rows in 8 bits

def check_rows(q, scale, y):
    """y in 64 bits.  The scale: at most 32 numbers a thread and 10 exchanges in the sum of
    squares (half of whose error reaches the root) and under 8 roundings more: 32 u.  A step:
    half a step, and 127 times the value's and the scale's errors (silu's exponential: 2 ulp)."""
    top = y.abs().amax(-1)
    live = top / 127 >= 2.0 ** -126
    want = torch.where(live, top / 127, 0.0)
    assert ((scale.double() - want).abs() <= 32 * U * want).all(), float(((scale.double() - want).abs() / want.clamp(min=1e-300)).max() / U)
    steps = torch.where(live[..., None], y / want.clamp(min=1e-300)[..., None], 0.0)
    assert ((q.double() - steps).abs() <= 0.5 + 127 * 80 * U).all(), float((q.double() - steps).abs().max())
    assert (q[..., :].abs().amax(-1)[live] == 127).all()


def rows_x(seed, shape, io, scale=1.0):
    g = rng(seed)
    x = randn(g, *shape) * scale
    x[..., 0] *= 20
    return x.to(io)


SHAPES = [(1, 1), (3, 7), (1, 8), (5, 1001), (2, 2048), (33, 64), (4, 4104), (2, 8192), (3, 16001), (2, 32768), (1, 32767)]


@pytest.mark.parametrize("io", [BF, F])
@pytest.mark.parametrize("shape", SHAPES)
def test_quantize(shape, io):
    x = rows_x(10, shape, io)
    q, scale = gdn.quantize_int8(x)
    assert q.shape == x.shape and q.dtype == torch.int8 and scale.shape == shape[:1]
    assert q.stride(0) % 16 == 0
    check_rows(q, scale, x.double())


@pytest.mark.parametrize("io,res,wt", [(BF, BF, F), (BF, F, BF), (F, F, F), (F, BF, None), (BF, None, BF), (F, None, F)])
@pytest.mark.parametrize("shape", SHAPES)
def test_norm(shape, io, res, wt):
    D, eps = shape[1], 1e-5
    x = rows_x(11, shape, io)
    r = None if res is None else rows_x(12, shape, res, 3.0)
    w = None if wt is None else (1 + 0.2 * randn(rng(13), D)).to(wt)
    q, scale, h = gdn.add_rms_norm_int8(x, w, r, eps=eps)
    full = x.float() if r is None else x.float() + r.float()
    if r is None:
        assert h is None
    else:
        assert h.dtype == res and torch.equal(h, full.to(res))     # one sum, one rounding
    y = full.double() / (full.double().pow(2).mean(-1, keepdim=True) + eps).sqrt()
    check_rows(q, scale, y if w is None else y * w.double())


@pytest.mark.parametrize("inplace", ["residual", "x"])
@pytest.mark.parametrize("D", [2048, 1001])
def test_norm_in_place(D, inplace):
    x, r = rows_x(14, (6, D), BF), rows_x(15, (6, D), BF)
    q0, s0, h0 = gdn.add_rms_norm_int8(x, None, r)
    x2, r2 = x.clone(), r.clone()
    q1, s1, h1 = gdn.add_rms_norm_int8(x2, None, r2, residual_out=r2 if inplace == "residual" else x2)
    assert h1 is (r2 if inplace == "residual" else x2)
    assert torch.equal(q0, q1) and torch.equal(s0, s1) and torch.equal(h0, h1)


@pytest.mark.parametrize("io", [BF, F])
@pytest.mark.parametrize("rows,H,d,packed", [(1, 1, 8, False), (3, 16, 128, True), (61, 5, 96, True), (7, 32, 64, False),
                                             (2, 3, 256, True), (4, 9, 40, False), (2, 128, 256, False), (2, 1024, 32, False)])
def test_gated(rows, H, d, packed, io):
    g = rng(16)
    x = (0.2 * randn(g, rows, H, d)).to(io)
    gate = randn(g, rows, (3 if packed else 1) * H * d + (8 if packed else 0)).to(io)[:, -H * d:].unflatten(1, (H, d))
    w = 1 + 0.2 * randn(g, d)
    q, scale = gdn.gated_rms_norm_int8(x, gate, w, eps=1e-6)
    assert q.shape == (rows, H * d) and scale.shape == (rows,)
    xd, gd = x.double(), gate.double()
    y = xd / (xd.pow(2).mean(-1, keepdim=True) + 1e-6).sqrt() * w.double() * gd * torch.sigmoid(gd)
    check_rows(q, scale, y.flatten(1))


def test_gated_unaligned_gate():
    g = rng(17)
    x, gate = randn(g, 5, 4, 32).to(BF), randn(g, 5, 129).to(BF)[:, 1:].unflatten(1, (4, 32))
    q, scale = gdn.gated_rms_norm_int8(x, gate)
    q2, scale2 = gdn.gated_rms_norm_int8(x, gate.contiguous())
    assert torch.equal(q, q2) and torch.equal(scale, scale2)


@pytest.mark.parametrize("D", [64, 1001])
def test_rows_of_zeros_tiny_and_not_finite(D):
    x = rows_x(18, (8, D), F)
    x[1] = 0
    x[2] *= 1e-39 / x[2].abs().max()              # a scale below 2^-126
    x[3] *= 1e-36 / x[3].abs().max()              # a small scale that is not
    x[4, D // 2] = math.inf
    x[5, D - 1] = math.nan
    x[6] *= 3e38 / x[6].abs().max()
    x[7] = -0.0
    q, scale = gdn.quantize_int8(x)
    bad = torch.tensor([4, 5], device="cuda")
    assert scale[bad].isnan().all() and not q[bad].any()
    assert (scale[[1, 2, 7]] == 0).all() and not q[[1, 2, 7]].any()
    good = torch.tensor([0, 1, 2, 3, 6, 7], device="cuda")
    check_rows(q[good], scale[good], x[good].double())
    q, scale, _ = gdn.add_rms_norm_int8(x[:6])
    assert scale[bad].isnan().all() and not q[bad].any() and scale[1] == 0 and not q[1].any()
    y = x[:4].double()
    y = y / (y.pow(2).mean(-1, keepdim=True) + 1e-6).sqrt()
    check_rows(q[[0, 1, 3]], scale[[0, 1, 3]], y[[0, 1, 3]])


def test_rows_with_other_strides_and_dimensions():
    g = rng(19)
    wide = randn(g, 6, 3, 300).to(BF)
    for x in (wide[:, 1, :200], wide[:, :, :77], wide[:, 2, 3:103], wide[2, 1], wide[:0, 0]):
        q, scale = gdn.quantize_int8(x)
        assert q.shape == x.shape and scale.shape == x.shape[:-1]
        if x.numel():
            check_rows(q, scale, x.double())
        q2, scale2, _ = gdn.add_rms_norm_int8(x)
        assert q2.shape == x.shape


def test_rows_past_32_bits():
    """More than 2^31 numbers; the rows on both sides of that border and the last."""
    R, D = 66001, 32768
    x = torch.empty(R, D, device="cuda", dtype=BF)
    x[0::2] = 1.0
    x[1::2] = -3.0
    some = [0, 65535, 65536, 65537, R - 1]
    for i in some:
        x[i] = rows_x(50 + i, (1, D), BF)[0]
    q, scale = gdn.quantize_int8(x)
    check_rows(q[some], scale[some], x[some].double())
    assert (q[2] == 127).all() and (q[R - 2] == -127).all()


# ------------------------------------------------------------------ int8_matmul

def check_product(out, x, xs, w, ws, bias, rows=None):
    """The sum is exact; then the sum's conversion, two products and the bias's sum round:
    4 u, and half a step of the output's type."""
    acc = x.double() @ w.double().t()
    y = acc * xs.double().reshape(-1)[:, None] * ws.double()
    mag = y.abs()
    if bias is not None:
        y = y + bias.double()
        mag = mag + bias.double().abs()
    tol = 4 * U * mag * 1.01 + (HALF[out.dtype] * y.abs() * 1.01 if out.dtype == BF else 0)
    assert ((out.double() - y).abs() <= tol).all(), float(((out.double() - y).abs() - tol).max())


def make_product(seed, M, N, K, pad=True, bias=False):
    g = rng(seed)
    width = (K + 15) // 16 * 16 if pad else K
    make = lambda r: torch.full((r, width), 99, dtype=torch.int8, device="cuda")[:, :K].copy_(  # noqa: E731
        torch.randint(-128, 128, (r, K), device="cuda", generator=g))
    return (make(M), torch.rand(M, device="cuda", generator=g) + 0.5, make(N), torch.rand(N, device="cuda", generator=g) * 0.01 + 0.001,
            randn(g, N) if bias else None)


@pytest.mark.parametrize("out_dtype", [BF, F])
@pytest.mark.parametrize("M,N,K", [(1, 1, 1), (1, 16, 16), (1, 129, 128), (2, 257, 2048), (16, 128, 127), (17, 300, 1537),
                                   (33, 1000, 129), (64, 513, 4096), (65, 128, 256), (127, 384, 640), (129, 257, 100),
                                   (200, 1001, 1000), (300, 130, 8192), (513, 2050, 320), (700, 8224, 272),
                                   (16, 8224, 2048), (9, 8192, 130), (2300, 2100, 130), (3001, 2900, 257), (4200, 4100, 300)])
def test_product(M, N, K, out_dtype):
    x, xs, w, ws, bias = make_product(20, M, N, K, bias=(M + N) % 2 == 0)
    out = gdn.int8_matmul(x, xs, w, ws, bias, out_dtype=out_dtype)
    gdn.device_check()
    assert out.shape == (M, N) and out.dtype == out_dtype
    check_product(out, x, xs, w, ws, bias)


@pytest.mark.parametrize("M,N,K", [(1, 3, 5), (5, 77, 333), (70, 130, 1537), (300, 500, 1)])
def test_product_of_unaligned_rows(M, N, K):
    x, xs, w, ws, bias = make_product(21, M, N, K, pad=False, bias=True)
    check_product(gdn.int8_matmul(x, xs, w, ws, bias, out_dtype=F), x, xs, w, ws, bias)
    x1, w1 = (torch.empty(t.shape[0], K + 17, dtype=torch.int8, device="cuda")[:, 1:K + 1].copy_(t) for t in (x, w))
    check_product(gdn.int8_matmul(x1, xs, w1, ws, bias, out_dtype=F), x, xs, w, ws, bias)
    wp = torch.zeros(N, (K + 15) // 16 * 16, dtype=torch.int8, device="cuda")[:, :K].copy_(w)
    check_product(gdn.int8_matmul(x1, xs, wp, ws, bias, out_dtype=F), x, xs, w, ws, bias)


def test_product_extremes_fill_32_bits():
    K = 131071
    x = torch.full((2, 131072), -128, dtype=torch.int8, device="cuda")[:, :K]
    w = torch.full((3, 131072), -128, dtype=torch.int8, device="cuda")[:, :K]
    w[1], w[2] = 127, 0
    one = lambda n: torch.ones(n, device="cuda")  # noqa: E731
    out = gdn.int8_matmul(x, one(2), w, one(3), out_dtype=F)
    want = torch.tensor([16384.0 * K, -16256.0 * K, 0.0], dtype=torch.float64, device="cuda")
    assert ((out.double() - want).abs() <= U * want.abs()).all()


def test_product_dimensions_output_and_rows_left_alone():
    x, xs, w, ws, bias = make_product(22, 6, 50, 64)
    whole = torch.full((8, 60), 3.0, device="cuda", dtype=BF)
    out = gdn.int8_matmul(x, xs, w, ws, out=whole[1:7, 4:54])
    check_product(out, x, xs, w, ws, None)
    mask = torch.ones_like(whole, dtype=torch.bool)
    mask[1:7, 4:54] = False
    assert (whole[mask] == 3).all()
    cube = gdn.int8_matmul(x.view(2, 3, 64), xs.view(2, 3), w, ws)
    assert torch.equal(cube.view(6, 50), out)
    row = gdn.int8_matmul(x[0], xs[0], w, ws)
    assert row.shape == (50,) and torch.equal(row, out[0])
    assert gdn.int8_matmul(x[:0], xs[:0], w, ws).shape == (0, 50)


def test_product_past_32_bits():
    """An output of more than 2^31 numbers."""
    M, N, K = 270001, 8192, 32
    x, xs, w, ws, _ = make_product(24, M, N, K)
    out = gdn.int8_matmul(x, xs, w, ws)
    gdn.device_check()
    for a in (0, 262143 - 128, M - 200):
        check_product(out[a:a + 200], x[a:a + 200], xs[a:a + 200], w, ws, None)


def test_product_of_rows_that_are_not_finite():
    x, xs, w, ws, _ = make_product(23, 3, 40, 64)
    xs[1] = math.nan
    out = gdn.int8_matmul(x, xs, w, ws)
    assert out[1].isnan().all() and not out[0].isnan().any() and not out[2].isnan().any()


# ------------------------------------------------------------------ together

def layer(hidden, residual, P, state, slots, cu):
    return bench.layer_step(P, hidden, residual.clone(), state, slots, cu)


def layer64(hidden, residual, P, state, slots, starts):
    """The same steps with the operators' definitions in 64 bits, rounded where the layer rounds."""
    H, d = P["H"], P["d"]

    def rows(y):
        s = y.abs().amax(-1, keepdim=True) / 127
        return torch.where(s > 0, (y / s.clamp(min=1e-300)).round(), 0.0), s

    def product(q, s, w, ws):
        return ((q @ w.double().t()) * s * ws.double()).to(BF)
    h = hidden.double() + residual.double()
    q, s = rows(h / (h.pow(2).mean(-1, keepdim=True) + 1e-6).sqrt() * P["norm"].double())
    row = product(q, s, *P["w_in"])
    q, k, v, gate, ab = row.split([H * d] * 4 + [2 * H], dim=1)
    q, k, v, gate = (t.unflatten(1, (H, d)) for t in (q, k, v, gate))
    alpha = torch.exp(-torch.nn.functional.softplus(ab[:, :H].float() - 4))
    beta = torch.sigmoid(ab[:, H:].float())
    o, pool, _ = rule64(q, k, v, alpha, beta, state, slots, starts, torch.zeros(q.shape, device="cuda"), 1e-6)
    o = o.to(BF).double()
    y = o / (o.pow(2).mean(-1, keepdim=True) + 1e-6).sqrt() * P["head"].double() * gate.double() * torch.sigmoid(gate.double())
    return product(*rows(y.flatten(1)), *P["w_out"]), h.to(residual.dtype), pool


def make_layer(seed=30):
    return bench.layer_weights(4, 128, 512, torch.device("cuda"), seed), rng(seed)


def test_layer_of_all_operators():
    """The five operators as they are used.  Both sides round the same values at the same
    places, except where a value lies within the other side's error of a tie: such a flip is
    one step of 8 bits (1/127 of its row's largest) or of bf16 in one of K inputs.  Flips
    touch a share of about 127 * 2 * 40 u of the values (6e-4 of them), each of size 1/127 of
    the largest, so the outputs agree to well under 2 steps of bf16 at the output's scale
    (2^-6 of its rms; the flips' own part is sqrt(6e-4) / 127 * 4 = 8e-4)."""
    P, g = make_layer()
    lens, slots = [3, 1, 0, 2, 1], [2, 0, 5, -1, 4]
    starts = [0, 3, 4, 4, 6, 7]
    hidden, residual, state = randn(g, 7, 512).to(BF), randn(g, 7, 512), 0.05 * randn(g, 6, 4, 128, 128)
    want, want_res, want_pool = layer64(hidden, residual, P, state.clone(), slots, starts)
    got, got_res = layer(hidden, residual, P, state, torch.tensor(slots, dtype=torch.int32, device="cuda"),
                         torch.tensor(starts, dtype=torch.int32, device="cuda"))
    gdn.device_check()
    assert torch.equal(got_res, want_res)
    rms = want.double().pow(2).mean().sqrt()
    assert (got.double() - want.double()).pow(2).mean().sqrt() <= 2.0 ** -6 * rms
    assert (state.double() - want_pool).pow(2).mean().sqrt() <= 2.0 ** -6 * want_pool.pow(2).mean().sqrt()


def test_layer_captured_replayed_and_on_another_stream():
    P, g = make_layer()
    hidden, residual = randn(g, 9, 512).to(BF), randn(g, 9, 512)
    start = 0.05 * randn(g, 9, 4, 128, 128)
    state = start.clone()
    want = [layer(hidden, residual, P, state, None, None) for _ in range(3)]
    after = state.clone()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        state.copy_(start)
        graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        out, res = layer(hidden, residual, P, state, None, None)
    state.copy_(start)
    for o, r in want:
        graph.replay()
        assert torch.equal(out, o) and torch.equal(res, r)
    assert torch.equal(state, after)


def test_calls_on_a_given_stream():
    x, xs, w, ws, bias = make_product(31, 40, 70, 33, pad=False)      # with a workspace
    q, k, v, al, be, state, starts = make_rule(32, [1] * 3, 1, 2, 64, 64)
    a, r = rows_x(33, (5, 256), BF), rows_x(34, (5, 256), BF)
    s0 = state.clone()
    plain = [gdn.int8_matmul(x, xs, w, ws), gdn.recurrent_fwd(q, k, v, al, be, s0), *gdn.quantize_int8(a),
             *gdn.add_rms_norm_int8(a, None, r), *gdn.gated_rms_norm_int8(a.view(5, 2, 128), r.view(5, 2, 128))]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    other = [gdn.int8_matmul(x, xs, w, ws, stream=side), gdn.recurrent_fwd(q, k, v, al, be, state, stream=side),
             *gdn.quantize_int8(a, stream=side), *gdn.add_rms_norm_int8(a, None, r, stream=side),
             *gdn.gated_rms_norm_int8(a.view(5, 2, 128), r.view(5, 2, 128), stream=side)]
    side.synchronize()
    for x, y in zip(plain, other):
        assert torch.equal(x, y)
    assert torch.equal(s0, state)


def test_the_same_call_twice_gives_the_same_bits():
    x, xs, w, ws, bias = make_product(35, 20, 600, 4096)
    one = gdn.int8_matmul(x, xs, w, ws, out_dtype=F)
    assert all(torch.equal(one, gdn.int8_matmul(x, xs, w, ws, out_dtype=F)) for _ in range(3))


def test_small_calls_back_to_back_wait_for_one_another():
    """Small launches begin before the one ahead has ended, and wait for it: the same bits as with
    the device idle between calls, in place, with buffers that each call reads and the next writes."""
    P, g = make_layer(37)
    first = randn(g, 3, 512).to(BF), randn(g, 3, 512), 0.05 * randn(g, 3, 4, 128, 128)
    wq, ws = gdn.quantize_int8(randn(g, 512, 511) / 512 ** 0.5)
    wq = wq.contiguous()                                         # rows off 16 bytes: copied in each call

    def run(wait):
        hidden, residual, state = (t.clone() for t in first)
        out, o = torch.empty(3, 512, device="cuda", dtype=BF), torch.empty(3, 4, 128, device="cuda", dtype=BF)
        for i in range(60):
            x, xs, _ = gdn.add_rms_norm_int8(hidden, P["norm"], residual, residual_out=residual)
            wait()
            row = gdn.int8_matmul(x, xs, *P["w_in"])
            wait()
            q, k, v, gate = (row[:, 512 * j:512 * (j + 1)].unflatten(1, (4, 128)) for j in range(4))
            gdn.recurrent_fwd(q, k, v, None, None, state, qk_norm_eps=1e-6, out=o)
            wait()
            y, ys = gdn.gated_rms_norm_int8(o, gate, P["head"])
            wait()
            gdn.int8_matmul(y, ys, *P["w_out"], out=out)
            wait()
            z, zs = gdn.quantize_int8(out[:, :511])
            wait()
            gdn.int8_matmul(z, zs, wq, ws, out=hidden)           # what the next round's norm reads
            wait()
        return hidden, residual, state

    want = run(torch.cuda.synchronize)
    for _ in range(5):
        assert all(torch.equal(a, b) for a, b in zip(run(lambda: None), want))
    assert all(t.isfinite().all() for t in want)
    gdn.device_check()


def test_product_with_copies_captured_twice():
    """Two graphs of one stream, each with copies of unaligned rows: they share no workspace."""
    a, b = make_product(36, 30, 70, 333, pad=False), make_product(37, 50, 90, 555, pad=False)
    want = [gdn.int8_matmul(*t[:4], out_dtype=F) for t in (a, b)]
    torch.cuda.synchronize()
    graphs, outs = [], []
    for t in (a, b):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(gdn.int8_matmul(*t[:4], out_dtype=F))
        graphs.append(g)
    s = [torch.cuda.Stream() for _ in graphs]
    for _ in range(5):
        for g, st in zip(graphs, s):
            with torch.cuda.stream(st):
                g.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(x, y) for x, y in zip(outs, want))


def test_calls_from_threads_on_their_own_streams():
    import threading
    P, g = make_layer()
    hidden, residual, start = randn(g, 6, 512).to(BF), randn(g, 6, 512), 0.05 * randn(g, 6, 4, 128, 128)
    s0 = start.clone()
    want = [layer(hidden, residual, P, s0, None, None) for _ in range(4)]
    torch.cuda.synchronize()
    errors = []

    def work():
        try:
            with torch.cuda.stream(torch.cuda.Stream()):
                state = start.clone()
                for o, r in want:
                    got = layer(hidden, residual, P, state, None, None)
                    assert torch.equal(got[0], o) and torch.equal(got[1], r)
                assert torch.equal(state, s0)
        except BaseException as e:      # noqa: B902 - handed to the test's own thread
            errors.append(e)
    threads = [threading.Thread(target=work) for _ in range(4)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    gdn.device_check()
    assert not errors, errors


def test_recurrent_gives_the_same_bits_alone_and_in_a_batch():
    """A sequence's result does not depend on its neighbours or its place."""
    lens = [5, 9, 1, 4]
    q, k, v, al, be, state, starts = make_rule(43, lens, 2, 4, 128, 128, BF)
    s0 = state.clone()
    o = gdn.recurrent_fwd(q, k, v, al, be, s0, None, torch.tensor(starts, dtype=torch.int32, device="cuda"))
    for i in range(4):
        a, e = starts[i], starts[i + 1]
        s1 = state[i:i + 1].clone()
        o1 = gdn.recurrent_fwd(q[a:e], k[a:e], v[a:e], al[a:e], be[a:e], s1, None, torch.tensor([0, e - a], dtype=torch.int32, device="cuda"))
        assert torch.equal(o1, o[a:e]) and torch.equal(s1[0], s0[i])


@pytest.mark.parametrize("quick", [True, False])
def test_both_ways_to_the_library(quick, monkeypatch):
    """Calls of every operator through the quick binding and without it."""
    import chunked_gated_delta_14_b200.layer as L
    from chunked_gated_delta_14_b200 import _layer
    gdn.quantize_int8(torch.ones(1, 8, device="cuda"))
    assert L._quick is _layer
    calls = []
    if quick:      # a call of the usual form does not reach the long way
        monkeypatch.setattr(L, "_launch", lambda *a: calls.append(a))
    else:
        monkeypatch.setattr(L, "_quick", L._NoQuick)
    a, r = rows_x(60, (5, 256), BF), rows_x(61, (5, 256), F)
    w = 1 + 0.1 * randn(rng(62), 256)
    check_rows(*gdn.quantize_int8(a), a.double())
    q, s, h = gdn.add_rms_norm_int8(a, w.to(BF), r, residual_out=r)
    assert h is r
    y = r.double()
    check_rows(q, s, y / (y.pow(2).mean(-1, keepdim=True) + 1e-6).sqrt() * w.to(BF).double())
    x, gate = a.view(5, 4, 64).double(), a.view(5, 4, 64).double()
    y = x / (x.pow(2).mean(-1, keepdim=True) + 1e-6).sqrt() * w[:64].double() * gate * torch.sigmoid(gate)
    check_rows(*gdn.gated_rms_norm_int8(a.view(5, 4, 64), a.view(5, 4, 64), w[:64]), y.flatten(1))
    for pad in (True, False):
        x, xs, wq, ws, bias = make_product(63, 9, 70, 130, pad=pad, bias=True)
        out = torch.empty(9, 70, device="cuda")
        assert gdn.int8_matmul(x, xs, wq, ws, bias, out_dtype=F, out=out) is out
        check_product(out, x, xs, wq, ws, bias)
        check_product(gdn.int8_matmul(x, xs, wq, ws, bias), x, xs, wq, ws, bias)
    lens, slots = [3, 0, 2], [1, 0, -1]
    q, k, v, al, be, state, starts = make_rule(64, lens, 1, 2, 64, 64, BF, packed=True)
    want = rule64(q, k, v, al, be, state, slots, starts, torch.zeros_like(v))
    o = gdn.recurrent_fwd(q, k, v, al, be, state, torch.tensor(slots, dtype=torch.int32, device="cuda"),
                          torch.tensor(starts, dtype=torch.int32, device="cuda"), o_dtype=F)
    assert o.dtype == F
    check_rule(o, state, want, slots, starts, q, 64, 3)
    with pytest.raises(gdn.GDNError, match="eps"):
        gdn.add_rms_norm_int8(a, eps=0.0)
    with pytest.raises(ValueError):
        gdn.int8_matmul(x, xs, wq[:, 1:], ws)
    gdn.device_check()
    assert not calls


def test_nothing_is_recorded_for_gradients_and_leaves_are_refused():
    x = randn(rng(44), 4, 64).requires_grad_()
    with pytest.raises(ValueError, match="gradient"):
        gdn.quantize_int8(x)
    with torch.no_grad():
        q, scale = gdn.quantize_int8(x)
        w = torch.nn.Parameter(torch.ones(64, device="cuda"))
        gdn.add_rms_norm_int8(x, w, x)
    assert not scale.requires_grad


def test_bench_line_of_the_layer(capsys):
    import json
    import types
    from test_bench_host import CONTRACT
    bench.run_decode_layer(types.SimpleNamespace(steps=3, warmup=3, e2e_steps=1, batch=4), 0, 1, 0)
    line = json.loads(capsys.readouterr().out.strip().splitlines()[-1])
    assert all(k in line for k in CONTRACT) and line["value"] > 0 and line["e2e"]["value"] > 0
