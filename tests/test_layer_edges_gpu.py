"""Decode-layer operators on the GPU where their kernels change over: every head size in every
variant, ties, the ends of the numbers' range, batches around a sequence, sizes near 2^31,
overlapping rows, captures over two streams.

Tolerances are those of test_layer_gpu.py, derived there beside each check.
"""
import math

import pytest
import torch

import chunked_gated_delta_14_b200 as gdn
from test_layer_gpu import BF, F, U, check_product, check_rows, check_rule, make_product, make_rule, randn, rng, rows_x, rule64

pytestmark = pytest.mark.gpu


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def off16(x):
    """The same numbers in rows and heads that start off 16 bytes."""
    return torch.empty(x.shape[0], x.shape[1], x.shape[2] + 1, device="cuda", dtype=x.dtype)[..., 1:].copy_(x)


# the variants that a batch's lengths choose: short sequences, long ones, long ones of whole heads by two column quads
LENGTHS = {"short": [2, 3, 4, 5, 6, 7, 8, 9, 1, 0], "long": [40, 17, 2, 1, 33, 9, 0, 24, 23, 21],
           "two quads": [40, 17, 2, 1, 33, 9, 0, 24, 23, 21] * 8}


@pytest.mark.parametrize("io", [BF, F])
@pytest.mark.parametrize("aligned", [True, False])
@pytest.mark.parametrize("lengths,dk,dv", [(n, dk, dv) for n in LENGTHS for dk in (16, 32, 64, 128) for dv in (32, 64, 96, 128)
                                           if n != "two quads" or dv == 128])
def test_recurrent_every_size_in_every_variant(lengths, dk, dv, aligned, io):
    lens = LENGTHS[lengths]
    H = 4 if lengths == "two quads" else 2
    q, k, v, al, be, state, starts = make_rule(70, lens, 2, H, dk, dv, io)
    assert (lengths == "short") == (starts[-1] < 16 * len(lens))
    S = range(len(lens))
    want = rule64(q, k, v, al, be, state, S, starts, torch.zeros_like(v))
    o = gdn.recurrent_fwd(*((q, k, v) if aligned else map(off16, (q, k, v))), al, be, state, None, i32(starts))
    gdn.device_check()
    check_rule(o, state, want, S, starts, q, dk, max(lens))


@pytest.mark.parametrize("io", [BF, F])
@pytest.mark.parametrize("D,pitch,off", [(1001, 1001, 0), (77, 79, 1), (2049, 2051, 3), (16001, 16001, 0), (2048, 2049, 1)])
def test_norm_in_place_of_rows_off_16_bytes(D, pitch, off, io):
    """The pieces that a thread reads hold numbers that its neighbours overwrite."""
    g = rng(82)
    make = lambda: randn(g, 300 * pitch + off).to(io)[off:].view(300, pitch)[:, :D]  # noqa: E731
    x, r = make(), make()
    want = gdn.add_rms_norm_int8(x.clone(), None, r.clone())
    for place in (r, x):
        keep = place.clone()
        for _ in range(3):
            place.copy_(keep)
            got = gdn.add_rms_norm_int8(x, None, r, residual_out=place)
            assert got[2] is place and all(torch.equal(a, b) for a, b in zip(got, want))
        place.copy_(keep)


@pytest.mark.parametrize("out_dtype", [BF, F])
@pytest.mark.parametrize("M,N,K", [(40, 7, 64), (64, 17, 4096), (130, 9, 130), (200, 2001, 512), (128, 2008, 128), (100, 1001, 2048),
                                   (257, 8221, 256), (1030, 4099, 640), (500, 33, 100), (2100, 2050, 128)])
def test_product_of_channels_that_end_inside_a_warp(M, N, K, out_dtype):
    """Several loads of the accumulator behind stores of some lanes, in tiles of every kind; what
    lies behind the channels is left as it was."""
    x, xs, w, ws, bias = make_product(83, M, N, K, bias=True)
    out = torch.full((M + 1, N + 3), 7.0, device="cuda", dtype=out_dtype)
    gdn.int8_matmul(x, xs, w, ws, bias, out_dtype=out_dtype, out=out[:M, :N])
    gdn.device_check()
    check_product(out[:M, :N], x, xs, w, ws, bias)
    assert (out[M] == 7).all() and (out[:, N:] == 7).all()


def test_rows_as_many_as_the_arguments_hold():
    """2^31 - 1 rows, in blocks of four: the last block's rows pass 2^31."""
    R = 2 ** 31 - 1
    q, scale = gdn.quantize_int8(torch.full((1, 1), -3.0, device="cuda").expand(R, 1))
    assert q.shape == (R, 1) and (q == -127).all()
    assert (scale == scale[0]).all() and scale[0] == 3.0 / 127
    del q, scale
    torch.cuda.empty_cache()


BIG = [1e18, 1e19, 1e25, 1e30, 1e38, 3e38]


@pytest.mark.parametrize("io", [BF, F])
@pytest.mark.parametrize("res", [None, BF, F])
@pytest.mark.parametrize("D", [8, 64, 300, 1001, 2048, 8192, 20001])
def test_norm_of_rows_whose_squares_pass_32_bits(D, res, io):
    x = rows_x(74, (len(BIG) + 2, D), F)
    x *= torch.tensor(BIG + [1.0, 1e20], device="cuda")[:, None] / x.abs().amax(1, keepdim=True)
    x[len(BIG) + 1, 1:] *= 1e-15
    x = x.to(io)
    r = None if res is None else (x.float() * -0.25).to(res)
    w = 1 + 0.2 * randn(rng(75), D)
    w /= w.abs().max()            # |h w| stays in range where |h| does
    q, scale, h = gdn.add_rms_norm_int8(x, w, r)
    full = (x.float() if r is None else x.float() + r.float()).double()
    assert full.abs().max() < 3.3e38
    check_rows(q, scale, full / (full.pow(2).mean(-1, keepdim=True) + 1e-6).sqrt() * w.double())


def test_norm_of_rows_past_the_range_have_scale_nan():
    x = torch.full((2, 64), 3e38, device="cuda")
    q, scale, _ = gdn.add_rms_norm_int8(x, torch.full((64,), 2.0, device="cuda"))
    assert scale.isnan().all() and not q.any()
    q, scale, h = gdn.add_rms_norm_int8(x, None, x)
    assert scale.isnan().all() and not q.any() and h.isinf().all()
    x = torch.zeros(2, 64, device="cuda")
    x[:, 5] = 1.0                                    # y = 8 w there
    q, scale, _ = gdn.add_rms_norm_int8(x, torch.full((64,), 1e38, device="cuda"))
    assert scale.isnan().all() and not q.any()


@pytest.mark.parametrize("io", [BF, F])
@pytest.mark.parametrize("H,d", [(1, 8), (3, 40), (16, 128), (5, 96), (128, 256)])
def test_gated_of_heads_whose_squares_pass_32_bits(H, d, io):
    g = rng(76)
    x = randn(g, len(BIG) + 1, H, d)
    x *= torch.tensor(BIG + [1.0], device="cuda")[:, None, None] / x.abs().amax((1, 2), keepdim=True)
    if H > 1:
        x[:, 1] *= 1e-17
    x, gate, w = x.to(io), randn(g, len(BIG) + 1, H, d).to(io), 1 + 0.2 * randn(g, d)
    q, scale = gdn.gated_rms_norm_int8(x, gate, w)
    xd, gd = x.double(), gate.double()
    y = xd / (xd.pow(2).mean(-1, keepdim=True) + 1e-6).sqrt() * w.double() * gd * torch.sigmoid(gd)
    check_rows(q, scale, y.flatten(1))


@pytest.mark.parametrize("width", [64, 1001, 2048, 9000])
def test_quantize_rounds_ties_to_even(width):
    """Of rows in bf16 many numbers are a tie (half the row's largest is 63.5 steps): each step is
    the definition's, rint(127 y / top).  In 64 bits 127 y is exact and so is a quotient that is a tie."""
    g = rng(73)
    R = 1024
    top = (1 + torch.arange(R, device="cuda") % 128 / 128) * 2.0 ** (torch.arange(R, device="cuda") // 128 * 30 - 100)
    x = (2 * torch.rand(R, width, device="cuda", generator=g) - 1) * top[:, None]
    x[:, 1::3] = top[:, None] / 2 ** torch.randint(0, 8, (R, width), device="cuda", generator=g)[:, 1::3]
    x = x.to(BF)
    x[:, 0], x[:, width // 2] = top.to(BF), -top.to(BF) / 2
    q, scale = gdn.quantize_int8(x)
    y = x.double()
    t = y.abs().amax(1, keepdim=True)
    want = (127 * y / t).round()
    assert torch.equal(q.double(), want)
    assert torch.equal(scale, (t[:, 0] / 127).float())           # rounded correctly: the quotient in 64 bits is far from a tie
    q, scale, _ = gdn.add_rms_norm_int8(x[512:])                  # the same ratios, and so the same steps
    assert torch.equal(q.double(), want[512:])


def test_quantize_of_fp32_takes_the_nearest_step():
    """y (f - over): the product's rounding and the sum's, 2^-18 of a step and half a step; ties as they are."""
    g = rng(86)
    x = randn(g, 2000, 1001)
    x[:, 7] = x.abs().amax(1) / 2
    q, scale = gdn.quantize_int8(x)
    t = x.double().abs().amax(1, keepdim=True)
    y = 127 * x.double() / t
    assert ((q.double() - y).abs() <= 0.5 + 2 ** -18).all()
    half = y[:, 7] == 63.5                                        # not where column 7 was the largest itself
    assert half.sum() > 1900 and (q[half, 7] == 64).all()
    assert torch.equal(scale, (t[:, 0] / 127).float())


@pytest.mark.parametrize("io", [BF, F])
@pytest.mark.parametrize("dk,dv,Hk,H", [(128, 128, 2, 4), (16, 64, 1, 4), (32, 96, 2, 2), (64, 32, 1, 2), (16, 128, 4, 4)])
def test_recurrent_gives_the_same_bits_whatever_is_beside_a_sequence(dk, dv, Hk, H, io):
    """Alone, in a batch of short sequences, beside long ones, and in one of so many that its
    blocks take whole heads; a single token without offsets too."""
    mine = [1, 2, 3, 4, 5, 8, 13, 31, 1]
    batches = [mine, mine + [2] * 40, mine + [300], [90, 0] + mine, mine + [40] * 90]
    q, k, v, al, be, state, starts = make_rule(71, mine, Hk, H, dk, dv, io)
    got = []
    for lens in batches:
        at = next(i for i in range(len(lens)) if lens[i:i + len(mine)] == mine)
        Q, K, V, A, B, s, st = make_rule(72, lens, Hk, H, dk, dv, io)
        a, e = st[at], st[at + len(mine)]
        for x, y in ((Q, q), (K, k), (V, v), (A, al), (B, be)):
            x[a:e] = y
        s[at:at + len(mine)] = state
        o = gdn.recurrent_fwd(Q, K, V, A, B, s, None, i32(st), qk_norm_eps=1e-6)
        got.append((o[a:e].clone(), s[at:at + len(mine)].clone()))
    for i, n in enumerate(mine):
        a, e = starts[i], starts[i + 1]
        s = state[i:i + 1].clone()
        o = gdn.recurrent_fwd(q[a:e], k[a:e], v[a:e], al[a:e], be[a:e], s, None, i32([0, n]), qk_norm_eps=1e-6)
        if n == 1:
            s1 = state[i:i + 1].clone()
            o1 = gdn.recurrent_fwd(q[a:e], k[a:e], v[a:e], al[a:e], be[a:e], s1, qk_norm_eps=1e-6)
            assert torch.equal(o, o1) and torch.equal(s, s1)
            P = 320 // H                                         # enough that a block takes more columns
            s2 = state[i:i + 1].repeat(P, 1, 1, 1)
            o2 = gdn.recurrent_fwd(*(x[a:e].repeat(P, *[1] * (x.dim() - 1)) for x in (q, k, v, al, be)), s2, qk_norm_eps=1e-6)
            assert torch.equal(o2, o.repeat(P, 1, 1)) and torch.equal(s2, s.repeat(P, 1, 1, 1))
        for j, (go, gs) in enumerate(got):
            assert torch.equal(go[a:e], o) and torch.equal(gs[i], s[0]), (n, j)


def test_other_threads_run_while_a_call_waits(tmp_path):
    """The quick binding over functions that wait 0.3 s, as a launch into a full queue does: Python's
    lock is free meanwhile."""
    import ctypes
    import subprocess
    import threading
    import time
    from chunked_gated_delta_14_b200 import _layer
    (tmp_path / "wait.c").write_text("#include <unistd.h>\nint waits(const void *a, void *s) { usleep(300000); return 1; }\n"
                                     "unsigned long long none(const void *a) { return 0; }\n")
    subprocess.check_call(["gcc", "-shared", "-fPIC", str(tmp_path / "wait.c"), "-o", str(tmp_path / "wait.so")])
    so = ctypes.CDLL(str(tmp_path / "wait.so"))
    at = lambda f: ctypes.cast(f, ctypes.c_void_p).value  # noqa: E731
    x, i8, s = torch.ones(4, 64, device="cuda"), torch.ones(4, 64, device="cuda", dtype=torch.int8), torch.ones(4, device="cuda")
    q, state = x.view(4, 1, 64), torch.zeros(4, 1, 64, 64, device="cuda")
    calls = [lambda: _layer.quantize_int8(x), lambda: _layer.add_rms_norm_int8(x, None, x, 1e-6, None),
             lambda: _layer.gated_rms_norm_int8(x.view(4, 2, 32), x.view(4, 2, 32), None, 1e-6),
             lambda: _layer.int8_matmul(i8, s, i8, s, None, F, None),
             lambda: _layer.recurrent_fwd(q, q, q, None, None, state, None, None, None, None, None)]
    turns, done = [0], threading.Event()

    def turn():
        while not done.is_set():
            turns[0] += 1
            time.sleep(0.002)
    thread = threading.Thread(target=turn)
    thread.start()
    try:
        _layer.bind(at(so.waits), at(so.waits), at(so.waits), at(so.none), gdn.abi_version())
        for call in calls:
            before = turns[0]
            assert call() == 1
            assert turns[0] - before > 20
    finally:
        done.set()
        thread.join()
        gdn.layer._bind_quick()
    assert type(_layer.quantize_int8(x)) is tuple
    gdn.device_check()


@pytest.mark.parametrize("quick", [True, False])
def test_rows_of_any_leading_dimensions(quick, monkeypatch):
    """One row, batches of rows, strides that are one run, dimensions of one, and rows that are not
    one run, through the quick binding and without it; the same numbers as of plain rows."""
    import chunked_gated_delta_14_b200.layer as L
    long_way = []
    if quick:
        launch = L._launch
        monkeypatch.setattr(L, "_launch", lambda *a: (long_way.append(a), launch(*a)))
    else:
        monkeypatch.setattr(L, "_quick", L._NoQuick)
    g = rng(87)
    wide = randn(g, 6, 4, 300)
    w = 1 + 0.1 * randn(g, 100)
    wq, ws = gdn.quantize_int8(randn(g, 40, 100))
    for io in (BF, F):
        for x in (wide[:, :, 3:103], wide[1, :, :100], wide[1, 2, 7:107], wide[:, None, 2:3, :100], wide[::2, 1:2, :100], wide[None, 3, 1:2, None, :100]):
            x = x.to(io) if x.is_contiguous() else torch.empty_strided(x.shape, x.stride(), device="cuda", dtype=io).copy_(x)
            flat = x.reshape(-1, 100).clone()
            lead = x.shape[:-1]
            for got, want in ((gdn.quantize_int8(x), gdn.quantize_int8(flat)),
                              (gdn.add_rms_norm_int8(x, w, x), gdn.add_rms_norm_int8(flat, w, flat)),
                              (gdn.add_rms_norm_int8(x, w, eps=1), gdn.add_rms_norm_int8(flat, w, eps=1.0))):
                assert got[0].shape == x.shape and got[1].shape == lead and got[0].stride(-1) == 1
                assert not lead or got[0].stride(-2) == 112 and got[0].data_ptr() % 16 == 0
                assert torch.equal(got[0].reshape(-1, 100), want[0]) and torch.equal(got[1].reshape(-1), want[1])
                if len(got) == 3 and want[2] is not None:
                    assert got[2].shape == x.shape and torch.equal(got[2].reshape(-1, 100), want[2])
            r = x.clone()
            q, s, h = gdn.add_rms_norm_int8(x, w, r, residual_out=r)
            assert h is r and torch.equal(h, (x + x)) and q.shape == x.shape
            out = gdn.int8_matmul(q, s, wq, ws, out_dtype=F)
            assert out.shape == (*lead, 40) and torch.equal(out.reshape(-1, 40), gdn.int8_matmul(q.reshape(-1, 100), s.reshape(-1), wq, ws, out_dtype=F))
            place = torch.full((*lead, 48), 5.0, device="cuda")[..., :40]
            assert gdn.int8_matmul(q, s, wq, ws, out_dtype=F, out=place) is place and torch.equal(place, out)
            if len(lead):
                y = x.unflatten(-1, (5, 20))[..., :16].contiguous()
                q, s = gdn.gated_rms_norm_int8(y, y)
                q2, s2 = gdn.gated_rms_norm_int8(y.view(-1, 5, 16), y.view(-1, 5, 16))
                assert q.shape == (*lead, 80) and torch.equal(q.reshape(-1, 80), q2) and torch.equal(s.reshape(-1), s2)
    gdn.gated_rms_norm_int8(randn(g, 3, 16), randn(g, 3, 16))
    assert not long_way
    for x in (wide[:, :3, :100], wide.transpose(0, 1)[..., :100]):         # not one run
        with pytest.raises(ValueError, match="one run"):
            gdn.quantize_int8(x)
    assert gdn.quantize_int8(wide[:0])[0].shape == (0, 4, 300)
    assert gdn.int8_matmul(wq.view(2, 20, 100)[:, :0], ws.view(2, 20)[:, :0], wq, ws).shape == (2, 0, 40)
    with pytest.raises(ValueError):
        gdn.add_rms_norm_int8(wide[0], None, wide[0, :3])
    with pytest.raises(gdn.GDNError, match="overlap"):
        gdn.add_rms_norm_int8(wide[:1].expand(3, 4, 300).reshape(12, 300)[:2], None, wide[0, :2].clone(),
                              residual_out=wide[5, 3:].expand(2, 300))
    gdn.device_check()


@pytest.mark.parametrize("quick", [True, False])
def test_tangents_are_refused_in_every_argument(quick, monkeypatch):
    import torch.autograd.forward_ad as fw
    import chunked_gated_delta_14_b200.layer as L
    if not quick:
        monkeypatch.setattr(L, "_quick", L._NoQuick)
    x, i8, s = torch.ones(4, 64, device="cuda"), torch.ones(4, 64, device="cuda", dtype=torch.int8), torch.ones(4, device="cuda")
    w, q, state, a = torch.ones(64, device="cuda"), x.view(4, 1, 64), torch.zeros(4, 1, 64, 64, device="cuda"), torch.ones(4, 1, device="cuda")
    calls = [(gdn.quantize_int8, [x]), (gdn.add_rms_norm_int8, [x, w, x]), (gdn.gated_rms_norm_int8, [x.view(4, 2, 32), x.view(4, 2, 32), w[:32]]),
             (gdn.int8_matmul, [i8, s, i8, s, s]), (gdn.recurrent_fwd, [q, q, q, a, a, state])]
    with fw.dual_level():
        for f, args in calls:
            for i, t in enumerate(args):
                if t.is_floating_point():
                    dual = fw.make_dual(t, torch.ones_like(t))
                    with torch.no_grad(), pytest.raises(ValueError, match="tangent"):
                        f(*args[:i], dual, *args[i + 1:])
            f(*args)                                 # the same without
    gdn.device_check()


@pytest.mark.parametrize("io", [BF, F])
@pytest.mark.parametrize("lo,hi,weight", [(-90, -80, 1.0), (-88.6, -87.4, 1.0), (-95, -86, 1e4), (-100, 100, 1e4), (60, 100, 1.0), (-3, 3, 1e-33)])
def test_gated_of_gates_far_below_zero(lo, hi, weight, io):
    """silu there is g e^g, small, but its rows have a scale.  The exponent is rounded once, to half
    of 2^-17 below 128, and its factor log2(e) is off by 0.23 u of it: 44 u + 21 u of the result; with
    the exponential's and the quotient's 2 units in the last place each and check_rows' 32 u: 110 u."""
    g = rng(88)
    x, gate = randn(g, 50, 4, 64).to(io), (lo + (hi - lo) * torch.rand(50, 4, 64, device="cuda", generator=g)).to(io)
    w = weight * (1 + 0.2 * randn(g, 64))
    q, scale = gdn.gated_rms_norm_int8(x, gate, w)
    xd, gd = x.double(), gate.double()
    y = (xd / (xd.pow(2).mean(-1, keepdim=True) + 1e-6).sqrt() * w.double() * gd * torch.sigmoid(gd)).flatten(1)
    want = y.abs().amax(1) / 127
    assert want.min() > 2.0 ** -126
    assert ((scale.double() - want).abs() <= 110 * U * want).all(), float(((scale.double() - want).abs() / want).max() / U)
    assert ((q.double() - y / want[:, None]).abs() <= 0.5 + 127 * 250 * U).all()
    assert (q.abs().amax(1) == 127).all()


@pytest.mark.parametrize("M,N,K,step", [(40, 30, 64, 16), (40, 30, 100, 48), (300, 200, 130, 32)])
def test_product_of_rows_that_overlap(M, N, K, step):
    g = rng(77)
    make = lambda r: torch.randint(-128, 128, ((r - 1) * step + K,), device="cuda", generator=g, dtype=torch.int8).as_strided((r, K), (step, 1))  # noqa: E731
    x, w = make(M), make(N)
    xs, ws = torch.rand(M, device="cuda", generator=g), torch.rand(N, device="cuda", generator=g)
    check_product(gdn.int8_matmul(x, xs, w, ws, out_dtype=F), x, xs, w, ws, None)


def test_captured_over_two_streams():
    """Operators on two streams of one capture, each launched right behind the other's event."""
    x, xs, w, ws, _ = make_product(78, 20, 512, 256)
    wu = w[:, 1:250]
    a, r = rows_x(79, (20, 512), BF), rows_x(80, (20, 512), F)
    q, k, v, al, be, state, starts = make_rule(81, [1] * 20, 2, 4, 64, 128)
    lens = i32(starts)
    s0 = state.clone()
    side = torch.cuda.Stream()

    def run(state):
        main = torch.cuda.current_stream()
        y = gdn.int8_matmul(x, xs, w, ws)
        side.wait_stream(main)
        with torch.cuda.stream(side):
            z, zs, h = gdn.add_rms_norm_int8(y, None, r)
            u = gdn.int8_matmul(z[:, :249], zs, wu[:, :249], ws)
        o = gdn.recurrent_fwd(q, k, v, al, be, state, None, lens)
        main.wait_stream(side)
        p, ps = gdn.gated_rms_norm_int8(o, u.view(20, 4, 128))
        side.wait_stream(main)
        with torch.cuda.stream(side):
            t, ts = gdn.quantize_int8(h)
        main.wait_stream(side)
        return gdn.int8_matmul(p, ps, t, ts, out_dtype=F), o, u
    want = run(s0)
    torch.cuda.synchronize()
    s1 = state.clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = run(s1)
    for _ in range(3):
        s1.copy_(state)
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want)) and torch.equal(s1, s0)
    gdn.device_check()


@pytest.mark.parametrize("quick", [True, False])
def test_eps_of_other_types(quick, monkeypatch):
    import chunked_gated_delta_14_b200.layer as L
    if not quick:
        monkeypatch.setattr(L, "_quick", L._NoQuick)
    x = randn(rng(89), 4, 64)
    q, state = x.view(4, 1, 64), torch.zeros(4, 1, 64, 64, device="cuda")
    for f in (lambda e: gdn.add_rms_norm_int8(x, eps=e), lambda e: gdn.gated_rms_norm_int8(q, q, eps=e),
              lambda e: gdn.recurrent_fwd(q, q, q, None, None, state, qk_norm_eps=e)):
        for eps in ("1e-6", [1.0]):
            with pytest.raises(TypeError):
                f(eps)
        for eps in (0, 0.0, -1, math.nan, 1e-60):
            with pytest.raises(gdn.GDNError, match="eps"):
                f(eps)
        for eps in (1, True, 1e60, 10 ** 400):
            try:
                f(eps)
            except OverflowError:
                assert eps == 10 ** 400
    gdn.device_check()
