"""Decode-layer operators: what the host refuses, before any launch.  No GPU needed."""
import ctypes
import re

import pytest
import torch

import chunked_gated_delta_14_b200 as gdn
import chunked_gated_delta_14_b200.layer as L
from chunked_gated_delta_14_b200.gdn import GDN_ERR_ALIGNMENT, GDN_ERR_INVALID_ARG, GDN_ERR_UNSUPPORTED
from test_abi import _c_layout

G = 1 << 36                      # addresses far enough apart never to overlap
INV, UNS, ALI = GDN_ERR_INVALID_ARG, GDN_ERR_UNSUPPORTED, GDN_ERR_ALIGNMENT


@pytest.mark.parametrize("struct,mirror", [("gdn_recurrent_args", gdn.RecurrentArgs), ("gdn_rows_args", gdn.RowsArgs),
                                           ("gdn_int8_matmul_args", gdn.Int8MatmulArgs)])
def test_mirrors_match_the_c_structs(struct, mirror, tmp_path):
    names = [f[0] for f in mirror._fields_]
    size, offsets = _c_layout(struct, names, tmp_path)
    assert ctypes.sizeof(mirror) == size
    assert [getattr(mirror, n).offset for n in names] == offsets


def test_packed_bytes_are_the_struct():
    values = list(range(1, len(gdn.RecurrentArgs._fields_) + 1))
    a = gdn.RecurrentArgs(*values)
    assert L._pack_recurrent(*values) == bytes(a)


def refused(call, args, status):
    with pytest.raises(gdn.GDNError) as e:
        call(args)
    assert e.value.status == status and gdn.last_error()


def recurrent(**kw):
    base = dict(rows=10, seqs=3, H=4, Hk=2, dk=128, dv=128, pool=5, io_dtype=1, o_dtype=1, q=G, k=2 * G, v=3 * G,
                q_row=256, q_head=128, k_row=256, k_head=128, v_row=512, v_head=128, alpha=4 * G, beta=5 * G,
                alpha_row=4, beta_row=4, cu_seqlens=6 * G, slots=7 * G, state=8 * G, o=9 * G)
    base.update(kw)
    return gdn.RecurrentArgs(**base)


@pytest.mark.parametrize("kw,status", [
    (dict(rows=-1), INV), (dict(seqs=-1), INV), (dict(H=0), INV), (dict(Hk=3), INV), (dict(Hk=0), INV), (dict(dk=48), INV),
    (dict(dk=256), INV), (dict(dv=16), INV), (dict(dv=256), INV), (dict(pool=0), INV), (dict(io_dtype=2), INV),
    (dict(o_dtype=-1), INV), (dict(qk_norm=2), INV), (dict(qk_norm=1), INV), (dict(qk_norm=1, qk_eps=float("nan")), INV),
    (dict(cu_seqlens=None), INV), (dict(slots=None, pool=2), INV), (dict(q_row=-1), INV), (dict(beta_row=-4), INV),
    (dict(q=None), INV), (dict(o=None), INV), (dict(state=None), INV), (dict(state=8 * G + 4), ALI), (dict(q=G + 1), ALI),
    (dict(alpha=4 * G + 2), ALI), (dict(slots=7 * G + 2), ALI), (dict(o=9 * G + 1), ALI),
    (dict(o=G), INV), (dict(o=G + 100), INV), (dict(o=8 * G + 1000), INV), (dict(v=8 * G + 16), INV), (dict(slots=8 * G), INV),
    (dict(seqs=2 ** 31 - 1, H=4096, Hk=1), INV),
])
def test_recurrent_refusals(kw, status):
    refused(gdn.call_recurrent, recurrent(**kw), status)


def rows(**kw):
    base = dict(op=1, rows=4, width=64, x_dtype=1, residual_dtype=1, weight_dtype=0, eps=1e-6, x=G, residual=2 * G,
                weight=3 * G, x_row=64, residual_row=64, residual_out_row=64, q_row=64, residual_out=4 * G, q=5 * G, scale=6 * G)
    base.update(kw)
    return gdn.RowsArgs(**base)


GATED = dict(op=2, residual=None, residual_out=None, gate=2 * G, gate_row=64, head=32)
PLAIN = dict(op=0, residual=None, residual_out=None, weight=None)


@pytest.mark.parametrize("kw,status", [
    (dict(op=3), INV), (dict(op=-1), INV), (dict(rows=-1), INV), (dict(width=0), INV), (dict(width=32769), UNS),
    (dict(x_dtype=5), INV), (dict(residual_dtype=5), INV), (dict(weight_dtype=5), INV), (dict(eps=0.0), INV),
    (dict(eps=float("nan")), INV), (dict(gate=7 * G), INV), (dict(residual_out=None), INV), (dict(residual=None), INV),
    (dict(x=None), INV), (dict(q=None), INV), (dict(scale=None), INV), (dict(x_row=-1), INV), (dict(q_row=63), INV),
    (dict(residual_out_row=32), INV), (dict(x=G + 1), ALI), (dict(scale=6 * G + 2), ALI), (dict(q=G + 8), INV),
    (dict(scale=5 * G + 4), INV), (dict(residual_out=2 * G + 2), INV), (dict(residual_out=G, residual_dtype=0), INV),
    (dict(residual_out=G, residual_out_row=128), INV), (dict(residual_out=3 * G, weight=3 * G), INV),
    (dict(residual_out=5 * G), INV), ({**PLAIN, "weight": 3 * G}, INV), ({**PLAIN, "residual": 2 * G}, INV),
    ({**GATED, "gate": None}, INV), ({**GATED, "head": 0}, INV), ({**GATED, "head": 12}, INV), ({**GATED, "head": 264}, INV),
    ({**GATED, "head": 24}, INV), ({**GATED, "residual": 4 * G}, INV), ({**GATED, "q": 2 * G}, INV),
    ({**GATED, "head": 40, "width": 32000, "x_row": 32000, "gate_row": 32000, "q_row": 32000}, UNS),
])
def test_rows_refusals(kw, status):
    refused(gdn.call_rows, rows(**kw), status)


def product(**kw):
    base = dict(M=5, N=7, K=33, out_dtype=1, x=G, w=2 * G, x_row=48, w_row=48, out_row=7, x_scale=3 * G, w_scale=4 * G,
                bias=5 * G, out=6 * G)
    base.update(kw)
    return gdn.Int8MatmulArgs(**base)


@pytest.mark.parametrize("kw,status", [
    (dict(M=-1), INV), (dict(N=0), INV), (dict(K=0), INV), (dict(K=131072), UNS), (dict(out_dtype=2), INV), (dict(x_row=-16), INV),
    (dict(x=None), INV), (dict(w=None), INV), (dict(out=None), INV), (dict(x_scale=None), INV), (dict(w_scale=None), INV),
    (dict(out_row=6), INV), (dict(out=6 * G + 1), ALI), (dict(bias=5 * G + 2), ALI), (dict(x_scale=3 * G + 1), ALI),
    (dict(out=G + 32), INV), (dict(out=3 * G), INV), (dict(M=2 ** 31 - 1, N=2 ** 30, out_row=2 ** 30), INV),
    (dict(x=G + 1), INV),                                                        # needs a workspace
    (dict(x=G + 1, workspace=7 * G, workspace_bytes=5 * 48 - 1), INV),
    (dict(x=G + 1, workspace=7 * G + 8, workspace_bytes=5 * 48), ALI),
    (dict(x=G + 1, workspace=2 * G, workspace_bytes=5 * 48), INV), (dict(x=G + 1, workspace=6 * G, workspace_bytes=5 * 48), INV),
])
def test_product_refusals(kw, status):
    refused(gdn.call_int8_matmul, product(**kw), status)


def test_product_workspace():
    ws = gdn.int8_matmul_workspace_bytes
    assert ws(product()) == 0
    assert ws(product(x_row=33)) == 5 * 48 and ws(product(w=2 * G + 8)) == 7 * 48
    assert ws(product(x_row=0, w_row=40)) == 12 * 48
    assert ws(product(M=1, x_row=33)) == 0                # one row has no stride
    assert ws(product(K=0)) == 0 and re.search("K", gdn.last_error())


def test_calls_of_no_rows_launch_nothing():
    gdn.call_recurrent(recurrent(rows=0, q=None))
    gdn.call_recurrent(recurrent(seqs=0))
    gdn.call_rows(rows(rows=0, x=None))
    gdn.call_int8_matmul(product(M=0, x=None))


def test_null_args():
    for f in ("gdn_recurrent_fwd", "gdn_rows_int8", "gdn_int8_matmul"):
        assert getattr(gdn.lib(), f)(None, None) == INV


def test_python_refuses_host_tensors():
    x, s = torch.zeros(4, 64, dtype=torch.bfloat16), torch.zeros(4)
    i8 = torch.zeros(4, 64, dtype=torch.int8)
    calls = [lambda: gdn.quantize_int8(x), lambda: gdn.add_rms_norm_int8(x), lambda: gdn.int8_matmul(i8, s, i8, s),
             lambda: gdn.gated_rms_norm_int8(x.view(4, 2, 32), x.view(4, 2, 32)),
             lambda: gdn.recurrent_fwd(x.view(4, 1, 64), x.view(4, 1, 64), x.view(4, 1, 64), None, None, torch.zeros(4, 1, 64, 64))]
    for c in calls:
        with pytest.raises(ValueError):
            c()
    with pytest.raises(TypeError):
        gdn.quantize_int8([1.0])


class OnDevice(torch.Tensor):
    """A host tensor that says it is on a CUDA device: for the checks before a launch."""
    @staticmethod
    def __new__(cls, t):
        return torch.Tensor._make_subclass(cls, t, t.requires_grad)

    @property
    def device(self):
        return torch.device("cuda", 0)

    def get_device(self):
        return 0


def dev(*shape, dtype=torch.float32, grad=False):
    return OnDevice(torch.zeros(*shape, dtype=dtype).requires_grad_(grad))


BF = torch.bfloat16


@pytest.mark.parametrize("call,error", [
    (lambda: gdn.quantize_int8(dev(4, 64, dtype=torch.float16)), TypeError),
    (lambda: gdn.quantize_int8(dev(4, 64, grad=True)), ValueError),
    (lambda: gdn.quantize_int8(OnDevice(torch.zeros(64, 4).t())), ValueError),
    (lambda: gdn.quantize_int8(OnDevice(torch.zeros(4, 3, 64)[:, :2])), ValueError),
    (lambda: gdn.add_rms_norm_int8(dev(4, 64), dev(63)), ValueError),
    (lambda: gdn.add_rms_norm_int8(dev(4, 64), None, dev(4, 63)), ValueError),
    (lambda: gdn.add_rms_norm_int8(dev(4, 64), None, torch.zeros(4, 64)), ValueError),
    (lambda: gdn.add_rms_norm_int8(dev(4, 64), None, None, residual_out=dev(4, 64)), ValueError),
    (lambda: gdn.add_rms_norm_int8(dev(4, 64), None, dev(4, 64), residual_out=dev(4, 64, dtype=BF)), TypeError),
    (lambda: gdn.gated_rms_norm_int8(dev(4, 2, 32), dev(4, 2, 32, dtype=BF)), TypeError),
    (lambda: gdn.gated_rms_norm_int8(dev(4, 2, 32), dev(4, 2, 32), dev(64)), ValueError),
    (lambda: gdn.gated_rms_norm_int8(OnDevice(torch.zeros(4, 2, 64)[..., :32]), dev(4, 2, 32)), ValueError),
    (lambda: gdn.int8_matmul(dev(4, 64), dev(4), dev(8, 64, dtype=torch.int8), dev(8)), TypeError),
    (lambda: gdn.int8_matmul(dev(4, 64, dtype=torch.int8), dev(4), dev(8, 63, dtype=torch.int8), dev(8)), ValueError),
    (lambda: gdn.int8_matmul(dev(4, 64, dtype=torch.int8), dev(4, 1), dev(8, 64, dtype=torch.int8), dev(8)), ValueError),
    (lambda: gdn.int8_matmul(dev(4, 64, dtype=torch.int8), dev(4), dev(8, 64, dtype=torch.int8), dev(8), out=dev(4, 8)), TypeError),
    (lambda: gdn.recurrent_fwd(dev(4, 2, 64), dev(4, 2, 64), dev(4, 2, 64), dev(4, 1), None, dev(4, 2, 64, 64)), ValueError),
    (lambda: gdn.recurrent_fwd(dev(4, 2, 64), dev(4, 2, 64), dev(4, 2, 64), None, None, dev(4, 2, 64, 64, dtype=BF)), TypeError),
    (lambda: gdn.recurrent_fwd(dev(4, 2, 64), dev(4, 2, 64), dev(4, 2, 64), None, None,
                               OnDevice(torch.zeros(4, 2, 64, 64).transpose(0, 1).contiguous().transpose(0, 1))), ValueError),
    (lambda: gdn.recurrent_fwd(dev(4, 2, 64), dev(4, 2, 64), dev(4, 2, 64), None, None, dev(4, 2, 64, 64), dev(4)), TypeError),
    (lambda: gdn.recurrent_fwd(dev(4, 2, 64), dev(4, 2, 64), dev(4, 2, 64, grad=True), None, None, dev(4, 2, 64, 64)), ValueError),
])
def test_python_refusals(call, error):
    with pytest.raises(error):
        call()


def test_quick_binding_builds_and_leaves_other_calls_alone():
    """_layer.so is built beside the library, binds to its ABI only, and gives None for what is
    not a plain device tensor."""
    from chunked_gated_delta_14_b200 import build as gbuild
    gbuild.build_binding()
    from chunked_gated_delta_14_b200 import _layer
    assert L._bind_quick() is _layer
    with pytest.raises(RuntimeError):
        _layer.bind(0, 0, 0, 0, 1)
    x = torch.zeros(4, 64)
    for a in (x, dev(4, 64), [1.0], None):
        assert _layer.quantize_int8(a) is None
        assert _layer.add_rms_norm_int8(a, None, None, 1e-6, None) is None
        assert _layer.gated_rms_norm_int8(a, a, None, 1e-6) is None
        assert _layer.int8_matmul(a, a, a, a, None, torch.float32, None) is None
        assert _layer.recurrent_fwd(a, a, a, None, None, a, None, None, None, None, None) is None
    assert _layer.quantize_int8() is None and _layer.int8_matmul(x) is None
