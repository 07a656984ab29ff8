"""Refusals of the 8-bit quantiser and product, the gate's gradient and the weight's
gradient: every bad argument is turned down on the host, before any launch."""
import ctypes

import pytest

E = pytest.importorskip("hashed_gram_conditional_amd")


def _gpu_visible():
    try:
        import torch
        return torch.cuda.device_count() > 0
    except Exception:
        return False


pytestmark = pytest.mark.skipif(_gpu_visible(), reason="fake device pointers: host-only test")

P = 0x10000        # aligned, never dereferenced on the host
BIG = 1 << 40


def _status(name, *args):
    return getattr(E.LIB, name)(*args)


QUANT = dict(src_type=E.F32, rows=4, cols=64, src_ld=0, out_cols=64, kind=E.SCALE_F32)


def _quantize(src=P, codes=P, scales=P, values=None, **kw):
    a = {**QUANT, **kw}
    return _status("engram_quantize_i8", src, a["src_type"], a["rows"], a["cols"], a["src_ld"],
                   a["out_cols"], a["kind"], codes, scales, values, None)


@pytest.mark.parametrize("kw,status", [
    (dict(src_type=E.I8), E.EINVAL), (dict(src_type=-1), E.EINVAL), (dict(kind=2), E.EINVAL),
    (dict(kind=-1), E.EINVAL), (dict(rows=-1), E.ESHAPE), (dict(rows=1 << 31), E.ESHAPE),
    (dict(cols=0), E.ESHAPE), (dict(cols=65), E.ESHAPE), (dict(out_cols=72), E.ESHAPE),
    (dict(out_cols=(1 << 20) + 16), E.ESHAPE), (dict(src_ld=63), E.ESHAPE), (dict(src_ld=1 << 31), E.ESHAPE),
    (dict(src_ld=-64), E.ESHAPE), (dict(rows=(1 << 31) - 1, out_cols=1 << 20), E.ESHAPE),
    (dict(src=None), E.EINVAL), (dict(codes=None), E.EINVAL), (dict(scales=None), E.EINVAL),
    (dict(src=P + 8), E.EINVAL), (dict(codes=P + 8), E.EINVAL), (dict(scales=P + 4), E.EINVAL),
    (dict(values=P + 8), E.EINVAL)])
def test_quantiser_refusals(kw, status):
    assert _quantize(**kw) == status
    assert _quantize(rows=0, src=None, codes=None, scales=None) == E.OK


SHAPES = [
    (dict(tokens=-1), E.ESHAPE), (dict(tokens=1 << 31), E.ESHAPE), (dict(in_dim=0), E.ESHAPE),
    (dict(in_dim=8), E.ESHAPE), (dict(in_dim=24), E.ESHAPE), (dict(in_dim=-16), E.ESHAPE),
    (dict(in_dim=E.MAX_I8_IN_DIM + 16), E.ESHAPE), (dict(out_dim=0), E.ESHAPE), (dict(out_dim=12), E.ESHAPE),
    (dict(out_dim=-8), E.ESHAPE), (dict(out_dim=1 << 31), E.ESHAPE),
    (dict(tokens=(1 << 31) - 1, out_dim=1 << 20), E.ESHAPE)]


def _project(ptrs=(P, P, P, P, P), ws=None, size=0, kv_type=E.BF16, tokens=4, in_dim=256, out_dim=64):
    return _status("engram_project_i8", *ptrs, kv_type, tokens, in_dim, out_dim, ws, size, None)


def _weight_grad(ptrs=(P, P, P, P), ws=None, size=0, grad_type=E.F32, accumulate=0, tokens=4, in_dim=256,
                 out_dim=64):
    return _status("engram_project_grad", *ptrs, grad_type, accumulate, tokens, in_dim, out_dim, ws, size,
                   None)


@pytest.mark.parametrize("kw,status", SHAPES)
def test_products_refuse_shapes(kw, status):
    assert _project(**kw) == status
    assert _weight_grad(**kw) == status
    assert E.engram_project_i8_workspace_size(*[kw.get(n, d) for n, d in (("tokens", 4), ("in_dim", 256),
                                                                          ("out_dim", 64))]) == 0
    assert E.engram_project_grad_workspace_size(*[kw.get(n, d) for n, d in (("tokens", 4), ("in_dim", 256),
                                                                            ("out_dim", 64))]) == 0


def test_weight_gradient_refuses_sizes_beyond_its_offsets():
    assert _weight_grad(out_dim=E.MAX_GRAD_OUT_DIM + 8, in_dim=16) == E.ESHAPE
    assert _weight_grad(tokens=E.MAX_GRAD_TOKENS + 1, in_dim=16, out_dim=8) == E.ESHAPE
    assert E.engram_project_grad_workspace_size(E.MAX_GRAD_TOKENS + 1, 16, 8) == 0


def test_products_refuse_types_pointers_and_workspaces():
    for t in (E.I8, -1):
        assert _project(kv_type=t) == E.EINVAL
        assert _weight_grad(grad_type=t) == E.EINVAL
    for acc in (-1, 2):
        assert _weight_grad(accumulate=acc) == E.EINVAL
    for bad in (None, P + 8):
        for k in range(5):
            ptrs = [P] * 5
            ptrs[k] = bad
            assert _project(ptrs) == E.EINVAL
        for k in range(4):
            ptrs = [P] * 4
            ptrs[k] = bad
            assert _weight_grad(ptrs) == E.EINVAL
    assert _project(ws=P + 64, size=BIG) == E.EWORKSPACE
    assert _weight_grad(ws=P + 64, size=BIG) == E.EWORKSPACE
    assert _project([None] * 5, tokens=0) == E.OK
    # no tokens: nothing to add, but zeros to write
    assert _weight_grad([None] * 4, tokens=0, accumulate=1) == E.OK
    assert _weight_grad([P, P, P, None], tokens=0) == E.EINVAL


def test_fine_gradients_are_the_weight_gradients_alone():
    assert _weight_grad([None] * 4, tokens=0, accumulate=1, grad_type=E.F32_FINE) == E.OK
    assert _weight_grad([P, P, P, None], tokens=0, grad_type=E.F32_FINE) == E.EINVAL
    assert _weight_grad(grad_type=E.F32_FINE + 1) == E.EINVAL
    assert _project(kv_type=E.F32_FINE) == E.EINVAL
    assert _quantize(src_type=E.F32_FINE) == E.EINVAL
    assert _gate(saved=_saved(kv_type=E.F32_FINE)) == E.EINVAL
    assert _gate(saved=_saved(h_type=E.F32_FINE)) == E.EINVAL
    for kw in (dict(table_type=E.F32_FINE), dict(out_type=E.F32_FINE)):
        d = E.embed_desc(10, 4, 16, **kw)
        assert _status("engram_embed", ctypes.byref(d), P, P, P, None) == E.EINVAL


def _desc(**kw):
    base = dict(batch=1, seq=4, hc=4, dim=64, table_rows=0, row_format=E.ROW_E4M3_E8M0_264, row_dim=256)
    base.update(kw)
    return E.forward_desc(**base)


def _saved(kv=P, kv_type=E.I8, kv_scales=P, h=P, h_type=E.I8, h_scales=P):
    return E.gate_saved(kv, kv_type, kv_scales, h, h_type, h_scales)


GATE = dict(ids=P, raw_vocab=100, q_w=P, k_w=P, d_out=P, d_h=P, d_kv=P, d_q_w=P, d_k_w=P, accumulate=0, ws=P,
            size=BIG)


def _gate(desc=None, saved=None, **kw):
    a = {**GATE, **kw}
    d = _desc() if desc is None else desc
    s = _saved() if saved is None else saved
    return _status("engram_gate_grad", ctypes.byref(d), a["ids"], a["raw_vocab"], ctypes.byref(s), a["q_w"],
                   a["k_w"], a["d_out"], a["d_h"], a["d_kv"], a["d_q_w"], a["d_k_w"], a["accumulate"], a["ws"],
                   a["size"], None)


@pytest.mark.parametrize("kw,status", [
    (dict(batch=-1), E.ESHAPE), (dict(seq=1 << 31), E.ESHAPE), (dict(hc=0), E.ESHAPE), (dict(hc=9), E.ESHAPE),
    (dict(dim=0), E.ESHAPE), (dict(dim=12), E.ESHAPE), (dict(dim=8200), E.ESHAPE),
    (dict(row_format=2), E.EINVAL), (dict(eps=-1.0), E.EINVAL), (dict(eps=float("nan")), E.EINVAL),
    (dict(gate_clamp=-1.0), E.EINVAL), (dict(gate_mode=2), E.EINVAL)])
def test_gate_gradient_refuses_a_bad_description(kw, status):
    assert _gate(_desc(**kw)) == status
    assert E.engram_gate_grad_workspace_size(_desc(**kw)) == 0


def test_gate_gradient_refuses_arguments():
    d = _desc()
    size = E.engram_gate_grad_workspace_size(d)
    assert size > 0
    assert _status("engram_gate_grad", None, P, 100, P, P, P, P, P, P, P, P, 0, P, BIG, None) == E.EINVAL
    assert _status("engram_gate_grad", ctypes.byref(d), P, 100, None, P, P, P, P, P, P, P, 0, P, BIG,
                   None) == E.EINVAL
    assert _gate(raw_vocab=0) == E.EINVAL
    for acc in (-1, 2):
        assert _gate(accumulate=acc) == E.EINVAL
    for name in ("ids", "q_w", "k_w", "d_out", "d_h", "d_kv"):
        for bad in (None, P + 2):
            assert _gate(**{name: bad}) == E.EINVAL
    for name in ("d_q_w", "d_k_w"):
        for bad in (None, P + 4):
            assert _gate(**{name: bad}) == E.EINVAL
    for ws, n in ((None, BIG), (P + 128, BIG), (P, size - 1)):
        assert _gate(ws=ws, size=n) == E.EWORKSPACE
    # a type that is neither the layer's own nor 8-bit codes; codes without scales
    for s in (_saved(kv_type=E.F32), _saved(h_type=E.F32), _saved(kv_type=3), _saved(h_type=-1),
              _saved(kv_scales=None), _saved(h_scales=None), _saved(kv_scales=P + 2), _saved(h_scales=P + 2),
              _saved(kv=None), _saved(h=None), _saved(kv=P + 8), _saved(h=P + 8)):
        assert _gate(saved=s) == E.EINVAL
    f32 = _desc(row_format=E.ROW_F32, row_dim=32)
    assert _gate(f32, _saved(kv_type=E.BF16)) == E.EINVAL
    assert _gate(f32, _saved(h_type=E.BF16)) == E.EINVAL


def test_gate_gradient_workspace_sizes():
    last = 0
    for seq in (0, 1, 100, 32768):
        size = E.engram_gate_grad_workspace_size(_desc(seq=seq))
        assert size >= last
        last = size
    assert E.engram_gate_grad_workspace_size(_desc(seq=1)) >= 4 * 64 * 4


def test_struct_layout_matches():
    assert E.LIB.engram_sizeof_gate_saved() == ctypes.sizeof(E.GateSaved)
