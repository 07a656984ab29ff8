"""Refusals of the scaled lookup, its gradient, the 4-bit quantiser and the 4-bit
product: every bad argument is turned down on the host, before any launch."""
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


def _desc(**kw):
    base = dict(table_rows=100, n_ids=10, dim=16, table_type=E.BF16, out_type=E.F32, scale=1.0)
    base.update(kw)
    return E.embed_desc(**base)


BAD_DESC = [
    (dict(table_rows=-1), E.ESHAPE), (dict(n_ids=-1), E.ESHAPE), (dict(dim=0), E.ESHAPE),
    (dict(dim=E.MAX_EMBED_DIM + 1), E.ESHAPE), (dict(table_type=2), E.EINVAL),
    (dict(out_type=-1), E.EINVAL), (dict(scale=float("nan")), E.EINVAL),
    (dict(scale=float("inf")), E.EINVAL), (dict(table_ld=15), E.ESHAPE), (dict(out_ld=15), E.ESHAPE),
    (dict(table_ld=1 << 31), E.ESHAPE), (dict(out_ld=-16), E.ESHAPE), (dict(n_ids=1 << 62), E.ESHAPE),
]


@pytest.mark.parametrize("kw,status", BAD_DESC)
def test_lookup_and_gradient_refuse_a_bad_description(kw, status):
    d = _desc(**kw)
    p = ctypes.byref(d)
    assert _status("engram_embed", p, P, P, P, None) == status
    assert _status("engram_embed_grad", p, P, P, P, P, P, P, BIG, None) == status
    assert _status("engram_embed_grad_dense", p, P, P, P, 0, P, BIG, None) == status
    assert E.engram_embed_grad_workspace_size(d) == 0


def test_lookup_refuses_bad_pointers():
    d = ctypes.byref(_desc())
    assert _status("engram_embed", None, P, P, P, None) == E.EINVAL
    for k in range(3):
        for bad in (None, P + 4):
            args = [P, P, P]
            args[k] = bad
            assert _status("engram_embed", d, *args, None) == E.EINVAL
    # a table address no device knows is refused as well
    assert _status("engram_embed", d, P, P, P, None) == E.EINVAL
    assert _status("engram_embed", ctypes.byref(_desc(n_ids=0)), None, None, None, None) == E.OK


def test_gradient_refuses_sizes_its_keys_cannot_hold():
    for kw in (dict(table_rows=2 ** 32 - 1), dict(n_ids=E.MAX_EMBED_GRAD_IDS + 1)):
        d = _desc(**kw)
        assert E.engram_embed_grad_workspace_size(d) == 0
        assert _status("engram_embed_grad", ctypes.byref(d), P, P, P, P, P, P, BIG, None) == E.ESHAPE
        assert _status("engram_embed_grad_dense", ctypes.byref(d), P, P, P, 0, P, BIG, None) == E.ESHAPE
    assert E.engram_embed_grad_workspace_size(_desc(table_rows=2 ** 32 - 2)) > 0


def test_gradient_refuses_bad_pointers_and_workspaces():
    d = _desc()
    p = ctypes.byref(d)
    size = E.engram_embed_grad_workspace_size(d)
    assert size > 0
    assert _status("engram_embed_grad", None, P, P, P, P, P, P, BIG, None) == E.EINVAL
    for k in range(5):
        for bad in (None, P + 4):
            args = [P] * 5
            args[k] = bad
            assert _status("engram_embed_grad", p, *args, P, size, None) == E.EINVAL
    for ws, n in ((None, size), (P + 128, size), (P, size - 1)):
        assert _status("engram_embed_grad", p, P, P, P, P, P, ws, n, None) == E.EWORKSPACE
        assert _status("engram_embed_grad_dense", p, P, P, P, 0, ws, n, None) == E.EWORKSPACE
    for k in range(3):
        args = [P] * 3
        args[k] = None
        assert _status("engram_embed_grad_dense", p, *args, 0, P, size, None) == E.EINVAL
    for acc in (-1, 2):
        assert _status("engram_embed_grad_dense", p, P, P, P, acc, P, size, None) == E.EINVAL
    # nothing to add, or no table: nothing to do
    assert _status("engram_embed_grad_dense", ctypes.byref(_desc(n_ids=0)), None, None, P, 1, None, 0, None) == E.OK
    assert _status("engram_embed_grad_dense", ctypes.byref(_desc(table_rows=0)), P, P, None, 0, None, 0, None) == E.OK


def test_workspace_sizes_grow_and_cover_small_calls():
    last = 0
    for n in (0, 1, 100, 16384, 16385, 100_000, E.MAX_EMBED_GRAD_IDS):
        size = E.engram_embed_grad_workspace_size(_desc(n_ids=n, dim=256))
        assert size > 0 and size >= last
        last = size


QUANT = dict(src_type=E.F32, rows=4, cols=64, src_ld=0, out_cols=64)


def _quantize(src=P, codes=P, scales=P, values=None, **kw):
    a = {**QUANT, **kw}
    return _status("engram_quantize_mx4", src, a["src_type"], a["rows"], a["cols"], a["src_ld"],
                   a["out_cols"], codes, scales, values, None)


@pytest.mark.parametrize("kw,status", [
    (dict(src_type=3), E.EINVAL), (dict(rows=-1), E.ESHAPE), (dict(rows=1 << 31), E.ESHAPE),
    (dict(cols=0), E.ESHAPE), (dict(cols=65), E.ESHAPE), (dict(out_cols=72), E.ESHAPE),
    (dict(out_cols=(1 << 20) + 32), E.ESHAPE), (dict(src_ld=63), E.ESHAPE), (dict(src_ld=1 << 31), E.ESHAPE),
    (dict(rows=(1 << 31) - 1, out_cols=1 << 20), E.ESHAPE), (dict(src=None), E.EINVAL),
    (dict(codes=None), E.EINVAL), (dict(scales=None), E.EINVAL), (dict(src=P + 8), E.EINVAL),
    (dict(codes=P + 8), E.EINVAL), (dict(scales=P + 2), E.EINVAL), (dict(values=P + 8), E.EINVAL)])
def test_quantiser_refusals(kw, status):
    assert _quantize(**kw) == status
    assert _quantize(rows=0, src=None, codes=None, scales=None) == E.OK


PROJ = dict(fmt=E.MX_E2M1, tokens=4, in_dim=256, out_dim=64)


def _project(ptrs=(P, P, P, P, P), ws=None, size=0, **kw):
    a = {**PROJ, **kw}
    return _status("engram_project_mx4", ptrs[0], ptrs[1], a["fmt"], ptrs[2], ptrs[3], ptrs[4],
                   a["tokens"], a["in_dim"], a["out_dim"], ws, size, None)


@pytest.mark.parametrize("kw,status", [
    (dict(fmt=2), E.EINVAL), (dict(tokens=-1), E.ESHAPE), (dict(tokens=1 << 31), E.ESHAPE),
    (dict(in_dim=0), E.ESHAPE), (dict(in_dim=64), E.ESHAPE), (dict(in_dim=192), E.ESHAPE),
    (dict(in_dim=(1 << 20) + 128), E.ESHAPE), (dict(out_dim=0), E.ESHAPE), (dict(out_dim=12), E.ESHAPE),
    (dict(out_dim=1 << 31), E.ESHAPE), (dict(tokens=(1 << 31) - 1, out_dim=1 << 20), E.ESHAPE)])
def test_product_refuses_shapes(kw, status):
    assert _project(**kw) == status


def test_product_refuses_pointers_and_small_workspaces():
    for k, off in enumerate((8, 2, 8, 2, 8)):
        for bad in (None, P + off):
            ptrs = [P] * 5
            ptrs[k] = bad
            assert _project(ptrs) == E.EINVAL
    assert _project(ws=P + 64, size=BIG) == E.EWORKSPACE
    assert _project([None] * 5, tokens=0) == E.OK
    assert E.engram_project_mx4_workspace_size(4, 100, 64, E.MX_E2M1) == 0
    assert E.engram_project_mx4_workspace_size(4, 256, 64, 7) == 0


def test_struct_layout_matches():
    assert E.LIB.engram_sizeof_embed_desc() == ctypes.sizeof(E.EmbedDesc)
