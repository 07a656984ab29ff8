"""The 8-bit quantiser and the product of 8-bit codes against references.

The quantiser's codes and scales match the definition exactly, and its values are q s
rounded once. The product's sum is a whole number, exact in 32 bits; converting it to fp32
and the two multiplications round as numpy's float32 does, so the result is compared bit
for bit."""
import numpy as np
import pytest

from tests.gpu_util import say

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("no GPU", allow_module_level=True)

import hashed_gram_conditional_amd as E  # noqa: E402

DEV = "cuda"
TYPES = {E.BF16: torch.bfloat16, E.F32: torch.float32}
KINDS = [E.SCALE_F32, E.SCALE_POW2]


def bf16_round(x):
    """float32 array -> nearest bf16 as float32 (torch rounds to nearest even)."""
    return torch.from_numpy(np.ascontiguousarray(x, dtype=np.float32)).to(torch.bfloat16).float().numpy()


def bf16_once(x):
    """float64 -> nearest bf16 as float64, by its 8 leading bits (normal numbers only; a
    conversion by way of float32 would round twice)."""
    part, exp = np.frexp(x)
    return np.ldexp(np.rint(part * 256) / 256, exp)


def quantize_reference(x, out_cols, kind):
    """Codes, scales (float32) and exact values (float64) of float64 rows by the definition.
    x times an fp32 factor has at most 48 bits and is exact in float64."""
    rows, cols = x.shape
    codes = np.zeros((rows, out_cols), np.int64)
    scales = np.zeros(rows, np.float32)
    values = np.zeros((rows, cols))
    for r in range(rows):
        amax = np.abs(x[r]).max()
        if not np.isfinite(amax):
            scales[r] = np.nan
            values[r] = np.nan
            continue
        if amax < 2.0 ** -119:
            continue
        if kind == E.SCALE_POW2:
            e = int(np.floor(np.log2(amax))) - 8
            while 127 * 2.0 ** e < amax:
                e += 1
            s, by = 2.0 ** e, 2.0 ** -e
        else:
            s, by = np.float32(amax / 127), float(np.float32(127 / amax))
            if 127 * float(s) > float(np.finfo(np.float32).max):
                s = np.nextafter(s, np.float32(0))
        scales[r] = s
        codes[r, :cols] = np.rint(x[r] * by)
        if 64 * float(s) > float(np.finfo(np.float32).max):
            codes[r] = np.clip(codes[r], -63, 63)
        values[r] = codes[r, :cols] * float(s)
    return codes, scales, values


def quantize(src, cols, ld=0, out_cols=None, kind=E.SCALE_F32, values="new"):
    rows = src.shape[0]
    out_cols = -(-cols // 16) * 16 if out_cols is None else out_cols
    st = E.F32 if src.dtype == torch.float32 else E.BF16
    # a row and a value more, to see that they are left alone
    codes = torch.full((rows + 1, out_cols), 85, dtype=torch.int8, device=DEV)
    scales = torch.full((rows + 1,), 77.0, device=DEV)
    v = torch.full_like(src, 9.0) if isinstance(values, str) else values
    E.engram_quantize_i8(src, st, rows, cols, ld, out_cols, kind, codes, scales, v)
    torch.cuda.synchronize()
    assert (codes[rows] == 85).all() and scales[rows] == 77.0
    return codes[:rows], scales[:rows], v


def check_quantize(x, cols, ld=0, out_cols=None, kind=E.SCALE_F32):
    src = x.to(DEV)
    codes, scales, values = quantize(src, cols, ld, out_cols, kind)
    ec, es, ev = quantize_reference(x[:, :cols].double().numpy(), codes.shape[1], kind)
    np.testing.assert_array_equal(scales.cpu().numpy(), es)
    np.testing.assert_array_equal(codes.cpu().numpy(), ec)
    # q s has 8 + 24 bits: exact in float64, rounded once
    want = ev.astype(np.float32).astype(np.float64) if x.dtype == torch.float32 else bf16_once(ev)
    got = values.cpu().double().numpy()
    np.testing.assert_array_equal(got[:, :cols], want)
    assert (got[:, cols:] == 9.0).all()


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("st", [E.BF16, E.F32])
@pytest.mark.parametrize("rows,cols,ld,out_cols", [
    (1, 1, 0, 16), (1, 16, 0, 16), (3, 15, 0, 48), (5, 17, 24, 64), (7, 128, 0, 256), (2, 1001, 1003, 1024),
    (257, 96, 104, 96), (300, 64, 0, 64), (33, 6144, 0, 6144), (4, 1000, 1000, 1152), (130, 8, 0, 128),
    (5, 512, 0, 512), (6, 520, 0, 528), (3, 2048, 0, 2048), (3, 4104, 0, 4112), (2, 8192, 8195, 8192),
    (2, 8200, 0, 8208), (2, 20001, 0, 20016), (1, 131072, 0, 131072),
    (41, 63, 0, 64), (77, 100, 101, 112), (19, 127, 129, 128), (23, 250, 0, 256), (50, 255, 255, 256),
    (100, 511, 513, 512), (9, 1023, 0, 1024), (6, 2047, 2049, 2048), (5, 6143, 6143, 6144), (1000, 24, 26, 32)])
def test_quantize_against_the_definition(kind, st, rows, cols, ld, out_cols):
    say("quantize_i8", kind, st, rows, cols, ld, out_cols)
    g = torch.Generator().manual_seed(rows + cols)
    x = torch.randn((rows, ld or cols), generator=g) * torch.exp2(torch.randn((rows, 1), generator=g) * 8)
    check_quantize(x.to(TYPES[st]), cols, ld, out_cols, kind)


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("st", [E.BF16, E.F32])
def test_quantize_ties_and_every_exponent(kind, st):
    """The largest value fixes the scale; the others are halves of it, one step off them
    and zeros of both signs, for every exponent of fp32 down to the subnormal ones."""
    say("quantize_i8: ties at every exponent", kind, st)
    halves = np.arange(-127, 127) + 0.5
    rows = []
    for e in range(-149, 121):
        for top in (64.0, 127.0, 126.5, 100.0):
            for delta in (0.0, 2.0 ** -23, -2.0 ** -23):
                rows.append(np.concatenate([[top], halves * (1 + delta), [0.0, -0.0]]) * 2.0 ** e)
    with np.errstate(over="ignore"):
        x = torch.from_numpy(np.array(rows)).float().to(TYPES[st])
    assert torch.isfinite(x).all()
    check_quantize(x, x.shape[1], kind=kind)


@pytest.mark.parametrize("st", [E.BF16, E.F32])
def test_quantize_products_beside_a_half(st):
    """Values that the scale's factor takes onto, or to within one step of, a half."""
    say("quantize_i8: beside a half", st)
    rng = np.random.default_rng(7)
    rows = []
    for _ in range(400):
        amax = np.float32(rng.uniform(1, 2))
        if st == E.BF16:
            amax = bf16_round(np.array([amax]))[0]
        by = np.float32(127 / float(amax))
        near = ((np.arange(-126, 126) + 0.5) / float(by)).astype(np.float32)
        near = np.concatenate([near, np.nextafter(near, np.float32(9)), np.nextafter(near, np.float32(-9))])
        rows.append(np.concatenate([[amax], near]))
    check_quantize(torch.from_numpy(np.array(rows, dtype=np.float32)).to(TYPES[st]), len(rows[0]))


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("st", [E.BF16, E.F32])
def test_quantize_infinities_nan_zeros_and_the_largest(kind, st):
    say("quantize_i8: special rows", kind, st)
    big = torch.finfo(TYPES[st]).max
    x = torch.randn((12, 600), generator=torch.Generator().manual_seed(3))
    x[0, 599] = float("inf")
    x[1, 0] = float("-inf")
    x[2, 300] = float("nan")
    x[3] = 0.0
    x[4] = -0.0
    x[5, 7] = big
    x[6] = big
    x[7] = -big
    x[8] *= 1e-40
    x[9] = 0.0
    x[9, 5] = 2.0 ** -119
    x[10] = 0.0
    x[10, 5] = float(np.nextafter(np.float32(2.0 ** -119), np.float32(0))) if st == E.F32 else 2.0 ** -120
    x = x.to(TYPES[st])
    check_quantize(x, 600, kind=kind)


def test_quantize_in_place_and_without_values():
    say("quantize_i8: in place, without values")
    x = torch.randn((37, 704), generator=torch.Generator().manual_seed(5)).to(torch.bfloat16).to(DEV)
    codes, scales, values = quantize(x, 700, 704)
    only, s2, _ = quantize(x, 700, 704, values=None)
    assert torch.equal(codes, only) and torch.equal(scales, s2)
    y = x.clone()
    c3, s3, _ = quantize(y, 700, 704, values=y)
    assert torch.equal(c3, codes) and torch.equal(s3, scales)
    assert torch.equal(y[:, :700], values[:, :700]) and torch.equal(y[:, 700:], x[:, 700:])


def test_quantize_offsets_beyond_32_bits():
    say("quantize_i8: offsets beyond 2^31 elements")
    rows, ld = 70000, 32768
    src = torch.zeros((rows, ld), dtype=torch.bfloat16, device=DEV)
    g = torch.Generator(device=DEV).manual_seed(1)
    src[-3:] = torch.randn((3, ld), generator=g, device=DEV).to(torch.bfloat16)
    codes = torch.empty((rows, ld), dtype=torch.int8, device=DEV)
    scales = torch.empty(rows, device=DEV)
    E.engram_quantize_i8(src, E.BF16, rows, ld, 0, ld, E.SCALE_POW2, codes, scales)
    torch.cuda.synchronize()
    ec, es, _ = quantize_reference(src[-3:].double().cpu().numpy(), ld, E.SCALE_POW2)
    np.testing.assert_array_equal(codes[-3:].cpu().numpy(), ec)
    np.testing.assert_array_equal(scales[-3:].cpu().numpy(), es)
    assert int(codes[:-3].abs().max()) == 0 and float(scales[:-3].abs().max()) == 0.0


def test_quantize_more_rows_than_a_launch_has_waves():
    say("quantize_i8: many rows")
    for rows, cols in (((1 << 23) + 5, 16), ((1 << 21) + 3, 1040)):
        src = torch.zeros((rows, cols), dtype=torch.bfloat16, device=DEV)
        g = torch.Generator(device=DEV).manual_seed(2)
        src[-7:] = torch.randn((7, cols), generator=g, device=DEV).to(torch.bfloat16)
        codes, scales, values = quantize(src, cols)
        ec, es, ev = quantize_reference(src[-7:].double().cpu().numpy(), cols, E.SCALE_F32)
        np.testing.assert_array_equal(codes[-7:].cpu().numpy(), ec)
        np.testing.assert_array_equal(scales[-7:].cpu().numpy(), es)
        assert int(codes[:-7].abs().max()) == 0 and float(scales[:-7].abs().max()) == 0.0
        assert float(values[:-7].abs().max()) == 0.0


# ---- the product -------------------------------------------------------------------

def codes_of(rows, cols, seed, full=False):
    g = torch.Generator().manual_seed(seed)
    lo = -128 if full else -127
    return torch.randint(lo, 128, (rows, cols), generator=g, dtype=torch.int16).to(torch.int8)


def scales_of(n, seed):
    return torch.exp2(torch.randn(n, generator=torch.Generator().manual_seed(seed)) * 4)


def project(e, es, w, ws, kv_type, workspace=True):
    m, k = e.shape
    n = w.shape[0]
    kv = torch.full((m * n + 64,), 9.0, dtype=TYPES[kv_type], device=DEV)
    size = E.engram_project_i8_workspace_size(m, k, n) if workspace else 0
    buf = torch.full((size + 256,), 0xAB, dtype=torch.uint8, device=DEV) if size else None
    E.engram_project_i8(e, es, w, ws, kv, kv_type, m, k, n, buf, size)
    torch.cuda.synchronize()
    assert (kv[m * n:] == 9.0).all()
    if size:
        assert (buf[size:] == 0xAB).all()
    return kv[:m * n].reshape(m, n)


def project_reference(e, es, w, ws):
    """float32 results in the kernel's order of operations; sums below 2^31 are exact in
    float64."""
    sums = e.double().numpy() @ w.double().numpy().T
    with np.errstate(over="ignore", invalid="ignore"):
        return (sums.astype(np.float32) * ws.numpy()[None]) * es.numpy()[:, None]


def check_project(m, k, n, kv_type, seed=0, full=True):
    e, w = codes_of(m, k, seed, full), codes_of(n, k, seed + 1, full)
    es, ws = scales_of(m, seed + 2), scales_of(n, seed + 3)
    want = torch.from_numpy(project_reference(e, es, w, ws)).to(TYPES[kv_type])
    dev = [x.to(DEV) for x in (e, es, w, ws)]
    got = project(*dev, kv_type).cpu()
    assert torch.equal(got, want), (got.float() - want.float()).abs().max()
    assert torch.equal(project(*dev, kv_type, workspace=False).cpu(), want)


@pytest.mark.parametrize("kv_type", [E.BF16, E.F32])
@pytest.mark.parametrize("m,k,n", [
    (1, 16, 8), (1, 6144, 264), (2, 48, 24), (5, 112, 40), (17, 128, 64), (31, 144, 72), (33, 256, 136),
    (64, 272, 128), (65, 1040, 200), (100, 384, 520), (128, 512, 256), (129, 640, 264), (200, 6144, 320),
    (256, 1024, 1000), (257, 896, 776), (300, 2064, 1288), (513, 176, 2056), (1003, 768, 1032)])
def test_project_every_bit(m, k, n, kv_type):
    say("project_i8", m, k, n, kv_type)
    check_project(m, k, n, kv_type, seed=m + n)


@pytest.mark.parametrize("k", [16 * x for x in (1, 2, 7, 8, 9, 15, 16, 17, 23, 24, 25, 31, 33, 40, 47, 48, 49, 63,
                                               65, 97)])
@pytest.mark.parametrize("m,n", [(3, 72), (70, 200), (300, 328)])
def test_project_step_counts(m, n, k):
    say("project_i8: inputs", m, n, k)
    check_project(m, k, n, E.F32, seed=k)


@pytest.mark.parametrize("k", [16, 144, 400])
@pytest.mark.parametrize("m,n", [(1, 25600), (256, 25600), (600, 5120), (1003, 25600), (2048, 12288)])
def test_project_wide(m, n, k):
    say("project_i8: wide", m, n, k)
    e, w = codes_of(m, k, 1), codes_of(n, k, 2)
    es, ws = scales_of(m, 3), scales_of(n, 4)
    want = torch.from_numpy(project_reference(e, es, w, ws)).to(torch.bfloat16)
    got = project(*[x.to(DEV) for x in (e, es, w, ws)], E.BF16).cpu()
    assert torch.equal(got, want)


def test_project_largest_sums():
    """The largest in_dim with codes of -128 throughout: 2147221504, below 2^31."""
    say("project_i8: largest sums")
    k = E.MAX_I8_IN_DIM
    for m, n in ((3, 16), (130, 264)):
        e = torch.full((m, k), -128, dtype=torch.int8, device=DEV)
        w = torch.full((n, k), -128, dtype=torch.int8, device=DEV)
        one_m, one_n = torch.ones(m, device=DEV), torch.ones(n, device=DEV)
        got = project(e, one_m, w, one_n, E.F32)
        assert (got == float(np.float32(k * 16384))).all()
        w[::2] = 127
        got = project(e, one_m, w, one_n, E.F32)
        assert (got[:, ::2] == float(np.float32(-k * 128 * 127))).all()


def test_project_scales_that_are_not_finite():
    """A NaN row of either operand makes its outputs NaN and no other."""
    say("project_i8: NaN and zero scales")
    for m, n in ((5, 64), (300, 520)):
        e, w = codes_of(m, 144, 1).to(DEV), codes_of(n, 144, 2).to(DEV)
        es, ws = torch.ones(m, device=DEV), torch.ones(n, device=DEV)
        base = project(e, es, w, ws, E.F32)
        es[1], ws[7], es[2], ws[9] = float("nan"), float("nan"), 0.0, 0.0
        got = project(e, es, w, ws, E.F32)
        assert torch.isnan(got[1]).all() and torch.isnan(got[:, 7]).all()
        rest = torch.ones_like(got, dtype=torch.bool)
        rest[1], rest[:, 7] = False, False
        base[2], base[:, 9] = 0.0, 0.0
        assert torch.equal(got[rest], base[rest])


def test_project_offsets_beyond_32_bits():
    say("project_i8: offsets beyond 2^31")
    m, k, n = 90000, 32, 25600         # 2.3e9 outputs
    e, w = codes_of(m, k, 1).to(DEV), codes_of(n, k, 2).to(DEV)
    es, ws = scales_of(m, 3).to(DEV), scales_of(n, 4).to(DEV)
    kv = torch.empty((m, n), dtype=torch.bfloat16, device=DEV)
    E.engram_project_i8(e, es, w, ws, kv, E.BF16, m, k, n)
    torch.cuda.synchronize()
    for at in (0, 83885, 83886, 89999):
        want = project_reference(e[at:at + 1].cpu(), es[at:at + 1].cpu(), w.cpu(), ws.cpu())
        assert torch.equal(kv[at].cpu(), torch.from_numpy(want[0]).to(torch.bfloat16))
    del kv
    m, k, n = 32800, 66000 // 16 * 16, 16      # 2.16e9 codes
    e = torch.zeros((m, k), dtype=torch.int8, device=DEV)
    e[-2:] = codes_of(2, k, 5).to(DEV)
    w, ws, es = codes_of(n, k, 6).to(DEV), scales_of(n, 7).to(DEV), scales_of(m, 8).to(DEV)
    kv = torch.empty((m, n), dtype=torch.float32, device=DEV)
    E.engram_project_i8(e, es, w, ws, kv, E.F32, m, k, n)
    torch.cuda.synchronize()
    want = project_reference(e[-2:].cpu(), es[-2:].cpu(), w.cpu(), ws.cpu())
    assert np.array_equal(kv[-2:].cpu().numpy(), want) and float(kv[:-2].abs().max()) == 0.0


def test_project_on_streams_at_once_and_replayed():
    """Two calls on two streams with their own workspaces, then both captured and replayed
    with other inputs in the same buffers."""
    say("project_i8: streams and graphs")
    shapes = [(3, 2048, 776), (200, 1040, 1288)]
    data = []
    for i, (m, k, n) in enumerate(shapes):
        e, w = codes_of(m, k, 10 + i).to(DEV), codes_of(n, k, 20 + i).to(DEV)
        es, ws = scales_of(m, 30 + i).to(DEV), scales_of(n, 40 + i).to(DEV)
        size = E.engram_project_i8_workspace_size(m, k, n)
        data.append((e, es, w, ws, torch.empty((m, n), device=DEV),
                     torch.empty(max(size, 256), dtype=torch.uint8, device=DEV), size))

    def call(d):
        E.engram_project_i8(*d[:5], E.F32, d[0].shape[0], d[0].shape[1], d[2].shape[0], d[5], d[6])

    want = [project(*d[:4], E.F32) for d in data]
    streams = [torch.cuda.Stream() for _ in data]
    torch.cuda.synchronize()
    for _ in range(5):
        for s, d in zip(streams, data):
            with torch.cuda.stream(s):
                call(d)
    torch.cuda.synchronize()
    for d, x in zip(data, want):
        assert torch.equal(d[4], x)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        for d in data:
            call(d)
    for turn in range(4):
        for i, d in enumerate(data):
            d[0].copy_(codes_of(*d[0].shape, 100 * turn + i))
            d[4].fill_(-1.0)
        graph.replay()
        torch.cuda.synchronize()
        got = [d[4].clone() for d in data]
        for d, x in zip(data, got):
            assert torch.equal(project(*d[:4], E.F32), x)


def test_quantised_codes_feed_the_product():
    """bf16 activations and an fp32 weight quantised and multiplied: within the error that
    half a step of either operand makes."""
    say("quantize_i8 then project_i8")
    m, k, n = 70, 1000, 136
    g = torch.Generator().manual_seed(9)
    x = torch.randn((m, k), generator=g).to(torch.bfloat16)
    w = torch.randn((n, k), generator=g) * 0.02
    kp = 1008
    qe, se, ve = quantize(x.to(DEV), k, 0, kp)
    qw, sw, vw = quantize(w.to(DEV), k, 0, kp)
    kv = project(qe.contiguous(), se.contiguous(), qw.contiguous(), sw.contiguous(), E.F32).cpu().double()
    exact = x.double() @ w.double().t()
    de = 0.5 * se.cpu().double()[:, None] * (1 + 2.0 ** -20)
    dw = 0.5 * sw.cpu().double()[:, None] * (1 + 2.0 ** -20)
    bound = (x.double().abs().sum(1, keepdim=True) * dw.t() + de * w.double().abs().sum(1)[None]
             + k * de * dw.t() + 2.0 ** -22 * exact.abs())
    assert ((kv - exact).abs() <= bound).all()
