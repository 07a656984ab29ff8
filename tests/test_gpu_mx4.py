"""The 4-bit block quantiser and the product with a 4-bit weight against 64-bit
references.

The quantiser's codes, scales and values match the formula exactly. The product of
codes is exact; its fp32 accumulation of K terms, each addition off by at most one
unit 2^-23 of the sum of magnitudes, plus the rounding to bf16 (2^-8):
|kv - exact| <= acc + 2^-8 (|exact| + acc) with acc = K 2^-23 sum|e w|.

With an E4M3 operand the instruction first adds the products of eight consecutive
inputs in fixed point, with the largest product's power of two 2^p as the leading
place and 2^(p - 13) as the last: measured with +L, -L and a small product 2^-k L in
one group of eight, the small one survives for k <= 13 and vanishes for k >= 14, and
survives always in another group. Cutting a product off there loses less than
2^(p - 13) <= 2^-13 of the group's largest product, and at most seven of the eight
are cut (the largest holds few enough bits): acc grows by 7 2^-13 sum over the groups
of the largest |e w|. E2M1 products span 2^-2 .. 2^5 and lose nothing.

Integer products whose sums stay below 2^24 are exact up to the bf16 rounding."""
import numpy as np
import pytest

from tests.gpu_util import say

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("no GPU", allow_module_level=True)

import hashed_gram_conditional_amd as E  # noqa: E402
from workloads import gen  # noqa: E402

DEV = "cuda"
TYPES = {E.BF16: torch.bfloat16, E.F32: torch.float32}
GRID = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])


def quantize_reference(x, out_cols):
    """Codes [rows, out_cols], E8M0 scales and values of float64 x by the definition:
    the nearest grid value, a tie to the even code."""
    rows, cols = x.shape
    pad = np.zeros((rows, out_cols))
    pad[:, :cols] = x
    blocks = pad.reshape(rows, -1, 32)
    top = np.abs(blocks).max(-1)
    bad = ~np.isfinite(top)
    safe = np.where(bad | (top == 0), 2.0 ** -149, top)
    exp = np.maximum(np.frexp(safe)[1] - 1 - 2, -127)
    scales = np.where(bad, 255, exp + 127).astype(np.uint8)
    with np.errstate(invalid="ignore"):
        y = np.abs(blocks) * 2.0 ** -exp[..., None].astype(np.float64)
        dist = np.abs(y[..., None] - GRID)
        near = dist.min(-1, keepdims=True)
        codes = np.where(dist == near, np.arange(8) % 2 * 10 + np.arange(8) / 8, 99).argmin(-1)
    sign = np.signbit(blocks)
    codes = np.where(bad[..., None], 0, codes + 8 * sign)
    values = np.where(bad[..., None], np.nan,
                      np.where(sign, -1.0, 1.0) * GRID[codes % 8] * 2.0 ** exp[..., None].astype(np.float64))
    return (codes.reshape(rows, -1).astype(np.uint8), scales.reshape(rows, -1),
            values.reshape(rows, -1)[:, :cols])


def quantize(src, cols, ld=0, out_cols=None, values="new"):
    rows = src.shape[0]
    out_cols = -(-cols // 32) * 32 if out_cols is None else out_cols
    st = E.F32 if src.dtype == torch.float32 else E.BF16
    codes = torch.full((rows, out_cols // 2), 0x55, dtype=torch.uint8, device=DEV)
    scales = torch.full((rows, out_cols // 32), 0x55, dtype=torch.uint8, device=DEV)
    v = torch.full_like(src, 9.0) if values == "new" else values
    E.engram_quantize_mx4(src, st, rows, cols, ld, out_cols, codes, scales, v)
    torch.cuda.synchronize()
    return codes, scales, v


def unpack(codes):
    c = codes.cpu().numpy()
    return np.stack((c & 15, c >> 4), -1).reshape(c.shape[0], -1)


def check_quantize(x, cols, ld=0, out_cols=None):
    src = x.to(DEV)
    codes, scales, values = quantize(src, cols, ld, out_cols)
    oc = codes.shape[1] * 2
    with np.errstate(over="ignore"):
        ec, es, ev = quantize_reference(x[:, :cols].double().numpy(), oc)
    assert np.array_equal(scales.cpu().numpy(), es)
    assert np.array_equal(unpack(codes), ec)
    got = values.cpu().double().numpy()
    np.testing.assert_array_equal(got[:, :cols], ev)
    assert np.array_equal(np.signbit(got[:, :cols])[np.isfinite(ev)], np.signbit(ev)[np.isfinite(ev)])
    assert (got[:, cols:] == 9.0).all()


@pytest.mark.parametrize("st", [E.BF16, E.F32])
@pytest.mark.parametrize("rows,cols,ld,out_cols", [
    (1, 1, 0, 32), (1, 32, 0, 32), (3, 31, 0, 64), (5, 33, 40, 64), (7, 128, 0, 256), (2, 1001, 1003, 1024),
    (257, 96, 104, 96), (1000, 64, 0, 64), (33, 6144, 0, 6144), (4, 1000, 1000, 1152), (130, 8, 0, 128)])
def test_quantize_against_the_definition(st, rows, cols, ld, out_cols):
    say("quantize", st, rows, cols, ld, out_cols)
    g = torch.Generator().manual_seed(rows + cols)
    x = torch.randn((rows, ld or cols), generator=g) * torch.exp2(torch.randn((rows, 1), generator=g) * 8)
    check_quantize(x.to(TYPES[st]), cols, ld, out_cols)


@pytest.mark.parametrize("st", [E.BF16, E.F32])
def test_quantize_ties_and_every_exponent(st):
    """Each block's largest value fixes its scale 2^e; the rest are the grid's values and
    midpoints (ties), one step off them, and zeros of both signs, for every exponent
    of fp32 with the subnormal ones."""
    say("quantize: ties at every exponent", st)
    marks = np.array([0.0, -0.0, 0.25, 0.5, 0.75, 1, 1.25, 1.5, 1.75, 2, 2.5, 3, 3.5, 4, 5, 6, 7.75])
    near = np.concatenate([marks, -marks])[:31]
    rows = []
    for e in range(-149, 126):
        for delta in (0.0, 2.0 ** -7, -2.0 ** -7):
            rows.append(np.concatenate([[4.0], near * (1 + delta)]) * 2.0 ** e)
    with np.errstate(over="ignore"):
        x = torch.from_numpy(np.array(rows, dtype=np.float64)).float().to(TYPES[st])
    assert torch.isfinite(x).all()
    check_quantize(x, 32)


@pytest.mark.parametrize("st", [E.BF16, E.F32])
def test_quantize_infinities_and_nan_mark_their_block_only(st):
    say("quantize: non-finite blocks", st)
    x = torch.randn((6, 96), generator=torch.Generator().manual_seed(2)).to(TYPES[st])
    x[0, 5], x[1, 40], x[2, 95] = float("inf"), float("-inf"), float("nan")
    x[3] = 0
    x[4] = torch.finfo(TYPES[st]).max
    x[5, :32] = torch.finfo(TYPES[st]).tiny / 4
    check_quantize(x, 96)


def test_quantize_in_place_without_values_and_empty():
    say("quantize: in place, no values, no rows")
    x = torch.randn((50, 64), generator=torch.Generator().manual_seed(4)).to(DEV)
    codes, scales, values = quantize(x, 64)
    c2, s2, _ = quantize(x, 64, values=None)
    y = x.clone()
    c3, s3, _ = quantize(y, 64, values=y)
    for a, b in ((c2, codes), (c3, codes), (s2, scales), (s3, scales), (y, values)):
        assert torch.equal(a, b)
    # its own values quantise to themselves: a block's maximum rounds to code 4 or 6,
    # which keeps the scale
    assert torch.equal(quantize(y, 64)[2], y)
    E.engram_quantize_mx4(None, E.F32, 0, 64, 0, 64, None, None, None)


@pytest.mark.parametrize("st", [E.BF16, E.F32])
def test_quantize_rows_far_apart(st):
    """A stride that takes the rows past 2^31 elements."""
    say("quantize: offsets beyond 2^31 elements", st)
    rows, ld = 1100, (1 << 21) + 8
    for cols in (40, 61):
        x = torch.randn((rows, cols), generator=torch.Generator().manual_seed(cols)).to(TYPES[st])
        src = torch.zeros((rows, ld), dtype=TYPES[st], device=DEV)
        src[:, :cols] = x.to(DEV)
        near = quantize(x.to(DEV), cols)
        far = quantize(src, cols, ld, values=src)
        assert torch.equal(far[0], near[0]) and torch.equal(far[1], near[1])
        assert torch.equal(src[:, :cols], near[2]) and (src[:, cols:cols + 64] == 0).all()
        del src, far


def test_quantize_on_streams_and_in_graphs():
    say("quantize: streams, graph replays")
    x = torch.randn((300, 1001), generator=torch.Generator().manual_seed(6)).to(torch.bfloat16).to(DEV)
    first = quantize(x, 1001, 0, 1024)
    streams = [torch.cuda.Stream() for _ in range(2)]
    outs = [[torch.full_like(t, 5) for t in first] for _ in streams]
    torch.cuda.synchronize()
    for _ in range(3):
        for s, o in zip(streams, outs):
            E.engram_quantize_mx4(x, E.BF16, 300, 1001, 0, 1024, *o, s)
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for o in outs for a, b in zip(o, first))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        E.engram_quantize_mx4(x, E.BF16, 300, 1001, 0, 1024, *outs[0])
    for _ in range(3):
        for t in outs[0]:
            t.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(outs[0], first))
        x.copy_(-x)                     # other values through the same graph
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(outs[0], quantize(x, 1001, 0, 1024)))
        x.copy_(-x)


# ---- product -----------------------------------------------------------------------

def e4m3_value(c):
    s, f, m = c >> 7, (c >> 3) & 15, c & 7
    v = np.where(f == 0, m / 8 * 2.0 ** -6, (1 + m / 8) * 2.0 ** (f.astype(np.float64) - 7))
    return np.where(s == 1, -v, v)


def operand(rows, K, fmt, seed, integer=False):
    """(bytes, scales, float64 values) of random block-scaled rows."""
    rng = np.random.default_rng(seed)
    scales = (np.full((rows, K // 32), 127, np.uint8) if integer
              else rng.integers(120, 132, (rows, K // 32)).astype(np.uint8))
    if fmt == E.MX_E2M1:
        codes = rng.integers(0, 16, (rows, K)).astype(np.uint8)
        values = np.where(codes & 8, -1.0, 1.0) * GRID[codes & 7]
        raw = (codes[:, 0::2] | (codes[:, 1::2] << 4)).astype(np.uint8)
    else:
        # magnitudes up to 28 (code 0x5E); small integers when asked for
        raw = (rng.choice(np.array([0x00, 0x38, 0x40, 0x44, 0x48]), (rows, K)) if integer
               else rng.integers(0, 0x5F, (rows, K))).astype(np.uint8)
        raw |= (rng.integers(0, 2, (rows, K)) << 7).astype(np.uint8)
        values = e4m3_value(raw.astype(np.int64))
    values = values * np.repeat(2.0 ** (scales.astype(np.float64) - 127), 32, axis=1)
    return raw, scales, values


def project(e, es, fmt, w, ws, tokens, K, N, workspace=True, stream=None):
    kv = torch.full((tokens, N), 7.0, dtype=torch.bfloat16, device=DEV)
    size = E.engram_project_mx4_workspace_size(tokens, K, N, fmt) if workspace else 0
    buf = torch.full((size,), 0xA5, dtype=torch.uint8, device=DEV) if size else None
    E.engram_project_mx4(e, es, fmt, w, ws, kv, tokens, K, N, buf, size, stream)
    torch.cuda.synchronize()
    return kv


def dev(a):
    return torch.from_numpy(np.ascontiguousarray(a)).to(DEV)


def assert_product(got, ev, wv, fmt):
    """kv against the float64 product of the operands' values, at the bound above."""
    K = ev.shape[1]
    ev, wv = (x if torch.is_tensor(x) else dev(x) for x in (ev, wv))
    ev, wv = ev.double(), wv.double()
    exact = ev @ wv.t().contiguous()
    acc = K * 2.0 ** -23 * (ev.abs() @ wv.abs().t().contiguous())
    if fmt == E.MX_E4M3:
        for g in range(0, K, 8):
            top = torch.zeros_like(acc)
            for k in range(g, g + 8):
                torch.maximum(top, torch.outer(ev[:, k].abs(), wv[:, k].abs()), out=top)
            acc += 7 * 2.0 ** -13 * top
    excess = (got.double() - exact).abs() - (acc + 2.0 ** -8 * (exact.abs() + acc))
    assert (excess <= 0).all(), float(excess.max())


def check_project(tokens, K, N, fmt, workspace=True):
    e, es, ev = operand(tokens, K, fmt, tokens + K)
    w, ws, wv = operand(N, K, E.MX_E2M1, N + K)
    assert_product(project(dev(e), dev(es), fmt, dev(w), dev(ws), tokens, K, N, workspace), ev, wv, fmt)


SHAPES = [(1, 128, 8), (1, 6144, 520), (2, 256, 40), (7, 384, 24), (31, 640, 264), (32, 128, 256),
          (33, 1152, 136), (64, 256, 512), (65, 2176, 72), (100, 384, 1000), (128, 512, 128),
          (129, 640, 392), (255, 1024, 520), (256, 6144, 1032), (257, 256, 264), (300, 384, 776),
          (513, 1280, 2056), (1003, 896, 520), (1, 20480, 32), (2500, 128, 264), (40, 256, 12808),
          (20, 1664, 16392), (100, 1920, 16400), (200, 1408, 16648), (2100, 128, 4104), (2049, 384, 4360),
          (2305, 1152, 4104), (2111, 1280, 4128), (130, 256, 33032), (300, 640, 20488)]


@pytest.mark.parametrize("fmt", [E.MX_E4M3, E.MX_E2M1])
@pytest.mark.parametrize("tokens,K,N", SHAPES)
def test_project_against_64_bits(fmt, tokens, K, N):
    say("project", fmt, tokens, K, N)
    check_project(tokens, K, N, fmt)


@pytest.mark.parametrize("fmt", [E.MX_E4M3, E.MX_E2M1])
@pytest.mark.parametrize("tokens,K,N", [(129, 640, 392), (513, 1280, 2056), (5, 6144, 264)])
def test_project_without_a_workspace(fmt, tokens, K, N):
    say("project, no workspace", fmt, tokens, K, N)
    check_project(tokens, K, N, fmt, workspace=False)


@pytest.mark.parametrize("fmt", [E.MX_E4M3, E.MX_E2M1])
@pytest.mark.parametrize("tokens,K,N", [(3, 384, 40), (70, 640, 136), (256, 1152, 520), (700, 512, 1288),
                                        (5000, 256, 3336), (2100, 640, 4104), (2305, 2176, 4360), (250, 4992, 16392),
                                        (30_000, 512, 2568)])
def test_project_integers_are_exact(fmt, tokens, K, N):
    """Codes of halves and integers at scale 1: every partial sum is a multiple of 1/4
    below 2^16, so fp32 holds it and only the bf16 rounding remains."""
    say("project: exact sums", fmt, tokens, K, N)
    e, es, ev = operand(tokens, K, fmt, 1, integer=True)
    w, ws, wv = operand(N, K, E.MX_E2M1, 2, integer=True)
    got = project(dev(e), dev(es), fmt, dev(w), dev(ws), tokens, K, N)
    exact = dev(ev) @ dev(wv).t()
    assert torch.equal(got, exact.float().to(torch.bfloat16))


@pytest.mark.parametrize("fmt", [E.MX_E4M3, E.MX_E2M1])
@pytest.mark.parametrize("tokens,K,N", [(4, 384, 40), (200, 640, 264), (600, 1152, 1032),
                                        (2100, 1408, 4104)])
def test_project_each_input_meets_its_own_weight(fmt, tokens, K, N):
    """e has one nonzero input per token, at its own scale: kv is one exact product."""
    say("project: one input per token", fmt, tokens, K, N)
    e, es, ev = operand(tokens, K, fmt, 3)
    pick = np.arange(tokens) * 37 % K
    mask = np.zeros((tokens, K), bool)
    mask[np.arange(tokens), pick] = True
    if fmt == E.MX_E2M1:
        keep = np.where(mask[:, 0::2], 0x0F, 0) | np.where(mask[:, 1::2], 0xF0, 0)
        e = e & keep.astype(np.uint8)
    else:
        e = np.where(mask, e, 0).astype(np.uint8)
    w, ws, wv = operand(N, K, E.MX_E2M1, 4)
    exact = np.where(mask, ev, 0.0) @ wv.T
    got = project(dev(e), dev(es), fmt, dev(w), dev(ws), tokens, K, N)
    assert torch.equal(got, dev(exact).float().to(torch.bfloat16))


@pytest.mark.parametrize("fmt", [E.MX_E4M3, E.MX_E2M1])
@pytest.mark.parametrize("tokens,K,N", [(3, 384, 40), (130, 384, 264), (700, 640, 520),
                                        (2100, 640, 4104), (90, 896, 16392)])
def test_project_nan_scales_stay_in_their_row(fmt, tokens, K, N):
    """A NaN block scale makes its own row's outputs NaN and no other's; the last block of
    a row lies next to the following row's first in memory."""
    say("project: NaN scales", fmt, tokens, K, N)
    e, es, ev = operand(tokens, K, fmt, 5)
    w, ws, wv = operand(N, K, E.MX_E2M1, 6)
    es[1, 0] = es[tokens - 1, -1] = 255
    ws[2, -1] = ws[N - 1, 0] = 255
    got = project(dev(e), dev(es), fmt, dev(w), dev(ws), tokens, K, N).cpu()
    bad = torch.zeros((tokens, N), dtype=torch.bool)
    bad[[1, tokens - 1]] = True
    bad[:, [2, N - 1]] = True
    assert torch.equal(torch.isnan(got), bad)


def test_project_extreme_scales():
    """Blocks near both ends of the scale range, meeting a factor that brings them back."""
    say("project: extreme scales")
    for lo, hi in ((1, 253), (253, 1), (90, 164)):
        e, es, _ = operand(40, 256, E.MX_E2M1, 7, integer=True)
        w, ws, _ = operand(64, 256, E.MX_E2M1, 8, integer=True)
        es[:], ws[:] = lo, hi
        ones = [np.full_like(s, 127) for s in (es, ws)]
        a = project(dev(e), dev(es), E.MX_E2M1, dev(w), dev(ws), 40, 256, 64)
        b = project(dev(e), dev(ones[0]), E.MX_E2M1, dev(w), dev(ones[1]), 40, 256, 64)
        assert torch.equal(a, b)


def test_project_zero_tokens_and_rows_behind():
    say("project: no tokens; rows behind the last token stay")
    E.engram_project_mx4(None, None, E.MX_E2M1, None, None, None, 0, 256, 64)
    e, es, _ = operand(70, 256, E.MX_E2M1, 9)
    w, ws, _ = operand(264, 256, E.MX_E2M1, 10)
    kv = torch.full((75, 264), 7.0, dtype=torch.bfloat16, device=DEV)
    E.engram_project_mx4(dev(e), dev(es), E.MX_E2M1, dev(w), dev(ws), kv, 70, 256, 264)
    torch.cuda.synchronize()
    assert (kv[70:] == 7.0).all()


@pytest.mark.parametrize("fmt", [E.MX_E4M3, E.MX_E2M1])
@pytest.mark.parametrize("tokens", [1, 40, 256, 600, 10_000])
def test_project_same_bits_on_streams_and_in_graphs(fmt, tokens):
    say("project: streams, graph replays", fmt, tokens)
    K, N = 640, 1032
    e, es, _ = (operand(tokens, K, fmt, 11))
    w, ws, _ = operand(N, K, E.MX_E2M1, 12)
    args = [dev(x) for x in (e, es, w, ws)]
    first = project(args[0], args[1], fmt, args[2], args[3], tokens, K, N)
    size = E.engram_project_mx4_workspace_size(tokens, K, N, fmt)
    streams = [torch.cuda.Stream() for _ in range(2)]
    outs = [torch.empty_like(first) for _ in streams]
    bufs = [torch.empty(max(size, 1), dtype=torch.uint8, device=DEV) for _ in streams]
    torch.cuda.synchronize()
    for s, o, b in zip(streams, outs, bufs):
        E.engram_project_mx4(args[0], args[1], fmt, args[2], args[3], o, tokens, K, N,
                             b if size else None, size, s)
    torch.cuda.synchronize()
    assert all(torch.equal(o, first) for o in outs)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        E.engram_project_mx4(args[0], args[1], fmt, args[2], args[3], outs[0], tokens, K, N,
                             bufs[0] if size else None, size)
    for k in range(3):
        outs[0].zero_()
        bufs[0].fill_(k)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(outs[0], first)


def test_project_full_layer_sizes():
    """6144 inputs to 25600 outputs: a sample of columns against float64."""
    say("project: the layer's sizes")
    K, N = 6144, 25600
    w, ws, wv = operand(N, K, E.MX_E2M1, 13)
    wd, wsd = dev(w), dev(ws)
    cols = np.random.default_rng(0).choice(N, 300, replace=False)
    for fmt, tokens in ((E.MX_E4M3, 1), (E.MX_E2M1, 1), (E.MX_E2M1, 40), (E.MX_E4M3, 256), (E.MX_E2M1, 256),
                        (E.MX_E4M3, 1003), (E.MX_E2M1, 2049)):
        e, es, ev = operand(tokens, K, fmt, 14)
        say(fmt, tokens)
        assert_product(project(dev(e), dev(es), fmt, wd, wsd, tokens, K, N)[:, cols], ev, wv[cols], fmt)


@pytest.mark.parametrize("fmt", [E.MX_E4M3, E.MX_E2M1])
@pytest.mark.parametrize("tokens,K,N", [(90_000, 128, 25600), (1_100_000, 2048, 16)])
def test_project_offsets_beyond_31_bits(fmt, tokens, K, N):
    """More than 2^31 outputs, and more than 2^31 bytes of E4M3 inputs (2^30 of E2M1):
    rows from every part against float64."""
    say("project: far offsets", fmt, tokens, K, N)
    width = K if fmt == E.MX_E4M3 else K // 2
    gen_ = torch.Generator(device=DEV).manual_seed(15)
    e = torch.randint(0, 256, (tokens, width), dtype=torch.uint8, device=DEV, generator=gen_)
    if fmt == E.MX_E4M3:
        e &= 0xD7                       # magnitudes up to 15, no NaN
    es = torch.full((tokens, K // 32), 126, dtype=torch.uint8, device=DEV)
    w, ws, wv = operand(N, K, E.MX_E2M1, 16)
    kv = project(e, es, fmt, dev(w), dev(ws), tokens, K, N)
    pick = torch.tensor([0, 1, tokens // 3, tokens // 2 + 5, tokens - 257, tokens - 1], device=DEV)
    raw = e[pick].cpu().numpy().astype(np.int64)
    if fmt == E.MX_E4M3:
        ev = e4m3_value(raw)
    else:
        codes = np.stack((raw & 15, raw >> 4), -1).reshape(len(pick), -1)
        ev = np.where(codes & 8, -1.0, 1.0) * GRID[codes & 7]
    assert_product(kv[pick], ev * 0.5, wv, fmt)


# ---- together ----------------------------------------------------------------------

def test_lookup_quantise_project_gate():
    """A step as it would be used: rows looked up from a bf16 table with a scale, quantised,
    projected with a quantised weight, and the gate applied to the result; every stage
    against float64 on the stage before it."""
    say("embed -> quantize -> project_mx4 -> gate")
    R, S, dim, hc, d, tokens = 4000, 6, 64, 2, 128, 50
    K, N = S * dim, (hc + 1) * d
    g = torch.Generator().manual_seed(1)
    table = torch.randn((R, dim), generator=g).to(torch.bfloat16).to(DEV)
    ids = torch.from_numpy(np.random.default_rng(2).integers(0, R, tokens * S)).to(DEV)
    e = torch.empty((tokens, K), dtype=torch.bfloat16, device=DEV)
    E.engram_embed(E.embed_desc(R, tokens * S, dim, E.BF16, E.BF16, 0.5), table, ids, e)
    assert torch.equal(e.reshape(-1, dim), (table[ids].float() * 0.5).to(torch.bfloat16))
    weight = torch.randn((N, K), generator=g) * 0.05
    ec, es, ev = quantize(e, K)
    wc, wsc, wv = quantize(weight.to(DEV), K)
    kv = project(ec, es, E.MX_E2M1, wc, wsc, tokens, K, N)
    assert_product(kv, ev, wv, E.MX_E2M1)
    desc = E.forward_desc(1, tokens, hc, d, R, E.ROW_E4M3_E8M0_264, 256)
    tok = torch.zeros(tokens, dtype=torch.int32, device=DEV)
    qw, kw = (torch.ones((hc, d), device=DEV) for _ in range(2))
    h = torch.randn((tokens, hc, d), generator=g).to(torch.bfloat16).to(DEV)
    before = h.clone().double()
    gates = torch.empty((tokens, hc), device=DEV)
    E.engram_gate(desc, tok, 10, kv, qw, kw, h, gates)
    torch.cuda.synchronize()
    value = kv[:, hc * d:].double()
    want = before + gates.double()[..., None] * value[:, None, :]
    assert ((h.double() - want).abs() <= 2.0 ** -8 * want.abs() + 1e-6).all()


def test_table_rows_codes_project_directly():
    """The table's own E4M3 rows, split by engram_gather_mx, against a 4-bit weight."""
    say("gather_mx -> project_mx4")
    R, S, tokens, N = 3000, 3, 37, 264
    raw = gen.table_rows(5, np.arange(R))
    ids = np.random.default_rng(3).integers(0, R, tokens * S).astype(np.int64)
    codes = torch.empty((tokens, S * 256), dtype=torch.uint8, device=DEV)
    scales = torch.empty((tokens, S * 8), dtype=torch.uint8, device=DEV)
    E.engram_gather_mx(dev(raw), R, dev(ids), ids.size, codes, scales)
    w, ws, wv = operand(N, S * 256, E.MX_E2M1, 20)
    kv = project(codes, scales, E.MX_E4M3, dev(w), dev(ws), tokens, S * 256, N)
    rows = raw[ids].astype(np.int64)
    vals = e4m3_value(rows[:, :256]) * np.repeat(2.0 ** (rows[:, 256:] - 127.0), 32, axis=1)
    assert_product(kv, vals.reshape(tokens, -1), wv, E.MX_E4M3)


@pytest.mark.parametrize("fmt", [E.MX_E4M3, E.MX_E2M1])
@pytest.mark.parametrize("tokens,K,N", [(1, 6144, 264), (129, 896, 392), (256, 1408, 16648), (2111, 1280, 4128)])
def test_project_leaves_a_given_workspace_alone(fmt, tokens, K, N):
    say("project: a real workspace", fmt, tokens, K, N)
    e, es, _ = operand(tokens, K, fmt, 31)
    w, ws, _ = operand(N, K, E.MX_E2M1, 32)
    args = [dev(x) for x in (e, es, w, ws)]
    plain = project(args[0], args[1], fmt, args[2], args[3], tokens, K, N, workspace=False)
    buf = torch.full((1 << 16,), 0xA5, dtype=torch.uint8, device=DEV)
    assert buf.data_ptr() % 256 == 0
    for size in (0, buf.numel()):
        kv = torch.full_like(plain, 7.0)
        E.engram_project_mx4(args[0], args[1], fmt, args[2], args[3], kv, tokens, K, N, buf, size)
        torch.cuda.synchronize()
        assert torch.equal(kv, plain) and (buf == 0xA5).all()


@pytest.mark.parametrize("fmt", [E.MX_E4M3, E.MX_E2M1])
@pytest.mark.parametrize("tokens,K,N", [(256, 6144, 25600), (1003, 6144, 25600), (256, 5888, 16400),
                                        (64, 2816, 12808), (40, 768, 264)])
def test_project_repeats_itself(fmt, tokens, K, N):
    """Twelve calls over outputs filled with something else each time, other work between."""
    say("project: repeats", fmt, tokens, K, N)
    g = torch.Generator(device=DEV).manual_seed(K)
    width = K if fmt == E.MX_E4M3 else K // 2
    e = torch.randint(0, 256, (tokens, width), dtype=torch.uint8, device=DEV, generator=g)
    if fmt == E.MX_E4M3:
        e &= 0xF7                       # no NaN
    w = torch.randint(0, 256, (N, K // 2), dtype=torch.uint8, device=DEV, generator=g)
    es = torch.randint(120, 132, (tokens, K // 32), dtype=torch.uint8, device=DEV, generator=g)
    ws = torch.randint(120, 132, (N, K // 32), dtype=torch.uint8, device=DEV, generator=g)
    first = project(e, es, fmt, w, ws, tokens, K, N)
    assert torch.isfinite(first).all()
    kv = torch.empty_like(first)
    for k in range(12):
        kv.fill_(float(k))
        E.engram_project_mx4(e, es, fmt, w, ws, kv, tokens, K, N)
        assert torch.equal(kv, first)


@pytest.mark.parametrize("fmt", [E.MX_E4M3, E.MX_E2M1])
@pytest.mark.parametrize("tokens,K,N", [(128, 384, 66056), (129, 384, 33032), (256, 768, 65800), (600, 896, 25608),
                                        (768, 1408, 25608), (900, 512, 25608), (1700, 640, 10248),
                                        (5000, 512, 10248)])
def test_project_rounds_of_tiles(fmt, tokens, K, N):
    """Shapes on both sides of the choice between tiles of 128 and 256 tokens, of one round of
    blocks to four, and tiles walked by a block: exact integer sums as above."""
    say("project: rounds", fmt, tokens, K, N)
    e, es, ev = operand(tokens, K, fmt, 41, integer=True)
    w, ws, wv = operand(N, K, E.MX_E2M1, 42, integer=True)
    got = project(dev(e), dev(es), fmt, dev(w), dev(ws), tokens, K, N)
    wt = dev(wv).float().t().contiguous()
    for m in range(0, tokens, 1024):        # sums of multiples of 1/4 below 2^16: fp32 holds them
        exact = dev(ev[m:m + 1024]).float() @ wt
        assert torch.equal(got[m:m + 1024], exact.to(torch.bfloat16))


# ---- the largest sizes, special codes -------------------------------------------------

def test_quantize_more_groups_than_one_sweep_of_threads():
    """2^28 + 12345 rows of one block: threads take a second turn, the codes pass 2^32 bytes."""
    say("quantize: 2^28 rows")
    rows, cols = (1 << 28) + 12345, 3
    src = torch.arange(rows * cols, device=DEV).remainder_(251).reshape(rows, cols).to(torch.bfloat16)
    codes = torch.full((rows, 16), 0x55, dtype=torch.uint8, device=DEV)
    scales = torch.full((rows, 1), 0x55, dtype=torch.uint8, device=DEV)
    E.engram_quantize_mx4(src, E.BF16, rows, cols, 0, 32, codes, scales)
    torch.cuda.synchronize()
    for a in (0, 70_000_000, 1 << 28, rows - 2000):
        part = slice(a, min(rows, a + 2000))
        ec, es, _ = quantize_reference(src[part].cpu().double().numpy(), 32)
        assert np.array_equal(scales[part].cpu().numpy(), es) and np.array_equal(unpack(codes[part]), ec)


@pytest.mark.parametrize("st", [E.BF16, E.F32])
def test_quantize_the_widest_rows(st):
    say("quantize: 2^20 columns", st)
    cols = (1 << 20) - 5
    x = torch.randn((3, cols + 8), generator=torch.Generator().manual_seed(7)).to(TYPES[st])
    check_quantize(x, cols, cols + 8, 1 << 20)


@pytest.mark.parametrize("fmt", [E.MX_E4M3, E.MX_E2M1])
@pytest.mark.parametrize("tokens,K,N", [(1, 1 << 20, 8), (130, 1 << 20, 264), (130, (1 << 20) - 128, 264),
                                        (2049, 1 << 20, 4104)])
def test_project_the_longest_sums(fmt, tokens, K, N):
    """2^20 inputs, one in 64 of them not zero: sums of small integers, exact."""
    say("project: long sums", fmt, tokens, K, N)
    g = torch.Generator(device=DEV).manual_seed(K + tokens)

    def codes(rows, e4m3):
        pick = torch.randint(0, 64, (rows, K), dtype=torch.uint8, device=DEV, generator=g)
        c = torch.tensor([0x38, 0x40, 0xB8, 0xC0] if e4m3 else [2, 4, 10, 12], dtype=torch.uint8, device=DEV)
        c = torch.where(pick < 4, c[(pick & 3).int()], 0)
        v = torch.tensor([1.0, 2.0, -1.0, -2.0], device=DEV)
        v = torch.where(pick < 4, v[(pick & 3).int()], 0.0)
        return (c if e4m3 else (c[:, 0::2] | (c[:, 1::2] << 4)).contiguous()), v

    e, ev = codes(tokens, fmt == E.MX_E4M3)
    w, wv = codes(N, False)
    es = torch.full((tokens, K // 32), 127, dtype=torch.uint8, device=DEV)
    ws = torch.full((N, K // 32), 127, dtype=torch.uint8, device=DEV)
    got = project(e, es, fmt, w, ws, tokens, K, N)
    exact = ev @ wv.t().contiguous()
    assert exact.abs().max() > 8 and torch.equal(got, exact.to(torch.bfloat16))


@pytest.mark.parametrize("tokens,K,N", [(3, 384, 40), (130, 896, 264), (600, 384, 25608), (2100, 640, 4104)])
def test_project_nan_codes_stay_in_their_token(tokens, K, N):
    """An E4M3 NaN among a token's inputs makes its outputs NaN and no other's, a zero weight
    beside it or not; in the first input and in the last."""
    say("project: NaN codes", tokens, K, N)
    e, es, _ = operand(tokens, K, E.MX_E4M3, 51)
    w, ws, _ = operand(N, K, E.MX_E2M1, 52)
    e[1, 0], e[tokens - 1, K - 1] = 0x7F, 0xFF
    w[:N // 2, 0] = 0
    got = project(dev(e), dev(es), E.MX_E4M3, dev(w), dev(ws), tokens, K, N).cpu()
    bad = torch.zeros((tokens, N), dtype=torch.bool)
    bad[[1, tokens - 1]] = True
    assert torch.equal(torch.isnan(got), bad)
