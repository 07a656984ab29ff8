"""The scaled lookup and its gradient by sorted row ids against 64-bit references.

Lookup: the fp32 product is off by at most half a step (2^-24), its rounding to
bf16 by another half step (2^-8).

Gradient: a term of a row's sum of m passes through at most m additions (through
fewer than 200 + m / 64 in a long sum), each off by at most half a step, and the
scaling by one more: (m + 2) 2^-24 of the sum of magnitudes."""
import numpy as np
import pytest

from tests.gpu_util import say

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("no GPU", allow_module_level=True)

import hashed_gram_conditional_amd as E  # noqa: E402

DEV = "cuda"
U32, UBF = 2.0 ** -24, 2.0 ** -8
TYPES = {E.BF16: torch.bfloat16, E.F32: torch.float32}


def _rand(shape, seed, dtype, scale=1.0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(shape, generator=g) * scale).to(dtype)


def _embed(table, ids, dim, tt, ot, scale, table_ld=0, out_ld=0, rows=None, fill=7.0):
    n = ids.numel()
    out = torch.full((n, out_ld or dim), fill, dtype=TYPES[ot], device=DEV)
    d = E.embed_desc(table.shape[0] if rows is None else rows, n, dim, tt, ot, scale, table_ld, out_ld)
    E.engram_embed(d, table, ids, out)
    torch.cuda.synchronize()
    return out


@pytest.mark.parametrize("tt", [E.BF16, E.F32])
@pytest.mark.parametrize("ot", [E.BF16, E.F32])
@pytest.mark.parametrize("n,dim,table_ld,out_ld", [
    (1, 1, 0, 0), (1, 256, 0, 0), (3, 8, 0, 0), (1000, 256, 0, 0), (257, 7, 0, 0), (513, 33, 40, 0),
    (100, 264, 0, 272), (77, 5120, 5128, 5120), (65, 24, 28, 24), (4099, 32, 0, 0), (9, 1001, 0, 1003)])
def test_embed_against_64_bits(tt, ot, n, dim, table_ld, out_ld):
    say("embed", tt, ot, n, dim, table_ld, out_ld)
    R, scale = 501, -0.37
    table = _rand((R, table_ld or dim), n + dim, TYPES[tt])
    ids = torch.from_numpy(np.random.default_rng(n).integers(-4, R + 4, n))
    ids[0] = R - 1
    got = _embed(table.to(DEV), ids.to(DEV), dim, tt, ot, scale, table_ld, out_ld).cpu()
    ok = (ids >= 0) & (ids < R)
    exp = torch.zeros((n, dim), dtype=torch.float64)
    exp[ok] = table[ids[ok], :dim].double() * float(np.float32(scale))
    tol = exp.abs() * (U32 + (UBF * (1 + U32) if ot == E.BF16 else 0.0))
    assert ((got[:, :dim].double() - exp).abs() <= tol).all()
    # dropped rows are +0 whatever the scale's sign, and the gaps stay as they were
    assert not torch.signbit(got[:, :dim][~ok]).any()
    assert (got[:, dim:] == 7.0).all()


def test_embed_scale_one_copies_every_bit_pattern():
    say("embed: all bf16 patterns, scale 1")
    bits = torch.arange(65536, dtype=torch.int32).to(torch.int16).reshape(256, 256)
    table = bits.view(torch.bfloat16).to(DEV)
    ids = torch.arange(256, device=DEV)
    got = _embed(table, ids, 256, E.BF16, E.BF16, 1.0).cpu()
    nan = torch.isnan(table.cpu())
    assert torch.equal(got.view(torch.int16)[~nan], bits[~nan]) and torch.isnan(got[nan]).all()


def test_embed_empty_and_empty_table():
    say("embed: no ids, no rows")
    ids = torch.zeros(3, dtype=torch.int64, device=DEV)
    out = torch.full((3, 16), 5.0, device=DEV)
    E.engram_embed(E.embed_desc(0, 3, 16, E.F32, E.F32), None, ids, out)
    E.engram_embed(E.embed_desc(10, 0, 16, E.F32, E.F32), None, None, None)
    torch.cuda.synchronize()
    assert (out == 0).all()


def test_embed_far_rows_and_pinned_table():
    say("embed: byte offsets beyond 2^32, pinned host table")
    R, dim = 4_500_000, 512                      # 4.6 GB of bf16
    table = torch.zeros((R, dim), dtype=torch.bfloat16, device=DEV)
    far = torch.tensor([R - 1, 4_194_305, 0, 2_097_153], device=DEV)
    table[far] = torch.arange(4 * dim, device=DEV).reshape(4, dim).remainder(251).to(torch.bfloat16)
    got = _embed(table, far, dim, E.BF16, E.F32, 2.0)
    assert torch.equal(got, table[far].float() * 2)
    small = _rand((1000, 72), 3, torch.float32)
    host = torch.empty((1000, 72), pin_memory=True)
    host.copy_(small)
    ids = torch.from_numpy(np.random.default_rng(1).integers(-2, 1003, 5000)).to(DEV)
    assert torch.equal(_embed(host, ids, 72, E.F32, E.BF16, 0.5),
                       _embed(small.to(DEV), ids, 72, E.F32, E.BF16, 0.5))


# ---- gradient ----------------------------------------------------------------------

def _reference(ids, d_out, R, scale):
    """Ascending rows, their float64 gradients, and the tolerance of each value."""
    ids = ids.numpy()
    ok = (ids >= 0) & (ids < R)
    rows, slot = np.unique(ids[ok], return_inverse=True)
    x = d_out[torch.from_numpy(ok)].double()
    slot = torch.from_numpy(slot.astype(np.int64))
    s = float(np.float32(scale))
    sums = torch.zeros((rows.size, d_out.shape[1]), dtype=torch.float64).index_add_(0, slot, x) * s
    mags = torch.zeros_like(sums).index_add_(0, slot, x.abs()) * abs(s)
    m = torch.bincount(slot, minlength=rows.size).double()
    return rows, sums, mags * ((m + 2) * U32)[:, None]


def _grad(ids, d_out, R, dim, ot, scale, out_ld=0, table_ld=0, dense=None):
    n = ids.numel()
    d = E.embed_desc(R, n, dim, E.F32, ot, scale, table_ld, out_ld)
    size = E.engram_embed_grad_workspace_size(d)
    ws = torch.full((size,), 0xA5, dtype=torch.uint8, device=DEV)
    d_out, ids = d_out.to(DEV), ids.to(DEV)
    if dense is not None:
        grad, accumulate = dense
        E.engram_embed_grad_dense(d, d_out, ids, grad, accumulate, ws, size)
        torch.cuda.synchronize()
        return grad
    rows = torch.full((n,), 99, dtype=torch.int64, device=DEV)
    grad = torch.full((n, dim), 7.0, device=DEV)
    count = torch.full((1,), 99, dtype=torch.int64, device=DEV)
    E.engram_embed_grad(d, d_out, ids, rows, grad, count, ws, size)
    torch.cuda.synchronize()
    return rows.cpu(), grad.cpu(), int(count)


def _check_sparse(ids, d_out, R, dim, ot, scale, out_ld=0):
    rows, grad, count = _grad(ids, d_out, R, dim, ot, scale, out_ld)
    er, es, tol = _reference(ids, d_out[:, :dim], R, scale)
    assert count == er.size
    assert np.array_equal(rows[:count].numpy(), er) and (rows[count:] == -1).all()
    assert ((grad[:count].double() - es).abs() <= tol).all()
    assert (grad[count:] == 7.0).all()
    return rows, grad


# (n, rows of the table, dim, ids): sizes around the small sort's parts and tiles, the
# merge's limit of 32768 and the large sort's tiles, runs on both sides of 64
SPREAD = [
    (1, 5, 8, "uniform"), (2, 1, 3, "uniform"), (63, 7, 256, "uniform"), (64, 1, 8, "uniform"),
    (65, 1, 8, "uniform"), (129, 2, 40, "uniform"), (1000, 100_000, 256, "uniform"),
    (1023, 40, 33, "zipf"), (4097, 300, 1, "zipf"), (12216, 2_400_000, 256, "zipf"),
    (16384, 100, 16, "zipf"), (16385, 100, 16, "zipf"), (16385, 50_000, 72, "uniform"),
    (20481, 384_006_168, 64, "uniform"), (40_000, 4_294_967_294, 8, "uniform"),
    (100_003, 1000, 24, "zipf"), (100_003, 1, 8, "uniform"), (300_000, 2_000_000, 8, "zipf"),
    (1024, 700, 16, "zipf"), (1025, 4_294_967_294, 16, "uniform"), (2048, 1, 16, "uniform"),
    (32768, 5000, 16, "zipf"), (32769, 5000, 16, "zipf"), (33_000, 3, 40, "zipf"),
    (30_000, 9, 7, "zipf"), (3000, 50, 5120, "zipf"), (500, 20, 2056, "zipf"), (400, 11, 1030, "zipf"),
    (2_200_000, 700_000, 4, "zipf")]


def _ids(n, R, kind, seed, drop=0.1):
    rng = np.random.default_rng(seed)
    if kind == "zipf":
        ids = np.minimum(rng.zipf(1.2, n) - 1, R - 1) * 7919 % R
    else:
        ids = rng.integers(0, R, n)
    bad = rng.random(n) < drop
    ids[bad] = rng.choice(np.array([-1, R, R + 5, 2 ** 40, -2 ** 62]), int(bad.sum()))
    return torch.from_numpy(ids.astype(np.int64))


@pytest.mark.parametrize("ot", [E.BF16, E.F32])
@pytest.mark.parametrize("n,R,dim,kind", SPREAD)
def test_grad_rows_against_64_bits(ot, n, R, dim, kind):
    say("grad", ot, n, R, dim, kind)
    _check_sparse(_ids(n, R, kind, n + dim), _rand((n, dim), n, TYPES[ot]), R, dim, ot, 0.75)


@pytest.mark.parametrize("lengths", [[64] * 9, [65] * 9, [63, 64, 65, 66, 1, 127, 128, 129, 200],
                                     [8] * 40, [7, 9] * 30, [1000, 1, 1000], [1] * 100 + [640] + [1] * 100])
def test_grad_run_lengths(lengths):
    say("grad: run lengths", lengths[:9])
    ids = np.repeat(np.arange(len(lengths)) * 3, lengths)
    perm = np.random.default_rng(5).permutation(ids.size)
    ids = torch.from_numpy(ids[perm].astype(np.int64))
    _check_sparse(ids, _rand((ids.numel(), 40), 9, torch.float32), 3 * len(lengths), 40, E.F32, 1.0)


@pytest.mark.parametrize("n", [0, 1, 500, 16384, 32768, 32769, 50_000])
def test_grad_no_id_in_the_table(n):
    say("grad: nothing kept", n)
    ids = torch.full((n,), -1, dtype=torch.int64)
    rows, grad, count = _grad(ids, _rand((n, 16), 1, torch.bfloat16), 10, 16, E.BF16, 1.0)
    assert count == 0 and (rows == -1).all() and (grad == 7.0).all()
    full = _grad(ids, _rand((n, 16), 1, torch.bfloat16), 10, 16, E.BF16, 1.0,
                 dense=(torch.full((10, 16), 3.0, device=DEV), 0))
    assert (full == 0).all()
    kept = _grad(ids, _rand((n, 16), 1, torch.bfloat16), 10, 16, E.BF16, 1.0,
                 dense=(torch.full((10, 16), 3.0, device=DEV), 1))
    assert (kept == 3.0).all()


@pytest.mark.parametrize("ot", [E.BF16, E.F32])
@pytest.mark.parametrize("n,R,dim,out_ld,table_ld", [
    (300, 50, 24, 0, 0), (300, 50, 24, 32, 28), (5000, 2000, 13, 17, 15), (20_000, 999, 64, 0, 0),
    (37_000, 3, 8, 8, 16), (40, 100_000, 256, 264, 256), (700, 30, 1032, 0, 1036)])
def test_grad_dense_written_and_added(ot, n, R, dim, out_ld, table_ld):
    say("grad dense", ot, n, R, dim, out_ld, table_ld)
    ids = _ids(n, R, "zipf", n)
    d_out = _rand((n, out_ld or dim), 2, TYPES[ot])
    er, es, tol = _reference(ids, d_out[:, :dim], R, 1.5)
    exp = torch.zeros((R, dim), dtype=torch.float64)
    bound = torch.zeros_like(exp)
    exp[er], bound[er] = es, tol
    start = _rand((R, table_ld or dim), 4, torch.float32)
    for accumulate in (0, 1):
        got = _grad(ids, d_out, R, dim, ot, 1.5, out_ld, table_ld, dense=(start.to(DEV), accumulate)).cpu()
        want, lim = (exp, bound) if not accumulate else (exp + start[:, :dim].double(), bound)
        if accumulate:       # one more rounding, of the sum with what was there
            lim = bound + U32 * (want.abs() + bound)
        assert ((got[:, :dim].double() - want).abs() <= lim).all()
        assert torch.equal(got[:, dim:], start[:, dim:])
        if accumulate:
            untouched = torch.ones(R, dtype=torch.bool)
            untouched[er] = False
            assert torch.equal(got[untouched], start[untouched])


def test_grad_padded_rows_and_stride():
    say("grad: strided d_out, NaN in the gaps")
    d_out = _rand((900, 48), 3, torch.bfloat16)
    d_out[:, 40:] = float("nan")
    _check_sparse(_ids(900, 60, "zipf", 1), d_out, 60, 40, E.BF16, 2.0, out_ld=48)


def test_grad_dropped_rows_do_not_reach_the_sums():
    say("grad: NaN and infinity at dropped ids")
    ids = _ids(20_000, 100, "zipf", 3, drop=0.3)
    d_out = _rand((20_000, 16), 3, torch.float32)
    bad = (ids < 0) | (ids >= 100)
    d_out[bad] = float("nan")
    d_out[bad.nonzero()[::2, 0]] = float("inf")
    rows, grad, count = _grad(ids, d_out, 100, 16, E.F32, 1.0)
    assert torch.isfinite(grad[:count]).all()


def test_grad_is_the_lookup_s_adjoint_and_difference():
    """<d_out, embed(T + dT) - embed(T)> = <grad, dT>: the lookup is linear, so the two
    sides are one sum of products in two orders."""
    say("grad: adjoint of the lookup")
    n, R, dim, scale = 5000, 300, 40, 0.5
    ids = _ids(n, R, "zipf", 8).to(DEV)
    table, step = _rand((R, dim), 1, torch.float32), _rand((R, dim), 2, torch.float32)
    d_out = _rand((n, dim), 3, torch.float32)
    # differences of values that fp32 holds exactly: multiples of 2^-10 below 8
    table, step = (torch.round(x * 1024).clamp(-4095, 4095) / 1024 for x in (table, step))
    moved = _embed((table + step).to(DEV), ids, dim, E.F32, E.F32, scale).double()
    diff = moved - _embed(table.to(DEV), ids, dim, E.F32, E.F32, scale).double()
    grad = _grad(ids.cpu(), d_out, R, dim, E.F32, scale,
                 dense=(torch.empty((R, dim), device=DEV), 0)).double().cpu()
    left = (d_out.double() * diff.cpu()).sum()
    right = (grad * step.double()).sum()
    _, _, tol = _reference(ids.cpu(), d_out, R, scale)
    assert abs(left - right) <= (tol.sum(0).max() * dim * 4).item() + 1e-9 * abs(left)


@pytest.mark.parametrize("n,R", [(900, 30), (3000, 40), (40_000, 40), (40_000, 1_000_000)])
def test_grad_same_bits_twice_and_in_a_graph(n, R):
    say("grad: repeat and replay", n, R)
    dim = 64
    ids, d_out = _ids(n, R, "zipf", 4).to(DEV), _rand((n, dim), 5, torch.bfloat16).to(DEV)
    d = E.embed_desc(R, n, dim, E.BF16, E.BF16, 0.5)
    size = E.engram_embed_grad_workspace_size(d)
    ws = torch.empty(size, dtype=torch.uint8, device=DEV)
    table = _rand((R, dim), 6, torch.bfloat16).to(DEV)
    out = torch.zeros((n, dim), dtype=torch.bfloat16, device=DEV)
    rows = torch.zeros(n, dtype=torch.int64, device=DEV)
    grad = torch.zeros((n, dim), device=DEV)
    count = torch.zeros(1, dtype=torch.int64, device=DEV)

    def step(stream=None):
        E.engram_embed(d, table, ids, out, stream)
        E.engram_embed_grad(d, d_out, ids, rows, grad, count, ws, size, stream)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    first = [t.clone() for t in (out, rows, grad, count)]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for k in range(3):
        for t in (out, rows, grad, count):
            t.zero_()
        ws.fill_(k)
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip((out, rows, grad, count), first):
            assert torch.equal(a, b)
        # other ids through the same graph, then the first ones again
        keep = ids.clone()
        ids.copy_(_ids(n, R, "uniform", 50 + k).to(DEV))
        graph.replay()
        torch.cuda.synchronize()
        er, es, tol = _reference(ids.cpu(), d_out.cpu(), R, 0.5)
        assert int(count) == er.size and np.array_equal(rows[:er.size].cpu().numpy(), er)
        assert ((grad[:er.size].cpu().double() - es).abs() <= tol).all()
        ids.copy_(keep)


def test_a_training_step_of_a_table():
    """Lookup, gradient of sum(out * c), and the update of the touched rows, against the
    same step in float64 on the host."""
    say("embed + grad: one step of gradient descent on the table")
    n, R, dim, scale, rate = 6144, 5000, 256, 0.5, 0.125
    ids = _ids(n, R, "zipf", 12)
    table, c = _rand((R, dim), 1, torch.float32), _rand((n, dim), 2, torch.float32)
    dev_table = table.to(DEV)
    out = _embed(dev_table, ids.to(DEV), dim, E.F32, E.F32, scale)
    rows, grad, count = _grad(ids, c, R, dim, E.F32, scale)
    dev_table[rows[:count].to(DEV)] -= rate * grad[:count].to(DEV)
    er, es, tol = _reference(ids, c, R, scale)
    exp = table.double()
    exp[er] -= rate * es
    lim = torch.zeros_like(exp)
    lim[er] = rate * tol * (1 + U32) + U32 * (rate * es).abs()
    lim += U32 * (exp.abs() + lim)
    assert ((dev_table.cpu().double() - exp).abs() <= lim).all()
    assert out.shape == (n, dim)


# ---- calls at once, replayed, and of the largest sizes ------------------------------

WIDE_LD = (1 << 21) + 8          # 1100 rows at this stride pass 2^31 elements


def test_rows_far_apart():
    """Strides that take the lookup's output, d_out and the dense gradient past 2^31
    elements give what dense rows give."""
    say("embed, grad: offsets beyond 2^31 elements")
    n, R, dim = 1100, 1100, 24
    ids = _ids(n, R, "uniform", 21).to(DEV)
    table = _rand((R, dim), 22, torch.bfloat16).to(DEV)
    near = _embed(table, ids, dim, E.BF16, E.BF16, 0.5)
    far = torch.zeros((n, WIDE_LD), dtype=torch.bfloat16, device=DEV)
    E.engram_embed(E.embed_desc(R, n, dim, E.BF16, E.BF16, 0.5, 0, WIDE_LD), table, ids, far)
    torch.cuda.synchronize()
    assert torch.equal(far[:, :dim], near)
    a = _grad(ids, near, R, dim, E.BF16, 0.75)
    b = _grad(ids, far, R, dim, E.BF16, 0.75, out_ld=WIDE_LD)
    assert a[2] == b[2] and torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    c = _grad(ids, near, R, dim, E.BF16, 0.75, dense=(torch.empty((R, dim), device=DEV), 0))
    for accumulate, start in ((0, 3.0), (1, 0.0)):
        wide = torch.full((R, WIDE_LD), start, device=DEV)
        _grad(ids, near, R, dim, E.BF16, 0.75, table_ld=WIDE_LD, dense=(wide, accumulate))
        assert torch.equal(wide[:, :dim], c) and (wide[:, dim:dim + 64] == start).all()
        assert (wide[-1, dim:] == start).all()
        del wide


def test_grad_of_the_most_ids():
    """2^28 ids, of which the first ones name a row twice: every gradient is 1 or 2."""
    say("grad: 2^28 ids")
    n, m, step = E.MAX_EMBED_GRAD_IDS, 200_000_003, 21
    ids = torch.arange(n, device=DEV).remainder_(m).mul_(step)
    R = m * step                                   # 4.2e9 rows
    d = E.embed_desc(R, n, 1, E.BF16, E.BF16)
    size = E.engram_embed_grad_workspace_size(d)
    ws = torch.empty(size, dtype=torch.uint8, device=DEV)
    d_out = torch.ones((n, 1), dtype=torch.bfloat16, device=DEV)
    rows = torch.empty(n, dtype=torch.int64, device=DEV)
    grad = torch.full((n, 1), 7.0, device=DEV)
    count = torch.zeros(1, dtype=torch.int64, device=DEV)
    E.engram_embed_grad(d, d_out, ids, rows, grad, count, ws, size)
    torch.cuda.synchronize()
    assert int(count) == m
    assert torch.equal(rows[:m], torch.arange(m, device=DEV).mul_(step)) and (rows[m:] == -1).all()
    assert (grad[:n - m] == 2).all() and (grad[n - m:m] == 1).all() and (grad[m:] == 7).all()


@pytest.mark.parametrize("n,R", [(700, 50), (12216, 3000), (60_000, 900)])
def test_calls_at_once_on_two_streams(n, R):
    say("grad: two streams at once", n, R)
    dim = 72
    cases = []
    for k in range(2):
        ids, d_out = _ids(n, R, "zipf", 30 + k), _rand((n, dim), 40 + k, torch.float32)
        want = _grad(ids, d_out, R, dim, E.F32, 0.5)
        full = _grad(ids, d_out, R, dim, E.F32, 0.5, dense=(torch.empty((R, dim), device=DEV), 0))
        cases.append((ids.to(DEV), d_out.to(DEV), want, full))
    d = E.embed_desc(R, n, dim, E.F32, E.F32, 0.5)
    size = E.engram_embed_grad_workspace_size(d)
    bufs = []
    for k in range(2):
        bufs.append((torch.empty(size, dtype=torch.uint8, device=DEV),
                     torch.zeros(n, dtype=torch.int64, device=DEV), torch.zeros((n, dim), device=DEV),
                     torch.zeros(1, dtype=torch.int64, device=DEV), torch.zeros((R, dim), device=DEV),
                     torch.cuda.Stream()))
    torch.cuda.synchronize()
    for _ in range(5):
        for (ids, d_out, _, _), (ws, rows, grad, count, full, stream) in zip(cases, bufs):
            # the two calls of a stream share its workspace
            E.engram_embed_grad(d, d_out, ids, rows, grad, count, ws, size, stream)
            E.engram_embed_grad_dense(d, d_out, ids, full, 0, ws, size, stream)
    torch.cuda.synchronize()
    for (_, _, (rows0, grad0, count0), full0), (_, rows, grad, count, full, _) in zip(cases, bufs):
        assert int(count) == count0 and torch.equal(rows.cpu(), rows0)
        assert torch.equal(grad[:count0].cpu(), grad0[:count0]) and torch.equal(full, full0)


@pytest.mark.parametrize("n,R,table_ld", [(900, 300, 0), (900, 300, 76), (40_000, 2000, 0)])
def test_dense_gradient_in_a_graph(n, R, table_ld):
    """Captured twice over, written and then added to: every replay, with eager work
    between, gives the bits of the eager calls."""
    say("grad dense: replays", n, R, table_ld)
    dim = 72
    ids, d_out = _ids(n, R, "zipf", 50).to(DEV), _rand((n, dim), 51, torch.bfloat16).to(DEV)
    d = E.embed_desc(R, n, dim, E.BF16, E.BF16, 0.5, table_ld)
    size = E.engram_embed_grad_workspace_size(d)
    ws = torch.empty(size, dtype=torch.uint8, device=DEV)
    grad = torch.full((R, table_ld or dim), 3.0, device=DEV)

    def step():
        E.engram_embed_grad_dense(d, d_out, ids, grad, 0, ws, size)
        E.engram_embed_grad_dense(d, d_out, ids, grad, 1, ws, size)

    step()
    torch.cuda.synchronize()
    first = grad.clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for k in range(3):
        grad[:, :dim] = float(k)
        ws.fill_(17 * k)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(grad, first)
        step()
        torch.cuda.synchronize()
        assert torch.equal(grad, first)


# ---- the order of a long sum --------------------------------------------------------

@pytest.mark.parametrize("ot", [E.BF16, E.F32])
@pytest.mark.parametrize("dim,m", [(1, 4096), (2, 2048), (3, 1400), (8, 2048), (16, 1024), (256, 4096),
                                   (1, 32768), (8, 40_000)])
def test_grad_additions_of_one_row(ot, dim, m):
    """One row named by every id: 1 and then, in every chunk of 8, one value just below
    half a step of 1. A value added to the 1 by itself is lost, so the error counts the
    additions that stand one behind another, of which there are fewer than 200 + m / 64."""
    say("grad: additions", ot, dim, m)
    d_out = torch.zeros((m, dim), dtype=TYPES[ot])
    d_out[::8] = 0.984375 * 2.0 ** -24               # 63 / 64, exact in bf16
    d_out[0] = 1.0
    rows, grad, count = _grad(torch.zeros(m, dtype=torch.int64), d_out, 1, dim, ot, 1.0)
    assert count == 1 and rows[0] == 0
    want = d_out.double().sum(0)
    assert ((grad[0].double() - want).abs() <= (200 + m / 64) * U32 * want).all()


# ---- longer chunks -------------------------------------------------------------------

def plan_chunk(n, per_chunk):
    """Positions of a chunk: 64, halved down to 8 until the chunks' threads (one per 8
    columns) number 2048 per CU."""
    chunk = 64
    while chunk > 8 and n // chunk * per_chunk < 256 * 2048:
        chunk //= 2
    return chunk


@pytest.mark.parametrize("ot", [E.BF16, E.F32])
@pytest.mark.parametrize("n,dim,chunk", [(40_000, 2048, 16), (30_000, 2824, 16), (70_000, 2048, 32),
                                         (786_432, 256, 32), (140_000, 2048, 64), (1_050_000, 256, 64)])
def test_grad_run_lengths_of_longer_chunks(ot, n, dim, chunk):
    """Runs of both sides of the longest that one thread sums (twice a chunk, at most 64), of
    16 pieces and of thousands, among rows named once or a few times: row ids, count and
    gradients, sparse and dense, a sample of columns against float64."""
    say("grad: chunk", chunk, ot, n, dim)
    assert plan_chunk(n, dim // 8) == chunk
    longest = min(2 * chunk, 64)
    marks = [longest - 1, longest, longest + 1, chunk - 1, chunk, chunk + 1, 15 * chunk, 16 * chunk,
             16 * chunk + 1, 17 * chunk, 18 * chunk + 3, 40 * chunk, 1, 2, 100 * chunk - 1]
    hot = n // 8
    rng = np.random.default_rng(n + dim)
    lengths = np.concatenate([np.repeat(marks, 3), [hot, hot // 3]])
    rest = rng.zipf(1.3, n - int(lengths.sum()) - 97)
    R = 3 * lengths.size + 5000
    ids = np.concatenate([np.repeat(rng.permutation(lengths.size) * 3, lengths),
                          3 * lengths.size + np.minimum(rest - 1, 4999),
                          np.full(97, -1)])
    ids = torch.from_numpy(rng.permutation(ids).astype(np.int64))
    g = torch.Generator(device=DEV).manual_seed(n)
    d_out = torch.empty((n, dim), dtype=TYPES[ot], device=DEV).normal_(generator=g)
    cols = torch.tensor([0, 1, 7, 8, 63, dim // 2 + 3, dim - 9, dim - 8, dim - 1], device=DEV)
    er, es, tol = _reference(ids, d_out[:, cols].cpu(), R, 0.75)
    d = E.embed_desc(R, n, dim, E.F32, ot, 0.75)
    size = E.engram_embed_grad_workspace_size(d)
    ws = torch.full((size,), 0xA5, dtype=torch.uint8, device=DEV)
    rows = torch.full((n,), 99, dtype=torch.int64, device=DEV)
    grad = torch.full((n, dim), 7.0, device=DEV)
    count = torch.full((1,), 99, dtype=torch.int64, device=DEV)
    dids = ids.to(DEV)
    E.engram_embed_grad(d, d_out, dids, rows, grad, count, ws, size)
    full = torch.full((R, dim), 3.0, device=DEV)
    E.engram_embed_grad_dense(d, d_out, dids, full, 0, ws, size)
    torch.cuda.synchronize()
    assert int(count) == er.size
    assert np.array_equal(rows[:er.size].cpu().numpy(), er) and (rows[er.size:] == -1).all()
    assert ((grad[:er.size][:, cols].double().cpu() - es).abs() <= tol).all()
    assert (grad[er.size:] == 7.0).all()
    touched = torch.from_numpy(er).to(DEV)
    assert torch.equal(full[touched], grad[:er.size])
    full[touched] = 0
    assert (full == 0).all()


# ---- the widest rows, the most values, special values --------------------------------

@pytest.mark.parametrize("ot", [E.BF16, E.F32])
@pytest.mark.parametrize("dim", [E.MAX_EMBED_DIM, E.MAX_EMBED_DIM - 1, 20_004, 16_392])
def test_the_widest_rows(ot, dim):
    """Rows of up to 32768 values: lookup, and gradients of a row named 1, 20 and 700 times."""
    say("embed, grad: wide rows", ot, dim)
    R, scale = 40, 1.25
    ids = np.repeat([39, 3, 17, 0, 22], [700, 20, 1, 130, 9])
    ids = torch.from_numpy(np.random.default_rng(dim).permutation(np.append(ids, [-1, R])).astype(np.int64))
    n = ids.numel()
    table = _rand((R, dim), 1, TYPES[ot])
    got = _embed(table.to(DEV), ids.to(DEV), dim, ot, ot, scale).cpu()
    ok = (ids >= 0) & (ids < R)
    want = (table[ids[ok]].float() * scale).to(TYPES[ot])
    assert torch.equal(got[ok], want) and (got[~ok] == 0).all()
    d_out = _rand((n, dim), 2, TYPES[ot])
    rows, grad = _check_sparse(ids, d_out, R, dim, ot, scale)
    full = _grad(ids, d_out, R, dim, ot, scale, dense=(torch.full((R, dim), 3.0, device=DEV), 0)).cpu()
    assert torch.equal(full[rows[:5]], grad[:5])


def test_embed_more_values_than_one_sweep_of_threads():
    """2.2e9 values one at a time: threads take a second turn, and the output passes 2^31."""
    say("embed: 2.2e9 values")
    n, dim, R = 314_600_003, 7, 1000
    ids = torch.arange(n, device=DEV).remainder_(R + 1)          # every 1001st outside the table
    table = _rand((R, dim), 4, torch.bfloat16).to(DEV)
    out = torch.full((n, dim), 9.0, dtype=torch.bfloat16, device=DEV)
    E.engram_embed(E.embed_desc(R, n, dim, E.BF16, E.BF16, 1.0), table, ids, out)
    torch.cuda.synchronize()
    padded = torch.cat((table, torch.zeros((1, dim), dtype=torch.bfloat16, device=DEV)))
    for a in list(range(0, n, 40_000_000)) + [n - 5000]:
        part = slice(a, min(n, a + 3_000_000))
        assert torch.equal(out[part], padded[ids[part]])


@pytest.mark.parametrize("n,dim", [(3000, 40), (3000, 7), (50_000, 24), (1_050_000, 256)])
def test_grad_special_values_stay_in_their_row_and_column(n, dim):
    """Infinities and NaN at kept ids reach the sums of their own row and column alone, in
    rows named once and thousands of times."""
    say("grad: NaN and infinity at kept ids", n, dim)
    R = 500
    ids = _ids(n, R, "zipf", 60, drop=0.05)
    g = torch.Generator(device=DEV).manual_seed(n)
    d_out = torch.empty((n, dim), device=DEV).normal_(generator=g)
    kept = ((ids >= 0) & (ids < R)).nonzero()[:, 0]
    spots = [(int(kept[k * len(kept) // 9]), (k * 5) % dim) for k in range(9)]
    bad = torch.zeros((R, dim), dtype=torch.bool)
    for k, (i, c) in enumerate(spots):
        d_out[i, c] = (float("nan"), float("inf"), float("-inf"))[k % 3]
        bad[ids[i], c] = True
    full = _grad(ids, d_out, R, dim, E.F32, 0.5, dense=(torch.empty((R, dim), device=DEV), 0)).cpu()
    assert torch.equal(~torch.isfinite(full), bad)
