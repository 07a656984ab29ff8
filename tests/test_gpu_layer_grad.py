"""The gate's gradient and the projection weight's gradient against 64-bit references.

Gate: every output is compared element by element with the formula in float64 from the same
saved values, within a bound added up from the roundings, with u = 2^-24. A sum over a row
passes a term through at most 30 fp32 additions (8 in a thread, 6 levels of a wave, up to
16 waves): 30 u of the sum of magnitudes. So the root mean squares are off by at most
17 u of their values (half of 30, the division and the root), s by 40 u plus what its sum D
loses, at most 2^-33 of the sum of its terms' magnitudes; alpha' by 80 u + 20 |z| u (half
of s in the root, z in the exponential, and single operations); d_out . v by 30 u of its
magnitudes. The result's own type adds half a step. The learned scales' gradients add the
tokens one by one within a block and then the blocks' parts: (tokens / 256 + 520) u of the
magnitudes.

Weight: e_scales e rounded to fp32 and then to bf16 is reproduced exactly; its products
with bf16 are exact, and each of the fp32 additions is off by at most 2^-23 of the sum of
magnitudes."""
import math

import numpy as np
import pytest

from tests.gpu_util import say

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("no GPU", allow_module_level=True)

import hashed_gram_conditional_amd as E  # noqa: E402

DEV = "cuda"
U = 2.0 ** -24
TYPES = {E.BF16: torch.bfloat16, E.F32: torch.float32}
VOCAB = 1000


def half_step(t):
    return torch.finfo(t).eps / 2


# ---- the gate ----------------------------------------------------------------------

def saved_of(shape, kind, seed, scale_kind=E.SCALE_F32, size=1.0):
    """(what the call gets, its scales, the values in float64)"""
    g = torch.Generator(device=DEV).manual_seed(seed)
    x = torch.randn(shape, generator=g, device=DEV) * torch.exp2(
        torch.randn((*shape[:-1], 1), generator=g, device=DEV)) * size
    if kind != E.I8:
        x = x.to(TYPES[kind])
        return x, None, x.double()
    dim, rows = shape[-1], math.prod(shape[:-1])
    out = -(-dim // 16) * 16
    codes = torch.empty((*shape[:-1], out), dtype=torch.int8, device=DEV)
    scales = torch.empty(shape[:-1], device=DEV)
    E.engram_quantize_i8(x, E.F32, rows, dim, 0, out, scale_kind, codes, scales)
    return codes, scales, codes[..., :dim].double() * scales.double()[..., None]


class Case:
    def __init__(self, tokens, hc, dim, fmt=E.BF16, kv=E.I8, h=E.I8, plain=False, clamp=0.0, dead=0.1, eps=1e-6,
                 scale_kind=E.SCALE_F32, seed=0, batch=1):
        self.t, self.hc, self.dim, self.fmt, self.plain, self.clamp, self.eps = tokens, hc, dim, fmt, plain, clamp, eps
        self.kv_type, self.h_type, self.type = kv, h, TYPES[fmt]
        self.kv, self.kv_scales, self.kv64 = saved_of((tokens, hc + 1, dim), kv, seed + 1, scale_kind)
        self.h, self.h_scales, self.h64 = saved_of((tokens, hc, dim), h, seed + 2, scale_kind)
        g = torch.Generator(device=DEV).manual_seed(seed)
        rand = lambda *s: torch.randn(s, generator=g, device=DEV)      # noqa: E731
        self.q_w, self.k_w = 1 + 0.3 * rand(hc, dim), 1 + 0.3 * rand(hc, dim)
        self.d_out = (0.01 * rand(tokens, hc, dim)).to(self.type)
        self.ids = torch.randint(0, VOCAB, (tokens,), generator=g, device=DEV, dtype=torch.int32)
        self.ids[torch.rand(tokens, generator=g, device=DEV) < dead] = -1
        self.desc = E.forward_desc(batch, tokens // batch, hc, dim, 0,
                                   E.ROW_F32 if fmt == E.F32 else E.ROW_E4M3_E8M0_264, 256, eps, clamp,
                                   E.GATE_PLAIN if plain else E.GATE_SIGNED_SQRT)

    def saved(self):
        return E.gate_saved(self.kv, self.kv_type, self.kv_scales, self.h, self.h_type, self.h_scales)

    def run(self, accumulate=0, d_q_w=None, d_k_w=None, in_place=False, weights=True):
        t, hc, dim = self.t, self.hc, self.dim
        pad = 64

        def guarded(n, dtype):
            return torch.full((n + pad,), 9.0, dtype=dtype, device=DEV)

        d_kv, d_h = guarded(t * (hc + 1) * dim, self.type), guarded(t * hc * dim, self.type)
        d_out = self.d_out
        if in_place:
            d_h[:-pad] = d_out.reshape(-1)
            d_out = d_h
        if weights and d_q_w is None:
            d_q_w, d_k_w = (torch.full((hc, dim), 5.0, device=DEV) for _ in range(2))
        size = E.engram_gate_grad_workspace_size(self.desc)
        ws = torch.full((size + 256,), 0xAB, dtype=torch.uint8, device=DEV) if weights else None
        E.engram_gate_grad(self.desc, self.ids, VOCAB, self.saved(), self.q_w, self.k_w, d_out, d_h, d_kv, d_q_w,
                           d_k_w, accumulate, ws, size if weights else 0)
        torch.cuda.synchronize()
        assert (d_kv[-pad:] == 9.0).all() and (d_h[-pad:] == 9.0).all()
        assert ws is None or (ws[size:] == 0xAB).all()
        return (d_h[:-pad].reshape(t, hc, dim), d_kv[:-pad].reshape(t, hc + 1, dim), d_q_w, d_k_w)

    def reference(self):
        """The gradients in float64 and how far each may be off before its rounding."""
        hc, dim = self.hc, self.dim
        h, k, v, d = self.h64, self.kv64[:, :hc], self.kv64[:, hc:], self.d_out.double()
        w = self.q_w.double() * self.k_w.double()
        rh = 1 / torch.sqrt(h.square().mean(-1) + self.eps)
        rk = 1 / torch.sqrt(k.square().mean(-1) + self.eps)
        D, mag = (h * w * k).sum(-1), (h * w * k).abs().sum(-1)
        s = D * rh * rk / math.sqrt(dim)
        on = (s.abs() > self.clamp) if not self.plain else torch.ones_like(s, dtype=torch.bool)
        root = torch.sqrt(torch.clamp(s.abs(), min=self.clamp))
        z = s if self.plain else torch.where(s < 0, -root, root)
        alpha = torch.sigmoid(z)
        slope = alpha * (1 - alpha)
        if not self.plain:
            slope = torch.where(on, slope / (2 * torch.where(on, root, 1.0)), 0.0)
        live = ((self.ids >= 0) & (self.ids < VOCAB))[:, None]
        alpha = torch.where(live, alpha, 0.0)
        dv, dv_mag = (d * v).sum(-1), (d * v).abs().sum(-1)
        norm = slope * rh * rk / math.sqrt(dim) * live
        c1 = dv * norm
        rel = 80 * U + 20 * z.abs() * U + (1 + z.abs()) * 2.0 ** -33 * mag / D.abs().clamp(min=1e-300)
        dc1 = c1.abs() * rel + norm.abs() * 30 * U * dv_mag
        Bh, Bk = D * rh * rh / dim, D * rk * rk / dim
        c1, dc1 = c1[..., None], dc1[..., None]
        th, tk = (k * w).abs() + (Bh[..., None] * h).abs(), (h * w).abs() + (Bk[..., None] * k).abs()
        d_h = d + c1 * (k * w - Bh[..., None] * h)
        d_k = c1 * (h * w - Bk[..., None] * k)
        e_h = dc1 * th + c1.abs() * 48 * U * th + 4 * U * (d.abs() + d_h.abs())
        e_k = dc1 * tk + c1.abs() * 48 * U * tk + 4 * U * d_k.abs()
        d_v = (alpha[..., None] * d).sum(1, keepdim=True)
        e_a = alpha * (8 * U + (1 - alpha) * (40 * z.abs() * U + 2.0 ** -33 * mag / D.abs().clamp(min=1e-300) * z.abs()))
        e_v = ((e_a + 8 * U * alpha)[..., None] * d.abs()).sum(1, keepdim=True)
        d_w = (c1 * h * k).sum(0)
        m_w = (c1 * h * k).abs()
        e_w = (dc1 * (h * k).abs()).sum(0) + (4 + self.t / 256 + 520) * U * m_w.sum(0)
        tiny = 1e-37       # products below the smallest fp32
        return dict(d_h=(d_h, e_h + tiny), d_kv=(torch.cat((d_k, d_v), 1), torch.cat((e_k, e_v), 1) + tiny),
                    d_q_w=(d_w * self.k_w.double(), e_w * self.k_w.abs().double() + tiny),
                    d_k_w=(d_w * self.q_w.double(), e_w * self.q_w.abs().double() + tiny))


def check_gate(case, **kw):
    got = dict(zip(("d_h", "d_kv", "d_q_w", "d_k_w"), case.run(**kw)))
    for name, (want, err) in case.reference().items():
        x = got[name]
        if x is None:
            continue
        tol = err * (1 + 2.0 ** -7) + half_step(x.dtype) * (want.abs() + err)
        off = (x.double() - want).abs()
        bad = ~(off <= tol)
        assert not bad.any(), (name, int(bad.sum()), bad.nonzero()[0].tolist(), float(off[bad][0]), float(tol[bad][0]))
    return got


@pytest.mark.parametrize("fmt,kv,h", [(f, kv, h) for f in (E.BF16, E.F32) for kv in (f, E.I8) for h in (f, E.I8)])
@pytest.mark.parametrize("tokens,hc,dim", [(1, 1, 8), (1, 4, 5120), (3, 2, 24), (7, 4, 64), (64, 1, 64), (130, 3, 520),
                                           (517, 4, 136), (1100, 2, 1000), (40, 8, 1024), (9, 5, 8192), (700, 4, 512),
                                           (2100, 8, 64), (600, 6, 2048), (33, 7, 3656), (300, 5, 4096), (5, 4, 6400),
                                           (1300, 2, 2056), (90, 3, 4616), (2, 8, 8192), (1500, 8, 32), (20, 8, 3200)])
def test_gate_gradient(tokens, hc, dim, fmt, kv, h):
    say("gate_grad", tokens, hc, dim, fmt, kv, h)
    check_gate(Case(tokens, hc, dim, fmt, kv, h, seed=tokens + dim))


@pytest.mark.parametrize("fmt", [E.BF16, E.F32])
@pytest.mark.parametrize("plain,clamp", [(True, 0.0), (False, 0.01), (False, 0.5), (False, 100.0)])
def test_gate_gradient_modes(plain, clamp, fmt):
    say("gate_grad: modes", plain, clamp, fmt)
    for scale_kind in (E.SCALE_F32, E.SCALE_POW2):
        check_gate(Case(211, 4, 256, fmt, E.I8, fmt, plain, clamp, scale_kind=scale_kind, seed=3))


@pytest.mark.parametrize("dead", [0.0, 1.0])
def test_gate_gradient_dead_positions(dead):
    """Every position DEAD: d_out passes, the rest is zero; none DEAD."""
    say("gate_grad: dead", dead)
    got = check_gate(Case(300, 3, 320, dead=dead, seed=5))
    if dead:
        assert not got["d_kv"].any() and not got["d_q_w"].any() and not got["d_k_w"].any()


def test_gate_gradient_dead_rows_may_hold_anything():
    say("gate_grad: NaN and infinities at DEAD positions")
    for kv, h in ((E.BF16, E.BF16), (E.I8, E.I8), (E.BF16, E.I8)):
        case = Case(90, 4, 136, E.BF16, kv, h, dead=0.4, seed=8)
        want = case.run()
        gone = (case.ids < 0).nonzero().flatten()
        for saved, scales in ((case.kv, case.kv_scales), (case.h, case.h_scales)):
            if scales is None:
                saved[gone[::2]] = float("nan")
                saved[gone[1::2]] = float("inf")
            else:
                scales[gone] = float("nan")
        for a, b in zip(case.run(), want):
            assert torch.equal(a, b)


@pytest.mark.parametrize("fmt,kv,h", [(E.BF16, E.I8, E.I8), (E.F32, E.I8, E.F32), (E.BF16, E.BF16, E.I8)])
@pytest.mark.parametrize("hc,dim", [(4, 136), (2, 1000), (5, 8192)])
def test_gate_gradient_of_rows_that_hold_nan(fmt, kv, h, hc, dim):
    """At a position that is not DEAD a key that holds a NaN makes the gradients of its stream and of the value
    NaN, and those of the learned scales; the position's other streams and the other positions keep theirs."""
    say("gate_grad: NaN in a key", fmt, kv, h, hc, dim)
    for plain in (False, True):
        case = Case(60, hc, dim, fmt, kv, h, plain=plain, dead=0.0, seed=17)
        want = case.run()
        if kv == E.I8:
            case.kv_scales[7, 1] = float("nan")
        else:
            case.kv[7, 1, 5] = float("nan")
        d_h, d_kv, d_q, d_k = case.run()
        assert torch.isnan(d_h[7, 1]).all() and torch.isnan(d_kv[7, 1]).all() and torch.isnan(d_kv[7, hc]).all()
        assert torch.isnan(d_q[1]).all() and torch.isnan(d_k[1]).all()
        d_h[7, 1], d_kv[7, 1], d_kv[7, hc] = want[0][7, 1], want[1][7, 1], want[1][7, hc]
        d_q[1], d_k[1] = want[2][1], want[3][1]
        for a, b in zip((d_h, d_kv, d_q, d_k), want):
            assert torch.equal(a, b)


def test_gate_gradient_raw_ids_outside_the_vocabulary():
    say("gate_grad: ids")
    case = Case(20, 2, 64, dead=0.0, seed=1)
    case.ids[3], case.ids[5], case.ids[7] = VOCAB, 2 ** 31 - 1, -2 ** 31
    got = check_gate(case)
    for t in (3, 5, 7):
        assert torch.equal(got["d_h"][t], case.d_out[t]) and not got["d_kv"][t].any()


def test_gate_gradient_in_place_without_weights_and_added():
    say("gate_grad: in place, without weights, accumulated")
    case = Case(333, 4, 512, dead=0.3, seed=11)
    d_h, d_kv, d_q, d_k = check_gate(case).values()
    a = case.run(in_place=True)
    assert torch.equal(a[0], d_h) and torch.equal(a[1], d_kv) and torch.equal(a[2], d_q)
    b = case.run(weights=False)
    assert torch.equal(b[0], d_h) and torch.equal(b[1], d_kv) and b[2] is None
    q0, k0 = torch.randn_like(d_q), torch.randn_like(d_k)
    c = case.run(accumulate=1, d_q_w=q0.clone(), d_k_w=k0.clone())
    assert torch.equal(c[2], q0 + d_q) and torch.equal(c[3], k0 + d_k)


def test_gate_gradient_zero_products_under_a_clamp():
    """s = 0 with a clamp above 0: the gate is sigmoid(sqrt(clamp)) there, as the forward pass has it,
    and the root's derivative 0, so that the streams' gradient is d_out and the keys' is 0."""
    say("gate_grad: s = 0 under a clamp")
    clamp = 0.04
    for hc, dim in ((2, 64), (5, 8192)):
        for kv in (E.BF16, E.I8):
            case = Case(8, hc, dim, E.BF16, kv, E.BF16, clamp=clamp, dead=0.0, seed=2)
            zero = [(1, 0), (2, 1), (3, 0)]
            case.kv[1, 0], case.kv64[1, 0] = 0, 0.0
            case.h[2, 1], case.h64[2, 1] = 0.0, 0.0
            case.kv[3, 0], case.kv64[3, 0] = 0, 0.0
            case.h[3, 0], case.h64[3, 0] = 0.0, 0.0
            if kv == E.BF16:                       # disjoint halves
                zero.append((4, 1))
                case.kv[4, 1, :dim // 2], case.kv64[4, 1, :dim // 2] = 0.0, 0.0
                case.h[4, 1, dim // 2:], case.h64[4, 1, dim // 2:] = 0.0, 0.0
            got = check_gate(case)
            for t, m in zero:
                assert torch.equal(got["d_h"][t, m], case.d_out[t, m]) and not got["d_kv"][t, m].any()
            if kv == E.BF16:
                alpha = torch.empty((8, hc), device=DEV)
                E.engram_gate(case.desc, case.ids, VOCAB, case.kv, case.q_w, case.k_w, case.h.clone(), alpha)
                torch.cuda.synchronize()
                # a root, an exponential of at most 1, a sum and a division
                want = 1 / (1 + math.exp(-math.sqrt(clamp)))
                assert all(abs(float(alpha[t, m]) - want) <= 16 * U for t, m in zero)


@pytest.mark.parametrize("fmt,kv,h", [(E.BF16, E.I8, E.I8), (E.F32, E.F32, E.I8), (E.BF16, E.BF16, E.BF16)])
@pytest.mark.parametrize("hc,dim", [(4, 136), (2, 1000), (5, 8192)])
def test_gate_gradient_of_streams_and_values_that_hold_nan(fmt, kv, h, hc, dim):
    """A NaN in a stream's saved row or scale does to the gradients what one in its key does. One in
    the value's row or scale makes those of the position's streams and keys NaN, and the learned scales';
    the value's own gradient, which does not depend on the value, and the other positions keep theirs."""
    say("gate_grad: NaN in a stream and in the value", fmt, kv, h, hc, dim)
    for plain in (False, True):
        for broken in ("stream", "value"):
            case = Case(60, hc, dim, fmt, kv, h, plain=plain, dead=0.0, seed=18)
            want = case.run()
            if broken == "stream":
                if h == E.I8:
                    case.h_scales[7, 1] = float("nan")
                else:
                    case.h[7, 1, 5] = float("nan")
            elif kv == E.I8:
                case.kv_scales[7, hc] = float("nan")
            else:
                case.kv[7, hc, 5] = float("nan")
            d_h, d_kv, d_q, d_k = case.run()
            streams = slice(1, 2) if broken == "stream" else slice(0, hc)
            assert torch.isnan(d_h[7, streams]).all() and torch.isnan(d_kv[7, streams]).all()
            assert torch.isnan(d_q[streams]).all() and torch.isnan(d_k[streams]).all()
            d_h[7, streams], d_kv[7, streams] = want[0][7, streams], want[1][7, streams]
            d_q[streams], d_k[streams] = want[2][streams], want[3][streams]
            if broken == "stream":
                assert torch.isnan(d_kv[7, hc]).all()
                d_kv[7, hc] = want[1][7, hc]
            for a, b in zip((d_h, d_kv, d_q, d_k), want):
                assert torch.equal(a, b)


@pytest.mark.parametrize("fmt,kv,h,t,hc,dim", [(E.BF16, E.I8, E.I8, 5000, 4, 136), (E.BF16, E.BF16, E.BF16, 1100, 4, 2056),
                                               (E.F32, E.I8, E.F32, 1300, 2, 2056), (E.BF16, E.I8, E.BF16, 700, 4, 6400),
                                               (E.BF16, E.I8, E.I8, 3000, 8, 32)])
def test_gate_gradient_in_place_over_many_turns(fmt, kv, h, t, hc, dim):
    """Several tokens a block, of which the next ones' rows are requested before this one's are stored."""
    say("gate_grad: in place, several tokens a block", fmt, kv, h, t, hc, dim)
    case = Case(t, hc, dim, fmt, kv, h, dead=0.2, seed=19)
    want = case.run()
    for a, b in zip(case.run(in_place=True), want):
        assert torch.equal(a, b)


def test_gate_gradient_of_no_tokens():
    say("gate_grad: no tokens")
    desc = E.forward_desc(2, 0, 2, 64, 0, E.ROW_E4M3_E8M0_264, 256)
    w = torch.ones((2, 64), device=DEV)
    empty = torch.empty(0, dtype=torch.bfloat16, device=DEV)
    saved = E.gate_saved(None, E.I8, None, None, E.I8, None)
    for accumulate, want in ((1, 5.0), (0, 0.0)):
        q, k = (torch.full((2, 64), 5.0, device=DEV) for _ in range(2))
        E.engram_gate_grad(desc, empty, VOCAB, saved, w, w, empty, empty, empty, q, k, accumulate, None, 0)
        torch.cuda.synchronize()
        assert (q == want).all() and (k == want).all()


def test_gate_gradient_zero_rows_and_zero_products():
    """Zero keys, zero streams and streams orthogonal to their keys: s = 0, where the
    root's derivative is taken as 0, and the plain gate's is 1/4."""
    say("gate_grad: s = 0")
    for plain in (False, True):
        for kv in (E.BF16, E.I8):
            case = Case(8, 2, 64, E.BF16, kv, E.BF16, plain=plain, dead=0.0, seed=2)
            case.kv[1, 0], case.kv64[1, 0] = 0, 0.0
            case.h[2, 1], case.h64[2, 1] = 0.0, 0.0
            case.kv[3, 0], case.kv64[3, 0] = 0, 0.0
            case.h[3, 0], case.h64[3, 0] = 0.0, 0.0
            if kv == E.BF16:                       # disjoint halves
                case.kv[4, 1, :32], case.kv64[4, 1, :32] = 0.0, 0.0
                case.h[4, 1, 32:], case.h64[4, 1, 32:] = 0.0, 0.0
            got = check_gate(case)
            assert all(torch.isfinite(x).all() for x in got.values())


def test_gate_gradient_where_the_terms_cancel():
    """s down to 1e-7 of its terms: the root's derivative needs D to many more digits
    than fp32 sums of it would keep."""
    say("gate_grad: cancellation")
    for kv, h in ((E.BF16, E.BF16), (E.I8, E.I8), (E.F32, E.F32)):
        fmt = E.F32 if kv == E.F32 else E.BF16
        case = Case(200, 2, 1024, fmt, kv, h, dead=0.0, seed=21)
        # weights of the second half that make D small: scaled so that the halves cancel
        w = case.q_w.double() * case.k_w.double()
        part = (case.h64 * w * case.kv64[:, :2])
        low, high = part[..., :512].sum(-1), part[..., 512:].sum(-1)
        case.k_w[0, 512:] *= float(-(low / high)[0, 0])
        case.k_w[1, 512:] *= float(-(low / high)[1, 1])
        w = case.q_w.double() * case.k_w.double()
        part = (case.h64 * w * case.kv64[:, :2])
        share = float((part.sum(-1).abs() / part.abs().sum(-1))[0, 0])
        assert share < 1e-6
        check_gate(case)


def test_gate_gradient_against_differences():
    """Directional derivatives of the forward formula in float64 by central differences,
    whose error falls with the fourth power of the step after one extrapolation."""
    say("gate_grad: differences")
    for plain in (False, True):
        case = Case(12, 3, 96, E.F32, E.F32, E.F32, plain=plain, dead=0.2, seed=4)
        d_h, d_kv, d_q, d_k = (x.double() for x in case.run())
        base = dict(h=case.h64, kv=case.kv64, q=case.q_w.double(), k=case.k_w.double())
        live = ((case.ids >= 0) & (case.ids < VOCAB))[:, None, None]

        def loss(p):
            h, k, v = p["h"], p["kv"][:, :3], p["kv"][:, 3:]
            nh = h / torch.sqrt(h.square().mean(-1, keepdim=True) + case.eps)
            nk = k / torch.sqrt(k.square().mean(-1, keepdim=True) + case.eps)
            s = (nh * nk * p["q"] * p["k"]).sum(-1, keepdim=True) / math.sqrt(96)
            z = s if plain else torch.sign(s) * torch.sqrt(s.abs())
            return ((h + torch.where(live, torch.sigmoid(z) * v, 0.0)) * case.d_out.double()).sum()

        g = torch.Generator(device=DEV).manual_seed(6)
        for name, grad in (("h", d_h), ("kv", d_kv), ("q", d_q), ("k", d_k)):
            u = torch.randn(base[name].shape, generator=g, device=DEV, dtype=torch.float64)
            slopes = []
            for step in (2e-5, 1e-5):
                up, down = (loss({**base, name: base[name] + x * step * u}) for x in (1, -1))
                slopes.append(float((up - down) / (2 * step)))
            want = (4 * slopes[1] - slopes[0]) / 3
            got = float((grad * u).sum())
            size = float((grad * u).abs().sum())
            assert abs(got - want) <= 1e-5 * size + 1e-8, (plain, name, got, want, size)


def test_gate_gradient_repeats_its_bits_on_streams_and_replays():
    say("gate_grad: streams and graphs")
    cases = [Case(300, 4, 1024, seed=31), Case(77, 2, 520, E.F32, E.I8, E.F32, seed=32)]
    want = [c.run() for c in cases]
    bufs = []
    for c, x in zip(cases, want):
        size = E.engram_gate_grad_workspace_size(c.desc)
        bufs.append((*[torch.empty_like(y) for y in x], torch.empty(size, dtype=torch.uint8, device=DEV), size))

    def call(c, b):
        E.engram_gate_grad(c.desc, c.ids, VOCAB, c.saved(), c.q_w, c.k_w, c.d_out, b[0], b[1], b[2], b[3], 0, b[4],
                           b[5])

    streams = [torch.cuda.Stream() for _ in cases]
    torch.cuda.synchronize()
    for _ in range(4):
        for s, c, b in zip(streams, cases, bufs):
            with torch.cuda.stream(s):
                call(c, b)
    torch.cuda.synchronize()
    for b, x in zip(bufs, want):
        assert all(torch.equal(p, q) for p, q in zip(b, x))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        for c, b in zip(cases, bufs):
            call(c, b)
    for turn in range(4):
        for c, b in zip(cases, bufs):
            c.d_out.copy_(torch.randn_like(c.d_out.float()) * 0.01)
            c.ids[turn] = -1
            for x in b[:4]:
                x.fill_(3.0)
        graph.replay()
        torch.cuda.synchronize()
        got = [[x.clone() for x in b[:4]] for b in bufs]
        for c, x in zip(cases, got):
            assert all(torch.equal(p, q) for p, q in zip(c.run(), x))


def test_gate_gradient_offsets_beyond_32_bits():
    """2.2e9 values of d_kv: the last tokens against the same tokens alone."""
    say("gate_grad: offsets beyond 2^31")
    t, hc, dim = 90000, 4, 5120
    case = Case(2, hc, dim, dead=0.0, seed=41)
    d_h2, d_kv2, _, _ = case.run(weights=False)
    big = Case.__new__(Case)
    kv = torch.zeros((t, hc + 1, dim), dtype=torch.int8, device=DEV)
    h = torch.zeros((t, hc, dim), dtype=torch.int8, device=DEV)
    kvs, hs = torch.zeros((t, hc + 1), device=DEV), torch.zeros((t, hc), device=DEV)
    kv[-2:], h[-2:], kvs[-2:], hs[-2:] = case.kv, case.h, case.kv_scales, case.h_scales
    d_out = torch.zeros((t, hc, dim), dtype=torch.bfloat16, device=DEV)
    d_out[-2:] = case.d_out
    ids = torch.full((t,), 1, dtype=torch.int32, device=DEV)
    desc = E.forward_desc(1, t, hc, dim, 0, E.ROW_E4M3_E8M0_264, 256)
    d_kv = torch.empty((t, hc + 1, dim), dtype=torch.bfloat16, device=DEV)
    E.engram_gate_grad(desc, ids, VOCAB, E.gate_saved(kv, E.I8, kvs, h, E.I8, hs), case.q_w, case.k_w, d_out, d_out,
                       d_kv, None, None, 0, None, 0)
    torch.cuda.synchronize()
    assert torch.equal(d_kv[-2:], d_kv2) and torch.equal(d_out[-2:], d_h2)
    assert not d_kv[:-2].any() and not d_out[:-2].any()
    del big


# ---- the projection's weight -------------------------------------------------------

def weight_case(t, k, n, seed=0, kind=E.SCALE_F32):
    g = torch.Generator(device=DEV).manual_seed(seed)
    d_kv = torch.randn((t, n), generator=g, device=DEV).to(torch.bfloat16)
    codes = torch.randint(-128, 128, (t, k), generator=g, device=DEV, dtype=torch.int16).to(torch.int8)
    scales = torch.exp2(torch.randn(t, generator=g, device=DEV))
    if kind == E.SCALE_POW2:
        scales = (scales.view(torch.int32) & 0x7F800000).view(torch.float32)
    return d_kv, codes, scales


def weight_grad(d_kv, codes, scales, grad_type, accumulate=0, grad=None, workspace=True):
    t, n = d_kv.shape
    k = codes.shape[1]
    out = torch.full((n * k + 64,), 9.0, dtype=TYPES[grad_type], device=DEV)
    if grad is not None:
        out[:n * k] = grad.reshape(-1)
    size = E.engram_project_grad_workspace_size(t, k, n) if workspace else 0
    ws = torch.full((size + 256,), 0xAB, dtype=torch.uint8, device=DEV) if size else None
    E.engram_project_grad(d_kv, codes, scales, out, grad_type, accumulate, t, k, n, ws, size)
    torch.cuda.synchronize()
    assert (out[n * k:] == 9.0).all()
    assert ws is None or (ws[size:] == 0xAB).all()
    return out[:n * k].reshape(n, k)


def check_weight(d_kv, codes, scales, grad_type, **kw):
    t = d_kv.shape[0]
    e = (scales[:, None] * codes.float()).to(torch.bfloat16).double()
    d = d_kv.double()
    dt = d.t().contiguous()
    want, mag = dt @ e, dt.abs() @ e.abs()
    err = (t + 8) * 2.0 ** -23 * mag
    tol = err + half_step(TYPES[grad_type]) * (want.abs() + err) + 1e-37
    got = weight_grad(d_kv, codes, scales, grad_type, **kw)
    off = (got.double() - want).abs()
    assert (off <= tol).all(), (float((off - tol).max()), (off > tol).nonzero()[0].tolist())
    return got


@pytest.mark.parametrize("grad_type", [E.BF16, E.F32])
@pytest.mark.parametrize("t,k,n", [
    (1, 16, 8), (2, 48, 24), (15, 112, 40), (16, 128, 64), (17, 144, 72), (31, 256, 136), (33, 272, 128),
    (63, 1040, 200), (64, 384, 520), (65, 512, 256), (100, 640, 264), (127, 6144, 320), (128, 1024, 1000),
    (129, 896, 776), (257, 2064, 1288), (509, 176, 2056), (1003, 768, 1032), (5000, 80, 48), (4096, 256, 512)])
def test_weight_gradient(t, k, n, grad_type):
    say("project_grad", t, k, n, grad_type)
    case = weight_case(t, k, n, seed=t + k)
    a = check_weight(*case, grad_type)
    check_weight(*case, grad_type, workspace=False)
    assert torch.equal(a, weight_grad(*case, grad_type))


@pytest.mark.parametrize("t", [1, 7, 33, 64, 96, 100, 128, 160, 192, 193, 224, 256, 300, 320, 384, 448, 511])
@pytest.mark.parametrize("k,n", [(48, 40), (304, 520)])
def test_weight_gradient_whole_numbers(t, k, n):
    """Whole numbers whose sums stay below 2^24 are exact, whatever the order."""
    say("project_grad: whole numbers", t, k, n)
    g = torch.Generator(device=DEV).manual_seed(t)
    d = torch.randint(-8, 9, (t, n), generator=g, device=DEV).to(torch.bfloat16)
    codes = torch.randint(-128, 128, (t, k), generator=g, device=DEV, dtype=torch.int16).to(torch.int8)
    one = torch.ones(t, device=DEV)
    want = d.double().t().contiguous() @ codes.double()
    got = weight_grad(d, codes, one, E.F32)
    assert torch.equal(got.double(), want)
    # a power of two is exact as well, and gradients are added to what is there
    base = torch.randint(-100, 100, (n, k), generator=g, device=DEV).float()
    got = weight_grad(d, codes, one * 0.25, E.F32, accumulate=1, grad=base)
    assert torch.equal(got.double(), want * 0.25 + base.double())


def test_weight_gradient_added_to_bf16():
    say("project_grad: accumulate in bf16")
    case = weight_case(200, 272, 264, seed=3, kind=E.SCALE_POW2)
    base = torch.randn((264, 272), device=DEV).to(torch.bfloat16)
    plain = weight_grad(*case, E.F32)
    got = weight_grad(*case, E.BF16, accumulate=1, grad=base)
    assert torch.equal(got, (plain + base.float()).to(torch.bfloat16))


TYPES[E.F32_FINE] = torch.float32


@pytest.mark.parametrize("grad_type", [E.BF16, E.F32, E.F32_FINE])
@pytest.mark.parametrize("kind", [E.SCALE_F32, E.SCALE_POW2])
@pytest.mark.parametrize("t,k,n", [(1, 48, 24), (65, 512, 256), (509, 176, 1032), (4096, 256, 512)])
def test_weight_gradient_of_the_unrounded_values(t, k, n, kind, grad_type):
    """Against e_scales e itself. Rounded to bf16, a value is off by at most 2^-8 of itself, and by
    2^-24 in fp32 before; powers of two leave it as it is. The second of two terms is what the first
    drops, at most 2^-8 of the value's power of two, so that a step of bf16 is at most 2^-16 there, and
    a rounding 2^-17. What the sum adds is at most 2^-23 of the terms' magnitudes for each of them, which
    are within 1 + 2^-7 of the unrounded values'."""
    say("project_grad: unrounded values", t, k, n, kind, grad_type)
    d_kv, codes, scales = weight_case(t, k, n, seed=t + k, kind=kind)
    e, dt = scales.double()[:, None] * codes.double(), d_kv.double().t().contiguous()
    want, mag = dt @ e, dt.abs() @ e.abs()
    fine = grad_type == E.F32_FINE
    part = 0.0 if kind == E.SCALE_POW2 else (2.0 ** -17 if fine else 2.0 ** -8) + 2.0 ** -23
    err = ((t + 8) * (2 if fine else 1) * 2.0 ** -23 * (1 + 2.0 ** -7) + part) * mag
    got = weight_grad(d_kv, codes, scales, grad_type)
    off = (got.double() - want).abs()
    tol = err + half_step(TYPES[grad_type]) * (want.abs() + err) + 1e-37
    print("  off by %.2e of the norm" % float(off.norm() / want.norm()), flush=True)
    assert (off <= tol).all(), (float((off - tol).max()), (off > tol).nonzero()[0].tolist())


@pytest.mark.parametrize("t", [1, 7, 31, 32, 33, 64, 65, 96, 100, 128, 129, 160, 192, 224, 256, 300, 511, 1500])
@pytest.mark.parametrize("k,n", [(16, 8), (48, 40), (304, 520)])
def test_weight_gradient_in_two_terms(t, k, n):
    """Whole numbers times 257 / 256 need 16 bits, which two terms hold and one does not. Their sums
    stay below 2^24 (in units of 1 / 256: 1500 x 3 x 14 x 257), so that every order gives the same."""
    say("project_grad: two terms", t, k, n)
    g = torch.Generator(device=DEV).manual_seed(t)
    d = torch.randint(-3, 4, (t, n), generator=g, device=DEV).to(torch.bfloat16)
    codes = torch.randint(-14, 15, (t, k), generator=g, device=DEV, dtype=torch.int16).to(torch.int8)
    scales = torch.full((t,), 257 / 256, device=DEV)
    scales[::3] = 1.0
    want = d.double().t().contiguous() @ (codes.double() * scales.double()[:, None])
    base = torch.randint(-100, 100, (n, k), generator=g, device=DEV).float()
    for workspace in (True, False):
        got = weight_grad(d, codes, scales, E.F32_FINE, workspace=workspace)
        assert torch.equal(got.double(), want)
        got = weight_grad(d, codes, scales, E.F32_FINE, accumulate=1, grad=base, workspace=workspace)
        assert torch.equal(got.double(), want + base.double())


def test_weight_gradient_in_two_terms_of_every_code():
    """The codes from -128 to 127 as whole columns, each against a single token's 1: what comes back is the
    sum of a code's two terms."""
    say("project_grad: two terms of every code")
    codes = torch.arange(-128, 128, device=DEV, dtype=torch.int16).to(torch.int8).repeat(40, 1)
    d = torch.eye(40, device=DEV).to(torch.bfloat16)
    scales = torch.exp2(torch.randn(40, generator=torch.Generator(device=DEV).manual_seed(1), device=DEV) * 20)
    got = weight_grad(d, codes, scales, E.F32_FINE)
    x = scales[:, None] * codes.float()
    high = x.to(torch.bfloat16).float()
    low = (x - high).to(torch.bfloat16).float()
    assert torch.equal(got, high + low)
    # powers of two are exact, as in one term
    scales = (scales.view(torch.int32) & 0x7F800000).view(torch.float32)
    assert torch.equal(weight_grad(d, codes, scales, E.F32_FINE), scales[:, None] * codes.float())


def test_weight_gradient_in_two_terms_not_finite():
    """What is infinite or NaN in one term is so in two: NaN and infinite scales, a product beyond
    fp32's range, one that only its rounding to bf16 takes beyond, and d_kv's own."""
    say("project_grad: two terms, not finite")
    for scale, code in ((3.4e38, 127), (3.4e38 / 64, 64), (float("inf"), -3), (float("nan"), 5)):
        d, c, s = weight_case(70, 160, 136, seed=5)
        d[30], c[30], s[30] = 1.0, code, scale
        got = weight_grad(d, c, s, E.F32_FINE)
        assert (torch.isnan(got) if math.isnan(scale) else got == math.copysign(math.inf, code)).all()
    d, c, s = weight_case(70, 160, 136, seed=5)
    base = weight_grad(d, c, s, E.F32_FINE)
    d[13, 9], d[20, 100] = float("nan"), float("inf")
    got = weight_grad(d, c, s, E.F32_FINE)
    keep = [i for i in range(136) if i not in (9, 100)]
    assert torch.equal(got[keep], base[keep]) and torch.isnan(got[9]).all()
    assert not torch.isfinite(got[100][c[20] != 0]).any()


def test_weight_gradient_in_two_terms_of_no_tokens_far_offsets_and_replays():
    say("project_grad: two terms, no tokens")
    d, c, s = (torch.empty((0, n), dtype=x, device=DEV) for n, x in ((40, torch.bfloat16), (48, torch.int8),
                                                                     (1, torch.float32)))
    one = torch.ones((40, 48), device=DEV)
    assert not weight_grad(d, c, s, E.F32_FINE, grad=one).any()
    assert (weight_grad(d, c, s, E.F32_FINE, accumulate=1, grad=one) == 1).all()

    say("project_grad: two terms, offsets beyond 2^31")
    t, k, n = 88000, 64, 25600           # 2.25e9 values of d_kv
    d = torch.zeros((t, n), dtype=torch.bfloat16, device=DEV)
    c = torch.zeros((t, k), dtype=torch.int8, device=DEV)
    s = torch.full((t,), 257 / 256, device=DEV)
    g = torch.Generator(device=DEV).manual_seed(1)
    d[-3:] = torch.randint(-8, 9, (3, n), generator=g, device=DEV).to(torch.bfloat16)
    c[-3:] = torch.randint(-128, 128, (3, k), generator=g, device=DEV, dtype=torch.int16).to(torch.int8)
    got = weight_grad(d, c, s, E.F32_FINE)
    assert torch.equal(got.double(), d[-3:].double().t().contiguous() @ c[-3:].double() * (257 / 256))
    del d

    say("project_grad: two terms, graphs")
    cases = [weight_case(700, 272, 264, 1), weight_case(333, 1040, 1288, 2)]
    bufs = []
    for d, c, s in cases:
        size = E.engram_project_grad_workspace_size(d.shape[0], c.shape[1], d.shape[1])
        bufs.append((torch.empty((d.shape[1], c.shape[1]), device=DEV),
                     torch.empty(max(size, 256), dtype=torch.uint8, device=DEV), size))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        for x, b in zip(cases, bufs):
            E.engram_project_grad(*x, b[0], E.F32_FINE, 0, x[0].shape[0], x[1].shape[1], x[0].shape[1], b[1], b[2])
    for turn in range(4):
        for x, b in zip(cases, bufs):
            x[0].copy_(torch.randn_like(x[0].float()))
            b[0].fill_(3.0)
        graph.replay()
        torch.cuda.synchronize()
        got = [b[0].clone() for b in bufs]
        for x, y in zip(cases, got):
            assert torch.equal(weight_grad(*x, E.F32_FINE), y)


@pytest.mark.parametrize("t", [300, 1500])
def test_weight_gradient_added_across_splits(t):
    """Few tiles and many tokens: with a workspace the tokens are split and joined. Whole
    numbers, so that every order gives the same."""
    say("project_grad: splits added to what is there", t)
    g = torch.Generator(device=DEV).manual_seed(t)
    k, n = 272, 136
    d = torch.randint(-3, 4, (t, n), generator=g, device=DEV).to(torch.bfloat16)
    codes = torch.randint(-20, 21, (t, k), generator=g, device=DEV, dtype=torch.int16).to(torch.int8)
    one = torch.ones(t, device=DEV)
    assert E.engram_project_grad_workspace_size(t, k, n) > 0
    base = torch.randint(-100, 100, (n, k), generator=g, device=DEV).float()
    want = d.double().t().contiguous() @ codes.double() + base.double()
    for workspace in (True, False):
        got = weight_grad(d, codes, one, E.F32, accumulate=1, grad=base, workspace=workspace)
        assert torch.equal(got.double(), want)
        got = weight_grad(d, codes, one, E.BF16, accumulate=1, grad=base.to(torch.bfloat16), workspace=workspace)
        assert torch.equal(got, want.to(torch.bfloat16))


def test_weight_gradient_of_no_tokens():
    say("project_grad: no tokens")
    d, c, s = (torch.empty((0, n), dtype=x, device=DEV) for n, x in ((40, torch.bfloat16), (48, torch.int8),
                                                                     (1, torch.float32)))
    for grad_type in (E.BF16, E.F32):
        assert not weight_grad(d, c, s, grad_type, grad=torch.ones((40, 48), device=DEV)).any()
        assert (weight_grad(d, c, s, grad_type, accumulate=1, grad=torch.ones((40, 48), device=DEV)) == 1).all()


def test_weight_gradient_not_finite():
    """A NaN scale (a row the quantiser could not hold) makes every gradient NaN; a NaN or
    infinity in one column of d_kv stays in its row of the gradient."""
    say("project_grad: not finite")
    d, c, s = weight_case(70, 160, 136, seed=5)
    base = weight_grad(d, c, s, E.F32)
    d2 = d.clone()
    d2[13, 9], d2[20, 100] = float("nan"), float("inf")
    got = weight_grad(d2, c, s, E.F32)
    keep = [i for i in range(136) if i not in (9, 100)]
    assert torch.equal(got[keep], base[keep]) and torch.isnan(got[9]).all()
    assert not torch.isfinite(got[100][c[20] != 0]).any()
    s[3] = float("nan")
    assert torch.isnan(weight_grad(d, c, s, E.F32)).all()


def test_weight_gradient_offsets_beyond_32_bits():
    say("project_grad: offsets beyond 2^31")
    t, k, n = 88000, 64, 25600           # 2.25e9 values of d_kv
    d = torch.zeros((t, n), dtype=torch.bfloat16, device=DEV)
    c = torch.zeros((t, k), dtype=torch.int8, device=DEV)
    s = torch.ones(t, device=DEV)
    g = torch.Generator(device=DEV).manual_seed(1)
    d[-3:] = torch.randint(-8, 9, (3, n), generator=g, device=DEV).to(torch.bfloat16)
    c[-3:] = torch.randint(-128, 128, (3, k), generator=g, device=DEV, dtype=torch.int16).to(torch.int8)
    got = weight_grad(d, c, s, E.F32)
    want = d[-3:].double().t().contiguous() @ c[-3:].double()
    assert torch.equal(got.double(), want)
    del d
    k, n, t = 100000, 25600, 3           # 2.56e9 gradients
    d = torch.randint(-8, 9, (t, n), generator=g, device=DEV).to(torch.bfloat16)
    c = torch.randint(-128, 128, (t, k), generator=g, device=DEV, dtype=torch.int16).to(torch.int8)
    got = weight_grad(d, c, torch.ones(t, device=DEV), E.BF16)
    for row in (0, 21474, 21475, 25599):
        want = (d[:, row:row + 1].double() * c.double()).sum(0)
        assert torch.equal(got[row], want.to(torch.bfloat16))


def test_weight_gradient_on_streams_and_replays():
    say("project_grad: streams and graphs")
    cases = [weight_case(700, 272, 264, 1), weight_case(333, 1040, 1288, 2)]
    bufs = []
    for d, c, s in cases:
        size = E.engram_project_grad_workspace_size(d.shape[0], c.shape[1], d.shape[1])
        bufs.append((torch.empty((d.shape[1], c.shape[1]), device=DEV),
                     torch.empty(max(size, 256), dtype=torch.uint8, device=DEV), size))

    def call(x, b):
        E.engram_project_grad(*x, b[0], E.F32, 0, x[0].shape[0], x[1].shape[1], x[0].shape[1], b[1], b[2])

    want = [weight_grad(*x, E.F32) for x in cases]
    streams = [torch.cuda.Stream() for _ in cases]
    torch.cuda.synchronize()
    for _ in range(4):
        for s, x, b in zip(streams, cases, bufs):
            with torch.cuda.stream(s):
                call(x, b)
    torch.cuda.synchronize()
    for b, w in zip(bufs, want):
        assert torch.equal(b[0], w)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        for x, b in zip(cases, bufs):
            call(x, b)
    for turn in range(4):
        for x, b in zip(cases, bufs):
            x[0].copy_(torch.randn_like(x[0].float()))
            b[0].fill_(3.0)
        graph.replay()
        torch.cuda.synchronize()
        got = [b[0].clone() for b in bufs]
        for x, y in zip(cases, got):
            assert torch.equal(weight_grad(*x, E.F32), y)


# ---- the operators together --------------------------------------------------------

def test_a_training_step_of_the_layer():
    """Rows looked up, quantised, projected in 8 bits and gated; then the gradients from the
    8-bit checkpoints back to the table, the weight and the gate's scales. Each stage is
    checked against 64 bits on the inputs that it was given."""
    say("a training step")
    t, seg, row_dim, hc, dim, rows = 150, 6, 32, 2, 128, 977
    k, n = seg * row_dim, (hc + 1) * dim
    g = torch.Generator(device=DEV).manual_seed(12)
    rand = lambda *s: torch.randn(s, generator=g, device=DEV)      # noqa: E731
    table, weight = rand(rows, row_dim), rand(n, k) * 0.05
    row_ids = torch.randint(0, rows, (t * seg,), generator=g, device=DEV)
    case = Case(t, hc, dim, E.BF16, E.I8, E.I8, seed=13)
    h = rand(t, hc, dim).to(torch.bfloat16)

    # forward
    e = torch.empty((t, k), dtype=torch.bfloat16, device=DEV)
    E.engram_embed(E.embed_desc(rows, t * seg, row_dim, E.F32, E.BF16), table, row_ids, e)
    ec, es = torch.empty((t, k), dtype=torch.int8, device=DEV), torch.empty(t, device=DEV)
    wc, wsc = torch.empty((n, k), dtype=torch.int8, device=DEV), torch.empty(n, device=DEV)
    E.engram_quantize_i8(e, E.BF16, t, k, 0, k, E.SCALE_POW2, ec, es)
    E.engram_quantize_i8(weight, E.F32, n, k, 0, k, E.SCALE_F32, wc, wsc)
    kv = torch.empty((t, n), dtype=torch.bfloat16, device=DEV)
    E.engram_project_i8(ec, es, wc, wsc, kv, E.BF16, t, k, n)
    exact = (ec.double() * es.double()[:, None]) @ (wc.double() * wsc.double()[:, None]).t().contiguous()
    assert ((kv.double() - exact).abs() <= (2.0 ** -8 + 4 * U) * exact.abs() * (1 + 2.0 ** -7)).all()
    case.kv, case.kv_scales = torch.empty((t, hc + 1, dim), dtype=torch.int8, device=DEV), torch.empty((t, hc + 1), device=DEV)
    case.h, case.h_scales = torch.empty((t, hc, dim), dtype=torch.int8, device=DEV), torch.empty((t, hc), device=DEV)
    E.engram_quantize_i8(kv, E.BF16, t * (hc + 1), dim, 0, dim, E.SCALE_F32, case.kv, case.kv_scales)
    E.engram_quantize_i8(h, E.BF16, t * hc, dim, 0, dim, E.SCALE_F32, case.h, case.h_scales)
    case.kv64, case.h64 = (c.double() * s.double()[..., None] for c, s in ((case.kv, case.kv_scales), (case.h, case.h_scales)))
    E.engram_gate(case.desc, case.ids, VOCAB, kv, case.q_w, case.k_w, h, None)

    # backward
    got = check_gate(case)
    d_kv = got["d_kv"].reshape(t, n)
    check_weight(d_kv, ec, es, E.F32)
    wt = torch.empty((k, n), dtype=torch.bfloat16, device=DEV)
    E.engram_transpose(weight.to(torch.bfloat16), wt, n, k, 0, 2)
    d_e = torch.empty((t, k), dtype=torch.bfloat16, device=DEV)
    E.engram_project(d_kv, wt, d_e, t, n, k, 0, False)
    w64 = weight.to(torch.bfloat16).double()
    exact, mag = d_kv.double() @ w64, d_kv.double().abs() @ w64.abs()
    err = (n + 8) * 2.0 ** -23 * mag
    assert ((d_e.double() - exact).abs() <= err + 2.0 ** -8 * (exact.abs() + err)).all()
    grad = torch.empty((rows, row_dim), device=DEV)
    desc = E.embed_desc(rows, t * seg, row_dim, E.F32, E.BF16)
    size = E.engram_embed_grad_workspace_size(desc)
    E.engram_embed_grad_dense(desc, d_e, row_ids, grad, 0, torch.empty(size, dtype=torch.uint8, device=DEV), size)
    torch.cuda.synchronize()
    terms = d_e.double().reshape(-1, row_dim)
    want = torch.zeros((rows, row_dim), dtype=torch.float64, device=DEV).index_add_(0, row_ids, terms)
    size = torch.zeros((rows, row_dim), dtype=torch.float64, device=DEV).index_add_(0, row_ids, terms.abs())
    assert ((grad.double() - want).abs() <= 200 * U * size).all()
    assert float(want.abs().max()) > 0


def test_calls_on_another_stream_than_their_buffers():
    """The operators run where they are told, behind what fills their inputs there."""
    say("8-bit operators: a stream handed over")
    s = torch.cuda.Stream()
    x = torch.randn((64, 256), device=DEV)
    codes, scales = torch.empty((64, 256), dtype=torch.int8, device=DEV), torch.empty(64, device=DEV)
    E.engram_quantize_i8(x, E.F32, 64, 256, 0, 256, E.SCALE_F32, codes, scales)
    torch.cuda.synchronize()
    c2, s2 = torch.zeros_like(codes), torch.zeros_like(scales)
    y = torch.empty_like(x)
    with torch.cuda.stream(s):
        torch.cuda._sleep(20_000_000)
        y.copy_(x)
    E.engram_quantize_i8(y, E.F32, 64, 256, 0, 256, E.SCALE_F32, c2, s2, None, s)
    s.synchronize()
    assert torch.equal(c2, codes) and torch.equal(s2, scales)
