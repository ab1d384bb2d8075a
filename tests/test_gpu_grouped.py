"""moe_grouped_gemm, moe_grouped_gemm_wgrad, moe_quantize_mxfp4, moe_grouped_gemm_mxfp4, moe_swiglu and
moe_swiglu_backward against plain float64 forms.

Products are tested on small whole numbers (MXFP4: on codes with few exponents), whose every partial sum fp32 holds
exactly: the results have to be equal, in whatever order they were added."""
import itertools

import pytest
import torch

from mixture_experts_ffn_topk_amd import MoEFFN, MoEError

pytestmark = pytest.mark.gpu

E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)
LEFT = 77.0  # what rows that a call does not write hold


def gen(seed):
    return torch.Generator().manual_seed(seed)


def routing(T, E, k, seed, skew=0.0, mask=0.0):
    """Expert ids [T, k], their pairs in plan order (stable by expert), and the experts' first rows."""
    g = gen(seed)
    pop = (1.0 / (1.0 + torch.arange(E)) ** skew).expand(max(T, 1), E)
    ids = torch.multinomial(pop, k, generator=g)[:T] if T else torch.zeros((0, k), dtype=torch.int64)
    ids = torch.where(torch.rand((T, k), generator=g) < mask, torch.full_like(ids, -1), ids)
    flat = ids.reshape(-1)
    pairs = torch.cat([(flat == e).nonzero().reshape(-1) for e in range(E)])
    start = [0] + torch.stack([(flat == e).sum() for e in range(E)]).cumsum(0).tolist()
    return ids, pairs, start


class Case:
    def __init__(self, T, E, k, seed=0, skew=0.0, mask=0.0, H=64, I=64, ids=None, **kw):
        self.T, self.E, self.k = T, E, k
        self.ids, self.pairs, self.start = routing(T, E, k, seed, skew, mask)
        self.rows = self.start[-1]
        self.moe = MoEFFN(H, I, E, k, max(T, 1), fmt="w4a8_mx", **kw)
        self.plan = self.moe.alloc_plan(T)
        self.moe.plan(T, self.plan, topk_idx=self.ids.cuda(), ws=self.moe.alloc_workspace(T))
        torch.cuda.synchronize()
        assert self.plan["src_info"][:self.rows].tolist() == self.pairs.tolist()

    def count(self, order):
        return self.T if order == "token" else self.T * self.k

    def pick(self, order):
        """The rows of a tensor in this order that the plan's rows stand for."""
        return {"plan": torch.arange(self.rows), "token": self.pairs // self.k, "pair": self.pairs}[order]

    def spans(self):
        return [(e, self.start[e], self.start[e + 1]) for e in range(self.E)]


def whole(g, *shape, top=3):
    return torch.randint(-top, top + 1, shape, generator=g).to(torch.bfloat16)


def product(c, a, w, a_rows, out_rows, n, kn=False):
    """The definition in float64, rows that no row of the plan reaches LEFT."""
    out = torch.full((c.T * c.k, n), LEFT, dtype=torch.float64)
    src, dst = c.pick(a_rows), c.pick(out_rows)
    for e, lo, hi in c.spans():
        we = w[e].double()
        out[dst[lo:hi]] = a[src[lo:hi]].double() @ (we if kn else we.T)
    return out


# (T, E, k, n, k of the product): one row, rows about the tiles' edges, several tiles an expert, ragged sides
SHAPES = [(1, 2, 1, 8, 8), (1, 8, 2, 256, 256), (3, 4, 2, 24, 40), (33, 3, 2, 264, 72), (70, 2, 1, 504, 136),
          (129, 4, 3, 256, 64), (300, 2, 2, 520, 200), (700, 3, 1, 296, 1032), (40, 128, 4, 96, 2880),
          (17, 5, 5, 7168, 128)]


@pytest.mark.parametrize("T,E,k,n,kk", SHAPES)
@pytest.mark.parametrize("kn", [False, True])
@pytest.mark.parametrize("f32", [False, True])
def test_grouped_gemm(T, E, k, n, kk, kn, f32):
    for i, (a_rows, out_rows) in enumerate(itertools.product(("plan", "token", "pair"), ("plan", "pair"))):
        c = Case(T, E, k, seed=T + i, skew=0.7 * (i % 2), mask=0.25 * (i % 3))
        g = gen(i)
        a, w = whole(g, c.count(a_rows), kk), whole(g, E, kk, n) if kn else whole(g, E, n, kk)
        out = torch.full((T * k, n), LEFT, dtype=torch.float32 if f32 else torch.bfloat16, device="cuda")
        c.moe.grouped_gemm(T, a.cuda(), w.cuda(), c.plan, out, a_rows=a_rows, out_rows=out_rows, w_kn=kn)
        want = product(c, a, w, a_rows, out_rows, n, kn).to(out.dtype)
        assert torch.equal(out.cpu(), want), (a_rows, out_rows)


@pytest.mark.parametrize("T,E,k,n,kk", SHAPES)
@pytest.mark.parametrize("f32", [False, True])
def test_grouped_gemm_wgrad(T, E, k, n, kk, f32):
    for i, (d_rows, a_rows) in enumerate(itertools.product(("plan", "token", "pair"), repeat=2)):
        if T * n * kk * 9 > 3e9 and i % 2:
            continue
        c = Case(T, E, k, seed=T + i, skew=0.7 * (i % 2), mask=0.25 * (i % 3))
        g = gen(i)
        d, a = whole(g, c.count(d_rows), n), whole(g, c.count(a_rows), kk)
        dw = torch.full((E, n, kk), LEFT, dtype=torch.float32 if f32 else torch.bfloat16, device="cuda")
        c.moe.grouped_gemm_wgrad(T, d.cuda(), a.cuda(), c.plan, dw, dout_rows=d_rows, a_rows=a_rows)
        di, ai = c.pick(d_rows), c.pick(a_rows)
        want = torch.stack([d[di[lo:hi]].float().T @ a[ai[lo:hi]].float() for _, lo, hi in c.spans()])
        assert torch.equal(dw.cpu(), want.to(dw.dtype)), (d_rows, a_rows)
        if f32:
            c.moe.grouped_gemm_wgrad(T, d.cuda(), a.cuda(), c.plan, dw, dout_rows=d_rows, a_rows=a_rows, accumulate=True)
            assert torch.equal(dw.cpu(), 2 * want)


def test_wgrad_reads_no_byte_past_the_rows_it_finds():
    """A tensor that takes a whole allocation (45 MiB, half of an allocation of 90): the last tile's columns past the last
    row's end lie past it."""
    torch.cuda.empty_cache()
    c = Case(8192, 2, 1)
    whole_segment = torch.empty(8192, 2880, 2, dtype=torch.bfloat16, device="cuda")
    del whole_segment
    halves = [torch.zeros(8192, 2880, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    dout = torch.zeros(8192, 264, dtype=torch.bfloat16, device="cuda")
    for a in halves:
        a[:, 2879] = 1.0
        dout[:] = 1.0
        dw = torch.empty(2, 264, 2880, device="cuda")
        c.moe.grouped_gemm_wgrad(c.T, dout, a, c.plan, dw, dout_rows="token", a_rows="token")
        counts = torch.tensor([hi - lo for _, lo, hi in c.spans()], dtype=torch.float32)
        assert torch.equal(dw[:, :, 2879].cpu(), counts[:, None].expand(2, 264))
        assert not dw[:, :, :2879].any()
        dw = torch.empty(2, 2880, 264, device="cuda")
        c.moe.grouped_gemm_wgrad(c.T, a, dout, c.plan, dw, dout_rows="token", a_rows="token")
        assert torch.equal(dw[:, 2879].cpu(), counts[:, None].expand(2, 264))
        assert not dw[:, :2879].any()


def codes(g, *shape):
    return torch.randint(0, 256, shape, generator=g, dtype=torch.uint8)


def value(q, sf):
    """MXFP4 codes [.., C/2] and scale bytes [.., C/32] in float64."""
    n = torch.stack([q & 15, q >> 4], -1).flatten(-2).long()
    v = torch.tensor(E2M1, dtype=torch.float64)[n & 7] * (1.0 - 2.0 * (n >> 3))
    s = torch.where(sf == 255, torch.full_like(sf, 0, dtype=torch.float64) + float("nan"), torch.exp2(sf.double() - 127))
    return v * s.repeat_interleave(32, -1)


MX_SHAPES = [(1, 2, 1, 8, 32), (1, 8, 2, 256, 256), (3, 4, 2, 24, 96), (33, 3, 2, 264, 544), (70, 2, 1, 504, 1024),
             (129, 4, 3, 256, 288), (300, 2, 2, 520, 160), (40, 128, 4, 96, 2880), (17, 5, 5, 7168, 128),
             (700, 3, 1, 296, 736)]


@pytest.mark.parametrize("T,E,k,n,kk", MX_SHAPES)
@pytest.mark.parametrize("f32", [False, True])
def test_grouped_gemm_mxfp4(T, E, k, n, kk, f32):
    for i, (a_rows, out_rows) in enumerate(itertools.product(("plan", "token", "pair"), ("plan", "pair"))):
        c = Case(T, E, k, seed=T + i, skew=0.7 * (i % 2), mask=0.25 * (i % 3))
        g = gen(i)
        R = c.count(a_rows)
        a, w = codes(g, R, kk // 2), codes(g, E, n, kk // 2)
        # exponents apart by at most 2: sums of multiples of 1/4 below 2^22
        asf = torch.randint(126, 128, (R, kk // 32), generator=g, dtype=torch.uint8)
        wsf = torch.randint(127, 129, (E, n, kk // 32), generator=g, dtype=torch.uint8)
        out = torch.full((T * k, n), LEFT, dtype=torch.float32 if f32 else torch.bfloat16, device="cuda")
        c.moe.grouped_gemm_mxfp4(T, a.cuda(), asf.cuda(), w.cuda(), wsf.cuda(), c.plan, out, a_rows=a_rows,
                                 out_rows=out_rows)
        want = product(c, value(a, asf), value(w, wsf), a_rows, out_rows, n).to(out.dtype)
        assert torch.equal(out.cpu(), want), (a_rows, out_rows)


def test_grouped_gemm_mxfp4_scales():
    """Every scale byte but the largest ones, whose products leave fp32; a NaN scale stays in its row or column."""
    c = Case(64, 2, 1, seed=3)
    g = gen(5)
    kk, n = 320, 48
    a, w = codes(g, 64, kk // 2), codes(g, 2, n, kk // 2)
    asf = torch.randint(60, 190, (64, kk // 32), generator=g, dtype=torch.uint8)
    wsf = torch.randint(100, 150, (2, n, kk // 32), generator=g, dtype=torch.uint8)
    asf[7, 9], wsf[1, 5, 3] = 255, 255
    out = torch.empty((64, n), dtype=torch.float32, device="cuda")
    c.moe.grouped_gemm_mxfp4(64, a.cuda(), asf.cuda(), w.cuda(), wsf.cuda(), c.plan, out, a_rows="token", out_rows="pair")
    av, wv = value(a, asf), value(w, wsf)
    want = product(c, av, wv, "token", "pair", n)
    size = product(c, av.abs(), wv.abs(), "token", "pair", n)
    got = out.cpu().double()
    assert torch.equal(torch.isnan(got), torch.isnan(want)) and torch.isnan(want).any() and not torch.isnan(want).all()
    fine = ~torch.isnan(want)
    # kk - 1 sums of fp32, each rounded (or cut) by less than 2^-23 of a partial sum, which is at most `size`
    assert ((got - want).abs() <= kk * 2.0 ** -23 * size)[fine].all()


@pytest.mark.parametrize("f32", [False, True])
@pytest.mark.parametrize("op", ["forward", "gradient", "wgrad"])
def test_grouped_rounding(op, f32):
    """Ordinary values: the fp32 sum of K products is off by at most K 2^-23 of the sum of magnitudes (each addition by
    less than 2^-23 of a partial sum), its rounding to bf16 by 2^-8 of the value."""
    T, E, k, n, kk = 260, 2, 2, 192, 320
    c = Case(T, E, k, seed=1)
    g = gen(2)
    dt, K = torch.float32 if f32 else torch.bfloat16, c.rows if op == "wgrad" else kk
    if op == "wgrad":
        d, a = (torch.randn(T * k, s, generator=g).to(torch.bfloat16) for s in (n, kk))
        got = torch.empty((E, n, kk), dtype=dt, device="cuda")
        c.moe.grouped_gemm_wgrad(T, d.cuda(), a.cuda(), c.plan, got)
        form = lambda x, y: torch.stack([x[lo:hi].double().T @ y[lo:hi].double() for _, lo, hi in c.spans()])  # noqa: E731
        want, size = form(d, a), form(d.abs(), a.abs())
    else:
        kn = op == "gradient"
        a = torch.randn(T * k, kk, generator=g).to(torch.bfloat16)
        w = torch.randn(*((E, kk, n) if kn else (E, n, kk)), generator=g).to(torch.bfloat16)
        got = torch.empty((T * k, n), dtype=dt, device="cuda")
        c.moe.grouped_gemm(T, a.cuda(), w.cuda(), c.plan, got, w_kn=kn)
        want, size = (product(c, x, y, "plan", "plan", n, kn) for x, y in ((a, w), (a.abs(), w.abs())))
    off = (got.cpu().double() - want).abs()
    assert (off <= K * 2.0 ** -23 * size * (1 + 2.0 ** -8) + (0 if f32 else 2.0 ** -8) * want.abs()).all()


def test_grouped_infinities_stay_in_their_rows():
    """Masked tails (rows past an expert's last, columns past K) multiply nothing: NaN and infinities of other rows, other
    experts and other columns do not leak."""
    T, E, k, n, kk = 40, 3, 1, 40, 72
    c = Case(T, E, k, seed=9)
    g = gen(4)
    a, w = whole(g, T, kk), whole(g, E, n, kk)
    r, e = 5, 1
    a[r, 3], a[r, 71], w[e, 7, 70] = float("inf"), float("nan"), float("nan")
    out = torch.empty((T, n), dtype=torch.float32, device="cuda")
    c.moe.grouped_gemm(T, a.cuda(), w.cuda(), c.plan, out)
    want = product(c, a, w, "plan", "plan", n).float()
    assert torch.equal(torch.isnan(out.cpu()), torch.isnan(want))
    assert torch.equal(out.cpu().nan_to_num(0.0), want.nan_to_num(0.0))
    d = whole(g, T, n)
    d[r, 2] = float("inf")
    dw = torch.empty((E, n, kk), dtype=torch.float32, device="cuda")
    a = whole(g, T, kk, top=3)
    a[a == 0] = 1
    c.moe.grouped_gemm_wgrad(T, d.cuda(), a.cuda(), c.plan, dw)
    want = torch.stack([d[lo:hi].float().T @ a[lo:hi].float() for _, lo, hi in c.spans()])
    assert torch.equal(torch.isnan(dw.cpu()), torch.isnan(want)) and torch.isinf(want).sum() == kk
    assert torch.equal(dw.cpu().nan_to_num(0.0), want.nan_to_num(0.0))


def test_no_rows():
    """A batch whose every slot is masked, and one of no tokens: nothing is written but zero weight gradients."""
    for T, mask in ((6, 1.0), (0, 0.0)):
        c = Case(T, 4, 2, mask=mask)
        z = lambda *s, dt=torch.bfloat16: torch.full(s, LEFT, dtype=dt, device="cuda")  # noqa: E731
        out, n = z(max(1, T * 2), 64), max(1, T * 2)
        c.moe.grouped_gemm(T, z(n, 64), z(4, 64, 64), c.plan, out)
        c.moe.swiglu(T, z(n, 128), c.plan, h=out)
        c.moe.swiglu_backward(T, z(n, 128), z(n, 64), c.plan, z(n, 128), h=out)
        c.moe.grouped_gemm_mxfp4(T, z(n, 64, dt=torch.uint8), z(n, 4, dt=torch.uint8), z(4, 64, 64, dt=torch.uint8),
                                 z(4, 64, 4, dt=torch.uint8), c.plan, out)
        assert (out == LEFT).all()
        dw = z(4, 64, 64, dt=torch.float32)
        c.moe.grouped_gemm_wgrad(T, z(n, 64), z(n, 64), c.plan, dw, accumulate=True)
        assert (dw == LEFT).all()
        c.moe.grouped_gemm_wgrad(T, z(n, 64), z(n, 64), c.plan, dw)
        assert (dw == 0).all()
    MoEFFN(32, 32, 1, 1, 1, fmt="w4a8_mx").quantize_mxfp4(z(0, 64), z(0, 32, dt=torch.uint8), z(0, 2, dt=torch.uint8))


# ------------------------------------------------------------------------------------------------ MXFP4
def quantised(x):
    """The definition: (codes one a byte, scale bytes, values) of float64 rows."""
    b = x.unflatten(-1, (-1, 32))
    top = b.abs().amax(-1)
    nan = torch.isnan(b).any(-1)
    m, e = torch.frexp(torch.where(torch.isinf(top) | nan | (top == 0), torch.ones_like(top), top))
    e = torch.where(m > 0.75, e - 2, e - 3)
    e = torch.where(torch.isinf(top), torch.full_like(e, 127), torch.where(top == 0, torch.full_like(e, -127), e))
    e = e.clamp(-127, 127)
    v = b / torch.exp2(e.double())[..., None]
    a = v.abs().clamp(max=6.0)
    step = torch.where(a < 2, 0.5, torch.where(a < 4, 1.0, 2.0)).double()
    r = torch.round(a / step) * step
    code = (r[..., None] > torch.tensor(E2M1, dtype=torch.float64)).sum(-1) | (torch.signbit(v).long() << 3)
    values = torch.copysign(r, v) * torch.exp2(e.double())[..., None]
    values = torch.where(nan[..., None], torch.full_like(values, float("nan")), values)
    return code.flatten(-2), torch.where(nan, torch.full_like(e, 255 - 127), e) + 127, values.flatten(-2), nan


def special_rows(kind, cols):
    """Rows of every size of number, ties, borders of the scale, zeros, infinities and NaNs."""
    g = gen(cols)
    x = torch.randn(60, cols, generator=g) * torch.exp2(torch.randint(-140, 120, (60, 1), generator=g).float())
    x[1] = 0.0
    x[2] = -0.0
    ties = torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 6.0, -0.25, -0.75, -5.0, -1.25, 0.2490234375, 0.251953125,
                         2.484375, 2.515625])
    for i, e in enumerate((-127, -126, -100, -61, -60, -59, 0, 3, 100, 125)):
        x[3 + i] = ties.repeat(cols // 16) * 2.0 ** e
        x[13 + i] = x[3 + i]
        x[13 + i, ::32] = 6.0 * 2.0 ** e * (1 + 2.0 ** -7)  # past 6: one exponent more
        x[23 + i, :] = 2.0 ** (e - 8) if e > -120 else 2.0 ** e
    x[40, 5], x[41, 33 % cols], x[42, 0] = float("inf"), float("-inf"), float("nan")
    x[43] = torch.finfo(kind).max
    x[44] = torch.finfo(kind).tiny
    x[45] = torch.finfo(kind).tiny / 4
    return x.to(kind)


@pytest.mark.parametrize("cols", [32, 96, 1024, 2880])
@pytest.mark.parametrize("kind", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("pad", [0, 8, 40])
def test_quantize_mxfp4(cols, kind, pad):
    x = special_rows(kind, cols)
    R = x.shape[0]
    wide = torch.full((R, cols + pad), float("nan"), dtype=kind, device="cuda")
    wide[:, :cols] = x.cuda()
    q, sf = (torch.full((R + 1, c), 77, dtype=torch.uint8, device="cuda") for c in (cols // 2, cols // 32))
    values = torch.full((R + 1, cols), LEFT, dtype=torch.bfloat16, device="cuda")
    moe = MoEFFN(32, 32, 1, 1, 1, fmt="w4a8_mx")
    moe.quantize_mxfp4(wide[:, :cols], q[:R], sf[:R], values=values[:R])
    code, scale, val, nan = quantised(x.double())
    assert torch.equal(sf[:R].cpu().long(), scale.long())
    got = torch.stack([q[:R] & 15, q[:R] >> 4], -1).flatten(-2).cpu().long()
    ok = ~nan.repeat_interleave(32, -1)
    assert torch.equal(got[ok], code[ok])
    v = values[:R].cpu()
    assert torch.equal(torch.isnan(v), ~ok) and torch.equal(v[ok], val.to(torch.bfloat16)[ok])
    assert torch.equal(torch.signbit(v[ok]), torch.signbit(val[ok]))
    assert (q[R] == 77).all() and (sf[R] == 77).all() and (values[R] == LEFT).all()


def test_quantize_mxfp4_in_place_and_many_rows():
    moe = MoEFFN(32, 32, 1, 1, 1, fmt="w4a8_mx")
    x = torch.randn(40000, 96, generator=gen(0)).to(torch.bfloat16)
    t = x.cuda()
    q, sf = torch.empty((40000, 48), dtype=torch.uint8, device="cuda"), torch.empty((40000, 3), dtype=torch.uint8, device="cuda")
    moe.quantize_mxfp4(t, q, sf, values=t)
    want = quantised(x.double())[2].to(torch.bfloat16)
    assert torch.equal(t.cpu(), want)
    wide = torch.zeros((40000, 128), dtype=torch.bfloat16, device="cuda")
    wide[:, 16:112] = x.cuda()
    q2 = torch.empty_like(q)
    moe.quantize_mxfp4(wide[:, 16:112], q2, sf)
    assert torch.equal(q, q2)


# ------------------------------------------------------------------------------------------------ SwiGLU
def swiglu64(gu, dh, clamp):
    I = gu.shape[1] // 2
    g, u = gu[:, :I].double(), gu[:, I:].double()
    gc, uc = torch.where(g > clamp, clamp, g), torch.where(u > clamp, clamp, torch.where(u < -clamp, -clamp, u))
    s = torch.sigmoid(gc)
    h = torch.where(gc == -float("inf"), torch.zeros_like(gc), gc * s) * uc
    if dh is None:
        return h
    d = dh.double()
    fin = gc.clamp(-1e30, 1e30)
    dg = torch.where(g > clamp, torch.zeros_like(d), d * uc * s * (1 + fin * (1 - s)))
    du = torch.where(u.abs() > clamp, torch.zeros_like(d), d * torch.where(gc == -float("inf"), torch.zeros_like(gc), gc * s))
    return h, torch.cat([dg, du], 1)


def near(got, want, extra):
    """Within half a bf16 step (2^-8 of the value, or half the smallest one) and `extra` of fp32 roundings."""
    got, want = got.cpu().double(), want.double()
    assert torch.equal(torch.isnan(got), torch.isnan(want))
    ok = ~torch.isnan(want)
    got, want, extra = got[ok], want[ok], (extra.expand_as(ok) if extra.dim() else extra.expand(ok.shape))[ok]
    fin = torch.isfinite(got)
    assert torch.equal(got[~fin], want[~fin].float().to(torch.bfloat16).double())
    assert ((got - want).abs()[fin] <= (2.0 ** -8 * want.abs() * (1 + 2.0 ** -8) + 2.0 ** -134 + 1.01 * extra)[fin]).all()


@pytest.mark.parametrize("I", [32, 96, 512, 2048, 2880])
@pytest.mark.parametrize("fast", [True, False])
@pytest.mark.parametrize("clamp", [10.0, 1.5, float("inf")])
def test_swiglu(I, fast, clamp):
    c = Case(37, 4, 2, seed=I, mask=0.2, H=64, I=I, fast_math=fast, activation_clamp=clamp)
    g = gen(I)
    R, rows = 74, c.rows
    gu = (torch.randn(R, 2 * I, generator=g) * 4).to(torch.bfloat16)
    dh = torch.randn(R, I, generator=g).to(torch.bfloat16)
    special = torch.tensor([0.0, -0.0, clamp if clamp < 1e9 else 3.0, -clamp if clamp < 1e9 else -3.0, 100.0, -100.0, 1e-30,
                            float("inf"), float("-inf"), float("nan"), 11.0, -11.0, -88.0, -90.0, 20.0, -3e38]).to(torch.bfloat16)
    gu[0, :16], gu[1, I:I + 16] = special, special
    z = lambda *s, dt=torch.bfloat16: torch.full(s, LEFT, dtype=dt, device="cuda")  # noqa: E731
    h, h2, dgu = z(R, I), z(R, I), z(R, 2 * I)
    q, sf = z(R, I // 2, dt=torch.uint8), z(R, I // 32, dt=torch.uint8)
    c.moe.swiglu(37, gu.cuda(), c.plan, h=h, q=q, sf=sf)
    c.moe.swiglu_backward(37, gu.cuda(), dh.cuda(), c.plan, dgu, h=h2)
    wh, wd = swiglu64(gu[:rows], dh[:rows], clamp)
    # fp32: the exponent -g log2(e) is rounded (2^-24 of up to 1.45 |g'|, times ln 2), exp2, 1 + e, the reciprocal and
    # three products each by at most 2^-23: (|g'| + 8) 2^-23 of the value; 1 + g' (1 - s) is formed of numbers up to
    # 1 + |g'|, whose errors do not shrink with the sum
    gp = torch.where(gu[:rows, :I].double() > clamp, clamp, gu[:rows, :I].double()).abs().nan_to_num(0.0).clamp(max=100.0)
    rel = (gp + 8) * 2.0 ** -23
    near(h[:rows], wh, rel * wh.abs().nan_to_num(0.0))
    assert torch.equal(h[:rows].view(torch.int16), h2[:rows].view(torch.int16))
    s = torch.sigmoid(torch.where(gu[:rows, :I].double() > clamp, clamp, gu[:rows, :I].double())).nan_to_num(0.0)
    uc = gu[:rows, I:].double().clamp(-clamp, clamp).abs().nan_to_num(0.0)
    size = dh[:rows].double().abs() * torch.cat([uc, gp], 1).unflatten(1, (2, I)).transpose(0, 1)
    big = torch.cat([(size[0] * s * (1 + gp)), size[1] * s], 1)
    near(dgu[:rows], wd, torch.cat([rel, rel], 1) * big.nan_to_num(0.0))
    for t in (h, h2, dgu):
        assert (t[rows:] == LEFT).all()
    assert (q[rows:] == 77).all() and (sf[rows:] == 77).all()
    # MXFP4 of the unrounded h: codes within one fp32 error of h of a rounding's border may go either way
    lo, hi = (quantised(wh * (1 + s_ * 2.0 ** -17)) for s_ in (-1.0, 1.0))
    same = (lo[1] == hi[1]) & ~lo[3]
    assert torch.equal(sf[:rows].cpu().long()[same], lo[1].long()[same])
    got = torch.stack([q[:rows] & 15, q[:rows] >> 4], -1).flatten(-2).cpu().long()
    sure = same.repeat_interleave(32, -1) & (lo[0] == hi[0])
    assert torch.equal(got[sure], lo[0][sure]) and sure.float().mean() > 0.9


def test_swiglu_gradient_is_the_difference_quotient():
    """The backward pass against differences of the forward definition in float64."""
    c = Case(8, 2, 1, I=64, activation_clamp=2.0)
    g = gen(3)
    gu, dh = torch.randn(8, 128, generator=g).to(torch.bfloat16) * 1.5, torch.randn(8, 64, generator=g).to(torch.bfloat16)
    dgu = torch.empty((8, 128), dtype=torch.bfloat16, device="cuda")
    c.moe.swiglu_backward(8, gu.cuda(), dh.cuda(), c.plan, dgu)
    step = 2.0 ** -20
    x = gu.double()
    diff = torch.zeros_like(x)
    for j in range(128):
        up, down = x.clone(), x.clone()
        up[:, j] += step
        down[:, j] -= step
        diff[:, j] = ((swiglu64(up, None, 2.0) - swiglu64(down, None, 2.0)) / (2 * step) * dh.double()).sum(1)
    edge = (x.abs() - 2.0).abs() < 2 * step
    # a difference is off by step^2 / 6 of the third derivative (below 4 here) and 2^-52 / step of the values
    assert ((dgu.cpu().double() - diff).abs() <= 2.0 ** -8 * diff.abs() * 1.01 + 2.0 ** -18)[~edge].all()


def test_in_place():
    c = Case(50, 4, 2, seed=2, I=96)
    g = gen(1)
    gu, dh = (torch.randn(100, s, generator=g).to(torch.bfloat16).cuda() for s in (192, 96))
    dgu, h = torch.empty_like(gu), torch.empty_like(dh)
    c.moe.swiglu_backward(50, gu, dh, c.plan, dgu, h=h)
    gu2, dh2 = gu.clone(), dh.clone()
    c.moe.swiglu_backward(50, gu2, dh2, c.plan, gu2, h=dh2)
    assert torch.equal(gu2[:c.rows], dgu[:c.rows]) and torch.equal(dh2[:c.rows], h[:c.rows])


# ------------------------------------------------------------------------------------------------ together
def test_training_step_gradients():
    """A layer's forward and backward by these calls and moe_combine, against autograd in float64 of the same values
    (each rounding to bf16 on the way is a relative 2^-8 of what it rounds)."""
    T, E, k, H, I = 70, 4, 2, 128, 96
    c = Case(T, E, k, seed=4, mask=0.1, H=H, I=I)
    g = gen(8)
    r = lambda s, *shape: (torch.randn(*shape, generator=g) * s).to(torch.bfloat16)  # noqa: E731
    x, w13, w2, dout = r(1.0, T, H), r(H ** -0.5, E, 2 * I, H), r(I ** -0.5, E, H, I), r(1.0, T, H)
    tw = torch.rand(T, k, generator=g)
    new = lambda *s, dt=torch.bfloat16: torch.zeros(s, dtype=dt, device="cuda")  # noqa: E731
    X, W13, W2, D, TW = (t.cuda() for t in (x, w13, w2, dout, tw))
    gu, h, y, out = new(T * k, 2 * I), new(T * k, I), new(T * k, H), new(T, H)
    c.moe.grouped_gemm(T, X, W13, c.plan, gu, a_rows="token")
    c.moe.swiglu(T, gu, c.plan, h=h)
    c.moe.grouped_gemm(T, h, W2, c.plan, y, out_rows="pair")
    c.moe.combine(T, y, TW, c.plan, out)
    dy = (D[:, None] * TW[..., None]).to(torch.bfloat16).view(T * k, H)
    dh, dgu, dxp, dx = new(T * k, I), new(T * k, 2 * I), new(T * k, H), new(T, H)
    dw2, dw13 = new(E, H, I, dt=torch.float32), new(E, 2 * I, H, dt=torch.float32)
    c.moe.grouped_gemm(T, dy, W2, c.plan, dh, a_rows="pair", w_kn=True)
    c.moe.grouped_gemm_wgrad(T, dy, h, c.plan, dw2, dout_rows="pair")
    c.moe.swiglu_backward(T, gu, dh, c.plan, dgu)
    c.moe.grouped_gemm(T, dgu, W13, c.plan, dxp, out_rows="pair", w_kn=True)
    c.moe.grouped_gemm_wgrad(T, dgu, X, c.plan, dw13, a_rows="token")
    c.moe.combine(T, dxp, torch.ones_like(TW), c.plan, dx)

    xd, ad, bd = (t.double().requires_grad_(True) for t in (x, w13, w2))
    total = torch.zeros(T, H, dtype=torch.float64)
    for t, j in itertools.product(range(T), range(k)):
        e = int(c.ids[t, j])
        if e >= 0:
            total[t] = total[t] + tw[t, j].double() * (bd[e] @ swiglu64((ad[e] @ xd[t])[None], None, 10.0)[0])
    grads = torch.autograd.grad(total, (xd, ad, bd), dout.double())
    for got, want in zip((out, dx, dw13, dw2), (total.detach(), *grads)):
        # at most six roundings to bf16 (gu, h or dh, dgu, y or dy, dxp, out) of 2^-8 each on the way to a value, and what
        # they meet is spread like the terms: the norm of the error is below 6 * 2^-8 of the norm of the result
        off = (got.cpu().double() - want).norm() / want.norm()
        assert off <= 6 * 2.0 ** -8, off


def test_mxfp4_layer():
    """Plan, quantisation, product, SwiGLU to MXFP4, product and combine, against the definition step by step in float64 on
    the library's own intermediates."""
    T, E, k, H, I = 45, 8, 2, 288, 160
    c = Case(T, E, k, seed=6, mask=0.1, H=H, I=I)
    g = gen(5)
    x = torch.randn(T, H, generator=g).to(torch.bfloat16)
    w13, w2 = torch.randn(E, 2 * I, H, generator=g) * H ** -0.5, torch.randn(E, H, I, generator=g) * I ** -0.5
    tw = torch.rand(T, k, generator=g)
    u8 = lambda *s: torch.zeros(s, dtype=torch.uint8, device="cuda")  # noqa: E731
    bf = lambda *s: torch.zeros(s, dtype=torch.bfloat16, device="cuda")  # noqa: E731
    Q13, S13, Q2, S2 = u8(E, 2 * I, H // 2), u8(E, 2 * I, H // 32), u8(E, H, I // 2), u8(E, H, I // 32)
    c.moe.quantize_mxfp4(w13.cuda(), Q13, S13)
    c.moe.quantize_mxfp4(w2.cuda(), Q2, S2)
    xq, xs, gu, hq, hs, y, out = u8(T, H // 2), u8(T, H // 32), bf(T * k, 2 * I), u8(T * k, I // 2), u8(T * k, I // 32), bf(T * k, H), bf(T, H)
    c.moe.quantize_mxfp4(x.cuda(), xq, xs)
    c.moe.grouped_gemm_mxfp4(T, xq, xs, Q13, S13, c.plan, gu, a_rows="token")
    c.moe.swiglu(T, gu, c.plan, q=hq, sf=hs)
    c.moe.grouped_gemm_mxfp4(T, hq, hs, Q2, S2, c.plan, y, out_rows="pair")
    c.moe.combine(T, y, tw.cuda(), c.plan, out)
    v = lambda q, s: value(q.cpu(), s.cpu())  # noqa: E731
    assert torch.equal(v(Q13, S13), quantised(w13.double())[2])
    for got, a, w, ar, orr, n in ((gu, v(xq, xs), v(Q13, S13), "token", "plan", 2 * I),
                                  (y, v(hq, hs), v(Q2, S2), "plan", "pair", H)):
        want, size = product(c, a, w, ar, orr, n), product(c, a.abs(), w.abs(), ar, orr, n)
        at = c.pick(orr)
        off = (got.cpu().double() - want).abs()[at]
        assert (off <= (2.0 ** -8 * want.abs() * 1.01 + H * 2.0 ** -23 * size)[at]).all()
    ref = torch.zeros(T, H, dtype=torch.float64)
    for t, j in itertools.product(range(T), range(k)):
        if c.ids[t, j] >= 0:
            ref[t] += tw[t, j].double() * y[t * k + j].cpu().double()
    assert ((out.cpu().double() - ref).abs() <= 2.0 ** -8 * ref.abs() * 1.01 + 2.0 ** -20).all()


def test_graph_of_two_steps_on_another_stream():
    """Captured on a side stream with other calls' buffers alive, replayed with eager work between the replays."""
    T, E, k, H, I = 33, 4, 2, 64, 64
    c = Case(T, E, k, seed=1, H=H, I=I)
    g = gen(2)
    x, w, d = whole(g, T, H).cuda(), whole(g, E, 2 * I, H).cuda(), whole(g, T * k, 2 * I).cuda()
    out, dw, q, sf = (torch.zeros(s, dtype=t, device="cuda") for s, t in
                      (((T * k, 2 * I), torch.bfloat16), ((E, 2 * I, H), torch.float32), ((T, H // 2), torch.uint8),
                       ((T, H // 32), torch.uint8)))

    def step():
        c.moe.grouped_gemm(T, x, w, c.plan, out, a_rows="token")
        c.moe.grouped_gemm_wgrad(T, d, x, c.plan, dw, a_rows="token")
        c.moe.quantize_mxfp4(x, q, sf)

    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        step()
    for i in range(4):
        x.copy_(whole(gen(10 + i), T, H))
        out.zero_()
        dw.fill_(5.0)
        graph.replay()
        torch.cuda.synchronize()
        got = [t.clone() for t in (out, dw, q, sf)]
        step()
        for a, b in zip(got, (out, dw, q, sf)):
            assert torch.equal(a, b)
        assert torch.equal(out.cpu().double(), product(c, x.cpu(), w.cpu(), "token", "plan", 2 * I).to(torch.bfloat16).double())


def test_refusals_of_the_binding():
    c = Case(4, 2, 1)
    b = torch.zeros((4, 64), dtype=torch.bfloat16, device="cuda")
    w = torch.zeros((2, 64, 64), dtype=torch.bfloat16, device="cuda")
    with pytest.raises(ValueError):
        c.moe.grouped_gemm(4, b, w, c.plan, b.clone(), a_rows="expert")
    with pytest.raises(MoEError, match="UNSUPPORTED"):
        c.moe.grouped_gemm(4, b, w, c.plan, b.clone(), out_rows="token")
    with pytest.raises(MoEError, match="INVALID"):
        c.moe.grouped_gemm(4, b, w, c.plan, b)
    with pytest.raises(MoEError, match="UNSUPPORTED"):
        c.moe.grouped_gemm_wgrad(4, b, b.clone(), c.plan, w, accumulate=True)
    with pytest.raises(ValueError):
        c.moe.grouped_gemm(4, b, w.cpu(), c.plan, b.clone())
    with pytest.raises(ValueError):
        c.moe.grouped_gemm(4, b.t(), w, c.plan, b.clone())
    with pytest.raises(TypeError):
        c.moe.grouped_gemm(4, b.float(), w, c.plan, b.clone())
