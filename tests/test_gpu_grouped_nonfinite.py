"""Infinities and NaNs in the products by expert whose tiles are 128 x 128 and 256 x 256: in the rows of masked slots, in
the next expert's first row and weights, in the columns right behind a tile, in the next row's first columns (which a K-step
that is longer than the row would reach), and MXFP4's NaN scales in the same places.  They show where the definition has
them and nowhere else; the other values are whole numbers whose sums fp32 holds, and have to be equal.  MXFP4's scales of
every size, on the 256 x 256 tile."""
import pytest
import torch

from test_gpu_grouped import LEFT, Case, codes, gen, product, value, whole
from test_gpu_grouped_paths import Fixed, even_ids

pytestmark = pytest.mark.gpu

INF, NAN = float("inf"), float("nan")


def same(got, want):
    """NaNs in the same places, the rest equal (infinities too)."""
    got, want = got.cpu(), want.to(got.dtype)
    nan = torch.isnan(want)
    assert torch.equal(torch.isnan(got), nan)
    assert torch.equal(got[~nan], want[~nan])
    assert nan.any() and not nan.all() and torch.isinf(want).any()


def masked_ids(T, E, k, seed):
    """Different experts for a token's slots, every expert as often, and some slots masked."""
    ids = (torch.arange(T)[:, None] + torch.arange(k)) % E
    return torch.where(torch.rand((T, k), generator=gen(seed)) < 0.1, torch.full_like(ids, -1), ids)


def poison_rows(c, t, order):
    """NaN in masked slots' rows; an infinity in the last column of expert 0's last row, NaN in the first of what lies
    behind it: expert 1's first row in the plan's order, the next row in memory in any."""
    if order == "pair":
        t[(c.ids.reshape(-1) < 0).nonzero().reshape(-1)] = NAN
    if order == "plan":
        t[c.rows:] = NAN
    at = c.pick(order)
    last, first = at[c.start[1] - 1], at[c.start[1]]
    t[last, -1] = INF
    t[first, 0] = NAN
    t[at[c.start[2] - 1], 1] = -INF
    if int(last) + 1 < len(t):
        t[last + 1, 0] = NAN


def nonzero(g, *shape):
    """Whole numbers without a zero: an infinity times them is one."""
    t = whole(g, *shape)
    return torch.where(t == 0, torch.ones_like(t), t)


# (T, E, k, n, k of the product): tiles of 128 x 128; of 256 x 256, with tails of rows, columns and summed columns
TILES = [(300, 3, 1, 1032, 136), (250, 3, 2, 1032, 72), (520, 2, 1, 25608, 72), (400, 3, 2, 25608, 136)]
ORDERS = [("token", "pair"), ("plan", "plan"), ("pair", "plan")]


@pytest.mark.parametrize("T,E,k,n,kk", TILES)
@pytest.mark.parametrize("kn", [False, True])
@pytest.mark.parametrize("a_rows,out_rows", ORDERS)
def test_products(T, E, k, n, kk, kn, a_rows, out_rows):
    c = Fixed(E, masked_ids(T, E, k, T))
    g = gen(kk)
    a = whole(g, c.count(a_rows), kk)
    w = nonzero(g, E, n, kk)
    poison_rows(c, a, a_rows)
    w[1, 0] = NAN          # what follows expert 0's last row
    w[0, 255, 3] = INF
    w[0, 256] = NAN        # what follows a tile's last column
    w[0, 128, 5] = -INF
    w[0, n - 1, kk - 1] = INF
    w[E - 1, :, 0][9] = NAN
    if kn:
        w = w.transpose(1, 2).contiguous()
        w[1, 0] = NAN      # what follows expert 0's last summed row
    out = torch.full((T * k, n), LEFT, device="cuda")
    c.moe.grouped_gemm(T, a.cuda(), w.cuda(), c.plan, out, a_rows=a_rows, out_rows=out_rows, w_kn=kn)
    same(out, product(c, a, w, a_rows, out_rows, n, kn))


# 128 x 128 and 256 x 256, rows of an expert that end inside a K-step, columns that end inside a tile
@pytest.mark.parametrize("T,E,k,n,kk", [(300, 3, 1, 520, 264), (410, 4, 2, 264, 136), (560, 6, 1, 2056, 1800)])
@pytest.mark.parametrize("d_rows,a_rows", [("plan", "token"), ("pair", "plan"), ("token", "pair"), ("plan", "plan")])
def test_weight_gradients(T, E, k, n, kk, d_rows, a_rows):
    c = Fixed(E, masked_ids(T, E, k, T + 1))
    g = gen(n)
    d, a = nonzero(g, c.count(d_rows), n), nonzero(g, c.count(a_rows), kk)
    poison_rows(c, d, d_rows)
    poison_rows(c, a, a_rows)
    d[c.pick(d_rows)[c.start[2] - 1], 256] = NAN
    a[c.pick(a_rows)[c.start[2] - 1], 128] = INF
    dw = torch.full((E, n, kk), LEFT, device="cuda")
    c.moe.grouped_gemm_wgrad(T, d.cuda(), a.cuda(), c.plan, dw, dout_rows=d_rows, a_rows=a_rows)
    di, ai = c.pick(d_rows), c.pick(a_rows)
    same(dw, torch.stack([d[di[lo:hi]].double().T @ a[ai[lo:hi]].double() for _, lo, hi in c.spans()]))


# scales of whole words and not, one to five K-steps, several tiles a workgroup
@pytest.mark.parametrize("T,E,k,n,kk", [(300, 2, 1, 264, 1024), (540, 3, 1, 264, 1056), (280, 2, 2, 520, 96),
                                        (500, 3, 1, 25608, 128), (460, 3, 1, 25608, 160)])
@pytest.mark.parametrize("a_rows,out_rows", ORDERS)
def test_mxfp4_scales_of_nan(T, E, k, n, kk, a_rows, out_rows):
    c = Fixed(E, masked_ids(T, E, k, T))
    g = gen(kk)
    R = c.count(a_rows)
    a, w = codes(g, R, kk // 2), codes(g, E, n, kk // 2)
    # (exponents apart by at most 2: sums of multiples of 1/8 below 2^21)
    asf = torch.randint(126, 128, (R, kk // 32), generator=g, dtype=torch.uint8)
    wsf = torch.randint(127, 129, (E, n, kk // 32), generator=g, dtype=torch.uint8)
    at = c.pick(a_rows)
    asf[at[c.start[1] - 1] + 1 if int(at[c.start[1] - 1]) + 1 < R else at[3], 0] = 255
    asf[at[c.start[1]], 0] = 255
    asf[at[5], -1] = 255
    asf[at[-1] if a_rows == "token" else R - 1, 0] = 255
    wsf[0, 256, 0] = 255   # what follows a tile's last row of weights, and row 255's last scale
    wsf[1, 0] = 255
    wsf[0, n - 1, -1] = 255
    if a_rows == "plan":
        asf[c.rows:] = 255
    if a_rows == "pair":
        asf[(c.ids.reshape(-1) < 0).nonzero().reshape(-1)] = 255
    out = torch.full((T * k, n), LEFT, device="cuda")
    c.moe.grouped_gemm_mxfp4(T, a.cuda(), asf.cuda(), w.cuda(), wsf.cuda(), c.plan, out, a_rows=a_rows,
                             out_rows=out_rows)
    want = product(c, value(a, asf), value(w, wsf), a_rows, out_rows, n).float()
    nan = torch.isnan(want)
    assert nan.any() and not nan.all()
    assert torch.equal(torch.isnan(out.cpu()), nan) and torch.equal(out.cpu()[~nan], want[~nan])


@pytest.mark.parametrize("kk", [320, 1024])
def test_mxfp4_scales_of_every_size(kk):
    """On the 256 x 256 tile: every scale byte but the largest, whose products leave fp32."""
    c = Fixed(2, even_ids(600, 2))
    g = gen(kk)
    n = 264
    a, w = codes(g, 600, kk // 2), codes(g, 2, n, kk // 2)
    asf = torch.randint(60, 190, (600, kk // 32), generator=g, dtype=torch.uint8)
    wsf = torch.randint(100, 150, (2, n, kk // 32), generator=g, dtype=torch.uint8)
    out = torch.empty((600, n), device="cuda")
    c.moe.grouped_gemm_mxfp4(600, a.cuda(), asf.cuda(), w.cuda(), wsf.cuda(), c.plan, out, a_rows="token",
                             out_rows="pair")
    av, wv = value(a, asf), value(w, wsf)
    want, size = (product(c, x, y, "token", "pair", n) for x, y in ((av, wv), (av.abs(), wv.abs())))
    # kk - 1 sums of fp32, each rounded (or cut) by less than 2^-23 of a partial sum, which is at most `size`
    assert ((out.cpu().double() - want).abs() <= kk * 2.0 ** -23 * size).all()


def test_gradient_of_masked_tokens_input():
    """The rows of masked slots are not written: what the buffer held there, a NaN too, stays out of the token's gradient
    where moe_combine adds the others up."""
    T, E, k, H, n = 90, 4, 3, 64, 128
    c = Case(T, E, k, seed=3, mask=0.3, H=H)
    assert (c.ids < 0).any(1).any() and c.rows < T * k
    g = gen(6)
    dgu, w = whole(g, T * k, n), whole(g, E, n, H)
    pairs = torch.full((T * k, H), NAN, dtype=torch.bfloat16, device="cuda")
    dx = torch.empty((T, H), dtype=torch.bfloat16, device="cuda")
    c.moe.grouped_gemm(T, dgu.cuda(), w.cuda(), c.plan, pairs, out_rows="pair", w_kn=True)
    c.moe.combine(T, pairs, torch.ones((T, k), device="cuda"), c.plan, dx)
    want = product(c, dgu, w, "plan", "pair", H, True).to(torch.bfloat16).double()
    masked = c.ids.reshape(-1) < 0
    assert torch.isnan(pairs.cpu()[masked]).all()
    want[masked] = 0.0
    assert torch.equal(dx.cpu(), want.view(T, k, H).sum(1).to(torch.bfloat16))  # (whole numbers: fp32 sums are exact)
