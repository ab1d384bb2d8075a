"""moe_swiglu and moe_swiglu_backward over the range of bf16: infinite gates and up columns, zeros, NaNs and far negative
gates, without a clamp and with one, element by element against float64.  Infinities and NaNs have to stand where the
definition has them."""
import itertools

import pytest
import torch

from test_gpu_grouped import Case, quantised

pytestmark = pytest.mark.gpu

INF, NAN = float("inf"), float("nan")
# (-174: from there on the sigmoid's square root leaves fp32's normal numbers)
GATES = (INF, -INF, 0.0, -0.0, 1.0, -1.0, 10.0, 20.0, -20.0, -88.0, -90.0, 3e38, -3e38, NAN)
UPS = (0.0, -0.0, 0.25, -0.25, 2.0, -2.0, 1000.0, -1e10, 1e30, INF, -INF, NAN)
GRADIENTS = (0.0, 0.25, -0.25, 3.0, INF, NAN)


def definition(g, u, d, clamp):
    """(h, dg, du) in float64; g s(g) and s(g) (1 + g (1 - s(g))) at -infinity are their limits, 0, and at +infinity the
    second's is 1."""
    gc = torch.where(g > clamp, clamp, g)
    uc = torch.where(u > clamp, clamp, torch.where(u < -clamp, -clamp, u))
    s = torch.sigmoid(gc)
    gs = torch.where(gc == -INF, torch.zeros_like(gc), gc * s)
    bounded = torch.where(gc.isinf(), gc.sign() * 1e30, gc)
    dg = torch.where(g > clamp, torch.zeros_like(d), d * uc * s * (1 + bounded * (1 - s)))
    return gs * uc, dg, torch.where(u.abs() > clamp, torch.zeros_like(d), d * gs)


def near(got, want, extra):
    """Infinities and NaNs as in want rounded to bf16 (no finite value here is within one rounding of the largest); else
    half a bf16 step (2^-8 of the value, or half the smallest one) and `extra`."""
    got, want = got.cpu().double(), want.double()
    far = want.float().to(torch.bfloat16).double()
    assert torch.equal(torch.isnan(got), torch.isnan(want))
    assert torch.equal(torch.isinf(got), torch.isinf(far))
    assert torch.equal(got[torch.isinf(far)], far[torch.isinf(far)])
    ok = torch.isfinite(far)
    off = (got - want).abs()[ok]
    assert (off <= (2.0 ** -8 * want.abs() * (1 + 2.0 ** -8) + 2.0 ** -134 + 1.01 * extra)[ok]).all()


def grid(gates, ups, gradients):
    """Rows, one for each gradient, of every pair of a gate and an up value: (gu, dh, I)."""
    pairs = list(itertools.product(gates, ups))
    pairs += [(1.0, 1.0)] * (-len(pairs) % 32)
    g, u = (torch.tensor(v) for v in zip(*pairs))
    rows = len(gradients)
    return (torch.cat([g, u]).to(torch.bfloat16).repeat(rows, 1),
            torch.tensor(gradients).to(torch.bfloat16)[:, None].repeat(1, len(pairs)), len(pairs))


def check(gates, ups, gradients, fast, clamp):
    gu, dh, I = grid(gates, ups, gradients)
    rows = len(gradients)
    c = Case(rows, 2, 1, seed=1, I=I, fast_math=fast, activation_clamp=clamp)
    h, h2 = (torch.empty((rows, I), dtype=torch.bfloat16, device="cuda") for _ in range(2))
    dgu = torch.empty((rows, 2 * I), dtype=torch.bfloat16, device="cuda")
    c.moe.swiglu(rows, gu.cuda(), c.plan, h=h)
    c.moe.swiglu_backward(rows, gu.cuda(), dh.cuda(), c.plan, dgu, h=h2)
    g, u, d = gu[:, :I].double(), gu[:, I:].double(), dh.double()
    wh, wg, wu = definition(g, u, d, clamp)
    # fp32: the exponent -|g'| log2(e) / 2 and its constant are each rounded (2^-24 of it), and the square doubles that:
    # |g'| 2^-23 of the sigmoid; exp2 (twice), 1 + e, the reciprocal and four products each by at most 2^-23.  1 + g' (1 - s)
    # is formed of numbers up to 1 + |g'|, whose errors do not shrink with the sum.
    gp = torch.where(g > clamp, clamp, g).abs().nan_to_num(0.0, posinf=0.0)
    gp = torch.where(gp > 1e30, torch.zeros_like(gp), gp)  # (the sigmoid is 0 or 1)
    rel = (gp + 9) * 2.0 ** -23
    finite = lambda v: v.abs().nan_to_num(0.0, posinf=0.0)  # noqa: E731
    near(h, wh, rel * finite(wh))
    assert torch.equal(h.view(torch.int16), h2.view(torch.int16))
    s = torch.sigmoid(torch.where(g > clamp, clamp, g)).nan_to_num(0.0)
    near(dgu[:, :I], wg, rel * finite(d) * finite(u.clamp(-clamp, clamp)) * s * (1 + gp))
    near(dgu[:, I:], wu, rel * finite(wu))


@pytest.mark.parametrize("fast", [True, False])
@pytest.mark.parametrize("clamp", [INF, 10.0, 1.5])
def test_whole_range(fast, clamp):
    check(GATES, UPS, GRADIENTS, fast, clamp)


@pytest.mark.parametrize("fast", [True, False])
def test_an_infinite_gate_shows_in_mxfp4(fast):
    """Without a clamp: sf of the largest exponent where a finite up column meets it, of NaN where a zero does."""
    c = Case(1, 2, 1, I=96, fast_math=fast, activation_clamp=INF)
    gu = torch.ones((1, 192), dtype=torch.bfloat16)
    gu[0, 3], gu[0, 96 + 3] = INF, -0.25
    gu[0, 40], gu[0, 96 + 40] = INF, 0.0
    q, sf = (torch.zeros((1, n), dtype=torch.uint8, device="cuda") for n in (48, 3))
    c.moe.swiglu(1, gu.cuda(), c.plan, q=q, sf=sf)
    h = definition(gu[:, :96].double(), gu[:, 96:].double(), torch.zeros(1, 96).double(), INF)[0]
    code, scale, _, nan = quantised(h)
    assert scale.tolist()[0][:2] == [254, 255] and nan.tolist() == [[False, True, False]]
    assert torch.equal(sf.cpu().long(), scale.long())
    got = torch.stack([q & 15, q >> 4], -1).flatten(-2).cpu().long()
    assert got[0, 3] == 15 and torch.equal(got[0, :32], code[0, :32]) and torch.equal(got[0, 64:], code[0, 64:])


@pytest.mark.parametrize("fast", [True, False])
def test_large_up_columns_at_far_negative_gates(fast):
    """g' s below fp32's normal numbers where h and its gradients are not."""
    check((-80.0, -95.0, -100.0, -103.0, -104.5, -107.0, -110.0, -130.0, -150.0, -174.0),
          (1000.0, -1e10, 1e20, -1e30, 1e35, INF), (0.25, -3.0, 1000.0), fast, INF)
