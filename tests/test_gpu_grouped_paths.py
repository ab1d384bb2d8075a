"""The kernels behind the products by expert: each choice by rows an expert and tiles, at its edges, with several tiles a
workgroup, more experts than lanes, gathered and scattered rows, long tensors, and calls side by side.  Whole numbers whose
sums fp32 holds, against float64: results have to be equal."""
import pytest
import torch

from mixture_experts_ffn_topk_amd import MoEFFN
from test_gpu_grouped import LEFT, Case, codes, product, value, whole

pytestmark = pytest.mark.gpu


def gen(seed):
    return torch.Generator().manual_seed(seed)


def even_ids(T, E):
    return (torch.arange(T) % E)[:, None]


class Fixed(Case):
    """A Case with these ids [T, k]."""

    def __init__(self, E, ids):
        self.T, self.k, self.E, self.ids = *ids.shape, E, ids
        flat = ids.reshape(-1)
        self.pairs = torch.cat([(flat == e).nonzero().reshape(-1) for e in range(E)])
        self.start = [0] + torch.stack([(flat == e).sum() for e in range(E)]).cumsum(0).tolist()
        self.rows = self.start[-1]
        self.moe = MoEFFN(64, 64, E, self.k, self.T, fmt="w4a8_mx")
        self.plan = self.moe.alloc_plan(self.T)
        self.moe.plan(self.T, self.plan, topk_idx=ids.cuda(), ws=self.moe.alloc_workspace(self.T))


def check_rows(c, n, kk, a_rows, out_rows, kn, f32, seed=0):
    g = gen(seed)
    a = whole(g, c.count(a_rows), kk)
    w = whole(g, c.E, *((kk, n) if kn else (n, kk)))
    out = torch.full((c.T * c.k, n), LEFT, dtype=torch.float32 if f32 else torch.bfloat16).cuda()
    c.moe.grouped_gemm(c.T, a.cuda(), w.cuda(), c.plan, out, a_rows=a_rows, out_rows=out_rows, w_kn=kn)
    want = product(c, a, w, a_rows, out_rows, n, kn).to(out.dtype)  # (sums below 2^24: one rounding)
    assert torch.equal(out.cpu(), want)


def check_mx(c, n, kk, a_rows, out_rows, f32, seed=0):
    g = gen(seed)
    q, w = codes(g, c.count(a_rows), kk // 2), codes(g, c.E, n, kk // 2)
    # (exponents apart by at most 2: sums of multiples of 1/8 below 2^21)
    sf = torch.randint(126, 128, (len(q), kk // 32), generator=g, dtype=torch.uint8)
    w_sf = torch.randint(127, 129, (c.E, n, kk // 32), generator=g, dtype=torch.uint8)
    out = torch.full((c.T * c.k, n), LEFT, dtype=torch.float32 if f32 else torch.bfloat16).cuda()
    c.moe.grouped_gemm_mxfp4(c.T, q.cuda(), sf.cuda(), w.cuda(), w_sf.cuda(), c.plan, out, a_rows=a_rows,
                             out_rows=out_rows)
    want = product(c, value(q, sf), value(w, w_sf), a_rows, out_rows, n).to(out.dtype)
    assert torch.equal(out.cpu(), want)


def check_wgrad(c, n, kk, d_rows, a_rows, f32, accumulate=False, seed=0):
    g = gen(seed)
    dout, a = whole(g, c.count(d_rows), n), whole(g, c.count(a_rows), kk)
    dw = torch.full((c.E, n, kk), LEFT, dtype=torch.float32 if f32 else torch.bfloat16).cuda()
    c.moe.grouped_gemm_wgrad(c.T, dout.cuda(), a.cuda(), c.plan, dw, dout_rows=d_rows, a_rows=a_rows,
                             accumulate=accumulate)
    ds, as_ = c.pick(d_rows), c.pick(a_rows)
    for e, lo, hi in c.spans():
        want = dout[ds[lo:hi]].double().T @ a[as_[lo:hi]].double() + (LEFT if accumulate else 0.0)
        assert torch.equal(dw[e].cpu(), want.to(dw.dtype)), e


# rows an expert about every change of kernel: 4 | 5 (forward), 12 | 13 and 24 | 25 (MXFP4), 48 | 49 and 64 | 65
@pytest.mark.parametrize("rows", [1, 4, 5, 6, 12, 13, 15, 16, 17, 24, 25, 32, 33, 48, 49, 64, 65, 128, 129, 257])
@pytest.mark.parametrize("n,kk", [(264, 96), (1032, 1056)])
def test_rows_an_expert(rows, n, kk):
    c = Fixed(3, even_ids(3 * rows, 3))
    assert c.start == [0, rows, 2 * rows, 3 * rows]
    check_rows(c, n, kk, "plan", "plan", False, False)
    check_rows(c, n, kk, "token", "pair", False, True)
    check_rows(c, n, kk, "pair", "pair", True, False)
    check_mx(c, n, kk, "token", "plan", False)
    check_mx(c, n, kk, "plan", "pair", True)
    check_wgrad(c, n, kk, "pair", "plan", False)
    check_wgrad(c, kk, n, "plan", "token", True, accumulate=True)


# (T, E, k, n, k of the product): more tiles than compute units of 256 x 256 and of 128 x 128, uneven experts, some of
# them empty; the last with more experts than lanes of a wave
MANY = [(900, 4, 1, 25608, 136), (300, 5, 1, 25608, 72), (2100, 70, 2, 2056, 96), (1300, 150, 4, 1048, 64)]


@pytest.mark.parametrize("T,E,k,n,kk", MANY)
@pytest.mark.parametrize("f32", [False, True])
def test_many_tiles(T, E, k, n, kk, f32):
    c = Case(T, E, k, seed=3, skew=1.2, mask=0.1)
    check_rows(c, n, kk, "token", "pair", False, f32)
    check_rows(c, n, kk, "plan", "plan", False, f32)
    check_rows(c, n, kk, "pair", "plan", True, f32)


@pytest.mark.parametrize("T,E,k,n,kk", [(900, 4, 1, 25608, 160), (2100, 70, 2, 2056, 96), (700, 3, 1, 25608, 544)])
@pytest.mark.parametrize("f32", [False, True])
def test_many_tiles_mxfp4(T, E, k, n, kk, f32):
    c = Case(T, E, k, seed=4, skew=1.2, mask=0.1)
    check_mx(c, n, kk, "token", "pair", f32)
    check_mx(c, n, kk, "plan", "plan", f32)


# several tiles a workgroup; 2048 x 2048: 64 tiles of 256 x 256, an expert's in chunks; 1800 x 1544: not in chunks
@pytest.mark.parametrize("T,E,k,n,kk", [(900, 6, 1, 2048, 2048), (1200, 9, 2, 1800, 1544), (500, 80, 2, 520, 264)])
@pytest.mark.parametrize("f32,accumulate", [(False, False), (True, False), (True, True)])
def test_many_tiles_wgrad(T, E, k, n, kk, f32, accumulate):
    c = Case(T, E, k, seed=5, skew=1.0, mask=0.1)
    for orders in (("plan", "plan"), ("pair", "plan"), ("plan", "token"), ("token", "pair")):
        check_wgrad(c, n, kk, *orders, f32, accumulate)


@pytest.mark.parametrize("kk", [32, 64, 128, 512, 640, 1152])
def test_mxfp4_k_steps(kk):
    """One to five K-steps of 256, scales of whole words or not, over several tiles a workgroup."""
    check_mx(Fixed(2, even_ids(600, 2)), 25608, kk, "token", "pair", False)
    check_mx(Fixed(2, even_ids(600, 2)), 264, kk, "plan", "plan", True)


def test_an_expert_with_all_rows():
    """The mean chooses the kernel for few rows, and one expert has them all."""
    c = Fixed(200, torch.full((600, 1), 7))
    check_rows(c, 264, 72, "token", "pair", False, False)
    check_rows(c, 264, 72, "plan", "plan", True, False)
    check_mx(c, 264, 96, "token", "pair", False)
    check_wgrad(c, 264, 136, "token", "plan", True)


@pytest.mark.parametrize("kk", [32, 64, 96, 2880, 4128])
def test_mxfp4_scales_at_the_tensors_end(kk):
    """Rows of scales that are not whole words, the last row's at the tensor's end."""
    for rows in (1, 9, 40):
        check_mx(Fixed(2, even_ids(2 * rows, 2)), 8, kk, "pair", "plan", True)


def test_rows_past_four_gigabytes():
    """Tensors in the plan's order may be any size: 2^19 + 300 rows of 8192 bytes, the last of them."""
    T, n, kk = (1 << 19) + 300, 16, 4096
    c = Fixed(2, torch.cat([torch.zeros(T - 40, 1, dtype=torch.int64), torch.ones(40, 1, dtype=torch.int64)]))
    a = torch.randint(-3, 4, (T, kk), dtype=torch.int8, device="cuda").to(torch.bfloat16)
    w = whole(gen(1), 2, n, kk)
    out = torch.empty(T, n, device="cuda")
    c.moe.grouped_gemm(T, a, w.cuda(), c.plan, out)
    lo, hi = T - 700, T - 40
    for rows, e in ((slice(0, 300), 0), (slice(lo, hi), 0), (slice(hi, T), 1)):
        assert torch.equal(out[rows].cpu().double(), a[rows].cpu().double() @ w[e].double().T)
    dw = torch.empty(2, n, kk, device="cuda")
    dout = torch.zeros(T, n, dtype=torch.bfloat16, device="cuda")
    dout[lo:] = whole(gen(2), T - lo, n).cuda()
    c.moe.grouped_gemm_wgrad(T, dout, a, c.plan, dw)
    for rows, e in ((slice(lo, hi), 0), (slice(hi, T), 1)):
        assert torch.equal(dw[e].cpu().double(), dout[rows].cpu().double().T @ a[rows].cpu().double())
    wide = torch.empty(T, kk, dtype=torch.bfloat16, device="cuda")  # an output of more than 4 GiB, from rows of 16
    wt = whole(gen(3), 2, kk, n)
    c.moe.grouped_gemm(T, dout, wt.cuda(), c.plan, wide)
    for rows, e in ((slice(lo, hi), 0), (slice(hi, T), 1)):
        assert torch.equal(wide[rows].cpu(), (dout[rows].cpu().double() @ wt[e].double().T).to(torch.bfloat16))


def test_calls_side_by_side_and_replayed():
    """Two streams at once and one graph of every kernel, replayed with other inputs, eager calls between."""
    cases = [(Fixed(3, even_ids(n * 3, 3)), n) for n in (2, 30, 200)]
    n, kk = 520, 264
    g = gen(9)
    jobs = []
    for c, _ in cases:
        a, d = whole(g, c.T, kk).cuda(), whole(g, c.T, n).cuda()
        w = whole(g, 3, n, kk).cuda()
        jobs.append((c, a, d, w, torch.empty(c.T, n, device="cuda"), torch.empty(c.T, kk, device="cuda"),
                     torch.empty(3, n, kk, device="cuda")))

    def run():
        for c, a, d, w, y, da, dw in jobs:
            c.moe.grouped_gemm(c.T, a, w, c.plan, y, a_rows="token", out_rows="pair")
            c.moe.grouped_gemm(c.T, d, w, c.plan, da, a_rows="pair", out_rows="pair", w_kn=True)
            c.moe.grouped_gemm_wgrad(c.T, d, a, c.plan, dw, dout_rows="pair", a_rows="token")

    def check():
        torch.cuda.synchronize()
        for c, a, d, w, y, da, dw in jobs:
            for e in range(3):
                A, D, W = a[e::3].cpu().double(), d[e::3].cpu().double(), w[e].cpu().double()
                assert torch.equal(y[e::3].cpu().double(), A @ W.T)
                assert torch.equal(da[e::3].cpu().double(), D @ W)
                assert torch.equal(dw[e].cpu().double(), D.T @ A)

    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    held = jobs
    for s, part in zip(streams, (held[:2], held[2:])):
        jobs = part
        with torch.cuda.stream(s):
            for _ in range(5):
                run()
    jobs = held
    check()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        run()
    for turn in range(3):
        for c, a, d, w, y, da, dw in jobs:
            a.copy_(whole(g, c.T, kk))
            d.copy_(whole(g, c.T, n))
            for t in (y, da, dw):
                t.fill_(LEFT)
        torch.cuda.synchronize()
        graph.replay()
        check()
        run()
        check()
