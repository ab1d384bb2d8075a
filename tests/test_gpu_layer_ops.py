"""GPU tests of moe_add_rmsnorm, moe_router_logits and moe_forward_few against the
float64 oracle."""
import numpy as np
import pytest
import torch

import moe_synth
import oracle
from gpu_util import dev, device_inputs, fwd_kwargs, geometry, make_moe, prepared
from mixture_experts_ffn_topk_amd import MoEFFN
from oracle import layer as ol

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():  # pragma: no cover
    pytest.skip("needs a GPU", allow_module_level=True)

BF16_HALF = 2.0 ** -8   # half a bf16 step, relative
E4M3_HALF, E4M3_SUB = 2.0 ** -4, 2.0 ** -10  # half a step, relative; below the smallest normal number
# the norm before its last rounding: at most ~64 fp32 roundings in the sum of
# squares (halved by the root), the addition, the reciprocal root and two products: under 2^-18
NORM_REL = 2.0 ** -18


def bits(t):
    return t.detach().float().cpu().numpy().astype(np.float64)


# ------------------------------------------------------------------ residual + RMS norm
def norm_case(fmt, T, H, xt, rt, wt, seed, scale=1.0, eps=1e-6, make=None, x_gs=1.0, x_norm=True, x_q=True):
    g = torch.Generator().manual_seed(seed)
    x = (torch.randn(T, H, generator=g) * scale).to(xt)
    r = None if rt is None else (torch.randn(T, H, generator=g) * 3 * scale).to(rt)
    w = (1 + 0.3 * torch.randn(H, generator=g)).to(wt)
    if make is not None:
        make(x, r, w)
    moe = MoEFFN(H, 128, 4, 2, max(T, 1), fmt=fmt)
    o = {"residual_out": None if r is None else torch.full_like(r, float("nan"), device="cuda"),
         "x_norm": torch.full((T, H), float("nan"), dtype=torch.bfloat16, device="cuda") if x_norm else None,
         "x_q": None, "x_sf": None}
    if x_q and fmt not in ("bf16", "nvfp4_w4a16"):
        o["x_q"] = torch.full((T, H // 2 if fmt == "nvfp4" else H), 0x7F, dtype=torch.uint8, device="cuda")
        o["x_sf"] = (torch.full((T, H // 128), float("nan"), device="cuda") if fmt == "fp8_block128" else
                     torch.full((T, H // (16 if fmt == "nvfp4" else 32)), 0xEE, dtype=torch.uint8, device="cuda"))
    moe.add_rmsnorm(T, x.cuda(), None if r is None else r.cuda(), w.cuda(), eps, x_global_scale=x_gs, **o)
    torch.cuda.synchronize()
    z, n = ol.add_rmsnorm(bits(x), None if r is None else bits(r), bits(w), eps)
    return o, z, n


def check_norm(fmt, o, z, n, x_gs=1.0):
    if o["residual_out"] is not None:
        half = BF16_HALF if o["residual_out"].dtype == torch.bfloat16 else 2.0 ** -24
        assert np.all(np.abs(bits(o["residual_out"]) - z) <= (half + 2.0 ** -24) * np.abs(z) * (1 + half))
    if o["x_norm"] is not None:
        assert np.all(np.abs(bits(o["x_norm"]) - n) <= (BF16_HALF + NORM_REL) * np.abs(n) * (1 + BF16_HALF) + 2.0 ** -133)
    if o["x_q"] is None:
        return
    q, sf = o["x_q"].cpu().numpy(), o["x_sf"].cpu().numpy()
    block = {"fp8_block128": 128, "w4a8_mx": 32, "nvfp4": 16}[fmt]
    amax = np.abs(n.reshape(n.shape[0], -1, block)).max(axis=2)
    if fmt == "fp8_block128":
        s = sf.astype(np.float64)
        want = ol.act_scales(fmt, n)
        assert np.all(np.abs(s - want) <= (NORM_REL + 2.0 ** -23) * want)
        v = oracle.e4m3_decode(q)
    elif fmt == "w4a8_mx":
        s = oracle.ue8m0_decode(sf)
        # the exponent of a maximum within the norm's error of the true one
        lo, hi = ol.act_scales(fmt, n * (1 - NORM_REL)), ol.act_scales(fmt, n * (1 + NORM_REL))
        assert np.all((s == lo) | (s == hi))
        v = oracle.e4m3_decode(q)
    else:
        s = oracle.e4m3_decode(sf)
        s6 = np.minimum(amax / (6.0 * x_gs), 448.0)
        assert np.all(np.abs(s - s6) <= np.maximum(E4M3_HALF * s6, E4M3_SUB) + 2 * NORM_REL * s6)
        v = oracle.e2m1_decode_nibbles(oracle.e2m1_unpack(q))
    den = np.repeat(s, block, axis=1) * (x_gs if fmt == "nvfp4" else 1.0)
    a = np.abs(np.where(den > 0, n / np.where(den > 0, den, 1.0), 0.0))
    err = np.abs(v - np.where(den > 0, n / np.where(den > 0, den, 1.0), 0.0))
    if fmt == "nvfp4":
        half = np.where(a <= 2.0, 0.25, np.where(a <= 4.0, 0.5, 1.0))
        ok = err <= half + 4 * NORM_REL * a
        ok |= (a > 6.0) & (np.abs(v) == 6.0)  # saturated
    else:
        # (448 is the largest code: a scale rounded down puts the maximum a hair above it)
        ok = err <= np.maximum(E4M3_HALF * a, E4M3_SUB) + 4 * NORM_REL * a
    assert np.all(ok)


@pytest.mark.parametrize("fmt,T,H", [
    ("fp8_block128", 1, 7168), ("fp8_block128", 3, 128), ("fp8_block128", 33, 384), ("fp8_block128", 2, 32768),
    ("fp8_block128", 5, 8320), ("w4a8_mx", 7, 2880), ("w4a8_mx", 1, 32), ("w4a8_mx", 130, 96), ("w4a8_mx", 2, 16416),
    ("bf16", 3, 4096), ("bf16", 1, 64), ("nvfp4_w4a16", 2, 192), ("nvfp4", 5, 448), ("nvfp4", 1, 7168)])
@pytest.mark.parametrize("types", ["bf16", "f32", "mixed", "none"])
def test_norm(fmt, T, H, types):
    b, f = torch.bfloat16, torch.float32
    xt, rt, wt = {"bf16": (b, b, b), "f32": (f, f, f), "mixed": (b, f, f), "none": (f, None, b)}[types]
    o, z, n = norm_case(fmt, T, H, xt, rt, wt, seed=T * 1000 + H, x_gs=0.0023)
    check_norm(fmt, o, z, n, x_gs=0.0023)


@pytest.mark.parametrize("fmt", ["fp8_block128", "w4a8_mx", "nvfp4"])
def test_norm_zero_rows_blocks_and_outliers(fmt):
    """A row of zeros, a block whose weights are zero, one huge channel, tiny values."""
    def make(x, r, w):
        x[1].zero_()
        r[1].zero_()
        w[128:256] = 0.0
        x[2, 5] = 3.0e4
        x[3] *= 2.0 ** -60
        r[3] *= 2.0 ** -60
    o, z, n = norm_case(fmt, 5, 512, torch.bfloat16, torch.bfloat16, torch.bfloat16, seed=3, make=make, x_gs=0.01)
    check_norm(fmt, o, z, n, x_gs=0.01)
    q = o["x_q"].cpu().numpy()
    assert not q[1].any()
    if fmt == "fp8_block128":
        assert float(o["x_sf"][1, 0]) == 1.0 and float(o["x_sf"][0, 1]) == 1.0
    if fmt == "w4a8_mx":
        assert int(o["x_sf"][1, 0]) == 0


def test_norm_scale_floor():
    """Weights so small that amax / 448 is below the smallest normal number: the scale is that number, all codes finite."""
    def make(x, r, w):
        w.fill_(2.0 ** -122)
    o, z, n = norm_case("fp8_block128", 2, 256, torch.float32, None, torch.float32, seed=9, make=make)
    assert np.all(o["x_sf"].cpu().numpy() == np.float32(2.0 ** -126))
    check_norm("fp8_block128", o, z, n)


@pytest.mark.parametrize("fmt", ["fp8_block128", "w4a8_mx", "bf16"])
@pytest.mark.parametrize("eps", [0.0, 1e-6])
def test_norm_rows_whose_squares_leave_fp32(fmt, eps):
    """Rows of 2^100 and, without eps, of 2^-100: their norms are those of the same rows at 1."""
    def make(x, r, w):
        x[1] *= 2.0 ** 100
        r[1] *= 2.0 ** 100
        if eps == 0.0:
            x[2] *= 2.0 ** -100
            r[2] *= 2.0 ** -100
    o, z, n = norm_case(fmt, 4, 512, torch.bfloat16, torch.bfloat16, torch.bfloat16, seed=6, make=make, eps=eps)
    check_norm(fmt, o, z, n)


def test_norm_mx_codes_are_those_of_the_unrounded_norm():
    """Codes of the fp64 norm, rounded once (the stream's sums are exact in fp32: small integers times 2^-6)."""
    T, H = 4096, 352
    g = torch.Generator().manual_seed(8)
    x = (torch.randint(-120, 121, (T, H), generator=g) * 2.0 ** -6).bfloat16()
    r = (torch.randint(-120, 121, (T, H), generator=g) * 2.0 ** -6).bfloat16()
    w = (1 + 0.3 * torch.randn(H, generator=g)).bfloat16()
    moe = MoEFFN(H, 32, 2, 1, T, fmt="w4a8_mx")
    q = torch.empty((T, H), dtype=torch.uint8, device="cuda")
    sf = torch.empty((T, H // 32), dtype=torch.uint8, device="cuda")
    ro = torch.empty_like(r, device="cuda")
    moe.add_rmsnorm(T, x.cuda(), r.cuda(), w.cuda(), 1e-6, residual_out=ro, x_q=q, x_sf=sf)
    _, n = ol.add_rmsnorm(bits(x), bits(r), bits(w), 1e-6)
    codes = oracle.e4m3_decode(q.cpu().numpy()).reshape(T, H // 32, 32)
    v = n.reshape(T, H // 32, 32) / oracle.ue8m0_decode(sf.cpu().numpy())[..., None]
    step = np.exp2(np.maximum(np.floor(np.log2(np.abs(v) + 1e-300)), -6.0) - 3.0)
    # half a step, and what two fp64 evaluations of the norm may differ by
    assert np.all(np.abs(codes - v) <= 0.5 * step * (1 + 2.0 ** -30))


@pytest.mark.parametrize("fmt", ["fp8_block128", "w4a8_mx", "nvfp4"])
def test_norm_nan_and_inf(fmt):
    """A NaN makes its row NaN, an infinity its own element (the rest of the row is finite / inf = 0); other rows keep
    their values; a block with a NaN has a NaN scale."""
    def make(x, r, w):
        x[1, 7] = float("nan")
        x[2, 300] = float("inf")
    o, _, _ = norm_case(fmt, 4, 512, torch.bfloat16, torch.bfloat16, torch.bfloat16, seed=4, make=make)
    ref, _, _ = norm_case(fmt, 4, 512, torch.bfloat16, torch.bfloat16, torch.bfloat16, seed=4)
    for name in ("x_norm", "x_q", "x_sf", "residual_out"):
        for row in (0, 3):
            assert torch.equal(o[name][row], ref[name][row])
    xn = o["x_norm"].float().cpu()
    assert torch.isnan(xn[1]).all()
    assert torch.isnan(xn[2, 300]) and not torch.isnan(xn[2, :300]).any() and (xn[2, :300] == 0).all()
    block = {"fp8_block128": 128, "w4a8_mx": 32, "nvfp4": 16}[fmt]
    sf = o["x_sf"].cpu().numpy()
    nan = np.isnan(sf) if fmt == "fp8_block128" else np.isnan(oracle.ue8m0_decode(sf) if fmt == "w4a8_mx" else oracle.e4m3_decode(sf))
    assert nan[1].all()
    assert nan[2, 300 // block] and nan[2].sum() == 1


def test_norm_in_place_matches():
    """residual_out = residual and x_norm = x give the bits of separate buffers; x_norm or x_q alone too."""
    T, H = 9, 768
    g = torch.Generator().manual_seed(11)
    x = torch.randn(T, H, generator=g).bfloat16().cuda()
    r = torch.randn(T, H, generator=g).bfloat16().cuda()
    w = torch.randn(H, generator=g).bfloat16().cuda()
    moe = MoEFFN(H, 128, 4, 2, T)
    ro, xn = torch.empty_like(r), torch.empty_like(x)
    q, sf = torch.empty((T, H), dtype=torch.uint8, device="cuda"), torch.empty((T, H // 128), device="cuda")
    moe.add_rmsnorm(T, x, r, w, 1e-5, residual_out=ro, x_norm=xn, x_q=q, x_sf=sf)
    q2, sf2, xn2 = torch.empty_like(q), torch.empty_like(sf), torch.empty_like(xn)
    moe.add_rmsnorm(T, x, r, w, 1e-5, residual_out=torch.empty_like(r), x_q=q2, x_sf=sf2)
    moe.add_rmsnorm(T, x, r, w, 1e-5, residual_out=torch.empty_like(r), x_norm=xn2)
    assert torch.equal(q, q2) and torch.equal(sf, sf2) and torch.equal(xn, xn2)
    moe.add_rmsnorm(T, x, r, w, 1e-5, residual_out=r, x_norm=x, x_q=q2.zero_(), x_sf=sf2.zero_())
    assert torch.equal(r, ro) and torch.equal(x, xn) and torch.equal(q, q2) and torch.equal(sf, sf2)


def test_norm_leaves_rows_behind_the_last():
    o, z, n = norm_case("fp8_block128", 4, 256, torch.bfloat16, torch.bfloat16, torch.bfloat16, seed=5)
    T, H = 2, 256
    moe = MoEFFN(H, 128, 4, 2, 4)
    x = torch.randn(4, H).bfloat16().cuda()
    xn = torch.full((4, H), 7.0, dtype=torch.bfloat16, device="cuda")
    moe.add_rmsnorm(T, x, None, torch.ones(H, dtype=torch.bfloat16, device="cuda"), 1e-6, x_norm=xn)
    assert (xn[T:] == 7.0).all() and not (xn[:T] == 7.0).all()
    moe.add_rmsnorm(0, x, None, torch.ones(H, dtype=torch.bfloat16, device="cuda"), 1e-6, x_norm=xn)


# ------------------------------------------------------------------ router logits
def router_tolerance(x, w, H):
    """fp32 sums: at most 32 additions inside an MFMA; a chain of 12 MFMAs per K-step of 64 (three terms of four) over
    a fourth of the K-steps, rounded up, where four groups share them, or over at most nine (the larger tiles: H up to
    1024 in two groups, 2112 in four parts, 192 in one); 8 for the groups' and splits' sums: each within 2^-23 of the
    running sum's bound.  The terms of an fp32 weight hold it exactly."""
    steps = -(-H // 64)
    return (40 + max(3 * (steps + 3), min(12 * steps, 108))) * 2.0 ** -23 * (np.abs(x) @ np.abs(w).T) + 1e-37


@pytest.mark.parametrize("T,H,E", [
    (1, 7168, 256), (1, 64, 1), (2, 96, 3), (3, 2880, 128), (5, 4096, 8), (8, 512, 40), (9, 512, 33), (16, 1056, 17),
    (31, 7168, 256), (64, 2880, 128), (100, 320, 512), (257, 7168, 64), (300, 32, 1000), (1000, 1024, 256),
    (2047, 2880, 128), (4099, 256, 8), (8192, 128, 257),
    (1500, 1056, 257), (4100, 1024, 128), (8500, 192, 260),
    (1111, 544, 256), (3000, 480, 200), (2500, 2080, 300), (5000, 2080, 129), (20000, 96, 40), (9000, 64, 64), (17000, 64, 8)])
@pytest.mark.parametrize("w32", [False, True])
def test_router_logits(T, H, E, w32):
    print(f"[router] T={T} H={H} E={E} w32={w32}", flush=True)
    g = torch.Generator().manual_seed(T + H + E)
    x = torch.randn(T, H, generator=g).bfloat16()
    w = torch.randn(E, H, generator=g) * H ** -0.5
    w = w if w32 else w.bfloat16()
    moe = MoEFFN(H, 64, E, 1, T, fmt="w4a8_mx")
    out = torch.full((T + 1, E), float("nan"), device="cuda")
    ws = moe.alloc_router_workspace(T)
    ws.fill_(0xFF)
    moe.router_logits(T, x.cuda(), w.cuda(), out, ws)
    torch.cuda.synchronize()
    ref = ol.router_logits(bits(x), bits(w))
    got = bits(out)
    assert np.isnan(got[T]).all()
    assert np.all(np.abs(got[:T] - ref) <= router_tolerance(bits(x), bits(w), H))
    again = torch.empty_like(out)
    moe.router_logits(T, x.cuda(), w.cuda(), again, ws)
    assert torch.equal(out[:T], again[:T])


@pytest.mark.parametrize("T,H,E", [(1, 96, 5), (4, 96, 5), (64, 192, 40), (1000, 224, 256), (1500, 128, 256), (4096, 2080, 256),
                                   (9000, 64, 300)])
@pytest.mark.parametrize("w32", [False, True])
def test_router_one_hot_rows_read_the_weights_exactly(T, H, E, w32):
    g = torch.Generator().manual_seed(H)
    w = torch.randn(E, H, generator=g) * torch.exp2(torch.randint(-60, 60, (E, H), generator=g).float())
    w = w if w32 else w.bfloat16()
    at = torch.randint(0, H, (T,), generator=g)
    x = torch.zeros(T, H, dtype=torch.bfloat16)
    x[torch.arange(T), at] = -2.0
    moe = MoEFFN(H, 64, E, 1, T, fmt="w4a8_mx")
    out = torch.empty(T, E, device="cuda")
    moe.router_logits(T, x.cuda(), w.cuda(), out, moe.alloc_router_workspace(T))
    assert torch.equal(out.cpu(), -2.0 * w.float()[:, at].T)


@pytest.mark.parametrize("T", [1, 6, 40, 700])
def test_router_nan_and_inf_stay_in_their_row_and_column(T):
    H, E = 640, 48
    g = torch.Generator().manual_seed(T)
    x = torch.randn(T, H, generator=g).bfloat16()
    w = torch.randn(E, H, generator=g)
    moe = MoEFFN(H, 64, E, 1, T, fmt="w4a8_mx")
    ws = moe.alloc_router_workspace(T)
    ref = torch.empty(T, E, device="cuda")
    moe.router_logits(T, x.cuda(), w.cuda(), ref, ws)
    x2, w2 = x.clone(), w.clone()
    x2[T - 1, 3] = float("nan")
    w2[5, 7] = float("inf")
    w2[6, 8] = float("nan")
    x2[0, 7] = 2.0
    got = torch.empty(T, E, device="cuda")
    moe.router_logits(T, x2.cuda(), w2.cuda(), got, ws)
    clean_w = torch.empty(T, E, device="cuda")
    w3 = w2.clone()
    w3[5:7] = 0
    x3 = x2.clone()
    x3[T - 1] = 0
    moe.router_logits(T, x3.cuda(), w3.cuda(), clean_w, ws)
    assert torch.isnan(got[T - 1]).all()
    if T > 1:
        assert torch.isinf(got[0, 5]) and torch.isnan(got[: T - 1, 6]).all()
        keep = [e for e in range(E) if e not in (5, 6)]
        assert torch.equal(got[: T - 1][:, keep], clean_w[: T - 1][:, keep])


@pytest.mark.parametrize("T,H,E", [(2, 640, 48), (6, 640, 48), (40, 640, 48), (700, 640, 48), (1500, 2112, 257), (4100, 1024, 128)])
@pytest.mark.parametrize("w32", [False, True])
def test_router_infinities_keep_their_sign(T, H, E, w32):
    """An infinite activation or weight gives infinities of the products' signs, NaN where both signs or 0 x inf meet."""
    g = torch.Generator().manual_seed(T)
    x = torch.randn(T, H, generator=g).bfloat16()
    w = torch.randn(E, H, generator=g)
    w[w == 0] = 1.0
    w[:, 9] = torch.where(w[:, 9].bfloat16() == 0, 1.0, w[:, 9])
    x[0, 9] = float("-inf")
    w[3, 9] = 0.0
    w[5, H - 1] = float("inf")
    w[6, 1], w[6, 2] = float("inf"), float("-inf")
    x[:, 1], x[:, 2] = 1.0, 2.0
    x[1, H - 1] = 0.0
    if not w32:
        w = w.bfloat16()
    moe = MoEFFN(H, 64, E, 1, T, fmt="w4a8_mx")
    out = torch.empty(T, E, device="cuda")
    moe.router_logits(T, x.cuda(), w.cuda(), out, moe.alloc_router_workspace(T))
    got = out.cpu().double()
    ref = torch.zeros(T, E, dtype=torch.float64)
    ref[0] = -torch.sign(w[:, 9].double()) * float("inf")
    ref[:, 5] = torch.sign(x[:, H - 1].double()) * float("inf")
    ref[0, 5] = ref[0, 5] - torch.sign(w[5, 9].double()) * float("inf")
    ref[:, 6] = float("nan")
    odd = ~torch.isfinite(ref)
    assert torch.equal(torch.isnan(got), torch.isnan(ref))
    inf = odd & ~torch.isnan(ref)
    assert torch.equal(got[inf], ref[inf]) and torch.isfinite(got[~odd]).all()


def test_norm_and_router_offsets_past_32_bits():
    """An fp32 stream of 8.3 GB and activations of 4.2 GB: the first, a middle and the last rows."""
    T, H, E = 290000, 7168, 8
    rows = [0, 1, T // 2, T - 2, T - 1]
    g = torch.Generator(device="cuda").manual_seed(1)
    x = torch.empty((T, H), device="cuda").normal_(generator=g)
    r = torch.empty((T, H), device="cuda").normal_(generator=g)
    w = torch.empty(H, device="cuda").normal_(generator=g)
    xs, rs = x[rows].clone(), r[rows].clone()
    moe = MoEFFN(H, 64, E, 1, T, fmt="w4a8_mx")
    xn = torch.empty((T, H), dtype=torch.bfloat16, device="cuda")
    q = torch.empty((T, H), dtype=torch.uint8, device="cuda")
    sf = torch.empty((T, H // 32), dtype=torch.uint8, device="cuda")
    moe.add_rmsnorm(T, x, r, w, 1e-6, residual_out=r, x_norm=xn, x_q=q, x_sf=sf)
    z, n = ol.add_rmsnorm(bits(xs), bits(rs), bits(w), 1e-6)
    check_norm("w4a8_mx", {"residual_out": r[rows], "x_norm": xn[rows], "x_q": q[rows], "x_sf": sf[rows]}, z, n)
    for w32 in (False, True):
        rw = torch.empty((E, H), device="cuda").normal_(generator=g)
        rw = rw if w32 else rw.bfloat16()
        out = torch.empty((T, E), device="cuda")
        moe.router_logits(T, xn, rw, out, moe.alloc_router_workspace(T))
        ref = ol.router_logits(bits(xn[rows]), bits(rw))
        assert np.all(np.abs(bits(out[rows]) - ref) <= router_tolerance(bits(xn[rows]), bits(rw), H))


# ------------------------------------------------------------------ the layer for few tokens
def shape(fmt, T, H, I, E, k, routing="precomputed", seed=1, **kw):
    return moe_synth.MoEShape(f"few_{fmt}", seed, T, H, I, E, k, fmt, routing, **kw)


def few_inputs(sh, ids=None, tw=None, add=False, bias=False, idx_dtype=torch.int64):
    inp = moe_synth.make_inputs(sh)
    d = device_inputs(inp, ids, tw, idx_dtype)
    kw, okw = {}, {}
    rng = np.random.default_rng(sh.seed + 77)
    if add:
        for n in ("shared", "residual"):
            t = torch.from_numpy(rng.standard_normal((sh.tokens, sh.hidden), dtype=np.float32)).bfloat16()
            kw[n], okw[n] = t.cuda(), bits(t)
    if bias:
        b = rng.standard_normal(sh.experts).astype(np.float32)
        kw["routing_bias"], okw["routing_bias"] = torch.from_numpy(b).cuda(), b
    return inp, d, kw, okw


def run_few(moe, d, T, kw, out=None, ws=None, stream=None):
    if out is None:
        out = torch.full((T + 1, moe.hidden), float("nan"), dtype=torch.float32 if moe.out_fp32 else torch.bfloat16,
                         device="cuda")
    if ws is None:
        ws = moe.alloc_few_workspace(T)
        ws.fill_(0xFF)  # NaN in every format
    moe.forward_few(T, d["x"], d["x_sf"], d["topk_idx"], d["topk_weights"],
                    d["logits"] if moe.route_mode == "from_logits" else None, prepared(moe, d), out, ws, stream=stream, **kw)
    return out


def oracle_few(inp, okw, ids=None, tw=None):
    sh = inp["shape"]
    r = dict(okw)
    if sh.routing == "precomputed":
        r["topk_idx"] = inp["topk_idx"] if ids is None else ids
        r["topk_weights"] = inp["topk_weights"] if tw is None else tw
    else:
        r["logits"] = inp["logits"]
    return oracle.forward(geometry(sh), inp["x"], inp["x_sf"], inp["w13"], inp["w13_sf"], inp["w2"], inp["w2_sf"],
                          **r, **fwd_kwargs(inp))


def flip_bound(inp, ref):
    """The most that one requantised element of h moves an output by when its code is the neighbouring one: a step
    of the top binade (E4M3 2^-3, E2M1 2^-1 ... of the value, bf16 2^-7) times the largest |weight x h x w2|."""
    sh, geo = inp["shape"], geometry(inp["shape"])
    step = {"fp8_block128": 2.0 ** -3, "w4a8_mx": 2.0 ** -3, "nvfp4": 0.5}.get(sh.fmt, 2.0 ** -7)
    most = 0.0
    xd = oracle.dequant_activations(geo, inp["x"], inp["x_sf"])
    w = np.asarray(ref["topk_weights"])
    for e in range(sh.experts):
        t, j = np.nonzero(np.asarray(ref["topk_idx"]) == e)
        if not t.size:
            continue
        gs = {k: v for k, v in fwd_kwargs(inp).items() if k != "c_scales"}
        sf = lambda n: None if inp[n] is None else inp[n]
        w13, w2 = oracle.dequant_expert(geo, inp["w13"], sf("w13_sf"), inp["w2"], sf("w2_sf"), e, gs.get("w13_gs"),
                                        gs.get("w2_gs"))
        I = sh.inter
        h = oracle.swiglu_clamped(xd[t] @ w13[:I].T, xd[t] @ w13[I:].T, sh.clamp)
        c = float(inp["c_scales"][e]) if "c_scales" in inp else 1.0
        most = max(most, float((np.abs(w[t, j])[:, None] * np.abs(h)).max()) / c * float(np.abs(w2).max()))
    return step * most


def check_few(got, inp, ref, T, out_fp32=False, addends=()):
    """Half a bf16 step of the output and, on the routed sum: relative L2 1e-2 for 8- and 4-bit intermediates (an
    8-bit MFMA sums 128 products to ~14 bits, so codes near a midpoint differ: the tolerance of the same path's
    parity tests), 2^-10 for bf16 ones (1 in 2^6 of the codes off by 2^-7 would give 2^-10); any one element within
    two neighbouring codes at the largest term."""
    r = ref["out"][:T]
    g = bits(got[:T])
    assert np.isfinite(g).all()
    routed = r - sum((np.asarray(a, np.float64).reshape(r.shape) for a in addends), np.zeros_like(r))
    half = 2.0 ** -24 if out_fp32 else BF16_HALF
    tight = inp["shape"].fmt in ("bf16", "nvfp4_w4a16")
    rel = 2.0 ** -10 if tight else 1e-2
    assert np.linalg.norm(g - r) <= half * np.linalg.norm(r) + rel * np.linalg.norm(routed) + 1e-30
    assert np.all(np.abs(g - r) <= half * np.abs(r) * (1 + half) + 2 * flip_bound(inp, ref) +
                  2.0 ** -14 * np.abs(routed).max() + 1e-30)


SIZES = {"fp8_block128": (384, 256), "bf16": (192, 320), "w4a8_mx": (416, 288), "nvfp4_w4a16": (320, 192),
         "nvfp4": (320, 192)}


@pytest.mark.parametrize("fmt", list(SIZES))
@pytest.mark.parametrize("T", [1, 2, 5, 16, 17, 32])
@pytest.mark.parametrize("routing", ["precomputed", "from_logits"])
def test_few(fmt, T, routing):
    H, I = SIZES[fmt]
    sh = shape(fmt, T, H, I, 11, 3, routing, seed=T)
    print(f"[few] {sh}", flush=True)
    add = T % 2 == 0
    inp, d, kw, okw = few_inputs(sh, add=add, bias=routing == "from_logits")
    moe = make_moe(sh)
    out = run_few(moe, d, T, kw)
    torch.cuda.synchronize()
    ref = oracle_few(inp, okw)
    assert np.isnan(bits(out[T])).all()
    check_few(out, inp, ref, T, addends=[okw[n] for n in ("shared", "residual") if n in okw])
    if routing == "from_logits":
        assert np.array_equal(d["topk_idx"].cpu().numpy(), ref["topk_idx"])
        # hardware exp2 and reciprocal: a few fp32 roundings each of arguments up to ~8
        assert np.abs(d["topk_weights"].cpu().numpy() - ref["topk_weights"]).max() <= 2.0 ** -18
    again = run_few(moe, d, T, kw)
    assert torch.equal(out[:T], again[:T])


@pytest.mark.parametrize("fmt,H,I,E,k,T", [
    ("fp8_block128", 128, 128, 1, 1, 1),       # one of everything
    ("fp8_block128", 256, 128, 1, 1, 32),      # every token to one expert
    ("fp8_block128", 7168, 256, 16, 8, 1),     # a thin shard of a wide layer (h in LDS)
    ("fp8_block128", 256, 4096, 64, 8, 3),     # whole 128-column blocks
    ("fp8_block128", 384, 1024, 8, 2, 3), ("fp8_block128", 2944, 640, 9, 3, 5),  # h in LDS, more than a round of workgroups
    ("fp8_block128", 1024, 1024, 2, 2, 24),    # few experts, h too large for LDS
    ("bf16", 64, 64, 7, 7, 4), ("bf16", 2048, 64, 2, 1, 3), ("bf16", 64, 4096, 3, 2, 20),
    ("w4a8_mx", 32, 32, 5, 2, 3), ("w4a8_mx", 2880, 96, 40, 4, 32), ("w4a8_mx", 96, 2880, 6, 3, 2),
    ("nvfp4_w4a16", 64, 64, 4, 2, 7), ("nvfp4_w4a16", 1216, 192, 9, 4, 1), ("nvfp4", 64, 64, 4, 2, 7),
    ("nvfp4", 192, 1088, 9, 4, 18), ("nvfp4_w4a16", 192, 1088, 9, 4, 18), ("nvfp4_w4a16", 2880, 64, 5, 2, 6),
    # twice the tiles per down workgroup, and the same H with short parts
    ("bf16", 2432, 1344, 7, 3, 4), ("bf16", 5248, 192, 9, 3, 20), ("fp8_block128", 4224, 640, 12, 3, 9),
    ("fp8_block128", 4224, 128, 3, 1, 3), ("fp8_block128", 2944, 1152, 5, 2, 3), ("nvfp4_w4a16", 2880, 1024, 20, 4, 8),
    ("nvfp4", 2880, 1024, 20, 4, 8), ("nvfp4", 2880, 64, 4, 2, 2),
    ("bf16", 64, 64, 1000, 32, 32),            # more experts and slots than any wave holds
    ("w4a8_mx", 64, 64, 40, 32, 32),
    ("w4a8_mx", 512, 64, 1000, 32, 32)])       # the largest tables and sums in LDS
def test_few_sizes(fmt, H, I, E, k, T):
    sh = shape(fmt, T, H, I, E, k, seed=H + I)
    print(f"[few] {sh}", flush=True)
    inp, d, kw, okw = few_inputs(sh)
    out = run_few(make_moe(sh), d, T, kw)
    torch.cuda.synchronize()
    check_few(out, inp, oracle_few(inp, okw), T)


@pytest.mark.parametrize("fmt", list(SIZES))
@pytest.mark.parametrize("idx_bits", [64, 32])
def test_few_masked_repeated_and_bad_ids(fmt, idx_bits):
    """Tokens without a valid slot, masked slots, ids out of range, one expert twice in a token."""
    H, I = SIZES[fmt]
    T, E, k = 9, 6, 4
    rng = np.random.default_rng(5)
    ids = rng.integers(0, E, size=(T, k))
    ids[0] = -1
    ids[1, 1:] = -1
    ids[2] = [3, 3, 3, 3]
    ids[3] = [E, 2, -5, 2]
    ids[4] = [1 << 40 if idx_bits == 64 else 1 << 30, -(1 << 31), 5, 0]
    ids[8] = -1
    tw = rng.random((T, k)).astype(np.float32)
    sh = shape(fmt, T, H, I, E, k, seed=8)
    idt = torch.int64 if idx_bits == 64 else torch.int32
    for add in (False, True):
        inp, d, kw, okw = few_inputs(sh, ids, tw, add=add, idx_dtype=idt)
        out = run_few(make_moe(sh, topk_idx_bits=idx_bits), d, T, kw)
        ref = oracle_few(inp, okw, ids, tw)
        check_few(out, inp, ref, T, addends=[okw[n] for n in okw])
        if not add:
            assert not out[0].any() and not out[8].any()
    # nothing valid at all
    none = np.full((T, k), -1)
    inp, d, kw, okw = few_inputs(sh, none, tw, add=True, idx_dtype=idt)
    out = run_few(make_moe(sh, topk_idx_bits=idx_bits), d, T, kw)
    want = (kw["shared"].float() + kw["residual"].float()).bfloat16()
    assert torch.equal(out[:T], want)


@pytest.mark.parametrize("fmt", list(SIZES))
@pytest.mark.parametrize("fast", [True, False])
def test_few_fp32_out_and_clamp(fmt, fast):
    H, I = SIZES[fmt]
    sh = shape(fmt, 6, H, I, 5, 2, "from_logits", seed=21, x_scale=6.0, clamp=4.0)
    inp, d, kw, okw = few_inputs(sh, add=True)
    moe = make_moe(sh, out_fp32=True, fast_math=fast)
    out = run_few(moe, d, 6, kw)
    check_few(out, inp, oracle_few(inp, okw), 6, out_fp32=True, addends=[okw[n] for n in okw])


@pytest.mark.parametrize("fmt", ["fp8_block128", "bf16", "w4a8_mx"])
@pytest.mark.parametrize("T", [3, 20])
def test_few_nan_stays_in_its_token(fmt, T):
    H, I = SIZES[fmt]
    sh = shape(fmt, T, H, I, 4, 2, seed=31)
    inp, d, kw, okw = few_inputs(sh)
    moe = make_moe(sh)
    clean = run_few(moe, d, T, kw)
    x = d["x"].clone()
    if fmt == "bf16":
        x.view(torch.bfloat16)[1, 5] = float("nan")
    else:
        x.view(torch.uint8)[1, 5] = 0x7F
    d["x"] = x
    got = run_few(moe, d, T, kw)
    assert torch.isnan(got[1]).all()
    keep = [t for t in range(T) if t != 1]
    assert torch.equal(got[keep], clean[keep])


@pytest.mark.parametrize("fmt", ["nvfp4_w4a16", "nvfp4"])
def test_few_nan_stays_in_its_token_nvfp4(fmt):
    H, I = SIZES[fmt]
    sh = shape(fmt, 5, H, I, 4, 2, seed=32)
    inp, d, kw, okw = few_inputs(sh)
    moe = make_moe(sh)
    clean = run_few(moe, d, 5, kw)
    if fmt == "nvfp4":
        d["x_sf"] = d["x_sf"].clone()
        d["x_sf"].view(torch.uint8)[1, 3] = 0x7F
    else:
        d["x"] = d["x"].clone()
        d["x"].view(torch.bfloat16)[1, H - 1] = float("nan")
    got = run_few(moe, d, 5, kw)
    assert torch.isnan(got[1]).all()
    keep = [0, 2, 3, 4]
    assert torch.equal(got[keep], clean[keep])


@pytest.mark.parametrize("fmt", list(SIZES))
def test_few_masked_slots_weights_are_not_read(fmt):
    """NaN and infinite router weights of masked slots change nothing; a valid slot's NaN stays in its token."""
    H, I = SIZES[fmt]
    T, E, k = 4, 5, 3
    ids = np.array([[0, -1, 2], [-1, -1, -1], [4, 4, E], [1, 2, 3]])
    tw = np.full((T, k), 0.25, np.float32)
    sh = shape(fmt, T, H, I, E, k, seed=14)
    inp, d, kw, _ = few_inputs(sh, ids, tw)
    moe = make_moe(sh)
    clean = run_few(moe, d, T, kw)
    bad = tw.copy()
    bad[0, 1] = bad[1, 0] = np.nan
    bad[1, 2] = bad[2, 2] = np.inf
    inp, d, kw, _ = few_inputs(sh, ids, bad)
    assert torch.equal(run_few(moe, d, T, kw)[:T], clean[:T])
    bad[3, 1] = np.nan
    inp, d, kw, _ = few_inputs(sh, ids, bad)
    got = run_few(moe, d, T, kw)
    assert torch.equal(got[:3], clean[:3]) and torch.isnan(got[3]).all()


@pytest.mark.parametrize("T", [4, 12])
def test_few_routes_odd_logits_as_the_top_k_does(T):
    """Rows of NaN, of infinities, of one value, of the type's lowest value: experts and weights as moe_forward has them,
    in the launch (4 tokens) and before it (12)."""
    sh = shape("w4a8_mx", T, 416, 288, 70, 3, "from_logits", seed=15)
    inp, d, kw, _ = few_inputs(sh)
    lg = d["logits"]
    lg[0] = float("nan")
    lg[1] = torch.finfo(torch.float32).min
    lg[1, 69] = 1.0
    lg[2] = float("-inf")
    lg[2, 65] = 0.5
    lg[3, 3] = float("nan")
    lg[3, 66] = float("inf")
    moe = make_moe(sh)
    run_few(moe, d, T, kw)
    ids, tw = torch.empty_like(d["topk_idx"]), torch.empty_like(d["topk_weights"])
    moe.forward(T, d["x"], d["x_sf"], ids, tw, lg, prepared(moe, d), torch.empty((T, 416), dtype=torch.bfloat16, device="cuda"),
                moe.alloc_workspace(T))
    assert torch.equal(d["topk_idx"], ids)
    assert torch.equal(d["topk_weights"].view(torch.int32), tw.view(torch.int32))


def test_few_infinite_weight_reaches_only_its_tokens():
    sh = shape("bf16", 5, 128, 128, 4, 2, seed=3)
    ids = np.array([[0, 1], [1, 2], [2, 3], [0, 3], [3, 2]])
    tw = np.full((5, 2), 0.5, np.float32)
    inp, d, kw, okw = few_inputs(sh, ids, tw)
    moe = make_moe(sh)
    clean = run_few(moe, d, 5, kw)
    w2 = d["weights"]["w2"] if not d.get("weights_prepared") else None
    inp2, d2, _, _ = few_inputs(sh, ids, tw)
    d2["weights"]["w2"].view(torch.bfloat16)[1, 9, 4] = float("inf")
    d2["weights"]["w13"].view(torch.bfloat16)[1, 130, 4] = float("inf")
    got = run_few(moe, d2, 5, kw)
    assert w2 is None
    for t in (2, 3, 4):
        assert torch.equal(got[t], clean[t])
    for t in (0, 1):
        assert not torch.isfinite(got[t].float()).all()


@pytest.mark.parametrize("fmt", list(SIZES))
def test_few_agrees_with_forward(fmt):
    """moe_forward and moe_forward_few compute one operator: they differ by moe_forward's bf16 y (half a step per
    slot), the two outputs' roundings, and codes of h at midpoints."""
    H, I = SIZES[fmt]
    sh = shape(fmt, 12, H, I, 7, 3, seed=2)
    inp, d, kw, okw = few_inputs(sh, add=True)
    moe = make_moe(sh)
    few = run_few(moe, d, 12, kw)
    out = torch.empty((12, H), dtype=torch.bfloat16, device="cuda")
    ws = moe.alloc_workspace(12)
    moe.forward(12, d["x"], d["x_sf"], d["topk_idx"], d["topk_weights"], None, prepared(moe, d), out, ws, **kw)
    diff = bits(few[:12]) - bits(out)
    assert np.linalg.norm(diff) <= (3 * BF16_HALF + 1e-2) * np.linalg.norm(bits(out))


@pytest.mark.parametrize("fmt,T,routing", [("fp8_block128", 2, "from_logits"), ("fp8_block128", 32, "from_logits"),
                                           ("bf16", 3, "precomputed"), ("w4a8_mx", 20, "from_logits")])
def test_block_of_operators_in_a_graph(fmt, T, routing):
    """norm -> router -> few-token layer with the new residual stream added, as a decode step runs them: against the
    oracle on what the step itself produced, on a stream of its own, then captured and replayed with eager work of
    the same buffers between the replays; two graphs share the workspaces."""
    H, I = SIZES[fmt]
    E, k = 9, 2
    sh = shape(fmt, T, H, I, E, k, routing, seed=6)
    inp, d, _, _ = few_inputs(sh)
    moe = make_moe(sh)
    w = prepared(moe, d)
    g = torch.Generator().manual_seed(1)
    x0 = torch.randn(T, H, generator=g).bfloat16().cuda()
    r0 = torch.randn(T, H, generator=g).bfloat16().cuda()
    nw = (1 + 0.1 * torch.randn(H, generator=g)).bfloat16().cuda()
    rw = (torch.randn(E, H, generator=g) * H ** -0.5).bfloat16().cuda()
    ro, xn = torch.empty_like(r0), torch.empty_like(x0)
    q = sf = None
    if fmt != "bf16":
        q = torch.empty((T, H), dtype=torch.uint8, device="cuda")
        sf = (torch.empty((T, H // 128), device="cuda") if fmt == "fp8_block128" else
              torch.empty((T, H // 32), dtype=torch.uint8, device="cuda"))
    logits = torch.empty((T, E), device="cuda")
    rws, fws = moe.alloc_router_workspace(T), moe.alloc_few_workspace(T)
    out = torch.empty((T, H), dtype=torch.bfloat16, device="cuda")
    ids, tw = d["topk_idx"], d["topk_weights"]
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())

    def step():
        moe.add_rmsnorm(T, x0, r0, nw, 1e-6, residual_out=ro, x_norm=xn, x_q=q, x_sf=sf, stream=s)
        moe.router_logits(T, xn, rw, logits, rws, stream=s)
        moe.forward_few(T, xn if q is None else q, sf, ids, tw, logits if routing == "from_logits" else None, w, out,
                        fws, residual=ro, stream=s)

    with torch.cuda.stream(s):
        step()
    torch.cuda.synchronize()
    eager = out.clone()
    act = {"x": xn.view(torch.int16).cpu().numpy().view(np.uint16) if q is None else q.cpu().numpy(),
           "x_sf": None if sf is None else sf.cpu().numpy()}
    inp2 = dict(inp, **act, logits=logits.cpu().numpy())
    check_few(out, inp2, oracle_few(inp2, {"residual": bits(ro)}), T, addends=[bits(ro)])
    graphs = []
    for _ in range(2):
        gr = torch.cuda.CUDAGraph()
        with torch.cuda.graph(gr, stream=s):
            step()
        graphs.append(gr)
    torch.cuda.synchronize()
    for r in range(4):
        out.zero_()
        fws.fill_(0xFF)
        torch.cuda.synchronize()
        graphs[r % 2].replay()
        torch.cuda.synchronize()
        assert torch.equal(out, eager), f"replay {r}"
        out.zero_()
        torch.cuda.synchronize()
        with torch.cuda.stream(s):
            step()
        torch.cuda.synchronize()
        assert torch.equal(out, eager)


def test_few_out_may_be_the_residual():
    sh = shape("fp8_block128", 4, 256, 128, 4, 2, seed=12)
    inp, d, kw, _ = few_inputs(sh, add=True)
    moe = make_moe(sh)
    want = run_few(moe, d, 4, kw)[:4].clone()
    run_few(moe, d, 4, kw, out=kw["residual"])
    assert torch.equal(kw["residual"], want)


def test_few_two_streams_with_their_own_workspaces():
    sh = shape("fp8_block128", 8, 512, 512, 8, 2, seed=13)
    inp, d, kw, _ = few_inputs(sh)
    moe = make_moe(sh)
    prepared(moe, d)
    want = run_few(moe, d, 8, kw)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    outs = [torch.zeros_like(want) for _ in streams]
    wss = [moe.alloc_few_workspace(8) for _ in streams]
    torch.cuda.synchronize()
    for _ in range(5):
        for st, o, ws in zip(streams, outs, wss):
            run_few(moe, d, 8, kw, out=o, ws=ws, stream=st)
    torch.cuda.synchronize()
    for o in outs:
        assert torch.equal(o[:8], want[:8])


def test_a_workspace_for_32_tokens_serves_fewer():
    sh = shape("fp8_block128", 32, 256, 256, 6, 2, seed=16)
    inp, d, kw, _ = few_inputs(sh)
    moe = make_moe(sh)
    ws = moe.alloc_few_workspace(32)
    whole = run_few(moe, d, 32, kw, ws=ws)
    for T in (1, 2, 9, 31):
        own = run_few(moe, d, T, kw)
        assert torch.equal(run_few(moe, d, T, kw, ws=ws)[:T], own[:T])
    assert torch.equal(run_few(moe, d, 32, kw, ws=ws)[:32], whole[:32])


def test_few_weights_past_32_bits():
    """The last expert of 14 GB of weights gives the bits of the same expert on its own."""
    H, I, E, T = 4096, 14336, 40, 3
    g = torch.Generator(device="cuda").manual_seed(2)
    w13 = torch.zeros((E, 2 * I, H), dtype=torch.bfloat16, device="cuda")
    w2 = torch.zeros((E, H, I), dtype=torch.bfloat16, device="cuda")
    w13[-1].normal_(0.0, H ** -0.5, generator=g)
    w2[-1].normal_(0.0, I ** -0.5, generator=g)
    x = torch.empty((T, H), dtype=torch.bfloat16, device="cuda").normal_(generator=g)
    tw = torch.rand((T, 1), generator=g, device="cuda")
    outs = []
    for first in (0, E - 1):
        moe = MoEFFN(H, I, E - first, 1, T, fmt="bf16")
        w = moe.prepare_weights({"w13": w13[first:], "w2": w2[first:]})
        ids = torch.full((T, 1), E - 1 - first, dtype=torch.int64, device="cuda")
        out = torch.empty((T, H), dtype=torch.bfloat16, device="cuda")
        moe.forward_few(T, x, None, ids, tw, None, w, out, moe.alloc_few_workspace(T))
        torch.cuda.synchronize()
        outs.append(out)
    assert outs[0].float().abs().max() > 0 and torch.equal(*outs)
