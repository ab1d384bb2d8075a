"""Host side of moe_add_rmsnorm, moe_router_logits and moe_forward_few: refusals before
any launch (fake addresses; nothing runs), workspace sizes, the binding's checks, and
pins of their float64 definitions."""
import ctypes

import numpy as np
import pytest
import torch

import mixture_experts_ffn_topk_amd as mx
from oracle import layer as ol

INVALID, UNSUPPORTED, WS_SMALL = 1, 2, 3


def handle(**kw):
    base = dict(hidden=7168, intermediate_hidden=2048, num_experts=32, num_topk=8, max_num_tokens=256,
                activation_clamp=10.0, format=0, route_mode=0, topk_idx_bits=64, fast_math=1, tile_regime=0)
    base.update(kw)
    lib, h = mx.load_library(), ctypes.c_void_p()
    assert lib.moe_create(ctypes.byref(mx._Config(**base)), ctypes.byref(h)) == 0
    return lib, h


M = 1 << 30  # fake, 16-byte aligned addresses, far apart


def norm(lib, h, **kw):
    a = dict(T=4, x=M, xf=0, r=2 * M, rf=0, w=3 * M, wf=0, eps=1e-6, ro=4 * M, xn=5 * M, xq=6 * M, sf=7 * M, gs=1.0)
    a.update(kw)
    return lib.moe_add_rmsnorm(h, a["T"], a["x"], a["xf"], a["r"], a["rf"], a["w"], a["wf"], a["eps"], a["ro"], a["xn"],
                               a["xq"], a["sf"], a["gs"], None)


ROW = 4 * 7168 * 2  # bytes of a [4, 7168] bf16 buffer


@pytest.mark.parametrize("kw", [
    dict(T=-1), dict(T=257), dict(x=None), dict(w=None), dict(xn=None, xq=None, sf=None), dict(r=None), dict(ro=None),
    dict(xq=None), dict(sf=None), dict(xf=2), dict(rf=-1), dict(wf=7), dict(eps=-1e-6), dict(eps=float("nan")),
    dict(eps=float("inf")), dict(x=M + 8), dict(r=2 * M + 4), dict(w=3 * M + 2), dict(ro=4 * M + 8), dict(xn=5 * M + 8),
    dict(xq=6 * M + 8), dict(sf=7 * M + 2),
    # overlaps other than an input's own elements
    dict(xn=M + 16), dict(ro=2 * M + ROW - 16), dict(xq=M), dict(sf=2 * M), dict(xn=3 * M), dict(xn=4 * M),
    dict(xf=1, xn=M), dict(rf=1, xn=2 * M), dict(sf=6 * M), dict(sf=5 * M + 64)])
def test_norm_refusals(kw):
    lib, h = handle()
    assert norm(lib, h, **kw) == INVALID
    lib.moe_destroy(h)


def test_norm_refusals_by_format():
    for fmt in (1, 3):  # bf16 activations: x_norm is the activation
        lib, h = handle(format=fmt)
        assert norm(lib, h) == INVALID
        lib.moe_destroy(h)
    lib, h = handle(format=4)
    for gs in (0.0, -1.0, float("nan"), float("inf")):
        assert norm(lib, h, gs=gs) == INVALID
    lib.moe_destroy(h)
    lib, h = handle(format=1, hidden=32768 + 64, intermediate_hidden=64)
    assert norm(lib, h, xq=None, sf=None) == UNSUPPORTED
    assert lib.moe_router_logits(h, 4, M, 2 * M, 0, 3 * M, None, 0, None) == UNSUPPORTED
    assert lib.moe_router_workspace_size(h, 4) == 0
    lib.moe_destroy(h)
    lib, h = handle(format=2, hidden=32, intermediate_hidden=32, num_experts=2, num_topk=1, max_num_tokens=1 << 25)
    assert norm(lib, h, T=1 << 25) == UNSUPPORTED
    lib.moe_destroy(h)


def test_no_tokens_is_a_no_op():
    lib, h = handle()
    assert norm(lib, h, T=0, x=None, r=None, w=None, ro=None, xn=None, xq=None, sf=None) == 0
    assert lib.moe_router_logits(h, 0, None, None, 0, None, None, 0, None) == 0
    w = mx._Weights(M, 2 * M, 3 * M, 4 * M)
    assert lib.moe_forward_few(h, 0, None, None, None, None, None, None, ctypes.byref(w), None, None, None, M, 0,
                               None) == 0
    lib.moe_destroy(h)


def test_router_refusals():
    lib, h = handle()
    big = 1 << 40
    ok = dict(T=4, x=M, w=2 * M, f=0, lg=3 * M, ws=4 * M, n=big)
    for kw in (dict(T=-1), dict(T=257), dict(x=None), dict(w=None), dict(lg=None), dict(f=2), dict(x=M + 8),
               dict(w=2 * M + 4), dict(lg=3 * M + 4), dict(ws=4 * M + 128)):
        a = dict(ok, **kw)
        assert lib.moe_router_logits(h, a["T"], a["x"], a["w"], a["f"], a["lg"], a["ws"], a["n"], None) == INVALID
    assert lib.moe_router_workspace_size(h, -1) == 0 and lib.moe_router_workspace_size(h, 257) == 0
    for T in range(1, 257):
        need = lib.moe_router_workspace_size(h, T)
        assert need % 256 == 0
        if need:
            assert lib.moe_router_logits(h, T, M, 2 * M, 0, 3 * M, 4 * M, need - 1, None) == WS_SMALL
            assert lib.moe_router_logits(h, T, M, 2 * M, 0, 3 * M, None, need, None) == WS_SMALL
    lib.moe_destroy(h)


def test_a_workspace_of_the_largest_step_serves_every_smaller_one():
    for fmt, kw in ((2, {}), (0, {}), (2, dict(num_experts=40, hidden=1024)), (2, dict(num_experts=1000, num_topk=1)),
                    (2, dict(num_experts=129, hidden=2048, num_topk=1)), (2, dict(num_experts=32)),
                    (2, dict(hidden=992, intermediate_hidden=96)), (0, dict(hidden=256, intermediate_hidden=128))):
        lib, h = handle(format=fmt, max_num_tokens=40000, **kw)
        router = [lib.moe_router_workspace_size(h, T) for T in range(0, 40001, 7)]
        assert router == sorted(router)
        few_sizes = [lib.moe_few_workspace_size(h, T) for T in range(33)]
        assert few_sizes == sorted(few_sizes), few_sizes
        lib.moe_destroy(h)


def few(lib, h, **kw):
    a = dict(T=4, x=M, sf=2 * M, ids=3 * M, tw=4 * M, lg=None, b=None, sh=None, rs=None, out=5 * M, ws=6 * M, n=1 << 40,
             w=mx._Weights(7 * M, 8 * M, 9 * M, 10 * M))
    a.update(kw)
    return lib.moe_forward_few(h, a["T"], a["x"], a["sf"], a["ids"], a["tw"], a["lg"], a["b"], ctypes.byref(a["w"]),
                               a["sh"], a["rs"], a["out"], a["ws"], a["n"], None)


def test_few_refusals():
    lib, h = handle()
    for kw in (dict(T=-1), dict(T=257), dict(x=None), dict(sf=None), dict(ids=None), dict(tw=None), dict(out=None),
               dict(b=M), dict(x=M + 8), dict(sf=2 * M + 2), dict(out=5 * M + 8), dict(sh=M + 4), dict(rs=M + 8),
               dict(ws=6 * M + 16), dict(w=mx._Weights(None, M, M, M)), dict(w=mx._Weights(M, None, M, M)),
               dict(w=mx._Weights(M + 8, M, M, M)), dict(w=mx._Weights(M, M + 2, M, M))):
        assert few(lib, h, **kw) == INVALID, kw
    assert few(lib, h, T=33) == UNSUPPORTED
    assert lib.moe_few_workspace_size(h, 33) == 0 and lib.moe_few_workspace_size(h, -1) == 0
    for T in (1, 4, 32):
        need = lib.moe_few_workspace_size(h, T)
        assert need > 0
        assert few(lib, h, T=T, n=need - 1) == WS_SMALL
        assert few(lib, h, T=T, ws=None, n=need) == WS_SMALL
    lib.moe_destroy(h)
    lib, h = handle(route_mode=1)
    assert few(lib, h, lg=None) == INVALID
    lib.moe_destroy(h)
    lib, h = handle(format=4)
    assert few(lib, h) == INVALID  # no per-expert scales
    lib.moe_destroy(h)


def test_few_workspace_holds_the_intermediate():
    """[T*k, I] of the format's intermediate with its scales (FP8 may keep it in fp32)."""
    for fmt, per in ((0, 1 + 4 / 128), (1, 2), (2, 1 + 1 / 32), (3, 2), (4, 2)):
        lib, h = handle(format=fmt)
        for T in (1, 3, 16, 32):
            assert lib.moe_few_workspace_size(h, T) >= T * 8 * 2048 * per
        lib.moe_destroy(h)


def test_binding_checks_tensors():
    moe = mx.MoEFFN(256, 128, 4, 2, 8)
    x, w = torch.zeros(4, 256, dtype=torch.bfloat16), torch.zeros(256, dtype=torch.bfloat16)
    xn = torch.zeros_like(x)
    with pytest.raises(ValueError, match="GPU"):
        moe.add_rmsnorm(4, x, None, w, 1e-6, x_norm=xn)
    with pytest.raises(TypeError, match="dtype"):
        moe.add_rmsnorm(4, x.half(), None, w, 1e-6, x_norm=xn)
    with pytest.raises(ValueError, match="contiguous"):
        moe.add_rmsnorm(4, torch.zeros(256, 4, dtype=torch.bfloat16).t(), None, w, 1e-6, x_norm=xn)
    with pytest.raises(ValueError, match="bytes"):
        moe.add_rmsnorm(5, x, None, w, 1e-6, x_norm=torch.zeros(5, 256, dtype=torch.bfloat16))
    with pytest.raises(ValueError, match="residual_out is required"):
        moe.add_rmsnorm(4, x, x, w, 1e-6, x_norm=xn)
    with pytest.raises(TypeError, match="residual_out"):
        moe.add_rmsnorm(4, x, x.float(), w, 1e-6, residual_out=xn, x_norm=xn)
    with pytest.raises(ValueError, match="x_sf is required"):
        moe.add_rmsnorm(4, x, None, w, 1e-6, x_q=torch.zeros(4, 256, dtype=torch.uint8))
    with pytest.raises(TypeError, match="x_sf"):
        moe.add_rmsnorm(4, x, None, w, 1e-6, x_q=torch.zeros(4, 256, dtype=torch.uint8),
                        x_sf=torch.zeros(4, 2, dtype=torch.bfloat16))
    lg = torch.zeros(4, 4)
    with pytest.raises(TypeError, match="router_w"):
        moe.router_logits(4, x, torch.zeros(4, 256, dtype=torch.float16), lg)
    with pytest.raises(ValueError, match="router_w"):
        moe.router_logits(4, x, torch.zeros(3, 256), lg)
    with pytest.raises(ValueError, match="GPU"):
        moe.router_logits(4, x, torch.zeros(4, 256), lg)
    with pytest.raises(ValueError, match="weights"):
        moe.forward_few(2, torch.zeros(2, 256, dtype=torch.uint8), torch.zeros(2, 2), torch.zeros(2, 2, dtype=torch.int64),
                        torch.zeros(2, 2), None, {"w13": None}, xn, None)


# ------------------------------------------------------------------ the definitions
def test_norm_definition():
    x = np.array([[3.0, 4.0, 0.0, 0.0]])
    z, n = ol.add_rmsnorm(x, None, np.ones(4), 0.0)
    assert np.allclose(n, x / 2.5)  # mean square 25 / 4
    z, n = ol.add_rmsnorm(x, np.full((1, 4), 1.0), np.array([1.0, 2.0, 0.0, 1.0]), 1e-3)
    t = torch.nn.functional.rms_norm(torch.tensor(x + 1.0), (4,), torch.tensor([1.0, 2.0, 0.0, 1.0], dtype=torch.float64), 1e-3)
    assert np.allclose(n, t.numpy()) and np.array_equal(z, x + 1)


def test_activation_codes():
    n = np.zeros((1, 128))
    n[0, :4] = [448.0, -224.0, 1.0, 17.0]
    s = ol.act_scales("fp8_block128", n)
    assert s[0, 0] == 1.0 and ol.act_codes("fp8_block128", n, s)[0, :4].tolist() == [448.0, -224.0, 1.0, 16.0]
    s = ol.act_scales("w4a8_mx", 2 * n)
    assert s[0].tolist() == [2.0] + [2.0 ** -127] * 3
    assert ol.act_scales("fp8_block128", 0 * n)[0, 0] == 1.0
    s = ol.act_scales("nvfp4", n / 448.0 * 6.0, 0.5)
    assert s[0].tolist() == [2.0] + [0.0] * 7
    assert ol.act_codes("nvfp4", n / 448.0 * 6.0, s, 0.5)[0, :4].tolist() == [6.0, -3.0, 0.0, 0.0]


def test_router_workspace_refusals_where_one_is_needed():
    """Sizes whose fp32 weights split K: a workspace too small by a byte, none, and a misaligned one are refused."""
    lib, h = handle(num_experts=256, max_num_tokens=8192)
    for T in (2100, 4100, 8192):
        need = lib.moe_router_workspace_size(h, T)
        assert need > 0 and need % 256 == 0
        assert lib.moe_router_logits(h, T, M, 2 * M, 1, 3 * M, 4 * M, need - 1, None) == WS_SMALL
        assert lib.moe_router_logits(h, T, M, 2 * M, 1, 3 * M, 4 * M, 0, None) == WS_SMALL
        assert lib.moe_router_logits(h, T, M, 2 * M, 1, 3 * M, None, need, None) == WS_SMALL
        assert lib.moe_router_logits(h, T, M, 2 * M, 1, 3 * M, 4 * M + 128, need, None) == INVALID
    lib.moe_destroy(h)


def test_few_refuses_an_output_that_overlaps_an_addend():
    """bf16: anything but the addend's own buffer; fp32 elements are never an addend's."""
    for fp32 in (0, 1):
        lib, h = handle(out_fp32=fp32)
        out = 5 * M
        for name in ("sh", "rs"):
            for at in (out + 16, out - 16, out + ROW - 16) + ((out, out + 2 * ROW - 16) if fp32 else ()):
                assert few(lib, h, **{name: at}) == INVALID, (fp32, name, at - out)
        # past the end: whatever else is wrong is found (here the workspace)
        assert few(lib, h, rs=out + ROW * (1 + fp32), n=0) == WS_SMALL
        if not fp32:
            assert few(lib, h, rs=out, sh=out, n=0) == WS_SMALL
        lib.moe_destroy(h)
