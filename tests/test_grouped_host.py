"""Host side of the products by expert, the MXFP4 quantisation and SwiGLU: refusals before any launch (fake addresses;
nothing runs), their limits, and the binding's checks."""
import ctypes

import pytest
import torch

import mixture_experts_ffn_topk_amd as mx

OK, INVALID, UNSUPPORTED = 0, 1, 2
PLAN, TOKEN, PAIR = 0, 1, 2
M = 1 << 36  # fake, 16-byte aligned addresses, far apart


def handle(**kw):
    base = dict(hidden=256, intermediate_hidden=128, num_experts=4, num_topk=2, max_num_tokens=64,
                activation_clamp=10.0, format=0, route_mode=0, topk_idx_bits=64, fast_math=1, tile_regime=0)
    base.update(kw)
    lib, h = mx.load_library(), ctypes.c_void_p()
    assert lib.moe_create(ctypes.byref(mx._Config(**base)), ctypes.byref(h)) == 0
    return lib, h


def plan(**kw):
    return ctypes.byref(mx._Plan(None, kw.get("start", 20 * M), None, None, kw.get("src", 21 * M)))


BASE = dict(T=8, n=256, k=128, a=M, ar=PLAN, w=2 * M, kn=0, plan={}, out=3 * M, f32=0, orr=PLAN)


def gemm(kw, **cfg):
    lib, h = handle(**cfg)
    a = {**BASE, **kw}
    r = lib.moe_grouped_gemm(h, a["T"], a["n"], a["k"], a["a"], a["ar"], a["w"], a["kn"],
                             None if a["plan"] is None else plan(**a["plan"]), a["out"], a["f32"], a["orr"], None)
    lib.moe_destroy(h)
    return r


def gemm_mx(kw, **cfg):
    lib, h = handle(**cfg)
    a = {**BASE, "asf": 4 * M, "wsf": 5 * M, **kw}
    r = lib.moe_grouped_gemm_mxfp4(h, a["T"], a["n"], a["k"], a["a"], a["asf"], a["ar"], a["w"], a["wsf"],
                                   None if a["plan"] is None else plan(**a["plan"]), a["out"], a["f32"], a["orr"], None)
    lib.moe_destroy(h)
    return r


def wgrad(kw, **cfg):
    lib, h = handle(**cfg)
    a = dict(T=8, n=256, k=128, d=M, dr=PLAN, a=2 * M, ar=PLAN, plan={}, dw=3 * M, f32=0, acc=0)
    a.update(kw)
    r = lib.moe_grouped_gemm_wgrad(h, a["T"], a["n"], a["k"], a["d"], a["dr"], a["a"], a["ar"],
                                   None if a["plan"] is None else plan(**a["plan"]), a["dw"], a["f32"], a["acc"], None)
    lib.moe_destroy(h)
    return r


PRODUCT = [
    dict(T=-1), dict(T=65), dict(n=0), dict(k=0), dict(n=-8), dict(n=12), dict(k=100), dict(a=None), dict(w=None),
    dict(out=None), dict(plan=None), dict(plan=dict(start=None)), dict(plan=dict(src=None)), dict(ar=3), dict(ar=-1),
    dict(orr=3), dict(f32=2), dict(f32=-1), dict(a=M + 8), dict(w=2 * M + 8), dict(out=3 * M + 8),
    # overlaps: of a row's end, of the weights' last expert
    dict(out=M), dict(out=2 * M), dict(a=3 * M + 16 * 256 * 2 - 16)]
SIDE = 1 << 20


@pytest.mark.parametrize("kw", PRODUCT + [dict(kn=2), dict(out=M + 16 * 128 * 2 - 16),
                                          dict(out=2 * M + 4 * 256 * 128 * 2 - 16),
                                          dict(out=M + 8 * 128 * 2 - 16, ar=TOKEN),
                                          dict(w=3 * M + 16 * 256 * 4 - 16, f32=1),
                                          # the plan's own arrays
                                          dict(out=20 * M), dict(out=21 * M + 48)])
def test_gemm_refusals(kw):
    assert gemm(kw) == INVALID


@pytest.mark.parametrize("kw", PRODUCT + [dict(k=48), dict(asf=None), dict(wsf=None), dict(asf=4 * M + 2),
                                          dict(wsf=5 * M + 1), dict(out=4 * M), dict(out=5 * M),
                                          dict(out=M + 16 * 128 // 2 - 16), dict(asf=3 * M), dict(out=20 * M)])
def test_gemm_mxfp4_refusals(kw):
    assert gemm_mx(kw) == INVALID


@pytest.mark.parametrize("kw", [
    dict(T=-1), dict(T=65), dict(n=0), dict(k=-8), dict(n=12), dict(k=100), dict(d=None), dict(a=None), dict(dw=None),
    dict(dw=None, T=0), dict(plan=None), dict(plan=dict(start=None)), dict(plan=dict(src=None)), dict(dr=3),
    dict(ar=-1), dict(f32=2), dict(acc=2, f32=1), dict(d=M + 8), dict(a=2 * M + 8), dict(dw=3 * M + 8), dict(dw=M),
    dict(dw=2 * M), dict(dw=M + 16 * 256 * 2 - 16), dict(a=3 * M + 4 * 256 * 128 * 2 - 16), dict(dw=20 * M),
    dict(dw=21 * M + 48)])
def test_wgrad_refusals(kw):
    assert wgrad(kw) == INVALID


@pytest.mark.parametrize("kw", [dict(orr=TOKEN), dict(n=SIDE + 8), dict(k=SIDE + 32)])
def test_product_limits(kw):
    assert gemm(kw) == UNSUPPORTED
    assert gemm_mx(kw) == UNSUPPORTED


def test_limits():
    assert wgrad(dict(acc=1)) == UNSUPPORTED  # bf16 sums do not add up
    assert wgrad(dict(n=SIDE + 8)) == UNSUPPORTED and wgrad(dict(k=SIDE + 8)) == UNSUPPORTED
    many = dict(max_num_tokens=1 << 24, num_topk=2, hidden=32, intermediate_hidden=32, format=2)
    far = dict(a=1 << 45, w=2 << 45, out=3 << 45)
    big = dict(T=1 << 21, n=8, k=1024, **far)  # 2^21 tokens' rows of 2 KB: 4 GiB
    assert gemm(dict(big, ar=TOKEN), **many) == UNSUPPORTED
    assert gemm(dict(big, T=1 << 20, ar=PAIR), **many) == UNSUPPORTED
    assert gemm(dict(big, n=1024, k=8, T=1 << 20, orr=PAIR), **many) == UNSUPPORTED
    assert gemm_mx(dict(big, T=1 << 23, ar=TOKEN), **many) == UNSUPPORTED  # of 512 bytes
    assert wgrad(dict(T=1 << 21, n=8, k=1024, d=1 << 45, a=2 << 45, dw=3 << 45, ar=TOKEN), **many) == UNSUPPORTED
    # tiles
    assert wgrad(dict(n=SIDE, k=SIDE, d=1 << 45, a=2 << 45, dw=3 << 52), num_experts=256) == UNSUPPORTED


def test_no_tokens():
    """Nothing runs: rows may be missing."""
    none = dict(T=0, a=None, w=None, out=None)
    assert gemm(none) == OK
    assert gemm_mx(dict(none, asf=None, wsf=None)) == OK


def quant(kw):
    lib, h = handle()
    a = dict(h=h, rows=4, cols=128, x=M, f32=0, stride=128, q=2 * M, sf=3 * M, v=4 * M)
    a.update(kw)
    r = lib.moe_quantize_mxfp4(a["h"], a["rows"], a["cols"], a["x"], a["f32"], a["stride"], a["q"], a["sf"], a["v"], None)
    lib.moe_destroy(h)
    return r


@pytest.mark.parametrize("kw", [
    dict(h=None), dict(rows=-1), dict(cols=0), dict(cols=48), dict(cols=-32), dict(f32=2), dict(stride=120),
    dict(stride=132), dict(stride=130, f32=1), dict(stride=-128), dict(x=None), dict(q=None), dict(sf=None),
    dict(x=M + 8), dict(q=2 * M + 8), dict(sf=3 * M + 2), dict(v=4 * M + 8), dict(rows=1 << 41), dict(stride=1 << 41),
    dict(rows=1 << 40, stride=1 << 40), dict(q=M), dict(sf=M + 1020), dict(q=3 * M), dict(v=2 * M), dict(v=3 * M),
    # values in place: of the same elements alone
    dict(v=M + 16), dict(v=M, f32=1), dict(v=M, stride=136)])
def test_quantize_refusals(kw):
    assert quant(kw) == INVALID


def test_quantize_no_rows():
    assert quant(dict(rows=0, x=None, q=None, sf=None, v=None)) == OK


def swiglu(kw, back):
    lib, h = handle()
    a = dict(T=8, gu=M, dh=2 * M, plan={}, dgu=3 * M, h=4 * M, q=5 * M, sf=6 * M)
    a.update(kw)
    p = None if a["plan"] is None else plan(**a["plan"])
    if back:
        r = lib.moe_swiglu_backward(h, a["T"], a["gu"], a["dh"], p, a["dgu"], a["h"], None)
    else:
        r = lib.moe_swiglu(h, a["T"], a["gu"], p, a["h"], a["q"], a["sf"], None)
    lib.moe_destroy(h)
    return r


ROWS = 16 * 128 * 2  # bytes of h


@pytest.mark.parametrize("kw", [
    dict(T=-1), dict(T=65), dict(gu=None), dict(plan=None), dict(plan=dict(start=None)), dict(h=None, q=None, sf=None),
    dict(q=None), dict(sf=None), dict(gu=M + 8), dict(h=4 * M + 8), dict(q=5 * M + 8), dict(sf=6 * M + 2), dict(h=M),
    dict(q=M), dict(sf=M + 4), dict(h=5 * M), dict(h=6 * M), dict(q=6 * M), dict(h=M + 2 * ROWS - 16), dict(h=20 * M),
    dict(q=20 * M), dict(sf=20 * M)])
def test_swiglu_refusals(kw):
    assert swiglu(kw, False) == INVALID


@pytest.mark.parametrize("kw", [
    dict(T=-1), dict(T=65), dict(gu=None), dict(dh=None), dict(dgu=None), dict(plan=None), dict(plan=dict(start=None)),
    dict(gu=M + 8), dict(dh=2 * M + 8), dict(dgu=3 * M + 8), dict(h=4 * M + 8), dict(dgu=M + 16), dict(dgu=2 * M),
    dict(h=M), dict(h=2 * M + 16), dict(h=3 * M), dict(dgu=2 * M + ROWS - 16), dict(dgu=20 * M), dict(h=20 * M)])
def test_swiglu_backward_refusals(kw):
    assert swiglu(kw, True) == INVALID


def test_swiglu_no_tokens():
    assert swiglu(dict(T=0, gu=None, dh=None, dgu=None, h=None, q=None, sf=None), True) == OK
    assert swiglu(dict(T=0, gu=None, h=None, q=None, sf=None), False) == OK


def test_the_binding_names_what_is_wrong():
    moe = mx.MoEFFN(256, 128, 4, 2, 64)
    p = {"expert_start_indices": 20 * M, "src_info": 21 * M}
    with pytest.raises(ValueError, match="a_rows"):
        moe.grouped_gemm(8, M, 2 * M, p, 3 * M, a_rows="rows", n=256, k=128)
    with pytest.raises(ValueError, match="n and k"):
        moe.grouped_gemm(8, M, 2 * M, p, 3 * M)
    with pytest.raises(ValueError, match="w must be"):
        moe.grouped_gemm(8, M, torch.zeros(3, 256, 128, dtype=torch.bfloat16), p, 3 * M)
    with pytest.raises(ValueError, match="out is required"):
        moe.grouped_gemm(8, M, 2 * M, p, None, n=256, k=128)
    with pytest.raises(ValueError, match="src_info"):
        moe.grouped_gemm(8, M, 2 * M, {"expert_start_indices": 20 * M}, 3 * M, n=256, k=128)
    with pytest.raises(ValueError, match="rows and cols"):
        moe.quantize_mxfp4(M, 2 * M, 3 * M)
