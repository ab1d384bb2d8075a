"""GPU tests of moe_add_rmsnorm at the ends of its range: rows whose root leaves fp32, infinite weights, ties."""
import math
from fractions import Fraction

import numpy as np
import pytest
import torch

import oracle
from mixture_experts_ffn_topk_amd import MoEFFN
from oracle import layer as ol
from test_gpu_layer_ops import bits

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():  # pragma: no cover
    pytest.skip("needs a GPU", allow_module_level=True)

BLOCK = {"fp8_block128": 128, "w4a8_mx": 32, "nvfp4": 16}


def norm(fmt, x, w, eps, x_gs=1.0):
    """(x_norm, codes' values, scales' values) of rows x without a residual."""
    T, H = x.shape
    moe = MoEFFN(H, 128, 4, 2, T, fmt=fmt)
    xn = torch.empty((T, H), dtype=torch.bfloat16, device="cuda")
    q = sf = None
    if fmt in BLOCK:
        q = torch.empty((T, H // 2 if fmt == "nvfp4" else H), dtype=torch.uint8, device="cuda")
        sf = torch.empty((T, H // BLOCK[fmt]), dtype=torch.float32 if fmt == "fp8_block128" else torch.uint8, device="cuda")
    moe.add_rmsnorm(T, x.cuda(), None, w.cuda(), eps, x_norm=xn, x_q=q, x_sf=sf, x_global_scale=x_gs)
    torch.cuda.synchronize()
    if q is None:
        return bits(xn), None, None
    q, sf = q.cpu().numpy(), sf.cpu().numpy()
    if fmt == "fp8_block128":
        return bits(xn), oracle.e4m3_decode(q), sf.astype(np.float64)
    if fmt == "w4a8_mx":
        return bits(xn), oracle.e4m3_decode(q), oracle.ue8m0_decode(sf)
    return bits(xn), oracle.e2m1_decode_nibbles(oracle.e2m1_unpack(q)), oracle.e4m3_decode(sf)


def half_step(v, mantissa, emin):
    """Half the step of a format with so many mantissa bits at |v| (emin: the smallest normal exponent)."""
    return 0.5 * np.exp2(np.maximum(np.floor(np.log2(np.abs(v) + 1e-300)), emin) - mantissa)


@pytest.mark.parametrize("fmt", ["bf16", "fp8_block128", "w4a8_mx"])
def test_norm_rows_at_the_ends_of_fp32(fmt):
    """Without eps a row's norm does not depend on its magnitude: subnormal rows (their 1 / rms is no fp32 number),
    rows of the smallest number, rows whose 1 / rms is subnormal."""
    T, H = 12, 512
    g = torch.Generator().manual_seed(41)
    x = torch.randn(T, H, generator=g)
    for t, e in enumerate((-126, -130, -135, -140, -145, 100, 110, 120, 124, 125, 126)):
        x[t] = (x[t].double().clamp(-3.0, 3.0) * 2.0 ** (e - (e > 0))).float()
    x[11] = 2.0 ** -149
    w = 1 + 0.3 * torch.randn(H, generator=g)
    xn, codes, sf = norm(fmt, x, w, 0.0)
    _, n = ol.add_rmsnorm(bits(x), None, bits(w), 0.0)
    assert np.isfinite(n).all()
    # rounded to fp32 (half a step: 2^-24), then to bf16
    assert np.all(np.abs(xn - n) <= half_step(n, 7, -126) + 2.0 ** -24 * np.abs(n))
    if codes is None:
        return
    v = n / np.repeat(sf, BLOCK[fmt], axis=1)
    # FP8: the norm and the quotient are rounded to fp32 before the code (2^-24 each)
    slack = 2.0 ** -30 * half_step(v, 3, -6) if fmt == "w4a8_mx" else 2.0 ** -23 * np.abs(v)
    assert np.all(np.abs(codes - v) <= half_step(v, 3, -6) + slack)


def test_norm_mx_codes_of_large_rows_are_those_of_the_unrounded_norm():
    """Rows of 2^127, whose 1 / rms has few bits in fp32: as at 1, each code is the fp64 norm's, rounded once."""
    T, H = 4096, 352
    g = torch.Generator().manual_seed(8)
    x = torch.randint(-240, 241, (T, H), generator=g).float() * 2.0 ** 120
    w = (1 + 0.3 * torch.randn(H, generator=g)).bfloat16()
    _, codes, sf = norm("w4a8_mx", x, w, 1e-6)
    _, n = ol.add_rmsnorm(bits(x), None, bits(w), 1e-6)
    v = n / np.repeat(sf, 32, axis=1)
    assert np.all(np.abs(codes - v) <= half_step(v, 3, -6) * (1 + 2.0 ** -30))


def test_norm_infinite_weights_give_infinities():
    """inf x n is the infinity of the product's sign, NaN only against a zero; other columns keep their values."""
    T, H = 64, 512
    g = torch.Generator().manual_seed(5)
    x = torch.randn(T, H, generator=g).bfloat16()
    x[3, 7] = 0.0
    w = (1 + 0.3 * torch.randn(H, generator=g)).bfloat16()
    clean, _, _ = norm("bf16", x, w, 1e-6)
    w[7], w[300] = float("inf"), float("-inf")
    xn, _, _ = norm("bf16", x, w, 1e-6)
    want = np.sign(bits(x))
    with np.errstate(invalid="ignore"):
        assert np.array_equal(xn[:, 7], want[:, 7] * np.inf, equal_nan=True)
        assert np.array_equal(xn[:, 300], want[:, 300] * -np.inf, equal_nan=True)
    keep = [c for c in range(H) if c not in (7, 300)]
    assert np.array_equal(xn[:, keep], clean[:, keep])


@pytest.mark.parametrize("a,b", [(1, 7), (7, 17), (7, 23)])
def test_norm_mx_ties_of_subnormal_codes(a, b):
    """Norms next to the ties of E4M3's subnormal and normal codes, nearer than fp32 can tell: half of the row's columns
    are a, half b, whose rms is a whole number, and the weights put n at a tie times 1 + at most 2^-24."""
    r = math.isqrt((a * a + b * b) // 2)
    assert 2 * r * r == a * a + b * b
    H = 1024
    x = torch.tensor([a, b] * (H // 2), dtype=torch.float32).reshape(1, H)
    ties = [Fraction(2 * k + 1, 1024) for k in range(8)] + [Fraction(2 * k + 1, 16) for k in range(8, 16)]
    w = np.zeros(H)
    for block in range(H // 32):
        scale = Fraction(2) ** (block - 16)
        for i in range(32):  # the largest, of the scale's binade; then each tie twice, for columns of a and of b
            c = block * 32 + i
            want = (440 if i == 0 else ties[i // 2] * (-1) ** (i // 4)) * scale
            w[c] = np.float32(float(want * r / (a, b)[c % 2]))
    _, codes, sf = norm("w4a8_mx", x, torch.from_numpy(w).float(), 0.0)
    assert np.array_equal(sf[0], 2.0 ** np.arange(-16, 16))
    wrong = []
    for c in range(H):
        v = Fraction(float(w[c])) * (a, b)[c % 2] / r / Fraction(float(sf[0, c // 32]))
        half = Fraction(2) ** (max(math.floor(math.log2(abs(v))), -6) - 4)
        if abs(Fraction(float(codes[0, c])) - v) > half * (1 + Fraction(1, 2 ** 30)):
            wrong.append((c, float(v), codes[0, c]))
    assert not wrong


@pytest.mark.parametrize("x_gs", [0.01, 1 / 3, 0.7, 3.1, 0.001, 11 / 2688])
def test_norm_nvfp4_ties_go_to_the_even_code(x_gs):
    """n / (s x_global_scale) exactly at E2M1's ties (rows of 1, so n is the weight; a global scale of 17 bits, so
    that the tie's n is an fp32 number)."""
    gs = float((np.float32([x_gs]).view(np.uint32) & np.uint32(0xFFFFFF80)).view(np.float32)[0])
    ties = [0.25, -0.75, 1.25, -1.75, 2.5, -3.5, 5.0, -0.25, 0.75, -1.25, 1.75, -2.5, 3.5, -5.0, 0.0]
    even = [0.0, -1.0, 1.0, -2.0, 2.0, -4.0, 4.0, 0.0, 1.0, -1.0, 2.0, -2.0, 4.0, -4.0, 0.0]
    scales = [1.0, 2.0, 0.5, 416.0, 0.875, 1.125, 13.0, 0.0625]
    w = np.array([[6.0, *ties]]) * (np.array(scales) * gs)[:, None]
    assert np.array_equal(w[:, 1:], w[:, 1:].astype(np.float32))
    x = torch.ones(2, w.size)
    _, codes, sf = norm("nvfp4", x, torch.from_numpy(w.reshape(-1)).float(), 0.0, gs)
    assert np.array_equal(sf, np.tile(scales, (2, 1)))
    assert np.array_equal(codes, np.tile(np.array([6.0, *even]), (2, len(scales))))


@pytest.mark.parametrize("x_gs", [2.0 ** -149, 3 * 2.0 ** -140, 2.0 ** -126, 1.7e-38, 1.0, 1.1e38, 3.4e38])
@pytest.mark.parametrize("spread", [0.0, 1.0, 40.0, 3000.0, 1e9])
def test_norm_nvfp4_takes_every_global_scale(x_gs, spread):
    """Global scales at both ends of fp32, with norms from below the smallest code to beyond the largest; zeros are
    zeros."""
    H, top = 512, float(np.finfo(np.float32).max)
    x_gs = float(np.float32(x_gs))
    g = torch.Generator().manual_seed(3)
    w = (torch.randn(H, generator=g).double() * x_gs * spread).clamp(-top, top).float()
    w[5::7] = 0.0
    w[64:96] = 0.0
    xn, codes, sf = norm("nvfp4", torch.ones(1, H), w, 0.0, x_gs)
    n = bits(w).reshape(-1, 16)
    s6 = np.minimum(np.abs(n).max(axis=1) / (6.0 * x_gs), 448.0)
    # 6 x_global_scale, the quotient: 2^-24 each
    assert np.all(np.abs(sf[0] - s6) <= half_step(s6, 3, -6) + 2.0 ** -23 * s6)
    den = sf[0][:, None] * x_gs
    v = np.clip(np.where(den > 0, n / np.where(den > 0, den, 1.0), 0.0), -6.0, 6.0)
    codes = codes.reshape(-1, 16)
    # s x_global_scale, the quotient: 2^-24 each
    assert np.all(np.abs(codes - v) <= half_step(v, 1, 0) + 2.0 ** -23 * np.abs(v))
    assert not codes[n == 0].any()


@pytest.mark.parametrize("fmt", ["bf16", "fp8_block128", "w4a8_mx", "nvfp4"])
def test_norm_outputs_are_one_rounding_from_the_definition(fmt):
    """x_norm and the codes within half of the step at each value, and what rounding n (MX: not), the quotient and
    NVFP4's product of the scales to fp32 adds, 2^-24 of the value each (the stream is exact in fp32: small integers)."""
    T, H, x_gs = 2048, 1920, 0.0019
    g = torch.Generator().manual_seed(17)
    x = torch.randint(-240, 241, (T, H), generator=g).float() * 2.0 ** -6
    w = (1 + 0.3 * torch.randn(H, generator=g)).bfloat16()
    xn, codes, sf = norm(fmt, x, w, 1e-6, x_gs)
    _, n = ol.add_rmsnorm(bits(x), None, bits(w), float(np.float32(1e-6)))
    assert np.all(np.abs(xn - n) <= half_step(n, 7, -126) + 2.0 ** -24 * np.abs(n))
    if codes is None:
        return
    den = np.repeat(sf, BLOCK[fmt], axis=1) * (float(np.float32(x_gs)) if fmt == "nvfp4" else 1.0)
    top, mantissa, emin = (6.0, 1, 0) if fmt == "nvfp4" else (448.0, 3, -6)
    v = np.clip(n / den, -top, top)
    slack = {"fp8_block128": 2 * 2.0 ** -24, "w4a8_mx": 2.0 ** -40, "nvfp4": 3 * 2.0 ** -24}[fmt]
    assert np.all(np.abs(codes - v) <= half_step(v, mantissa, emin) + slack * np.abs(v))


def test_norm_fp8_codes_beside_an_infinity_are_zero():
    """A block with an infinite weight has an infinite scale: the codes of its finite elements are those of n / inf."""
    H = 512
    g = torch.Generator().manual_seed(6)
    x = torch.randn(8, H, generator=g)
    w = 1 + 0.3 * torch.randn(H, generator=g)
    _, clean, clean_sf = norm("fp8_block128", x, w, 1e-6)
    w[130] = float("inf")
    _, codes, sf = norm("fp8_block128", x, w, 1e-6)
    assert np.isposinf(sf[:, 1]).all()
    assert not codes[:, [c for c in range(128, 256) if c != 130]].any()
    other = [c for c in range(H) if not 128 <= c < 256]
    assert np.array_equal(codes[:, other], clean[:, other]) and np.array_equal(sf[:, [0, 2, 3]], clean_sf[:, [0, 2, 3]])
