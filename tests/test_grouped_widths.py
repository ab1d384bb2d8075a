"""The binding's products by expert take n and k from one tensor and check the others' rows against them: a tensor with more
elements than the call needs has to have rows of that many (its last dimension, or its last ones together; k of them side
by side where the rows are a token's pairs).  One dimension is a buffer of rows one behind the other."""
import pytest
import torch

import mixture_experts_ffn_topk_amd as mx

T, E, K, N, D = 6, 4, 2, 64, 96  # tokens, experts, slots, columns out and summed
RIGHT = "must be a GPU tensor"   # what CPU tensors of the right widths are refused for


def bf(*shape, dt=torch.bfloat16):
    return torch.zeros(shape, dtype=dt)


def u8(*shape):
    return bf(*shape, dt=torch.uint8)


def calls():
    moe = mx.MoEFFN(64, 96, E, K, 16, fmt="w4a8_mx")  # I = 96
    plan = {"expert_start_indices": bf(E + 1, dt=torch.int32), "src_info": bf(16 * K, dt=torch.int32)}
    R = T * K
    return {
        "gemm": (moe.grouped_gemm, dict(a=bf(R, D), w=bf(E, N, D), plan=plan, out=bf(R, N)), dict(num_tokens=T)),
        "wgrad": (moe.grouped_gemm_wgrad, dict(dout=bf(R, N), a=bf(R, D), plan=plan, dw=bf(E, N, D)), dict(num_tokens=T)),
        "mx": (moe.grouped_gemm_mxfp4, dict(a=u8(R, 48), a_sf=u8(R, 3), w=u8(E, N, 48), w_sf=u8(E, N, 3), plan=plan,
                                            out=bf(R, N)), dict(num_tokens=T)),
        "quantize": (moe.quantize_mxfp4, dict(x=bf(R, D), q=u8(R, 48), sf=u8(R, 3), values=bf(R, D)), {}),
        "swiglu": (moe.swiglu, dict(gu=bf(R, 192), plan=plan, h=bf(R, 96), q=u8(R, 48), sf=u8(R, 3)), dict(num_tokens=T)),
        "backward": (moe.swiglu_backward, dict(gu=bf(R, 192), dh=bf(R, 96), plan=plan, dgu=bf(R, 192), h=bf(R, 96)),
                     dict(num_tokens=T)),
    }


ROWS = [("gemm", "a"), ("gemm", "out"), ("wgrad", "dout"), ("wgrad", "a"), ("mx", "a"), ("mx", "a_sf"), ("mx", "w_sf"),
        ("mx", "out"), ("quantize", "q"), ("quantize", "sf"), ("quantize", "values"), ("swiglu", "gu"), ("swiglu", "h"),
        ("swiglu", "q"), ("swiglu", "sf"), ("backward", "gu"), ("backward", "dh"), ("backward", "dgu"), ("backward", "h")]


def refused(name, match, **change):
    f, tensors, rest = calls()[name]
    with pytest.raises(ValueError, match=match):
        f(**{**rest, **tensors, **change})


@pytest.mark.parametrize("name,which", ROWS)
def test_rows_of_another_width(name, which):
    t = calls()[name][1][which]
    R = T * K
    wide = bf(*t.shape[:-1], t.shape[-1] + 8, dt=t.dtype)
    refused(name, f"{which} must have rows of {t.shape[-1]}", **{which: wide})
    narrow = bf(*t.shape[:-2], t.shape[-2] * 3, max(1, t.shape[-1] // 2 + 1), dt=t.dtype)
    refused(name, f"{which} must have rows of {t.shape[-1]}", **{which: narrow})
    refused(name, RIGHT, **{which: t})
    if which == "w_sf":
        refused(name, RIGHT, w_sf=bf(E * N + 8, 3, dt=t.dtype))
        return
    for shape in ((R + 5, t.shape[-1]), (R * t.shape[-1],), (R * t.shape[-1] + 32,), (T, K, t.shape[-1]),
                  (3, 2, K, t.shape[-1]), (R // 3, 3 * t.shape[-1])):
        refused(name, RIGHT, **{which: bf(*shape, dt=t.dtype)})
    if t.shape[-1] % 2 == 0:
        refused(name, RIGHT, **{which: bf(R + 1, 2, t.shape[-1] // 2, dt=t.dtype)})
    if name != "quantize":
        refused(name, RIGHT, **{which: bf(T + 1, K * t.shape[-1], dt=t.dtype)})  # a token's rows side by side


def test_rows_by_token():
    refused("gemm", RIGHT, a=bf(T, D), a_rows="token")
    refused("gemm", f"a must have rows of {D}", a=bf(T, K * D), a_rows="token")
    refused("wgrad", f"a must have rows of {D}", a=bf(T, K * D), a_rows="token")
    refused("wgrad", f"dout must have rows of {N}", dout=bf(T, K * N), dout_rows="token")
    refused("mx", "a_sf must have rows of 3", a_sf=u8(T, 6), a_rows="token")


def test_too_small_is_said_first():
    refused("gemm", "bytes", a=bf(T * K - 1, D))


def test_k_beside_mxfp4_weights():
    refused("mx", RIGHT, k=96)
    refused("mx", "k = 96", k=97)
    refused("mx", "k = 96", k=64)


@pytest.mark.gpu
def test_layouts_of_the_same_rows():
    """Buffers with room for more rows, rows in several dimensions, flat ones: the same product."""
    moe = mx.MoEFFN(64, 96, E, K, 16, fmt="w4a8_mx")
    plan = moe.alloc_plan(T)
    ids = (torch.arange(T * K).view(T, K) % E).cuda()
    moe.plan(T, plan, topk_idx=ids, ws=moe.alloc_workspace(T))
    g = torch.Generator().manual_seed(1)
    a = torch.randint(-3, 4, (T * K, D), generator=g).to(torch.bfloat16).cuda()
    w = torch.randint(-3, 4, (E, N, D), generator=g).to(torch.bfloat16).cuda()
    want = torch.empty(T * K, N, dtype=torch.bfloat16, device="cuda")
    moe.grouped_gemm(T, a, w, plan, want, a_rows="pair", out_rows="pair")
    pad = torch.cat([a, a])
    for rows in (a.view(T, K, D), pad, pad.view(-1, 4, D // 4), pad.view(-1), pad.view(-1, K * D)):
        for shape in ((T * K + 3, N), (T + 2, K, N), (T + 1, K * N), (T * K * N + 8,)):
            out = torch.zeros(shape, dtype=torch.bfloat16, device="cuda")
            moe.grouped_gemm(T, rows, w, plan, out, a_rows="pair", out_rows="pair")
            assert torch.equal(out.view(-1)[:want.numel()], want.view(-1)) and not out.view(-1)[want.numel():].any()
    for e in range(E):
        mine = (ids.view(-1) == e).cpu()
        assert torch.equal(want.cpu()[mine].double(), a.cpu()[mine].double() @ w[e].cpu().double().T)
