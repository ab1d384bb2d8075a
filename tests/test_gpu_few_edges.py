"""GPU tests of moe_forward_few where its down kernel takes the most LDS."""
import pytest
import torch

from gpu_util import make_moe
from test_gpu_layer_ops import check_few, few_inputs, oracle_few, run_few, shape

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():  # pragma: no cover
    pytest.skip("needs a GPU", allow_module_level=True)


@pytest.mark.parametrize("fmt,H,I,E,k,T", [
    ("fp8_block128", 4224, 128, 200, 10, 32),  # h in LDS, sums of four tiles for 32 tokens, tables of 200 experts
    ("fp8_block128", 384, 1024, 16, 1, 32),    # h in LDS with two units for some experts
    ("nvfp4", 2880, 64, 300, 8, 32)])
def test_few_largest_lds(fmt, H, I, E, k, T):
    sh = shape(fmt, T, H, I, E, k, seed=H + E)
    print(f"[few] {sh}", flush=True)
    inp, d, kw, okw = few_inputs(sh, add=True)
    moe = make_moe(sh)
    out = run_few(moe, d, T, kw)
    torch.cuda.synchronize()
    check_few(out, inp, oracle_few(inp, okw), T, addends=[okw[n] for n in okw])
    assert torch.equal(run_few(moe, d, T, kw)[:T], out[:T])
