"""The operators next to the routed half on the GPU where exactness, extreme values or a failure path is the point."""
import pytest
import torch

from tests import ops_ref as R
from tests.test_ops_gpu import BF16, FP16, FP32, gen

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def B():
    from quantized_moe_routed_router_b200 import build
    build.build()
    from quantized_moe_routed_router_b200 import binding
    return binding


# ----------------------------------------------------------------------------- codes are rounded quotients

def codes(v):
    """(codes, scales) of float32 v from the definition: scale = max(amax, 2^-100) / 448, code = e4m3(v / scale), each
    quotient rounded to float32."""
    M, K = v.shape
    p = torch.nn.functional.pad(v.cpu(), (0, R.blocks(K) * 128 - K)).view(M, -1, 128)
    s = p.abs().amax(-1).clamp_min(2.0 ** -100) / 448.0
    return (p / s[..., None]).view(M, -1)[:, :K].to(torch.float8_e4m3fn), s


def same_codes(q, s, v):
    """-0 and 0 are one value: compared as numbers."""
    wq, ws = codes(v)
    assert torch.equal(s.cpu(), ws)
    assert torch.equal(q.float().cpu(), wq.float()), (q.float().cpu() != wq.float()).sum()


@pytest.mark.parametrize("M,H", [(2000, 4096), (1100, 8192), (40, 16384), (300, 1001)])
def test_norm_codes_are_the_quotients(B, M, H):
    """From the kernel's own float32 rows: 16-bit inputs put some values in a thousand exactly between two codes, where an
    approximate quotient takes the wrong one."""
    r = gen(M)
    resid, gamma = (r(M, H) * torch.exp(r(M, 1))).to(BF16), (1 + 0.2 * r(H)).to(BF16)
    y, q, s = torch.empty(M, H, device="cuda"), R.rows8(M, H), torch.empty(M, R.blocks(H), device="cuda")
    B.rmsnorm(resid, gamma, 1e-5, y=y, q=q, q_scale=s)
    same_codes(q, s, y)


@pytest.mark.parametrize("M,inter", [(1500, 4096), (200, 129)])
@pytest.mark.parametrize("dtype", [BF16, FP32])
def test_act_codes_are_the_quotients(B, M, inter, dtype):
    """sigmoid(64) is 1 in float32, so v = 64 up exactly; rows from 2^-130 (below the smallest scale's amax) to 2^115."""
    size = torch.exp2(torch.linspace(-130, 115, M, device="cuda").round())[:, None]
    up = (gen(inter)(M, inter) * size).to(dtype)
    gate = torch.full_like(up, 64.0)
    q, s = R.rows8(M, inter), torch.empty(M, R.blocks(inter), device="cuda")
    B.act_quant(gate, up, 0, q, s)
    same_codes(q, s, 64.0 * up.float())
