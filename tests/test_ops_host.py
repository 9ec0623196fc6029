"""Refusals of the operators next to the routed half, through the C ABI, on a machine without a GPU: every check
comes before any CUDA call."""
import ctypes as C

import pytest
import torch

from quantized_moe_routed_router_b200 import build

P = 1 << 20          # an address that no check may read
BIG = (1 << 24) + 1


@pytest.fixture(scope="module")
def B():
    build.build()
    from quantized_moe_routed_router_b200 import binding
    return binding


def norm_args(B, **over):
    a = B.RmsnormArgs(rows=2, hidden=64, resid_type=0, delta_type=2, gamma_type=2, y_type=0, eps=1e-5, resid=P, ld_resid=64,
                      delta=P, ld_delta=64, gamma=P, resid_out=P, ld_resid_out=64, y=P, ld_y=64, q=P, ld_q=64, q_scale=P,
                      qs_row=1, qs_group=1)
    for k, v in over.items():
        setattr(a, k, v)
    return a


def act_args(B, **over):
    a = B.ActQuantArgs(rows=2, inter=64, act=1, in_type=0, act_alpha=1.7, act_limit=7.0, gate=P, ld_gate=64, up=P, ld_up=64,
                       q=P, ld_q=64, q_scale=P, qs_row=1, qs_group=1)
    for k, v in over.items():
        setattr(a, k, v)
    return a


def matmul_args(B, **over):
    a = B.Fp8MatmulArgs(rows=2, n=32, k=64, num_groups=4, out_type=0, reserved=0, a=P, ld_a=64, a_scale=P, as_row=1, as_block=1,
                        b=P, ld_b=64, b_group=64 * 32, b_scale=P, bs_group=1, bs_row=1, bs_block=1, offsets=P, add=P, ld_add=32,
                        out=P, ld_out=32)
    for k, v in over.items():
        setattr(a, k, v)
    return a


def balance_args(B, **over):
    a = B.BalanceArgs(rows=2, experts=8, top_k=2, score=1, dtype=2, coef=1.0, logits=P, ld_logits=8, idx=P, ld_idx=2, mask=P,
                      dloss=P, loss=P, prob=P, counts=P, offsets=P, dlogits=P, ld_dlogits=8, workspace=P, workspace_bytes=1 << 20)
    for k, v in over.items():
        setattr(a, k, v)
    return a


NAN, INF = float("nan"), float("inf")


def refused(B, fn, args, frag):
    st = fn(C.byref(args) if args is not None else None, None)
    msg = B.lib.ts_moe_last_error(None).decode()
    assert st == 1, (st, msg)
    assert frag in msg


@pytest.mark.parametrize("over,frag", [
    (dict(rows=-1), "rows"), (dict(rows=BIG), "rows"), (dict(hidden=0), "hidden"), (dict(hidden=16385), "hidden"),
    (dict(resid_type=3), "type"), (dict(delta_type=-1), "type"), (dict(gamma_type=9), "type"), (dict(y_type=7), "type"),
    (dict(eps=-1e-6), "eps"), (dict(eps=NAN), "eps"), (dict(eps=INF), "eps"), (dict(y=None, q=None, q_scale=None), "both NULL"),
    (dict(q_scale=None), "together"), (dict(q=None), "together"), (dict(delta=None), "resid_out"), (dict(resid=None), "resid"),
    (dict(ld_resid=63), "stride"), (dict(ld_delta=63), "stride"), (dict(ld_resid_out=63), "stride"), (dict(ld_y=1), "stride"),
    (dict(ld_q=0), "stride"), (dict(ld_resid_out=72), "in place"),
])
def test_rmsnorm_refusals(B, over, frag):
    refused(B, B.lib.ts_moe_rmsnorm, norm_args(B, **over), frag)


@pytest.mark.parametrize("over,frag", [
    (dict(rows=-1), "rows"), (dict(rows=BIG), "rows"), (dict(inter=0), "inter"), (dict(inter=65537), "inter"), (dict(act=2), "act"),
    (dict(in_type=3), "type"), (dict(act_alpha=NAN), "alpha"), (dict(act_limit=0.0), "limit"), (dict(act_limit=NAN), "limit"),
    (dict(gate=None), "NULL"), (dict(up=None), "NULL"), (dict(q=None), "NULL"), (dict(q_scale=None), "NULL"),
    (dict(ld_gate=63), "stride"), (dict(ld_up=63), "stride"), (dict(ld_q=63), "stride"),
])
def test_act_quant_refusals(B, over, frag):
    refused(B, B.lib.ts_moe_act_quant, act_args(B, **over), frag)


@pytest.mark.parametrize("over,frag", [
    (dict(rows=-1), "rows"), (dict(rows=BIG), "rows"), (dict(n=0), "n and k"), (dict(k=0), "n and k"), (dict(n=(1 << 20) + 1), "n and k"),
    (dict(k=(1 << 20) + 1), "n and k"), (dict(num_groups=0), "num_groups"), (dict(num_groups=257), "num_groups"),
    (dict(offsets=None), "offsets"), (dict(out_type=4), "type"), (dict(reserved=1), "reserved"), (dict(a=None), "NULL"),
    (dict(a_scale=None), "NULL"), (dict(b=None), "NULL"), (dict(b_scale=None), "NULL"), (dict(out=None), "NULL"),
    (dict(ld_a=48), "stride"), (dict(ld_b=48), "stride"), (dict(ld_out=31), "stride"), (dict(ld_add=31), "stride"),
    (dict(a=P + 8), "16-byte"), (dict(b=P + 4), "16-byte"), (dict(ld_a=72), "16-byte"), (dict(ld_b=65), "16-byte"),
    (dict(b_group=64 * 32 + 8), "16-byte"), (dict(b_group=64 * 16), "b_group"), (dict(ld_add=40), "in place"),
])
def test_fp8_matmul_refusals(B, over, frag):
    refused(B, B.lib.ts_moe_fp8_matmul, matmul_args(B, **over), frag)


@pytest.mark.parametrize("over,frag", [
    (dict(rows=-1), "rows"), (dict(rows=BIG), "rows"), (dict(experts=0), "experts"), (dict(experts=257), "experts"),
    (dict(top_k=0), "top_k"), (dict(top_k=9, experts=16, ld_logits=16), "top_k"), (dict(top_k=5, experts=4), "top_k"),
    (dict(score=3), "score"), (dict(dtype=5), "type"), (dict(coef=INF), "coef"), (dict(loss=None), "loss"), (dict(counts=None), "counts"),
    (dict(logits=None), "logits"), (dict(idx=None), "idx"), (dict(ld_logits=7), "stride"), (dict(ld_idx=1), "stride"),
    (dict(ld_dlogits=7), "stride"), (dict(workspace=None), "workspace"), (dict(workspace=P + 8), "workspace"),
    (dict(workspace_bytes=64), "too small"),
])
def test_balance_refusals(B, over, frag):
    refused(B, B.lib.ts_moe_balance, balance_args(B, **over), frag)


def test_null_args_and_no_rows(B):
    for f in ("rmsnorm", "act_quant", "fp8_matmul", "balance"):
        refused(B, getattr(B.lib, "ts_moe_" + f), None, "NULL")
    for f, a in (("rmsnorm", norm_args(B, rows=0)), ("act_quant", act_args(B, rows=0)), ("fp8_matmul", matmul_args(B, rows=0))):
        assert getattr(B.lib, "ts_moe_" + f)(C.byref(a), None) == 0


def test_balance_workspace_is_bounded(B):
    w = B.lib.ts_moe_balance_workspace
    assert w(-1, 8) == 0 and w(4, 0) == 0 and w(4, 257) == 0
    assert 0 < w(0, 1) <= w(1 << 24, 256) < 1 << 20


def test_binding_checks_tensors(B):
    z = torch.zeros(4, 64)
    q, s = torch.zeros(4, 64, dtype=torch.uint8), torch.zeros(4, 1)
    with pytest.raises(B.TsMoeError, match="CUDA device"):
        B.rmsnorm(z, None, 1e-5, y=z.clone())
    with pytest.raises(B.TsMoeError, match="shape"):
        B.rmsnorm(z, None, 1e-5, y=torch.zeros(4, 65))
    with pytest.raises(B.TsMoeError, match="bfloat16"):
        B.rmsnorm(z.double(), None, 1e-5, y=z)
    with pytest.raises(B.TsMoeError, match="contiguous"):
        B.rmsnorm(torch.zeros(64, 4).t(), None, 1e-5, y=z)
    with pytest.raises(B.TsMoeError, match="float8"):
        B.rmsnorm(z, None, 1e-5, q=z, q_scale=s)
    with pytest.raises(B.TsMoeError, match="q_scale"):
        B.act_quant(z, z, 0, q, torch.zeros(4, 2))
    with pytest.raises(B.TsMoeError, match="one type"):
        B.act_quant(z, z.half(), 0, q, s)
    with pytest.raises(B.TsMoeError, match="b_scale"):
        B.fp8_matmul(q, s, q, torch.zeros(2, 1), torch.zeros(4, 4))
    with pytest.raises(B.TsMoeError, match="add"):
        B.fp8_matmul(q, s, q, torch.zeros(1, 1), torch.zeros(4, 4), add=torch.zeros(4, 4).half())
    with pytest.raises(B.TsMoeError, match="int32"):
        B.balance(torch.zeros(4, 8), torch.zeros(4, 2, dtype=torch.int64), 1, torch.zeros(1), torch.zeros(8, dtype=torch.int32))
    with pytest.raises(B.TsMoeError, match="counts"):
        B.balance(torch.zeros(4, 8), torch.zeros(4, 2, dtype=torch.int32), 1, torch.zeros(1), torch.zeros(9, dtype=torch.int32))
    with pytest.raises(B.TsMoeError, match="CUDA device"):
        B.balance(torch.zeros(4, 8), torch.zeros(4, 2, dtype=torch.int32), 1, torch.zeros(1), torch.zeros(8, dtype=torch.int32))
