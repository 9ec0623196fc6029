"""Further host logic and refusals of the operators next to the routed half, on a machine without a GPU."""
import ctypes as C
import math
import random

import pytest
import torch

from tests.test_ops_host import P, B, act_args, balance_args, matmul_args, norm_args, refused  # noqa: F401  (B is a fixture)


@pytest.mark.parametrize("cta,wait_us,frag", [(-1, 1, "cta"), (0, 2_000_001, "wait_us")])
def test_held_product_refusals(B, cta, wait_us, frag):  # noqa: F811
    st = B.lib.ts_moe_debug_fp8_matmul_held(C.byref(matmul_args(B)), cta, wait_us, None)
    assert st == 1 and frag in B.lib.ts_moe_last_error(None).decode()


def test_a_split_product_has_a_cluster_for_every_item(B):  # noqa: F811
    """The cluster's join takes one item: wherever K is split, the grid has as many clusters as there can be items (row
    tiles of all groups at their most, times column tiles), and its CTAs fit two an SM."""
    rng = random.Random(7)
    seen = set()
    for _ in range(20000):
        size = lambda low, high: int(math.exp(rng.uniform(math.log(low), math.log(high + 1))))  # noqa: E731
        G = rng.choice((0, 0, 1, 2, 8, 32, 100, 256))
        M, N, K, sms = size(1, 8192), size(1, 20000), size(1, 20000), rng.choice((148, 148, 132, 16))
        a = matmul_args(B, rows=M, n=N, k=K, num_groups=max(G, 1), ld_out=N, out_type=rng.choice((0, 2)))
        if not G:
            a.offsets = None
        if rng.random() < 0.7:
            a.add = None
        plan = (C.c_int32 * 4)()
        B.lib.ts_moe_debug_fp8_matmul_plan(C.byref(a), sms, plan)
        kind, bt, splits, grid = plan
        seen.add((kind, splits))
        assert splits >= 1 and grid >= 1
        if kind != 1:
            assert splits == 1
            continue
        # groups of sizes that leave the most row tiles: one row each, and the rest in one
        reached = min(max(G, 1), M)
        items = (reached - 1 + -(-(M - reached + 1) // bt)) * -(-N // 128)
        assert splits <= min(4, -(-K // 128)) and grid * splits <= 2 * sms
        assert splits == 1 or grid >= items, (M, N, K, G, sms, list(plan))
    assert {(0, 1), (1, 1), (1, 2), (1, 4), (2, 1)} <= seen
    B.lib.ts_moe_debug_fp8_matmul_plan(C.byref(matmul_args(B, rows=0)), 148, plan)
    assert plan[3] == 0


def test_binding_refuses_tensors_of_other_dimensions(B):  # noqa: F811
    """As TsMoeError, like every other refusal."""
    z, q, s = torch.zeros(4, 64), torch.zeros(4, 64, dtype=torch.uint8), torch.zeros(4, 1)
    line, cube = torch.zeros(64), torch.zeros(2, 4, 64)
    i32 = torch.int32
    for call in (lambda: B.rmsnorm(line, None, 1e-5, y=line), lambda: B.rmsnorm(cube, None, 1e-5, y=cube),
                 lambda: B.rmsnorm(z, None, 1e-5, y=cube), lambda: B.act_quant(line, line, 0, q, s), lambda: B.act_quant(cube, cube, 0, q, s),
                 lambda: B.fp8_matmul(q[0], s, q, s, z), lambda: B.fp8_matmul(q, s, q, s, line), lambda: B.fp8_matmul(q, s, q[None], s, z),
                 lambda: B.fp8_matmul(q, s, q[:0][None][:0], torch.zeros(0, 1, 1), z, offsets=torch.zeros(1, dtype=i32)),
                 lambda: B.balance(line, torch.zeros(64, 2, dtype=i32), 1, torch.zeros(1), torch.zeros(8, dtype=i32)),
                 lambda: B.balance(z, torch.zeros(4, dtype=i32), 1, torch.zeros(1), torch.zeros(64, dtype=i32)),
                 lambda: B.balance(z, torch.zeros((), dtype=i32), 1, torch.zeros(1), torch.zeros(64, dtype=i32))):
        with pytest.raises(B.TsMoeError):
            call()


@pytest.mark.parametrize("op,over", [
    ("rmsnorm", dict(resid=P + 1, resid_out=P + 1)), ("rmsnorm", dict(resid_type=2, resid=P + 2, resid_out=P + 4)), ("rmsnorm", dict(delta=P + 2)),
    ("rmsnorm", dict(gamma=P + 6)), ("rmsnorm", dict(y=P + 3)), ("rmsnorm", dict(resid_out=P + 1)), ("rmsnorm", dict(q_scale=P + 2)),
    ("act_quant", dict(gate=P + 1)), ("act_quant", dict(in_type=2, up=P + 2)), ("act_quant", dict(q_scale=P + 1)),
    ("fp8_matmul", dict(out=P + 1)), ("fp8_matmul", dict(out_type=2, out=P + 2)), ("fp8_matmul", dict(add=P + 1)),
    ("fp8_matmul", dict(a_scale=P + 2)), ("fp8_matmul", dict(b_scale=P + 1)), ("fp8_matmul", dict(offsets=P + 2)),
    ("balance", dict(logits=P + 2)), ("balance", dict(dtype=0, dlogits=P + 1)), ("balance", dict(idx=P + 2)), ("balance", dict(dloss=P + 2)),
    ("balance", dict(loss=P + 1)), ("balance", dict(prob=P + 2)), ("balance", dict(counts=P + 2)), ("balance", dict(offsets=P + 1)),
])
def test_pointers_off_their_elements_are_refused(B, op, over):  # noqa: F811
    """A load there would fault the GPU."""
    args = dict(rmsnorm=norm_args, act_quant=act_args, fp8_matmul=matmul_args, balance=balance_args)[op](B, **over)
    refused(B, getattr(B.lib, "ts_moe_" + op), args, "aligned to its elements")


@pytest.mark.parametrize("rows,cols,qs_row,qs_group", [(2, 300, 0, 1), (2, 300, 3, 0), (1, 129, 5, 0), (5, 100, 0, 1), (4, 300, 1, 1),
                                                       (4, 300, 1, 3), (4, 300, 4, 2), (3, 300, -2, 1), (2, 200, 0, 0)])
def test_scales_that_would_overlap_are_refused(B, rows, cols, qs_row, qs_group):  # noqa: F811
    places = [r * qs_row + g * qs_group for r in range(rows) for g in range(-(-cols // 128))]
    assert len(set(places)) < len(places)
    wide = dict(rows=rows, qs_row=qs_row, qs_group=qs_group, ld_q=cols)
    refused(B, B.lib.ts_moe_rmsnorm, norm_args(B, hidden=cols, ld_resid=cols, ld_delta=cols, ld_resid_out=cols, ld_y=cols, **wide), "q_scale overlap")
    refused(B, B.lib.ts_moe_act_quant, act_args(B, inter=cols, ld_gate=cols, ld_up=cols, **wide), "q_scale overlap")


# the kernels' times for these groups lie 8 to 190 % apart: stream where K can be shared or tiles would mostly be empty
@pytest.mark.parametrize("G,M,N,K,kind", [
    (32, 64, 5760, 2880, 1), (32, 640, 5760, 2880, 1), (64, 1280, 2816, 2048, 1), (8, 200, 512, 4096, 1), (2, 100, 512, 4096, 1),
    (4, 256, 1024, 2048, 1), (8, 1024, 1408, 2048, 2), (32, 2048, 5760, 2880, 2), (64, 24576, 2816, 2048, 2), (4, 400, 14336, 4096, 2)])
def test_grouped_products_take_the_faster_kernel(B, G, M, N, K, kind):  # noqa: F811
    a = matmul_args(B, rows=M, n=N, k=K, num_groups=G, ld_out=N, add=None)
    plan = (C.c_int32 * 4)()
    B.lib.ts_moe_debug_fp8_matmul_plan(C.byref(a), 148, plan)
    assert plan[0] == kind, list(plan)
