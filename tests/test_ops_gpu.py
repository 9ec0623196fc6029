"""The operators next to the routed half on the GPU, against their formulas in 64 bits (tests/ops_ref.py)."""
import math
import os
import subprocess
import sys

import pytest
import torch

from quantized_moe_routed_router_b200 import synth
from tests import ops_ref as R

pytestmark = pytest.mark.gpu

BF16, FP16, FP32 = torch.bfloat16, torch.float16, torch.float32


@pytest.fixture(scope="module")
def B():
    from quantized_moe_routed_router_b200 import build
    build.build()
    from quantized_moe_routed_router_b200 import binding
    return binding


def gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return lambda *s: torch.randn(*s, generator=g, device="cuda")


def wide(t, pad, shift=0):
    """t's values in rows `pad` elements longer, starting `shift` elements in."""
    M, K = t.shape
    w = torch.zeros(M, K + pad + shift, dtype=t.dtype, device=t.device)[:, shift:shift + K]
    w.copy_(t)
    return w


# ----------------------------------------------------------------------------- norm

# v is rounded in: the additions of a row's squares (at most 32 in a thread, 5 + 32 across threads; all positive, so the
# relative error adds up, and halves under the root), the division, the root, the reciprocal, and two products
NORM_REL = (69 / 2 + 8) * 2 * R.F32


@pytest.mark.parametrize("M", [1, 5, 1500])
@pytest.mark.parametrize("H,rt,dt,gt,yt,q", [
    (2880, BF16, FP32, FP32, BF16, True), (64, BF16, BF16, BF16, None, True), (4096, FP16, None, None, FP16, False),
    (1, BF16, BF16, None, FP32, True), (127, FP32, FP16, BF16, FP32, True), (129, BF16, None, FP16, BF16, True),
    (2047, BF16, FP32, BF16, None, True), (16384, BF16, BF16, BF16, BF16, True), (16383, FP32, FP32, FP32, FP32, True),
    (8200, BF16, BF16, FP32, BF16, True),
])
def test_rmsnorm(B, M, H, rt, dt, gt, yt, q):
    if M > 5 and H > 9000:
        M = 1100      # past the launch rule's bound, and no more than the 64-bit check needs
    r = gen(H + M)
    resid = (r(M, H) * torch.exp(r(M, 1))).to(rt)
    delta = r(M, H).to(dt) if dt else None
    gamma = (1 + 0.2 * r(H)).to(gt) if gt else None
    out = torch.empty_like(resid) if dt else None
    y = torch.empty(M, H, dtype=yt, device="cuda") if yt else None
    q8, qs = (R.rows8(M, H), torch.empty(M, R.blocks(H), device="cuda")) if q else (None, None)
    B.rmsnorm(resid, gamma, 1e-5, delta=delta, resid_out=out, y=y, q=q8, q_scale=qs)
    want_r, v = R.rmsnorm(resid, gamma, 1e-5, delta)
    if dt:
        assert torch.equal(out.cpu(), want_r)
    if yt:
        assert ((R.d64(y) - v).abs() <= R.rounding(v, yt) + v.abs() * NORM_REL).all()
    if q:
        R.check_rows8(q8, qs, v, NORM_REL)


@pytest.mark.parametrize("H", [256, 250])
def test_rmsnorm_strides_and_in_place(B, H):
    """Rows inside larger buffers, scales with the rows innermost, the residual in place; what lies around stays."""
    r = gen(3)
    M = 7
    resid, delta = r(M, H).to(BF16), r(M, H)
    want_r, v = R.rmsnorm(resid, None, 1e-6, delta)
    buf = torch.full((M + 2, H + 24), 9.0, dtype=BF16, device="cuda")
    buf[1:-1, 8:8 + H] = resid
    at = buf[1:-1, 8:8 + H]
    ybuf = torch.full((M, H + 3), 5.0, device="cuda")
    qbuf = torch.full((M + 1, 512), 77, dtype=torch.uint8, device="cuda")
    qs = torch.full((R.blocks(H), M + 5), -1.0, device="cuda")
    B.rmsnorm(at, None, 1e-6, delta=wide(delta, 5, 1), resid_out=at, y=ybuf[:, 1:1 + H], q=qbuf[:M, 8:8 + H], q_scale=qs[:, :M].t())
    assert torch.equal(at.cpu(), want_r)
    assert ((R.d64(ybuf[:, 1:1 + H]) - v).abs() <= R.rounding(v, FP32) + v.abs() * NORM_REL).all()
    R.check_rows8(qbuf[:M, 8:8 + H].view(torch.float8_e4m3fn), qs[:, :M].t(), v, NORM_REL)
    assert (buf[0] == 9).all() and (buf[-1] == 9).all() and (buf[:, :8] == 9).all() and (buf[:, 8 + H:] == 9).all()
    assert (ybuf[:, 0] == 5).all() and (ybuf[:, 1 + H:] == 5).all()
    assert (qbuf[M] == 77).all() and (qbuf[:, :8] == 77).all() and (qbuf[:, 8 + H:] == 77).all() and (qs[:, M:] == -1).all()


def test_rmsnorm_zero_and_non_finite_rows(B):
    M, H = 5, 300
    x = gen(4)(M, H)
    x[0] = 0
    x[1, 130:] = 0          # a group of zeros beside others
    x[2, 7] = float("nan")
    x[3, 290] = float("inf")
    y, q, s = torch.empty(M, H, device="cuda"), R.rows8(M, H), torch.empty(M, 3, device="cuda")
    B.rmsnorm(x, None, 1e-5, y=y, q=q, q_scale=s)
    _, v = R.rmsnorm(x, None, 1e-5, None)
    for m in (0, 1, 4):
        assert ((R.d64(y[m:m + 1]) - v[m]).abs() <= v[m].abs() * (NORM_REL + R.F32)).all()
        R.check_rows8(q[m:m + 1], s[m:m + 1], v[m:m + 1], NORM_REL)
    assert (s[0] == 2.0 ** -100 / 448).all() and (q[0].float() == 0).all()
    assert y[2].isnan().all() and s[2].isnan().all() and q[2].float().isnan().all()
    # an infinite mean: the infinity over it is NaN, every other value over it is 0
    assert y[3, 290].isnan() and (y[3, :290] == 0).all() and s[3, 2].isnan() and s[3, 0] == 2.0 ** -100 / 448


# ----------------------------------------------------------------------------- activation

# the sigmoid's exponential (2 ulp), sum and reciprocal (2 ulp); alpha g is rounded once, which the exponential turns
# into |alpha g| half steps: at most 90 of them before the value itself is below any scale's reach; three products
ACT_REL = (2 + 1 + 2 + 4) * 2 * R.F32 + 90 * R.F32


@pytest.mark.parametrize("M", [1, 3, 700])
@pytest.mark.parametrize("inter,kind,dtype", [(2880, 1, BF16), (128, 0, FP16), (1, 0, FP32), (1408, 0, BF16), (1001, 1, FP32),
                                              (14336, 0, BF16), (17, 1, FP16)])
def test_act_quant(B, M, inter, kind, dtype):
    both = (4 * gen(inter + M)(M, 2 * inter)).to(dtype)
    gate, up = both[:, :inter], both[:, inter:]
    q, s = R.rows8(M, inter), torch.empty(M, R.blocks(inter), device="cuda")
    B.act_quant(gate, up, kind, q, s)
    R.check_rows8(q, s, R.act(gate, up, kind), ACT_REL)


def test_act_quant_non_finite_and_strides(B):
    M, inter = 4, 200
    r = gen(8)
    g, u = r(M, inter), r(M, inter)
    g[0, 3], u[1, 150], g[2, 5], u[2, 6] = float("nan"), float("nan"), float("inf"), -float("inf")
    q, s = R.rows8(M, 512)[:, 64:64 + inter], torch.full((2, 9), -1.0, device="cuda")
    B.act_quant(wide(g, 3), wide(u, 1), 1, q, s[:, :M].t(), act_alpha=1.5, act_limit=2.0)
    v = R.act(g, u, 1, 1.5, 2.0)
    got = s[:, :M].t()
    assert got[0, 0].isnan() and got[1, 1].isnan()
    for m, c in ((0, 1), (1, 0), (2, 0), (2, 1), (3, 0), (3, 1)):     # the clamp makes the infinities finite
        cols = slice(c * 128, min(inter, c * 128 + 128))
        R.check_rows8(q[m:m + 1, cols], got[m:m + 1, c:c + 1], v[m:m + 1, cols], ACT_REL)
    assert (s[:, M:] == -1).all()
    B.act_quant(g, u, 0, q, s[:, :M].t())
    assert s[0, 2].isinf() and q[2, 5].float().isnan()      # silu(inf) * u: the group's scale is infinite


# ----------------------------------------------------------------------------- product

def check_matmul(B, M, N, K, out_type, add=None, seed=0, a=None, b=None, out=None):
    r = gen(seed + M * 7 + N * 3 + K)
    a, sa = a or R.encode_rows(r(M, K) * torch.exp(0.5 * r(M, 1)))
    b, sb = b or R.encode_matrix(0.05 * r(N, K))
    out = torch.full((M, N), 3.0, dtype=out_type, device="cuda") if out is None else out
    plus = None
    if add == "in place":
        out.copy_(r(M, N).to(out_type))
        plus = out
    elif add:
        plus = r(M, N).to(out_type)
    before = R.d64(plus) if plus is not None else 0.0
    B.fp8_matmul(a, sa, b, sb, out, add=plus)
    v, mags = R.matmul(R.dequant_rows(a, sa), R.dequant_matrix(b, sb))
    if plus is not None:
        v, mags = v + before, mags + before.abs()
    err = (R.d64(out) - v).abs()
    assert (err <= R.matmul_tol(v, mags, K, out_type)).all(), (err - R.matmul_tol(v, mags, K, out_type)).max()


@pytest.mark.parametrize("M", [1, 2, 8, 16, 17, 33, 64, 65, 128, 130, 300, 1100])
@pytest.mark.parametrize("N,K", [(128, 128), (256, 512), (1000, 1408), (33, 129), (1, 1), (2047, 100), (2880, 2880)])
def test_fp8_matmul(B, M, N, K):
    check_matmul(B, M, N, K, (BF16, FP16, FP32)[(M + N) % 3], add=(None, True, "in place")[(M + K) % 3])


@pytest.mark.parametrize("M,N,K", [(1, 4096, 4096), (16, 5760, 2880), (3, 512, 14336), (2000, 1100, 300), (513, 4096, 1000), (4100, 1300, 300),
                                   (2500, 2049, 1), (2500, 2303, 129), (19000, 64, 1408), (700, 8200, 640)])
def test_fp8_matmul_larger(B, M, N, K):
    check_matmul(B, M, N, K, BF16)


@pytest.mark.parametrize("M", [3, 40, 700])
def test_fp8_matmul_strides(B, M):
    """Rows inside larger buffers, scales in either order, outputs at odd places; what lies around stays."""
    N, K = 391, 450
    r = gen(M)
    qa, sa = R.encode_rows(r(M, K))
    qb, sb = R.encode_matrix(r(N, K))
    abuf = torch.full((M + 3, 560), 0x7F, dtype=torch.uint8, device="cuda").view(torch.float8_e4m3fn)   # NaN around the rows
    a = abuf[2:2 + M, 16:16 + K]
    a.copy_(qa)
    bbuf = torch.full((N + 1, 496), 0x7F, dtype=torch.uint8, device="cuda").view(torch.float8_e4m3fn)
    b = bbuf[:N, 32:32 + K]
    b.copy_(qb)
    obuf = torch.full((M + 2, N + 10), 7.0, dtype=BF16, device="cuda")
    out = obuf[1:-1, 3:3 + N]
    wsa = torch.full((R.blocks(K), M + 3), float("nan"), device="cuda")[:, :M].t()
    wsa.copy_(sa)
    wsb = torch.full((R.blocks(K), R.blocks(N) + 1), float("nan"), device="cuda")[:, :-1].t()
    wsb.copy_(sb)
    check_matmul(B, M, N, K, BF16, a=(a, wsa), b=(b, wsb), out=out)
    assert (obuf[0] == 7).all() and (obuf[-1] == 7).all() and (obuf[:, :3] == 7).all() and (obuf[:, 3 + N:] == 7).all()


@pytest.mark.parametrize("M", [5, 200])
def test_fp8_matmul_nan_stays_in_its_row(B, M):
    N, K = 260, 384
    r = gen(M)
    qa, sa = R.encode_rows(r(M, K))
    qb, sb = R.encode_matrix(r(N, K))
    clean, out = torch.empty(M, N, device="cuda"), torch.empty(M, N, device="cuda")
    B.fp8_matmul(qa, sa, qb, sb, clean)
    qa.view(torch.uint8)[1, 200] = 0x7F
    sa[3, 1] = float("inf")
    qb.view(torch.uint8)[77, 5] = 0xFF
    B.fp8_matmul(qa, sa, qb, sb, out)
    hit = torch.zeros(M, N, dtype=torch.bool, device="cuda")
    hit[1], hit[3], hit[:, 77] = True, True, True
    assert torch.equal(out[~hit], clean[~hit])
    assert out[1].isnan().all() and out[:, 77].isnan().all() and not out[3].isfinite().any()


def grouped(B, sizes, N, K, out_type, tail=0, add=False, offsets=None, seed=0):
    G, M = len(sizes), sum(sizes) + tail
    r = gen(seed + M + N + K + G)
    a, sa = R.encode_rows(r(M, K))
    b = torch.zeros(G, N, -(-K // 16) * 16, dtype=torch.uint8, device="cuda").view(torch.float8_e4m3fn)[..., :K]
    sb = torch.empty(G, R.blocks(N), R.blocks(K), device="cuda")
    for g in range(G):
        q, s = R.encode_matrix(0.05 * r(N, K))
        b[g].copy_(q)
        sb[g].copy_(s)
    if offsets is None:
        offsets = [0]
        for s in sizes:
            offsets.append(offsets[-1] + s)
    plus = r(M, N).to(out_type) if add else None
    out = torch.full((M, N), 3.0, dtype=out_type, device="cuda")
    B.fp8_matmul(a, sa, b, sb, out, add=plus, offsets=torch.tensor(offsets, dtype=torch.int32, device="cuda"))
    # the documented reading of the offsets
    edge, top = [], 0
    for o in offsets:
        top = max(top, min(o, M))
        edge.append(top)
    da = R.dequant_rows(a, sa)
    got = R.d64(out)
    held = torch.zeros(M, dtype=torch.bool)
    for g in range(G):
        lo, hi = edge[g], edge[g + 1]
        held[lo:hi] = True
        if hi > lo:
            v, mags = R.matmul(da[lo:hi], R.dequant_matrix(b[g], sb[g]))
            if add:
                v, mags = v + R.d64(plus[lo:hi]), mags + R.d64(plus[lo:hi]).abs()
            err = (got[lo:hi] - v).abs()
            assert (err <= R.matmul_tol(v, mags, K, out_type)).all(), g
    assert (got[~held] == 3).all()


@pytest.mark.parametrize("sizes,N,K,tail", [
    ([3, 0, 1, 17, 0], 300, 200, 2), ([0, 0, 0], 64, 128, 5), ([1], 128, 64, 0), ([0, 40], 130, 1408, 0),
    ([129, 0, 256, 1, 400], 520, 390, 3), ([700, 5], 257, 256, 0), ([2] * 32, 576, 288, 0), ([1] * 256, 64, 64, 1),
    ([0] * 200 + [300] + [0] * 50, 384, 129, 0), ([64] * 8, 1000, 640, 0), ([100, 700, 90, 128, 0, 130], 768, 512, 50),
    ([500, 0, 1300, 129, 2000, 3], 1300, 300, 9), ([0, 3000, 1, 700], 2049, 260, 1), ([128, 256, 384, 2100], 1800, 128, 0),
])
def test_fp8_matmul_grouped(B, sizes, N, K, tail):
    grouped(B, sizes, N, K, (BF16, FP32, FP16)[len(sizes) % 3], tail=tail, add=len(sizes) % 2 == 0)


@pytest.mark.parametrize("M", [40, 600])
def test_fp8_matmul_offsets_out_of_range(B, M):
    """Offsets that fall, are negative or pass the end are read as documented, within the buffers."""
    grouped(B, [M // 4] * 4, 200, 256, FP32, offsets=[-5, M // 2, M // 4, M + 1000, M])
    grouped(B, [M // 4] * 4, 200, 256, FP32, offsets=[M // 4, M // 2, M // 2, 2 ** 31 - 1, 0])
    grouped(B, [M // 4] * 4, 200, 256, FP32, offsets=[0, -(2 ** 31), 0, 0, -1])


# ----------------------------------------------------------------------------- balance

def run_balance(B, logits, idx, score, mask=None, coef=1.0, dloss=None, grad=True, **kw):
    M, E = logits.shape
    loss, prob = torch.full((1,), 7.0, device="cuda"), torch.full((E,), 7.0, device="cuda")
    counts = torch.full((E,), 7, dtype=torch.int32, device="cuda")
    offsets = torch.full((E + 1,), 7, dtype=torch.int32, device="cuda")
    d = torch.full_like(logits, 7.0) if grad else None
    B.balance(logits, idx, score, loss, counts, prob=prob, mask=mask, dlogits=d, coef=coef, offsets=offsets,
              dloss=torch.tensor([dloss], device="cuda") if dloss is not None else None, **kw)
    return loss, prob, counts, offsets, d


def check_balance(B, logits, idx, score, mask=None, coef=1.0, dloss=None, grad=True):
    loss, prob, counts, offsets, d = run_balance(B, logits, idx, score, mask, coef, dloss, grad)
    wl, wp, wc, wd = R.balance(logits, idx, score, mask, coef, 1.0 if dloss is None else dloss)
    M, E = logits.shape
    assert torch.equal(counts.cpu().long(), wc)
    assert torch.equal(offsets.cpu().long(), torch.nn.functional.pad(wc.cumsum(0), (1, 0)))
    # p: two exponentials, a logarithm's value (at most 90 in size) and a sum of E positive terms, E / 32 + 5 deep per lane
    prel = (90 + 8 + 5 + 12) * 2 * R.F32
    # sums of positive terms: rows of a lane, 5 + 8 across the CTA, the CTAs after one another
    srel = prel + (M / 592 / 8 + 64 + 13 + 592) * R.F32
    assert ((R.d64(prob) - wp).abs() <= wp * srel + 1e-37).all()
    assert abs(float(loss) - wl) <= abs(wl) * (srel + 16 * R.F32) + 1e-37
    if grad:
        # f - sum f p: f and the sum are each within prel of themselves, and at most the largest load
        T = max(1, int(mask.sum()) if mask is not None else M)
        f = wc.double().max() * E / (idx.shape[1] * T)
        tol = abs(coef * (1 if dloss is None else dloss)) / T * f * 4 * prel
        assert ((R.d64(d) - wd).abs() <= R.rounding(wd, logits.dtype) + tol * 1.0).all()
    return loss, prob, counts, d


def routed(M, E, K, dtype=FP32, seed=0):
    r = gen(seed + M + E * 3 + K)
    l = 1.5 * r(M, E) + r(E)
    return l.to(dtype), l.topk(K, -1).indices.to(torch.int32)


@pytest.mark.parametrize("score", [0, 1, 2])
@pytest.mark.parametrize("M,E,K,dtype", [(1, 1, 1, FP32), (1, 8, 2, BF16), (16, 32, 4, FP32), (17, 60, 6, FP16), (64, 64, 6, BF16),
                                         (333, 100, 8, FP32), (1000, 256, 8, FP32), (4099, 129, 3, BF16), (9000, 7, 2, FP32)])
def test_balance(B, score, M, E, K, dtype):
    l, idx = routed(M, E, K, dtype)
    check_balance(B, l, idx, score, coef=0.01, dloss=-3.0)
    check_balance(B, l, idx, score, grad=False)


@pytest.mark.parametrize("M", [40, 5000])
def test_balance_mask_strides_and_odd_entries(B, M):
    E, K = 36, 3
    l, idx = routed(M, E, K)
    mask = torch.rand(M, generator=torch.Generator().manual_seed(1)).cuda() > 0.3
    wl = wide(l, 3, 1)
    widx = torch.full((M, 8), 5, dtype=torch.int32, device="cuda")[:, 2:2 + K]
    widx.copy_(idx)
    widx[0] = torch.tensor([-1, E, 2 ** 31 - 1])      # entries that name no expert
    widx[1] = 4                                       # one expert named three times
    mask[:2] = True
    for score in (1, 2):
        check_balance(B, wl, widx, score, mask=mask)
        check_balance(B, wl, widx, score, mask=mask.to(torch.uint8), grad=False)
    none = torch.zeros(M, dtype=torch.bool, device="cuda")
    loss, prob, counts, offsets, d = run_balance(B, wl, widx, 1, none)
    assert loss.item() == 0 and not prob.any() and not counts.any() and not offsets.any() and not d.any()


@pytest.mark.parametrize("M", [6, 3000])
def test_balance_masked_and_extreme_logits(B, M):
    E, K = 40, 4
    l, idx = routed(M, E, K)
    l[1] = -float("inf")                              # nothing left in the row
    l[2] = torch.finfo(FP32).min
    l[3] = -300.0                                     # sigmoids that underflow; their shares do not
    l[4] = 1e30 * l[4]
    l[:, 7] = -float("inf")
    for score in (1, 2):
        loss, prob, counts, d = check_balance(B, l, idx, score)
        assert not d[1].any() and not d[:, 7].any()
    l[5, 3] = float("nan")
    loss, prob, counts, offsets, d = run_balance(B, l, idx, 1)
    assert loss.isnan().all() and d[5].isnan().all() and d[:5].isfinite().all()


def test_balance_no_rows(B):
    loss, prob, counts, offsets, d = run_balance(B, torch.empty(0, 9, device="cuda"), torch.empty(0, 2, dtype=torch.int32, device="cuda"), 1)
    assert loss.item() == 0 and not prob.any() and not counts.any() and not offsets.any()


@pytest.mark.parametrize("score", [1, 2])
def test_balance_gradient_against_differences(B, score):
    """Central differences of the loss in 64 bits along random directions (idx, so the load, held fixed): their own
    error is h^2 / 6 times a third derivative of at most a few times the loss, and rounding / h."""
    M, E, K, h = 12, 20, 3, 1e-4
    l, idx = routed(M, E, K)
    *_, d = run_balance(B, l, idx, score, coef=0.5)
    l64 = l.double().cpu()
    for seed in range(4):
        u = torch.randn(M, E, generator=torch.Generator().manual_seed(seed), dtype=torch.float64)
        up, down = (R.balance(l64 + s * h * u, idx, score, coef=0.5)[0] for s in (1, -1))
        got = float((R.d64(d) * u).sum())
        scale = float((R.d64(d).abs() * u.abs()).sum())
        assert abs(got - (up - down) / (2 * h)) <= 1e-6 * scale + 1e-7 * abs(up)


def test_balance_equal_calls_give_equal_bits(B):
    l, idx = routed(20000, 64, 6)
    first = run_balance(B, l, idx, 2)
    for _ in range(3):
        for x, y in zip(first, run_balance(B, l, idx, 2)):
            assert torch.equal(x, y)


# ----------------------------------------------------------------------------- together

def expert_layer(B, moe, shape, W, resid, delta, gamma):
    """One routed half in 8 bits: norm, route, load, the experts' two products over the routes sorted by expert."""
    (gu, gus), (dn, dns) = W
    M, H = resid.shape
    E, K, inter = shape.num_experts, shape.top_k, shape.moe_inter
    dev = resid.device
    x, xq, xs = torch.empty_like(resid), R.rows8(M, H), torch.empty(M, R.blocks(H), device=dev)
    B.rmsnorm(resid, gamma, 1e-5, delta=delta, resid_out=resid, y=x, q=xq, q_scale=xs)
    idx, w = torch.empty(M, K, dtype=torch.int32, device=dev), torch.empty(M, K, device=dev)
    logits = torch.empty(M, E, device=dev)
    moe.route(0, x, idx, w, logits)
    loss, counts, offsets = torch.empty(1, device=dev), torch.empty(E, dtype=torch.int32, device=dev), torch.empty(E + 1, dtype=torch.int32, device=dev)
    dlogits = torch.empty_like(logits)
    B.balance(logits, idx, shape.score, loss, counts, offsets=offsets, dlogits=dlogits)
    order = torch.argsort(idx.view(-1), stable=True)
    rows = order // K
    a = R.rows8(M * K, H)
    a.view(torch.uint8).copy_(xq.view(torch.uint8)[rows])
    both = torch.empty(M * K, 2 * inter, dtype=BF16, device=dev)
    B.fp8_matmul(a, xs[rows], gu, gus, both, offsets=offsets)
    h, hs = R.rows8(M * K, inter), torch.empty(M * K, R.blocks(inter), device=dev)
    B.act_quant(both[:, :inter], both[:, inter:], shape.act, h, hs, shape.act_alpha, shape.act_limit)
    y = torch.empty(M * K, H, device=dev)
    B.fp8_matmul(h, hs, dn, dns, y, offsets=offsets)
    parts = torch.empty_like(y)
    parts[order] = y * w.view(-1)[order][:, None]
    return dict(x=x, xq=xq, xs=xs, idx=idx, w=w, logits=logits, loss=loss, counts=counts, both=both, h=h, hs=hs,
                y=parts.view(M, K, H).sum(1), dlogits=dlogits)


def layer_setup(B, M, seed=0):
    shape = synth.MoEShape("chain", 320, 160, 12, 3, cfg_id=611, max_tokens=256, act=synth.ACT_SWIGLU_CLAMPED)
    L = synth.make_layer(shape, 0, device="cuda")
    moe = B.MoE(shape, [L])
    r = gen(seed)

    def matrices(N, K):
        q = torch.zeros(shape.num_experts, N, K, dtype=torch.uint8, device="cuda").view(torch.float8_e4m3fn)
        s = torch.empty(shape.num_experts, R.blocks(N), R.blocks(K), device="cuda")
        for e in range(shape.num_experts):
            qe, se = R.encode_matrix(0.05 * r(N, K))
            q[e].copy_(qe)
            s[e].copy_(se)
        return q, s

    W = matrices(2 * shape.moe_inter, shape.hidden), matrices(shape.hidden, shape.moe_inter)
    return shape, moe, W, r(M, shape.hidden).to(BF16), r(M, shape.hidden), (1 + 0.1 * r(shape.hidden)).to(BF16)


@pytest.mark.parametrize("M", [1, 16, 200])
def test_layer_of_8_bit_experts(B, M):
    """The operators as a layer uses them, against the formulas on the same 8-bit values, step by step; the sum at the
    end against a run in 64 bits from the 8-bit inputs of each product."""
    shape, moe, W, resid, delta, gamma = layer_setup(B, M)
    want_r, v = R.rmsnorm(resid, gamma, 1e-5, delta)
    o = expert_layer(B, moe, shape, W, resid, delta, gamma)
    moe.device_status()
    assert torch.equal(resid.cpu(), want_r)
    R.check_rows8(o["xq"], o["xs"], v, NORM_REL)
    assert torch.equal(o["counts"].cpu(), torch.bincount(o["idx"].view(-1).cpu(), minlength=shape.num_experts).int())
    wl, _, _, wd = R.balance(o["logits"], o["idx"], shape.score)
    assert abs(float(o["loss"]) - wl) <= 1e-4 * wl
    x = R.dequant_rows(o["xq"], o["xs"])
    order = torch.argsort(o["idx"].view(-1), stable=True).cpu()
    hq = R.dequant_rows(o["h"], o["hs"])
    want = torch.zeros(M, shape.hidden, dtype=torch.float64)
    tol = torch.zeros_like(want)
    idx, w = o["idx"].cpu(), R.d64(o["w"])
    for pos, route in enumerate(order.tolist()):
        t, e = route // shape.top_k, int(idx.view(-1)[route])
        g, mags = R.matmul(x[t:t + 1], R.dequant_matrix(W[0][0][e], W[0][1][e]))
        err = (R.d64(o["both"][pos]) - g[0]).abs()
        assert (err <= R.matmul_tol(g, mags, shape.hidden, BF16)[0]).all()
        y, mags = R.matmul(hq[pos:pos + 1], R.dequant_matrix(W[1][0][e], W[1][1][e]))
        want[t] += w.view(-1)[route] * y[0]
        tol[t] += w.view(-1)[route] * R.matmul_tol(y, mags, shape.moe_inter, FP32)[0] + 4 * R.F32 * (w.view(-1)[route] * y[0]).abs()
    assert ((R.d64(o["y"]) - want).abs() <= tol + 4 * R.F32 * want.abs()).all()
    moe.close()


def test_norm_feeds_the_routed_half(B):
    """The norm's y as ts_moe_forward's x, its y joined to the stream by the next norm."""
    shape, moe, _, resid, delta, gamma = layer_setup(B, 24, seed=5)
    x, resid2 = torch.empty_like(resid), torch.empty_like(resid)
    B.rmsnorm(resid, gamma, 1e-5, delta=delta, resid_out=resid2, y=x)
    y, inplace = torch.empty(24, shape.hidden, device="cuda"), resid2.clone()
    moe.forward(0, x, resid=inplace, y=y)
    x2, stream = torch.empty_like(x), torch.empty_like(resid)
    B.rmsnorm(resid2, gamma, 1e-5, delta=y, resid_out=stream, y=x2)
    assert torch.equal(stream, inplace)         # bf16(resid + y) either way
    x3 = torch.empty_like(x)
    B.rmsnorm(inplace, gamma, 1e-5, y=x3)
    assert torch.equal(x2, x3)                  # a fused addition is an addition followed by a norm
    moe.device_status()
    moe.close()


def test_captured_and_replayed(B):
    """The whole run in a graph: replays on new inputs equal eager runs, bit for bit."""
    shape, moe, W, resid, delta, gamma = layer_setup(B, 100)
    fresh = [(gen(s)(100, shape.hidden).to(BF16), gen(s + 50)(100, shape.hidden)) for s in (21, 22)]
    eager = []
    for r0, d0 in fresh:
        eager.append({k: v.clone() for k, v in expert_layer(B, moe, shape, W, r0.clone(), d0, gamma).items()})
    sr, sd = resid.clone(), delta.clone()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        expert_layer(B, moe, shape, W, sr, sd, gamma)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        o = expert_layer(B, moe, shape, W, sr, sd, gamma)
    for _ in range(2):
        for (r0, d0), want in zip(fresh, eager):
            sr.copy_(r0)
            sd.copy_(d0)
            graph.replay()
            for k, v in want.items():
                assert torch.equal(o[k].view(torch.uint8) if o[k].dtype == torch.float8_e4m3fn else o[k],
                                   v.view(torch.uint8) if v.dtype == torch.float8_e4m3fn else v), k
    del graph
    moe.device_status()
    moe.close()


def test_two_streams_at_once(B):
    """Calls on two streams, with outputs (and torch's workspaces) of their own, equal calls one after another."""
    M, N, K, E = 600, 1024, 1024, 64
    r = gen(31)
    a, sa = R.encode_rows(r(M, K))
    b, sb = R.encode_matrix(r(N, K))
    small, ssmall = a[:8], sa[:8]
    l, idx = routed(20000, E, 6)

    def work(stream=None):
        out, dec = torch.empty(M, N, device="cuda"), torch.empty(8, N, device="cuda")
        loss, counts, d = torch.empty(1, device="cuda"), torch.empty(E, dtype=torch.int32, device="cuda"), torch.empty_like(l)
        y, q, s = torch.empty(M, K, device="cuda"), R.rows8(M, K), torch.empty(M, K // 128, device="cuda")
        for _ in range(10):
            B.fp8_matmul(a, sa, b, sb, out, stream=stream)
            B.fp8_matmul(small, ssmall, b, sb, dec, stream=stream)
            B.balance(l, idx, 2, loss, counts, dlogits=d, stream=stream)
            B.rmsnorm(out, None, 1e-5, y=y, q=q, q_scale=s, stream=stream)
        return out, dec, loss, counts, d, y, q.view(torch.uint8), s

    want = work()
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    got = []
    for s in streams:
        with torch.cuda.stream(s):
            got.append(work())
    torch.cuda.synchronize()
    for g in got:
        for x, y in zip(g, want):
            assert torch.equal(x, y)
    given = work(streams[0])
    torch.cuda.synchronize()
    for x, y in zip(given, want):
        assert torch.equal(x, y)


def test_row_offsets_past_32_bits(B):
    """Rows whose byte offsets pass 2^32: the last rows of a tall buffer."""
    H = 16384
    M = (1 << 32) // (2 * H) + 3
    buf = torch.zeros(M, H, dtype=BF16, device="cuda")
    tail = gen(1)(3, H).to(BF16)
    buf[-3:] = tail
    q, s = R.rows8(M, H), torch.empty(M, H // 128, device="cuda")
    B.rmsnorm(buf, None, 1e-5, q=q, q_scale=s)
    _, v = R.rmsnorm(tail, None, 1e-5, None)
    R.check_rows8(q[-3:], s[-3:], v, NORM_REL)
    B.act_quant(buf[:, :8192], buf[:, 8192:], 0, q[:, :8192], s[:, :64])
    R.check_rows8(q[-3:, :8192], s[-3:, :64], R.act(tail[:, :8192], tail[:, 8192:], 0), ACT_REL)


# ----------------------------------------------------------------------------- kernels and paths by size

def nan_padded(q, pad, shift):
    """8-bit rows in a buffer that holds NaN codes around them."""
    M, K = q.shape
    ld = -(-(K + pad + shift) // 16) * 16
    buf = torch.full((M, ld), 0x7F, dtype=torch.uint8, device="cuda").view(torch.float8_e4m3fn)
    at = buf[:, shift:shift + K]
    at.copy_(q)
    return at


@pytest.mark.parametrize("M", [1, 2, 5, 7, 8, 9])
@pytest.mark.parametrize("N,K", [(1, 1), (15, 17), (16, 16), (17, 127), (31, 144), (2049, 129), (640, 4096), (1000, 1100), (48, 14336)])
def test_fp8_matmul_a_step_of_decode(B, M, N, K):
    """Few rows, with NaN codes behind every row of both operands."""
    r = gen(M + N + K)
    qa, sa = R.encode_rows(r(M, K))
    qb, sb = R.encode_matrix(0.05 * r(N, K))
    check_matmul(B, M, N, K, (BF16, FP16, FP32)[(M + K) % 3], add=(None, True, "in place")[(M + N) % 3],
                 a=(nan_padded(qa, 5, 16), sa), b=(nan_padded(qb, 33, 0), sb))


@pytest.mark.parametrize("out_type", [BF16, FP16, FP32])
@pytest.mark.parametrize("add", [None, True, "in place"])
@pytest.mark.parametrize("N", [2049, 2050, 2056])
def test_fp8_matmul_tiles_at_odd_places(B, N, add, out_type):
    """Tiles whose rows start at 2-, 4- and 16-byte places, plain and added to."""
    check_matmul(B, 2500, N, 1408, out_type, add=add)


@pytest.mark.parametrize("out_type", [BF16, FP32])
@pytest.mark.parametrize("shift", [0, 1, 3, 6])
def test_fp8_matmul_tiles_leave_their_surroundings(B, out_type, shift):
    """Groups whose last rows end inside a tile, written into a wider buffer: nothing beside them changes."""
    sizes, N, K = [200, 0, 333, 1, 150], 300, 256
    M = sum(sizes) + 7
    r = gen(shift)
    a, sa = R.encode_rows(r(M, K))
    b = torch.zeros(len(sizes), N, K, dtype=torch.uint8, device="cuda").view(torch.float8_e4m3fn)
    sb = torch.empty(len(sizes), R.blocks(N), R.blocks(K), device="cuda")
    for g in range(len(sizes)):
        q, s = R.encode_matrix(0.05 * r(N, K))
        b[g].copy_(q)
        sb[g].copy_(s)
    edge = [0]
    for s in sizes:
        edge.append(edge[-1] + s)
    buf = torch.full((M + 2, N + 12), 7.0, dtype=out_type, device="cuda")
    out = buf[1:-1, shift:shift + N]
    B.fp8_matmul(a, sa, b, sb, out, offsets=torch.tensor(edge, dtype=torch.int32, device="cuda"))
    da = R.dequant_rows(a, sa)
    for g in range(len(sizes)):
        lo, hi = edge[g], edge[g + 1]
        v, mags = R.matmul(da[lo:hi], R.dequant_matrix(b[g], sb[g]))
        assert ((R.d64(out[lo:hi]) - v).abs() <= R.matmul_tol(v, mags, K, out_type)).all(), g
    assert (out[edge[-1]:] == 7).all() and (buf[0] == 7).all() and (buf[-1] == 7).all()
    assert (buf[:, :shift] == 7).all() and (buf[:, shift + N:] == 7).all()


@pytest.mark.parametrize("M,H,rt,dt", [(2000, 512, BF16, FP32), (1300, 4096, BF16, BF16), (1100, 8192, FP32, FP32), (1200, 5120, FP16, BF16)])
def test_rmsnorm_many_rows_in_place(B, M, H, rt, dt):
    """More rows than CTAs, the residual in place and rows inside a wider buffer."""
    r = gen(M + H)
    buf = torch.full((M, H + 16), 9.0, dtype=rt, device="cuda")
    at = buf[:, 8:8 + H]
    at.copy_((r(M, H) * torch.exp(r(M, 1))).to(rt))
    delta, gamma = r(M, H).to(dt), (1 + 0.2 * r(H)).to(BF16)
    want_r, v = R.rmsnorm(at, gamma, 1e-5, delta)
    y, q, s = torch.empty(M, H, dtype=BF16, device="cuda"), R.rows8(M, H), torch.empty(M, R.blocks(H), device="cuda")
    B.rmsnorm(at, gamma, 1e-5, delta=delta, resid_out=at, y=y, q=q, q_scale=s)
    assert torch.equal(at.cpu(), want_r)
    assert ((R.d64(y) - v).abs() <= R.rounding(v, BF16) + v.abs() * NORM_REL).all()
    R.check_rows8(q, s, v, NORM_REL)
    assert (buf[:, :8] == 9).all() and (buf[:, 8 + H:] == 9).all()


@pytest.mark.parametrize("dtype", [FP32, BF16])
@pytest.mark.parametrize("E", [8, 60, 129, 256])
def test_balance_rows_of_unlike_size(B, E, dtype):
    """Rows whose sigmoids all but vanish beside ordinary ones, in one warp and far from E = a multiple of four."""
    l, idx = routed(700, E, 4)
    l[::3] -= 30
    l[1::5] -= 95
    l[7] = -1e4
    l[8, 1:] = -float("inf")
    l = l.to(dtype)
    mask = torch.rand(700, generator=torch.Generator().manual_seed(E)).cuda() > 0.2
    for score in (1, 2):
        check_balance(B, l, idx, score, mask=mask, coef=0.3)
        check_balance(B, l[:20], idx[:20], score)


def test_balance_masked_rows_may_hold_anything(B):
    """Rows that the mask leaves out may hold NaN and infinities: they touch nothing."""
    l, idx = routed(600, 64, 6)
    mask = torch.ones(600, dtype=torch.bool, device="cuda")
    mask[100:140] = False
    for score in (1, 2):
        want = run_balance(B, torch.where(mask[:, None], l, torch.zeros_like(l)), idx, score, mask)
        bad = l.clone()
        bad[100:120], bad[120:130], bad[130:140] = float("nan"), float("inf"), -float("inf")
        got = run_balance(B, bad, idx, score, mask)
        for x, y in zip(got, want):
            assert torch.equal(x, y)
        assert not got[-1][100:140].any()


def test_two_graphs_replayed_in_turn(B):
    """Two captured calls of one size, each with its own inputs: replays in turn equal eager calls."""
    cases = []
    for seed in (1, 2):
        l, idx = routed(9000, 64, 6, seed=seed)
        a, sa = R.encode_rows(gen(seed)(300, 512))
        b, sb = R.encode_matrix(gen(seed + 9)(700, 512))
        out, loss = torch.empty(300, 700, device="cuda"), torch.empty(1, device="cuda")
        counts, d = torch.empty(64, dtype=torch.int32, device="cuda"), torch.empty_like(l)

        def call(l=l, idx=idx, a=a, sa=sa, b=b, sb=sb, out=out, loss=loss, counts=counts, d=d):
            B.balance(l, idx, 2, loss, counts, dlogits=d)
            B.fp8_matmul(a, sa, b, sb, out)
            return out, loss, counts, d

        want = [t.clone() for t in call()]
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            got = call()
        cases.append((graph, got, want, call))   # call keeps the inputs alive
    for _ in range(3):
        for graph, got, *_ in cases:
            for t in got:
                t.zero_()
            graph.replay()
        torch.cuda.synchronize()
        for _, got, want, _ in cases:
            for x, y in zip(got, want):
                assert torch.equal(x, y)


FIRST_CALL = """
import torch
from quantized_moe_routed_router_b200 import binding as B
from tests import ops_ref as R
M, N, K, E = {M}, 2304, 512, 64
g = torch.Generator(device="cuda")
g.manual_seed(1)
r = lambda *s: torch.randn(*s, generator=g, device="cuda")
a, sa = R.encode_rows(r(M, K))
b, sb = R.encode_matrix(r(N, K))
x, l = r(M, N), r(M, E)
idx = l.topk(4, -1).indices.to(torch.int32)
out, y, q, s = torch.empty(M, N, device="cuda"), torch.empty(M, N, device="cuda"), R.rows8(M, N), torch.empty(M, N // 128, device="cuda")
loss, counts, d = torch.empty(1, device="cuda"), torch.empty(E, dtype=torch.int32, device="cuda"), torch.empty_like(l)


def run():
    B.fp8_matmul(a, sa, b, sb, out)
    B.rmsnorm(out, None, 1e-5, delta=x, y=y)
    B.act_quant(y, x, 0, q, s)
    B.balance(l, idx, 2, loss, counts, dlogits=d)
    return out, y, q.view(torch.uint8), s, loss, counts, d


torch.cuda.synchronize()
graph = torch.cuda.CUDAGraph()
with torch.cuda.graph(graph):
    run()
graph.replay()
torch.cuda.synchronize()
got = [t.clone() for t in (out, y, q.view(torch.uint8), s, loss, counts, d)]
for t, u in zip(got, run()):
    assert torch.equal(t, u)
torch.cuda.synchronize()
print("equal")
"""


@pytest.mark.parametrize("M", [4, 60, 3000])
def test_first_call_of_a_process_is_captured(B, M):
    """Nothing a first call sets up stands in the way of a capture."""
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    p = subprocess.run([sys.executable, "-c", FIRST_CALL.format(M=M)], cwd=root, capture_output=True, text=True, timeout=120)
    assert p.returncode == 0 and "equal" in p.stdout, p.stderr[-2000:]
