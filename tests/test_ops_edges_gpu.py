"""The operators next to the routed half on the GPU where exactness, extreme values or a failure path is the point."""
import ctypes as C

import pytest
import torch

from tests import ops_ref as R
from tests.test_ops_gpu import BF16, FP16, FP32, gen, grouped, routed, run_balance

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def B():
    from quantized_moe_routed_router_b200 import build
    build.build()
    from quantized_moe_routed_router_b200 import binding
    return binding


# ----------------------------------------------------------------------------- codes are rounded quotients

def codes(v):
    """(codes, scales) of float32 v from the definition: scale = max(amax, 2^-100) * (1 / 448), code = e4m3(v / scale), the
    reciprocal, the product and the quotient each rounded to float32."""
    M, K = v.shape
    p = torch.nn.functional.pad(v.cpu(), (0, R.blocks(K) * 128 - K)).view(M, -1, 128)
    s = p.abs().amax(-1).clamp_min(2.0 ** -100) * torch.tensor(1.0 / 448.0)
    return (p / s[..., None]).view(M, -1)[:, :K].to(torch.float8_e4m3fn), s


def same_codes(q, s, v):
    """-0 and 0 are one value: compared as numbers."""
    wq, ws = codes(v)
    assert torch.equal(s.cpu(), ws)
    assert torch.equal(q.float().cpu(), wq.float()), (q.float().cpu() != wq.float()).sum()


@pytest.mark.parametrize("M,H", [(2000, 4096), (1100, 8192), (40, 16384), (300, 1001)])
def test_norm_codes_are_the_quotients(B, M, H):
    """From the kernel's own float32 rows: 16-bit inputs put some values in ten thousand exactly between two codes, where an
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


# ----------------------------------------------------------------------------- a wait that runs out

def held_product(B, cta, a, sa, b, sb, out, offsets=None, wait_us=1000):
    """fp8_matmul in which one CTA issues no copies and gives its waits up after a millisecond; contiguous tensors."""
    M, K, N = a.shape[0], a.shape[1], out.shape[1]
    G = 1 if offsets is None else b.shape[0]
    args = B.Fp8MatmulArgs(rows=M, n=N, k=K, num_groups=G, out_type={BF16: 0, FP16: 1, FP32: 2}[out.dtype], reserved=0,
                           a=a.data_ptr(), ld_a=a.stride(0), a_scale=sa.data_ptr(), as_row=sa.stride(0), as_block=sa.stride(1),
                           b=b.data_ptr(), ld_b=b.stride(-2), b_group=b.stride(0) if G > 1 else 0, b_scale=sb.data_ptr(),
                           bs_group=sb.stride(0) if G > 1 else 0, bs_row=sb.stride(-2), bs_block=sb.stride(-1),
                           offsets=None if offsets is None else offsets.data_ptr(), add=None, ld_add=0,
                           out=out.data_ptr(), ld_out=out.stride(0))
    st = B.lib.ts_moe_debug_fp8_matmul_held(C.byref(args), cta, wait_us, torch.cuda.current_stream().cuda_stream)
    assert st == 0, B.lib.ts_moe_last_error(None)


def lost_tiles(out, want, starts, rows, cols):
    """Of the tiles (rows from each of `starts`, `cols` columns), the ones that are NaN; the others have to equal `want`."""
    lost = []
    for r0, r1 in starts:
        for m in range(r0, r1, rows):
            for n in range(0, out.shape[1], cols):
                t, w = out[m:min(m + rows, r1), n:n + cols], want[m:min(m + rows, r1), n:n + cols]
                if t.isnan().all():
                    lost.append((m, n))
                else:
                    assert torch.equal(t, w), (m, n)
    return lost


# K split over 2 and 3 CTAs of a cluster; tiles of 128 x 256 that a CTA takes one after another
@pytest.mark.parametrize("M,N,K,rows,cols", [(64, 4096, 4096, 32, 128), (16, 5760, 2880, 16, 128), (2000, 5000, 300, 128, 256)])
@pytest.mark.parametrize("cta", [0, 1, 5])
def test_fp8_matmul_wait_that_runs_out_gives_nan(B, M, N, K, rows, cols, cta):
    """A CTA whose copies never come: the outputs that need its sums are NaN, all others are as ever, and so is the next call."""
    r = gen(M)
    a, sa = R.encode_rows(r(M, K))
    b, sb = R.encode_matrix(r(N, K))
    want, out = torch.empty(M, N, device="cuda"), torch.full((M, N), 3.0, device="cuda")
    B.fp8_matmul(a, sa, b, sb, want)
    held_product(B, cta, a, sa, b, sb, out)
    torch.cuda.synchronize()
    tiles = -(-M // rows) * -(-N // cols)
    lost = lost_tiles(out, want, [(0, M)], rows, cols)
    assert 1 <= len(lost) <= -(-tiles // 148), lost
    B.fp8_matmul(a, sa, b, sb, out)
    assert torch.equal(out, want)


def test_fp8_matmul_wait_that_runs_out_in_a_group(B):
    """The same where a CTA takes whole items of small groups, K unsplit."""
    G, each, N, K = 32, 2, 1024, 512
    r = gen(2)
    a, sa = R.encode_rows(r(G * each, K))
    b = torch.empty(G, N, K, dtype=torch.uint8, device="cuda").view(torch.float8_e4m3fn)
    sb = torch.empty(G, R.blocks(N), R.blocks(K), device="cuda")
    for g in range(G):
        q, s = R.encode_matrix(r(N, K))
        b[g].copy_(q)
        sb[g].copy_(s)
    offsets = torch.arange(0, G * each + 1, each, dtype=torch.int32, device="cuda")
    want, out = torch.empty(G * each, N, device="cuda"), torch.full((G * each, N), 3.0, device="cuda")
    B.fp8_matmul(a, sa, b, sb, want, offsets=offsets)
    held_product(B, 7, a, sa, b, sb, out, offsets)
    torch.cuda.synchronize()
    lost = lost_tiles(out, want, [(g * each, g * each + each) for g in range(G)], 16, 128)
    assert len(lost) == 1, lost
    B.fp8_matmul(a, sa, b, sb, out, offsets=offsets)
    assert torch.equal(out, want)


@pytest.mark.parametrize("sizes,N,K,tail", [
    ([20] * 32, 300, 260, 1), ([1, 60, 0, 33, 32, 31, 65, 0], 520, 512, 3), ([25] * 8, 512, 1408, 0), ([90, 10], 391, 1300, 2),
    ([0, 255, 0, 1], 1024, 520, 5)])
def test_fp8_matmul_groups_of_medium_size(B, sizes, N, K, tail):
    """Groups that end inside a tile of 32 rows, K whole and shared."""
    for t, add in ((BF16, False), (FP32, True)):
        grouped(B, sizes, N, K, t, tail=tail, add=add)


# ----------------------------------------------------------------------------- far below the sigmoid's own range

# e^x from an exponent rounded once, which turns into |x| half steps (|x| <= 180 here), two exponentials of 2 ulp and four
# products; the clamped form's alpha g adds its own rounding, another |x| half steps
FAR_REL = (2 * 180 + 2 * 4 + 8) * R.F32


@pytest.mark.parametrize("inter", [256, 250])
@pytest.mark.parametrize("dtype", [BF16, FP32])
@pytest.mark.parametrize("kind,alpha,limit", [(0, 1.0, 7.0), (1, 1.0, 1e38), (1, 2.0, 1e36)])
def test_act_quant_of_gates_far_below_zero(B, inter, dtype, kind, alpha, limit):
    """silu(g) up with g from -60 to -180 and up large enough for values that a scale reaches: e^g alone is below the
    smallest float32 from -104 on, the product is not.  One far gate among ordinary ones in the last rows."""
    M = 24
    r = gen(inter)
    g = -torch.linspace(60, 170, M, device="cuda")[:, None] / alpha * (1 + 0.05 * torch.rand(M, inter, device="cuda"))
    u = torch.where(r(M, inter) > 0, 1.0, -1.0) * torch.exp2(120 + 2 * torch.rand(M, inter, device="cuda"))
    u[:4] *= 2.0 ** -100
    g[20:, :128], u[20:, :128] = r(4, 128), r(4, 128)
    g[20:, 5] = -90.0 / alpha
    u[20:, 5] = 1e30
    g, u = g.to(dtype), u.to(dtype)
    q, s = R.rows8(M, inter), torch.empty(M, R.blocks(inter), device="cuda")
    B.act_quant(g, u, kind, q, s, act_alpha=alpha, act_limit=limit)
    v = R.act(g, u, kind, alpha, limit)
    R.check_rows8(q, s, v, FAR_REL)
    assert (q[:12].float() != 0).any(1).all()


def test_act_quant_of_infinite_gates(B):
    """silu(-inf) is no number, as its formula has it, in the group that holds it and nowhere else."""
    g, u = gen(1)(3, 256), gen(2)(3, 256)
    g[1, 200] = -float("inf")
    q, s = R.rows8(3, 256), torch.empty(3, 2, device="cuda")
    B.act_quant(g, u, 0, q, s)
    assert s[1, 1].isnan() and s.isnan().sum() == 1


# ----------------------------------------------------------------------------- rows of a router's batch

@pytest.mark.parametrize("E", [8, 60, 256])
def test_balance_gradient_of_a_row_does_not_depend_on_its_neighbours(B, E):
    """With one idx (so one load), other rows' logits change nothing in a row's gradient, not even its last bits: rows of
    negative logits beside ones whose sigmoids all but vanish."""
    M = 640
    l = gen(E)(M, E) - 3.0
    idx = l.topk(4, -1).indices.to(torch.int32)

    def gradient(logits):
        loss, counts, d = torch.empty(1, device="cuda"), torch.empty(E, dtype=torch.int32, device="cuda"), torch.empty_like(logits)
        B.balance(logits, idx, 2, loss, counts, dlogits=d)
        return d

    beside = l.clone()
    beside[1::3] -= 40.0
    want, got = gradient(l), gradient(beside)
    assert torch.equal(got[0::3], want[0::3]) and torch.equal(got[2::3], want[2::3])


def gradient_bound(logits, idx, score, mask, coef, dloss):
    """(gradient in 64 bits, what float32 may leave it off by), element by element and in proportion to p (1 - sigmoid):

    p = t / sum t.  t: an exponential (2 ulp = 4 half steps) whose argument d (l - max, or l) is rounded as a difference, by
    the constant and as a product, 3 |d| half steps; for sigmoids also a sum and a reciprocal, 1 + 4.  The sum: at most
    8 + 5 additions of positive terms.  The quotient: a reciprocal and a product, 4 + 1.  1 - sigmoid: as t, and a product.
    f: 3 roundings.  sum f p: as p, f, and 13 additions.  The rest: 3 of coef dloss / T, and 4 products and a difference."""
    l = R.d64(logits)
    M, E = l.shape
    *_, counts, grad = R.balance(logits, idx, score, mask, coef, dloss)
    T = max(1, M if mask is None else int(mask.sum()))
    f = counts.double() * E / (idx.shape[1] * T)
    t = torch.nn.functional.logsigmoid(l) if score == 2 else l
    p = torch.softmax(t, 1)
    slope = torch.sigmoid(-l) if score == 2 else torch.ones_like(l)
    d = float((l - l.max(1, keepdim=True).values).abs().max()) if score != 2 else float(l.abs().max())
    trel = (3 * d + 4 + (5 if score == 2 else 0)) * R.F32
    prel = 2 * trel + (13 + 5) * R.F32
    srel = trel + R.F32 if score == 2 else 0.0
    fp = (p * f).sum(1, keepdim=True)
    c = abs(coef * dloss) / T
    bound = c * p * slope * ((f - fp).abs() * (prel + srel + 8 * R.F32) + 3 * R.F32 * f + fp * (prel + 16 * R.F32))
    return grad, bound + R.rounding(grad, logits.dtype) + c * f.max() * 2.0 ** -124


@pytest.mark.parametrize("score", [0, 1, 2])
@pytest.mark.parametrize("M,E,K,dtype", [(3, 8, 2, FP32), (65, 40, 4, FP16), (333, 100, 8, FP32), (1000, 256, 8, FP32), (4099, 129, 3, BF16),
                                         (20000, 64, 6, FP32), (3000, 200, 8, FP16)])
def test_balance_gradient_element_by_element(B, score, M, E, K, dtype):
    l, idx = routed(M, E, K, dtype)
    mask = torch.rand(M, generator=torch.Generator().manual_seed(M)).cuda() > 0.2
    for m in (None, mask):
        *_, d = run_balance(B, l, idx, score, m, coef=0.5, dloss=-3.0)
        want, tol = gradient_bound(l, idx, score, m, 0.5, -3.0)
        err = (R.d64(d) - want).abs()
        assert (err <= tol).all(), (err / tol).max()


@pytest.mark.parametrize("score", [1, 2])
@pytest.mark.parametrize("M,E,K", [(400, 256, 8), (1500, 130, 4)])
def test_balance_gradient_against_differences_over_many_ctas(B, score, M, E, K):
    """Central differences of the loss in 64 bits, the load held fixed.  Their own error: h^2 / 6 times the third derivative,
    at most 6 (2 V)^3 times the largest load for shares that move by V (a sigmoid's slope is at most 1; a factor 4 for
    its own derivatives), and a rounding of the loss over h."""
    l, idx = routed(M, E, K)
    *_, d = run_balance(B, l, idx, score, coef=0.5)
    _, tol = gradient_bound(l, idx, score, None, 0.5, 1.0)
    f = torch.bincount(idx.flatten().cpu().long(), minlength=E).max().double() * E / (K * M)
    h, l64 = 1e-6, l.double().cpu()
    for seed in range(3):
        u = torch.randn(M, E, generator=torch.Generator().manual_seed(seed), dtype=torch.float64)
        up, down = (R.balance(l64 + s * h * u, idx, score, coef=0.5)[0] for s in (1, -1))
        got, want = float((R.d64(d) * u).sum()), (up - down) / (2 * h)
        room = 0.5 * f * h * h / 6 * 4 * 6 * (2 * u.abs().max()) ** 3 + abs(up) * 2.0 ** -50 / h
        assert abs(got - want) <= float((tol * u.abs()).sum() + room), (got, want, float(room))
        assert abs(want) > 20 * float(room)      # the differences say something


# ----------------------------------------------------------------------------- the binding's stream

def test_current_stream_without_torchs_private_name(B, monkeypatch):
    """The binding loads and runs on the current stream where torch lacks the direct call."""
    import importlib.util
    monkeypatch.delattr(torch._C, "_cuda_getCurrentRawStream")
    spec = importlib.util.spec_from_file_location("quantized_moe_routed_router_b200.binding_again", B.__file__)
    again = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(again)
    x, y = gen(1)(5, 256), torch.empty(5, 256, device="cuda")
    for s in (torch.cuda.current_stream(), torch.cuda.Stream()):
        with torch.cuda.stream(s):
            assert again._current_stream(0) == s.cuda_stream
            again.rmsnorm(x, None, 1e-5, y=y)
        torch.cuda.synchronize()
        want = torch.empty_like(y)
        B.rmsnorm(x, None, 1e-5, y=want)
        assert torch.equal(y, want)
        y.zero_()
        torch.cuda.synchronize()
