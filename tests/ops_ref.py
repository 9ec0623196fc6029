"""The operators next to the routed half from their formulas, in 64 bits on the CPU, and what a result may be off by.

A rounding to type t is off by at most eps(t) / 2 relative to the value; E4M3
codes by 2^-4 of the value, or by half their smallest step (2^-10) of the scale."""
import torch

BLOCK = 128
F32 = 2.0 ** -24       # half a step of float32, relative
E4M3_HALF, E4M3_SUB = 2.0 ** -4, 2.0 ** -10
HALF = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11, torch.float32: 2.0 ** -24}
FP16_SUB = 2.0 ** -25  # half fp16's smallest step


def blocks(n):
    return -(-n // BLOCK)


def d64(t):
    return t.detach().cpu().double()


def rows8(M, K, device="cuda", fill=0):
    """[M, K] E4M3 rows at 16-byte boundaries."""
    t = torch.full((M, -(-K // 16) * 16), fill, dtype=torch.uint8, device=device)
    return t.view(torch.float8_e4m3fn)[:, :K]


def rounding(v, dtype):
    """Largest error of rounding v (64 bits) to dtype."""
    return v.abs() * HALF[dtype] + (FP16_SUB if dtype == torch.float16 else 0.0)


def group_scale(v):
    """Scale of each 128-column group of v, and the scale spread over the columns."""
    M, K = v.shape
    p = torch.nn.functional.pad(v, (0, blocks(K) * BLOCK - K)).view(M, -1, BLOCK)
    s = p.abs().amax(-1).clamp_min(2.0 ** -100) / 448.0
    return s, s.repeat_interleave(BLOCK, 1)[:, :K]


def check_rows8(q, q_scale, v, rel):
    """q * q_scale against v, itself computed to within rel: the scale to rel and its own two roundings,
    each value to half a code step of the scale that was stored."""
    s, _ = group_scale(v)
    got = d64(q_scale)
    assert ((got - s).abs() <= s * (rel + 4 * F32)).all()
    wide = got.repeat_interleave(BLOCK, 1)[:, :v.shape[1]]
    back = d64(q.float()) * wide
    tol = v.abs() * (E4M3_HALF + rel + 4 * F32) + wide * E4M3_SUB
    assert ((back - v).abs() <= tol).all(), ((back - v).abs() - tol).max()


def rmsnorm(resid, gamma, eps, delta):
    """(r, v): r in resid's type, v in 64 bits."""
    r = resid.detach().cpu()
    if delta is not None:
        # the float32 sum rounded to the type: both steps are the operator's definition
        r = (r.float() + delta.detach().cpu().float()).to(r.dtype)
    x = r.double()
    v = x / torch.sqrt((x * x).mean(1, keepdim=True) + eps)
    return r, v if gamma is None else v * d64(gamma)


def act(gate, up, kind, alpha=1.702, limit=7.0):
    g, u = d64(gate), d64(up)
    if kind == 0:
        return g / (1 + torch.exp(-g)) * u
    g, u = g.clamp(max=limit), u.clamp(-limit, limit)
    return g / (1 + torch.exp(-alpha * g)) * (u + 1)


def dequant_rows(q, s):
    return d64(q.float()) * d64(s).repeat_interleave(BLOCK, 1)[:, :q.shape[1]]


def dequant_matrix(q, s):
    N, K = q.shape
    return d64(q.float()) * d64(s).repeat_interleave(BLOCK, 0)[:N].repeat_interleave(BLOCK, 1)[:, :K]


def matmul(a, b):
    """(value, sum of magnitudes) of dequantised a [M, K] and b [N, K]."""
    return a @ b.t(), a.abs() @ b.abs().t()


def matmul_tol(value, mags, K, dtype):
    """K products in float32, 128 to a block and the blocks after one another or split and joined: each of a value's
    additions and scalings is off by at most one step (2^-23) of the magnitudes' sum."""
    return mags * ((min(K, BLOCK) + blocks(K) + 12) * 2.0 ** -23) + rounding(value, dtype)


def encode_rows(x):
    """float32 [M, K] to E4M3 rows and scales on x's device."""
    M, K = x.shape
    p = torch.nn.functional.pad(x, (0, blocks(K) * BLOCK - K)).view(M, -1, BLOCK)
    s = p.abs().amax(-1).clamp_min(2.0 ** -100) / 448.0
    q = rows8(M, K, x.device)
    q.copy_((p / s[..., None]).view(M, -1)[:, :K].to(torch.float8_e4m3fn))
    return q, s


def encode_matrix(w):
    N, K = w.shape
    p = torch.nn.functional.pad(w, (0, blocks(K) * BLOCK - K, 0, blocks(N) * BLOCK - N)).view(blocks(N), BLOCK, -1, BLOCK)
    s = p.abs().amax((1, 3)).clamp_min(2.0 ** -100) / 448.0
    q = rows8(N, K, w.device)
    q.copy_((p / s[:, None, :, None]).view(blocks(N) * BLOCK, -1)[:N, :K].to(torch.float8_e4m3fn))
    return q, s


def balance(logits, idx, score, mask=None, coef=1.0, dloss=1.0):
    """(loss, prob, counts, dlogits) in 64 bits.  Rows of -inf alone have p = 0."""
    l = d64(logits)
    M, E = l.shape
    idx = idx.cpu().long()
    keep = torch.ones(M, dtype=torch.bool) if mask is None else mask.cpu().bool()
    T = int(keep.sum())
    sel = idx[keep].reshape(-1)
    sel = sel[(sel >= 0) & (sel < E)]
    counts = torch.bincount(sel, minlength=E)
    if T == 0:
        z = torch.zeros(E, dtype=torch.float64)
        return 0.0, z, counts, torch.zeros_like(l)
    f = counts.double() * E / (idx.shape[1] * T)
    if score == 2:
        t = torch.nn.functional.logsigmoid(l)
        slope = torch.sigmoid(-l)
    else:
        t, slope = l, torch.ones_like(l)
    empty = (t == -torch.inf).all(1, keepdim=True)
    p = torch.where(empty, 0.0, torch.softmax(torch.where(empty, 0.0, t), 1))
    prob = p[keep].sum(0) / T
    grad = p * slope * (f - (p * f).sum(1, keepdim=True)) * (coef * dloss / T)
    grad[~keep] = 0
    return coef * float((f * prob).sum()), prob, counts, grad
