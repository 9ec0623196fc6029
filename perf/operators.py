"""The operators next to the routed half, as they are measured: what a call takes, its plain form and its work.

Four operators surround the routed experts in a decoder layer:

* ``norm``: the residual's addition and the root-mean-square norm that makes the routed half's input, in 16 bits and in
  8 bits (e4m3) with one scale per 128 columns of a row;
* ``act``: SwiGLU (or the clamped form) with the same 8-bit output, between an expert's two products;
* ``matmul``: the product of such 8-bit rows with an e4m3 matrix that has one scale per 128 x 128 block, dense (a
  projection) or grouped (row runs of an expert-sorted batch, one matrix per expert);
* ``balance``: the router's per-expert counts, its balance loss and the loss's gradient.

``run`` computes them in their plain form in 32 bits, or with ``own`` set through the library's binding.
"""
import math

import torch

own = False

BLOCK = 128          # columns of a row, and rows and columns of a matrix, that share a scale
E4M3_MAX = 448.0
AMAX_FLOOR = 2.0 ** -100  # smallest magnitude a scale is formed from: an all-zero group gets a normal scale

DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
SIZES = {"bf16": 2, "fp16": 2, "fp32": 4}
SOFTMAX, SIGMOID = 1, 2   # the library's TS_SCORE_SOFTMAX_ALL_NORENORM and TS_SCORE_SIGMOID_RENORM
SWIGLU, CLAMPED = 0, 1    # TS_ACT_SWIGLU, TS_ACT_SWIGLU_CLAMPED
ALPHA, LIMIT = 1.702, 7.0


def listed():
    return [
        # a decode micro-batch of the gpt-oss-shaped stack: the FP32 sum of one half joins the residual
        dict(name="norm 16x2880", op="norm", M=16, H=2880, resid="bf16", delta="fp32", gamma="fp32", y=True, q=True),
        # a prompt's rows at the Mixtral-shaped width: both forms of the normed rows are wanted
        dict(name="norm 16384x4096", op="norm", M=16384, H=4096, resid="bf16", delta="bf16", gamma="bf16", y=True, q=True),
        # 16 tokens x 4 experts of the gpt-oss-shaped layer, clamped SwiGLU
        dict(name="act 64x2880", op="act", M=64, I=2880, act=CLAMPED, dtype="bf16"),
        # a prompt through the Mixtral-shaped width
        dict(name="act 8192x14336", op="act", M=8192, I=14336, act=SWIGLU, dtype="bf16"),
        # one token through a square projection: latency
        dict(name="matmul 1x4096x4096", op="matmul", M=1, N=4096, K=4096, out="bf16", add=False),
        # a decode micro-batch through the gpt-oss-shaped gate and up: the last scale block is half full
        dict(name="matmul 16x5760x2880", op="matmul", M=16, N=5760, K=2880, out="bf16", add=False),
        # a ragged chunk of a prompt, added to an FP32 stream, at odd sizes
        dict(name="matmul 333x2047x1408", op="matmul", M=333, N=2047, K=1408, out="fp32", add=True),
        # a long prompt through the Mixtral-shaped dense width
        dict(name="matmul 8192x14336x4096", op="matmul", M=8192, N=14336, K=4096, out="bf16", add=False),
        # a decode micro-batch's routes over 32 experts, some of which get none
        dict(name="experts 64x5760x2880 of 32", op="matmul", G=32, M=64, N=5760, K=2880, tail=0, skew=0.0, out="bf16", add=False),
        # a prompt's routes over 64 experts of the deepseek2-lite shape, unevenly loaded, with rows behind the last expert's
        dict(name="experts 24576x2816x2048 of 64", op="matmul", G=64, M=24576, N=2816, K=2048, tail=100, skew=0.7, out="bf16", add=False),
        # the load of a decode micro-batch's routing
        dict(name="balance 16x32", op="balance", M=16, E=32, K=4, score=SOFTMAX, dtype="fp32", mask=False, grad=False),
        # a training batch with padding, the largest router, with the gradient
        dict(name="balance 65536x256", op="balance", M=65536, E=256, K=8, score=SIGMOID, dtype="fp32", mask=True, grad=True),
    ]


def _size(rng, low, high, step=1):
    """A size spread over its logarithm; odd ones come up as often as round ones."""
    n = int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))
    if rng.random() < 0.5:
        n = n // 16 * 16
    return max(low, min(high, n)) // step * step


def draw(rng):
    op = rng.choice(("norm", "act", "matmul", "matmul", "experts", "balance"))
    if op == "norm":
        H = _size(rng, 64, 16384)
        y = rng.random() < 0.7
        return dict(op="norm", M=_size(rng, 1, 16384 * 4096 // max(H, 4096)), H=H, resid=rng.choice(("bf16", "bf16", "fp16", "fp32")),
                    delta=rng.choice(("bf16", "fp32", "none")), gamma=rng.choice(("bf16", "fp32")), y=y, q=not y or rng.random() < 0.7)
    if op == "act":
        inter = _size(rng, 64, 14336)
        return dict(op="act", M=_size(rng, 1, 8192), I=inter, act=rng.choice((SWIGLU, CLAMPED)), dtype=rng.choice(("bf16", "fp16", "fp32")))
    if op == "matmul":
        return dict(op="matmul", M=_size(rng, 1, 8192), N=_size(rng, 64, 14336), K=_size(rng, 64, 4096),
                    out=rng.choice(("bf16", "bf16", "fp16", "fp32")), add=rng.random() < 0.3)
    if op == "experts":
        G, N, K = rng.choice((8, 32, 64, 100)), _size(rng, 64, 5760), _size(rng, 64, 4096)
        G = max(2, min(G, 530_000_000 // (N * K)))
        return dict(op="matmul", G=G, M=_size(rng, 1, 8192), N=N, K=K, tail=rng.choice((0, 1, 37)), skew=rng.choice((0.0, 0.7)),
                    out=rng.choice(("bf16", "fp16", "fp32")), add=rng.random() < 0.3)
    E = rng.choice((8, 32, 60, 64, 100, 256))
    return dict(op="balance", M=_size(rng, 1, 65536), E=E, K=rng.choice((1, 2, 4, 6, 8)), score=rng.choice((SOFTMAX, SIGMOID)),
                dtype=rng.choice(("fp32", "fp32", "bf16")), mask=rng.random() < 0.5, grad=rng.random() < 0.6)


# ----------------------------------------------------------------------------- inputs

def _blocks(n):
    return -(-n // BLOCK)


def _rows8(M, K):
    """[M, K] bytes whose rows start 16-byte aligned, as the library's 8-bit rows do."""
    return torch.empty(M, -(-K // 16) * 16, dtype=torch.uint8, device="cuda")[:, :K].view(torch.float8_e4m3fn)


def _encode_rows(x):
    """fp32 [M, K] to e4m3 rows and their scales, one per 128 columns."""
    M, K = x.shape
    x = torch.nn.functional.pad(x, (0, _blocks(K) * BLOCK - K)).view(M, -1, BLOCK)
    s = x.abs().amax(-1).clamp_min(AMAX_FLOOR) / E4M3_MAX
    q = _rows8(M, K)
    q.copy_((x / s[..., None]).view(M, -1)[:, :K].to(torch.float8_e4m3fn))
    return q, s


def _encode_matrix(w):
    """fp32 [N, K] to e4m3 and one scale per 128 x 128 block."""
    N, K = w.shape
    w = torch.nn.functional.pad(w, (0, _blocks(K) * BLOCK - K, 0, _blocks(N) * BLOCK - N)).view(_blocks(N), BLOCK, -1, BLOCK)
    s = w.abs().amax((1, 3)).clamp_min(AMAX_FLOOR) / E4M3_MAX
    q = _rows8(N, K)
    q.copy_((w / s[:, None, :, None]).view(_blocks(N) * BLOCK, -1)[:N, :K].to(torch.float8_e4m3fn))
    return q, s


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)

    def randn(*shape):
        return torch.randn(*shape, generator=g, device="cuda")

    s = dict(case)
    M = case["M"]
    if case["op"] == "norm":
        H = case["H"]
        # rows of a residual stream: a few columns much larger than the rest, rows of unlike size
        size = torch.exp(randn(M, 1))
        column = torch.exp(0.5 * randn(H))
        s["r"] = (randn(M, H) * size * column).to(DTYPES[case["resid"]])
        s["d"] = (randn(M, H) * column).to(DTYPES[case["delta"]]) if case["delta"] != "none" else None
        s["g"] = (1 + 0.2 * randn(H)).to(DTYPES[case["gamma"]])
        s["r_out"] = torch.empty_like(s["r"]) if s["d"] is not None else None
        s["y_out"] = torch.empty(M, H, dtype=torch.bfloat16, device="cuda") if case["y"] else None
        s["q_out"] = _rows8(M, H) if case["q"] else None
        s["s_out"] = torch.empty(M, _blocks(H), device="cuda") if case["q"] else None
    elif case["op"] == "act":
        inter = case["I"]
        # one product makes gate and up side by side
        both = (2 * randn(M, 2 * inter)).to(DTYPES[case["dtype"]])
        s["gate"], s["up"] = both[:, :inter], both[:, inter:]
        s["q_out"], s["s_out"] = _rows8(M, inter), torch.empty(M, _blocks(inter), device="cuda")
    elif case["op"] == "matmul":
        N, K, G, tail = case["N"], case["K"], case.get("G", 0), case.get("tail", 0)
        s["a"], s["a_scale"] = _encode_rows(randn(M + tail, K) * torch.exp(0.5 * randn(M + tail, 1)))
        if G:
            # rows sorted by expert; `skew` makes some experts' share larger than others'
            share = torch.softmax(case["skew"] * randn(G), 0)
            count = torch.bincount(torch.multinomial(share, M, replacement=True, generator=g), minlength=G)
            s["offsets"] = torch.nn.functional.pad(count.cumsum(0), (1, 0)).to(torch.int32)
            s["most"] = int(count.max())
            s["b"] = torch.empty(G, N, -(-K // 16) * 16, dtype=torch.uint8, device="cuda")[..., :K].view(torch.float8_e4m3fn)
            s["b_scale"] = torch.empty(G, _blocks(N), _blocks(K), device="cuda")
            for e in range(G):
                q, sc = _encode_matrix(0.02 * randn(N, K))
                s["b"][e].copy_(q)
                s["b_scale"][e].copy_(sc)
        else:
            s["b"], s["b_scale"] = _encode_matrix(0.02 * randn(N, K))
            s["offsets"] = None
        s["plus"] = randn(M + tail, N).to(DTYPES[case["out"]]) if case["add"] else None
        s["out_"] = torch.full((M + tail, N), 0.25, dtype=DTYPES[case["out"]], device="cuda")
    else:
        E, K = case["E"], case["K"]
        logits = randn(M, E) * 1.5 + 0.5 * randn(E)
        s["idx"] = logits.topk(min(K, E), dim=-1).indices.to(torch.int32)
        s["logits"] = logits.to(DTYPES[case["dtype"]])
        # padded rows stand behind the texts of a batch: about one in eight
        s["mask_"] = torch.rand(M, generator=g, device="cuda") > 0.125 if case["mask"] else None
        s["loss"] = torch.empty(1, device="cuda")
        s["prob"] = torch.empty(E, device="cuda")
        s["counts"] = torch.empty(E, dtype=torch.int32, device="cuda")
        s["dlogits"] = torch.empty_like(s["logits"]) if case["grad"] else None
    return s


# ----------------------------------------------------------------------------- one pass

def run(s):
    if own:
        return _own(s)
    return {"norm": _plain_norm, "act": _plain_act, "matmul": _plain_matmul, "balance": _plain_balance}[s["op"]](s)


def _own(s):
    from quantized_moe_routed_router_b200 import binding
    if s["op"] == "norm":
        binding.rmsnorm(s["r"], s["g"], 1e-5, delta=s["d"], resid_out=s["r_out"], y=s["y_out"], q=s["q_out"], q_scale=s["s_out"])
        return {"resid": s["r_out"] if s["d"] is not None else s["r"], "y": s["y_out"], "q": s["q_out"], "q_scale": s["s_out"]}
    if s["op"] == "act":
        binding.act_quant(s["gate"], s["up"], s["act"], s["q_out"], s["s_out"], act_alpha=ALPHA, act_limit=LIMIT)
        return {"q": s["q_out"], "q_scale": s["s_out"]}
    if s["op"] == "matmul":
        binding.fp8_matmul(s["a"], s["a_scale"], s["b"], s["b_scale"], s["out_"], add=s["plus"], offsets=s["offsets"])
        return s["out_"]
    binding.balance(s["logits"], s["idx"], s["score"], s["loss"], s["counts"], prob=s["prob"], mask=s["mask_"], dlogits=s["dlogits"])
    return {"loss": s["loss"], "prob": s["prob"], "counts": s["counts"], "dlogits": s["dlogits"]}


def _plain_rows8(v):
    """fp32 [M, K] to e4m3 rows and their scales."""
    M, K = v.shape
    groups = torch.nn.functional.pad(v, (0, _blocks(K) * BLOCK - K)).view(M, -1, BLOCK)
    scale = groups.abs().amax(-1).clamp_min(AMAX_FLOOR) / E4M3_MAX
    q = (groups / scale[..., None]).view(M, -1)[:, :K].to(torch.float8_e4m3fn)
    return q, scale


def _plain_norm(s):
    r = s["r"]
    if s["d"] is not None:
        r = (r.float() + s["d"].float()).to(r.dtype)  # the stream is kept in its own type, and the norm reads what is kept
    x = r.float()
    v = x * torch.rsqrt(x.square().mean(-1, keepdim=True) + 1e-5) * s["g"].float()
    q, scale = _plain_rows8(v) if s["q_out"] is not None else (None, None)
    return {"resid": r, "y": v.to(torch.bfloat16) if s["y_out"] is not None else None, "q": q, "q_scale": scale}


def _plain_act(s):
    g, u = s["gate"].float(), s["up"].float()
    if s["act"] == CLAMPED:
        g, u = g.clamp(max=LIMIT), u.clamp(-LIMIT, LIMIT)
        v = g * torch.sigmoid(ALPHA * g) * (u + 1)
    else:
        v = g * torch.sigmoid(g) * u
    q, scale = _plain_rows8(v)
    return {"q": q, "q_scale": scale}


def _plain_matmul(s):
    K, N = s["K"], s["N"]
    a = s["a"].float() * s["a_scale"].repeat_interleave(BLOCK, 1)[:, :K]
    b = s["b"].float() * s["b_scale"].repeat_interleave(BLOCK, -2)[..., :N, :].repeat_interleave(BLOCK, -1)[..., :K]
    if s["offsets"] is None:
        out = a @ b.t()
    else:
        # rows of a group side by side in a slab of the longest group's length
        G, M = b.shape[0], a.shape[0]
        row = torch.arange(M, device=a.device)
        group = torch.searchsorted(s["offsets"][1:].long(), row, right=True)
        held = group < G
        group = group.clamp_max(G - 1)
        place = torch.where(held, row - s["offsets"][group], s["most"])
        slab = torch.zeros(G, s["most"] + 1, K, device=a.device)
        slab[group, place] = a
        out = torch.bmm(slab, b.transpose(1, 2))[group, place]
    if s["plus"] is not None:
        out = out + s["plus"].float()
    out = out.to(s["out_"].dtype)
    return out if s["offsets"] is None else torch.where(held[:, None], out, s["out_"])


def _plain_balance(s):
    E = s["E"]
    l = s["logits"].float()
    M, K = s["idx"].shape
    keep = s["mask_"] if s["mask_"] is not None else torch.ones(M, dtype=torch.bool, device=l.device)
    tokens = keep.sum().clamp_min(1)
    counts = ((s["idx"][..., None] == torch.arange(E, device=l.device)).any(1) & keep[:, None]).sum(0)
    load = counts * (E / K) / tokens
    if s["score"] == SIGMOID:
        sig = torch.sigmoid(l)
        p = sig / sig.sum(-1, keepdim=True)
        slope = p * torch.sigmoid(-l)
    else:
        p = torch.exp(l - l.amax(-1, keepdim=True))
        p = p / p.sum(-1, keepdim=True)
        slope = p
    prob = (p * keep[:, None]).sum(0) / tokens
    grad = None
    if s["dlogits"] is not None:
        grad = slope * (load - (p * load).sum(-1, keepdim=True)) * (keep[:, None] / tokens)
        grad = grad.to(s["dlogits"].dtype)
    return {"loss": (load * prob).sum().view(1), "prob": prob, "counts": counts.to(torch.int32), "dlogits": grad}


# ----------------------------------------------------------------------------- values and work

def exact(case, seed):
    """The values in 64 bits, before any rounding to an output's type."""
    s = prepare(case, seed)
    if case["op"] == "norm":
        r = s["r"].double()
        if s["d"] is not None:
            r = (r + s["d"].double()).to(s["r"].dtype).double()
        rms = ((r ** 2).sum(1) / case["H"] + 1e-5) ** 0.5
        v = r / rms[:, None] * s["g"].double()
        q, scale = _exact_rows8(v) if case["q"] else (None, None)
        return {"resid": r, "y": v if case["y"] else None, "q": q, "q_scale": scale}
    if case["op"] == "act":
        g, u = s["gate"].double(), s["up"].double()
        if case["act"] == CLAMPED:
            g, u = torch.minimum(g, g.new_tensor(LIMIT)), torch.maximum(torch.minimum(u, u.new_tensor(LIMIT)), u.new_tensor(-LIMIT))
            v = g / (1 + torch.exp(-ALPHA * g)) * (1 + u)
        else:
            v = g / (1 + torch.exp(-g)) * u
        q, scale = _exact_rows8(v)
        return {"q": q, "q_scale": scale}
    if case["op"] == "matmul":
        N, K = case["N"], case["K"]
        col = torch.arange(K, device="cuda") // BLOCK
        line = torch.arange(N, device="cuda") // BLOCK
        a = s["a"].double() * s["a_scale"].double()[:, col]
        plus = s["plus"].double() if s["plus"] is not None else torch.zeros((), dtype=torch.float64, device="cuda")
        if s["offsets"] is None:
            return a @ (s["b"].double() * s["b_scale"].double()[line][:, col]).t() + plus
        out, edge = s["out_"].double(), s["offsets"].tolist()
        for e in range(case["G"]):
            if edge[e + 1] > edge[e]:
                rows = slice(edge[e], edge[e + 1])
                out[rows] = a[rows] @ (s["b"][e].double() * s["b_scale"][e].double()[line][:, col]).t()
                if s["plus"] is not None:
                    out[rows] += plus[rows]
        return out
    l, E, K = s["logits"].double(), case["E"], s["idx"].shape[1]
    keep = s["mask_"].double() if s["mask_"] is not None else torch.ones(case["M"], dtype=torch.float64, device="cuda")
    tokens = max(1.0, float(keep.sum()))
    counts = torch.zeros(E, dtype=torch.float64, device="cuda").index_add_(0, s["idx"].reshape(-1).long(), keep.repeat_interleave(K))
    load = counts * E / (K * tokens)
    if case["score"] == SIGMOID:
        e = 1 / (1 + torch.exp(-l))
        p, slope = e / e.sum(1)[:, None], 1 - e
    else:
        p, slope = torch.softmax(l, 1), torch.ones_like(l)
    prob = keep @ p / tokens
    grad = p * slope * (load[None] - (p @ load)[:, None]) * keep[:, None] / tokens if case["grad"] else None
    return {"loss": (load @ prob).view(1), "prob": prob, "counts": counts.to(torch.int32), "dlogits": grad}


def _exact_rows8(v):
    M, K = v.shape
    group = (torch.arange(K, device=v.device) // BLOCK).expand(M, K)
    top = torch.zeros(M, _blocks(K), dtype=torch.float64, device=v.device).scatter_reduce_(1, group, v.abs(), "amax")
    scale = torch.clamp(top, min=AMAX_FLOOR) / E4M3_MAX
    return v / scale.gather(1, group), scale


def work(case):
    M = case["M"]
    if case["op"] == "norm":
        H, e = case["H"], SIZES[case["resid"]]
        per = e + (SIZES[case["delta"]] + e if case["delta"] != "none" else 0) + (2 if case["y"] else 0) + (1 if case["q"] else 0)
        return {"bytes": M * H * per + (4 * M * _blocks(H) if case["q"] else 0) + H * SIZES[case["gamma"]], "flops": 8 * M * H}
    if case["op"] == "act":
        inter = case["I"]
        return {"bytes": M * inter * (2 * SIZES[case["dtype"]] + 1) + 4 * M * _blocks(inter), "flops": 10 * M * inter}
    if case["op"] == "matmul":
        N, K, G = case["N"], case["K"], case.get("G", 0)
        reached = G * (1 - (1 - 1 / G) ** M) if G else 1  # matrices that get a row at all, on average
        return {"bytes": reached * (N * K + 4 * _blocks(N) * _blocks(K)) + M * (K + 4 * _blocks(K)) + M * N * SIZES[case["out"]] * (2 if case["add"] else 1),
                "flops": 2 * M * N * K}
    E, e = case["E"], SIZES[case["dtype"]]
    return {"bytes": M * (E * e * (2 if case["grad"] else 1) + 4 * min(case["K"], E) + (1 if case["mask"] else 0)) + 8 * E, "flops": 12 * M * E}
