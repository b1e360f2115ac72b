"""The operators around a layer's quantized products, for measurement: the root-mean-square norm with the residual's
addition (to f32, f16, or 8 bits with scales for the integer products), the routing of tokens to experts, and the
products with bias, activation, elementwise factor and residual in their epilogue.

``run`` makes either the library's calls (``own``) or the same results from elementary torch operations.  Both work on
the same GGUF bytes; where a program keeps its weights in the library's repacked order, so does the state here
(``_repacked`` spells that order out), and the plain form reads the weights back out of it.
"""
import math

import torch

own = False

DEV = "cuda"
F16, F32, F64 = torch.float16, torch.float32, torch.float64
EPS = 1e-5


# ---------------------------------------------------------------------------
# Cases
# ---------------------------------------------------------------------------
def listed():
    return [
        # One token between two layers: the projection's f32 result joins the residual stream, the norm feeds the next
        # product in f16.  A launch's latency.
        dict(name="norm_1_token", op="norm", T=1, H=1, D=4096, x="f32", res="f32", out="f16"),
        # The heads of a prompt's queries, each normed by itself before the rotation: many short rows, a slice of the
        # projection's output.
        dict(name="norm_heads", op="norm", T=4999, H=32, D=128, x="f16", res="none", out="f16"),
        # A prompt's hidden states: the largest.
        dict(name="norm_prompt", op="norm", T=8192, H=1, D=4096, x="f32", res="f32", out="f16"),
        # One token through the norm in 8 bits and the integer product that reads it, four-bit weights.
        dict(name="i8_1_token", op="i8", T=1, D=4096, N=4096, kind="Q4_0", x="f32", res="f32", bias=False, act="none"),
        # Seven sequences' tokens, eight-bit weights, a bias and an activation behind the product.
        dict(name="i8_7_tokens", op="i8", T=7, D=4096, N=11008, kind="Q8_0", x="f16", res="f16", bias=True, act="silu"),
        # One token over 128 experts, eight chosen: latency.
        dict(name="route_1_token", op="route", M=1, E=128, k=8, score="softmax", bias=False, groups=1, keep=1, top=1,
             norm=True, scale=1.0, dtype="f32", pad=0),
        # A ragged batch padded to a captured step's size, an odd number of experts, f16 logits.
        dict(name="route_batch", op="route", M=333, E=60, k=4, score="softmax", bias=False, groups=1, keep=1, top=1,
             norm=False, scale=1.0, dtype="f16", pad=13),
        # A long prompt over 256 experts in eight groups, a bias for balance: the largest.
        dict(name="route_prompt", op="route", M=16384, E=256, k=8, score="sigmoid", bias=True, groups=8, keep=4, top=2,
             norm=True, scale=2.5, dtype="f32", pad=0),
        # One token's gate projection, times its up projection: the decode step's largest product.
        dict(name="product_1_token", op="product", M=1, N=14336, K=4096, kind="Q4_K", packed=False, a="f16",
             bias=False, act="silu", mul="f32", res="none", out="f16"),
        # Eight tokens' down projection into the f32 residual stream.
        dict(name="product_8_tokens", op="product", M=8, N=4096, K=14336, kind="Q6_K", packed=False, a="f16",
             bias=False, act="none", mul="none", res="f32", out="f32"),
        # A prompt of odd length through a layer with biases, repacked eight-bit weights.
        dict(name="product_499_tokens", op="product", M=499, N=4096, K=4096, kind="Q8_0", packed=True, a="f16",
             bias=True, act="gelu", mul="none", res="f16", out="f16"),
        # A long prompt's gate projection times its up projection: the largest.
        dict(name="product_prompt", op="product", M=2048, N=14336, K=4096, kind="Q4_K", packed=False, a="f16",
             bias=False, act="silu", mul="f16", res="none", out="f16"),
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(("norm", "i8", "route", "product", "product"))
    if op == "norm":
        H = rng.choice((1, 1, 1, rng.randint(2, 64)))
        D = rng.choice((64, 96, 128, 256)) if H > 1 else _log(rng, 64, 16384)
        return dict(op=op, T=_log(rng, 1, max(1, (1 << 25) // (H * D))), H=H, D=D, x=rng.choice(("f32", "f16")),
                    res=rng.choice(("f32", "f16", "none")) if H == 1 else "none", out=rng.choice(("f32", "f16")))
    if op == "i8":
        D = 256 * _log(rng, 2, 40)
        return dict(op=op, T=rng.randint(1, min(8, 262144 // D)), D=D, N=_log(rng, 64, 16384),
                    kind=rng.choice(("Q8_0", "Q4_0")), x=rng.choice(("f32", "f16")),
                    res=rng.choice(("f32", "f16", "none")), bias=rng.random() < 0.5,
                    act=rng.choice(("none", "relu", "silu", "gelu", "gelu_tanh")))
    if op == "route":
        groups = rng.choice((1, 1, 4, 8))
        E = groups * _log(rng, 4, 512 // groups)
        keep = rng.randint(1, groups)
        M = _log(rng, 1, (1 << 22) // E)
        return dict(op=op, M=M, E=E, k=rng.randint(1, min(16, E // groups * keep)),
                    score=rng.choice(("softmax", "sigmoid")), bias=rng.random() < 0.5, groups=groups, keep=keep,
                    top=rng.choice((1, 2)), norm=rng.random() < 0.7, scale=rng.choice((1.0, 2.5)),
                    dtype=rng.choice(("f32", "f16")), pad=rng.choice((0, 0, M // 8)))
    kind = rng.choice(("Q4_0", "Q8_0", "Q4_K", "Q6_K"))
    packed = kind in ("Q4_0", "Q8_0") and rng.random() < 0.5
    M = rng.choice((rng.randint(1, 8), _log(rng, 9, 2048)))
    N, K = _log(rng, 64, 14336), 256 * _log(rng, 2, 56)
    M = max(1, min(M, (2048 * 14336 * 4096) // (N * K)))
    # Up to eight tokens the products are exact to f32 for f16 activations; the larger ones round weights to f16, so
    # their results go on in f16.
    a = rng.choice(("f16", "f32"))
    out = rng.choice(("f16", "f32")) if M <= 8 and a == "f16" else "f16"
    return dict(op=op, M=M, N=N, K=K, kind=kind, packed=packed, a=a, bias=rng.random() < 0.5,
                act=rng.choice(("none", "relu", "silu", "gelu", "gelu_tanh")), mul=rng.choice(("none", "none", "f16", "f32")),
                res=rng.choice(("none", "f16", "f32")), out=out)


SIZE = {"f16": 2, "f32": 4, "none": 0}
BLOCK = {"Q4_0": (18, 32), "Q8_0": (34, 32), "Q4_K": (144, 256), "Q6_K": (210, 256)}


def _row_bytes(kind, K):
    return K // BLOCK[kind][1] * BLOCK[kind][0]


def work(c):
    if c["op"] == "norm":
        n = c["T"] * c["H"] * c["D"]
        return {"bytes": n * (SIZE[c["x"]] + 2 * SIZE[c["res"]] + SIZE[c["out"]]) + 4 * c["D"], "flops": 4 * n}
    if c["op"] == "i8":
        n = c["T"] * c["D"]
        return {"bytes": n * (SIZE[c["x"]] + 2 * SIZE[c["res"]]) + 4 * c["D"] + c["N"] * _row_bytes(c["kind"], c["D"])
                + 4 * c["T"] * c["N"] + 4 * c["N"] * c["bias"], "flops": 2 * n * c["N"] + 4 * n}
    if c["op"] == "route":
        n = c["M"] * c["E"]
        return {"bytes": n * SIZE[c["dtype"]] + 4 * c["E"] * c["bias"] + 4 * c["M"] + 8 * c["M"] * c["k"], "flops": 4 * n}
    n = c["M"] * c["N"]
    return {"bytes": c["N"] * _row_bytes(c["kind"], c["K"]) + c["M"] * c["K"] * SIZE[c["a"]] + 4 * c["N"] * c["bias"]
            + n * (SIZE[c["mul"]] + SIZE[c["res"]] + SIZE[c["out"]]), "flops": 2 * n * c["K"]}


# ---------------------------------------------------------------------------
# Weights: GGUF blocks, and the repacked order of two kinds
# ---------------------------------------------------------------------------
def _gen(seed, what):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed * 16 + what)
    return g


def _dt(name):
    return {"f16": F16, "f32": F32}[name]


def _weights(kind, N, K, seed):
    """Rows of random blocks [N, blocks, block bytes] whose products with unit activations have unit size."""
    g = _gen(seed, 7)
    size, elems = BLOCK[kind]
    w = torch.randint(0, 256, (N, K // elems, size), generator=g, device=DEV, dtype=torch.uint8)
    rms = {"Q4_0": 4.6, "Q8_0": 74.0, "Q4_K": 258.0, "Q6_K": 1370.0}[kind]
    d = (0.5 + torch.rand((N, K // elems, 1), generator=g, device=DEV)) / (rms * math.sqrt(K))
    if kind == "Q4_K":
        w[..., :4] = torch.cat((d, 7.5 * d), dim=-1).to(F16).view(torch.uint8)
    elif kind == "Q6_K":
        w[..., 208:] = d.to(F16).view(torch.uint8)
    else:
        w[..., :2] = d.to(F16).view(torch.uint8)
    return w


def _repacked(kind, w):
    """The blocks [N, K/32, bytes] in the library's order, flat: tiles of 16 rows by 8 blocks, their codes first (by
    section, lane group, row and byte), then their scales (by row)."""
    N, nb, size = w.shape
    w = torch.cat((w, torch.zeros((-N % 16, nb, size), device=DEV, dtype=torch.uint8)))
    w = w.reshape(-1, 16, nb // 8, 8, size).transpose(1, 2)  # tile, k-block, row, block, byte
    codes = w[..., 2:]
    if kind == "Q8_0":
        codes = codes.unflatten(3, (4, 2)).unflatten(5, (4, 8))  # t b j c s G i
    else:
        codes = codes.unflatten(3, (2, 4)).unflatten(5, (4, 4))
    codes = codes.permute(0, 1, 3, 5, 2, 4, 6).flatten(2)  # t b (c G j s i)
    return torch.cat((codes, w[..., :2].flatten(2)), dim=-1).reshape(-1)


def _unpacked(kind, p, N, K):
    """The native blocks [N, K/32, bytes] back out of the repacked order."""
    size = BLOCK[kind][0]
    rec = p.reshape(-1, K // 256, 16 * 8 * size)
    at = 16 * 8 * (size - 2)
    d = rec[..., at:].unflatten(2, (16, 8, 2))
    if kind == "Q8_0":
        codes = rec[..., :at].unflatten(2, (4, 4, 16, 2, 8))  # t b c G j s i
    else:
        codes = rec[..., :at].unflatten(2, (2, 4, 16, 4, 4))
    codes = codes.permute(0, 1, 4, 2, 5, 3, 6).flatten(5).flatten(3, 4)  # t b j (c s) (G i)
    return torch.cat((d, codes), dim=-1).transpose(1, 2).reshape(-1, K // 32, size)[:N]


def _half(b):
    return b.contiguous().view(F16).float()


def _values(kind, w):
    """The blocks' values [N, K] in f32."""
    if kind == "Q8_0":
        v = _half(w[..., :2]) * w[..., 2:].contiguous().view(torch.int8).float()
    elif kind == "Q4_0":
        q = w[..., 2:]
        v = _half(w[..., :2]) * (torch.cat((q & 15, q >> 4), dim=-1).float() - 8)
    elif kind == "Q4_K":
        s, q = w[..., 4:16], w[..., 16:].unflatten(-1, (4, 32))
        a, b, c = s[..., :4], s[..., 4:8], s[..., 8:]
        sc = torch.cat((a & 63, (c & 15) | ((a >> 6) << 4)), dim=-1).float()
        m = torch.cat((b & 63, (c >> 4) | ((b >> 6) << 4)), dim=-1).float()
        q = torch.stack((q & 15, q >> 4), dim=-2).flatten(-3, -2).float()  # eight sub-blocks of 32
        v = (_half(w[..., :2]) * sc).unsqueeze(-1) * q - (_half(w[..., 2:4]) * m).unsqueeze(-1)
        v = v.flatten(-2)
    else:
        ql, qh = w[..., :128].unflatten(-1, (2, 2, 32)), w[..., 128:192].unflatten(-1, (2, 1, 32))
        low = torch.cat((ql & 15, ql >> 4), dim=-2)  # [half, quarter, 32]
        high = torch.cat((qh & 3, (qh >> 2) & 3, (qh >> 4) & 3, qh >> 6), dim=-2)
        q = (low | (high << 4)).float() - 32
        sc = w[..., 192:208].contiguous().view(torch.int8).float()
        v = ((_half(w[..., 208:]) * sc).unsqueeze(-1) * q.flatten(-3).unflatten(-1, (16, 16))).flatten(-2)
    return v.flatten(1)


# ---------------------------------------------------------------------------
# What a program has in hand
# ---------------------------------------------------------------------------
def _rows(T, D, dtype, g, spread=0.5):
    """Hidden states: channels of different sizes, a few far larger than the others."""
    x = torch.randn((T, D), generator=g, device=DEV)
    x *= torch.exp(spread * torch.randn((1, D), generator=g, device=DEV))
    return x.to(_dt(dtype))


def prepare(case, seed):
    c = dict(case)
    s = {"c": c}
    g = _gen(seed, 1)
    if c["op"] == "norm":
        if c["H"] > 1:  # the first heads of a projection's output that holds as many again behind them
            x = _rows(c["T"], 2 * c["H"] * c["D"], c["x"], g)
            s["x"] = x[:, :c["H"] * c["D"]].unflatten(1, (c["H"], c["D"]))
        else:
            s["x"] = _rows(c["T"], c["D"], c["x"], g)
        s["res"] = None if c["res"] == "none" else _rows(c["T"], c["D"], c["res"], g, 1.0)
        s["w"] = 1 + 0.2 * torch.randn((c["D"],), generator=g, device=DEV)
    elif c["op"] == "i8":
        s["x"] = _rows(c["T"], c["D"], c["x"], g)
        s["res"] = None if c["res"] == "none" else _rows(c["T"], c["D"], c["res"], g, 1.0)
        s["w"] = 1 + 0.2 * torch.randn((c["D"],), generator=g, device=DEV)
        s["W"] = _repacked(c["kind"], _weights(c["kind"], c["N"], c["D"], seed))
        s["bias"] = torch.randn((c["N"],), generator=g, device=DEV) if c["bias"] else None
    elif c["op"] == "route":
        s["logits"] = (2 * torch.randn((c["M"], c["E"]), generator=g, device=DEV)).to(_dt(c["dtype"]))
        s["bias"] = 0.1 * torch.randn((c["E"],), generator=g, device=DEV) if c["bias"] else None
        s["slots"] = None
        if c["pad"]:
            s["slots"] = torch.arange(c["M"], device=DEV, dtype=torch.int32)
            s["slots"][c["M"] - c["pad"]:] = -1
    else:
        s["A"] = _rows(c["M"], c["K"], c["a"], g)
        W = _weights(c["kind"], c["N"], c["K"], seed)
        s["W"] = _repacked(c["kind"], W) if c["packed"] else W.reshape(-1)
        s["bias"] = torch.randn((c["N"],), generator=g, device=DEV) if c["bias"] else None
        for name in ("mul", "res"):
            s[name] = None if c[name] == "none" else torch.randn((c["M"], c["N"]), generator=g, device=DEV).to(_dt(c[name]))
    return s


# ---------------------------------------------------------------------------
# One pass
# ---------------------------------------------------------------------------
def _norm(x, res, w):
    """The sum and its norm.  The mean of the squares and the product in 64 bits: what the 8-bit form rounds next lies
    beside borders."""
    h = x.float() if res is None else x.float() + res.float()
    h2 = h.double()
    return h, (h2 * torch.rsqrt(h2.square().mean(-1, keepdim=True) + EPS) * w.double()).float()


def _activated(act, v):
    if act == "relu":
        return torch.clamp(v, min=0)
    if act == "silu":
        return v / (1 + torch.exp(-v))
    if act == "gelu":
        return 0.5 * v * (1 + torch.erf(v * math.sqrt(0.5)))
    if act == "gelu_tanh":
        return 0.5 * v * (1 + torch.tanh(math.sqrt(2 / math.pi) * (v + 0.044715 * v * v * v)))
    return v


def _in_eight_bits(y):
    """The values that 8 bits a piece and a scale per 32 keep of y."""
    y = y.unflatten(-1, (-1, 32))
    d = (y.abs().amax(-1, keepdim=True).double() / 127).float()
    q = torch.where(d == 0, 0.0, torch.round((y.double() / torch.where(d == 0, 1.0, d.double())).float()))
    return (q * d).flatten(-2)


def _route(s, c):
    l = s["logits"].float()
    # In 64 bits where scores are added to something: values that differ by less than f32 holds decide the choice.
    sc = torch.sigmoid(l.double()) if c["score"] == "sigmoid" else torch.softmax(l.double(), -1)
    pick = sc if s["bias"] is None else sc + s["bias"].double()
    if c["groups"] > 1:
        in_groups = pick.unflatten(-1, (c["groups"], -1))
        best = in_groups.sort(dim=-1, descending=True).values[..., :c["top"]].sum(-1)
        kept = best.sort(dim=-1, descending=True, stable=True).indices[:, :c["keep"]]
        on = torch.zeros_like(best, dtype=torch.bool).scatter(1, kept, True)
        pick = torch.where(on.unsqueeze(-1), in_groups, -math.inf).flatten(-2)
    ids = pick.sort(dim=-1, descending=True, stable=True).indices[:, :c["k"]]
    w = sc.gather(1, ids)
    if c["norm"]:
        w = w / w.sum(-1, keepdim=True)
    w = w * c["scale"]
    if s["slots"] is not None:
        skipped = (s["slots"] < 0).unsqueeze(-1)
        ids, w = torch.where(skipped, -1, ids), torch.where(skipped, 0.0, w)
    return {"ids": ids.to(torch.int32), "weights": w.float()}


def run(s):
    c = s["c"]
    if own:
        return _run_own(s, c)
    if c["op"] == "norm":
        h, y = _norm(s["x"], s["res"], s["w"])
        y = y.to(_dt(c["out"]))
        return {"y": y} if s["res"] is None else {"y": y, "sum": h.to(_dt(c["res"]))}
    if c["op"] == "i8":
        h, y = _norm(s["x"], s["res"], s["w"])
        v = torch.matmul(_in_eight_bits(y), _values(c["kind"], _unpacked(c["kind"], s["W"], c["N"], c["D"])).t())
        v = _activated(c["act"], v if s["bias"] is None else v + s["bias"])
        return {"y": v} if s["res"] is None else {"y": v, "sum": h.to(_dt(c["res"]))}
    if c["op"] == "route":
        return _route(s, c)
    blocks = _unpacked(c["kind"], s["W"], c["N"], c["K"]) if c["packed"] else s["W"].reshape(c["N"], -1, BLOCK[c["kind"]][0])
    v = torch.matmul(s["A"].float(), _values(c["kind"], blocks).t())
    v = _activated(c["act"], v if s["bias"] is None else v + s["bias"])
    if s["mul"] is not None:
        v = v * s["mul"].float()
    if s["res"] is not None:
        v = v + s["res"].float()
    return v.to(_dt(c["out"]))


def _run_own(s, c):
    import gguf_block_quantized_kind_amd as qmm
    if c["op"] == "norm":
        got = qmm.rmsnorm(s["x"], s["w"], EPS, residual=s["res"], out_dtype=_dt(c["out"]))
        return {"y": got} if s["res"] is None else {"y": got[0], "sum": got[1]}
    if c["op"] == "i8":
        got = qmm.rmsnorm_q8(c["kind"], s["x"], s["w"], EPS, residual=s["res"])
        acts, h = (got, None) if s["res"] is None else got
        y = qmm.gemv_q8(c["kind"], s["W"], acts, c["N"], bias=s["bias"], act=c["act"])
        return {"y": y} if h is None else {"y": y, "sum": h}
    if c["op"] == "route":
        ids, w = qmm.moe_route(s["logits"], c["k"], score=c["score"], bias=s["bias"], n_group=c["groups"],
                               topk_group=c["keep"], group_top=c["top"], normalize=c["norm"], scale=c["scale"],
                               slots=s["slots"])
        return {"ids": ids, "weights": w}
    product = qmm.matmul_packed_ep if c["packed"] else qmm.matmul_ep
    return product(c["kind"], s["W"], s["A"], c["N"], bias=s["bias"], act=c["act"], mul=s["mul"], residual=s["res"],
                   out_dtype=_dt(c["out"]))


# ---------------------------------------------------------------------------
# The definitions in 64 bits
# ---------------------------------------------------------------------------
def _exact_values(kind, w):
    """Values [N, K] in 64 bits, element by element: where each element's bits lie, and its block's rule."""
    N, nb, _ = w.shape
    e = torch.arange(BLOCK[kind][1], device=DEV)

    def at(i):
        return w[:, :, i].long()

    def half(i):
        return w[:, :, i:i + 2].contiguous().view(F16).double()

    def signed(x):
        return torch.where(x > 127, x - 256, x)

    if kind == "Q8_0":
        v = half(0) * signed(at(2 + e))
    elif kind == "Q4_0":
        v = half(0) * (((at(2 + e % 16) >> (4 * (e // 16))) & 15) - 8)
    elif kind == "Q4_K":
        j = e // 32
        q = (at(16 + 32 * (e // 64) + e % 32) >> (4 * (j % 2))) & 15
        low, top = at(4 + j % 4), at(8 + j % 4)
        both = at(12 + j % 4)
        sc = torch.where(j < 4, low & 63, (both & 15) + 16 * (low >> 6))
        m = torch.where(j < 4, top & 63, (both >> 4) + 16 * (top >> 6))
        v = half(0) * sc * q - half(2) * m
    else:
        h, r = e // 128, e % 128
        q = (at(64 * h + r % 64) >> (4 * (r // 64))) & 15
        q = q + 16 * ((at(128 + 32 * h + r % 32) >> (2 * (r // 32))) & 3) - 32
        v = half(208) * signed(at(192 + e // 16)) * q
    return v.reshape(N, -1)


def _exact_act(act, v):
    zero = torch.zeros((), dtype=F64, device=DEV)
    if act == "relu":
        return torch.maximum(v, zero)
    if act == "silu":
        return v * torch.sigmoid(v)
    if act == "gelu":
        return v * torch.special.ndtr(v)
    if act == "gelu_tanh":
        return v * torch.sigmoid(2 * math.sqrt(2 / math.pi) * (v + 0.044715 * v ** 3))
    return v


def _exact_norm(s):
    h = s["x"].double()
    if s["res"] is not None:
        h = (h + s["res"].double()).float().double()  # the sum is a number in f32
    size = torch.sqrt((h * h).sum(-1, keepdim=True) / h.shape[-1] + EPS)
    return h, h / size * s["w"].double()


def _exact_route(c, l, bias):
    l = l.double()
    if c["score"] == "sigmoid":
        sc = 1 / (1 + torch.exp(-l))
    else:
        sc = torch.exp(l - l.amax(-1, keepdim=True))
        sc = sc / sc.sum(-1, keepdim=True)
    pick = sc if bias is None else sc + bias.double()

    def place(v):  # how many come before each one
        i = torch.arange(v.shape[-1], device=DEV)
        a, b = v.unsqueeze(-1), v.unsqueeze(-2)
        return ((b > a) | ((b == a) & (i < i.unsqueeze(-1)))).sum(-1)

    if c["groups"] > 1:
        g = pick.reshape(l.shape[0], c["groups"], -1)
        best = torch.where(place(g) < c["top"], g, 0.0).sum(-1)
        pick = torch.where((place(best) < c["keep"]).unsqueeze(-1), g, -math.inf).reshape(l.shape)
    p = place(pick)
    ids = torch.where(p < c["k"], p, c["k"])
    ids = torch.zeros((l.shape[0], c["k"] + 1), dtype=torch.long, device=DEV).scatter(
        1, ids, torch.arange(c["E"], device=DEV).expand(l.shape).contiguous())[:, :c["k"]]
    w = torch.take_along_dim(sc, ids, 1)
    if c["norm"]:
        w = w / w.sum(1, keepdim=True)
    return ids.to(torch.int32), w * c["scale"]


def exact(case, seed):
    c = dict(case)
    s = prepare(c, seed)
    if c["op"] == "norm":
        h, y = _exact_norm(s)
        return {"y": y} if s["res"] is None else {"y": y, "sum": h}
    if c["op"] == "route":
        parts = [_exact_route(c, l, s["bias"]) for l in s["logits"].split(max(1, (1 << 26) // (c["E"] * c["E"])))]
        ids, w = (torch.cat(x) for x in zip(*parts))
        live = c["M"] - c["pad"]
        ids[live:], w[live:] = -1, 0
        return {"ids": ids, "weights": w}
    if c["op"] == "i8":
        h, y = _exact_norm(s)
        # What is kept of each 32: the numbers are defined with a scale and a quotient in f32.
        b = y.float().reshape(c["T"], -1, 32).double()
        d = (b.abs().max(-1, keepdim=True).values / 127).float().double()
        q = torch.where(d > 0, (b / torch.where(d > 0, d, 1.0)).float().double(), 0.0).round()
        v = torch.matmul((q * d).reshape(c["T"], -1),
                         _exact_values(c["kind"], _weights(c["kind"], c["N"], c["D"], seed)).t().contiguous())
        v = _exact_act(c["act"], v if s["bias"] is None else v + s["bias"].double())
        return {"y": v} if s["res"] is None else {"y": v, "sum": h}
    W = _exact_values(c["kind"], _weights(c["kind"], c["N"], c["K"], seed))
    v = torch.matmul(s["A"].double(), W.t().contiguous())
    if s["bias"] is not None:
        v = v + s["bias"].double()
    v = _exact_act(c["act"], v)
    if s["mul"] is not None:
        v = v * s["mul"].double()
    return v if s["res"] is None else v + s["res"].double()
