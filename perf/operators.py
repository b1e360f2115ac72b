"""The attention-side operators of a decode step, for measurement: rotary positions, the block-quantised paged
key/value cache (written and read back), the fused append of a step's new tokens, and attention of one new token
per sequence over that cache.

``run`` makes either the library's calls (``own``) or the same results from elementary torch operations.  Both work
on the same bytes: the cache pages in the library's layout, which the functions under "The cache's layout" spell out
with views and permutations.
"""
import math
import random

import torch

own = False

DEV = "cuda"
F16, F32 = torch.float16, torch.float32


# ---------------------------------------------------------------------------
# Cases
# ---------------------------------------------------------------------------
def listed():
    return [
        # One token's 32 query and 8 key heads: a launch's latency.
        dict(name="rope_1_token", op="rope", T=1, H=40, D=128, n_rot=128, layout="half", dtype="f16", out="f16",
             yarn=1.0, far=4096),
        # Half of each head rotated, interleaved pairs, f32 projections, positions up to a million.
        dict(name="rope_partial_far", op="rope", T=777, H=9, D=96, n_rot=48, layout="interleaved", dtype="f32",
             out="f32", yarn=1.0, far=1000000),
        # A prompt's queries, f32 as the GEMM leaves them, f16 for attention, a context stretched eight times.
        dict(name="rope_prompt", op="rope", T=8192, H=32, D=128, n_rot=128, layout="half", dtype="f32", out="f16",
             yarn=8.0, far=131072),
        # A prompt of odd length quantised into the cache and read back.
        dict(name="cache_prompt", op="cache", T=5003, n_kv=8, D=128, k_kind="Q8_0", v_kind="Q4_0", page=64,
             dtype="f16", out="f32", scattered=False),
        # A long prompt in four bits: the largest write.
        dict(name="cache_large", op="cache", T=32768, n_kv=8, D=128, k_kind="Q4_0", v_kind="Q4_0", page=256,
             dtype="f32", out="f16", scattered=False),
        # One sequence's decode step: rotate q and k, write one token.
        dict(name="append_1_token", op="append", T=1, n_q=32, n_kv=8, D=128, n_rot=128, layout="half",
             k_kind="Q8_0", v_kind="Q8_0", page=64, dtype="f16", scattered=True, far=4096),
        # A batch of sequences, each at its own place in the cache; small heads, f32 projections.
        dict(name="append_batch", op="append", T=131, n_q=64, n_kv=8, D=64, n_rot=64, layout="half", k_kind="F16",
             v_kind="Q4_0", page=32, dtype="f32", scattered=True, far=131072),
        # One short chat, full-precision cache: latency.
        dict(name="attn_1_short", op="attn", B=1, L=1000, n_q=32, n_kv=8, D=128, k_kind="F16", v_kind="F16",
             page=64, dtype="f16", window=0, sinks=False),
        # One very long context: the split over the length carries it.
        dict(name="attn_1_long", op="attn", B=1, L=131071, n_q=32, n_kv=8, D=128, k_kind="Q8_0", v_kind="Q8_0",
             page=256, dtype="f16", window=0, sinks=False),
        # A serving batch of ragged lengths, keys in eight and values in four bits.
        dict(name="attn_batch", op="attn", B=64, L=8192, n_q=32, n_kv=8, D=128, k_kind="Q8_0", v_kind="Q4_0",
             page=64, dtype="f16", window=0, sinks=False),
        # One key head per query head, f32 queries and results.
        dict(name="attn_mha_f32", op="attn", B=16, L=4001, n_q=32, n_kv=32, D=128, k_kind="F16", v_kind="F16",
             page=32, dtype="f32", window=0, sinks=False),
        # Small heads in groups of eight, four-bit cache, a sliding window and a sink logit per head.
        dict(name="attn_window_sinks", op="attn", B=48, L=20000, n_q=64, n_kv=8, D=64, k_kind="Q4_0",
             v_kind="Q4_0", page=128, dtype="f16", window=4096, sinks=True),
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(("rope", "cache", "append", "attn", "attn"))
    D = rng.choice((64, 96, 128, 128, 192, 256))
    kinds = ("F16", "Q8_0", "Q4_0")
    page = rng.choice((32, 64, 128, 256))
    if op == "rope":
        H = rng.randint(1, 64)
        T = _log(rng, 1, max(1, (1 << 25) // (H * D)))
        return dict(op=op, T=T, H=H, D=D, n_rot=rng.choice((D, D, D // 2, 2 * rng.randint(1, D // 2))),
                    layout=rng.choice(("half", "interleaved")), dtype=rng.choice(("f16", "f32")),
                    out=rng.choice(("f16", "f32")), yarn=rng.choice((1.0, 4.0, 8.0)), far=_log(rng, 64, 1000000))
    if op == "cache":
        n_kv = rng.randint(1, 16)
        return dict(op=op, T=_log(rng, 1, max(1, (1 << 24) // (n_kv * D))), n_kv=n_kv, D=D,
                    k_kind=rng.choice(kinds), v_kind=rng.choice(kinds), page=page, dtype=rng.choice(("f16", "f32")),
                    out=rng.choice(("f16", "f32")), scattered=rng.random() < 0.25)
    if op == "append":
        n_kv = rng.randint(1, 8)
        n_q = n_kv * rng.randint(1, 8)
        return dict(op=op, T=_log(rng, 1, 2048), n_q=n_q, n_kv=n_kv, D=D, n_rot=rng.choice((D, D // 2)),
                    layout=rng.choice(("half", "interleaved")), k_kind=rng.choice(("F16", "Q8_0")),
                    v_kind=rng.choice(kinds), page=page, dtype=rng.choice(("f16", "f32")),
                    scattered=rng.random() < 0.5, far=_log(rng, 64, 1000000))
    n_kv = rng.choice((1, 2, 4, 8, 8, 16))
    n_q = n_kv * rng.choice((1, 2, 4, 7, 8, 16))
    B = _log(rng, 1, 64)
    L = _log(rng, 16, min(131072, max(64, (1 << 27) // (B * n_kv * D))))
    return dict(op=op, B=B, L=L, n_q=n_q, n_kv=n_kv, D=D, k_kind=rng.choice(kinds), v_kind=rng.choice(kinds),
                page=page, dtype=rng.choice(("f16", "f16", "f32")),
                window=rng.choice((0, 0, max(1, L // 3))), sinks=rng.random() < 0.3)


def _lens(c):
    """The sequences' lengths: the longest first, then spread over the range, an empty row and a row of one among
    them."""
    L = [c["L"]] + [int(c["L"] * ((b * 0.6180339887) % 1.0)) for b in range(1, c["B"])]
    if c["B"] >= 8:
        L[3], L[5] = 0, 1
    return L


def _row_bytes(kind, D):
    return D * 2 if kind == "F16" else D // 32 * (34 if kind == "Q8_0" else 18)


def work(c):
    size = {"f16": 2, "f32": 4}
    if c["op"] == "rope":
        n = c["T"] * c["H"] * c["D"]
        return {"bytes": n * (size[c["dtype"]] + size[c["out"]]) + 4 * c["T"] + 4 * c["n_rot"],
                "flops": 3 * c["T"] * c["H"] * c["n_rot"]}
    if c["op"] == "attn":
        seen = sum(min(n, c["window"]) if c["window"] else n for n in _lens(c))
        rows = _row_bytes(c["k_kind"], c["D"]) + _row_bytes(c["v_kind"], c["D"])
        return {"bytes": seen * c["n_kv"] * rows + 2 * c["B"] * c["n_q"] * c["D"] * size[c["dtype"]],
                "flops": 4 * seen * c["n_q"] * c["D"]}
    n = c["T"] * c["n_kv"] * c["D"]
    rows = c["T"] * c["n_kv"] * (_row_bytes(c["k_kind"], c["D"]) + _row_bytes(c["v_kind"], c["D"]))
    if c["op"] == "cache":
        return {"bytes": 2 * n * (size[c["dtype"]] + size[c["out"]]) + 2 * rows, "flops": 8 * n}
    nq = c["T"] * c["n_q"] * c["D"]
    return {"bytes": 2 * n * (size[c["dtype"]] + 2) + 2 * rows + 2 * nq * size[c["dtype"]], "flops": 3 * nq + 11 * n}


# ---------------------------------------------------------------------------
# The cache's layout: [page][kv head][group of 32 tokens][codes of D/32 blocks, then f16 scales [D/32][32]]
# ---------------------------------------------------------------------------
def _codes(kind, x):
    """Codes and f16 scales of values x [..., D], 32 elements to a block."""
    if kind == "F16":
        return x.to(F16), None
    x = x.float().unflatten(-1, (-1, 32))
    hi, lo = x.amax(-1), x.amin(-1)
    # (A tensor divisor: torch multiplies by the reciprocal of a number.)
    d = torch.maximum(hi, -lo) / torch.full((), 127.0 if kind == "Q8_0" else 8.0, device=x.device)
    h = d.to(F16).clamp(max=65504.0)
    up = (h.float() < d) & (h < 65504.0)
    h = (h.view(torch.int16) + up.to(torch.int16)).view(F16)  # rounded up: no code leaves its range
    if kind == "Q4_0":
        h = torch.where((hi >= -lo) & (h != 0), -h, h)
    q = torch.round(x / torch.where(h == 0, torch.ones_like(h), h).float().unsqueeze(-1))
    q = torch.where((h == 0).unsqueeze(-1), torch.zeros_like(q), q)
    q = q.clamp(-127, 127) + 128 if kind == "Q8_0" else (q + 8).clamp(0, 15)
    return q.to(torch.uint8).flatten(-2), h


def _values(kind, codes, h):
    if kind == "F16":
        return codes.float()
    off = 128.0 if kind == "Q8_0" else 8.0
    return ((codes.float() - off).unflatten(-1, (-1, 32)) * h.float().unsqueeze(-1)).flatten(-2)


def _to_bytes(kind, is_v, codes, h):
    """Page bytes [n, page_bytes] of codes [n, H, P, D] and scales [n, H, P, D/32]."""
    n, H, P, D = codes.shape
    x = codes.reshape(n, H, P // 32, 32, D // 32, 32)
    if not is_v:  # token = 8a + 4m + r, element = (x, G, e)
        x = x.unflatten(3, (4, 2, 4))  # n H g a m r b c
        if kind == "F16":
            x = x.unflatten(7, (4, 8)).permute(0, 1, 2, 6, 4, 7, 3, 5, 8)  # b m G a r e
        elif kind == "Q8_0":
            x = x.unflatten(7, (4, 8)).permute(0, 1, 2, 6, 7, 3, 5, 4, 8)  # b G a r m e
        else:
            x = x.unflatten(7, (2, 4, 4)).permute(7, 0, 1, 2, 6, 8, 3, 5, 4, 9)  # x | b G a r m e
            x = x[0] | (x[1] << 4)
    else:  # token = 8G + e, element = 16x + j
        x = x.unflatten(3, (4, 8)).unflatten(6, (2, 16))  # n H g G e b x j
        if kind == "F16":
            x = x.permute(0, 1, 2, 5, 6, 3, 7, 4)  # b x G j e
        elif kind == "Q8_0":
            x = x.permute(0, 1, 2, 5, 3, 7, 6, 4)  # b G j x e
        else:
            x = x.permute(6, 0, 1, 2, 5, 3, 7, 4)  # x | b G j e
            x = x[0] | (x[1] << 4)
    x = x.contiguous().view(torch.uint8).reshape(n, H, P // 32, -1)
    if kind != "F16":
        s = h.reshape(n, H, P // 32, 32, D // 32).transpose(3, 4).contiguous().view(torch.uint8)
        x = torch.cat((x, s.reshape(n, H, P // 32, -1)), dim=-1)
    return x.reshape(n, -1)


def _from_bytes(kind, is_v, pages, H, P, D):
    """Values [n, H, P, D] in f32 of page bytes [n, page_bytes]."""
    n, NB = pages.shape[0], D // 32
    x = pages.reshape(n, H, P // 32, -1)
    h = None
    if kind != "F16":
        at = x.shape[-1] - NB * 64
        h = x[..., at:].contiguous().view(F16).reshape(n, H, P // 32, NB, 32).transpose(3, 4).reshape(n, H, P, NB)
        x = x[..., :at]
    x = x.contiguous()
    if kind == "F16":
        x = x.view(F16)
    elif kind == "Q4_0":
        x = torch.stack((x & 15, x >> 4))
    s = (n, H, P // 32, NB)
    if not is_v:
        if kind == "F16":
            x = x.reshape(*s, 2, 4, 4, 4, 8).permute(0, 1, 2, 6, 4, 7, 3, 5, 8)  # n H g a m r b G e
        elif kind == "Q8_0":
            x = x.reshape(*s, 4, 4, 4, 2, 8).permute(0, 1, 2, 5, 7, 6, 3, 4, 8)
        else:
            x = x.reshape(2, *s, 4, 4, 4, 2, 4).permute(1, 2, 3, 6, 8, 7, 4, 0, 5, 9)  # n H g a m r b x G e
    else:
        if kind == "F16":
            x = x.reshape(*s, 2, 4, 16, 8).permute(0, 1, 2, 5, 7, 3, 4, 6)  # n H g G e b x j
        elif kind == "Q8_0":
            x = x.reshape(*s, 4, 16, 2, 8).permute(0, 1, 2, 4, 7, 3, 6, 5)
        else:
            x = x.reshape(2, *s, 4, 16, 8).permute(1, 2, 3, 5, 7, 4, 0, 6)
    return _values(kind, x.reshape(n, H, P, D), h)


def _places(kind, is_v, slots, H, P, D):
    """Where a token's codes and scales lie: element indices into the pages as codes (halves for F16, else bytes)
    [T, H, D] (D/2 bytes of two elements for Q4_0) and into the pages as halves for the scales [T, H, D/32]."""
    NB = D // 32
    row = _row_bytes(kind, D)
    s = slots.long()
    head = torch.arange(H, device=s.device)
    group = ((s // P)[:, None] * H + head) * (P // 32) + ((s % P) // 32)[:, None]  # [T, H]
    r = (s % 32)[:, None]
    b = torch.arange(NB, device=s.device)[:, None]
    c = torch.arange(16 if kind == "Q4_0" else 32, device=s.device)
    if not is_v:
        i, m = 4 * (r // 8) + r % 4, (r // 4) % 2
        i, m = i[:, :, None], m[:, :, None]
        if kind == "F16":
            at = ((b * 2 + m) * 4 + c // 8) * 128 + i * 8 + c % 8
        elif kind == "Q8_0":
            at = b * 1024 + ((c // 8 * 16 + i) * 2 + m) * 8 + c % 8
        else:
            at = b * 512 + ((c // 4 * 16 + i) * 2 + m) * 4 + c % 4
    else:
        G, e = (r // 8)[:, :, None], (r % 8)[:, :, None]
        if kind == "F16":
            at = ((b * 2 + c // 16) * 4 + G) * 128 + c % 16 * 8 + e
        elif kind == "Q8_0":
            at = b * 1024 + ((G * 16 + c % 16) * 2 + c // 16) * 8 + e
        else:
            at = b * 512 + (G * 16 + c) * 8 + e
    unit = row * 32 // (2 if kind == "F16" else 1)
    at = group[:, :, None] * unit + at.reshape(s.shape[0], 1, -1)
    if kind == "F16":
        return at, None
    codes = NB * (1024 if kind == "Q8_0" else 512)
    return at, group[:, :, None] * (row * 16) + codes // 2 + b[:, 0] * 32 + r[:, :, None]


def _write(kind, is_v, pages, slots, x, P):
    T, H, D = x.shape
    codes, h = _codes(kind, x)
    at, sat = _places(kind, is_v, slots, H, P, D)
    if kind == "F16":
        pages.view(-1).view(F16)[at.view(-1)] = codes.reshape(-1)
        return
    if kind == "Q4_0":
        codes = codes.unflatten(-1, (-1, 2, 16))
        codes = (codes[..., 0, :] | (codes[..., 1, :] << 4)).flatten(-2)
    pages.view(-1)[at.view(-1)] = codes.reshape(-1)
    pages.view(-1).view(F16)[sat.reshape(-1)] = h.reshape(-1)


def _read(kind, is_v, pages, slots, H, P, D, out):
    at, sat = _places(kind, is_v, slots, H, P, D)
    if kind == "F16":
        return pages.view(-1).view(F16)[at].to(out)
    codes = pages.view(-1)[at]
    if kind == "Q4_0":
        codes = codes.unflatten(-1, (-1, 1, 16))
        codes = torch.cat((codes & 15, codes >> 4), dim=-2).flatten(-3)
    return _values(kind, codes, pages.view(-1).view(F16)[sat]).to(out)


# ---------------------------------------------------------------------------
# What a program has in hand
# ---------------------------------------------------------------------------
def _gen(seed, what):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed * 16 + what)
    return g


def _dt(name):
    return {"f16": F16, "f32": F32}[name]


def _freqs(n_rot, yarn):
    """Radians per position of each pair, and the factor on the rotated elements (a context stretched `yarn` times
    from 4096 positions)."""
    i = torch.arange(n_rot // 2, dtype=torch.float64)
    f = 10000.0 ** (-2 * i / n_rot)
    if yarn == 1.0:
        return f.to(DEV), 1.0
    turns = [n_rot * math.log(4096 / (beta * 2 * math.pi)) / (2 * math.log(10000.0)) for beta in (32.0, 1.0)]
    low, high = max(math.floor(turns[0]), 0), min(math.ceil(turns[1]), n_rot - 1)
    ramp = ((i - low) / max(high - low, 0.001)).clamp(0, 1)
    return (f * (1 - ramp) + f / yarn * ramp).to(DEV), 0.1 * math.log(yarn) + 1.0


def _token_slots(c, seed):
    """Distinct slots of T tokens: a prompt fills whole pages in random order from some place inside the first one,
    a batch has each token in a page of its own."""
    r = random.Random(seed)
    T, P = c["T"], c["page"]
    if c["scattered"]:
        n = T + 3
        pages = r.sample(range(n), T)
        return [p * P + r.randrange(P) for p in pages], n
    first = r.randrange(P)
    n = (first + T + P - 1) // P + 2
    order = r.sample(range(n), n)
    return [order[(first + t) // P] * P + (first + t) % P for t in range(T)], n


def _kv_inputs(c, seed):
    g, dt = _gen(seed, 1), _dt(c["dtype"])
    n_q = c.get("n_q", 0)
    # One projection's result holds q, k and v side by side: the operators get strided views of it.
    row = (n_q + 2 * c["n_kv"]) * c["D"]
    x = torch.randn((c["T"], row), generator=g, device=DEV)
    x *= torch.exp(0.5 * torch.randn((1, row), generator=g, device=DEV))  # channels of different sizes
    x = x.to(dt)
    q = x[:, :n_q * c["D"]].unflatten(1, (-1, c["D"])) if n_q else None
    k, v = x[:, n_q * c["D"]:].unflatten(1, (2, c["n_kv"], c["D"])).unbind(1)
    return q, k, v


def _contents(c, seed):
    """Codes and scales [n_pages, n_kv, page, D] of a filled cache, the block table and the lengths."""
    P, lens = c["page"], _lens(c)
    pages = [(n + P - 1) // P for n in lens]
    n, wide = sum(pages) + 2, max(1, max(pages))
    order = random.Random(seed).sample(range(n), n)
    table, at = [], 0
    for p in pages:
        table.append(order[at:at + p] + [-1] * (wide - p))
        at += p
    g = _gen(seed, 2)
    parts = []
    for kind, spread in ((c["k_kind"], 0.6), (c["v_kind"], 0.2)):
        x = torch.randn((n, c["n_kv"], P, c["D"]), generator=g, device=DEV)
        x *= torch.exp(spread * torch.randn((1, c["n_kv"], 1, c["D"]), generator=g, device=DEV))
        parts.append(_codes(kind, x))
        del x
    return parts, torch.tensor(table, dtype=torch.int32), lens


def prepare(case, seed):
    c = dict(case)
    s = {"c": c}
    if c["op"] in ("rope", "append"):
        s["freqs"], s["mscale"] = _freqs(c["n_rot"], c.get("yarn", 1.0))
        s["pos"] = torch.randint(0, c["far"], (c["T"],), generator=_gen(seed, 3), device=DEV, dtype=torch.int32)
    if c["op"] == "rope":
        s["x"] = torch.randn((c["T"], c["H"], c["D"]), generator=_gen(seed, 1), device=DEV).to(_dt(c["dtype"]))
    elif c["op"] in ("cache", "append"):
        s["q"], s["k"], s["v"] = _kv_inputs(c, seed)
        slots, n = _token_slots(c, seed)
        s["slots"] = torch.tensor(slots, dtype=torch.int32, device=DEV)
        for name, kind in (("k_pages", c["k_kind"]), ("v_pages", c["v_kind"])):
            s[name] = torch.zeros((n, c["page"] * c["n_kv"] * _row_bytes(kind, c["D"])), dtype=torch.uint8, device=DEV)
    else:
        (k, v), table, lens = _contents(c, seed)
        s["k_pages"] = _to_bytes(c["k_kind"], False, *k)
        s["v_pages"] = _to_bytes(c["v_kind"], True, *v)
        s["table"] = table.to(DEV)
        s["lens"] = torch.tensor(lens, dtype=torch.int32, device=DEV)
        g = _gen(seed, 4)
        s["q"] = torch.randn((c["B"], c["n_q"], c["D"]), generator=g, device=DEV).to(_dt(c["dtype"]))
        s["sinks"] = torch.randn((c["n_q"],), generator=g, device=DEV) if c["sinks"] else None
    return s


# ---------------------------------------------------------------------------
# One pass
# ---------------------------------------------------------------------------
def _rotate(x, pos, freqs, layout, mscale):
    n = 2 * freqs.shape[0]
    phi = pos.double()[:, None] * freqs
    cos, sin = (phi.cos() * mscale).float()[:, None, :], (phi.sin() * mscale).float()[:, None, :]
    x = x.float()
    part = x[..., :n]
    a, b = (part[..., : n // 2], part[..., n // 2:]) if layout == "half" else (part[..., 0::2], part[..., 1::2])
    y = (a * cos - b * sin, a * sin + b * cos)
    y = torch.cat(y, dim=-1) if layout == "half" else torch.stack(y, dim=-1).flatten(-2)
    return torch.cat((y, x[..., n:]), dim=-1)


def _attend(s):
    c = s["c"]
    B, G, D = c["B"], c["n_q"] // c["n_kv"], c["D"]
    at = s["table"].long().clamp(min=0)
    k, v = (_from_bytes(kind, is_v, pages[at].flatten(0, 1), c["n_kv"], c["page"], D)
            .unflatten(0, at.shape).transpose(1, 2).flatten(2, 3)
            for kind, is_v, pages in ((c["k_kind"], False, s["k_pages"]), (c["v_kind"], True, s["v_pages"])))
    q = s["q"].float().reshape(B, c["n_kv"], G, D)
    score = torch.matmul(q, k.transpose(2, 3).contiguous()) / math.sqrt(D)  # [B, n_kv, G, tokens]
    t, n = torch.arange(score.shape[-1], device=DEV), s["lens"].long()[:, None]
    seen = (t < n) & (t >= n - c["window"]) if c["window"] else t < n
    score = torch.where(seen[:, None, None, :], score, -math.inf)
    top = score.amax(-1, keepdim=True)
    if s["sinks"] is not None:
        sink = s["sinks"].reshape(1, c["n_kv"], G, 1)
        top = torch.maximum(top, sink)
    top = torch.where(top == -math.inf, 0.0, top)
    p = torch.exp(score - top)
    total = p.sum(-1, keepdim=True)
    if s["sinks"] is not None:
        total = total + torch.exp(sink - top)
    out = torch.matmul(p, v) / torch.where(total == 0, 1.0, total)
    return out.reshape(B, c["n_q"], D).to(s["q"].dtype)


def run(s):
    c = s["c"]
    if own:
        return _run_own(s, c)
    if c["op"] == "rope":
        return _rotate(s["x"], s["pos"], s["freqs"], c["layout"], s["mscale"]).to(_dt(c["out"]))
    if c["op"] == "attn":
        return _attend(s)
    k, q = s["k"], None
    if c["op"] == "append":
        q = _rotate(s["q"], s["pos"], s["freqs"], c["layout"], s["mscale"]).to(_dt(c["dtype"]))
        k = _rotate(k, s["pos"], s["freqs"], c["layout"], s["mscale"])
    _write(c["k_kind"], False, s["k_pages"], s["slots"], k, c["page"])
    _write(c["v_kind"], True, s["v_pages"], s["slots"], s["v"], c["page"])
    out = _dt(c.get("out", "f16"))
    got = {"k": _read(c["k_kind"], False, s["k_pages"], s["slots"], c["n_kv"], c["page"], c["D"], out),
           "v": _read(c["v_kind"], True, s["v_pages"], s["slots"], c["n_kv"], c["page"], c["D"], out)}
    return got if q is None else {"q": q, **got}


def _run_own(s, c):
    import gguf_block_quantized_kind_amd as qmm
    if c["op"] == "rope":
        return qmm.rope(s["x"], s["pos"], s["freqs"], layout=c["layout"], mscale=s["mscale"], out_dtype=_dt(c["out"]))
    if c["op"] == "attn":
        return qmm.attn_decode(s["q"], s["k_pages"], s["v_pages"], s["table"], s["lens"], c["k_kind"], c["v_kind"],
                               c["page"], c["n_kv"], window=c["window"], sinks=s["sinks"])
    got = {}
    if c["op"] == "append":
        got["q"] = qmm.kv_append(s["q"], s["k"], s["v"], s["pos"], s["slots"], s["k_pages"], s["v_pages"],
                                 c["k_kind"], c["v_kind"], c["page"], s["freqs"], layout=c["layout"],
                                 mscale=s["mscale"])
    else:
        qmm.kv_write(s["k"], s["v"], s["slots"], s["k_pages"], s["v_pages"], c["k_kind"], c["v_kind"], c["page"])
    got["k"], got["v"] = qmm.kv_read(s["slots"], s["k_pages"], s["v_pages"], c["k_kind"], c["v_kind"], c["page"],
                                     c["n_kv"], c["D"], dtype=_dt(c.get("out", "f16")))
    return got


# ---------------------------------------------------------------------------
# The definitions in 64 bits
# ---------------------------------------------------------------------------
def _exact_rope(x, pos, n_rot, layout, yarn):
    freqs, m = _freqs(n_rot, yarn)
    y = x.double().clone()
    phi = (pos.double()[:, None] * freqs).unsqueeze(1)
    pair = torch.arange(n_rot // 2, device=DEV)
    a, b = (pair, pair + n_rot // 2) if layout == "half" else (2 * pair, 2 * pair + 1)
    xa, xb = x.double()[..., a], x.double()[..., b]
    y[..., a] = m * (xa * torch.cos(phi) - xb * torch.sin(phi))
    y[..., b] = m * (xa * torch.sin(phi) + xb * torch.cos(phi))
    return y


def _exact_cache(kind, x):
    x = x.double()
    if kind == "F16":
        return x.to(F16).double()
    blocks = x.unflatten(-1, (-1, 32))
    big = blocks.abs().amax(-1)
    step = big / (127 if kind == "Q8_0" else 8)
    # The smallest f16 number at or above the step.
    h = step.to(F16)
    h = torch.where(h.double() < step, (h.view(torch.int16) + 1).view(F16), h).double()
    if kind == "Q4_0":
        h = torch.where(blocks.amax(-1) == big, -h, h)
    h = h.unsqueeze(-1)
    q = torch.round(blocks / torch.where(h == 0, 1.0, h))
    q = q.clamp(-127, 127) if kind == "Q8_0" else q.clamp(-8, 7)
    return (q * h).flatten(-2)


def exact(case, seed):
    c = dict(case)
    if c["op"] == "attn":
        (k, v), table, lens = _contents(c, seed)
        s = prepare(c, seed)
        G = c["n_q"] // c["n_kv"]
        out = torch.zeros((c["B"], c["n_q"], c["D"]), dtype=torch.float64, device=DEV)

        def rows(kind, part, pages, lo, hi):
            x = part[0][pages].transpose(1, 2).flatten(0, 1)[lo:hi].double()  # [tokens, n_kv, D]
            if kind == "F16":
                return x
            h = part[1][pages].transpose(1, 2).flatten(0, 1)[lo:hi].double()
            return (x - (128 if kind == "Q8_0" else 8)) * h.repeat_interleave(32, dim=-1)

        for b, n in enumerate(lens):
            lo = max(0, n - c["window"]) if c["window"] else 0
            if n == 0:
                continue
            pages = table[b, : (n + c["page"] - 1) // c["page"]].long().to(DEV)
            kk, vv = rows(c["k_kind"], k, pages, lo, n), rows(c["v_kind"], v, pages, lo, n)
            for h in range(c["n_q"]):
                e = torch.mv(kk[:, h // G].contiguous(), s["q"][b, h].double()) / math.sqrt(c["D"])
                top = e.max()
                p = torch.exp(e - top)
                total = p.sum()
                if s["sinks"] is not None:
                    total = total + torch.exp(s["sinks"][h].double() - top)
                out[b, h] = torch.mv(vv[:, h // G].t().contiguous(), p) / total
        return out
    s = prepare(c, seed)
    if c["op"] == "rope":
        return _exact_rope(s["x"], s["pos"], c["n_rot"], c["layout"], c["yarn"])
    k, v = s["k"], s["v"]
    if c["op"] == "cache":
        return {"k": _exact_cache(c["k_kind"], k), "v": _exact_cache(c["v_kind"], v)}
    k = _exact_rope(k, s["pos"], c["n_rot"], c["layout"], 1.0)
    return {"q": _exact_rope(s["q"], s["pos"], c["n_rot"], c["layout"], 1.0),
            "k": _exact_cache(c["k_kind"], k), "v": _exact_cache(c["v_kind"], v)}
