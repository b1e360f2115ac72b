"""Rotary positions, the paged block-quantized key/value cache and attention
of one token over it, on the GPU against the numpy definitions of
oracle/attention.py.

Tolerances (none measured): the cache's bytes and values exactly; a rotation
2^-21 mscale (|x_a| + |x_b|), plus half a step of an f16 result; attention the
header's bound, (r + 2 e) sum w|v|, plus half a step of an f16 result.
"""
import numpy as np
import pytest

import workloads as wl
from oracle import attention as oa

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
import gguf_block_quantized_kind_amd as qmm  # noqa: E402

KINDS = ["F16", "Q8_0", "Q4_0"]
PAIRS = [(k, v) for k in KINDS for v in KINDS]
NP = {"f16": np.float16, "f32": np.float32}


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    qmm.load_library()


def dev(a):
    return torch.from_numpy(np.ascontiguousarray(a)).cuda()


def half_step(y, dt):
    """Half a step of the result's type: 2^-11 |y| and half the smallest f16."""
    return 2.0 ** -11 * np.abs(y) + 2.0 ** -25 if dt == "f16" else 0.0


def check(got, want, tol, what):
    got = got.astype(np.float64)
    assert np.all(np.isfinite(got)), f"{what}: not finite"
    err = np.abs(got - want)
    ratio = np.divide(err, tol, out=np.where(err == 0, 0.0, np.inf), where=tol > 0)
    at = np.unravel_index(np.argmax(ratio), ratio.shape)
    assert ratio[at] <= 1.0, f"{what}: |err| / tol = {ratio[at]:.3g} at {at}: got {got[at]}, want {want[at]}"


# -- rotary positions ----------------------------------------------------------
@pytest.mark.parametrize("layout", ["half", "interleaved"])
@pytest.mark.parametrize("xd,yd", [("f16", "f16"), ("f16", "f32"), ("f32", "f16"), ("f32", "f32")])
@pytest.mark.parametrize("T,H,D,n_rot", [(1, 1, 2, 2), (1, 40, 128, 128), (7, 3, 96, 48), (33, 5, 80, 34), (130, 2, 256, 64)])
def test_rope(layout, xd, yd, T, H, D, n_rot):
    g = wl.rng("rope", f"{layout}{xd}{yd}{T}{D}")
    x = g.normal(size=(T, H + 2, D)).astype(NP[xd])
    pos = g.integers(-5, 1 << 20, T).astype(np.int32)
    pos[0] = 0 if T > 1 else 1 << 20
    freqs, m = qmm.rope_freqs(n_rot, factor=4.0, orig_ctx=4096)
    view = dev(x)[:, 1:1 + H]                                 # a row stride above H * D
    y = qmm.rope(view, dev(pos), freqs, layout, m, out_dtype=getattr(torch, {"f16": "float16", "f32": "float32"}[yd]))
    f = freqs.cpu().numpy()
    want = oa.rope(x[:, 1:1 + H], pos, f, layout, m)
    tol = 2.0 ** -21 * oa.rope_bound(x[:, 1:1 + H], n_rot, layout, m) + half_step(want, yd)
    check(y.cpu().numpy(), want, tol, "rope")
    if xd == yd:                                              # in place, and only the rows given
        buf = dev(x)
        qmm.rope(buf[:, 1:1 + H], dev(pos), freqs, layout, m, out=buf[:, 1:1 + H])
        assert torch.equal(buf[:, 1:1 + H], y)
        assert torch.equal(buf[:, 0], dev(x)[:, 0]) and torch.equal(buf[:, H + 1], dev(x)[:, H + 1])


def test_rope_far_positions():
    """The largest positions and an angle per position above a turn."""
    pos = np.array([2 ** 31 - 1, -2 ** 31, 123456789, 1], np.int32)
    f = np.array([1.0, 1e-3, 7.123456789, 1e-9])
    x = wl.rng("rope", "far").normal(size=(4, 2, 8)).astype(np.float32)
    y = qmm.rope(dev(x), dev(pos), dev(f)).cpu().numpy()
    want = oa.rope(x, pos, f)
    # Beside the bound, the 64-bit angle itself: |phi| 2^-52 of both sides.
    tol = (2.0 ** -21 + np.abs(np.outer(pos.astype(float), f)).max() * 2.0 ** -51) * oa.rope_bound(x, 8)
    check(y, want, tol, "far")


@pytest.mark.parametrize("layout", ["half", "interleaved"])
@pytest.mark.parametrize("D", [8, 2])
def test_rope_turns_by_the_rounded_cosine_and_sine(layout, D):
    """The vector (1, 0) turned is mscale (cos, sin), each rounded once to f32: half a step of the value itself, beside
    the 64-bit angle's |phi| 2^-51 and 2^-35 of the series.  Positions and angles of every size, zeros of both."""
    g = wl.rng("rope", f"unit{layout}{D}")
    pos = np.concatenate([np.arange(700), g.integers(-2 ** 31, 2 ** 31, 300)]).astype(np.int32)
    f = np.exp(g.uniform(np.log(1e-6), np.log(10), D // 2))
    f[0] = np.pi / 8
    x = np.zeros((1000, 1, D), np.float32)
    a = np.arange(D // 2) if layout == "half" else 2 * np.arange(D // 2)
    x[..., a] = 1
    m = np.float32(1.2079442)
    y = qmm.rope(dev(x), dev(pos), dev(f), layout, float(m)).cpu().numpy()
    want, phi = oa.rope(x, pos, f, layout, float(m)), np.zeros((1000, 1, D))
    phi[:, 0, a] = phi[:, 0, a + (D // 2 if layout == "half" else 1)] = np.abs(np.outer(pos.astype(float), f))
    check(y, want, 2.0 ** -24 * np.abs(want) + m * (phi * 2.0 ** -51 + 2.0 ** -35), "unit")


@pytest.mark.parametrize("T,H,D,n_rot,layout", [(1, 40, 128, 128, "half"), (130, 2, 256, 64, "interleaved")])
def test_rope_bound(T, H, D, n_rot, layout):
    """f32 rows within the header's 2^-22 mscale (|x_a| + |x_b|)."""
    g = wl.rng("rope", f"bound{T}")
    x, pos = g.normal(size=(T, H, D)).astype(np.float32), g.integers(0, 1 << 20, T).astype(np.int32)
    freqs, m = qmm.rope_freqs(n_rot, factor=8.0, orig_ctx=4096)
    y = qmm.rope(dev(x), dev(pos), freqs, layout, m).cpu().numpy()
    check(y, oa.rope(x, pos, freqs.cpu().numpy(), layout, m), 2.0 ** -22 * oa.rope_bound(x, n_rot, layout, m), "rope")


# -- writing and reading the cache -----------------------------------------------
def values_for(g, shape, dt):
    """Rows of very different sizes with some far outliers."""
    x = g.normal(size=shape) * np.exp(g.normal(size=shape[:-1] + (1,)) * 2)
    x[..., 0::37] *= 20
    with np.errstate(over="ignore"):
        return x.astype(NP[dt])


def some_slots(g, n_pages, P, T, skip=True):
    s = g.permutation(n_pages * P)[:T].astype(np.int32)
    if skip and T > 3:
        s[1], s[T - 1] = -1, n_pages * P
        s[T // 2] = -2 ** 31
    return s


def run_slots(n_pages, P, start, T):
    """Consecutive tokens through pages in descending order."""
    t = start + np.arange(T)
    return ((n_pages - 1 - t // P) * P + t % P).astype(np.int32)


@pytest.mark.parametrize("kk,vk", PAIRS)
@pytest.mark.parametrize("dt", ["f16", "f32"])
@pytest.mark.parametrize("D,P,H,case", [(128, 64, 2, "random"), (64, 32, 3, "run"), (96, 96, 1, "one"), (256, 32, 2, "run"),
                                        (192, 64, 5, "aligned")])
def test_kv_write_bytes_and_read(kk, vk, dt, D, P, H, case):
    n_pages = 6
    g = wl.rng("kv", f"{kk}{vk}{dt}{D}")
    if case == "random":
        slots = some_slots(g, n_pages, P, 45)
    elif case == "run":
        slots = run_slots(n_pages, P, 13, 101)
        slots[50] = -1
    elif case == "aligned":
        slots = run_slots(n_pages, P, 32, 4 * P)
    else:
        slots = np.array([77], np.int32)
    T = len(slots)
    qkv = values_for(g, (T, 1 + 2 * H, D), dt)
    if T > 4:
        qkv[2] = 0                                             # zero blocks
        qkv[3, :, :32] = 1e-7 if dt == "f32" else 6e-8         # below the smallest scale's range
        qkv[4, :, 32:64] = 60000.0
    x = dev(qkv)
    pages = {s: g.integers(0, 256, (n_pages, oa.page_bytes(k, P, H, D)), dtype=np.uint8) for s, k in (("k", kk), ("v", vk))}
    kp, vp = dev(pages["k"]), dev(pages["v"])
    qmm.kv_write(x[:, 1:1 + H], x[:, 1 + H:], dev(slots), kp, vp, kk, vk, P)
    for s, kind, part in (("k", kk, qkv[:, 1:1 + H]), ("v", vk, qkv[:, 1 + H:])):
        codes, h = oa.quantize(kind, part)
        for t, slot in enumerate(slots):
            if 0 <= slot < n_pages * P:
                oa.store(kind, s == "v", pages[s], P, int(slot), codes[t], None if h is None else h[t])
    same = [np.array_equal(p.cpu().numpy(), pages[s]) for p, s in ((kp, "k"), (vp, "v"))]
    assert same == [True, True]
    for od in ("f32", "f16"):
        got = qmm.kv_read(dev(slots), kp, vp, kk, vk, P, H, D, dtype=getattr(torch, {"f16": "float16", "f32": "float32"}[od]))
        for s, kind, t in (("k", kk, got[0]), ("v", vk, got[1])):
            want = np.zeros((T, H, D))
            for i, slot in enumerate(slots):
                if 0 <= slot < n_pages * P:
                    want[i] = oa.load(kind, s == "v", pages[s], P, int(slot), H, D)
            # An f16 input beyond 65504 is an infinity, whose block reads back as NaN.
            with np.errstate(over="ignore"):
                same = np.array_equal(t.cpu().numpy(), want.astype(NP[od]), equal_nan=True)
            assert same, (s, od)


@pytest.mark.parametrize("kk,vk", [("Q8_0", "Q4_0"), ("F16", "Q8_0"), ("Q4_0", "F16")])
def test_kv_large_calls_equal_small_ones(kk, vk):
    """Sizes whose waves take several heads each: the same bytes and values as calls of 777 tokens."""
    P, H, D, T = 64, 8, 64, 70001
    n_pages = T // P + 3
    g = torch.Generator(device="cuda")
    g.manual_seed(5)
    x = torch.randn((T, 2 * H, D), generator=g, device="cuda").half()
    order = torch.randperm(n_pages, generator=g, device="cuda").int()
    t = torch.arange(T, device="cuda") + 13
    slots = order[t // P] * P + (t % P).int()
    slots[5000] = -1
    pages = [[torch.full((n_pages, oa.page_bytes(k, P, H, D)), 0x33, dtype=torch.uint8, device="cuda") for k in (kk, vk)]
             for _ in range(2)]
    qmm.kv_write(x[:, :H], x[:, H:], slots, *pages[0], kk, vk, P)
    for i in range(0, T, 777):
        qmm.kv_write(x[i:i + 777, :H], x[i:i + 777, H:], slots[i:i + 777], *pages[1], kk, vk, P)
    assert torch.equal(pages[0][0], pages[1][0]) and torch.equal(pages[0][1], pages[1][1])
    k, v = qmm.kv_read(slots, *pages[0], kk, vk, P, H, D)
    for i in range(0, T, 777):
        a, b = qmm.kv_read(slots[i:i + 777], *pages[0], kk, vk, P, H, D)
        assert torch.equal(a, k[i:i + 777]) and torch.equal(b, v[i:i + 777])


@pytest.mark.parametrize("dt", ["f16", "f32"])
def test_odd_strides_and_offsets(dt):
    """Rows at odd element offsets and strides give what packed rows give, in every operator."""
    T, nq, H, D, P = 37, 4, 2, 128, 32
    g = wl.rng("attn", f"odd{dt}")
    x = g.normal(size=(T, nq + 2 * H, D)).astype(NP[dt])
    row = (nq + 2 * H) * D + 3
    buf = torch.zeros(T * row + 1, dtype=getattr(torch, {"f16": "float16", "f32": "float32"}[dt]), device="cuda")
    odd = buf[1:].view(T, row)[:, :row - 3].unflatten(1, (nq + 2 * H, D))
    odd.copy_(dev(x))
    pos, slots = dev(np.arange(T, dtype=np.int32) * 999), dev(g.permutation(4 * P)[:T].astype(np.int32))
    freqs, m = qmm.rope_freqs(D)
    got = []
    for y in (dev(x), odd):
        kp, vp = qmm.kv_pages("Q8_0", 4, P, H, D), qmm.kv_pages("Q4_0", 4, P, H, D)
        kp.zero_()
        vp.zero_()
        q = qmm.kv_append(y[:, :nq], y[:, nq:nq + H], y[:, nq + H:], pos, slots, kp, vp, "Q8_0", "Q4_0", P, freqs, mscale=m)
        r = qmm.rope(y, pos, freqs, "interleaved")
        table, lens = dev(np.arange(4, dtype=np.int32).reshape(1, 4).repeat(T, 0)), dev(np.arange(T, dtype=np.int32) * 3)
        got.append((kp, vp, q, r, qmm.attn_decode(y[:, :nq], kp, vp, table, lens, "Q8_0", "Q4_0", P, H)))
    assert all(torch.equal(a, b) for a, b in zip(*got))


def test_kv_write_nonfinite_blocks():
    g = wl.rng("kv", "nonfinite")
    x = g.normal(size=(3, 2, 64)).astype(np.float32)
    x[0, 0, 5], x[1, 1, 40], x[2, 0, 0] = np.inf, np.nan, -np.inf
    for kind in ("Q8_0", "Q4_0"):
        kp, vp = (qmm.kv_pages(kind, 1, 32, 2, 64) for _ in range(2))
        slots = dev(np.array([3, 9, 31], np.int32))
        qmm.kv_write(dev(x), dev(x), slots, kp, vp, kind, kind, 32)
        for t in qmm.kv_read(slots, kp, vp, kind, kind, 32, 2, 64, dtype=torch.float32):
            nan = np.isnan(t.cpu().numpy()).reshape(3, 2, 2, 32)
            assert nan[0, 0, 0].all() and nan[1, 1, 1].all() and nan[2, 0, 0].all() and nan.sum() == 96


@pytest.mark.parametrize("kk,vk", [("F16", "Q4_0"), ("Q8_0", "Q8_0"), ("Q4_0", "F16")])
@pytest.mark.parametrize("dt,qd", [("f16", "f16"), ("f32", "f16"), ("f32", "f32")])
@pytest.mark.parametrize("T,nq,H,D,n_rot,layout", [(1, 8, 2, 128, 128, "half"), (70, 3, 3, 64, 32, "interleaved"),
                                                   (37, 4, 1, 192, 96, "half"), (300, 4, 2, 96, 96, "half")])
def test_kv_append(kk, vk, dt, qd, T, nq, H, D, n_rot, layout):
    P, n_pages = 64, 7
    g = wl.rng("append", f"{kk}{vk}{dt}{T}")
    x = np.clip(values_for(g, (T, nq + 2 * H, D), dt), -20000, 20000)
    slots = some_slots(g, n_pages, P, T) if T < 100 else run_slots(n_pages, P, 5, T)
    pos = g.integers(0, 100000, T).astype(np.int32)
    freqs, m = qmm.rope_freqs(n_rot, factor=2.0, orig_ctx=1000)
    kp, vp = qmm.kv_pages(kk, n_pages, P, H, D), qmm.kv_pages(vk, n_pages, P, H, D)
    kp.fill_(0x5a)
    vp.fill_(0x5a)
    xt = dev(x)
    q, k, v = xt[:, :nq], xt[:, nq:nq + H], xt[:, nq + H:]
    out = qmm.kv_append(q, k, v, dev(pos), dev(slots), kp, vp, kk, vk, P, freqs, layout, m,
                        out_dtype=getattr(torch, {"f16": "float16", "f32": "float32"}[qd]))
    f = freqs.cpu().numpy()
    want = oa.rope(x[:, :nq], pos, f, layout, m)
    tol = 2.0 ** -21 * oa.rope_bound(x[:, :nq], n_rot, layout, m)
    check(out.cpu().numpy(), want, tol + half_step(want, qd), "q")
    # v's bytes exactly; a value of k within half its block's step (a whole step where a Q4_0 code was cut) of the
    # rotated value, itself known to 2^-21, and steps within one f16 unit of the exact rotated block's.
    pages = np.full((n_pages, oa.page_bytes(vk, P, H, D)), 0x5a, np.uint8)
    codes, h = oa.quantize(vk, x[:, nq + H:])
    ok = (slots >= 0) & (slots < n_pages * P)
    for t in np.flatnonzero(ok):
        oa.store(vk, True, pages, P, int(slots[t]), codes[t], None if h is None else h[t])
    same = np.array_equal(vp.cpu().numpy(), pages)
    assert same, "value pages"
    kw = oa.rope(x[:, nq:nq + H], pos, f, layout, m)
    rt = 2.0 ** -21 * oa.rope_bound(x[:, nq:nq + H], n_rot, layout, m)
    got = np.stack([oa.load(kk, False, kp.cpu().numpy(), P, int(s), H, D) for s in slots[ok]])
    kw, rt = kw[ok], rt[ok]
    if kk == "F16":
        check(got, kw, rt + half_step(kw, "f16") + 2.0 ** -11 * rt, "k")
    else:
        big = np.abs(kw).reshape(*kw.shape[:-1], -1, 32).max(-1).repeat(32, -1)
        rb = rt.reshape(*kw.shape[:-1], -1, 32).max(-1).repeat(32, -1)
        step = ((big + rb) / (127 if kk == "Q8_0" else 8)) * (1 + 2.0 ** -10) + 2.0 ** -24
        near = np.abs(kw) > big - 2 * step if kk == "Q4_0" else np.zeros_like(kw, bool)   # may be cut to code 15
        check(got, kw, rt + np.where(near, step, step / 2), "k")
    if dt == qd:                                              # in place
        q2 = qmm.kv_append(q, k, v, dev(pos), dev(slots), kp, vp, kk, vk, P, freqs, layout, m, out=q)
        assert torch.equal(q2, out)


# -- attention ---------------------------------------------------------------
class Case:
    """A cache filled through kv_write in scattered pages, everything else in it garbage; the oracle reads the stored
    values back from the bytes."""

    def __init__(self, kk, vk, D, P, n_kv, lens, seed="", wide=None, spread=1.0):
        g = self.g = wl.rng("attn", f"{kk}{vk}{D}{P}{n_kv}{lens[:4]}{seed}")
        self.kk, self.vk, self.D, self.P, self.n_kv, self.lens = kk, vk, D, P, n_kv, lens
        need = [(n + P - 1) // P for n in lens]
        n_pages = sum(need) + 3
        order = g.permutation(n_pages)
        wide = wide or max(1, max(need))
        self.table = np.full((len(lens), wide), -7, np.int32)
        at, slots = 0, []
        for b, n in enumerate(lens):
            self.table[b, :need[b]] = order[at:at + need[b]]
            at += need[b]
            t = np.arange(n)
            slots.append(self.table[b, t // P] * P + t % P if n else np.zeros(0, np.int64))
        T = sum(lens)
        self.k = (g.normal(size=(T, n_kv, D)) * spread * np.exp(0.5 * g.normal(size=(1, n_kv, D)))).astype(np.float32)
        self.v = (g.normal(size=(T, n_kv, D)) * np.exp(g.normal(size=(T, n_kv, 1)))).astype(np.float32)
        self.kp, self.vp = (torch.full((n_pages, oa.page_bytes(kind, P, n_kv, D)), 0xFF, dtype=torch.uint8, device="cuda")
                            for kind in (kk, vk))              # 0xFFFF: NaN halves and scales
        if T:
            qmm.kv_write(dev(self.k), dev(self.v), dev(np.concatenate(slots).astype(np.int32)), self.kp, self.vp, kk, vk, P)
        self.kx, self.vx = (oa.dequantize(kind, *oa.quantize(kind, x)) for kind, x in ((kk, self.k), (vk, self.v)))
        self.first = np.concatenate([[0], np.cumsum(lens)])

    def run(self, q, **kw):
        return qmm.attn_decode(q, self.kp, self.vp, dev(self.table), dev(np.array(kw.pop("lens", self.lens), np.int32)),
                               self.kk, self.vk, self.P, self.n_kv, **kw)

    def want(self, q, dt, scale=None, window=0, sinks=None, drop=()):
        B, nq, D = q.shape
        G = nq // self.n_kv
        out, tol = np.zeros(q.shape), np.zeros(q.shape)
        for b, n in enumerate(self.lens):
            t = np.arange(max(0, n - window) if window else 0, n)
            t = t[~np.isin(t // self.P, [p for bb, p in drop if bb == b])]
            rows = self.first[b] + t
            for h in range(nq):
                out[b, h], tol[b, h] = oa.attend(q[b, h], self.kx[rows, h // G], self.vx[rows, h // G],
                                                 D ** -0.5 if scale is None else scale,
                                                 None if sinks is None else sinks[h], dt == "f16")
        return out, tol + half_step(out, dt)


@pytest.mark.parametrize("kk,vk", PAIRS)
@pytest.mark.parametrize("dt", ["f16", "f32"])
@pytest.mark.parametrize("D,G", [(64, 8), (96, 3), (128, 4), (192, 1), (256, 2)])
def test_attn_kinds_and_sizes(kk, vk, dt, D, G):
    c = Case(kk, vk, D, 64, 2, [1, 0, 31, 32, 33, 64, 65, 200, 700])
    q = c.g.normal(size=(9, 2 * G, D)).astype(NP[dt])
    check(c.run(dev(q)).cpu().numpy(), *c.want(q, dt), f"{kk} {vk} D={D}")


@pytest.mark.parametrize("n_kv,G", [(1, 1), (1, 16), (2, 17), (1, 40), (3, 7), (5, 32)])
@pytest.mark.parametrize("dt", ["f16", "f32"])
def test_attn_head_groups(n_kv, G, dt):
    c = Case("Q8_0", "Q4_0", 64, 32, n_kv, [300, 5, 0, 1000])
    q = c.g.normal(size=(4, n_kv * G, 64)).astype(NP[dt])
    sinks = c.g.normal(size=n_kv * G).astype(np.float32) * 3
    check(c.run(dev(q), sinks=dev(sinks)).cpu().numpy(), *c.want(q, dt, sinks=sinks), f"G={G}")


@pytest.mark.parametrize("window", [1, 2, 31, 32, 33, 100, 5000])
@pytest.mark.parametrize("kk,vk", [("F16", "F16"), ("Q4_0", "Q8_0"), ("Q8_0", "Q4_0")])
def test_attn_window(window, kk, vk):
    c = Case(kk, vk, 128, 32, 2, [1, 40, 64, 129, 900, 0])
    q = c.g.normal(size=(6, 8, 128)).astype(np.float16)
    check(c.run(dev(q), window=window).cpu().numpy(), *c.want(q, "f16", window=window), f"window={window}")


@pytest.mark.parametrize("B", [1, 2, 63, 64, 65, 130, 300, 1500])
def test_attn_many_sequences(B):
    """Counts of sequences around the 64 that a wave plans and the 1024 that a workgroup plans at a time, most of them
    short, one long."""
    g = wl.rng("attn", f"many{B}")
    lens = [int(x) for x in g.integers(0, 70, B)]
    lens[B // 2] = 3000
    c = Case("Q8_0", "Q8_0", 64, 32, 2, lens)
    q = c.g.normal(size=(B, 4, 64)).astype(np.float16)
    a = c.run(dev(q))
    check(a.cpu().numpy(), *c.want(q, "f16"), f"B={B}")
    assert torch.equal(a, c.run(dev(q)))                       # the same bits again


@pytest.mark.parametrize("kk,vk", [("F16", "F16"), ("Q8_0", "Q8_0"), ("Q4_0", "Q4_0")])
@pytest.mark.parametrize("dt", ["f16", "f32"])
def test_attn_long(kk, vk, dt):
    """One sequence long enough for splits of several groups per wave, of odd length, in large pages."""
    c = Case(kk, vk, 64, 256, 1, [150001], spread=2.0)
    q = c.g.normal(size=(1, 8, 64)).astype(NP[dt])
    check(c.run(dev(q)).cpu().numpy(), *c.want(q, dt), "long")


def test_attn_strided_q_scale_out_and_workspace():
    c = Case("Q8_0", "F16", 128, 64, 2, [100, 257, 12])
    big = c.g.normal(size=(3, 12, 128)).astype(np.float16)
    q = dev(big)[:, 2:10]
    out = torch.full((3, 8, 128), 7.0, dtype=torch.float16, device="cuda")
    ws = torch.full((qmm.qmm_attn_decode_workspace_bytes(3, 8, 2, 128),), 0xFF, dtype=torch.uint8, device="cuda")
    got = c.run(q, scale=0.3, out=out, workspace=ws)
    assert got is out
    check(out.cpu().numpy(), *c.want(big[:, 2:10], "f16", scale=0.3), "strided")
    with pytest.raises(qmm.QmmError, match="workspace"):
        c.run(q, workspace=ws[:-1])


@pytest.mark.parametrize("dt", ["f16", "f32"])
def test_attn_into_its_queries(dt):
    c = Case("Q8_0", "Q4_0", 128, 64, 2, [300, 31, 0, 2000])
    q = dev(c.g.normal(size=(4, 40, 128)).astype(NP[dt]))
    want = c.run(q)
    assert c.run(q, out=q) is q and torch.equal(q, want)


@pytest.mark.parametrize("kk,vk", [("F16", "F16"), ("Q8_0", "Q4_0")])
def test_attn_strong_and_tiny_values(kk, vk):
    """Scores that leave one token all the weight, scores far below zero, tiny and large values, sinks that outweigh
    every token."""
    c = Case(kk, vk, 64, 32, 1, [500, 500, 500, 500])
    q = c.g.normal(size=(4, 2, 64)).astype(np.float16)
    for amount, scale in ((1.0, 20.0), (2.0 ** -13, 0.125), (300.0, 0.125)):
        c.v = (c.v / np.abs(c.v).max() * amount).astype(np.float32)
        slots = np.concatenate([c.table[b, np.arange(n) // 32] * 32 + np.arange(n) % 32 for b, n in enumerate(c.lens)])
        qmm.kv_write(dev(c.k), dev(c.v), dev(slots.astype(np.int32)), c.kp, c.vp, kk, vk, 32)
        c.vx = oa.dequantize(vk, *oa.quantize(vk, c.v))
        for sinks in (None, np.array([-1000.0, 60.0], np.float32)):
            got = c.run(dev(q), scale=scale, sinks=None if sinks is None else dev(sinks))
            check(got.cpu().numpy(), *c.want(q, "f16", scale=scale, sinks=sinks), f"{amount} {scale}")


@pytest.mark.parametrize("P,wide", [(32, 1), (32, 4), (64, 2), (128, 1), (32, 5)])
@pytest.mark.parametrize("B", [1, 3, 70])
def test_attn_small_tables(P, wide, B):
    """Tables of one split's tokens, and of one page more."""
    full = P * wide
    c = Case("Q8_0", "Q8_0", 64, P, 2, ([full, 1, full - 1] * 24)[:B], seed=str(wide), wide=wide)
    q = c.g.normal(size=(B, 6, 64)).astype(np.float16)
    check(c.run(dev(q)).cpu().numpy(), *c.want(q, "f16"), "out")


def test_attn_lengths_beyond_the_table_and_bad_pages():
    """Lengths are cut to the table, negative ones are empty, pages outside the cache count as absent."""
    c = Case("Q8_0", "Q4_0", 64, 32, 2, [96, 70, 200, 33], wide=7)
    q = c.g.normal(size=(4, 4, 64)).astype(np.float16)
    c.table[2, 3] = 10 ** 6
    c.table[3, 0] = -1
    want, tol = c.want(q, "f16", drop=[(2, 3), (3, 0)])
    want[1], tol[1] = 0, 0
    check(c.run(dev(q), lens=[96, -5, 200, 33]).cpu().numpy(), want, tol, "bad pages")
    c2 = Case("F16", "F16", 64, 32, 1, [64, 64])
    q = c2.g.normal(size=(2, 1, 64)).astype(np.float16)
    check(c2.run(dev(q), lens=[2 ** 31 - 1, 65]).cpu().numpy(), *c2.want(q, "f16"), "cut lengths")
    c2.table[:] = -1                                           # nothing left
    assert torch.equal(c2.run(dev(q)), torch.zeros((2, 1, 64), dtype=torch.float16, device="cuda"))


def test_cache_beyond_32_bit_offsets():
    """Pages at the end of a cache of more than 2^32 bytes."""
    P, H, D = 256, 8, 128
    pb = oa.page_bytes("F16", P, H, D)
    n_pages = (5 << 30) // pb
    kp, vp = (qmm.kv_pages("F16", n_pages, P, H, D) for _ in range(2))
    g = wl.rng("attn", "far")
    n = 300
    table = np.array([[n_pages - 1, 0, 5], [n_pages - 3, n_pages - 2, 1]], np.int32)
    k, v = (g.normal(size=(2 * n, H, D)).astype(np.float16) for _ in range(2))
    slots = np.concatenate([table[b, np.arange(n) // P].astype(np.int64) * P + np.arange(n) % P for b in (0, 1)]).astype(np.int32)
    qmm.kv_write(dev(k), dev(v), dev(slots), kp, vp, "F16", "F16", P)
    rk, rv = qmm.kv_read(dev(slots), kp, vp, "F16", "F16", P, H, D)
    assert torch.equal(rk, dev(k)) and torch.equal(rv, dev(v))
    q = g.normal(size=(2, H, D)).astype(np.float16)
    got = qmm.attn_decode(dev(q), kp, vp, dev(table), dev(np.array([n, n], np.int32)), "F16", "F16", P, H).cpu().numpy()
    for b in (0, 1):
        for h in range(H):
            w, tol = oa.attend(q[b, h], k[b * n:(b + 1) * n, h].astype(float), v[b * n:(b + 1) * n, h].astype(float), D ** -0.5)
            check(got[b, h], w, tol + half_step(w, "f16"), f"far {b} {h}")


@pytest.mark.parametrize("kk,vk", [("F16", "F16"), ("Q8_0", "Q8_0"), ("Q4_0", "Q4_0")])
@pytest.mark.parametrize("dt", ["f16", "f32"])
@pytest.mark.parametrize("scale", [-0.2, 0.0])
def test_attn_negative_and_zero_scale(kk, vk, dt, scale):
    c = Case(kk, vk, 64, 32, 2, [90, 1, 400])
    q = c.g.normal(size=(3, 6, 64)).astype(NP[dt])
    check(c.run(dev(q), scale=scale).cpu().numpy(), *c.want(q, dt, scale=scale), f"scale={scale}")


@pytest.mark.parametrize("kk,vk", [("F16", "F16"), ("Q8_0", "Q8_0"), ("Q4_0", "Q4_0")])
def test_attn_extreme_queries_and_sinks(kk, vk):
    """f32 queries near the ends of their range, and results far below one through sinks: relative to themselves."""
    c = Case(kk, vk, 64, 32, 1, [70, 300])
    q = c.g.normal(size=(2, 2, 64)).astype(np.float32)
    for size in (1e-36, 1e36):
        check(c.run(dev(q * np.float32(size)), scale=0.125 / size).cpu().numpy(),
              *c.want(q * np.float32(size), "f32", scale=0.125 / size), f"{size}")
    c.v = (c.v * 2.0 ** -12).astype(np.float32)
    slots = np.concatenate([c.table[b, np.arange(n) // 32] * 32 + np.arange(n) % 32 for b, n in enumerate(c.lens)])
    qmm.kv_write(dev(c.k), dev(c.v), dev(slots.astype(np.int32)), c.kp, c.vp, kk, vk, 32)
    c.vx = oa.dequantize(vk, *oa.quantize(vk, c.v))
    sinks = np.array([55.0, 60.0], np.float32)
    check(c.run(dev(q), sinks=dev(sinks)).cpu().numpy(), *c.want(q, "f32", sinks=sinks), "far below one")


@pytest.mark.parametrize("kk,vk", PAIRS)
@pytest.mark.parametrize("dt,size", [("f16", 2.0 ** 12), ("f32", 2.0 ** 16), ("f32", 2.0 ** 60), ("f32", 2.0 ** 100)])
@pytest.mark.parametrize("sign", [1, -1])
def test_attn_far_scores_pick_one_token(kk, vk, dt, size, sign):
    """Scores whose f32 neighbours are far apart: all the weight is on the largest (the next one lies below it by more
    than both errors and 100), which has the exact weight 1."""
    c = Case(kk, vk, 64, 64, 1, [1, 40, 150, 333], spread=300.0)
    q = (c.g.normal(size=(4, 3, 64)) * size).astype(NP[dt])
    got = c.run(dev(q), scale=sign * 0.125).cpu().numpy()
    want = np.zeros(q.shape)
    for b in range(4):
        k, v = c.kx[c.first[b]:c.first[b + 1], 0], c.vx[c.first[b]:c.first[b + 1], 0]
        for h in range(3):
            s = sign * 0.125 * (k @ q[b, h].astype(np.float64))
            e = 2.0 ** -17 * (0.125 * np.abs(q[b, h].astype(np.float64)).reshape(2, 32).sum(-1)
                              @ np.abs(k).reshape(-1, 2, 32).max(-1).T + np.abs(s) + 40)
            top = np.argmax(s)
            assert np.all(np.delete(s + e, top) + 100 < s[top] - e[top])
            want[b, h] = v[top]
    check(got, want, 2.0 ** (-11 if dt == "f16" else -18) * np.abs(want) + half_step(want, dt), "out")


@pytest.mark.parametrize("kk,vk", [("F16", "F16"), ("Q8_0", "Q8_0"), ("Q4_0", "Q4_0")])
def test_attn_vanishing_scores(kk, vk):
    c = Case(kk, vk, 64, 64, 1, [1, 0, 40, 150])
    q = (c.g.normal(size=(4, 3, 64)) * 2.0 ** -115).astype(np.float32)
    check(c.run(dev(q), scale=2.0 ** -40).cpu().numpy(), *c.want(q, "f32", scale=2.0 ** -40), "out")


@pytest.mark.parametrize("vk", ["F16", "Q8_0", "Q4_0"])
def test_attn_nonfinite_value_stays_in_its_elements(vk):
    """A NaN in an attended value reaches the elements that share its place (its block of a quantized kind) and no
    others."""
    c = Case("Q8_0", vk, 96, 32, 2, [200, 40])
    row, el = 77, 40                                           # sequence 0, key head 1, block 1
    c.v[row, 1, el] = np.nan
    slots = np.concatenate([c.table[b, np.arange(n) // 32] * 32 + np.arange(n) % 32 for b, n in enumerate(c.lens)])
    qmm.kv_write(dev(c.k), dev(c.v), dev(slots.astype(np.int32)), c.kp, c.vp, "Q8_0", vk, 32)
    q = c.g.normal(size=(2, 4, 96)).astype(np.float16)
    got = c.run(dev(q)).cpu().numpy().astype(np.float64)
    hit = np.zeros(got.shape, bool)
    hit[0, 2:, el if vk == "F16" else slice(32, 64)] = True
    assert np.array_equal(np.isnan(got), hit)
    c.vx[np.isnan(c.vx)] = 0
    want, tol = c.want(q, "f16")
    got[hit] = want[hit] = 0
    check(got, want, tol, "the other elements")


@pytest.mark.parametrize("dt", ["f16", "f32"])
def test_attn_sinks_at_the_ends_of_their_range(dt):
    """Infinite sinks and those whose base-2 logarithm overflows take all the weight or none; a NaN is one head's own."""
    c = Case("Q8_0", "Q4_0", 64, 32, 1, [40, 1, 0, 3000])
    q = c.g.normal(size=(4, 6, 64)).astype(NP[dt])
    sinks = np.array([np.inf, 3e38, -np.inf, -3.4e38, np.nan, 1.0], np.float32)
    got = c.run(dev(q), sinks=dev(sinks)).cpu().numpy()
    want, tol = c.want(q, dt, sinks=[-1e30, -1e30, -1e30, -1e30, 0.0, 1.0])
    want[:, :2] = tol[:, :2] = 0
    assert np.isnan(got[[0, 1, 3], 4]).all()
    got[:, 4] = want[:, 4] = 0
    check(got, want, tol, "sinks")


def rewrite_kv(c):
    """c.k and c.v, changed, into the cache and as the oracle's exact values."""
    t = [np.arange(n) for n in c.lens]
    slots = np.concatenate([c.table[b, x // c.P] * c.P + x % c.P for b, x in enumerate(t)]).astype(np.int32)
    qmm.kv_write(dev(c.k), dev(c.v), dev(slots), c.kp, c.vp, c.kk, c.vk, c.P)
    c.kx, c.vx = (oa.dequantize(kind, *oa.quantize(kind, x)) for kind, x in ((c.kk, c.k), (c.vk, c.v)))


def want_with_floor(c, q, dt):
    """c.want(q, dt), with what f16 weights may lose (the header's term a)."""
    out, tol = c.want(q, dt)
    if dt == "f16":
        scales = None if c.vk == "F16" else oa.quantize(c.vk, c.v)[1]
        for b, n in enumerate(c.lens):
            rows = slice(c.first[b], c.first[b] + n)
            for h in range(q.shape[1]):
                g = h // (q.shape[1] // c.n_kv)
                s = c.kx[rows, g] @ q[b, h].astype(np.float64) * c.D ** -0.5
                w = np.exp(s - s.max())
                tol[b, h] += oa.f16_floor(c.vx[rows, g], None if scales is None else scales[rows, g], w / w.sum())
    return out, tol


def lone_score(c, b, t, q, gap):
    """Sets the key of token t of sequence b so that q scores `gap` (scale D^-0.5)."""
    c.k[c.first[b] + t, 0] = q * (gap * c.D ** 0.5 / np.dot(q, q))


@pytest.mark.parametrize("kk", ["F16", "Q4_0"])
@pytest.mark.parametrize("vk", KINDS)
@pytest.mark.parametrize("dt", ["f16", "f32"])
@pytest.mark.parametrize("D,below,G", [(64, 16, 6), (128, 12, 2), (256, 16, 12), (96, 16, 4)])
def test_attn_blocks_of_unequal_size(kk, vk, dt, D, below, G):
    """Every second block of the values 2^-below of the others and nearly zero in the strongest token: the bound holds for
    each element by its own values."""
    c = Case(kk, vk, D, 64, 1, [1024, 100])
    q = c.g.normal(size=(2, 1, D)).astype(np.float32) * (1 - np.arange(G, dtype=np.float32)[:, None] / 64)
    q = q.astype(NP[dt])
    blocks = c.v.reshape(-1, D // 32, 32)
    blocks *= 2.0 ** 9 / np.abs(blocks).max()
    blocks[:, 1::2] *= np.float32(2.0 ** -below)
    for b, t in ((0, 700), (1, 31)):
        lone_score(c, b, t, q[b, 0].astype(np.float32), 14.0)
        blocks[c.first[b] + t, 1::2] *= np.float32(2.0 ** -9)
    rewrite_kv(c)
    check(c.run(dev(q)).cpu().numpy(), *want_with_floor(c, q, dt), f"{kk} {vk} D={D}")


@pytest.mark.parametrize("kk", ["F16", "Q8_0"])
@pytest.mark.parametrize("vk", KINDS)
@pytest.mark.parametrize("dt,gap,size", [("f16", 20.0, 30000.0), ("f32", 20.0, 1.0), ("f32", 30.0, 1.0), ("f32", 60.0, 0.01)])
def test_attn_strongest_token_of_zero_value(kk, vk, dt, gap, size):
    """The token with nearly all the weight has the value 0 in some elements: what the others add there is exact to the
    bound relative to itself."""
    c = Case(kk, vk, 64, 32, 1, [500, 40], seed=str(gap))
    q = c.g.normal(size=(2, 2, 64)).astype(np.float32)
    q[:, 1] = q[:, 0] * np.float32(0.96875)
    q = q.astype(NP[dt])
    c.v = (c.v / np.abs(c.v).max() * size).astype(np.float32)
    for b, t in ((0, 333), (1, 39)):
        lone_score(c, b, t, q[b, 0].astype(np.float32), gap)
        c.v[c.first[b] + t, 0, ::2] = 0
        c.v[c.first[b] + t, 0, 32:] = 0
    rewrite_kv(c)
    check(c.run(dev(q)).cpu().numpy(), *want_with_floor(c, q, dt), f"{kk} {vk} gap={gap}")


@pytest.mark.parametrize("vk", KINDS)
def test_attn_far_weights_of_the_smallest_blocks(vk):
    """Tokens 2^-98 below the strongest in blocks of the smallest scale, 2^-24, where f32's own range nearly ends."""
    c = Case("Q8_0", vk, 64, 32, 1, [500, 40])
    q = c.g.normal(size=(2, 2, 64)).astype(np.float32)
    q[:, 1] = q[:, 0] * np.float32(0.96875)
    c.v = (c.v / np.abs(c.v).max() * 4e-6).astype(np.float32)
    for b, t in ((0, 333), (1, 39)):
        lone_score(c, b, t, q[b, 0], 68.0)
        c.v[c.first[b] + t] = 0
    rewrite_kv(c)
    check(c.run(dev(q)).cpu().numpy(), *c.want(q, "f32"), vk)


@pytest.mark.parametrize("kk,vk", [("F16", "F16"), ("Q4_0", "Q8_0")])
def test_attn_results_far_below_a_sink(kk, vk):
    """e^-80 of the values, relative to itself."""
    c = Case(kk, vk, 64, 32, 1, [70, 3000])
    q = c.g.normal(size=(2, 2, 64)).astype(np.float32)
    sinks = np.array([80.0, 75.0], np.float32)
    check(c.run(dev(q), sinks=dev(sinks)).cpu().numpy(), *c.want(q, "f32", sinks=sinks), "far below")


@pytest.mark.parametrize("kk,vk", [("F16", "F16"), ("Q8_0", "Q4_0"), ("Q4_0", "Q8_0")])
@pytest.mark.parametrize("G", [1, 6])
@pytest.mark.parametrize("dt", ["f16", "f32"])
def test_attn_long_splits(kk, vk, G, dt):
    """A million tokens in one split (1024 key heads leave no room for more), of nearly equal weight: every entry of the
    table names the same page, so that the sums repeat the same few additions, whose roundings all go one way."""
    n, D, H, P = (1 << 20) + 37, 64, 1024, 32
    g = wl.rng("attn", f"long{kk}{vk}{G}{dt}")
    q = (g.normal(size=(1, H, 1, D)) * np.linspace(1.0, 0.9, G)[:, None]).astype(NP[dt]).reshape(1, H * G, D)
    first = q[0, ::G].astype(np.float64)
    score = np.full((P, 1), -0.41)
    score[0] = 0.7
    k = (score[:, :, None] * first * (D ** 0.5 / (first * first).sum(-1, keepdims=True))).astype(np.float32)
    v = np.abs(g.normal(size=(P, H, D))).astype(np.float32)
    kp, vp = qmm.kv_pages(kk, 1, P, H, D), qmm.kv_pages(vk, 1, P, H, D)
    qmm.kv_write(dev(k), dev(v), dev(np.arange(P, dtype=np.int32)), kp, vp, kk, vk, P)
    kx, vx = (oa.dequantize(kind, *oa.quantize(kind, x)) for kind, x in ((kk, k), (vk, v)))
    got = qmm.attn_decode(dev(q), kp, vp, torch.zeros((1, n // P + 1), dtype=torch.int32, device="cuda"),
                          dev(np.array([n], np.int32)), kk, vk, P, H).cpu().numpy()
    counts = n // P + (np.arange(P) < n % P)
    for h in range(0, H * G, 97):
        w, tol = oa.attend(q[0, h], kx[:, h // G], vx[:, h // G], D ** -0.5, f16=dt == "f16", counts=counts)
        check(got[0, h], w, tol + half_step(w, dt), f"head {h}")


@pytest.mark.parametrize("D", [192, 256])
@pytest.mark.parametrize("dt", ["f16", "f32"])
def test_attn_many_heads_of_large_size(D, dt):
    c = Case("Q8_0", "Q8_0", D, 32, 1, [700, 33])
    q = c.g.normal(size=(2, 16, D)).astype(NP[dt])
    check(c.run(dev(q)).cpu().numpy(), *c.want(q, dt), f"D={D}")


def test_two_streams_at_once():
    """Calls on two streams, each with its own workspace, and the stream argument with outputs allocated by the call."""
    cases = [Case("Q8_0", "Q4_0", 128, 64, 2, [3000, 100]), Case("F16", "F16", 64, 32, 1, [5000])]
    qs = [dev(c.g.normal(size=(len(c.lens), 4, c.D)).astype(np.float16)) for c in cases]
    want = [c.run(q) for c, q in zip(cases, qs)]
    streams = [torch.cuda.Stream() for _ in cases]
    tables = [(dev(c.table), dev(np.array(c.lens, np.int32))) for c in cases]
    torch.cuda.synchronize()
    got = [[], []]
    for _ in range(20):
        for i, (c, q) in enumerate(zip(cases, qs)):
            got[i].append(qmm.attn_decode(q, c.kp, c.vp, *tables[i], c.kk, c.vk, c.P, c.n_kv, stream=streams[i]))
    torch.cuda.synchronize()
    for i in (0, 1):
        assert all(torch.equal(x, want[i]) for x in got[i])


# -- the operators together ----------------------------------------------------------
def test_outputs_of_a_call_on_another_stream_are_its_own():
    """Memory that the current stream's pending work still writes is not handed to a call on another stream."""
    T, H, D = 1000, 7, 128
    x = dev(wl.rng("stream", "own").normal(size=(T, H, D)).astype(np.float32))
    pos, (freqs, m) = dev(np.arange(T, dtype=np.int32)), qmm.rope_freqs(D)
    want = qmm.rope(x, pos, freqs, mscale=m).clone()
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    late = torch.empty_like(x)
    torch.cuda._sleep(50_000_000)
    late.fill_(5.0)
    del late
    got = qmm.rope(x, pos, freqs, mscale=m, stream=side)
    torch.cuda.synchronize()
    assert torch.equal(got, want)


def test_operands_of_a_call_on_another_stream_outlive_it():
    """An operand freed after the call is not handed out while the other stream has still to read it."""
    T, H, D = 1000, 9, 128
    x = dev(wl.rng("stream", "operand").normal(size=(T, H, D)).astype(np.float32))
    pos, (freqs, m) = dev(np.arange(T, dtype=np.int32)), qmm.rope_freqs(D)
    want, side = qmm.rope(x, pos, freqs, mscale=m), torch.cuda.Stream()
    brief = x.clone()
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        torch.cuda._sleep(50_000_000)
    got = qmm.rope(brief, pos, freqs, mscale=m, stream=side)
    del brief
    torch.empty_like(x).fill_(5.0)
    torch.cuda.synchronize()
    assert torch.equal(got, want)


def test_decode_steps_through_a_layer(oracle_mod):
    """Prompt, then decode steps: q, k, v from a Q4_0 projection (qmm_matmul), append, attention, output projection.
    Each part against its definition on the previous part's actual output."""
    B, nq, H, D, P, K = 3, 8, 2, 64, 32, 256
    g = wl.rng("attn", "layer")
    rows = (nq + 2 * H) * D
    W, Wo = wl.random_weights("Q4_0", rows, K, g), wl.random_weights("Q4_0", K, nq * D, g)
    Wd, Wod = dev(W), dev(Wo)
    kp, vp = qmm.kv_pages("Q8_0", 16, P, H, D), qmm.kv_pages("Q4_0", 16, P, H, D)
    kp.fill_(0xFF)
    vp.fill_(0xFF)
    table = np.arange(15).reshape(5, 3).T.copy().astype(np.int32)
    freqs, m = qmm.rope_freqs(D)
    lens = np.array([40, 0, 64])
    for step in range(4):
        if step == 0:                                          # the prompts, as one ragged batch
            seq = np.concatenate([np.full(n, b) for b, n in enumerate(lens)]).astype(int)
            pos = np.concatenate([np.arange(n) for n in lens]).astype(np.int32)
        else:
            seq, pos = np.arange(B), lens.astype(np.int32)
            lens = lens + 1
        slots = (table[seq, pos // P] * P + pos % P).astype(np.int32)
        x = wl.activations((len(seq), K), np.float16, g)
        y = qmm.matmul("Q4_0", Wd, dev(x))
        qkv = y.view(len(seq), nq + 2 * H, D)
        q = qmm.kv_append(qkv[:, :nq], qkv[:, nq:nq + H], qkv[:, nq + H:], dev(pos), dev(slots), kp, vp, "Q8_0", "Q4_0", P,
                          freqs, mscale=m, out_dtype=torch.float16)
        ref = qkv.cpu().numpy()
        want = oa.rope(ref[:, :nq], pos, freqs.cpu().numpy())
        check(q.cpu().numpy(), want, 2.0 ** -21 * oa.rope_bound(ref[:, :nq], D) + half_step(want, "f16"), "q")
        if step == 0:
            continue
        out = qmm.attn_decode(q, kp, vp, dev(table), dev(lens.astype(np.int32)), "Q8_0", "Q4_0", P, H)
        qn, on = q.cpu().numpy(), out.cpu().numpy()
        for b in range(B):
            t = np.arange(lens[b])
            kk, vv = qmm.kv_read(dev((table[b, t // P] * P + t % P).astype(np.int32)), kp, vp, "Q8_0", "Q4_0", P, H, D,
                                 dtype=torch.float32)
            kk, vv = kk.cpu().numpy().astype(float), vv.cpu().numpy().astype(float)
            for h in range(nq):
                w, tol = oa.attend(qn[b, h], kk[:, h // 4], vv[:, h // 4], D ** -0.5)
                check(on[b, h], w, tol + half_step(w, "f16"), f"step {step} row {b} head {h}")
        z = qmm.matmul("Q4_0", Wod, out.view(B, nq * D)).cpu().numpy()
        Y, bound = oracle_mod.matmul("Q4_0", Wo, nq * D, on.reshape(B, nq * D))
        check(z, Y, 1e-3 * bound + 1e-6, "output projection")


def test_captured_steps_replay_with_other_lengths():
    """Append and attention in one captured graph, replayed with positions, slots, lengths and tables changed in place
    and eager calls between the replays; every replay equals the eager result bit for bit."""
    c = Case("Q8_0", "Q4_0", 128, 32, 2, [50, 3, 400, 1], wide=14)
    B, nq = 4, 8
    g = c.g
    freqs, _ = qmm.rope_freqs(128)
    x = dev(g.normal(size=(B, nq + 4, 128)).astype(np.float16))
    pos, lens = (torch.zeros(B, dtype=torch.int32, device="cuda") for _ in range(2))
    slots = torch.full((B,), -1, dtype=torch.int32, device="cuda")
    table = dev(c.table)
    q_out, out = (torch.empty((B, nq, 128), dtype=torch.float16, device="cuda") for _ in range(2))
    ws = torch.empty(qmm.qmm_attn_decode_workspace_bytes(B, nq, 2, 128), dtype=torch.uint8, device="cuda")

    def step(kp, vp, q_out, out):
        qmm.kv_append(x[:, :nq], x[:, nq:nq + 2], x[:, nq + 2:], pos, slots, kp, vp, "Q8_0", "Q4_0", 32, freqs, out=q_out)
        qmm.attn_decode(q_out, kp, vp, table, lens, "Q8_0", "Q4_0", 32, 2, out=out, workspace=ws)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):                              # another stream than the tensors' own
        step(c.kp, c.vp, q_out, out)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step(c.kp, c.vp, q_out, out)
    kp, vp = c.kp.clone(), c.vp.clone()
    for r in range(4):
        n = np.array([50, 3, 400, 1]) + r + 1
        x.copy_(dev(g.normal(size=(B, nq + 4, 128)).astype(np.float16)))
        pos.copy_(dev((n - 1).astype(np.int32)))
        lens.copy_(dev((n if r < 3 else np.array([0, 4, 10, 2])).astype(np.int32)))
        need = c.table.copy()
        for b in range(B):
            if need[b, (n[b] - 1) // 32] < 0:
                need[b, (n[b] - 1) // 32] = c.kp.shape[0] - 1
        table.copy_(dev(need))
        slots.copy_(dev((need[np.arange(B), (n - 1) // 32] * 32 + (n - 1) % 32).astype(np.int32)))
        graph.replay()
        torch.cuda.synchronize()
        q2, o2 = torch.empty_like(q_out), torch.empty_like(out)
        step(kp, vp, q2, o2)
        assert torch.equal(q2, q_out) and torch.equal(o2, out), f"replay {r}"
        assert torch.equal(kp, c.kp) and torch.equal(vp, c.vp), f"replay {r}: cache"
