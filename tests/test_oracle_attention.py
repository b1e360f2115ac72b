"""The numpy definitions of the attention-side operators against hand-worked
values, and the library's host-side calls (page sizes, rotary angles, refusals
in the documented order) without a GPU."""
import ctypes
import math
import os

import numpy as np
import pytest

import gguf_block_quantized_kind_amd as qmm
from oracle import attention as oa

OK, EMPTY, KIND, KALIGN, DTYPE, ARG, HIP, WS = range(8)
FAKE = 0x1000  # never dereferenced: every call below is refused first


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(qmm.LIBRARY):
        import gguf_block_quantized_kind_amd._build as b
        b.build()
    return qmm.load_library()


# -- the definitions -----------------------------------------------------------
def test_quantizer_hand_values():
    x = np.zeros(32, np.float32)
    x[:4] = [127.0, -63.5, 0.5, 1.5]                       # d = 1: ties to even
    c, h = oa.quantize("Q8_0", x)
    assert h[0] == 1.0 and list(c[:5].astype(int) - 128) == [127, -64, 0, 2, 0]
    x[0] = 127.0 * (1 + 2.0 ** -12)                        # the step is rounded up, never down
    c, h = oa.quantize("Q8_0", x)
    assert h[0] == np.float16(1 + 2.0 ** -10) and c[0] - 128 == 127
    y = np.zeros(32, np.float32)
    y[:5] = [-8.0, 7.0, 7.6, 0.5, 8.0]                     # the positive extreme wins the tie: d = -1
    c, h = oa.quantize("Q4_0", y)
    assert h[0] == -1.0 and list(c[:6]) == [15, 1, 0, 8, 0, 8]
    assert list(oa.dequantize("Q4_0", c, h)[:5]) == [-7.0, 7.0, 8.0, 0.0, 8.0]
    for kind in ("Q8_0", "Q4_0"):
        c, h = oa.quantize(kind, np.zeros(32, np.float32))
        assert h.view(np.uint16)[0] == 0 and np.all(oa.dequantize(kind, c, h) == 0)
        for bad in (np.inf, -np.inf, np.nan):
            z = np.ones(64, np.float32)
            z[3] = bad
            v = oa.dequantize(kind, *oa.quantize(kind, z))
            assert np.isnan(v[:32]).all() and np.isfinite(v[32:]).all()


@pytest.mark.parametrize("kind", list(oa.KINDS))
@pytest.mark.parametrize("is_v", [False, True])
@pytest.mark.parametrize("D", [64, 96])
def test_layout_places_every_byte_once(kind, is_v, D):
    """All tokens and elements of a group land on distinct bytes (nibbles) that fill the codes exactly, and a token
    stored reads back."""
    seen = {}
    for r in range(32):
        for d in range(D):
            key = (int(oa.code_at(kind, is_v, r, np.array([d]))[0]), d % 32 // 16 if kind == "Q4_0" else 0)
            assert key not in seen
            seen[key] = (r, d)
    size = D // 32 * oa.UNIT[kind]
    per = 2 if kind == "F16" else 1
    assert {k[0] for k in seen} == set(range(0, size, per))
    g = np.random.default_rng(1)
    pages = g.integers(0, 256, (2, oa.page_bytes(kind, 64, 3, D)), dtype=np.uint8)
    x = g.normal(size=(3, D)).astype(np.float32)
    c, h = oa.quantize(kind, x)
    oa.store(kind, is_v, pages, 64, 64 + 37, c, h)
    assert np.array_equal(oa.load(kind, is_v, pages, 64, 64 + 37, 3, D), oa.dequantize(kind, c, h))


def test_rope_hand_values():
    x = np.zeros((1, 1, 6))
    x[0, 0] = [1, 2, 3, 4, 5, 6]
    y = oa.rope(x, np.array([3]), np.array([math.pi / 6, 0.0]))     # a quarter turn of (x0, x2)
    assert np.allclose(y[0, 0], [-3, 2, 1, 4, 5, 6])
    y = oa.rope(x, np.array([3]), np.array([math.pi / 6, 0.0]), "interleaved", 2.0)
    assert np.allclose(y[0, 0], [-4, 2, 6, 8, 5, 6])


def test_attend_hand_values():
    k = np.array([[0.0] * 32, [1.0] + [0.0] * 31])
    v = np.array([[1.0] * 32, [3.0] * 32])
    q = np.array([math.log(3.0)] + [0.0] * 31)
    o, _ = oa.attend(q, k, v, 1.0)                            # weights 1/4, 3/4
    assert np.allclose(o, 2.5)
    o, _ = oa.attend(q, k, v, 1.0, sink=math.log(4.0))        # weights 1/8, 3/8
    assert np.allclose(o, 1.25)


# -- host-side calls -------------------------------------------------------------
def test_page_bytes(lib):
    for kind, kid in oa.KINDS.items():
        for P, H, D in ((32, 1, 64), (64, 8, 128), (65536, 3, 256)):
            assert lib.qmm_kv_page_bytes(kid, P, H, D) == oa.page_bytes(kind, P, H, D)
    for bad in ((0, 32, 1, 64), (12, 32, 1, 64), (8, 48, 1, 64), (8, 0, 1, 64), (8, 32, 0, 64), (8, 32, 1, 80),
                (8, 32, 1, 160), (8, 65568, 1, 64), (8, 32, 1025, 64)):
        assert lib.qmm_kv_page_bytes(*bad) == -1
    assert qmm.kv_page_bytes("Q8_0", 32, 2, 64) == 32 * 2 * 68
    with pytest.raises(qmm.QmmError):
        qmm.kv_page_bytes("Q5_0", 32, 2, 64)


def test_rope_freqs_plain_linear_factors_and_yarn(lib):
    n = 64
    i = np.arange(n // 2)
    plain = 10000.0 ** (-2.0 * i / n)
    f, m = qmm.rope_freqs(n, device="cpu")
    assert m == 1.0 and np.allclose(f.numpy(), plain, rtol=1e-14)
    f, m = qmm.rope_freqs(n, base=5e5, factor=4.0, device="cpu")
    assert m == 1.0 and np.allclose(f.numpy(), 5e5 ** (-2.0 * i / n) / 4, rtol=1e-14)
    fac = (1 + i / 8).astype(np.float32)
    f, _ = qmm.rope_freqs(n, factors=fac, device="cpu")
    assert np.allclose(f.numpy(), plain / fac, rtol=1e-14)
    f, m = qmm.rope_freqs(n, factor=8.0, orig_ctx=4096, device="cpu")
    assert abs(m - (0.1 * math.log(8.0) + 1)) < 1e-7
    # Pairs that turn more than 32 times over the 4096 positions keep their angle, those that turn less than once are
    # interpolated; in between, the ramp in the pair number.
    turns = plain * 4096 / (2 * math.pi)
    low = math.floor(n * math.log(4096 / (32 * 2 * math.pi)) / (2 * math.log(10000.0)))
    high = math.ceil(n * math.log(4096 / (2 * math.pi)) / (2 * math.log(10000.0)))
    assert np.all(turns[:low] > 32) and np.all(turns[high + 1:] < 1) and 0 < low < high < n // 2
    got = f.numpy()
    assert np.allclose(got[:low + 1], plain[:low + 1], rtol=1e-14)
    assert np.allclose(got[high:], plain[high:] / 8, rtol=1e-14)
    ramp = (i - low) / (high - low)
    mid = slice(low, high)
    assert np.allclose(got[mid], (plain * (1 - ramp) + plain / 8 * ramp)[mid], rtol=1e-13)


def test_rope_freqs_refusals(lib):
    buf = (ctypes.c_double * 8)()
    f = lib.qmm_rope_freqs
    assert f(buf, None, 0, 1e4, None, 1.0, 0, 32.0, 1.0) == EMPTY
    assert f(buf, None, 7, 1e4, None, 1.0, 0, 32.0, 1.0) == ARG
    assert f(None, None, 8, 1e4, None, 1.0, 0, 32.0, 1.0) == ARG
    for base in (1.0, -3.0, math.nan, math.inf):
        assert f(buf, None, 8, base, None, 1.0, 0, 32.0, 1.0) == ARG
    for factor in (0.5, math.nan, math.inf):
        assert f(buf, None, 8, 1e4, None, factor, 0, 32.0, 1.0) == ARG
    assert f(buf, None, 8, 1e4, None, 2.0, -1, 32.0, 1.0) == ARG
    assert f(buf, None, 8, 1e4, None, 2.0, 4096, 1.0, 1.0) == ARG
    assert f(buf, None, 8, 1e4, None, 2.0, 4096, 32.0, 0.0) == ARG
    assert f(buf, None, 8, 1e4, None, 2.0, 4096, 32.0, 1.0) == OK


def test_rope_refusals_in_order(lib):
    base = dict(freqs=FAKE, n_rot=64, layout=0, m=1.0, pos=FAKE, x=FAKE, xd=1, xs=256, y=FAKE + 0x10000, yd=1, ys=256,
                T=3, H=2, D=128, s=None)

    def call(**kw):
        return lib.qmm_rope(*dict(base, **kw).values())

    for zero in ("T", "H", "D"):
        assert call(**{zero: 0}, xd=9) == EMPTY
    assert call(xd=9, layout=7) == DTYPE
    assert call(yd=9) == DTYPE
    for bad in (dict(layout=2), dict(D=127, n_rot=2), dict(n_rot=63), dict(n_rot=130), dict(n_rot=0), dict(freqs=None),
                dict(pos=None), dict(x=None), dict(y=None), dict(x=FAKE + 1), dict(y=FAKE + 1), dict(pos=FAKE + 2),
                dict(freqs=FAKE + 4), dict(xs=255), dict(ys=255), dict(T=1 << 25, xs=1 << 20, ys=1 << 20),
                dict(y=FAKE, yd=0), dict(y=FAKE, ys=512)):
        assert call(**bad) == ARG, bad


CACHE = dict(kk=8, vk=2, kp=FAKE, vp=FAKE, n=4, P=64, H=2, D=128)


def cache(kw):
    c = dict(CACHE)
    for k in list(kw):
        if k in c:
            c[k] = kw.pop(k)
    return list(c.values())


CACHE_ARG = (dict(D=160), dict(D=32), dict(P=48), dict(P=1 << 17), dict(H=2000), dict(n=1 << 26), dict(kp=None),
             dict(vp=None), dict(kp=FAKE + 8), dict(vp=FAKE + 4))


def test_kv_write_refusals_in_order(lib):
    base = dict(k=FAKE, ks=256, v=FAKE, vs=256, dt=1, slots=FAKE, T=5, s=None)

    def call(**kw):
        c = cache(kw)
        return lib.qmm_kv_write(*c, *dict(base, **kw).values())

    for zero in ("n", "P", "H", "D", "T"):
        assert call(**{zero: 0}, kk=5) == EMPTY
    assert call(kk=6, D=80) == KIND and "Q8_0" in qmm.qmm_last_error()
    assert call(vk=39) == KIND
    assert call(D=80, dt=7) == KALIGN
    assert call(dt=7, P=48) == DTYPE
    for bad in CACHE_ARG + (dict(k=None), dict(v=None), dict(k=FAKE + 1), dict(v=FAKE + 1), dict(ks=255), dict(vs=255),
                            dict(slots=None), dict(slots=FAKE + 2), dict(T=1 << 23)):
        assert call(**bad) == ARG, bad


def test_kv_append_refusals(lib):
    head = dict(freqs=FAKE, n_rot=64, layout=0, m=1.0, pos=FAKE, q=FAKE, qs=512, n_q=4, qo=FAKE + 0x10000, qd=1, qos=512)
    tail = dict(k=FAKE, ks=256, v=FAKE, vs=256, dt=1, slots=FAKE, T=5, s=None)

    def call(**kw):
        c = cache(kw)
        h = dict(head, **{k: kw.pop(k) for k in list(kw) if k in head})
        return lib.qmm_kv_append(*h.values(), *c, *dict(tail, **kw).values())

    assert call(n_q=0) == EMPTY
    assert call(T=0) == EMPTY
    assert call(kk=4) == KIND
    assert call(qd=3) == DTYPE
    for bad in CACHE_ARG + (dict(layout=-1), dict(n_rot=130), dict(n_rot=3), dict(freqs=None), dict(pos=None),
                            dict(q=None), dict(qo=None), dict(qs=511), dict(qos=511), dict(qo=FAKE, qos=1024),
                            dict(slots=None), dict(T=1 << 22)):
        assert call(**bad) == ARG, bad


def test_kv_read_refusals(lib):
    base = dict(slots=FAKE, T=5, ko=FAKE, vo=FAKE, dt=0, s=None)

    def call(**kw):
        c = cache(kw)
        return lib.qmm_kv_read(*c, *dict(base, **kw).values())

    assert call(T=0) == EMPTY
    assert call(vk=1000) == KIND
    assert call(dt=2) == DTYPE
    for bad in CACHE_ARG + (dict(slots=None), dict(ko=None), dict(vo=None), dict(ko=FAKE + 4), dict(T=1 << 23)):
        assert call(**bad) == ARG, bad


def test_attn_decode_refusals_in_order(lib):
    need = lib.qmm_attn_decode_workspace_bytes(3, 8, 2, 128)
    assert need > 0
    for bad in ((0, 8, 2, 128), (3, 0, 2, 128), (3, 8, 0, 128), (3, 8, 3, 128), (3, 8, 2, 80), (1 << 20, 64, 2, 128)):
        assert lib.qmm_attn_decode_workspace_bytes(*bad) == 0
    base = dict(q=FAKE, dt=1, qs=8 * 128, n_q=8, bt=FAKE, mp=7, sl=FAKE, B=3, scale=0.1, window=0, sinks=None, out=FAKE,
                ws=FAKE, wsb=need, s=None)

    def call(**kw):
        c = cache(kw)
        return lib.qmm_attn_decode(*c, *dict(base, **kw).values())

    for zero in ("n", "P", "H", "D", "B", "n_q", "mp"):
        assert call(**{zero: 0}, dt=9) == EMPTY
    assert call(kk=0, D=80) == KIND
    assert call(D=80, dt=9) == KALIGN
    assert call(dt=9, n_q=7) == DTYPE
    for bad in CACHE_ARG + (dict(n_q=7), dict(mp=1 << 26), dict(scale=math.nan), dict(scale=math.inf), dict(window=-1),
                            dict(q=None), dict(q=FAKE + 1), dict(qs=1023), dict(bt=None), dict(sl=None),
                            dict(bt=FAKE + 1), dict(sinks=FAKE + 2), dict(out=None), dict(out=FAKE + 8)):
        assert call(**bad) == ARG, bad
    assert call(ws=None) == WS
    assert call(wsb=need - 1) == WS
    assert call(ws=FAKE + 8) == WS
    assert "workspace" in qmm.qmm_last_error()


def test_python_checks_before_the_library():
    torch = pytest.importorskip("torch")
    k = torch.zeros((5, 2, 128), dtype=torch.float16)
    slots = torch.zeros(5, dtype=torch.int32)
    kp, vp = (torch.zeros((4, qmm.kv_page_bytes(x, 64, 2, 128)), dtype=torch.uint8) for x in ("Q8_0", "Q4_0"))
    good = (k, k, slots, kp, vp, "Q8_0", "Q4_0", 64)

    def swap(i, v):
        return good[:i] + (v,) + good[i + 1:]

    with pytest.raises(ValueError, match="on one GPU"):
        qmm.kv_write(*good)                                         # host tensors
    with pytest.raises(ValueError):
        qmm.kv_write(*swap(1, k[:, :1]))
    with pytest.raises(TypeError):
        qmm.kv_write(*swap(1, k.float()))
    with pytest.raises(TypeError):
        qmm.kv_write(*swap(2, slots.long()))
    with pytest.raises(ValueError):
        qmm.kv_write(*swap(2, slots[:4]))
    with pytest.raises(ValueError):
        qmm.kv_write(*swap(3, vp))                                  # pages of another kind
    with pytest.raises(ValueError):
        qmm.kv_write(*swap(4, vp[:3]))
    with pytest.raises(qmm.QmmError):
        qmm.kv_write(*swap(5, "Q6_K"))
    with pytest.raises(ValueError, match="packed"):
        qmm.kv_write(*swap(0, k.transpose(0, 1).contiguous().transpose(0, 1)))
    with pytest.raises(qmm.QmmError):
        qmm.kv_pages("Q8_0", 3, 48, 2, 128, device="cpu")
    with pytest.raises(ValueError):
        qmm.rope_freqs(8, factors=[1.0], device="cpu")


def test_python_checks_of_other_operands(lib):
    torch = pytest.importorskip("torch")
    x = torch.zeros((3, 2, 64), dtype=torch.float16)
    pos, (f, m) = torch.arange(3, dtype=torch.int32), qmm.rope_freqs(64, device="cpu")
    for bad, error in [((x.numpy(), pos, f), TypeError), ((x[0], pos, f), ValueError), ((x, pos.long(), f), TypeError),
                       ((x, pos[:2], f), ValueError), ((x, pos, f.float()), TypeError), ((x, None, f), TypeError),
                       ((x, pos, f, "other"), qmm.QmmError), ((x, pos, f, "half", "1"), TypeError),
                       ((x, pos, f), ValueError)]:                      # the last: host tensors
        with pytest.raises(error):
            qmm.rope(*bad)
    kp = torch.zeros((4, qmm.kv_page_bytes("F16", 32, 2, 64)), dtype=torch.uint8)
    table, lens = torch.zeros((3, 2), dtype=torch.int32), torch.ones(3, dtype=torch.int32)
    good = [x, kp, kp, table, lens, "F16", "F16", 32, 2]
    for at, value, error in [(3, table[:2], ValueError), (3, table.long(), TypeError), (4, lens[:2], ValueError),
                             (1, kp[:, :-1], TypeError), (1, kp[:3], ValueError), (7, 64, ValueError), (8, 3, ValueError),
                             (8, 2.5, TypeError), (5, "Q6_K", qmm.QmmError), (0, x, ValueError)]:
        with pytest.raises(error):
            qmm.attn_decode(*good[:at], value, *good[at + 1:])
    for kw in (dict(sinks=torch.zeros(3)), dict(out=x[:1]), dict(window="a"), dict(workspace=1)):
        with pytest.raises((ValueError, TypeError)):
            qmm.attn_decode(*good, **kw)
    with pytest.raises(TypeError):
        qmm._load_ops().rope(x)                                         # too few arguments


def test_an_output_tensor_of_another_type_than_asked_for_is_refused(lib):
    """Not written in its own type without a word."""
    torch = pytest.importorskip("torch")
    x = torch.zeros((3, 2, 64), dtype=torch.float16)
    pos, (f, m) = torch.arange(3, dtype=torch.int32), qmm.rope_freqs(64, device="cpu")
    kp = torch.zeros((4, qmm.kv_page_bytes("F16", 32, 2, 64)), dtype=torch.uint8)
    cache = (kp, kp, "F16", "F16", 32)
    for call in (lambda t: qmm.rope(x, pos, f, out=x, out_dtype=t),
                 lambda t: qmm.kv_append(x, x, x, pos, pos, *cache, f, out=x, out_dtype=t),
                 lambda t: qmm.kv_read(pos, *cache, 2, 64, dtype=t, k_out=x, v_out=x)):
        with pytest.raises(TypeError, match="asked for"):
            call(torch.float32)
        with pytest.raises(ValueError, match="on one GPU"):             # host tensors, refused after the types
            call(torch.float16)


def test_rope_factors_that_leave_no_angle_are_refused(lib):
    """A zero or non-finite per-pair divisor made infinite or NaN angles, and so NaN rows."""
    for bad in (0.0, math.inf, -math.inf, math.nan):
        with pytest.raises(qmm.QmmError, match="factors"):
            qmm.rope_freqs(8, factors=[1.0, 2.0, bad, 1.0], device="cpu")
    f, _ = qmm.rope_freqs(8, factors=[1.0, 2.0, -4.0, 1.0], device="cpu")
    assert np.allclose(f.numpy(), 10000.0 ** (-np.arange(4) / 4) / [1, 2, -4, 1], rtol=1e-14)
