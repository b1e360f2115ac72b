"""The numpy definitions of what stands around a layer's products against
hand-worked values, and the library's refusals in the documented order, without
a GPU."""
import ctypes
import math
import os

import numpy as np
import pytest

import gguf_block_quantized_kind_amd as qmm
from oracle import layer

OK, EMPTY, KIND, KALIGN, DTYPE, ARG, HIP, WS = range(8)
FAKE = 0x1000  # never dereferenced: every call below is refused first


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(qmm.LIBRARY):
        import gguf_block_quantized_kind_amd._build as b
        b.build()
    return qmm.load_library()


# -- the definitions -----------------------------------------------------------
def test_rmsnorm_hand_values():
    h, y = layer.rmsnorm(np.array([[3.0, 4.0]], np.float16), np.array([[0.0, 0.0]], np.float32), eps=0.0)
    assert h.dtype == np.float32 and np.allclose(y, np.array([[3.0, 4.0]]) / math.sqrt(12.5), rtol=1e-15)
    h, y = layer.rmsnorm(np.array([1.0], np.float32), np.array([2.0 ** -25], np.float32), np.array([2.0]), eps=0.0)
    assert h[0] == 1.0 and y[0] == 2.0                      # the sum is a number in f32
    assert np.all(layer.rmsnorm(np.zeros((2, 3), np.float32), eps=0.0)[1] == 0)
    big = layer.rmsnorm(np.array([1e38, -1e38], np.float32), eps=0.0)[1]
    assert np.allclose(big, [1.0, -1.0], rtol=1e-15)        # squares beyond f32
    bad = layer.rmsnorm(np.array([np.inf, 2.0], np.float32))[1]
    assert np.isnan(bad[0]) and bad[1] == 0


def test_eight_bits_orders():
    y = np.zeros((1, 64), np.float32)
    y[0, :32] = np.arange(32)
    y[0, 31] = 127.0
    for kind in ("Q8_0", "Q4_0"):
        codes, d, sums = layer.eight_bits(kind, y)
        assert d.tolist() == [[1.0, 0.0]] and sums.tolist() == [[sum(range(31)) + 127, 0]]
        first = codes[0, :32].tolist()
        want = list(range(31)) + [127]
        if kind == "Q4_0":                                  # 0..3, 16..19, 4..7, 20..23, ...
            want = [want[16 * h + 4 * G + j] for G in range(4) for h in range(2) for j in range(4)]
        assert first == want and not codes[0, 32:].any()


def test_activation_hand_values():
    v = np.array([-30.0, -1.0, 0.0, 1.0, 30.0])
    assert np.allclose(layer.activation("silu", v), [-30 * math.exp(-30), -1 / (1 + math.e), 0, 1 / (1 + 1 / math.e), 30], rtol=1e-12)
    phi = 0.5 * (1 + math.erf(1 / math.sqrt(2)))
    assert np.allclose(layer.activation("gelu", v), [0, -(1 - phi), 0, phi, 30], rtol=1e-12, atol=1e-150)
    u = math.sqrt(2 / math.pi) * 1.044715
    assert np.allclose(layer.activation("gelu_tanh", v[1:4]), [-0.5 * (1 - math.tanh(u)), 0, 0.5 * (1 + math.tanh(u))], rtol=1e-12)
    assert layer.activation("relu", v).tolist() == [0, 0, 0, 1, 30]
    for act, slope in layer.SLOPE.items():                  # the slopes that tolerances count with
        x = np.linspace(-10, 10, 20001)
        assert np.max(np.abs(np.diff(layer.activation(act, x)))) <= slope * 0.001 * (1 + 1e-9)


def test_route_hand_values():
    l = np.log(np.array([[1.0, 4.0, 2.0, 1.0]]))
    ids, w = layer.route(l, 2)
    assert ids.tolist() == [[1, 2]] and np.allclose(w, [[4 / 6, 2 / 6]])
    ids, w = layer.route(l, 3, normalize=False, scale=2.0)
    assert ids.tolist() == [[1, 2, 0]] and np.allclose(w, [[1.0, 0.5, 0.25]])          # a tie: the lowest index
    ids, w = layer.route(l, 1, bias=[0, 0, 0, 9.0], normalize=False)
    assert ids.tolist() == [[3]] and np.allclose(w, [[1 / 8]])                          # the bias does not weigh
    # Groups {0, 1} and {2, 3}: by their largest, by their two largest.
    s = np.array([[0.9, 0.1, 0.6, 0.6]])
    l = np.log(s / (1 - s))
    assert layer.route(l, 2, "sigmoid", n_group=2, topk_group=1)[0].tolist() == [[0, 1]]
    ids, w = layer.route(l, 2, "sigmoid", n_group=2, topk_group=1, group_top=2)
    assert ids.tolist() == [[2, 3]] and np.allclose(w, 0.5)
    l = np.array([[-math.inf, math.nan, 0.0], [-math.inf] * 3, [0.0, 1.0, 2.0], [math.inf, 0.0, math.inf]])
    ids, w = layer.route(l, 2, slots=[0, 0, -1, 5])
    assert ids.tolist() == [[2, -1], [-1, -1], [-1, -1], [0, 2]] and w.tolist() == [[1, 0], [0, 0], [0, 0], [0.5, 0.5]]
    low = np.full((1, 4), np.finfo(np.float32).min)
    for score in ("softmax", "sigmoid"):
        ids, w = layer.route(low, 2, score)
        assert ids.tolist() == [[0, 1]] and w.tolist() == [[0.5, 0.5]]


# -- refusals ------------------------------------------------------------------
def ep(**kw):
    e = qmm.Epilogue()
    for k, v in dict(dict(act=0), **kw).items():
        setattr(e, k, v)
    return e


def product(fn, **kw):
    a = dict(kind=2, W=FAKE, A=FAKE, dt=1, ep=None, out=FAKE, odt=0, os=None, M=2, N=16, K=256)
    a.update(kw)
    e = None if a["ep"] is None else ctypes.byref(a["ep"])
    return fn(a["kind"], a["W"], a["A"], a["dt"], e, a["out"], a["odt"], a["N"] if a["os"] is None else a["os"], a["M"],
              a["N"], a["K"], a.get("ws"), a.get("wsb", 0), None)


@pytest.mark.parametrize("packed", [False, True])
def test_product_refusals_in_order(lib, packed):
    f = lib.qmm_matmul_packed_ep if packed else lib.qmm_matmul_ep
    assert product(f, M=0, kind=3, K=48) == EMPTY
    assert product(f, kind=3, K=48, dt=9) == KIND
    assert product(f, K=272, dt=9) == KALIGN
    assert product(f, dt=9, W=None) == DTYPE
    assert product(f, odt=2, W=None) == DTYPE
    assert product(f, ep=ep(mul=FAKE, mul_dtype=5, mul_stride=16), W=None) == DTYPE
    assert product(f, ep=ep(residual=FAKE, residual_dtype=-1, residual_stride=16), W=None) == DTYPE
    for bad in (dict(W=None), dict(A=None), dict(A=FAKE + 1), dict(out=None), dict(out=FAKE + 2), dict(odt=1, out=FAKE + 1),
                dict(os=15), dict(os=-16), dict(os=1 << 40), dict(ep=ep(act=5)), dict(ep=ep(act=-1)),
                dict(ep=ep(bias=FAKE + 2)), dict(ep=ep(mul=FAKE + 2, mul_stride=16)),
                dict(ep=ep(mul=FAKE + 1, mul_stride=16, mul_dtype=1)), dict(ep=ep(mul=FAKE, mul_stride=15)),
                dict(ep=ep(residual=FAKE, residual_stride=0)), dict(ep=ep(residual=FAKE, residual_stride=16, residual_dtype=1)),
                dict(ep=ep(residual=FAKE, residual_stride=17)), dict(N=1 << 31)):
        assert product(f, **bad) == ARG, bad
    assert product(f, M=65535 * 64 + 1) == ARG
    assert product(f, M=9, A=FAKE + 8) == ARG               # more than eight tokens: whole 16-byte pieces
    if packed:
        assert product(f, W=FAKE + 8) == ARG
        assert product(f, kind=8, M=1 << 21, K=1024) == ARG
        assert product(f, kind=8, M=100, N=(1 << 31) // 272 + 16) == WS  # beyond the GEMM over records: decoded once
    # The workspace last, where one is used: many tokens, or records that no GEMM multiplies directly.
    big = dict(kind=12, M=4096, N=4096, K=4096)
    need = lib.qmm_matmul_ep_workspace_bytes(12, int(packed), 4096, 4096, 4096, 1)
    assert need == 4096 * 4096 * 2
    assert lib.qmm_matmul_ep_workspace_bytes(12, int(packed), 4096, 4096, 4096, 0) == need + 4096 * 4096 * 4
    assert product(f, **big) == WS and product(f, ws=FAKE, wsb=need - 1, **big) == WS
    assert product(f, ws=FAKE + 128, wsb=need, **big) == WS and product(f, out=None, **big) == ARG
    for bad in ((12, 9, 0, 16, 256, 1), (12, 9, 16, 16, 257, 1), (3, 4096, 4096, 4096, 4096, 1), (12, 4096, 4096, 4096, 4096, 7),
                (12, 8, 4096, 4096, 1, 1), (12, 65535 * 64 + 1, 4096, 4096, 256, 1)):
        k, M, N, K, _, dt = bad
        assert lib.qmm_matmul_ep_workspace_bytes(k, int(packed), M, N, bad[4], dt) == 0, bad


def test_gemv_q8_refusals_in_order(lib):
    def f(**kw):
        a = dict(kind=8, P=FAKE, q=FAKE, d=FAKE, s=FAKE, ep=None, out=FAKE, odt=0, os=16, M=2, N=16, K=256)
        a.update(kw)
        return lib.qmm_gemv_q8(a["kind"], a["P"], a["q"], a["d"], a["s"], None if a["ep"] is None else ctypes.byref(a["ep"]),
                               a["out"], a["odt"], a["os"], a["M"], a["N"], a["K"], None)
    assert f(M=0, kind=99) == EMPTY
    assert f(kind=99, K=288) == KIND and f(kind=12, odt=9) == KIND
    assert f(K=288, odt=9) == KALIGN
    assert f(odt=9, P=None) == DTYPE
    for bad in (dict(P=None), dict(P=FAKE + 8), dict(q=None), dict(q=FAKE + 8), dict(d=None), dict(d=FAKE + 2), dict(s=None),
                dict(s=FAKE + 1), dict(M=9), dict(M=8, K=65536), dict(out=None), dict(os=15), dict(ep=ep(act=7))):
        assert f(**bad) == ARG, bad


def norm(lib, **kw):
    a = dict(x=FAKE, xd=0, xs=64, r=FAKE * 2, rd=0, rs=64, w=FAKE, eps=1e-6, s=FAKE * 3, ss=64, y=FAKE * 4, yd=1, ys=64,
             T=2, H=2, D=32)
    a.update(kw)
    return lib.qmm_rmsnorm(a["x"], a["xd"], a["xs"], a["r"], a["rd"], a["rs"], a["w"], a["eps"], a["s"], a["ss"], a["y"],
                           a["yd"], a["ys"], a["T"], a["H"], a["D"], None)


def test_rmsnorm_refusals_in_order(lib):
    assert norm(lib, T=0, xd=9) == EMPTY and norm(lib, H=0) == EMPTY and norm(lib, D=-1) == EMPTY
    for bad in (dict(xd=2), dict(rd=3), dict(yd=-1)):
        assert norm(lib, D=1 << 20, **bad) == DTYPE
    for bad in (dict(D=32769, xs=1 << 17, rs=1 << 17, ss=1 << 17, ys=1 << 17), dict(eps=-1e-9), dict(eps=math.nan), dict(eps=math.inf), dict(r=None), dict(x=None),
                dict(y=None), dict(x=FAKE + 2), dict(yd=1, y=FAKE + 1), dict(w=FAKE + 2), dict(xs=63), dict(rs=63), dict(ss=63),
                dict(ys=63), dict(ys=1 << 41), dict(y=FAKE * 3, yd=0), dict(y=FAKE), dict(y=FAKE, yd=0, ys=65),
                dict(y=FAKE * 2, yd=0, ys=65), dict(s=FAKE, ss=65), dict(s=FAKE * 2, ss=65), dict(s=FAKE, xd=1),
                dict(T=1 << 31), dict(T=1 << 20, H=1 << 12, xs=1 << 18, rs=1 << 18, ss=1 << 18, ys=1 << 18)):
        assert norm(lib, **bad) == ARG, bad


def test_rmsnorm_q8_refusals_in_order(lib):
    def f(**kw):
        a = dict(kind=2, x=FAKE, xd=0, xs=64, r=None, rd=0, rs=0, w=None, eps=1e-6, s=None, ss=0, q=FAKE, d=FAKE, c=FAKE, T=2,
                 D=64)
        a.update(kw)
        return lib.qmm_rmsnorm_q8(a["kind"], a["x"], a["xd"], a["xs"], a["r"], a["rd"], a["rs"], a["w"], a["eps"], a["s"],
                                  a["ss"], a["q"], a["d"], a["c"], a["T"], a["D"], None)
    assert f(T=0, kind=12) == EMPTY and f(kind=12, D=48) == KIND and f(D=48, xd=7) == KALIGN and f(xd=7, q=None) == DTYPE
    for bad in (dict(q=None), dict(q=FAKE + 8), dict(d=None), dict(c=FAKE + 2), dict(x=None), dict(xs=63), dict(s=FAKE, ss=64),
                dict(eps=-1.0)):
        assert f(**bad) == ARG, bad


def test_moe_route_refusals_in_order(lib):
    def f(**kw):
        a = dict(l=FAKE, dt=0, st=64, b=None, M=2, E=64, k=4, sc=0, g=4, kg=2, top=2, nm=1, scale=1.0, sl=None, i=FAKE, w=FAKE)
        a.update(kw)
        return lib.qmm_moe_route(a["l"], a["dt"], a["st"], a["b"], a["M"], a["E"], a["k"], a["sc"], a["g"], a["kg"], a["top"],
                                 a["nm"], a["scale"], a["sl"], a["i"], a["w"], None)
    for bad in (dict(M=0), dict(E=0), dict(k=0), dict(g=0)):
        assert f(dt=9, **bad) == EMPTY
    assert f(dt=9, E=5000) == DTYPE
    for bad in (dict(E=4100, st=5000), dict(k=65, E=256, st=256), dict(g=65, E=650, st=650), dict(g=3), dict(kg=0), dict(kg=5),
                dict(top=0), dict(top=3), dict(k=33), dict(sc=2), dict(nm=2), dict(nm=-1), dict(scale=math.inf),
                dict(scale=math.nan), dict(l=None), dict(l=FAKE + 2), dict(st=63), dict(b=FAKE + 2), dict(sl=FAKE + 1),
                dict(i=None), dict(w=None), dict(i=FAKE + 2), dict(w=FAKE + 2), dict(M=1 << 31)):
        assert f(**bad) == ARG, bad


def test_python_refusals(lib):
    """Checks of operands before the library is called (host tensors: nothing reaches a GPU)."""
    torch = pytest.importorskip("torch")
    z = torch.zeros
    with pytest.raises(ValueError, match="one GPU"):
        qmm.rmsnorm(z(2, 64), z(64))
    with pytest.raises(ValueError, match="one GPU"):
        qmm.rmsnorm_q8("Q8_0", z(2, 64))
    with pytest.raises(ValueError, match="one GPU"):
        qmm.moe_route(z(2, 8), 2)
    with pytest.raises(qmm.QmmError, match="score"):
        qmm.moe_route(z(2, 8), 2, score="tanh")
    with pytest.raises(ValueError, match="one GPU"):
        qmm.matmul_ep("Q4_0", z(18 * 4, dtype=torch.uint8), z(1, 32))
    with pytest.raises(ValueError, match="needs 144"):
        qmm.matmul_ep("Q4_0", z(18 * 4, dtype=torch.uint8), z(1, 32), 8)
    with pytest.raises(TypeError, match="byte tensor"):
        qmm.matmul_ep("Q4_0", z(18 * 4), z(1, 32), 4)
    with pytest.raises(qmm.QmmError, match="eleven"):
        qmm.matmul_ep("Q4_1", z(18 * 4, dtype=torch.uint8), z(1, 32), 4)
    with pytest.raises(ValueError, match="codes must be"):
        qmm.gemv_q8("Q8_0", z(1, dtype=torch.uint8), (z(2, 256), z(2, 8), z(2, 8, dtype=torch.int32)), 16)
