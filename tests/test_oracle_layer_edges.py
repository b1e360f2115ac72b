"""The edges of what stands around a layer's products, without a GPU: what the tolerances of the definitions let pass,
and calls of the library that end before it reaches one."""
import math

import numpy as np
import pytest

from oracle import layer


# -- tolerances ------------------------------------------------------------------
def test_how_far_an_activation_moves():
    """Against a fine grid of the sums within reach, the minimum among them."""
    for act in layer.ACTS:
        for u, err in ((-1.3, 0.2), (-0.75, 1e-3), (-0.7518, 1e-9), (-6.0, 0.5), (2.0, 0.25), (0.0, 3.0), (-88.0, 1.0)):
            grid = u + err * np.linspace(-1, 1, 20001)
            far = np.abs(layer.activation(act, grid) - layer.activation(act, u)).max()
            got = float(layer.moved(act, np.array(u), err))
            assert far * (1 - 1e-12) <= got <= far * (1 + 1e-3) + 1e-18, (act, u, got, far)
    for act, low in layer.LOWEST.items():
        x = low + np.array([-1e-4, 0.0, 1e-4])
        assert np.argmin(layer.activation(act, x)) == 1, act


@pytest.mark.parametrize("act,where", [("silu", (-103.0, -5.0)), ("gelu", (-13.0, -3.0)), ("gelu_tanh", (-10.0, -3.0))])
def test_tails_that_are_lost_are_outside_the_tolerance(act, where):
    """Mistakes planted in the result: a tail of zeros, one off by a thousandth, and the tail of an exponential that
    overflows; sums known to their rounding alone, the result in f32."""
    v = np.linspace(*where, 1001)
    want, tol = layer.epilogue(v, 0.0, act=act)
    far = np.abs(want) > 2.0 ** -125
    assert np.any(far) and np.all(np.abs(want[far]) > tol[far])
    # (A rounding of the sum moves a tail by up to |v| (silu) or v^2 (gelu) steps; a thousandth is far beyond.)
    clear = np.abs(want) > 2.0 ** -114                      # a thousandth of it is a normal number
    assert np.any(clear) and np.all(np.abs(1e-3 * want[clear]) > tol[clear])
    assert np.all(np.abs(want * (1 + 2.0 ** -21) - want) <= tol)
    if act == "silu":
        over = (v < -88.73) & far
        assert np.any(over) and np.all(np.abs(want[over]) > tol[over])


def test_tolerance_covers_sums_that_lie_across_the_minimum():
    g = np.random.default_rng(7)
    for act in ("silu", "gelu", "gelu_tanh"):
        u = g.uniform(-3, 1, 4000)
        err = np.exp(g.uniform(math.log(1e-7), math.log(2.0), 4000))
        want, tol = layer.epilogue(u, err, act=act)
        off = u + err * g.uniform(-1, 1, 4000)
        assert np.all(np.abs(layer.activation(act, off) - want) <= tol)


# -- the library's answers about sizes ---------------------------------------------
OK, EMPTY, KIND, KALIGN, DTYPE, ARG, HIP, WS = range(8)
FAKE = 0x1000  # never dereferenced: every call below is refused first


@pytest.fixture(scope="module")
def lib():
    import os

    import gguf_block_quantized_kind_amd as qmm
    if not os.path.exists(qmm.LIBRARY):
        import gguf_block_quantized_kind_amd._build as b
        b.build()
    return qmm.load_library()


def product(lib, packed, kind, M, N, K, dt=1, ws=None, wsb=0):
    fn = lib.qmm_matmul_packed_ep if packed else lib.qmm_matmul_ep
    return fn(kind, FAKE, FAKE, dt, None, FAKE, 0, N, M, N, K, ws, wsb, None)


@pytest.mark.parametrize("kind,N,K", [(8, 100352, 20480), (2, 65536, 65536), (20, 131072, 32768)])
def test_weights_beyond_32_bits_at_any_number_of_tokens(lib, kind, N, K):
    """Records of 2^31 bytes and more are beyond the GEMM over records: decoded once, whether the tokens are few or many.
    (Every call ends at the missing workspace.)"""
    for M in (9, 16, 17, 64, 65, 100, 512, 513, 600, 2000):
        for dt in (0, 1):
            assert lib.qmm_matmul_ep_workspace_bytes(kind, 1, M, N, K, dt) >= 2 * N * K, (M, dt)
            assert product(lib, True, kind, M, N, K, dt) == WS, (M, dt)


@pytest.mark.parametrize("packed,kind,M,N,K", [
    (1, 8, 1 << 21, 64, 1024),                               # M K of 2^31
    (1, 12, 9, 16, 1 << 21), (1, 14, 100, 4096, 1 << 21),    # decoded weights of more than 2^20 columns
    (1, 8, 9, 16, (1 << 30) + 256), (0, 8, 9, 16, (1 << 30) + 32), (0, 8, 100, (1 << 31), 32), (1, 8, 100, (1 << 31), 256),
    (1, 8, 100, 1 << 28, 1 << 20),                           # 2^40 bytes of records
    (1, 12, 1 << 21, 1 << 21, 256), (0, 14, 65535 * 64 + 1, 64, 256), (1, 3, 100, 8192, 256), (0, 12, 100, 8192, 288)])
def test_no_workspace_for_what_is_refused(lib, packed, kind, M, N, K):
    for dt in (0, 1):
        assert product(lib, packed, kind, M, N, K, dt) not in (OK, WS, HIP)
        assert lib.qmm_matmul_ep_workspace_bytes(kind, packed, M, N, K, dt) == 0, dt


# -- eight bits ------------------------------------------------------------------
def test_eight_bits_of_subnormal_blocks():
    """Where the scale has few bits left the quotient of the largest can be beyond 127: its code is cut there, with its
    sign, and the code sum is that of the codes."""
    from oracle import int8
    unit = np.float32(2.0 ** -149)
    y = np.zeros((1, 64), np.float32)
    y[0, :4] = np.array([190, -190, 100, 63], np.float32) * unit     # d = 190 / 127 rounds to one unit
    y[0, 32:35] = np.array([-63, 40, 5], np.float32) * unit          # d rounds to none
    q, d = int8.quantize(y)
    assert d.tolist() == [[float(unit), 0.0]]
    assert q[0, :4].tolist() == [127, -127, 100, 63] and not q[0, 4:].any()
    assert layer.eight_bits("Q8_0", y)[2].tolist() == [[163, 0]]
    for n in range(1, 127 * 127 + 2000, 37):                          # every other scale: codes within half a step of 127
        q, d = int8.quantize(np.full((1, 32), n, np.float32) * unit)
        k = round(float(d[0, 0]) / 2.0 ** -149)
        assert k == int(np.rint(np.float32(n) / np.float32(127))) and np.all(q == (min(127, round(n / k)) if k else 0))


def test_norm_refuses_more_heads_than_it_names(lib):
    f = lambda H: lib.qmm_rmsnorm(FAKE, 0, 4 * H, None, 0, 0, None, 1e-6, None, 0, FAKE + 2, 0, 4 * H, 1, H, 4, None)  # noqa: E731
    assert f(65536) == f(65537) == ARG                       # y is misaligned: refused either way, by their own words
    import gguf_block_quantized_kind_amd as qmm
    f(65536)
    assert b"aligned" in lib.qmm_last_error()
    f(65537)
    assert b"H=65537" in lib.qmm_last_error()
    assert "H > 65536" in open(__import__("os").path.join(__import__("os").path.dirname(__import__("os").path.dirname(qmm.__file__)),
                                                          "include", "qmm.h")).read()
