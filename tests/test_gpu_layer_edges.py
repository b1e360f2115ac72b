"""What stands around a layer's products on the GPU, at the edges of its numerics and of its sizes, against the
definitions of oracle/layer.py.

Activations: 2^-20 of the value, or 2^-126 (where the value leaves f32's normal range), as include/qmm.h states it, on
sums whose f32 value is known exactly.
"""
import numpy as np
import pytest

import workloads as wl
from oracle import layer

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
import gguf_block_quantized_kind_amd as qmm  # noqa: E402


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    qmm.load_library()


def dev(a):
    return torch.from_numpy(np.ascontiguousarray(a)).cuda()


def host(t):
    return t.cpu().numpy()


# -- activations -----------------------------------------------------------------
def far_and_near(n, g):
    """n numbers of f32: tails down to where each activation leaves f32's normal range and past it, what lies between,
    and far ones."""
    parts = [(-104, -87), (-92, -88), (-15, -12.5), (-14, -3), (-11, -9), (-3, 3), (3, 14), (14, 92)]
    special = [0.0, -0.0, 1e-40, -1e-40, 2.0 ** -126, -88.722839, -88.72284, -91.85, 88.722839, 1e30, -1e30, 3e38, -3e38]
    each = -(-(n - len(special)) // len(parts))
    v = np.concatenate([special] + [g.uniform(a, b, each) for a, b in parts])[:n].astype(np.float32)
    return g.permutation(v)


@pytest.mark.parametrize("act", ["silu", "gelu", "gelu_tanh"])
@pytest.mark.parametrize("kind,packed,M,N,K", [
    ("Q4_K", False, 1, 4099, 256), ("Q6_K", False, 8, 4099, 1536), ("Q8_0", True, 1, 4099, 256), ("Q8_0", True, 5, 9001, 256),
    ("Q4_0", False, 3, 4099, 96), ("Q4_K", False, 33, 4099, 256), ("Q4_K", False, 130, 4099, 256), ("Q8_0", False, 64, 8203, 64),
    ("Q8_0", True, 300, 4099, 256), ("Q8_0", False, 70, 4099, 64), ("Q6_K", True, 70, 16403, 256)])
def test_activations_of_known_sums(act, kind, packed, M, N, K):
    """Activations of zeros: the sum is the bias itself, through every kernel that ends in an epilogue."""
    g = wl.rng("edges", f"{act}{kind}{M}{N}")
    b = far_and_near(N, g)
    W = dev(wl.random_weights(kind, N, K, g))
    W = qmm.repack(kind, W, N, K) if packed else W
    fn = qmm.matmul_packed_ep if packed else qmm.matmul_ep
    got = host(fn(kind, W, torch.zeros((M, K), dtype=torch.float16, device="cuda"), N, bias=dev(b), act=act)).astype(np.float64)
    want = layer.activation(act, b)
    ratio = np.abs(got - want) / (2.0 ** -20 * np.abs(want) + 2.0 ** -126)
    at = np.unravel_index(np.argmax(ratio), ratio.shape)
    assert ratio[at] <= 1.0, f"{ratio[at]:.3g} of the bound at {b[at[1]]}: got {got[at]}, want {want[at[1]]}"


@pytest.mark.parametrize("act", ["silu", "gelu", "gelu_tanh"])
def test_activations_of_known_sums_behind_the_integer_product(act):
    g = wl.rng("edges", f"q8{act}")
    N, K = 5003, 512
    b = far_and_near(N, g)
    P = qmm.repack("Q4_0", dev(wl.random_weights("Q4_0", N, K, g)), N, K)
    acts = qmm.rmsnorm_q8("Q4_0", torch.zeros((3, K), device="cuda"), None, 0.0)
    got = host(qmm.gemv_q8("Q4_0", P, acts, N, bias=dev(b), act=act)).astype(np.float64)
    want = layer.activation(act, b)
    assert np.all(np.abs(got - want) <= 2.0 ** -20 * np.abs(want) + 2.0 ** -126)


# -- sizes -----------------------------------------------------------------------
def test_packed_weights_of_more_than_2_31_bytes():
    """Few tokens over records beyond 32-bit offsets, against the same rows taken a few at a time: sums that are exact
    in f32, so the ways give the same bits."""
    N, K = 100352, 20480
    assert qmm.qmm_packed_bytes("Q8_0", N, K) >= 1 << 31
    g = torch.Generator(device="cuda")
    g.manual_seed(5)
    W = torch.randint(-3, 4, (N, K // 32, 34), generator=g, device="cuda", dtype=torch.int8).view(torch.uint8)
    W[..., 0], W[..., 1] = 0, 0x24                          # 2^-6 in f16
    P = qmm.repack("Q8_0", W.reshape(-1), N, K)
    A = torch.randint(-2, 3, (64, K), generator=g, device="cuda").half()
    for M in (9, 64):
        out = qmm.matmul_packed_ep("Q8_0", P, A[:M], N)
        for n in (0, 50000, N - 1040):
            part = qmm.matmul_ep("Q8_0", W[n:n + 1040].reshape(-1), A[:M], 1040)
            assert torch.equal(out[:, n:n + 1040], part), (M, n)
    del W, P, out
    torch.cuda.empty_cache()


# -- eight bits ------------------------------------------------------------------
def subnormal_rows(g, T, D):
    """f32 rows whose blocks have largest magnitudes of 1 to 20000 times the smallest f32, both signs."""
    top = np.exp(g.uniform(0, np.log(20000), (T, D // 32, 1)))
    n = np.rint(g.uniform(-1, 1, (T, D // 32, 32)) * top)
    n[:, :, 5] = np.rint(np.where(g.random((T, D // 32)) < 0.5, -1, 1) * top[:, :, 0])
    n[0, 0, :4] = [190, -190, 100, 63]
    n[0, 0, 4:] = 0
    return (n.reshape(T, D) * 2.0 ** -149).astype(np.float32)


@pytest.mark.parametrize("kind", ["Q8_0", "Q4_0"])
def test_eight_bits_of_subnormal_rows(kind):
    """The norm's 8 bits are those of its f32 rows where these are subnormal: codes, scales and code sums."""
    g = wl.rng("edges", f"subnormal{kind}")
    T, D = 7, 1312
    w = subnormal_rows(g, 1, D)[0]                           # h / sqrt(mean h^2) = 1, -1: the rows are the weight
    x = np.where(g.random((T, D)) < 0.5, -3.0, 3.0).astype(np.float32)
    y = host(qmm.rmsnorm(dev(x), dev(w), 0.0))
    assert np.array_equal(np.abs(y), np.broadcast_to(np.abs(w), y.shape))
    codes, d, sums = layer.eight_bits(kind, y)
    got = qmm.rmsnorm_q8(kind, dev(x), dev(w), 0.0)
    assert np.array_equal(host(got[1]), d) and np.array_equal(host(got[0]), codes) and np.array_equal(host(got[2]), sums)


@pytest.mark.parametrize("kind", ["Q8_0", "Q5_0"])
def test_integer_product_of_subnormal_activations(kind):
    """The workspace of the quantizing product: the oracle's codes, scales and code sums."""
    g = wl.rng("edges", f"subnormal i8 {kind}")
    M, N, K = 5, 32, 1024
    X = subnormal_rows(g, M, K)
    P = qmm.repack(kind, dev(wl.random_weights(kind, N, K, g)), N, K)
    ws = torch.empty(qmm.qmm_gemv_i8_workspace_bytes(M, K), dtype=torch.uint8, device="cuda")
    y = torch.empty((M, N), device="cuda")
    qmm.qmm_gemv_i8(kind, P, dev(X), y, M, N, K, ws)
    raw = host(ws)
    at = [0]
    for n in (M * K, M * K // 8):
        at.append((at[-1] + n + 255) // 256 * 256)
    codes, d, sums = layer.eight_bits(kind, X)
    assert np.array_equal(raw[at[1]:at[1] + M * K // 8].view(np.float32).reshape(M, K // 32), d)
    assert np.array_equal(raw[:M * K].view(np.int8).reshape(M, K), codes)
    assert np.array_equal(raw[at[2]:at[2] + M * K // 8].view(np.int32).reshape(M, K // 32), sums)


# -- the outputs' tensors ----------------------------------------------------------
def calls():
    """One call of every function that makes its outputs itself, as (name, function, how many tensors it makes)."""
    g = wl.rng("edges", "calls")
    x = dev(g.normal(size=(3, 256)).astype(np.float32))
    W = dev(wl.random_weights("Q8_0", 64, 256, g))
    P = qmm.repack("Q8_0", W, 64, 256)
    acts = qmm.rmsnorm_q8("Q8_0", x, None)
    heads, pos = x.view(3, 4, 64), dev(np.arange(3, dtype=np.int32))
    freqs = torch.ones(32, dtype=torch.float64, device="cuda")
    pages = torch.zeros((2, qmm.kv_page_bytes("F16", 32, 4, 64)), dtype=torch.uint8, device="cuda")
    table, lens = dev(np.zeros((3, 1), np.int32)), dev(np.array([1, 2, 3], np.int32))
    return [("rmsnorm", lambda: qmm.rmsnorm(x, None), 1), ("rmsnorm with a residual", lambda: qmm.rmsnorm(x, None, residual=x), 2),
            ("rmsnorm_q8", lambda: qmm.rmsnorm_q8("Q8_0", x, None), 3), ("moe_route", lambda: qmm.moe_route(x, 4), 2),
            ("matmul_ep", lambda: qmm.matmul_ep("Q8_0", W, x, 64), 1), ("matmul_packed_ep", lambda: qmm.matmul_packed_ep("Q8_0", P, x, 64), 1),
            ("gemv_q8", lambda: qmm.gemv_q8("Q8_0", P, acts, 64), 1), ("rope", lambda: qmm.rope(heads, pos, freqs), 1),
            ("kv_read", lambda: qmm.kv_read(pos, pages, pages, "F16", "F16", 32, 4, 64), 2),
            ("attn_decode", lambda: qmm.attn_decode(heads, pages, pages, table, lens, "F16", "F16", 32, 4), 2)]


def tensors(got):
    return [t for part in got for t in tensors(part)] if isinstance(got, tuple) else [got]


def test_dispatch_modes_see_the_outputs():
    """A mode that watches torch's operators sees every tensor that a call makes, and may replace it."""
    from torch.utils._python_dispatch import TorchDispatchMode

    class Watch(TorchDispatchMode):
        def __init__(self):
            super().__init__()
            self.made = []

        def __torch_dispatch__(self, func, types, args=(), kwargs=None):
            out = func(*args, **(kwargs or {}))
            self.made.append((func.name().split(".")[0], out))
            return out

    for name, call, n in calls():
        want = tensors(call())
        with Watch() as w:
            got = tensors(call())
        made = [t for f, t in w.made if f == "aten::empty"]
        assert len(made) == n, (name, w.made)
        assert all(any(t is m for m in made) for t in got), name
        assert all(torch.equal(a, b) for a, b in zip(got, want)), name


def test_deterministic_fill_reaches_the_outputs():
    """With torch's filling of new memory on, the tensors are made by the operator that fills them; the results stay."""
    from torch.profiler import ProfilerActivity, profile
    assert torch.utils.deterministic.fill_uninitialized_memory
    for name, call, n in calls():
        want = tensors(call())
        torch.use_deterministic_algorithms(True)
        try:
            with profile(activities=[ProfilerActivity.CPU]) as p:
                got = tensors(call())
        finally:
            torch.use_deterministic_algorithms(False)
        fills = sum(e.count for e in p.key_averages() if e.key == "aten::empty")
        assert fills >= n, (name, [e.key for e in p.key_averages()])
        assert all(torch.equal(a, b) for a, b in zip(got, want)), name


def test_outputs_that_a_mode_replaces_are_looked_at():
    """A mode that answers with a tensor the kernels cannot write to (on the host, of another type or shape) ends the
    call; what the caller gives is looked at as before."""
    from torch.utils._python_dispatch import TorchDispatchMode

    class Replace(TorchDispatchMode):
        def __init__(self, change):
            super().__init__()
            self.change = change

        def __torch_dispatch__(self, func, types, args=(), kwargs=None):
            out = func(*args, **(kwargs or {}))
            return self.change(out) if func.name().startswith("aten::empty") else out

    changes = [lambda t: torch.zeros(t.shape, dtype=t.dtype), lambda t: t.double(), lambda t: t.reshape(-1)[:1],
               lambda t: torch.zeros((*t.shape, 2), dtype=t.dtype, device=t.device)[..., 0]]
    for name, call, _ in calls():
        for i, change in enumerate(changes):
            with Replace(change), pytest.raises(TypeError, match="new tensor"):
                call()
    torch.cuda.synchronize()
