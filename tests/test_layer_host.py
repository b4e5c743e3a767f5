"""The operators around the grouped GEMM, without a GPU: the fp64 definitions against
differences, torch and brute force, and the refusals of the C ABI and the binding."""
import ctypes

import numpy as np
import pytest
import torch

import oracle.layer as ol

FAKE = ctypes.c_void_p(4096)
OFF = ctypes.c_void_p(4100)   # 4-byte aligned, not 16


@pytest.fixture(scope="module")
def lib():
    from moe_grouped_gemm_ragged_b200 import _build
    _build.build()
    import moe_grouped_gemm_ragged_b200 as gg
    return gg.lib()


# -------------------------------------------------------------------------- definitions

def _difference(f, x, i, h=1e-6):
    a, b = x.copy(), x.copy()
    a[i] += h
    b[i] -= h
    return (f(a) - f(b)) / (2 * h)


@pytest.mark.parametrize("sigmoid", [False, True])
@pytest.mark.parametrize("renorm", [False, True])
def test_gate_gradient_equals_differences(sigmoid, renorm):
    """Central differences with h = 1e-6 are off by h^2 times the third derivative (below 10
    here) and 2^-52 / h from rounding: 1e-9 bounds both."""
    rng = np.random.default_rng(3)
    x = rng.normal(size=(4, 9))
    x[1, 2] = -np.inf
    x[2] = -np.inf
    x[3, 3:] = -np.inf
    dw = rng.normal(size=(4, 5))
    ids, _ = ol.gate(x, 5, sigmoid, renorm, 2.5)
    assert (ids[2] == -1).all() and (ids[3, 3:] == -1).all()
    dx = ol.gate_backward(x, ids, dw, sigmoid, renorm, 2.5)

    def loss(z):
        return (2.5 * ol._weights(z, ids, sigmoid, renorm) * dw).sum()

    for i in np.ndindex(x.shape):
        if np.isneginf(x[i]):
            assert dx[i] == 0
        else:
            assert abs(_difference(loss, x, i) - dx[i]) < 1e-9


def test_gate_equals_torch_and_sums_to_scale():
    x = torch.randn(50, 13, dtype=torch.float64, generator=torch.Generator().manual_seed(1))
    ids, w = ol.gate(x.numpy(), 4, scale=1.0, renorm=False)
    tw, tids = torch.softmax(x, 1).topk(4)
    np.testing.assert_array_equal(ids, tids.numpy())
    np.testing.assert_allclose(w, tw.numpy(), rtol=1e-13)
    for sig in (False, True):
        np.testing.assert_allclose(ol.gate(x.numpy(), 4, sig, True, 3.0)[1].sum(1), 3.0,
                                   rtol=1e-13)
    ids, _ = ol.gate(np.zeros((2, 6)), 3)
    assert ids.tolist() == [[0, 1, 2]] * 2  # ties to the lowest


def test_unroute_inverts_a_routing():
    """Weights 1/k of copies of a token's own row bring the row back; gradients against
    differences of a linear map (exact up to rounding: 1e-8)."""
    import oracle
    import workloads
    ids, X = workloads.make_routing(20, 3, 5, 8, seed=2)
    offs, row_of, Ap, _ = oracle.route(ids, X, 5)
    Y = oracle.bf16_to_f64(Ap)
    w = np.full((20, 3), 1 / 3)
    np.testing.assert_allclose(ol.unroute(Y, row_of, 3, w), oracle.bf16_to_f64(oracle.as_u16(X)),
                               rtol=1e-14)
    rng = np.random.default_rng(0)
    d, w = rng.normal(size=(20, 8)), rng.normal(size=(20, 3))
    row_of[4] = -1
    dY, dw = ol.unroute_backward(d, Y, row_of, 3, w)
    for i in [(0, 0), (17, 3), (40, 7)]:
        got = _difference(lambda z: (ol.unroute(z, row_of, 3, w) * d).sum(), Y, i)
        assert abs(got - dY[i]) < 1e-8
    for i in [(0, 0), (1, 1), (19, 2)]:
        got = _difference(lambda z: (ol.unroute(Y, row_of, 3, z) * d).sum(), w, i)
        assert abs(got - dw[i]) < 1e-8
    assert dw[1, 1] == 0


@pytest.mark.parametrize("concat", [False, True])
def test_silu_mul_gradient_equals_differences(concat):
    rng = np.random.default_rng(5)
    H, d, w = rng.normal(size=(2, 256)), rng.normal(size=(2, 128)), rng.normal(size=2)
    dH, dw = ol.silu_mul_backward(d, H, concat, w)
    for i in [(0, 0), (0, 127), (0, 128), (1, 200), (1, 255)]:
        got = _difference(lambda z: (ol.silu_mul(z, concat, w) * d).sum(), H, i)
        assert abs(got - dH[i]) < 1e-8
    for i in range(2):
        got = _difference(lambda z: (ol.silu_mul(H, concat, z) * d).sum(), w, i)
        assert abs(got - dw[i]) < 1e-8


def test_e4m3_rounding_equals_torch():
    v = torch.cat([torch.linspace(-448, 448, 20001), torch.logspace(-12, 8, 4001, base=2.0),
                   torch.tensor(ol.E4M3), torch.tensor((ol.E4M3[1:] + ol.E4M3[:-1]) / 2)])
    v = v.float()
    np.testing.assert_array_equal(ol.round_e4m3(v.double().numpy()),
                                  v.to(torch.float8_e4m3fn).double().numpy())
    assert ol.E4M3[-1] == 448


def test_pack8_scale_is_the_least_that_fits():
    x = np.zeros((5, 40))
    x[0, 0], x[1, 3], x[2, 5], x[3, 39] = 448.0, 449.0, 2.0 ** -130, 3.38e38
    x[4, 0], x[4, 1] = np.inf, 1.0
    val, code = ol.pack8(x)
    assert code[0].tolist() == [127, 9] and code[1, 0] == 128 and code[2, 0] == 9
    assert code[3, 1] == 247 and np.isnan(val[4, 0]) and val[4, 1] == 1 and code[4, 0] == 119
    rng = np.random.default_rng(1)
    y = rng.normal(size=(64, 96)) * np.exp2(rng.integers(-20, 20, (64, 1)))
    val, code = ol.pack8(y)
    s = np.repeat(np.exp2(code - 127.0), 32, 1)
    assert (np.abs(val - y) <= np.maximum(np.abs(y) * 2.0 ** -4, 2.0 ** -10 * s)).all()
    assert (np.abs(val) <= 448 * s).all()
    tight = np.abs(y).reshape(64, 3, 32).max(2) > 224 * np.exp2(code - 127.0)
    assert tight.all()


# ----------------------------------------------------------------------------- refusals

def test_gate_refusals(lib):
    f, b = lib.gg_gate_topk, lib.gg_gate_topk_backward

    def fwd(T=4, E=8, k=2, bias=None, score=0, flags=0, scale=1.0, x=FAKE, ids=FAKE, w=FAKE,
            num=None, st=None):
        return f(x, T, E, k, bias, score, flags, scale, num, ids, w, st, None)

    for bad in (dict(T=-1), dict(E=0), dict(k=0), dict(k=9), dict(score=2), dict(flags=4),
                dict(scale=float("inf")), dict(scale=float("nan")), dict(x=None), dict(ids=None),
                dict(w=None), dict(bias=FAKE)):
        assert fwd(**bad) == 1, bad
    odd = ctypes.c_void_p(4097)
    for bad in (dict(E=1025), dict(E=64, k=33), dict(T=1 << 31), dict(x=odd), dict(ids=odd),
                dict(w=odd), dict(num=odd), dict(st=odd), dict(bias=odd, score=1),
                dict(x=ctypes.c_void_p(4098), flags=2)):
        assert fwd(**bad) == 2, bad
    assert b(FAKE, 4, 8, 2, 0, 0, 1.0, FAKE, None, FAKE, None, None) == 1
    assert b(FAKE, 4, 8, 2, 0, 0, 1.0, FAKE, FAKE, odd, None, None) == 2
    assert b(FAKE, 4, 8, 9, 0, 0, 1.0, FAKE, FAKE, FAKE, None, None) == 1


def test_unroute_refusals(lib):
    f, b = lib.gg_unroute, lib.gg_unroute_backward

    def fwd(Y=FAKE, rows=8, row_of=FAKE, w=None, res=None, T=4, k=2, N=16, out=FAKE, st=None):
        return f(Y, rows, row_of, w, res, T, k, N, out, st, None)

    for bad in (dict(Y=None), dict(rows=-1), dict(row_of=None), dict(T=-1), dict(k=0), dict(N=0),
                dict(out=None)):
        assert fwd(**bad) == 1, bad
    for bad in (dict(N=12), dict(Y=OFF), dict(res=OFF), dict(out=OFF), dict(rows=1 << 31),
                dict(T=1 << 30, k=2), dict(w=ctypes.c_void_p(4098))):
        assert fwd(**bad) == 2, bad

    def bwd(d=FAKE, Y=FAKE, rows=8, row_of=FAKE, w=None, T=4, k=2, N=16, used=None, flags=0,
            dY=FAKE, dw=FAKE):
        return b(d, Y, rows, row_of, w, T, k, N, used, flags, dY, dw, None, None)

    for bad in (dict(d=None), dict(Y=None), dict(row_of=None), dict(dY=None, dw=None),
                dict(flags=1), dict(flags=2), dict(flags=1, used=FAKE, dY=None)):
        assert bwd(**bad) == 1, bad
    for bad in (dict(d=OFF), dict(Y=OFF), dict(dY=OFF), dict(dw=ctypes.c_void_p(4098)),
                dict(used=ctypes.c_void_p(4098)), dict(N=4)):
        assert bwd(**bad) == 2, bad


def test_silu_mul_and_rows8_refusals(lib):
    def fwd(H=FAKE, rows=4, N=256, used=None, row_of=None, n=0, w=None, flags=0, act=FAKE,
            H8=None, s=None):
        return lib.gg_silu_mul(H, rows, N, used, row_of, n, w, flags, act, H8, s, None, None)

    for bad in (dict(H=None), dict(rows=-1), dict(N=0), dict(n=-1), dict(n=4), dict(act=None),
                dict(H8=FAKE), dict(s=FAKE), dict(flags=1), dict(flags=2), dict(flags=8)):
        assert fwd(**bad) == 1, bad
    for bad in (dict(N=128), dict(N=264), dict(N=24, flags=4), dict(H=OFF), dict(act=OFF),
                dict(H8=OFF, s=FAKE), dict(rows=1 << 30), dict(row_of=FAKE, n=1 << 30),
                dict(w=ctypes.c_void_p(4098))):
        assert fwd(**bad) == 2, bad

    def bwd(d=FAKE, H=None, H8=FAKE, s=FAKE, rows=4, N=256, dH=FAKE, act=None, flags=0):
        return lib.gg_silu_mul_backward(d, H, H8, s, rows, N, None, None, 0, None, flags, dH,
                                        act, None, None, None)

    for bad in (dict(d=None), dict(H8=None), dict(s=None), dict(H=FAKE), dict(dH=None),
                dict(H8=None, s=None)):
        assert bwd(**bad) == 1, bad
    for bad in (dict(d=OFF), dict(H8=OFF), dict(dH=OFF), dict(act=OFF)):
        assert bwd(**bad) == 2, bad
    p, u = lib.gg_pack8, lib.gg_unpack8
    assert p(None, 4, 8, None, FAKE, FAKE, None, None) == 1
    assert p(FAKE, 4, 0, None, FAKE, FAKE, None, None) == 1
    assert p(FAKE, 4, 12, None, FAKE, FAKE, None, None) == 2
    assert p(OFF, 4, 8, None, FAKE, FAKE, None, None) == 2
    assert u(FAKE, None, 4, 8, None, 0, FAKE, None, None) == 1
    assert u(FAKE, FAKE, 4, 8, None, 1, FAKE, None, None) == 1   # a tail needs a count
    assert u(FAKE, FAKE, 4, 8, None, 4, FAKE, None, None) == 1
    assert u(FAKE, FAKE, 4, 8, None, 0, OFF, None, None) == 2


def test_binding_refuses_host_tensors_and_types():
    import moe_grouped_gemm_ragged_b200 as gg
    bf = torch.zeros(4, 256, dtype=torch.bfloat16)
    i32 = torch.zeros(8, dtype=torch.int32)
    with pytest.raises(TypeError):
        gg.gate_topk(torch.zeros(4, 8, dtype=torch.float16), 2)
    for call in (lambda: gg.gate_topk(bf, 2), lambda: gg.unroute(bf, i32, 2),
                 lambda: gg.unroute_backward(bf, i32, 2, bf), lambda: gg.silu_mul(bf),
                 lambda: gg.silu_mul_backward(bf, H=bf), lambda: gg.pack8(bf),
                 lambda: gg.unpack8(torch.zeros(4, 32, dtype=torch.float8_e4m3fn), bf)):
        with pytest.raises(ValueError, match="must be a CUDA tensor"):
            call()


def test_native_module_takes_only_what_it_can_check(lib):
    """Anything but device tensors (and too few arguments, or none bound) is left to the Python
    checks: None, and no error set."""
    from moe_grouped_gemm_ragged_b200 import _layer
    n = _layer._native
    assert n is not None, "csrc/binding.cpp has not been built for this interpreter"
    bf, i32 = torch.zeros(4, 256, dtype=torch.bfloat16), torch.zeros(4, dtype=torch.int32)
    assert n.unroute(bf, i32, 1, bf, None, None, None, None) is None
    assert n.unroute(bf) is None and n.pack8() is None
    assert n.gate_topk(bf, 2, 0, True, 1.0, None, None, None, None, None, None) is None
    assert n.gate_topk("x", None, 0, 1, 1, None, None, None, None, None, None) is None
    assert n.silu_mul(None, *[None] * 10) is None
    with pytest.raises(ValueError):
        n.bind("gg_forward", 1)
    with pytest.raises(ValueError):
        n.bind("gg_unroute")
    with pytest.raises(TypeError):
        n.bind("gg_unroute", "1")
