"""The operators around the grouped GEMM against their fp64 definitions.

Tolerances count roundings: u = 2^-24 is half a step of fp32, 2^-8 half a step of bf16, both
relative to the value. An fp32 sum of n products is off by at most n u sum |products| in any
order; expf, divisions and the fast exponential of the activation by a few units of 2^-23 each
(the fast one by 2 + 1.17 |x| of them). What a test adds on top of the final rounding is written
beside it.
"""
import ctypes

import numpy as np
import pytest
import torch

import oracle
import oracle.layer as ol
import workloads
from conftest import cuda_ok
from helpers import assert_close, is_sentinel, sentinel, to_f64

pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not cuda_ok(), reason="needs a CUDA device")]

gg = pytest.importorskip("moe_grouped_gemm_ragged_b200")

U, B = 2.0 ** -24, 2.0 ** -8
BF16_TINY, F32_TINY = 2.0 ** -133, 2.0 ** -126


def _near(got, ref, bound, what):
    assert got.shape == ref.shape, (what, got.shape, ref.shape)
    assert np.isfinite(got).all(), what
    over = np.abs(got - ref) - bound
    assert (over <= 0).all(), (what, np.unravel_index(np.argmax(over), over.shape), over.max())


def _status():
    return torch.zeros(1, dtype=torch.int32, device="cuda")


def _bf16(a):
    return torch.as_tensor(np.asarray(a, np.float32)).to(torch.bfloat16)


# -------------------------------------------------------------------------------- gate

def _check_gate(x, k, sigmoid, renorm, scale, bias=None, num=None, flagged=0):
    """Forward and backward of logits x (a torch tensor on the host) against the definition."""
    T, E = x.shape
    st = _status()
    how = dict(score=gg.GATE_SIGMOID if sigmoid else gg.GATE_SOFTMAX, renorm=renorm, scale=scale)
    xd = x.cuda()
    nt = None if num is None else torch.tensor([num], dtype=torch.int32, device="cuda")
    ids, w = gg.gate_topk(xd, k, bias=None if bias is None else bias.cuda(), num_tokens=nt,
                          status=st, **how)
    x64 = x.double().numpy()
    rids, rw = ol.gate(x64, k, sigmoid, renorm, scale,
                       None if bias is None else bias.double().numpy(), num)
    np.testing.assert_array_equal(ids.cpu().numpy(), rids)
    # exp of a rounded difference of up to ~50 (u each), sums of E terms, a division
    xs = np.where(rids >= 0, np.take_along_axis(x64, np.maximum(rids, 0), 1), 0)
    finite = np.where(np.isfinite(x64), x64, 0)
    far = np.abs(finite).max(1, keepdims=True) + np.abs(xs)
    rel = (far + 16 + E / 8) * 2 * U
    _near(w.cpu().double().numpy(), rw, np.abs(rw) * rel + F32_TINY, "weights")
    assert int(st.item()) & gg.DEV_ERROR_MASK == flagged
    # backward
    rng = np.random.default_rng(T + E)
    dw = rng.normal(size=(T, k)).astype(np.float32)
    dx = gg.gate_topk_backward(xd, ids, torch.from_numpy(dw).cuda(), **how)
    rdx = ol.gate_backward(x64, rids, dw.astype(np.float64), sigmoid, renorm, scale)
    # the terms of a logit's gradient before they cancel: |g| v and v sum |g v|, v <= 1
    g = np.abs(scale * dw) * (rids >= 0)
    v = np.abs(rw) / abs(scale)
    mean = (g * v).sum(1, keepdims=True)
    size = np.abs(np.zeros((T, E)))
    for s in range(k):
        rows = np.nonzero(rids[:, s] >= 0)[0]
        size[rows, rids[rows, s]] += (v * (g + mean))[rows, s]
    if not sigmoid and not renorm:
        size += mean * ol._softmax(ol._mask(x64))
    bound = size * (far.max(1, keepdims=True) + 32 + E / 8) * 4 * U + F32_TINY
    if x.dtype is torch.bfloat16:
        bound = bound + np.abs(rdx) * B * (1 + 2 * B) + bound * B
    _near(dx.cpu().double().numpy(), rdx, bound, "dlogits")


@pytest.mark.parametrize("T,E,k", [(1, 1, 1), (1, 64, 8), (5, 7, 7), (33, 32, 32), (130, 33, 3),
                                   (257, 64, 1), (64, 160, 6), (40, 256, 8), (9, 257, 5),
                                   (7, 1024, 32), (3, 1000, 1), (30, 96, 4), (30, 192, 8),
                                   (10, 384, 8), (8, 600, 6), (20, 128, 8)])
@pytest.mark.parametrize("sigmoid,renorm", [(False, False), (False, True), (True, False),
                                            (True, True)])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_gate(T, E, k, sigmoid, renorm, dtype):
    gen = torch.Generator().manual_seed(T * E + k)
    x = (2 * torch.randn(T, E, generator=gen)).to(dtype)  # bf16: many ties of neighbours
    _check_gate(x, k, sigmoid, renorm, 1.0 if renorm else 2.5)
    if sigmoid:
        _check_gate(x, k, True, renorm, 1.0, bias=0.3 * torch.randn(E, generator=gen))


@pytest.mark.parametrize("E,k,dtype", [(5, 5, torch.bfloat16), (33, 4, torch.float32),
                                       (64, 8, torch.bfloat16), (64, 6, torch.float32),
                                       (100, 3, torch.bfloat16), (128, 8, torch.float32),
                                       (160, 8, torch.bfloat16), (256, 6, torch.float32),
                                       (400, 2, torch.bfloat16), (1000, 32, torch.float32),
                                       # half as many experts a lane again
                                       (72, 8, torch.bfloat16), (96, 3, torch.float32),
                                       (90, 8, torch.float32), (136, 2, torch.float32),
                                       (192, 8, torch.bfloat16), (320, 6, torch.float32),
                                       (384, 8, torch.bfloat16), (264, 32, torch.bfloat16),
                                       (520, 8, torch.bfloat16), (768, 4, torch.float32)])
def test_gate_of_many_tokens(E, k, dtype):
    """Several tokens a warp (above 4096), the last group of them short, some not in use."""
    gen = torch.Generator().manual_seed(E)
    x = (2 * torch.randn(4099, E, generator=gen)).to(dtype)
    x[torch.rand(4099, E, generator=gen) < 0.2] = -float("inf")
    _check_gate(x, k, False, E % 2 == 0, 1.5, num=4090)
    _check_gate(x, k, True, E % 3 == 0, 1.0, num=4090,
                bias=0.3 * torch.randn(E, generator=gen) if E % 2 == 0 else None)


@pytest.mark.parametrize("sigmoid,renorm", [(False, False), (False, True), (True, False),
                                            (True, True)])
def test_gate_masks_and_far_values(sigmoid, renorm):
    """Tokens with every expert masked, with fewer than k left, masks of the type's lowest value
    (ordinary logits), scores far below what fp32 holds, both zeros, and large logits."""
    x = torch.randn(12, 40, generator=torch.Generator().manual_seed(7))
    x[0] = -float("inf")
    x[1, 2:] = -float("inf")
    x[2, 3:] = torch.finfo(torch.float32).min
    x[3] = torch.finfo(torch.float32).min
    x[4] = -40.0 + 0.5 * x[4]
    x[5] = 40.0 + 0.5 * x[5]
    x[6] = 0.0
    x[6, ::2] = -0.0
    x[7, :39] = -float("inf")
    num = 11
    x[11] = float("nan")  # not in use
    if sigmoid:  # the lowest value's score is 0 in 64 bits too: shares of nothing
        x[2, 3:], x[3] = -80.0, -80.0
    else:  # exp of (x - m) is 0 or 1 whatever |x| is: no rounding grows with it
        _check_far_softmax(x[2:4].clone(), renorm)
        x[2, 3:], x[3] = -60.0, -60.0
    _check_gate(x, 6, sigmoid, renorm, 1.5, num=num)


def _check_far_softmax(x, renorm):
    ids, w = gg.gate_topk(x.cuda(), 6, renorm=renorm)
    assert ids[0].tolist()[3:] == [3, 4, 5] and w[0, 3:].tolist() == [0.0] * 3
    assert abs(float(w[0].sum()) - 1) < 32 * U
    assert ids[1].tolist() == list(range(6))
    share = 1 / 6 if renorm else 1 / 40
    assert (w[1].cpu().double() - share).abs().max() < 32 * U * share
    dx = gg.gate_topk_backward(x.cuda(), ids, torch.ones_like(w), renorm=renorm)
    assert bool(torch.isfinite(dx).all())
    # p = 1/40 for all: dx_j = p ([j chosen] - 6 p); a renormalised sum of weights is constant
    want = torch.zeros(40, dtype=torch.float64)
    if not renorm:
        want -= 6 / 1600
        want[:6] += 1 / 40
    assert (dx[1].cpu().double() - want).abs().max() < 64 * U


def test_gate_flags_bad_logits_and_counts():
    x = torch.randn(6, 16, generator=torch.Generator().manual_seed(2))
    x[1, 3] = float("nan")
    x[2, 0] = float("inf")
    x[3, 7] = torch.tensor([-1], dtype=torch.int32).view(torch.float32)[0]  # NaN, sign set
    for z in (x, x.to(torch.bfloat16)):
        for renorm in (False, True):
            _check_gate(z, 4, False, renorm, 1.0, flagged=gg.DEV_BAD_LOGIT)
            _check_gate(z, 4, True, renorm, 1.0, flagged=gg.DEV_BAD_LOGIT)
    z = x.to(torch.bfloat16)
    z[3, 7], z[1, 3], z[2, 0] = 0.0, 1.0, 2.0
    z.view(torch.int16)[3, 7] = -1
    _check_gate(z, 4, False, False, 1.0, flagged=gg.DEV_BAD_LOGIT)
    x[3, 7] = 0.5
    bias = torch.zeros(16)
    bias[5] = float("nan")
    bias[6] = -float("inf")  # a mask, as such no error
    _check_gate(x[3:], 4, True, True, 1.0, bias=bias, flagged=gg.DEV_BAD_LOGIT)
    for num in (-3, 9):
        _check_gate(x[3:], 2, False, True, 1.0, num=num, flagged=gg.DEV_BAD_COUNT)
    ids = torch.tensor([[0, 16], [-1, 3]], dtype=torch.int32, device="cuda")
    st = _status()
    dx = gg.gate_topk_backward(x[3:5].cuda(), ids, torch.ones(2, 2, device="cuda"), renorm=False,
                               status=st)
    assert int(st.item()) == gg.DEV_BAD_ROUTE and bool(torch.isfinite(dx).all())
    ref = ol.gate_backward(x[3:5].double().numpy(), np.array([[0, -1], [-1, 3]]), np.ones((2, 2)),
                           renorm=False)
    _near(dx.cpu().double().numpy(), ref, 128 * U, "dlogits of valid ids")


def test_gate_bias_decides_close_calls():
    """Scores + bias that fp32 cannot tell apart: the choice follows 64 bits."""
    T, E = 64, 256
    gen = torch.Generator().manual_seed(11)
    x = torch.randn(T, E, generator=gen)
    want = torch.sigmoid(x[0].double())
    bias = (0.7 - want).float()  # every sum of token 0 lies within 2^-25 of 0.7
    _check_gate(x, 8, True, True, 1.0, bias=bias)


@pytest.mark.parametrize("E,k", [(33, 8), (64, 6), (200, 8), (300, 4), (1000, 32)])
def test_gate_neighbours_and_ties(E, k):
    """Logits that differ in their last bits only, logits of few distinct values, and biases of
    0: the order is that of the values, ties to the lowest expert."""
    gen = torch.Generator().manual_seed(E)
    near = 1.0 + torch.randint(0, 64, (40, E), generator=gen).float() * 2.0 ** -23
    few = torch.randint(-3, 4, (40, E), generator=gen).float()
    one = few.clone()
    one[:, E // 2:] = near[:, E // 2:]
    for x in (near, few, one, -near):
        _check_gate(x, k, False, True, 1.0)
        _check_gate(x, k, True, False, 1.0, bias=torch.zeros(E))
        _check_gate(x, k, True, True, 1.0, bias=0.125 * torch.randint(-1, 2, (E,), generator=gen))
    _check_gate(few.to(torch.bfloat16), k, False, False, 1.0)
    _check_gate(few.to(torch.bfloat16), k, True, True, 1.0, bias=torch.zeros(E))


# ----------------------------------------------------------------------------- unroute

def _routing(T, k, E, seed, dropped=0.1):
    """(row_of, offs, rows in use) of T tokens over E experts, some slots dropped."""
    rng = np.random.default_rng(seed)
    ids = np.stack([rng.permutation(E)[:k] for _ in range(T)]) if T else np.zeros((0, k), int)
    ids[rng.random(ids.shape) < dropped] = -1
    offs, row_of, _, _ = oracle.route(ids.astype(np.int32), torch.zeros(T, 8, dtype=torch.bfloat16),
                                      E)
    return row_of, offs, int(offs[-1])


@pytest.mark.parametrize("T,k,E,N", [(1, 1, 4, 8), (1, 8, 8, 2048), (3, 2, 5, 16), (37, 3, 6, 136),
                                     (130, 8, 16, 1160), (65, 10, 12, 264), (20, 33, 40, 520),
                                     (5, 8, 64, 7168), (2, 4, 16, 8200),
                                     # several tokens a thread (above 1184) of 1 to 9 slots
                                     (1301, 1, 4, 72), (1303, 2, 6, 264), (1250, 3, 6, 40),
                                     (1191, 4, 8, 1096), (1200, 5, 8, 24), (1187, 9, 12, 16),
                                     (600, 1, 4, 2312)])
@pytest.mark.parametrize("weighted,residual", [(False, False), (True, False), (True, True)])
def test_unroute(T, k, E, N, weighted, residual):
    row_of, offs, n = _routing(T, k, E, seed=T + N)
    rows = T * k
    gen = torch.Generator().manual_seed(T * N)
    Y = torch.randn(rows, N, generator=gen).to(torch.bfloat16)
    Y[n:] = float("nan")  # rows that nothing names
    w = torch.randn(T, k, generator=gen) if weighted else None
    if weighted:
        w[torch.from_numpy(row_of.reshape(T, k) < 0)] = float("nan")  # weights of dropped slots
    res = torch.randn(T, N, generator=gen).to(torch.bfloat16) if residual else None
    st = _status()
    rd, Yd = torch.from_numpy(row_of).cuda(), Y.cuda()
    wd = None if w is None else w.cuda()
    out = gg.unroute(Yd, rd, k, sentinel((T, N)), weights=wd,
                     residual=None if res is None else res.cuda(), status=st)
    w64 = None if w is None else w.double().numpy()
    r64 = None if res is None else to_f64(res)
    ref = ol.unroute(to_f64(Y), row_of, k, w64, r64)
    size = ol.unroute(np.abs(to_f64(Y)), row_of, k, None if w is None else np.abs(w64),
                      None if res is None else np.abs(r64))
    _near(to_f64(out), ref, np.abs(ref) * B + size * (k + 2) * U * (1 + B) + BF16_TINY, "out")
    # gradients
    d = torch.randn(T, N, generator=gen).to(torch.bfloat16)
    dY = sentinel((rows, N))
    dw = torch.full((T, k), 7.0, device="cuda") if weighted else None
    gg.unroute_backward(d.cuda(), rd, k, dY, Y=Yd if weighted else None, weights=wd, dweights=dw,
                        status=st)
    Yz = np.nan_to_num(to_f64(Y))
    rdY, rdw = ol.unroute_backward(to_f64(d), Yz, row_of, k, w64)
    _near(to_f64(dY[:n]), rdY[:n], np.abs(rdY[:n]) * (B + 2 * U) + BF16_TINY, "dY")
    assert bool(is_sentinel(dY[n:]).all())
    if weighted:
        size = ol.unroute_backward(np.abs(to_f64(d)), np.abs(Yz), row_of, k)[1]
        # a thread's chain of products, then the tree over threads
        _near(dw.cpu().double().numpy(), rdw, size * (N / 32 + 16) * U + F32_TINY, "dweights")
        only = torch.empty_like(dw)  # either gradient alone
        gg.unroute_backward(d.cuda(), rd, k, None, Y=Yd, dweights=only)
        assert torch.equal(only, dw)
    tail = sentinel((rows, N))
    gg.unroute_backward(d.cuda(), rd, k, tail, weights=wd, offs=torch.from_numpy(offs).cuda(),
                        zero_tail=True, status=st)
    assert torch.equal(tail[:n].view(torch.int16), dY[:n].view(torch.int16))
    assert bool((tail[n:].view(torch.int16) == 0).all())
    assert int(st.item()) == 0


def test_unroute_of_nothing_in_place_and_bad_rows():
    empty = torch.empty(0, 64, dtype=torch.bfloat16, device="cuda")
    none = torch.empty(0, dtype=torch.int32, device="cuda")
    assert gg.unroute(empty, none, 4).shape == (0, 64)
    # every slot dropped: the residual itself, in place; without it zeros
    row_of = torch.full((6,), -1, dtype=torch.int32, device="cuda")
    x = torch.randn(3, 64, device="cuda").to(torch.bfloat16)
    keep = x.clone()
    assert gg.unroute(empty, row_of, 2, x, residual=x) is x and torch.equal(x, keep)
    assert bool((gg.unroute(empty, row_of, 2).view(torch.int16) == 0).all())
    # a row past Y is dropped and flagged, in every direction
    Y = torch.randn(4, 64, device="cuda").to(torch.bfloat16)
    row_of = torch.tensor([0, 4, 3, -5, 2 ** 31 - 1, 1], dtype=torch.int32, device="cuda")
    st = _status()
    out = gg.unroute(Y, row_of, 2, status=st)
    assert int(st.item()) == gg.DEV_BAD_ROUTE
    assert torch.equal(out, Y[[0, 3, 1]])
    st.zero_()
    dY, dw = sentinel((4, 64)), torch.full((3, 2), 9.0, device="cuda")
    gg.unroute_backward(x, row_of, 2, dY, Y=Y, dweights=dw, status=st)
    assert int(st.item()) == gg.DEV_BAD_ROUTE
    assert torch.equal(dY[[0, 3, 1]], x) and bool(is_sentinel(dY[2]).all())
    assert (dw.cpu() == 0).tolist() == [[False, True], [False, True], [True, False]]


def test_unroute_same_row_twice_and_shared_tokens():
    """Forward reads may repeat a row; the sum is that of the slots."""
    Y = torch.randn(2, 32, device="cuda").to(torch.bfloat16)
    row_of = torch.tensor([1, 1, 0, 0], dtype=torch.int32, device="cuda")
    out = gg.unroute(Y, row_of, 2, weights=torch.full((2, 2), 0.5, device="cuda"))
    assert torch.equal(out, Y.flip(0))


def test_unroute_past_32_bit_offsets():
    """The last row of a Y of more than 2^31 elements."""
    rows, N = 270000, 8192
    Y = torch.empty(rows, N, dtype=torch.bfloat16, device="cuda")
    Y[rows - 2:] = torch.randn(2, N, device="cuda").to(torch.bfloat16)
    row_of = torch.tensor([rows - 1, rows - 2], dtype=torch.int32, device="cuda")
    out = gg.unroute(Y, row_of, 1)
    assert torch.equal(out, Y[rows - 2:].flip(0))
    d = torch.randn(2, N, device="cuda").to(torch.bfloat16)
    gg.unroute_backward(d, row_of, 1, Y)
    assert torch.equal(Y[rows - 2:].flip(0), d)


# ------------------------------------------------------------------- 8-bit rows, SiLU-and-mul

def _wild_rows(R, C, seed):
    """bf16 rows whose blocks span the exponents, with zero blocks, the largest and the
    smallest numbers."""
    rng = np.random.default_rng(seed)
    x = rng.normal(size=(R, C)) * np.exp2(rng.integers(-30, 30, (R, 1)))
    x[rng.random((R, C)) < 0.1] *= 2.0 ** -12
    x[rng.random((R, C)) < 0.05] = 0.0
    x = _bf16(x)
    x[0, :16] = 0.0
    if R > 3:
        x[1] = 2.0 ** -133
        x[2, 0] = 3.38e38
        x[3] = -0.0
    return x


@pytest.mark.parametrize("R,C", [(1, 8), (1, 2048), (5, 32), (3, 40), (65, 136), (130, 1160),
                                 (4, 8200), (7, 56),
                                 (1201, 264), (1190, 1160)])  # a warp a row of several pieces
def test_rows8_bit_exact(R, C):
    x = _wild_rows(R, C, R + C)
    blocks = -(-C // 32)
    for used in (R, R // 2, 0):
        offs = torch.tensor([0, used], dtype=torch.int32, device="cuda")
        x8 = torch.full((R, C), 0x55, dtype=torch.uint8, device="cuda").view(torch.float8_e4m3fn)
        sc = torch.full((R, blocks), 0x55, dtype=torch.uint8, device="cuda").view(
            torch.float8_e8m0fnu)
        st = _status()
        gg.pack8(x.cuda(), x8, sc, offs=offs, status=st)
        ref, codes = ol.pack8(to_f64(x))
        np.testing.assert_array_equal(sc.view(torch.uint8)[:used].cpu().numpy(), codes[:used])
        assert bool((sc.view(torch.uint8)[used:] == 0x55).all())
        assert bool((x8.view(torch.uint8)[used:] == 0x55).all())
        back = gg.unpack8(x8, sc, sentinel((R, C)), offs=offs, status=st)
        np.testing.assert_array_equal(to_f64(back[:used]), ref[:used])
        assert bool(is_sentinel(back[used:]).all())
        # what the two tensors stand for, by torch's own types
        mean = x8.float() * sc.float().repeat_interleave(32, 1)[:, :C]
        np.testing.assert_array_equal(mean[:used].double().cpu().numpy(), ref[:used])
        gg.unpack8(x8, sc, back, offs=offs, zero_tail=True, status=st)
        assert bool((back[used:].view(torch.int16) == 0).all())
        assert int(st.item()) == 0


def test_rows8_not_finite_and_bad_count():
    x = torch.randn(2, 64, generator=torch.Generator().manual_seed(1)).to(torch.bfloat16)
    x[0, 3], x[0, 40], x[1, 0] = float("nan"), float("inf"), -float("inf")
    x8, sc = gg.pack8(x.cuda())
    ref, codes = ol.pack8(to_f64(x))
    np.testing.assert_array_equal(sc.view(torch.uint8).cpu().numpy(), codes)
    np.testing.assert_array_equal(to_f64(gg.unpack8(x8, sc)), ref)  # NaN where x is not finite
    for count, used in ((-1, 0), (3, 2)):
        st = _status()
        back = gg.unpack8(x8, sc, sentinel((2, 64)), status=st,
                          offs=torch.tensor([count], dtype=torch.int32, device="cuda"))
        assert int(st.item()) == gg.DEV_BAD_COUNT and bool(is_sentinel(back[used:]).all())


def _silu_bounds(H, d, concat, w):
    """How far fp32 arithmetic may be off in act, dH and dweights' terms: relative to each
    product before any cancels. sigma: 2 + 1.17 |g| units of 2^-23 from the exponential, 3 from
    the quotient; 8 more products and sums."""
    cg, cu = ol.halves(H.shape[1], concat)
    g, u = H[:, cg], H[:, cu]
    with np.errstate(over="ignore"):
        q = 1 / (1 + np.exp(-g))
    rel = (16 + 1.2 * np.abs(g)) * 2 * U
    s = 1.0 if w is None else np.abs(w)[:, None]
    act = np.abs(g * q * u) * rel
    dH = np.empty(H.shape)
    dH[:, cg] = s * np.abs(d * u) * (q + np.abs(g) * q * (1 - q)) * rel * 2
    # 1 - q from a rounded q is off by 2^-24 and q's error whatever its size
    dH[:, cg] += s * np.abs(d * u * g) * q * q * rel
    dH[:, cu] = s * np.abs(d * g) * q * rel
    return s * act, dH, (np.abs(d) * act).sum(1), (np.abs(d * g * u) * q).sum(1)


# sigma below 2^-126 is 0 in the kernels: g u sigma is then below 2^-118 for |g u| < 2^8
FLUSHED = 2.0 ** -100


@pytest.mark.parametrize("rows,N,concat", [(1, 256, False), (8, 1536, True), (37, 512, False),
                                           (5, 16, True), (9, 80, True), (33, 1040, True),
                                           (3, 4096, False), (2, 16400, True),
                                           # a warp a row of several pieces
                                           (1195, 528, True), (1190, 2048, False),
                                           (1186, 2576, True)])
@pytest.mark.parametrize("weighted", [False, True])
@pytest.mark.parametrize("ckpt", [False, True])
def test_silu_mul(rows, N, concat, weighted, ckpt):
    """Rows before a count, forward and backward, from bf16 and from the 8-bit form."""
    used = rows - rows // 4
    rng = np.random.default_rng(rows * N)
    H = _bf16(3 * rng.normal(size=(rows, N)))
    H[0, :8] = _bf16([0, -0.0, 90, -90, -1.28, 20, -20, 1e-30])
    H[used:] = float("nan")
    d = _bf16(rng.normal(size=(rows, N // 2)))
    d[used:] = float("nan")
    w = torch.from_numpy(rng.normal(size=rows).astype(np.float32)) if weighted else None
    wd = None if w is None else w.cuda()
    w64 = None if w is None else w.double().numpy()[:used]
    offs = torch.tensor([0, used, used], dtype=torch.int32, device="cuda")
    st = _status()
    H8 = s8 = None
    if ckpt:
        H8 = torch.zeros(rows, N, dtype=torch.uint8, device="cuda").view(torch.float8_e4m3fn)
        s8 = torch.zeros(rows, 2 * -(-N // 64), dtype=torch.uint8, device="cuda").view(
            torch.float8_e8m0fnu)
    how = dict(offs=offs, weights=wd, gate_up_concat=concat, status=st)
    act = gg.silu_mul(H.cuda(), sentinel((rows, N // 2)), H8=H8, H8_scale=s8, **how)
    h64, d64 = to_f64(H)[:used], to_f64(d)[:used]
    ref = ol.silu_mul(h64, concat, w64)
    b_act = _silu_bounds(h64, d64, concat, w64)[0]
    _near(to_f64(act[:used]), ref, np.abs(ref) * B + b_act * 2 + FLUSHED, "act")
    assert bool(is_sentinel(act[used:]).all())
    if ckpt:
        h64 = ol.pack8_halves(h64, concat)
        assert bool((H8.view(torch.uint8)[used:] == 0).all())
    dH, again = sentinel((rows, N)), sentinel((rows, N // 2))
    dw = torch.full((rows,), 7.0, device="cuda") if weighted else None
    gg.silu_mul_backward(d.cuda(), dH, H=None if ckpt else H.cuda(), H8=H8, H8_scale=s8,
                         act=again, dweights=dw, **how)
    rdH, rdw = ol.silu_mul_backward(d64, h64, concat, w64)
    ref = ol.silu_mul(h64, concat, w64)
    b_act, b_dH, b_dot, size = _silu_bounds(h64, d64, concat, w64)
    _near(to_f64(dH[:used]), rdH, np.abs(rdH) * B + b_dH * 2 + FLUSHED, "dH")
    _near(to_f64(again[:used]), ref, np.abs(ref) * B + b_act * 2 + FLUSHED, "act again")
    assert bool(is_sentinel(dH[used:]).all()) and bool(is_sentinel(again[used:]).all())
    if weighted:
        bound = b_dot + size * (N / 64 + 16) * U + FLUSHED
        _near(dw[:used].cpu().double().numpy(), rdw, bound, "dweights")
        assert bool((dw[used:] == 7).all())
    # the tail cleared instead
    gg.silu_mul(H.cuda(), act, zero_tail=True, **how)
    gg.silu_mul_backward(d.cuda(), dH, H=None if ckpt else H.cuda(), H8=H8, H8_scale=s8,
                         act=again, zero_tail=True, **how)
    for t in (act, dH, again):
        assert bool((t[used:].view(torch.int16) == 0).all())
    assert int(st.item()) == 0


@pytest.mark.parametrize("T,k,E,N,concat", [(1, 8, 8, 256, False), (29, 3, 6, 528, True),
                                            (50, 4, 9, 1024, False), (700, 2, 5, 784, True)])
def test_silu_mul_by_assignment(T, k, E, N, concat):
    """row_of and weights in the order of the gate equal the same weights by row, bit for bit;
    dropped slots (weights NaN) get gradient 0, an entry past the rows in use is flagged."""
    row_of, offs, n = _routing(T, k, E, seed=T, dropped=0.2)
    rng = np.random.default_rng(T)
    rows = T * k
    H, d = _bf16(rng.normal(size=(rows, N))).cuda(), _bf16(rng.normal(size=(rows, N // 2))).cuda()
    w = torch.from_numpy(rng.normal(size=(T, k)).astype(np.float32))
    live = torch.from_numpy(row_of >= 0)
    w.view(-1)[~live] = float("nan")
    by_row = torch.zeros(rows)
    by_row[torch.from_numpy(row_of[row_of >= 0]).long()] = w.view(-1)[live]
    offs_d, rd = torch.from_numpy(offs).cuda(), torch.from_numpy(row_of).cuda()
    st = _status()
    runs = []
    for kw in (dict(row_of=rd, weights=w.cuda()), dict(weights=by_row.cuda())):
        kw |= dict(offs=offs_d, gate_up_concat=concat, zero_tail=True, status=st)
        H8 = torch.zeros(rows, N, dtype=torch.uint8, device="cuda").view(torch.float8_e4m3fn)
        s8 = torch.zeros(rows, 2 * -(-N // 64), dtype=torch.uint8, device="cuda").view(
            torch.float8_e8m0fnu)
        act = gg.silu_mul(H, sentinel((rows, N // 2)), H8=H8, H8_scale=s8, **kw)
        again, dw = sentinel((rows, N // 2)), torch.full_like(kw["weights"], 7.0)
        dH = gg.silu_mul_backward(d, sentinel((rows, N)), H8=H8, H8_scale=s8, act=again,
                                  dweights=dw, **kw)
        runs.append([t.view(torch.uint8) for t in (act, H8, s8, again, dH)] + [dw.cpu()])
    for a, b in zip(runs[0][:-1], runs[1][:-1]):
        assert torch.equal(a, b)
    dw = runs[0][-1].view(-1)
    assert torch.equal(dw[live], runs[1][-1][torch.from_numpy(row_of[row_of >= 0]).long()])
    assert bool((dw[~live] == 0).all())
    assert int(st.item()) == 0
    bad = rd.clone()
    bad[0] = n  # past the rows in use
    gg.silu_mul(H, sentinel((rows, N // 2)), offs=offs_d, row_of=bad, gate_up_concat=concat,
                status=st)
    assert int(st.item()) == gg.DEV_BAD_ROUTE


def test_rows8_and_silu_mul_past_32_bit_offsets():
    """The last rows of an H of more than 2^31 elements."""
    rows, N = 270000, 8192
    H = torch.empty(rows, N, dtype=torch.bfloat16, device="cuda")
    H[rows - 2:] = torch.randn(2, N, device="cuda").to(torch.bfloat16)
    want8 = ol.pack8_halves(to_f64(H[rows - 2:]), False)
    H8 = torch.empty(rows, N, dtype=torch.float8_e4m3fn, device="cuda")
    s8 = torch.empty(rows, N // 32, dtype=torch.float8_e8m0fnu, device="cuda")
    row_of = torch.tensor([rows - 1, rows - 2], dtype=torch.int32, device="cuda")
    act = gg.silu_mul(H, row_of=row_of, H8=H8, H8_scale=s8)
    small = gg.silu_mul(H[rows - 2:].clone())
    assert torch.equal(act[rows - 2:], small)
    dH = gg.silu_mul_backward(act, H8=H8, H8_scale=s8, row_of=row_of)
    assert torch.equal(dH[rows - 2:], gg.silu_mul_backward(
        small, H8=H8[rows - 2:].clone(), H8_scale=s8[rows - 2:].clone()))
    del act, dH
    H[:rows - 2] = 0
    gg.pack8(H, H8, s8)
    gg.unpack8(H8, s8, H)
    np.testing.assert_array_equal(to_f64(H[rows - 2:]), want8)  # blocks of 32 either way
    assert bool((H[:rows - 2:4999] == 0).all())


def test_silu_mul_of_no_assignment():
    """An empty row_of names no row, whatever the rows in use are; the tail is cleared all the
    same."""
    H, d = (torch.randn(6, n, device="cuda").to(torch.bfloat16) for n in (256, 128))
    none = torch.empty(0, dtype=torch.int32, device="cuda")
    offs = torch.tensor([4], dtype=torch.int32, device="cuda")
    for kw in (dict(), dict(offs=offs), dict(offs=offs, zero_tail=True)):
        act = gg.silu_mul(H, sentinel((6, 128)), row_of=none, **kw)
        dH = gg.silu_mul_backward(d, sentinel((6, 256)), H=H, row_of=none, **kw)
        kept = 4 if "zero_tail" in kw else 6
        for t in (act, dH):
            assert bool(is_sentinel(t[:kept]).all())
            assert bool((t[kept:].view(torch.int16) == 0).all())


# ---------------------------------------------------------------------------- run together

def _layer_inputs(T=96, K=256, E=8, k=3, N=512, K2=256, seed=17):
    gen = torch.Generator().manual_seed(seed)
    X = torch.randn(T, K, generator=gen).to(torch.bfloat16)
    x = torch.randn(T, E, generator=gen)
    x[5] = -float("inf")   # a token without experts
    x[9, 2:] = -float("inf")
    W1 = (torch.randn(E, K, N, generator=gen) / 16).to(torch.bfloat16)
    W2 = (torch.randn(E, N // 2, K2, generator=gen) / 16).to(torch.bfloat16)
    res = torch.randn(T, K2, generator=gen).to(torch.bfloat16)
    dout = torch.randn(T, K2, generator=gen).to(torch.bfloat16)
    return X, x, W1, W2, res, dout


@pytest.mark.parametrize("ckpt8", [False, True])
@pytest.mark.parametrize("where", ["activation", "combine"])
def test_layer_forward_and_gradients(ckpt8, where):
    """gate -> dispatch -> expert products -> combine as a layer uses them, against the layer in
    64 bits, rounded where the layer stores bf16. Off by the last rounding (2^-8) and by single
    neighbours' roundings inside the sums; the bound is that of the grouped GEMM's own tests
    (1e-2 relative plus 1e-2)."""
    X, x, W1, W2, res, dout = _layer_inputs()
    T, k, E = 96, 3, 8
    leaves = [t.cuda().requires_grad_(True) for t in (X, x, W1, W2, res)]
    Xd, xd, W1d, W2d, rd = leaves
    st = _status()
    ids, w = gg.gate(xd, k, status=st)
    A, row_of, offs = gg.dispatch(Xd, ids, E, status=st)
    if where == "activation":
        Y = gg.expert_mlp(A, W1d, W2d, offs, row_of=row_of, weights=w, ckpt8=ckpt8, status=st)
        out = gg.combine(Y, row_of, k, residual=rd, offs=offs, status=st)
    else:
        H = gg.grouped_mm(A, W1d, offs, ckpt8=ckpt8)
        Y = gg.grouped_mm(gg.swiglu(H, offs, ckpt8=ckpt8, status=st), W2d, offs, ckpt8=ckpt8)
        out = gg.combine(Y, row_of, k, weights=w, residual=rd, offs=offs, status=st)
    grads = torch.autograd.grad(out, leaves, dout.cuda())
    assert int(st.item()) & gg.DEV_ERROR_MASK == 0

    def r16(a):  # as stored
        return oracle.bf16_to_f64(oracle.round_bf16(a))

    x64 = x.double().numpy()
    rids, rw = ol.gate(x64, k)
    np.testing.assert_array_equal(ids.cpu().numpy(), rids)
    roffs, rrow, rA, _ = oracle.route(rids.astype(np.int32), X, E)
    n = int(roffs[-1])
    seg = np.repeat(np.arange(E), np.diff(np.concatenate([[0], roffs])))
    A64 = oracle.bf16_to_f64(rA)
    W164, W264 = to_f64(W1), to_f64(W2)
    live = rrow >= 0
    wrow = np.zeros(n)
    wrow[rrow[live]] = rw.reshape(-1)[live]
    H64 = r16(np.einsum("rk,rkn->rn", A64, W164[seg]))
    inside = wrow if where == "activation" else None
    act = r16(ol.silu_mul(H64, False, inside))
    Y64 = r16(np.einsum("rj,rjk->rk", act, W264[seg]))
    outer = None if where == "activation" else rw
    ref = ol.unroute(Y64, rrow, k, outer, to_f64(res))
    assert_close(to_f64(out.detach()), ref, "out")
    # backward
    d64 = to_f64(dout)
    dY64, dw64 = ol.unroute_backward(d64, Y64, rrow, k, outer)
    dY64 = r16(dY64)
    dact = r16(np.einsum("rk,rjk->rj", dY64, W264[seg]))
    Hb = ol.pack8_halves(H64, False) if ckpt8 else H64
    dH64, dwr = ol.silu_mul_backward(dact, Hb, False, inside)
    dH64 = r16(dH64)
    if where == "activation":
        again = r16(ol.silu_mul(Hb, False, inside))
        dw64 = np.zeros((T, k))
        dw64.reshape(-1)[live] = dwr[rrow[live]]
    else:
        again = ol.pack8(act)[0] if ckpt8 else act
    dA = r16(np.einsum("rn,rkn->rk", dH64, W164[seg]))
    Ab = ol.pack8(A64)[0] if ckpt8 else A64
    dW1, dW2 = np.zeros(W164.shape), np.zeros(W264.shape)
    for e in range(E):
        m = seg == e
        dW1[e], dW2[e] = Ab[m].T @ dH64[m], again[m].T @ dY64[m]
    assert_close(to_f64(grads[0]), ol.unroute(dA, rrow, k), "dX")
    assert_close(grads[1].cpu().double().numpy(), ol.gate_backward(x64, rids, dw64), "dlogits")
    assert_close(to_f64(grads[2]), dW1, "dW1")
    assert_close(to_f64(grads[3]), dW2, "dW2")
    assert torch.equal(grads[4].cpu(), dout)


@pytest.mark.parametrize("ckpt8", [False, True])
@pytest.mark.parametrize("T,used", [(0, 0), (1, 1), (5, 0), (40, 13)])
def test_layer_of_few_and_of_unused_tokens(T, used, ckpt8):
    """No token, one, a padded batch without any and with some: outputs and gradients of unused
    tokens are the residual's and zeros, those of the others as if the batch were not padded."""
    X, x, W1, W2, res, dout = (t.cuda() for t in _layer_inputs())
    x[5], x[9] = x[6], x[7]
    k, E = 3, 8

    def layer(n, num):
        leaves = [t.clone().requires_grad_(True) for t in (X[:n], x[:n], W1, W2, res[:n])]
        st = _status()
        ids, w = gg.gate(leaves[1], k, num_tokens=num, status=st)
        A, row_of, offs = gg.dispatch(leaves[0], ids, E, status=st)
        Y = gg.expert_mlp(A, leaves[2], leaves[3], offs, row_of=row_of, weights=w, ckpt8=ckpt8,
                          status=st)
        out = gg.combine(Y, row_of, k, residual=leaves[4], offs=offs, status=st)
        grads = torch.autograd.grad(out, leaves, dout[:n])
        assert int(st.item()) & gg.DEV_ERROR_MASK == 0
        return out.detach(), grads

    num = torch.tensor([used], dtype=torch.int32, device="cuda")
    out, grads = layer(T, num)
    want, wgrads = layer(used, None)
    assert torch.equal(out[:used], want) and torch.equal(out[used:], res[used:T])
    for i in (0, 1):
        assert torch.equal(grads[i][:used], wgrads[i])
        assert bool((grads[i][used:] == 0).all())
    for i in (2, 3):
        assert torch.equal(grads[i], wgrads[i])
    if used == 0:
        assert bool((grads[2] == 0).all()) and bool((grads[3] == 0).all())


def test_expert_mlp_equals_its_parts():
    """expert_mlp without and with weights by row, W stored [E, N, K], both column layouts, with
    and without the 8-bit checkpoint, equals grouped_mm, swiglu and grouped_mm bit for bit."""
    rng = np.random.default_rng(12)
    offs = torch.tensor([0, 70, 70, 201], dtype=torch.int32, device="cuda")
    A = _bf16(rng.normal(size=(210, 128))).cuda()
    A[201:] = float("nan")
    W1, W2 = _bf16(rng.normal(size=(4, 128, 512)) / 8).cuda(), _bf16(
        rng.normal(size=(4, 256, 136)) / 8).cuda()
    w = torch.rand(210, device="cuda")
    dY = _bf16(rng.normal(size=(210, 136))).cuda()
    for nk in (False, True):
        ws = [t.transpose(1, 2).contiguous() if nk else t for t in (W1, W2)]
        for concat in (False, True):
            for weights in (None, w):
                for ckpt8 in (False, True):
                    runs = []
                    for whole in (True, False):
                        leaves = [t.detach().clone().requires_grad_(True)
                                  for t in [A, *ws] + ([w] if weights is not None else [])]
                        wt = leaves[3] if weights is not None else None
                        if whole:
                            Y = gg.expert_mlp(leaves[0], leaves[1], leaves[2], offs, weights=wt,
                                              gate_up_concat=concat, w_nk=nk, ckpt8=ckpt8)
                        else:
                            H = gg.grouped_mm(leaves[0], leaves[1], offs, w_nk=nk, ckpt8=ckpt8)
                            act = gg.swiglu(H, offs, weights=wt, gate_up_concat=concat,
                                            ckpt8=ckpt8)
                            Y = gg.grouped_mm(act, leaves[2], offs, w_nk=nk)
                        runs.append([Y.detach(), *torch.autograd.grad(Y, leaves, dY)])
                    for i, (a, b) in enumerate(zip(*runs)):
                        if i == 3 and ckpt8:
                            continue  # W2's gradient: from the activation's second computation
                        assert torch.equal(a, b), (nk, concat, ckpt8, i)


def test_checkpoints_in_8_bits_take_half_the_memory():
    rows, K, N = 4096, 512, 1024
    offs = torch.tensor([rows // 2, rows], dtype=torch.int32, device="cuda")
    A = torch.randn(rows, K, device="cuda").to(torch.bfloat16).requires_grad_(True)
    W1 = torch.randn(2, K, N, device="cuda").to(torch.bfloat16).requires_grad_(True)
    W2 = torch.randn(2, N // 2, K, device="cuda").to(torch.bfloat16).requires_grad_(True)
    kept = []
    for ckpt8 in (False, True):
        before = torch.cuda.memory_allocated()
        # A is the caller's to free: a copy that only the layer holds
        Y = gg.expert_mlp(A * 1, W1, W2, offs, ckpt8=ckpt8)
        kept.append(torch.cuda.memory_allocated() - before - Y.nbytes)
        del Y
    whole = 2 * rows * (K + N)
    assert whole <= kept[0] < 1.01 * whole
    assert kept[1] <= whole * 33 / 64 + (1 << 16)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("score", ["GATE_SOFTMAX", "GATE_SIGMOID"])
def test_gate_gradient_of_an_only_expert_is_zero(score, dtype):
    """A renormalised weight of one slot is the scale whatever the logits: no rounding is left."""
    for T, E in ((5, 16), (300, 64), (5000, 160)):
        x = 3 * torch.randn(T, E, device="cuda").to(dtype)
        ids, w = gg.gate_topk(x, 1, score=getattr(gg, score), scale=2.5)
        assert bool((w == 2.5).all())
        dx = gg.gate_topk_backward(x, ids, torch.randn_like(w), score=getattr(gg, score),
                                   scale=2.5)
        assert bool((dx == 0).all())


@pytest.mark.parametrize("biased", [False, True])
@pytest.mark.parametrize("shift", [0.0, -10.0, -14.0, -16.0, -60.0, -86.0, -300.0])
def test_gate_shares_of_scores_far_below_one(shift, biased):
    """Sigmoid shares keep their precision however small the scores are. In units of U: e^-x 4, the
    sum under it 1, the quotient 4, their sum as much and its 4 additions, the share's quotient and
    the scale 2; the difference to the largest, at most 16, moves a share by 16."""
    gen = torch.Generator().manual_seed(9)
    x = torch.randn(300, 48, generator=gen) + shift
    bias = torch.randn(48, generator=gen) if biased else None
    ids, w = gg.gate_topk(x.cuda(), 5, score=gg.GATE_SIGMOID, scale=2.5,
                          bias=None if bias is None else bias.cuda())
    s = np.take_along_axis(x.double().numpy(), ids.cpu().numpy().astype(np.int64), 1)
    s = -np.logaddexp(0.0, -s)  # their logarithms
    s = np.exp(s - s.max(1, keepdims=True))
    ref = 2.5 * s / s.sum(1, keepdims=True)
    _near(w.cpu().double().numpy(), ref, 48 * U * ref + F32_TINY, "weights")


@pytest.mark.parametrize("sigmoid", [False, True])
def test_gate_gradient_of_gains_that_hardly_differ(sigmoid):
    """Renormalised weights whose gradients differ in their last bits: dx_i = v_i (g_i - sum g v),
    the differences of the g in full."""
    gen = torch.Generator().manual_seed(6)
    x = torch.randn(200, 32, generator=gen)
    dw = 1.0 + 2.0 ** -20 * torch.randint(-8, 9, (200, 4), generator=gen)
    score = gg.GATE_SIGMOID if sigmoid else gg.GATE_SOFTMAX
    ids, _ = gg.gate_topk(x.cuda(), 4, score=score)
    dx = gg.gate_topk_backward(x.cuda(), ids, dw.cuda(), score=score)
    ref = ol.gate_backward(x.double().numpy(), ids.cpu().numpy(), (dw.double() - 1).numpy(),
                           sigmoid)
    # |g| up to 2^-17; a few dozen roundings of products of that size
    _near(dx.cpu().double().numpy(), ref, 64 * U * 2.0 ** -16 + F32_TINY, "dlogits")


@pytest.mark.parametrize("sigmoid", [False, True])
def test_gate_gradient_with_a_large_gain_of_a_small_share(sigmoid):
    """A first slot of next to no share (a balancing bias can make one) and a large gain takes
    nothing from the others' gradients; a slot whose logit is masked counts for nothing at all."""
    gen = torch.Generator().manual_seed(7)
    T, E, k = 100, 16, 5
    x = torch.randn(T, E, generator=gen)
    ids = torch.arange(k, dtype=torch.int32).repeat(T, 1)
    dw = torch.randn(T, k, generator=gen)
    x[:, 0], dw[:, 0] = -25.0, 1e8
    x[50:, 2], dw[50:, 2] = -float("inf"), float("inf")
    score = gg.GATE_SIGMOID if sigmoid else gg.GATE_SOFTMAX
    dx = gg.gate_topk_backward(x.cuda(), ids.cuda(), dw.cuda(), score=score)
    live = np.where(np.isfinite(dw.numpy()), dw.double().numpy(), 0.0)
    ref = ol.gate_backward(x.double().numpy(), ids.numpy(), live, sigmoid)
    v = np.where(np.isfinite(x.numpy()), x.double().numpy(), -700.0)[:, :k]
    v = 1 / (1 + np.exp(-v)) if sigmoid else np.exp(v)
    v /= v.sum(1, keepdims=True)
    # each share is off by a few roundings and its exponent's, 25 U; the mean by those of its terms
    mean = (v * np.abs(live)).sum(1, keepdims=True)
    bound = np.full((T, E), F32_TINY)
    bound[:, :k] += 64 * U * v * (np.abs(live) + mean)
    _near(dx.cpu().double().numpy(), ref, bound, "dlogits")


def test_gate_gradient_of_an_expert_named_twice():
    """ids that gate_topk would not make: both slots add to their expert, in order."""
    x = torch.randn(3, 40, generator=torch.Generator().manual_seed(8))
    ids = torch.tensor([[4, 4, 4], [1, 2, 1], [39, -1, 39]], dtype=torch.int32)
    dw = torch.randn(3, 3, generator=torch.Generator().manual_seed(9))
    for score in (gg.GATE_SOFTMAX, gg.GATE_SIGMOID):
        for renorm in (False, True):
            dx = gg.gate_topk_backward(x.cuda(), ids.cuda(), dw.cuda(), score=score, renorm=renorm)
            ref = ol.gate_backward(x.double().numpy(), ids.numpy(), dw.double().numpy(),
                                   score == gg.GATE_SIGMOID, renorm)
            # |dw| below 4, a few dozen roundings
            _near(dx.cpu().double().numpy(), ref, 256 * U, "dlogits")
            again = gg.gate_topk_backward(x.cuda(), ids.cuda(), dw.cuda(), score=score,
                                          renorm=renorm)
            assert torch.equal(dx, again)


def test_captured_autograd_layer():
    """The autograd forms captured with their backward pass (leaves without an eager graph),
    replayed on new inputs, equal eager ones bit for bit."""
    inputs = [t.cuda() for t in _layer_inputs()]
    k, E = 3, 8

    def layer(leaves, dout):
        ids, w = gg.gate(leaves[1], k, score=gg.GATE_SIGMOID, scale=2.0)
        A, row_of, offs = gg.dispatch(leaves[0], ids, E)
        Y = gg.expert_mlp(A, leaves[2], leaves[3], offs, row_of=row_of, weights=w, ckpt8=True)
        out = gg.combine(Y, row_of, k, residual=leaves[4], offs=offs)
        return [out.detach(), *torch.autograd.grad(out, leaves, dout)]

    static = [t.clone().requires_grad_(i < 5) for i, t in enumerate(inputs)]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        for _ in range(2):
            layer(static[:5], static[5])
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        got = layer(static[:5], static[5])
    for seed in (1, 2):
        gen = torch.Generator(device="cuda").manual_seed(seed)
        with torch.no_grad():
            for s, t in zip(static, inputs):
                s.copy_(t.flip(0) + 0.25 * torch.randn(t.shape, generator=gen, device="cuda"))
        graph.replay()
        torch.cuda.synchronize()
        got_now = [t.clone() for t in got]
        fresh = [t.detach().clone().requires_grad_(i < 5) for i, t in enumerate(static)]
        for a, b in zip(got_now, layer(fresh[:5], fresh[5])):
            assert torch.equal(a, b)


def test_swiglu_weights_and_partial_gradients():
    """Gradients asked for one by one equal those asked for together; an expanded and a
    misaligned gradient are taken."""
    rng = np.random.default_rng(4)
    offs = torch.tensor([3, 11], dtype=torch.int32, device="cuda")
    H = _bf16(rng.normal(size=(16, 256))).cuda().requires_grad_(True)
    w = torch.rand(16, device="cuda", requires_grad=True)
    act = gg.swiglu(H, offs, weights=w, ckpt8=True)
    assert bool((act[11:] == 0).all())
    d = torch.ones((), dtype=torch.bfloat16, device="cuda").expand(16, 128)
    both = torch.autograd.grad(act, (H, w), d, retain_graph=True)
    odd = torch.ones(16 * 128 + 1, dtype=torch.bfloat16, device="cuda")[1:].view(16, 128)
    assert torch.equal(torch.autograd.grad(act, H, odd, retain_graph=True)[0], both[0])
    assert torch.equal(torch.autograd.grad(act, w, d)[0], both[1])
    assert bool((both[0][11:] == 0).all()) and bool((both[1][11:] == 0).all())
    Y = _bf16(rng.normal(size=(6, 64))).cuda().requires_grad_(True)
    row_of = torch.tensor([4, -1, 0, 2], dtype=torch.int32, device="cuda")
    out = gg.combine(Y, row_of, 2)
    (dY,) = torch.autograd.grad(out, Y, torch.ones_like(out))
    assert dY[:, 0].tolist() == [1, 0, 1, 0, 1, 0]  # rows that no slot names: 0


def test_captured_layer_step_replays_on_new_inputs():
    """Forward and backward of the operators in one CUDA graph, replayed on changed inputs,
    equal eager calls bit for bit (no allocation, no host read, workspaces of the caller)."""
    T, K, E, k, N = 64, 256, 8, 2, 512
    gen = torch.Generator(device="cuda").manual_seed(3)
    W1 = (torch.randn(E, K, N, generator=gen, device="cuda") / 16).to(torch.bfloat16)
    x = torch.empty(T, E, device="cuda")
    X = torch.empty(T, K, dtype=torch.bfloat16, device="cuda")
    num = torch.empty(1, dtype=torch.int32, device="cuda")
    dout = torch.randn(T, N // 2, generator=gen, device="cuda").to(torch.bfloat16)
    n = T * k
    bufs = dict(ids=(T, k, torch.int32), w=(T, k, torch.float32), A=(n, K, torch.bfloat16),
                H=(n, N, torch.bfloat16), act=(n, N // 2, torch.bfloat16),
                out=(T, N // 2, torch.bfloat16), dact=(n, N // 2, torch.bfloat16),
                dH=(n, N, torch.bfloat16), dw=(T, k, torch.float32), dx=(T, E, torch.float32),
                H8=(n, N, torch.uint8), s8=(n, N // 32, torch.uint8))
    b = {key: torch.zeros(r, c, dtype=t, device="cuda") for key, (r, c, t) in bufs.items()}
    row_of = torch.zeros(n, dtype=torch.int32, device="cuda")
    offs = torch.zeros(E, dtype=torch.int32, device="cuda")
    ws = torch.empty(max(4, gg.route_workspace_bytes(n, E)), dtype=torch.uint8, device="cuda")
    H8, s8 = b["H8"].view(torch.float8_e4m3fn), b["s8"].view(torch.float8_e8m0fnu)

    def step():
        gg.gate_topk(x, k, num_tokens=num, topk_ids=b["ids"], weights=b["w"])
        gg.route(b["ids"], X, E, A_packed=b["A"], row_of=row_of, offs=offs, workspace=ws)
        gg.forward(b["A"], W1, offs, b["H"])
        gg.silu_mul(b["H"], b["act"], offs=offs, H8=H8, H8_scale=s8)
        gg.unroute(b["act"], row_of, k, b["out"], weights=b["w"])
        gg.unroute_backward(dout, row_of, k, b["dact"], Y=b["act"], weights=b["w"],
                            dweights=b["dw"], offs=offs, zero_tail=True)
        gg.silu_mul_backward(b["dact"], b["dH"], H8=H8, H8_scale=s8, offs=offs)
        gg.gate_topk_backward(x, b["ids"], b["dw"], b["dx"])

    def fill(seed, used):
        g = torch.Generator(device="cuda").manual_seed(seed)
        x.copy_(torch.randn(T, E, generator=g, device="cuda"))
        X.copy_(torch.randn(T, K, generator=g, device="cuda"))
        num.fill_(used)
        for t in b.values():
            t.zero_()

    fill(1, T)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for seed, used in ((2, T), (3, 17), (4, 0)):
        fill(seed, used)
        graph.replay()
        torch.cuda.synchronize()
        got = {key: t.clone() for key, t in b.items()}
        fill(seed, used)
        step()
        torch.cuda.synchronize()
        for key, t in b.items():
            assert torch.equal(got[key].view(torch.uint8), t.view(torch.uint8)), (key, used)
        assert int(offs[-1]) == used * k
        assert bool((b["out"][used:].view(torch.int16) == 0).all())


def test_captured_branches_that_fork_and_join():
    """Calls on two branches of one capture, joined by a call that reads both, and two replays of
    two such graphs at the same time."""
    gen = torch.Generator(device="cuda").manual_seed(33)
    T, k, N = 500, 2, 1024
    x = torch.randn(T, 64, generator=gen, device="cuda")
    Y = torch.randn(T * k, N, generator=gen, device="cuda").to(torch.bfloat16)
    row_of = torch.randperm(T * k, generator=gen, device="cuda").to(torch.int32)

    def make():
        ids = torch.zeros(T, k, dtype=torch.int32, device="cuda")
        w, back = torch.zeros(T, k, device="cuda"), torch.zeros_like(Y)
        x8 = torch.zeros(T * k, N, dtype=torch.uint8, device="cuda").view(torch.float8_e4m3fn)
        s8 = torch.zeros(T * k, N // 32, dtype=torch.uint8, device="cuda").view(
            torch.float8_e8m0fnu)
        out = torch.zeros(T, N, dtype=torch.bfloat16, device="cuda")
        main, side = torch.cuda.Stream(), torch.cuda.Stream()

        def step():
            side.wait_stream(main)
            gg.gate_topk(x, k, topk_ids=ids, weights=w, stream=main)
            gg.pack8(Y, x8, s8, stream=side)
            gg.unpack8(x8, s8, back, stream=side)
            main.wait_stream(side)
            gg.unroute(back, row_of, k, out, weights=w, stream=main)

        torch.cuda.synchronize()
        step()
        torch.cuda.synchronize()
        want = out.clone()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=main):
            step()
        for t in (w, back, out):
            t.zero_()
        torch.cuda.synchronize()
        return graph, out, want

    a, b = make(), make()
    streams = torch.cuda.Stream(), torch.cuda.Stream()
    for _ in range(10):
        for (graph, _, _), stream in zip((a, b), streams):
            with torch.cuda.stream(stream):
                graph.replay()
    torch.cuda.synchronize()
    for _, out, want in (a, b):
        assert torch.equal(out.view(torch.int16), want.view(torch.int16))
    ids, w = gg.gate_topk(x, k)
    x8, s8 = gg.pack8(Y)
    assert torch.equal(a[2], gg.unroute(gg.unpack8(x8, s8), row_of, k, weights=w))


def test_chain_of_calls_needs_no_synchronisation():
    """Each call reads what the one before wrote, on one stream (a kernel may be scheduled while
    the one before it ends): the same bits as with a synchronisation after every call."""
    gen = torch.Generator(device="cuda").manual_seed(21)
    T, k, E, N = 900, 2, 64, 512
    x0 = torch.randn(T, E, generator=gen, device="cuda")
    Y0 = torch.randn(T * k, N, generator=gen, device="cuda").to(torch.bfloat16)
    row_of = torch.randperm(T * k, generator=gen, device="cuda").to(torch.int32)
    offs = torch.tensor([T * k - 5], dtype=torch.int32, device="cuda")

    def chain(sync):
        x, Y, seen = x0.clone(), Y0.clone(), []
        wait = torch.cuda.synchronize if sync else lambda: None
        out = torch.zeros(T, N, dtype=torch.bfloat16, device="cuda")
        dY, dw = torch.zeros_like(Y), torch.zeros(T, k, device="cuda")
        act = torch.zeros(T * k, N // 2, dtype=torch.bfloat16, device="cuda")
        dH, dx = torch.zeros_like(Y), torch.zeros_like(x)
        H8 = torch.zeros(T * k, N, dtype=torch.uint8, device="cuda").view(torch.float8_e4m3fn)
        s8 = torch.zeros(T * k, N // 32, dtype=torch.uint8, device="cuda").view(
            torch.float8_e8m0fnu)
        ids = torch.zeros(T, k, dtype=torch.int32, device="cuda")
        w = torch.zeros(T, k, device="cuda")
        for _ in range(6):
            for call in (lambda: gg.gate_topk(x, k, topk_ids=ids, weights=w),
                         lambda: gg.unroute(Y, row_of, k, out, weights=w),
                         lambda: gg.unroute_backward(out, row_of, k, dY, Y=Y, weights=w,
                                                     dweights=dw),
                         lambda: gg.gate_topk_backward(x, ids, dw, dx),
                         lambda: gg.silu_mul(dY, act, offs=offs, H8=H8, H8_scale=s8),
                         lambda: gg.silu_mul_backward(act, dH, H8=H8, H8_scale=s8, offs=offs),
                         lambda: gg.pack8(dH, H8, s8, offs=offs),
                         lambda: gg.unpack8(H8, s8, Y, offs=offs),
                         lambda: x.add_(dx, alpha=1e-3)):
                call()
                wait()
            seen += [t.clone() for t in (ids, w, out, dw, dx, Y)]
        torch.cuda.synchronize()
        return seen

    want = chain(True)
    for _ in range(3):
        for a, b in zip(chain(False), want):
            assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))


def test_calls_on_another_stream_own_their_buffers():
    """Buffers that a call allocates belong to the stream it runs on; results on a side stream
    equal those on the current one, also while both run."""
    gen = torch.Generator(device="cuda").manual_seed(5)
    x = torch.randn(300, 48, generator=gen, device="cuda")
    Y = torch.randn(600, 256, generator=gen, device="cuda").to(torch.bfloat16)
    row_of = torch.randperm(600, generator=gen, device="cuda").to(torch.int32)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()

    def calls(**kw):
        ids, w = gg.gate_topk(x, 2, **kw)
        x8, s = gg.pack8(Y, **kw)
        return [ids, w, gg.unroute(Y, row_of, 2, weights=w, **kw), gg.silu_mul(Y, **kw),
                gg.unpack8(x8, s, **kw)]

    here = calls()
    there = calls(stream=side)
    by_handle = calls(stream=side.cuda_stream)
    torch.cuda.synchronize()
    for a, b, c in zip(here, there, by_handle):
        assert torch.equal(a, b) and torch.equal(a, c)


def test_binding_refuses_shapes_strides_and_missing_arguments():
    Y = torch.zeros(8, 256, dtype=torch.bfloat16, device="cuda")
    row_of = torch.zeros(8, dtype=torch.int32, device="cuda")
    f32 = torch.zeros(4, 2, device="cuda")
    e8 = torch.zeros(8, 256, dtype=torch.float8_e4m3fn, device="cuda")
    for call, text in [
            (lambda: gg.unroute(Y, row_of, 3), "k entries"),
            (lambda: gg.unroute(Y.t(), row_of, 2), "contiguous"),
            (lambda: gg.unroute(Y, row_of, 2, weights=f32.view(2, 4)), "weights must have"),
            (lambda: gg.unroute_backward(Y[:4], row_of, 2), "one of dY"),
            (lambda: gg.unroute_backward(Y[:4], row_of, 2, dweights=f32), "needs Y"),
            (lambda: gg.unroute_backward(Y[:4], row_of, 2, Y, zero_tail=True), "needs offs"),
            (lambda: gg.unroute_backward(Y, row_of, 2, Y), "a row for each token"),
            (lambda: gg.silu_mul(Y, H8=e8), "go together"),
            (lambda: gg.silu_mul(Y, weights=f32[:3]), "hold 8 values"),
            (lambda: gg.silu_mul_backward(Y, H=None), "exactly one"),
            (lambda: gg.gate_topk(f32, 0), "positive"),
            (lambda: gg.gate_topk(f32, 1, score=5), "score must"),
            (lambda: gg.gate_topk_backward(f32, row_of.view(8, 1), f32), "disagree"),
            (lambda: gg.pack8(Y, offs=row_of[:0]), "not be empty")]:
        with pytest.raises(ValueError, match=text):
            call()
    with pytest.raises(gg.GGError, match="INVALID_ARG"):
        gg.gate_topk(f32, 3)
    with pytest.raises(gg.GGError, match="UNSUPPORTED"):
        gg.unroute(Y.view(-1)[1:1 + 4 * 256].view(4, 256), row_of[:4], 2)  # not on 16 bytes
    with pytest.raises(gg.GGError, match="UNSUPPORTED"):
        gg.silu_mul(Y[:, :128].contiguous())


def _calls(T=6, k=2, E=16, N=512):
    """Every call with all of its buffers: (function, positional, keywords)."""
    def t(*shape, dtype=torch.bfloat16):
        if dtype in (torch.bfloat16, torch.float32):
            gen = torch.Generator(device="cuda").manual_seed(sum(shape))
            return torch.randn(shape, generator=gen, device="cuda").to(dtype)
        if dtype is torch.int32:
            return torch.zeros(shape, dtype=dtype, device="cuda")
        return torch.zeros(shape, dtype=torch.uint8, device="cuda").view(dtype)

    f32, i32, e4, e8 = torch.float32, torch.int32, torch.float8_e4m3fn, torch.float8_e8m0fnu
    n = T * k
    row_of = torch.arange(n, dtype=i32, device="cuda")
    num = torch.tensor([T], dtype=i32, device="cuda")
    offs = torch.tensor([3, n], dtype=i32, device="cuda")
    st = t(1, dtype=i32)
    ids = torch.tensor([[1, 0]] * T, dtype=i32, device="cuda")
    by = dict(offs=offs, row_of=row_of, weights=t(T, k, dtype=f32), status=st)
    return [
        (gg.gate_topk, [t(T, E, dtype=f32), k],
         dict(score=gg.GATE_SIGMOID, bias=t(E, dtype=f32), num_tokens=num,
              topk_ids=t(T, k, dtype=i32), weights=t(T, k, dtype=f32), status=st)),
        (gg.gate_topk, [t(T, E), k], dict(topk_ids=t(T, k, dtype=i32),
                                          weights=t(T, k, dtype=f32))),
        (gg.gate_topk_backward, [t(T, E, dtype=f32), ids, t(T, k, dtype=f32),
                                 t(T, E, dtype=f32)], dict(status=st)),
        (gg.unroute, [t(n, N), row_of, k, t(T, N)],
         dict(weights=t(T, k, dtype=f32), residual=t(T, N), status=st)),
        (gg.unroute_backward, [t(T, N), row_of, k, t(n, N)],
         dict(Y=t(n, N), weights=t(T, k, dtype=f32), dweights=t(T, k, dtype=f32), offs=offs,
              zero_tail=True, status=st)),
        (gg.silu_mul, [t(n, N), t(n, N // 2)],
         dict(H8=t(n, N, dtype=e4), H8_scale=t(n, N // 32, dtype=e8), zero_tail=True, **by)),
        (gg.silu_mul, [t(n, N), t(n, N // 2)], dict(weights=t(n, dtype=f32),
                                                    gate_up_concat=True)),
        (gg.silu_mul_backward, [t(n, N // 2), t(n, N)],
         dict(H8=t(n, N, dtype=e4), H8_scale=t(n, N // 32, dtype=e8), act=t(n, N // 2),
              dweights=t(T, k, dtype=f32), **by)),
        (gg.silu_mul_backward, [t(n, N // 2), t(n, N)], dict(H=t(n, N), gate_up_concat=True)),
        (gg.pack8, [t(n, N), t(n, N, dtype=e4), t(n, N // 32, dtype=e8)],
         dict(offs=offs, status=st)),
        (gg.unpack8, [t(n, N, dtype=e4), t(n, N // 32, dtype=e8), t(n, N)],
         dict(offs=offs, zero_tail=True, status=st)),
    ]


def _tensors(fn, args, kw):
    """What a call was given and has written, as bytes."""
    fn(*args, **kw)
    return [t.clone().view(torch.uint8) for t in [*args, *kw.values()]
            if isinstance(t, torch.Tensor)]


def test_calls_without_the_native_module(monkeypatch):
    """The quick way into a call and the one through ctypes do the same."""
    from moe_grouped_gemm_ragged_b200 import _layer
    assert _layer._native is not None
    quick = [_tensors(*c) for c in _calls()]
    monkeypatch.setattr(_layer, "_native", None)
    for a, b in zip(quick, [_tensors(*c) for c in _calls()]):
        assert all(torch.equal(x, y) for x, y in zip(a, b))


@pytest.mark.parametrize("native", [True, False])
@pytest.mark.parametrize("call", range(11))
def test_every_tensor_argument_is_checked(call, native, monkeypatch):
    """Another type, one row more, strides, the host, a list in its place: each refused with a
    Python error, by either way into the call."""
    from moe_grouped_gemm_ragged_b200 import _layer
    if not native:
        monkeypatch.setattr(_layer, "_native", None)
    fn, args, kw = _calls()[call]
    names = [i for i, a in enumerate(args) if isinstance(a, torch.Tensor)]
    names += [key for key, a in kw.items() if isinstance(a, torch.Tensor)]
    for name in names:
        good = args[name] if isinstance(name, int) else kw[name]
        raw = good.view(torch.uint8) if good.element_size() == 1 else good
        longer = torch.cat([raw, raw[:1]]).view(good.dtype)
        bad = [raw.double(), good.cpu(), raw.tolist()]
        if name not in ("offs", "status") and not (fn is gg.unroute and name == 0):
            bad.append(longer)  # those are of any length
        if not (name in ("weights", "dweights") and fn in (gg.silu_mul, gg.silu_mul_backward)):
            bad.append(good[None])  # those are of any shape
        if good.numel() > 1 and good.element_size() > 1:
            bad.append(torch.stack([good, good], -1).select(-1, 0))
        for b in bad:
            a2, k2 = list(args), dict(kw)
            if isinstance(name, int):
                a2[name] = b
            else:
                k2[name] = b
            with pytest.raises((ValueError, TypeError)):
                fn(*a2, **k2)
