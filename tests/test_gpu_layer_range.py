"""The layer's operators at the ends of their value ranges, against their fp64 definitions.

Tolerances count roundings as in test_gpu_layer.py: u = 2^-24 is half a step of fp32, 2^-8 half a
step of bf16, both relative to the value.
"""
import numpy as np
import pytest
import torch

import oracle.layer as ol
from conftest import cuda_ok
from helpers import to_f64

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


def _bf16(a):
    return torch.as_tensor(np.asarray(a, np.float32)).to(torch.bfloat16)


# ----------------------------------------------------------------------------- SiLU-and-mul

def _check_silu_mul(g, u, d, w, concat, ckpt, units):
    """Both directions of rows with gates g, ups u and gradients d, weighted by w. A product is off
    by `units` u before its last rounding, and by bf16's smallest step where that is above it."""
    rows, half = g.shape
    cg, cu = ol.halves(2 * half, concat)
    H = torch.empty(rows, 2 * half, dtype=torch.bfloat16)
    H[:, cg], H[:, cu] = _bf16(g), _bf16(u)
    d, w = _bf16(d), torch.from_numpy(w.astype(np.float32))
    h64, d64, w64 = to_f64(H), to_f64(d), w.double().numpy()
    H8 = s8 = None
    if ckpt:
        H8 = torch.empty(rows, 2 * half, dtype=torch.float8_e4m3fn, device="cuda")
        s8 = torch.empty(rows, 2 * -(-half // 32), dtype=torch.uint8, device="cuda").view(
            torch.float8_e8m0fnu)
    how = dict(weights=w.cuda(), gate_up_concat=concat)
    act = gg.silu_mul(H.cuda(), H8=H8, H8_scale=s8, **how)
    ref = ol.silu_mul(h64, concat, w64)
    _near(to_f64(act), ref, np.abs(ref) * (B + units * U) + BF16_TINY, "act")
    if ckpt:
        h64 = ol.pack8_halves(h64, concat)
    again = torch.empty(rows, half, dtype=torch.bfloat16, device="cuda")
    dw = torch.empty(rows, device="cuda")
    dH = gg.silu_mul_backward(d.cuda(), H=None if ckpt else H.cuda(), H8=H8, H8_scale=s8,
                              act=again, dweights=dw, **how)
    ref = ol.silu_mul(h64, concat, w64)
    _near(to_f64(again), ref, np.abs(ref) * (B + units * U) + BF16_TINY, "act again")
    ref, rdw = ol.silu_mul_backward(d64, h64, concat, w64)
    _near(to_f64(dH), ref, np.abs(ref) * (B + units * U) + BF16_TINY, "dH")
    size = np.abs(d64 * ol.silu_mul(h64, concat)).sum(1)
    _near(dw.cpu().double().numpy(), rdw, size * (units + half) * U + F32_TINY, "dweights")


# four and eight lanes a row, a block a row, a warp a row of several pieces
@pytest.mark.parametrize("rows,N,concat", [(33, 256, False), (33, 80, True), (33, 4096, False),
                                           (11, 1040, True), (3, 16400, True), (1300, 1040, True)])
@pytest.mark.parametrize("ckpt", [False, True])
def test_silu_mul_of_large_gates(rows, N, concat, ckpt):
    """Above 2^8 sigma is 1 or 0, the slope of SiLU too: dg = w d u for every positive gate. A row
    has gates of one size, which its 8-bit blocks keep; ups and gradients are small enough for the
    products of 2^100. A handful of fp32 roundings in each product."""
    rng = np.random.default_rng(N)
    sizes = np.exp2([8, 16, 20, 22, 23, 24, 25, 26, 30, 60, 100])[np.arange(rows) % 11, None]
    g = sizes * rng.uniform(1, 2, (rows, N // 2)) * rng.choice([-1, 1], (rows, N // 2))
    u, d = (2.0 ** -20 * rng.normal(size=(rows, N // 2)) for _ in range(2))
    _check_silu_mul(g, u, d, rng.normal(size=rows), concat, ckpt, 8)


# four and eight lanes a row, a block a row, a warp a row of several pieces
@pytest.mark.parametrize("rows,N,concat", [(33, 256, False), (33, 80, True), (33, 4096, False),
                                           (11, 1040, True), (3, 16400, True), (1300, 1040, True)])
@pytest.mark.parametrize("ckpt", [False, True])
def test_silu_mul_of_far_negative_gates(rows, N, concat, ckpt):
    """Gates whose sigma is below fp32's normal numbers (-87.3) and then below fp32 itself: bf16
    holds g sigma(g) u down to 2^-133. sigma's power is off by 4 U for each of the factors that it
    is made of (four at most) and 1.3 times its argument, and there are a dozen products."""
    rng = np.random.default_rng(N)
    g = -np.array([60, 80, 87, 88, 89, 92, 100, 120, 150, 172, 180])[np.arange(rows) % 11, None]
    g = g * rng.uniform(1, 1.06, (rows, N // 2))
    u = np.exp2(rng.uniform(80, 126, (rows, N // 2))) * rng.choice([-1, 1], (rows, N // 2))
    d = 2.0 ** -3 * rng.normal(size=(rows, N // 2))
    _check_silu_mul(g, u, d, rng.normal(size=rows) / 16, concat, ckpt, 16 + 1.3 * 192 + 16)


# ------------------------------------------------------------------------------------- gate

@pytest.mark.parametrize("T,E,k", [(40, 7, 2), (64, 64, 4), (30, 160, 6), (12, 1000, 8),
                                   (4200, 64, 1), (4200, 64, 8), (4200, 200, 5)])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_gate_gradient_of_a_confident_expert(T, E, k, dtype):
    """Softmax over all experts with one of them 8 to 20 above the rest: its gradient
    p (g - sum p_i g_i) = p sum p_i (g - g_i) is many times smaller than g. In units of U: a power
    is off by 4 and 1.3 times its argument (25 at most), the total and the mean by one of these each,
    by E / 8 additions in a lane and 5 + 5 over the lanes, and there are a few products."""
    gen = torch.Generator().manual_seed(E + k)
    x = torch.randn(T, E, generator=gen).clamp(-2.5, 2.5)
    top = torch.randint(0, E, (T, 1), generator=gen)
    x.scatter_(1, top, 2.5 + 8 + 12 * torch.rand(T, 1, generator=gen))
    x = (x + torch.randn(T, 1, generator=gen)).to(dtype)
    for gains in (torch.ones(T, k), torch.randn(T, k, generator=gen)):
        ids, _ = gg.gate_topk(x.cuda(), k, renorm=False, scale=2.5)
        dx = gg.gate_topk_backward(x.cuda(), ids, gains.cuda(), renorm=False, scale=2.5)
        ids = ids.cpu().numpy()
        assert (ids[:, :1] == top.numpy()).all()
        x64, g64 = x.double().numpy(), gains.double().numpy()
        ref = ol.gate_backward(x64, ids, g64, renorm=False, scale=2.5)
        p, g = ol._softmax(x64), np.zeros((T, E))
        np.put_along_axis(g, ids.astype(np.int64), g64, 1)
        far = np.abs(g - g64[:, :1])  # gains as they differ from the confident expert's
        size = 2.5 * p * (far + (p * far).sum(1, keepdims=True))
        units = 3 * (4 + 1.3 * 25) + E / 8 + 26
        bound = size * units * U + F32_TINY
        if dtype is torch.bfloat16:
            bound = bound + np.abs(ref) * B
        _near(dx.cpu().double().numpy(), ref, bound, "dlogits")


def test_gate_gradient_of_infinite_and_missing_gains():
    """An infinite gain of the best expert takes every other gradient to minus infinity, as the
    formula has it; a token without ids has zeros whatever its gains are."""
    x = torch.randn(3, 64, generator=torch.Generator().manual_seed(3)).cuda()
    ids, w = gg.gate_topk(x, 4, renorm=False)
    ids[1] = -1
    dw = torch.ones_like(w)
    dw[0, 0], dw[1] = float("inf"), float("nan")
    dx = gg.gate_topk_backward(x, ids, dw, renorm=False)
    others = torch.arange(64, device="cuda") != ids[0, 0]
    assert bool((dx[0][others] == -float("inf")).all()) and bool(dx[0][~others].isnan())
    assert bool((dx[1] == 0).all()) and bool(torch.isfinite(dx[2]).all())


# ------------------------------------------------------------------------------- autograd

@pytest.mark.parametrize("ckpt8", [False, True])
def test_grouped_mm_refuses_a_second_derivative(ckpt8):
    """The gradients are not functions that can be differentiated again: asking for it is an
    error, not a gradient without those terms."""
    A = torch.randn(32, 64, device="cuda").to(torch.bfloat16).requires_grad_(True)
    W = torch.randn(2, 64, 64, device="cuda").to(torch.bfloat16).requires_grad_(True)
    offs = torch.tensor([16, 32], dtype=torch.int32, device="cuda")
    out = gg.grouped_mm(A, W, offs, ckpt8=ckpt8)
    dA, dW = torch.autograd.grad(out.float().pow(2).sum(), (A, W), create_graph=True)
    with pytest.raises(RuntimeError, match="once_differentiable"):
        (dA.float().sum() + dW.float().sum() + A.float().sum()).backward()
