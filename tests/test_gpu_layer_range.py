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


@pytest.mark.parametrize("rows,N,concat", [(33, 256, False), (33, 80, True), (1300, 1040, True)])
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
