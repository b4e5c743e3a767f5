"""Arrays of a call that share memory where they must not: refused on the host."""
import ctypes

import pytest

from conftest import cuda_ok


@pytest.fixture(scope="module")
def lib():
    from moe_grouped_gemm_ragged_b200 import _build
    _build.build()
    import moe_grouped_gemm_ragged_b200 as gg
    return gg.lib()


@pytest.mark.parametrize("f32", [False, True])
def test_gate_backward_in_place_is_refused(lib, f32):
    """4 x 8 logits: the gradient in their place, or with its first or last number among them. Apart,
    the arguments are in order, and the call gets as far as looking for a device."""
    T, E, size = 4, 8, 4 if f32 else 2
    at = 1 << 20
    for score in (0, 1):
        for flags in (0, 1):
            flags |= 2 if f32 else 0

            def call(d, n=T):
                P = ctypes.c_void_p
                return lib.gg_gate_topk_backward(P(at), n, E, 2, score, flags, 1.0, P(64), P(64),
                                                 P(at + d), None, None)

            whole = T * E * size
            for d in (0, size, -size, whole - size, size - whole):
                assert call(d) == 1, d
            if not cuda_ok():  # these are never made where they would run
                assert call(whole) not in (0, 1) and call(-whole) not in (0, 1)
                assert call(0, 0) != 1
