"""Forward-mode differentiation of the autograd forms: there is none, and a call says so instead of
returning a result without a tangent."""
import pytest
import torch
from torch.autograd import forward_ad

import moe_grouped_gemm_ragged_b200 as gg

BF16 = torch.bfloat16
I32 = torch.int32


def _calls():
    """(function, arguments, keywords) of every form, on the host: without a tangent a call gets as
    far as the check of the device."""
    x, ids = torch.zeros(4, 8, dtype=BF16), torch.zeros(4, 2, dtype=I32)
    row_of, offs, w = torch.zeros(8, dtype=I32), torch.zeros(8, dtype=I32), torch.zeros(4, 2)
    H, A = torch.zeros(8, 256, dtype=BF16), torch.zeros(8, 64, dtype=BF16)
    W1, W2 = torch.zeros(8, 64, 256, dtype=BF16), torch.zeros(8, 128, 64, dtype=BF16)
    return [
        (gg.gate, [x, 2], {}, [0]),
        (gg.dispatch, [x, ids, 8], {}, [0]),
        (gg.combine, [A, row_of, 2], dict(weights=w, residual=A[:4], offs=offs),
         [0, "weights", "residual"]),
        (gg.swiglu, [H, offs], dict(row_of=row_of, weights=w), [0, "weights"]),
        (gg.expert_mlp, [A, W1, W2, offs], dict(row_of=row_of, weights=w), [0, 1, 2, "weights"]),
        (gg.grouped_mm, [A, W1, offs], {}, [0, 1]),
    ]


@pytest.mark.parametrize("call", range(6))
@pytest.mark.parametrize("grad", [True, False])
def test_a_tangent_is_refused(call, grad):
    fn, args, kw, names = _calls()[call]
    for name in names:
        a2, k2 = list(args), dict(kw)
        with forward_ad.dual_level(), torch.set_grad_enabled(grad):
            old = args[name] if isinstance(name, int) else kw[name]
            dual = forward_ad.make_dual(old, torch.ones_like(old))
            if isinstance(name, int):
                a2[name] = dual
            else:
                k2[name] = dual
            with pytest.raises(NotImplementedError, match="forward-mode"):
                fn(*a2, **k2)
            with pytest.raises(ValueError, match="CUDA"):  # others beside it are not concerned
                fn(*args, **kw)
    with pytest.raises(ValueError, match="CUDA"):
        fn(*args, **kw)
