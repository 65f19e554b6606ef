"""The bounds that hold the hidden values of the mixture of experts to
float32 reject what holds them in fewer bits."""
import numpy as np
import pytest
import torch

from . import _moe_h_ref as H
from . import _w4g_ref as R


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
def test_cancelling_bound_sees_two_parts_of_h(dtype):
    M, K, F = 6, 128, 64
    x, r, gate, up, down, p = H.cancelling(M, K, F, 2, 32, dtype, False, [m % 2 for m in range(M)])
    y, tol = H.expected(x, K, F, p)
    # the layer is what the formula says, and float32's h is inside
    ref, ids, *_ = R.moe(x, r, gate, up, down, 1, True)
    assert np.allclose(ref, y, rtol=1e-9) and (ids[:, 0] == np.arange(M) % 2).all()
    to = lambda v: torch.from_numpy(v).to(dtype).double().numpy()
    for parts, inside in ((1, False), (2, False), (3, True)):
        got = to(H.expected(x, K, F, p, lambda h: H.bf16_parts(h, parts))[0])
        assert (np.abs(got - y) <= tol).all() == inside, parts


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
def test_norm_limit_sees_one_part_of_h(dtype):
    rng = np.random.default_rng(0)
    h = rng.normal(size=(16, 512)) * rng.normal(size=(16, 512))
    w = rng.integers(-8, 8, size=(512, 256)) * 0.01
    y = h @ w
    to = lambda v: torch.from_numpy(v).to(dtype).double().numpy()
    limit = H.norm_limit(y, dtype)
    assert np.linalg.norm(to(H.bf16_parts(h, 3) @ w) - y) <= limit
    one = torch.from_numpy(h).to(dtype).double().numpy()
    assert np.linalg.norm(to(one @ w) - y) > limit
