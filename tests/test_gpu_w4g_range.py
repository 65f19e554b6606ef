"""GPU: the operators on 4-bit weights with group scales at the ends of the
types' ranges, against their 64-bit definitions (_w4g_ref.py)."""
import numpy as np
import pytest
import torch

import rotated_bit_quantized_convrot_amd as crp

from . import _w4g_ref as R
from .test_gpu_moe import run as run_moe
from .test_gpu_w4g import activations, dev

pytestmark = pytest.mark.gpu
BF16 = torch.bfloat16
# rows of x that reach every height of the linear's tiles, with columns that are few and many
TILES = [(1, 40), (5, 8200), (20, 100), (20, 4100), (40, 100), (40, 8200), (76, 100), (100, 9731), (300, 9731),
         (1000, 4090)]


@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("zeros", [False, True])
@pytest.mark.parametrize("M,N", TILES)
def test_linear_with_the_largest_scales(group, zeros, M, N):
    """From 2^124 to bf16's largest number, over activations so small that nothing overflows."""
    c, s, z = R.stored((N,), 256, group, BF16, zeros, M)
    s = torch.full_like(s, 2.0 ** 124)
    s[1::2] = torch.finfo(BF16).max
    x = (activations(M, 256, BF16, 1).float() * 2.0 ** -115).to(BF16)
    ref, tol = R.linear(x, (c, s, z))
    y = crp.linear_w4g(x.cuda(), crp.pack_weight_w4g(*map(dev, (c, s, z))), N, group, zeros=zeros)
    assert (np.abs(y.cpu().double().numpy() - ref) <= tol).all()


@pytest.mark.parametrize("zeros", [False, True])
@pytest.mark.parametrize("M,K,F,E,topk", [(1, 128, 64, 4, 2), (9, 128, 256, 16, 4), (40, 256, 2176, 4, 2),
                                          (64, 4224, 128, 2, 1)])
@pytest.mark.parametrize("which", ["gate_up", "down"])
def test_moe_with_the_largest_scales(zeros, M, K, F, E, topk, which):
    rng = np.random.default_rng(M)
    small = 2.0 ** -124 if which == "gate_up" else 1.0
    x = torch.from_numpy(rng.normal(size=(M, K)) * small).to(BF16)
    r = torch.from_numpy(rng.normal(size=(E, K)) * 1.5 / np.sqrt(K) / small).to(BF16)
    gate, up, down = (R.stored(shape, k, 64, BF16, zeros, i) for i, (shape, k) in
                      enumerate((((E, F), K), ((E, F), K), ((E, K), F))))
    if which == "gate_up":
        gate[1].fill_(2.0 ** 124)
        up[1].fill_(2.0 ** 124)
    else:
        gate[1].fill_(2.0 ** -60)
        up[1].fill_(2.0 ** -60)
        down[1].fill_(2.0 ** 125)
    y, ids, _ = run_moe(x, r, gate, up, down, topk, True, routing=True)
    ref, rids, _, _, tol = R.moe(x, r, gate, up, down, topk, True)
    assert np.array_equal(ids.cpu().numpy(), rids) and np.isfinite(ref).all()
    assert (np.abs(y.cpu().double().numpy() - ref) <= tol).all()
