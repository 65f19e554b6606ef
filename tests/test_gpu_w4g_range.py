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


def defined(x, w):
    """x W^T term by term in float64: an infinity times 0 is a NaN, as are two of either sign."""
    W, _ = R.dequantise(*w)
    xd = x.double().numpy()
    with np.errstate(invalid="ignore", over="ignore"):
        return np.stack([(xd[m][None, :] * W).sum(-1) for m in range(len(xd))])


@pytest.mark.parametrize("dtype", [BF16, torch.float16])
@pytest.mark.parametrize("group,K", [(32, 96), (32, 416), (64, 320), (128, 384)])
@pytest.mark.parametrize("zeros", [False, True])
@pytest.mark.parametrize("M,N", [(1, 40), (13, 40), (30, 4100), (76, 100), (300, 1003)])
def test_linear_infinities_and_nan_are_the_definition_s(dtype, group, K, zeros, M, N):
    """An infinity gives infinities of the definition's signs, wherever in the row it stands (in the last 8
    values of a K that is no multiple of 128, too), two of either sign and a NaN give NaN."""
    w = R.stored((N,), K, group, dtype, zeros, M)
    x = activations(M, K, dtype, 1)
    rows = [m % M for m in range(0, 9 * 7, 7)][:min(9, M)]
    for i, m in enumerate(rows):
        at = [K - 1, 0, K - 8, K // 2, 31, K - 3, 7, K - 40, 64][i]
        x[m, at] = float("-inf") if i % 3 == 1 else float("inf")
        if i == 5:
            x[m, 0] = float("-inf")
        if i == 6:
            x[m, K - 2] = float("nan")
    y = crp.linear_w4g(x.cuda(), crp.pack_weight_w4g(*map(dev, w)), N, group, zeros=zeros).cpu().double().numpy()
    want = defined(x[rows], w)
    assert np.array_equal(y[rows], want, equal_nan=True)
    assert np.isinf(want[0]).any()
    keep = [m for m in range(M) if m not in rows]
    if keep:
        ref, tol = R.linear(x[keep], w)
        assert (np.abs(y[keep] - ref) <= tol).all()


@pytest.mark.parametrize("group,K", [(32, 416), (64, 320), (128, 384)])
@pytest.mark.parametrize("zeros", [False, True])
@pytest.mark.parametrize("M,N", [(1, 40), (13, 40), (40, 8200), (76, 100), (300, 1003)])
def test_linear_of_the_largest_activations(group, K, zeros, M, N):
    """Sums of a group that pass float32's range where their product with the scale does not."""
    c, s, z = R.stored((N,), K, group, BF16, zeros, M)
    s = torch.full_like(s, 2.0 ** -40)
    x = torch.full((M, K), 2.0 ** 127, dtype=BF16)
    x[:, 1::3] = torch.finfo(BF16).max
    ref, tol = R.linear(x, (c, s, z))
    y = crp.linear_w4g(x.cuda(), crp.pack_weight_w4g(*map(dev, (c, s, z))), N, group, zeros=zeros)
    assert (np.abs(y.cpu().double().numpy() - ref) <= tol).all()


@pytest.mark.parametrize("zeros", [False, True])
@pytest.mark.parametrize("M,K,F,E,topk", [(1, 128, 96, 4, 2), (9, 128, 256, 16, 4), (40, 256, 2176, 4, 2),
                                          (64, 4224, 128, 2, 1), (70, 160, 96, 5, 2), (9, 128, 2176, 8, 8),
                                          (40, 256, 2176, 8, 2), (20, 160, 1088, 8, 3)])
@pytest.mark.parametrize("which", ["x", "h"])
def test_moe_of_the_largest_values(zeros, M, K, F, E, topk, which):
    """The same for the experts' x and h: sums beyond float32, results within it."""
    rng = np.random.default_rng(M)
    big = 2.0 ** 124 if which == "x" else 1.0
    x = torch.from_numpy(np.abs(rng.normal(size=(M, K))) * big).to(BF16).clamp(max=2.0 ** 127)
    r = torch.from_numpy(rng.normal(size=(E, K)) * 1.5 / np.sqrt(K) / big).to(BF16)
    gate, up, down = (R.stored(shape, k, 32, BF16, zeros, i) for i, (shape, k) in
                      enumerate((((E, F), K), ((E, F), K), ((E, K), F))))
    if which == "x":
        gate[1].fill_(2.0 ** -122)
        up[1].fill_(2.0 ** -122)
    else:   # g up to 2^67, u up to 2^59 in either sign, h under 2^126
        gate[1].fill_(2.0 ** 64 / K)
        up[1].fill_(2.0 ** 57 / K)
        down[1].fill_(2.0 ** -90)
    y, ids, _ = run_moe(x, r, gate, up, down, topk, True, routing=True)
    with np.errstate(over="ignore"):
        ref, rids, _, _, tol = R.moe(x, r, gate, up, down, topk, True)
    assert np.array_equal(ids.cpu().numpy(), rids) and np.isfinite(ref).all()
    assert (np.abs(y.cpu().double().numpy() - ref) <= tol).all()


@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("zeros", [False, True])
def test_encode_the_largest_weights(group, zeros):
    """Weights up to bf16's largest number in either sign: the codes of the same weights 2^-10 times as large,
    scales 2^10 times theirs; and the linear on them."""
    rng = np.random.default_rng(group)
    w = torch.from_numpy(rng.uniform(-1, 1, size=(33, 256)) * 2.0 ** 127).to(BF16)
    w[:, ::group] = torch.finfo(BF16).max
    w[1:, 5::group] = torch.finfo(BF16).min
    c, s, z = crp.encode_w4g(w.cuda(), group, zeros)
    c1, s1, z1 = crp.encode_w4g((w.float() * 2.0 ** -10).to(BF16).cuda(), group, zeros)
    for a, b in zip((c1, s1, z1), R.encode((w.float() * 2.0 ** -10).to(BF16), group, zeros)):
        assert (a is None) == (b is None) and (a is None or torch.equal(a.cpu(), b))
    assert torch.isfinite(s.float()).all()
    assert torch.equal(c, c1) and torch.equal(s.float(), s1.float() * 2.0 ** 10)
    assert z is None or torch.equal(z, z1)
    x = (activations(3, 256, BF16, 1).float() * 2.0 ** -20).to(BF16)
    ref, tol = R.linear(x, tuple(None if t is None else t.cpu() for t in (c, s, z)))
    y = crp.linear_w4g(x.cuda(), crp.pack_weight_w4g(c, s, z), 33, group, zeros=zeros)
    assert (np.abs(y.cpu().double().numpy() - ref) <= tol).all()
