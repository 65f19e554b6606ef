"""GPU: every tile of the group-scaled linear and every form of the mixture of
experts over several turns of its loops, in all types, against 64-bit results
(_w4g_tiled.py).  Each case first works out, as the library does, that the
form it is meant for is the one that runs."""
import numpy as np
import pytest
import torch

from . import _moe_h_ref as H
from . import _w4g_tiled as T
from .test_gpu_w4g import activations

pytestmark = pytest.mark.gpu
DT = {"bf16": torch.bfloat16, "fp16": torch.float16}


def up(a, b):
    return -(-a // b)


# --------------------------------------------------------------------- linear

def tile(M, N, units):
    """(MT, NT, WM, WN, KG) of the linear's tile."""
    tiles = up(N, 16)
    if M <= 16:
        return (1, 1, 1, 1, 4 if tiles > 512 else 16 if units > 40 else 10)
    if M <= 32:
        return (2, 1, 1, 2, 4) if (tiles + 1) // 2 >= 128 else (2, 1, 1, 1, 8)
    if M <= 48:
        return (3, 1, 1, 4, 4) if (tiles + 3) // 4 >= 128 else (3, 1, 1, 1, 6)
    shapes = {(5, 1, 1, 1, 4): (80, 16, 2), (5, 1, 1, 4, 4): (80, 64, 3), (7, 2, 1, 4, 2): (112, 128, 7),
              (8, 2, 1, 4, 2): (128, 128, 8)}
    return min(shapes, key=lambda t: shapes[t][2] * up(up(M, shapes[t][0]) * up(N, shapes[t][1]), 256))


CASES = [((1, 1, 1, 1, 4), (1, 5, 16), 8200), ((1, 1, 1, 1, 10), (1, 5, 16), 1003), ((1, 1, 1, 1, 16), (1, 5, 16), 1003),
         ((2, 1, 1, 2, 4), (17, 32), 4105), ((2, 1, 1, 1, 8), (17, 32), 1003), ((3, 1, 1, 4, 4), (33, 48), 8200),
         ((3, 1, 1, 1, 6), (33, 48), 1003), ((5, 1, 1, 1, 4), (49, 80), 1003), ((5, 1, 1, 4, 4), (100, 150), 9731),
         ((7, 2, 1, 4, 2), (300, 331), 9731), ((8, 2, 1, 4, 2), (1000,), 4090)]


@pytest.mark.parametrize("dtype", DT)
@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("zeros", [False, True])
@pytest.mark.parametrize("want,rows,N", CASES)
def test_linear_turns(dtype, group, zeros, want, rows, N):
    """Four or five turns of K for each group of waves, the last for some of them only, the last unit not full
    (groups of 128: a whole one)."""
    turns = 3 if want[4] == 10 else 4        # ten groups of waves take no more than 40 units
    K = (turns * want[4] + (0 if want[4] != 10 else 8)) * 128 + group
    units = up(K, 128)
    assert up(units, want[4]) == turns + 1 and units % want[4]
    w = T.Linear(N, K, group, DT[dtype], zeros, seed=K)
    for M in rows:
        assert tile(M, N, units) == want
        x = activations(M, K, DT[dtype], M)
        assert torch.equal(w.check(x), w.check(x))


# ----------------------------------------------------------------- experts

def share(M, E, topk):
    return M > 16 and M * topk >= 5 * E


def gate_up(M, K, F, E, topk):
    """"many" or the number of waves that share a tile's K."""
    pairs, tiles, units = M * topk, F // 16, up(K, 128)
    rows = pairs if pairs < E else E
    if share(M, E, topk) and rows * up(tiles, 4) >= 256:
        return "many"
    ks = 1
    while ks < 8 and not (rows * tiles * ks >= 1024 and (rows * tiles * ks >= 4096 or units // (2 * ks) < 8)):
        ks *= 2
    return ks


def wide(M, K, E, topk):
    pairs, blocks = M * topk, up(K // 16, 4) * 8
    return blocks >= 256 if pairs >= 12 * E else pairs >= 5 * E and blocks >= 352


def inputs(M, K, E, dtype, seed, favourite=None):
    rng = np.random.default_rng(seed)
    x = torch.from_numpy(rng.normal(size=(M, K))).to(dtype)
    r = torch.from_numpy(rng.normal(size=(E, K)) * 1.5 / np.sqrt(K)).to(dtype)
    if favourite is not None:   # every token's first choice
        r[favourite] = torch.sign(x.float().mean(0) + 1e-3).to(dtype)
        x = (x.float().abs() * torch.sign(r[favourite].float())).to(dtype)
    return x, r


UP = [(1, 12, 416, 1056, 16, 8, None), (1, 8, 416, 272, 128, 8, None), (1, 40, 416, 272, 64, 2, 61),
      (1, 16, 2080, 1040, 64, 8, None), (2, 12, 1056, 560, 16, 8, None), (2, 24, 672, 560, 20, 2, 3),
      (4, 3, 2080, 464, 64, 4, None), (4, 20, 1312, 336, 16, 3, None), (8, 1, 4128, 272, 8, 2, None),
      (8, 18, 4128, 48, 24, 2, 5), ("many", 17, 672, 2080, 8, 3, None), ("many", 33, 800, 2080, 8, 2, 6),
      ("many", 64, 1312, 1056, 16, 6, None), ("many", 70, 672, 2192, 8, 2, None)]


@pytest.mark.parametrize("dtype", DT)
@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("zeros", [False, True])
@pytest.mark.parametrize("want,M,K,F,E,topk,favourite", UP)
def test_gate_up_turns(dtype, group, zeros, want, M, K, F, E, topk, favourite):
    """Every number of waves on a tile's K, and rows shared, over several units, the last one not full; blocks
    whose last tiles do not exist; experts of more tokens than one operand takes."""
    K, F = up(K, group) * group, up(F, group) * group
    assert gate_up(min(M, 64), K, F, E, topk) == want
    x, r = inputs(M, K, E, DT[dtype], M + K, favourite)
    experts = T.Experts(K, F, E, group, DT[dtype], zeros, seed=K)
    got = experts.check(x, r, topk, zeros)
    if favourite is not None:
        assert (got[1][:, 0] == favourite).all()
    assert np.linalg.norm(got[0].cpu().double().numpy() - experts.exact) <= H.norm_limit(experts.exact, DT[dtype])


DOWN = [(False, 1, 416, 2080, 8, 2, None), (False, 3, 4128, 800, 60, 4, None), (False, 16, 2080, 800, 128, 8, None),
        (False, 40, 416, 1312, 64, 2, 61), (False, 64, 1056, 2080, 8, 4, None), (False, 64, 2080, 416, 60, 8, None),
        (True, 5, 4128, 1312, 2, 2, None), (True, 16, 2080, 1312, 8, 8, None), (True, 20, 4128, 1312, 8, 3, None),
        (True, 40, 2848, 1312, 8, 2, 6), (True, 64, 2080, 2080, 8, 2, None), (True, 64, 4096, 800, 60, 8, 3),
        (True, 131, 4128, 672, 5, 2, None)]


@pytest.mark.parametrize("dtype", DT)
@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("zeros", [False, True])
@pytest.mark.parametrize("want,M,K,F,E,topk,favourite", DOWN)
def test_down_turns(dtype, group, zeros, want, M, K, F, E, topk, favourite):
    """Blocks of columns apart and wide, over several units and passes, passes cut between blocks, sums joined
    by the last block; the same call gives the same bits."""
    K, F = up(K, group) * group, up(F, group) * group
    assert wide(min(M, 64), K, E, topk) == want
    x, r = inputs(M, K, E, DT[dtype], M + F, favourite)
    experts = T.Experts(K, F, E, group, DT[dtype], zeros, seed=F)
    got = experts.check(x, r, topk, not zeros)
    assert np.linalg.norm(got[0].cpu().double().numpy() - experts.exact) <= H.norm_limit(experts.exact, DT[dtype])
    for _ in range(3):
        assert all(torch.equal(a, b) for a, b in zip(got, experts.run(x, r, topk, not zeros)))


def test_rows_of_a_batch_that_goes_in_passes():
    """The same 40 tokens four times in a row, over passes of 64, 64 and 32: every copy within the bound, one
    choice; the first pass's the same bits whatever rows the later ones hold."""
    x, r = inputs(40, 544, 24, torch.bfloat16, 1)
    experts = T.Experts(544, 416, 24, 32, torch.bfloat16, True, seed=2)
    y, ids, c = experts.check(x.repeat(4, 1), r, 4, True)
    assert torch.equal(ids.view(4, 40, 4)[1:], ids.view(4, 40, 4)[:3]) and torch.equal(c[:40], c[120:])
    other = torch.cat((x, x[:24], x.flip(0), x.flip(0)[:56]))
    y2, *_ = experts.check(other, r, 4, True)
    assert torch.equal(y[:64], y2[:64])
