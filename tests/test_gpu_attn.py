"""GPU: attention over whole prompts against its 64-bit definition
(_attn_ref.py states the bounds)."""
import numpy as np
import pytest
import torch

import rotated_bit_quantized_convrot_amd as crp

from . import _attn_ref as R

pytestmark = pytest.mark.gpu
DT = {"bf16": torch.bfloat16, "fp16": torch.float16}


def starts(lens):
    return [0] + list(np.cumsum(lens))


def make(lens, Hq, Hkv, D, dtype, seed=0, gain=1.5, extra=0):
    """q, k, v as the parts of one projection's output."""
    gen = torch.Generator().manual_seed(seed)
    x = torch.randn((sum(lens) + extra, Hq + 2 * Hkv, D), generator=gen)
    x[:, :Hq] *= gain
    return x.to(dtype).cuda().split((Hq, Hkv, Hkv), 1)


def check(q, k, v, lens, causal, dtype, scale=None, first=0):
    cu = [first + c for c in starts(lens)]
    y = crp.attn_prompt(q, k, v, torch.tensor(cu, dtype=torch.int32).cuda(), causal=causal, scale=scale)
    want, tol = R.prompt(q, k, v, cu, causal, q.shape[-1] ** -0.5 if scale is None else scale, dtype)
    got = y.double().cpu().numpy()[cu[0]:cu[-1]]
    want, tol = want[cu[0]:cu[-1]], tol[cu[0]:cu[-1]]
    assert np.isfinite(got).all()
    assert (np.abs(got - want) / tol).max(initial=0) <= 1
    return y


@pytest.mark.parametrize("dtype", DT)
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("Hq,Hkv", [(1, 1), (6, 2), (7, 7), (16, 1)])
def test_heads_and_types(dtype, D, causal, Hq, Hkv):
    lens = [37, 0, 1, 130, 64]
    check(*make(lens, Hq, Hkv, D, DT[dtype], seed=Hq + D), lens, causal, DT[dtype])


@pytest.mark.parametrize("n", [1, 2, 15, 16, 17, 31, 32, 33, 63, 64, 65, 95, 127, 128, 129, 191, 192, 193, 255, 256,
                               257, 300, 511, 513])
@pytest.mark.parametrize("causal", [True, False])
def test_lengths(n, causal):
    check(*make([n], 2, 1, 128, torch.bfloat16, seed=n), [n], causal, torch.bfloat16)


@pytest.mark.parametrize("dtype", DT)
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("lens,Hq,Hkv", [([700], 40, 5), ([130, 700, 1, 257, 64], 48, 4), ([500, 333, 129], 16, 16),
                                         ([65], 300, 100), ([60] * 20, 64, 8), ([1500], 48, 2), ([700, 600], 80, 8)])
def test_many_blocks(dtype, D, causal, lens, Hq, Hkv):
    """Enough rows and heads for every way that the rows and keys are split
    over blocks and waves."""
    check(*make(lens, Hq, Hkv, D, DT[dtype], seed=Hq), lens, causal, DT[dtype])


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("causal", [True, False])
def test_many_short_sequences(D, causal):
    rng = np.random.default_rng(3)
    lens = list(rng.integers(0, 9, size=150)) + [0, 0] + list(rng.integers(1, 140, size=9))
    check(*make(lens, 2, 2, D, torch.float16, seed=D), lens, causal, torch.float16)


@pytest.mark.parametrize("dtype", DT)
@pytest.mark.parametrize("gain", [0.0, 6.0, 40.0])
@pytest.mark.parametrize("D", [64, 128, 256])
def test_flat_and_peaked_weights(dtype, gain, D):
    """Equal weights, and weights that one key holds almost alone: the running
    maximum moves often."""
    lens = [333, 70]
    q, k, v = make(lens, 4, 2, D, DT[dtype], seed=5, gain=gain)
    # later keys larger: every tile raises the maximum
    k = (k.float() * torch.linspace(0.1, 2.0, sum(lens), device="cuda")[:, None, None]).to(DT[dtype])
    check(q, k, v, lens, True, DT[dtype])


def test_scores_far_from_zero():
    """All scores of a row large and of one sign."""
    lens = [200]
    q, k, v = make(lens, 2, 1, 128, torch.bfloat16, seed=8)
    k = (k.float() * 0.05 + 1.0).to(torch.bfloat16)
    for sign in (2.0, -2.0):
        check((q.float() * 0.05 + sign).to(torch.bfloat16), k, v, lens, True, torch.bfloat16)


@pytest.mark.parametrize("scale", [1.0, 0.01, -0.1, 0.0])
def test_scale(scale):
    lens = [100, 29]
    check(*make(lens, 2, 1, 64, torch.bfloat16, seed=1, gain=0.3), lens, True, torch.bfloat16, scale=scale)


def test_layouts():
    """[heads, T, D] in memory, broadcast keys, a stride that is no power of two."""
    lens, dtype = [90, 41], torch.bfloat16
    q, k, v = make(lens, 4, 2, 128, dtype, seed=2)
    want = check(q, k, v, lens, True, dtype)
    turned = [t.transpose(0, 1).contiguous().transpose(0, 1) for t in (q, k, v)]
    assert torch.equal(check(*turned, lens, True, dtype), want)
    wide = torch.empty((131, 4, 128 + 24), dtype=dtype, device="cuda")
    wide[..., :128] = q
    assert torch.equal(check(wide[..., :128], turned[1], v, lens, True, dtype), want)
    one = k[:, :1].expand(-1, 2, -1)
    check(q, one, v, lens, True, dtype)
    same = k[:1].expand(131, -1, -1)
    check(q, same, v, lens, True, dtype)


def test_rows_outside_the_sequences():
    """Rows before the first and behind the last sequence: not read (NaN
    there), not written."""
    lens, dtype = [50, 33], torch.bfloat16
    q, k, v = make(lens, 4, 2, 128, dtype, seed=3, extra=40)
    for t in (q, k, v):
        t[:10] = float("nan")
        t[93:] = float("nan")
    cu = torch.tensor([10, 60, 93], dtype=torch.int32).cuda()
    out = torch.full((123, 4, 128), 7.0, dtype=dtype, device="cuda")
    y = crp.attn_prompt(q, k, v, cu, out=out)
    assert y is out
    assert (out[:10] == 7).all() and (out[93:] == 7).all()
    want, tol = R.prompt(q, k, v, [10, 60, 93], True, 128 ** -0.5, dtype)
    assert (np.abs(out[10:93].double().cpu().numpy() - want[10:93]) <= tol[10:93]).all()


def special(D, Hq=4, Hkv=2, n=300, dtype=torch.bfloat16):
    return make([n], Hq, Hkv, D, dtype, seed=D)


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("bad", [float("nan"), float("inf"), float("-inf")])
@pytest.mark.parametrize("where", ["k", "v"])
@pytest.mark.parametrize("heads", [2, 60, 110, 200])   # of each half: ways of test_many_blocks
def test_a_bad_token_reaches_only_rows_that_see_it(D, bad, where, heads):
    q, k, v = special(D)
    q = q.repeat_interleave(heads // 2, 1)
    clean = crp.attn_prompt(q, k, v, torch.tensor([0, 150, 300], dtype=torch.int32).cuda())
    (k if where == "k" else v)[77, 1, 5] = bad
    y = crp.attn_prompt(q, k, v, torch.tensor([0, 150, 300], dtype=torch.int32).cuda())
    # heads 0, 1 and rows before it, and the other sequence, as they were (to the weights' rounding)
    near = lambda a, b: (a.float() - b.float()).abs().max() <= 4 * torch.finfo(torch.bfloat16).eps
    H = heads
    assert near(y[:, :H], clean[:, :H]) and near(y[:77], clean[:77]) and near(y[150:], clean[150:])
    seen = y[77:150, H:].float()
    if where == "v":
        others = [d for d in range(D) if d != 5]
        assert near(y[77:150, H:][..., others], clean[77:150, H:][..., others])
        assert (seen[..., 5] == bad).all() if bad == bad else seen[..., 5].isnan().all()
    elif bad != bad:
        assert seen.isnan().all()
    else:
        # a score of +-infinity: NaN, or a key with no weight
        up = (q[77:150, H:, 5].float() * bad) > 0
        assert seen[up].isnan().all() and seen[~up].isfinite().all()


def test_bad_rows_of_q():
    q, k, v = special(128)
    q[40, 1, 3] = float("nan")
    q[200, 2, 3] = float("inf")
    y = crp.attn_prompt(q, k, v, torch.tensor([0, 300], dtype=torch.int32).cuda())
    bad = y.isnan().any(-1).nonzero().tolist()
    assert bad == [[40, 1], [200, 2]]


def test_in_a_larger_memory():
    """A token stride that takes offsets past 32 bits."""
    T, D = 300, 128
    big = torch.empty((T, 8_000_000), dtype=torch.bfloat16, device="cuda")   # 4.8 GB
    q, k, v = make([T], 1, 1, D, torch.bfloat16, seed=4)
    big[:, :D], big[:, 4_000_000:4_000_000 + D], big[:, -D:] = q[:, 0], k[:, 0], v[:, 0]
    parts = [big[:, None, :D], big[:, None, 4_000_000:4_000_000 + D], big[:, None, -D:]]
    check(*parts, [T], True, torch.bfloat16)


def test_repeatable_on_other_streams_and_in_graphs():
    lens, dtype = [120, 1, 64, 333], torch.bfloat16
    q, k, v = make(lens, 8, 2, 128, dtype, seed=6)
    cu = torch.tensor(starts(lens), dtype=torch.int32).cuda()
    want = crp.attn_prompt(q, k, v, cu).clone()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        y = crp.attn_prompt(q, k, v, cu)
    side.synchronize()
    assert torch.equal(y, want)
    graph = torch.cuda.CUDAGraph()
    out = torch.empty_like(want)
    with torch.cuda.graph(graph):
        crp.attn_prompt(q, k, v, cu, out=out)
    for turn in range(3):
        out.fill_(0)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want)
        eager = crp.attn_prompt(q, k, v, cu)
        assert torch.equal(eager, want)


def test_no_rows():
    q, k, v = make([0], 2, 1, 64, torch.bfloat16)
    assert crp.attn_prompt(q, k, v, torch.zeros(3, dtype=torch.int32).cuda()).shape == (0, 2, 64)
    q, k, v = make([5], 2, 1, 64, torch.bfloat16)
    out = torch.full((5, 2, 64), 3.0, dtype=torch.bfloat16, device="cuda")
    crp.attn_prompt(q, k, v, torch.zeros(1, dtype=torch.int32).cuda(), out=out)
    crp.attn_prompt(q, k, v, torch.zeros(4, dtype=torch.int32).cuda(), out=out)
    assert (out == 3).all()
