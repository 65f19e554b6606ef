"""GPU: attention over prompts at the ends of the types' ranges: keys that
score minus infinity, a scale of 0, scores and values as large as the types
hold, against the definition in 64 bits."""
import numpy as np
import pytest
import torch

import rotated_bit_quantized_convrot_amd as crp

from . import _attn_ref as R

pytestmark = pytest.mark.gpu
DT = {"bf16": torch.bfloat16, "fp16": torch.float16}
# (lengths, query heads): every way of splitting rows and keys over blocks and waves, for heads of 64, 128 and 256
WAYS = [([300], 4), ([300], 128), ([300], 240), ([600], 100), ([100] * 12, 128)]


def make(lens, D, dtype=torch.bfloat16, seed=0):
    """q [T, 4, D], k and v [T, 2, D]."""
    gen = torch.Generator().manual_seed(seed)
    return (torch.randn((sum(lens), h, D), generator=gen).to(dtype).cuda() for h in (4, 2, 2))


def attend(q, k, v, lens, heads, causal, scale=None):
    """The call with every query head `heads` / 4 times, which all give the
    same: y [T, 4, D]."""
    cu = torch.tensor([0] + list(np.cumsum(lens)), dtype=torch.int32).cuda()
    y = crp.attn_prompt(q.repeat_interleave(heads // 4, 1), k, v, cu, causal=causal, scale=scale)
    y = y.view(q.shape[0], 4, heads // 4, -1)
    assert torch.equal(y.view(torch.int16), y[:, :, :1].expand_as(y).contiguous().view(torch.int16))
    return y[:, :, 0].double().cpu().numpy()


def reference(q, k, v, seen, scale, dtype, score_error=None):
    """One sequence whose row r sees the first seen[r] of the keys: y and the
    tolerance, which _attn_ref.prompt derives, with its error of the scores or
    this one."""
    q, k, v = (t.double().cpu().numpy() for t in (q, k, v))
    y, tol = np.zeros(q.shape), np.zeros(q.shape)
    half = torch.finfo(dtype).eps / 2
    for h in range(q.shape[1]):
        y[:, h], (A, ds, span, n, total) = R.attend(q[:, h], k[:, h // 2], v[:, h // 2], seen, scale)
        e = 2 * ((ds if score_error is None else score_error) + 4 * R.U * (span + 1) + 2 * n * R.U)
        tol[:, h] = (half + e)[:, None] * A + half * np.abs(y[:, h]) * (1 + 1e-3) + 2.0 ** -126
        if dtype == torch.float16:
            tol[:, h] += (n * 2.0 ** -25 / total)[:, None] * np.abs(v).max() + 2.0 ** -25
    return y, tol


def pieces(lens):
    at = 0
    for n in lens:
        yield slice(at, at + n), n
        at += n


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("lens,heads", WAYS)
@pytest.mark.parametrize("at,bad", [(0, 64), (0, 65), (0, 128), (64, 64)])
def test_keys_that_score_minus_infinity(D, causal, lens, heads, at, bad):
    """An infinite channel of some keys next to each other, against the sign of
    q: weights of 0, a softmax over the others, NaN where there is no other."""
    if at + bad >= lens[0]:
        at, bad = 0, lens[0] - 2
    q, k, v = make(lens, D, seed=D + bad)
    q[..., 5] = -q[..., 5].abs().clamp(min=0.25)
    for one, n in pieces(lens):
        k[one][at:at + bad, :, 5] = float("inf")
    got = attend(q, k, v, lens, heads, causal)
    for one, n in pieces(lens):
        i = np.arange(n) if causal else np.full(n, n - 1)
        seen = np.minimum(i + 1, at) + np.maximum(i + 1 - at - bad, 0)
        rest = torch.cat((k[one][:at], k[one][at + bad:])), torch.cat((v[one][:at], v[one][at + bad:]))
        want, tol = reference(q[one], *rest, seen, D ** -0.5, torch.bfloat16)
        assert np.isnan(got[one][seen == 0]).all()
        assert (np.abs(got[one] - want) <= tol)[seen > 0].all()


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("lens,heads", WAYS)
@pytest.mark.parametrize("size", [1e15, 2.0 ** 63])
def test_a_scale_of_0(D, causal, lens, heads, size):
    """The mean of the values, however large q and k are (at 2^63 their
    products pass float32); a row of q with an infinity gives NaN."""
    q, k, v = make(lens, D, seed=D)
    q, k = ((x.float() * size).to(torch.bfloat16) for x in (q, k))
    q[7, 1, 3], q[9, 2, 4] = float("inf"), float("nan")
    got = attend(q, k, v, lens, heads, causal, scale=0.0)
    assert np.isnan(got[7, 1]).all() and np.isnan(got[9, 2]).all()
    got[7, 1] = got[9, 2] = 0
    q, k = q.nan_to_num(0, 0, 0), k
    for one, n in pieces(lens):
        seen = np.arange(1, n + 1) if causal else np.full(n, n)
        want, tol = reference(q[one], k[one], v[one], seen, 0.0, torch.bfloat16)
        off = np.abs(got[one] - want) <= tol
        if one.start == 0:
            off[7, 1] = off[9, 2] = True
        assert off.all()


@pytest.mark.parametrize("dtype,D", [("fp16", 64), ("bf16", 128), ("fp16", 128), ("bf16", 256)])
@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("lens,heads", WAYS)
@pytest.mark.parametrize("size", [2.0 ** 11, 2.0 ** 24, 2.0 ** 32, 1e30])
def test_scores_as_large_as_float32_holds(dtype, D, causal, lens, heads, size):
    """Rows whose weight goes to one key, or to some with the same score: q and
    k along one direction, where float32 has the scores exactly."""
    dt = DT[dtype]
    q, k, v = make(lens, D, dt, seed=D)
    gen = torch.Generator().manual_seed(D)
    u = torch.randint(0, 2, (D,), generator=gen).mul(2).sub(1).float().cuda()
    sign = torch.randint(0, 2, q.shape[:2], generator=gen).mul(2).sub(1).float()
    q = ((1 + torch.rand(q.shape[:2], generator=gen)) * sign).cuda()[..., None].mul(u).to(dt)
    r = (2 * torch.rand(k.shape[:2], generator=gen) - 1).cuda()
    k = r[..., None].mul(u).to(dt)
    scale = size / D
    got = attend(q, k, v, lens, heads, causal, scale=scale)
    for one, n in pieces(lens):
        seen = np.arange(1, n + 1) if causal else np.full(n, n)
        # scale and log2 e are rounded once more each, and their product with a score of up to twice `size`; from 2^20
        # on keys of other scores have no weight, and equal ones the same error
        ds = 6 * R.U * size if size < 2.0 ** 20 else 0.0
        want, tol = reference(q[one], k[one], v[one], seen, float(np.float32(scale)), dt, ds)
        assert (np.abs(got[one] - want) <= tol).all()


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("lens,heads", WAYS)
@pytest.mark.parametrize("sign", [False, True])
def test_values_as_large_as_the_type_holds(D, causal, lens, heads, sign):
    """Averages of v close to bf16's largest number, of one sign or of both, next
    to channels of ordinary size."""
    q, k, v = make(lens, D, seed=D)
    v[..., ::2] = (v[..., ::2].float().abs().clamp(0, 1).mul(0.25).add(0.75) * torch.finfo(torch.bfloat16).max *
                   (v[..., ::2].float().sign() if sign else 1)).to(torch.bfloat16)
    v[1, 0, 0] = v[0, 0, 0] = 2e38
    assert v.isfinite().all()
    got = attend(q, k, v, lens, heads, causal)
    for one, n in pieces(lens):
        seen = np.arange(1, n + 1) if causal else np.full(n, n)
        want, tol = reference(q[one], k[one], v[one], seen, D ** -0.5, torch.bfloat16)
        assert (np.abs(got[one] - want) <= tol).all()


@pytest.mark.parametrize("D", [64, 128, 256])
def test_infinite_values_of_keys_of_little_weight(D):
    """exp underflows in float32, not in the definition: a weight that is not 0
    times infinity is infinity; with a score of -infinity it is 0, and NaN."""
    q, k, v = make([200], D, seed=1)
    q[..., 5], k[..., 5] = 1.0, 0.0
    k[60, 0, 5] = -200 * D ** 0.5
    k[70, 1, 5] = float("-inf")
    v[60, 0, 9] = v[70, 1, 9] = float("inf")
    got = attend(q, k, v, [200], 4, True)
    assert np.isposinf(got[60:, :2, 9]).all() and np.isnan(got[70:, 2:, 9]).all()
    v[60, 0, 9] = v[70, 1, 9] = 0
    want, tol = reference(q, k.nan_to_num(0, 0, -200 * D ** 0.5), v, np.arange(1, 201), D ** -0.5, torch.bfloat16)
    clean = np.ones(got.shape, bool)
    clean[60:, :2, 9] = clean[70:, 2:, 9] = False
    assert (np.abs(got - want) <= tol)[clean].all()
