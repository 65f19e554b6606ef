"""GPU: attention over the 4-bit cache at the ends of the types' ranges: signs
and sizes of the scale, scores, queries and values as large as the types
hold, against the definition in 64 bits."""
import numpy as np
import pytest
import torch

import rotated_bit_quantized_convrot_amd as crp

from . import _attn_ref as R
from .test_gpu_kv4 import Setup, ints, starts

pytestmark = pytest.mark.gpu
DT = {"bf16": torch.bfloat16, "fp16": torch.float16}
# (lengths, new tokens, query heads of 2 key heads, pages of a table beyond what is needed): one span or several, tiles of
# 8 rows, of 16, and two or three of those
WAYS = [([300, 37], [1, 1], 6, 2), ([3000, 500], [1, 1], 6, 40), ([300, 90], [3, 3], 10, 2), ([2500, 90], [3, 3], 10, 40),
        ([700, 90], [7, 7], 10, 40)]


def reference(s, q, new, scale, score_error=None):
    """Setup.reference; with `score_error` in the place of the scores' error
    that it derives."""
    if score_error is None:
        # its bound is written for scales that are not negative: the sign to q
        return s.reference(-q if scale < 0 else q, new, abs(scale))
    y, tol = np.zeros(q.shape), np.zeros(q.shape)
    a, c = starts(new), starts(s.lens)
    rot = R.hadamard(s.D) if s.rotate else np.eye(s.D)
    kv = [(R.values(*w, s.group), (w[0] + 16.0) * (w[1] & np.uint32(0xFFFFFFF0)).view(np.float32).astype(float).repeat(s.group, -1))
          for w in (R.encode(s.k, s.group, s.rotate), R.encode(s.v, s.group, s.rotate))]
    (k, _), (v, v_big) = kv
    x = q.double().cpu().numpy()
    for b, n in enumerate(s.lens):
        rows, one = slice(a[b], a[b + 1]), slice(c[b], c[b + 1])
        seen = np.clip(n - new[b] + 1 + np.arange(new[b]), 0, n)
        for h in range(x.shape[1]):
            g = h // (x.shape[1] // s.H)
            o, (A, _, span, m, total) = R.attend(x[rows, h] @ rot, k[one, g], v[one, g], seen, scale)
            big = R.attend(x[rows, h] @ rot, k[one, g], v_big[one, g], seen, scale)[0]
            e = 2 * (score_error + 4 * R.U * (span + 1) + 2 * m * R.U) + 2.0 ** -17
            off = e[:, None] * A + 2 * (m + 4)[:, None] * R.U * big
            y[rows, h] = o @ rot
            tol[rows, h] = (off @ np.abs(rot) + 20 * R.U * np.abs(o) @ np.abs(rot) +
                            torch.finfo(s.dtype).eps / 2 * np.abs(y[rows, h]) * (1 + 1e-3) + 2.0 ** -25)
    return y, tol


@pytest.mark.parametrize("rotate", [True, False])
@pytest.mark.parametrize("D,group", [(64, 64), (128, 32), (256, 64)])
@pytest.mark.parametrize("lens,new,Hq,spare", WAYS)
@pytest.mark.parametrize("scale", [-0.1, 0.0])
def test_signs_of_the_scale(rotate, D, group, lens, new, Hq, spare, scale):
    s = Setup(lens, 2, D, group, 64, rotate, torch.bfloat16, seed=D, spare=spare).fill()
    q = s.queries(new, Hq)
    y, tol = reference(s, q, new, scale)
    assert (np.abs(s.attend(q, new, scale=scale).double().cpu().numpy() - y) <= tol).all()


@pytest.mark.parametrize("rotate", [True, False])
@pytest.mark.parametrize("lens,new,Hq,spare", WAYS)
@pytest.mark.parametrize("size", [1e15, 2.0 ** 63])
def test_a_scale_of_0(rotate, lens, new, Hq, spare, size):
    """The mean of the values, however large q and k are (at 2^63 their
    products pass float32); a row of q with an infinity gives NaN."""
    s = Setup(lens, 2, 128, 64, 64, rotate, torch.bfloat16, seed=3, spare=spare)
    s.k *= size
    s.fill()
    q = (s.queries(new, Hq).float() * size).to(torch.bfloat16)
    want, tol = reference(s, q, new, 0.0)
    q[0, 1, 3], q[1, 2, 4] = float("inf"), float("nan")
    got = s.attend(q, new, scale=0.0).double().cpu().numpy()
    assert np.isnan(got[0, 1]).all() and np.isnan(got[1, 2]).all()
    off = np.abs(got - want) <= tol
    off[0, 1] = off[1, 2] = True
    assert off.all()


@pytest.mark.parametrize("rotate", [True, False])
@pytest.mark.parametrize("dtype,D,group", [("fp16", 64, 32), ("bf16", 128, 128), ("bf16", 256, 64)])
@pytest.mark.parametrize("lens,new,Hq,spare", WAYS)
@pytest.mark.parametrize("size", [2.0 ** 11, 2.0 ** 24, 2.0 ** 32, 1e30])
def test_scores_as_large_as_float32_holds(dtype, rotate, D, group, lens, new, Hq, spare, size):
    """Rows whose weight goes to one token, or to some with the same codes: q
    and k along one direction, which the rotation turns into one channel."""
    s = Setup(lens, 2, D, group, 64, rotate, DT[dtype], seed=D, spare=spare)
    r = 2 * torch.rand(s.k.shape[:2], generator=s.gen) - 1
    s.k.copy_(r[..., None].expand(*s.k.shape))
    s.fill()
    q = 1 + torch.rand((sum(new), Hq), generator=s.gen)
    q[:, ::2] *= -1
    q = q[..., None].expand(-1, -1, D).to(s.dtype).cuda()
    scale = size / D
    # Scores of up to twice `size` (a little more after rounding): scale and log2 e are rounded once each, q (2^-17), the
    # sums and three products; from 2^20 on tokens of other scores have no weight, and equal ones the same error.
    ds = 2.1 * size * (2.0 ** -17 + (31 * (D + 4) + 8) * R.U) if size < 2.0 ** 20 else 0.0
    y, tol = reference(s, q, new, float(np.float32(scale)), ds)
    assert (np.abs(s.attend(q, new, scale=scale).double().cpu().numpy() - y) <= tol).all()


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("seed", range(4))
def test_rows_that_see_nothing_change_no_bit_of_others(D, seed):
    s = Setup([40], 2, D, 32, 64, True, torch.float16, seed=seed).fill()
    q = s.queries([47], 4)
    want = crp.attn_kv4(q[7:], s.cache, s.table, ints([40]), ints([0, 40]))
    got = crp.attn_kv4(q, s.cache, s.table, ints([40]), ints([0, 47]))
    assert (got[:7] == 0).all() and torch.equal(got[7:], want)


def large_values(s, size):
    s.v.copy_((s.v.float().sign() * (0.5 + 0.5 * torch.rand(s.v.shape, generator=s.gen).cuda()) * size).to(torch.bfloat16))
    assert s.v.isfinite().all()


@pytest.mark.parametrize("D,group", [(64, 32), (128, 32), (128, 128), (256, 64)])
@pytest.mark.parametrize("lens,new,Hq,spare", WAYS)
@pytest.mark.parametrize("size", [2.0 ** 79, 2.0 ** 84, 2.0 ** 127])
def test_values_as_large_as_the_type_holds(D, group, lens, new, Hq, spare, size):
    """Without a rotation: values of up to 2^127; where there are several groups
    one of them holds ordinary ones, which lose nothing."""
    s = Setup(lens, 2, D, group, 64, False, torch.bfloat16, seed=D + group, spare=spare)
    plain = s.v.clone()
    large_values(s, size)
    s.v[:, 0] = s.v[:, 0].abs()   # of one sign: the average is as large
    if D > group:
        s.v[..., group:2 * group] = plain[..., group:2 * group]
    s.fill()
    s.check(new, Hq, gain=0.5)


@pytest.mark.parametrize("D,group", [(64, 32), (128, 64), (256, 128)])
@pytest.mark.parametrize("lens,new,Hq,spare", WAYS)
def test_large_values_late(D, group, lens, new, Hq, spare):
    """Ordinary tokens, then some of up to 2^120: the sums before them count for
    nothing next to them, and where a group has none they are as they were."""
    s = Setup(lens, 2, D, group, 64, False, torch.bfloat16, seed=D, spare=spare)
    at = starts(s.lens)
    for b, n in enumerate(s.lens):
        s.v[at[b] + n // 2:at[b] + n // 2 + 3, :, :group] *= 2.0 ** 120
    s.fill()
    s.check(new, Hq)


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("lens,new,Hq,spare", WAYS)
@pytest.mark.parametrize("spike", [False, True])
def test_large_values_rotated(D, lens, new, Hq, spare, spike):
    """Values whose rotation float32 holds: all of up to 2^127 / dim, or one of
    2^127 a head."""
    s = Setup(lens, 2, D, 64, 64, True, torch.bfloat16, seed=D, spare=spare)
    if spike:
        s.v[:] = 0
        s.v[..., 17] = 2.0 ** 127
    else:
        large_values(s, 2.0 ** 127 / D)
    s.fill()
    s.check(new, Hq)


def test_a_bad_token_among_large_values():
    """A group of NaN beside groups of large values: only its channels, only the
    rows that see it."""
    s = Setup([2000, 100], 2, 128, 64, 64, False, torch.bfloat16, seed=4, spare=40)
    large_values(s, 2.0 ** 126)
    s.fill()
    q = s.queries([6, 1], 4)
    want, tol = reference(s, q, [6, 1], 128 ** -0.5)
    s.v[1997, 1, 70] = float("inf")
    y = s.fill().attend(q, [6, 1]).double().cpu().numpy()
    bad = np.zeros(y.shape, bool)
    bad[3:6, 2:, 64:] = True
    assert np.array_equal(np.isnan(y), bad) and (np.abs(y - want) <= tol)[~bad].all()


@pytest.mark.parametrize("rotate", [True, False])
@pytest.mark.parametrize("D,group", [(64, 32), (128, 128), (256, 64)])
@pytest.mark.parametrize("lens,new,Hq,spare", WAYS)
@pytest.mark.parametrize("size", [2.0 ** 111, 2.0 ** 125])
def test_queries_as_large_as_the_type_holds(rotate, D, group, lens, new, Hq, spare, size):
    """Large q against small k: scores of ordinary size."""
    s = Setup(lens, 2, D, group, 64, rotate, torch.bfloat16, seed=D, spare=spare)
    s.k *= 2.0 ** -60
    s.fill()
    q = s.queries(new, Hq).float().clamp(-4, 4).mul(size / 4).to(torch.bfloat16)
    assert q.isfinite().all()
    scale = 4 * D ** -0.5 * 2.0 ** 60 / size
    y, tol = reference(s, q, new, scale)
    assert (np.abs(s.attend(q, new, scale=scale).double().cpu().numpy() - y) <= tol).all()


@pytest.mark.parametrize("rotate", [True, False])
@pytest.mark.parametrize("D,group", [(64, 32), (128, 128), (256, 64)])
@pytest.mark.parametrize("lens,new,Hq,spare", WAYS)
@pytest.mark.parametrize("others", [0, 1, 20, 85])
def test_scores_below_what_float32_holds(rotate, D, group, lens, new, Hq, spare, others):
    """Tokens whose scores are -infinity weigh nothing beside others; a row
    that sees no other gives NaN, not what a row gives that sees no token."""
    s = Setup(lens, 2, D, group, 64, rotate, torch.bfloat16, seed=D, spare=spare)
    s.k[:] = -2.0 ** 100
    at = starts(s.lens)
    others = min(others, min(lens) - 1)
    for b in range(len(lens)):
        s.k[at[b]:at[b] + others:2], s.k[at[b + 1] - others:at[b + 1]] = 0, 0
    s.fill()
    q = torch.full((sum(new), Hq, D), 2.0 ** 100, dtype=torch.bfloat16, device="cuda")
    got = s.attend(q, new).double().cpu().numpy()
    if others == 0:
        assert np.isnan(got).all()
    else:
        y, tol = reference(s, q, new, D ** -0.5, 0.0)
        assert (np.abs(got - y) <= tol).all()
