"""Attention and the 4-bit cache in float64 (NumPy), written from their
definitions in include/convrot.h, and the bounds that tests hold kernels to.

Bounds.  eps(T) / 2 is half a step of the 16-bit type, u = 2^-24 float32's.

prompt: y = sum p v / sum p.  Each weight p is rounded to T (half a step,
  relative) and y to T; a score is off by its sums, (D + 2) u sum |q k| scale
  at most, and by the exponential's argument, 2 u |score - top| (two
  roundings) and its own 2 u (the instruction's error, under 1 ulp), all of
  which are relative errors of p; the sums over n keys by n u each.  Hence
      |y' - y| <= (eps(T)/2 + e) A + eps(T)/2 |y|,   A = sum p |v| / sum p,
      e = 2 (ds + 4 u (span + 1) + 2 n u),
  ds the largest score error and span the largest |score - top| of the row
  (numerator and denominator each, hence the 2); fp16 weights below 2^-14
  of the largest carry an absolute error instead, 2^-25 of the largest, n of
  which sum to no more than n 2^-25 / sum p of max |v| (sum p >= 1 at the top).
decode: values of the cache are exact in the operands; q and p are each held
  in two bf16 of 8 bits, off by 2^-17 of each; the same with 2^-17 in the place
  of eps(T)/2, and 16 codes' offset in a sum makes its terms up to 31 / 1 of
  a code's size, which the bound has as A with (c + 16) in the place of |c - z|.
"""
import numpy as np
import torch

U = 2.0 ** -24


def hadamard(n):
    h = np.ones((1, 1))
    while h.shape[0] < n:
        h = np.block([[h, h], [h, -h]])
    return h / np.sqrt(n)


def _softmax(s, keep):
    s = np.where(keep, s, -np.inf)
    top = s.max(-1, keepdims=True)
    with np.errstate(invalid="ignore"):
        p = np.where(keep, np.exp(s - top), 0.0)
    return s, top, p


def attend(q, k, v, seen, scale):
    """One head: q [n, D], k, v [m, D] float64; row r sees the first seen[r]
    keys.  (y, bound's parts): A, ds, span, keys, p's sum."""
    n, m = q.shape[0], k.shape[0]
    keep = np.arange(m)[None, :] < np.asarray(seen)[:, None]
    s = q @ k.T * scale
    ds = np.where(keep, np.abs(q) @ np.abs(k).T * abs(scale), 0.0).max(-1, initial=0.0) * (q.shape[1] + 2) * U
    y = np.zeros((n, v.shape[1]))
    A, span, total = np.zeros_like(y), np.zeros(n), np.ones(n)
    some = keep.any(-1)
    if some.any():
        s, top, p = _softmax(s[some], keep[some])
        total[some] = p.sum(-1)
        y[some] = p @ v / total[some][:, None]
        A[some] = p @ np.abs(v) / total[some][:, None]
        span[some] = np.where(keep[some], top - s, 0.0).max(-1)
    return y, (A, ds, np.minimum(span, 40.0), keep.sum(-1), total)


def prompt(q, k, v, cu, causal, scale, dtype):
    """float64 y [T, Hq, D] (NaN where no sequence is) and its tolerance."""
    q, k, v = (t.double().cpu().numpy() for t in (q, k, v))
    T, Hq, D = q.shape
    G = Hq // k.shape[1]
    half = torch.finfo(dtype).eps / 2
    y, tol = np.full(q.shape, np.nan), np.zeros(q.shape)
    for a, b in zip(cu, cu[1:]):
        for h in range(Hq):
            kk, vv = k[a:b, h // G], v[a:b, h // G]
            seen = np.arange(1, b - a + 1) if causal else np.full(b - a, b - a)
            y[a:b, h], (A, ds, span, n, total) = attend(q[a:b, h], kk, vv, seen, scale)
            e = 2 * (ds + 4 * U * (span + 1) + 2 * n * U)
            tol[a:b, h] = (half + e)[:, None] * A + half * np.abs(y[a:b, h]) * (1 + 1e-3)
            if dtype == torch.float16 and b > a:
                # subnormal weights, and a subnormal result
                tol[a:b, h] += (n * 2.0 ** -25 / total)[:, None] * np.abs(vv).max() + 2.0 ** -25
            elif b > a:
                tol[a:b, h] += 2.0 ** -126
    return y, tol


# ---------------------------------------------------------------------------
# The cache
# ---------------------------------------------------------------------------

def rotate32(x):
    """float32 butterflies of strides 1, 2, .. over the last axis."""
    x = x.astype(np.float32)
    D, h = x.shape[-1], 1
    while h < D:
        y = x.reshape(*x.shape[:-1], D // (2 * h), 2, h)
        x = np.stack((y[..., 0, :] + y[..., 1, :], y[..., 0, :] - y[..., 1, :]), -2).reshape(x.shape)
        h *= 2
    return x * np.float32(1 / np.sqrt(D))


def encode(x, group, rotate):
    """16-bit [T, H, D] -> codes [T, H, D] uint8, words uint32 [T, H, D / g]."""
    x = x.float().cpu().numpy()
    with np.errstate(all="ignore"):
        x = rotate32(x) if rotate else x
        x = x.reshape(*x.shape[:-1], -1, group)
        bad = ~np.isfinite(x).all(-1)
        x = np.where(bad[..., None], np.float32(0), x)
        lo, hi = np.minimum(x.min(-1), np.float32(0)), np.maximum(x.max(-1), np.float32(0))
        s = hi / np.float32(15) - lo / np.float32(15)
        w = (s.view(np.uint32) + np.uint32(8)) & np.uint32(0xFFFFFFF0)
        s = w.view(np.float32)
        z = np.where(s > 0, np.clip(np.rint(-lo / s), 0, 15), 0).astype(np.float32)
        c = np.where(s[..., None] > 0, np.clip(np.rint(x / s[..., None]) + z[..., None], 0, 15), 0)
    w = np.where(bad, np.uint32(0x7FC00000), w | z.astype(np.uint32))
    return c.astype(np.uint8).reshape(*c.shape[:-2], -1), w


def values(codes, words, group):
    """float64 x' that codes and words stand for."""
    s = (words & np.uint32(0xFFFFFFF0)).view(np.float32).astype(np.float64)
    z = (words & np.uint32(15)).astype(np.float64)
    return (codes - z.repeat(group, -1)) * s.repeat(group, -1)


def read_cache(codes, words, which, page, D, group):
    """Cache bytes [pages, 2, H, ..] -> codes [pages, H, page, D] and words
    [pages, H, page, D / g], by the layout's description, d by d."""
    P, _, H, _ = codes.shape
    c = codes[:, which]
    out = np.zeros((P, H, page, D), np.uint8)
    r = np.arange(page)
    for d in range(D):
        if which == 0:
            bit = 4 * (d % 8 // 2) + 16 * (d % 2)
            at = r * (D // 2) + 4 * ((d // 8 % 4) * (D // 32) + d // 32) + bit // 8
            out[..., d] = c[..., at] >> (bit % 8) & 15
        else:
            at = (r // 16) * 8 * D + (16 * (d // 32) + d % 16) * 16 + r % 16
            out[..., d] = c[..., at] >> (4 if d % 32 >= 16 else 0) & 15
    return out, words[:, which].reshape(P, H, page, D // group).view(np.uint32)


def decode(q, kc, kw, vc, vw, group, rotate, seen, scale, dtype):
    """One sequence: q [n, Hq, D] 16-bit; codes and words [m, H, ..] of its m
    tokens.  float64 y [n, Hq, D] and its tolerance."""
    D = q.shape[-1]
    q = q.double().cpu().numpy()
    G = q.shape[1] // kc.shape[1]
    H = hadamard(D) if rotate else np.eye(D)
    k, v = values(kc, kw, group), values(vc, vw, group)
    # |x'| with a code's offset of 16 in the sums
    v_big = (vc + 16.0) * (vw & np.uint32(0xFFFFFFF0)).view(np.float32).repeat(group, -1)
    k_big = (kc + 16.0) * (kw & np.uint32(0xFFFFFFF0)).view(np.float32).repeat(group, -1)
    y, tol = np.zeros(q.shape), np.zeros(q.shape)
    half = torch.finfo(dtype).eps / 2
    for h in range(q.shape[1]):
        qr = q[:, h] @ H
        o, (A, ds, span, n, total) = attend(qr, k[:, h // G], v[:, h // G], seen, scale)
        y[:, h] = o @ H
        # two bf16 hold 16 bits: 2^-17 of |q|, summed against k; rotation in float32: log2 D + 1 roundings of |q| H
        ds = (2.0 ** -17 + 12 * U + (D + 4) * U) * scale * (np.abs(q[:, h]) @ np.abs(H) @ k_big[:, h // G].T).max(-1, initial=0)
        big = attend(qr, k[:, h // G], v_big[:, h // G], seen, scale)[0]
        e = 2 * (ds + 4 * U * (span + 1) + 2 * n * U) + 2.0 ** -17
        off = e[:, None] * A + 2 * (n + 4)[:, None] * U * big
        tol[:, h] = off @ np.abs(H) + 20 * U * np.abs(o) @ np.abs(H) + half * np.abs(y[:, h]) * (1 + 1e-3)
        tol[:, h] += 2.0 ** -25 if dtype == torch.float16 else 2.0 ** -126
    return y, tol
