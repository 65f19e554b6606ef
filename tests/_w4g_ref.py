"""64-bit definitions of the operators on 4-bit weights with group scales, and
the error bounds their kernels have to stay under.

Roundings counted: products of two 16-bit values are exact in float32; a
group's sum takes at most 128 additions, each off by at most one step of
float32 (2^-23 relative, which allows for additions that truncate) of the
absolute sum; the scaled group sums are added with 2 roundings each; the
16-bit output is off by half a step."""
import numpy as np
import torch

F32 = 2.0 ** -23


def half_step(dtype):
    return torch.finfo(dtype).eps / 2


def stored(shape, K, group, dtype, zeros, seed):
    """Random codes, scales and zero points; scales positive, around 0.008."""
    rng = np.random.default_rng(seed)
    q = rng.integers(0, 16, size=(*shape, K), dtype=np.uint8)
    codes = torch.from_numpy(q[..., 0::2] | (q[..., 1::2] << 4))
    s = torch.from_numpy(np.exp(rng.normal(-4.8, 0.3, size=(*shape, K // group))).astype(np.float32)).to(dtype)
    z = torch.from_numpy(rng.integers(0, 16, size=(*shape, K // group), dtype=np.uint8)) if zeros else None
    return codes, s, z


def dequantise(codes, s, z):
    """(W, B) in float64: the weight, and per element s (16 + q + 16 + z), the
    absolute size of what the kernel adds up for it."""
    c = codes.cpu().numpy()
    q = np.stack((c & 15, c >> 4), -1).reshape(*c.shape[:-1], -1).astype(np.float64)
    g = q.shape[-1] // s.shape[-1]
    sf = np.repeat(s.cpu().double().numpy(), g, -1)
    zf = 8.0 if z is None else np.repeat((z.cpu().numpy() & 15).astype(np.float64), g, -1)
    return (q - zf) * sf, (32.0 + q + zf) * sf


def sum_bound(xabs, B, group):
    """Bound of the float32 error of x W^T: xabs [M, K], B [N, K]."""
    K = B.shape[-1]
    return F32 * (min(group, 128) + 8 + 2 * (K // group)) * (xabs @ B.T)


def linear(x, w, bias=None):
    """(y, bound) of the linear; w the stored triple."""
    W, B = dequantise(*w)
    group = W.shape[-1] // w[1].shape[-1]
    xd = x.cpu().double().numpy()
    y = xd @ W.T
    err = sum_bound(np.abs(xd), B, group)
    if bias is not None:
        b = bias.cpu().double().numpy()
        y = y + b
        err = err + F32 * (np.abs(b) + np.abs(y))
    tiny = float(torch.finfo(x.dtype).smallest_normal) * torch.finfo(x.dtype).eps
    return y, err + half_step(x.dtype) * (np.abs(y) + err) + tiny


def route(x, router, topk, norm):
    """ids [M, topk], weights [M, topk] and the relative error of a float32
    softmax: its argument's rounding, exp and division (2 steps each), the sum."""
    logits = x.cpu().double().numpy() @ router.cpu().double().numpy().T
    E = logits.shape[1]
    order = np.argsort(-logits, axis=1, kind="stable")[:, :topk]
    top = np.take_along_axis(logits, order, 1)
    arg = logits - top[:, :1]
    p = np.exp(arg)
    chosen = np.take_along_axis(p, order, 1)
    total = (chosen if norm else p).sum(1, keepdims=True)
    rel = F32 * (np.abs(np.take_along_axis(arg, order, 1)) + 4 + E + topk)
    return order, chosen / total, rel


def moe(x, router, gate, up, down, topk, norm):
    """(y, ids, weights, weight error, bound) of the layer."""
    dtype = x.dtype
    ids, c, c_rel = route(x, router, topk, norm)
    xd = x.cpu().double().numpy()
    xa = np.abs(xd)
    M, K = xd.shape
    y, err = np.zeros((M, K)), np.zeros((M, K))
    hs = half_step(dtype)
    tiny = float(torch.finfo(dtype).smallest_normal) * torch.finfo(dtype).eps
    steps = 0
    for e in sorted(set(ids.ravel().tolist())):
        m, r = np.nonzero(ids == e)
        pick = [tuple(None if t is None else t[e] for t in w) for w in (gate, up, down)]
        (Wg, Bg), (Wu, Bu), (Wd, Bd) = (dequantise(*w) for w in pick)
        group = Wg.shape[1] // pick[0][1].shape[1]
        g, u = xd[m] @ Wg.T, xd[m] @ Wu.T
        dg, du = sum_bound(xa[m], Bg, group), sum_bound(xa[m], Bu, group)
        silu = g / (1 + np.exp(-g))
        w = c[m, r][:, None]
        h = w * silu * u
        # |silu'| < 1.1; exp, division and the products: 8 steps, and |g| of exp's argument
        dh = w * (1.1 * dg * (np.abs(u) + du) + np.abs(silu) * du) + np.abs(h) * (c_rel[m, r][:, None] + F32 * (8 + np.abs(g)))
        dh = dh + hs * (np.abs(h) + dh) + tiny
        y[m] += h @ Wd.T
        steps += 2 * (Wd.shape[1] // group)
        err[m] += dh @ np.abs(Wd).T + F32 * (group + 8 + 2 * (Wd.shape[1] // group)) * ((np.abs(h) + dh) @ Bd.T)
    err += F32 * 2 * topk * np.abs(y)
    # below 2^-126 float32 values lie 2^-149 apart: exp within 3 of those, over a sum of at least 1
    # (it contains exp(0)), and the quotient within half a one
    return y, ids, c, c * c_rel + 3.5 * 2.0 ** -149, err + hs * (np.abs(y) + err) + tiny


def encode(w, group, zeros):
    """(codes, scales, zeros) as tensors, by float32 NumPy arithmetic."""
    v = w.cpu().float().numpy()
    v = v.reshape(*v.shape[:-1], -1, group)
    f = np.float32
    with np.errstate(divide="ignore", invalid="ignore"):
        if zeros:
            lo, hi = np.minimum(v.min(-1), f(0)), np.maximum(v.max(-1), f(0))
            s16 = torch.from_numpy((hi - lo) / f(15)).to(w.dtype)
            s = s16.float().numpy()
            z = np.where(s > 0, np.clip(np.rint(-lo / s), 0, 15), 0).astype(np.float32)
            q = np.where(s[..., None] > 0, np.clip(np.rint(v / s[..., None]) + z[..., None], 0, 15), 0)
            zt = torch.from_numpy(z.astype(np.uint8))
        else:
            s16 = torch.from_numpy(np.abs(v).max(-1) / f(7)).to(w.dtype)
            s = s16.float().numpy()
            q = np.where(s[..., None] > 0, np.clip(np.rint(v / s[..., None]), -8, 7) + 8, 8)
            zt = None
    q = q.astype(np.uint8).reshape(*w.shape)
    return torch.from_numpy(q[..., 0::2] | (q[..., 1::2] << 4)), s16, zt
