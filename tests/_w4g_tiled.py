"""Large weights of few different rows, and their 64-bit results with bounds:
row n of a weight is row (a + n) mod B of B stored ones (B a prime), so that
every row of every tile is checked at the cost of B.

The bounds count what the kernels sum (in units of float32's step, 2^-23,
which allows for additions that truncate): (q - z) s x, or for bf16 operands
of a weight with zero points (q - 8) s x and (8 - z) s x; a group's additions,
the scaled groups', the joining of waves and blocks; and the output's half
step."""
import numpy as np
import torch

import rotated_bit_quantized_convrot_amd as crp

from . import _w4g_ref as R

BASE = 61


def rows(triple, index):
    """The stored weight of rows `index` (any shape, appended to the front), on the GPU."""
    at = torch.as_tensor(index).cuda()
    return [None if t is None else t.cuda()[at].contiguous() for t in triple]


def operands(triple, bf16):
    """(W, A) of a stored weight in float64: the weight, and the absolute size of what is summed for it."""
    codes, s, z = triple
    c = codes.numpy()
    q = np.stack((c & 15, c >> 4), -1).reshape(*c.shape[:-1], -1).astype(np.float64)
    sf = np.repeat(s.double().numpy(), q.shape[-1] // s.shape[-1], -1)
    if z is None:
        return (q - 8) * sf, np.abs(q - 8) * sf
    zf = np.repeat((z.numpy() & 15).astype(np.float64), q.shape[-1] // s.shape[-1], -1)
    return (q - zf) * sf, ((np.abs(q - 8) + np.abs(8 - zf)) if bf16 else np.abs(q - zf)) * sf


def product(x, W, A, group, parts=1):
    """x W^T and its float32 error; x [M, K] float64."""
    steps = parts * group + 2 * (W.shape[1] // group) + 24
    return x @ W.T, R.F32 * steps * (np.abs(x) @ A.T)


def rounded(y, err, dtype):
    tiny = float(torch.finfo(dtype).smallest_normal) * torch.finfo(dtype).eps
    return err + R.half_step(dtype) * (np.abs(y) + err) + tiny


class Linear:
    def __init__(self, N, K, group, dtype, zeros, seed):
        self.N, self.group, self.dtype, self.zeros = N, group, dtype, zeros
        self.base = R.stored((BASE,), K, group, dtype, zeros, seed)
        self.index = np.arange(N) % BASE
        self.packed = crp.pack_weight_w4g(*rows(self.base, self.index))

    def check(self, x):
        y = crp.linear_w4g(x.cuda(), self.packed, self.N, self.group, zeros=self.zeros)
        ref, err = product(x.double().numpy(), *operands(self.base, self.dtype is torch.bfloat16), self.group)
        tol = rounded(ref, err, self.dtype)
        off = np.abs(y.cpu().double().numpy() - ref[:, self.index]) / tol[:, self.index]
        assert off.max() <= 1, (off.max(), np.unravel_index(off.argmax(), off.shape))
        return y


class Experts:
    def __init__(self, K, F, E, group, dtype, zeros, seed):
        self.K, self.F, self.E, self.group, self.dtype, self.zeros = K, F, E, group, dtype, zeros
        self.base = [R.stored((BASE,), k, group, dtype, zeros, seed + i) for i, k in enumerate((K, K, F))]
        self.index = [(7 * np.arange(E)[:, None] + 3 * i + np.arange(n)) % BASE for i, n in enumerate((F, F, K))]
        self.packed = [crp.pack_weight_w4g(*rows(b, i)) for b, i in zip(self.base, self.index)]

    def run(self, x, r, topk, norm, **kw):
        return crp.moe_w4g(x.cuda(), r.cuda(), *self.packed, self.F, self.group, topk, zeros=self.zeros, norm=norm,
                           routing=True, **kw)

    def check(self, x, r, topk, norm):
        """Runs the layer and compares it; returns (y, ids, weights)."""
        got = self.run(x, r, topk, norm)
        ids, c, c_rel = R.route(x, r, topk, norm)
        xd, bf16 = x.double().numpy(), self.dtype is torch.bfloat16
        (G, dG), (U, dU) = (product(xd, *operands(b, bf16), self.group) for b in self.base[:2])
        Wd, Ad = operands(self.base[2], True)
        y, err = np.zeros((len(x), self.K)), np.zeros((len(x), self.K))
        for rank in range(topk):
            e = ids[:, rank]
            gi, ui, di = (i[e] for i in self.index)
            take = np.take_along_axis
            g, dg, u, du = take(G, gi, 1), take(dG, gi, 1), take(U, ui, 1), take(dU, ui, 1)
            silu = g / (1 + np.exp(-g))
            h = silu * u
            # |silu'| < 1.1; exp, division and the products: 8 steps, and |g| of exp's argument
            dh = 1.1 * dg * (np.abs(u) + du) + np.abs(silu) * du + R.F32 * (8 + np.abs(g)) * np.abs(h)
            v, dv = product(h, Wd, Ad, self.group, 3)
            dv = dv + dh @ np.abs(Wd).T
            w = c[:, rank:rank + 1]
            rel = c_rel[:, rank:rank + 1] + R.F32 * (topk + 16)
            y += take(w * v, di, 1)
            err += take(w * (dv + rel * (np.abs(v) + dv) + R.F32 * 24 * (np.abs(h) @ Ad.T)), di, 1)
        assert np.array_equal(got[1].cpu().numpy(), ids)
        assert (np.abs(got[2].cpu().double().numpy() - c) <= c * c_rel + 3.5 * 2.0 ** -149).all()
        off = np.abs(got[0].cpu().double().numpy() - y) / rounded(y, err, self.dtype)
        assert off.max() <= 1, (off.max(), np.unravel_index(off.argmax(), off.shape))
        self.exact = y
        return got
