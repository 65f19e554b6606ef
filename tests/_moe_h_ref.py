"""A mixture-of-experts layer whose output shows how exactly the hidden values
h = silu(g) u are held, and the norm that a lost part of h exceeds.

``cancelling``: x = (a, b, +-1, 0, ...), every scale 1.  Gate rows read a only;
up row f reads p a, and b besides where f is odd (p the same for the rows 2 j
and 2 j + 1); down column k takes h[2 j + 1] - h[2 j] for one j.  So
y = silu(a) b, while the two h that it is the difference of are up to
7 a / b = 7168 times as large (b = 2^-9).  The third value of x picks the
expert.  All products and sums before silu are exact in float32."""
import numpy as np
import torch

from . import _w4g_ref as R

B = 2.0 ** -9


def cancelling(M, K, F, E, group, dtype, zeros, pick):
    """x, router, gate, up, down (stored triples) and p [F]; token m on expert pick[m]."""
    rng = np.random.default_rng(M * 1000 + K)
    # the down product's zero points are 8: others would add half of every h of the group to both sides
    z = (*rng.integers(1, 8, size=2), 8) if zeros else (8, 8, 8)

    def stored(q, zero):
        codes = torch.from_numpy((q[..., 0::2] | (q[..., 1::2] << 4)).astype(np.uint8))
        s = torch.ones((*q.shape[:-1], q.shape[-1] // group), dtype=dtype)
        return codes, s, torch.full(s.shape, int(zero), dtype=torch.uint8) if zeros else None

    gate = np.full((E, F, K), z[0], dtype=np.int64)
    gate[..., 0] += 1
    up = np.full((E, F, K), z[1], dtype=np.int64)
    p = 1 + (np.arange(F) // 2) % 7
    up[..., 0] += p
    up[:, 1::2, 1] += 1
    down = np.full((E, K, F), z[2], dtype=np.int64)
    j = np.arange(K) % (F // 2)
    for e in range(E):
        down[e, np.arange(K), 2 * j] -= 1
        down[e, np.arange(K), 2 * j + 1] += 1
    x = torch.zeros((M, K), dtype=torch.float64)
    x[:, 0] = torch.from_numpy(1 + rng.integers(0, 128, size=M) / 128.0)
    x[:, 1] = B
    r = torch.zeros((E, K), dtype=torch.float64)
    for e in range(E):   # logits 4 and below: exact, far apart
        r[e, 2 + e % 4] = 4.0 * (1 if e < 4 else -1)
    for m in range(M):
        x[m, 2 + pick[m] % 4] = 1 if pick[m] < 4 else -1
    return x.to(dtype), r.to(dtype), stored(gate, z[0]), stored(up, z[1]), stored(down, z[2]), p


def expected(x, K, F, p, h_of=None):
    """(y, tol) [M, K]; ``h_of`` rounds float64 h to what a kernel would hold.

    tol: h is off by a rounding of its own (2^-24 of it; silu's error, of some
    2^-21, is common to both), the sums of the parts stay under 2^-7 of h and
    take 6 additions: together under 2^-23 of both h; the output by half a
    step."""
    a = x[:, 0].double().numpy()[:, None]
    silu = a / (1 + np.exp(-a))
    f = np.arange(F)
    h = silu * (a * p + B * (f % 2))
    if h_of is not None:
        h = h_of(h)
    j = np.arange(K) % (F // 2)
    y = silu * B * np.ones((1, K)) if h_of is None else h[:, 2 * j + 1] - h[:, 2 * j]
    size = np.abs(h[:, 2 * j + 1]) + np.abs(h[:, 2 * j])
    err = 2.0 ** -23 * size + 2.0 ** -20 * np.abs(y)
    return y, err + R.half_step(x.dtype) * (np.abs(y) + err)


def bf16_parts(h, parts):
    """h as the sum of so many rounded bf16 values."""
    left = torch.from_numpy(np.ascontiguousarray(h)).float()
    out = torch.zeros_like(left, dtype=torch.float64)
    for _ in range(parts):
        v = left.bfloat16().float()
        out += v.double()
        left = left - v
    return out.numpy()


def norm_limit(y, dtype):
    """Limit of the norm of (output - y): the rounding of y itself, and 2 % for
    what float32 sums add (their error e adds e^2 to the square: up to a fifth
    of the rounding's, 2^-13 of y in fp16, hundreds of float32's steps)."""
    rounded = torch.from_numpy(y).to(dtype).double().numpy()
    return 1.02 * np.linalg.norm(rounded - y)
