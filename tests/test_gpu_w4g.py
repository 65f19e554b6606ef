"""GPU: the group encoder, and the linear on 4-bit weights with group scales,
against their 64-bit definitions (_w4g_ref.py states the bounds)."""
import numpy as np
import pytest
import torch

import rotated_bit_quantized_convrot_amd as crp

from . import _w4g_ref as R

pytestmark = pytest.mark.gpu
DT = {"bf16": torch.bfloat16, "fp16": torch.float16}


def dev(t):
    return None if t is None else t.cuda()


def activations(M, K, dtype, seed):
    rng = np.random.default_rng(seed)
    x = rng.normal(size=(M, K))
    x[:, rng.choice(K, max(1, K // 200), replace=False)] *= 20.0
    return torch.from_numpy(x.astype(np.float32)).to(dtype)


def check_linear(M, N, K, group, dtype, zeros, bias, seed=0):
    w = R.stored((N,), K, group, dtype, zeros, seed)
    x = activations(M, K, dtype, seed + 1)
    b = torch.randn(N, generator=torch.Generator().manual_seed(seed)).to(dtype) if bias else None
    packed = crp.pack_weight_w4g(*map(dev, w))
    y = crp.linear_w4g(x.cuda(), packed, N, group, zeros=zeros, bias=dev(b))
    assert y.dtype == dtype and tuple(y.shape) == (M, N)
    ref, tol = R.linear(x, w, b)
    off = np.abs(y.cpu().double().numpy() - ref) / tol
    assert off.max() <= 1, (off.max(), np.unravel_index(off.argmax(), off.shape))


# --------------------------------------------------------------------- encoder

@pytest.mark.parametrize("dtype", DT)
@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("zeros", [False, True])
def test_encode_equals_the_definition(dtype, group, zeros):
    rng = np.random.default_rng(group)
    w = rng.normal(0, 0.02, size=(37, 3 * 128)).astype(np.float32)
    w[0] = 0                             # empty groups
    w[1] = np.abs(w[1]) + 0.01           # one sign: the zero point at an end
    w[2] = -np.abs(w[2]) - 0.01
    w[3] = 0.5                           # all equal
    w[4, ::group] = 40.0                 # one large value a group: codes at 0
    w[5] *= 1e-6                         # small, subnormal scales in fp16
    w[6] = np.tile([3.5, 0.5, 1.5, 2.5, -0.5, -1.5, -2.5, -3.5], 48) / 8   # ties
    w[6, ::group] = 7.0 / 8
    w = torch.from_numpy(w).to(DT[dtype])
    got = crp.encode_w4g(w.cuda(), group, zeros)
    for g, r, name in zip(got, R.encode(w, group, zeros), ("codes", "scales", "zeros")):
        assert (g is None) == (r is None)
        if g is not None:
            assert torch.equal(g.cpu().view(torch.uint8), r.view(torch.uint8)), name


def test_encode_stacked_and_empty():
    w = (torch.randn(3, 5, 64) * 0.02).half().cuda()
    c, s, z = crp.encode_w4g(w, 32, True)
    for e in range(3):
        for a, b in zip((c[e], s[e], z[e]), crp.encode_w4g(w[e].contiguous(), 32, True)):
            assert torch.equal(a, b)
    c, s, z = crp.encode_w4g(w[:, :0], 32)
    assert tuple(c.shape) == (3, 0, 32) and tuple(s.shape) == (3, 0, 2) and z is None
    # more rows than one call of the library takes
    tall = (torch.randn((1 << 20) + 3, 32, device="cuda") * 0.02).bfloat16()
    c, s, _ = crp.encode_w4g(tall, 32)
    c1, s1, _ = crp.encode_w4g(tall[-40:].contiguous(), 32)
    assert torch.equal(c[-40:], c1) and torch.equal(s[-40:], s1)


def test_encode_keeps_to_half_a_step():
    """|w - W| <= s/2 plus what the rounding of s and clipping cost."""
    w = (torch.randn(64, 512) * 0.02).bfloat16()
    for zeros, levels in ((False, 7), (True, 15)):
        c, s, z = crp.encode_w4g(w.cuda(), 64, zeros)
        W, _ = R.dequantise(c, s, z)
        step = np.repeat(s.cpu().double().numpy(), 64, -1)
        # a scale rounded down by half a step of bf16 leaves the largest value levels * 2^-8 of a step
        # outside; the rounded zero point moves the range by at most half a step more
        slack = 0.5 + levels * R.half_step(torch.bfloat16) + (0.5 if zeros else 0) + 1e-6
        assert (np.abs(W - w.double().numpy()) <= slack * step).all()


# --------------------------------------------------------------------- linear

@pytest.mark.parametrize("dtype", DT)
@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("zeros", [False, True])
@pytest.mark.parametrize("M", [1, 3, 16, 17, 76])
def test_linear_types(dtype, group, zeros, M):
    check_linear(M, 200, 3 * 128, group, DT[dtype], zeros, bias=zeros, seed=M)


@pytest.mark.parametrize("N", [1, 2, 15, 16, 17, 63, 129])
@pytest.mark.parametrize("M", [1, 2, 15, 33])
def test_linear_odd_rows(M, N):
    check_linear(M, N, 160, 32, torch.bfloat16, True, True, seed=N)


@pytest.mark.parametrize("K,group", [(32, 32), (64, 32), (96, 32), (64, 64), (192, 64), (128, 128), (640, 128),
                                     (2720, 32), (4160, 64), (9728, 128), (20480, 128)])
@pytest.mark.parametrize("M", [1, 8, 40])
def test_linear_depths(K, group, M):
    check_linear(M, 48, K, group, torch.float16 if K % 64 else torch.bfloat16, False, False, seed=K)


@pytest.mark.parametrize("M", [4, 5, 31, 32, 48, 63, 64, 65, 127, 128, 129, 255, 256, 257, 300, 513])
def test_linear_row_counts(M):
    check_linear(M, 272, 512, 64, torch.bfloat16, M % 2 == 1, M % 3 == 0, seed=M)


@pytest.mark.parametrize("dtype", DT)
@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("zeros", [False, True])
@pytest.mark.parametrize("M,N", [(20, 4105), (40, 8200), (130, 4101), (300, 9731), (1000, 4090)])
def test_linear_wide_tiles(dtype, group, zeros, M, N):
    """Every tile that takes many columns, in all its types, with a last one that is not full."""
    check_linear(M, N, 3 * 128 if group == 128 else 3 * 128 + group, group, DT[dtype], zeros, bias=zeros, seed=N)


@pytest.mark.parametrize("M,N,K,group,dtype", [(1, 2560, 2560, 128, "bf16"), (1, 9728, 2560, 64, "fp16"),
                                               (76, 2560, 2560, 128, "fp16"), (1220, 512, 2560, 128, "bf16"),
                                               (200, 4000, 1056, 32, "fp16"), (700, 1100, 1280, 64, "bf16")])
def test_linear_layers(M, N, K, group, dtype):
    check_linear(M, N, K, group, DT[dtype], True, True, seed=5)


def test_linear_rows_do_not_depend_on_each_other():
    """A row's result is the same bits whatever the other rows hold, and a NaN
    or an infinity in one stays in it (an infinity times a code at its zero
    point is a NaN, as in the definition)."""
    w = R.stored((100,), 384, 64, torch.bfloat16, False, 3)
    packed = crp.pack_weight_w4g(*map(dev, w))
    for M in (16, 70, 300):
        x = activations(M, 384, torch.bfloat16, 4).cuda()
        y = crp.linear_w4g(x, packed, 100, 64)
        x2 = x.clone()
        x2[M // 2, 7] = float("nan")
        x2[M // 3, 100] = float("inf")
        y2 = crp.linear_w4g(x2, packed, 100, 64)
        assert torch.isnan(y2[M // 2]).all() and not torch.isfinite(y2[M // 3]).any()
        keep = [m for m in range(M) if m not in (M // 2, M // 3)]
        assert torch.equal(y[keep], y2[keep])
        assert torch.equal(y, crp.linear_w4g(x, packed, 100, 64))


@pytest.mark.parametrize("M,N", [(1, 33), (5, 16), (20, 100), (140, 50)])
def test_linear_writes_only_its_output(M, N):
    """Memory behind y and behind every input keeps its values, and inputs that
    end where their allocation's guard begins are read no further: guards
    hold NaN."""
    K, dtype = 96, torch.bfloat16
    w = R.stored((N,), K, 32, dtype, True, 1)
    packed = crp.pack_weight_w4g(*map(dev, w))
    x = activations(M, K, dtype, 2)
    xg = torch.full((M * K + 4096,), float("nan"), dtype=dtype, device="cuda")
    xg[:M * K] = x.cuda().view(-1)
    pg = torch.full((packed.numel() + 8192,), 0xFF, dtype=torch.uint8, device="cuda")
    pg[:packed.numel()] = packed
    yg = torch.full((M * N + 4096,), 7.0, dtype=dtype, device="cuda")
    crp.linear_w4g(xg[:M * K].view(M, K), pg[:packed.numel()], N, 32, zeros=True, out=yg[:M * N].view(M, N))
    assert (yg[M * N:] == 7.0).all()
    ref, tol = R.linear(x, w)
    assert (np.abs(yg[:M * N].view(M, N).cpu().double().numpy() - ref) <= tol).all()


def test_linear_zero_rows_and_convenience():
    w = (torch.randn(96, 256) * 0.02).half()
    pw = crp.pack_linear(w.cuda(), torch.ones(96, dtype=torch.float16, device="cuda"), w4g=64, zeros=True)
    assert pw.kind == crp.W4G and pw.scale is None
    assert tuple(crp.linear(torch.empty((0, 256), dtype=torch.float16, device="cuda"), pw).shape) == (0, 96)
    x = activations(9, 256, torch.float16, 0)
    ref, tol = R.linear(x, tuple(t.cpu() for t in crp.encode_w4g(w.cuda(), 64, True)), torch.ones(96).half())
    assert (np.abs(crp.linear(x.cuda(), pw).cpu().double().numpy() - ref) <= tol).all()


def test_linear_small_and_large_values():
    """Scales at the ends of the type's range: subnormal fp16, large bf16."""
    for dtype, size in ((torch.float16, 3e-7), (torch.float16, 6e4), (torch.bfloat16, 1e-30), (torch.bfloat16, 1e30)):
        c, s, z = R.stored((40,), 128, 32, dtype, True, 9)
        s = torch.full_like(s, size)
        x = (activations(3, 128, dtype, 1).float() * (1e-3 if size > 1 else 1.0)).to(dtype)
        if dtype is torch.float16 and size > 1:
            x = (x.float() * 1e-3).to(dtype)
        packed = crp.pack_weight_w4g(dev(c), dev(s), dev(z))
        ref, tol = R.linear(x, (c, s, z))
        y = crp.linear_w4g(x.cuda(), packed, 40, 32, zeros=True).cpu().double().numpy()
        inside = np.abs(ref) < float(torch.finfo(dtype).max) * 0.99
        assert (np.abs(y - ref)[inside] <= tol[inside]).all(), (dtype, size)


def test_linear_on_another_stream():
    w = R.stored((64,), 256, 128, torch.bfloat16, False, 3)
    x = activations(5, 256, torch.bfloat16, 4)
    ref, tol = R.linear(x, w)
    st = torch.cuda.Stream()
    with torch.cuda.stream(st):
        packed = crp.pack_weight_w4g(*map(dev, w))
        y = crp.linear_w4g(x.cuda(), packed, 64, 128)
    st.synchronize()
    assert (np.abs(y.cpu().double().numpy() - ref) <= tol).all()


@pytest.mark.parametrize("M", [1, 40, 200])
def test_linear_and_encode_in_a_graph(M):
    """Captured calls replayed on new inputs, with eager work in between."""
    K, N = 512, 200
    x = activations(M, K, torch.bfloat16, 1).cuda()
    w = (torch.randn(N, K) * 0.02).bfloat16().cuda()

    def step():
        c, s, z = crp.encode_w4g(w, 64, True)
        return c, crp.linear_w4g(x, crp.pack_weight_w4g(c, s, z), N, 64, zeros=True)
    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        codes, y = step()
    for i in range(4):
        x.copy_(activations(M, K, torch.bfloat16, 10 + i))
        w.copy_((torch.randn(N, K) * 0.02).bfloat16())
        want = step()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(codes, want[0]) and torch.equal(y, want[1])
