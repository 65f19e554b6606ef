"""GPU: the mixture-of-experts layer on 4-bit weights with group scales against
its 64-bit definition (_w4g_ref.py states the bounds)."""
import numpy as np
import pytest
import torch

import rotated_bit_quantized_convrot_amd as crp

from . import _w4g_ref as R

pytestmark = pytest.mark.gpu
DT = {"bf16": torch.bfloat16, "fp16": torch.float16}


def dev(w):
    return [None if t is None else t.cuda() for t in w]


def layer(M, K, F, E, group, dtype, zeros, seed=0):
    rng = np.random.default_rng(seed)
    x = torch.from_numpy(rng.normal(size=(M, K)).astype(np.float32)).to(dtype)
    r = torch.from_numpy((rng.normal(size=(E, K)) * 1.5 / np.sqrt(K)).astype(np.float32)).to(dtype)
    return (x, r, R.stored((E, F), K, group, dtype, zeros, seed + 1), R.stored((E, F), K, group, dtype, zeros, seed + 2),
            R.stored((E, K), F, group, dtype, zeros, seed + 3))


def run(x, r, gate, up, down, topk, norm, **kw):
    F = gate[0].shape[1]
    group = x.shape[1] // gate[1].shape[-1]
    packed = [crp.pack_weight_w4g(*dev(w)) for w in (gate, up, down)]
    return crp.moe_w4g(x.cuda(), r.cuda(), *packed, F, group, topk, zeros=gate[2] is not None, norm=norm, **kw)


def compare(got, want, dtype):
    y, ids, c = (t.cpu() for t in got)
    ry, rids, rc, ctol, ytol = want
    assert np.array_equal(ids.numpy(), rids)
    assert (np.abs(c.double().numpy() - rc) <= ctol).all()
    off = np.abs(y.double().numpy() - ry)
    assert (off / ytol).max() <= 1
    # rounding h and rounding y are off by half a step of each element at most, the first one's
    # errors independent of each other: together under one step of y's norm, whatever the sizes
    if ry.size > 64:
        assert np.linalg.norm(off) <= torch.finfo(dtype).eps * np.linalg.norm(ry)


@pytest.mark.parametrize("dtype", DT)
@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("zeros", [False, True])
@pytest.mark.parametrize("M,norm", [(1, True), (7, False), (30, True), (64, False)])
def test_moe_types(dtype, group, zeros, M, norm):
    args = layer(M, 256, 384, 12, group, DT[dtype], zeros, seed=M)
    compare(run(*args, 3, norm, routing=True), R.moe(*args, 3, norm), DT[dtype])


@pytest.mark.parametrize("M", [1, 2, 5, 16, 17, 33, 63, 64, 65, 130])
@pytest.mark.parametrize("E,topk", [(1, 1), (8, 2), (60, 4), (130, 8)])
def test_moe_batches_and_experts(M, E, topk):
    args = layer(M, 160, 96, E, 32, torch.bfloat16, M % 2 == 0, seed=E)
    compare(run(*args, topk, True, routing=True), R.moe(*args, topk, True), torch.bfloat16)


@pytest.mark.parametrize("E,topk", [(16, 16), (17, 1), (64, 7), (65, 16), (256, 8), (1000, 16), (1024, 3)])
@pytest.mark.parametrize("norm", [True, False])
def test_moe_choices(E, topk, norm):
    args = layer(9, 64, 32, E, 32, torch.float16, False, seed=E)
    compare(run(*args, topk, norm, routing=True), R.moe(*args, topk, norm), torch.float16)


@pytest.mark.parametrize("K,F", [(32, 32), (32, 1024), (1376, 96), (2048, 768), (544, 2016)])
def test_moe_widths(K, F):
    args = layer(6, K, F, 5, 32, torch.bfloat16, True, seed=K)
    compare(run(*args, 2, True, routing=True), R.moe(*args, 2, True), torch.bfloat16)


@pytest.mark.parametrize("dtype", DT)
@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("zeros", [False, True])
@pytest.mark.parametrize("M,E,F,topk", [(17, 8, 2176, 3), (100, 8, 2176, 2), (64, 5, 3328, 3)])
def test_moe_wide_experts(dtype, group, zeros, M, E, F, topk):
    """Many hidden columns and some tokens an expert (up to more than two operands of them): gate and up
    with shared rows, the last block not full in groups of 32."""
    args = layer(M, 128 + group, F - 32 * (group == 32), E, group, DT[dtype], zeros, seed=M)
    compare(run(*args, topk, zeros, routing=True), R.moe(*args, topk, zeros), DT[dtype])


@pytest.mark.parametrize("dtype", DT)
@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("zeros", [False, True])
@pytest.mark.parametrize("M,E", [(17, 6), (40, 6), (64, 2), (131, 3)])
def test_moe_wide_outputs(dtype, group, zeros, M, E):
    """Many columns and some tokens an expert: the down product's wide blocks, the last one not full."""
    args = layer(M, 4096 + group, 256 + group, E, group, DT[dtype], zeros, seed=M)
    compare(run(*args, 2, zeros, routing=True), R.moe(*args, 2, zeros), DT[dtype])


def test_all_tokens_on_one_expert():
    """One expert takes every token (more than one tile of them), the others none."""
    x, r, g, u, d = layer(64, 128, 128, 10, 64, torch.bfloat16, False)
    r = torch.zeros_like(r)
    r[7] = torch.sign(x.float().mean(0) + 1e-3).to(r.dtype)
    x = (x.float().abs() * torch.sign(r[7].float())).to(x.dtype)
    got = run(x, r, g, u, d, 1, False, routing=True)
    assert (got[1] == 7).all()
    compare(got, R.moe(x, r, g, u, d, 1, False), torch.bfloat16)


@pytest.mark.parametrize("E", [64, 200])
def test_most_tokens_on_one_of_many_experts(E):
    """Few tokens per expert on average, and one that has three tiles of them."""
    x, r, g, u, d = layer(40, 128, 96, E, 32, torch.bfloat16, True, seed=E)
    r[E - 3] = torch.sign(x.float().mean(0) + 1e-3).to(r.dtype)
    x = (x.float().abs() * torch.sign(r[E - 3].float())).to(x.dtype)
    got = run(x, r, g, u, d, 2, True, routing=True)
    assert (got[1][:, 0] == E - 3).all()
    compare(got, R.moe(x, r, g, u, d, 2, True), torch.bfloat16)


def test_ties_go_to_the_lowest_index():
    x, r, g, u, d = layer(5, 128, 64, 70, 64, torch.bfloat16, False)
    r[:] = r[0]                              # every logit of a row equal
    got = run(x, r, g, u, d, 6, True, routing=True)
    assert (got[1].cpu() == torch.arange(6, dtype=torch.int32)).all()
    assert (got[2].cpu() - 1 / 6).abs().max() <= 4 * R.F32
    compare(got, R.moe(x, r, g, u, d, 6, True), torch.bfloat16)
    r[:] = 0                                 # and zeros of either sign
    r[3] = -r[3]
    assert (run(x, r, g, u, d, 6, True, routing=True)[1].cpu() == torch.arange(6, dtype=torch.int32)).all()


def test_nan_and_infinite_rows_stay_in_their_rows():
    args = layer(20, 128, 64, 16, 64, torch.bfloat16, False)
    want = R.moe(*args, 3, True)
    y, ids, c = run(*args, 3, True, routing=True)
    x = args[0].clone()
    x[4, 9] = float("nan")
    x[11, 0] = float("inf")
    y2, ids2, c2 = run(x, *args[1:], 3, True, routing=True)
    assert torch.isnan(y2[4]).all() and torch.isnan(y2[11]).all()
    assert (ids2 >= 0).all() and (ids2 < 16).all()
    assert all(len(set(row)) == 3 for row in ids2.cpu().tolist())
    assert (ids2[4].cpu() == torch.arange(3, dtype=torch.int32)).all()     # all NaN: by index
    keep = [m for m in range(20) if m not in (4, 11)]
    assert torch.equal(y[keep], y2[keep]) and torch.equal(ids[keep], ids2[keep]) and torch.equal(c[keep], c2[keep])
    assert np.array_equal(ids.cpu().numpy(), want[1])


def test_moe_is_repeatable_and_independent_of_the_workspace():
    x, r, g, u, d = layer(40, 256, 128, 24, 128, torch.bfloat16, False)
    packed = [crp.pack_weight_w4g(*dev(w)) for w in (g, u, d)]
    x, r = x.cuda(), r.cuda()
    need = crp.moe_w4g_workspace_bytes(40, 256, 128, 24, 4, 128)
    first = None
    for fill in (0, 0xFF, 0x7F, 0x80):
        ws = torch.full((need + 4096,), fill, dtype=torch.uint8, device="cuda")
        out = torch.full((41, 256), 3.0, dtype=torch.bfloat16, device="cuda")
        crp.moe_w4g(x, r, *packed, 128, 128, 4, out=out[:40], workspace=ws[:need])
        assert (out[40] == 3.0).all() and (ws[need:] == fill).all()
        first = out if first is None else first
        assert torch.equal(first, out)
    # a row alone, and in a batch that goes in passes: the same choice, the same sums within the bound
    y, ids, c = crp.moe_w4g(x.repeat(4, 1), r, *packed, 128, 128, 4, routing=True)
    assert torch.equal(y[:40], y[40:80]) or np.allclose(y[:40].cpu().float(), y[40:80].cpu().float(), rtol=2 ** -6)
    assert torch.equal(ids.view(4, 40, 4)[0], ids.view(4, 40, 4)[3]) and torch.equal(c[:40], c[120:])


def test_moe_zero_rows_and_convenience():
    torch.manual_seed(0)
    E, F, K = 6, 64, 128
    w = [(torch.randn(s) * 0.05).half() for s in ((E, F, K), (E, F, K), (E, K, F))]
    pe = crp.pack_experts(*(t.cuda() for t in w), group=64, zeros=True)
    r = torch.randn(E, K).half()
    y, ids, c = crp.moe(torch.empty((0, K), dtype=torch.float16, device="cuda"), r.cuda(), pe, 2, routing=True)
    assert tuple(y.shape) == (0, K) and tuple(ids.shape) == (0, 2) and tuple(c.shape) == (0, 2)
    x = torch.randn(3, K).half()
    st = [tuple(t.cpu() for t in crp.encode_w4g(v.cuda(), 64, True)) for v in w]
    compare(crp.moe(x.cuda(), r.cuda(), pe, 2, routing=True), R.moe(x, r, *st, 2, True), torch.float16)
    assert torch.equal(crp.moe(x.cuda(), r.cuda(), pe, 2), crp.moe(x.cuda(), r.cuda(), pe, 2, routing=True)[0])


@pytest.mark.parametrize("M", [3, 64, 100])
def test_moe_in_place_and_on_another_stream(M):
    """y in x's place; and the same layers on two streams at once, a workspace each."""
    x, r, *w = layer(M, 512, 256, 16, 64, torch.bfloat16, False, seed=M)
    packed = [crp.pack_weight_w4g(*dev(v)) for v in w]
    xs = [x.cuda(), x.flip(0).cuda()]
    r = r.cuda()
    want = [crp.moe_w4g(t, r, *packed, 256, 64, 4, routing=True) for t in xs]
    y = xs[0].clone()
    crp.moe_w4g(y, r, *packed, 256, 64, 4, out=y)
    assert torch.equal(y, want[0][0])
    need = crp.moe_w4g_workspace_bytes(M, 512, 256, 16, 4, 64)
    ws = [torch.empty(need, dtype=torch.uint8, device="cuda") for _ in xs]
    streams = [torch.cuda.Stream() for _ in xs]
    torch.cuda.synchronize()
    got = [[], []]
    for _ in range(8):
        for i, st in enumerate(streams):
            with torch.cuda.stream(st):
                got[i].append(crp.moe_w4g(xs[i], r, *packed, 256, 64, 4, workspace=ws[i], routing=True))
    torch.cuda.synchronize()
    for i in range(2):
        for g in got[i]:
            assert all(torch.equal(a, b) for a, b in zip(g, want[i]))


@pytest.mark.parametrize("M", [1, 12, 64])
def test_moe_in_two_graphs(M):
    """Two captured layers on one workspace, replayed in turn on new inputs on
    one stream, with eager calls between."""
    layers = []
    K, F, E = 256, 128, 20
    ws = torch.empty(crp.moe_w4g_workspace_bytes(M, K, F, E, 4, 64), dtype=torch.uint8, device="cuda")
    for s in range(2):
        x, r, *w = layer(M, K, F, E, 64, torch.bfloat16, False, seed=s)
        packed = [crp.pack_weight_w4g(*dev(v)) for v in w]
        layers.append((x.cuda(), r.cuda(), packed))

    def step(i, workspace=None):
        x, r, packed = layers[i]
        return crp.moe_w4g(x, r, *packed, F, 64, 4, workspace=workspace, routing=True)
    step(0), step(1)
    torch.cuda.synchronize()
    graphs = []
    for i in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            got = step(i, ws)
        graphs.append((g, got))
    for n in range(4):
        for i in range(2):
            layers[i][0].copy_(torch.randn(M, K))
            want = step(i)
            graphs[i][0].replay()
            torch.cuda.synchronize()
            for a, b in zip(graphs[i][1], want):
                assert torch.equal(a, b)


def test_decoder_block_of_linears_and_experts():
    """Encoded weights through the linear, then the experts, as a decoder layer
    runs them while it generates, against 64 bits at every step."""
    torch.manual_seed(1)
    K, F, E = 256, 128, 8
    proj = (torch.randn(K, K) / 16).bfloat16()
    ws = [(torch.randn(s) * 0.08).bfloat16() for s in ((E, F, K), (E, F, K), (E, K, F))]
    r = (torch.randn(E, K) / 8).bfloat16()
    pw = crp.pack_linear(proj.cuda(), w4g=128)
    pe = crp.pack_experts(*(w.cuda() for w in ws), group=64)
    x = torch.randn(2, K).bfloat16()
    stored = tuple(None if t is None else t.cpu() for t in crp.encode_w4g(proj.cuda(), 128))
    experts = [tuple(None if t is None else t.cpu() for t in crp.encode_w4g(w.cuda(), 64)) for w in ws]
    for _ in range(3):
        a = crp.linear(x.cuda(), pw)
        ref, tol = R.linear(x, stored)
        assert (np.abs(a.cpu().double().numpy() - ref) <= tol).all()
        got = crp.moe(a, r.cuda(), pe, 2, routing=True)
        compare(got, R.moe(a.cpu(), r, *experts, 2, True), torch.bfloat16)
        x = torch.nn.functional.layer_norm((a + got[0]).float().cpu(), (K,)).bfloat16()
