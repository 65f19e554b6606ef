"""GPU: the 4-bit key / value cache: its writer, code for code, and attention
over it against the 64-bit definition (_attn_ref.py states the bounds)."""
import numpy as np
import pytest
import torch

import rotated_bit_quantized_convrot_amd as crp

from . import _attn_ref as R

pytestmark = pytest.mark.gpu
DT = {"bf16": torch.bfloat16, "fp16": torch.float16}
FORMS = [(64, 32), (64, 64), (128, 32), (128, 64), (128, 128), (256, 32), (256, 64), (256, 128)]


def starts(lens):
    return [0] + [int(c) for c in np.cumsum(lens)]


def ints(x):
    return torch.tensor(x, dtype=torch.int32).cuda()


class Setup:
    """Sequences of some lengths whose pages lie anywhere in the cache."""

    def __init__(self, lens, H, D, group, page, rotate, dtype, seed=0, spare=2):
        gen = torch.Generator().manual_seed(seed)
        self.lens, self.H, self.D, self.group, self.page, self.dtype = list(lens), H, D, group, page, dtype
        self.rotate = rotate
        need = [-(-n // page) for n in lens]
        order = torch.randperm(sum(need) + 3, generator=gen).tolist()
        at = starts(need)
        wide = max(need + [1]) + spare
        self.table = ints([order[at[b]:at[b + 1]] + [-1] * (wide - n) for b, n in enumerate(need)])
        self.k = torch.randn((sum(lens), H, D), generator=gen).to(dtype).cuda()
        self.v = torch.randn((sum(lens), H, D), generator=gen).to(dtype).cuda()
        # a key head's loud channels
        self.k[:, :, 3] *= 6
        self.cache = crp.kv4_cache(sum(need) + 3, page, H, D, group=group, rotate=rotate)
        # what was never written is not to be read
        self.cache.codes.fill_(0xA5)
        self.cache.scales.fill_(0x7FC00000)
        self.gen = gen

    def fill(self):
        crp.kv4_append(self.k, self.v, self.cache, self.table, ints(self.lens), ints(starts(self.lens)))
        return self

    def queries(self, new, Hq, gain=1.5):
        q = torch.randn((sum(new), Hq, self.D), generator=self.gen) * gain
        q[:, :, 3] /= 6
        return q.to(self.dtype).cuda()

    def reference(self, q, new, scale=None):
        scale = self.D ** -0.5 if scale is None else scale
        y, tol = np.zeros(q.shape), np.zeros(q.shape)
        a, c = starts(new), starts(self.lens)
        kc, kw = R.encode(self.k, self.group, self.rotate)
        vc, vw = R.encode(self.v, self.group, self.rotate)
        for b, n in enumerate(self.lens):
            one = slice(c[b], c[b + 1])
            seen = np.clip(n - new[b] + 1 + np.arange(new[b]), 0, n)
            y[a[b]:a[b + 1]], tol[a[b]:a[b + 1]] = R.decode(q[a[b]:a[b + 1]], kc[one], kw[one], vc[one], vw[one],
                                                            self.group, self.rotate, seen, scale, self.dtype)
        return y, tol

    def attend(self, q, new, **kw):
        return crp.attn_kv4(q, self.cache, self.table, ints(self.lens), ints(starts(new)), **kw)

    def check(self, new, Hq, gain=1.5, scale=None, **kw):
        q = self.queries(new, Hq, gain)
        got = self.attend(q, new, scale=scale, **kw)
        y, tol = self.reference(q, new, scale)
        off = np.abs(got.double().cpu().numpy() - y)
        assert (off / tol).max(initial=0) <= 1
        return q, got


# ---------------------------------------------------------------------------
# The writer
# ---------------------------------------------------------------------------

def cached(s):
    """Codes and words of every token of the sequences, as the cache has them."""
    out = []
    codes, words = s.cache.codes.cpu().numpy(), s.cache.scales.cpu().numpy()
    table = s.table.cpu().numpy()
    for which in (0, 1):
        c, w = R.read_cache(codes, words, which, s.page, s.D, s.group)
        at = [(table[b, p // s.page], p % s.page) for b, n in enumerate(s.lens) for p in range(n)]
        pages, rows = (np.array([x[i] for x in at], dtype=int) for i in (0, 1))
        out += [c[pages, :, rows], w[pages, :, rows]]
    return out


@pytest.mark.parametrize("dtype", DT)
@pytest.mark.parametrize("D,group", FORMS)
@pytest.mark.parametrize("rotate", [True, False])
@pytest.mark.parametrize("page", [16, 64])
def test_append(dtype, D, group, rotate, page):
    s = Setup([37, 0, 1, 130, 16], 3, D, group, page, rotate, DT[dtype], seed=D + group).fill()
    kc, kw, vc, vw = cached(s)
    for x, c, w in ((s.k, kc, kw), (s.v, vc, vw)):
        wc, ww = R.encode(x, group, rotate)
        assert np.array_equal(w, ww) and np.array_equal(c, wc)


@pytest.mark.parametrize("rotate", [True, False])
def test_append_step_by_step(rotate):
    """The same tokens a few at a time: the same cache, and rows that were not
    named as they were."""
    whole = Setup([50, 33, 7], 2, 128, 64, 16, rotate, torch.bfloat16, seed=9).fill()
    parts = Setup([50, 33, 7], 2, 128, 64, 16, rotate, torch.bfloat16, seed=9)
    done, at = [0, 0, 0], starts(whole.lens)
    while done != whole.lens:
        new = [min(n - d, k) for n, d, k in zip(whole.lens, done, (17, 1, 3))]
        rows = torch.cat([torch.arange(at[b] + done[b], at[b] + done[b] + new[b]) for b in range(3)]).cuda()
        done = [d + n for d, n in zip(done, new)]
        crp.kv4_append(parts.k[rows], parts.v[rows], parts.cache, parts.table, ints(done), ints(starts(new)))
    assert torch.equal(parts.cache.codes, whole.cache.codes)
    assert torch.equal(parts.cache.scales, whole.cache.scales)


def test_append_edges():
    """Zero groups, one sign only, the types' largest and smallest values,
    infinities and NaN."""
    for dtype in (torch.bfloat16, torch.float16):
        for rotate in (True, False):
            s = Setup([24], 2, 128, 32, 16, rotate, dtype, seed=1)
            big, tiny = torch.finfo(dtype).max, 2.0 ** -133 if dtype == torch.bfloat16 else 2.0 ** -24
            s.k[0] = 0
            s.k[1] = s.k[1].abs()
            s.k[2] = -s.k[2].abs()
            s.k[3] = big
            s.k[4] = big * torch.sign(s.k[4])
            s.k[5] = tiny * torch.sign(s.k[5])
            s.k[6, 0, 40] = float("nan")
            s.k[7, 1, 70] = float("inf")
            s.k[8, 1, 1] = float("-inf")
            s.k[9] = 0
            s.k[9, :, 5] = 1.0
            s.k[10] *= 2.0 ** -100 if dtype == torch.bfloat16 else 2.0 ** -12
            s.v.copy_(s.k.flip(1))
            s.fill()
            kc, kw, vc, vw = cached(s)
            for x, c, w in ((s.k, kc, kw), (s.v, vc, vw)):
                wc, ww = R.encode(x, 32, rotate)
                assert np.array_equal(w, ww) and np.array_equal(c, wc)


def test_append_leaves_out_rows_without_a_place():
    s = Setup([40, 20], 2, 64, 32, 16, True, torch.bfloat16, seed=2)
    table = s.table.clone()
    table[0, 1], table[1, 0] = -1, 1 << 20
    before = s.cache.codes.clone()
    crp.kv4_append(s.k, s.v, s.cache, table, ints(s.lens), ints(starts(s.lens)))
    torch.cuda.synchronize()
    gone = [int(s.table[0, 1]), int(s.table[1, 0])]
    assert torch.equal(s.cache.codes[gone], before[gone])
    there = [int(s.table[0, 0]), int(s.table[1, 1])]
    assert not torch.equal(s.cache.codes[there], before[there])
    # fewer tokens in the cache than rows: the first rows come before token 0
    s2 = Setup([40], 2, 64, 32, 16, True, torch.bfloat16, seed=2)
    crp.kv4_append(s2.k, s2.v, s2.cache, s2.table, ints([10]), ints([0, 40]))
    want = R.encode(s2.k[30:], 32, True)
    s2.lens = [10]
    kc, kw, _, _ = cached(s2)
    assert np.array_equal(kc, want[0]) and np.array_equal(kw, want[1])


def test_append_views():
    s = Setup([45], 2, 128, 128, 32, True, torch.bfloat16, seed=4).fill()
    fused = torch.cat((torch.zeros_like(s.k), s.k, s.v), 1)
    other = Setup([45], 2, 128, 128, 32, True, torch.bfloat16, seed=4)
    crp.kv4_append(fused[:, 2:4], fused[:, 4:], other.cache, other.table, ints([45]), ints([0, 45]))
    assert torch.equal(other.cache.codes, s.cache.codes) and torch.equal(other.cache.scales, s.cache.scales)
    turned = [t.transpose(0, 1).contiguous().transpose(0, 1) for t in (s.k, s.v)]
    crp.kv4_append(*turned, other.cache, other.table, ints([45]), ints([0, 45]))
    assert torch.equal(other.cache.codes, s.cache.codes)


# ---------------------------------------------------------------------------
# Attention over it
# ---------------------------------------------------------------------------

@pytest.mark.parametrize("dtype", DT)
@pytest.mark.parametrize("D,group", FORMS)
@pytest.mark.parametrize("rotate", [True, False])
@pytest.mark.parametrize("spare", [2, 40])   # tables of up to 1024 tokens, and longer ones: one span, or several
def test_decode_forms(dtype, D, group, rotate, spare):
    s = Setup([37, 1, 600, 64], 2, D, group, 64, rotate, DT[dtype], seed=D + group, spare=spare).fill()
    s.check([1, 1, 1, 1], 6)


@pytest.mark.parametrize("dtype", DT)
@pytest.mark.parametrize("D,group", FORMS)
@pytest.mark.parametrize("rotate", [True, False])
@pytest.mark.parametrize("new,Hq,spare", [([4, 4], 10, 2), ([7, 7], 10, 40), ([30, 2], 6, 40)])
def test_chunk_forms(dtype, D, group, rotate, new, Hq, spare):
    """Several tiles of rows: 20, 35 and 48 rows a key head on average, in
    blocks of one to three tiles."""
    s = Setup([700, 90], 2, D, group, 64, rotate, DT[dtype], seed=D + group, spare=spare).fill()
    s.check(new, Hq)


@pytest.mark.parametrize("H,Hq", [(1, 4), (8, 8), (3, 6)])
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("lens", [[5000, 3, 700, 2600, 1, 0, 513], [257] * 70 + [9000], [1, 2, 3], [20000], [4096] * 9])
def test_spans(H, Hq, D, lens):
    """Ragged contexts in spans over the chip: more and fewer sequences than 64,
    than the blocks that run at once; joined, or whole in tables that are wide."""
    s = Setup(lens, H, D, 64, 128, True, torch.bfloat16, seed=H + D, spare=30).fill()
    s.check([min(1, n) for n in lens], Hq)


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("lens", [[20000, 300, 4000, 2, 900, 6000], [400] * 68 + [9000, 3], [9000] * 4])
def test_uneven_spans(D, lens):
    """Many key heads leave few blocks a head, whose shares are long: uneven
    sequences in spans that follow each other, even ones as they are."""
    H = 64
    s = Setup(lens, H, D, 64, 128, True, torch.bfloat16, seed=D, spare=30)
    few = s.k[:, :2].contiguous(), s.v[:, :2].contiguous()
    s.k, s.v = (x.repeat(1, H // 2, 1) for x in few)
    s.fill()
    new = [1] * len(lens)
    q = s.queries(new, 4)
    got = s.attend(q.repeat(1, H // 2, 1), new)
    s.k, s.v = few
    y, tol = s.reference(q, new)
    assert (np.abs(got[:, :4].double().cpu().numpy() - y) / tol).max() <= 1
    assert torch.equal(got, got[:, :4].repeat(1, H // 2, 1))


def test_two_workspaces_at_once():
    """Two calls on two streams, a workspace each."""
    s = Setup([3000, 100, 1500], 2, 128, 64, 64, True, torch.bfloat16, seed=20).fill()
    t = Setup([2000, 1800], 2, 64, 32, 16, False, torch.float16, seed=21).fill()
    q, p = s.queries([1, 1, 1], 8), t.queries([2, 1], 8)
    args = [(q, s, ints([0, 1, 2, 3])), (p, t, ints([0, 2, 3]))]
    lens = [ints(s.lens), ints(t.lens)]
    want = [crp.attn_kv4(x, c.cache, c.table, n, cu).clone() for (x, c, cu), n in zip(args, lens)]
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    got = [[], []]
    for turn in range(10):
        for i, ((x, c, cu), n) in enumerate(zip(args, lens)):
            with torch.cuda.stream(streams[i]):
                got[i].append(crp.attn_kv4(x, c.cache, c.table, n, cu))
    torch.cuda.synchronize()
    for g, w in zip(got, want):
        assert all(torch.equal(y, w) for y in g)


@pytest.mark.parametrize("n", [1, 2, 15, 16, 17, 31, 33, 63, 64, 65, 127, 128, 129, 255, 256, 257, 511, 512, 513, 1000,
                               1025, 2047, 2049, 4100])
@pytest.mark.parametrize("page", [16, 128])
def test_decode_lengths(n, page):
    s = Setup([n], 1, 128, 64, page, True, torch.bfloat16, seed=n).fill()
    s.check([1], 4)


@pytest.mark.parametrize("Hq,H", [(1, 1), (8, 8), (4, 1), (5, 1), (14, 2), (16, 1), (17, 1), (32, 2), (40, 1)])
@pytest.mark.parametrize("new", [1, 3])
def test_decode_heads(Hq, H, new):
    s = Setup([200, 90], H, 64, 32, 32, True, torch.float16, seed=Hq).fill()
    s.check([new, new], Hq)


@pytest.mark.parametrize("new", [[2, 2], [5, 1], [0, 7], [16, 33], [100, 64], [200, 90]])
@pytest.mark.parametrize("page", [16, 256])
def test_chunks(new, page):
    s = Setup([200, 90], 2, 128, 64, page, True, torch.bfloat16, seed=7).fill()
    s.check(new, 6)


@pytest.mark.parametrize("page", [16, 32, 64, 128, 256, 512, 1024])
def test_pages(page):
    s = Setup([1030, 5, 700], 2, 64, 64, page, False, torch.bfloat16, seed=page).fill()
    s.check([1, 1, 1], 4)


@pytest.mark.parametrize("dtype", DT)
@pytest.mark.parametrize("gain", [0.0, 8.0, 60.0])
def test_flat_and_peaked_weights(dtype, gain):
    s = Setup([777, 2500], 2, 128, 128, 64, True, DT[dtype], seed=3)
    # later keys larger: the maximum moves all the time
    s.k.copy_((s.k.float() * torch.cat([torch.linspace(0.1, 2, n) for n in s.lens]).cuda()[:, None, None]).to(DT[dtype]))
    s.fill().check([1, 2], 4, gain=gain)


@pytest.mark.parametrize("size", [2.0 ** -60, 2.0 ** 60])
def test_values_far_from_one(size):
    s = Setup([300], 2, 128, 64, 64, True, torch.bfloat16, seed=5)
    s.v *= size
    s.k *= size
    s.fill()
    s.check([1], 4, scale=128 ** -0.5 / size)


def test_many_sequences():
    rng = np.random.default_rng(1)
    lens = [int(n) for n in rng.integers(1, 400, size=130)]
    lens[5] = 0
    s = Setup(lens, 2, 64, 32, 16, True, torch.bfloat16, seed=11).fill()
    new = [min(1, n) for n in lens]
    s.check(new, 4)


def test_a_row_that_sees_nothing():
    s = Setup([20, 0], 2, 64, 32, 16, True, torch.bfloat16, seed=12).fill()
    q = s.queries([1, 1], 4)
    y = crp.attn_kv4(q, s.cache, s.table, ints([20, 0]), ints([0, 1, 2]))
    assert (y[1] == 0).all() and y[0].isfinite().all()
    # more rows than tokens: the first rows come before token 0
    q = s.queries([25], 4)
    y = crp.attn_kv4(q, s.cache, s.table[:1], ints([20]), ints([0, 25]))
    assert (y[:5] == 0).all()
    want = crp.attn_kv4(q[5:], s.cache, s.table[:1], ints([20]), ints([0, 20]))
    assert torch.equal(y[5:], want)


def test_pages_that_are_none_hold_nothing():
    """A sequence whose second page is no page: as if its tokens were not there."""
    s = Setup([48], 2, 64, 32, 16, True, torch.bfloat16, seed=13).fill()
    q = s.queries([1], 4)
    for none in (-1, 1 << 20, -(1 << 31)):
        table = s.table.clone()
        table[0, 1] = none
        y = crp.attn_kv4(q, s.cache, table, ints([48]), ints([0, 1]))
        kc, kw = R.encode(s.k, 32, True)
        vc, vw = R.encode(s.v, 32, True)
        rest = np.r_[0:16, 32:48]
        want, tol = R.decode(q, kc[rest], kw[rest], vc[rest], vw[rest], 32, True, [32], 64 ** -0.5, torch.bfloat16)
        assert (np.abs(y.double().cpu().numpy() - want) <= tol).all()
    y = crp.attn_kv4(q, s.cache, torch.full_like(s.table, -1), ints([48]), ints([0, 1]))
    assert (y == 0).all()


def test_a_bad_token_reaches_only_rows_that_see_it():
    for where in "kv":
        s = Setup([200, 100], 2, 128, 64, 16, False, torch.bfloat16, seed=14)
        clean = Setup([200, 100], 2, 128, 64, 16, False, torch.bfloat16, seed=14).fill()
        getattr(s, where)[197, 1, 70] = float("inf")
        s.fill()
        q = s.queries([6, 1], 4)
        y, want = s.attend(q, [6, 1]), clean.attend(q, [6, 1])
        # rows 0..2 of the first sequence are before token 197; heads 0, 1 read the other key head
        assert torch.equal(y[:3], want[:3]) and torch.equal(y[6], want[6]) and torch.equal(y[:, :2], want[:, :2])
        bad = y[3:6, 2:].isnan()
        assert bad.all() if where == "k" else bad[..., 64:].all() and not bad[..., :64].any()


def test_rows_outside_the_sequences():
    s = Setup([30, 44], 2, 128, 64, 16, True, torch.bfloat16, seed=15).fill()
    q = s.queries([9], 4)
    q[:2] = float("nan")
    q[6:] = float("nan")
    out = torch.full_like(q, 7.0)
    y = crp.attn_kv4(q, s.cache, s.table, ints(s.lens), ints([2, 3, 6]), out=out)
    assert y is out and (out[:2] == 7).all() and (out[6:] == 7).all()
    # (bits may differ from a call of other sizes: how rows are tiled goes by T)
    want, tol = s.reference(q[2:6], [1, 3])
    assert (np.abs(out[2:6].double().cpu().numpy() - want) <= tol).all()


def test_a_long_cache():
    """Codes past 4 GiB, and a context over most of it."""
    n, page, H, D = 9000, 1024, 8, 128
    pages = (5 << 30) // (H * page * D)
    cache = crp.kv4_cache(pages, page, H, D, group=128, rotate=True)
    assert cache.codes.numel() > 1 << 32
    order = torch.randperm(pages, generator=torch.Generator().manual_seed(1)).tolist()
    order = [pages - 1] + [p for p in order if p != pages - 1]
    need = -(-n // page)
    s = Setup([n], H, D, 128, page, True, torch.bfloat16, seed=16)
    s.cache, s.table = cache, ints([order[:need]])
    s.fill().check([1], 16)


def test_repeatable_on_other_streams_and_in_graphs():
    """Eager, on another stream, in two graphs that share a workspace (one
    after the other), and with garbage in the workspace: the same bits."""
    s = Setup([3000, 100, 1500], 2, 128, 64, 64, True, torch.bfloat16, seed=17).fill()
    new = [1, 1, 1]
    q = s.queries(new, 8)
    lens, cu = ints(s.lens), ints(starts(new))
    need = crp.attn_kv4_workspace_bytes(3, 8, s.cache, s.table.shape[1], 3)
    ws = torch.full((max(need, 256),), 0xFF, dtype=torch.uint8, device="cuda")
    want = crp.attn_kv4(q, s.cache, s.table, lens, cu).clone()
    assert torch.equal(crp.attn_kv4(q, s.cache, s.table, lens, cu, workspace=ws), want)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        y = crp.attn_kv4(q, s.cache, s.table, lens, cu)
    side.synchronize()
    assert torch.equal(y, want)
    graphs, outs = [], []
    q2 = s.queries(new, 8)
    want2 = crp.attn_kv4(q2, s.cache, s.table, lens, cu).clone()
    for x in (q, q2):
        g, out = torch.cuda.CUDAGraph(), torch.empty_like(q)
        with torch.cuda.graph(g):
            crp.attn_kv4(x, s.cache, s.table, lens, cu, out=out, workspace=ws)
        graphs.append(g)
        outs.append(out)
    for turn in range(3):
        for g, out, w in zip(graphs, outs, (want, want2)):
            out.fill_(0)
            g.replay()
            torch.cuda.synchronize()
            assert torch.equal(out, w)
        assert torch.equal(crp.attn_kv4(q, s.cache, s.table, lens, cu, workspace=ws), want)


def test_a_graph_follows_its_lengths():
    """One captured step, replayed while the sequences grow: lens and table are
    read on the device."""
    s = Setup([300, 40], 2, 64, 32, 16, True, torch.bfloat16, seed=18)
    lens, cu = ints([0, 0]), ints([0, 1, 2])
    k, v = torch.empty((2, 2, 64), dtype=torch.bfloat16, device="cuda"), torch.empty((2, 2, 64), dtype=torch.bfloat16, device="cuda")
    q, out = s.queries([1, 1], 4), torch.empty((2, 4, 64), dtype=torch.bfloat16, device="cuda")
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        crp.kv4_append(k, v, s.cache, s.table, lens, cu)
        crp.attn_kv4(q, s.cache, s.table, lens, cu, out=out)
    for step in range(40):
        n = [step + 1 + 260 * (step == 39), step + 1]
        if step == 39:   # the first sequence gets a prompt of 260 on the way
            crp.kv4_append(s.k[39:299], s.v[39:299], s.cache, s.table[:1], ints([299]), ints([0, 260]))
        for i, b in enumerate((0, 300)):
            k[i], v[i] = s.k[b + n[i] - 1], s.v[b + n[i] - 1]
        lens.copy_(ints(n))
        g.replay()
        want = crp.attn_kv4(q, s.cache, s.table, lens, cu)
        assert torch.equal(out, want)


def test_prompt_then_tokens():
    """A run of the three: a prompt's attention in 16 bits while its keys and
    values go to the cache, then tokens one at a time, between linears."""
    H, Hq, D, width = 2, 8, 64, 256
    gen = torch.Generator().manual_seed(19)
    w = [torch.randn((n, width), generator=gen).mul_(width ** -0.5).to(torch.bfloat16).cuda()
         for n in ((Hq + 2 * H) * D, width)]
    qkv, proj = crp.pack_linear(w[0], w4g=64), None
    proj = crp.pack_linear(torch.randn((width, Hq * D), generator=gen).mul_((Hq * D) ** -0.5).to(torch.bfloat16).cuda(), w4g=64)
    x = torch.randn((90, width), generator=gen).to(torch.bfloat16).cuda()
    cache = crp.kv4_cache(8, 16, H, D, group=32)
    table = ints([[3, 1, 6, 0, 5, 2]])
    n = 83
    parts = crp.linear(x, qkv).view(90, Hq + 2 * H, D).split((Hq, H, H), 1)
    q, k, v = parts
    y = crp.attn_prompt(q[:n], k[:n], v[:n], ints([0, n]))
    crp.kv4_append(k[:n], v[:n], cache, table, ints([n]), ints([0, n]))
    out = crp.linear(y.reshape(n, -1), proj)
    assert out.shape == (n, width) and out.isfinite().all()
    steps = []
    for t in range(n, 90):
        row = slice(t, t + 1)
        crp.kv4_append(k[row], v[row], cache, table, ints([t + 1]), ints([0, 1]))
        steps.append(crp.attn_kv4(q[row], cache, table, ints([t + 1]), ints([0, 1])))
    got = torch.cat(steps)
    # the same rows over the 16-bit keys and values: off by what 4 bits lose
    want = crp.attn_prompt(q, k, v, ints([0, 90]))[n:]
    kc, kw = R.encode(k, 32, True)
    vc, vw = R.encode(v, 32, True)
    ref, tol = R.decode(q[n:], kc, kw, vc, vw, 32, True, np.arange(n + 1, 91), D ** -0.5, torch.bfloat16)
    assert (np.abs(got.double().cpu().numpy() - ref) <= tol).all()
    assert (got.float() - want.float()).norm() < 0.35 * want.float().norm()
    # and all seven at once, as a chunk
    chunk = crp.attn_kv4(q[n:], cache, table, ints([90]), ints([0, 7]))
    assert (np.abs(chunk.double().cpu().numpy() - ref) <= tol).all()
