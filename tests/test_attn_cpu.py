"""Sizes and refusals of the attention calls, and where the 4-bit cache's
kernels go for its pages, whatever their tables say (no GPU needed)."""
import ctypes

import numpy as np
import pytest
import torch

import rotated_bit_quantized_convrot_amd as crp

from . import _attn_ref as R

OK, NULL, SHAPE, GROUP, ALIGN, WORKSPACE, KIND = 0, 1, 2, 3, 4, 5, 8
P, ODD = ctypes.c_void_p(1 << 20), ctypes.c_void_p((1 << 20) + 8)   # never dereferenced
FAR = ctypes.c_void_p(1 << 40)
NAN, INF = float("nan"), float("inf")


@pytest.fixture(scope="module")
def L():
    return crp.lib()


def cache(pages=8, page=64, heads=2, dim=128, group=64, rotate=1, codes=1 << 21, scales=1 << 22):
    return ctypes.byref(crp._Kv4(codes, scales, pages, page, heads, dim, group, rotate))


def test_sizes(L):
    assert L.cr_kv4_codes_bytes(cache()) == 8 * 2 * 2 * 64 * 64
    assert L.cr_kv4_scales_bytes(cache()) == 8 * 2 * 2 * 64 * 2 * 4
    assert L.cr_kv4_codes_bytes(cache(pages=1 << 20, page=1024, heads=8)) == (1 << 20) * 16 * 1024 * 64
    bad = [dict(page=8), dict(page=48), dict(page=2048), dict(page=0), dict(page=-16), dict(pages=0), dict(pages=-1),
           dict(heads=0), dict(heads=1025), dict(dim=96), dict(dim=512), dict(group=16), dict(group=256), dict(group=0),
           dict(dim=64, group=128)]
    for b in bad:
        assert L.cr_kv4_codes_bytes(cache(**b)) == 0 and L.cr_kv4_scales_bytes(cache(**b)) == 0
        assert L.cr_attn_kv4_workspace_bytes(1, 4, cache(**b), 4, 1) == 0
    assert L.cr_kv4_codes_bytes(None) == 0
    ws = L.cr_attn_kv4_workspace_bytes
    assert ws(1, 4, cache(), 4, 1) >= 256
    for T, Hq, width, B in ((-1, 4, 4, 1), (1, 3, 4, 1), (1, 0, 4, 1), (1, 4, 0, 1), (1, 4, 4, -1), (1, 2048, 4, 1),
                            (1, 4, 4, 1 << 17), (1 << 21, 4, 4, 1), (1, 4, 1 << 21, 1)):
        assert ws(T, Hq, cache(), width, B) == 0


def prompt(L, dtype=0, q=P, q_row=512, q_head=128, k=P, k_row=256, k_head=128, v=P, v_row=256, v_head=128, T=10, Hq=4,
           Hkv=2, D=128, cu=P, B=1, causal=1, scale=0.1, y=FAR):
    return L.cr_attn_prompt(dtype, q, q_row, q_head, k, k_row, k_head, v, v_row, v_head, T, Hq, Hkv, D, cu, B, causal,
                            scale, y, None)


def test_prompt_refusals(L):
    for status, cases in {
        KIND: [dict(dtype=2), dict(dtype=-1)],
        SHAPE: [dict(T=-1), dict(T=(1 << 20) + 1), dict(D=96), dict(D=0), dict(Hq=3), dict(Hkv=0), dict(Hq=0),
                dict(Hq=2048, Hkv=1024), dict(B=-1), dict(B=65537), dict(scale=NAN), dict(scale=INF), dict(scale=-INF), dict(scale=2e30), dict(scale=-2e30),
                dict(q_row=1 << 24), dict(k_head=1 << 41),
                dict(y=P), dict(y=ctypes.c_void_p((1 << 20) + 512 * 2 * 9 + 512 * 2 - 16)),
                dict(y=ctypes.c_void_p((1 << 20) - 10 * 512 * 2 + 16))],
        NULL: [dict(q=None), dict(k=None), dict(v=None), dict(cu=None), dict(y=None)],
        ALIGN: [dict(q=ODD), dict(k=ODD), dict(v=ODD), dict(y=ODD), dict(cu=ctypes.c_void_p(1026)), dict(q_row=516),
                dict(k_head=130), dict(v_row=-256), dict(q_head=-128)],
    }.items():
        for c in cases:
            assert prompt(L, **c) == status, c
            assert L.cr_last_error()
    # nothing to do: no pointer is looked at
    assert prompt(L, T=0, q=None, k=None, v=None, cu=None, y=None) == OK
    assert prompt(L, B=0, cu=None) == OK


def append(L, dtype=0, k=P, k_row=256, k_head=128, v=P, v_row=256, v_head=128, T=3, c=None, table=P, width=4, lens=P,
           cu=P, B=1, **kv):
    return L.cr_kv4_append(dtype, k, k_row, k_head, v, v_row, v_head, T, c or cache(**kv), table, width, lens, cu, B, None)


def attend(L, dtype=0, q=P, q_row=512, q_head=128, T=3, Hq=4, c=None, table=P, width=4, lens=P, cu=P, B=1, scale=0.1,
           y=FAR, ws=P, ws_bytes=1 << 30, **kv):
    return L.cr_attn_kv4(dtype, q, q_row, q_head, T, Hq, c or cache(**kv), table, width, lens, cu, B, scale, y, ws,
                         ws_bytes, None)


def test_kv4_refusals(L):
    common = {
        KIND: [dict(dtype=2)],
        SHAPE: [dict(T=-1), dict(B=-1), dict(width=0), dict(width=1 << 21), dict(page=24), dict(dim=96), dict(heads=0),
                dict(pages=0)],
        GROUP: [dict(group=16), dict(group=96), dict(dim=64, group=128)],
        NULL: [dict(table=None), dict(lens=None), dict(cu=None), dict(codes=None), dict(scales=None)],
        ALIGN: [dict(table=ctypes.c_void_p(1025)), dict(lens=ctypes.c_void_p(1025)), dict(cu=ctypes.c_void_p(1025)),
                dict(codes=(1 << 21) + 4), dict(scales=(1 << 22) + 4)],
    }
    for call in (append, attend):
        for status, cases in common.items():
            for c in cases:
                assert call(L, **c) == status, (call, c)
        assert call(L, T=0, table=None, lens=None, cu=None) == OK
        assert call(L, B=0, table=None, lens=None, cu=None) == OK
    for status, cases in {NULL: [dict(k=None), dict(v=None)], ALIGN: [dict(k=ODD), dict(v=ODD), dict(k_row=4), dict(v_head=-8)],
                          SHAPE: [dict(k_row=1 << 24)]}.items():
        for c in cases:
            assert append(L, **c) == status, c
    for status, cases in {NULL: [dict(q=None), dict(y=None), dict(ws=None, width=100)],
                          ALIGN: [dict(q=ODD), dict(y=ODD), dict(ws=ODD), dict(q_row=4), dict(q_head=-8)],
                          SHAPE: [dict(Hq=3), dict(Hq=0), dict(scale=NAN), dict(y=P)],
                          WORKSPACE: [dict(ws_bytes=0, width=100), dict(ws_bytes=256, width=100)]}.items():
        for c in cases:
            assert attend(L, **c) == status, c
    assert L.cr_attn_kv4(0, P, 512, 128, 3, 4, None, P, 4, P, P, 1, 0.1, FAR, P, 1 << 30, None) == NULL


def test_python_refusals():
    q = torch.zeros((4, 4, 64), dtype=torch.bfloat16)
    cu = torch.zeros(2, dtype=torch.int32)
    with pytest.raises(ValueError, match="float32"):
        crp.attn_prompt(q.float(), q, q, cu)
    with pytest.raises(ValueError):   # not on a device
        crp.attn_prompt(q, q, q, cu)
    for kw, status in ((dict(page=24), 2), (dict(dim=80), 2), (dict(group=48), 3), (dict(heads=0), 2)):
        with pytest.raises(crp.ConvRotError) as e:
            crp.kv4_cache(**{**dict(pages=2, page=16, heads=1, dim=64, group=32, device="cpu"), **kw})
        assert e.value.status == status
    with pytest.raises(ValueError):
        crp.kv4_cache(2, 16, 1, 64, group=32, device="cpu")   # no CPU path


# ---------------------------------------------------------------------------
# Where the kernels go
# ---------------------------------------------------------------------------

def places(lens, cu, table, T, pages=5, page=16, heads=3, dim=64, group=32, head=2):
    t = [torch.tensor(x, dtype=torch.int32) for x in (table, lens, cu)]
    return [crp.dbg_kv4_place(pages, page, heads, dim, group, *t, T, row, head) for row in range(T)]


LOW, HIGH = -(1 << 31), (1 << 31) - 1


@pytest.mark.parametrize("seed", range(40))
def test_places_stay_inside(seed):
    """Arrays of any numbers: rows, tokens, pages and offsets stay in range."""
    rng = np.random.default_rng(seed)
    pages, page, heads, dim, group = 5, 16, 3, 64, 32
    B, T, width = 4, 23, 3
    odd = np.array([LOW, HIGH, -1, 0, 1, 5, 15, 16, 17, 22, 23, 24, 47, 48, 49, 1 << 20])
    pick = lambda shape: rng.choice(odd, size=shape).tolist()
    codes, words = pages * 2 * heads * page * dim // 2, pages * 2 * heads * page * dim // group
    for p in places(pick(B), pick(B + 1), pick((B, width)), T, pages, page, heads, dim, group):
        assert -1 <= p["sequence"] < B
        if p["sequence"] < 0:
            continue
        assert p["token"] < p["tokens"] <= width * page
        assert -1 <= p["page"] < pages
        if p["token"] < 0:
            assert p["page"] == -1
        if p["page"] >= 0:
            assert 0 <= p["k_codes"] <= codes - dim // 2
            assert 0 <= p["v_codes"] and p["v_codes"] + 16 * (dim // 2 - 1) < codes
            assert 0 <= p["k_scales"] and p["k_scales"] + dim // group <= words
            assert 0 <= p["v_scales"] and p["v_scales"] + dim // group <= words
        else:
            assert p["k_codes"] == p["v_codes"] == p["k_scales"] == p["v_scales"] == -1


def test_places():
    got = places([20, 0, 33], [1, 4, 4, 6], [[4, 2, -1], [0, 0, 0], [1, 9, 3]], 7)
    assert [p["sequence"] for p in got] == [-1, 0, 0, 0, 2, 2, -1]
    assert [p["token"] for p in got[1:6]] == [17, 18, 19, 31, 32]
    assert [p["page"] for p in got[1:6]] == [2, 2, 2, -1, 3]     # token 31 is on page 9 of 5: none
    p = got[1]
    # page 2, K and V of head 2 of 3, row 1
    assert p["k_codes"] == ((2 * 2 + 0) * 3 + 2) * 16 * 32 + 32 and p["v_codes"] == ((2 * 2 + 1) * 3 + 2) * 16 * 32 + 1
    assert p["k_scales"] == ((2 * 2 + 0) * 3 + 2) * 16 * 2 + 2 and p["v_scales"] == ((2 * 2 + 1) * 3 + 2) * 16 * 2 + 2
    # offsets past 32 bits
    t = [torch.tensor(x, dtype=torch.int32) for x in ([[1 << 19]], [40], [0, 1])]
    p = crp.dbg_kv4_place((1 << 19) + 1, 1024, 8, 128, 64, *t, 1, 0, 7)
    assert p["v_codes"] == (((1 << 19) * 2 + 1) * 8 + 7) * 1024 * 64 + (39 // 16) * 1024 + 39 % 16
    # a table wider than 32 bits of tokens
    t = [torch.zeros((1, 1 << 20), dtype=torch.int32), torch.tensor([HIGH], dtype=torch.int32),
         torch.tensor([0, 1], dtype=torch.int32)]
    p = crp.dbg_kv4_place(1, 1024, 1, 64, 32, *t, 1, 0, 0)
    assert p["tokens"] == 1 << 30 and p["token"] == (1 << 30) - 1 and p["page"] == 0


# ---------------------------------------------------------------------------
# The reference itself
# ---------------------------------------------------------------------------

def test_reference_codes():
    """The rotation is the Hadamard matrix; codes stand for the values to half
    a step, and a planted mistake is seen."""
    rng = np.random.default_rng(0)
    x = torch.from_numpy(rng.normal(size=(7, 2, 128)).astype(np.float32)).to(torch.bfloat16)
    r = R.rotate32(x.float().numpy())
    assert np.allclose(r, x.double().numpy() @ R.hadamard(128), atol=1e-5)
    c, w = R.encode(x, 32, True)
    step = (w & np.uint32(0xFFFFFFF0)).view(np.float32).repeat(32, -1)
    # half a step, and what clamping at a rounded zero point can add to it
    assert (np.abs(R.values(c, w, 32) - r) <= step * 1.001).all()
    assert not np.array_equal(R.encode(x, 32, False)[0], c)


def test_reference_attention():
    """Against torch's softmax in float64, grouped heads, causal."""
    rng = np.random.default_rng(1)
    q, k, v = (torch.from_numpy(rng.normal(size=(9, h, 64))) for h in (4, 2, 2))
    y, tol = R.prompt(q, k, v, [0, 5, 9], True, 0.125, torch.bfloat16)
    for a, b in ((0, 5), (5, 9)):
        for h in range(4):
            s = q[a:b, h] @ k[a:b, h // 2].t() * 0.125
            s = s.masked_fill(torch.ones_like(s).triu(1).bool(), -INF)
            want = torch.softmax(s, -1) @ v[a:b, h // 2]
            assert np.abs(y[a:b, h] - want.numpy()).max() < 1e-12
    # rounding y is inside the bound; weights that are off by a percent are not
    assert (np.abs(torch.from_numpy(y).to(torch.bfloat16).double().numpy() - y) <= tol).all()
    off, _ = R.prompt(q * 1.1, k, v, [0, 5, 9], True, 0.125, torch.bfloat16)
    assert (np.abs(off - y) > tol).any()
