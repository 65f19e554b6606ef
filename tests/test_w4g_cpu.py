"""Sizes and refusals of the calls on 4-bit weights with group scales: every
one is detected before a launch (no GPU needed)."""
import ctypes

import pytest
import torch

import rotated_bit_quantized_convrot_amd as crp

OK, NULL, SHAPE, GROUP, ALIGN, WORKSPACE, KIND = 0, 1, 2, 3, 4, 5, 8
P, ODD = ctypes.c_void_p(256), ctypes.c_void_p(264)   # never dereferenced


@pytest.fixture(scope="module")
def L():
    return crp.lib()


def test_packed_bytes(L):
    # 16-row, 128-k tiles: codes, 16-bit scales, zero points, in 256-byte blocks
    assert L.cr_w4g_packed_bytes(128, 0, 2560, 2560) == 2560 * 2560 // 2 + 2560 * 20 * 2
    assert L.cr_w4g_packed_bytes(32, 0, 64, 256) == 64 * 128 + 64 * 8 * 2
    assert L.cr_w4g_packed_bytes(32, 1, 64, 256) == 64 * 128 + 64 * 8 * 2 + 64 * 8 // 2
    assert L.cr_w4g_packed_bytes(64, 1, 64, 256) == -(-(64 * 128 + 64 * 4 * 2 + 64 * 4 // 2) // 256) * 256
    # one row, a quarter of a unit: padded to a whole tile
    assert L.cr_w4g_packed_bytes(32, 0, 1, 32) == 1024 + 256
    for g, N, K in ((16, 64, 256), (256, 64, 256), (0, 64, 256), (128, 64, 192), (32, 64, 40), (32, 0, 32),
                    (32, 16, 0), (32, (1 << 20) + 1, 32), (-32, 64, 64)):
        assert L.cr_w4g_packed_bytes(g, 0, N, K) == 0


def test_generic_calls_refuse_the_kind(L):
    assert crp.W4G == 7
    assert L.cr_packed_bytes(crp.W4G, 256, 256) == 0
    assert L.cr_quantize_activations(crp.W4G, P, 4, 256, P, 1 << 20, None) == KIND


def test_encode_and_pack_refusals(L):
    enc, pack = L.cr_encode_w4g, L.cr_pack_weight_w4g
    assert enc(2, P, 64, 256, 128, P, P, None, None) == KIND
    assert enc(0, P, 64, 200, 128, P, P, None, None) == GROUP
    assert enc(0, P, 64, 256, 96, P, P, None, None) == GROUP
    assert enc(0, P, 0, 256, 128, P, P, None, None) == SHAPE
    assert enc(0, P, 1 << 20, 1 << 15, 128, P, P, None, None) == SHAPE      # 2^35 weights
    assert enc(0, None, 64, 256, 128, P, P, None, None) == NULL
    assert enc(0, P, 64, 256, 128, None, P, None, None) == NULL
    assert enc(0, P, 64, 256, 128, P, None, None, None) == NULL
    assert enc(0, ODD, 64, 256, 128, P, P, None, None) == ALIGN
    assert enc(0, P, 64, 256, 128, P, P, ODD, None) == ALIGN
    assert pack(P, P, None, 0, 64, 256, 128, P, None) == SHAPE
    assert pack(P, P, None, 1 << 20, 1 << 10, 1 << 10, 128, P, None) == SHAPE
    assert pack(P, P, None, 1, 64, 256, 48, P, None) == GROUP
    assert pack(P, None, None, 1, 64, 256, 128, P, None) == NULL
    assert pack(P, P, None, 1, 64, 256, 128, None, None) == NULL
    assert pack(P, P, ODD, 1, 64, 256, 128, P, None) == ALIGN


def test_linear_refusals(L):
    lin = L.cr_linear_w4g
    assert lin(2, P, 4, 256, P, 128, 0, 64, None, P, None) == KIND
    assert lin(0, P, -1, 256, P, 128, 0, 64, None, P, None) == SHAPE
    assert lin(0, P, (1 << 20) + 1, 256, P, 128, 0, 64, None, P, None) == SHAPE
    assert lin(0, P, 4, 256, P, 128, 0, 0, None, P, None) == SHAPE
    assert lin(0, P, 4, 160, P, 64, 0, 64, None, P, None) == GROUP
    assert b"160" in L.cr_last_error()
    assert lin(0, P, 4, 256, None, 128, 0, 64, None, P, None) == NULL
    assert lin(0, None, 4, 256, P, 128, 0, 64, None, P, None) == NULL
    assert lin(0, P, 4, 256, P, 128, 0, 64, None, None, None) == NULL
    for at in (1, 4, 8, 9):   # x, weight, bias, y
        args = [0, P, 4, 256, P, 128, 0, 64, P, P, None]
        args[at] = ODD
        assert lin(*args) == ALIGN
    assert lin(0, None, 0, 256, P, 128, 0, 64, None, None, None) == OK


def test_outputs_over_their_inputs_are_refused(L):
    def at(a):
        return ctypes.c_void_p(a)
    # x is 4 x 256 and y 4 x 64 elements of 2 bytes
    for y in (4096, 4096 + 2032, 4096 - 496):
        assert L.cr_linear_w4g(0, at(4096), 4, 256, P, 128, 0, 64, None, at(y), None) == SHAPE
        assert b"overlaps" in L.cr_last_error()
    # a mixture of experts may write its rows over x, but over no others
    need = L.cr_moe_w4g_workspace_bytes(4, 256, 128, 8, 2, 128)
    for y in (4096 + 512, 4096 - 2032):
        assert L.cr_moe_w4g(0, at(4096), 4, 256, P, 8, 2, 1, P, P, P, 128, 128, 0, at(y), None, None, P, need,
                            None) == SHAPE
    # next to each other they may lie: the next check's turn
    for y in (4096 + 2048, 4096, 4096 - 2048):
        assert L.cr_moe_w4g(0, at(4096), 4, 256, P, 8, 2, 1, P, P, P, 128, 128, 0, at(y), None, None, P, need - 1,
                            None) == WORKSPACE


def test_pack_linear_refuses_mixed_formats(host):
    w = torch.zeros((64, 256), dtype=torch.bfloat16)
    for k in (dict(int8=True), dict(regular=True), dict(group=64)):
        with pytest.raises(ValueError, match="of its own"):
            crp.pack_linear(w, w4g=64, **k)
    with pytest.raises(ValueError, match="zeros needs"):
        crp.pack_linear(w, zeros=True)


def test_moe_refusals(L):
    need = L.cr_moe_w4g_workspace_bytes(4, 256, 128, 8, 2, 128)
    good = dict(dtype=0, x=P, M=4, K=256, router=P, E=8, topk=2, norm=1, wg=P, wu=P, wd=P, F=128, group=128, zeros=0,
                y=P, ids=None, weights=None, ws=P, ws_bytes=need, stream=None)

    def call(**k):
        return L.cr_moe_w4g(*{**good, **k}.values())

    assert need >= 4 * 8 * 8 + 4 * 2 * 128 * 2
    assert call(dtype=3) == KIND
    assert call(M=-1) == SHAPE
    assert call(E=0) == SHAPE and call(E=1025) == SHAPE
    assert call(topk=0) == SHAPE and call(topk=9) == SHAPE and call(E=64, topk=17) == SHAPE
    assert call(K=200) == GROUP and call(F=100) == GROUP and call(group=256) == GROUP
    assert call(K=65536 + 128) == SHAPE and call(F=65536 + 128) == SHAPE
    for k in ("router", "wg", "wu", "wd", "x", "y", "ws"):
        assert call(**{k: None}) == NULL, k
    for k in ("router", "wg", "wu", "wd", "x", "y", "ws", "ids", "weights"):
        assert call(**{k: ODD}) == ALIGN, k
    assert call(ws_bytes=need - 1) == WORKSPACE
    assert call(M=0, x=None, y=None, ws=None, ws_bytes=0) == OK
    for bad in ((4, 256, 128, 8, 9, 128), (4, 256, 100, 8, 2, 128), (-1, 256, 128, 8, 2, 128)):
        assert L.cr_moe_w4g_workspace_bytes(*bad) == 0
    # a long batch goes in passes over one pass's workspace
    assert L.cr_moe_w4g_workspace_bytes(1000, 256, 128, 8, 2, 128) == L.cr_moe_w4g_workspace_bytes(64, 256, 128, 8, 2, 128)


def test_host_tensors_and_types_are_refused():
    x = torch.zeros((4, 256), dtype=torch.bfloat16)
    u8 = torch.zeros(1 << 16, dtype=torch.uint8)
    with pytest.raises(ValueError, match="device tensor"):
        crp.encode_w4g(x)
    with pytest.raises(ValueError, match="device tensor"):
        crp.linear_w4g(x, u8, 16, 128)
    with pytest.raises(ValueError, match="device tensor"):
        crp.moe_w4g(x, x, u8, u8, u8, 128, 128, 1)
    with pytest.raises(ValueError, match="bfloat16 or"):
        crp.encode_w4g(x.float())
    with pytest.raises(ValueError, match="bfloat16 or"):
        crp.linear_w4g(x.float(), u8, 16, 128)


@pytest.fixture
def host(monkeypatch, L):
    """The binding with its device check off, so that its shape checks run on
    host tensors; a call that would launch fails the test."""
    def host_ok(t, name, dtype=None):
        if dtype is not None and t.dtype != dtype:
            raise ValueError(f"{name} must be {dtype}")

    def no_launch(*a, **k):
        raise AssertionError("a launching call was reached")
    monkeypatch.setattr(crp, "_dev", host_ok)
    monkeypatch.setattr(crp, "_call_on", no_launch)


def test_binding_shape_checks(host):
    b = torch.bfloat16
    w = torch.zeros((64, 256), dtype=b)
    for g in (16, 96, 256):
        with pytest.raises(crp.ConvRotError, match="group"):
            crp.encode_w4g(w, g)
    with pytest.raises(crp.ConvRotError, match="group"):
        crp.encode_w4g(torch.zeros((64, 200), dtype=b), 128)
    codes, s = torch.zeros((64, 128), dtype=torch.uint8), torch.ones((64, 2), dtype=b)
    with pytest.raises(ValueError, match="leading dimension"):
        crp.pack_weight_w4g(codes, s[:32])
    with pytest.raises(ValueError, match="shape of scales"):
        crp.pack_weight_w4g(codes, s, torch.zeros((64, 4), dtype=torch.uint8))
    with pytest.raises(crp.ConvRotError):
        crp.pack_weight_w4g(codes, torch.ones((64, 16), dtype=b))          # groups of 16
    with pytest.raises(crp.ConvRotError):
        crp.pack_weight_w4g(codes, torch.ones((64, 0), dtype=b))
    x = torch.zeros((4, 256), dtype=b)
    packed = torch.zeros(crp.w4g_packed_bytes(128, False, 64, 256), dtype=torch.uint8)
    with pytest.raises(ValueError, match="packed has"):
        crp.linear_w4g(x, packed[:-256], 64, 128)
    with pytest.raises(ValueError, match="packed has"):
        crp.linear_w4g(x, packed, 64, 128, zeros=True)
    with pytest.raises(ValueError, match="bias must have N"):
        crp.linear_w4g(x, packed, 64, 128, bias=torch.zeros(63, dtype=b))
    with pytest.raises(ValueError, match="bias must be"):
        crp.linear_w4g(x, packed, 64, 128, bias=torch.zeros(64))
    with pytest.raises(ValueError, match="out must be"):
        crp.linear_w4g(x, packed, 64, 128, out=torch.zeros((4, 63), dtype=b))
    with pytest.raises(ValueError, match="x must be"):
        crp.linear_w4g(x[0], packed, 64, 128)
    pw = crp.PackedWeight(crp.W4G, 64, 256, packed, None, w4g=128, dtype=torch.float16)
    with pytest.raises(ValueError, match="type of the weight's scales"):
        crp.linear(x, pw)


def test_moe_binding_shape_checks(host):
    b = torch.bfloat16
    E, F, K = 4, 128, 256
    x, r = torch.zeros((3, K), dtype=b), torch.zeros((E, K), dtype=b)
    up = torch.zeros(E * crp.w4g_packed_bytes(128, False, F, K), dtype=torch.uint8)
    down = torch.zeros(E * crp.w4g_packed_bytes(128, False, K, F), dtype=torch.uint8)
    with pytest.raises(ValueError, match="gate has"):
        crp.moe_w4g(x, r, up[:-256], up, down, F, 128, 2)
    with pytest.raises(ValueError, match="down has"):
        crp.moe_w4g(x, r, up, up, down[:-256], F, 128, 2)
    with pytest.raises(ValueError, match="router"):
        crp.moe_w4g(x, r[:, :128], up, up, down, F, 128, 2)
    with pytest.raises(ValueError, match="router must be"):
        crp.moe_w4g(x, r.half(), up, up, down, F, 128, 2)
    with pytest.raises(ValueError, match="out must be"):
        crp.moe_w4g(x, r, up, up, down, F, 128, 2, out=torch.zeros((4, K), dtype=b))
    pe = crp.PackedExperts(E, K, F, 128, False, torch.float16, up, up, down)
    with pytest.raises(ValueError, match="experts' scales"):
        crp.moe(x, r, pe, 2)
    with pytest.raises(ValueError, match="router must be"):
        crp.moe(x.half(), r.half()[:3], pe, 2)
    with pytest.raises(ValueError, match="gate and up"):
        crp.pack_experts(torch.zeros((E, F, K), dtype=b), torch.zeros((E, F, K), dtype=b),
                         torch.zeros((E, F, K), dtype=b))
