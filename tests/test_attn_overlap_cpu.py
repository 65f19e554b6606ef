"""Outputs of the attention calls that share bytes with an input, or with each
other, are refused (no GPU needed)."""
import ctypes

import pytest

import rotated_bit_quantized_convrot_amd as crp

from .test_attn_cpu import FAR, NULL, P, SHAPE, WORKSPACE, append, attend, cache, prompt

BASE = 1 << 20            # the address that P holds
CODES, SCALES = 1 << 21, 1 << 22
CODE_BYTES, WORD_BYTES = 8 * 2 * 2 * 64 * 64, 8 * 2 * 2 * 64 * 2 * 4   # of the default cache


@pytest.fixture(scope="module")
def L():
    return crp.lib()


def at(address):
    return ctypes.c_void_p(address)


def refused(status, L):
    return status == SHAPE and b"overlap" in L.cr_last_error()


def test_prompt_output_on_cu(L):
    # y: 10 rows of 4 heads of 128, 16-bit
    y = 1 << 30
    for cu in (y, y - 4 * 3, y + 10 * 4 * 128 * 2 - 4):
        assert refused(prompt(L, cu=at(cu), B=3, y=at(y)), L), cu


def test_attend_outputs(L):
    y, n = 1 << 30, 3 * 4 * 128 * 2
    B, width = 2, 5
    for name, size in (("table", 4 * B * width), ("lens", 4 * B), ("cu", 4 * (B + 1))):
        for address in (y, y - size + 4, y + n - 4):
            assert refused(attend(L, B=B, width=width, y=at(y), **{name: at(address)}), L), (name, address)
    for address in (CODES, CODES + CODE_BYTES - 16, CODES - n + 16, SCALES, SCALES + WORD_BYTES - 16, SCALES - n + 16):
        assert refused(attend(L, y=at(address)), L), address
    # beside them: the next refusal is the workspace's
    for address in (CODES + CODE_BYTES, CODES - n, SCALES + WORD_BYTES, SCALES - n):
        assert attend(L, y=at(address), width=100, ws_bytes=0) == WORKSPACE


def test_attend_workspace(L):
    width, B = 100, 2
    need = L.cr_attn_kv4_workspace_bytes(3, 4, cache(), width, B)
    ws, q_bytes = 1 << 30, (2 * 512 + 3 * 128 + 128) * 2
    assert need > 256
    go = lambda **kw: attend(L, **{**dict(ws=at(ws), ws_bytes=need, width=width, B=B), **kw})
    for name, size in (("q", q_bytes), ("y", 3 * 4 * 128 * 2), ("table", 4 * B * width), ("lens", 4 * B), ("cu", 4 * (B + 1)),
                       ("codes", CODE_BYTES), ("scales", WORD_BYTES)):
        step = 16 if name in ("q", "y", "codes", "scales") else 4
        for address in (ws, ws + need - step, ws - size + step):
            assert refused(go(**{name: address if name in ("codes", "scales") else at(address)}), L), (name, address)
    # of a table that needs none, no workspace overlaps anything
    assert attend(L, ws=None, y=None) == NULL


def test_append_outputs(L):
    B, width = 2, 5
    span = (2 * 256 + 128 + 128) * 2
    for out, size in ((CODES, CODE_BYTES), (SCALES, WORD_BYTES)):
        for name, n, step in (("k", span, 16), ("v", span, 16), ("table", 4 * B * width, 4), ("lens", 4 * B, 4), ("cu", 4 * (B + 1), 4)):
            for address in (out, out + size - step, out - n + step):
                assert refused(append(L, B=B, width=width, **{name: at(address)}), L), (name, address)
    for scales in (CODES, CODES + CODE_BYTES - 16, CODES - WORD_BYTES + 16):
        assert refused(append(L, scales=scales), L), scales
