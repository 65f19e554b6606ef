"""Packed weights with group scales that were packed otherwise than a call
says are refused by their size (no GPU needed)."""
import pytest
import torch

import rotated_bit_quantized_convrot_amd as crp

from .test_w4g_cpu import L, host  # noqa: F401 (fixtures)

FORMS = [(g, z) for g in (32, 64, 128) for z in (False, True)]


def packed(N, K, group, zeros, count=1):
    return torch.zeros(count * crp.w4g_packed_bytes(group, zeros, N, K), dtype=torch.uint8)


@pytest.mark.parametrize("N,K", [(64, 512), (2560, 2560), (9728, 2560)])
@pytest.mark.parametrize("group,zeros", FORMS)
def test_linear_refuses_another_packing(host, N, K, group, zeros):
    x = torch.zeros((2, K), dtype=torch.bfloat16)
    for g, z in FORMS:
        if (g, z) == (group, zeros):   # the one that is right goes on to launch
            with pytest.raises(AssertionError, match="launching"):
                crp.linear_w4g(x, packed(N, K, g, z), N, group, zeros=zeros)
        else:
            with pytest.raises(ValueError, match="packed has"):
                crp.linear_w4g(x, packed(N, K, g, z), N, group, zeros=zeros)
    with pytest.raises(ValueError, match="packed has"):
        crp.linear_w4g(x, packed(N, K, group, zeros, 2), N, group, zeros=zeros)


@pytest.mark.parametrize("at,name", [(0, "gate"), (1, "up"), (2, "down")])
def test_moe_refuses_another_packing(host, at, name):
    E, F, K = 4, 256, 512
    x, r = torch.zeros((3, K), dtype=torch.bfloat16), torch.zeros((E, K), dtype=torch.bfloat16)
    right = [packed(F, K, 64, True, E), packed(F, K, 64, True, E), packed(K, F, 64, True, E)]

    def call(w):
        return crp.moe_w4g(x, r, *w, F, 64, 2, zeros=True, workspace=torch.zeros(1 << 20, dtype=torch.uint8))
    with pytest.raises(AssertionError, match="launching"):
        call(right)
    shape = (K, F) if name == "down" else (F, K)
    for wrong in (packed(*shape, 32, True, E), packed(*shape, 128, True, E), packed(*shape, 64, False, E),
                  packed(*shape, 64, True, E + 1)):
        with pytest.raises(ValueError, match=name + " has"):
            call([wrong if i == at else t for i, t in enumerate(right)])
