"""GPU: the mixture of experts holds its hidden values in float32 (_moe_h_ref.py)."""
import numpy as np
import pytest
import torch

import rotated_bit_quantized_convrot_amd as crp

from . import _moe_h_ref as H
from . import _w4g_ref as R
from .test_gpu_moe import layer, run

pytestmark = pytest.mark.gpu
DT = {"bf16": torch.bfloat16, "fp16": torch.float16}


@pytest.mark.parametrize("dtype", DT)
@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("zeros", [False, True])
@pytest.mark.parametrize("M,K,F,E", [(1, 128, 256, 2), (5, 256, 128, 3), (16, 128, 384, 2), (33, 256, 128, 8),
                                     (20, 4224, 128, 2), (64, 4224, 256, 2), (67, 128, 128, 5)])
def test_differences_of_hidden_values(dtype, group, zeros, M, K, F, E):
    pick = [(m * m + m // 3) % E for m in range(M)]
    x, r, gate, up, down, p = H.cancelling(M, K, F, E, group, DT[dtype], zeros, pick)
    y, ids, c = run(x, r, gate, up, down, 1, True, routing=True)
    assert ids.cpu()[:, 0].tolist() == pick and (c == 1).all()
    want, tol = H.expected(x, K, F, p)
    off = np.abs(y.cpu().double().numpy() - want) / tol
    assert off.max() <= 1, (off.max(), np.unravel_index(off.argmax(), off.shape))


@pytest.mark.parametrize("dtype", DT)
@pytest.mark.parametrize("zeros", [False, True])
@pytest.mark.parametrize("M,K,F,E,topk,group", [(1, 2048, 768, 16, 8, 128), (16, 1024, 512, 32, 4, 64),
                                                (5, 1376, 1408, 8, 4, 32), (64, 512, 256, 60, 8, 128),
                                                (64, 4096, 640, 4, 2, 64), (130, 512, 512, 6, 2, 32)])
def test_error_is_the_rounding_of_y(dtype, zeros, M, K, F, E, topk, group):
    args = layer(M, K, F, E, group, DT[dtype], zeros, seed=M)
    y = run(*args, topk, True)
    want = R.moe(*args, topk, True)[0]
    assert np.linalg.norm(y.cpu().double().numpy() - want) <= H.norm_limit(want, DT[dtype])
