"""Appends of blocks without a finite value."""

import numpy as np
import pytest
import torch

import oracle.cache_ops as co
from test_gpu_cache_append import Setup, status
from test_gpu_qk_prep import BF, F32, np64, randn

pytestmark = pytest.mark.gpu
E4 = torch.float8_e4m3fn


@pytest.fixture(scope="module", autouse=True)
def _lib():
    from programmable_block_sparse_b200 import build
    build.build()


@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "fp32"])
@pytest.mark.parametrize("block,E", [(1, 64), (1, 20), (16, 64), (64, 128), (128, 64)])
def test_infinities_without_a_finite_value(block, E, dtype):
    """Such a block has scale 0: zeros stay zeros, an infinity becomes +-448
    times that, NaN stays NaN; and a token after it takes the scale it needs."""
    import programmable_block_sparse_b200 as fa
    page, N = max(block, 16), max(block, 2) - 1
    s = Setup(1, 2, N, E, E, E4, page, 2, block=block, seed=3)
    s.k, s.v = torch.zeros((2, 1, 2, N, E), dtype=dtype, device="cuda")
    s.v[0, 1, 0, 3], s.v[0, 1, 0, 4], s.v[0, 1, 0, 5] = float("inf"), float("-inf"), float("nan")
    fa.flexattn_cache_append(s.k, s.v, s.spec([0]))
    assert status() == 0
    o = s.rows[0][0]
    v = s.vp[o].float()
    assert s.vs[o, :, 0].abs().max().item() == 0.0 and s.ks[o, :, 0].abs().max().item() == 0.0
    assert s.kp[o, :, :N].float().abs().max().item() == 0.0
    assert v[1, 0, 3] == 448 and v[1, 0, 4] == -448 and v[1, 0, 5].isnan()
    v[1, 0, 3:6] = 0
    assert v[:, :N].abs().max().item() == 0.0
    if block > 1:
        s.k, s.v = randn(5, 1, 2, 1, E, dtype=dtype).cuda(), randn(6, 1, 2, 1, E, dtype=dtype).cuda()
        fa.flexattn_cache_append(s.k, s.v, s.spec([N]))
        assert status() == 0
        assert s.vs[o, 1, 0].item() == co.block_scale(np.abs(np64(s.v[0, 1])).max())
        v = s.vp[o, 1, 0].float()
        assert v[5].isnan() and v[[i for i in range(E) if i != 5]].abs().max().item() == 0.0
