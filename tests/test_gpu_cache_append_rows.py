"""Appends of fp32 rows, and of blocks without a finite value, vs the fp64 plain
form (tolerances: test_gpu_cache_append.py)."""

import numpy as np
import pytest
import torch

import oracle.cache_ops as co
from test_gpu_cache_append import Setup, run_and_check, status
from test_gpu_qk_prep import BF, F32, half_step, inv_freq, np64, pair_size, randn

pytestmark = pytest.mark.gpu
E4 = torch.float8_e4m3fn


@pytest.fixture(scope="module", autouse=True)
def _lib():
    from programmable_block_sparse_b200 import build
    build.build()


def fp32_setup(*args, **kw):
    s = Setup(*args, **kw)
    s.k, s.v = (randn(i, *t.shape, dtype=F32).cuda() for i, t in ((31, s.k), (32, s.v)))
    return s


@pytest.mark.parametrize("pool,block", [(BF, 0), (F32, 0), (E4, 16), (E4, 64), (E4, 128)],
                         ids=["bf16", "fp32", "e4m3_16", "e4m3_64", "e4m3_128"])
@pytest.mark.parametrize("E,Ev,rot,inter", [(128, 128, 128, False), (64, 64, 32, True), (80, 128, 40, False),
                                            (128, 64, 0, False), (13, 7, 6, False)])
@pytest.mark.parametrize("N,start,count", [(1, [0, 5, 127], None), (37, [60, 0, 9], [37, 0, 30])])
def test_fp32_rows(pool, block, E, Ev, rot, inter, N, start, count):
    page = max(block, 16)
    s = fp32_setup(3, 2, N, E, Ev, pool, page, -(-170 // page), block=block, seed=E + N)
    rope = {"inv_freq": inv_freq(rot).cuda(), "interleaved": inter} if rot else None
    run_and_check(s, start, count, k_norm={"weight": (1 + randn(9, E, dtype=F32)).cuda()}, rope=rope)


@pytest.mark.parametrize("D", [64, 128, 20])
def test_fp32_queries_in_the_same_launch(D):
    import programmable_block_sparse_b200 as fa
    N, start = 21, [9, 0]
    s = fp32_setup(2, 2, N, D, D, E4, 32, 2, block=32, seed=D)
    q = randn(11, 2, N, 6, D, dtype=F32).cuda().transpose(1, 2)
    w, f = (1 + randn(12, D)).cuda(), inv_freq(D).cuda()
    pos = np.array(start)[:, None] + np.arange(N)
    ref = co.norm_rope(np64(q), pos, np64(f), norm=True, weight=np64(w))
    size = pair_size(co.norm_rope(np64(q), norm=True, weight=np64(w)), D, False)
    for out in (None, torch.empty(q.shape, dtype=BF, device="cuda")):
        got = fa.flexattn_cache_append(s.k, s.v, s.spec(start), rope={"inv_freq": f}, q=q, q_norm={"weight": w}, q_out=out)
        assert got.dtype == (F32 if out is None else BF)
        assert np.all(np.abs(np64(got) - ref) <= 2.0 ** -20 * size + half_step(got.dtype, ref)) and status() == 0


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
