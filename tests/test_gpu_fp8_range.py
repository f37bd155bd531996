"""Attention over an e4m3 cache where its numbers lie far apart: keys that take
most of the weight, value scales far from one another, far positions, lists that
reach past a sequence's end.

Tolerances are those of test_gpu_fp8.py: with A_i = sum_j p_ij |v_j|, 2^-8 + 2^-12
of A_i for out (a weight is good to 2^-8 of itself while it is above 2^-27 of its
row's largest, and to 2^-34 of that one below: 2^-14 of A over 2^20 such keys),
half a bf16 step of the result, and 1e-3 for lse and max_scores.
"""

import numpy as np
import pytest
import torch

from test_gpu_fp8 import BF, E4, F32, Fp8Case

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    from programmable_block_sparse_b200 import build
    build.build()


def finish(c, page=0, seed=0):
    """The case's values, pools and device tensors after its codes or scales were changed."""
    for i in range(2):
        s = c.scales[i].double().repeat_interleave(c.block, -1)[..., :c.S, None]
        c.vals[i] = c.codes[i].double().numpy() * s.numpy()
        if c.kv_len is not None:
            for b, n in enumerate(c.kv_len):
                c.vals[i][b, :, n:] = 0
    if page:
        c.page = page
        c._page(torch.Generator().manual_seed(seed))
    c.dev = [t.cuda() for t in c.codes]
    c.quant = {"k_scale": c.scales[0].cuda(), "v_scale": c.scales[1].cuda(), "scale_block": c.block}
    return c


def sink_case(L, S, code, tail, page=0, E=128, B=1, seed=0):
    """The first key's score is (64 / sqrt(E)) * code * 2^-7 for every query, its
    value 0; the other keys' scores are N(0, 0.9) or all 0, their values 0.5 on
    average."""
    c = Fp8Case(B, 8, 2, L, S, E, block=64, seed=seed)
    g = torch.Generator().manual_seed(seed + 1)
    c.q[..., 0] = 64
    k = c.codes[0].float()
    if tail == "equal":
        k.zero_()
    k[..., 0] = 0
    k[:, :, 0] = 0
    k[:, :, 0, 0] = code
    v = torch.randn(c.codes[1].shape, generator=g) * 60 + 60
    v[:, :, 0] = 0
    c.codes = [k.clamp(-448, 448).to(E4), v.clamp(-448, 448).to(E4)]
    c.scales = [torch.full_like(s, 2.0 ** -7) for s in c.scales]
    return finish(c, page, seed)


@pytest.mark.parametrize("split_kv", [1, 0])
@pytest.mark.parametrize("page", [0, 64])
@pytest.mark.parametrize("L", [1, 2, 4, 20])  # 4, 8, 16 rows a group of heads, five chunks of 16
@pytest.mark.parametrize("code", [224, 288, 320, 352])  # 9.9, 12.7, 14.1 and 15.6 nats
def test_many_keys_far_below_a_sink(code, L, page, split_kv):
    c = sink_case(L, 8192, code, "normal", page)
    c.check(c.run(split_kv=split_kv, out_dtype=F32))


@pytest.mark.parametrize("L,S", [(1, 65536), (4, 32768)])
@pytest.mark.parametrize("code", [192, 256, 288])
def test_equal_keys_far_below_a_sink(code, L, S):
    """Equal weights are rounded alike, so their errors add up."""
    c = sink_case(L, S, code, "equal", E=64)  # 12, 16 and 18 nats
    c.check(c.run(split_kv=1, out_dtype=F32))


@pytest.mark.parametrize("log2", [10, 16, -16])
@pytest.mark.parametrize("L", [1, 4])
def test_one_block_of_values_far_from_the_others(L, log2):
    """A block whose value scale is far from the others', its values in one channel."""
    c = Fp8Case(2, 8, 2, L, 4096, 128, block=64, kv_len=[4096, 3000], seed=L, tail_nan=False)
    v = c.codes[1].float()
    v[:, :, 320:384] = 0
    v[:, :, 320:384, 3] = 100
    c.codes[1] = v.to(E4)
    c.scales[1][:, :, 5] = 2.0 ** (log2 - 7)
    finish(c)
    for split in (1, 0):
        c.check(c.run(split_kv=split, out_dtype=F32))


@pytest.mark.parametrize("L", [1, 4])
def test_blocks_of_scale_zero_beside_large_scales(L):
    """Keys whose values are nothing keep their share of the softmax, a sixth,
    beside a value scale of 2^20: 4032 of them 10 nats below the first."""
    c = sink_case(L, 4096, 224, "equal")
    c.scales[1][:, :, 0] = 2.0 ** 20
    c.scales[1][:, :, 1:] = 0
    v = c.codes[1].float()
    v[:, :, 0] = 100
    c.codes[1] = v.to(E4)
    finish(c)
    c.check(c.run(split_kv=1, out_dtype=F32))


@pytest.mark.parametrize("L", [1, 2, 4])
def test_scales_of_zero_over_many_keys(L):
    """All values nothing: out is 0 and lse finite, however many keys."""
    c = Fp8Case(1, 8, 2, L, 1 << 17, 64, block=128, seed=L)
    c.codes[0].view(torch.uint8).zero_()
    c.scales[1].zero_()
    finish(c)
    out, lse, _ = c.run(split_kv=1)
    assert out.abs().max().item() < 1e-20
    want = np.log((1 << 17) - (L - 1) + np.arange(L))
    assert np.abs(lse.double().cpu().numpy() - want).max() <= 1e-3


@pytest.mark.parametrize("L", [1, 2, 4])
def test_distance_bias_at_far_positions(L):
    """lse and max_scores of a distance bias over 2^19 keys: the bias is taken
    from the distance, so that the size of the positions does not matter."""
    S = 1 << 19
    c = Fp8Case(1, 8, 1, L, S, 16, block=64, score={"kind": "alibi"}, seed=L)
    out, lse, mx = c.run()
    q, (k, v) = c.q.double().numpy(), c.vals
    near = 1 << 15  # slopes of 2^-8 and more: e^-128 beyond
    sub = Fp8Case.__new__(Fp8Case)
    sub.__dict__.update(c.__dict__)
    sub.S, sub.vals = near, [x[:, :, -near:] for x in c.vals]
    sub.check((out, lse, mx))


@pytest.mark.parametrize("split_kv", [2, 5])
def test_explicit_splits_of_more_rows(split_kv):
    """More than one split is a request for the decode kernel, at every batch."""
    for B, L in ((1, 48), (8, 48), (8, 100)):
        c = Fp8Case(B, 16, 4, L, 640, 64, block=64, page=64, kv_len=[640 - 9 * b for b in range(B)], seed=L + B)
        c.check(c.run(split_kv=split_kv))


@pytest.mark.parametrize("L,qtype,E,BN", [(5, F32, 64, 128), (40, BF, 40, 128), (300, BF, 128, 128), (300, F32, 24, 100),
                                          (3, BF, 64, 64)])
@pytest.mark.parametrize("page", [0, 20])
def test_lists_that_reach_past_the_end(L, qtype, E, BN, page):
    """Lists made for the whole capacity and used at shorter lengths, over a
    workspace of NaN: what lies past kv_len is not read as a number."""
    import programmable_block_sparse_b200 as fa
    S = 1000
    c = Fp8Case(2, 4, 2, L, S, E, block=4 if page else 16, kv_len=[S, S], qtype=qtype, seed=E, tail_nan=False,
                mask={"kind": "none"})
    bm = c.block_mask(128, BN)
    short = Fp8Case(2, 4, 2, L, S, E, block=4 if page else 16, page=page, kv_len=[410, 33], qtype=qtype, seed=E,
                    mask={"kind": "none"})
    n = fa.flexattn_forward_fp8_workspace_size(short.q.cuda(), short.dev[0], short.dev[1], bm, short.quant,
                                               paged=short.paged)
    ws = torch.full((max(n, 1),), 255, dtype=torch.uint8, device="cuda")
    short.check(short.run(bm, workspace=ws), restored=True)


@pytest.mark.parametrize("L", [1, 4])
def test_wait_budget_does_run_out(L):
    """A budget of one cycle gives up in every part of the kernel (one and two
    sets of softmax warps), and the next call is as good as ever."""
    import programmable_block_sparse_b200 as fa
    c = Fp8Case(2, 8, 2, L, 4096, 128, block=64, kv_len=[4096, 4000], seed=1)
    bm = c.block_mask()
    fa.flexattn_forward_fp8(c.q.cuda(), c.dev[0], c.dev[1], bm, c.quant, mask_mod=c.dev_mask, enable_gqa=True,
                            wait_cycles=1)
    torch.cuda.synchronize()
    assert fa.flexattn_poll_device_status() == 13
    c.check(c.run(bm))


@pytest.mark.parametrize("L,BM", [(48, 48), (100, 112)])
def test_smaller_query_tiles_of_many_rows(L, BM):
    c = Fp8Case(8, 16, 4, L, 640, 64, block=64, page=64, kv_len=[640 - 9 * b for b in range(8)], seed=L)
    c.check(c.run(c.block_mask(BM)))
