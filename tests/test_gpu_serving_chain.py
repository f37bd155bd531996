"""The operators together, as a user runs them: a training step (norm and
rotation, attention, their gradients) and serving (a prompt appended in
chunks, then single tokens, each attending over the e4m3 cache)."""

import math

import numpy as np
import pytest
import torch

import oracle.cache_ops as co
import oracle.flex_oracle as o
from test_gpu_qk_prep import BF, F32, inv_freq, np64, randn

pytestmark = pytest.mark.gpu
E4 = torch.float8_e4m3fn


@pytest.fixture(scope="module", autouse=True)
def _lib():
    from programmable_block_sparse_b200 import build
    build.build()


def test_training_step():
    """Gradients of sum(attention(prep(x)) * dout) for x, against the fp64
    chain; the intermediate tensors are those the kernels stored."""
    import programmable_block_sparse_b200 as fa
    B, Hq, Hkv, N, D = 1, 4, 2, 256, 64
    qkv = randn(1, B, N, Hq + 2 * Hkv, D).cuda().transpose(1, 2)
    q, k, v = qkv[:, :Hq], qkv[:, Hq:Hq + Hkv], qkv[:, Hq + Hkv:]
    qw, kw = (1 + 0.1 * randn(2, D, dtype=F32)).cuda(), (1 + 0.1 * randn(3, D, dtype=F32)).cuda()
    f = inv_freq(D).cuda()
    spec = dict(q_norm={"weight": qw}, k_norm={"weight": kw}, rope={"inv_freq": f})
    mask = {"kind": "causal"}
    bm = fa.flexattn_build_block_mask(mask, 1, 1, N, N)
    qr, kr = fa.flexattn_qk_norm_rope(q, k, **spec)
    out, lse = fa.flexattn_forward(qr, kr, v, bm, mask_mod=mask, enable_gqa=True)
    dout = randn(4, B, Hq, N, D).cuda()
    dqr, dkr, dv = fa.flexattn_backward(qr, kr, v, out, dout, lse, bm, mask_mod=mask, enable_gqa=True, grad_dtype=F32)
    dq, dk, dqw, dkw = fa.flexattn_qk_norm_rope_backward(q, k, dqr, dkr, grad_dtype=BF, **spec)
    assert fa.flexattn_poll_device_status() == 0
    pos = np.arange(N)[None]
    kwq = dict(pos=pos, inv_freq=np64(f), norm=True)
    scale = float(np.float32(1 / math.sqrt(D)))
    gq, gk, gv = o.backward(np64(qr), np64(kr), np64(v), np64(dout), scale, mask, {"kind": "none"}, enable_gqa=True,
                            out=np64(out))
    for x, g, got, gw, w in ((q, gq, dq, dqw, qw), (k, gk, dk, dkw, kw)):
        rx, rw = co.norm_rope_backward(np64(x), g, weight=np64(w), **kwq)
        # the attention gradients carry bf16 products (2^-8 of their terms); what
        # follows is linear in them, so errors stay at that share of the norm
        for a, b in ((np64(got), rx), (np64(gw), rw)):
            assert np.linalg.norm(a - b) <= 2.0 ** -6 * np.linalg.norm(b)


@pytest.mark.parametrize("page,block", [(64, 64), (16, 16)])
def test_prompt_then_tokens(page, block):
    import programmable_block_sparse_b200 as fa
    B, Hq, Hkv, D, prompt, steps, chunk = 2, 8, 2, 128, 300, 6, 150
    pps = -(-(prompt + steps) // page)
    total = prompt + steps
    x = randn(1, B, total, Hq + 2 * Hkv, D).cuda().transpose(1, 2)
    f, kw = inv_freq(D).cuda(), (1 + 0.1 * randn(2, D, dtype=F32)).cuda()
    norm, rope = {"weight": kw}, {"inv_freq": f}
    table = torch.randperm(B * pps, generator=torch.Generator().manual_seed(3)).to(torch.int32).reshape(B, pps).cuda()
    pools = [torch.full((B * pps, Hkv, page, D), 0x7F, dtype=torch.uint8, device="cuda").view(E4) for _ in range(2)]
    scales = [torch.full((B * pps, Hkv, page // block), float("nan"), device="cuda") for _ in range(2)]
    lens = torch.zeros(B, dtype=torch.int32, device="cuda")
    cache = {"k": pools[0], "v": pools[1], "k_scale": scales[0], "v_scale": scales[1], "scale_block": block,
             "page_table": table, "cache_len": lens}
    quant = {"k_scale": scales[0], "v_scale": scales[1], "scale_block": block}
    paged = {"page_table": table, "page_size": page}
    S = pps * page
    at = 0
    for n in [chunk, chunk] + [1] * steps:
        sl = x[:, :, at:at + n]
        q = fa.flexattn_cache_append(sl[:, Hq:Hq + Hkv], sl[:, Hq + Hkv:], cache, k_norm=norm, rope=rope, q=sl[:, :Hq],
                                     q_norm=norm)
        lens.add_(n)
        at += n
        mask = {"kind": "causal", "kv_len": lens}
        bm = fa.flexattn_build_block_mask(mask, B, 1, n, S)
        out, lse = fa.flexattn_forward_fp8(q, pools[0], pools[1], bm, quant, mask_mod=mask, enable_gqa=True, paged=paged)
        torch.cuda.synchronize()
        assert fa.flexattn_poll_device_status() == 0
        # the cache holds the normed, turned keys and the values within e4m3's rounding (older
        # codes of a block may have been rounded again, by half a step of the larger scale)
        dense = []
        for pool, sc in zip(pools, scales):
            t = table.long()
            d = pool.float()[t] * sc[t].repeat_interleave(block, -1)[..., None]
            dense.append(np64(d.permute(0, 2, 1, 3, 4).flatten(2, 3)[:, :, :at]))
        kref = co.norm_rope(np64(x[:, Hq:Hq + Hkv, :at]), np.arange(at)[None], np64(f), norm=True, weight=np64(kw))
        vref = np64(x[:, Hq + Hkv:, :at])
        for got, ref in ((dense[0], kref), (dense[1], vref)):
            assert np.all(np.abs(got - ref) <= 2 * 2.0 ** -4 * np.abs(ref) + 2.0 ** -9 * np.abs(ref).max((-1, -2), keepdims=True))
        # and attention is over what the cache holds
        scale = float(np.float32(1 / math.sqrt(D)))
        ro, rl = o.forward(np64(q), dense[0], dense[1], scale, {"kind": "causal"}, {"kind": "none"}, enable_gqa=True)
        A, _ = o.forward(np64(q), dense[0], np.abs(dense[1]), scale, {"kind": "causal"}, {"kind": "none"}, enable_gqa=True)
        assert np.all(np.abs(np64(out) - ro) <= (2.0 ** -8 + 2.0 ** -12) * A + 2.0 ** -8 * np.abs(ro) + 1e-6)
        assert np.abs(np64(lse) - rl).max() <= 1e-3
