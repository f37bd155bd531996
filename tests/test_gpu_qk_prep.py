"""Per-head norm with rotation, and its gradients, vs the fp64 plain forms.

Tolerances.  fp32 arithmetic on rotated, normed values u (pair magnitude
P = |u_a| + |u_b|): the angle is off by 2 pi 2^-25 < 2^-22 and sincos by 2^-23,
r by 2^-22, the products by a few 2^-24: together below 2^-20 P.  A bf16
output adds half a step, 2^-8 of the value.
"""

import numpy as np
import pytest
import torch

import oracle.cache_ops as co

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module", autouse=True)
def _lib():
    from programmable_block_sparse_b200 import build
    build.build()


def randn(seed, *shape, dtype=BF):
    g = torch.Generator().manual_seed(seed)
    return torch.randn(shape, generator=g).to(dtype)


def np64(t):
    return t.detach().cpu().double().numpy()


def pair_size(u, rot, interleaved):
    """|u_a| + |u_b| at both places of each pair."""
    p = np.abs(u)
    if rot:
        a, b = co.pairs(rot, interleaved)
        s = p[..., a] + p[..., b]
        p[..., a], p[..., b] = s, s
    return p


def half_step(dtype, ref):
    return 2.0 ** -8 * np.abs(ref) if dtype == BF else 0.0


def inv_freq(rot):
    return (10000.0 ** (-torch.arange(rot // 2, dtype=torch.float64) * 2 / rot)).float()


def check_forward(x, y, norm, weight, pos, f, interleaved):
    kw = dict(norm=norm, weight=None if weight is None else np64(weight))
    ref = co.norm_rope(np64(x), None if f is None else pos.cpu().numpy(), None if f is None else np64(f), interleaved, **kw)
    u = co.norm_rope(np64(x), **kw)
    tol = 2.0 ** -20 * pair_size(u, 0 if f is None else 2 * f.numel(), interleaved) + half_step(y.dtype, ref)
    err = np.abs(np64(y) - ref)
    assert np.all(err <= tol + 1e-30), (err - tol).max()


CASES = [  # B, Hq, Hkv, N, D, rot, interleaved
    (2, 4, 2, 5, 128, 128, False), (1, 8, 1, 1, 128, 128, False), (3, 5, 3, 33, 64, 64, False),
    (2, 3, 1, 7, 80, 80, False), (2, 2, 2, 9, 96, 32, True), (1, 2, 1, 17, 64, 6, True), (2, 3, 2, 6, 20, 20, False),
    (1, 2, 2, 4, 7, 6, False), (1, 1, 1, 3, 1, 0, False), (2, 2, 1, 11, 128, 36, False), (1, 16, 4, 1500, 64, 64, False),
]


@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "fp32"])
@pytest.mark.parametrize("norm", [True, False])
@pytest.mark.parametrize("B,Hq,Hkv,N,D,rot,inter", CASES)
def test_forward(B, Hq, Hkv, N, D, rot, inter, norm, dtype):
    import programmable_block_sparse_b200 as fa
    if not norm and not rot:
        pytest.skip("nothing to do is refused")
    q, k = randn(1, B, Hq, N, D, dtype=dtype).cuda(), randn(2, B, Hkv, N, D, dtype=dtype).cuda()
    qw, kw = (1 + randn(3, D, dtype=F32)).cuda(), (1 + randn(4, D)).cuda()  # fp32 and bf16 weights
    pos = torch.randint(0, 131072, (B, N), generator=torch.Generator().manual_seed(5)).to(torch.int32).cuda()
    f = inv_freq(rot).cuda() if rot else None
    rope = {"inv_freq": f, "interleaved": inter, "pos": pos} if rot else None
    qo, ko = fa.flexattn_qk_norm_rope(q, k, q_norm={"weight": qw} if norm else None,
                                      k_norm={"weight": kw} if norm else None, rope=rope)
    check_forward(q, qo, norm, qw, pos, f, inter)
    check_forward(k, ko, norm, kw, pos, f, inter)


def test_far_positions():
    """Angles of positions near 2^31 keep their precision."""
    import programmable_block_sparse_b200 as fa
    x = randn(1, 1, 2, 4, 64, dtype=F32).cuda()
    pos = torch.tensor([[2 ** 31 - 1, 2 ** 30 + 3, -5, 1 << 24]], dtype=torch.int32).cuda()
    f = inv_freq(64).cuda()
    y, _ = fa.flexattn_qk_norm_rope(x, None, rope={"inv_freq": f, "pos": pos})
    check_forward(x, y, False, None, pos, f, False)


@pytest.mark.parametrize("offset", [0, 1], ids=["aligned", "odd_base"])
def test_strides_types_and_in_place(offset):
    """Slices of a fused projection, odd bases, one side only, an fp32 result
    of bf16 rows, positions that a batch shares, implied positions, outputs in
    place of the inputs; the value part of the projection keeps its bits."""
    import programmable_block_sparse_b200 as fa
    B, N, Hq, Hkv, D = 2, 13, 6, 2, 64
    flat = randn(7, B * N * (Hq + 2 * Hkv) * D + offset).cuda()
    qkv = flat[offset:].view(B, N, Hq + 2 * Hkv, D).transpose(1, 2)
    keep = qkv.clone()
    q, k = qkv[:, :Hq], qkv[:, Hq:Hq + Hkv]
    f = inv_freq(D).cuda()
    pos = torch.arange(40, 40 + N, dtype=torch.int32).cuda()
    w = randn(8, D, dtype=F32).cuda()
    spec = dict(q_norm={"weight": w, "eps": 1e-5}, rope={"inv_freq": f, "pos": pos})
    q32, none = fa.flexattn_qk_norm_rope(q, None, q_out=torch.empty(q.shape, dtype=F32, device="cuda"), **spec)
    assert none is None
    ref = co.norm_rope(np64(q), pos[None].cpu().numpy(), np64(f), norm=True, weight=np64(w), eps=1e-5)
    size = pair_size(co.norm_rope(np64(q), norm=True, weight=np64(w), eps=1e-5), D, False)
    assert np.all(np.abs(np64(q32) - ref) <= 2.0 ** -20 * size)
    _, k1 = fa.flexattn_qk_norm_rope(None, k, rope={"inv_freq": f})  # token n at position n
    check_forward(k, k1, False, None, torch.arange(N)[None], f, False)
    got, _ = fa.flexattn_qk_norm_rope(q, None, q_out=q, **spec)
    assert got is q
    assert np.all(np.abs(np64(q) - ref) <= 2.0 ** -20 * size + half_step(BF, ref))
    assert torch.equal(qkv[:, Hq:], keep[:, Hq:])


def check_backward(x, dy, dx, dw, norm, weight, pos, f, interleaved):
    w = None if weight is None else np64(weight)
    xr, g = np64(x), np64(dy)
    rx, rw = co.norm_rope_backward(xr, g, pos.cpu().numpy(), np64(f), interleaved, norm, w)
    turned = pair_size(g, 2 * f.numel(), interleaved)  # bounds the turned gradient's rounding
    if norm:
        wv = np.ones(xr.shape[-1]) if w is None else np.abs(w)
        r = 1 / np.sqrt((xr * xr).mean(-1, keepdims=True) + 1e-6)
        size = r * (turned * wv + np.abs(xr) * r ** 2 * (turned * wv * np.abs(xr)).mean(-1, keepdims=True))
    else:
        size = turned
    err = np.abs(np64(dx) - rx)
    assert np.all(err <= 2.0 ** -18 * size + half_step(dx.dtype, rx) + 1e-30)
    if norm:
        # terms good to 2^-19, their sum in fp32 over chains of at most 2^6 terms and a tree
        total = (turned * np.abs(xr) * r).sum((0, 1, 2))
        assert np.all(np.abs(np64(dw) - rw) <= (2.0 ** -18 + 2.0 ** -18) * total)
    else:
        assert dw is None


@pytest.mark.parametrize("dtype,gtype", [(BF, BF), (F32, F32), (BF, F32)], ids=["bf16", "fp32", "mixed"])
@pytest.mark.parametrize("norm", [True, False])
@pytest.mark.parametrize("B,Hq,Hkv,N,D,rot,inter", [c for c in CASES if c[5]])
def test_backward(B, Hq, Hkv, N, D, rot, inter, norm, dtype, gtype):
    import programmable_block_sparse_b200 as fa
    q, k = randn(1, B, Hq, N, D, dtype=dtype).cuda(), randn(2, B, Hkv, N, D, dtype=dtype).cuda()
    gq, gk = randn(3, B, Hq, N, D, dtype=gtype).cuda(), randn(4, B, Hkv, N, D, dtype=gtype).cuda()
    qw = (1 + randn(5, D, dtype=F32)).cuda()
    pos = torch.randint(0, 131072, (1, N), generator=torch.Generator().manual_seed(6)).to(torch.int32).cuda()
    f = inv_freq(rot).cuda()
    rope = {"inv_freq": f, "interleaved": inter, "pos": pos}
    args = dict(q_norm={"weight": qw} if norm else None, k_norm={} if norm else None, rope=rope, grad_dtype=dtype)
    dq, dk, dqw, dkw = fa.flexattn_qk_norm_rope_backward(q, k, gq, gk, **args)
    check_backward(q, gq, dq, dqw, norm, qw, pos, f, inter)
    check_backward(k, gk, dk, dkw, norm, None, pos, f, inter)
    again = fa.flexattn_qk_norm_rope_backward(q, k, gq, gk, **args)
    for a, b in zip((dq, dk, dqw, dkw), again):
        assert (a is None and b is None) or torch.equal(a, b), "equal calls give equal bits"


def test_backward_of_shared_and_broadcast_inputs():
    """A key tensor expanded over heads and a broadcast output gradient are
    read through their zero strides; dq may take dq_out's place."""
    import programmable_block_sparse_b200 as fa
    B, H, N, D = 2, 4, 9, 64
    k1 = randn(1, B, 1, N, D, dtype=F32).cuda()
    k, g = k1.expand(B, H, N, D), randn(2, B, H, N, 1, dtype=F32).cuda().expand(B, H, N, D).contiguous()
    g1 = randn(3, 1, 1, N, D, dtype=F32).cuda().expand(B, H, N, D)
    f = inv_freq(D).cuda()
    pos = torch.arange(N, dtype=torch.int32).cuda()[None]
    for dy in (g, g1):
        _, dk, _, dw = fa.flexattn_qk_norm_rope_backward(None, k, None, dy, k_norm={}, rope={"inv_freq": f})
        check_backward(k, dy, dk, dw, True, None, pos, f, False)
    buf = g.clone()
    out = fa.flexattn_qk_norm_rope_backward(k, None, buf, None, dq=buf, q_norm={}, rope={"inv_freq": f},
                                            weight_grads=False)
    assert out[0] is buf and out[2] is None
    check_backward(k, g, buf, fa.flexattn_qk_norm_rope_backward(k, None, g, None, q_norm={}, rope={"inv_freq": f})[2],
                   True, None, pos, f, False)


@pytest.mark.parametrize("N,H,D", [(5, 3, 64), (33, 5, 128), (1, 1, 80)])
def test_backward_without_eps(N, H, D):
    """eps = 0: places that a block of tokens or heads leaves empty add nothing."""
    import programmable_block_sparse_b200 as fa
    x, g = randn(1, 2, H, N, D).cuda(), randn(2, 2, H, N, D).cuda()
    f = inv_freq(D).cuda()
    dx, _, dw, _ = fa.flexattn_qk_norm_rope_backward(x, None, g, None, q_norm={"eps": 0.0}, rope={"inv_freq": f})
    rx, rw = co.norm_rope_backward(np64(x), np64(g), np.arange(N)[None], np64(f), False, True, None, 0.0)
    assert np.linalg.norm(np64(dx) - rx) <= 2.0 ** -8 * np.linalg.norm(rx)
    assert np.linalg.norm(np64(dw) - rw) <= 2.0 ** -17 * np.abs(np64(g) * np64(x)).sum()


def test_gradient_against_differences():
    """Central differences of the kernel's own fp32 forward: a step of 2^-7
    leaves a rounding of 2^-20 / 2^-7 and a third-order term of 2^-14 a value."""
    import programmable_block_sparse_b200 as fa
    q, g = randn(1, 1, 1, 2, 16, dtype=F32).cuda(), randn(2, 1, 1, 2, 16, dtype=F32).cuda()
    w = (1 + randn(3, 16, dtype=F32)).cuda()
    rope = {"inv_freq": inv_freq(16).cuda(), "pos": torch.tensor([3, 70], dtype=torch.int32).cuda()}
    norm = {"weight": w, "eps": 0.5}
    dq, _, dw, _ = fa.flexattn_qk_norm_rope_backward(q, None, g, None, q_norm=norm, rope=rope)

    def loss(x, wt):
        y, _ = fa.flexattn_qk_norm_rope(x, None, q_norm={"weight": wt, "eps": 0.5}, rope=rope)
        return (y.double() * g.double()).sum().item()

    h = 2.0 ** -7
    size = g.abs().sum().item() * 8
    for n, e in [(0, 0), (1, 5), (0, 15)]:
        d = torch.zeros_like(q)
        d[0, 0, n, e] = h
        assert abs((loss(q + d, w) - loss(q - d, w)) / (2 * h) - dq[0, 0, n, e].item()) <= 2.0 ** -12 * size
        dwt = torch.zeros_like(w)
        dwt[e] = h
        assert abs((loss(q, w + dwt) - loss(q, w - dwt)) / (2 * h) - dw[e].item()) <= 2.0 ** -12 * size


def test_infinities_and_nan_stay_in_their_rows():
    import programmable_block_sparse_b200 as fa
    q = randn(1, 1, 2, 6, 64).cuda()
    clean, _ = fa.flexattn_qk_norm_rope(q, None, q_norm={}, rope={"inv_freq": inv_freq(32).cuda()})
    bad = q.clone()
    bad[0, 0, 2, 3], bad[0, 1, 4, 60] = float("inf"), float("nan")
    got, _ = fa.flexattn_qk_norm_rope(bad, None, q_norm={}, rope={"inv_freq": inv_freq(32).cuda()})
    keep = torch.ones(1, 2, 6, dtype=torch.bool)
    keep[0, 0, 2] = keep[0, 1, 4] = False
    assert torch.equal(got[keep.cuda()], clean[keep.cuda()]) and got[0, 1, 4].isnan().all()
    # without a norm the elements past the rotation pass through as they are
    turned, _ = fa.flexattn_qk_norm_rope(bad, None, rope={"inv_freq": inv_freq(32).cuda()})
    assert torch.equal(turned[0, 0, 2, 32:], bad[0, 0, 2, 32:]) and turned[0, 1, 4, 60].isnan()


def test_streams_and_graphs():
    """Another stream, and a captured graph replayed on new inputs, give the
    eager call's bits; two graphs hold workspaces of their own."""
    import programmable_block_sparse_b200 as fa
    B, H, N, D = 1, 4, 40, 128
    rope = {"inv_freq": inv_freq(D).cuda()}
    x, g = randn(1, B, H, N, D).cuda(), randn(2, B, H, N, D).cuda()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        y1, _ = fa.flexattn_qk_norm_rope(x, None, q_norm={}, rope=rope)
    y2, _ = fa.flexattn_qk_norm_rope(x, None, q_norm={}, rope=rope, stream=side)
    side.synchronize()
    y0, _ = fa.flexattn_qk_norm_rope(x, None, q_norm={}, rope=rope)
    assert torch.equal(y0, y1) and torch.equal(y0, y2)
    graphs, outs = [], []
    for _ in range(2):
        gr = torch.cuda.CUDAGraph()
        with torch.cuda.graph(gr):
            outs.append(fa.flexattn_qk_norm_rope_backward(x, None, g, None, q_norm={}, rope=rope))
        graphs.append(gr)
    x.copy_(randn(5, B, H, N, D))
    g.copy_(randn(6, B, H, N, D))
    for gr in graphs:
        gr.replay()
    want = fa.flexattn_qk_norm_rope_backward(x, None, g, None, q_norm={}, rope=rope)
    torch.cuda.synchronize()
    for o in outs:
        assert torch.equal(o[0], want[0]) and torch.equal(o[2], want[2])


def test_many_heads_and_sequences():
    """Grid extents past a block's groups: 300 heads, 700 sequences."""
    import programmable_block_sparse_b200 as fa
    f = inv_freq(64).cuda()
    for B, H, N in [(1, 300, 3), (700, 1, 2)]:
        x = randn(B, B, H, N, 64).cuda()
        y, _ = fa.flexattn_qk_norm_rope(x, None, q_norm={}, rope={"inv_freq": f})
        check_forward(x, y, True, None, torch.arange(N)[None], f, False)
