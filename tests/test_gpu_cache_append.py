"""Appending to dense and paged caches vs the fp64 plain form.

bf16 and fp32 caches: the tolerances of the preparation (2^-20 of the pair,
plus half a bf16 step).  e4m3: a code stands for its quotient y / s within half
an e4m3 step, plus the fp32 error of the quotient (2^-19 of it); values that
take no arithmetic (v) have to match bit for bit, scales always.
"""

import numpy as np
import pytest
import torch

import oracle.cache_ops as co
from test_gpu_qk_prep import BF, F32, half_step, inv_freq, np64, pair_size, randn

pytestmark = pytest.mark.gpu
E4 = torch.float8_e4m3fn


@pytest.fixture(scope="module", autouse=True)
def _lib():
    from programmable_block_sparse_b200 import build
    build.build()


def status():
    import programmable_block_sparse_b200 as fa
    return fa.flexattn_poll_device_status()


class Setup:
    """A cache with random contents and a page table in shuffled order."""

    def __init__(self, B, Hkv, N, E, Ev, pool, page, pps, block=0, dense=False, seed=0, scale_pow2=True):
        g = torch.Generator().manual_seed(seed)
        self.B, self.H, self.N, self.page, self.block, self.pool = B, Hkv, N, page, block, pool
        outer = B if dense else B * pps + 2
        self.k, self.v = randn(seed + 1, B, Hkv, N, E).cuda(), randn(seed + 2, B, Hkv, N, Ev).cuda()
        if dense:
            self.table = None
            self.rows = [[b] for b in range(B)]
        else:
            self.table = torch.randperm(outer, generator=g)[:B * pps].to(torch.int32).reshape(B, pps)
            self.rows = self.table.tolist()
            self.table = self.table.cuda()
        shape = (outer, Hkv, page)
        if pool == E4:
            self.kp = (torch.randn(shape + (E,), generator=g) * 100).clamp(-448, 448).to(E4).cuda()
            self.vp = (torch.randn(shape + (Ev,), generator=g) * 100).clamp(-448, 448).to(E4).cuda()
            nb = -(-page // block)
            self.ks, self.vs = (torch.ldexp(torch.ones(outer, Hkv, nb), torch.randint(-12, -6, (outer, Hkv, nb), generator=g)).cuda()
                                for _ in range(2))
        else:
            self.kp, self.vp = randn(seed + 3, *shape, E, dtype=pool).cuda(), randn(seed + 4, *shape, Ev, dtype=pool).cuda()
            self.ks = self.vs = None

    def spec(self, start, count=None):
        c = {"k": self.kp, "v": self.vp, "cache_len": torch.tensor(start, dtype=torch.int32).cuda(),
             "page_table": self.table}
        if count is not None:
            c["new_len"] = torch.tensor(count, dtype=torch.int32).cuda()
        if self.pool == E4:
            c.update(k_scale=self.ks, v_scale=self.vs, scale_block=self.block)
        return c


def run_and_check(s, start, count=None, k_norm=None, rope=None):
    import programmable_block_sparse_b200 as fa
    cnt = [s.N] * s.B if count is None else count
    before = {n: None if t is None else t.clone() for n, t in dict(kp=s.kp, vp=s.vp, ks=s.ks, vs=s.vs).items()}
    fa.flexattn_cache_append(s.k, s.v, s.spec(start, count), k_norm=k_norm, rope=rope)
    assert status() == 0
    f = None if rope is None else np64(rope["inv_freq"])
    inter = bool(rope and rope.get("interleaved"))
    for name, new, pool, scale in (("k", s.k, s.kp, s.ks), ("v", s.v, s.vp, s.vs)):
        is_k = name == "k"
        D = new.shape[-1]
        ref = np64(before[name + "p"])
        rscale = None if scale is None else np64(before[name + "s"])
        tol = np.zeros_like(ref)
        for b in range(s.B):
            pos = (np.arange(s.N) + start[b])[None] if rope is None or rope.get("pos") is None else \
                np64(rope["pos"])[b if rope["pos"].shape[0] > 1 else 0][None]
            x = np64(new[b:b + 1])
            kw = dict(norm=is_k and k_norm is not None)
            if kw["norm"]:
                kw.update(weight=None if k_norm.get("weight") is None else np64(k_norm["weight"]), eps=k_norm.get("eps", 1e-6))
            rows = co.norm_rope(x, pos, f if is_k else None, inter, **kw)[0][:, :cnt[b]]
            size = pair_size(co.norm_rope(x, **kw), 2 * f.size if is_k and f is not None else 0, inter)[0][:, :cnt[b]]
            wrote = co.append(rows, ref, rscale, s.block, s.rows[b], s.page, start[b], cnt[b])
            for n in range(cnt[b]):
                j = start[b] + n
                o, at = s.rows[b][j // s.page], j % s.page
                exact = not (is_k and (k_norm is not None or f is not None))
                if scale is None:
                    tol[o, :, at] = half_step(pool.dtype, ref[o, :, at]) + (0 if exact else 2.0 ** -20 * size[:, n])
                elif not exact:
                    q = wrote[j]
                    # compared against the unrounded quotient
                    ref[o, :, at] = np.clip(q, -448, 448)
                    sc = rscale[o, :, at // s.block][:, None]
                    tol[o, :, at] = 0.5 * co.e4m3_step(q) + np.where(sc > 0, 2.0 ** -19 * size[:, n] / np.where(sc > 0, sc, 1), 0)
        got = np64(pool)
        err = np.abs(got - ref)
        assert np.all(err <= tol + 1e-30), (name, (err - tol).max(), np.argwhere(err > tol)[0])
        if scale is not None:
            assert np.array_equal(np64(scale), rscale), name


@pytest.mark.parametrize("pool", [BF, F32], ids=["bf16", "fp32"])
@pytest.mark.parametrize("dense", [False, True], ids=["paged", "dense"])
@pytest.mark.parametrize("N,start,count", [(1, [0, 5, 63], None), (7, [60, 0, 9], [7, 0, 3]), (50, [1, 13, 0], [50, 31, 17])])
def test_plain_pools(pool, dense, N, start, count):
    s = Setup(3, 2, N, 64, 64, pool, 100 if dense else 16, 1 if dense else 7, dense=dense, seed=N)
    run_and_check(s, start, count, k_norm={"weight": (1 + randn(9, 64, dtype=F32)).cuda()},
                  rope={"inv_freq": inv_freq(64).cuda()})


@pytest.mark.parametrize("block,page", [(1, 16), (8, 16), (16, 16), (32, 64), (64, 64), (128, 128), (16, 48)])
@pytest.mark.parametrize("N,start,count", [(1, [0, 5, 127], None), (33, [60, 0, 9], [33, 0, 30]), (150, [1, 100, 64], None)])
def test_e4m3_pools(block, page, N, start, count):
    s = Setup(3, 2, N, 128, 128, E4, page, -(-300 // page), block=block, seed=block + N)
    run_and_check(s, start, count, rope={"inv_freq": inv_freq(128).cuda()})


@pytest.mark.parametrize("E,Ev", [(64, 64), (80, 128), (40, 24), (13, 7), (128, 64)])
@pytest.mark.parametrize("dense", [False, True], ids=["paged", "dense"])
def test_head_dims(E, Ev, dense):
    """Unequal and odd head dims; a dense cache whose length is no multiple of the block."""
    rope = {"inv_freq": inv_freq(E // 4 * 2).cuda(), "interleaved": E == 40,
            "pos": torch.randint(0, 90000, (2, 21), generator=torch.Generator().manual_seed(1)).to(torch.int32).cuda()}
    s = Setup(2, 3, 21, E, Ev, E4, 77 if dense else 32, 1 if dense else 3, block=16, dense=dense, seed=E)
    run_and_check(s, [3, 50], [21, 20], k_norm={"weight": None, "eps": 1e-5}, rope=rope)
    s = Setup(2, 3, 21, E, Ev, BF, 77 if dense else 32, 1 if dense else 3, dense=dense, seed=E)
    run_and_check(s, [3, 50], None, rope=rope)


def test_growth_keeps_and_rescales_older_tokens():
    """Token by token with rising magnitudes: every scale growth re-rounds the
    block's older codes, and nothing else moves."""
    s = Setup(2, 2, 1, 64, 64, E4, 16, 2, block=16, seed=5)
    for step in range(20):
        s.k = randn(100 + step, 2, 2, 1, 64).cuda() * 2.0 ** (step % 7)
        s.v = randn(200 + step, 2, 2, 1, 64).cuda() * 2.0 ** -(step % 5)
        run_and_check(s, [step, step + 7])


def test_zeros_infinities_and_nan():
    """A block of zeros has scale 0; an infinity becomes the largest code, NaN
    stays NaN, and neither moves the scale."""
    import programmable_block_sparse_b200 as fa
    s = Setup(1, 1, 16, 16, 16, E4, 16, 2, block=16, seed=6)
    s.k.zero_()
    s.v[0, 0, 3, 5], s.v[0, 0, 4, 6], s.v[0, 0, 5, 7] = float("inf"), float("-inf"), float("nan")
    fa.flexattn_cache_append(s.k, s.v, s.spec([0]))
    assert status() == 0
    o = s.rows[0][0]
    assert s.ks[o, 0, 0].item() == 0.0 and s.kp[o].float().abs().max().item() == 0.0
    fin = np64(s.v)[np.isfinite(np64(s.v))]
    assert s.vs[o, 0, 0].item() == co.block_scale(np.abs(fin).max())
    v = s.vp[o, 0].float().cpu()
    assert v[3, 5] == 448 and v[4, 6] == -448 and v[5, 7].isnan() and torch.isfinite(v).sum() == v.numel() - 1
    # a token after a block of zeros takes the scale it needs
    s2 = Setup(1, 1, 1, 16, 16, E4, 16, 2, block=16, seed=7)
    s2.kp, s2.ks, s2.table, s2.rows = s.kp, s.ks, s.table, s.rows
    fa.flexattn_cache_append(s2.k[:, :, :1] * 1e-3, s2.v, s2.spec([15]))
    assert s.ks[o, 0, 0].item() == co.block_scale(np.abs(np64(s2.k * 1e-3)).max()) and status() == 0


def test_refused_tokens_write_nothing():
    """Bad pages, full caches and bad lengths: the status word says so, the
    other sequences are appended, and no byte outside the named slots moves."""
    import programmable_block_sparse_b200 as fa
    for what in ("page", "page_negative", "full", "past", "start", "count"):
        s = Setup(2, 2, 8, 64, 64, E4, 16, 2, block=16, seed=8)
        start, count = [10, 4], [8, 8]
        if what.startswith("page"):
            s.table[0, 1] = 10 ** 6 if what == "page" else -1
        if what == "full":
            start[0] = 30  # two slots left
        if what == "past":
            start[0] = 10 ** 9
        if what == "start":
            start[0] = -3
        if what == "count":
            count[0] = 9
        before = s.kp.clone().view(torch.uint8)
        fa.flexattn_cache_append(s.k, s.v, s.spec(start, count))
        assert status() == 9, what
        now = s.kp.view(torch.uint8)
        moved = (now != before).flatten(2).any(-1).any(1).nonzero().flatten().tolist()
        own = {"page": [s.rows[0][0]], "page_negative": [s.rows[0][0]], "full": [s.rows[0][1]], "past": [], "start": [],
               "count": [s.rows[0][0], s.rows[0][1]]}[what]
        assert set(moved) <= set(own + [s.rows[1][0]]) and s.rows[1][0] in moved, what


def test_queries_in_the_same_launch():
    import programmable_block_sparse_b200 as fa
    for N, start in ((1, [9, 0]), (45, [3, 70])):
        s = Setup(2, 2, N, 64, 64, E4, 32, 4, block=32, seed=N)
        q = randn(11, 2, N, 6, 64).cuda().transpose(1, 2)
        w = (1 + randn(12, 64)).cuda()
        f = inv_freq(64).cuda()
        got = fa.flexattn_cache_append(s.k, s.v, s.spec(start, [N, 0]), rope={"inv_freq": f}, q=q, q_norm={"weight": w})
        pos = np.array(start)[:, None] + np.arange(N)
        ref = co.norm_rope(np64(q), pos, np64(f), norm=True, weight=np64(w))
        size = pair_size(co.norm_rope(np64(q), norm=True, weight=np64(w)), 64, False)
        assert np.all(np.abs(np64(got) - ref) <= 2.0 ** -20 * size + half_step(BF, ref)) and status() == 0


def test_strided_pools_streams_and_graphs():
    """Pools stored (pages, slots, heads, D); a captured append replayed at new
    lengths; a side stream."""
    import programmable_block_sparse_b200 as fa
    s = Setup(2, 2, 3, 64, 64, E4, 16, 4, block=16, seed=13)
    kt = s.kp.view(torch.uint8).transpose(1, 2).contiguous().transpose(1, 2).view(E4)
    vt = s.vp.view(torch.uint8).transpose(1, 2).contiguous().transpose(1, 2).view(E4)
    s.kp, s.vp = kt, vt
    assert not s.kp.is_contiguous()
    run_and_check(s, [14, 30], rope={"inv_freq": inv_freq(64).cuda()})
    twin = Setup(2, 2, 3, 64, 64, E4, 16, 4, block=16, seed=13)
    spec = twin.spec([0, 0])
    fa.flexattn_cache_append(twin.k, twin.v, spec)  # first call outside the capture
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        fa.flexattn_cache_append(twin.k, twin.v, spec)
    eager = Setup(2, 2, 3, 64, 64, E4, 16, 4, block=16, seed=13)
    espec = eager.spec([0, 0])
    fa.flexattn_cache_append(eager.k, eager.v, espec)
    side = torch.cuda.Stream()
    for i in range(4):
        for sp in (spec, espec):
            sp["cache_len"].fill_(3 * i + 3)
        graph.replay()
        side.wait_stream(torch.cuda.current_stream())
        fa.flexattn_cache_append(eager.k, eager.v, espec, stream=side)
        torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    assert torch.equal(twin.kp.view(torch.uint8), eager.kp.view(torch.uint8)) and torch.equal(twin.ks, eager.ks)
    assert torch.equal(twin.vp.view(torch.uint8), eager.vp.view(torch.uint8)) and status() == 0


def test_slots_past_four_gigabytes():
    """Offsets of a pool above 2^32 bytes."""
    import programmable_block_sparse_b200 as fa
    pages, H, page, D = 4100, 8, 1024, 128  # 4.3 GB of codes
    kp = torch.zeros((pages, H, page, D), dtype=torch.uint8, device="cuda").view(E4)
    vp = torch.zeros((pages, H, page, D), dtype=torch.uint8, device="cuda").view(E4)
    ks, vs = (torch.zeros((pages, H, page // 64), device="cuda") for _ in range(2))
    k, v = randn(1, 1, H, 5, D).cuda(), randn(2, 1, H, 5, D).cuda()
    table = torch.tensor([[0, 4099]], dtype=torch.int32).cuda()
    fa.flexattn_cache_append(k, v, {"k": kp, "v": vp, "k_scale": ks, "v_scale": vs, "scale_block": 64,
                                    "page_table": table, "cache_len": torch.tensor([2040], dtype=torch.int32).cuda()})
    assert status() == 0
    got = vp[4099, :, 1016:1021].float() * vs[4099, :, 15][:, None, None]
    assert torch.all((got - v[0].float()).abs() <= v[0].float().abs() * 2.0 ** -4 + vs[4099, :, 15][:, None, None] * 2.0 ** -10)
    assert kp.view(torch.uint8)[:4099].max().item() == 0
