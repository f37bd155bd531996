"""Attention over an e4m3 cache vs the fp64 oracle on the restored values.

Tolerance.  With A_i = sum_j p_ij |v_j| (the oracle run on |v|): the softmax
weights are rounded by at most 2^-8 each (decode kernel: two e4m3 terms;
tensor-core prefill: bf16), fp32 scores and sums by less than 2^-12 of each
term, a bf16 output by 2^-8 of the value.  Where the restored cache is rounded
(scales that are no powers of two), keys and values move by 2^-8: a score by
2^-8 sum |q k| scale, a value by 2^-8 of itself.  lse is fp32: 1e-3, the
framework's bound.
"""

import math

import numpy as np
import pytest
import torch

import oracle.flex_oracle as o
import workloads as wl

pytestmark = pytest.mark.gpu
BF, F32, E4 = torch.bfloat16, torch.float32, torch.float8_e4m3fn


@pytest.fixture(scope="module", autouse=True)
def _lib():
    from programmable_block_sparse_b200 import build
    build.build()


class Fp8Case:
    def __init__(self, B, Hq, Hkv, L, S, E, Ev=None, block=16, page=0, kv_len=None, mask=None, score=None, seed=0,
                 pow2=True, qtype=BF, tail_nan=True):
        Ev = Ev or E
        g = torch.Generator().manual_seed(seed)
        self.B, self.Hq, self.Hkv, self.L, self.S, self.block, self.page, self.pow2 = B, Hq, Hkv, L, S, block, page, pow2
        self.q = torch.randn((B, Hq, L, E), generator=g).to(qtype)
        nb = -(-S // block)
        self.kv_len = None if kv_len is None else np.asarray(kv_len, np.int32)
        self.codes, self.scales, self.vals = [], [], []
        for D in (E, Ev):
            c = (torch.randn((B, Hkv, S, D), generator=g) * 120).clamp(-448, 448).to(E4)
            s = torch.ldexp(torch.ones(B, Hkv, nb), torch.randint(-8, -5, (B, Hkv, nb), generator=g))
            if not pow2:
                s = s * (1 + torch.rand(s.shape, generator=g))
            self.codes.append(c)
            self.scales.append(s)
            self.vals.append(c.double().numpy() * s.double().repeat_interleave(block, -1)[..., :S, None].numpy())
        if tail_nan and self.kv_len is not None:  # unused slots: NaN codes and scales
            for c, s in zip(self.codes, self.scales):
                for b, n in enumerate(self.kv_len):
                    c[b, :, n:] = float("nan")
                    s[b, :, -(-int(n) // block):] = float("nan")
            for v in self.vals:
                for b, n in enumerate(self.kv_len):
                    v[b, :, n:] = 0
        self.mask, self.score = dict(mask or {"kind": "causal"}), dict(score or {"kind": "none"})
        self.dev_mask, self.dev_score = dict(self.mask), dict(self.score)
        if self.kv_len is not None:
            self.dev_mask["kv_len"] = torch.from_numpy(self.kv_len).cuda()
        if self.mask["kind"] == "document" or self.score.get("pos") == "in_doc":
            lens = wl.doc_lengths(S, max(1, S // 16), max(2, S // 4), seed)
            ids = wl.doc_ids_from_lengths(lens)
            if self.mask["kind"] == "document":
                self.mask["doc_id"], self.dev_mask["doc_id"] = ids, torch.from_numpy(ids).cuda().reshape(1, S)
            if self.score.get("pos") == "in_doc":
                self.score["doc_id"] = ids
                self.dev_score["pos"] = torch.from_numpy(wl.in_doc_positions(lens)).cuda().reshape(1, S)
        if self.dev_score.get("pos") == "global":
            self.dev_score["pos"] = None
        self.paged = None
        if page:
            self._page(g)
        self.dev = [t.cuda() for t in self.codes]
        self.quant = {"k_scale": self.scales[0].cuda(), "v_scale": self.scales[1].cuda(), "scale_block": block}

    def _page(self, g):
        """The same cache in shuffled pages; entries past the last page in use are -1."""
        B, S, page = self.B, self.S, self.page
        pps = S // page
        ids = torch.randperm(B * pps + 3, generator=g)[:B * pps].reshape(B, pps)
        for i in range(2):
            D = self.codes[i].shape[-1]
            pool = torch.full((B * pps + 3, self.Hkv, page, D), float("nan")).to(E4)
            scale = torch.full((B * pps + 3, self.Hkv, page // self.block), float("nan"))
            c = self.codes[i].view(torch.uint8).reshape(B, self.Hkv, pps, page, D).permute(0, 2, 1, 3, 4)
            pool.view(torch.uint8)[ids.flatten()] = c.reshape(B * pps, self.Hkv, page, D)
            scale[ids.flatten()] = self.scales[i].reshape(B, self.Hkv, pps, -1).permute(0, 2, 1, 3).reshape(
                B * pps, self.Hkv, -1)
            self.codes[i], self.scales[i] = pool, scale
        table = ids.to(torch.int32)
        if self.kv_len is not None:
            for b, n in enumerate(self.kv_len):
                table[b, -(-int(n) // page):] = -1
        self.paged = {"page_table": table.cuda(), "page_size": page}

    def block_mask(self, BM=128, BN=128, heads=1):
        import programmable_block_sparse_b200 as fa
        B = self.B if self.kv_len is not None else 1
        return fa.flexattn_build_block_mask(self.dev_mask, B, heads, self.L, self.S, BM, BN)

    def run(self, bm=None, **kw):
        import programmable_block_sparse_b200 as fa
        kw.setdefault("max_scores", True)
        res = fa.flexattn_forward_fp8(self.q.cuda(), self.dev[0], self.dev[1], bm or self.block_mask(), self.quant,
                                      score_mod=self.dev_score, mask_mod=self.dev_mask, enable_gqa=self.Hq != self.Hkv,
                                      paged=self.paged, **kw)
        torch.cuda.synchronize()
        assert fa.flexattn_poll_device_status() == 0
        return res

    def check(self, res, restored=False):
        scale = float(np.float32(1 / math.sqrt(self.q.shape[-1])))
        q, (k, v) = self.q.double().numpy(), self.vals
        kw = dict(kv_len=self.kv_len, enable_gqa=self.Hq != self.Hkv)
        ro, rl, rm = o.forward(q, k, v, scale, self.mask, self.score, aux=True, **kw)
        A, _ = o.forward(q, k, np.abs(v), scale, self.mask, self.score, **kw)
        out, lse = res[0], res[1]
        fp32 = self.q.dtype == F32
        tol = (2.0 ** -14 if fp32 else 2.0 ** -8 + 2.0 ** -12) * A + 1e-7
        ltol = 1e-3
        if restored and not self.pow2 and not fp32:
            kmax = np.repeat(np.abs(k), self.Hq // self.Hkv, 1)
            move = 2.0 ** -8 * scale * np.einsum("bhle,bhse->bhls", np.abs(q), kmax).max((-1, -2))[..., None, None]
            tol = tol + (2.0 ** -8 + 2 * move) * A
            ltol = ltol + move.max()
        if out.dtype == BF:
            tol = tol + 2.0 ** -8 * np.abs(ro)
        got = out.double().cpu().numpy()
        assert np.isfinite(got).all()
        err = np.abs(got - ro)
        assert np.all(err <= tol), (err.max(), np.argwhere(err > tol)[0].tolist())
        for a, b in ((lse, rl), (res[2] if len(res) > 2 else lse, rm if len(res) > 2 else rl)):
            a = a.double().cpu().numpy()
            fin = np.isfinite(b)
            assert np.array_equal(np.isfinite(a), fin) and np.all(a[~fin] == -np.inf)
            assert not fin.any() or np.abs(a[fin] - b[fin]).max() <= ltol


@pytest.mark.parametrize("split_kv", [0, 3, 1])
@pytest.mark.parametrize("L,Hq,Hkv", [(1, 8, 2), (4, 8, 2), (16, 4, 4), (2, 32, 4), (3, 6, 2), (20, 3, 1), (100, 2, 2)])
@pytest.mark.parametrize("E", [64, 128])
def test_decode_paged(L, Hq, Hkv, E, split_kv):
    c = Fp8Case(4, Hq, Hkv, L, 1536, E, block=16, page=64, kv_len=[1500, 700, 129, 64], score={"kind": "softcap", "cap": 50.0},
                seed=L + E)
    c.check(c.run(split_kv=split_kv))


MASKS = [{"kind": "none"}, {"kind": "sliding_window", "window": 200, "n_sink": 4}, {"kind": "chunked", "chunk": 300},
         {"kind": "prefix_lm", "prefix": 100}, {"kind": "document"}]
SCORES = [{"kind": "none"}, {"kind": "softcap", "cap": 2.0}, {"kind": "alibi"},
          {"kind": "cap_then_bias", "cap": 30.0, "pos": "global"}, {"kind": "cap_then_bias", "cap": 20.0, "pos": "in_doc"}]


@pytest.mark.parametrize("mask", MASKS, ids=lambda m: m["kind"])
@pytest.mark.parametrize("score", SCORES, ids=lambda s: s["kind"] + ("_doc" if s.get("pos") == "in_doc" else ""))
def test_decode_rules(mask, score):
    c = Fp8Case(3, 8, 2, 4, 1000, 128, block=32, kv_len=[1000, 555, 77], mask=mask, score=score, seed=4)
    c.check(c.run(split_kv=4))


@pytest.mark.parametrize("E,Ev", [(16, 16), (48, 96), (80, 80), (112, 64), (128, 16)])
@pytest.mark.parametrize("page,block", [(16, 16), (8, 1), (48, 16), (128, 128), (256, 64), (0, 128)])
def test_decode_dims_and_pages(E, Ev, page, block):
    S = 768
    c = Fp8Case(2, 4, 1, 2, S, E, Ev, block=block, page=page, kv_len=[701, 33], seed=E + page)
    c.check(c.run())


@pytest.mark.parametrize("out_dtype", [BF, F32])
def test_scales_of_any_value(out_dtype):
    """Scales that are no powers of two, a scale of 0, and scales 2^20 apart
    between blocks of values."""
    c = Fp8Case(2, 8, 2, 1, 512, 128, block=16, kv_len=[512, 300], pow2=False, seed=3, tail_nan=False)
    for i in (0, 1):
        c.scales[i][:, :, 3] = 0
        c.scales[i][:, :, 5] *= 2.0 ** (-20 * i)
        c.scales[1][:, :, 7] *= 2.0 ** 5
        c.vals[i] = c.codes[i].double().numpy() * c.scales[i].double().repeat_interleave(16, -1)[..., None].numpy()
    c.quant = {"k_scale": c.scales[0].cuda(), "v_scale": c.scales[1].cuda(), "scale_block": 16}
    c.check(c.run(out_dtype=out_dtype))
    c.check(c.run(out_dtype=out_dtype, split_kv=1))


def test_all_value_scales_zero():
    c = Fp8Case(1, 4, 1, 1, 300, 64, block=128, seed=3)
    c.quant["v_scale"].zero_()
    out, lse, _ = c.run()
    assert out.abs().max().item() < 1e-20 and torch.isfinite(lse).all()


def test_rows_without_keys_and_empty_sequences():
    """kv_len 0, 1 and below L: rows without a key give (0, -inf)."""
    c = Fp8Case(4, 4, 2, 8, 256, 64, page=64, kv_len=[256, 5, 0, 1], seed=6)
    for split in (0, 1, 2):
        out, lse, mx = c.run(split_kv=split)
        assert torch.all(lse[1, :, :3] == -np.inf) and torch.all(out[1, :, :3] == 0)
        assert torch.all(lse[2] == -np.inf) and torch.all(out[2] == 0) and torch.all(mx[2] == -np.inf)
        c.check((out, lse, mx))


def test_head_dependent_rule():
    import programmable_block_sparse_b200 as fa
    rule = fa.and_masks({"kind": "causal"}, fa.or_masks({"kind": "head_below", "value": 3},
                                                        {"kind": "distance_below", "value": 100}))
    for L in (1, 20):
        c = Fp8Case(2, 8, 2, L, 512, 128, kv_len=[512, 200], mask=rule, seed=L)
        c.check(c.run(c.block_mask(heads=8)))


def test_document_rule_with_lists_per_head():
    """Fixed rules may come with per-head lists: the last chunk of 20 rows a
    head is not full, and its empty rows read no document id."""
    c = Fp8Case(2, 4, 2, 20, 384, 64, mask={"kind": "document"}, kv_len=[384, 384], seed=5)
    c.check(c.run(c.block_mask(heads=4)))


@pytest.mark.parametrize("kv_len", [[64, 700, 1500, 129, 700], [(37 * i) % 900 + 40 for i in range(40)]],
                         ids=["ties", "forty_sequences"])
def test_sequence_order(kv_len):
    c = Fp8Case(len(kv_len), 8, 2, 1, 1536, 128, block=64, page=64, kv_len=kv_len, seed=1)
    c.check(c.run())


def test_large_and_tiny_queries():
    """Rows 2^30 apart, values 2^-16 of their row's largest, a row of zeros."""
    c = Fp8Case(1, 8, 1, 1, 400, 128, seed=9)
    c.q[:, 0] *= 2.0 ** -20
    c.q[:, 1] *= 2.0 ** 4
    c.q[:, 2, :, 3:] *= 2.0 ** -16
    c.q[:, 3] = 0
    c.check(c.run())


def test_nan_query_rows_stay_alone():
    c = Fp8Case(1, 4, 1, 2, 300, 64, seed=2)
    clean, lse0, _ = c.run()
    c.q[0, 1, 0, 5], c.q[0, 2, 1, 7] = float("nan"), float("inf")
    out, lse, _ = c.run()
    for h in range(4):
        for i in range(2):
            if (h, i) in ((1, 0), (2, 1)):
                assert out[0, h, i].isnan().all() and lse[0, h, i].isnan()
            else:
                assert torch.equal(out[0, h, i], clean[0, h, i]) and torch.equal(lse[0, h, i], lse0[0, h, i])


@pytest.mark.parametrize("L,Hq,Hkv,E,Ev,page,block,qtype,pow2", [
    (200, 8, 2, 128, 128, 64, 64, BF, True), (130, 4, 4, 64, 64, 0, 128, BF, True), (33, 4, 1, 40, 24, 16, 16, BF, True),
    (5, 4, 2, 64, 64, 48, 16, F32, True), (300, 2, 1, 128, 128, 16, 8, BF, False), (7, 2, 2, 13, 5, 0, 32, F32, False),
    (4, 4, 2, 128, 128, 20, 4, BF, True)])
def test_restored_calls(L, Hq, Hkv, E, Ev, page, block, qtype, pow2):
    """Long or fp32 queries, other head dims and odd pages: the cache is
    restored to the query's type and the forward pass runs on it."""
    S = 720 if page != 64 else 768
    c = Fp8Case(2, Hq, Hkv, L, S, E, Ev, block=block, page=page, kv_len=[S - 9, 150], seed=L, qtype=qtype, pow2=pow2)
    c.check(c.run(), restored=True)


@pytest.mark.parametrize("BM,BN", [(64, 64), (32, 100), (128, 64)])
def test_other_tiles(BM, BN):
    c = Fp8Case(2, 4, 2, 4, 700, 64, block=64, kv_len=[650, 101], seed=BN)
    c.check(c.run(c.block_mask(BM, BN)), restored=True)


def test_strided_pools_and_outputs():
    """Pools stored (pages, slots, heads, D), queries as slices of a projection, an output with gaps."""
    c = Fp8Case(2, 8, 2, 1, 512, 128, block=64, page=64, kv_len=[500, 77], seed=12)
    c.dev = [t.view(torch.uint8).transpose(1, 2).contiguous().transpose(1, 2).view(E4).cuda() for t in c.codes]
    wide = torch.full((2, 8, 1, 256), 7.0, dtype=BF, device="cuda")
    res = c.run(out=wide[..., :128])
    c.check(res)
    assert torch.all(wide[..., 128:] == 7.0)
    # an odd base: not the decode kernel's alignment
    flat = torch.zeros(c.codes[0].numel() + 8, dtype=torch.uint8, device="cuda")
    flat[8:] = c.codes[0].view(torch.uint8).flatten().cuda()
    c.dev[0] = flat[8:].view(c.codes[0].shape).view(E4)
    c.check(c.run(), restored=True)


def test_streams_graphs_and_repeats():
    """A side stream and replays of two graphs with workspaces of their own
    give the eager bits, replays follow the cache and its lengths."""
    import programmable_block_sparse_b200 as fa
    c = Fp8Case(3, 8, 2, 1, 1024, 128, block=64, page=64, kv_len=[1000, 64, 700], seed=20)
    q = c.q.cuda()
    bm = c.block_mask()

    def call(**kw):
        fa.flexattn_build_block_mask(c.dev_mask, 3, 1, 1, 1024, 128, 128, out=bm)
        return fa.flexattn_forward_fp8(q, c.dev[0], c.dev[1], bm, c.quant, mask_mod=c.dev_mask, enable_gqa=True,
                                       paged=c.paged, split_kv=5, **kw)

    want = call()
    again = call()
    assert torch.equal(want[0], again[0]) and torch.equal(want[1], again[1])
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        other = call()
    side.synchronize()
    assert torch.equal(want[0], other[0])
    graphs = []
    for _ in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            res = call()
        graphs.append((g, res))
    c.dev_mask["kv_len"].copy_(torch.tensor([130, 64, 700], dtype=torch.int32))
    want = call()
    want = want[0].clone(), want[1].clone()
    for g, res in graphs:
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(res[0], want[0]) and torch.equal(res[1], want[1])
    assert fa.flexattn_poll_device_status() == 0


def test_two_calls_at_once():
    """Calls on two streams, each with a workspace of its own, do not touch one another."""
    import programmable_block_sparse_b200 as fa
    cases = [Fp8Case(4, 8, 2, 1, 4096, 128, block=64, page=64, kv_len=[4096, 3000, 64, 2000], seed=s) for s in (1, 2)]
    want = [c.run(split_kv=7) for c in cases]
    streams = [torch.cuda.Stream() for _ in cases]
    bms = [c.block_mask() for c in cases]
    qs = [c.q.cuda() for c in cases]
    torch.cuda.synchronize()
    got = [None, None]
    for _ in range(5):
        for i, c in enumerate(cases):
            with torch.cuda.stream(streams[i]):
                got[i] = fa.flexattn_forward_fp8(qs[i], c.dev[0], c.dev[1], bms[i], c.quant, score_mod=c.dev_score,
                                                 mask_mod=c.dev_mask, enable_gqa=True, paged=c.paged, split_kv=7)
    torch.cuda.synchronize()
    for g, w in zip(got, want):
        assert torch.equal(g[0], w[0]) and torch.equal(g[1], w[1])


def test_workspace_of_a_named_stream():
    """A call on a stream that is still busy, its workspace allocated inside:
    work that the current stream is given meanwhile does not get that memory."""
    import programmable_block_sparse_b200 as fa
    c = Fp8Case(4, 8, 2, 1, 4096, 128, block=64, page=64, kv_len=[4096, 3000, 64, 2000], seed=3)
    want = c.run(split_kv=7, max_scores=None)
    bm, q = c.block_mask(), c.q.cuda()
    size = fa.flexattn_forward_fp8_workspace_size(q, c.dev[0], c.dev[1], bm, c.quant, 7, c.paged)
    side = torch.cuda.Stream()

    def call():
        return fa.flexattn_forward_fp8(q, c.dev[0], c.dev[1], bm, c.quant, mask_mod=c.dev_mask, enable_gqa=True,
                                       paged=c.paged, split_kv=7, stream=side)

    # The first allocations reach the driver, which may wait for the device:
    # both streams' pools hold what is needed before the stream is made busy.
    torch.cuda.synchronize()
    kept = [call(), [torch.full((size,), 255, dtype=torch.uint8, device="cuda") for _ in range(8)]]
    torch.cuda.synchronize()
    side_done = torch.cuda.Event()
    side_done.record(side)
    kept.clear()
    with torch.cuda.stream(side):
        torch.cuda._sleep(400_000_000)  # about 0.2 s
    out, lse = call()
    side_done.record(side)
    junk = [torch.full((size,), 255, dtype=torch.uint8, device="cuda") for _ in range(8)]
    busy = not side_done.query()
    torch.cuda.synchronize()
    assert len(junk) == 8 and busy
    assert torch.equal(out, want[0]) and torch.equal(lse, want[1])


def test_threads():
    """Calls from several host threads at once, each on its own stream; a call
    that is refused in between tells its own thread only."""
    from concurrent.futures import ThreadPoolExecutor
    import programmable_block_sparse_b200 as fa
    cases = [Fp8Case(2, 8, 2, 1 + i, 1024, 128, block=64, page=64, kv_len=[1024, 700 + i], seed=20 + i)
             for i in range(4)]
    wants = [c.run(split_kv=0, max_scores=None) for c in cases]
    args = [(c.q.cuda(), c.dev[0], c.dev[1], c.block_mask()) for c in cases]
    streams = [torch.cuda.Stream() for _ in cases]
    torch.cuda.synchronize()

    def work(i):
        q, k, v, bm = args[i]
        outs = []
        for _ in range(20):
            outs.append(fa.flexattn_forward_fp8(q, k, v, bm, cases[i].quant, mask_mod=cases[i].dev_mask,
                                                enable_gqa=True, paged=cases[i].paged, stream=streams[i]))
            with pytest.raises(fa.FlexAttnError):
                fa.flexattn_forward_fp8(q, k, v, bm, cases[i].quant, enable_gqa=True, paged=[], stream=streams[i])
        streams[i].synchronize()
        return outs

    with ThreadPoolExecutor(len(cases)) as pool:
        results = list(pool.map(work, range(len(cases))))
    for want, outs in zip(wants, results):
        assert all(torch.equal(o, want[0]) and torch.equal(l, want[1]) for o, l in outs)


def test_python_refusals():
    """Rule tensors, scales and tables of other types, extents or devices."""
    import programmable_block_sparse_b200 as fa
    c = Fp8Case(2, 4, 2, 1, 256, 64, block=16, page=64, kv_len=[256, 100], seed=1)
    bm = c.block_mask()

    def status(quant=c.quant, mask=c.dev_mask, paged=c.paged, **kw):
        with pytest.raises(fa.FlexAttnError) as e:
            fa.flexattn_forward_fp8(c.q.cuda(), c.dev[0], c.dev[1], bm, quant, mask_mod=mask, enable_gqa=True,
                                    paged=paged, **kw)
        return e.value.status

    assert status(mask=dict(c.dev_mask, kv_len=c.dev_mask["kv_len"].long())) == 6
    assert status(mask=dict(c.dev_mask, kv_len=c.dev_mask["kv_len"][:1])) == 2
    assert status(mask=dict(c.dev_mask, kv_len=c.dev_mask["kv_len"].cpu())) == 9
    assert status(quant=dict(c.quant, k_scale=c.quant["k_scale"][:-1])) == 2
    assert status(quant=dict(c.quant, v_scale=c.quant["v_scale"].double())) == 6
    assert status(quant=dict(c.quant, scale_block=32)) == 2
    assert status(paged=dict(c.paged, page_table=c.paged["page_table"][:1])) == 2
    assert status(paged=dict(c.paged, page_table=c.paged["page_table"].t().contiguous().t())) == 8
    assert status(lse=torch.empty(2, 4, 2, device="cuda")) == 2
    assert status(paged=[c.paged["page_table"]]) == 9
    assert status(split_kv=2, workspace=torch.empty(1 << 20, dtype=torch.uint8)) == 9
    assert status(split_kv=2, workspace=torch.empty((1 << 10, 2), device="cuda")[:, 0]) == 8
    host = fa.BlockMask(**{k: v.cpu() if torch.is_tensor(v) else v for k, v in vars(bm).items()})
    with pytest.raises(fa.FlexAttnError):
        fa.flexattn_forward_fp8(c.q.cuda(), c.dev[0], c.dev[1], host, c.quant, mask_mod=c.dev_mask, enable_gqa=True,
                                paged=c.paged)
    assert status(score_mod={"kind": "cap_then_bias", "cap": 5.0, "pos": torch.zeros(7, dtype=torch.int32).cuda()}) == 2


def test_bad_page_ids_are_reported():
    """An id outside the pool in a page that is in use: nothing outside the
    pool is read and the status word says so, on both paths."""
    import programmable_block_sparse_b200 as fa
    for L in (1, 200):
        c = Fp8Case(1, 2, 1, L, 512, 64, block=64, page=64, kv_len=[500], seed=1)
        c.paged["page_table"][0, 2] = 1 << 30
        fa.flexattn_forward_fp8(c.q.cuda(), c.dev[0], c.dev[1], c.block_mask(), c.quant, mask_mod=c.dev_mask,
                                enable_gqa=True, paged=c.paged)
        torch.cuda.synchronize()
        assert fa.flexattn_poll_device_status() == 9
        assert fa.flexattn_poll_device_status() == 0


def test_wait_budget_runs_out():
    """A tiny wait budget gives a timeout status, and the context stays usable."""
    import programmable_block_sparse_b200 as fa
    c = Fp8Case(2, 8, 2, 1, 4096, 128, block=64, kv_len=[4096, 4000], seed=1)
    bm = c.block_mask()
    fa.flexattn_forward_fp8(c.q.cuda(), c.dev[0], c.dev[1], bm, c.quant, mask_mod=c.dev_mask, enable_gqa=True,
                            wait_cycles=1)
    torch.cuda.synchronize()
    assert fa.flexattn_poll_device_status() in (0, 13)
    c.check(c.run(bm))


def test_long_cache_offsets():
    """A dense cache above 4 GB of codes: the last sequence's keys are read where they are."""
    import programmable_block_sparse_b200 as fa
    B, H, S, D = 3, 8, 1 << 19, 128  # 512 MB a sequence and tensor x 3
    codes = [torch.zeros((B, H, S, D), dtype=torch.uint8, device="cuda").view(E4) for _ in range(2)]
    scales = [torch.ones((B, H, S // 128), device="cuda") for _ in range(2)]
    v1 = torch.randint(0, 100, (H, D), generator=torch.Generator().manual_seed(1), dtype=torch.uint8).cuda()
    codes[1].view(torch.uint8)[2, :, S - 2] = v1
    codes[0].view(torch.uint8)[2, :, S - 2, 0] = 0x7E  # 448: this key takes all the weight
    q = torch.zeros((B, H, 1, D), dtype=BF, device="cuda")
    q[..., 0] = 8
    mask = {"kind": "causal"}
    bm = fa.flexattn_build_block_mask(mask, 1, 1, 1, S, 128, 128)
    out, lse = fa.flexattn_forward_fp8(q, codes[0], codes[1], bm, {"k_scale": scales[0], "v_scale": scales[1],
                                                                    "scale_block": 128}, mask_mod=mask)
    assert torch.equal(out[2, :, 0].float(), v1.view(E4).float()) and out[:2].abs().max().item() == 0
    assert fa.flexattn_poll_device_status() == 0
