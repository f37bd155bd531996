"""Refusals of the preparation, cache and 8-bit attention entry points: host
checks that return before any CUDA work (no GPU needed)."""

import ctypes as C

import pytest
import torch

import programmable_block_sparse_b200 as fa
from programmable_block_sparse_b200 import _abi
from test_abi_cpu import FAKE, _bm, _t

BF, F32, E4 = _abi.FA_DTYPE_BF16, _abi.FA_DTYPE_F32, _abi.FA_DTYPE_E4M3
NULL, SHAPE, HEADS, BATCH, MASK_SHAPE, DTYPE, HEADDIM, ALIGN, PARAM, WORKSPACE = 1, 2, 3, 4, 5, 6, 7, 8, 9, 10


@pytest.fixture(scope="module")
def lib():
    from programmable_block_sparse_b200 import build
    build.build()
    return fa.load_library()


def ref(s):
    return None if s is None else C.byref(s)


def norm(weight=FAKE, dtype=F32, eps=1e-6):
    return _abi.fa_head_norm(weight, dtype, eps)


def rope(inv=FAKE, pos=None, rot=64, inter=0, pos_batch=0, reserved=0):
    return _abi.fa_rope(inv, pos, rot, inter, pos_batch, reserved)


def prep(lib, q=None, k=None, qo=None, ko=None, qn=None, kn=None, rp=None):
    return lib.flexattn_qk_norm_rope(ref(q), ref(k), ref(qo), ref(ko), ref(qn), ref(kn), ref(rp), None)


def test_struct_sizes():
    assert C.sizeof(_abi.fa_head_norm) == 16
    assert C.sizeof(_abi.fa_rope) == 32
    assert C.sizeof(_abi.fa_kv_quant) == 24
    assert C.sizeof(_abi.fa_kv_cache) == 2 * 80 + 5 * 8 + 8


def test_prep_refusals(lib):
    q, k = _t(2, 4, 7, 64), _t(2, 2, 7, 64)
    n, r = norm(), rope()
    assert prep(lib, rp=r) == NULL
    assert prep(lib, q=q, qo=q) == NULL                                   # nothing to do
    assert prep(lib, q=q, rp=r) == NULL                                   # no output
    assert prep(lib, q=q, qo=_t(2, 4, 8, 64), rp=r) == SHAPE
    assert prep(lib, q=q, qo=q, k=_t(2, 2, 8, 64), ko=_t(2, 2, 8, 64), rp=r) == SHAPE
    assert prep(lib, q=q, qo=q, k=_t(3, 2, 7, 64), ko=_t(3, 2, 7, 64), rp=r) == BATCH
    assert prep(lib, q=q, qo=q, k=_t(2, 2, 7, 32), ko=_t(2, 2, 7, 32), rp=r) == SHAPE
    assert prep(lib, q=_t(2, 4, 7, 136), qo=_t(2, 4, 7, 136), rp=r) == HEADDIM
    assert prep(lib, q=_t(2, 4, 7, 64, dtype=E4), qo=q, rp=r) == DTYPE
    assert prep(lib, q=_t(2, 4, 7, 64, addr=0), qo=q, rp=r) == NULL
    assert prep(lib, q=_t(70000, 1, 1, 64), qo=_t(70000, 1, 1, 64), rp=r) == SHAPE
    # an output with two elements in one place
    assert prep(lib, q=q, qo=_t(2, 4, 7, 64, stride=(0, 448, 64, 1)), rp=r) == ALIGN
    for bad in (dict(rot=0), dict(rot=3), dict(rot=66), dict(inter=2), dict(reserved=1)):
        assert prep(lib, q=q, qo=q, rp=rope(**bad)) == PARAM, bad
    assert prep(lib, q=q, qo=q, rp=rope(inv=None)) == NULL
    assert prep(lib, q=q, qo=q, rp=rope(pos=FAKE, pos_batch=3)) == BATCH
    assert prep(lib, q=q, qo=q, rp=rope(pos=FAKE + 2, pos_batch=2)) == ALIGN
    for eps in (-1.0, float("nan"), float("inf")):
        assert prep(lib, q=q, qo=q, qn=norm(eps=eps)) == PARAM
    assert prep(lib, q=q, qo=q, qn=norm(dtype=E4)) == DTYPE
    assert prep(lib, q=q, qo=q, qn=norm(weight=FAKE + 1, dtype=BF)) == ALIGN


def bwd(lib, q=None, k=None, gq=None, gk=None, oq=None, ok=None, wq=None, wk=None, qn=None, kn=None, rp=None, ws=FAKE,
        n=1 << 30):
    return lib.flexattn_qk_norm_rope_backward(ref(q), ref(k), ref(gq), ref(gk), ref(oq), ref(ok), wq, wk, ref(qn),
                                              ref(kn), ref(rp), ws, n, None)


def test_prep_backward_refusals(lib):
    q, nq, r = _t(2, 4, 7, 64), norm(), rope()
    assert bwd(lib, rp=r) == NULL
    assert bwd(lib, gq=q, oq=q) == NULL
    assert bwd(lib, gq=q, rp=r) == NULL
    assert bwd(lib, gq=q, oq=q, qn=nq) == NULL                             # the norm's input
    assert bwd(lib, q=_t(2, 4, 6, 64), gq=q, oq=q, qn=nq) == SHAPE
    assert bwd(lib, gq=q, oq=q, rp=r, wq=FAKE) == PARAM                    # a weight gradient without a norm
    assert bwd(lib, q=q, gq=q, oq=q, qn=nq, wk=FAKE) == PARAM
    assert bwd(lib, q=q, gq=q, oq=q, qn=nq, wq=FAKE, ws=None, n=0) == WORKSPACE
    assert bwd(lib, q=q, gq=q, oq=q, qn=nq, wq=FAKE, n=16) == WORKSPACE
    assert bwd(lib, q=q, gq=q, oq=q, qn=nq, wq=FAKE, ws=FAKE + 4) == ALIGN
    assert bwd(lib, q=q, gq=q, oq=q, qn=nq, wq=FAKE + 2) == ALIGN
    assert bwd(lib, q=q, gq=q, oq=_t(2, 4, 7, 64, stride=(1792, 0, 64, 1)), qn=nq) == ALIGN
    n = C.c_size_t(7)
    size = lib.flexattn_qk_norm_rope_backward_workspace_size
    assert size(64, 1, C.byref(n)) == 0 and n.value > 0
    assert size(64, 0, C.byref(n)) == 0 and n.value == 0
    assert size(64, 1, None) == NULL and size(0, 1, C.byref(n)) == SHAPE and size(200, 1, C.byref(n)) == HEADDIM


def cache(kp, vp, table=FAKE, pps=4, lens=FAKE, ks=None, vs=None, block=0):
    c = _abi.fa_kv_cache()
    c.k, c.v = kp, vp
    c.page_table, c.pages_per_seq, c.cache_len = table, pps, lens
    c.k_scale, c.v_scale, c.scale_block = ks, vs, block
    return c


def app(lib, k, v, c, q=None, qo=None, kn=None, qn=None, rp=None):
    return lib.flexattn_cache_append(ref(k), ref(v), ref(c), ref(kn), ref(rp), ref(q), ref(qo), ref(qn), None)


def test_append_refusals(lib):
    k, v = _t(2, 2, 5, 64), _t(2, 2, 5, 64)
    pool, codes = _t(9, 2, 16, 64), _t(9, 2, 16, 64, dtype=E4)
    assert app(lib, k, v, None) == NULL
    assert app(lib, k, None, cache(pool, pool)) == NULL
    assert app(lib, k, _t(3, 2, 5, 64), cache(pool, pool)) == BATCH
    assert app(lib, k, _t(2, 2, 6, 64), cache(pool, pool)) == SHAPE
    assert app(lib, _t(2, 2, 5, 136), v, cache(pool, pool)) == HEADDIM
    assert app(lib, k, v, cache(pool, codes)) == DTYPE
    assert app(lib, k, v, cache(_t(9, 4, 16, 64), pool)) == HEADS
    assert app(lib, k, v, cache(_t(9, 2, 16, 32), pool)) == SHAPE
    assert app(lib, k, v, cache(_t(8, 2, 16, 64), pool)) == SHAPE
    assert app(lib, k, v, cache(pool, pool, lens=None)) == NULL
    assert app(lib, k, v, cache(pool, pool, pps=0)) == PARAM
    assert app(lib, k, v, cache(pool, pool, pps=1 << 28)) == SHAPE
    assert app(lib, k, v, cache(pool, pool, table=None)) == BATCH          # a dense cache of 9 sequences
    assert app(lib, k, v, cache(pool, pool, ks=FAKE)) == PARAM             # scales without codes
    assert app(lib, k, v, cache(_t(9, 2, 16, 64, stride=(0, 1024, 64, 1)), pool)) == ALIGN
    assert app(lib, k, v, cache(codes, codes, block=16)) == NULL           # codes without scales
    for block, want in ((0, PARAM), (3, PARAM), (256, PARAM), (32, PARAM)):
        assert app(lib, k, v, cache(codes, codes, ks=FAKE, vs=FAKE, block=block)) == want
    assert app(lib, k, v, cache(codes, codes, ks=FAKE + 2, vs=FAKE, block=16)) == ALIGN
    assert app(lib, k, v, cache(pool, pool), q=_t(2, 4, 5, 64)) == NULL
    assert app(lib, k, v, cache(pool, pool), q=_t(2, 4, 4, 64), qo=_t(2, 4, 4, 64)) == SHAPE
    assert app(lib, k, v, cache(pool, pool), q=_t(1, 4, 5, 64), qo=_t(1, 4, 5, 64)) == BATCH
    assert app(lib, k, v, cache(pool, pool), rp=rope(rot=66)) == PARAM
    assert app(lib, k, v, cache(pool, pool), kn=norm(eps=-1)) == PARAM
    big = _t(1, 40000, 1, 64)
    assert app(lib, big, big, cache(_t(9, 40000, 16, 64), _t(9, 40000, 16, 64))) == SHAPE


def fp8(lib, q, k, v, o, bm, quant="default", opts=None, gqa=1, split=0, mask=None, score=None, ws=FAKE, n=1 << 40):
    if quant == "default":
        quant = _abi.fa_kv_quant(FAKE, FAKE, 16, 0)
    score = score or _abi.fa_score_mod(kind=0)
    mask = mask or _abi.fa_mask_mod(kind=1)
    return lib.flexattn_forward_fp8(ref(q), ref(k), ref(v), ref(quant), ref(o), None, 0.0, gqa, C.byref(score),
                                    C.byref(mask), C.byref(bm), split, ref(opts), ws, n, None)


def test_forward_fp8_refusals(lib):
    q, o = _t(2, 4, 1, 64), _t(2, 4, 1, 64)
    k = _t(2, 2, 256, 64, dtype=E4)
    bm = _bm(2, 1, 1, 256, 128, 128)
    assert fp8(lib, q, k, k, None, bm) == NULL
    assert fp8(lib, q, _t(2, 2, 256, 64), k, o, bm) == DTYPE
    assert fp8(lib, _t(2, 4, 1, 64, dtype=E4), k, k, o, bm) == DTYPE
    assert fp8(lib, q, k, k, o, bm, quant=None) == NULL
    assert fp8(lib, q, k, k, o, bm, quant=_abi.fa_kv_quant(None, FAKE, 16, 0)) == NULL
    assert fp8(lib, q, k, k, o, bm, quant=_abi.fa_kv_quant(FAKE, FAKE, 16, 1)) == PARAM
    assert fp8(lib, q, k, k, o, bm, quant=_abi.fa_kv_quant(FAKE, FAKE, 12, 0)) == PARAM
    assert fp8(lib, q, k, k, o, bm, quant=_abi.fa_kv_quant(FAKE + 1, FAKE, 16, 0)) == ALIGN
    assert fp8(lib, q, k, k, o, bm, gqa=0) == HEADS
    assert fp8(lib, q, _t(3, 2, 256, 64, dtype=E4), k, o, bm) == BATCH
    assert fp8(lib, q, k, k, o, _bm(2, 1, 1, 255, 128, 128)) == MASK_SHAPE
    assert fp8(lib, q, k, k, o, bm, split=-1) == PARAM
    assert fp8(lib, q, k, k, o, bm, mask=_abi.fa_mask_mod(kind=2, window=0)) == PARAM
    assert fp8(lib, q, k, k, o, bm, score=_abi.fa_score_mod(kind=1, cap=-1.0)) == PARAM
    assert fp8(lib, q, k, k, _t(2, 4, 1, 64, stride=(0, 64, 64, 1)), bm) == ALIGN
    assert fp8(lib, q, k, k, o, bm, split=2, ws=None, n=0) == WORKSPACE
    assert fp8(lib, q, k, k, o, bm, split=2, ws=FAKE + 8) == ALIGN
    # a call that restores the cache needs its workspace too
    long_q, long_o = _t(2, 4, 256, 64), _t(2, 4, 256, 64)
    assert fp8(lib, long_q, k, k, long_o, _bm(2, 1, 256, 256, 128, 128), ws=None, n=0) == WORKSPACE
    # pages that the scale blocks do not divide
    pool = _t(9, 2, 24, 64, dtype=E4)
    opts = _abi.fa_forward_options(page_table=FAKE, page_size=24, pages_per_seq=4)
    assert fp8(lib, q, pool, pool, o, _bm(2, 1, 1, 96, 128, 128), opts=opts) == PARAM
    assert fp8(lib, q, _t(9, 2, 16, 64, dtype=E4), pool, o, _bm(2, 1, 1, 96, 128, 128), opts=opts) == SHAPE


def test_forward_fp8_workspace(lib):
    """Decode calls need scratch for their splits only, others the restored cache."""
    def size(q, k, bm, split=0):
        n = C.c_size_t()
        quant = _abi.fa_kv_quant(FAKE, FAKE, 16, 0)
        rc = lib.flexattn_forward_fp8_workspace_size(C.byref(q), C.byref(k), C.byref(k), C.byref(quant), C.byref(bm),
                                                     split, None, C.byref(n))
        assert rc == 0, fa.flexattn_last_error()
        return n.value
    k = _t(2, 2, 4096, 64, dtype=E4)
    assert size(_t(2, 4, 1, 64), k, _bm(2, 1, 1, 4096, 128, 128), split=1) == 0
    assert size(_t(2, 4, 1, 64), k, _bm(2, 1, 1, 4096, 128, 128), split=4) == 2 * 4 * 1 * 4 * 66 * 4
    restored = 2 * 2 * 2 * 4096 * 64 * 2
    assert size(_t(2, 4, 512, 64), k, _bm(2, 1, 512, 4096, 128, 128)) == restored
    assert size(_t(2, 4, 1, 64, dtype=F32), k, _bm(2, 1, 1, 4096, 128, 128)) == 2 * restored
    # the plain entry points keep refusing codes
    q, bm = _t(2, 4, 1, 64), _bm(2, 1, 1, 4096, 128, 128)
    score, mask = _abi.fa_score_mod(kind=0), _abi.fa_mask_mod(kind=1)
    assert lib.flexattn_forward(C.byref(q), C.byref(k), C.byref(k), C.byref(q), None, 0.0, 1, C.byref(score),
                                C.byref(mask), C.byref(bm), 0, None, None, 0, None) == DTYPE


def test_python_checks_come_before_the_library():
    """Tensors on the host, of other types or extents, never reach the library."""
    x = torch.zeros((1, 1, 2, 8), dtype=torch.bfloat16)
    with pytest.raises(fa.FlexAttnError):
        fa.flexattn_qk_norm_rope(x, None, rope={"inv_freq": torch.zeros(4)})
    with pytest.raises(fa.FlexAttnError):
        fa.flexattn_qk_norm_rope(None, None)
    with pytest.raises(fa.FlexAttnError):
        fa.flexattn_cache_append(x, x, {"k": x, "v": x, "cache_len": torch.zeros(1, dtype=torch.int32)})
    with pytest.raises(fa.FlexAttnError) as e:
        fa.flexattn_qk_norm_rope(x.half(), None)
    assert e.value.status == DTYPE
