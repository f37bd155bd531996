"""Which way a call of attention over an e4m3 cache goes, seen in the workspace it
asks for (no GPU needed)."""

import ctypes as C

import pytest

import programmable_block_sparse_b200 as fa
from programmable_block_sparse_b200 import _abi
from test_abi_cpu import FAKE, _bm, _t

E4 = _abi.FA_DTYPE_E4M3


@pytest.fixture(scope="module")
def lib():
    from programmable_block_sparse_b200 import build
    build.build()
    return fa.load_library()


def workspace(lib, B, Hq, Hkv, L, S, D, split=0, BM=128):
    n = C.c_size_t()
    q, k = _t(B, Hq, L, D), _t(B, Hkv, S, D, dtype=E4)
    quant, bm = _abi.fa_kv_quant(FAKE, FAKE, 16, 0), _bm(B, 1, L, S, BM, 128)
    rc = lib.flexattn_forward_fp8_workspace_size(C.byref(q), C.byref(k), C.byref(k), C.byref(quant), C.byref(bm), split,
                                                 None, C.byref(n))
    assert rc == 0, fa.flexattn_last_error()
    return n.value


@pytest.mark.parametrize("B", [1, 2, 8, 32])
@pytest.mark.parametrize("L", [17, 32, 48, 128])
def test_explicit_splits_take_the_decode_kernel(lib, B, L):
    """Scratch for the splits' partial results, at every batch and up to a tile of rows."""
    for split in (2, 4):
        assert workspace(lib, B, 16, 4, L, 4096, 64, split) == B * 16 * L * split * (64 + 2) * 4


@pytest.mark.parametrize("L,BM", [(48, 48), (48, 64), (100, 100), (33, 33)])
def test_query_tiles_without_a_tensor_core_prefill_stay_on_the_decode_kernel(lib, L, BM):
    """Where 128-row tiles go to the prefill over the restored cache, smaller
    ones would only find the general kernel there."""
    restored = 2 * 64 * 4 * 4096 * 64 * 2
    assert workspace(lib, 64, 16, 4, L, 4096, 64) == restored
    assert workspace(lib, 64, 16, 4, L, 4096, 64, BM=BM) < restored
