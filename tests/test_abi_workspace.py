"""CPU checks of the workspace sizes that callers of the C ABI allocate to.

A size that a caller once allocated has to stay enough: the backward's sizes
are pinned (256 compute units, which the library also assumes without a
device), and a backward from a checkpoint asks for no more than the plain one.
"""

import ctypes
import os

import pytest

P = ctypes.c_void_p(1 << 20)   # non-NULL and aligned; never dereferenced on error paths


@pytest.fixture(scope="module")
def lib():
    from bit_quantized_fine_qlora_amd import _lib
    if not os.path.exists(_lib.LIB_PATH):
        pytest.fail("libqlora.so is not built (run __graft_entry__.build())")
    return _lib.load()


# M, n, m, r; bytes of the backward, and of the backward with dropout
SIZES = [(8192, 8192, 8192, 64, 41943040, 310378496), (8192, 8192, 8192, 128, 67108864, 335544320),
         (4096, 4096, 14336, 16, 27000832, 94109696), (8192, 8192, 28672, 64, 48234496, 316669952),
         (2048, 4096, 4096, 32, 46925056, 80479488), (2468, 128, 1, 32, 2062848, 3326464),
         (7535, 64, 1, 64, 11109632, 13038592)]


@pytest.mark.parametrize("M,n,m,r,plain,dropout", SIZES)
def test_backward_needs_no_more_than_it_did(lib, M, n, m, r, plain, dropout):
    assert 0 < lib.qlora_workspace_bytes(1, M, n, m, r) <= plain
    assert 0 < lib.qlora_workspace_bytes(2, M, n, m, r) <= dropout


@pytest.mark.parametrize("M,n,m,r,plain,dropout", SIZES)
def test_checkpointed_backward_takes_the_plain_size(lib, M, n, m, r, plain, dropout):
    """The size check comes after the others: one byte less is refused for its size, not accepted and not otherwise."""
    need = lib.qlora_workspace_bytes(1, M, n, m, r)
    st = lib.qlora_linear_bwd_ckpt(M, n, m, r, 1.0, P, P, P, P, P, P, P, P, P, P, P, P, None, P, need - 1, None)
    assert st == -5
