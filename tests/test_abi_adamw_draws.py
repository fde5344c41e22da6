"""CPU checks of qlora_adamw_step_ex: the arguments that qlora_adamw_step refuses are refused with a seed too, before
anything is launched."""

import ctypes
import os

import pytest

P = ctypes.c_void_p(1 << 20)   # non-NULL and aligned; never dereferenced on error paths
MIS = ctypes.c_void_p((1 << 20) + 4)
NAN, INF = float("nan"), float("inf")


@pytest.fixture(scope="module")
def lib():
    from bit_quantized_fine_qlora_amd import _lib
    if not os.path.exists(_lib.LIB_PATH):
        pytest.fail("libqlora.so is not built (run __graft_entry__.build())")
    return _lib.load()


@pytest.mark.parametrize("seed", [None, 0, 2 ** 64 - 1])
def test_refusals(lib, seed):
    from bit_quantized_fine_qlora_amd import _lib

    def handle(plan=1 << 20, tensors=1, chunks=1):
        return ctypes.byref(_lib.AdamWHandle(plan, tensors, chunks, 0))

    def step(h=handle(), lr=1e-3, b1=0.9, b2=0.999, eps=1e-8, wd=0.0, t=1, clip=P):
        s = None if seed is None else ctypes.pointer(ctypes.c_uint64(seed))
        return lib.qlora_adamw_step_ex(h, lr, b1, b2, eps, wd, t, clip, s, None)

    assert step(h=None) == -1 and step(h=handle(plan=None)) == -1 and step(h=handle(plan=(1 << 20) + 8)) == -4
    assert step(h=handle(tensors=0)) == -2 and step(h=handle(chunks=0)) == -2 and step(h=handle(chunks=1 << 31)) == -2
    for kw in (dict(lr=NAN), dict(lr=-1.0), dict(b1=1.0), dict(b1=NAN), dict(b2=1.0), dict(b2=-0.1), dict(eps=0.0),
               dict(eps=1e-39), dict(eps=INF), dict(wd=NAN), dict(wd=INF), dict(t=0), dict(t=-1)):
        assert step(**kw) == -7, kw
    assert step(clip=MIS) == -4
