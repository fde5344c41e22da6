"""CPU checks of the C ABI of the experts' layer and the optimizer step over
many tensors: bad arguments are rejected before anything is launched; and what
the binding itself refuses."""

import ctypes
import os

import pytest
import torch

P = ctypes.c_void_p(1 << 20)   # non-NULL and aligned; never dereferenced on error paths
MIS = ctypes.c_void_p((1 << 20) + 4)
ODD = ctypes.c_void_p((1 << 20) + 2)
NAN, INF = float("nan"), float("inf")


@pytest.fixture(scope="module")
def lib():
    from bit_quantized_fine_qlora_amd import _lib
    if not os.path.exists(_lib.LIB_PATH):
        pytest.fail("libqlora.so is not built (run __graft_entry__.build())")
    return _lib.load()


SHAPES = [  # sizes that both directions refuse, with the status
    (dict(M=0), -2), (dict(M=-5), -2), (dict(M=1 << 22), -2), (dict(E=0), -2), (dict(E=-1), -2), (dict(E=1025), -2),
    (dict(n=100), -2), (dict(n=0), -2), (dict(m=0), -2), (dict(E=1024, m=1 << 21), -2), (dict(r=0), -3),
    (dict(r=129), -3), (dict(s=NAN), -7), (dict(s=INF), -7), (dict(M=1 << 20, m=1 << 10), -2),
    (dict(m=1 << 22, n=512), -2), (dict(E=1024, M=(1 << 14) - 1, n=1 << 16, m=1 << 15), -2)]


def test_experts_fwd(lib):
    def f(M=32, E=4, n=256, m=256, r=8, s=1.0, x=P, off=P, c=P, a=P, c2=P, A=P, B=P, h=P, u=P, ws=P, wsb=1 << 40):
        return lib.qlora_experts_fwd(M, E, n, m, r, s, x, off, c, a, c2, A, B, h, u, ws, wsb, None)

    for kw, status in SHAPES:
        assert f(**kw) == status, kw
    for name in ("x", "off", "c", "a", "c2", "A", "B", "h"):
        assert f(**{name: None}) == -1, name
    for name in ("x", "off", "c", "a", "c2", "A", "B", "h", "u", "ws"):
        assert f(**{name: MIS}) == -4, name
    need = lib.qlora_experts_workspace_bytes(0, 32, 4, 256, 256, 8)
    assert need > 0 and f(wsb=need - 1) == -5 and f(ws=None) == -5


def test_experts_bwd(lib):
    def f(M=32, E=4, n=256, m=256, r=8, s=1.0, x=P, g=P, off=P, c=P, a=P, c2=P, A=P, B=P, u=P, gx=P, gA=P, gB=P, ws=P,
          wsb=1 << 40):
        return lib.qlora_experts_bwd(M, E, n, m, r, s, x, g, off, c, a, c2, A, B, u, gx, gA, gB, ws, wsb, None)

    for kw, status in SHAPES:
        assert f(**kw) == status, kw
    for name in ("x", "g", "off", "c", "a", "c2", "A", "B", "gA", "gB"):
        assert f(**{name: None}) == -1, name
    for name in ("x", "g", "off", "c", "a", "c2", "A", "B", "u", "gx", "gA", "gB", "ws"):
        assert f(**{name: MIS}) == -4, name
    need = lib.qlora_experts_workspace_bytes(1, 32, 4, 256, 256, 8)
    assert need > 0 and f(wsb=need - 1) == -5 and f(ws=None) == -5


def test_experts_workspace(lib):
    f = lib.qlora_experts_workspace_bytes
    for op in (0, 1):
        for kw, status in SHAPES:
            if "s" in kw:
                continue
            a = dict(M=32, E=4, n=256, m=256, r=8, **{}) | kw
            assert f(op, a["M"], a["E"], a["n"], a["m"], a["r"]) == 0, kw
    assert f(2, 32, 4, 256, 256, 8) == 0 and f(-1, 32, 4, 256, 256, 8) == 0


def tensor(_lib, count=100, p=P, p16=P, g=P, m=P, v=P, md=P, vd=P, gt=0, mom=1):
    return _lib.AdamWTensor(count, p, p16, g, m, v, md, vd, gt, mom)


BAD = [(dict(count=0), -2), (dict(count=-1), -2), (dict(count=1 << 40), -2), (dict(gt=2), -7), (dict(gt=-1), -7),
       (dict(mom=2), -7), (dict(mom=-1), -7), (dict(p=None), -1), (dict(g=None), -1), (dict(m=None), -1),
       (dict(v=None), -1), (dict(md=None), -1), (dict(vd=None), -1), (dict(p=MIS), -4), (dict(p16=MIS), -4),
       (dict(g=MIS), -4), (dict(m=MIS), -4), (dict(v=MIS), -4), (dict(md=ODD), -4), (dict(vd=ODD), -4)]


def test_adamw_plan(lib):
    from bit_quantized_fine_qlora_amd import _lib
    h = _lib.AdamWHandle()

    def f(tensors, count=None, plan=P, nbytes=1 << 40, handle=ctypes.byref(h)):
        arr = (_lib.AdamWTensor * max(1, len(tensors)))(*tensors)
        return lib.qlora_adamw_plan(arr, len(tensors) if count is None else count, plan, nbytes, handle, None)

    good = tensor(_lib)
    for kw, status in BAD:
        bad = tensor(_lib, **kw)
        assert f([bad]) == status and f([good, bad]) == status and f([bad, good]) == status, kw
        arr = (_lib.AdamWTensor * 2)(good, bad)
        assert lib.qlora_adamw_plan_bytes(arr, 2) == 0, kw
    assert f([good], count=0) == -2 and f([good], count=-3) == -2
    assert f([tensor(_lib, count=(1 << 40) - 1)] * 4) == -2   # 2^31 chunks of 2048 together
    arr = (_lib.AdamWTensor * 1)(good)
    need = lib.qlora_adamw_plan_bytes(arr, 1)
    assert need > 0 and f([good], nbytes=need - 1) == -5 and f([good], plan=None) == -5 and f([good], plan=MIS) == -4
    assert lib.qlora_adamw_plan(arr, 1, P, need, None, None) == -1
    assert lib.qlora_adamw_plan(None, 1, P, need, ctypes.byref(h), None) == -1
    assert lib.qlora_adamw_plan_bytes(None, 1) == 0
    # 32-bit moments have no steps
    arr = (_lib.AdamWTensor * 1)(tensor(_lib, mom=0, md=None, vd=None))
    assert lib.qlora_adamw_plan_bytes(arr, 1) == need


def test_adamw_step_and_clip(lib):
    from bit_quantized_fine_qlora_amd import _lib

    def handle(plan=1 << 20, tensors=1, chunks=1):
        return ctypes.byref(_lib.AdamWHandle(plan, tensors, chunks, 0))

    def step(h=handle(), lr=1e-3, b1=0.9, b2=0.999, eps=1e-8, wd=0.0, t=1, clip=P):
        return lib.qlora_adamw_step(h, lr, b1, b2, eps, wd, t, clip, None)

    def clip(h=handle(), most=1.0, out=P):
        return lib.qlora_grad_clip(h, most, out, None)

    for f in (step, clip):
        assert f(h=None) == -1 and f(h=handle(plan=None)) == -1 and f(h=handle(plan=(1 << 20) + 8)) == -4
        assert f(h=handle(tensors=0)) == -2 and f(h=handle(chunks=0)) == -2 and f(h=handle(chunks=1 << 31)) == -2
    for kw in (dict(lr=NAN), dict(lr=-1.0), dict(lr=INF), dict(b1=1.0), dict(b1=-0.1), dict(b1=NAN), dict(b2=1.0),
               dict(b2=NAN), dict(eps=0.0), dict(eps=-1e-8), dict(eps=1e-39), dict(eps=NAN), dict(eps=INF),
               dict(eps=1e39), dict(wd=NAN), dict(wd=INF), dict(t=0), dict(t=-1)):
        assert step(**kw) == -7, kw
    assert step(clip=MIS) == -4
    assert clip(most=0.0) == -7 and clip(most=-1.0) == -7 and clip(most=NAN) == -7
    assert clip(out=None) == -1 and clip(out=MIS) == -4


def test_moment8_values(lib):
    f = lib.qlora_moment8_values
    assert f(2, 8, P, P, P, None) == -7 and f(-1, 8, P, P, P, None) == -7
    assert f(0, 0, P, P, P, None) == -2 and f(0, 1 << 40, P, P, P, None) == -2
    for i in range(3):
        assert f(0, 8, *[None if j == i else P for j in range(3)], None) == -1
        assert f(1, 8, *[(ODD if i == 1 else MIS) if j == i else P for j in range(3)], None) == -4


def test_binding_refuses_host_tensors_and_wrong_moments():
    import bit_quantized_fine_qlora_amd as Q
    f, b = torch.zeros(256), torch.zeros(256, dtype=torch.bfloat16)

    def m8(signed, n=256):
        return Q.Moment8(torch.zeros(n, dtype=torch.uint8), torch.zeros(-(-n // 128)), signed)

    def make(p=f, p16=b, g=b, m=f, v=f):
        return Q.AdamWStep([(p, p16, g, m, v)])

    with pytest.raises(ValueError, match="no tensors"):
        Q.AdamWStep([])
    with pytest.raises(ValueError, match="GPU or in pinned"):
        make()
    with pytest.raises(ValueError, match="GPU or in pinned"):
        make(m=m8(True), v=m8(False))
    for kw in (dict(p=b), dict(p16=f), dict(g=torch.zeros(256, dtype=torch.float16)), dict(m=b), dict(v=b),
               dict(m=m8(True)), dict(v=m8(False))):
        with pytest.raises(TypeError):
            make(**kw)
    for kw in (dict(g=b[:255]), dict(m=f[:100]), dict(p=torch.zeros(512)[::2]), dict(m=m8(False), v=m8(True)),
               dict(m=m8(True, 255), v=m8(False)),
               dict(m=Q.Moment8(torch.zeros(256, dtype=torch.uint8), torch.zeros(3), True), v=m8(False))):
        with pytest.raises(ValueError):
            make(**kw)


def test_binding_refuses_experts_of_other_shapes():
    import bit_quantized_fine_qlora_amd as Q
    E, M, n, m, r = 3, 10, 64, 8, 4
    bf = dict(dtype=torch.bfloat16)
    q = Q.QuantizedWeight(torch.zeros(E * m * n // 2, dtype=torch.uint8), torch.zeros(E * m * n // 64, dtype=torch.uint8),
                          torch.zeros(1), E * m, n)
    x, off = torch.zeros(M, n, **bf), torch.zeros(E + 1, dtype=torch.int32)
    A, B = torch.zeros(E, r, n, **bf), torch.zeros(E, m, r, **bf)
    for args in ((x, off, q, A[0], B, 1.0), (x, off, q, A[:2], B[:2], 1.0), (x, off, q, A[:0], B, 1.0),
                 (x, off[:3], q, A, B, 1.0), (x[:, :32], off, q, A, B, 1.0), (x, off, q, A, B[:, :4], 1.0)):
        with pytest.raises(ValueError):
            Q.experts_fwd(*args)
    with pytest.raises(TypeError):
        Q.experts_fwd(x.float(), off, q, A, B, 1.0)
    with pytest.raises(TypeError, match="Checkpoint8"):
        Q.experts_bwd(Q.alloc_checkpoint(M, n, "cpu"), torch.zeros(M, m, **bf), off, q, A, B, 1.0)
    with pytest.raises(ValueError, match="device tensor"):
        Q.experts_fwd(x, off, q, A, B, 1.0)
