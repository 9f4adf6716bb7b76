"""Refusals of the training and expert calls (no GPU): every call below fails
validation or has no work, so nothing launches."""
import ctypes

import pytest
import torch

from combine_fp32_router_amd import binding as B

OK, NULL, SHAPE, ALIGN, WORKSPACE, HIP, ALIAS = range(7)
F = ctypes.c_void_p(0x10000)  # aligned, never dereferenced
G = ctypes.c_void_p(0x20000)
H = ctypes.c_void_p(0x30000)
ODD = ctypes.c_void_p(0x10002)
EIGHT = ctypes.c_void_p(0x40008)


@pytest.fixture(scope="module")
def lib():
    return B.load()


def test_balance_loss(lib):
    n = ctypes.c_size_t(0)
    f = lambda T, seg, E, k, *p, ws=F, size=1 << 30: lib.moe_balance_loss(  # noqa: E731
        *p[:3], T, seg, E, k, *p[3:], ws, ctypes.byref(ctypes.c_size_t(size)), None)
    ok = (F, F, None, F, F, F, F)
    assert lib.moe_balance_loss(None, None, None, 100, 10, 8, 2, None, None, None, None, None, ctypes.byref(n), None) == OK
    assert n.value > 0 and n.value % 256 == 0 and n.value == B.balance_workspace_bytes(100, 10, 8, 2)
    assert lib.moe_balance_loss(None, None, None, 100, 10, 8, 2, None, None, None, None, None, None, None) == NULL
    assert f(-1, 1, 8, 2, *ok) == SHAPE
    assert f(4, 0, 8, 2, *ok) == SHAPE
    assert f(4, -1, 8, 2, *ok) == SHAPE
    assert f(4, 4, 0, 1, *ok) == SHAPE
    assert f(4, 4, 1025, 1, *ok) == SHAPE
    assert f(4, 4, 8, 9, *ok) == SHAPE
    assert f(4, 4, 64, 17, *ok) == SHAPE
    assert f(66000, 1, 8, 2, *ok) == SHAPE      # more than 65535 segments
    assert f(2 ** 62, 2 ** 61, 8, 2, *ok) == SHAPE  # T*k
    assert f(100, 10, 8, 2, *ok, size=n.value - 1) == WORKSPACE
    assert f(100, 10, 8, 2, *ok, ws=ODD) == ALIGN
    for i in (0, 1, 3, 4, 5, 6):
        assert f(100, 10, 8, 2, *(None if j == i else p for j, p in enumerate(ok))) == NULL
        assert f(100, 10, 8, 2, *(ODD if j == i else p for j, p in enumerate(ok))) == ALIGN


def test_route_grad(lib):
    f = lambda *p, T=10, seg=5, E=8, k=2: lib.moe_route_grad(*p[:8], T, seg, E, k, p[8], None)  # noqa: E731
    ok = (F, F, F, F, None, F, F, F, F)
    assert f(*ok, T=-1) == SHAPE and f(*ok, seg=0) == SHAPE and f(*ok, E=1025) == SHAPE and f(*ok, k=9) == SHAPE
    assert f(*ok, T=66000, seg=1) == SHAPE
    assert f(*ok, T=2 ** 30, seg=2 ** 30, E=8, k=1) == SHAPE  # grid
    for i in (0, 1, 2, 6, 7, 8):
        assert f(*(None if j == i else p for j, p in enumerate(ok))) == NULL
    assert f(F, F, F, None, None, None, F, F, F) == NULL      # neither part
    for i in (0, 1, 2, 3, 5, 6, 7, 8):
        assert f(*(ODD if j == i else p for j, p in enumerate(ok))) == ALIGN
    assert f(*([None] * 9), T=0) == OK


def test_combine_grad(lib):
    f = lambda d, r, s, q, p, w, o, dw, T=4, H=32, k=2: lib.moe_combine_grad(d, r, s, q, p, w, T, H, k, o, dw, None)  # noqa: E731
    assert f(F, G, None, 0, F, F, H, F, T=-1) == SHAPE and f(F, G, None, 0, F, F, H, F, H=24) == SHAPE
    assert f(F, G, None, 4, F, F, H, F) == SHAPE and f(F, G, F, 2, F, F, H, F, H=48) == SHAPE
    assert f(F, G, None, 0, F, F, H, F, k=17) == SHAPE
    assert f(F, G, None, 0 | B.MOE_PACK_STREAM, F, F, H, F) == SHAPE
    assert f(F, G, None, 0, F, F, H, F, T=2 ** 30, H=65536, k=1) == SHAPE  # grid
    assert f(None, G, None, 0, F, F, H, F) == NULL and f(F, None, None, 0, F, F, H, F) == NULL
    assert f(F, G, None, 0, None, F, H, F) == NULL and f(F, G, None, 0, F, None, H, F) == NULL
    assert f(F, G, None, 0, F, F, None, None) == NULL and f(F, G, None, 1, F, F, H, F) == NULL
    assert f(EIGHT, G, None, 0, F, F, H, F) == ALIGN and f(F, EIGHT, None, 0, F, F, H, F) == ALIGN
    assert f(F, G, None, 0, ODD, F, H, F) == ALIGN and f(F, G, None, 0, F, ODD, H, F) == ALIGN
    assert f(F, G, None, 0, F, F, EIGHT, F) == ALIGN and f(F, G, None, 0, F, F, H, ODD) == ALIGN
    assert f(F, G, ODD, 3, F, F, H, F) == ALIGN
    assert f(F, G, None, 0, F, F, F, F) == ALIAS and f(F, G, None, 0, F, F, G, F) == ALIAS
    assert f(None, None, None, 0, None, None, None, None, T=0) == OK


def test_expert_matmul(lib):
    def f(x=F, off=F, w=G, b=None, act=0, res=None, E=2, rows=4, K=32, N=32, out=H, pre=None, ws=None, size=None):
        return lib.moe_expert_matmul(x, off, w, b, act, res, E, rows, K, N, out, pre, ws, size, None)
    for bad in (dict(E=0), dict(E=1025), dict(rows=-1), dict(rows=2 ** 31), dict(K=0), dict(K=24), dict(K=65552),
                dict(N=8), dict(N=40), dict(N=65552), dict(act=-1), dict(act=5)):
        assert f(**bad) == SHAPE, bad
    for p in ("x", "off", "w", "out"):
        assert f(**{p: None}) == NULL
    for p in ("x", "w", "b", "res", "out", "pre"):
        assert f(**{p: EIGHT}) == ALIGN
    assert f(off=ODD) == ALIGN
    assert f(out=F) == ALIAS and f(out=G) == ALIAS and f(pre=H) == ALIAS and f(pre=F) == ALIAS and f(pre=G) == ALIAS
    assert f(res=ctypes.c_void_p(0x50000), pre=ctypes.c_void_p(0x50000)) == ALIAS
    assert f(None, None, None, out=None, rows=0) == OK


def test_expert_matmul_gradients(lib):
    def dx(dy=F, off=F, w=G, act=0, z=None, E=2, rows=4, K=32, N=32, out=H, ws=None, size=None):
        return lib.moe_expert_matmul_dx(dy, off, w, act, z, E, rows, K, N, out, ws, size, None)
    for bad in (dict(E=0), dict(rows=-1), dict(rows=2 ** 31), dict(K=24), dict(K=65552), dict(N=24), dict(N=131088),
                dict(act=7)):
        assert dx(**bad) == SHAPE, bad
    for p in ("dy", "off", "w", "out"):
        assert dx(**{p: None}) == NULL
    assert dx(act=2) == NULL
    for p in ("dy", "w", "z", "out"):
        assert dx(**{p: EIGHT}) == ALIGN
    assert dx(off=ODD) == ALIGN and dx(out=F) == ALIAS and dx(out=G) == ALIAS
    assert dx(None, None, None, out=None, rows=0) == OK

    def dw(dy=F, x=G, off=F, E=2, rows=4, K=32, N=32, flags=0, out=H, db=None, ws=None, size=None):
        return lib.moe_expert_matmul_dw(dy, x, off, E, rows, K, N, flags, out, db, ws, size, None)
    for bad in (dict(E=0), dict(rows=-1), dict(K=24), dict(K=65552), dict(N=0), dict(flags=2), dict(flags=0x101),
                dict(flags=-1)):
        assert dw(**bad) == SHAPE, bad
    for p in ("dy", "x", "off", "out"):
        assert dw(**{p: None}) == NULL
    for p in ("dy", "x", "out", "db"):
        assert dw(**{p: EIGHT}) == ALIGN
    assert dw(off=ODD) == ALIGN and dw(out=F) == ALIAS and dw(out=G) == ALIAS


def test_expert_gradient_workspaces(lib):
    n = ctypes.c_size_t(7)
    none = [None] * 3
    q = {"moe_expert_matmul": lambda E, rows, K, N, s=n: lib.moe_expert_matmul(
             *none, None, 0, None, E, rows, K, N, None, None, None, ctypes.byref(s), None),
         "moe_expert_matmul_dx": lambda E, rows, K, N, s=n: lib.moe_expert_matmul_dx(
             *none, 0, None, E, rows, K, N, None, None, ctypes.byref(s), None),
         "moe_expert_matmul_dw": lambda E, rows, K, N, s=n: lib.moe_expert_matmul_dw(
             *none, E, rows, K, N, 0, None, None, None, ctypes.byref(s), None)}
    for name, f in q.items():
        assert f(1, 8192, 65552, 65552) == SHAPE
        for sizes in ((1, 0, 64, 64), (8, 8192, 7168, 7168), (300, 300, 16, 8192), (2, 64, 64, 64)):
            assert f(*sizes) == OK and n.value == 0 == B.expert_workspace_bytes(name, *sizes)
    assert q["moe_expert_matmul_dx"](2, 200, 128, 8192) == OK and n.value > 0 and n.value % 256 == 0
    few = ctypes.c_size_t(n.value - 1)
    assert q["moe_expert_matmul"](2, 4000, 8192, 128) == OK and n.value > 0
    few = ctypes.c_size_t(n.value - 1)
    call = lambda ws, size: lib.moe_expert_matmul(  # noqa: E731
        F, F, G, None, 0, None, 2, 4000, 8192, 128, H, None, ws, size, None)
    assert call(F, ctypes.byref(few)) == WORKSPACE and call(F, None) == WORKSPACE
    assert call(EIGHT, ctypes.byref(n)) == ALIGN
    assert q["moe_expert_matmul_dx"](2, 200, 128, 8192) == OK
    few = ctypes.c_size_t(n.value - 1)
    call = lambda ws, size: lib.moe_expert_matmul_dx(  # noqa: E731
        F, F, G, 0, None, 2, 200, 128, 8192, H, ws, size, None)
    assert call(F, ctypes.byref(few)) == WORKSPACE and call(F, None) == WORKSPACE
    assert call(EIGHT, ctypes.byref(n)) == ALIGN
    assert q["moe_expert_matmul_dw"](2, 20000, 128, 128) == OK and n.value > 0
    few = ctypes.c_size_t(n.value - 1)
    call = lambda ws, size: lib.moe_expert_matmul_dw(  # noqa: E731
        F, G, F, 2, 20000, 128, 128, 0, H, None, ws, size, None)
    assert call(F, ctypes.byref(few)) == WORKSPACE and call(F, None) == WORKSPACE
    assert call(EIGHT, ctypes.byref(n)) == ALIGN


def test_binding_refuses_host_tensors_and_wrong_shapes():
    """ValueError before the library is called: dtypes, shapes, devices."""
    bf = lambda *s: torch.zeros(*s, dtype=torch.bfloat16)  # noqa: E731
    i32 = lambda *s: torch.zeros(*s, dtype=torch.int32)  # noqa: E731
    x, w, off, out = bf(4, 32), bf(2, 48, 32), i32(3), bf(4, 48)
    for a in ((bf(4, 16), off, w, None, 0, None, out), (x, i32(2), w, None, 0, None, out),
              (x, off, bf(48, 32), None, 0, None, out), (x, off, w, None, 0, None, bf(4, 32)),
              (x, off, w, None, 4, None, out), (x, off, w, torch.zeros(2, 32), 0, None, out),
              (x, off, w, bf(2, 48), 0, None, out), (x, off, w, None, 0, bf(3, 48), out),
              (x.float(), off, w, None, 0, None, out), (x, off.long(), w, None, 0, None, out),
              (x, off, w, None, 0, None, out)):  # the last only lacks a device
        with pytest.raises(ValueError):
            B.moe_expert_matmul(*a, stream=0)
    with pytest.raises(ValueError):
        B.moe_expert_matmul_dx(bf(4, 48), off, w, 2, None, x, stream=0)
    with pytest.raises(ValueError):
        B.moe_expert_matmul_dw(bf(4, 48), x, off, torch.zeros(2, 48, 32, dtype=torch.float64), stream=0)
    z, idx = torch.zeros(4, 8), i32(4, 2)
    bal = B.alloc_balance(4, 2, 8, 2, "cpu")
    assert bal.loss.shape == (2,) and bal.expert_counts.shape == (2, 8)
    for a in ((z.double(), idx, None, bal), (z, idx.long(), None, bal), (z, i32(8), None, bal), (z, idx, i32(4), bal),
              (z, idx, torch.zeros(3, dtype=torch.uint8), bal), (z, idx, None, B.alloc_balance(4, 4, 8, 2, "cpu")._replace(seg_tokens=2)),
              (z, idx, None, bal)):
        with pytest.raises(ValueError):
            B.moe_balance_loss(*a, stream=0)
    w2, d_w, d_loss = torch.zeros(4, 2), torch.zeros(4, 2), torch.zeros(2)
    for a in ((z, idx, None, d_w, None, None, None, z), (None, idx, w2, d_w, None, d_loss, bal, z),
              (z, idx, w2, d_w, None, torch.zeros(1), bal, z), (z, idx, w2, torch.zeros(3, 2), None, None, None, z)):
        with pytest.raises(ValueError):
            B.moe_route_grad(*a, stream=0)
    with pytest.raises(ValueError):
        B.moe_combine_grad(bf(4, 16), None, None, 0, i32(8), torch.zeros(4, 2), 4, 32, 2, bf(8, 32), None, stream=0)
