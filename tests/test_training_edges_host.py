"""Refusals and sizes at the edges of the training and expert calls (no GPU):
nothing below launches."""
import ctypes

import pytest
import torch

from combine_fp32_router_amd import binding as B
from combine_fp32_router_amd import epgroup
from combine_fp32_router_amd.epgroup import EPGroup
from combine_fp32_router_amd.experts import ExpertMLP

OK, NULL, SHAPE, ALIGN, WORKSPACE, HIP, ALIAS = range(7)
F = ctypes.c_void_p(0x10000)  # aligned, never dereferenced
G = ctypes.c_void_p(0x20000)
H = ctypes.c_void_p(0x30000)


@pytest.fixture(scope="module")
def lib():
    return B.load()


def test_the_flag_of_masked_gates_is_no_size(lib):
    flag = B.MOE_ROUTE_MASKED_GATES
    f = lambda k, T=10: lib.moe_route_grad(F, F, F, F, None, F, F, F, T, 5, 8, k, None, None)  # noqa: E731
    assert f(2) == NULL and f(2 | flag) == NULL  # no output: past the sizes
    for k in (9, 0, -1, 2 | flag << 1):
        assert f(k) == SHAPE and f(k | flag) == SHAPE
    assert f(2 | flag, T=0) == OK
    assert lib.moe_balance_loss(None, None, None, 10, 5, 8, 2 | flag, None, None, None, None, None,
                                ctypes.byref(ctypes.c_size_t(0)), None) == SHAPE


def bf16(*s):
    return torch.zeros(*s, dtype=torch.bfloat16)


@pytest.fixture
def launches(monkeypatch):
    """Every launch of a layer replaced by its name in a list."""
    calls = []
    for module, names in ((B, B.EXPORTS), (epgroup.HN, ("moe_exchange_blocks",))):
        for name in names:
            if hasattr(module, name) and name not in ("moe_status_string", "moe_row_bytes"):
                monkeypatch.setattr(module, name, lambda *a, _name=name, **kw: calls.append(_name))
    monkeypatch.setattr(torch.cuda, "current_stream", lambda *a: None)
    return calls


def experts(E=4, H=32, I=16, max_rows=64):
    return ExpertMLP(bf16(E, I, H), bf16(E, H, I), B.MOE_ACT_SILU, max_rows=max_rows, train=True)


def test_experts_refuse_a_backward_of_another_forward(launches):
    m, off, x = experts(), torch.zeros(5, dtype=torch.int32), bf16(8, 32)
    with pytest.raises(ValueError, match="before"):
        m.backward(x, x, off, None, None)
    assert m.forward(x, off, x) is x
    first = m.forwards
    m.backward(x, x, off, None, None)
    m.backward(x, x, off, None, None, forward=first)
    with pytest.raises(ValueError, match="9 rows"):
        m.backward(bf16(9, 32), bf16(9, 32), off, None, None)
    m.forward(x, off, x)
    launches.clear()
    with pytest.raises(ValueError, match="again"):
        m.backward(x, x, off, None, None, forward=first)
    assert not launches
    m.backward(x, x, off, None, None)


def test_a_forward_that_fails_half_way_keeps_nothing(launches, monkeypatch):
    m, off, x = experts(), torch.zeros(5, dtype=torch.int32), bf16(8, 32)
    m.forward(x, off, x)

    def fail(*a, **kw):
        raise B.MoeError("moe_expert_matmul", HIP)

    monkeypatch.setattr(B, "moe_expert_matmul", fail)
    with pytest.raises(B.MoeError):
        m.forward(x, off, x)
    with pytest.raises(ValueError, match="before"):
        m.backward(x, x, off, None, None)


def test_groups_that_share_their_experts(launches):
    """A group's backward is refused once the experts ran for another group or
    call; what needs no experts (the logits' gradient) still goes."""
    m = experts()
    one, two = (EPGroup(16, 32, 4, 2, 2, device="cpu", experts=m) for _ in range(2))
    z, x = torch.zeros(16, 4), bf16(16, 32)
    one.run(z, x, x)
    one.backward(x, x, z)
    two.run(z, x, x)
    two.backward(x, x, z, m.alloc_grads())
    for kw in (dict(d_x=x), dict(d_x=None, grads=m.alloc_grads())):
        launches.clear()
        with pytest.raises(ValueError, match="again"):
            one.backward(x, d_logits=z, **kw)
        assert not launches
    one.backward(x, None, z)
    m.forward(bf16(8, 32), torch.zeros(5, dtype=torch.int32), bf16(8, 32))
    with pytest.raises(ValueError, match="again"):
        two.backward(x, x, z)
    two.run(z, x, x)
    two.backward(x, x, z)


@pytest.mark.parametrize("name", ["moe_recv_layout", "moe_recv_ungroup", "moe_combine"])
def test_a_run_that_fails_half_way_is_not_gone_back_through(launches, monkeypatch, name):
    m = experts()
    group, z, x = EPGroup(16, 32, 4, 2, 2, device="cpu", experts=m), torch.zeros(16, 4), bf16(16, 32)
    group.run(z, x, x)
    group.backward(x, x, z)

    def fail(*a, **kw):
        raise B.MoeError(name, HIP)

    with monkeypatch.context() as patch:
        patch.setattr(B, name, fail)
        with pytest.raises(B.MoeError):
            group.run(z, x, x)
    with pytest.raises(ValueError, match="before run"):
        group.backward(x, x, z)
    group.run(z, x, x)
    group.backward(x, x, z)


def test_most_rows_of_a_product(lib):
    """Up to 2^31 - 256 rows: beyond, a run rounded up to whole tiles, or two
    stages past its end, would pass 32 bits."""
    none, n = [None] * 3, ctypes.c_size_t(0)
    calls = (lambda rows: lib.moe_expert_matmul(*none, None, 0, None, 1, rows, 16, 16, None, None, None, ctypes.byref(n), None),
             lambda rows: lib.moe_expert_matmul_dx(*none, 0, None, 1, rows, 16, 16, None, None, ctypes.byref(n), None),
             lambda rows: lib.moe_expert_matmul_dw(*none, 1, rows, 16, 16, 0, None, None, None, ctypes.byref(n), None))
    for call in calls:
        assert call(2 ** 31 - 256) == OK
        for rows in (2 ** 31 - 255, 2 ** 31 - 1, 2 ** 31, 2 ** 62):
            assert call(rows) == SHAPE


@pytest.mark.parametrize("dtype", [torch.float16, torch.float32, torch.uint8, torch.int32])
def test_rows_of_another_type_are_refused(dtype):
    """Two bytes do not make bf16: float16 is refused like the rest."""
    off, w, x, y = torch.zeros(3, dtype=torch.int32), bf16(2, 48, 32), bf16(4, 32), bf16(4, 48)
    other = lambda t: torch.zeros(t.shape, dtype=dtype)  # noqa: E731
    for a in ((other(x), off, w, None, 0, None, y), (x, off, other(w), None, 0, None, y), (x, off, w, None, 0, other(y), y),
              (x, off, w, None, 0, None, other(y)), (x, off, w, None, 0, None, y, other(y))):
        with pytest.raises(ValueError, match="bf16"):
            B.moe_expert_matmul(*a, stream=0)
    for a in ((other(y), off, w, 1, x, x), (y, off, other(w), 1, x, x), (y, off, w, 1, other(x), x), (y, off, w, 1, x, other(x))):
        with pytest.raises(ValueError, match="bf16"):
            B.moe_expert_matmul_dx(*a, stream=0)
    for a in ((other(y), x, off), (y, other(x), off)):
        with pytest.raises(ValueError, match="bf16"):
            B.moe_expert_matmul_dw(*a, torch.zeros(2, 48, 32), stream=0)
    with pytest.raises(ValueError, match="bf16"):
        ExpertMLP(other(w), bf16(2, 32, 48), B.MOE_ACT_SILU)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.int16, torch.uint16])
def test_bits_of_bf16_are_taken(dtype):
    """Past the types; the host's tensors are refused further in."""
    x, off, w = torch.zeros(4, 32).to(dtype), torch.zeros(3, dtype=torch.int32), torch.zeros(2, 48, 32).to(dtype)
    with pytest.raises(ValueError, match="device tensor"):
        B.moe_expert_matmul(x, off, w, None, 0, None, torch.zeros(4, 48).to(dtype), stream=0)


def test_rows_of_the_combine_gradient():
    """d_recv takes rows of 2 H bytes: a payload's own buffer, or another type,
    would be written past its end or left as garbage."""
    T, H, k = 4, 32, 2
    pos, w, d_out = torch.zeros(8, dtype=torch.int32), torch.zeros(4, 2), bf16(T, H)
    u8 = lambda *s: torch.zeros(*s, dtype=torch.uint8)  # noqa: E731

    def call(d_recv, d_out=d_out, recv=None, quant=0, scales=None, d_w=None):
        with pytest.raises(ValueError) as e:
            B.moe_combine_grad(d_out, recv, scales, quant, pos, w, T, H, k, d_recv, d_w, stream=0)
        return "device tensor" not in str(e.value)  # else past the rows' checks

    for bad in (torch.zeros(8, H), torch.zeros(8, H, dtype=torch.float16), torch.zeros(8, H, dtype=torch.int8), u8(8, H), u8(8 * H),
                u8(8, H // 2), bf16(8, H // 2), bf16(7 * H), u8(7 * 2 * H), bf16(8, H - 16)):
        assert call(bad), bad.shape
    for good in (bf16(8, H), bf16(5, H), bf16(8 * H), bf16(20, H), u8(8, 2 * H), u8(3, 2 * H), u8(8 * 2 * H), bf16(8, H).view(torch.int16),
                 u8(16, H)):
        assert not call(good), good.shape
    assert call(bf16(8, H), d_out=torch.zeros(T, H, dtype=torch.float16))
    d_w, scales = torch.zeros(T, k), torch.zeros(8)
    assert call(None, recv=torch.zeros(8, H), d_w=d_w)
    assert call(None, recv=bf16(8, H), quant=1, scales=scales, d_w=d_w)
    assert call(None, recv=torch.zeros(8, H, dtype=torch.int8), quant=1, d_w=d_w)  # no scales
    assert not call(None, recv=torch.zeros(8, H, dtype=torch.int8), quant=1, scales=scales, d_w=d_w)
    assert not call(None, recv=u8(8, 2 * H), d_w=d_w) and not call(None, recv=bf16(8, H), d_w=d_w)
