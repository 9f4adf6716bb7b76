"""Refusals of the norm, of the quantisers and of the E4M3 products, on the host:
nothing is launched, so made-up addresses stand for device arrays."""
import ctypes

import pytest
import torch

from combine_fp32_router_amd import binding as B

OK, NULL, SHAPE, ALIGN, WORKSPACE, HIP, ALIAS = range(7)


@pytest.fixture(scope="module")
def lib():
    return B.load()


def at(i):
    return ctypes.c_void_p(0x100000 * (i + 1))


def call(fn, defaults, **other):
    args = dict(defaults)
    assert set(other) <= set(args)
    args.update(other)
    return fn(*args.values())


NORM = dict(x=at(0), residual=at(1), weight=at(2), eps=1e-6, T=4, H=64, sum=at(3), y=at(4), block=128, codes=at(5),
            scales=at(6), stream=None)


@pytest.mark.parametrize("other,status", [
    (dict(T=-1), SHAPE), (dict(T=1 << 31), SHAPE), (dict(H=8), SHAPE), (dict(H=24), SHAPE), (dict(H=65552), SHAPE),
    (dict(eps=-1.0), SHAPE), (dict(eps=float("nan")), SHAPE), (dict(block=64), SHAPE), (dict(x=None), NULL),
    (dict(y=None, codes=None), NULL), (dict(scales=None), NULL), (dict(x=0x100008), ALIGN), (dict(weight=0x100004), ALIGN),
    (dict(codes=0x100008), ALIGN), (dict(scales=0x100002), ALIGN), (dict(y=at(3)), ALIAS), (dict(codes=at(0)), ALIAS),
    (dict(codes=at(4)), ALIAS), (dict(T=0, x=None), OK)])
def test_norm(lib, other, status):
    assert call(lib.moe_add_norm, NORM, **other) == status


GRAD = dict(d_y=at(0), d_sum=at(1), sum=at(2), weight=at(3), eps=1e-6, T=4, H=64, d_x=at(4), d_weight=at(5), accumulate=0,
            workspace=at(6), workspace_bytes=None, stream=None)


@pytest.mark.parametrize("other,status", [
    (dict(T=-1), SHAPE), (dict(H=40), SHAPE), (dict(eps=-1.0), SHAPE), (dict(accumulate=2), SHAPE), (dict(d_y=None), NULL),
    (dict(sum=None), NULL), (dict(d_x=None), NULL), (dict(d_sum=0x100002), ALIGN), (dict(d_weight=0x100004), ALIGN),
    (dict(workspace=0x100080), ALIGN)])
def test_norm_grad(lib, other, status):
    n = ctypes.c_size_t(1 << 30)
    assert call(lib.moe_add_norm_grad, GRAD, workspace_bytes=ctypes.byref(n), **other) == status


def test_norm_grad_workspace(lib):
    n = ctypes.c_size_t(0)
    assert call(lib.moe_add_norm_grad, GRAD, workspace=None, workspace_bytes=ctypes.byref(n)) == OK
    need = n.value
    assert need >= 64 * 4 and need == B.add_norm_grad_workspace_bytes(4, 64)
    n = ctypes.c_size_t(need - 1)
    assert call(lib.moe_add_norm_grad, GRAD, workspace_bytes=ctypes.byref(n)) == WORKSPACE
    assert call(lib.moe_add_norm_grad, GRAD) == WORKSPACE
    assert call(lib.moe_add_norm_grad, GRAD, workspace=None) == WORKSPACE
    assert call(lib.moe_add_norm_grad, GRAD, T=0, d_weight=None, workspace=None) == OK
    for T in (1, 3, 1000, 1 << 20, (1 << 31) - 1):  # bounded, whatever T
        assert B.add_norm_grad_workspace_bytes(T, 7168) <= 64 << 20


ROWS = dict(x=at(0), offsets=at(1), E=2, max_rows=4, H=64, halves=1, codes=at(2), scales=at(3), stream=None)


@pytest.mark.parametrize("other,status", [
    (dict(halves=0), SHAPE), (dict(halves=3), SHAPE), (dict(H=16, halves=2), SHAPE), (dict(H=48, halves=2), SHAPE),
    (dict(H=131072), SHAPE), (dict(H=131072 + 32, halves=2), SHAPE), (dict(E=0), SHAPE), (dict(E=1025), SHAPE),
    (dict(max_rows=-1), SHAPE), (dict(max_rows=(1 << 31) - 255), SHAPE), (dict(x=None), NULL), (dict(codes=None), NULL),
    (dict(scales=None), NULL), (dict(x=0x100008), ALIGN), (dict(offsets=0x100002), ALIGN), (dict(codes=at(0)), ALIAS),
    (dict(max_rows=0), OK)])
def test_quant_rows(lib, other, status):
    assert call(lib.moe_quant_rows, ROWS, **other) == status


WEIGHTS = dict(w=at(0), E=2, N=64, K=64, halves=1, codes=at(1), scales=at(2), codes_t=at(3), scales_t=at(4), stream=None)


@pytest.mark.parametrize("other,status", [
    (dict(halves=0), SHAPE), (dict(E=0), SHAPE), (dict(N=24), SHAPE), (dict(K=0), SHAPE), (dict(K=65552), SHAPE),
    (dict(E=1024, N=65536, K=65536), SHAPE), (dict(w=None), NULL), (dict(codes_t=None), NULL), (dict(scales_t=None), NULL),
    (dict(w=0x100008), ALIGN), (dict(codes_t=0x100008), ALIGN), (dict(codes=at(0)), ALIAS), (dict(codes_t=at(1)), ALIAS),
    (dict(scales_t=at(2)), ALIAS)])
def test_quant_weights(lib, other, status):
    assert call(lib.moe_quant_weights, WEIGHTS, **other) == status


PRODUCT = dict(x=at(0), x_scales=at(1), x_scale_cols=2, offsets=at(2), w=at(3), w_scales=at(4), bias=at(5), act=4,
               residual=at(6), E=2, max_rows=8, K=144, N=64, out=at(7), codes=at(8), scales=at(9), preact=at(10),
               workspace=None, workspace_bytes=None, stream=None)


@pytest.mark.parametrize("other,status", [
    (dict(E=0), SHAPE), (dict(E=1025), SHAPE), (dict(max_rows=-1), SHAPE), (dict(max_rows=(1 << 31) - 255), SHAPE),
    (dict(K=24), SHAPE), (dict(N=8), SHAPE), (dict(act=5), SHAPE), (dict(act=-1), SHAPE), (dict(x_scale_cols=3), SHAPE),
    (dict(x_scale_cols=0), SHAPE), (dict(max_rows=1 << 30, N=65536), SHAPE), (dict(x=None), NULL), (dict(x_scales=None), NULL),
    (dict(offsets=None), NULL), (dict(w_scales=None), NULL), (dict(out=None, codes=None), NULL), (dict(scales=None), NULL),
    (dict(x=0x100008), ALIGN), (dict(bias=0x100004), ALIGN), (dict(scales=0x100001), ALIGN), (dict(out=at(0)), ALIAS),
    (dict(codes=at(0)), ALIAS), (dict(codes=at(7)), ALIAS), (dict(preact=at(7)), ALIAS), (dict(preact=at(6)), ALIAS),
    (dict(scales=at(1)), ALIAS), (dict(max_rows=0), OK)])
def test_product(lib, other, status):
    assert call(lib.moe_expert_matmul_fp8, PRODUCT, **other) == status


DX = dict(dy=at(0), dy_scales=at(1), offsets=at(2), w_t=at(3), w_t_scales=at(4), halves=1, act=4, preact=at(5), E=2,
          max_rows=8, K=144, N=64, dx=at(6), codes=at(7), scales=at(8), workspace=None, workspace_bytes=None, stream=None)


@pytest.mark.parametrize("other,status", [
    (dict(E=0), SHAPE), (dict(halves=3), SHAPE), (dict(K=24), SHAPE), (dict(N=65552), SHAPE), (dict(act=9), SHAPE),
    (dict(dy=None), NULL), (dict(w_t_scales=None), NULL), (dict(dx=None, codes=None), NULL), (dict(preact=None), NULL),
    (dict(scales=None), NULL), (dict(dx=0x100008), ALIGN), (dict(dx=at(0)), ALIAS), (dict(codes=at(6)), ALIAS),
    (dict(codes=at(5)), ALIAS), (dict(scales=at(4)), ALIAS), (dict(max_rows=0), OK)])
def test_dx(lib, other, status):
    assert call(lib.moe_expert_matmul_fp8_dx, DX, **other) == status


def test_binding_refuses():
    """Wrong types and shapes, before the library is asked."""
    f, h, u = torch.zeros(4, 2), torch.zeros(4, 256, dtype=torch.bfloat16), torch.zeros(4, 256, dtype=torch.uint8)
    off = torch.zeros(3, dtype=torch.int32)
    w, ws = torch.zeros(2, 64, 256, dtype=torch.uint8), torch.zeros(2, 1, 2)
    out = torch.zeros(4, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="codes and scales"):
        B.moe_add_norm(h, None, None, 1e-6, None, None, u)
    with pytest.raises(ValueError, match="scales: expected shape"):
        B.moe_add_norm(h, None, None, 1e-6, None, None, u, torch.zeros(4, 3))
    with pytest.raises(ValueError, match="E4M3"):
        B.moe_add_norm(h, None, None, 1e-6, None, None, torch.zeros(4, 256, dtype=torch.int8), f)
    with pytest.raises(ValueError, match="weight"):
        B.moe_add_norm(h, None, torch.zeros(256, dtype=torch.bfloat16), 1e-6, None, h)
    with pytest.raises(ValueError, match="d_x"):
        B.moe_add_norm_grad(h, None, h, None, 1e-6, torch.zeros(4, 128, dtype=torch.bfloat16))
    with pytest.raises(ValueError, match="halves"):
        B.moe_quant_rows(h, u, f, halves=3)
    with pytest.raises(ValueError, match="scales"):
        B.moe_quant_rows(h, u, f, halves=2)
    with pytest.raises(ValueError, match="come together"):
        B.moe_quant_weights(w.to(torch.bfloat16), w, ws, codes_t=torch.zeros(2, 256, 64, dtype=torch.uint8))
    with pytest.raises(ValueError, match="x_scales"):
        B.moe_expert_matmul_fp8(u, torch.zeros(4, 3), off, w, ws, None, 0, None, out)
    with pytest.raises(ValueError, match="w_scales"):
        B.moe_expert_matmul_fp8(u, f, off, w, torch.zeros(2, 2, 2), None, 0, None, out)
    with pytest.raises(ValueError, match="offsets"):
        B.moe_expert_matmul_fp8(u, f, off[:2], w, ws, None, 0, None, out)
    with pytest.raises(ValueError, match="needs preact"):
        B.moe_expert_matmul_fp8_dx(u, f, off, torch.zeros(2, 64, 256, dtype=torch.uint8), ws, 2, None, out)
    with pytest.raises(ValueError, match="device tensor"):
        B.moe_expert_matmul_fp8(u, f, off, w, ws, None, 0, None, out)
