"""Experts in E4M3 codes on other streams than the one that their codes are made on."""
import pytest
import torch

from combine_fp32_router_amd.experts import ExpertMLP8
from test_gpu_fp8_products import SWIGLU, normal, offsets_of

pytestmark = pytest.mark.gpu

E, H, I, ROWS = 4, 528, 272, 300
SPIN = 50_000_000  # cycles: some ten ms or more, in which everything after is queued


def weights(seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return normal(g, E, 2 * I, H, scale=H ** -0.5), normal(g, E, H, I, scale=I ** -0.5)


def inputs():
    g = torch.Generator(device="cuda").manual_seed(7)
    return normal(g, ROWS, H), offsets_of([100, 0, 199, 1]), normal(g, ROWS, H)


def alone(w, x, off, d_out):
    mlp = ExpertMLP8(*w, SWIGLU, max_rows=ROWS, train=True)
    out, d_x = torch.empty_like(x), torch.empty_like(x)
    mlp.forward(x, off, out)
    mlp.backward(d_out, x, off, d_x, None)
    torch.cuda.synchronize()
    return out, d_x


@pytest.mark.parametrize("given", ["stream", "handle", "current"])
def test_calls_wait_for_the_codes(given):
    w, (x, off, d_out) = weights(1), inputs()
    want, d_want = alone(w, x, off, d_out)
    out, d_x, side = torch.zeros_like(x), torch.zeros_like(x), torch.cuda.Stream()
    torch.cuda.synchronize()
    torch.cuda._sleep(SPIN)
    mlp = ExpertMLP8(*w, SWIGLU, max_rows=ROWS, train=True)  # its codes come behind that
    busy = torch.cuda.current_stream()
    stream = dict(stream=side, handle=side.cuda_stream, current=None)[given]
    with torch.cuda.stream(side if given == "current" else busy):
        mlp.forward(x, off, out, stream=stream)
        mlp.backward(d_out, x, off, d_x, None, stream=stream)
    assert not busy.query()  # (or this has shown nothing)
    torch.cuda.synchronize()
    assert torch.equal(out, want) and torch.equal(d_x, d_want)


def test_calls_wait_for_codes_taken_again():
    first, second, (x, off, d_out) = weights(1), weights(2), inputs()
    want, d_want = alone(second, x, off, d_out)
    maker, side = torch.cuda.Stream(), torch.cuda.Stream()
    mlp = ExpertMLP8(*first, SWIGLU, max_rows=ROWS, train=True, stream=maker)
    out, d_x = torch.zeros_like(x), torch.zeros_like(x)
    mlp.forward(x, off, out)
    mlp.w_up.copy_(second[0]), mlp.w_down.copy_(second[1])
    torch.cuda.synchronize()
    with torch.cuda.stream(maker):
        torch.cuda._sleep(SPIN)
    mlp.quantize(maker)
    mlp.forward(x, off, out, stream=side)
    mlp.backward(d_out, x, off, d_x, None, stream=side)
    assert not maker.query()
    torch.cuda.synchronize()
    assert torch.equal(out, want) and torch.equal(d_x, d_want)


@pytest.mark.parametrize("handle", [False, True])
def test_made_on_another_stream(handle):
    """Behind what the current stream does with the weights and the buffers' memory."""
    w, late, (x, off, d_out) = weights(1), weights(2), inputs()
    want, d_want = alone(late, x, off, d_out)
    maker, out, d_x = torch.cuda.Stream(), torch.zeros_like(x), torch.zeros_like(x)
    torch.cuda.synchronize()
    torch.cuda._sleep(SPIN)
    w[0].copy_(late[0]), w[1].copy_(late[1])
    stream = maker.cuda_stream if handle else maker
    mlp = ExpertMLP8(*w, SWIGLU, max_rows=ROWS, train=True, stream=stream)
    mlp.forward(x, off, out, stream=stream)
    mlp.backward(d_out, x, off, d_x, None, stream=stream)
    assert not torch.cuda.current_stream().query()
    torch.cuda.synchronize()
    assert torch.equal(out, want) and torch.equal(d_x, d_want)


def test_captured_with_codes_of_another_stream():
    w, (x, off, d_out) = weights(1), inputs()
    want, d_want = alone(w, x, off, d_out)
    mlp = ExpertMLP8(*(t.clone() for t in w), SWIGLU, max_rows=ROWS, train=True)
    out, d_x = torch.zeros_like(x), torch.zeros_like(x)
    graph, again = torch.cuda.CUDAGraph(), torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        mlp.forward(x, off, out)
        mlp.backward(d_out, x, off, d_x, None)
    with torch.cuda.graph(again):
        mlp.quantize()
    other = weights(2)
    for w, (a, b) in ((w, (want, d_want)), (other, alone(other, x, off, d_out)), (w, (want, d_want))):
        mlp.w_up.copy_(w[0]), mlp.w_down.copy_(w[1])
        again.replay()
        for t in (out, d_x):
            t.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, a) and torch.equal(d_x, b)
        mlp.forward(x, off, out), mlp.backward(d_out, x, off, d_x, None)  # eager, beside the graphs
        torch.cuda.synchronize()
        assert torch.equal(out, a) and torch.equal(d_x, b)
