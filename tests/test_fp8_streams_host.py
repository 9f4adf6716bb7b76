"""In which order the E4M3 experts' calls reach their streams, on the host with
streams that only write down what they are given."""
import pytest
import torch

from combine_fp32_router_amd import binding as B
from combine_fp32_router_amd import experts
from test_fp8_experts_host import bf16, mlp


class Stream:
    capturing = False

    def __init__(self, handle, log):
        self.cuda_stream, self.log = handle, log

    def record_event(self):
        self.log.append((self.cuda_stream, "made"))
        return "made"

    def wait_event(self, event):
        self.log.append((self.cuda_stream, "waits"))


@pytest.fixture
def log(monkeypatch):
    log = []
    # (names of what may be missing: calls then fail in their order, not here)
    monkeypatch.setattr(B, "stream_handle", lambda s, device: s.cuda_stream, raising=False)
    monkeypatch.setattr(B, "stream_of", lambda s, device: s, raising=False)
    monkeypatch.setattr(experts, "_capturing", lambda s: s.capturing, raising=False)
    for name in ("moe_quant_weights", "moe_quant_rows", "moe_expert_matmul_fp8", "moe_expert_matmul_fp8_dx", "moe_expert_matmul_dw"):
        def call(*args, stream=None, **kw):
            s = stream or next(a for a in args if isinstance(a, Stream))
            log.append((s.cuda_stream, "launch"))

        monkeypatch.setattr(B, name, call)
    return log


def test_other_streams_wait_once(log):
    m, off, x = mlp(train=True), torch.zeros(5, dtype=torch.int32), bf16(8, 144)
    a, b, c = (Stream(i, log) for i in range(3))
    m.quantize(a)
    m.forward(x, off, bf16(8, 144), stream=a)
    assert (0, "waits") not in log
    m.forward(x, off, bf16(8, 144), stream=b)
    assert [what for s, what in log if s == 1][:2] == ["waits", "launch"]
    m.backward(x, x, off, bf16(8, 144), None, stream=c)
    assert [what for s, what in log if s == 2][:2] == ["waits", "launch"]
    m.forward(x, off, bf16(8, 144), stream=b)
    assert log.count((1, "waits")) == 1
    m.quantize(b)  # codes of another stream: all others wait again
    for s in (a, b, c):
        log.clear()
        m.forward(x, off, bf16(8, 144), stream=s)
        assert (log[0] == (s.cuda_stream, "waits")) == (s is not b)


def test_captured_calls_neither_record_nor_wait(log):
    m, off, x = mlp(), torch.zeros(5, dtype=torch.int32), bf16(8, 144)
    a, b = (Stream(i, log) for i in range(2))
    m.quantize(a)
    b.capturing = True
    log.clear()
    m.forward(x, off, bf16(8, 144), stream=b)
    m.quantize(b)
    assert {what for _, what in log} == {"launch"}
    b.capturing = False  # the same stream, eager: not behind the codes yet
    m.forward(x, off, bf16(8, 144), stream=b)
    assert (1, "waits") in log
