"""A raw stream handle says nothing about its device: what a layer allocates for a call on it has to be allocated for
that stream on the tensors' device, whatever the current device is. Checked without a GPU: torch's stream
classes are replaced by recorders, and the calls end at the refusal of CPU tensors."""
import contextlib

import pytest
import torch

import quantized_gemm_moe_b200 as qe


@pytest.fixture
def made(monkeypatch):
    """The (handle, device) of every external stream that is made, and those that were current at an allocation."""
    log, current, at = [], [], []

    class External:
        def __init__(self, handle, like):
            self.cuda_stream, self.device = handle, like.device
            log.append((handle, like.device))

    @contextlib.contextmanager
    def stream(s):
        current.append(s)
        yield
        current.pop()

    scratch = qe._scratch

    def record(*a):
        at.append(current[-1] if current else None)
        return scratch(*a)

    monkeypatch.setattr(qe, "_external", External)
    monkeypatch.setattr(torch.cuda, "stream", stream)
    monkeypatch.setattr(qe, "_scratch", record)
    from quantized_gemm_moe_b200 import build
    build.build()
    return log, at


def tensors():
    X = torch.zeros(4, 256, dtype=torch.bfloat16)
    layer = qe.Mx4Layer(torch.zeros(8, 128, dtype=torch.uint8), torch.zeros(1024, dtype=torch.uint8))
    return X, layer


def calls():
    X, layer = tensors()
    codes, scales = torch.zeros(4, 128, dtype=torch.uint8), torch.zeros(1024, dtype=torch.uint8)
    c8, sa = torch.zeros(4, 256, dtype=torch.int8), torch.zeros(4)
    some = torch.zeros(16, dtype=torch.uint8)
    qel = qe.QELayer(qe.make_desc(256, 256, 64, 4, 8, 8, 4, 4), some, some, some, some)
    return {"forward": lambda s: layer.forward(X, stream=s), "forward_codes": lambda s: layer.forward_codes(codes, scales, stream=s),
            "from_float": lambda s: qe.Mx4Layer.from_float(X, stream=s),
            "qe forward_codes": lambda s: qel.forward_codes(X, c8, sa, stream=s)}


@pytest.mark.parametrize("name", list(calls()))
def test_raw_handle_belongs_to_the_tensors_device(made, name):
    log, at = made
    with pytest.raises(qe.QEError):  # CPU tensors are refused behind the allocations
        calls()[name](0x7000)
    assert log == [(0x7000, torch.device("cpu"))]
    assert at and all(s is not None and s.cuda_stream == 0x7000 for s in at)


@pytest.mark.parametrize("name", list(calls()))
def test_stream_object_is_taken_as_it_is(made, name):
    log, at = made

    class Own:
        cuda_stream, device = 0x8000, torch.device("cpu")

    own = Own()
    with pytest.raises(qe.QEError):
        calls()[name](own)
    assert log == [] and at and all(s is own for s in at)


def test_raw_handle_and_a_cpu_tensor_are_refused():
    X, layer = tensors()
    with pytest.raises(qe.QEError):
        layer.forward(X, stream=0x7000)


@pytest.mark.gpu
def test_external_stream_carries_the_device():
    X = torch.zeros(1, device="cuda")
    handle = torch.cuda.Stream().cuda_stream
    made = qe._external(handle, X)
    assert made.cuda_stream == handle and made.device == X.device
