"""Where the binding makes its own buffers and on which device and stream it launches, without a GPU: tensors that say
they are on device 1 while device 0 is current, a library whose launching calls only note their arguments, and
stand-ins for torch's stream and device contexts that keep a journal."""

import contextlib

import pytest
import torch

from block_quantized_matmul_mq_amd import mq

RAW = {0: 1000, 1: 1001}      # the current stream's handle of each device
M, N, K, E, F, TOPK = 40, 100, 8192, 4, 256, 2


class OnDevice1(torch.Tensor):
    is_cuda = True

    def get_device(self):
        return 1


class Journal:
    def __init__(self):
        self.contexts, self.made, self.launches = [], [], []

    @contextlib.contextmanager
    def enter(self, what):
        self.contexts.append(what)
        yield
        self.contexts.pop()

    def here(self):
        return self.contexts[-1] if self.contexts else "current"


@pytest.fixture
def journal(monkeypatch):
    j = Journal()
    real = mq.load()

    class Library:
        def __getattr__(self, name):
            fn = getattr(real, name)
            if fn.restype is not mq.ctypes.c_int:
                return fn

            def launch(*args):
                stream = args[-1]
                device = next((c[1] for c in reversed(j.contexts) if c[0] == "device"), 0)
                j.launches.append((name, device, (stream.value or 0) if isinstance(stream, mq.ctypes.c_void_p) else stream))
                return 0
            return launch

    library = Library()
    monkeypatch.setattr(mq, "load", lambda: library)
    monkeypatch.setattr(mq, "_same_device", lambda fn, *tensors: None)
    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: 0, raising=False)
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda device: RAW[device], raising=False)
    monkeypatch.setattr(torch.cuda, "device", lambda d: j.enter(("device", d)))
    monkeypatch.setattr(torch.cuda, "stream", j.enter)

    def external(handle, device=None):
        assert handle != 0, "a stream object of handle 0 is a new stream, not the default one"
        return ("stream", handle)

    monkeypatch.setattr(torch.cuda, "ExternalStream", external)
    monkeypatch.setattr(torch.cuda, "default_stream", lambda device=None: ("stream", 0))

    def noted(make):
        def call(*a, **k):
            j.made.append(j.here())
            return make(*a, **k).as_subclass(OnDevice1)
        return call

    for name in ("empty", "zeros"):
        monkeypatch.setattr(torch, name, noted(getattr(torch, name)))
    monkeypatch.setattr(OnDevice1, "new_empty",
                        lambda self, shape, dtype=None: noted(torch.Tensor.new_empty)(self, shape, dtype=dtype), raising=False)
    return j


def tensor(*shape, dtype=torch.float32):
    return torch.ones(shape, dtype=dtype).as_subclass(OnDevice1)


def payload(qtype, rows, cols):
    return tensor(mq.weight_bytes(qtype, rows, cols), dtype=torch.uint8)


FEED_FORWARD = {
    "gemv_ep": lambda **k: mq.gemv_ep(payload(mq.Q4_K, N, K), mq.Q4_K, tensor(K), N, K, **k),
    "gemm_ep": lambda **k: mq.gemm_ep(payload(mq.Q4_K, N, K), mq.Q4_K, plane(), M, N, K, **k),
    "moe_route": lambda **k: mq.moe_route(tensor(M, K), tensor(E, K), TOPK, **k),
    "moe_ffn": lambda **k: mq.moe_ffn(payload(mq.Q4_K, E * F, K), payload(mq.Q4_K, E * F, K), mq.Q4_K, payload(mq.Q4_K, E * K, F),
                                      mq.Q4_K, tensor(M, K), tensor(M, TOPK, dtype=torch.int32), tensor(M, TOPK), E, F, **k),
}


def plane():
    return tensor(mq.act_bytes(M, K), dtype=torch.uint8)


@pytest.mark.parametrize("handle", [0, 77])
@pytest.mark.parametrize("name", FEED_FORWARD)
def test_buffers_are_made_on_the_given_stream(journal, name, handle):
    """Outputs and workspaces of a call that is given a stream handle, the default stream's 0 too."""
    FEED_FORWARD[name](stream=handle)
    assert journal.made and all(where == ("stream", handle) for where in journal.made), journal.made
    assert journal.launches == [("mq_" + name, 1, handle)]


@pytest.mark.parametrize("name", FEED_FORWARD)
def test_without_a_stream_the_devices_current_one(journal, name):
    FEED_FORWARD[name]()
    assert journal.made and all(where == "current" for where in journal.made)
    assert journal.launches == [("mq_" + name, 1, RAW[1])]


@pytest.mark.parametrize("handle", [0, 77])
def test_quantize_act_makes_its_plane_on_the_given_stream(journal, handle):
    mq.quantize_act(tensor(M, K), stream=handle)
    assert journal.made == [("stream", handle)]
    assert journal.launches == [("mq_quantize_act", 1, handle)]


PRODUCTS = {
    "gemv": lambda **k: mq.gemv(payload(mq.Q4_K, N, K), mq.Q4_K, tensor(K), N, K, **k),
    "gemm": lambda **k: mq.gemm(payload(mq.Q4_K, N, K), mq.Q4_K, plane(), M, N, K, **k),      # (K cut: with a workspace)
    "repack": lambda **k: mq.repack(payload(mq.Q4_K, N, K), mq.Q4_K, N, K, **k),
    "gemm_blockdots": lambda **k: mq.gemm_blockdots(payload(mq.Q4_K, N, K), mq.Q4_K, plane(), M, N, K, **k),
}


@pytest.mark.parametrize("handle", [0, 77])
@pytest.mark.parametrize("name", PRODUCTS)
def test_buffers_of_the_products_are_made_on_the_given_stream(journal, name, handle):
    """A workspace cleared on another stream than the product's may be cleared after the product starts."""
    PRODUCTS[name](stream=handle)
    assert journal.made and all(where == ("stream", handle) for where in journal.made), journal.made
    assert len(journal.made) == (2 if name == "gemm" else 1)
    assert journal.launches[0][2] == handle


@pytest.mark.parametrize("stream", [None, 0, 77])
@pytest.mark.parametrize("name", [*PRODUCTS, "gemm_noalloc", "quantize_act"])
def test_products_launch_on_the_tensors_device(journal, name, stream):
    """With another device current: on the tensors' device, on its current stream where none is given."""
    call = {**PRODUCTS, "quantize_act": lambda **k: mq.quantize_act(tensor(M, K), **k),
            "gemm_noalloc": lambda **k: mq.gemm_noalloc(payload(mq.Q4_K, N, K), mq.Q4_K, plane(), M, N, K, tensor(M, N), **k)}[name]
    call(stream=stream)
    entry = "mq_debug_gemm_blockdots" if name == "gemm_blockdots" else "mq_" + name
    assert journal.launches == [(entry, 1, RAW[1] if stream is None else stream)]
