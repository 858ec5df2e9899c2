"""What the Python calls of the attention sublayer refuse by themselves (no GPU)."""

import pytest
import torch

from tensor_comm_gemm_gb300 import build as tb
from tensor_comm_gemm_gb300 import tpoverlap as t

BF16 = torch.bfloat16


@pytest.fixture(scope="module", autouse=True)
def lib():
    tb.build()
    return t.lib()


class OnDevice:
    """A tensor as the binding sees it, on a device that this machine lacks."""

    is_cuda = True

    def __init__(self, device, *shape, dtype=BF16):
        self.shape, self.dtype, self.device = torch.Size(shape), dtype, device
        self.like = torch.empty(shape, dtype=dtype, device="meta")

    def get_device(self):
        return self.device

    def stride(self):
        return self.like.stride()

    def numel(self):
        return self.like.numel()

    def is_contiguous(self):
        return self.like.is_contiguous()

    def data_ptr(self):
        return 0x10000


@pytest.fixture
def cuda_tensors(monkeypatch):
    """Calls get as far as the library, which refuses the handle (None) last."""
    monkeypatch.setattr(t, "_RAW_STREAM", lambda device: 0)
    monkeypatch.setattr(t, "_CURRENT_DEVICE", lambda: 0)


def attention(**kw):
    a = dict(q=OnDevice(0, 5, 4, 16), k=OnDevice(0, 9, 2, 16), v=OnDevice(0, 9, 2, 16), out=OnDevice(0, 5, 4, 16))
    a.update(kw)
    t.tpo_attention(None, **a)


def attention_bwd(**kw):
    a = dict(dout=OnDevice(0, 5, 4, 16), q=OnDevice(0, 5, 4, 16), k=OnDevice(0, 9, 2, 16), v=OnDevice(0, 9, 2, 16),
             out=OnDevice(0, 5, 4, 16), lse=OnDevice(0, 5, 4, dtype=torch.float32), dq=OnDevice(0, 5, 4, 16),
             dk=OnDevice(0, 9, 2, 16), dv=OnDevice(0, 9, 2, 16))
    a.update(kw)
    t.tpo_attention_bwd(None, **a)


def rotary(**kw):
    a = dict(x=OnDevice(0, 5, 4, 16), table=OnDevice(0, 8, dtype=torch.int64), y=OnDevice(0, 5, 4, 16))
    a.update(kw)
    t.tpo_rotary(None, **a)


def test_heads_of_no_elements_are_refused_by_the_library(cuda_tensors):
    """Also where the scale follows from their number."""
    q, k = OnDevice(0, 5, 4, 0), OnDevice(0, 9, 2, 0)
    with pytest.raises(t.TpoError, match="dim=0"):
        attention(q=q, k=k, v=k, out=q)
    with pytest.raises(t.TpoError, match="dim=0"):
        attention_bwd(dout=q, q=q, k=k, v=k, out=q, dq=q, dk=k, dv=k)


def test_calls_on_one_device_get_to_the_library(cuda_tensors):
    starts = OnDevice(0, 2, dtype=torch.int32)
    for call in (attention, attention_bwd):
        with pytest.raises(t.TpoError, match="handle"):
            call(q_start=starts, k_start=starts, k_len=OnDevice(0, 1, dtype=torch.int32))
    with pytest.raises(t.TpoError, match="handle"):
        rotary(pos=OnDevice(0, 5, dtype=torch.int32))


def int32(*shape):
    return lambda device: OnDevice(device, *shape, dtype=torch.int32)


Q, K = (lambda device: OnDevice(device, 5, 4, 16)), (lambda device: OnDevice(device, 9, 2, 16))
LSE = lambda device: OnDevice(device, 5, 4, dtype=torch.float32)  # noqa: E731
TABLE = lambda device: OnDevice(device, 8, dtype=torch.int64)  # noqa: E731


@pytest.mark.parametrize("call,name,make", [
    (attention, "q", Q), (attention, "k", K), (attention, "v", K), (attention, "out", Q), (attention, "lse", LSE),
    (attention, "q_start", int32(2)), (attention, "k_start", int32(2)), (attention, "k_len", int32(1)),
    (attention_bwd, "dout", Q), (attention_bwd, "q", Q), (attention_bwd, "k", K), (attention_bwd, "v", K),
    (attention_bwd, "out", Q), (attention_bwd, "lse", LSE), (attention_bwd, "dq", Q), (attention_bwd, "dk", K),
    (attention_bwd, "dv", K), (attention_bwd, "q_start", int32(2)), (rotary, "x", Q), (rotary, "table", TABLE),
    (rotary, "y", Q), (rotary, "pos", int32(5)), (rotary, "rows", int32(5))])
def test_tensors_of_another_device_are_refused(cuda_tensors, call, name, make):
    """The kernels run on the current device: another's memory would fault there."""
    with pytest.raises(t.TpoError, match="%s is on device 1, the current device is 0" % name):
        call(**{name: make(1)})
