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
    monkeypatch.setattr(t, "_CURRENT_DEVICE", lambda: 0, raising=False)


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
