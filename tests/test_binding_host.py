"""What the binding hands out on the host, without a GPU."""

import ctypes

import pytest
import torch

from nvfp4_block_scaled_topk_gb300 import megamoe


@pytest.mark.parametrize("kind", [megamoe.Forward, megamoe.ShardForward])
def test_workspace_addresses_are_ctypes_pointers(kind):
    fwd = kind.__new__(kind)
    fwd.ws, fwd.ws_off = torch.empty(512, dtype=torch.uint8), 64
    assert isinstance(fwd.ws_ptr, ctypes.c_void_p)
    assert fwd.ws_ptr.value == fwd.ws.data_ptr() + 64


def test_streams_without_the_internal_function(monkeypatch):
    class Stream:
        cuda_stream = 1234

    monkeypatch.setattr(torch.cuda, "current_stream", lambda device: Stream)
    monkeypatch.delattr(torch._C, "_cuda_getCurrentRawStream", raising=False)
    assert megamoe._raw_stream_of()(0) == 1234
