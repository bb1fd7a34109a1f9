"""Calls of the block's operators that the binding refuses, on the host: tensors of the CPU stand in for the current device's."""
import pytest

import fsdp_sharded_mixed_pass_gb300 as fsp
from fsdp_sharded_mixed_pass_gb300 import fsp as B
from fsdp_sharded_mixed_pass_gb300 import ops

torch = pytest.importorskip("torch")


@pytest.fixture(autouse=True)
def on_the_host(monkeypatch):
    import os
    if not os.path.exists(B.LIB_PATH):
        from fsdp_sharded_mixed_pass_gb300 import build
        build.build()
    ops._ready()
    monkeypatch.setattr(ops, "_current", lambda: -1)   # where the CPU's tensors say they are
    monkeypatch.setattr(ops, "_handle", lambda stream, device: None)


def test_a_call_beyond_64_bits_is_refused():
    """2^64 would give call 0's masks, 2^63 those of -2^63."""
    x = torch.zeros(4, 8)
    for call in (1 << 63, 1 << 64, -(1 << 63) - 1, 1 << 80):
        with pytest.raises(ValueError, match="call"):
            fsp.dropout(x, 0.5, 1, call)
        with pytest.raises(ValueError, match="call"):
            fsp.dropout_backward(x, 0.5, 1, call)
    for call in ((1 << 63) - 1, -(1 << 63), 0):
        with pytest.raises(fsp.FspError):   # past the checks of the arguments: this memory is not the device's
            fsp.dropout(x, 0.5, 1, call)
