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


def test_workspaces_without_memory_of_their_own_are_refused():
    """An expanded or a strided tensor has more elements than adjacent bytes: a call would write over its neighbours."""
    x, stats, dw = torch.zeros(4000, 8), torch.zeros(4000, 2), torch.zeros(8)
    tokens, table = torch.zeros(64, dtype=torch.int64), torch.zeros(100, 8)
    need = max(fsp.layer_norm_backward_workspace_bytes(4000, 8), fsp.embedding_backward_workspace_bytes(100, 8, 64))
    for bad in (torch.zeros(1, dtype=torch.uint8).expand(need), torch.zeros(2 * need, dtype=torch.uint8)[::2], torch.zeros(need, 2, dtype=torch.uint8)[:, :1]):
        with pytest.raises(ValueError, match="workspace"):
            fsp.layer_norm_backward(x, stats, x, grad_weight=dw, workspace=bad)
        with pytest.raises(ValueError, match="workspace"):
            fsp.embedding_backward(tokens, x[:64], table, workspace=bad)
    good = torch.zeros(need, dtype=torch.uint8)
    for call in (lambda: fsp.layer_norm_backward(x, stats, x, grad_weight=dw, workspace=good), lambda: fsp.embedding_backward(tokens, x[:64], table, workspace=good)):
        with pytest.raises(fsp.FspError):   # past the checks of the arguments
            call()


def test_a_host_step_refuses_such_a_workspace():
    plan = fsp.plan_layout([(8, 8)], 2)
    work = torch.zeros(1, dtype=torch.uint8).expand(fsp.host_step_workspace_bytes(plan))
    with pytest.raises(ValueError, match="workspace"):
        state = [torch.zeros(plan.state_len_total) for _ in range(3)]
        fsp.sharded_step_host(plan, [torch.zeros(plan.full_len_padded) for _ in range(2)], *state,
                              [torch.zeros(plan.full_len_padded, dtype=torch.bfloat16) for _ in range(2)],
                              dict(lr=1e-3, beta1=0.9, beta2=0.95, eps=1e-8, weight_decay=0.1), 1, work)
