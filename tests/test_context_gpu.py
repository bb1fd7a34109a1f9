"""Calls from a thread whose CUDA context another library changed between them."""
import ctypes
import threading

import pytest
import torch

import fsdp_sharded_mixed_pass_gb300 as fsp

from gpu_cases import HP, ensure_built

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    ensure_built()


def test_a_thread_left_without_a_context_is_served():
    cuda = ctypes.CDLL("libcuda.so.1")
    w = torch.randn(10, 16, device="cuda")
    ids = torch.tensor([3, 1, 4], device="cuda")
    out = torch.zeros(2, 3, 16, device="cuda")
    plan = fsp.plan_layout([(40, 16)], 1, "fsdp2")
    grad = torch.ones(plan.full_len_padded, device="cuda")
    params = torch.zeros(plan.full_len_padded, device="cuda", dtype=torch.bfloat16)
    state = [torch.zeros(plan.state_len_total, device="cuda") for _ in range(3)]
    torch.cuda.synchronize()
    failed = []

    def calls():
        try:
            for i in range(2):
                fsp.embedding(w, ids, out=out[i])
                assert cuda.cuCtxSetCurrent(None) == 0
                fsp.sharded_step(plan, [grad], *state, [params], HP, i + 1)
                assert cuda.cuCtxSetCurrent(None) == 0
        except BaseException as e:   # (to the test's own thread)
            failed.append(e)
    t = threading.Thread(target=calls)
    t.start()
    t.join()
    torch.cuda.synchronize()
    assert not failed, failed
    assert torch.equal(out[0], w[ids]) and torch.equal(out[1], w[ids])
    n = 40 * 16
    assert float(state[1][:n].min()) > 0 and float(params[:n].float().max()) < 0
