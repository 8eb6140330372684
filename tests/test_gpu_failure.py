"""Failure detection on the GPU without a fault: bounded waits that expire set
a status the host reads, and the context stays usable afterwards."""
import pytest
import torch

import moe_expert_layer_06_gb300 as m

pytestmark = pytest.mark.gpu


def test_expired_wait_is_reported_and_context_survives():
    m.moe_set_wait_limit_ns(2_000_000)  # 2 ms
    try:
        m.moe_debug_expire_wait()
        assert m.moe_check_status() == m.MOE_ERR_DEVICE_TIMEOUT
        assert "wait" in m.last_error()
        assert m.moe_check_status() == m.MOE_OK  # read clears it
    finally:
        m.moe_set_wait_limit_ns(2_000_000_000)
    a = torch.arange(1000, device="cuda", dtype=torch.float32)
    assert float(a.sum().item()) == 499500.0


@pytest.mark.parametrize("limit_ns", [1_000, 200_000, 20_000_000])
def test_a_group_of_warps_gives_up_together(limit_ns):
    """Half of the probe's threads wait for what never comes, half for what has come: the vote that the
    adapter kernels' workers take makes all of them give up, none stays behind in a barrier, and the
    next kernels run as ever."""
    p = m.Adapter(264, 392, 3, 16)
    g = torch.Generator().manual_seed(1)
    x, w, a, b = ((torch.randn(*s, generator=g) * 0.1).to(torch.bfloat16).cuda()
                  for s in ((300, 264), (392, 264), (3, 16, 264), (3, 392, 16)))
    of = torch.randint(-1, 3, (300,), generator=g).int().cuda()
    ws = torch.empty(m.moe_adapter_workspace_size(p, 300), dtype=torch.uint8, device="cuda")
    outs = [torch.empty(300, 392, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    m.moe_adapter_project(p, 300, x, w, a, b, None, of, outs[0], None, ws)
    assert m.moe_check_status() == m.MOE_OK
    m.moe_set_wait_limit_ns(limit_ns)
    try:
        for _ in range(5):
            m.moe_debug_expire_wait()
            assert m.moe_check_status() == m.MOE_ERR_DEVICE_TIMEOUT
    finally:
        m.moe_set_wait_limit_ns(2_000_000_000)
    m.moe_adapter_project(p, 300, x, w, a, b, None, of, outs[1], None, ws)
    assert m.moe_check_status() == m.MOE_OK and torch.equal(outs[0], outs[1])
