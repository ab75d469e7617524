"""The bounded waits of the tensor-core path: a wait that nothing ends gives up, the status word says so, and the device goes on."""
import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("B,T", [(1, 40), (2, 700), (1, 3000), (40, 130)])
def test_wait_that_gives_up(d, B, T):
    import uncertainty_aware_delta_gb300 as kdn

    H = 2
    q, k, v, dO = (torch.randn(B, T, H, d, device="cuda").bfloat16() * d ** -0.5 for _ in range(4))
    l = torch.tensor([-0.01, -0.2], device="cuda")
    good = kdn.kdn_decay_forward(q, k, v, l)
    ws = torch.empty(kdn.decay_workspace_size(B, B * T, H, d, d), dtype=torch.uint8, device="cuda")
    kdn.kdn_decay_forward(q, k, v, l, workspace=ws, flags=kdn.KDN_FLAG_TIMEOUT_PROBE)
    assert kdn.kdn_read_device_status(ws) == 8
    back = torch.empty(kdn.decay_backward_workspace_size(B, B * T, H, d, d), dtype=torch.uint8, device="cuda")
    kdn.kdn_decay_backward(q, k, v, l, None, dO, workspace=back, flags=kdn.KDN_FLAG_TIMEOUT_PROBE)
    assert kdn.kdn_read_device_status(back) == 8
    again = kdn.kdn_decay_forward(q, k, v, l, workspace=ws)
    assert kdn.kdn_read_device_status(ws) == 0
    assert all(torch.equal(a, b) for a, b in zip(good, again))
