"""The bounded waits of the tcgen05 prompt kernel, driven without a fault (see test_timeout_probe.py)."""
import pytest

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("d,H,hkv", [(128, 4, 2), (64, 3, 3)])
def test_timeout_is_reported_and_recovered(d, H, hkv):
    import torch
    import uncertainty_aware_delta_gb300 as kdn

    g = torch.Generator().manual_seed(1)
    q, k, v = (torch.randn((700, h, d), generator=g).to(torch.bfloat16).cuda() for h in (H, hkv, hkv))
    cu = torch.tensor([0, 600, 700], dtype=torch.int32, device="cuda")
    ws = torch.empty(kdn.prompt_attention_workspace_size(2, 700, H, hkv, d), dtype=torch.uint8, device="cuda")
    want = kdn.kdn_prompt_attention(q, k, v, cu)
    kdn.kdn_prompt_attention(q, k, v, cu, workspace=ws, flags=kdn.KDN_FLAG_TIMEOUT_PROBE)
    assert kdn.kdn_read_device_status(ws) == 8
    got = kdn.kdn_prompt_attention(q, k, v, cu, workspace=ws)
    assert kdn.kdn_read_device_status(ws) == 0
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
