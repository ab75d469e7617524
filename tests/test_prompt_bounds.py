"""Bounds out of range past the sequences whose rows a call has room for."""
import pytest
import torch

from test_prompt_attention import _inputs

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("d,io", [(32, "bf16"), (64, "f32"), (64, "bf16"), (128, "bf16")])
@pytest.mark.parametrize("n", [33, 100, 3000])
def test_last_bound(n, d, io):
    import uncertainty_aware_delta_gb300 as kdn

    # 32 sequences of one token, then none; the last one's bounds run backwards
    lens = [1] * 32 + [0] * (n - 32)
    q, k, v, cu, _ = _inputs(lens, lens, 2, 1, d, io)
    ws = torch.empty(kdn.prompt_attention_workspace_size(n, 32, 2, 1, d, 1 if io == "bf16" else 0), dtype=torch.uint8, device="cuda")
    want, _ = kdn.kdn_prompt_attention(q, k, v, cu, cu, workspace=ws)
    assert kdn.kdn_read_device_status(ws) == 0
    back = cu.clone()
    back[-1] = 31
    for cu_q, cu_k in ((back, cu), (cu, back)):
        o, _ = kdn.kdn_prompt_attention(q, k, v, cu_q, cu_k, workspace=ws)
        assert kdn.kdn_read_device_status(ws) == 9
        assert torch.equal(o, want)
