"""Windows as long as an int holds: the same as none."""
import pytest
import torch

from test_prompt_attention import _inputs

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("window", [2 ** 31 - 1, 2 ** 31 - 100, 2 ** 30])
@pytest.mark.parametrize("lq,lk,H,hkv,d,io", [
    ([200], [100], 2, 1, 64, "bf16"), ([200], [100], 2, 2, 128, "bf16"), ([200], [100], 2, 1, 64, "f32"),
    ([400, 30, 5], [90, 30, 700], 4, 2, 64, "bf16"), ([400, 30, 5], [90, 30, 700], 4, 2, 32, "bf16"),
    ([1], [6000], 2, 1, 128, "bf16"), ([257, 2], [7000, 6700], 3, 1, 128, "bf16"), ([250] * 16, [4000] * 16, 4, 1, 64, "bf16"),
    ([40] * 40, [20] * 40, 2, 1, 64, "bf16")])
def test_long_windows(lq, lk, H, hkv, d, io, window):
    import uncertainty_aware_delta_gb300 as kdn

    q, k, v, cu_q, cu_k = _inputs(lq, lk, H, hkv, d, io)
    want = kdn.kdn_prompt_attention(q, k, v, cu_q, cu_k)
    out = torch.full_like(q, 7.0), torch.full(q.shape[:2], 7.0, device="cuda")
    kdn.kdn_prompt_attention(q, k, v, cu_q, cu_k, window=window, out=out)
    assert torch.equal(out[0], want[0]) and torch.equal(out[1], want[1])
