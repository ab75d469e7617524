"""Few prompts with many keys, whose rows are split over the keys and joined, against fp64 row by row."""
import pytest
import torch

import attention_oracle as ref
from test_prompt_attention import _expect, _inputs, _np, _run

pytestmark = pytest.mark.gpu

CASES = [([130, 1, 300, 0, 77], [2130, 4000, 300, 40, 2500], 4, 2, 64), ([1], [6000], 2, 1, 128), ([257, 2], [1800, 2100], 3, 1, 128),
         ([64, 500, 3], [3000, 20, 2], 2, 2, 64), ([200] * 5 + [1] * 27, [1100] * 5 + [1700] * 27, 2, 1, 128)]


@pytest.mark.parametrize("lq,lk,H,hkv,d", CASES)
@pytest.mark.parametrize("window", [0, 1, 1600])
def test_long_keys(lq, lk, H, hkv, d, window):
    _run(lq, lk, H, hkv, d, "bf16", window)


@pytest.mark.parametrize("d,hkv", [(128, 1), (64, 2)])
def test_rising_scores_and_special_values(d, hkv):
    """Later keys dominate by far, and values that are not finite stand where some rows see them."""
    import uncertainty_aware_delta_gb300 as kdn

    q, k, v, cu_q, cu_k = _inputs([140, 9], [3000, 2600], 2, hkv, d, "bf16", gain=1.0)
    k *= (1 + 3 * torch.arange(k.shape[0], device="cuda") / k.shape[0]).to(k.dtype)[:, None, None]
    v[2950, :, 5] = float("inf")
    v[2940, :, 6] = float("nan")
    v[3000 + 2598, :, 7] = -float("inf")
    v[2999, :, 8] = float("inf")
    want = _expect(q, k, v, cu_q, cu_k, 0)
    o, lse = kdn.kdn_prompt_attention(q, k, v, cu_q, cu_k)
    got = _np(o)
    for at, want_o in enumerate(want[0]):
        for h in range(2):
            special = ~(abs(want_o[h]) < float("inf"))
            assert ((got[at, h] == want_o[h]) | (got[at, h] != got[at, h]) & (want_o[h] != want_o[h]))[special].all()
    keep = [i for i in range(d) if i not in (5, 6, 7, 8)]
    ref.check(got[..., keep], _np(lse), (want[0][..., keep], want[1], want[2][..., keep], want[3]), "bf16")


def test_workspace_reused_and_invalid_bounds():
    import uncertainty_aware_delta_gb300 as kdn

    q, k, v, cu_q, cu_k = _inputs([100, 30], [2000, 2500], 4, 2, 64, "bf16")
    ws = torch.randint(0, 256, (kdn.prompt_attention_workspace_size(2, 130, 4, 2, 64),), dtype=torch.uint8, device="cuda")
    a = kdn.kdn_prompt_attention(q, k, v, cu_q, cu_k, workspace=ws)
    b = kdn.kdn_prompt_attention(q, k, v, cu_q, cu_k, workspace=ws)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    bad = cu_k.clone()
    bad[1] = 9000     # past the keys: both sequences are left out
    o = torch.full_like(q, 3.0)
    kdn.kdn_prompt_attention(q, k, v, cu_q, bad, workspace=ws, out=(o, torch.empty_like(a[1])))
    assert kdn.kdn_read_device_status(ws) == 9 and bool((o == 3).all())


@pytest.mark.parametrize("lq,lk,H,hkv,d", [([130, 1, 300, 0, 77], [6130, 9000, 300, 40, 7500], 2, 1, 64), ([1], [9001], 2, 2, 128),
                                           ([257, 2], [7000, 6700], 3, 1, 128), ([3, 140], [100, 20000], 2, 1, 128)])
@pytest.mark.parametrize("window", [0, 6000])
def test_longer_keys(lq, lk, H, hkv, d, window):
    _run(lq, lk, H, hkv, d, "bf16", window)


@pytest.mark.parametrize("d,hkv", [(128, 1), (64, 2)])
def test_special_values_in_parts(d, hkv):
    import uncertainty_aware_delta_gb300 as kdn

    q, k, v, cu_q, cu_k = _inputs([140, 9], [9000, 7600], 2, hkv, d, "bf16", seed=4)
    k *= (1 + 3 * torch.arange(k.shape[0], device="cuda") / k.shape[0]).to(k.dtype)[:, None, None]
    v[8950, :, 5] = float("inf")      # in the masked tiles, seen by the last rows
    v[8940, :, 6] = float("nan")
    v[9000 + 7598, :, 7] = -float("inf")
    v[8999, :, 8] = float("inf")
    want = _expect(q, k, v, cu_q, cu_k, 0)
    o, lse = kdn.kdn_prompt_attention(q, k, v, cu_q, cu_k)
    got = _np(o)
    for c in (5, 6, 7, 8):
        a, b = got[..., c], want[0][..., c]
        odd = ~(abs(b) < float("inf"))
        assert odd.any() and ((a == b) | (a != a) & (b != b))[odd].all()
    keep = [i for i in range(d) if i not in (5, 6, 7, 8)]
    ref.check(got[..., keep], _np(lse), (want[0][..., keep], want[1], want[2][..., keep], want[3]), "bf16")
    ws = torch.randint(0, 256, (kdn.prompt_attention_workspace_size(2, 149, 2, hkv, d),), dtype=torch.uint8, device="cuda")
    again = kdn.kdn_prompt_attention(q, k, v, cu_q, cu_k, workspace=ws)
    assert torch.equal(again[0].nan_to_num(), o.nan_to_num()) and torch.equal(again[1], lse)
    with pytest.raises(ValueError):
        kdn.kdn_prompt_attention(q, k, v, cu_q, cu_k, workspace=ws[:-1])


def test_timeout_of_parts():
    import uncertainty_aware_delta_gb300 as kdn

    q, k, v, cu_q, cu_k = _inputs([3], [9000], 4, 2, 128, "bf16")
    ws = torch.empty(kdn.prompt_attention_workspace_size(1, 3, 4, 2, 128), dtype=torch.uint8, device="cuda")
    want = kdn.kdn_prompt_attention(q, k, v, cu_q, cu_k)
    kdn.kdn_prompt_attention(q, k, v, cu_q, cu_k, workspace=ws, flags=kdn.KDN_FLAG_TIMEOUT_PROBE)
    assert kdn.kdn_read_device_status(ws) == 8
    got = kdn.kdn_prompt_attention(q, k, v, cu_q, cu_k, workspace=ws)
    assert kdn.kdn_read_device_status(ws) == 0
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


def test_overlapping_bounds():
    """Bounds out of order: more row tiles than queries; what the calls leave unwritten stays so, and nothing else is written."""
    import uncertainty_aware_delta_gb300 as kdn

    n, T, C = 31, 512, 9000
    cu_q = torch.tensor([0, T] * 16, dtype=torch.int32, device="cuda")       # 0 .. T and, backwards, T .. 0
    cu_k = torch.tensor([0, C] * 16, dtype=torch.int32, device="cuda")
    q, k, v, _, _ = _inputs([T], [C], 4, 2, 64, "bf16")
    need = kdn.prompt_attention_workspace_size(n, T, 4, 2, 64)
    ws = torch.full((need + 4096,), 7, dtype=torch.uint8, device="cuda")
    o, lse = kdn.kdn_prompt_attention(q, k, v, cu_q, cu_k, workspace=ws[:need])
    assert kdn.kdn_read_device_status(ws) == 9 and bool((ws[need:] == 7).all())
    one, lse_one = kdn.kdn_prompt_attention(q, k, v, cu_q[:2], cu_k[:2])
    assert bool(((o.float() - one.float()).abs() <= 0.02).all()) and bool(((lse - lse_one).abs() < 1e-4).all())
