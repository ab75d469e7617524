"""The serving example's calls against the 64-bit definitions, on the tensors that it passes them."""
import os
import sys

import pytest
import torch

import attention_oracle as ao
from test_cache_attention import _expect, _floor

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))
pytestmark = pytest.mark.gpu


def f64(t):
    return t.detach().double().cpu().numpy()


@pytest.mark.parametrize("window", [0, 40])
def test_two_turns(window, monkeypatch):
    import uncertainty_aware_delta_gb300 as kdn
    from hybrid_serve import Server, norm

    R, d, page = 3, 32, 16
    s = Server(R, 40, layers=2, heads=4, kv_heads=2, d=d, page=page, table_width=12, window=window)
    gen = torch.Generator(device="cuda").manual_seed(3)
    seen = {"prompt": 0, "cache": 0}
    prompt, cached = kdn.kdn_prompt_attention, kdn.kdn_cache_attention

    def check_prompt(q, k, v, cu_q, cu_k, window):
        o, lse = prompt(q, k, v, cu_q, cu_k, window=window)
        ref = ao.prompt(f64(q), f64(k), f64(v), cu_q.tolist(), cu_k.tolist(), window, d ** -0.5)
        ao.check(f64(o), f64(lse), ref, "bf16")
        seen["prompt"] += 1
        return o, lse

    def check_cache(q, cache, table, lens, window):
        o, lse = cached(q, cache, table, lens, window=window)
        ao.check(f64(o), f64(lse), _expect(q, cache, table, lens, window), "bf16", True, _floor(cache, lens.tolist()))
        seen["cache"] += 1
        return o, lse

    monkeypatch.setattr(kdn, "kdn_prompt_attention", check_prompt)
    monkeypatch.setattr(kdn, "kdn_cache_attention", check_cache)
    for new in ([33, 1, 50], [0, 20, 17]):
        y, granted = s.prefill(torch.randn(sum(new), s.dim, generator=gen, device="cuda").bfloat16(), new)
        assert granted == [1, 1, 1] and bool(torch.isfinite(y).all())
        x = torch.randn(R, s.dim, generator=gen, device="cuda").bfloat16()
        for _ in range(3):
            x = norm(s.decode(x))
        assert bool(torch.isfinite(x).all())
    assert s.context.tolist() == [39, 27, 73] and seen == {"prompt": 4, "cache": 12}
    # a prompt that the free pages cannot hold is refused and changes nothing of its request
    S, free = s.layers[0]["S"].clone(), int(s.n_free)
    s.table = torch.cat([s.table, torch.full((R, 60), -1, dtype=torch.int32, device="cuda")], 1)
    with pytest.raises(ValueError):
        s.prefill(torch.zeros(1200, s.dim, device="cuda").bfloat16(), [0, 1200, 0])
    new = [0, 700, 0]
    _, granted = s.prefill(torch.zeros(700, s.dim, device="cuda").bfloat16(), new)
    assert granted == [1, 0, 1] and s.context.tolist() == [39, 27, 73] and int(s.n_free) == free
    assert torch.equal(S, s.layers[0]["S"])
    for r in range(R):
        s.release(r)
    assert int(s.n_free) == 40 and sorted(s.free.tolist()) == list(range(40))


def test_command(monkeypatch, capsys):
    import hybrid_serve

    monkeypatch.setattr(sys, "argv", ["hybrid_serve.py", "--requests", "3", "--prompt", "70", "--steps", "4"])
    hybrid_serve.main()
    out = capsys.readouterr().out
    assert "outputs finite: True" in out and "pages free" in out
