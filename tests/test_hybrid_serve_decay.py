"""The serving example with decayed memories in place of the KDN mixer: its calls against the 64-bit definitions, on the tensors that
it passes them."""
import os
import sys

import pytest
import torch

import retention_oracle as ref

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))
pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("d", [32, 64])
def test_two_turns(d, monkeypatch):
    import uncertainty_aware_delta_gb300 as kdn
    from hybrid_serve import Server, norm

    R = 3
    s = Server(R, 40, layers=2, heads=4, kv_heads=2, d=d, page=16, table_width=12, mixer="decay")
    gen = torch.Generator(device="cuda").manual_seed(3)
    seen = {"forward": 0, "step": 0, "norm": 0}
    forward, step, group_norm = kdn.kdn_decay_forward, kdn.kdn_decay_step, kdn.kdn_group_norm

    def check_forward(q, k, v, l, S0, cu):
        o, S = forward(q, k, v, l, S0, cu=cu)
        want, size = ref.forward(q, k, v, l, S0, cu.tolist())
        ref.check(o, want[0], size[0], d == 64, "o")
        ref.check(S, want[1], size[1], False, "S")
        seen["forward"] += 1
        return o, S

    def check_step(q, k, v, l, S):
        want, size = ref.forward(*(t[:, None] for t in (q, k, v)), l, S)
        o = step(q, k, v, l, S)
        ref.check(o, want[0][:, 0], size[0][:, 0], False, "step")
        ref.check(S, want[1], size[1], False, "S")
        seen["step"] += 1
        return o

    def check_norm(x, w, b, gate, act):
        y = group_norm(x, w, b, gate=gate, act=act)
        ref.check_norm(y, ref.norm(x, w, b, gate, act, 1e-5)["y"], "norm")
        seen["norm"] += 1
        return y

    monkeypatch.setattr(kdn, "kdn_decay_forward", check_forward)
    monkeypatch.setattr(kdn, "kdn_decay_step", check_step)
    monkeypatch.setattr(kdn, "kdn_group_norm", check_norm)
    for new in ([33, 1, 50], [0, 20, 17]):
        y, granted = s.prefill(torch.randn(sum(new), s.dim, generator=gen, device="cuda").bfloat16(), new)
        assert granted == [1, 1, 1] and bool(torch.isfinite(y).all())
        x = torch.randn(R, s.dim, generator=gen, device="cuda").bfloat16()
        for _ in range(3):
            x = norm(s.decode(x))
        assert bool(torch.isfinite(x).all())
    assert seen == {"forward": 4, "step": 12, "norm": 16}
    # a prompt that the free pages cannot hold changes nothing of its request
    S = s.layers[0]["S"].clone()
    s.table = torch.cat([s.table, torch.full((R, 60), -1, dtype=torch.int32, device="cuda")], 1)
    new = [5, 700, 0]
    _, granted = s.prefill(torch.randn(705, s.dim, generator=gen, device="cuda").bfloat16(), new)
    assert granted == [1, 0, 1]
    assert torch.equal(S[1:], s.layers[0]["S"][1:]) and not torch.equal(S[0], s.layers[0]["S"][0])
    for r in range(R):
        s.release(r)
    assert int(s.n_free) == 40 and not bool(s.layers[0]["S"].any())


def test_command(monkeypatch, capsys):
    import hybrid_serve

    monkeypatch.setattr(sys, "argv", ["hybrid_serve.py", "--requests", "3", "--prompt", "70", "--steps", "4", "--mixer", "decay"])
    hybrid_serve.main()
    out = capsys.readouterr().out
    assert "outputs finite: True" in out and "pages free" in out


def test_unknown_mixer():
    from hybrid_serve import Server

    with pytest.raises(ValueError, match="mixer"):
        Server(1, 2, mixer="none")
