"""Group norm of values whose squares leave fp32's range (tolerances: retention_oracle.py; nothing in them depends on the size of x)."""
import pytest
import torch

import retention_oracle as ref
from test_group_norm import inputs

pytestmark = pytest.mark.gpu


def check(x, dy, z, w, b, act, eps):
    import uncertainty_aware_delta_gb300 as kdn

    y = kdn.kdn_group_norm(x, w, b, gate=z, act=act, eps=eps)
    ref.check_norm(y, ref.norm(x, w, b, z, act, eps)["y"], "y")
    got, want = kdn.kdn_group_norm_backward(x, dy, w, b, gate=z, act=act, eps=eps), ref.norm(x, w, b, z, act, eps, dy)
    for name in want:
        ref.check_norm(got[name], want[name], name)
    return y, got


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("d", [64, 128, 72])
@pytest.mark.parametrize("gate", [False, True])
@pytest.mark.parametrize("by,eps", [(2.0 ** 64, 1e-5), (2.0 ** 110, 1e-5), (2.0 ** 70, 0.0), (2.0 ** -70, 0.0), (2.0 ** -100, 0.0),
                                    (2.0 ** -64, 2.0 ** -110)])
def test_large_and_small_values(io, d, gate, by, eps):
    """In some rows, among others: those are as they are without them, bit for bit."""
    import uncertainty_aware_delta_gb300 as kdn

    x, dy, z, w, b = inputs(40, 3, d, io, gate, 3)
    before = kdn.kdn_group_norm(x, w, b, gate=z, act="silu", eps=eps), kdn.kdn_group_norm_backward(x, dy, w, b, gate=z, act="silu", eps=eps)
    odd = torch.zeros(40, 3, dtype=torch.bool)
    odd[::3, 1] = odd[5] = odd[17, 0] = True
    x[odd.cuda()] *= by                       # (powers of two: exact)
    y, g = check(x, dy, z, w, b, "silu", eps)
    same = (~odd).cuda()
    assert torch.equal(y[same], before[0][same]) and torch.equal(g["x"][same], before[1]["x"][same])


@pytest.mark.parametrize("io", ["f32", "bf16"])
def test_rows_of_zeros(io):
    """Padding: the bias, and gradients that are finite; with eps = 0 the definition's 0 / 0."""
    import uncertainty_aware_delta_gb300 as kdn

    x, dy, z, w, b = inputs(40, 3, 64, io, True, 3)
    x[::2] = 0
    check(x, dy, z, w, b, "silu", 1e-5)
    assert bool(torch.isnan(kdn.kdn_group_norm(x, eps=0.0)[::2]).all())


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("bad", [float("inf"), -float("inf"), float("nan")])
def test_not_finite_beside_large(io, bad):
    import uncertainty_aware_delta_gb300 as kdn

    x, dy, z, w, b = inputs(40, 3, 64, io, True, 3)
    x[3] *= 2.0 ** 100
    x[3, 1, 7] = bad
    y, g = kdn.kdn_group_norm(x, w, b, gate=z, act="silu"), kdn.kdn_group_norm_backward(x, dy, w, b, gate=z, act="silu")
    assert bool(torch.isnan(y[3, 1]).all()) and bool(torch.isnan(g["x"][3, 1]).all())
    assert bool(torch.isfinite(y[3, ::2]).all()) and bool(torch.isfinite(g["x"][3, ::2]).all())
