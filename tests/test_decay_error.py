"""How large the errors are beside the results, in the mean over a tensor: what the roundings on the way allow, and no more.

A rounding to bf16 is off by a number spread evenly over a step: 2^-8 / sqrt(3) of the value in the mean square, at most.  Outputs are
rounded once; on tensor cores the weights and the state go into their products rounded, too, whose terms are of either sign here and
uncorrelated, so that their errors add up to 2^-8 / sqrt(3) of the norm of the sum: sqrt(2) 2^-8 / sqrt(3) in all, and a tenth for the
terms' few correlations.  fp32 outputs and all states: three sums or products of 2^-22 each and their powers, 2^-20.
"""
import pytest
import torch

import retention_oracle as ref
from test_decay import inputs, on_tensor_cores

pytestmark = pytest.mark.gpu


def far(got, want):
    return float((got.cpu().double() - want).norm() / want.norm())


@pytest.mark.parametrize("io,dk,dv", [("bf16", 128, 128), ("bf16", 64, 64), ("bf16", 64, 128), ("bf16", 128, 64), ("bf16", 32, 32), ("f32", 128, 128),
                                      ("f32", 64, 32)])
@pytest.mark.parametrize("lengths,packed", [([333, 333], False), ([1700], False), ([40, 1, 300], True)])
def test_error(io, dk, dv, lengths, packed):
    import uncertainty_aware_delta_gb300 as kdn

    x = inputs(lengths, 3, dk, dv, io, packed)
    q, k, v, l, S0, cu = (x[n] for n in ("q", "k", "v", "log_decay", "S0", "cu"))
    bounds, half = None if cu is None else cu.tolist(), 2.0 ** -8 / 3 ** 0.5
    rows = 2.0 ** -20 if io == "f32" else 1.1 * half * (2 ** 0.5 if on_tensor_cores(io, dk, dv) else 1)
    o, S = kdn.kdn_decay_forward(q, k, v, l, S0, cu=cu)
    want, _ = ref.forward(q, k, v, l, S0, bounds)
    assert far(o, want[0]) <= rows and far(S, want[1]) <= 2.0 ** -20
    g = kdn.kdn_decay_backward(q, k, v, l, S0, x["dO"], x["dS"], cu=cu)
    want, _ = ref.backward(q, k, v, l, S0, x["dO"], x["dS"], bounds)
    for i, name in enumerate(("q", "k", "v")):
        assert far(g[name], want[i]) <= rows, name
    assert far(g["S0"], want[3]) <= 2.0 ** -20
