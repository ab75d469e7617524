"""Keys, queries and values as large as fp32 holds (such as a mask's lowest value), against the definition in 64 bits.
A TF32 part holds 11 bits, so the nearest one to such a number is infinite."""
import numpy as np
import pytest
import torch

import attention_oracle as ref
from test_prompt_attention import _expect, _inputs, _np

pytestmark = pytest.mark.gpu
LOW = torch.finfo(torch.float32).min


@pytest.mark.parametrize("d", [16, 32, 64, 128])
@pytest.mark.parametrize("window", [0, 70])
def test_largest_values(d, window):
    import uncertainty_aware_delta_gb300 as kdn

    q, k, v, cu, _ = _inputs([150, 90], [150, 90], 2, 1, d, "f32", seed=7)
    clean, clean_lse = kdn.kdn_prompt_attention(q, k, v, cu, window=window)
    v[60, 0, 3], v[200, 0, 0], v[201, 0, 1] = LOW, -LOW, LOW * (1 - 2.0 ** -12)
    o, lse = kdn.kdn_prompt_attention(q, k, v, cu, window=window)
    seen = np.zeros(240, bool)
    for place, end in ((60, 150), (200, 240), (201, 240)):
        seen[place:min(place + window, end) if window else end] = True
    assert torch.equal(lse, clean_lse) and torch.equal(o[~seen], clean[~seen])
    ref.check(_np(o), _np(lse), _expect(q, k, v, cu, cu, window), "f32")


@pytest.mark.parametrize("d", [16, 32, 64, 128])
def test_largest_keys_and_queries(d):
    """Scores of 1e37 and more: the largest has all the weight, or none where its sign is the other."""
    import uncertainty_aware_delta_gb300 as kdn

    q, k, v, cu, _ = _inputs([150, 90], [150, 90], 2, 1, d, "f32", seed=8)
    q.clamp_(-0.9, 0.9)       # (a product past 32 bits' range would be infinite)
    k.clamp_(-0.9, 0.9)
    k[60, 0, 3], k[200, 0, 1] = LOW, -LOW
    q[20, 0, 5], q[230, 1, 7] = LOW, -LOW * (1 - 2.0 ** -13)
    q[230, 1, 1], k[200, 0, 7] = 0.25, 0.1
    o, lse = kdn.kdn_prompt_attention(q, k, v, cu)
    want = _expect(q, k, v, cu, cu, 0)
    assert np.isfinite(want[0]).all() and np.isfinite(want[1]).all()
    ref.check(_np(o), _np(lse), want, "f32")
    # the bounds are wide where scores are, so rows by their score's sign: the value itself, in two TF32 parts (2^-23
    # of it lost) and a sum that cuts off (2^-22), or none of it
    x = _np(q)[60:150, 0, 3] * _np(k)[60, 0, 3]
    assert np.allclose(_np(o)[60:150, 0][x > 0], _np(v)[60, 0], rtol=2.0 ** -21, atol=0)
    assert (np.abs(_np(lse)[60:150, 0][x < 0]) < 20).all() and (x < 0).any()
