"""Keys, queries and values that are infinite or as large as the type holds, where rows see them: against the definition
in 64 bits, in which a key whose score is -infinity has a weight of 0."""
import numpy as np
import pytest
import torch

import attention_oracle as ref
from test_prompt_attention import _inputs, _np

pytestmark = pytest.mark.gpu
PATHS = [("bf16", 64, 0), ("bf16", 128, 0), ("bf16", 64, 1), ("bf16", 128, 1), ("f32", 64, 0), ("f32", 128, 0), ("bf16", 32, 0),
         ("f32", 16, 0)]


def _expect(q, k, v, cu, window):
    """(o, lse, A, E) row by row; rows with a score of +infinity or NaN are NaN, keys at -infinity are left out."""
    q, k, v = _np(q), _np(k), _np(v)
    n, H, d = q.shape
    o, A = np.zeros((2, n, H, d))
    lse, E = np.full((n, H), -np.inf), np.zeros((n, H))
    for a, b in zip(cu, cu[1:]):
        for i in range(a, b):
            lo = max(a, i - window + 1) if window else a
            for h in range(H):
                kk, vv = k[lo:i + 1, h * k.shape[1] // H], v[lo:i + 1, h * k.shape[1] // H]
                with np.errstate(invalid="ignore"):
                    x = (kk * q[i, h]).sum(1)
                if np.isnan(x).any() or (x == np.inf).any():
                    o[i, h] = lse[i, h] = np.nan
                    continue
                keep = np.isfinite(x)
                if keep.any():
                    o[i, h], lse[i, h], A[i, h], E[i, h] = ref.attend(q[i, h], kk[keep], vv[keep], d ** -0.5, 0, int(keep.sum()))
    return o, lse, A, E


def _compare(q, k, v, cu, window, flags, io):
    import uncertainty_aware_delta_gb300 as kdn

    o, lse = kdn.kdn_prompt_attention(q, k, v, cu, window=window, flags=flags)
    want = _expect(q, k, v, cu.tolist(), window)
    assert np.isfinite(want[0]).any()
    ref.check(_np(o), _np(lse), want, io)
    return want


@pytest.mark.parametrize("io,d,flags", PATHS)
@pytest.mark.parametrize("bad", [float("inf"), -float("inf")])
@pytest.mark.parametrize("window", [0, 70])
def test_infinite_keys(bad, window, io, d, flags):
    q, k, v, cu, _ = _inputs([150, 90, 200], [150, 90, 200], 2, 1, d, io, seed=5)
    for place in (10, 149, 150, 200, 300):
        k[place, 0, 3] = bad
    k[305, 0, 1], k[305, 0, 2] = bad, -bad      # of opposite signs in one key
    want = _compare(q, k, v, cu, window, flags, io)
    seen = np.isnan(want[0]).any((1, 2))
    assert seen[10:80].any() and not seen[:10].any()


@pytest.mark.parametrize("io,d,flags", PATHS)
def test_infinite_queries(io, d, flags):
    """A row of its own: the others keep their results, and one whose only score is -infinity has no weights at all."""
    q, k, v, cu, _ = _inputs([150, 90], [150, 90], 2, 1, d, io, seed=6)
    q[0, 0, 2] = -float("inf") if float(k[0, 0, 2]) > 0 else float("inf")
    q[7, 1, 5], q[160, 0, 0] = float("inf"), -float("inf")
    want = _compare(q, k, v, cu, 0, flags, io)
    assert want[1][0, 0] == -np.inf and np.isnan(want[1][7, 1]) and np.isfinite(want[1][7, 0])


@pytest.mark.parametrize("io,d,flags", PATHS)
@pytest.mark.parametrize("bad", [float("inf"), -float("inf"), float("nan")])
def test_channels_beside_a_bad_value(bad, io, d, flags):
    """A value that is not finite reaches its own channel of the rows that see it, and no other."""
    import uncertainty_aware_delta_gb300 as kdn

    q, k, v, cu, _ = _inputs([150, 90, 200], [150, 90, 200], 2, 1, d, io, seed=5)
    want = _expect(q, k, v, cu.tolist(), 70)
    for place, channel in ((10, 3), (149, 0), (150, 1), (200, d - 1), (300, 7)):
        v[place, 0, channel] = bad
        end = min(place + 70, [e for e in cu.tolist() if e > place][0])
        want[0][place:end, :, channel] = bad
    o, lse = kdn.kdn_prompt_attention(q, k, v, cu, window=70, flags=flags)
    got, odd = _np(o), ~np.isfinite(want[0])
    assert np.array_equal(got[odd], want[0][odd], equal_nan=True)
    ref.check(np.where(odd, 0, got), _np(lse), (np.where(odd, 0, want[0]), *want[1:]), io)
