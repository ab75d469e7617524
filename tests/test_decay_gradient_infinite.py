"""Gradients with a value that is not finite at one place: what depends on it is not finite, everything else has the same bits.

With R_t = sum_{s >= t} g^(s - t) q_s dO_s^T + g^(last - t) dS_T and S_t = sum_{s <= t} g^(t - s) k_s v_s^T + g^(t + 1) S0 along a sequence:
dq_t = S_t dO_t, dk_t = R_t v_t, dv_t = R_t^T k_t, dS0 = g R_0.
"""
import pytest
import torch

from test_decay import inputs

pytestmark = pytest.mark.gpu
HEAD, I, J = 1, 5, 7       # head, key channel, value channel


def depends(name, x, first, at, end, seq):
    """Masks of what depends on `name` at token `at` of the sequence `seq` (tokens first .. end - 1)."""
    m = {n: torch.zeros(x[n].shape, dtype=torch.bool, device="cuda") for n in ("q", "k", "v", "S0")}
    late, early, here, whole = slice(at, end), slice(first, at + 1), slice(at, at + 1), slice(first, end)
    if name == "q":             # R's row I from here to the front
        m["k"][early, HEAD, I] = m["v"][early, HEAD] = m["S0"][seq, HEAD, I] = True
    elif name == "k":           # S's row I from here on; dv here
        m["q"][late, HEAD, I] = m["v"][here, HEAD] = True
    elif name == "v":           # S's column J from here on; dk here
        m["q"][late, HEAD] = m["k"][here, HEAD] = True
    elif name == "dO":          # dq here; R's column J from here to the front
        m["q"][here, HEAD] = m["k"][early, HEAD] = m["v"][early, HEAD, J] = m["S0"][seq, HEAD, :, J] = True
    elif name == "dS":          # R's element (I, J) everywhere
        m["k"][whole, HEAD, I] = m["v"][whole, HEAD, J] = m["S0"][seq, HEAD, I, J] = True
    else:                       # S0: S's element (I, J) everywhere
        m["q"][whole, HEAD, I] = True
    return m


def check(lengths, dk, dv, io, flags, names, places):
    """A value in the second sequence, at places from its first token on."""
    import uncertainty_aware_delta_gb300 as kdn

    x = inputs(lengths, 2, dk, dv, io, True, lo=1e-3, hi=1e-2)
    back = lambda: kdn.kdn_decay_backward(*(x[n] for n in ("q", "k", "v", "log_decay", "S0", "dO", "dS")), cu=x["cu"], flags=flags)   # noqa: E731
    good = back()
    assert all(bool(torch.isfinite(t).all()) for t in good.values())
    first, end = lengths[0], lengths[0] + lengths[1]
    for name in names:
        for at in places if name not in ("S0", "dS") else (0,):
            at = first + at % lengths[1]
            place = (1, HEAD, I, J) if name in ("S0", "dS") else (at, HEAD, I if name in ("q", "k") else J)
            value = x[name][place].clone()
            for bad in (float("inf"), float("nan")):
                x[name][place] = bad
                got, mask = back(), depends(name, x, first, at, end, 1)
                for n, t in got.items():
                    assert torch.equal(t[~mask[n]], good[n][~mask[n]]), (name, at - first, bad, n)
                    assert not bool(torch.isfinite(t[mask[n]]).any()), (name, at - first, bad, n)
            x[name][place] = value


PATHS = pytest.mark.parametrize("io,dk,dv,flags", [("f32", 32, 32, 0), ("f32", 64, 128, 0), ("bf16", 64, 64, 0), ("bf16", 128, 128, 0),
                                                   ("bf16", 64, 128, 0), ("bf16", 128, 64, 2), ("bf16", 128, 128, 1)])


@PATHS
@pytest.mark.parametrize("name", ["q", "k", "v", "dO", "dS", "S0"])
def test_one_place(io, dk, dv, flags, name):
    """Chunks of 32 and of 64: the first token, both halves of a whole chunk, the short one and the last token.  The short chunk shares
    its rows with the next sequence's first, the first chunk comes after the sequence before."""
    check([75, 150, 70], dk, dv, io, flags, [name], [0, 10, 45, 84, 131, -1])


@PATHS
def test_in_segments(io, dk, dv, flags):
    """A long sequence, cut (but for KDN_FLAG_NO_SPLIT)."""
    import uncertainty_aware_delta_gb300 as kdn

    lengths = [75, 2500, 70] + [20] * 5
    assert flags & 2 or kdn.decay_backward_workspace_size(8, sum(lengths), 2, dk, dv, int(io == "bf16"), flags) >= 256 + 4 * 3 * 2 * dk * dv * 8
    check(lengths, dk, dv, io, flags, ["q", "k", "v", "dO", "dS", "S0"], [700, -1])
