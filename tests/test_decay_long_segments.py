"""Segments of many chunks (more than a ring of the tensor-core path has stages, twice over) with a short last one, and whole walks
from the end of as many, against the recurrence in 64 bits (tolerances: retention_oracle.py)."""
import pytest
import torch

import retention_oracle as ref
from test_decay import inputs, on_tensor_cores

pytestmark = pytest.mark.gpu
HEADS = slice(0, 16, 9)        # the ones that are checked


def cut(n, tok, H, dk, dv, jobs, io="bf16"):
    """Segments that have a state, by the size of the workspace."""
    import uncertainty_aware_delta_gb300 as kdn

    size = kdn.decay_backward_workspace_size if jobs == 3 else kdn.decay_workspace_size
    return (size(n, tok, H, dk, dv, int(io == "bf16")) - 256) // (4 * jobs * H * dk * dv)


def check(x, dk, dv, io, flags=0):
    import uncertainty_aware_delta_gb300 as kdn

    q, k, v, l, S0, dO, dS, cu = (x[n] for n in ("q", "k", "v", "log_decay", "S0", "dO", "dS", "cu"))
    few = lambda t: t[..., HEADS, :].contiguous()   # noqa: E731
    state = lambda t: t[:, HEADS].contiguous()      # noqa: E731
    tc, bounds = on_tensor_cores(io, dk, dv, flags), None if cu is None else cu.tolist()
    o, S = kdn.kdn_decay_forward(q, k, v, l, S0, cu=cu, flags=flags)
    want, size = ref.forward(few(q), few(k), few(v), l[HEADS], state(S0), bounds)
    ref.check(few(o), want[0], size[0], tc, "o")
    ref.check(state(S), want[1], size[1], False, "S_T")
    g = kdn.kdn_decay_backward(q, k, v, l, S0, dO, dS, cu=cu, flags=flags)
    want, size = ref.backward(few(q), few(k), few(v), l[HEADS], state(S0), few(dO), state(dS), bounds)
    for i, name in enumerate(("q", "k", "v")):
        ref.check(few(g[name]), want[i], size[i], tc, "gradient of " + name)
    ref.check(state(g["S0"]), want[3], size[3], False, "gradient of S0")


@pytest.mark.parametrize("dk,dv,T", [(64, 64, 7900), (64, 128, 7900), (128, 64, 7900), (128, 128, 7900), (64, 64, 7873)])
def test_dense(dk, dv, T):
    segments, back = cut(1, T, 16, dk, dv, 1), cut(1, T, 16, dk, dv, 3)
    for n in (segments, back):
        per = -(-T // n // 64)                              # chunks of a segment, at least
        assert n > 1 and per > 12 and T % 64 != 0
    check(inputs([T], 16, dk, dv, "bf16", False, lo=1e-3, hi=0.3), dk, dv, "bf16")


@pytest.mark.parametrize("dk,dv", [(64, 64), (128, 128)])
def test_packed(dk, dv):
    """Nine short sequences and a long one, which alone is cut."""
    lengths = [30] * 4 + [8001] + [50, 0, 64, 1, 30]
    slots = cut(10, sum(lengths), 8, dk, dv, 1)              # (the tokens over a segment's, and as many or the sequences more)
    assert slots >= 4 and 8001 // (slots // 2 + 1) > 12 * 64
    x = inputs(lengths, 8, dk, dv, "bf16", True, lo=1e-3, hi=0.3)
    check(x, dk, dv, "bf16")


@pytest.mark.parametrize("io,dk,dv", [("bf16", 64, 64), ("bf16", 128, 128), ("f32", 32, 32)])
@pytest.mark.parametrize("T", [1000, 1024])
def test_whole(io, dk, dv, T):
    check(inputs([T], 10, dk, dv, io, False, lo=1e-3, hi=0.3), dk, dv, io, 2)
