"""Packed bounds that are wrong, in calls whose long sequences are cut into segments: every sequence's are looked at, and the ones
that are right keep their results."""
import pytest
import torch

from test_decay import inputs

pytestmark = pytest.mark.gpu
LONG, N = 1600, 40                 # one long sequence and 39 of 20 tokens: more than a warp looks at in one go
LENGTHS = [LONG] + [20] * (N - 1)
FORMS = pytest.mark.parametrize("io,d", [("f32", 64), ("bf16", 64), ("bf16", 128)])


def run(x, cu, io, d, back, tok):
    """Outputs (rows of no sequence left at 7) and the status word."""
    import uncertainty_aware_delta_gb300 as kdn

    size = kdn.decay_backward_workspace_size if back else kdn.decay_workspace_size
    need = size(len(cu) - 1, tok, 1, d, d, int(io == "bf16"))
    assert need >= 256 + 4 * d * d * (3 if back else 1) * 4      # cut: there are segments' states
    ws = torch.empty(need, dtype=torch.uint8, device="cuda")
    cu = torch.tensor(cu, dtype=torch.int32, device="cuda")
    args = tuple(x[n] for n in ("q", "k", "v", "log_decay", "S0"))
    if back:
        g = kdn.kdn_decay_backward(*args, x["dO"], x["dS"], cu=cu, workspace=ws)
        out = [g[n] for n in ("q", "k", "v")], g["S0"]
    else:
        o, S = torch.full_like(x["v"], 7), torch.full_like(x["S0"], 7)
        kdn.kdn_decay_forward(*args, cu=cu, out=(o, S), workspace=ws)
        out = [o], S
    return out, kdn.kdn_read_device_status(ws)


def bounds():
    cu = [0]
    for m in LENGTHS:
        cu.append(cu[-1] + m)
    return cu


@FORMS
@pytest.mark.parametrize("back", [False, True])
@pytest.mark.parametrize("what", ["last", "middle", "first"])
def test_reported_wherever_they_are(io, d, back, what):
    x, cu = inputs(LENGTHS, 1, d, d, io, True), bounds()
    tok = cu[-1]
    good, status = run(x, cu, io, d, back, tok)
    assert status == 0
    if what == "last":          # past the tokens
        cu[N], bad = tok + 1, [N - 1]
    elif what == "middle":      # backwards; the next sequence takes its first token from before
        cu[36], bad = cu[35] - 1, [35]
    else:
        cu[0], bad = -1, [0]
    got, status = run(x, cu, io, d, back, tok)
    assert status == 9
    initial = x["dS"] if back else x["S0"]
    right = [s for s in range(N) if s not in bad + ([34, 36] if what == "middle" else [])]
    assert torch.equal(got[1][right], good[1][right]) and torch.equal(got[1][bad], initial[bad])
    first = cu[1] if what == "first" else 0
    upto = cu[34] if what == "middle" else cu[N - 1]
    assert all(torch.equal(a[first:upto], b[first:upto]) for a, b in zip(got[0], good[0]))
    if what == "last" and not back:
        assert bool((got[0][0][cu[N - 1]:] == 7).all())


@FORMS
@pytest.mark.parametrize("back", [False, True])
def test_sequences_behind_bounds_that_run_backwards(io, d, back):
    """The long sequence's rows in four of them: more segments than the tokens have.  Those behind share no row with them."""
    x = inputs(LENGTHS, 1, d, d, io, True)
    tail = [LONG + 20 * i for i in range(N - 6)]
    wrong = [0, LONG, 0, LONG, 0, LONG, 0] + tail
    right = [0, LONG, LONG, LONG, LONG, LONG, LONG] + tail
    right[1:7] = [0, 0, 0, 0, 0, 0]
    assert len(wrong) == len(right) == N + 1
    tok = sum(LENGTHS)
    good, status = run(x, right, io, d, back, tok)
    assert status == 0
    got, status = run(x, wrong, io, d, back, tok)
    assert status == 9
    assert torch.equal(got[1][7:], good[1][7:])
    assert all(torch.equal(a[LONG:tail[-1]], b[LONG:tail[-1]]) for a, b in zip(got[0], good[0]))
    if not back:
        assert bool((got[0][0][tail[-1]:] == 7).all())
