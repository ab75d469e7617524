"""Sizes of the retention layer's tensors that do not fit the library's 32-bit arguments are refused, not cut off.  (Views whose rows
are all the same one: no memory is needed, and no GPU.)"""
import pytest
import torch

BIG = 2 ** 32 + 2      # cut off: 2


def view(*shape):
    return torch.zeros(1).expand(*shape)


def calls(q, v, H, dk, dv, n):
    import uncertainty_aware_delta_gb300 as kdn

    l, S = view(H), view(n, H, dk, dv)
    yield lambda: kdn.kdn_decay_forward(q, q, v, l)
    yield lambda: kdn.kdn_decay_backward(q, q, v, l, None, v)
    if q.shape[1] == 1:
        yield lambda: kdn.kdn_decay_step(q[:, 0], q[:, 0], v[:, 0], l, S)


@pytest.mark.parametrize("n,H,dk,dv", [(1, BIG, 64, 64), (1, 2, BIG + 62, 64), (1, 2, 64, BIG + 62), (BIG, 2, 64, 64)])
def test_memory(n, H, dk, dv):
    for call in calls(view(n, 1, H, dk), view(n, 1, H, dv), H, dk, dv, n):
        with pytest.raises(ValueError, match="does not fit 32 bits"):
            call()


def test_sequences():
    import uncertainty_aware_delta_gb300 as kdn

    q, cu = view(5, 2, 64), torch.zeros(1, dtype=torch.int32).expand(BIG + 1)
    for call in (lambda: kdn.kdn_decay_forward(q, q, q, view(2), cu=cu), lambda: kdn.kdn_decay_backward(q, q, q, view(2), None, q, cu=cu)):
        with pytest.raises(ValueError, match="does not fit 32 bits"):
            call()
    q = view(BIG, 0, 2, 64)    # no tokens at all
    with pytest.raises(ValueError, match="does not fit 32 bits"):
        kdn.kdn_decay_forward(q, q, q, view(2))


@pytest.mark.parametrize("rows,groups,d", [(1, BIG, 64), (1, 2, BIG + 62), (BIG, 2, 64)])
def test_norm(rows, groups, d):
    import uncertainty_aware_delta_gb300 as kdn

    x = view(rows, groups, d)
    for call in (lambda: kdn.kdn_group_norm(x), lambda: kdn.kdn_group_norm(x[None]), lambda: kdn.kdn_group_norm_backward(x, x)):
        with pytest.raises(ValueError, match="does not fit 32 bits"):
            call()
