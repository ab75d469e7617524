"""States carried over many tokens by the decay alone: the factors of chunks, segments and steps must not add up their roundings.

Over n factors, each rounded to fp32, a state would be off by up to n 2^-24 of itself, always to the same side.  What may remain:
log_decay times a count is rounded once (2^-24 of log_decay T), exp(x) - 1 is good to a unit in the last place (2^-23 of it, so
again 2^-23 of log_decay T over all factors), the last factor's rounding (2^-24), and the roundings of the state itself at every factor.
These are of either sign: the mean of the m elements of a head is off by more than 2^-24 sqrt(2 n log(2e12) / m) with a probability
below 1e-12 (Hoeffding).
"""
import math

import pytest
import torch

pytestmark = pytest.mark.gpu
IO = {"f32": torch.float32, "bf16": torch.bfloat16}


def drift(S, S0, l, T):
    """Mean of S / (exp(l T) S0) - 1 of every head, in 64 bits, for S and S0 [H, dk, dv]."""
    want = torch.exp(l.cpu().double() * T)[:, None, None] * S0.cpu().double()
    return (S.cpu().double() / want - 1).mean((-1, -2)).abs()


def allowed(l, T, n, m):
    return 2.0 ** -24 * (3 * l.cpu().double().abs() * T + 2 + math.sqrt(2 * n * math.log(2e12) / m))


def states(H, d):
    g = torch.Generator().manual_seed(5)
    return ((1 + torch.rand(H, d, d, generator=g)) * (1 - 2 * torch.randint(0, 2, (H, d, d), generator=g))).cuda()


@pytest.mark.parametrize("io,d", [("f32", 64), ("bf16", 64), ("bf16", 128)])
@pytest.mark.parametrize("T", [51200, 51199])
def test_chunks(io, d, T):
    """One walk along all tokens, forward and from the end."""
    import uncertainty_aware_delta_gb300 as kdn

    H = 16
    l = -1e-4 * (1 + torch.arange(H, device="cuda") / H)
    S0, x = states(H, d), torch.zeros(1, T, H, d, dtype=IO[io], device="cuda")
    _, S = kdn.kdn_decay_forward(x, x, x, l, S0[None], flags=kdn.KDN_FLAG_NO_SPLIT)
    limit = allowed(l, T, T / 32 + 1, d * d)
    assert bool((drift(S[0], S0, l, T) <= limit).all())
    g = kdn.kdn_decay_backward(x, x, x, l, None, x, S0[None], flags=kdn.KDN_FLAG_NO_SPLIT)
    assert bool((drift(g["S0"][0], S0, l, T) <= limit).all())


@pytest.mark.parametrize("io,d", [("f32", 64), ("bf16", 64), ("bf16", 128)])
def test_segments(io, d):
    """Some hundred segments, chained."""
    import uncertainty_aware_delta_gb300 as kdn

    T = 204700
    size = kdn.decay_workspace_size(1, T, 1, d, d, int(io == "bf16"))
    assert size >= 256 + 4 * d * d * 60
    S0, x = states(1, d), torch.zeros(1, T, 1, d, dtype=IO[io], device="cuda")
    for i in range(16):
        l = torch.full((1,), -1e-5 * (1 + i / 16), device="cuda")
        limit = allowed(l, T, T / 64 + 1, d * d)
        _, S = kdn.kdn_decay_forward(x, x, x, l, S0[None])
        assert bool((drift(S[0], S0, l, T) <= limit).all()), i
        g = kdn.kdn_decay_backward(x, x, x, l, None, x, S0[None])
        assert bool((drift(g["S0"][0], S0, l, T) <= limit).all()), i


@pytest.mark.parametrize("io,d", [("f32", 64), ("bf16", 128)])
def test_steps(io, d):
    """Decoding: one token a call."""
    import uncertainty_aware_delta_gb300 as kdn

    H, n, once = 16, 16384, 512
    l = -1e-4 * (1 + torch.arange(H, device="cuda") / H)
    S0, x = states(H, d), torch.zeros(1, H, d, dtype=IO[io], device="cuda")
    S, o = S0[None].clone(), torch.empty_like(x)
    side, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph, stream=side):
        for _ in range(once):
            kdn.kdn_decay_step(x, x, x, l, S, o=o)
    for _ in range(n // once):
        graph.replay()
    torch.cuda.synchronize()
    assert bool((drift(S[0], S0, l, n) <= allowed(l, n, n, d * d)).all())


@pytest.mark.parametrize("log_decay", [0.0, -0.3, -0.6, -20.0, -float("inf")])
def test_steps_of_any_decay(log_decay):
    """exp(log_decay) S + k v^T.  Of k v^T the product is rounded, its sum with what the factor's small part gives, and the whole sum: three
    times 2^-24.  Of the old state the whole sum (and 2^-48 of the small part), and its factor is good to two units in the last place, 2^-22."""
    import uncertainty_aware_delta_gb300 as kdn

    g = torch.Generator().manual_seed(1)
    q, k, v = (torch.randn(2, 3, 64, generator=g).cuda() for _ in range(3))
    S0, l = torch.randn(2, 3, 64, 64, generator=g).cuda(), torch.full((3,), log_decay, device="cuda")
    S = S0.clone()
    kdn.kdn_decay_step(q, k, v, l, S)
    own, old = k.cpu().double()[..., :, None] * v.cpu().double()[..., None, :], math.exp(log_decay) * S0.cpu().double()
    assert bool(((S.cpu().double() - own - old).abs() <= 2.0 ** -24 * (3 * own.abs() + 6 * old.abs())).all())
