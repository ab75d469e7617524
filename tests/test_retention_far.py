"""Retention layer calls whose offsets pass 2^31 elements: rows far apart, and outputs and states that are that large."""
import pytest
import torch

import retention_oracle as ref
from test_decay import IO, on_tensor_cores

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("io,d", [("bf16", 128), ("bf16", 32), ("f32", 32)])
def test_rows_far_apart(io, d):
    """40 rows, 2^26 elements between one and the next."""
    import uncertainty_aware_delta_gb300 as kdn

    T, H, step = 40, 2, 1 << 26
    base = torch.empty(T * step, dtype=IO[io], device="cuda")
    gen = torch.Generator(device="cuda").manual_seed(0)
    far = []
    for i in range(4):
        t = base.as_strided((T, H, d), (step, d, 1), i * 1024)
        t.copy_(torch.randn(T, H, d, generator=gen, device="cuda") * d ** -0.5)
        far.append(t)
    near = [t.contiguous() for t in far]
    cu = torch.tensor([0, 13, T], dtype=torch.int32, device="cuda")
    l, S0 = torch.tensor([-0.01, -0.4], device="cuda"), torch.randn(2, H, d, d, device="cuda")
    for a, b in zip(kdn.kdn_decay_forward(*far[:3], l, S0, cu=cu), kdn.kdn_decay_forward(*near[:3], l, S0, cu=cu)):
        assert torch.equal(a, b)
    a, b = (kdn.kdn_decay_backward(*x[:3], l, S0, x[3], S0, cu=cu) for x in (far, near))
    assert all(torch.equal(a[n], b[n]) for n in a)
    assert torch.equal(kdn.kdn_group_norm(far[0], gate=far[1], act="silu"), kdn.kdn_group_norm(near[0], gate=near[1], act="silu"))
    a, b = (kdn.kdn_group_norm_backward(x[0], x[2], gate=x[1], act="silu") for x in (far, near))
    assert torch.equal(a["x"], b["x"]) and torch.equal(a["gate"], b["gate"])


@pytest.mark.parametrize("io,d,H", [("bf16", 128, 128), ("bf16", 32, 512)])
def test_large_outputs(io, d, H):
    """2^31 elements and some more: the last sequence's rows and state, against the definition."""
    import uncertainty_aware_delta_gb300 as kdn

    tok = (1 << 31) // (H * d) + 70
    g = torch.Generator(device="cuda").manual_seed(0)
    q, k, v = ((torch.randn(tok, H, d, generator=g, device="cuda", dtype=IO[io]) * d ** -0.5) for _ in range(3))
    cu = torch.tensor([0, tok - 75, tok - 70, tok], dtype=torch.int32, device="cuda")
    l, S0 = -torch.rand(H, device="cuda") * 0.1, torch.randn(3, H, d, d, device="cuda")
    o, S = kdn.kdn_decay_forward(q, k, v, l, S0, cu=cu)
    at, heads = slice(tok - 70, tok), slice(H - 4, H)
    want, size = ref.forward(*(t[at, heads] for t in (q, k, v)), l[heads], S0[2:, heads], [0, 70])
    ref.check(o[at, heads], want[0], size[0], on_tensor_cores(io, d, d), "o")
    ref.check(S[2:, heads], want[1], size[1], False, "S")
    y = kdn.kdn_group_norm(o, act="silu")
    ref.check_norm(y[at, heads], ref.norm(o[at, heads], None, None, None, "silu", 1e-5)["y"], "norm")
