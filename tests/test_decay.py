"""Linear attention with a decay for each head against its definition in 64 bits (tolerances: retention_oracle.py)."""
import pytest
import torch

import retention_oracle as ref

pytestmark = pytest.mark.gpu
IO = {"f32": torch.float32, "bf16": torch.bfloat16}


def inputs(lengths, H, dk, dv, io, packed, seed=0, lo=1e-3, hi=1.0):
    g = torch.Generator().manual_seed(seed)
    n, tok = len(lengths), sum(lengths)
    lead = (tok,) if packed else (n, lengths[0])
    rand = lambda *s: torch.randn(s, generator=g)   # noqa: E731
    x = {"q": rand(*lead, H, dk) * dk ** -0.5, "k": rand(*lead, H, dk) * dk ** -0.5, "v": rand(*lead, H, dv), "dO": rand(*lead, H, dv)}
    x = {name: t.to(IO[io]).cuda() for name, t in x.items()}
    x["log_decay"] = -(lo * (hi / lo) ** torch.rand(H, generator=g)).cuda()
    x["S0"], x["dS"] = rand(n, H, dk, dv).cuda(), rand(n, H, dk, dv).cuda()
    cu = [0]
    for m in lengths:
        cu.append(cu[-1] + m)
    x["cu"] = torch.tensor(cu, dtype=torch.int32, device="cuda") if packed else None
    return x


def on_tensor_cores(io, dk, dv, flags=0):
    return io == "bf16" and min(dk, dv) >= 64 and not flags & 1


def check_all(lengths, H, dk, dv, io, packed, flags=0, seed=0, **decays):
    import uncertainty_aware_delta_gb300 as kdn

    x = inputs(lengths, H, dk, dv, io, packed, seed, **decays)
    q, k, v, l, S0, cu = (x[n] for n in ("q", "k", "v", "log_decay", "S0", "cu"))
    tc, bounds = on_tensor_cores(io, dk, dv, flags), None if cu is None else cu.tolist()
    o, S = kdn.kdn_decay_forward(q, k, v, l, S0, cu=cu, flags=flags)
    want, size = ref.forward(q, k, v, l, S0, bounds)
    ref.check(o, want[0], size[0], tc, "o")
    ref.check(S, want[1], size[1], False, "S_T")
    g = kdn.kdn_decay_backward(q, k, v, l, S0, x["dO"], x["dS"], cu=cu, flags=flags)
    want, size = ref.backward(q, k, v, l, S0, x["dO"], x["dS"], bounds)
    for i, name in enumerate(("q", "k", "v", "S0")):
        ref.check(g[name], want[i], size[i], tc and name != "S0", "gradient of " + name)


@pytest.mark.parametrize("dk,dv", [(16, 16), (128, 128), (64, 64), (32, 128), (128, 16), (16, 64)])
@pytest.mark.parametrize("T", [1, 31, 32, 33, 64, 65, 200])
def test_fp32(dk, dv, T):
    check_all([T] * 2, 3, dk, dv, "f32", False)


@pytest.mark.parametrize("dk,dv", [(128, 128), (64, 64), (64, 128), (128, 64), (32, 32), (128, 16)])
@pytest.mark.parametrize("T", [1, 63, 64, 65, 128, 333])
def test_bf16(dk, dv, T):
    check_all([T] * 2, 3, dk, dv, "bf16", False)


@pytest.mark.parametrize("T", [1, 5, 31, 32])
def test_short_sequences(T):
    """Dense, heads of 64: the same bits as on CUDA cores, which work on them; packed ones are on tensor cores."""
    import uncertainty_aware_delta_gb300 as kdn

    check_all([T] * 5, 3, 64, 64, "bf16", True)
    x = inputs([T] * 5, 3, 64, 64, "bf16", False)
    args, dO, dS = tuple(x[n] for n in ("q", "k", "v", "log_decay", "S0")), x["dO"], x["dS"]
    for a, b in zip(*(kdn.kdn_decay_forward(*args, flags=f) for f in (0, kdn.KDN_FLAG_PORTABLE))):
        assert torch.equal(a, b)
    a, b = (kdn.kdn_decay_backward(*args, dO, dS, flags=f) for f in (0, kdn.KDN_FLAG_PORTABLE))
    assert all(torch.equal(a[n], b[n]) for n in a)
    want, size = ref.forward(*args)
    o, S = kdn.kdn_decay_forward(*args)
    ref.check(o, want[0], size[0], False, "o")
    ref.check(S, want[1], size[1], False, "S_T")


@pytest.mark.parametrize("io,dk,dv,flags", [("f32", 64, 32, 0), ("bf16", 128, 128, 0), ("bf16", 64, 64, 0), ("bf16", 128, 64, 1)])
def test_packed(io, dk, dv, flags):
    check_all([5, 0, 130, 1, 64, 97, 0], 2, dk, dv, io, True, flags)


@pytest.mark.parametrize("io,dk,dv,packed", [("f32", 16, 32, False), ("bf16", 128, 128, False), ("bf16", 64, 128, True), ("f32", 64, 64, True)])
def test_segments(io, dk, dv, packed):
    """Few long sequences: cut into segments, the last of them short."""
    check_all([1400, 700] if packed else [1400], 1, dk, dv, io, packed)


@pytest.mark.parametrize("io,dk,dv", [("f32", 32, 64), ("bf16", 64, 64), ("bf16", 128, 64)])
def test_long_sequences_among_short_ones(io, dk, dv):
    """Packed: only the long ones are cut into segments (more than 32 sequences: the forward alone)."""
    lengths = [3, 40, 0, 1700, 64, 1] + [17 + 9 * (i % 4) for i in range(5)] + [1000, 65, 0]
    check_all(lengths, 1, dk, dv, io, True)
    check_all(lengths + [30] * 24, 1, dk, dv, io, True)


def test_bounds_out_of_order_with_segments():
    """More segments than there is room for: nothing outside is written, the status word says so."""
    import uncertainty_aware_delta_gb300 as kdn

    n, H, d = 40, 1, 64
    x = inputs([1600] + [20] * 39, H, d, d, "bf16", True)
    tok = x["q"].shape[0]
    cu = torch.tensor([0 if i % 2 == 0 else tok for i in range(n + 1)], dtype=torch.int32, device="cuda")
    need = kdn.decay_workspace_size(n, tok, H, d, d, 1)
    assert need > 4096
    room = torch.full((need + 65536,), 7, dtype=torch.uint8, device="cuda")
    o, S = torch.full((tok + 64, H, d), 7, dtype=torch.bfloat16, device="cuda"), torch.empty_like(x["S0"])
    kdn.kdn_decay_forward(x["q"], x["k"], x["v"], x["log_decay"], x["S0"], cu=cu, out=(o[:tok], S), workspace=room[:need])
    assert kdn.kdn_read_device_status(room) == 9
    assert bool((room[need:] == 7).all()) and bool((o[tok:] == 7).all())


@pytest.mark.parametrize("io,d", [("f32", 32), ("bf16", 128)])
@pytest.mark.parametrize("log_decay", [0.0, -1e-6, -30.0, -float("inf")])
def test_extreme_decays(io, d, log_decay):
    import uncertainty_aware_delta_gb300 as kdn

    x = inputs([150] * 2, 2, d, d, io, False)
    l = torch.full((2,), log_decay, device="cuda")
    o, S = kdn.kdn_decay_forward(x["q"], x["k"], x["v"], l, x["S0"])
    want, size = ref.forward(x["q"], x["k"], x["v"], l, x["S0"])
    ref.check(o, want[0], size[0], on_tensor_cores(io, d, d), "o")
    ref.check(S, want[1], size[1], False, "S_T")
    g = kdn.kdn_decay_backward(x["q"], x["k"], x["v"], l, x["S0"], x["dO"], x["dS"])
    want, size = ref.backward(x["q"], x["k"], x["v"], l, x["S0"], x["dO"], x["dS"])
    for i, name in enumerate(("q", "k", "v", "S0")):
        ref.check(g[name], want[i], size[i], on_tensor_cores(io, d, d) and name != "S0", name)


@pytest.mark.parametrize("io", ["f32", "bf16"])
def test_without_states(io):
    import uncertainty_aware_delta_gb300 as kdn

    x = inputs([77], 2, 64, 64, io, False)
    zero = torch.zeros_like(x["S0"])
    for got, want in zip(kdn.kdn_decay_forward(x["q"], x["k"], x["v"], x["log_decay"]),
                         kdn.kdn_decay_forward(x["q"], x["k"], x["v"], x["log_decay"], zero)):
        assert torch.equal(got, want)
    a = kdn.kdn_decay_backward(x["q"], x["k"], x["v"], x["log_decay"], None, x["dO"])
    b = kdn.kdn_decay_backward(x["q"], x["k"], x["v"], x["log_decay"], zero, x["dO"], zero)
    assert all(torch.equal(a[n], b[n]) for n in a)


@pytest.mark.parametrize("io,d", [("f32", 64), ("bf16", 128), ("bf16", 64)])
def test_strided_rows(io, d):
    """q, k and v as slices of one projection, dO with rows apart."""
    import uncertainty_aware_delta_gb300 as kdn

    H, T = 2, 100
    z = torch.randn(2, T, 3 * H, d, device="cuda").to(IO[io])
    q, k, v = z.split(H, 2)
    wide = torch.randn(2, T, H, 2 * d, device="cuda").to(IO[io])
    dO, S0, dS = wide[..., d:], torch.randn(2, H, d, d, device="cuda"), torch.randn(2, H, d, d, device="cuda")
    l = torch.tensor([-0.01, -0.3], device="cuda")
    dense = [t.contiguous() for t in (q, k, v)]
    for a, b in zip(kdn.kdn_decay_forward(q, k, v, l, S0), kdn.kdn_decay_forward(*dense, l, S0)):
        assert torch.equal(a, b)
    a, b = kdn.kdn_decay_backward(q, k, v, l, S0, dO, dS), kdn.kdn_decay_backward(*dense, l, S0, dO.contiguous(), dS)
    assert all(torch.equal(a[n], b[n]) for n in a)


@pytest.mark.parametrize("io,d", [("f32", 64), ("bf16", 128), ("bf16", 64)])
def test_heads_outermost(io, d):
    """[H, tokens, d] in memory; one head, and one token a sequence, whose strides mean nothing."""
    import uncertainty_aware_delta_gb300 as kdn

    H, T = 3, 130
    q, k, v, dO = (torch.randn(H, T, d, device="cuda").to(IO[io]).transpose(0, 1)[None] for _ in range(4))
    l, S0 = torch.tensor([-0.01, -0.3, 0.0], device="cuda"), torch.randn(1, H, d, d, device="cuda")
    dense = [t.contiguous() for t in (q, k, v)]
    for a, b in zip(kdn.kdn_decay_forward(q, k, v, l, S0), kdn.kdn_decay_forward(*dense, l, S0)):
        assert torch.equal(a, b)
    a, b = kdn.kdn_decay_backward(q, k, v, l, S0, dO, S0), kdn.kdn_decay_backward(*dense, l, S0, dO.contiguous(), S0)
    assert all(torch.equal(a[n], b[n]) for n in a)
    wide = torch.randn(5, 1, 1, 3 * d, device="cuda").to(IO[io])
    args = lambda t: (t[..., :d], t[..., d:2 * d], t[..., 2 * d:])   # noqa: E731
    S0 = torch.randn(5, 1, d, d, device="cuda")
    for a, b in zip(kdn.kdn_decay_forward(*args(wide), l[:1], S0), kdn.kdn_decay_forward(*(t.contiguous() for t in args(wide)), l[:1], S0)):
        assert torch.equal(a, b)
    # rows that overlap, or sequences that do not lie one after another, are refused
    with pytest.raises((ValueError, kdn.KDNError)):
        kdn.kdn_decay_forward(dense[0].expand(2, T, H, d), *(t.expand(2, T, H, d) for t in dense[1:]), l)
    two = torch.randn(2, 200, H, d, device="cuda").to(IO[io])[:, :T]
    with pytest.raises(ValueError, match="one after another"):
        kdn.kdn_decay_forward(two, two, two, l)


@pytest.mark.parametrize("io,dk,dv", [("f32", 128, 128), ("bf16", 128, 128), ("bf16", 64, 128), ("f32", 16, 32)])
def test_steps_continue_a_prompt(io, dk, dv):
    """A prompt, its last tokens one at a time: the whole sequence's outputs and state."""
    import uncertainty_aware_delta_gb300 as kdn

    x = inputs([90] * 3, 4, dk, dv, io, False)
    q, k, v, l = (x[n] for n in ("q", "k", "v", "log_decay"))
    want, size = ref.forward(q, k, v, l, x["S0"])
    o, S = kdn.kdn_decay_forward(*(t[:, :80].contiguous() for t in (q, k, v)), l, x["S0"])
    ref.check(o, want[0][:, :80], size[0][:, :80], on_tensor_cores(io, dk, dv), "o")
    for t in range(80, 90):
        o = kdn.kdn_decay_step(*(y[:, t].contiguous() for y in (q, k, v)), l, S)
        ref.check(o, want[0][:, t], size[0][:, t], False, "step")
    ref.check(S, want[1], size[1], False, "S")


def test_resumed_in_place():
    import uncertainty_aware_delta_gb300 as kdn

    for io, T in (("f32", 40), ("bf16", 40), ("bf16", 1200)):
        x = inputs([T], 1, 128, 128, io, False)
        o, S = kdn.kdn_decay_forward(x["q"], x["k"], x["v"], x["log_decay"], x["S0"])
        state = x["S0"].clone()
        o2, S2 = kdn.kdn_decay_forward(x["q"], x["k"], x["v"], x["log_decay"], state, out=(torch.empty_like(o), state))
        assert torch.equal(o, o2) and torch.equal(S, S2) and S2 is state


@pytest.mark.parametrize("io,d,flags", [("f32", 32, 0), ("bf16", 128, 0), ("bf16", 64, 0), ("bf16", 128, 1)])
@pytest.mark.parametrize("name", ["q", "k", "v"])
@pytest.mark.parametrize("bad", [float("inf"), float("nan")])
def test_what_is_not_finite(io, d, flags, name, bad):
    """A value at one token leaves earlier tokens, the other head and the other sequence as they were, and shows where it is seen."""
    import uncertainty_aware_delta_gb300 as kdn

    lengths, at = [75, 70], 75 - 35     # (in the middle of a chunk; the second sequence begins in the first's last chunk)
    x = inputs(lengths, 2, d, d, io, True)
    args = lambda: (x["q"], x["k"], x["v"], x["log_decay"], x["S0"])   # noqa: E731
    o, S = kdn.kdn_decay_forward(*args(), cu=x["cu"], flags=flags)
    x[name][at, 1, 5] = bad
    o2, S2 = kdn.kdn_decay_forward(*args(), cu=x["cu"], flags=flags)
    same = torch.ones(o.shape, dtype=torch.bool, device="cuda")
    if name == "q":
        same[at, 1] = False
    elif name == "k":
        same[at:75, 1] = False
    else:
        same[at:75, 1, 5] = False
    assert torch.equal(o[same], o2[same]) and not bool(torch.isfinite(o2[~same]).any())
    assert torch.equal(S[1], S2[1]) and torch.equal(S[0, 0], S2[0, 0])
    assert bool(torch.isfinite(S2[0, 1]).all()) == (name == "q")
    # the second sequence's first tokens share a chunk's rows with the first's last
    x[name][at, 1, 5] = 0.5
    x[name][75, 1, 5] = bad
    o2, S2 = kdn.kdn_decay_forward(*args(), cu=x["cu"], flags=flags)
    x[name][75, 1, 5] = 0.5
    o3, S3 = kdn.kdn_decay_forward(*args(), cu=x["cu"], flags=flags)
    assert torch.equal(o2[:75], o3[:75]) and torch.equal(S2[0], S3[0])


@pytest.mark.parametrize("io,d", [("f32", 64), ("bf16", 128)])
def test_rows_of_no_sequence(io, d):
    import uncertainty_aware_delta_gb300 as kdn

    x = inputs([70, 60], 2, d, d, io, True)
    cu = torch.tensor([10, 45, 110], dtype=torch.int32, device="cuda")
    o, S = torch.full_like(x["v"], 7), torch.empty_like(x["S0"])
    kdn.kdn_decay_forward(x["q"], x["k"], x["v"], x["log_decay"], x["S0"], cu=cu, out=(o, S))
    assert bool((o[:10] == 7).all()) and bool((o[110:] == 7).all())
    want, size = ref.forward(*(x[n][10:110] for n in ("q", "k", "v")), x["log_decay"], x["S0"], [0, 35, 100])
    ref.check(o[10:110], want[0], size[0], on_tensor_cores(io, d, d), "o")
    ref.check(S, want[1], size[1], False, "S_T")


@pytest.mark.parametrize("io,d", [("f32", 64), ("bf16", 128)])
def test_bounds_out_of_order(io, d):
    """Such a sequence counts as empty; the status word says so.  (Rows 60 to 70 of the first bounds lie in two sequences.)"""
    import uncertainty_aware_delta_gb300 as kdn

    x = inputs([70, 60, 20], 2, d, d, io, True)
    good = kdn.kdn_decay_forward(x["q"], x["k"], x["v"], x["log_decay"], x["S0"], cu=x["cu"])
    for bad, rows in (([0, 70, 60, 150], slice(0, 60)), ([-1, 70, 130, 151], slice(70, 130)), ([0, 70, 130, 1 << 30], slice(0, 130))):
        cu = torch.tensor(bad, dtype=torch.int32, device="cuda")
        ws = torch.empty(kdn.decay_workspace_size(3, 150, 2, d, d, int(io == "bf16")), dtype=torch.uint8, device="cuda")
        o, S = torch.full_like(x["v"], 7), torch.empty_like(x["S0"])
        kdn.kdn_decay_forward(x["q"], x["k"], x["v"], x["log_decay"], x["S0"], cu=cu, out=(o, S), workspace=ws)
        assert kdn.kdn_read_device_status(ws) == 9
        assert torch.equal(o[rows], good[0][rows])
    assert torch.equal(S[2], x["S0"][2]) and torch.equal(S[:2], good[1][:2]) and bool((o[130:] == 7).all())


@pytest.mark.parametrize("io,d", [("f32", 32), ("f32", 128), ("bf16", 64), ("bf16", 128)])
@pytest.mark.parametrize("T", [1, 40, 1300])
def test_status_word(io, d, T):
    """Whatever the workspace held before: nothing found is zero, on every path, whole and in segments."""
    import uncertainty_aware_delta_gb300 as kdn

    x = inputs([T], 1, d, d, io, False)
    args = tuple(x[n] for n in ("q", "k", "v", "log_decay", "S0"))
    sizes = (1, T, 1, d, d, int(io == "bf16"))
    ws = torch.full((kdn.decay_workspace_size(*sizes),), 255, dtype=torch.uint8, device="cuda")
    kdn.kdn_decay_forward(*args, workspace=ws)
    assert kdn.kdn_read_device_status(ws) == 0
    ws = torch.full((kdn.decay_backward_workspace_size(*sizes),), 255, dtype=torch.uint8, device="cuda")
    kdn.kdn_decay_backward(*args, x["dO"], x["dS"], workspace=ws)
    assert kdn.kdn_read_device_status(ws) == 0


def test_nothing_to_do():
    import uncertainty_aware_delta_gb300 as kdn

    for io in ("f32", "bf16"):
        for B, T, H in ((0, 5, 2), (2, 0, 2), (2, 5, 0)):
            q = torch.zeros(B, T, H, 128, dtype=IO[io], device="cuda")
            l, S0 = -torch.ones(H, device="cuda"), torch.randn(B, H, 128, 128, device="cuda")
            o, S = kdn.kdn_decay_forward(q, q, q, l, S0)
            assert o.shape == q.shape and torch.equal(S, S0)
            g = kdn.kdn_decay_backward(q, q, q, l, S0, q, S0)
            assert torch.equal(g["S0"], S0)
        assert kdn.kdn_decay_step(q[:, 0], q[:, 0], q[:, 0], l, S0).shape == (2, 0, 128)


@pytest.mark.parametrize("io,d", [("f32", 64), ("bf16", 128)])
def test_gradients_against_differences(io, d):
    """L(x + e u) - L(x - e u) of the definition for a direction u of every input."""
    import uncertainty_aware_delta_gb300 as kdn

    x = inputs([70], 2, d, d, io, False)
    g = kdn.kdn_decay_backward(x["q"], x["k"], x["v"], x["log_decay"], x["S0"], x["dO"], x["dS"])
    host = {n: x[n].cpu().double() for n in ("q", "k", "v", "S0")}
    _, size = ref.backward(*(x[n] for n in ("q", "k", "v", "log_decay", "S0", "dO", "dS")))

    def loss(y):
        o, S = ref.walk(y["q"][0], y["k"][0], y["v"][0], x["log_decay"].cpu(), y["S0"][0])
        return float((o * x["dO"].cpu().double()[0]).sum() + (S * x["dS"].cpu().double()[0]).sum())

    for i, name in enumerate(("q", "k", "v", "S0")):
        u = torch.randn(host[name].shape, generator=torch.Generator().manual_seed(i), dtype=torch.float64)
        e = 1e-3                  # (L is linear in each input alone: no error of the difference but 2^-53 / e)
        d1 = (loss({**host, name: host[name] + e * u}) - loss({**host, name: host[name] - e * u})) / (2 * e)
        tol = (ref.FP32 + ref.HALF[g[name].dtype] + (2 ** -7 if io == "bf16" and name != "S0" else 0)) * float((u.abs() * size[i]).sum())
        assert abs(float((g[name].cpu().double() * u).sum()) - d1) <= tol + 1e-9 * abs(d1), name
