"""The retention layer's operators as a layer uses them together: memory, norm and gate, and their gradients back; in CUDA graphs,
on other streams, and two calls at once.  (Tolerances: retention_oracle.py, each operator on the tensors that it was given.)"""
import pytest
import torch

import retention_oracle as ref
from test_decay import IO, inputs, on_tensor_cores

pytestmark = pytest.mark.gpu


def layer(x, gate, w, b, dy, flags=0):
    """Outputs and gradients of a layer's core."""
    import uncertainty_aware_delta_gb300 as kdn

    o, S = kdn.kdn_decay_forward(x["q"], x["k"], x["v"], x["log_decay"], x["S0"], cu=x["cu"], flags=flags)
    y = kdn.kdn_group_norm(o, w, b, gate=gate, act="silu")
    g = kdn.kdn_group_norm_backward(o, dy, w, b, gate=gate, act="silu")
    m = kdn.kdn_decay_backward(x["q"], x["k"], x["v"], x["log_decay"], x["S0"], g["x"], x["dS"], cu=x["cu"], flags=flags)
    return {"o": o, "S": S, "y": y, "dgate": g["gate"], "dw": g["weight"], "db": g["bias"], "do": g["x"], **{"d" + n: t for n, t in m.items()}}


def make(lengths, H, dk, dv, io, packed, seed=0):
    x = inputs(lengths, H, dk, dv, io, packed, seed)
    gen = torch.Generator().manual_seed(seed + 100)
    gate, dy = (torch.randn(x["v"].shape, generator=gen).to(IO[io]).cuda() for _ in range(2))
    return x, gate, 1 + 0.1 * torch.randn(H, dv, generator=gen).cuda(), 0.1 * torch.randn(H, dv, generator=gen).cuda(), dy


@pytest.mark.parametrize("lengths,packed", [([90, 90], False), ([70, 1, 129], True), ([1300], False)])
@pytest.mark.parametrize("io,dk,dv", [("f32", 32, 64), ("bf16", 128, 128), ("bf16", 64, 128), ("bf16", 32, 32)])
def test_layer(lengths, packed, io, dk, dv):
    x, gate, w, b, dy = make(lengths, 2, dk, dv, io, packed)
    got = layer(x, gate, w, b, dy)
    tc, bounds = on_tensor_cores(io, dk, dv), None if x["cu"] is None else x["cu"].tolist()
    want, size = ref.forward(x["q"], x["k"], x["v"], x["log_decay"], x["S0"], bounds)
    ref.check(got["o"], want[0], size[0], tc, "o")
    ref.check(got["S"], want[1], size[1], False, "S")
    flat = lambda t: t.reshape(-1, *t.shape[-2:])   # noqa: E731
    ref.check_norm(flat(got["y"]), ref.norm(flat(got["o"]), w, b, flat(gate), "silu", 1e-5)["y"], "y")
    want = ref.norm(flat(got["o"]), w, b, flat(gate), "silu", 1e-5, flat(dy))
    for mine, name in (("do", "x"), ("dgate", "gate"), ("dw", "weight"), ("db", "bias")):
        ref.check_norm(got[mine].reshape(want[name][0].shape), want[name], mine)
    want, size = ref.backward(x["q"], x["k"], x["v"], x["log_decay"], x["S0"], got["do"], x["dS"], bounds)
    for i, name in enumerate(("dq", "dk", "dv", "dS0")):
        ref.check(got[name], want[i], size[i], tc and name != "dS0", name)


@pytest.mark.parametrize("lengths,packed", [([90, 90], False), ([70, 1, 129], True), ([1300], False), ([900, 20], True)])
@pytest.mark.parametrize("io,d", [("f32", 32), ("bf16", 128), ("bf16", 64)])
def test_in_a_graph(lengths, packed, io, d):
    """Captured once, replayed on new inputs, beside an eager call: the same bits."""
    a, b = make(lengths, 1, d, d, io, packed), make(lengths, 1, d, d, io, packed, seed=1)
    want = layer(*b)
    side, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    with torch.cuda.stream(side):
        layer(*a)
    torch.cuda.synchronize()
    with torch.cuda.graph(graph, stream=side):
        got = layer(*a)
    for s, t in zip([*a[0].values(), *a[1:]], [*b[0].values(), *b[1:]]):
        if s is not None:
            s.copy_(t)
    for _ in range(2):
        for t in got.values():
            t.fill_(7)
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(got[n], want[n]) for n in want)


def test_step_in_a_graph():
    import uncertainty_aware_delta_gb300 as kdn

    x = inputs([20] * 3, 2, 128, 64, "bf16", False)
    q, k, v = (x[n][:, 0].contiguous() for n in ("q", "k", "v"))
    S, o = x["S0"].clone(), torch.empty_like(v)
    side, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    with torch.cuda.stream(side):
        kdn.kdn_decay_step(q, k, v, x["log_decay"], S.clone(), o=o)
    torch.cuda.synchronize()
    with torch.cuda.graph(graph, stream=side):
        kdn.kdn_decay_step(q, k, v, x["log_decay"], S, o=o)
    want, size = ref.forward(x["q"], x["k"], x["v"], x["log_decay"], x["S0"])
    for t in range(20):
        for s, name in ((q, "q"), (k, "k"), (v, "v")):
            s.copy_(x[name][:, t])
        graph.replay()
        torch.cuda.synchronize()
        ref.check(o, want[0][:, t], size[0][:, t], False, "step")
    ref.check(S, want[1], size[1], False, "S")


@pytest.mark.parametrize("io,d,T", [("f32", 32, 300), ("bf16", 128, 300), ("bf16", 128, 1500)])
def test_on_another_stream(io, d, T):
    """Inputs made on the current stream, calls on another one; results read after the current stream waits for it."""
    import uncertainty_aware_delta_gb300 as kdn

    x, gate, w, b, dy = make([T], 2, d, d, io, False)
    want = layer(x, gate, w, b, dy)
    side = torch.cuda.Stream()
    for _ in range(3):
        torch.cuda._sleep(2_000_000)
        y = {n: None if t is None else t.clone() for n, t in x.items()}      # (not there yet when the calls are made)
        args = (y["q"], y["k"], y["v"], y["log_decay"], y["S0"])
        o, S = kdn.kdn_decay_forward(*args, stream=side)
        z = kdn.kdn_group_norm(o, w, b, gate=gate, act="silu", stream=side)
        g = kdn.kdn_group_norm_backward(o, dy, w, b, gate=gate, act="silu", stream=side)
        m = kdn.kdn_decay_backward(*args, g["x"], y["dS"], stream=side)
        state = y["S0"].clone()
        step = kdn.kdn_decay_step(y["q"][:, 0].contiguous(), y["k"][:, 0].contiguous(), y["v"][:, 0].contiguous(), y["log_decay"], state,
                                  stream=side)
        torch.cuda.current_stream().wait_stream(side)
        got = {"o": o, "S": S, "y": z, "dgate": g["gate"], "dw": g["weight"], "db": g["bias"], "do": g["x"], **{"d" + n: t for n, t in m.items()}}
        assert all(torch.equal(got[n], want[n]) for n in want)
        one, size = ref.forward(*(x[n][:, :1] for n in ("q", "k", "v")), x["log_decay"], x["S0"])
        ref.check(step, one[0][:, 0], size[0][:, 0], False, "step")
        ref.check(state, one[1], size[1], False, "S")


@pytest.mark.parametrize("io,d", [("f32", 64), ("bf16", 128)])
def test_two_calls_at_once(io, d):
    """On two streams, each with a workspace of its own."""
    import uncertainty_aware_delta_gb300 as kdn

    both = [make([1200, 1200], 2, d, d, io, False, seed)[0] for seed in (0, 1)]
    want = [kdn.kdn_decay_backward(*(x[n] for n in ("q", "k", "v", "log_decay", "S0", "dO", "dS"))) for x in both]
    streams = [torch.cuda.Stream() for _ in both]
    torch.cuda.synchronize()
    for _ in range(3):
        got = []
        for x, s in zip(both, streams):
            with torch.cuda.stream(s):
                got.append(kdn.kdn_decay_backward(*(x[n] for n in ("q", "k", "v", "log_decay", "S0", "dO", "dS"))))
        torch.cuda.synchronize()
        assert all(torch.equal(a[n], b[n]) for a, b in zip(got, want) for n in a)


def test_two_graphs_share_a_workspace():
    """Replayed one after another on one stream."""
    import uncertainty_aware_delta_gb300 as kdn

    both = [inputs([1300], 1, 128, 128, "bf16", False, seed) for seed in (0, 1)]
    args = [tuple(x[n] for n in ("q", "k", "v", "log_decay", "S0")) for x in both]
    want = [kdn.kdn_decay_forward(*a) for a in args]
    ws = torch.empty(kdn.decay_workspace_size(1, 1300, 1, 128, 128), dtype=torch.uint8, device="cuda")
    out = [tuple(torch.empty_like(t) for t in w) for w in want]
    side, graphs = torch.cuda.Stream(), [torch.cuda.CUDAGraph() for _ in both]
    torch.cuda.synchronize()
    for g, a, o in zip(graphs, args, out):
        with torch.cuda.graph(g, stream=side):
            kdn.kdn_decay_forward(*a, out=o, workspace=ws)
    for order in ((0, 1), (1, 0)):
        for i in order:
            graphs[i].replay()
        torch.cuda.synchronize()
        assert kdn.kdn_read_device_status(ws) == 0
        for o, w in zip(out, want):
            assert all(torch.equal(a, b) for a, b in zip(o, w))


def test_bounds_change_under_a_graph():
    """Packed lengths are device data: the same captured call on other lengths."""
    import uncertainty_aware_delta_gb300 as kdn

    x = inputs([700, 500], 1, 64, 64, "bf16", True)
    args = (x["q"], x["k"], x["v"], x["log_decay"], x["S0"])
    out = torch.empty_like(x["v"]), torch.empty_like(x["S0"])
    side, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    with torch.cuda.stream(side):
        kdn.kdn_decay_forward(*args, cu=x["cu"], out=out)
    torch.cuda.synchronize()
    with torch.cuda.graph(graph, stream=side):
        kdn.kdn_decay_forward(*args, cu=x["cu"], out=out)
    for middle in (700, 0, 1200, 13, 1199):
        x["cu"].copy_(torch.tensor([0, middle, 1200], dtype=torch.int32))
        graph.replay()
        torch.cuda.synchronize()
        want, size = ref.forward(*args, [0, middle, 1200])
        ref.check(out[0], want[0], size[0], True, "o")
        ref.check(out[1], want[1], size[1], False, "S")
