"""Group norm with an activation, and its gradients, against their definition in 64 bits (tolerances: retention_oracle.py)."""
import pytest
import torch

import retention_oracle as ref

pytestmark = pytest.mark.gpu
IO = {"f32": torch.float32, "bf16": torch.bfloat16}


def inputs(rows, G, d, io, gate, affine, seed=0):
    g = torch.Generator().manual_seed(seed)
    rand = lambda *s: torch.randn(s, generator=g)   # noqa: E731
    x = ((rand(rows, G, d) + 0.5 * rand(1, G, d)) * torch.exp(rand(rows, G, 1))).to(IO[io]).cuda()
    z, dy = (rand(rows, G, d).to(IO[io]).cuda() for _ in range(2))
    w, b = 1 + 0.2 * rand(G, d).cuda(), 0.2 * rand(G, d).cuda()
    return x, dy, z if gate else None, w if affine & 1 else None, b if affine & 2 else None


def check_all(rows, G, d, io, act, gate, affine, eps=1e-5):
    import uncertainty_aware_delta_gb300 as kdn

    x, dy, z, w, b = inputs(rows, G, d, io, gate, affine)
    y = kdn.kdn_group_norm(x, w, b, gate=z, act=act, eps=eps)
    ref.check_norm(y, ref.norm(x, w, b, z, act, eps)["y"], "y")
    got, want = kdn.kdn_group_norm_backward(x, dy, w, b, gate=z, act=act, eps=eps), ref.norm(x, w, b, z, act, eps, dy)
    assert {n for n, t in got.items() if t is not None} == set(want)
    for name in want:
        ref.check_norm(got[name], want[name], name)


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("act", ["none", "silu", "sigmoid"])
@pytest.mark.parametrize("gate", [False, True])
@pytest.mark.parametrize("affine", [0, 1, 2, 3])
def test_forms(io, act, gate, affine):
    check_all(37, 3, 64, io, act, gate, affine)


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("rows,G,d", [(1, 1, 8), (1, 1, 256), (5, 33, 16), (1000, 1, 24), (3, 70, 40), (2, 9, 128), (300, 17, 72),
                                      (11, 4, 248), (2, 300, 8), (4001, 2, 32), (9, 12, 256)])
def test_sizes(io, rows, G, d):
    check_all(rows, G, d, io, "silu", True, 3)


@pytest.mark.parametrize("io", ["f32", "bf16"])
def test_strided_rows(io):
    import uncertainty_aware_delta_gb300 as kdn

    z = torch.randn(2, 50, 8, 192, device="cuda").to(IO[io])
    x, gate, dy = z[:, :, :3, 64:128], z[:, :, 3:6, :64], z[:, :, 5:8, 128:]
    w, b = torch.randn(3, 64, device="cuda"), torch.randn(3, 64, device="cuda")
    dense = [t.contiguous() for t in (x, dy, gate)]
    assert torch.equal(kdn.kdn_group_norm(x, w, b, gate=gate, act="sigmoid"), kdn.kdn_group_norm(dense[0], w, b, gate=dense[2], act="sigmoid"))
    a = kdn.kdn_group_norm_backward(x, dy, w, b, gate=gate, act="sigmoid")
    c = kdn.kdn_group_norm_backward(dense[0], dense[1], w, b, gate=dense[2], act="sigmoid")
    assert all(torch.equal(a[n], c[n]) for n in a)


@pytest.mark.parametrize("eps", [0.0, 1e-3, 10.0])
def test_eps(eps):
    check_all(20, 2, 64, "f32", "silu", False, 3, eps)


def test_constant_groups():
    """Deviations of zero: the norm is the bias, and the gradient is not divided by zero."""
    import uncertainty_aware_delta_gb300 as kdn

    x, b = torch.full((4, 2, 64), 3.0, device="cuda"), torch.randn(2, 64, device="cuda")
    assert torch.equal(kdn.kdn_group_norm(x, None, b), b.expand(4, 2, 64))
    dy = torch.randn(4, 2, 64, device="cuda")
    g = kdn.kdn_group_norm_backward(x, dy, None, b)
    ref.check_norm(g["x"], ref.norm(x, None, b, None, "none", 1e-5, dy)["x"])


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("bad", [float("inf"), float("nan")])
def test_what_is_not_finite(io, bad):
    """stays in its group of its row."""
    import uncertainty_aware_delta_gb300 as kdn

    x, dy, z, w, b = inputs(40, 5, 72, io, True, 3)
    y, g = kdn.kdn_group_norm(x, w, b, gate=z, act="silu"), kdn.kdn_group_norm_backward(x, dy, w, b, gate=z, act="silu")
    x[7, 2, 3] = bad
    y2, g2 = kdn.kdn_group_norm(x, w, b, gate=z, act="silu"), kdn.kdn_group_norm_backward(x, dy, w, b, gate=z, act="silu")
    same = torch.ones(40, 5, dtype=torch.bool, device="cuda")
    same[7, 2] = False
    assert torch.equal(y[same], y2[same]) and bool(torch.isnan(y2[7, 2]).all())
    assert all(torch.equal(g[n][same], g2[n][same]) for n in ("x", "gate"))
    assert all(torch.equal(g[n][[0, 1, 3, 4]], g2[n][[0, 1, 3, 4]]) for n in ("weight", "bias"))


def test_large_gates():
    import uncertainty_aware_delta_gb300 as kdn

    x = torch.randn(8, 2, 64, device="cuda")
    gate = torch.linspace(-200, 200, 1024, device="cuda").view(8, 2, 64)
    for act in ("silu", "sigmoid"):
        ref.check_norm(kdn.kdn_group_norm(x, gate=gate, act=act), ref.norm(x, None, None, gate, act, 1e-5)["y"])
        g, want = kdn.kdn_group_norm_backward(x, x, gate=gate, act=act), ref.norm(x, None, None, gate, act, 1e-5, x)
        for n in ("x", "gate"):
            ref.check_norm(g[n], want[n], n)


def test_nothing_to_do():
    import uncertainty_aware_delta_gb300 as kdn

    x, w = torch.empty(0, 3, 64, device="cuda"), torch.ones(3, 64, device="cuda")
    assert kdn.kdn_group_norm(x, w).shape == x.shape
    g = kdn.kdn_group_norm_backward(x, x, w, w)
    assert bool((g["weight"] == 0).all()) and bool((g["bias"] == 0).all())


def test_sums_do_not_depend_on_the_run():
    import uncertainty_aware_delta_gb300 as kdn

    x, dy, z, w, b = inputs(5000, 3, 64, "bf16", True, 3)
    a, c = (kdn.kdn_group_norm_backward(x, dy, w, b, gate=z, act="silu") for _ in range(2))
    assert all(torch.equal(a[n], c[n]) for n in a)


@pytest.mark.parametrize("act,gate", [("silu", False), ("sigmoid", True)])
def test_gradients_against_differences(act, gate):
    import uncertainty_aware_delta_gb300 as kdn

    x, dy, z, w, b = inputs(6, 2, 32, "f32", gate, 3)
    got = kdn.kdn_group_norm_backward(x, dy, w, b, gate=z, act=act)
    host = {"x": x, "gate": z, "weight": w, "bias": b}
    host = {n: t.cpu().double() for n, t in host.items() if t is not None}

    def loss(t):
        y, _ = ref.norm(t["x"], t["weight"], t["bias"], t.get("gate"), act, 1e-5)["y"]
        return float((y * dy.cpu().double()).sum())

    for i, name in enumerate(host):
        u = torch.randn(host[name].shape, generator=torch.Generator().manual_seed(i), dtype=torch.float64)
        e = 1e-5
        d = (loss({**host, name: host[name] + e * u}) - loss({**host, name: host[name] - e * u})) / (2 * e)
        mine = float((got[name].cpu().double() * u).sum())
        tol = ref.norm(x, w, b, z, act, 1e-5, dy)[name]
        # fp32's part, and of the difference e^2 of the third derivative and 2^-53 / e of the loss
        assert abs(mine - d) <= float(((tol[1] + 2.0 ** -24 * tol[0].abs()) * u.abs()).sum()) + 1e-6 * abs(d) + 1e-7
