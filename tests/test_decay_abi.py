"""Host-side checks of the retention layer's entry points and binding: refused before anything is enqueued, so no GPU is needed."""
import ctypes

import pytest
import torch

from test_attention_abi import lib  # noqa: F401

vp = lambda x: None if x is None else ctypes.c_void_p(x)   # noqa: E731
MB = 1 << 20


def test_sizes(lib):  # noqa: F811
    for size in (lib.kdn_decay_workspace_size, lib.kdn_decay_backward_workspace_size):
        assert size(2, 200, 4, 64, 128, 1, 0) >= 256 and size(0, 0, 0, 16, 16, 0, 0) >= 256
        # few long sequences: their segments' states
        assert size(1, 65536, 2, 128, 128, 1, 0) >= 256 + 2 * 4 * 128 * 128 * 10
        assert size(1, 65536, 2, 128, 128, 1, 2) == 256
        for bad in ((-1, 200, 4, 64, 64, 1, 0), (2, -1, 4, 64, 64, 1, 0), (2, 200, -1, 64, 64, 1, 0), (2, 200, 4, 48, 64, 1, 0),
                    (2, 200, 4, 64, 256, 1, 0), (2, 200, 4, 64, 64, 2, 0), (2, 200, 4, 64, 64, 1, 4), (2, 200, 70000, 64, 64, 1, 0),
                    (2, 2 ** 31 - 1, 4, 64, 64, 1, 0)):
            assert size(*bad) == 0, bad
    norm = lib.kdn_group_norm_backward_workspace_size
    assert norm(1000, 8, 64, 1) >= 256 + 2 * 4 * 8 * 64 and norm(0, 8, 64, 0) >= 256
    for bad in ((-1, 8, 64, 1), (10, -1, 64, 1), (10, 8, 0, 1), (10, 8, 12, 1), (10, 8, 264, 1), (10, 8, 64, 3), (10, 70000, 8, 1)):
        assert norm(*bad) == 0, bad


def forward(lib, n=2, tok=8, H=2, dk=64, dv=128, io=1, flags=0, wsb=MB, strides=None, **ptr):  # noqa: F811
    p = dict(q=MB, k=2 * MB, v=3 * MB, l=4 * MB, S0=5 * MB, cu=None, o=6 * MB, S=7 * MB, ws=8 * MB)
    p.update(ptr)
    st = {"q": (H * dk, dk), "k": (H * dk, dk), "v": (H * dv, dv), **(strides or {})}
    return lib.kdn_decay_forward(n, tok, H, dk, dv, io, flags, vp(p["q"]), *st["q"], vp(p["k"]), *st["k"], vp(p["v"]), *st["v"],
                                 vp(p["l"]), vp(p["S0"]), vp(p["cu"]), vp(p["o"]), vp(p["S"]), vp(p["ws"]), wsb, None)


def test_forward_refusals(lib):  # noqa: F811
    f = lambda **a: forward(lib, **a)   # noqa: E731
    assert f(io=2) == 3 and f(n=-1) == 2 and f(tok=-2) == 2 and f(H=-1) == 2 and f(tok=9) == 2 and f(n=0) == 2
    assert f(dk=48) == 6 and f(dv=256) == 6 and f(flags=4) == 6 and f(flags=0x200) == 6
    assert f(ws=None) == 5 and f(wsb=128) == 5
    for name in ("q", "k", "v", "l", "o", "S"):
        assert f(**{name: None}) == 1, name
    for name in ("q", "k", "v", "l", "S0", "o", "S", "ws", "cu"):
        assert f(**{name: 12 * MB + 8}) == 4, name
    assert f(strides={"q": (64, 64)}) == 2 and f(strides={"k": (0, 64)}) == 2 and f(strides={"v": (256, 64)}) == 2
    assert f(strides={"q": (132, 64)}) == 4 and f(strides={"v": (1024, 132)}) == 4
    # outputs over inputs and over each other; the states may be resumed in place but not over half of each other
    assert f(o=MB) == 10 and f(S=MB + 512) == 10 and f(ws=6 * MB) == 10 and f(S=5 * MB + 64 * 128 * 4) == 10 and f(o=4 * MB) == 10
    assert f(cu=6 * MB) == 10


def test_step_refusals(lib):  # noqa: F811
    def step(B=3, H=2, dk=64, dv=32, io=0, **ptr):
        p = dict(q=MB, k=2 * MB, v=3 * MB, l=4 * MB, S=5 * MB, o=6 * MB)
        p.update(ptr)
        return lib.kdn_decay_step(B, H, dk, dv, io, *(vp(x) for x in p.values()), None)

    assert step(B=0) == 0 and step(H=0) == 0
    assert step(io=2) == 3 and step(B=-1) == 2 and step(dk=8) == 6 and step(dv=96) == 6
    for name in ("q", "k", "v", "l", "S", "o"):
        assert step(**{name: None}) == 1 and step(**{name: 8 * MB + 4}) == 4
    assert step(o=5 * MB) == 10 and step(S=MB) == 10 and step(o=3 * MB) == 10


def test_backward_refusals(lib):  # noqa: F811
    def back(n=2, tok=8, H=2, dk=64, dv=64, io=1, flags=0, wsb=MB, **ptr):
        p = dict(q=MB, k=2 * MB, v=3 * MB, l=4 * MB, S0=5 * MB, cu=None, dO=6 * MB, dS=7 * MB, gq=8 * MB, gk=9 * MB, gv=10 * MB,
                 gS=11 * MB, ws=12 * MB)
        p.update(ptr)
        s = (H * dk, dk)
        return lib.kdn_decay_backward(n, tok, H, dk, dv, io, flags, vp(p["q"]), *s, vp(p["k"]), *s, vp(p["v"]), *s, vp(p["l"]), vp(p["S0"]),
                                      vp(p["cu"]), vp(p["dO"]), *s, vp(p["dS"]), vp(p["gq"]), vp(p["gk"]), vp(p["gv"]), vp(p["gS"]),
                                      vp(p["ws"]), wsb, None)

    assert back(io=3) == 3 and back(tok=7) == 2 and back(dk=40) == 6 and back(flags=8) == 6 and back(ws=None) == 5 and back(wsb=0) == 5
    for name in ("q", "k", "v", "l", "dO", "gq", "gk", "gv", "gS"):
        assert back(**{name: None}) == 1, name
    for name in ("q", "dO", "dS", "gq", "gS", "ws", "S0"):
        assert back(**{name: 14 * MB + 8}) == 4, name
    assert back(gq=8 * MB, gk=8 * MB) == 10 and back(gq=MB) == 10 and back(gS=7 * MB) == 10 and back(ws=6 * MB) == 10


def test_norm_refusals(lib):  # noqa: F811
    def norm(rows=4, G=2, d=64, act=1, eps=1e-5, io=1, s=(128, 64), gs=(128, 64), **ptr):
        p = dict(x=MB, w=2 * MB, b=3 * MB, gate=4 * MB, y=5 * MB)
        p.update(ptr)
        return lib.kdn_group_norm(rows, G, d, act, eps, io, vp(p["x"]), *s, vp(p["w"]), vp(p["b"]), vp(p["gate"]), *gs, vp(p["y"]), None)

    assert norm(rows=0) == 0 and norm(G=0) == 0
    assert norm(io=2) == 3 and norm(rows=-1) == 2 and norm(d=60) == 6 and norm(d=264) == 6 and norm(d=0) == 6
    assert norm(act=3) == 6 and norm(act=-1) == 6 and norm(eps=-1.0) == 2 and norm(eps=float("inf")) == 2 and norm(eps=float("nan")) == 2
    assert norm(x=None) == 1 and norm(y=None) == 1 and norm(x=6 * MB + 8) == 4 and norm(gate=6 * MB + 2) == 4
    assert norm(s=(64, 64)) == 2 and norm(gs=(130, 64)) == 4 and norm(y=MB) == 10 and norm(y=4 * MB) == 10 and norm(y=2 * MB) == 10

    def back(rows=4, G=2, d=64, act=1, eps=1e-5, io=1, wsb=MB, **ptr):
        p = dict(x=MB, w=2 * MB, b=3 * MB, gate=4 * MB, dy=5 * MB, gx=6 * MB, gg=7 * MB, gw=8 * MB, gb=9 * MB, ws=10 * MB)
        p.update(ptr)
        s = (128, 64)
        return lib.kdn_group_norm_backward(rows, G, d, act, eps, io, vp(p["x"]), *s, vp(p["w"]), vp(p["b"]), vp(p["gate"]), *s, vp(p["dy"]), *s,
                                           vp(p["gx"]), vp(p["gg"]), vp(p["gw"]), vp(p["gb"]), vp(p["ws"]), wsb, None)

    assert back(io=2) == 3 and back(d=20) == 6 and back(eps=-1.0) == 2 and back(ws=None) == 5 and back(wsb=256) == 5
    for name in ("x", "dy", "gx", "gg", "gw", "gb"):
        assert back(**{name: None}) == 1, name
    assert back(gx=MB) == 10 and back(gx=7 * MB) == 10 and back(gw=9 * MB) == 10 and back(ws=5 * MB) == 10 and back(dy=12 * MB + 8) == 4


def test_binding_refuses(lib):  # noqa: F811
    import uncertainty_aware_delta_gb300 as kdn

    x, l, S = torch.zeros(2, 4, 2, 64), torch.zeros(2), torch.zeros(2, 2, 64, 64)
    cu = torch.zeros(3, dtype=torch.int32)
    for call in (lambda: kdn.kdn_decay_forward(x, x, x, l), lambda: kdn.kdn_decay_forward(x[0], x[0], x[0], l, cu=cu),
                 lambda: kdn.kdn_decay_step(x[:, 0], x[:, 0], x[:, 0], l, S), lambda: kdn.kdn_decay_backward(x, x, x, l, None, x),
                 lambda: kdn.kdn_group_norm(x), lambda: kdn.kdn_group_norm_backward(x, x)):
        with pytest.raises(TypeError, match="must be a CUDA tensor"):
            call()
    with pytest.raises(ValueError, match="need cu"):
        kdn.kdn_decay_forward(x[0], x[0], x[0], l)
    with pytest.raises(ValueError, match="packed"):
        kdn.kdn_decay_forward(x, x, x, l, cu=cu)
    with pytest.raises(ValueError, match=r"\[tokens, heads, d\]"):
        kdn.kdn_decay_forward(x[0, 0], x[0, 0], x[0, 0], l)
    with pytest.raises(ValueError, match="cu must be"):
        kdn.kdn_decay_forward(x[0], x[0], x[0], l, cu=cu[None])
    with pytest.raises(ValueError, match="act must be"):
        kdn.kdn_group_norm(x, act="gelu")
    with pytest.raises(TypeError, match="bfloat16 or float32"):
        kdn.kdn_group_norm(x.half())
    for big in (2 ** 31, 2 ** 32, -2 ** 31 - 1):
        with pytest.raises(ValueError, match="flags"):
            kdn.kdn_decay_forward(x, x, x, l, flags=big)
        with pytest.raises(ValueError, match="n_tok"):
            kdn.decay_workspace_size(1, big, 2, 64, 64)
        with pytest.raises(ValueError, match="rows"):
            kdn.group_norm_backward_workspace_size(big, 2, 64)
