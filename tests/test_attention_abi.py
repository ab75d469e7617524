"""Host-side checks of the attention entry points: refused before anything is enqueued, so no GPU is needed."""
import ctypes

import pytest


@pytest.fixture(scope="module")
def lib():
    from uncertainty_aware_delta_gb300.build import build_library
    import uncertainty_aware_delta_gb300 as kdn

    build_library()
    return kdn.library()


vp = lambda x: None if x is None else ctypes.c_void_p(x)   # noqa: E731
MB = 1 << 20


def test_sizes(lib):
    assert lib.kdn_cache_size(3, 64, 2, 128) == 3 * 2 * 64 * 144   # 4.5 bits a value, keys and values
    for page, d in ((8, 64), (24, 64), (2048, 64), (16, 16), (16, 96), (0, 64)):
        assert lib.kdn_cache_size(3, page, 2, d) == 0
    assert lib.kdn_cache_size(-1, 16, 2, 64) == 0
    ws = lib.kdn_cache_attention_workspace_size
    assert ws(4, 8, 2, 64, 100, 0) >= 256 and ws(4, 8, 2, 64, 10 ** 6, 0) >= 256
    assert ws(4, 8, 3, 64, 100, 0) == 0 and ws(4, 8, 2, 48, 100, 0) == 0 and ws(-1, 8, 2, 64, 100, 0) == 0
    ps = lib.kdn_prompt_attention_workspace_size
    assert ps(2, 100, 8, 2, 64, 1, 0) >= 256
    assert ps(2, 100, 8, 3, 64, 1, 0) == 0 and ps(2, 100, 8, 2, 48, 1, 0) == 0 and ps(2, 100, 8, 2, 64, 2, 0) == 0


def test_plan_refusals(lib):
    def call(n=4, page=16, width=8, n_free=20, cap=64, wsb=256, **ptr):
        p = dict(ctx=MB, new=2 * MB, table=3 * MB, free=4 * MB, count=5 * MB, slot=6 * MB, pos=7 * MB, cu=8 * MB, lens=9 * MB,
                 gr=10 * MB, left=11 * MB, ws=12 * MB)
        p.update(ptr)
        a = [vp(x) for x in p.values()]
        return lib.kdn_cache_plan(n, page, width, n_free, cap, *a, wsb, None)

    assert call(n=-1) == 2 and call(cap=-1) == 2 and call(width=1 << 28) == 2
    assert call(page=24) == 6 and call(page=0) == 6 and call(n=16385) == 6
    assert call(ws=None) == 5 and call(wsb=128) == 5
    for name in ("ctx", "new", "table", "free", "count", "slot", "pos", "cu", "lens", "gr", "left"):
        assert call(**{name: None}) == 1, name
    assert call(slot=6 * MB + 8) == 4
    assert call(slot=3 * MB) == 10 and call(lens=MB) == 10 and call(left=5 * MB) == 10


def test_write_and_read_refusals(lib):
    def write(n=4, pages=3, page=16, heads=2, d=64, io=1, k=MB, kr=128, kh=64, v=2 * MB, vr=128, vh=64, slot=3 * MB, cache=4 * MB):
        return lib.kdn_cache_write(n, pages, page, heads, d, io, vp(k), kr, kh, vp(v), vr, vh, vp(slot), vp(cache), None)

    assert write(io=2) == 3 and write(n=-1) == 2 and write(d=96) == 6 and write(page=20) == 6
    for name in ("k", "v", "slot", "cache"):
        assert write(**{name: None}) == 1
        assert write(**{name: 5 * MB + 8}) == 4
    assert write(kr=0) == 2 and write(kr=-128) == 2 and write(kh=32) == 2 and write(kr=64) == 2
    assert write(kr=132) == 4 and write(vh=68, vr=1000) == 4
    assert write(cache=MB) == 10 and write(slot=4 * MB + 64) == 10
    assert write(n=0, k=None) == 0

    def read(n=4, pages=3, page=16, heads=2, d=64, io=1, cache=4 * MB, slot=3 * MB, k=MB, v=2 * MB):
        return lib.kdn_cache_read(n, pages, page, heads, d, io, vp(cache), vp(slot), vp(k), vp(v), None)

    assert read(io=7) == 3 and read(d=16) == 6 and read(k=None) == 1 and read(v=2 * MB + 4) == 4
    assert read(k=2 * MB + 16) == 10 and read(v=4 * MB) == 10 and read(n=0) == 0


def test_cache_attention_refusals(lib):
    def call(n=3, H=4, hkv=2, d=64, page=16, pages=9, width=4, top=60, window=0, scale=0.0, io=1, q=MB, row=256, head=64,
             cache=2 * MB, table=3 * MB, lens=4 * MB, o=5 * MB, lse=6 * MB, ws=7 * MB, wsb=MB):
        return lib.kdn_cache_attention(n, H, hkv, d, page, pages, width, top, window, scale, io, vp(q), row, head, vp(cache),
                                       vp(table), vp(lens), vp(o), vp(lse), vp(ws), wsb, None)

    assert call(io=2) == 3 and call(H=5) == 2 and call(hkv=0) == 2 and call(window=-1) == 2 and call(top=-1) == 2
    assert call(scale=-1.0) == 2 and call(scale=float("inf")) == 2 and call(scale=float("nan")) == 2
    assert call(d=16) == 6 and call(page=40) == 6 and call(ws=None) == 5 and call(wsb=0) == 5
    for name in ("q", "cache", "table", "lens", "o", "lse"):
        assert call(**{name: None}) == 1, name
        assert call(**{name: 8 * MB + 8}) == 4, name
    assert call(row=64) == 2 and call(row=260) == 4
    assert call(o=MB) == 10 and call(lse=5 * MB) == 10 and call(ws=2 * MB) == 10


def test_prompt_attention_refusals(lib):
    def call(n=2, nq=40, nk=40, H=4, hkv=2, d=64, window=0, scale=0.0, io=1, flags=0, q=MB, qr=256, qh=64, k=2 * MB, kr=128,
             kh=64, v=3 * MB, vr=128, vh=64, cq=4 * MB, ck=5 * MB, o=6 * MB, lse=7 * MB, ws=8 * MB, wsb=MB):
        return lib.kdn_prompt_attention(n, nq, nk, H, hkv, d, window, scale, io, flags, vp(q), qr, qh, vp(k), kr, kh, vp(v), vr,
                                        vh, vp(cq), vp(ck), vp(o), vp(lse), vp(ws), wsb, None)

    assert call(io=2) == 3 and call(H=3) == 2 and call(n=-1) == 2 and call(window=-2) == 2 and call(scale=-0.1) == 2
    assert call(d=48) == 6 and call(flags=2) == 6 and call(ws=None) == 5 and call(wsb=100) == 5
    for name in ("q", "k", "v", "cq", "o", "lse"):
        assert call(**{name: None}) == 1, name
    for name in ("q", "k", "v", "cq", "ck", "o", "lse"):
        assert call(**{name: 9 * MB + 8}) == 4, name
    assert call(qr=128) == 2 and call(kh=0) == 2 and call(vr=132) == 4 and call(kr=-128) == 2
    assert call(nk=39, ck=None) == 2
    assert call(o=MB) == 10 and call(lse=6 * MB + 64) == 10 and call(ws=3 * MB) == 10 and call(o=4 * MB - 64) == 10
