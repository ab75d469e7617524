"""Attention of one token per sequence over the 4-bit cache, against fp64 on the cache's own values."""
import math

import numpy as np
import pytest

import attention_oracle as ref

pytestmark = pytest.mark.gpu


def _setup(lens, H, hkv, d, page, io, seed=0, gain=1.0, v_gain=1.0, extra=2):
    import torch
    import uncertainty_aware_delta_gb300 as kdn

    rng = np.random.default_rng(seed)
    lens = np.asarray(lens)
    held = -(-lens // page)
    pages = int(held.sum()) + extra
    width = int(held.max(initial=0)) + 1
    g = torch.Generator().manual_seed(seed)
    dt = torch.bfloat16 if io == "bf16" else torch.float32
    n = pages * page
    k = torch.randn((n, hkv, d), generator=g) * gain
    v = torch.randn((n, hkv, d), generator=g) * torch.exp(torch.randn((n, hkv, 1), generator=g)) * v_gain
    q = torch.randn((len(lens), H, d), generator=g)
    cache = kdn.cache_alloc(pages, page, hkv, d)
    kdn.kdn_cache_write(k.to(dt).cuda(), v.to(dt).cuda(), torch.arange(n).cuda(), cache)
    ids = rng.permutation(pages)
    table = np.full((len(lens), width), -1, np.int64)
    for r, h in enumerate(held):
        table[r, :h], ids = ids[:h], ids[h:]
    return q.to(dt).cuda(), cache, torch.from_numpy(table.astype(np.int32)).cuda(), torch.from_numpy(
        lens.astype(np.int32)).cuda()


def _expect(q, cache, table, lens, window, scale=None, drop=()):
    d = q.shape[2]
    ck, sk, cv, sv = ref.unpack(cache.cpu().numpy(), d)
    k, v = ref.values(ck, sk), ref.values(cv, sv)      # [pages, heads, page, d]
    qn, table, lens = q.double().cpu().numpy(), table.cpu().numpy(), lens.cpu().numpy()
    rep, out = q.shape[1] // cache.shape[1], []
    page = k.shape[2]
    for r in range(len(lens)):
        n = max(int(lens[r]), 0)
        ids = table[r, :-(-n // page)]
        for h in range(q.shape[1]):
            kk = np.concatenate([k[i, h // rep] for i in ids] or [k[0, 0][:0]])[:n]
            vv = np.concatenate([v[i, h // rep] for i in ids] or [v[0, 0][:0]])[:n]
            out.append(ref.attend(qn[r, h], kk, vv, scale or 1 / math.sqrt(d), max(0, n - window) if window else 0, n))
    shape = q.shape[:2]
    return (np.array([o for o, _, _, _ in out]).reshape(q.shape), np.array([x for _, x, _, _ in out]).reshape(shape),
            np.array([a for _, _, a, _ in out]).reshape(q.shape), np.array([e for _, _, _, e in out]).reshape(shape))


def _floor(cache, lens):
    """What fp16's subnormal range may lose of a row (attention_oracle's derivation), over all keys of the cache."""
    d = cache.shape[3] // 18
    _, _, code, s = ref.unpack(cache.cpu().numpy(), d)
    s = np.nan_to_num(s)
    return max(lens) * 2.0 ** -34 * 7 * s.max() * max(1.0, 2.0 ** -5 / max(s.max(), 2.0 ** -24))


def _run(lens, H, hkv, d, page, io, window=0, max_len=None, scale=None, **more):
    import torch
    import uncertainty_aware_delta_gb300 as kdn

    q, cache, table, n = _setup(lens, H, hkv, d, page, io, **more)
    top = max(max(lens), 0) if max_len is None else max_len
    ws = torch.empty(kdn.cache_attention_workspace_size(len(lens), H, hkv, d, top, window), dtype=torch.uint8, device="cuda")
    o, lse = kdn.kdn_cache_attention(q, cache, table, n, max_len=top, window=window, scale=scale, workspace=ws)
    ref.check(o.double().cpu().numpy(), lse.double().cpu().numpy(), _expect(q, cache, table, n, window, scale), io, True,
              _floor(cache, lens))
    assert kdn.kdn_read_device_status(ws) == 0
    again = kdn.kdn_cache_attention(q, cache, table, n, max_len=top, window=window, scale=scale)
    assert torch.equal(again[0], o) and torch.equal(again[1], lse)


LENS = [0, 1, 15, 16, 17, 63, 64, 65, 130, 257]


@pytest.mark.parametrize("io", ["bf16", "f32"])
@pytest.mark.parametrize("H,hkv,d,page", [(1, 1, 32, 16), (8, 1, 64, 16), (6, 2, 128, 48), (12, 1, 128, 64), (16, 4, 64, 32),
                                          (40, 2, 32, 128), (5, 5, 128, 1024)])
@pytest.mark.parametrize("window", [0, 1, 50])
def test_lengths(H, hkv, d, page, io, window):
    _run(LENS, H, hkv, d, page, io, window)


@pytest.mark.parametrize("io", ["bf16", "f32"])
@pytest.mark.parametrize("lens,window", [([5000], 0), ([3001, 7, 12345], 0), ([9000, 100], 4097), ([20000], 0)])
def test_long(lens, window, io):
    _run(lens, 4, 2, 64 if window else 128, 64, io, window)


def test_loose_bound_and_scale():
    _run([100, 3, 700], 8, 2, 64, 32, "bf16", max_len=50000)
    _run([100, 3, 700], 8, 2, 64, 32, "bf16", scale=0.7)


@pytest.mark.parametrize("io", ["bf16", "f32"])
@pytest.mark.parametrize("gain,v_gain", [(1e-4, 1e-4), (20.0, 300.0), (1.0, 1e4), (1e3, 1e-2)])
def test_magnitudes(gain, v_gain, io):
    """Scores far apart, and values whose scales lie near fp16's ends."""
    _run([300, 40], 4, 2, 64, 32, io, gain=gain, v_gain=v_gain)


def test_garbage_outside_the_sequence_has_no_influence():
    import torch
    import uncertainty_aware_delta_gb300 as kdn

    for d in (32, 64, 128):
        q, cache, table, n = _setup([33, 70, 16], 8, 2, d, 32, "bf16")
        want = kdn.kdn_cache_attention(q, cache, table, n, max_len=70, window=20)
        dirty = torch.full_like(cache, 0xff)   # NaN scales
        place = torch.zeros(cache.shape[0], cache.shape[2], 16, dtype=torch.bool)
        for r, m in enumerate(n.tolist()):
            for t in range(max(0, m - 20), m):
                place[table[r, t // 32], t % 32 // 16, t % 16] = True
        # copy the seen tokens only
        slots = place.flatten().nonzero().flatten().cuda()
        k, v = kdn.kdn_cache_read(cache, slots, dtype=torch.float32)
        kdn.kdn_cache_write(k, v, slots, dirty)
        k2, v2 = kdn.kdn_cache_read(dirty, slots, dtype=torch.float32)
        ref_o = _expect(q, dirty, table, n, 20)
        got = kdn.kdn_cache_attention(q, dirty, table, n, max_len=70, window=20)
        ref.check(got[0].double().cpu().numpy(), got[1].double().cpu().numpy(), ref_o, "bf16", True)
        assert torch.isfinite(got[0].float()).all() and want[0].shape == got[0].shape


def test_visible_nan_reaches_its_rows_only():
    import torch
    import uncertainty_aware_delta_gb300 as kdn

    q, cache, table, n = _setup([40, 40], 4, 2, 64, 32, "f32")
    x = torch.randn(1, 2, 64, device="cuda")
    x[0, 1, 5] = float("nan")
    slot = table[1, 0].long() * 32 + 3
    kdn.kdn_cache_write(x, x, slot.view(1), cache)
    o, _ = kdn.kdn_cache_attention(q, cache, table, n, max_len=40)
    assert torch.isnan(o[1, 2:]).all() and torch.isfinite(o[1, :2]).all() and torch.isfinite(o[0]).all()


def test_out_of_range_lengths_and_pages():
    import torch
    import uncertainty_aware_delta_gb300 as kdn

    q, cache, table, n = _setup([40, 40, 40, 40], 4, 2, 64, 16, "bf16")
    ws = torch.empty(kdn.cache_attention_workspace_size(4, 4, 2, 64, 45, 0), dtype=torch.uint8, device="cuda")
    clean = kdn.kdn_cache_attention(q, cache, table, n, max_len=45, workspace=ws)
    assert kdn.kdn_read_device_status(ws) == 0
    m = n.clone()
    m[0], m[1] = -5, 10 ** 6
    t = table.clone()
    t[2, 1], t[1, 2] = cache.shape[0], -7
    o, lse = kdn.kdn_cache_attention(q, cache, t, m, max_len=45, workspace=ws)
    assert kdn.kdn_read_device_status(ws) == 9
    assert torch.equal(o[3], clean[0][3]) and not o[0].any() and torch.isinf(lse[0]).all()
    assert torch.isfinite(o.float()).all()


def test_strided_queries_and_other_stream():
    import torch
    import uncertainty_aware_delta_gb300 as kdn

    q, cache, table, n = _setup([100, 37], 8, 2, 64, 32, "bf16")
    want = kdn.kdn_cache_attention(q, cache, table, n, max_len=100)
    fused = torch.zeros(2, 12, 64, device="cuda", dtype=torch.bfloat16)
    fused[:, :8] = q
    side = torch.cuda.Stream()
    got = kdn.kdn_cache_attention(fused[:, :8], cache, table, n, max_len=100, stream=side)
    side.synchronize()
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    got = kdn.kdn_cache_attention(q.transpose(0, 1).contiguous().transpose(0, 1), cache, table, n, max_len=100)
    assert torch.equal(got[0], want[0])


def test_graph_capture():
    import torch
    import uncertainty_aware_delta_gb300 as kdn

    q, cache, table, n = _setup([3000, 37], 8, 2, 64, 32, "bf16")
    want = kdn.kdn_cache_attention(q, cache, table, n, max_len=3000)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=side):
        got = kdn.kdn_cache_attention(q, cache, table, n, max_len=3000)
    for _ in range(3):
        got[0].zero_()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


def test_refusals():
    import torch
    import uncertainty_aware_delta_gb300 as kdn

    q, cache, table, n = _setup([20, 30], 4, 2, 64, 32, "bf16")
    for bad in (dict(q=q.half()), dict(q=q.cpu()), dict(block_table=table.long()), dict(seq_len=n[:1]),
                dict(q=q[..., :32]), dict(cache=cache.float()), dict(workspace=torch.empty(8, dtype=torch.uint8, device="cuda"))):
        a = dict(q=q, cache=cache, block_table=table, seq_len=n)
        a.update(bad)
        with pytest.raises((TypeError, ValueError)):
            kdn.kdn_cache_attention(**a)
    for bad, status in ((dict(scale=float("nan")), 2), (dict(scale=-1.0), 2), (dict(window=-1), 2), (dict(max_len=-1), 2)):
        with pytest.raises((kdn.KDNError, ValueError)):
            kdn.kdn_cache_attention(q, cache, table, n, **bad)
    with pytest.raises(kdn.KDNError) as e:
        kdn.kdn_cache_attention(q[:, :3].contiguous(), cache, table, n)
    assert e.value.status == 2
