"""Tokens quantised into the 4-bit cache and read back: codes, scales and places, exactly."""
import numpy as np
import pytest

import attention_oracle as ref

pytestmark = pytest.mark.gpu


def _inputs(n, hkv, d, io, seed):
    import torch

    g = torch.Generator().manual_seed(seed)
    x = torch.randn((2, n, hkv, d), generator=g) * torch.exp(2 * torch.randn((2, n, hkv, 1), generator=g))
    return x.to(torch.bfloat16 if io == "bf16" else torch.float32).cuda()


def _numpy(t):
    return t.double().cpu().numpy()


def _expect(x):
    """The format's arithmetic as the library states it: fp32 division and rounding."""
    g = x.astype(np.float32).reshape(*x.shape[:-1], -1, 32)
    s = np.minimum(np.abs(g).max(-1) / np.float32(7), np.float32(ref.F16_MAX)).astype(np.float16).astype(np.float32)
    f = s[..., None]
    code = np.where(f > 0, np.clip(np.rint(g / np.where(f > 0, f, np.float32(1))), -7, 7), 0).astype(np.int64) + 8
    return code.reshape(x.shape), s.astype(np.float64)


@pytest.mark.parametrize("d", [32, 64, 128])
@pytest.mark.parametrize("io", ["bf16", "f32"])
@pytest.mark.parametrize("n,hkv,page,order", [(1, 1, 16, "scattered"), (50, 3, 48, "scattered"), (4100, 5, 64, "pages"),
                                              (4099, 5, 64, "scattered"), (9000, 3, 128, "shifted")])
def test_write_and_read(n, hkv, page, order, io, d):
    import torch
    import uncertainty_aware_delta_gb300 as kdn

    k, v = _inputs(n, hkv, d, io, n + d)
    pages = n // page + 3
    rng = np.random.default_rng(n)
    if order == "scattered":
        slots = rng.permutation(pages * page)[:n]
    else:
        ids = rng.permutation(pages - 1)
        at = np.arange(n) + (5 if order == "shifted" else 0)
        slots = np.append(ids, pages - 1)[at // page] * page + at % page
    skip = rng.random(n) < 0.02
    slots[skip] = rng.choice([-1, -page, pages * page, 2 ** 40], skip.sum())
    cache = kdn.cache_alloc(pages, page, hkv, d)
    cache.fill_(0x5a)
    st = torch.from_numpy(slots).cuda()
    kdn.kdn_cache_write(k, v, st, cache)
    got = ref.unpack(cache.cpu().numpy(), d)
    untouched = ref.unpack(np.full(cache.shape, 0x5a, np.uint8), d)
    keep = ~skip
    at = slots[keep]
    for x, (code, scale), (code0, scale0) in ((k, got[:2], untouched[:2]), (v, got[2:], untouched[2:])):
        wc, ws = _expect(_numpy(x))
        if io == "bf16":   # for 8-bit significands the quotients never come near a tie without being one
            wc64, ws64 = ref.quantise(_numpy(x))
            assert np.array_equal(wc, wc64) and np.array_equal(ws, ws64)
        code0, scale0 = code0.copy(), scale0.copy()
        code0[at // page, :, at % page] = wc[keep]
        scale0[at // page, :, at % page] = ws[keep]
        assert np.array_equal(code, code0) and np.array_equal(scale, scale0)
    for dtype in (torch.float32, torch.bfloat16):
        for x, y in zip((k, v), kdn.kdn_cache_read(cache, st, dtype=dtype)):
            want = ref.values(*_expect(_numpy(x)))
            want[skip] = 0
            assert np.array_equal(_numpy(y), _numpy(torch.from_numpy(want).float().to(dtype)))


def test_special_values():
    import torch
    import uncertainty_aware_delta_gb300 as kdn

    x = torch.randn(12, 1, 64)
    x[0] = 0
    x[1, 0, 3] = float("nan")
    x[2, 0, 40] = float("inf")
    x[3, 0, 63] = -float("inf")
    x[4] *= 1e30
    x[5] *= 1e-30
    x[6] *= 1e-6
    x[7, 0, :32] = torch.arange(32).float() * 0.5 - 7.5     # ties: 7 is the largest code
    x[7, 0, 0] = -7.0
    x[8] = 3.4e38
    x[9, 0, 1:] = 0
    for dtype in (torch.float32, torch.bfloat16):
        k = x.to(dtype).cuda()
        cache = kdn.cache_alloc(1, 16, 1, 64)
        slots = torch.arange(12, device="cuda")
        kdn.kdn_cache_write(k, k, slots, cache)
        code, s = ref.quantise(_numpy(k))
        want = ref.values(code, s)
        for y in kdn.kdn_cache_read(cache, slots, dtype=torch.float32):
            assert np.array_equal(_numpy(y), want, equal_nan=True)


def test_strided_operands():
    import torch
    import uncertainty_aware_delta_gb300 as kdn

    qkv = torch.randn(40, 4 + 2 + 2, 64, device="cuda").to(torch.bfloat16)   # a fused projection's rows
    k, v = qkv[:, 4:6], qkv[:, 6:]
    by_head = torch.randn(2, 40, 64, device="cuda").to(torch.bfloat16).transpose(0, 1)
    slots = torch.randperm(48, device="cuda")[:40]
    for a, b in ((k, v), (by_head, v), (k, by_head)):
        one, two = kdn.cache_alloc(3, 16, 2, 64), kdn.cache_alloc(3, 16, 2, 64)
        kdn.kdn_cache_write(a, b, slots, one)
        kdn.kdn_cache_write(a.contiguous(), b.contiguous(), slots, two)
        assert torch.equal(one, two) and one.any()


def test_refusals():
    import torch
    import uncertainty_aware_delta_gb300 as kdn

    cache = kdn.cache_alloc(3, 16, 2, 64)
    k = torch.zeros(4, 2, 64, device="cuda", dtype=torch.bfloat16)
    s = torch.arange(4, device="cuda")
    for bad in (dict(k=k.half()), dict(v=k.float()), dict(k=k.cpu()), dict(slot_map=s.int()), dict(k=k[:, :1]),
                dict(cache=cache[:, :, :, :100]), dict(cache=cache.view(3, 2, -1)), dict(k=k[..., :32]),
                dict(k=torch.zeros(4, 2, 128, device="cuda", dtype=torch.bfloat16)[..., ::2])):
        a = dict(k=k, v=k, slot_map=s, cache=cache)
        a.update(bad)
        with pytest.raises((TypeError, ValueError)):
            kdn.kdn_cache_write(**a)
    with pytest.raises(kdn.KDNError) as e:
        kdn.kdn_cache_write(torch.zeros(4, 2 * 64 + 4, device="cuda", dtype=torch.bfloat16)[:, :128].unflatten(1, (2, 64)), k, s, cache)
    assert e.value.status == 4
    with pytest.raises(kdn.KDNError) as e:
        kdn.kdn_cache_write(torch.zeros(1, 1, 64, device="cuda", dtype=torch.bfloat16).expand(4, 2, 64), k, s, cache)
    assert e.value.status == 2
    with pytest.raises(kdn.KDNError):
        kdn.cache_alloc(3, 17, 2, 64)
    with pytest.raises(kdn.KDNError):
        kdn.cache_alloc(3, 16, 2, 96)


@pytest.mark.parametrize("io", ["bf16", "f32"])
@pytest.mark.parametrize("n,hkv,d,page,order", [(70001, 1, 128, 64, "pages"), (70000, 1, 128, 32, "shifted"),
                                                (46000, 3, 64, 128, "pages"), (131077, 2, 32, 16, "scattered")])
def test_large_write_and_read(n, hkv, d, page, order, io):
    test_write_and_read(n, hkv, page, order, io, d)
