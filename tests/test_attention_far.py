"""Attention operators on offsets past 32 bits: a cache of more than 2^32 bytes, rows more than 2^32 elements apart."""
import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("io", ["bf16", "f32"])
def test_far_pages(io):
    import uncertainty_aware_delta_gb300 as kdn

    dt = torch.bfloat16 if io == "bf16" else torch.float32
    page, hkv, d, H, lens = 1024, 8, 128, 16, [2500, 1, 1024]
    per_page = kdn.cache_alloc(1, page, hkv, d).numel()
    pages = 2 ** 32 // per_page + 8
    gen = torch.Generator(device="cuda").manual_seed(5)
    k, v = (torch.randn(sum(lens), hkv, d, generator=gen, device="cuda").to(dt) for _ in range(2))
    q = torch.randn(3, H, d, generator=gen, device="cuda").to(dt)
    ids = [pages - 1, 2 ** 31 // per_page, pages - 3, 1, 2 ** 32 // per_page]     # 3 pages, 1 and 1
    near = {p: i for i, p in enumerate(ids)}
    n = torch.tensor(lens, dtype=torch.int32, device="cuda")
    results = []
    for size, name in ((pages, lambda p: p), (len(ids), near.get)):
        cache = kdn.cache_alloc(size, page, hkv, d)
        own = [[name(p) for p in ids[:3]], [name(ids[3])], [name(ids[4])]]
        table = torch.tensor([(o + [-1, -1])[:3] for o in own], dtype=torch.int32, device="cuda")
        slots = torch.cat([table[r, torch.arange(m, device="cuda") // page].long() * page + torch.arange(m, device="cuda") % page
                           for r, m in enumerate(lens)])
        kdn.kdn_cache_write(k, v, slots, cache)
        used = torch.tensor([name(p) for p in ids], device="cuda")
        results.append([cache[used], *kdn.kdn_cache_read(cache, slots, dtype=dt),
                        *kdn.kdn_cache_attention(q, cache, table, n)])
        if size == pages:     # nothing else was written
            cache[used] = 0
            assert not bool(cache.view(torch.int64).any())
        del cache
    assert bool(results[0][0].any())
    for far, close in zip(*results):
        assert torch.equal(far, close)


@pytest.mark.parametrize("d,io", [(128, "bf16"), (64, "bf16"), (32, "f32")])
def test_far_rows(d, io):
    import uncertainty_aware_delta_gb300 as kdn

    dt = torch.bfloat16 if io == "bf16" else torch.float32
    rows, H, hkv = 600, 4, 2
    base = torch.zeros(rows, 2 ** 23, dtype=dt, device="cuda")
    gen = torch.Generator(device="cuda").manual_seed(6)
    base[:, :(H + 2 * hkv) * d] = torch.randn(rows, (H + 2 * hkv) * d, generator=gen, device="cuda").to(dt)
    q, k, v = base[:, :(H + 2 * hkv) * d].unflatten(1, (H + 2 * hkv, d)).split([H, hkv, hkv], 1)
    assert q.stride(0) == 2 ** 23
    cu = torch.tensor([0, 250, 600], dtype=torch.int32, device="cuda")
    far = kdn.kdn_prompt_attention(q, k, v, cu)
    near = kdn.kdn_prompt_attention(q.contiguous(), k.contiguous(), v.contiguous(), cu)
    slots = torch.arange(rows, device="cuda")
    caches = [kdn.kdn_cache_write(a, b, slots, kdn.cache_alloc(10, 64, hkv, d))
              for a, b in ((k, v), (k.contiguous(), v.contiguous()))]
    assert torch.equal(far[0], near[0]) and torch.equal(far[1], near[1]) and torch.equal(*caches)
    assert bool(far[0].any())
