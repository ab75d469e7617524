"""Plans of contexts whose place is near the largest int, with a page that is no power of two."""
import pytest

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("page", [48, 1008, 1024])
def test_long_context(page):
    import torch
    import uncertainty_aware_delta_gb300 as kdn

    i32 = dict(dtype=torch.int32, device="cuda")
    width = (2 ** 31 - 1) // page
    most = width * page
    table = torch.arange(width, **i32)[None]
    free, ws = torch.tensor([5, 7], **i32), torch.empty(256, dtype=torch.uint8, device="cuda")
    for ctx, new, pages in ((most, 0, 0), (most - 1, 1, 0), (most - page, 3, 1), (most - page - 1, page, 1)):
        t = table.clone()
        p = kdn.kdn_cache_plan(torch.tensor([ctx], **i32), torch.tensor([new], **i32), t, free, torch.tensor([2], **i32),
                               page=page, capacity=page, workspace=ws)
        assert kdn.kdn_read_device_status(ws) == 0
        assert p.granted.tolist() == [1] and p.seq_len.tolist() == [ctx + new] and p.free_left.tolist() == [2 - pages]
        if pages:
            table[0, -1] = 7
        assert torch.equal(t, table)
        place = torch.arange(ctx, ctx + new, device="cuda")
        assert torch.equal(p.position[:new].long(), place)
        assert torch.equal(p.slot_map[:new], table[0, place // page].long() * page + place % page) and bool((p.slot_map[new:] == -1).all())
        table[0, -1] = width - 1
