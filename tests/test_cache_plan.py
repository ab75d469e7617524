"""Block tables and slot maps built on the GPU, against a request-by-request walk."""
import numpy as np
import pytest

import attention_oracle as ref

pytestmark = pytest.mark.gpu


def _run(ctx, new, page, free_share=1.0, capacity=None, width=None, count=None, seed=0):
    import torch
    import uncertainty_aware_delta_gb300 as kdn

    rng = np.random.default_rng(seed)
    ctx, new = np.asarray(ctx, np.int64), np.asarray(new, np.int64)
    held = -(-np.maximum(ctx, 0) // page)
    need = np.maximum(-(-np.maximum(ctx + new, 0) // page) - held, 0)
    width = int((held + need).max(initial=0)) + 1 if width is None else width
    ids = rng.permutation(int(held.sum() + need.sum()) + 5)
    table = np.full((len(ctx), width), -1, np.int64)
    for r in range(len(ctx)):
        n = min(int(held[r]), width)
        table[r, :n], ids = ids[:n], ids[n:]
    free = ids
    count = int(free_share * need.sum()) if count is None else count
    capacity = int(np.maximum(new, 0).sum()) + 3 if capacity is None else capacity
    want = ref.plan(ctx, new, table, free, count, page, capacity)
    i32 = lambda x: torch.from_numpy(np.asarray(x).astype(np.int32)).cuda()
    t = i32(table).reshape(len(ctx), width)
    ws = torch.empty(256, dtype=torch.uint8, device="cuda")
    for _ in range(2):   # a repeated call gives the same
        got = kdn.kdn_cache_plan(i32(ctx), i32(new), t, i32(free), i32([count]), page=page, capacity=capacity, workspace=ws)
        assert np.array_equal(t.cpu().numpy(), want["table"])
        for name in got._fields:
            assert np.array_equal(getattr(got, name).cpu().numpy(), want[name]), name
        assert kdn.kdn_read_device_status(ws) == (9 if want["bad"] else 0)
    return want


@pytest.mark.parametrize("n,hi_ctx,hi_new,page", [(1, 0, 1, 16), (7, 100, 1, 16), (300, 500, 40, 32), (1500, 20, 9, 1024),
                                                  (33, 4000, 700, 48), (513, 64, 64, 64), (16384, 40, 3, 16)])
@pytest.mark.parametrize("share", [0.0, 0.6, 1.0])
def test_plan(n, hi_ctx, hi_new, page, share):
    rng = np.random.default_rng(n)
    w = _run(rng.integers(0, hi_ctx + 1, n), rng.integers(0, hi_new + 1, n), page, share)
    if share == 1.0:
        assert w["granted"].all() and w["free_left"] == 0


def test_plan_edges():
    _run([], [], 16, capacity=5, width=0)
    _run([0, 16, 15, 17], [0, 0, 1, 0], 16)                       # nothing needs a page
    _run([0, 0], [0, 0], 16, capacity=0)
    _run([16, 16], [1, 16], 16, capacity=2)                       # more tokens than the map holds
    _run([5, -3, 7, 100], [3, 4, -2, 9], 16, width=3)             # lengths out of range are refused alone
    _run([0, 0, 40, 0], [40, 1, 1, 500], 16, count=1)             # the first wants too much: those after it wait,
    _run([0] * 9, [16] * 9, 16, count=10 ** 6)                    # a count past the list
    _run([0] * 9, [16] * 9, 16, count=-4)


def test_refused_request_leaves_its_row_alone():
    w = _run([10, 0], [100, 1], 16, count=1)
    assert list(w["granted"]) == [0, 0] and (w["table"][0, 1:] == -1).all() and w["free_left"] == 1
