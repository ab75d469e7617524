"""The serving example where pages run out."""
import os
import sys

import pytest
import torch

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))
pytestmark = pytest.mark.gpu


def test_decode_refused_and_repeated():
    from hybrid_serve import Server

    new, outs = [15, 16, 20], []
    for pages in (5, 20):
        s = Server(3, pages, layers=2, heads=4, kv_heads=2, d=32, page=16, table_width=4)
        gen = torch.Generator(device="cuda").manual_seed(4)
        x = [torch.randn(n, s.dim, generator=gen, device="cuda").bfloat16() for n in (sum(new), 3, 3, 3)]
        _, granted = s.prefill(x[0], new)
        assert granted == [1, 1, 1]
        s.decode(x[1])
        if pages == 5:      # the first request needs a page, the others do not
            for _ in range(2):
                with pytest.raises(RuntimeError):
                    s.decode(x[2])
                assert s.context.tolist() == [16, 17, 21] and int(s.n_free) == 0
        s.release(2)
        outs.append([s.decode(x[2]), s.decode(x[3]), s.context])
    for a, b in zip(*outs):
        assert torch.equal(a, b)


def test_status_of_the_plan_is_read():
    """What the plan's status word tells of is an error, whatever was granted, and nothing changes."""
    from hybrid_serve import Server

    s = Server(2, 8, layers=1, heads=2, kv_heads=1, d=32, page=16, table_width=4)
    x = torch.zeros(20, s.dim, device="cuda").bfloat16()
    s.prefill(x, [20, 0])
    for broken in (9, -1):     # a free count outside the list of 8 pages
        good, s.n_free = s.n_free, torch.full_like(s.n_free, broken)
        with pytest.raises(RuntimeError, match="range"):
            s.decode(x[:2])
        with pytest.raises(RuntimeError, match="range"):
            s.prefill(x[:2], [0, 2])
        assert int(s.n_free) == broken and s.context.tolist() == [20, 0]
        s.n_free = good
    s.decode(x[:2])
    s.context = torch.tensor([64, 1], dtype=torch.int32, device="cuda")     # a full row of the table
    with pytest.raises(RuntimeError):
        s.decode(x[:2])
    assert s.context.tolist() == [64, 1]
