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
