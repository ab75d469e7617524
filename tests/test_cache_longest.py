"""Attention over a cache of as many tokens as an int counts: a table that names one page again and again."""
import math

import numpy as np
import pytest
import torch

import attention_oracle as ref

pytestmark = pytest.mark.gpu
PAGE, MOST = 1024, 2 ** 31 - 1024


@pytest.mark.parametrize("io", ["bf16", "f32"])
@pytest.mark.parametrize("n,max_len,window", [(2 ** 31 - 1, 2 ** 31 - 1, 0), (MOST, 2 ** 31 - 1, 0), (2 ** 31 - 1, 2 ** 31 - 1, 1024),
                                              (MOST, MOST, 3000), (5000, 2 ** 31 - 1, 0)])
def test_longest(n, max_len, window, io):
    import uncertainty_aware_delta_gb300 as kdn

    dt, d = torch.bfloat16 if io == "bf16" else torch.float32, 32
    gen = torch.Generator(device="cuda").manual_seed(9)
    k, v = (torch.randn(PAGE, 1, d, generator=gen, device="cuda").to(dt) for _ in range(2))
    q = torch.randn(1, 2, d, generator=gen, device="cuda").to(dt)
    cache = kdn.kdn_cache_write(k, v, torch.arange(PAGE, device="cuda"), kdn.cache_alloc(1, PAGE, 1, d))
    table = torch.zeros(1, 2 ** 31 // PAGE, dtype=torch.int32, device="cuda")
    ws = torch.empty(kdn.cache_attention_workspace_size(1, 2, 1, d, max_len, window), dtype=torch.uint8, device="cuda")
    out = torch.full_like(q, 7.0), torch.full((1, 2), 7.0, device="cuda")
    kdn.kdn_cache_attention(q, cache, table, torch.tensor([n], dtype=torch.int32, device="cuda"), max_len=max_len, window=window,
                            out=out, workspace=ws)
    assert kdn.kdn_read_device_status(ws) == (9 if n > MOST else 0)
    kk, vv = (t.double().cpu().numpy()[:, 0] for t in kdn.kdn_cache_read(cache, torch.arange(PAGE, device="cuda"), dtype=torch.float32))
    n = min(n, MOST)
    lo = max(n - window, 0) if window else 0
    # how often each place of the page is seen, as whole turns and a rest from `lo` on
    turns = np.full(PAGE, (n - lo) // PAGE)
    turns[(lo + np.arange((n - lo) % PAGE)) % PAGE] += 1
    # a row has at most 127 whole parts, of four warps that add 16 tokens a step; a step is off by 2^-23 of the sum
    # (rounded) or 2^-22 (cut off by the MMAs), all of one sign at worst
    steps = max(turns.sum() / 127 / 4 / 16, 48)
    for h in range(2):
        x = kk @ q[0, h].double().cpu().numpy() / math.sqrt(d)
        w = turns * np.exp(x - x.max())
        p, lse = w / w.sum(), x.max() + math.log(w.sum())
        o, A = p @ vv, p @ np.abs(vv)
        E = (np.abs(kk) @ np.abs(q[0, h].double().cpu().numpy())).max() / math.sqrt(d)
        bound, lb = ref.bounds(o, A, np.array(E), io, True)
        assert np.all(np.abs(out[0][0, h].double().cpu().numpy() - o) <= bound + A * steps * 2.0 ** -21)
        assert abs(float(out[1][0, h]) - lse) <= lb + steps * 2.0 ** -22 + 2.0 ** -22 * abs(lse)
