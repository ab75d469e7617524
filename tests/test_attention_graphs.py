"""The attention calls captured in a CUDA graph and replayed on new inputs, and prompts over prefixes in batches of more than
32 sequences."""
import pytest
import torch

import attention_oracle as ref
from test_prompt_attention import _expect, _inputs, _np, _run

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("n", [33, 40])
@pytest.mark.parametrize("d,H,hkv", [(64, 2, 1), (128, 3, 1)])
@pytest.mark.parametrize("window", [0, 300])
def test_many_sequences_over_prefixes(n, d, H, hkv, window):
    """One with a long prefix among short ones."""
    lq = [1 + 7 * (i % 5) for i in range(n)]
    lk = [x + 13 * (i % 3) for i, x in enumerate(lq)]
    lk[3] += 5000
    lk[n - 1] = 0
    _run(lq, lk, H, hkv, d, "bf16", window)


@pytest.mark.parametrize("io,lq,lk", [("bf16", [70, 5], [70, 5]), ("f32", [70, 5], [170, 5]), ("bf16", [3, 1], [9000, 20])])
def test_prompts_in_a_graph(io, lq, lk):
    import uncertainty_aware_delta_gb300 as kdn

    q, k, v, cu_q, cu_k = _inputs(lq, lk, 4, 2, 64, io)
    fresh = _inputs(lq, lk, 4, 2, 64, io, seed=1)
    out = torch.empty_like(q), torch.empty(q.shape[:2], device="cuda")
    ws = torch.empty(kdn.prompt_attention_workspace_size(2, q.shape[0], 4, 2, 64, 1 if io == "bf16" else 0), dtype=torch.uint8,
                     device="cuda")
    side, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    with torch.cuda.stream(side):
        kdn.kdn_prompt_attention(q, k, v, cu_q, cu_k, out=out, workspace=ws)
    torch.cuda.synchronize()
    with torch.cuda.graph(graph, stream=side):
        kdn.kdn_prompt_attention(q, k, v, cu_q, cu_k, out=out, workspace=ws)
    for a, b in zip((q, k, v), fresh):
        a.copy_(b)
    for _ in range(2):
        out[0].fill_(7)
        graph.replay()
        torch.cuda.synchronize()
        assert kdn.kdn_read_device_status(ws) == 0
        ref.check(_np(out[0]), _np(out[1]), _expect(q, k, v, cu_q, cu_k, 0), io)


def test_plan_write_and_read_in_a_graph():
    import uncertainty_aware_delta_gb300 as kdn

    i32 = dict(dtype=torch.int32, device="cuda")
    ctx, new, table = torch.tensor([0, 20], **i32), torch.tensor([18, 3], **i32), torch.tensor([[-1, -1], [4, 5]], **i32)
    free, count = torch.tensor([7, 2, 3], **i32), torch.tensor([3], **i32)
    k, v = (torch.randn(21, 2, 64, device="cuda") for _ in range(2))
    cache, ws = kdn.cache_alloc(8, 16, 2, 64), torch.empty(256, dtype=torch.uint8, device="cuda")
    plan = kdn.kdn_cache_plan(ctx, new, table, free, count, page=16, capacity=21, workspace=ws)
    out = torch.empty_like(k), torch.empty_like(v)

    def step():
        kdn.kdn_cache_plan(ctx, new, table, free, count, page=16, capacity=21, out=plan, workspace=ws)
        kdn.kdn_cache_write(k, v, plan.slot_map, cache)
        kdn.kdn_cache_read(cache, plan.slot_map, out=out)

    side, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    with torch.cuda.stream(side):
        step()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph, stream=side):
        step()
    for _ in range(2):
        k.normal_()
        v.normal_()
        graph.replay()
        torch.cuda.synchronize()
        assert kdn.kdn_read_device_status(ws) == 0 and table.tolist() == [[3, 2], [4, 5]]
        assert plan.slot_map.tolist() == [48 + i for i in range(16)] + [32, 33] + [84, 85, 86]
        for got, x in zip(out, (k, v)):
            want = ref.values(*ref.quantise(x.cpu().numpy()))
            assert torch.equal(got.double().cpu(), torch.from_numpy(want))
