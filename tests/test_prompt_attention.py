"""Attention over packed prompts, against fp64 row by row."""
import math

import numpy as np
import pytest

import attention_oracle as ref

pytestmark = pytest.mark.gpu


def _inputs(lq, lk, H, hkv, d, io, seed=0, gain=1.0, pad=0):
    import torch

    g = torch.Generator().manual_seed(seed)
    dt = torch.bfloat16 if io == "bf16" else torch.float32
    cu = lambda n: torch.tensor(np.concatenate([[0], np.cumsum(n)]).astype(np.int32)).cuda()
    nq, nk = int(sum(lq)) + pad, int(sum(lk)) + pad
    q = (torch.randn((nq, H, d), generator=g) * gain).to(dt).cuda()
    k = torch.randn((nk, hkv, d), generator=g).to(dt).cuda()
    v = torch.randn((nk, hkv, d), generator=g).to(dt).cuda()
    return q, k, v, cu(lq), cu(lk)


def _np(t):
    return t.double().cpu().numpy()


def _expect(q, k, v, cu_q, cu_k, window, scale=None):
    return ref.prompt(_np(q), _np(k), _np(v), cu_q.tolist(), cu_k.tolist(), window, scale or 1 / math.sqrt(q.shape[2]))


def _run(lq, lk, H, hkv, d, io, window=0, flags=0, scale=None, gain=1.0):
    import torch
    import uncertainty_aware_delta_gb300 as kdn

    q, k, v, cu_q, cu_k = _inputs(lq, lk, H, hkv, d, io, gain=gain)
    ws = torch.empty(kdn.prompt_attention_workspace_size(len(lq), q.shape[0], H, hkv, d, 1 if io == "bf16" else 0, flags),
                     dtype=torch.uint8, device="cuda")
    o, lse = kdn.kdn_prompt_attention(q, k, v, cu_q, cu_k, window=window, flags=flags, scale=scale, workspace=ws)
    assert kdn.kdn_read_device_status(ws) == 0
    ref.check(_np(o), _np(lse), _expect(q, k, v, cu_q, cu_k, window, scale), io)
    again = kdn.kdn_prompt_attention(q, k, v, cu_q, cu_k, window=window, flags=flags, scale=scale)
    assert torch.equal(again[0], o) and torch.equal(again[1], lse)
    return o, lse


SIZES = [([1], 1, 1, 64), ([1, 2, 3, 0, 5], 2, 2, 64), ([127, 128, 129], 2, 1, 128), ([300, 17], 4, 2, 64),
         ([63, 64, 65, 1, 255, 256, 257], 2, 1, 64), ([513], 3, 1, 128), ([200, 40], 6, 2, 128)]


@pytest.mark.parametrize("io", ["bf16", "f32"])
@pytest.mark.parametrize("lens,H,hkv,d", SIZES + [([70, 5], 2, 1, 16), ([70, 5], 2, 2, 32)])
@pytest.mark.parametrize("window", [0, 1, 100])
def test_packed(lens, H, hkv, d, io, window):
    _run(lens, lens, H, hkv, d, io, window)


@pytest.mark.parametrize("lens,H,hkv,d", SIZES[2:4])
def test_portable_path_in_bf16(lens, H, hkv, d):
    import uncertainty_aware_delta_gb300 as kdn

    _run(lens, lens, H, hkv, d, "bf16", 50, kdn.KDN_FLAG_PORTABLE)


@pytest.mark.parametrize("io", ["bf16", "f32"])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("lq,lk,window", [([1, 1, 1], [400, 1, 129], 0), ([50, 130], [450, 131], 0), ([60, 300], [20, 0], 0),
                                          ([50, 130], [450, 300], 65), ([200, 7], [10, 700], 33), ([0, 3], [40, 0], 0)])
def test_prefixes_and_rows_without_keys(lq, lk, window, d, io):
    _run(lq, lk, 4, 2, d, io, window)


@pytest.mark.parametrize("io", ["bf16", "f32"])
def test_scores_far_apart(io):
    _run([260, 70], [260, 70], 2, 1, 64, io, gain=40.0)
    _run([260, 70], [260, 70], 2, 1, 128, io, scale=1e-3)


def test_longer(tmp_path):
    """Rows of a longer prompt, where the running maximum moves over many tiles; a few rows are checked."""
    import uncertainty_aware_delta_gb300 as kdn

    for d, H, hkv in ((128, 4, 2), (64, 3, 3)):
        q, k, v, cu_q, cu_k = _inputs([2500, 901], [2500, 901], H, hkv, d, "bf16", seed=3)
        o, lse = kdn.kdn_prompt_attention(q, k, v, cu_q, cu_k)
        qn, kn, vn = _np(q), _np(k), _np(v)
        for i in (0, 127, 128, 1000, 1407, 2047, 2303, 2499, 2500, 2633, 3400):
            k0, place = (0, i) if i < 2500 else (2500, i - 2500)
            for h in range(H):
                w = ref.attend(qn[i, h], kn[k0:, h * hkv // H], vn[k0:, h * hkv // H], 1 / math.sqrt(d), 0, place + 1)
                w = tuple(np.asarray(x)[None] for x in w)
                ref.check(_np(o[i, h])[None], _np(lse[i, h]).reshape(1), w, "bf16")


@pytest.mark.parametrize("d,H,hkv,lens", [(128, 4, 2, [100] * 700 + [300] * 100), (64, 3, 3, [1, 40, 129, 300] * 120),
                                          (128, 2, 1, [700, 5, 260] * 110), (64, 8, 1, [128, 256, 384] * 60)])
@pytest.mark.parametrize("window", [0, 90])
def test_many_prompts(d, H, hkv, lens, window):
    """Many more row tiles than SMs, of one key tile and of several, against the CUDA-core path."""
    import torch
    import uncertainty_aware_delta_gb300 as kdn

    q, k, v, cu, _ = _inputs(lens, lens, H, hkv, d, "bf16", seed=9)
    ws = torch.empty(kdn.prompt_attention_workspace_size(len(lens), q.shape[0], H, hkv, d), dtype=torch.uint8, device="cuda")
    o, lse = kdn.kdn_prompt_attention(q, k, v, cu, window=window, workspace=ws)
    assert kdn.kdn_read_device_status(ws) == 0
    want, want_lse = kdn.kdn_prompt_attention(q, k, v, cu, window=window, flags=kdn.KDN_FLAG_PORTABLE)
    # the weights' rounding to bf16 (2^-8 of at most max |v|) and both outputs' own
    top = float(v.abs().max())
    assert float((o.float() - want.float()).abs().max()) <= 3 * 2.0 ** -8 * top
    assert float((o.float() - want.float()).norm() / want.float().norm()) <= 2.0 ** -8
    assert float((lse - want_lse).abs().max()) <= 1e-4
    again = kdn.kdn_prompt_attention(q, k, v, cu, window=window)
    assert torch.equal(again[0], o) and torch.equal(again[1], lse)


@pytest.mark.parametrize("io", ["bf16", "f32"])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf")])
def test_special_values_reach_only_rows_that_see_them(bad, d, io):
    import torch
    import uncertainty_aware_delta_gb300 as kdn

    lens = [150, 90, 200]
    for what in ("k", "v"):
        for place in (10, 149, 150, 200, 300, 439):
            q, k, v, cu, _ = _inputs(lens, lens, 2, 1, d, io, seed=5, pad=16)
            clean, clean_lse = kdn.kdn_prompt_attention(q, k, v, cu, window=70)
            x = k if what == "k" else v
            x[place, 0, 3] = bad
            x[440:] = bad                     # rows of no sequence
            o, lse = kdn.kdn_prompt_attention(q, k, v, cu, window=70)
            s = np.searchsorted(np.cumsum(lens), place, side="right")
            rows = torch.zeros(q.shape[0], dtype=torch.bool)
            rows[place:min(place + 70, int(np.sum(lens[:s + 1])))] = True
            live = torch.arange(q.shape[0]) < 440
            same = (live & ~rows).cuda()
            assert torch.equal(o[same], clean[same]) and torch.equal(lse[same], clean_lse[same])
            if what == "v":
                assert not torch.isfinite(o[rows.cuda()][:, :, 3]).any()
                assert torch.equal(lse[rows.cuda()], clean_lse[rows.cuda()])
                others = [c for c in range(d) if c != 3]
                assert torch.equal(o[rows.cuda()][:, :, others], clean[rows.cuda()][:, :, others]) or io == "bf16"
                assert torch.isfinite(o[rows.cuda()][:, :, others]).all()
            elif bad != bad:
                assert torch.isnan(o[rows.cuda()]).all()


def test_strided_operands_and_other_stream():
    import torch
    import uncertainty_aware_delta_gb300 as kdn

    for d, dt in ((64, torch.bfloat16), (128, torch.bfloat16), (64, torch.float32)):
        fused = torch.randn(230, 4 + 2 + 2, d, device="cuda").to(dt)
        q, k, v = fused[:, :4], fused[:, 4:6], fused[:, 6:]
        cu = torch.tensor([0, 100, 230], dtype=torch.int32, device="cuda")
        want = kdn.kdn_prompt_attention(q.contiguous(), k.contiguous(), v.contiguous(), cu)
        side = torch.cuda.Stream()
        got = kdn.kdn_prompt_attention(q, k, v, cu, stream=side)
        side.synchronize()
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
        heads_first = [x.transpose(0, 1).contiguous().transpose(0, 1) for x in (q, k, v)]
        got = kdn.kdn_prompt_attention(*heads_first, cu)
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


def test_rows_of_no_sequence_are_left_alone():
    import torch
    import uncertainty_aware_delta_gb300 as kdn

    for d in (64, 32):
        q, k, v, cu, _ = _inputs([140, 9], [140, 9], 2, 2, d, "bf16", pad=40)
        cu = cu + 11
        o, lse = torch.full_like(q, 7.0), torch.full(q.shape[:2], 7.0, device="cuda")
        kdn.kdn_prompt_attention(q, k, v, cu, out=(o, lse))
        assert (o[:11] == 7).all() and (o[160:] == 7).all() and (lse[160:] == 7).all() and not (o[11:160] == 7).any()


def test_bounds_out_of_range():
    import torch
    import uncertainty_aware_delta_gb300 as kdn

    for d in (64, 32):
        q, k, v, cu, _ = _inputs([100, 50, 60], [100, 50, 60], 2, 2, d, "bf16")
        ws = torch.empty(kdn.prompt_attention_workspace_size(3, 210, 2, 2, d), dtype=torch.uint8, device="cuda")
        clean, _ = kdn.kdn_prompt_attention(q, k, v, cu)
        for bad in ([0, 100, 90, 210], [-1, 100, 150, 210], [0, 100, 150, 211], [0, 100, 150, 2 ** 31 - 1]):
            o = torch.zeros_like(q)
            lse = torch.zeros(q.shape[:2], device="cuda")
            kdn.kdn_prompt_attention(q, k, v, torch.tensor(bad, dtype=torch.int32, device="cuda"), out=(o, lse), workspace=ws)
            assert kdn.kdn_read_device_status(ws) == 9
            if bad[:3] == [0, 100, 150]:
                assert torch.equal(o[:150], clean[:150])


def test_empty_batches():
    import torch
    import uncertainty_aware_delta_gb300 as kdn

    for dt in (torch.bfloat16, torch.float32):
        e = torch.empty(0, 2, 64, dtype=dt, device="cuda")
        cu = torch.zeros(3, dtype=torch.int32, device="cuda")
        o, lse = kdn.kdn_prompt_attention(e, e, e, cu)
        assert o.shape == (0, 2, 64) and lse.shape == (0, 2)
        q = torch.randn(5, 2, 64, device="cuda").to(dt)
        o, lse = kdn.kdn_prompt_attention(q, e, e, torch.tensor([0, 3, 5], dtype=torch.int32, device="cuda"), cu)
        assert not o.any() and (lse == -math.inf).all()


def test_refusals():
    import torch
    import uncertainty_aware_delta_gb300 as kdn

    q, k, v, cu, _ = _inputs([20], [20], 4, 2, 64, "bf16")
    for bad in (dict(q=q.half()), dict(k=k.float()), dict(v=v[:10]), dict(cu_q=cu.long()), dict(k=k.cpu()),
                dict(cu_k=cu[:1])):
        a = dict(q=q, k=k, v=v, cu_q=cu)
        a.update(bad)
        with pytest.raises((TypeError, ValueError)):
            kdn.kdn_prompt_attention(**a)
    for a, status in (((q[:, :3].contiguous(), k, v, cu), 2), ((q, k[:10].contiguous(), v[:10].contiguous(), cu), 2)):
        with pytest.raises(kdn.KDNError) as e:
            kdn.kdn_prompt_attention(*a)
        assert e.value.status == status
    for kw, status in ((dict(window=-1), 2), (dict(scale=math.inf), 2), (dict(flags=kdn.KDN_FLAG_NO_SPLIT), 6)):
        with pytest.raises(kdn.KDNError) as e:
            kdn.kdn_prompt_attention(q, k, v, cu, **kw)
        assert e.value.status == status


@pytest.mark.parametrize("d,io", [(64, "bf16"), (128, "bf16"), (64, "f32")])
def test_outputs_aligned_to_16_bytes(d, io):
    import torch
    import uncertainty_aware_delta_gb300 as kdn

    q, k, v, cu_q, cu_k = _inputs([130, 3], [130, 3], 2, 1, d, io)
    want = kdn.kdn_prompt_attention(q, k, v, cu_q, cu_k)
    spare, off = torch.zeros(q.numel() + 64, dtype=q.dtype, device="cuda"), 16 // q.element_size()
    o, lse = spare[off:off + q.numel()].view(q.shape), torch.empty_like(want[1])
    assert o.data_ptr() % 32 == 16
    kdn.kdn_prompt_attention(q, k, v, cu_q, cu_k, out=(o, lse))
    assert torch.equal(o, want[0]) and torch.equal(lse, want[1])
    assert not bool(spare[:off].any()) and not bool(spare[off + q.numel():].any())
