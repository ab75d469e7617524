"""Workloads of a retention layer's operators: linear attention with a decay for each head (whole sequences, one token
a sequence, gradients), and the group norm with activation that follows it (with its gradients).  Each case runs either in a
plain form (elementary torch operations in fp32) or through the library (``own``)."""
import math

import numpy as np
import torch

own = False

DEV = "cuda"
TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
BLOCK = 128   # tokens a block of the plain form
DECAYS = {"short": (1e-3, 0.1), "long": (1e-4, 1e-2), "wide": (1e-5, 2.0)}   # -log of the heads' decays


def listed():
    return [
        # the framework's small shape: latency
        dict(name="forward-1x64-f32", op="forward", n=1, T=64, ragged=False, H=2, dk=16, dv=16, io="f32", decay="short"),
        # the framework's training shape (8 sequences of 4096 tokens, 16 heads of 128)
        dict(name="forward-8x4096", op="forward", n=8, T=4096, ragged=False, H=16, dk=128, dv=128, io="bf16",
             decay="short"),
        # the framework's long context, one sequence
        dict(name="forward-1x65536", op="forward", n=1, T=65536, ragged=False, H=16, dk=128, dv=128, io="bf16",
             decay="long"),
        # prompts of all lengths packed together, continuing from states, heads of 64
        dict(name="forward-24-ragged", op="forward", n=24, T=4095, ragged=True, H=16, dk=64, dv=64, io="bf16",
             decay="wide"),
        # one request decoded alone: latency
        dict(name="step-1", op="step", n=1, H=16, dk=128, dv=128, io="bf16", decay="long"),
        # the framework's decode batch, fp32 as there
        dict(name="step-256-f32", op="step", n=256, H=16, dk=128, dv=128, io="f32", decay="short"),
        # gradients of a small odd batch in full precision
        dict(name="backward-3x777-f32", op="backward", n=3, T=777, ragged=False, H=4, dk=64, dv=128, io="f32",
             decay="wide"),
        # gradients at the training shape
        dict(name="backward-8x4096", op="backward", n=8, T=4096, ragged=False, H=16, dk=128, dv=128, io="bf16",
             decay="short"),
        # one decode step of 256 sequences: norm, then the gate
        dict(name="norm-256-gate", op="norm", rows=256, G=16, d=128, act="silu", gate=True, affine=True, io="bf16"),
        # the training shape's outputs
        dict(name="norm-32768-gate", op="norm", rows=32768, G=16, d=128, act="silu", gate=True, affine=True, io="bf16"),
        # gradients of an odd batch in full precision, groups that are no power of two, the activation on the norm itself
        dict(name="norm-backward-1001-f32", op="norm_backward", rows=1001, G=8, d=72, act="silu", gate=False, affine=True,
             io="f32"),
        # gradients at the training shape
        dict(name="norm-backward-32768", op="norm_backward", rows=32768, G=16, d=128, act="silu", gate=True, affine=True,
             io="bf16"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["forward", "forward", "forward", "step", "backward", "backward", "norm", "norm_backward"])
    io = rng.choice(["bf16", "bf16", "bf16", "f32"])
    if op in ("norm", "norm_backward"):
        G, d = _log(rng, 1, 32), 8 * _log(rng, 1, 32)
        most = 32768 * 16 * 128 // (G * d) // (1 if io == "bf16" else 2)
        return dict(op=op, rows=min(_log(rng, 1, 65536), most), G=G, d=d, act=rng.choice(["none", "silu", "sigmoid"]),
                    gate=rng.choice([True, False]), affine=rng.choice([True, True, False]), io=io)
    H = _log(rng, 1, 32)
    dk, dv = rng.choice([(128, 128), (128, 128), (64, 64), (64, 128), (128, 64), (32, 32), (16, 64)])
    decay = rng.choice(list(DECAYS))
    most = 8 * 16 * 4096 * 128 // (H * max(dk, dv)) // (1 if io == "bf16" else 4)
    if op == "step":
        return dict(op=op, n=max(1, min(_log(rng, 1, 512), 256 * 16 * 128 * 128 // (H * dk * dv))), H=H, dk=dk, dv=dv,
                    io=io, decay=decay)
    T = min(_log(rng, 1, 65536), most)
    return dict(op=op, n=max(1, min(_log(rng, 1, 64), most // T)), T=T, ragged=rng.choice([True, False]), H=H, dk=dk, dv=dv,
                io=io, decay=decay)


# ------------------------------------------------------------------ sizes that follow from the case alone

def _lengths(c):
    """Tokens of the sequences: all T, or spread over the logarithm of 1 .. T with T among them."""
    if not c["ragged"]:
        return np.full(c["n"], c["T"], np.int64)
    u = np.modf((np.arange(c["n"]) + 1) * 0.6180339887498949)[0]
    x = np.rint(np.exp(u * math.log(c["T"]))).astype(np.int64).clip(1, c["T"])
    x[c["n"] // 2] = c["T"]
    return x


def work(c):
    e = 2 if c["io"] == "bf16" else 4
    if c["op"] in ("norm", "norm_backward"):
        values = float(c["rows"]) * c["G"] * c["d"]
        params = (8.0 if c["affine"] else 0.0) * c["G"] * c["d"]
        if c["op"] == "norm":
            return {"bytes": e * values * (3 if c["gate"] else 2) + params, "flops": 10 * values}
        return {"bytes": e * values * (5 if c["gate"] else 3) + 2 * params, "flops": 25 * values}
    H, dk, dv = c["H"], c["dk"], c["dv"]
    state = 4.0 * c["n"] * H * dk * dv
    if c["op"] == "step":
        return {"bytes": 2 * state + e * c["n"] * H * (2.0 * dk + 2 * dv) + 4 * H, "flops": 5.0 * c["n"] * H * dk * dv}
    tok = float(_lengths(c).sum()) * H
    if c["op"] == "forward":
        return {"bytes": e * tok * (2 * dk + 2 * dv) + 2 * state, "flops": 4.0 * tok * dk * dv}
    return {"bytes": e * tok * (4 * dk + 3 * dv) + 3 * state, "flops": 10.0 * tok * dk * dv}


# ------------------------------------------------------------------ inputs

def _int(x):
    return torch.from_numpy(np.ascontiguousarray(x)).to(device=DEV, dtype=torch.int32)


def _cu(n):
    return np.concatenate([[0], np.cumsum(n)])


def prepare(case, seed):
    c, g, io = case, torch.Generator(device=DEV).manual_seed(seed), TYPES[case["io"]]
    normal = lambda *shape: torch.randn(shape, generator=g, device=DEV)   # noqa: E731
    s = {"case": c}
    if c["op"] in ("norm", "norm_backward"):
        shape = (c["rows"], c["G"], c["d"])
        # a memory's outputs: tokens and heads of different size, and means away from zero
        s["x"] = ((normal(*shape) + 0.3 * normal(1, c["G"], c["d"])) * torch.exp(normal(c["rows"], c["G"], 1))).to(io)
        s["gate"] = normal(*shape).to(io) if c["gate"] else None
        s["w"] = 1 + 0.2 * normal(c["G"], c["d"]) if c["affine"] else None
        s["b"] = 0.2 * normal(c["G"], c["d"]) if c["affine"] else None
        if c["op"] == "norm_backward":
            s["dy"] = normal(*shape).to(io)
        return s
    H, dk, dv = c["H"], c["dk"], c["dv"]
    lo, hi = (math.log(x) for x in DECAYS[c["decay"]])
    s["log_decay"] = -torch.exp(lo + (hi - lo) * torch.rand(H, generator=g, device=DEV))
    unit = lambda x: torch.nn.functional.normalize(x, dim=-1)   # noqa: E731
    if c["op"] == "step":
        s.update(q=unit(normal(c["n"], H, dk)).to(io), k=unit(normal(c["n"], H, dk)).to(io), v=normal(c["n"], H, dv).to(io),
                 S=normal(c["n"], H, dk, dv))
        return s
    n = _lengths(c)
    lead = (int(n.sum()),) if c["ragged"] else (c["n"], c["T"])
    s.update(q=unit(normal(*lead, H, dk)).to(io), k=unit(normal(*lead, H, dk)).to(io), v=normal(*lead, H, dv).to(io),
             S0=normal(c["n"], H, dk, dv), cu=_int(_cu(n)) if c["ragged"] else None, longest=int(n.max()))
    if c["op"] == "backward":
        s.update(dO=normal(*lead, H, dv).to(io), dS=normal(c["n"], H, dk, dv))
    return s


# ------------------------------------------------------------------ the library's calls

def _own(s):
    import uncertainty_aware_delta_gb300 as kdn

    op = s["case"]["op"]
    if op == "forward":
        return kdn.kdn_decay_forward(s["q"], s["k"], s["v"], s["log_decay"], s["S0"], cu=s["cu"])
    if op == "step":
        return kdn.kdn_decay_step(s["q"], s["k"], s["v"], s["log_decay"], s["S"]), s["S"]
    if op == "backward":
        g = kdn.kdn_decay_backward(s["q"], s["k"], s["v"], s["log_decay"], s["S0"], s["dO"], s["dS"], cu=s["cu"])
        return tuple(g[n] for n in ("q", "k", "v", "S0"))
    if op == "norm":
        return kdn.kdn_group_norm(s["x"], s["w"], s["b"], gate=s["gate"], act=s["case"]["act"])
    g = kdn.kdn_group_norm_backward(s["x"], s["dy"], s["w"], s["b"], gate=s["gate"], act=s["case"]["act"])
    return {n: t for n, t in g.items() if t is not None}


# ------------------------------------------------------------------ the plain forms

def _places(s, back):
    """Token indices [n, longest] in a flat token axis, the last token first where `back`; which of them exist; lengths."""
    c, L = s["case"], s["longest"]
    cu = s["cu"].long() if c["ragged"] else torch.arange(c["n"] + 1, device=DEV) * c["T"]
    n = cu[1:] - cu[:-1]
    i = torch.arange(L, device=DEV)
    at = n[:, None] - 1 - i if back else i[None, :].expand(c["n"], -1)
    return (cu[:-1, None] + at.clamp(min=0)).clamp(max=int(s["q"].numel() // s["q"].shape[-1] // c["H"]) - 1), i < n[:, None], n


def _power(log_decay, n):
    """exp(log_decay n) for every head and whole number, [H, ...]: the product in 64 bits."""
    return torch.exp(log_decay.double().view(-1, *[1] * n.dim()) * n.double()).float()


def _memory(s, q, k, v, S0, back=False, late=1):
    """o_t = sum_{j <= t} g^(t - j) (q_t k_j) v_j + g^(t + late) S0^T q_t along every sequence, from its end where `back`, and
    sum_j g^(last - j) k_j v_j^T + g^(last + late) S0."""
    at, live, n = _places(s, back)
    H, l = q.shape[-2], s["log_decay"]
    pad = -at.shape[1] % BLOCK
    fit = lambda t: torch.nn.functional.pad(   # noqa: E731  [n, H, blocks, BLOCK, d]
        (t.float().flatten(0, -3)[at] * live[..., None, None]).movedim(2, 1), (0, 0, 0, pad)).unflatten(2, (-1, BLOCK))
    qq, kk, vv = fit(q), fit(k), fit(v)
    i = torch.arange(BLOCK, device=DEV)
    gap = i[:, None] - i
    near = torch.where(gap >= 0, _power(l, gap.clamp(min=0)), 0.0)[:, None]
    o = torch.matmul(torch.matmul(qq, kk.transpose(-1, -2)) * near, vv)
    # what every block adds to the state, and the states that the blocks begin with
    own_part = torch.matmul((kk * _power(l, BLOCK - 1 - i)[:, None, :, None]).transpose(-1, -2), vv).flatten(3)
    b = torch.arange(own_part.shape[2], device=DEV)
    gap = (b[:, None] - 1 - b) * BLOCK
    far = torch.where(gap >= 0, _power(l, gap.clamp(min=0)), 0.0)
    begin = torch.matmul(far, own_part) + _power(l, b * BLOCK + late - 1)[..., None] * S0.flatten(2).unsqueeze(2)
    o = o + torch.matmul(qq, begin.unflatten(3, S0.shape[2:])) * _power(l, i + 1)[:, None, :, None]
    t = torch.arange(kk.shape[2] * BLOCK, device=DEV)
    left = n[:, None] - 1 - t
    weight = torch.where(left >= 0, _power(l, left.clamp(min=0)), 0.0).transpose(0, 1)
    end = torch.matmul((kk.flatten(2, 3) * weight[..., None]).transpose(-1, -2), vv.flatten(2, 3))
    end = end + _power(l, n - 1 + late).transpose(0, 1)[..., None, None] * S0
    flat = torch.empty((q.numel() // q.shape[-1] // H, H, v.shape[-1]), dtype=q.dtype, device=DEV)
    flat[at[live]] = o.flatten(2, 3)[:, :, : at.shape[1]].movedim(1, 2)[live].to(q.dtype)
    return flat.view(v.shape), end


def _plain_backward(s):
    q, k, v, dO, S0, dS = (s[n] for n in ("q", "k", "v", "dO", "S0", "dS"))
    dq, _ = _memory(s, dO, v, k, S0.transpose(-1, -2))
    dk, _ = _memory(s, v, dO, q, dS.transpose(-1, -2), back=True, late=0)
    dv, first = _memory(s, k, q, dO, dS, back=True, late=0)
    return dq, dk, dv, first * torch.exp(s["log_decay"])[:, None, None]


def _plain_step(s):
    q, k, v = (s[n].float() for n in ("q", "k", "v"))
    S = s["S"]
    S.copy_(S * torch.exp(s["log_decay"])[:, None, None] + k[..., :, None] * v[..., None, :])
    return torch.matmul(q[..., None, :], S).squeeze(-2).to(s["q"].dtype), S


def _act(kind, x):
    """The activation's value and slope."""
    if kind == "none":
        return x, torch.ones_like(x)
    h = torch.sigmoid(x)
    return (h, h * (1 - h)) if kind == "sigmoid" else (x * h, h * (1 + x * (1 - h)))


def _normed(s):
    x = s["x"].float()
    x = x - x.mean(-1, keepdim=True)
    r = torch.rsqrt((x * x).mean(-1, keepdim=True) + 1e-5)
    x = x * r
    return x, r, x * s["w"] + s["b"] if s["w"] is not None else x


def _plain_norm(s):
    kind = s["case"]["act"]
    _, _, n = _normed(s)
    y = _act(kind, n)[0] if s["gate"] is None else n * _act(kind, s["gate"].float())[0]
    return y.to(s["x"].dtype)


def _plain_norm_backward(s):
    kind, dy = s["case"]["act"], s["dy"].float()
    x, r, n = _normed(s)
    out = {}
    if s["gate"] is None:
        dn = dy * _act(kind, n)[1]
    else:
        a, slope = _act(kind, s["gate"].float())
        dn = dy * a
        out["gate"] = (dy * n * slope).to(s["x"].dtype)
    dx = dn
    if s["w"] is not None:
        out.update(weight=(dn * x).sum(0), bias=dn.sum(0))
        dx = dn * s["w"]
    dx = r * (dx - dx.mean(-1, keepdim=True) - x * (dx * x).mean(-1, keepdim=True))
    return {"x": dx.to(s["x"].dtype), **out}


def run(state):
    if own:
        return _own(state)
    op = state["case"]["op"]
    if op == "forward":
        return _memory(state, state["q"], state["k"], state["v"], state["S0"])
    return {"step": _plain_step, "backward": _plain_backward, "norm": _plain_norm,
            "norm_backward": _plain_norm_backward}[op](state)


# ------------------------------------------------------------------ the definitions, in 64 bits

def _walk(q, k, v, g, S, step=256):
    """The recurrence over [m, T, H, d] tokens, `step` of them at a time: outputs and the last state."""
    out = []
    for t in range(0, q.shape[1], step):
        a, b, x = (y[:, t:t + step].transpose(1, 2) for y in (q, k, v))
        m = torch.arange(a.shape[2], device=DEV, dtype=torch.float64)
        gap = m[:, None] - m
        w = torch.exp(g[:, None, None] * gap.clamp(min=0)) * (gap >= 0)
        carried = torch.einsum("nhtd,nhde->nhte", a, S) * torch.exp(g[:, None] * (m + 1))[..., None]
        out.append((torch.einsum("nhts,nhse->nhte", torch.einsum("nhtd,nhsd->nhts", a, b) * w, x) + carried).transpose(1, 2))
        late = torch.exp(g[:, None] * (m[-1] - m))[..., None]
        S = S * torch.exp(g * a.shape[2])[:, None, None] + torch.einsum("nhsd,nhse->nhde", b * late, x)
    return torch.cat(out, 1), S


def _exact_memory(c, s):
    g = s["log_decay"].double()
    names = ["q", "k", "v"] + (["dO"] if c["op"] == "backward" else [])
    n = _cu(_lengths(c)) if c["ragged"] else None
    # one sequence at a time where they differ in length, else all at once
    parts = [(slice(i, i + 1), slice(int(n[i]), int(n[i + 1]))) for i in range(c["n"])] if c["ragged"] else [(slice(None), None)]
    rows = []
    for seq, tok in parts:
        x = [(s[name] if tok is None else s[name][tok][None]).double() for name in names]
        S0 = s["S0"][seq].double()
        if c["op"] == "forward":
            o, S = _walk(*x, g, S0)
            rows.append((o, S))
            continue
        leaves = [t.requires_grad_() for t in (*x[:3], S0)]
        with torch.enable_grad():
            o, S = _walk(*leaves[:3], g, leaves[3])
            loss = (o * x[3]).sum() + (S * s["dS"][seq].double()).sum()
        rows.append(torch.autograd.grad(loss, leaves))
    whole = [torch.cat(t, 0) if not c["ragged"] else None for t in zip(*rows)]
    if not c["ragged"]:
        return tuple(whole)
    return tuple(torch.cat([r[i][0] if i < len(rows[0]) - 1 else r[i] for r in rows], 0) for i in range(len(rows[0])))


def _exact_norm(c, s):
    x, w, b, gate = (s[n].double() if s[n] is not None else None for n in ("x", "w", "b", "gate"))
    leaves = {"x": x, "weight": w, "bias": b, "gate": gate}
    f = {"none": lambda t: t, "silu": torch.nn.functional.silu, "sigmoid": torch.sigmoid}[c["act"]]
    used = {n: t.requires_grad_() for n, t in leaves.items() if t is not None}
    with torch.enable_grad():
        n = torch.nn.functional.layer_norm(x, (c["d"],), eps=1e-5)
        n = n * w + b if w is not None else n
        y = f(n) if gate is None else n * f(gate)
    if c["op"] == "norm":
        return y.detach()
    return dict(zip(used, torch.autograd.grad((y * s["dy"].double()).sum(), list(used.values()))))


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] in ("norm", "norm_backward"):
        return _exact_norm(case, s)
    if case["op"] == "step":
        q, k, v, S = (s[n].double() for n in ("q", "k", "v", "S"))
        S = S * torch.exp(s["log_decay"].double())[:, None, None] + torch.einsum("nhd,nhe->nhde", k, v)
        return torch.einsum("nhd,nhde->nhe", q, S), S
    return _exact_memory(case, s)
