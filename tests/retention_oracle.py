"""Definitions of a retention layer's operators in 64 bits, token by token, and how far fp32 and bf16 may be from them.

Half a step of a type is torch.finfo(type).eps / 2 of the value: 2^-8 for bf16, 2^-24 for fp32.

Memory.  FP32 = 2^-17 of the sum of the absolute values of all terms (the same recurrence on absolute values): two products
follow one another (weights, then their product with v; what goes into the state, then its product with q), and each has
operands in two TF32 parts (dropped and rounded rest at most 2 x 2^-22 of a term) or three bf16 parts (2^-24), up to 14 sums
inside the matrix instructions, cut off at 2^-22 at most, and as many in fp32 at 2^-24: 2 x 16 x 2^-22.  Powers of the decay are
within |n log_decay| 2^-24, 128 x 2^-24 = 2^-17 of their own term at the far end of a chunk, where the term itself has
decayed by e^-128.  On the bf16 tensor-core path the weights, or the state, are rounded to bf16 for their product:
2^-8 of a term more.  Outputs in bf16 are rounded once: 2^-8 of the value.

Norm.  With s = 2^-19 and a = mean|x| / sigma: a mean of up to 256 values has 11 roundings of 2^-24 of mean|x|, the deviation
and the variance as many again, the square root and the exponential a few: xh is within s (|xh| + a + 1).  That goes into n
(times |w|) and into y by the slope of the activation, at most 1.1; sums of gradients over rows have a rounding a row of a
thread, at most 64 in these tests (2^-18 of the sum of absolute values).
"""
import torch

FP32 = 2.0 ** -17
HALF = {torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}


def walk(q, k, v, log_decay, S0, back=False):
    """One sequence, [T, H, d] in 64 bits: o_t = S_t^T q_t, S_t = g S_{t-1} + k_t v_t^T; from the end where `back`, S0 then
    added at the last token.  Returns o and the state after the last token (from the end: decayed once more)."""
    g = torch.exp(log_decay.double())[:, None, None]
    S, o = S0.double(), torch.empty(v.shape, dtype=torch.float64)
    order = range(q.shape[0] - 1, -1, -1) if back else range(q.shape[0])
    for i, t in enumerate(order):
        S = (S if back and i == 0 else g * S) + k[t][:, :, None] * v[t][:, None, :]
        o[t] = torch.einsum("hk,hkv->hv", q[t], S)
    return o, (g * S if back and q.shape[0] else S)


def sequences(x, cu):
    """The sequences' tokens of [B, T, H, d] or packed [tokens, H, d], on the host in 64 bits."""
    x = x.detach().cpu().double()
    return list(x) if cu is None else [x[int(a):int(b)] for a, b in zip(cu[:-1], cu[1:])]


def forward(q, k, v, log_decay, S0, cu=None):
    """(o, S_T) and (the same of absolute values)."""
    l = log_decay.detach().cpu()
    out = []
    for f in (lambda t: t, torch.abs):
        rows = [walk(f(a), f(b), f(c), l, f(s)) for a, b, c, s in zip(*(sequences(t, cu) for t in (q, k, v)), S0.detach().cpu().double())]
        o = [r[0] for r in rows]
        out.append((torch.stack(o) if cu is None else torch.cat(o), torch.stack([r[1] for r in rows])))
    return out


def backward(q, k, v, log_decay, S0, dO, dS, cu=None):
    """Gradients of q, k, v and S0, and the same of absolute values."""
    l = log_decay.detach().cpu()
    out = []
    for f in (lambda t: t, torch.abs):
        rows = []
        for a, b, c, d, s, e in zip(*(sequences(t, cu) for t in (q, k, v, dO)), S0.detach().cpu().double(), dS.detach().cpu().double()):
            a, b, c, d, s, e = (f(t) for t in (a, b, c, d, s, e))
            dq, _ = walk(d, c, b, l, s.transpose(1, 2))
            dk, _ = walk(c, d, a, l, e.transpose(1, 2), back=True)
            dv, first = walk(b, a, d, l, e, back=True)
            rows.append((dq, dk, dv, first))
        join = torch.stack if cu is None else torch.cat
        out.append(tuple(join([r[i] for r in rows]) for i in range(3)) + (torch.stack([r[3] for r in rows]),))
    return out


def check(got, want, size, rounded=False, what=""):
    """`got` within what its type and fp32 sums allow of `want`; `rounded`: terms went through bf16."""
    tol = HALF[got.dtype] * want.abs() + (FP32 + (2.0 ** -8 * (1 + 2.0 ** -8) if rounded else 0.0)) * size
    d = (got.detach().cpu().double() - want).abs()
    assert got.shape == want.shape
    worst = float((d / tol.clamp(min=1e-300)).max()) if d.numel() else 0.0
    assert bool((d <= tol).all()), f"{what}: {worst:.2f} of the tolerance"


def act(kind, x):
    if kind == "none":
        return x, torch.ones_like(x)
    h = torch.sigmoid(x)
    return (h, h * (1 - h)) if kind == "sigmoid" else (x * h, h * (1 + x * (1 - h)))


def norm(x, w, b, gate, kind, eps, dy=None):
    """{name: (value, tolerance without the type's own rounding)} of y, or of the gradients for dy."""
    x, w, b, gate, dy = (None if t is None else t.detach().cpu().double() for t in (x, w, b, gate, dy))
    s = 2.0 ** -19
    mean = x.mean(-1, keepdim=True)
    sigma = ((x - mean) ** 2).mean(-1, keepdim=True).add(eps).sqrt()
    xh, a = (x - mean) / sigma, x.abs().mean(-1, keepdim=True) / sigma
    big = xh.abs() + a + 1
    ww, bb = (torch.ones_like(x[0]) if w is None else w), (torch.zeros_like(x[0]) if b is None else b)
    n = xh * ww + bb
    en = s * (ww.abs() * big + bb.abs())
    if gate is None:
        f, slope = act(kind, n)
        if dy is None:
            return {"y": (f, 1.1 * en + s * f.abs())}
        dn, edn = dy * slope, dy.abs() * (0.5 * en + s * 1.1)     # (second derivatives are at most 1/2)
    else:
        f, slope = act(kind, gate)
        if dy is None:
            return {"y": (n * f, f.abs() * en + s * (n * f).abs() + s * n.abs())}
        dn, edn = dy * f, s * (dy * f).abs() + s * dy.abs()
    out = {}
    if gate is not None:
        out["gate"] = (dy * n * slope, dy.abs() * (1.1 * en + 2 * s * n.abs() + s))
    dxh, edx = dn * ww, edn * ww.abs() + s * (dn * ww).abs()
    m1, m2 = dxh.mean(-1, keepdim=True), (dxh * xh).mean(-1, keepdim=True)
    e1 = edx.mean(-1, keepdim=True) + s * dxh.abs().mean(-1, keepdim=True)
    e2 = (edx * big + 2 * s * dxh.abs() * big).mean(-1, keepdim=True)
    dx = (dxh - m1 - xh * m2) / sigma
    out["x"] = (dx, (edx + e1 + big * e2 + s * big * m2.abs() + 2 * s * (dxh.abs() + m1.abs() + (xh * m2).abs())) / sigma)
    if w is not None:
        out["weight"] = ((dn * xh).sum(0), (edn * big + s * dn.abs() * big).sum(0) + 2 * s * (dn * xh).abs().sum(0))
    if b is not None:
        out["bias"] = (dn.sum(0), edn.sum(0) + 2 * s * dn.abs().sum(0))
    return out


def check_norm(got, want, what=""):
    value, tol = want
    tol = tol + HALF[got.dtype] * (value.abs() + tol)
    d = (got.detach().cpu().double() - value).abs()
    assert got.shape == value.shape
    worst = float((d / tol.clamp(min=1e-300)).max()) if d.numel() else 0.0
    assert bool((d <= tol).all()), f"{what}: {worst:.2f} of the tolerance"
