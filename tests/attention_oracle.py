"""Plain 64-bit definitions of the attention operators and of the 4-bit cache, for the tests.

Written from include/kdn.h with numpy, one request and one head at a time; shares no code
with the library.

Tolerances (derived, not fitted).  With A = sum_j p_j |v_j| (p the exact softmax) and
E = max_j scale sum_d |q_d k_jd| of a row:
  scores: products are exact or 3xTF32 (2^-21 of each product), summed in fp32 in at most 48
    steps that each round by at most 2^-23 of the partial sum: |dx| <= 2^-17 E; doubled
    for the exponent's own rounding of the same size: dx = 2^-16 E + 2^-20.
  a score error dx changes the output by at most 2 dx A.
  weights rounded to bf16 (unit roundoff 2^-8; prompts in bf16): 2^-8 A; to fp16 after the product with the
    value scale (cache): 2^-10 A, with the whole weight in two parts for fp32: 2^-20 A; both
    while the weight is a normal fp16 number.  Below, each key adds an absolute 2^-34 of the largest
    weight times V, the largest |v|, or 2^-34 (2^-5 / s) V where the largest value scale s is
    below 2^-5 (the kernel brings the largest weight to 2^10 or 2^15, fp16's spacing ends at 2^-24).
  output rounded to bf16: 2^-8 |o|.
  the sum over the keys in fp32: 2^-18 A.
"""
import numpy as np

F16_MAX = 65504.0


def attend(q, k, v, scale, lo, hi):
    """One query row over keys lo..hi-1: (o, lse, A, E) in fp64."""
    d = v.shape[1]
    if hi <= lo:
        return np.zeros(d), -np.inf, np.zeros(d), 0.0
    q, k, v = q.astype(np.float64), k[lo:hi].astype(np.float64), v[lo:hi].astype(np.float64)
    with np.errstate(invalid="ignore", over="ignore"):
        x = scale * (k @ q)
        m = x.max()
        p = np.exp(x - m)
        l = p.sum()
        p = p / l
        return p @ v, m + np.log(l), p @ np.abs(v), scale * (np.abs(k) @ np.abs(q)).max()


def prompt(q, k, v, cu_q, cu_k, window, scale):
    """(o, lse, A, E) of packed prompts; rows of no sequence are NaN."""
    nq, H, d = q.shape
    rep = H // k.shape[1]
    o, A = np.full((nq, H, d), np.nan), np.full((nq, H, d), np.nan)
    lse, E = np.full((nq, H), np.nan), np.full((nq, H), np.nan)
    for s in range(len(cu_q) - 1):
        q0, q1, k0, k1 = cu_q[s], cu_q[s + 1], cu_k[s], cu_k[s + 1]
        for i in range(q0, q1):
            place = (k1 - k0) - (q1 - q0) + (i - q0)
            lo = max(0, place - window + 1) if window else 0
            for h in range(H):
                kk, vv = k[k0:k1, h // rep], v[k0:k1, h // rep]
                o[i, h], lse[i, h], A[i, h], E[i, h] = attend(q[i, h], kk, vv, scale, lo, place + 1)
    return o, lse, A, E


def quantise(x):
    """Codes [..., d] and scales [..., d / 32] (as fp64) of values x: the format's arithmetic."""
    g = x.astype(np.float64).reshape(*x.shape[:-1], -1, 32)
    with np.errstate(invalid="ignore", over="ignore"):
        top = np.abs(g).max(-1)
        s = np.minimum(top / 7, F16_MAX).astype(np.float16).astype(np.float64)
        bad = ~np.isfinite(g).all(-1)
        s[bad] = np.nan
        f = s[..., None]
        code = np.where(f > 0, np.clip(np.rint(np.where(f > 0, g, 0) / np.where(f > 0, f, 1)), -7, 7), 0) + 8
    return code.reshape(x.shape).astype(np.int64), s


def values(code, s):
    return ((code.reshape(*code.shape[:-1], -1, 32) - 8) * s[..., None]).reshape(code.shape)


def unpack(cache, d):
    """Codes and scales [pages, heads, tokens, ...] of cache bytes [pages, heads, page / 16, 18 d],
    place by place from the layout's statement."""
    n, H, nb, _ = cache.shape
    G = d // 32
    ck, cv = np.zeros((2, n, H, nb * 16, d), np.int64)
    sk, sv = np.zeros((2, n, H, nb * 16, G))
    for b in range(nb):
        blk = np.ascontiguousarray(cache[:, :, b])
        kw = np.ascontiguousarray(blk[:, :, :8 * d]).view(np.uint32).reshape(n, H, 16, 4 * G)
        ks = np.ascontiguousarray(blk[:, :, 8 * d:9 * d]).view(np.float16).reshape(n, H, 16, G)
        vw = np.ascontiguousarray(blk[:, :, 9 * d:17 * d]).view(np.uint32).reshape(n, H, 2, 8, 4, G)
        vs = np.ascontiguousarray(blk[:, :, 17 * d:]).view(np.float16).reshape(n, H, 2, 4, G, 2)
        for t in range(16):
            at = b * 16 + t
            for g in range(G):
                sk[:, :, at, g] = ks[:, :, t, g]
                sv[:, :, at, g] = vs[:, :, t // 8, t // 2 % 4, g, t % 2]
                for c in range(4):
                    for e in range(8):
                        ck[:, :, at, 32 * g + 8 * c + e] = (kw[:, :, t, c * G + g] >> np.uint32(4 * e)) & 15
                for i in range(8):
                    for e in range(4):
                        w = vw[:, :, t // 8, i, t // 2 % 4, g]
                        cv[:, :, at, 32 * g + 8 * e + i] = (w >> np.uint32(16 * (t % 2) + 4 * e)) & 15
    return ck, sk, cv, sv


def plan(ctx, new, table, free, count, page, capacity):
    table = table.copy()
    R, width = table.shape
    stack = list(free[:min(max(count, 0), len(free))])
    left, wanted = len(stack), 0
    bad = count != left
    slots, pos, cu, lens, granted = [], [], [0], [], []
    for r in range(R):
        c, a = int(ctx[r]), max(int(new[r]), 0)
        ok = ctx[r] >= 0 and new[r] >= 0 and ctx[r] + new[r] <= width * page
        bad |= not ok
        held, need = 0, 0
        if ok:
            held = -(-c // page)
            need = -(-(c + a) // page) - held
        wanted += need
        g = ok and (need == 0 or wanted <= left)
        if g:
            for p in range(held, held + need):
                table[r, p] = stack.pop()
        for p in range(c, c + a):
            slots.append(int(table[r, p // page]) * page + p % page if g else -1)
            pos.append(p)
        cu.append(cu[-1] + a)
        lens.append(c + a if g else c)
        granted.append(int(g))
    bad |= cu[-1] > capacity
    slots, pos = (slots + [-1] * capacity)[:capacity], (pos + [0] * max(0, capacity - len(pos)))[:capacity]
    return dict(table=table, slot_map=np.array(slots, np.int64), position=np.array(pos, np.int64),
                cu_new=np.array(cu), seq_len=np.array(lens, np.int64), granted=np.array(granted, np.int64),
                free_left=np.array([len(stack)]), bad=bad)


def bounds(o, A, E, io, cached, floor=0.0):
    """Largest allowed |error| of the outputs, and of lse, from the derivation above."""
    dx = 2.0 ** -16 * E + 2.0 ** -20
    weight = (2.0 ** -10 if cached else 2.0 ** -8) if io == "bf16" else (2.0 ** -20 if cached else 0.0)
    out = A * (2 * dx[..., None] + weight + 2.0 ** -18) + (2.0 ** -8 * np.abs(o) if io == "bf16" else 0.0)
    return out * 1.01 + floor + 1e-30, dx + 2.0 ** -20


def check(got_o, got_lse, ref, io, cached=False, floor=0.0):
    """Assert outputs against (o, lse, A, E), special values in the same places."""
    o, lse, A, E = ref
    live = np.isfinite(o) & np.isfinite(A)
    assert np.array_equal(np.isnan(o), np.isnan(got_o))
    ob, lb = bounds(np.where(live, o, 0), np.where(live, A, 0), np.where(np.isfinite(E), E, 0), io, cached, floor)
    err = np.abs(np.where(live, got_o, 0) - np.where(live, o, 0))
    assert np.all(err <= ob), (float((err / ob).max()), np.argwhere(err > ob)[:3])
    fin = np.isfinite(lse)
    assert np.array_equal(np.isnan(lse), np.isnan(got_lse))
    assert np.array_equal(lse[~fin & ~np.isnan(lse)], got_lse[~fin & ~np.isnan(lse)])
    el = np.abs(got_lse[fin] - lse[fin])
    lb = lb[fin] + 2.0 ** -22 * np.abs(lse[fin])
    assert np.all(el <= lb), float((el / lb).max())
