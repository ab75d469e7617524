"""Binding of a retention layer's operators (include/kdn.h): linear attention with a decay for each head (whole sequences,
one token a sequence, gradients), and the group norm with activation that a memory's outputs go through (with its gradients).
Argument marshalling only, as in :mod:`.binding`; outputs carry no history: the gradients are calls of their own.
"""
from __future__ import annotations

import torch

from .attention import _call, _int, _io, _refuse, _tensor, _workspace
from .binding import KDN_BF16, library

_ACT = {"none": 0, "silu": 1, "sigmoid": 2}


def _fits(t, name):
    """The sizes of a tensor as 32-bit arguments (ctypes would cut them off; those of one with few elements need no look)."""
    if not 0 < t.numel() <= 0x7fffffff and max(t.shape) > 0x7fffffff:
        raise ValueError(f"a size of {name}, {max(t.shape)}, does not fit 32 bits")
    return t.shape


def _tokens(t, name):
    """Tokens, heads and channels of [B, T, heads, d] or [tokens, heads, d]."""
    if not isinstance(t, torch.Tensor) or t.dim() not in (3, 4):
        raise ValueError(f"{name} must be a tensor [B, T, heads, d] or [tokens, heads, d]")
    s = _fits(t, name)
    return (_int(s[0] * s[1], "tokens"), s[2], s[3]) if len(s) == 4 else s


def _operand(t, name, dtype, shape, device):
    """Pointer, row stride and head stride of a [B, T, heads, d] or [tokens, heads, d] operand of this shape (no view of it is
    made: that would take longer than the checks)."""
    if isinstance(t, torch.Tensor) and t.dtype is dtype and t.device == device and t.is_cuda and t.shape == shape:
        if len(shape) == 3:
            row, head, one = t.stride()
        else:
            seq, row, head, one = t.stride()
            if shape[1] == 1:
                row = seq
            elif shape[0] > 1 and seq != row * shape[1] and t.numel():
                raise ValueError(f"the sequences of {name} must lie one after another")
        if one == 1 or shape[-1] <= 1 or t.numel() == 0:
            return t.data_ptr(), row, head
    _refuse(t, name, dtype, shape, device, False)


def _maybe(t, name, dtype, shape, device):
    return None if t is None else _tensor(t, name, dtype, shape, device)


def _sequences(q, cu, device):
    """Sequences and the pointer of their bounds."""
    if cu is None:
        if q.dim() != 4:
            raise ValueError("tokens packed as [tokens, H, d] need cu")
        return q.shape[0], None
    if q.dim() != 3:
        raise ValueError("with cu, tokens are packed as [tokens, H, d]")
    if not isinstance(cu, torch.Tensor) or cu.dim() != 1 or cu.shape[0] < 1:
        raise ValueError("cu must be a tensor [sequences + 1]")
    return _int(cu.shape[0] - 1, "sequences"), _tensor(cu, "cu", torch.int32, cu.shape, device)


def decay_workspace_size(n_seq, n_tok, H, dk, dv, io=KDN_BF16, flags=0) -> int:
    names = ("n_seq", "n_tok", "H", "dk", "dv", "io", "flags")
    return int(library().kdn_decay_workspace_size(*map(_int, (n_seq, n_tok, H, dk, dv, io, flags), names)))


def decay_backward_workspace_size(n_seq, n_tok, H, dk, dv, io=KDN_BF16, flags=0) -> int:
    names = ("n_seq", "n_tok", "H", "dk", "dv", "io", "flags")
    return int(library().kdn_decay_backward_workspace_size(*map(_int, (n_seq, n_tok, H, dk, dv, io, flags), names)))


def kdn_decay_forward(q, k, v, log_decay, S0=None, *, cu=None, flags=0, out=None, workspace=None, stream=None):
    """S_t = exp(log_decay) S_{t-1} + k_t v_t^T, o_t = S_t^T q_t along every sequence.  Returns (o, S_T).

    q, k [B, T, H, dk], v [B, T, H, dv] fp32 or bf16, or packed: [tokens, H, d] with cu [sequences + 1] int32;
    log_decay [H], S0 and S_T [sequences, H, dk, dv] fp32.  ``out=(o, S_T)`` writes into tensors (S_T may be S0).
    """
    lib = library()
    device, io, flags = q.device, _io(q, "q"), _int(flags, "flags")
    tok, H, dk = _tokens(q, "q")
    n, cu_ptr = _sequences(q, cu, device)
    keys, dv, f32 = q.shape, _fits(v, "v")[-1], torch.float32
    shape, dt = (*keys[:-1], dv), q.dtype
    states = (n, H, dk, dv)
    if out is None:
        made = [torch.empty(shape, dtype=dt, device=device), torch.empty(states, dtype=f32, device=device)]
        o, S_T = made
        outs = o.data_ptr(), S_T.data_ptr()
    else:
        made, (o, S_T) = [], out
        outs = _tensor(o, "o", dt, shape, device), _tensor(S_T, "S_T", f32, states, device)
    need = lib.kdn_decay_workspace_size(n, tok, H, dk, dv, io, flags)
    ws, ws_bytes = _workspace(workspace, need, device, made)
    _call(lib.kdn_decay_forward, device, stream,
          (n, tok, H, dk, dv, io, flags, *_operand(q, "q", dt, keys, device), *_operand(k, "k", dt, keys, device),
           *_operand(v, "v", dt, shape, device), _tensor(log_decay, "log_decay", f32, (H,), device),
           _maybe(S0, "S0", f32, states, device), cu_ptr, *outs, ws, ws_bytes), made)
    return o, S_T


def kdn_decay_step(q, k, v, log_decay, S, *, o=None, stream=None):
    """One token of the same recurrence per sequence: q, k [B, H, dk], v [B, H, dv]; S [B, H, dk, dv] fp32 is updated in
    place.  Returns o [B, H, dv]."""
    device, io = q.device, _io(q, "q")
    B, H, dk = _fits(q, "q")
    dv, made = _fits(v, "v")[-1], []
    if o is None:
        o = torch.empty((B, H, dv), dtype=q.dtype, device=device)
        made.append(o)
        out = o.data_ptr()
    else:
        out = _tensor(o, "o", q.dtype, (B, H, dv), device)
    _call(library().kdn_decay_step, device, stream,
          (B, H, dk, dv, io, _tensor(q, "q", q.dtype, (B, H, dk), device), _tensor(k, "k", q.dtype, (B, H, dk), device),
           _tensor(v, "v", q.dtype, (B, H, dv), device), _tensor(log_decay, "log_decay", torch.float32, (H,), device),
           _tensor(S, "S", torch.float32, (B, H, dk, dv), device), out), made)
    return o


def kdn_decay_backward(q, k, v, log_decay, S0=None, dO=None, dS_T=None, *, cu=None, flags=0, workspace=None, stream=None):
    """Gradients of sum(dO o) + sum(dS_T S_T) of :func:`kdn_decay_forward` with these inputs.  Returns a dict: q, k, v (in
    the type of the inputs) and S0 (fp32)."""
    lib = library()
    device, io, flags = q.device, _io(q, "q"), _int(flags, "flags")
    tok, H, dk = _tokens(q, "q")
    n, cu_ptr = _sequences(q, cu, device)
    keys, dv, f32 = q.shape, _fits(v, "v")[-1], torch.float32
    values, dt = (*keys[:-1], dv), q.dtype
    states = (n, H, dk, dv)
    grads = {name: torch.empty(shape, dtype=dt, device=device) for name, shape in (("q", keys), ("k", keys), ("v", values))}
    grads["S0"] = torch.empty(states, dtype=f32, device=device)
    made = list(grads.values())
    need = lib.kdn_decay_backward_workspace_size(n, tok, H, dk, dv, io, flags)
    ws, ws_bytes = _workspace(workspace, need, device, made)
    _call(lib.kdn_decay_backward, device, stream,
          (n, tok, H, dk, dv, io, flags, *_operand(q, "q", dt, keys, device), *_operand(k, "k", dt, keys, device),
           *_operand(v, "v", dt, values, device), _tensor(log_decay, "log_decay", f32, (H,), device),
           _maybe(S0, "S0", f32, states, device), cu_ptr, *_operand(dO, "dO", dt, values, device),
           _maybe(dS_T, "dS_T", f32, states, device), *(grads[name].data_ptr() for name in ("q", "k", "v", "S0")), ws, ws_bytes), made)
    return grads


def _activation(act):
    if act not in _ACT:
        raise ValueError(f"act must be one of {sorted(_ACT)}, not {act!r}")
    return _ACT[act]


def kdn_group_norm(x, weight=None, bias=None, *, gate=None, act="none", eps=1e-5, out=None, stream=None):
    """Norm of every row's groups of channels, n = (x - mean) / sqrt(var + eps) weight + bias, and act(n), or n act(gate).

    x, gate [rows, groups, d] or [B, T, groups, d] fp32 or bf16; weight, bias [groups, d] fp32; act "none", "silu" or "sigmoid".
    """
    shape, device, io, kind = x.shape, x.device, _io(x, "x"), _activation(act)
    rows, G, d = _tokens(x, "x")
    made = []
    if out is None:
        out = torch.empty(shape, dtype=x.dtype, device=device)
        made.append(out)
        y = out.data_ptr()
    else:
        y = _tensor(out, "out", x.dtype, shape, device)
    gates = (None, 0, 0) if gate is None else _operand(gate, "gate", x.dtype, shape, device)
    _call(library().kdn_group_norm, device, stream,
          (rows, G, d, kind, eps, io, *_operand(x, "x", x.dtype, shape, device),
           _maybe(weight, "weight", torch.float32, (G, d), device), _maybe(bias, "bias", torch.float32, (G, d), device), *gates,
           y), made)
    return out


def group_norm_backward_workspace_size(rows, groups, d, io=KDN_BF16) -> int:
    return int(library().kdn_group_norm_backward_workspace_size(*map(_int, (rows, groups, d, io), ("rows", "groups", "d", "io"))))


def kdn_group_norm_backward(x, dy, weight=None, bias=None, *, gate=None, act="none", eps=1e-5, workspace=None, stream=None):
    """Gradients of sum(dy y) of :func:`kdn_group_norm` with these inputs.  Returns a dict: x, gate (in the type of the
    inputs), weight, bias (fp32); None for what was not given."""
    lib = library()
    shape, device, io, kind = x.shape, x.device, _io(x, "x"), _activation(act)
    rows, G, d = _tokens(x, "x")
    f32 = dict(dtype=torch.float32, device=device)
    grads = {"x": torch.empty(shape, dtype=x.dtype, device=device),
             "gate": None if gate is None else torch.empty(shape, dtype=x.dtype, device=device),
             "weight": None if weight is None else torch.empty((G, d), **f32),
             "bias": None if bias is None else torch.empty((G, d), **f32)}
    made = [t for t in grads.values() if t is not None]
    gates = (None, 0, 0) if gate is None else _operand(gate, "gate", x.dtype, shape, device)
    ws, ws_bytes = _workspace(workspace, lib.kdn_group_norm_backward_workspace_size(rows, G, d, io), device, made)
    _call(lib.kdn_group_norm_backward, device, stream,
          (rows, G, d, kind, eps, io, *_operand(x, "x", x.dtype, shape, device),
           _maybe(weight, "weight", torch.float32, (G, d), device), _maybe(bias, "bias", torch.float32, (G, d), device), *gates,
           *_operand(dy, "dy", x.dtype, shape, device),
           *(None if grads[name] is None else grads[name].data_ptr() for name in ("x", "gate", "weight", "bias")), ws, ws_bytes), made)
    return grads
