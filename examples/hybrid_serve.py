"""Serve requests with a hybrid stack: KDN memories beside attention over a paged 4-bit cache.

Every layer is a Diagonal KDN mixer followed by causal attention (through a sliding window, or none)
with fewer key heads than query heads; weights are random.  One plan a call gives pages to all layers'
caches.  Prompts run packed one after another, the attention over what the cache holds of them already
and over their new tokens; then every request gets a token a step.

    python examples/hybrid_serve.py --requests 8 --prompt 700 --steps 32
"""
import argparse
import os
import sys

import torch
import torch.nn.functional as F

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import uncertainty_aware_delta_gb300 as kdn  # noqa: E402


def norm(x):
    return F.rms_norm(x.float(), x.shape[-1:]).to(x.dtype)


class Server:
    """`requests` places; each holds a request's KDN states, its pages and its length."""

    def __init__(self, requests, pages, *, layers=2, heads=8, kv_heads=2, d=128, page=64, table_width=64, window=0,
                 seed=0, device="cuda"):
        self.R, self.H, self.Hkv, self.d, self.page, self.window = requests, heads, kv_heads, d, page, window
        self.dim = heads * d
        g = torch.Generator(device=device).manual_seed(seed)

        def weight(n_in, n_out):
            return (torch.randn(n_in, n_out, generator=g, device=device) * n_in ** -0.5).bfloat16()

        self.layers = [dict(mix=weight(self.dim, 5 * self.dim + heads), mix_out=weight(self.dim, self.dim),
                            qkv=weight(self.dim, (heads + 2 * kv_heads) * d), out=weight(self.dim, self.dim),
                            S=torch.zeros(requests, heads, d, d, device=device),
                            p=torch.ones(requests, heads, d, device=device),
                            cache=kdn.cache_alloc(pages, page, kv_heads, d, device)) for _ in range(layers)]
        ints = dict(dtype=torch.int32, device=device)
        self.table = torch.full((requests, table_width), -1, **ints)
        self.free = torch.arange(pages - 1, -1, -1, **ints)     # a stack: the next page is its last
        self.n_free = torch.tensor([pages], **ints)
        self.context = torch.zeros(requests, **ints)
        self.plan_ws = torch.empty(256, dtype=torch.uint8, device=device)   # its status word
        self.device = self.table.device

    def _plan(self, new, capacity):
        # (table entries past a request's length mean nothing: until a plan is taken, another may be made in its place)
        plan = kdn.kdn_cache_plan(self.context, new, self.table, self.free, self.n_free, page=self.page, capacity=capacity,
                                  workspace=self.plan_ws)
        status = kdn.kdn_read_device_status(self.plan_ws)   # (waits, as reading what was granted would)
        if status:
            raise RuntimeError(f"the requests' lengths or the free pages: {kdn.status_string(status)}")
        return plan

    def _take(self, plan):
        self.n_free, self.context = plan.free_left, plan.seq_len

    def _mixer_inputs(self, layer, x):
        """q, k, v, log_alpha, omega, r of tokens x [n, dim]."""
        n = x.shape[0]
        z = norm(x) @ layer["mix"]
        q, k, v, a, w = z[:, :5 * self.dim].view(n, 5, self.H, self.d).unbind(1)
        r = F.softplus(z[:, 5 * self.dim:].float()) + 1e-3
        q, k = (F.normalize(t.float(), dim=-1).bfloat16() for t in (q, k))
        return [t.contiguous() for t in (q, k, v, F.logsigmoid(a.float() + 4.6), F.softplus(w.float() - 6.0), r)]

    def _attention_inputs(self, layer, x):
        z = (norm(x) @ layer["qkv"]).view(x.shape[0], self.H + 2 * self.Hkv, self.d)
        return z.split([self.H, self.Hkv, self.Hkv], 1)     # strided rows: taken as they are

    def prefill(self, x, new):
        """Tokens x [sum(new), dim] of the requests' prompts, packed.  Returns (their outputs, the granted requests);
        a request that got no pages keeps its state, and its outputs mean nothing."""
        ctx, cu = self.context.tolist(), [0]
        if max(c + n for c, n in zip(ctx, new)) > self.table.shape[1] * self.page:
            raise ValueError("a request is longer than its row of the block table")
        for n in new:
            cu.append(cu[-1] + n)
        plan = self._plan(torch.tensor(new, dtype=torch.int32, device=self.device), cu[-1])
        granted = plan.granted.tolist()
        self._take(plan)
        # every request's tokens, cached and new, in one row each; the new ones are not read back from the cache
        seq = [c + n for c, n in zip(ctx, new)]
        request = torch.repeat_interleave(torch.tensor(seq)).to(self.device)
        cu_k = F.pad(torch.tensor(seq).cumsum(0), (1, 0)).to(self.device, torch.int32)
        place = torch.arange(sum(seq), device=self.device) - cu_k.long()[request]
        known = self.table[request, place // self.page].long() * self.page + place % self.page
        mine = (place >= torch.tensor(ctx, device=self.device)[request]).nonzero()[:, 0]
        for layer in self.layers:
            mixed = torch.zeros_like(x).view(-1, self.H, self.d)
            z = self._mixer_inputs(layer, x)
            for r in range(self.R):
                if new[r] and granted[r]:
                    o, S, p = kdn.kdn_diag_forward(*(t[None, cu[r]:cu[r + 1]] for t in z),
                                                   layer["S"][r:r + 1], layer["p"][r:r + 1])
                    mixed[cu[r]:cu[r + 1]], layer["S"][r], layer["p"][r] = o[0], S[0], p[0]
            x = x + mixed.view_as(x) @ layer["mix_out"]
            q, k, v = self._attention_inputs(layer, x)
            if any(ctx):
                keys, vals = kdn.kdn_cache_read(layer["cache"], known)
                keys[mine], vals[mine] = k, v
            else:
                keys, vals = k, v
            kdn.kdn_cache_write(k, v, plan.slot_map, layer["cache"])
            o, _ = kdn.kdn_prompt_attention(q, keys, vals, plan.cu_new, cu_k, window=self.window)
            x = x + o.view_as(x) @ layer["out"]
        return x, granted

    def decode(self, x):
        """One token x [requests, dim] for every request.  Returns its output.  Where pages run out nothing changes:
        the call may be repeated once a request has been released."""
        plan = self._plan(torch.ones_like(self.context), self.R)
        if not bool(plan.granted.all()):
            raise RuntimeError("the cache is out of pages: release a request")
        self._take(plan)
        for layer in self.layers:
            o = kdn.kdn_step("diag", *self._mixer_inputs(layer, x), layer["S"], layer["p"])
            x = x + o.view_as(x) @ layer["mix_out"]
            q, k, v = self._attention_inputs(layer, x)
            kdn.kdn_cache_write(k, v, plan.slot_map, layer["cache"])
            o, _ = kdn.kdn_cache_attention(q, layer["cache"], self.table, plan.seq_len, window=self.window)
            x = x + o.view_as(x) @ layer["out"]
        return x

    def release(self, r):
        """Give a finished request's pages back and clear its place."""
        held, count = -(-int(self.context[r]) // self.page), int(self.n_free)
        self.free[count:count + held] = self.table[r, :held]
        self.n_free = self.n_free + held
        self.context = self.context.clone()
        self.context[r], self.table[r] = 0, -1
        for layer in self.layers:
            layer["S"][r], layer["p"][r] = 0, 1


def main():
    ap = argparse.ArgumentParser(description=__doc__.split("\n")[0])
    ap.add_argument("--requests", type=int, default=8)
    ap.add_argument("--prompt", type=int, default=700, help="longest prompt")
    ap.add_argument("--steps", type=int, default=32, help="tokens generated for each request")
    ap.add_argument("--window", type=int, default=0)
    a = ap.parse_args()
    gen = torch.Generator(device="cuda").manual_seed(1)
    width = -(-(2 * a.prompt + 2 * a.steps) // 64)
    s = Server(a.requests, a.requests * width, table_width=width, window=a.window)

    def tokens(n):
        return torch.randn(n, s.dim, generator=gen, device="cuda").bfloat16()

    def last(y, new):     # the next token is made from a prompt's last output
        return norm(y[torch.tensor(new, device="cuda").cumsum(0) - 1])

    first = [1 + (a.prompt - 1) * (r + 1) // a.requests for r in range(a.requests)]
    for turn, new in enumerate((first, first[::-1])):     # a second turn continues over the cached first
        y, granted = s.prefill(tokens(sum(new)), new)
        x = last(y, new)
        start, end = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
        start.record()
        for _ in range(a.steps):
            x = norm(s.decode(x))
        end.record()
        end.synchronize()
        print(f"turn {turn}: {sum(new)} prompt tokens of {sum(granted)} requests, then {a.steps} steps of "
              f"{a.requests} tokens at {start.elapsed_time(end) / a.steps:.2f} ms")
    held = int(s.context.sum())
    size = sum(layer["cache"].numel() for layer in s.layers)
    print(f"{held} tokens cached; caches of {size / 2 ** 20:.1f} MiB (bf16: {size * 32 / 9 / 2 ** 20:.1f} MiB); "
          f"outputs finite: {bool(torch.isfinite(x).all())}")
    for r in range(a.requests):
        s.release(r)
    print(f"{int(s.n_free)} of {a.requests * width} pages free")


if __name__ == "__main__":
    main()
