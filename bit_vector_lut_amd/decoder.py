"""A small decoder stack out of the library's parts, served step by step (an example).

    python -m bit_vector_lut_amd.decoder

makes a seeded random model, prefills three prompts in one step and then decodes tokens for all of
them.  Every step takes the new tokens of all requests packed one after another:

    plan   PagePlanner        block tables, slots and row starts from the requests' lengths
    mixer  LUTProjection      -> PagedCache.store and .attention (every `full_every`-th layer), or
                              -> LinearAttention with its state per request (the other layers)
    norm   BlockNorm          norm of the mixer's or MLP's output, FP32 residual sum, norm for the next
    MLP    MLP                the three-bit vector-LUT MLP
    head   LUTProjection.argmax

Lengths, tables, states and the free list stay on the device; the host knows only how many tokens it
hands in.  The weights are random, so the tokens mean nothing.
"""
from __future__ import annotations

import numpy as np

from . import synth, vqmlp


class Decoder:
    """Weights, caches and states for up to `requests` requests of up to `max_len` tokens each."""

    def __init__(self, H=1024, I=2816, layers=4, full_every=4, heads=8, kv_heads=2, D=128, k_heads=4,
                 v_heads=8, Dk=64, Dv=128, vocab=4096, requests=3, max_len=512, page_size=16, t_max=256,
                 seed=0, device="cuda"):
        import torch

        rng = np.random.default_rng(seed)
        dev = torch.device(device, torch.cuda.current_device()) if device == "cuda" else torch.device(device)
        self.H, self.heads, self.kv_heads, self.D = H, heads, kv_heads, D
        self.k_heads, self.v_heads, self.Dk, self.Dv = k_heads, v_heads, Dk, Dv
        self.R, self.max_len, self.t_max, self.device = requests, max_len, t_max, dev

        def weight(n, at=1.0, spread=0.1):
            return torch.from_numpy((at + spread * rng.standard_normal(n)).astype(np.float16)).to(dev)

        def project(N, K, rank=64):
            return vqmlp.LUTProjection.from_proj(synth.lut_projection(rng, 4, N, K, rank, 1024), dev)

        self.embed = torch.from_numpy(rng.standard_normal((vocab, H)).astype(np.float16)).to(dev)
        self.head = project(vocab, H, rank=0)  # the argmax head takes no factors
        width = -(-max_len // page_size)
        pages = requests * width
        i32 = dict(dtype=torch.int32, device=dev)
        self.table = torch.full((requests, width), -1, **i32)
        free = torch.from_numpy(rng.permutation(pages).astype(np.int32)).to(dev)
        self.free_head = [torch.zeros(1, **i32), torch.zeros(1, **i32)]  # of this step and the next
        self.planners = [vqmlp.PagePlanner(self.table, free, page_size, pages, t_max, free_head=h)
                         for h in self.free_head]
        self.ctx_len = torch.zeros(requests, **i32)
        self.errors = torch.zeros(1, **i32)  # the error bits of all plans so far

        self.layers = []
        pre = [weight(H) for _ in range(2 * layers + 1)]  # norms in front of each mixer, MLP, the head
        self.first = vqmlp.BlockNorm(pre[0])
        for i in range(layers):
            layer = dict(full=(i + 1) % full_every == 0)
            if layer["full"]:
                layer["into"] = project((heads + 2 * kv_heads) * D, H)
                layer["out"] = project(H, heads * D)
                layer["cache"] = vqmlp.PagedCache.empty(pages, kv_heads, page_size, D, torch.float16, dev)
            else:
                gates = -(-v_heads // 64) * 64
                layer["into"] = project(2 * k_heads * Dk + v_heads * Dv + gates, H)
                layer["out"] = project(H, v_heads * Dv)
                layer["linear"] = vqmlp.LinearAttention(k_heads, v_heads, Dk, Dv)
                layer["state"] = layer["linear"].state(requests, dev)
                # queries and keys of length one: an RMS norm with weights Dk^-1/2
                layer["unit"] = vqmlp.BlockNorm(weight(Dk, Dk ** -0.5, 0.0))
                layer["bias"] = torch.from_numpy(rng.uniform(-5, 0, v_heads).astype(np.float32)).to(dev)
            layer["mlp"] = vqmlp.MLP.from_layer(synth.mlp_layer(H, I, 1, seed=rng), dev, t_max=t_max)
            layer["mid"] = vqmlp.BlockNorm(pre[2 * i + 1], post_weight=weight(H))
            layer["end"] = vqmlp.BlockNorm(pre[2 * i + 2], post_weight=weight(H))
            self.layers.append(layer)

    def _attend(self, layer, x, plan):
        h, k, D, T = self.heads, self.kv_heads, self.D, x.shape[0]
        qkv = layer["into"].forward(x).unflatten(1, (h + 2 * k, D))
        layer["cache"].store(qkv[:, h:h + k], qkv[:, h + k:], plan.slot)
        y = layer["cache"].attention(qkv[:, :h], self.table, plan.cu_q, plan.seq_len)
        return layer["out"].forward(y.view(T, h * D))

    def _recur(self, layer, x, plan, longest):
        import torch

        T, n = x.shape[0], self.k_heads * self.Dk
        z = layer["into"].forward(x)
        qk = layer["unit"].forward(z[:, :2 * n].reshape(-1, self.Dk))[1].view(T, 2 * self.k_heads, self.Dk)
        v = z[:, 2 * n:2 * n + self.v_heads * self.Dv].unflatten(1, (self.v_heads, self.Dv))
        gate = z[:, 2 * n + self.v_heads * self.Dv:][:, :self.v_heads].float()
        g = -torch.nn.functional.softplus(gate + layer["bias"])
        y, _ = layer["linear"].forward(qk[:, :self.k_heads], qk[:, self.k_heads:], v, g, layer["state"],
                                       plan.cu_q, ctx_len=self.ctx_len, max_q=longest,
                                       state_out=layer["state"])
        return layer["out"].forward(y.view(T, self.v_heads * self.Dv))

    def step(self, tokens, lens):
        """tokens: the requests' new tokens one after another (device, [sum of lens]); lens: how many each
        request brings (host).  Returns (hidden states [T, H] in front of the head, the PagePlan).  A plan
        that fails (a request beyond max_len) leaves the requests as they are and its bits in `errors`."""
        import torch

        T = tokens.shape[0]
        if T != sum(lens) or len(lens) != self.R or T > self.t_max:
            raise ValueError("tokens do not fit lens, requests or t_max")
        now, then = self.free_head
        planner = self.planners[0]
        q_len = torch.tensor(lens, dtype=torch.int32, device=self.device)
        plan = planner.forward(self.ctx_len, q_len, free_head_out=then)
        self.errors |= plan.status[:1]
        self.free_head.reverse()
        self.planners.reverse()
        r = self.embed[tokens].float()
        x = self._first(r)
        for layer in self.layers:
            y = self._attend(layer, x, plan) if layer["full"] else self._recur(layer, x, plan, max(lens))
            r, x = layer["mid"].forward(y, r, residual_out=r)
            r, x = layer["end"].forward(layer["mlp"].forward(x), r, residual_out=r)
        self.ctx_len = plan.seq_len
        return x, plan

    def _first(self, r):
        return self.first.forward(None, r)[1]

    def next_tokens(self, x, plan):
        """Greedy next token of each request from the hidden states of its last row; -1 for a request
        without new tokens in this step, and for all of them after a plan that failed (int32)."""
        import torch

        end = plan.cu_q[1:]
        tokens = self.head.argmax(x[(end - 1).clamp(min=0).long()].contiguous())[0]
        return torch.where(end > plan.cu_q[:-1], tokens, -1)


def main(steps=16, seed=0):
    import torch

    lens = [37, 5, 70]
    model = Decoder(requests=len(lens), seed=seed)
    tokens = torch.randint(0, 4096, (sum(lens),), device=model.device)
    out = []
    for i in range(steps + 1):
        x, plan = model.step(tokens, lens)
        tokens, lens = model.next_tokens(x, plan).long(), [1] * len(lens)
        out.append(tokens)
    if model.errors.item():
        raise RuntimeError("a plan failed, error bits %d" % model.errors.item())
    print("status of the last plan (errors, tokens, new pages, 0):", plan.status.tolist())
    for r, row in enumerate(torch.stack(out, 1).tolist()):
        print("request %d:" % r, row)


if __name__ == "__main__":
    main()
