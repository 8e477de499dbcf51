"""Operators in front of and inside a decoder's mixers: what is measured.

Three operators of a serving step over requests packed one after another (``cu_q`` holds their first
rows): the gated delta rule with its state per head, the append of new keys and values to a paged cache
with the heads' norms and the position rotation on the way, and the short causal convolution with its
state that feeds the delta rule.  ``run`` computes them in plain torch operations where ``own`` is false
and through ``bit_vector_lut_amd.vqmlp`` where it is true.
"""
import math

import torch

own = False

DEV = "cuda"
DTYPES = {"f16": torch.float16, "bf16": torch.bfloat16}
EPS = 1e-6


# ------------------------------------------------------------------ cases


def _text(pairs):
    return ",".join("%d:%d" % tuple(p) for p in pairs)


def _lens(case):
    """Per request: (new tokens, tokens before them)."""
    return [tuple(int(x) for x in p.split(":")) for p in case["lens"].split(",")]


def listed():
    return [
        # one request's eight drafted tokens through a recurrent layer: latency alone
        dict(name="delta_t8", op="delta", dtype="f16", lens="8:900", k_heads=16, v_heads=48, Dk=128, Dv=128),
        # one token for each of 64 requests, one of them new: the states' bytes
        dict(name="delta_r64", op="delta", dtype="bf16", lens=_text([1, 40 * int(i != 5)] for i in range(64)),
             k_heads=16, v_heads=48, Dk=128, Dv=128),
        # three packed prompts, two of them continued
        dict(name="delta_prompts", op="delta", dtype="f16", lens="5003:0,1021:512,2049:77", k_heads=16,
             v_heads=48, Dk=128, Dv=128),
        # a long prompt through one of eight shares of a layer's heads
        dict(name="delta_share", op="delta", dtype="bf16", lens="8000:0", k_heads=2, v_heads=6, Dk=128, Dv=128),
        # one request's eight drafted tokens at the end of a 64K context, a quarter of each head rotated
        dict(name="append_t8", op="append", dtype="f16", lens="8:65464", heads=24, kv_heads=4, D=256, rot=64,
             pairs="half", norm=True, page=64),
        # one new token for each of 64 requests, whole heads rotated
        dict(name="append_r64", op="append", dtype="bf16", lens=_text([1, 61 + 257 * i] for i in range(64)),
             heads=40, kv_heads=8, D=128, rot=128, pairs="half", norm=False, page=16),
        # a long packed batch of prompts
        dict(name="append_t8192", op="append", dtype="bf16", lens="5000:0,3191:1000,1:20000", heads=24,
             kv_heads=4, D=256, rot=64, pairs="half", norm=True, page=64),
        # a 512-token prompt chunk, neighbouring elements rotated
        dict(name="append_t512", op="append", dtype="f16", lens="512:32489", heads=40, kv_heads=8, D=128,
             rot=128, pairs="next", norm=False, page=16),
        # what stands in front of delta_t8
        dict(name="conv_t8", op="conv", dtype="f16", lens="8:900", C=10240, W=4, unit=32, unit_dim=128),
        # ... of delta_r64
        dict(name="conv_r64", op="conv", dtype="bf16", lens=_text([1, 40 * int(i != 5)] for i in range(64)),
             C=10240, W=4, unit=32, unit_dim=128),
        # ... of delta_prompts
        dict(name="conv_prompts", op="conv", dtype="f16", lens="5003:0,1021:512,2049:77", C=10240, W=4,
             unit=32, unit_dim=128),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def _draw_lens(rng, total, ctx):
    """Single tokens and drafts of many requests, or a few prompts."""
    if rng.random() < 0.5:
        return [[rng.randint(1, 8), rng.choice([0, _log_int(rng, 1, ctx)])] for _ in range(_log_int(rng, 1, 64))]
    R = rng.randint(1, 5)
    return [[_log_int(rng, 17, total // R), rng.choice([0, _log_int(rng, 1, ctx)])] for _ in range(R)]


def draw(rng):
    op = rng.choice(["delta", "delta", "append", "conv"])
    dt = rng.choice(["f16", "bf16"])
    if op == "delta":
        k_heads = rng.choice([1, 2, 4, 8, 16])
        return dict(op=op, dtype=dt, lens=_text(_draw_lens(rng, 8000, 30000)), k_heads=k_heads,
                    v_heads=k_heads * rng.choice([1, 2, 3]), Dk=rng.choice([64, 96, 128]),
                    Dv=rng.choice([64, 72, 128]))
    if op == "append":
        D = rng.choice([64, 80, 96, 128, 256])
        kv_heads = rng.choice([1, 2, 4])
        return dict(op=op, dtype=dt, lens=_text(_draw_lens(rng, 8000, 60000)),
                    heads=kv_heads * rng.choice([1, 3, 5, 6]), kv_heads=kv_heads, D=D,
                    rot=rng.choice([D, D, D // 4 // 8 * 8 + 8]), pairs=rng.choice(["half", "half", "next"]),
                    norm=rng.random() < 0.5, page=rng.choice([16, 32, 64, 128]))
    dim = rng.choice([64, 96, 128])
    unit = rng.choice([0, 2, 8, 32])
    return dict(op=op, dtype=dt, lens=_text(_draw_lens(rng, 8000, 30000)),
                C=unit * dim + 8 * _log_int(rng, 8, 700), W=rng.choice([2, 3, 4, 4]), unit=unit, unit_dim=dim)


def work(case):
    op = case["op"]
    T, R, old = sum(n for n, _ in _lens(case)), len(_lens(case)), sum(c > 0 for _, c in _lens(case))
    if op == "delta":
        hk, hv, dk, dv = case["k_heads"], case["v_heads"], case["Dk"], case["Dv"]
        return {"bytes": T * (4 * hk * dk + 4 * hv * dv + 8 * hv) + 4 * (R + old) * hv * dk * dv,
                "flops": 7 * T * hv * dk * dv}
    if op == "append":
        h, hk, D = case["heads"], case["kv_heads"], case["D"]
        turned = T * (h + hk) * (3 * case["rot"] + (4 * D if case["norm"] else 0))
        return {"bytes": T * (4 * (h + 2 * hk) * D + 8), "flops": turned}
    C, W = case["C"], case["W"]
    return {"bytes": 4 * T * C + 2 * C * W + 2 * (R + old) * (W - 1) * C,
            "flops": T * (C * (2 * W + 4) + 3 * case["unit"] * case["unit_dim"])}


# ------------------------------------------------------------------ inputs


def _normal(g, shape, dtype, std=1.0):
    return (torch.randn(shape, generator=g, device=DEV) * std).to(dtype)


def _ints(values):
    return torch.tensor(values, dtype=torch.int32, device=DEV)


def _inputs(case, seed):
    """The state without the library's handles: also what ``exact`` reads."""
    g = torch.Generator(device=DEV).manual_seed(int(seed) % (1 << 62))
    s, dt, lens = dict(case), DTYPES[case["dtype"]], _lens(case)
    starts = [0]
    for n, _ in lens:
        starts.append(starts[-1] + n)
    T, R = starts[-1], len(lens)
    s.update(starts=starts, cu_q=_ints(starts), ctx=_ints([c for _, c in lens]), max_q=max(n for n, _ in lens))
    if case["op"] == "delta":
        hk, hv, dk, dv = case["k_heads"], case["v_heads"], case["Dk"], case["Dv"]
        # q, k and v lie side by side, as the convolution in front leaves them: q and k of length one
        qk = torch.randn((T, 2 * hk, dk), generator=g, device=DEV)
        qk = (qk / qk.norm(dim=-1, keepdim=True)).to(dt).view(T, -1)
        z = torch.cat([qk, _normal(g, (T, hv * dv), dt)], 1)
        heads = torch.rand((hv,), generator=g, device=DEV) * 6 - 6.5  # decays of one to hundreds of tokens
        s.update(q=z[:, :hk * dk].unflatten(1, (hk, dk)), k=z[:, hk * dk:2 * hk * dk].unflatten(1, (hk, dk)),
                 v=z[:, 2 * hk * dk:].unflatten(1, (hv, dv)),
                 g=-torch.nn.functional.softplus(torch.randn((T, hv), generator=g, device=DEV) + heads),
                 beta=torch.sigmoid(torch.randn((T, hv), generator=g, device=DEV) * 1.5),
                 state=torch.randn((R, hv, dk, dv), generator=g, device=DEV) * 0.3)
        return s
    if case["op"] == "append":
        h, hk, D, page = case["heads"], case["kv_heads"], case["D"], case["page"]
        pages = sum((n + page - 1) // page + 1 for n, _ in lens)
        # a request's new positions lie in pages anywhere in the cache
        perm = torch.randperm(pages, generator=g, device=DEV)
        slot, position, at = [], [], 0
        for n, c in lens:
            p = torch.arange(c, c + n, device=DEV)
            at_page = p // page - c // page
            slot.append(perm[at + at_page] * page + p % page)
            position.append(p)
            at += (n + page - 1) // page + 1
        base = 1e6 if D >= 128 else 1e4
        half = case["rot"] // 2
        qkv = _normal(g, (T, h + 2 * hk, D), dt, 1.5)  # one projection's output
        s.update(q=qkv[:, :h], k=qkv[:, h:h + hk], v=qkv[:, h + hk:],
                 slot=torch.cat(slot).to(torch.int32), position=torch.cat(position).to(torch.int32),
                 inv_freq=(base ** (-torch.arange(half, device=DEV).double() / half)).float(),
                 q_weight=_normal(g, (D,), dt, 0.2) + 1 if case["norm"] else None,
                 k_weight=_normal(g, (D,), dt, 0.2) + 1 if case["norm"] else None,
                 k_cache=torch.zeros((pages, hk, page, D), dtype=dt, device=DEV),
                 v_cache=torch.zeros((pages, hk, D, page), dtype=dt, device=DEV))
        return s
    C, W = case["C"], case["W"]
    s.update(x=_normal(g, (T, C), dt), weight=_normal(g, (C, W), dt, W ** -0.5),
             state=_normal(g, (R, W - 1, C), dt))
    return s


def prepare(case, seed):
    s = _inputs(case, seed)
    if own:
        from bit_vector_lut_amd import vqmlp

        if case["op"] == "delta":
            s["plan"] = vqmlp.DeltaRule(case["k_heads"], case["v_heads"], case["Dk"], case["Dv"])
        elif case["op"] == "append":
            s["plan"] = vqmlp.PagedCache(s["k_cache"], s["v_cache"])
            s["rotary"] = vqmlp.Rotary(s["inv_freq"], interleaved=case["pairs"] == "next",
                                       q_weight=s["q_weight"], k_weight=s["k_weight"], eps=EPS)
        else:
            s["plan"] = vqmlp.ShortConv(s["weight"], unit_heads=case["unit"], unit_dim=case["unit_dim"], eps=EPS)
    return s


# ------------------------------------------------------------------ one pass


def run(s):
    return (_own if own else _plain)[s["op"]](s)


def _own_delta(s):
    y, state = s["plan"].forward(s["q"], s["k"], s["v"], s["g"], s["beta"], s["state"], s["cu_q"],
                                 ctx_len=s["ctx"], max_q=s["max_q"])
    return {"y": y, "state": state}


def _own_append(s):
    q = s["plan"].append(s["q"], s["k"], s["v"], s["position"], s["slot"], s["rotary"])
    return {"q": q, "k_cache": s["k_cache"], "v_cache": s["v_cache"]}


def _own_conv(s):
    y, state = s["plan"].forward(s["x"], s["state"], s["cu_q"], ctx_len=s["ctx"])
    return {"y": y, "state": state}


def _plain_delta(s):
    """Chunks of 64 tokens, requests of one length together."""
    hk, hv, dk, dv = s["k_heads"], s["v_heads"], s["Dk"], s["Dv"]
    y = torch.empty((s["q"].shape[0], hv, dv), dtype=s["q"].dtype, device=DEV)
    state = torch.empty_like(s["state"])
    groups = {}
    for r, n in enumerate(b - a for a, b in zip(s["starts"], s["starts"][1:])):
        groups.setdefault(n, []).append(r)
    for n, members in groups.items():
        rr = _ints(members).long()
        rows = s["cu_q"].long()[rr][:, None] + torch.arange(n, device=DEV)[None, :]
        S = torch.where((s["ctx"][rr] > 0)[:, None, None, None], s["state"][rr], 0.0)
        for c in range(0, n, 64):
            i = rows[:, c:c + 64]
            m = i.shape[1]
            rep = lambda x: (x[i].float().transpose(1, 2).repeat_interleave(hv // hk, 1))  # noqa: E731
            q, k, v = rep(s["q"]) / math.sqrt(dk), rep(s["k"]), s["v"][i].float().transpose(1, 2)
            beta = s["beta"][i].transpose(1, 2)[..., None]
            b = s["g"][i].double().cumsum(1).transpose(1, 2)
            eb = b.float().exp()[..., None]
            low = torch.ones((m, m), dtype=torch.bool, device=DEV).tril()
            d = torch.where(low, b[..., :, None] - b[..., None, :], -math.inf).float().exp()
            kt = k.transpose(2, 3).contiguous()
            # (1 - N)^-1 = (1 + N) (1 + N^2) (1 + N^4) .. for N = -A, whose power m vanishes
            N = -(torch.matmul(k, kt) * d * beta).tril(-1)
            u = beta * (v - eb * torch.matmul(k, S))
            u = u + torch.matmul(N, u)
            for _ in range(max(0, (m - 1).bit_length() - 1)):
                N = torch.matmul(N, N)
                u = u + torch.matmul(N, u)
            o = torch.matmul(torch.matmul(q, kt) * d, u) + eb * torch.matmul(q, S)
            tail = (b[..., -1:] - b).float().exp()
            S = S * b[..., -1].float().exp()[..., None, None] + torch.matmul(kt * tail[..., None, :], u)
            y[i.reshape(-1)] = o.transpose(1, 2).reshape(-1, hv, dv).to(y.dtype)
        state[rr] = S
    return {"y": y, "state": state}


def _plain_append(s):
    D, rot, page = s["D"], s["rot"], s["page"]
    half = rot // 2
    turns = s["position"].double()[:, None] * s["inv_freq"].double()[None]
    cos, sin = turns.cos().float()[:, None], turns.sin().float()[:, None]

    def turned(x, w):
        z = x.float()
        if w is not None:
            z = z * torch.rsqrt((z * z).mean(dim=-1, keepdim=True) + EPS) * w.float()
        a, b = (z[..., :half], z[..., half:rot]) if s["pairs"] == "half" else (z[..., 0:rot:2], z[..., 1:rot:2])
        a, b = a * cos - b * sin, b * cos + a * sin
        front = torch.cat([a, b], -1) if s["pairs"] == "half" else torch.stack([a, b], -1).flatten(-2)
        return torch.cat([front, z[..., rot:]], -1).to(x.dtype)

    slot = s["slot"].long()
    at, off = slot // page, slot % page
    s["k_cache"][at, :, off] = turned(s["k"], s["k_weight"])
    s["v_cache"][at, :, :, off] = s["v"]
    return {"q": turned(s["q"], s["q_weight"]), "k_cache": s["k_cache"], "v_cache": s["v_cache"]}


def _plain_conv(s):
    C, W, T, R = s["C"], s["W"], s["x"].shape[0], s["ctx"].shape[0]
    cu = s["cu_q"].long()
    t = torch.arange(T, device=DEV)
    r = torch.searchsorted(cu[1:], t, right=True)
    old = torch.where((s["ctx"] > 0)[:, None, None], s["state"], 0)
    # rows in front of a request's first are its state's last
    rows = torch.cat([s["x"], old.reshape(R * (W - 1), C)])
    z = torch.zeros((T, C), device=DEV)
    for w in range(W):
        at = t - (W - 1) + w
        src = torch.where(at >= cu[r], at, T + r * (W - 1) + (at - cu[r]) + W - 1)
        z += rows[src].float() * s["weight"][:, w].float()
    y = z / (1 + torch.exp(-z))
    n = s["unit"] * s["unit_dim"]
    if n:
        front = y[:, :n].unflatten(1, (s["unit"], s["unit_dim"]))
        front = front * torch.rsqrt((front * front).sum(dim=-1, keepdim=True) + EPS)
        y = torch.cat([front.flatten(1), y[:, n:]], 1)
    at = cu[1:, None] - (W - 1) + torch.arange(W - 1, device=DEV)[None]
    first = cu[:-1, None]
    src = torch.where(at >= first, at, T + torch.arange(R, device=DEV)[:, None] * (W - 1) + at - first + W - 1)
    return {"y": y.to(s["x"].dtype), "state": rows[src]}


_own = dict(delta=_own_delta, append=_own_append, conv=_own_conv)
_plain = dict(delta=_plain_delta, append=_plain_append, conv=_plain_conv)


# ------------------------------------------------------------------ the definitions in 64 bits


def exact(case, seed):
    s = _inputs(case, seed)
    starts = s["starts"]
    if case["op"] == "delta":
        # A head at a time over blocks of 128 tokens: the tokens' updates solve a triangular system.
        hk, hv, dk = case["k_heads"], case["v_heads"], case["Dk"]
        y = torch.zeros(s["v"].shape, dtype=torch.float64, device=DEV)
        state = torch.zeros(s["state"].shape, dtype=torch.float64, device=DEV)
        heads = torch.arange(hv, device=DEV) // (hv // hk)
        for r, (n, old) in enumerate(_lens(case)):
            S = s["state"][r].double() * (1.0 if old else 0.0)
            for c in range(0, n, 128):
                i = slice(starts[r] + c, starts[r] + min(n, c + 128))
                q = s["q"][i].double()[:, heads].permute(1, 0, 2).contiguous()
                k = s["k"][i].double()[:, heads].permute(1, 0, 2).contiguous()
                v, beta = s["v"][i].double().permute(1, 0, 2), s["beta"][i].double().T
                b = s["g"][i].double().T.cumsum(1)
                d = torch.exp((b[:, :, None] - b[:, None, :]).clamp(max=0.0)).tril()
                kt = k.transpose(1, 2).contiguous()
                eye = torch.eye(b.shape[1], dtype=torch.float64, device=DEV)
                system = eye + beta[:, :, None] * (torch.bmm(k, kt) * d).tril(-1)
                rhs = beta[..., None] * (v - torch.exp(b)[..., None] * torch.bmm(k, S))
                u = torch.linalg.solve_triangular(system, rhs, upper=False, unitriangular=True)
                o = torch.exp(b)[..., None] * torch.bmm(q, S) + torch.bmm(torch.bmm(q, kt) * d, u)
                y[i] = (o / math.sqrt(dk)).permute(1, 0, 2)
                S = torch.exp(b[:, -1])[:, None, None] * S + torch.bmm(kt, torch.exp(b[:, -1:] - b)[..., None] * u)
            state[r] = S
        return {"y": y, "state": state}
    if case["op"] == "append":
        D, rot, page = case["D"], case["rot"], case["page"]
        # a rotation is a product of complex numbers
        turn = torch.polar(torch.ones((), dtype=torch.float64, device=DEV),
                           s["position"].double()[:, None] * s["inv_freq"].double())
        p = torch.arange(rot // 2, device=DEV)
        one, two = (p, p + rot // 2) if case["pairs"] == "half" else (2 * p, 2 * p + 1)

        def turned(x, w):
            z = x.double()
            if w is not None:
                z = z / (z.pow(2).sum(2, keepdim=True) / D + EPS).sqrt() * w.double()
            z = z.clone()
            c = torch.complex(z[:, :, one], z[:, :, two]) * turn[:, None]
            z[:, :, one], z[:, :, two] = c.real, c.imag
            return z

        kc = torch.zeros(s["k_cache"].shape, dtype=torch.float64, device=DEV)
        vc = torch.zeros(s["v_cache"].shape, dtype=torch.float64, device=DEV)
        pg, off = torch.div(s["slot"].long(), page, rounding_mode="floor"), s["slot"].long() % page
        kc[pg, :, off] = turned(s["k"], s["k_weight"])
        vc[pg, :, :, off] = s["v"].double()
        return {"q": turned(s["q"], s["q_weight"]), "k_cache": kc, "v_cache": vc}
    C, W, n = case["C"], case["W"], case["unit"] * case["unit_dim"]
    y = torch.zeros(s["x"].shape, dtype=torch.float64, device=DEV)
    state = torch.zeros(s["state"].shape, dtype=torch.float64, device=DEV)
    w = s["weight"].double()
    for r, (m, old) in enumerate(_lens(case)):
        seq = torch.cat([s["state"][r].double() * (1.0 if old else 0.0), s["x"][starts[r]:starts[r + 1]].double()])
        z = (seq.unfold(0, W, 1) * w[None]).sum(-1)
        z = z * torch.special.expit(z)
        if n:
            head = z[:, :n].reshape(m, case["unit"], -1)
            z[:, :n] = (head / (head.pow(2).sum(2, keepdim=True) + EPS).sqrt()).reshape(m, n)
        y[starts[r]:starts[r + 1]] = z
        state[r] = seq[seq.shape[0] - (W - 1):]
    return {"y": y, "state": state}
