"""The operators around the quantized MLP: what is measured.

Five operators of a serving step over requests packed one after another (``cu_q`` holds their first
rows): the norms and the residual between two blocks, the block tables and slot maps of a paged
key/value cache, storing new keys and values into it, attention of the new tokens over it, and
linear attention with a decay per head and token.  ``run`` computes them in plain torch operations
where ``own`` is false and through ``bit_vector_lut_amd.vqmlp`` where it is true.
"""
import math

import torch

own = False

DEV = "cuda"
DTYPES = {"f16": torch.float16, "bf16": torch.bfloat16, "f32": torch.float32}


# ------------------------------------------------------------------ cases


def _text(pairs):
    return ",".join("%d:%d" % tuple(p) for p in pairs)


def _lens(case):
    """Per request: (new tokens, keys with them) for attention, (new tokens, has a state) for linear."""
    return [tuple(int(x) for x in p.split(":")) for p in case["lens"].split(",")]


def listed():
    return [
        # one verify step's eight rows between two blocks of a 5120-wide model
        dict(name="norm_t8", op="norm", dtype="f16", res="f16", T=8, H=5120, kind="rms", post=True,
             gate="none", bias=False, scale=1.0),
        # a large prompt batch with an FP32 residual, per-token gates and mean/variance norms
        dict(name="norm_t8192", op="norm", dtype="bf16", res="f32", T=8192, H=5120, kind="layer",
             post=True, gate="token", bias=True, scale=0.5),
        # four requests, each verifying eight drafted tokens: latency alone
        dict(name="pages_r4", op="pages", R=4, q_lo=8, q_hi=8, ctx_hi=65464, page=16),
        # a crowded step: 512 requests, most with few tokens, some with prompts
        dict(name="pages_r512", op="pages", R=512, q_lo=1, q_hi=257, ctx_hi=20000, page=16),
        # one new token for each of 64 requests
        dict(name="store_t64", op="store", dtype="f16", T=64, kv_heads=8, D=128, page=16, pages=1024),
        # the keys and values of a long packed prompt
        dict(name="store_t8192", op="store", dtype="bf16", T=8192, kv_heads=4, D=256, page=64,
             pages=256),
        # one request verifying eight drafted tokens at the end of a 64K context
        dict(name="attn_verify_64k", op="attn", dtype="f16", lens="8:65472", heads=24, kv_heads=4,
             D=256, page=64, window=0),
        # 64 requests of ragged lengths, one token each
        dict(name="attn_decode_r64", op="attn", dtype="bf16",
             lens=_text([1, 61 + 257 * i] for i in range(64)), heads=40, kv_heads=8, D=128, page=16,
             window=0),
        # a 512-row prompt chunk in a long context
        dict(name="attn_chunk_512", op="attn", dtype="f16", lens="512:33001", heads=40,
             kv_heads=8, D=128, page=16, window=0),
        # one request's eight drafted tokens through a recurrent layer
        dict(name="linear_t8", op="linear", dtype="f16", lens="8:1", k_heads=16, v_heads=48,
             Dk=128, Dv=128),
        # one token for each of 64 requests, one of them new
        dict(name="linear_r64", op="linear", dtype="bf16", lens=_text([1, int(i != 5)] for i in range(64)),
             k_heads=16, v_heads=48, Dk=128, Dv=128),
        # three packed prompts, two of them continued
        dict(name="linear_prompts", op="linear", dtype="f16", lens="5003:0,1021:1,2049:1",
             k_heads=16, v_heads=48, Dk=128, Dv=128),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["norm", "pages", "store", "attn", "attn", "linear", "linear"])
    dt = rng.choice(["f16", "bf16"])
    if op == "norm":
        H = _log_int(rng, 64, 8192)
        if rng.random() < 0.6:
            H = (H + 7) // 8 * 8
        return dict(op=op, dtype=dt, res=rng.choice([dt, "f32"]), T=_log_int(rng, 1, 4096), H=H,
                    kind=rng.choice(["rms", "layer"]), post=rng.random() < 0.5,
                    gate=rng.choice(["none", "channel", "token"]), bias=rng.random() < 0.5,
                    scale=rng.choice([1.0, 0.25, 1.7]))
    if op == "pages":
        q_lo = rng.choice([0, 1, 8])
        return dict(op=op, R=_log_int(rng, 1, 512), q_lo=q_lo, q_hi=q_lo + _log_int(rng, 1, 256),
                    ctx_hi=_log_int(rng, 16, 30000), page=rng.choice([16, 32, 64, 128]))
    if op == "store":
        page = rng.choice([16, 32, 64, 128])
        T = _log_int(rng, 1, 8192)
        return dict(op=op, dtype=dt, T=T, kv_heads=rng.choice([1, 2, 4]), D=rng.choice([64, 80, 128, 256]),
                    page=page, pages=(T + page - 1) // page + rng.randrange(1, 64))
    if op == "attn":
        D = rng.choice([64, 96, 128, 256])
        kv_heads = rng.choice([1, 2, 4, 8]) if D <= 128 else rng.choice([1, 2, 4])
        heads = kv_heads * rng.choice([1, 2, 3, 5, 8])
        if rng.random() < 0.6:  # single tokens and drafts
            R = _log_int(rng, 1, 64)
            top = max(64, min(65000, 400000 // R))
            lens = [[rng.randint(1, 8), _log_int(rng, 9, top)] for _ in range(R)]
        else:
            R = rng.randint(1, 4)
            lens = []
            for _ in range(R):
                n = _log_int(rng, 16, 512)
                lens.append([n, n + _log_int(rng, 1, 24000 // R)])
        return dict(op=op, dtype=dt, lens=_text(lens), heads=heads, kv_heads=kv_heads, D=D,
                    page=rng.choice([16, 32, 64, 128]), window=rng.choice([0, 0, 0, 1000]))
    k_heads = rng.choice([1, 2, 4, 8, 16])
    v_heads = k_heads * rng.choice([1, 2, 3])
    D = rng.choice([64, 96, 128])
    if rng.random() < 0.5:
        lens = [[rng.randint(1, 8), rng.randrange(2)] for _ in range(_log_int(rng, 1, 64))]
    else:
        R = rng.randint(1, 5)
        lens = [[_log_int(rng, 20, 8000 // R), rng.randrange(2)] for _ in range(R)]
    return dict(op=op, dtype=dt, lens=_text(lens), k_heads=k_heads, v_heads=v_heads, Dk=D,
                Dv=rng.choice([D, 128]))


def work(case):
    op = case["op"]
    if op == "norm":
        n, e = case["T"] * case["H"], 4 if case["res"] == "f32" else 2
        g = n * 2 if case["gate"] == "token" else 0
        return {"bytes": n * (2 + 2 * e + 2) + g, "flops": 16 * n}
    if op == "pages":
        T = case["R"] * case["q_hi"]  # the slot map's rows, padding among them
        return {"bytes": 16 * case["R"] + 8 * T + 8 * (T // case["page"] + case["R"]), "flops": 4 * T}
    if op == "store":
        return {"bytes": case["T"] * (8 * case["kv_heads"] * case["D"] + 4), "flops": 0}
    if op == "attn":
        h, hk, D, w = case["heads"], case["kv_heads"], case["D"], case["window"]
        pairs = keys = T = 0
        for n, kv in _lens(case):
            T += n
            first = max(0, kv - n - w + 1) if w else 0
            keys += kv - first
            for i in range(n):
                p = kv - n + i + 1
                pairs += min(p, w) if w else p
        return {"bytes": 4 * keys * hk * D + 4 * T * h * D + 4 * T * h, "flops": 4 * pairs * h * D}
    T, R = sum(n for n, _ in _lens(case)), len(_lens(case))
    old = sum(c > 0 for _, c in _lens(case))
    hk, hv, dk, dv = case["k_heads"], case["v_heads"], case["Dk"], case["Dv"]
    return {"bytes": T * (4 * hk * dk + 4 * hv * dv + 4 * hv) + 4 * (R + old) * hv * dk * dv,
            "flops": 5 * T * hv * dk * dv}


# ------------------------------------------------------------------ inputs


def _gen(seed):
    return torch.Generator(device=DEV).manual_seed(int(seed) % (1 << 62))


def _normal(g, shape, dtype, std=1.0):
    return (torch.randn(shape, generator=g, device=DEV) * std).to(dtype)


def _ints(values):
    return torch.tensor(values, dtype=torch.int32, device=DEV)


def _starts(lens):
    at = [0]
    for n in lens:
        at.append(at[-1] + n)
    return at


def _inputs(case, seed):
    """The state without the library's handles: also what ``exact`` reads."""
    g, op = _gen(seed), case["op"]
    s = dict(case)
    if "lens" in s:
        s["pairs"] = _lens(case)
    if op == "norm":
        dt, T, H = DTYPES[case["dtype"]], case["T"], case["H"]
        s.update(y=_normal(g, (T, H), dt, 1.5), res=_normal(g, (T, H), DTYPES[case["res"]], 2.0),
                 pre_w=_normal(g, (H,), dt, 0.2) + 1, pre_b=None, post_w=None, post_b=None, gates=None)
        if case["post"]:
            s["post_w"] = _normal(g, (H,), dt, 0.2) + 1
        if case["bias"]:
            s["pre_b"] = _normal(g, (H,), dt, 0.1)
            s["post_b"] = _normal(g, (H,), dt, 0.1) if case["post"] else None
        if case["gate"] != "none":
            s["gates"] = _normal(g, (H,) if case["gate"] == "channel" else (T, H), dt, 0.5)
        return s
    if op == "pages":
        R, page = case["R"], case["page"]
        ctx = torch.randint(0, case["ctx_hi"] + 1, (R,), generator=g, device=DEV, dtype=torch.int32)
        q = torch.randint(case["q_lo"], case["q_hi"] + 1, (R,), generator=g, device=DEV, dtype=torch.int32)
        width = (case["ctx_hi"] + case["q_hi"] + page - 1) // page
        pages = R * width
        # pages in use stand in the requests' rows, the others on the free list, in any order
        perm = torch.randperm(pages, generator=g, device=DEV).to(torch.int32)
        table = perm.view(R, width).clone()
        held = (ctx + page - 1) // page
        unused = torch.arange(width, device=DEV)[None, :] >= held[:, None]
        free = table[unused]
        free = free[torch.randperm(free.numel(), generator=g, device=DEV)].contiguous()
        table[unused] = -1
        s.update(ctx=ctx, q=q, table=table, free=free, pages=pages, cap=R * case["q_hi"])
        return s
    if op == "store":
        dt, T, h, D = DTYPES[case["dtype"]], case["T"], case["kv_heads"], case["D"]
        n, page = case["pages"], case["page"]
        s.update(k=_normal(g, (T, h, D), dt), v=_normal(g, (T, h, D), dt),
                 slot=torch.randperm(n * page, generator=g, device=DEV)[:T].sort().values.to(torch.int32),
                 k_cache=torch.zeros((n, h, page, D), dtype=dt, device=DEV),
                 v_cache=torch.zeros((n, h, D, page), dtype=dt, device=DEV))
        return s
    if op == "attn":
        dt, h, hk, D, page = (DTYPES[case["dtype"]], case["heads"], case["kv_heads"], case["D"],
                              case["page"])
        R = len(_lens(case))
        need = [(kv + page - 1) // page for _, kv in _lens(case)]
        n = sum(need) + 3
        perm = torch.randperm(n, generator=g, device=DEV).to(torch.int32)
        table = torch.full((R, max(need) + 1), -1, dtype=torch.int32, device=DEV)
        at = 0
        for r, m in enumerate(need):
            table[r, :m] = perm[at:at + m]
            at += m
        starts = _starts([q for q, _ in _lens(case)])
        s.update(q=_normal(g, (starts[-1], h, D), dt, 1.5),
                 k_cache=torch.randn((n, hk, page, D), generator=g, device=DEV, dtype=dt),
                 v_cache=torch.randn((n, hk, D, page), generator=g, device=DEV, dtype=dt),
                 table=table, starts=starts, cu_q=_ints(starts),
                 kv_len=_ints([kv for _, kv in _lens(case)]), max_kv=max(kv for _, kv in _lens(case)))
        return s
    dt, hk, hv, dk, dv = (DTYPES[case["dtype"]], case["k_heads"], case["v_heads"], case["Dk"], case["Dv"])
    starts = _starts([n for n, _ in _lens(case)])
    T, R = starts[-1], len(_lens(case))
    unit = lambda x: (x / x.norm(dim=-1, keepdim=True)).to(dt)  # noqa: E731
    heads = torch.rand((hv,), generator=g, device=DEV) * 6 - 6.5  # decays of one to hundreds of tokens
    s.update(q=unit(torch.randn((T, hk, dk), generator=g, device=DEV)),
             k=unit(torch.randn((T, hk, dk), generator=g, device=DEV)),
             v=_normal(g, (T, hv, dv), dt),
             g=-torch.nn.functional.softplus(torch.randn((T, hv), generator=g, device=DEV) + heads),
             state=torch.randn((R, hv, dk, dv), generator=g, device=DEV) * 0.3,
             starts=starts, cu_q=_ints(starts), ctx=_ints([c for _, c in _lens(case)]),
             max_q=max(n for n, _ in _lens(case)))
    return s


def prepare(case, seed):
    s = _inputs(case, seed)
    if own:
        from bit_vector_lut_amd import vqmlp

        if case["op"] == "norm":
            s["plan"] = vqmlp.BlockNorm(
                s["pre_w"], s["pre_b"], post_weight=s["post_w"], post_bias=s["post_b"],
                kind=case["kind"], eps=1e-6, residual_scale=case["scale"])
        elif case["op"] == "pages":
            s["plan"] = vqmlp.PagePlanner(s["table"], s["free"], case["page"], s["pages"], s["cap"])
        elif case["op"] in ("store", "attn"):
            s["plan"] = vqmlp.PagedCache(s["k_cache"], s["v_cache"])
        else:
            s["plan"] = vqmlp.LinearAttention(case["k_heads"], case["v_heads"], case["Dk"], case["Dv"])
    return s


# ------------------------------------------------------------------ one pass


def run(s):
    return (_own if own else _plain)[s["op"]](s)


def _own_norm(s):
    r, x = s["plan"].forward(s["y"], s["res"], gate=s["gates"])
    return {"residual": r, "x": x}


def _own_pages(s):
    p = s["plan"].forward(s["ctx"], s["q"])
    return {"table": s["table"], "seq_len": p.seq_len, "cu_q": p.cu_q, "slot": p.slot,
            "position": p.position, "status": p.status}


def _own_store(s):
    s["plan"].store(s["k"], s["v"], s["slot"])
    return {"k_cache": s["k_cache"], "v_cache": s["v_cache"]}


def _own_attn(s):
    y, lse = s["plan"].attention(s["q"], s["table"], s["cu_q"], s["kv_len"], window=s["window"],
                                 max_kv=s["max_kv"], with_lse=True)
    return {"y": y, "lse": lse}


def _own_linear(s):
    y, state = s["plan"].forward(s["q"], s["k"], s["v"], s["g"], s["state"], s["cu_q"],
                                 ctx_len=s["ctx"], max_q=s["max_q"])
    return {"y": y, "state": state}


def _norm(x, w, b, kind, eps):
    if kind == "layer":
        x = x - x.mean(dim=-1, keepdim=True)
    x = x * torch.rsqrt((x * x).mean(dim=-1, keepdim=True) + eps) * w.float()
    return x if b is None else x + b.float()


def _plain_norm(s):
    u = s["y"].float()
    if s["post_w"] is not None:
        u = _norm(u, s["post_w"], s["post_b"], s["kind"], 1e-6)
    if s["gates"] is not None:
        u = u * s["gates"].float()
    r = s["res"].float() + s["scale"] * u
    x = _norm(r, s["pre_w"], s["pre_b"], s["kind"], 1e-6)
    return {"residual": r.to(s["res"].dtype), "x": x.to(s["y"].dtype)}


def _plain_pages(s):
    page, table, cap = s["page"], s["table"], s["cap"]
    R = s["R"]
    ctx, q = s["ctx"].long(), s["q"].long()
    seq = ctx + q
    held, need = (ctx + page - 1) // page, (seq + page - 1) // page
    new = need - held
    first_new = new.cumsum(0) - new
    cols = torch.arange(table.shape[1], device=DEV)[None, :]
    takes = (cols >= held[:, None]) & (cols < need[:, None])
    at = (first_new[:, None] + cols - held[:, None]).clamp(0, max(0, s["free"].numel() - 1))
    table.copy_(torch.where(takes, s["free"][at], table))
    cu = torch.zeros(R + 1, dtype=torch.int64, device=DEV)
    cu[1:] = q.cumsum(0)
    t = torch.arange(cap, device=DEV)
    r = torch.searchsorted(cu[1:], t, right=True).clamp(max=R - 1)
    real = t < cu[R]
    pos = torch.where(real, ctx[r] + t - cu[r], 0)
    slot = table[r, pos // page].long() * page + pos % page
    zero = torch.zeros((), dtype=torch.int64, device=DEV)
    return {"table": table, "seq_len": seq.int(), "cu_q": cu.int(),
            "slot": torch.where(real, slot, -1).int(), "position": torch.where(real, pos, -1).int(),
            "status": torch.stack([zero, cu[R], new.sum(), zero]).int()}


def _plain_store(s):
    slot = s["slot"].long()
    page, off = slot // s["page"], slot % s["page"]
    s["k_cache"][page, :, off] = s["k"]
    s["v_cache"][page, :, :, off] = s["v"]
    return {"k_cache": s["k_cache"], "v_cache": s["v_cache"]}


def _plain_attn(s):
    h, hk, D, page, w = s["heads"], s["kv_heads"], s["D"], s["page"], s["window"]
    y = torch.empty_like(s["q"])
    lse = torch.empty((s["q"].shape[0], h), device=DEV)
    for r, (n, kv) in enumerate(s["pairs"]):
        rows = slice(s["starts"][r], s["starts"][r + 1])
        pages = s["table"][r, :(kv + page - 1) // page].long()
        k = s["k_cache"][pages].transpose(0, 1).reshape(hk, -1, D)[:, :kv].float()
        v = s["v_cache"][pages].permute(1, 0, 3, 2).reshape(hk, -1, D)[:, :kv].float()
        q = s["q"][rows].float().view(n, hk, h // hk, D).transpose(0, 1).reshape(hk, -1, D)
        p = torch.matmul(q, k.transpose(1, 2).contiguous()).view(hk, n, h // hk, kv) / math.sqrt(D)
        at = torch.arange(kv - n, kv, device=DEV)[:, None]
        j = torch.arange(kv, device=DEV)[None, :]
        out = j > at
        if w:
            out = out | (j <= at - w)
        p.masked_fill_(out[None, :, None, :], -math.inf)
        m = p.amax(dim=-1, keepdim=True)
        p = torch.exp(p.sub_(m))
        l = p.sum(dim=-1, keepdim=True)
        o = torch.matmul(p.view(hk, -1, kv), v).view(hk, n, h // hk, D) / l
        y[rows] = o.transpose(0, 1).reshape(n, h, D).to(y.dtype)
        lse[rows] = (m + l.log()).view(hk, n, h // hk).transpose(0, 1).reshape(n, h)
    return {"y": y, "lse": lse}


def _plain_linear(s):
    hk, hv, dk, dv = s["k_heads"], s["v_heads"], s["Dk"], s["Dv"]
    y = torch.empty((s["q"].shape[0], hv, dv), dtype=s["q"].dtype, device=DEV)
    state = torch.empty_like(s["state"])
    groups = {}  # requests of one length go through together
    for r, (n, _) in enumerate(s["pairs"]):
        groups.setdefault(n, []).append(r)
    for n, members in groups.items():
        rr = _ints(members).long()
        rows = s["cu_q"].long()[rr][:, None] + torch.arange(n, device=DEV)[None, :]
        S = torch.where((s["ctx"][rr] > 0)[:, None, None, None], s["state"][rr], 0.0)
        for c in range(0, n, 64):
            i = rows[:, c:c + 64]
            C = i.shape[1]
            rep = lambda x: (x[i].float().transpose(1, 2).repeat_interleave(hv // hk, 1))  # noqa: E731
            q, k, v = rep(s["q"]) / math.sqrt(dk), rep(s["k"]), s["v"][i].float().transpose(1, 2)
            b = s["g"][i].double().cumsum(1).transpose(1, 2)
            a = torch.matmul(q, k.transpose(2, 3).contiguous())
            low = torch.ones((C, C), dtype=torch.bool, device=DEV).tril()
            d = torch.where(low, (b[..., :, None] - b[..., None, :]), -math.inf).float().exp()
            o = torch.matmul(a * d, v) + torch.matmul(q * b.float().exp()[..., None], S)
            tail = (b[..., -1:] - b).float().exp()
            kt = (k * tail[..., None]).transpose(2, 3).contiguous()
            S = S * b[..., -1].float().exp()[..., None, None] + torch.matmul(kt, v)
            y[i.reshape(-1)] = o.transpose(1, 2).reshape(-1, hv, dv).to(y.dtype)
        state[rr] = S
    return {"y": y, "state": state}


_own = dict(norm=_own_norm, pages=_own_pages, store=_own_store, attn=_own_attn, linear=_own_linear)
_plain = dict(norm=_plain_norm, pages=_plain_pages, store=_plain_store, attn=_plain_attn,
              linear=_plain_linear)


# ------------------------------------------------------------------ the definitions in 64 bits


def exact(case, seed):
    if case["op"] in ("pages", "store"):
        return None
    s = _inputs(case, seed)
    if case["op"] == "norm":
        d = {k: (v.double() if torch.is_tensor(v) else v) for k, v in s.items()}

        def normed(x, w, b):
            mu = x.sum(1) / case["H"] if case["kind"] == "layer" else torch.zeros_like(x[:, 0])
            var = ((x - mu[:, None]) ** 2).sum(1) / case["H"]
            z = (x - mu[:, None]) / (var + 1e-6).sqrt()[:, None] * w[None]
            return z if b is None else z + b[None]

        u = normed(d["y"], d["post_w"], d["post_b"]) if case["post"] else d["y"]
        u = u if d["gates"] is None else u * d["gates"]
        r = d["res"] + case["scale"] * u
        return {"residual": r, "x": normed(r, d["pre_w"], d["pre_b"])}
    if case["op"] == "attn":
        h, hk, D, page = case["heads"], case["kv_heads"], case["D"], case["page"]
        y = torch.zeros(s["q"].shape, dtype=torch.float64, device=DEV)
        lse = torch.zeros((y.shape[0], h), dtype=torch.float64, device=DEV)
        for r, (n, kv) in enumerate(_lens(case)):
            pos = torch.arange(kv, device=DEV)
            pg, off = s["table"][r].long()[pos // page], pos % page
            i = pos[kv - n:, None]
            see = pos[None] <= i
            if case["window"]:
                see &= pos[None] > i - case["window"]
            for a in range(hk):
                k, v = s["k_cache"][pg, a, off].double(), s["v_cache"][pg, a, :, off].double()
                for b in range(a * (h // hk), (a + 1) * (h // hk)):
                    z = s["q"][s["starts"][r]:s["starts"][r + 1], b].double() @ k.T / math.sqrt(D)
                    z = torch.where(see, z, -math.inf)
                    c = torch.logsumexp(z, 1)
                    lse[s["starts"][r]:s["starts"][r + 1], b] = c
                    y[s["starts"][r]:s["starts"][r + 1], b] = torch.exp(z - c[:, None]) @ v
        return {"y": y, "lse": lse}
    # the recurrence unrolled over blocks of 256 tokens, a head at a time
    hk, hv, dk = case["k_heads"], case["v_heads"], case["Dk"]
    y = torch.zeros(s["v"].shape, dtype=torch.float64, device=DEV)
    state = torch.zeros(s["state"].shape, dtype=torch.float64, device=DEV)
    for r, (n, old) in enumerate(_lens(case)):
        t0 = s["starts"][r]
        S = s["state"][r].double() * (1.0 if old else 0.0)
        heads = torch.arange(hv, device=DEV) // (hv // hk)
        for c in range(0, n, 256):
            i = slice(t0 + c, t0 + min(n, c + 256))
            q, k = s["q"][i].double()[:, heads].permute(1, 0, 2), s["k"][i].double()[:, heads].permute(1, 0, 2)
            v, b = s["v"][i].double().permute(1, 0, 2), s["g"][i].double().T.cumsum(1)
            D = torch.exp((b[:, :, None] - b[:, None, :]).clamp(max=0.0)).tril()
            o = torch.bmm(torch.bmm(q, k.transpose(1, 2).contiguous()) * D, v)
            o = o + torch.exp(b)[..., None] * torch.bmm(q, S)
            y[i] = (o / math.sqrt(dk)).permute(1, 0, 2)
            left = torch.exp(b[:, -1:] - b)[..., None] * v
            S = torch.exp(b[:, -1])[:, None, None] * S + torch.bmm(k.transpose(1, 2).contiguous(), left)
        state[r] = S
    return {"y": y, "state": state}
