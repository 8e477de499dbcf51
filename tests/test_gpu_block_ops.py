"""GPU: the operators around the MLP against plain 64-bit forms on the same inputs.

Tolerances.  u = eps / 2 of the 16-bit type is one rounding, w = 2^-24 one of FP32.
  norm       one rounding of the output, and FP32 sums: 40 w of the terms' absolute values.
  attention  the output's rounding, one of each probability (u times the softmax mean of |v|), and
             of the scores' FP32 sums: (D + 8) w of sum |q_i k_i| scale, which moves a probability by
             that factor up or down (so twice over: numerator and sum).
  linear     the same through the recurrence of absolute values (z = the output with |q|, |k|, |v|):
             score and state operands each rounded once to 16 bits, so 2 u z, and FP32 terms; the
             state is FP32 throughout: its bound counts FP32 roundings only.
"""
import math

import numpy as np
import pytest

pytestmark = pytest.mark.gpu

W = 2.0 ** -24


@pytest.fixture(scope="module")
def torch_dev():
    import torch

    assert torch.cuda.is_available(), "GPU tests need a GPU"
    return torch


@pytest.fixture(scope="module")
def vq(torch_dev):
    from bit_vector_lut_amd import vqmlp

    vqmlp.lib()
    return vqmlp


def _t(torch, name):
    return {"f16": torch.float16, "bf16": torch.bfloat16, "f32": torch.float32}[name]


def _u(torch, dt):
    return torch.finfo(dt).eps / 2


def _randn(torch, shape, dt, seed, std=1.0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(shape, generator=g) * std).to(dt)


def _close(torch, got, ref, tol, name):
    got = got.double().cpu()
    assert got.shape == ref.shape, (got.shape, ref.shape)
    same = (got == ref) | (got.isnan() & ref.isnan())
    over = ((got - ref).abs() / tol.clamp(min=1e-30)).masked_fill(same, 0.0)
    worst = over.max().item() if over.numel() else 0.0
    print("%s: worst error %.3f of its bound" % (name, worst), flush=True)
    assert not over.isnan().any(), name
    assert worst <= 1.0, (name, worst, over.argmax().item())


# ------------------------------------------------------------------ norm


def _norm64(x, w, b, kind, eps, off):
    """Value and bound on its FP32 error."""
    mu = x.mean(1, keepdim=True) if kind == "layer" else 0.0
    z = x - mu
    rs = 1 / ((z * z).mean(1, keepdim=True) + eps).sqrt()
    y = z * rs * (w + off)
    scale = (x.abs() + (mu.abs() if kind == "layer" else 0.0)) * rs * (w + off).abs()
    if b is not None:
        y, scale = y + b, scale + b.abs()
    return y, 40 * W * scale


NORM_CASES = [
    # dtype, res, T, H, kind, post, gate, bias, offset
    ("f16", "f16", 1, 8, "rms", True, None, False, 0.0),
    ("bf16", "f32", 3, 1, "rms", False, None, False, 0.0),
    ("f16", "f32", 5, 37, "layer", True, "token", True, 1.0),
    ("bf16", "bf16", 2, 512, "rms", True, "channel", True, 0.0),
    ("f16", "f32", 7, 520, "layer", False, "token", True, 0.0),
    ("bf16", "f32", 4, 2056, "rms", True, None, False, 1.0),
    ("f16", "f16", 9, 5120, "layer", True, "channel", True, 0.0),
    ("bf16", "bf16", 3, 8184, "rms", False, None, True, 0.0),
    ("f16", "f32", 2, 16384, "layer", True, "token", False, 0.0),
    ("f16", "f16", 2, 16392, "rms", True, None, False, 0.0),
    ("bf16", "f32", 300, 1023, "layer", True, "token", True, 0.0),
]


@pytest.mark.parametrize("dtype,res,T,H,kind,post,gate,bias,off", NORM_CASES)
def test_block_norm(vq, torch_dev, dtype, res, T, H, kind, post, gate, bias, off):
    torch = torch_dev
    dt, rt = _t(torch, dtype), _t(torch, res)
    y, r = _randn(torch, (T, H), dt, 1, 2.0) + 3, _randn(torch, (T, H), rt, 2, 3.0)
    ws = [_randn(torch, (H,), dt, 3 + i, 0.3) for i in range(4)]
    gates = None if gate is None else _randn(torch, (H,) if gate == "channel" else (T, H), dt, 9)
    cu = lambda t: None if t is None else t.cuda()  # noqa: E731
    op = vq.BlockNorm(cu(ws[0]), cu(ws[1]) if bias else None, post_weight=cu(ws[2]) if post else None,
                      post_bias=cu(ws[3]) if bias and post else None, kind=kind, eps=1e-5,
                      residual_scale=0.75, weight_offset=off)
    print("norm", dtype, res, T, H, kind, flush=True)
    r2, x = op.forward(cu(y), cu(r), cu(gates))
    d = lambda t: t.double()  # noqa: E731
    u, ue = d(y), torch.zeros(T, H, dtype=torch.float64)
    if post:
        u, ue = _norm64(u, d(ws[2]), d(ws[3]) if bias else None, kind, 1e-5, off)
    if gates is not None:
        u, ue = u * d(gates), ue * d(gates).abs() + W * (u * d(gates)).abs()
    ref = d(r) + 0.75 * u
    err = 0.75 * ue + 2 * W * (d(r).abs() + (0.75 * u).abs())
    half = _u(torch, rt)
    _close(torch, r2, ref, err + half * ref.abs() + 2.0 ** -25, "r")
    refx, ex = _norm64(ref, d(ws[0]), d(ws[1]) if bias else None, kind, 1e-5, off)
    # an error of r moves x by its own share and through the spread
    rs = 1 / ((ref - (ref.mean(1, keepdim=True) if kind == "layer" else 0)).square().mean(1, keepdim=True)
              + 1e-5).sqrt()
    slope = rs * (d(ws[0]) + off).abs()
    ex = ex + slope * (err + err.mean(1, keepdim=True)) + refx.abs() * rs * err.square().mean(1, keepdim=True).sqrt()
    _close(torch, x, refx, 2 * ex + _u(torch, dt) * refx.abs() + 2.0 ** -25, "x")


@pytest.mark.parametrize("H,pad", [(64, 8), (64, 3), (1000, 24)])
def test_block_norm_strides_in_place_and_parts(vq, torch_dev, H, pad):
    """Row strides, r over res and x over y, one-sided calls: all give the plain call's values."""
    torch = torch_dev
    T, dt = 5, torch.float16
    w, pw = _randn(torch, (H,), dt, 1).cuda(), _randn(torch, (H,), dt, 2).cuda()
    y, r = _randn(torch, (T, H), dt, 3).cuda(), _randn(torch, (T, H), dt, 4).cuda()
    op = vq.BlockNorm(w, post_weight=pw)
    r2, x = op.forward(y, r)
    wide = lambda t: torch.cat([t, torch.full((T, pad), 7.0, dtype=dt, device="cuda")], 1)  # noqa: E731
    yw, rw = wide(y), wide(r)
    ro, xo = op.forward(yw[:, :H], rw[:, :H], residual_out=rw[:, :H], out=yw[:, :H])
    # the element-wise kernel sums in another order than the vector kernel: one step apart at most
    for a, b in ((ro, r2), (xo, x)):
        assert ((a.double() - b.double()).abs() <= 2 * torch.finfo(dt).eps * b.double().abs() + 2.0 ** -24).all()
    assert (yw[:, H:] == 7).all() and (rw[:, H:] == 7).all()
    # only the sum; only the norm of the residual; no residual
    s, none = vq.BlockNorm(post_weight=pw).forward(y, r)
    assert none is None and torch.equal(s, r2)
    same, xr = vq.BlockNorm(w).forward(None, r)
    assert torch.equal(same, r)
    y2, xy = vq.BlockNorm(w).forward(r)
    assert torch.equal(y2, r) and torch.equal(xy, xr)


def test_block_norm_zero_and_infinite_rows(vq, torch_dev):
    torch = torch_dev
    y = torch.zeros(4, 64, dtype=torch.float16, device="cuda")
    y[1, 3] = float("inf")
    y[2, 3] = float("nan")
    y[3] = 65504.0
    w = torch.ones(64, dtype=torch.float16, device="cuda")
    r, x = vq.BlockNorm(w).forward(y)
    assert (x[0] == 0).all() and x[2].isnan().all() and torch.equal(r.nan_to_num(5.0), y.nan_to_num(5.0))
    assert x[1, 3].isnan() and (x[1, :3] == 0).all()
    assert (x[3] == 1).all()
    assert vq.BlockNorm(w).forward(y[:0])[1].shape == (0, 64)


# ------------------------------------------------------------------ page plan


def _plan_ref(ctx, q, table, free, page, n_pages, cap, head=0):
    R, width = table.shape
    table = table.copy()
    bits, tokens, taken, rows = 0, 0, 0, []
    for c, n in zip(ctx.tolist(), q.tolist()):
        if c < 0 or n < 0 or c + n > width * page:
            bits |= 1
            tokens += max(n, 0)
        else:
            tokens += n
            taken += -(-(c + n) // page) - -(-c // page)
    if head < 0 or head > len(free) or taken > len(free) - head:
        bits |= 2
    if tokens > cap:
        bits |= 4
    slot, pos = np.full(cap, -1), np.full(cap, -1)
    cu, seq, t, at = np.zeros(R + 1, int), ctx.copy(), 0, head
    if not bits:
        for r in range(R):
            for i in range(-(-ctx[r] // page), -(-(ctx[r] + q[r]) // page)):
                table[r, i] = free[at]
                at += 1
            for p in range(ctx[r], ctx[r] + q[r]):
                pg = table[r, p // page]
                pos[t], slot[t] = p, pg * page + p % page if 0 <= pg < n_pages else -1
                t += 1
            cu[r + 1] = t
        seq = ctx + q
    top = 2 ** 31 - 1
    return table, seq, cu, slot, pos, np.array([bits, min(tokens, top), min(taken, top), 0]), at


def _plan_case(R, page, width, q_hi, seed):
    rng = np.random.default_rng(seed)
    q = rng.integers(0, q_hi + 1, R)
    ctx = rng.integers(0, max(1, width * page - q_hi), R)
    table = np.full((R, width), -7)
    perm = rng.permutation(R * width)
    at = 0
    for r in range(R):
        n = -(-ctx[r] // page)
        table[r, :n] = perm[at:at + n]
        at += n
    return ctx, q, table, perm[at:]


def _run_plan(vq, torch, ctx, q, table, free, page, n_pages, cap, head=None):
    i = lambda a: torch.from_numpy(np.ascontiguousarray(a).astype(np.int32)).cuda()  # noqa: E731
    tb = i(table)
    pl = vq.PagePlanner(tb, i(free), page, n_pages, cap, free_head=None if head is None else i([head]))
    out = torch.zeros(1, dtype=torch.int32, device="cuda")
    p = pl.forward(i(ctx), i(q), free_head_out=out)
    torch.cuda.synchronize()
    got = [x.cpu().numpy() for x in (tb, p.seq_len, p.cu_q, p.slot, p.position, p.status)]
    return got + [out.item()]


@pytest.mark.parametrize("R,page,width,q_hi,extra", [
    (1, 16, 1, 1, 0), (1, 8, 9, 70, 3), (3, 16, 5, 0, 4), (17, 32, 6, 40, 100), (1, 16, 700, 9000, 0),
    (300, 16, 20, 33, 7), (1025, 8, 12, 3, 0), (4096, 1024, 2, 5, 1),
])
@pytest.mark.parametrize("head", [None, 2])
def test_page_plan(vq, torch_dev, R, page, width, q_hi, extra, head):
    ctx, q, table, free = _plan_case(R, page, width, q_hi, R + page)
    free = np.concatenate([[5, 6], free]) if head else free
    cap, n_pages = int(q.sum()) + extra, R * width
    print("plan", R, page, width, q_hi, flush=True)
    ref = _plan_ref(ctx, q, table, free, page, n_pages, cap, head or 0)
    got = _run_plan(vq, torch_dev, ctx, q, table, free, page, n_pages, cap, head)
    assert ref[5][0] == 0
    for name, a, b in zip(("table", "seq", "cu", "slot", "pos", "status", "head"), got, ref):
        assert np.array_equal(a, b), name


@pytest.mark.parametrize("kind,bits", [("negative", 1), ("long", 1), ("free", 2), ("head", 2), ("cap", 4),
                                       ("all", 7)])
def test_page_plan_errors_change_nothing(vq, torch_dev, kind, bits):
    ctx, q, table, free = _plan_case(9, 16, 6, 30, 3)
    q[4] = 20
    ctx[4] = 16
    cap, head = int(q.sum()), 1
    free = np.concatenate([[0], free])
    if kind in ("negative", "all"):
        ctx[2] = -1
    if kind == "long":
        ctx[2], q[2], cap = 96, 1, cap + 1
    if kind == "free":
        free = free[:2]
    if kind == "head":
        head = -3
    if kind == "all":
        head, cap = len(free) + 1, 3
    if kind == "cap":
        cap -= 1
    ref = _plan_ref(ctx, q, table, free, 16, 54, cap, head)
    got = _run_plan(vq, torch_dev, ctx, q, table, free, 16, 54, cap, head)
    assert ref[5][0] == bits
    for name, a, b in zip(("table", "seq", "cu", "slot", "pos", "status", "head"), got, ref):
        assert np.array_equal(a, b), name
    assert np.array_equal(got[0], table)


def test_page_plan_pages_outside_the_cache_have_no_slot(vq, torch_dev):
    ctx, q, table, free = _plan_case(5, 16, 4, 20, 8)
    ctx[1], q[1] = 17, 20
    table[1, 1] = -1
    table[1, 0] = 99999
    free[:] = free[:] + 12
    ref = _plan_ref(ctx, q, table, free, 16, 20, int(q.sum()))
    got = _run_plan(vq, torch_dev, ctx, q, table, free, 16, 20, int(q.sum()))
    for a, b in zip(got, ref):
        assert np.array_equal(a, b)
    assert (got[3] == -1).any() and (got[3] >= 0).any()


# ------------------------------------------------------------------ store


@pytest.mark.parametrize("dtype,T,heads,D,page", [
    ("f16", 1, 1, 8, 8), ("bf16", 7, 3, 80, 16), ("f16", 64, 2, 128, 32), ("bf16", 65, 1, 256, 1024),
    ("f16", 300, 4, 72, 16),
])
def test_paged_store(vq, torch_dev, dtype, T, heads, D, page):
    torch = torch_dev
    dt = _t(torch, dtype)
    n = -(-T // page) + 3
    g = torch.Generator().manual_seed(T)
    slot = torch.randperm(n * page, generator=g)[:T].to(torch.int32)
    if T > 5:  # skipped tokens
        slot[2], slot[4], slot[5] = -1, n * page, 2 ** 31 - 1
    # keys and values as parts of one wider projection row
    rows = _randn(torch, (T, 3 * heads * D), dt, 5).cuda()
    k = rows[:, heads * D:2 * heads * D].unflatten(1, (heads, D))
    v = rows[:, 2 * heads * D:].unflatten(1, (heads, D))
    cache = vq.PagedCache(torch.full((n, heads, page, D), 9.0, dtype=dt, device="cuda"),
                          torch.full((n, heads, D, page), 9.0, dtype=dt, device="cuda"))
    cache.store(k, v, slot.cuda())
    ek, ev = torch.full((n, heads, page, D), 9.0, dtype=dt), torch.full((n, heads, D, page), 9.0, dtype=dt)
    for t, s in enumerate(slot.tolist()):
        if 0 <= s < n * page:
            ek[s // page, :, s % page] = k[t].cpu()
            ev[s // page, :, :, s % page] = v[t].cpu()
    assert torch.equal(cache.k.cpu(), ek) and torch.equal(cache.v.cpu(), ev)


# ------------------------------------------------------------------ attention


def _attn_case(torch, dt, lens, heads, kv_heads, D, page, seed, spare=2):
    g = torch.Generator().manual_seed(seed)
    need = [max(1, -(-kv // page)) for _, kv in lens]
    n = sum(need) + 2
    perm = torch.randperm(n, generator=g)
    table = torch.full((len(lens), max(need) + spare), -1, dtype=torch.int32)
    at = 0
    for r, m in enumerate(need):
        table[r, :m] = perm[at:at + m]
        at += m
    cu = [0]
    for q, _ in lens:
        cu.append(cu[-1] + q)
    k = torch.randn((n, kv_heads, page, D), generator=g).to(dt)
    v = torch.randn((n, kv_heads, D, page), generator=g).to(dt)
    # what no request has stored may be anything
    seen = torch.zeros(n, page, dtype=torch.bool)
    for r, (_, kv) in enumerate(lens):
        for j in range(kv):
            seen[table[r, j // page], j % page] = True
    k.masked_fill_(~seen[:, None, :, None], float("nan"))
    v.masked_fill_(~seen[:, None, None, :], float("nan"))
    q = (torch.randn((cu[-1], heads, D), generator=g) * 1.5).to(dt)
    return q, k, v, table, cu


def _attn_ref(torch, q, k, v, table, cu, kv_len, window, scale):
    T, heads, D = q.shape
    kv_heads, page = k.shape[1], k.shape[2]
    u = _u(torch, q.dtype)
    y, tol = torch.zeros(T, heads, D, dtype=torch.float64), torch.zeros(T, heads, D, dtype=torch.float64)
    lse, ltol = torch.full((T, heads), -math.inf, dtype=torch.float64), torch.zeros(T, heads, dtype=torch.float64)
    for r, kv in enumerate(kv_len):
        n = cu[r + 1] - cu[r]
        if n == 0:
            continue
        j = torch.arange(max(0, min(kv, table.shape[1] * page)))
        pg = table[r].long()[j // page]
        there = (pg >= 0) & (pg < k.shape[0])
        pg = pg.clamp(0, k.shape[0] - 1)
        p = torch.arange(kv - n, kv)[:, None]
        see = (j[None] <= p) & there[None]
        if window:
            see &= j[None] > p - window
        kk = k[pg, :, j % page].double().nan_to_num(0.0)
        vv = v[pg, :, :, j % page].double().nan_to_num(0.0)
        for h in range(heads):
            a = h // (heads // kv_heads)
            qq = q[cu[r]:cu[r + 1], h].double()
            s = (qq @ kk[:, a].T) * scale
            size = (qq.abs() @ kk[:, a].abs().T) * scale
            delta = ((D + 8) * W * size.masked_fill(~see, 0.0)).amax(1, keepdim=True) if len(j) else torch.zeros(n, 1)
            s = s.masked_fill(~see, -math.inf)
            if not len(j):
                continue
            c = torch.logsumexp(s, 1, keepdim=True)
            w = torch.exp(s - c.masked_fill(c == -math.inf, 0.0))
            rows = slice(cu[r], cu[r + 1])
            y[rows, h] = w @ vv[:, a]
            tol[rows, h] = u * y[rows, h].abs() + (u + 2 * delta + 2.0 ** -18) * (w @ vv[:, a].abs()) + 2.0 ** -25
            lse[rows, h] = c[:, 0]
            ltol[rows, h] = (delta[:, 0] + 2.0 ** -20) + 4 * W * c[:, 0].nan_to_num(0, 0, 0).abs()
    return y, tol, lse, ltol


def _attn_check(vq, torch, dt, lens, heads, kv_heads, D, page, window=0, seed=0, max_kv=None, pad=0,
                edit=None, stream=None):
    q, k, v, table, cu = _attn_case(torch, dt, lens, heads, kv_heads, D, page, seed)
    kv_len = [kv for _, kv in lens]
    if edit:
        edit(table, kv_len)
    if pad:
        q = torch.cat([q, torch.full((pad, heads, D), float("nan"), dtype=dt)])
    i = lambda a: torch.tensor(a, dtype=torch.int32, device="cuda")  # noqa: E731
    cache = vq.PagedCache(k.cuda(), v.cuda())
    scale = 0.9 / math.sqrt(D)
    print("attn", dt, lens[:4], heads, kv_heads, D, page, window, flush=True)
    args = (q.cuda(), table.cuda(), i(cu), i(kv_len))
    torch.cuda.synchronize()
    y, lse = cache.attention(*args, scale=scale, window=window, max_kv=max_kv, with_lse=True, stream=stream)
    torch.cuda.synchronize()
    ry, tol, rl, ltol = _attn_ref(torch, q, k, v, table, cu, kv_len, window, scale)
    _close(torch, y, ry, tol, "y")
    _close(torch, lse, rl, ltol, "lse")
    return y, lse


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("lens,heads,kv_heads,D,page,window", [
    ([(1, 1)], 1, 1, 64, 16, 0),
    ([(1, 33), (1, 7), (1, 200)], 8, 1, 128, 16, 0),
    ([(8, 77), (3, 3), (0, 50), (5, 640)], 6, 2, 256, 32, 0),
    ([(8, 8), (1, 900)], 5, 5, 96, 8, 17),
    ([(40, 100), (1, 64), (17, 17)], 4, 2, 80, 64, 0),
    ([(130, 300)], 10, 2, 128, 16, 33),
    ([(70, 70), (129, 500)], 3, 1, 64, 1024, 0),
    ([(33, 64), (2, 130)], 4, 4, 8, 16, 1),
    ([(300, 300), (1, 1100)], 8, 2, 256, 16, 0),
    ([(2, 5), (64, 1000)], 64, 1, 128, 128, 0),
])
def test_paged_attention(vq, torch_dev, dtype, lens, heads, kv_heads, D, page, window):
    _attn_check(vq, torch_dev, _t(torch_dev, dtype), lens, heads, kv_heads, D, page, window, seed=D)


# many rows (keys in LDS), few rows of D > 128 (keys in registers), key splits, odd page and head sizes
TILE_CASES = [
    ([(128, 128)], 1, 1, 64, 16, 0), ([(129, 4100)], 3, 1, 128, 16, 0), ([(64, 2049)], 10, 2, 256, 32, 0),
    ([(17, 4000), (200, 200)], 8, 8, 72, 8, 0), ([(90, 3000)], 5, 1, 136, 64, 700),
    ([(33, 6000)], 4, 4, 128, 1024, 64), ([(1, 9000), (2, 17)], 12, 2, 256, 16, 0),
    ([(3, 5000)], 5, 1, 200, 8, 1000), ([(1, 0), (1, 1), (1, 31), (1, 32), (1, 33), (1, 65)], 2, 1, 128, 16, 0),
    ([(0, 7), (250, 260), (0, 0), (1, 64)], 6, 3, 96, 16, 1),
]


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("lens,heads,kv_heads,D,page,window", TILE_CASES)
def test_paged_attention_tiles(vq, torch_dev, dtype, lens, heads, kv_heads, D, page, window):
    _attn_check(vq, torch_dev, _t(torch_dev, dtype), lens, heads, kv_heads, D, page, window, seed=D + 1, pad=3)


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("D", [72, 80, 96, 104, 136, 160, 192, 208])
def test_paged_attention_tiles_of_odd_heads(vq, torch_dev, dtype, D):
    """Heads that leave a part of a tile's row empty, a little or more than a quarter."""
    _attn_check(vq, torch_dev, _t(torch_dev, dtype), [(150, 700), (70, 70), (1, 9)], 4, 2, D, 16, seed=D, pad=2)
    _attn_check(vq, torch_dev, _t(torch_dev, dtype), [(129, 300)], 2, 2, D, 32, window=50, seed=D + 1)


@pytest.mark.parametrize("lens,D", [([(150, 700), (40, 900)], 128), ([(60, 1500)], 256), ([(2, 1500)], 256)])
def test_paged_attention_tiles_skip_pages_outside_the_cache(vq, torch_dev, lens, D):
    """Holes inside a request's keys, at its start and at its end, next to whole tiles."""

    def edit(table, kv_len):
        for r in range(len(kv_len)):
            last = (kv_len[r] + 15) // 16 - 1
            table[r, 0], table[r, 7], table[r, 20], table[r, 21] = -1, 2 ** 31 - 1, 10 ** 6, -2 ** 31
            table[r, last] = -5

    _attn_check(vq, torch_dev, torch_dev.float16, lens, 4, 2, D, 16, edit=edit, seed=9)


@pytest.mark.parametrize("rows", [1, 40])
@pytest.mark.parametrize("D", [64, 256])
def test_paged_attention_far_pages(vq, torch_dev, D, rows):
    """Pages whose first element lies beyond 2^32 elements of the cache give what near ones give."""
    torch = torch_dev
    dt, page = torch.bfloat16, 1024
    n = 2 ** 32 // (page * D) + 4
    k = torch.empty((n, 1, page, D), dtype=dt, device="cuda")
    v = torch.empty((n, 1, D, page), dtype=dt, device="cuda")
    g = torch.Generator(device="cuda").manual_seed(1)
    for near, far in ((0, n - 1), (1, n - 3)):
        k[near].normal_(generator=g)
        v[near].normal_(generator=g)
        k[far], v[far] = k[near], v[near]
    q = torch.randn((rows, 2, D), generator=g, device="cuda").to(dt)
    i = lambda a: torch.tensor(a, dtype=torch.int32, device="cuda")  # noqa: E731
    cache, cu, kv = vq.PagedCache(k, v), i([0, rows]), i([2000])
    near = cache.attention(q, i([[0, 1]]), cu, kv)
    assert torch.equal(near, cache.attention(q, i([[n - 1, n - 3]]), cu, kv))
    # and the store reaches them
    kv_new = torch.randn((1, 1, D), generator=g, device="cuda").to(dt)
    cache.store(kv_new, kv_new, i([(n - 1) * page + 5]))
    assert torch.equal(k[n - 1, 0, 5], kv_new[0, 0]) and torch.equal(v[n - 1, 0, :, 5], kv_new[0, 0])


def test_paged_attention_rows_that_see_nothing(vq, torch_dev):
    """More rows than keys, no keys at all, rows behind the last request (NaN queries)."""
    torch = torch_dev
    y, lse = _attn_check(vq, torch, torch.float16, [(9, 4), (3, 0), (20, 1)], 4, 2, 64, 16, pad=37)
    assert (y[:5] == 0).all() and (lse[:5] == -math.inf).all() and (y[9:12] == 0).all()
    assert (y[32:] == 0).all() and (lse[32:] == -math.inf).all()


@pytest.mark.parametrize("bad", [-1, -2 ** 31, 2 ** 31 - 1, 1000])
def test_paged_attention_skips_pages_outside_the_cache(vq, torch_dev, bad):
    torch = torch_dev

    def edit(table, kv_len):
        table[0, 1] = bad
        table[1, :] = bad
        kv_len[2] = 10 ** 6  # beyond the table: the keys end where it ends, the rows see them all

    _attn_check(vq, torch, torch.bfloat16, [(5, 100), (3, 40), (4, 48)], 4, 2, 128, 16, edit=edit)


@pytest.mark.parametrize("max_kv", [0, 1, 100, 10 ** 6])
def test_paged_attention_any_key_bound(vq, torch_dev, max_kv):
    """max_kv only chooses the split: below the truth and far above it the values hold."""
    torch = torch_dev
    _attn_check(vq, torch, torch.float16, [(3, 2100), (1, 5)], 6, 2, 128, 16, max_kv=max_kv)
    _attn_check(vq, torch, torch.float16, [(200, 1500)], 6, 2, 64, 16, max_kv=max_kv)


@pytest.mark.parametrize("lens,heads,D", [([(1, 9000)], 10, 128), ([(3, 9000), (1, 4000)], 4, 256),
                                          ([(150, 3000), (9, 9)], 4, 64)])
def test_paged_attention_windows_over_long_contexts(vq, torch_dev, lens, heads, D):
    """Windows from one key to more than there are, in one cache; a workspace made without the window holds."""
    torch = torch_dev
    for window in (1, 63, 64, 1000, 5000, 2 ** 31 - 1):
        _attn_check(vq, torch, torch.float16, lens, heads, 2, D, 16, window=window, seed=window % 100)
    q, k, v, table, cu = _attn_case(torch, torch.float16, lens, heads, 2, D, 16, 3)
    i = lambda a: torch.tensor(a, dtype=torch.int32, device="cuda")  # noqa: E731
    cache = vq.PagedCache(k.cuda(), v.cuda())
    args = (q.cuda(), table.cuda(), i(cu), i([n for _, n in lens]))
    small = cache.attention(*args, window=100)
    whole = cache.attention(*args)
    n = cache.workspace_bytes(q.shape[0], len(lens), heads, table.shape[1])
    ws = torch.empty(max(n, 1), dtype=torch.uint8, device="cuda")
    assert torch.equal(small, cache.attention(*args, window=100, workspace=ws))
    assert torch.equal(whole, cache.attention(*args, workspace=ws))


def test_paged_attention_extreme_scores(vq, torch_dev):
    """One key far above the others, all keys equal, and scores of thousands."""
    torch = torch_dev
    dt, D = torch.float16, 64
    k = torch.zeros(4, 1, 16, D, dtype=dt)
    v = torch.arange(64).view(4, 1, 1, 16).expand(4, 1, D, 16).contiguous().to(dt)
    q = torch.ones(3, 1, D, dtype=dt)
    i = lambda a: torch.tensor(a, dtype=torch.int32, device="cuda")  # noqa: E731
    table, cu, kv = i([[0, 1, 2, 3]]), i([0, 3]), i([64])
    k[2, 0, 5] = 100.0
    y = vq.PagedCache(k.cuda(), v.cuda()).attention(q.cuda(), table, cu, kv, scale=1.0)
    assert (y == 37).all()
    k[:] = 30.0
    y, lse = vq.PagedCache(k.cuda(), v.cuda()).attention(q.cuda(), table, cu, kv, scale=1.0, with_lse=True)
    ref = torch.tensor([30.5, 31.0, 31.5])  # means of 0 .. 61, 62, 63
    assert (y[:, 0, 0].float().cpu() - ref).abs().max() <= 31.5 * 2.0 ** -10
    want = 30.0 * D + torch.log(torch.tensor([62.0, 63.0, 64.0]))
    assert (lse[:, 0].cpu() - want).abs().max() <= 1920 * 4 * W


def test_paged_attention_many_far_keys_count(vq, torch_dev):
    """65,000 keys each 2^-20 of the one at the top carry 6% of the weight together."""
    torch = torch_dev
    dt, D, n = torch.float16, 64, 65008
    k = torch.zeros(n // 16, 1, 16, D, dtype=dt, device="cuda")
    k[7, 0, 3, 0] = 20 * math.log(2)
    v = torch.ones(n // 16, 1, D, 16, dtype=dt, device="cuda")
    v[7, 0, :, 3] = -1.0
    q = torch.zeros(1, 1, D, dtype=dt, device="cuda")
    q[0, 0, 0] = 1.0
    i = lambda a: torch.tensor(a, dtype=torch.int32, device="cuda")  # noqa: E731
    table = torch.arange(n // 16, dtype=torch.int32, device="cuda")[None]
    y = vq.PagedCache(k, v).attention(q, table, i([0, 1]), i([n]), scale=1.0)
    top = math.exp(float(k[7, 0, 3, 0]))
    ref = (n - 1 - top) / (n - 1 + top)
    assert abs(float(y[0, 0, 0]) - ref) <= 3 * 2.0 ** -11, (float(y[0, 0, 0]), ref)


@pytest.mark.parametrize("lens", [[(3, 40)], [(2, 3000)], [(200, 700)]])
def test_paged_attention_nan_queries_give_nan(vq, torch_dev, lens):
    """A NaN query makes its own outputs NaN, with and without a split of the keys; others keep theirs."""
    torch = torch_dev
    q, k, v, table, cu = _attn_case(torch, torch.bfloat16, lens, 4, 2, 64, 16, 6)
    i = lambda a: torch.tensor(a, dtype=torch.int32, device="cuda")  # noqa: E731
    cache = vq.PagedCache(k.cuda(), v.cuda())
    args = (table.cuda(), i(cu), i([kv for _, kv in lens]))
    y, lse = cache.attention(q.cuda(), *args, with_lse=True)
    q[1, 2, 5] = float("nan")
    y2, lse2 = cache.attention(q.cuda(), *args, with_lse=True)
    assert y2[1, 2].isnan().all() and lse2[1, 2].isnan()
    keep = torch.ones(y.shape[:2], dtype=torch.bool, device="cuda")
    keep[1, 2] = False
    assert torch.equal(y2[keep], y[keep]) and torch.equal(lse2[keep], lse[keep])


def test_paged_attention_strides_streams_and_graphs(vq, torch_dev):
    torch = torch_dev
    dt = torch.bfloat16
    q, k, v, table, cu = _attn_case(torch, dt, [(5, 300), (70, 90)], 8, 2, 128, 16, 4)
    i = lambda a: torch.tensor(a, dtype=torch.int32, device="cuda")  # noqa: E731
    cache, qd, tb, cud, kv = vq.PagedCache(k.cuda(), v.cuda()), q.cuda(), table.cuda(), i(cu), i([300, 90])
    want = cache.attention(qd, tb, cud, kv)
    # queries inside a wider projection row, outputs into one
    wide = torch.zeros(75, 20, 128, dtype=dt, device="cuda")
    wide[:, 4:12] = qd
    out = torch.full((75, 10, 128), 3.0, dtype=dt, device="cuda")
    cache.attention(wide[:, 4:12], tb, cud, kv, y=out[:, 1:9])
    assert torch.equal(out[:, 1:9], want) and (out[:, 0] == 3).all() and (out[:, 9] == 3).all()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    y = cache.attention(qd, tb, cud, kv, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(y, want)
    # a graph replayed with other lengths reads them anew
    y, work = torch.empty_like(want), torch.empty(
        cache.workspace_bytes(75, 2, 8, tb.shape[1]), dtype=torch.uint8, device="cuda")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        cache.attention(qd, tb, cud, kv, y=y, workspace=work)
    for lens, starts in (([300, 90], cu), ([111, 80], cu), ([290, 85], [0, 30, 75]), ([300, 90], cu)):
        kv.copy_(i(lens))
        cud.copy_(i(starts))
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(y, cache.attention(qd, tb, cud, kv)), lens
    assert torch.equal(y, want)


# ------------------------------------------------------------------ linear attention


def _linear_ref(torch, q, k, v, g, state, cu, ctx, index, scale, n_states):
    T, hk, dk = q.shape
    hv, dv = v.shape[1:]
    rep = hv // hk
    y, z = torch.zeros(T, hv, dv, dtype=torch.float64), torch.zeros(T, hv, dv, dtype=torch.float64)
    out, size = state.double().clone(), torch.zeros(state.shape, dtype=torch.float64)
    kd, qd = k.double().repeat_interleave(rep, 1), q.double().repeat_interleave(rep, 1)
    vd, e = v.double(), torch.exp(g.double())
    for r in range(len(cu) - 1):
        s = r if index is None else index[r]
        if not 0 <= s < n_states:
            s = -1
        S = state[s].double().clone() if s >= 0 and (ctx is None or ctx[r] > 0) else torch.zeros(hv, dk, dv).double()
        A = S.abs()
        for t in range(cu[r], cu[r + 1]):
            S = e[t][:, None, None] * S + kd[t][:, :, None] * vd[t][:, None, :]
            A = e[t][:, None, None] * A + kd[t].abs()[:, :, None] * vd[t].abs()[:, None, :]
            y[t] = scale * (S * qd[t][:, :, None]).sum(1)
            z[t] = abs(scale) * (A * qd[t].abs()[:, :, None]).sum(1)
        if s >= 0:
            out[s], size[s] = S, A
    return y, z, out, size


def _linear_check(vq, torch, dtype, lens, hk, hv, dk, dv, max_q=None, ctx=None, index=None, n_states=None,
                  pad=0, g=None, std=1.0, in_place=False, scale=None, seed=0):
    dt = _t(torch, dtype)
    cu = [0]
    for n in lens:
        cu.append(cu[-1] + n)
    T, R = cu[-1] + pad, len(lens)
    n_states = R if n_states is None else n_states
    q, k = _randn(torch, (T, hk, dk), dt, seed, dk ** -0.5), _randn(torch, (T, hk, dk), dt, seed + 1, dk ** -0.5)
    v = _randn(torch, (T, hv, dv), dt, seed + 2, std)
    if g is None:
        g = -torch.nn.functional.softplus(_randn(torch, (T, hv), torch.float32, seed + 3) * 2 - 3)
    state = _randn(torch, (n_states, hv, dk, dv), torch.float32, seed + 4, 0.5 * std)
    i = lambda a: None if a is None else torch.tensor(a, dtype=torch.int32, device="cuda")  # noqa: E731
    op = vq.LinearAttention(hk, hv, dk, dv, scale)
    sd = state.cuda()
    print("linear", dtype, lens[:5], hk, hv, dk, dv, max_q, flush=True)
    y, out = op.forward(q.cuda(), k.cuda(), v.cuda(), g.cuda(), sd, i(cu), ctx_len=i(ctx),
                        state_index=i(index), max_q=max_q, state_out=sd if in_place else None)
    torch.cuda.synchronize()
    if not in_place:
        assert torch.equal(sd.cpu(), state)
    ry, z, rs, size = _linear_ref(torch, q, k, v, g, state, cu, ctx, index, op.scale, n_states)
    u = _u(torch, dt)
    n = max(lens + [1])
    # FP32: a sum per chunk and one per token in it, and the exponents' arguments (largest sum of
    # decays within 64 tokens times W, in a product of decays once per chunk)
    gs = g.clamp(min=-80.0).abs()
    span = max([float(gs[a:a + 64].sum(0).max()) for a in range(0, max(1, T), 64)] + [0.0])
    _close(torch, y[:cu[-1]], ry[:cu[-1]],
           u * ry[:cu[-1]].abs() + (2 * u + (100 + n / 16 + 4 * span) * W) * z[:cu[-1]] + 2.0 ** -25, "y")
    assert (y[cu[-1]:] == 0).all()
    _close(torch, out, rs, (100 + n / 8) * W * size + 2.0 ** -100, "state")
    return y, out


LINEAR_SHAPES = [(1, 1, 64, 64), (2, 6, 128, 128), (2, 2, 96, 40), (1, 3, 8, 128), (3, 3, 128, 72)]


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("hk,hv,dk,dv", LINEAR_SHAPES)
@pytest.mark.parametrize("lens,max_q", [
    ([1], 1), ([8, 1, 0, 3], 8), ([16, 2], 16),             # the recurrence
    ([20, 1, 0, 70], 16),                                   # the same beyond its bound
    ([1, 64, 65, 0, 130], 130), ([17, 300], None),          # chunks
])
def test_linear_attention(vq, torch_dev, dtype, hk, hv, dk, dv, lens, max_q):
    _linear_check(vq, torch_dev, dtype, lens, hk, hv, dk, dv, max_q)


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("in_place", [False, True])
def test_linear_attention_segments(vq, torch_dev, dtype, in_place):
    """Long requests go through in segments whose states are joined; in place too."""
    _linear_check(vq, torch_dev, dtype, [1500, 0, 601, 1], 1, 2, 64, 64, ctx=[3, 1, 0, 9], in_place=in_place)
    _linear_check(vq, torch_dev, dtype, [1290], 1, 1, 128, 128, max_q=512, in_place=in_place)


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("dk,dv", [(72, 40), (40, 128), (128, 40), (128, 128), (64, 64)])
def test_linear_attention_segments_of_odd_heads(vq, torch_dev, dtype, dk, dv):
    _linear_check(vq, torch_dev, dtype, [1290, 77, 700], 1, 2, dk, dv, ctx=[2, 0, 1], seed=11, pad=1)


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("dk,dv", [(128, 128), (104, 96), (72, 40), (128, 8)])
def test_linear_attention_recurrence_few_and_many_waves(vq, torch_dev, dtype, dk, dv):
    _linear_check(vq, torch_dev, dtype, [8, 1, 0, 16], 1, 2, dk, dv, 16, ctx=[1, 0, 3, 7], seed=12, pad=2)
    _linear_check(vq, torch_dev, dtype, [1, 2, 0] * 23, 2, 16, dk, dv, 2, seed=13)


@pytest.mark.parametrize("lens,max_q", [([5, 1, 3], 8), ([100, 1, 66], 100)])
def test_linear_attention_slots_and_fresh_requests(vq, torch_dev, lens, max_q):
    torch = torch_dev
    for index, n in (([4, 0, 2], 5), ([1, -1, 7], 3)):
        _linear_check(vq, torch, "f16", lens, 2, 4, 64, 32, max_q, ctx=[1, 5, 0], index=index, n_states=n, pad=13)


@pytest.mark.parametrize("max_q", [16, 200])
def test_linear_attention_decays(vq, torch_dev, max_q):
    """No decay, full decay at some tokens (-inf and the type's lowest value), strong decays."""
    torch = torch_dev
    T = 200
    g = torch.zeros(T, 4)
    g[:, 1] = -5.0
    g[::7, 2] = -math.inf
    g[5::31, 2] = torch.finfo(torch.float32).min
    g[:, 2] -= 0.01
    g[:, 3] = -torch.rand(T, generator=torch.Generator().manual_seed(1)) * 60
    for dtype in ("f16", "bf16"):
        _linear_check(vq, torch, dtype, [T], 2, 4, 64, 64, max_q, g=g)


@pytest.mark.parametrize("max_q", [16, 150])
@pytest.mark.parametrize("std", [2.0 ** -12, 1000.0])
def test_linear_attention_scales(vq, torch_dev, std, max_q):
    """Small and large values and states keep FP32 accuracy in the state, and y its type's."""
    _linear_check(vq, torch_dev, "f16", [150, 3], 1, 2, 128, 64, max_q, std=std,
                  scale=1.0 if std < 1 else 0.01)


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("max_q", [16, 900])
def test_linear_attention_growing_states(vq, torch_dev, dtype, max_q):
    """Keys that all point one way and no decay: the state outgrows the values by the number of tokens;
    then values of one part in a million: it stays while they come in."""
    torch = torch_dev
    dt, T = _t(torch, dtype), 900
    k = torch.full((T, 1, 64), 0.125, dtype=dt)
    q = _randn(torch, (T, 1, 64), dt, 1, 0.125)
    v = _randn(torch, (T, 2, 64), dt, 2).abs() + 1
    v[600:] *= 2.0 ** -14
    g = torch.zeros(T, 2)
    g[:, 1] = -1e-3
    i = lambda a: torch.tensor(a, dtype=torch.int32, device="cuda")  # noqa: E731
    op = vq.LinearAttention(1, 2, 64, 64)
    state = op.state(1)
    y, out = op.forward(q.cuda(), k.cuda(), v.cuda(), g.cuda(), state, i([0, T]), max_q=max_q)
    ry, z, rs, size = _linear_ref(torch, q, k, v, g, state.cpu(), [0, T], None, None, op.scale, 1)
    u = _u(torch, dt)
    _close(torch, y, ry, u * ry.abs() + (2 * u + (100 + T / 16) * W) * z + 2.0 ** -25, "y")
    _close(torch, out, rs, (100 + T / 8) * W * size, "state")


@pytest.mark.parametrize("hk,hv", [(3, 9), (16, 16), (5, 5)])
def test_linear_attention_many_heads_and_requests(vq, torch_dev, hk, hv):
    """Every workgroup number meets its request, segment and head, whatever divides by what."""
    _linear_check(vq, torch_dev, "f16", [70, 3, 0, 65, 130, 64, 1, 257, 40], hk, hv, 24, 16, seed=5, pad=5)
    _linear_check(vq, torch_dev, "bf16", [1100, 700], hk, hv, 16, 8, seed=6)


def test_linear_attention_strides_streams_and_graphs(vq, torch_dev):
    torch = torch_dev
    i = lambda a: torch.tensor(a, dtype=torch.int32, device="cuda")  # noqa: E731
    op = vq.LinearAttention(2, 4, 64, 64)
    for lens, max_q, other in (([3, 8, 1], 8, [8, 0, 4]), ([700, 30, 600], 700, [600, 700, 30])):
        T = sum(lens)
        rows = _randn(torch, (T, 2 * 128 + 256 + 8), torch.float16, 3, 0.2).cuda()
        q, k = rows[:, :128].unflatten(1, (2, 64)), rows[:, 128:256].unflatten(1, (2, 64))
        v = rows[:, 256:512].unflatten(1, (4, 64))
        g = -torch.rand(T, 6, device="cuda")
        state = torch.randn(3, 4, 64, 64, device="cuda")
        start = lambda ls: i(np.concatenate([[0], np.cumsum(ls)]).tolist())  # noqa: E731
        cu = start(lens)
        args = (q.contiguous(), k.contiguous(), v.contiguous(), g[:, 1:5].contiguous())
        y, s = op.forward(*args, state, cu, max_q=max_q)
        y2, s2 = op.forward(q, k, v, g[:, 1:5], state, cu, max_q=max_q)
        assert torch.equal(y, y2) and torch.equal(s, s2)
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        y3, s3 = op.forward(*args, state, cu, max_q=max_q, stream=side)
        torch.cuda.current_stream().wait_stream(side)
        assert torch.equal(y, y3) and torch.equal(s, s3)
        out = torch.empty_like(s)
        work = torch.empty(max(1, op.workspace_bytes(T, 3, max_q)), dtype=torch.uint8, device="cuda")
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            op.forward(*args, state, cu, max_q=max_q, state_out=out, y=y2, workspace=work)
        for ls in (lens, other, lens):
            cu.copy_(start(ls))
            graph.replay()
            torch.cuda.synchronize()
            y4, s4 = op.forward(*args, state, cu, max_q=max_q)
            assert torch.equal(y2, y4) and torch.equal(out, s4), ls
        assert torch.equal(y2, y)


# ------------------------------------------------------------------ together


def test_poisoned_workspaces_change_nothing(vq, torch_dev):
    """Workspaces need no fill: all bits set gives the values of a fresh call, with short requests (done
    in one split) next to long ones, and with segments."""
    torch = torch_dev
    i = lambda a: torch.tensor(a, dtype=torch.int32, device="cuda")  # noqa: E731
    for lens, D in (([(1, 5000), (1, 20), (2, 700), (0, 9)], 64), ([(150, 4000), (3, 30)], 128),
                    ([(2, 3000), (1, 10)], 256)):
        q, k, v, table, cu = _attn_case(torch, torch.float16, lens, 4, 2, D, 16, 7)
        cache = vq.PagedCache(k.cuda(), v.cuda())
        args = (q.cuda(), table.cuda(), i(cu), i([kv for _, kv in lens]))
        want = cache.attention(*args, with_lse=True)
        work = torch.full((cache.workspace_bytes(q.shape[0], len(lens), 4, table.shape[1]),), 255,
                          dtype=torch.uint8, device="cuda")
        assert work.numel() > 0
        for _ in range(2):
            got = cache.attention(*args, with_lse=True, workspace=work)
            assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    op = vq.LinearAttention(1, 2, 64, 64)
    x = [_randn(torch, (2600, h, 64), torch.float16, s, 0.2).cuda() for h, s in ((1, 1), (1, 2), (2, 3))]
    g = -torch.rand(2600, 2, device="cuda")
    state = torch.randn(2, 2, 64, 64, device="cuda")
    want = op.forward(*x, g, state, i([0, 2000, 2600]))
    work = torch.full((op.workspace_bytes(2600, 2, 2600),), 255, dtype=torch.uint8, device="cuda")
    assert work.numel() > 0
    got = op.forward(*x, g, state, i([0, 2000, 2600]), workspace=work)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


def test_small_workspaces_are_refused(vq, torch_dev):
    torch = torch_dev
    q, k, v, table, cu = _attn_case(torch, torch.float16, [(2, 3000)], 2, 1, 64, 16, 0)
    i = lambda a: torch.tensor(a, dtype=torch.int32, device="cuda")  # noqa: E731
    cache = vq.PagedCache(k.cuda(), v.cuda())
    small = torch.empty(256, dtype=torch.uint8, device="cuda")
    with pytest.raises(vq.VqmlpError) as e:
        cache.attention(q.cuda(), table.cuda(), i(cu), i([3000]), workspace=small)
    assert e.value.status == vq.ERR_WORKSPACE
    op = vq.LinearAttention(1, 1, 64, 64)
    z = torch.zeros(2000, 1, 64, dtype=torch.float16, device="cuda")
    with pytest.raises(vq.VqmlpError) as e:
        op.forward(z, z, z, torch.zeros(2000, 1, device="cuda"), op.state(1), i([0, 2000]), workspace=small)
    assert e.value.status == vq.ERR_WORKSPACE


def test_block_ops_trace(vq, torch_dev, capfd, monkeypatch):
    torch = torch_dev
    monkeypatch.setenv("VQMLP_TRACE", "1")
    w = torch.ones(64, dtype=torch.float16, device="cuda")
    capfd.readouterr()
    vq.BlockNorm(w).forward(torch.zeros(3, 64, dtype=torch.float16, device="cuda"))
    op = vq.LinearAttention(1, 1, 64, 64)
    z = torch.zeros(2, 1, 64, dtype=torch.float16, device="cuda")
    op.forward(z, z, z, torch.zeros(2, 1, device="cuda"), op.state(1),
               torch.tensor([0, 2], dtype=torch.int32, device="cuda"))
    torch.cuda.synchronize()
    lines = [x for x in capfd.readouterr().err.splitlines() if x.startswith("vqmlp: ")]
    assert len(lines) == 2 and "block_norm T=3 H=64: vector kernel" in lines[0] and "recurrence" in lines[1], lines
