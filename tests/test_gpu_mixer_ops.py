"""GPU: the operators in front of and inside the mixers (gated delta rule, append with norm and rotation,
short convolution) against plain 64-bit forms on the same inputs.

Tolerances.  u = eps / 2 of the 16-bit type is one rounding, W = 2^-24 one of FP32.
  delta   Keys of length one and beta in [0, 1] make the step S -> e (S - beta k (S^T k)^T) no longer than
          it was, so an error of a column of S is carried on and not enlarged.  Each token adds to a column at
          most C W (|S'| + |v|), |S'| the length of the decayed column: sums over Dk rows (and the chunks'
          sums over 64 tokens) in FP32, C = Dk + 64.  Z sums that up with the decays.  A chunk applies the
          step's factors in another order: its triangular system has norm 1, which doubles C.  An output
          takes the state's error times scale |q|, one rounding of its own and, in chunks, one each of the state,
          the scores and the updates u as 16-bit operands, together 2 u of scale |q| times B = the decayed sum
          of |S_0| and all |u_t|.
  append  one rounding of the output; of norm and rotation 32 W of |a| + |b|.
  conv    one rounding of the output; sums of W + 1 terms, and |z| W of the exponential; brought to length
          one, the same of the head's length.
"""
import math

import numpy as np
import pytest

from test_gpu_block_ops import _close, _randn, _t, _u, torch_dev, vq  # noqa: F401

pytestmark = pytest.mark.gpu

W = 2.0 ** -24


def _i(torch, a):
    return None if a is None else torch.tensor(a, dtype=torch.int32, device="cuda")


def _starts(lens):
    return np.concatenate([[0], np.cumsum(lens)]).astype(int).tolist()


# ------------------------------------------------------------------ gated delta rule


def _delta_ref(torch, q, k, v, g, beta, state, cu, ctx, index, scale):
    T, hk, dk = q.shape
    hv, dv = v.shape[1:]
    rep, n_states = hv // hk, state.shape[0]
    y, ty, tz = (torch.zeros(T, hv, dv, dtype=torch.float64) for _ in range(3))
    out, ts = state.double().clone(), torch.zeros(state.shape, dtype=torch.float64)
    kd, qd = k.double().repeat_interleave(rep, 1), q.double().repeat_interleave(rep, 1)
    vd, e, bd = v.double(), torch.exp(g.double().clamp(min=-80.0)), beta.double()
    for r in range(len(cu) - 1):
        s = r if index is None else index[r]
        if not 0 <= s < n_states:
            s = -1
        old = s >= 0 and (ctx is None or ctx[r] > 0)
        S = state[s].double().clone() if old else torch.zeros(hv, dk, dv).double()
        B = S.norm(dim=1)
        Z = torch.zeros_like(B)
        for t in range(cu[r], cu[r + 1]):
            S = e[t][:, None, None] * S
            u = bd[t][:, None] * (vd[t] - torch.einsum("hkv,hk->hv", S, kd[t]))
            Z = e[t][:, None] * Z + S.norm(dim=1) + vd[t].abs()
            B = e[t][:, None] * B + u.abs()
            S = S + kd[t][:, :, None] * u[:, None, :]
            y[t] = scale * torch.einsum("hkv,hk->hv", S, qd[t])
            length = abs(scale) * qd[t].norm(dim=1)[:, None]
            ty[t], tz[t] = length * B, length * Z
        if s >= 0:
            out[s] = S
            ts[s] = Z[:, None, :].expand(hv, dk, dv)
    return y, ty, tz, out, ts


def _unit(x, dt):
    return (x / x.norm(dim=-1, keepdim=True)).to(dt)


def _delta_inputs(torch, dt, T, hk, hv, dk, dv, seed, std=1.0):
    q = _unit(_randn(torch, (T, hk, dk), torch.float32, seed), dt)
    k = _unit(_randn(torch, (T, hk, dk), torch.float32, seed + 1), dt)
    v = _randn(torch, (T, hv, dv), dt, seed + 2, std)
    g = -torch.nn.functional.softplus(_randn(torch, (T, hv), torch.float32, seed + 3) * 2 - 3)
    beta = torch.sigmoid(_randn(torch, (T, hv), torch.float32, seed + 4) * 1.5)
    return q, k, v, g, beta


def _delta_check(vq, torch, dtype, lens, hk, hv, dk, dv, max_q=None, ctx=None, index=None, n_states=None, pad=0,
                 inputs=None, std=1.0, in_place=False, scale=None, seed=0, state=None):
    dt = _t(torch, dtype)
    cu = _starts(lens)
    T, R = cu[-1] + pad, len(lens)
    n_states = R if n_states is None else n_states
    q, k, v, g, beta = inputs or _delta_inputs(torch, dt, T, hk, hv, dk, dv, seed, std)
    if state is None:
        state = _randn(torch, (n_states, hv, dk, dv), torch.float32, seed + 5, 0.5 * std)
    op = vq.DeltaRule(hk, hv, dk, dv, scale)
    sd = state.cuda()
    print("delta", dtype, lens[:5], hk, hv, dk, dv, max_q, flush=True)
    y, out = op.forward(q.cuda(), k.cuda(), v.cuda(), g.cuda(), beta.cuda(), sd, _i(torch, cu), ctx_len=_i(torch, ctx),
                        state_index=_i(torch, index), max_q=max_q, state_out=sd if in_place else None)
    torch.cuda.synchronize()
    if not in_place:
        assert torch.equal(sd.cpu(), state)
    ry, B, Z, rs, ts = _delta_ref(torch, q, k, v, g, beta, state, cu, ctx, index, op.scale)
    u, c, n = _u(torch, dt), 2 * (dk + 64) * W, cu[-1]
    _close(torch, y[:n], ry[:n], u * ry[:n].abs() + (2 * u + c) * B[:n] + c * Z[:n] + 2.0 ** -25, "y")
    assert (y[n:] == 0).all()
    _close(torch, out, rs, c * ts + 2.0 ** -100, "state")
    return y, out


DELTA_SHAPES = [(1, 1, 64, 64), (2, 6, 128, 128), (2, 2, 96, 40), (1, 3, 8, 128), (3, 3, 128, 72)]


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("hk,hv,dk,dv", DELTA_SHAPES)
@pytest.mark.parametrize("lens,max_q", [
    ([1], 1), ([8, 1, 0, 3], 8), ([16, 2], 16),      # short requests
    ([20, 1, 0, 70], 16),                            # longer than they were said to be
    ([1, 64, 65, 0, 130], 130), ([17, 300], None),   # prompts
])
def test_delta_rule(vq, torch_dev, dtype, hk, hv, dk, dv, lens, max_q):
    _delta_check(vq, torch_dev, dtype, lens, hk, hv, dk, dv, max_q)


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("in_place", [False, True])
def test_delta_rule_long_requests(vq, torch_dev, dtype, in_place):
    _delta_check(vq, torch_dev, dtype, [1500, 0, 601, 1], 1, 2, 64, 64, ctx=[3, 1, 0, 9], in_place=in_place)
    _delta_check(vq, torch_dev, dtype, [1290], 1, 1, 128, 128, max_q=512, in_place=in_place)


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("dk,dv", [(128, 128), (104, 96), (72, 40), (128, 8)])
def test_delta_rule_few_and_many_waves(vq, torch_dev, dtype, dk, dv):
    _delta_check(vq, torch_dev, dtype, [3], 1, 2, dk, dv, 8)
    _delta_check(vq, torch_dev, dtype, [2, 1, 3] * 20, 4, 16, dk, dv, 8)


@pytest.mark.parametrize("lens,max_q", [([5, 1, 3], 8), ([100, 1, 66], 100)])
def test_delta_rule_slots_and_fresh_requests(vq, torch_dev, lens, max_q):
    """Slots in any order, one outside the array, requests that start anew, rows behind the last."""
    _delta_check(vq, torch_dev, "f16", lens, 2, 4, 64, 64, max_q, ctx=[4, 0, 7], index=[3, 0, 5], n_states=5, pad=3)
    _delta_check(vq, torch_dev, "bf16", lens, 2, 4, 64, 64, max_q, ctx=[0, 9, 1], index=[-1, 2, 1], n_states=3, pad=70)


@pytest.mark.parametrize("max_q", [16, 200])
@pytest.mark.parametrize("dtype", ["f16", "bf16"])
def test_delta_rule_decays_and_gates(vq, torch_dev, max_q, dtype):
    """No decay, decays that forget at once, -inf, and beta of 0 and 1."""
    torch = torch_dev
    T = 200
    q, k, v, g, beta = _delta_inputs(torch, _t(torch, dtype), T, 1, 4, 64, 64, 11)
    g[:, 0] = 0.0
    g[:, 1] = -100.0
    g[5::7, 2] = -math.inf
    g[60:70, 3] = -30.0
    beta[::3] = 0.0
    beta[1::3] = 1.0
    _delta_check(vq, torch, dtype, [T - 90, 90], 1, 4, 64, 64, max_q, inputs=(q, k, v, g, beta))


@pytest.mark.parametrize("max_q", [16, 200])
@pytest.mark.parametrize("dtype", ["f16", "bf16"])
def test_delta_rule_repeated_keys(vq, torch_dev, max_q, dtype):
    """One key for all tokens, and beta 1: each update replaces the one before, the triangular system is full."""
    torch = torch_dev
    T, dt = 150, _t(torch, dtype)
    q, k, v, g, beta = _delta_inputs(torch, dt, T, 1, 2, 64, 64, 12)
    k[:] = 0.0
    k[:, :, 3] = 1.0
    beta[:] = 1.0
    g[:, 0] = 0.0
    y, out = _delta_check(vq, torch, dtype, [T], 1, 2, 64, 64, max_q, inputs=(q, k, v, g, beta))
    assert (out[0, :, 3].cpu() - v[-1].float()).abs().max() <= 200 * W * v.float().abs().max()


@pytest.mark.parametrize("max_q", [16, 300])
@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("std", [2.0 ** -12, 1000.0])
def test_delta_rule_value_sizes(vq, torch_dev, max_q, dtype, std):
    _delta_check(vq, torch_dev, dtype, [130, 70, 1], 1, 2, 64, 64, max_q, std=std, seed=3)


@pytest.mark.parametrize("max_q", [16, 300])
@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("apart", [14, 20])
def test_delta_rule_value_columns_far_apart(vq, torch_dev, max_q, dtype, apart):
    """Columns 2^14 and 2^20 apart keep their own accuracy."""
    torch = torch_dev
    q, k, v, g, beta = _delta_inputs(torch, _t(torch, dtype), 180, 1, 2, 64, 72, 4)
    v[:, :, ::2] *= 2.0 ** (apart // 2)
    v[:, :, 1::2] *= 2.0 ** (apart // 2 - apart)
    state = _randn(torch, (1, 2, 64, 72), torch.float32, 8) * (v[0, 0].float().abs().clamp(min=2.0 ** -apart))
    _delta_check(vq, torch, dtype, [180], 1, 2, 64, 72, max_q, inputs=(q, k, v, g, beta), state=state)


@pytest.mark.parametrize("max_q", [16, 300])
@pytest.mark.parametrize("dtype", ["f16", "bf16"])
def test_delta_rule_large_values_that_decay_at_once(vq, torch_dev, max_q, dtype):
    """Tokens of 2^12 times the others' values, forgotten right behind."""
    torch = torch_dev
    q, k, v, g, beta = _delta_inputs(torch, _t(torch, dtype), 200, 1, 2, 64, 64, 5)
    for t in (0, 17, 63, 64, 100, 127):
        v[t] *= 4096.0
        g[t + 1] = -60.0
    _delta_check(vq, torch, dtype, [200], 1, 2, 64, 64, max_q, inputs=(q, k, v, g, beta))


@pytest.mark.parametrize("max_q", [16, 300])
@pytest.mark.parametrize("scale", [1e-6, 1.0, -300.0])
def test_delta_rule_scales(vq, torch_dev, max_q, scale):
    _delta_check(vq, torch_dev, "f16", [70, 100], 1, 2, 64, 64, max_q, scale=scale, std=0.1 if scale > 0 else 1e-2)


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("max_q", [16, 300])
@pytest.mark.parametrize("qstd,kstd", [(2.0 ** -10, 2.0 ** -4), (64.0, 1.0)])
def test_delta_rule_other_lengths_of_keys(vq, torch_dev, dtype, max_q, qstd, kstd):
    """Keys shorter than one and queries of any length."""
    torch = torch_dev
    q, k, v, g, beta = _delta_inputs(torch, _t(torch, dtype), 170, 2, 2, 128, 64, 6, 0.1)
    _delta_check(vq, torch, dtype, [100, 70], 2, 2, 128, 64, max_q, inputs=(q * qstd, k * kstd, v, g, beta))


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("max_q", [16, 300])
@pytest.mark.parametrize("what", ["k", "v", "q", "g", "beta"])
@pytest.mark.parametrize("bad", [math.nan, math.inf])
def test_delta_rule_values_that_are_not_finite(vq, torch_dev, dtype, max_q, what, bad):
    """They reach their own token and those behind (a query's: its token; a value's: its column), no other."""
    torch = torch_dev
    if what in "g" and bad == math.inf:
        pytest.skip("a decay above 1 without bound is no input")
    dt = _t(torch, dtype)
    q, k, v, g, beta = _delta_inputs(torch, dt, 150, 1, 2, 64, 72, 7)
    args = [x.cuda() for x in (q, k, v, g, beta)]
    op = vq.DeltaRule(1, 2, 64, 72)
    state = _randn(torch, (2, 2, 64, 72), torch.float32, 9).cuda()
    cu = _i(torch, [0, 110, 150])
    y0, s0 = op.forward(*args, state, cu, max_q=max_q)
    for t in (0, 5, 37, 70, 109):
        new = [x.clone() for x in args]
        cols = slice(None)
        hit = torch.zeros_like(y0, dtype=torch.bool)
        if what == "v":
            new[2][t, 1, 20] = bad
            hit[t:110, 1, 20] = True
        elif what == "k":
            new[1][t, 0, 9] = bad
            hit[t:110] = True
        elif what == "q":
            new[0][t, 0, 9] = bad
            hit[t] = True
        else:
            new[3 if what == "g" else 4][t, 1] = bad
            hit[t:110, 1] = True
        y, s = op.forward(*new, state, cu, max_q=max_q)
        assert torch.equal(y[~hit], y0[~hit]), t
        if what in ("v", "q"):  # an infinity may also stay one
            assert not y[hit].isfinite().any(), t
        else:
            assert y[hit].isnan().all() if bad != bad else not y[hit].isfinite().any(), t
        lost = torch.zeros_like(s0, dtype=torch.bool)
        if what == "v":
            lost[0, 1, :, 20] = True
        elif what == "k":
            lost[0] = True
        elif what != "q":
            lost[0, 1] = True
        assert torch.equal(s[~lost], s0[~lost]), t
        assert not s[lost].isfinite().any(), t


@pytest.mark.parametrize("hk,hv", [(3, 9), (16, 16), (5, 5)])
def test_delta_rule_many_heads_and_requests(vq, torch_dev, hk, hv):
    _delta_check(vq, torch_dev, "f16", [70, 3, 0, 65, 130, 64, 1, 257, 40], hk, hv, 24, 16, seed=5, pad=5)
    _delta_check(vq, torch_dev, "bf16", [400, 300], hk, hv, 16, 8, seed=6)


def test_delta_rule_many_requests_find_their_rows(vq, torch_dev):
    """More than 64 and more than 4096 requests in a launch, empty ones among them."""
    torch = torch_dev
    for R, seed in ((70, 1), (4500, 2)):
        lens = np.random.default_rng(seed).integers(0, 4, R).tolist()
        _delta_check(vq, torch, "f16", lens, 1, 1, 8, 8, 64, seed=seed, pad=3)


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("hk,hv,dk,dv", [(2, 24, 64, 40), (12, 12, 128, 128)])
def test_delta_rule_short_and_long_requests_together(vq, torch_dev, dtype, hk, hv, dk, dv):
    """Enough heads and requests that the short ones go token by token beside the others' chunks."""
    lens = [1, 0, 200, 1, 28, 29, 2, 64, 1, 0, 65, 3] + [1] * 20
    R, n = len(lens), len(lens) + 3
    index = [(11 * r + 2) % n for r in range(R)]  # 11 and n share no factor: no slot twice
    index[0], index[2], index[8] = -1, n, n + 5
    ctx = [r % 3 for r in range(R)]
    _delta_check(vq, torch_dev, dtype, lens, hk, hv, dk, dv, 200, ctx=ctx, index=index, n_states=n, pad=7)
    _delta_check(vq, torch_dev, dtype, lens, hk, hv, dk, dv, 200, ctx=ctx, in_place=True)
    lens = [1] * 63 + [70, 1, 41] + [2, 0] * 90 + [29, 40, 130] + [1] * 10  # more than 64 requests
    _delta_check(vq, torch_dev, dtype, lens, hk, hv, dk, dv, 200, in_place=True, pad=2)


def test_delta_rule_recurrence_and_chunks_agree_in_a_graph(vq, torch_dev):
    """Which requests are short may change between replays."""
    torch = torch_dev
    R, T = 40, 700
    op = vq.DeltaRule(4, 8, 64, 64)
    args = [x.cuda() for x in _delta_inputs(torch, torch.float16, T, 4, 8, 64, 64, 3)]
    state, s = torch.randn(R, 8, 64, 64, device="cuda"), torch.empty(R, 8, 64, 64, device="cuda")
    first, other = [1] * 39 + [661], [300, 361] + [1] * 37 + [0]
    cu, y = _i(torch, _starts(first)), torch.empty_like(args[2])
    work = torch.full((op.workspace_bytes(T, R, T),), 255, dtype=torch.uint8, device="cuda")
    op.forward(*args, state, cu, max_q=T, state_out=s, y=y, workspace=work)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        op.forward(*args, state, cu, max_q=T, state_out=s, y=y, workspace=work)
    for lens in (first, other, [17] * 40, first):
        cu.copy_(_i(torch, _starts(lens)))
        y.fill_(7.0)
        work.fill_(255)
        graph.replay()
        torch.cuda.synchronize()
        y1, s1 = op.forward(*args, state, cu, max_q=T)
        assert torch.equal(y, y1) and torch.equal(s, s1), lens
        assert (y[sum(lens):] == 0).all()


def test_delta_rule_more_threads_than_a_launch_holds(vq, torch_dev):
    """65,535 requests of 1,200 heads: 5.0e9 threads for the recurrence."""
    torch = torch_dev
    R, hv = 65535, 1200
    q, k, v, g, beta = _delta_inputs(torch, torch.float16, 3, 1, hv, 8, 8, 2)
    cu = torch.zeros(R + 1, dtype=torch.int32)
    cu[-1], cu[-2] = 3, 1  # the first token to the last request but one, two to the last
    op = vq.DeltaRule(1, hv, 8, 8)
    print("delta", R, hv, flush=True)
    y, _ = op.forward(*(x.cuda() for x in (q, k, v, g, beta)), torch.empty(0, hv, 8, 8, device="cuda"), cu.cuda(), max_q=4)
    state = torch.zeros(2, hv, 8, 8)
    ry, B, Z, _, _ = _delta_ref(torch, q, k, v, g, beta, state, [0, 1, 3], None, None, op.scale)
    u, c = _u(torch, torch.float16), 2 * (8 + 64) * W
    _close(torch, y, ry, u * ry.abs() + (2 * u + c) * B + c * Z + 2.0 ** -25, "y")


def test_delta_rule_strides_streams_and_graphs(vq, torch_dev):
    torch = torch_dev
    op = vq.DeltaRule(2, 4, 64, 64)
    for lens, max_q, other in (([3, 8, 1], 8, [8, 0, 4]), ([700, 30, 600], 700, [600, 700, 30])):
        T = sum(lens)
        q, k, v, g, beta = _delta_inputs(torch, torch.float16, T, 2, 4, 64, 64, 3)
        rows = torch.cat([q.flatten(1), k.flatten(1), v.flatten(1), torch.zeros(T, 8, dtype=q.dtype)], 1).cuda()
        wide = torch.cat([g, beta, g], 1).cuda()
        state = torch.randn(3, 4, 64, 64, device="cuda")
        cu = _i(torch, _starts(lens))
        args = [x.cuda() for x in (q, k, v, g, beta)]
        y, s = op.forward(*args, state, cu, max_q=max_q)
        views = (rows[:, :128].unflatten(1, (2, 64)), rows[:, 128:256].unflatten(1, (2, 64)),
                 rows[:, 256:512].unflatten(1, (4, 64)), wide[:, :4], wide[:, 4:8])
        y2, s2 = op.forward(*views, state, cu, max_q=max_q)
        assert torch.equal(y, y2) and torch.equal(s, s2)
        out = torch.full((T, 6, 64), 3.0, dtype=torch.float16, device="cuda")
        op.forward(*args, state, cu, max_q=max_q, y=out[:, 1:5])
        assert torch.equal(out[:, 1:5], y) and (out[:, 0] == 3).all() and (out[:, 5] == 3).all()
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        y3, s3 = op.forward(*args, state, cu, max_q=max_q, stream=side)
        torch.cuda.current_stream().wait_stream(side)
        assert torch.equal(y, y3) and torch.equal(s, s3)
        sout = torch.empty_like(s)
        work = torch.full((max(1, op.workspace_bytes(T, 3, max_q)),), 255, dtype=torch.uint8, device="cuda")
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            op.forward(*args, state, cu, max_q=max_q, state_out=sout, y=y2, workspace=work)
        for ls in (lens, other, lens):
            cu.copy_(_i(torch, _starts(ls)))
            graph.replay()
            torch.cuda.synchronize()
            y4, s4 = op.forward(*args, state, cu, max_q=max_q)
            assert torch.equal(y2, y4) and torch.equal(sout, s4), ls
        assert torch.equal(y2, y)


def _in_segments(vq, dtype, T, R, hk, hv, dk, dv, max_q):
    """Whether the workspace holds states and factors of segments besides the chunks' own."""
    chunks = T // 64 + R + 1
    own = chunks * (hv * 20480 + hk * (1 if dtype == "f16" else 2) * 64 * (64 if dk <= 64 else 128) * 2)
    return vq.DeltaRule(hk, hv, dk, dv).workspace_bytes(T, R, max_q) > own


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("lens,hk,hv,dk,dv,extra", [
    ([4000], 1, 1, 128, 128, {}),
    ([3001, 0, 1700, 1], 1, 2, 128, 72, dict(ctx=[5, 1, 0, 9], index=[4, 0, 2, 1], n_states=5, pad=70)),
    ([2560, 2560], 2, 2, 64, 64, dict(in_place=True)),
    ([64, 5000, 130], 1, 1, 40, 16, dict(in_place=True, ctx=[1, 0, 3], index=[2, -1, 0], n_states=3)),
    ([2113, 2049, 3071], 1, 2, 96, 104, dict(in_place=True)),
])
def test_delta_rule_segments(vq, torch_dev, dtype, lens, hk, hv, dk, dv, extra):
    """Few heads and long requests: segments of a request at once."""
    T = sum(lens) + extra.get("pad", 0)
    assert _in_segments(vq, dtype, T, len(lens), hk, hv, dk, dv, max(lens))
    _delta_check(vq, torch_dev, dtype, lens, hk, hv, dk, dv, max(lens), **extra)
    # said to be as long as one of them when they are not
    _delta_check(vq, torch_dev, dtype, lens, hk, hv, dk, dv, T, **extra)


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
def test_delta_rule_segments_decays_and_repeated_keys(vq, torch_dev, dtype):
    torch = torch_dev
    T = 4100
    q, k, v, g, beta = _delta_inputs(torch, _t(torch, dtype), T, 1, 4, 64, 64, 11)
    g[:, 0] = 0.0
    g[:, 1] = -100.0
    g[5::700, 2] = -math.inf
    g[2000:2070, 3] = -30.0
    beta[::3] = 0.0
    beta[1::3] = 1.0
    assert _in_segments(vq, dtype, T, 1, 1, 4, 64, 64, T)
    _delta_check(vq, torch, dtype, [T], 1, 4, 64, 64, T, inputs=(q, k, v, g, beta))
    k[:] = 0.0
    k[:, :, 3] = 1.0
    beta[:] = 1.0
    _delta_check(vq, torch, dtype, [T], 1, 4, 64, 64, T, inputs=(q, k, v, g, beta))


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("what", ["k", "v", "q", "g", "beta", "state"])
def test_delta_rule_segments_values_that_are_not_finite(vq, torch_dev, dtype, what):
    torch = torch_dev
    n, T = 2600, 4300
    q, k, v, g, beta = _delta_inputs(torch, _t(torch, dtype), T, 1, 2, 64, 72, 7)
    args = [x.cuda() for x in (q, k, v, g, beta, _randn(torch, (2, 2, 64, 72), torch.float32, 9))]
    op = vq.DeltaRule(1, 2, 64, 72)
    cu = _i(torch, [0, n, T])
    assert _in_segments(vq, dtype, T, 2, 1, 2, 64, 72, n)
    y0, s0 = op.forward(*args, cu, max_q=n)
    for t in (0, 1500, n - 1):
        new = [x.clone() for x in args]
        hit, lost = torch.zeros_like(y0, dtype=torch.bool), torch.zeros_like(s0, dtype=torch.bool)
        if what == "state":
            new[5][0, 1, 7, 20] = math.nan
            hit[:n, 1, 20] = lost[0, 1, :, 20] = True
        elif what == "v":
            new[2][t, 1, 20] = math.nan
            hit[t:n, 1, 20] = lost[0, 1, :, 20] = True
        elif what == "k":
            new[1][t, 0, 9] = math.nan
            hit[t:n] = lost[0] = True
        elif what == "q":
            new[0][t, 0, 9] = math.nan
            hit[t] = True
        else:
            new[3 if what == "g" else 4][t, 1] = math.nan
            hit[t:n, 1] = lost[0, 1] = True
        y, s = op.forward(*new, cu, max_q=n)
        assert torch.equal(y[~hit], y0[~hit]) and y[hit].isnan().all(), t
        assert torch.equal(s[~lost], s0[~lost]) and s[lost].isnan().all(), t


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
def test_delta_rule_segments_beside_short_requests(vq, torch_dev, dtype):
    lens = [1] * 30 + [3000] + [5, 0, 300] * 5
    R, n = len(lens), len(lens) + 1
    assert _in_segments(vq, dtype, sum(lens), R, 1, 6, 64, 64, 3000)
    index, ctx = [(5 * r + 3) % n for r in range(R)], [r % 4 for r in range(R)]  # 5 and 47 share no factor
    assert len(set(index)) == R
    _delta_check(vq, torch_dev, dtype, lens, 1, 6, 64, 64, 3000, ctx=ctx, index=index, n_states=n, pad=5)
    _delta_check(vq, torch_dev, dtype, lens, 1, 6, 64, 64, 3000, ctx=ctx, in_place=True)


@pytest.mark.parametrize("max_q", [1, 300])
def test_no_tokens_at_all(vq, torch_dev, max_q):
    """States pass through, or start from zero; nothing else happens."""
    torch = torch_dev
    _delta_check(vq, torch, "f16", [0, 0, 0], 2, 4, 64, 64, max_q, ctx=[1, 0, 2])
    _delta_check(vq, torch, "bf16", [0, 0], 2, 4, 64, 64, max_q, pad=70, in_place=True)
    conv = vq.ShortConv(torch.zeros(64, 4, dtype=torch.float16, device="cuda"))
    state = torch.randn(2, 3, 64, device="cuda").half()
    x = torch.empty(0, 64, dtype=torch.float16, device="cuda")
    y, new = conv.forward(x, state, _i(torch, [0, 0, 0]), ctx_len=_i(torch, [1, 0]))
    assert y.shape == (0, 64) and torch.equal(new[0], state[0]) and (new[1] == 0).all()


def test_delta_rule_segments_in_a_graph(vq, torch_dev):
    """A poisoned workspace, other lengths and values between the replays."""
    torch = torch_dev
    T, lens = 4200, [4200, 0]
    op = vq.DeltaRule(1, 2, 64, 64)
    args = [x.cuda() for x in _delta_inputs(torch, torch.bfloat16, T, 1, 2, 64, 64, 3)]
    state, cu = torch.randn(2, 2, 64, 64, device="cuda"), _i(torch, _starts(lens))
    work = torch.full((op.workspace_bytes(T, 2, T),), 255, dtype=torch.uint8, device="cuda")
    assert _in_segments(vq, "bf16", T, 2, 1, 2, 64, 64, T)
    y, s = torch.empty_like(args[2]), torch.empty_like(state)
    op.forward(*args, state, cu, max_q=T, state_out=s, y=y, workspace=work)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        op.forward(*args, state, cu, max_q=T, state_out=s, y=y, workspace=work)
    for ls in (lens, [1000, 3200], [0, 4200], [4100, 63]):
        cu.copy_(_i(torch, _starts(ls)))
        args[2].mul_(0.5)
        work.fill_(255)
        graph.replay()
        torch.cuda.synchronize()
        y1, s1 = op.forward(*args, state, cu, max_q=T)
        assert torch.equal(y, y1) and torch.equal(s, s1), ls


# ------------------------------------------------------------------ append


def _append_ref(torch, x, w, eps, off, freq, pos, next_):
    z = x.double()
    if w is not None:
        z = z / ((z * z).mean(-1, keepdim=True) + eps).sqrt() * (w.double() + off)
    half = len(freq)
    f = pos.double()[:, None] * freq.double()
    c, s = f.cos()[:, None], f.sin()[:, None]
    p = torch.arange(half)
    i, j = (2 * p, 2 * p + 1) if next_ else (p, p + half)
    out, size = z.clone(), z.abs()
    out[..., i], out[..., j] = z[..., i] * c - z[..., j] * s, z[..., j] * c + z[..., i] * s
    size[..., i] = size[..., j] = z[..., i].abs() + z[..., j].abs()
    return out, size


@pytest.mark.parametrize("dtype,T,heads,kv,D,rot,next_,norm,page", [
    ("f16", 1, 1, 1, 8, 8, False, False, 8), ("bf16", 7, 6, 2, 80, 80, False, True, 16),
    ("f16", 64, 5, 1, 128, 128, True, False, 32), ("bf16", 65, 4, 4, 256, 64, False, True, 64),
    ("f16", 300, 3, 3, 72, 24, False, True, 16), ("bf16", 130, 2, 1, 136, 0, False, True, 16),
    ("f16", 40, 9, 2, 64, 32, True, True, 1024), ("bf16", 33, 0, 2, 96, 96, True, False, 16),
    ("f16", 600, 40, 8, 128, 128, False, False, 16), ("bf16", 500, 24, 4, 256, 256, True, True, 64),
    ("f16", 9, 300, 70, 16, 8, False, True, 16),
    ("bf16", 1100, 24, 9, 256, 64, False, True, 64), ("f16", 1100, 17, 17, 256, 256, True, False, 16),
])
def test_paged_append(vq, torch_dev, dtype, T, heads, kv, D, rot, next_, norm, page):
    torch = torch_dev
    dt = _t(torch, dtype)
    n = -(-T // page) + 3
    gen = torch.Generator().manual_seed(T)
    slot = torch.randperm(n * page, generator=gen)[:T].to(torch.int32)
    pos = torch.randint(0, 200000, (T,), generator=gen).to(torch.int32)
    if T > 8:  # skipped, not stored, far
        slot[2], slot[4], slot[5], pos[6], pos[7] = -1, n * page, 2 ** 31 - 1, -1, -2 ** 31
        pos[0], pos[1], pos[8] = 0, 2 ** 31 - 1, 2 ** 24 + 1
    # queries interleaved with gates, keys and values in one wider row
    wide = _randn(torch, (T, max(heads, 1), 2 * D), dt, 5, 1.5).cuda()
    q = wide[:, :heads, :D] if heads else None
    rows = _randn(torch, (T, 2 * kv + 1, D), dt, 6, 1.5).cuda()
    k, v = rows[:, :kv], rows[:, kv:2 * kv]
    freq = (1e4 ** (-torch.arange(rot // 2).double() / max(1, rot // 2))).float()
    qw = _randn(torch, (D,), dt, 7, 0.2) if norm else None
    kw = _randn(torch, (D,), dt, 8, 0.2) if norm else None
    if norm or rot:
        rotary = vq.Rotary(freq.cuda() if rot else None, interleaved=next_, q_weight=qw.cuda() if norm else None,
                           k_weight=kw.cuda() if norm else None, eps=1e-5, weight_offset=1.0)
    cache = vq.PagedCache(torch.full((n, kv, page, D), 9.0, dtype=dt, device="cuda"),
                          torch.full((n, kv, D, page), 9.0, dtype=dt, device="cuda"))
    q_out = torch.full((T, heads, D), 7.0, dtype=dt, device="cuda") if heads else None
    print("append", dtype, T, heads, kv, D, rot, flush=True)
    got = cache.append(q, k, v, pos.cuda(), slot.cuda(), rotary, q_out=q_out)
    torch.cuda.synchronize()
    u = _u(torch, dt)
    live = pos >= 0
    if heads:
        ref, size = _append_ref(torch, q.cpu(), qw, 1e-5, 1.0, freq, pos, next_)
        ref[~live] = 7.0
        _close(torch, got, ref, u * ref.abs() + 32 * W * size + 2.0 ** -25, "q")
        assert got is q_out
    else:
        assert got is None
    ref, size = _append_ref(torch, k.cpu(), kw, 1e-5, 1.0, freq, pos, next_)
    ek, tol = torch.full(cache.k.shape, 9.0).double(), torch.zeros(cache.k.shape).double()
    ev = torch.full(cache.v.shape, 9.0, dtype=dt)
    for t, s in enumerate(slot.tolist()):
        if live[t] and 0 <= s < n * page:
            ek[s // page, :, s % page] = ref[t]
            tol[s // page, :, s % page] = u * ref[t].abs() + 32 * W * size[t] + 2.0 ** -25
            ev[s // page, :, :, s % page] = v[t].cpu()
    _close(torch, cache.k, ek, tol, "k")
    assert torch.equal(cache.v.cpu(), ev)


def test_paged_append_without_rotation_or_norm_is_store(vq, torch_dev):
    """One of the two norms alone: the other operand and the values are copied bit for bit, NaN among them."""
    torch = torch_dev
    dt, T = torch.float16, 50
    q, k, v = (_randn(torch, (T, h, 64), dt, h).cuda() for h in (4, 2, 2))
    k[3, 1, 5], v[7, 0, 2], v[9] = math.nan, math.inf, math.nan
    slot = torch.arange(T, dtype=torch.int32, device="cuda")
    pos = slot + 1000
    one, two = (vq.PagedCache(torch.zeros(4, 2, 16, 64, dtype=dt, device="cuda"),
                              torch.zeros(4, 2, 64, 16, dtype=dt, device="cuda")) for _ in range(2))
    one.store(k, v, slot)
    two.append(q, k, v, pos, slot, vq.Rotary(q_weight=torch.ones(64, dtype=dt, device="cuda")))
    same = lambda a, b: torch.equal(a.view(torch.int16), b.view(torch.int16))  # noqa: E731
    assert same(one.k.nan_to_num(5.0), two.k.nan_to_num(5.0)) and same(one.v, two.v)
    assert torch.equal(one.k.isnan(), two.k.isnan())


def test_paged_append_in_place_streams_and_graphs(vq, torch_dev):
    torch = torch_dev
    dt, T, h, kv, D = torch.bfloat16, 90, 6, 2, 128
    q0, k, v = (_randn(torch, (T, n, D), dt, n).cuda() for n in (h, kv, kv + 0))
    freq = torch.rand(32, device="cuda")
    w = (torch.rand(D, device="cuda") + 0.5).to(dt)
    rotary = vq.Rotary(freq, q_weight=w, k_weight=w)
    slot = torch.arange(T, dtype=torch.int32, device="cuda")
    pos = slot + 7

    def fresh():
        return vq.PagedCache(torch.zeros(8, kv, 16, D, dtype=dt, device="cuda"),
                             torch.zeros(8, kv, D, 16, dtype=dt, device="cuda"))

    cache = fresh()
    want = cache.append(q0, k, v, pos, slot, rotary)
    other = fresh()
    q = q0.clone()
    assert other.append(q, k, v, pos, slot, rotary, q_out=q) is q and torch.equal(q, want)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    third = fresh()
    side.wait_stream(torch.cuda.current_stream())
    got = third.append(q0, k, v, pos, slot, rotary, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    for c in (other, third):
        assert torch.equal(got, want) and torch.equal(c.k, cache.k) and torch.equal(c.v, cache.v)
    graph, replayed = torch.cuda.CUDAGraph(), fresh()
    with torch.cuda.graph(graph):
        replayed.append(q0, k, v, pos, slot, rotary, q_out=q)
    for shift in (0, 20, 0):
        pos.copy_(torch.arange(T, device="cuda") + 7 + shift)
        slot.copy_((torch.arange(T, device="cuda") + shift) % 128)
        replayed.k.zero_(), replayed.v.zero_()
        graph.replay()
        torch.cuda.synchronize()
        eager = fresh()
        want = eager.append(q0, k, v, pos, slot, rotary)
        assert torch.equal(q, want) and torch.equal(replayed.k, eager.k) and torch.equal(replayed.v, eager.v), shift


# ------------------------------------------------------------------ short convolution


def _conv_ref(torch, x, weight, bias, state, cu, ctx, index, silu, heads, dim, eps):
    T, C = x.shape
    taps, n_states = weight.shape[1], state.shape[0]
    y, tol = torch.zeros(T, C, dtype=torch.float64), torch.zeros(T, C, dtype=torch.float64)
    out, w = state.clone(), weight.double()
    for r in range(len(cu) - 1):
        s = r if index is None else index[r]
        if not 0 <= s < n_states:
            s = -1
        old = s >= 0 and (ctx is None or ctx[r] > 0)
        seq = torch.cat([state[s] if old else torch.zeros_like(state[0]), x[cu[r]:cu[r + 1]]])
        n = cu[r + 1] - cu[r]
        if s >= 0:
            out[s] = seq[n:]
        if not n:
            continue
        win = seq.double().unfold(0, taps, 1)
        z = (win * w[None]).sum(-1)
        d = (win * w[None]).abs().sum(-1)
        if bias is not None:
            z, d = z + bias.double(), d + bias.double().abs()
        d = (taps + 2) * W * d
        if silu:
            v = z * torch.sigmoid(z)
            d = 1.1 * d + v.abs() * (8 + 2 * z.abs()) * W
            z = v
        m = heads * dim
        if m:
            h, e = z[:, :m].reshape(n, heads, dim), d[:, :m].reshape(n, heads, dim)
            length = ((h * h).sum(-1, keepdim=True) + eps).sqrt()
            e = e / length + h.abs() / length * (e.norm(dim=-1, keepdim=True) / length + (dim + 8) * W)
            z[:, :m], d[:, :m] = (h / length).reshape(n, m), e.reshape(n, m)
        y[cu[r]:cu[r + 1]], tol[cu[r]:cu[r + 1]] = z, d
    return y, tol, out


def _conv_check(vq, torch, dtype, lens, C, taps, heads=0, dim=0, silu=True, bias=False, ctx=None, index=None,
                n_states=None, pad=0, in_place=False, seed=0, eps=1e-6):
    dt = _t(torch, dtype)
    cu = _starts(lens)
    T, R = cu[-1] + pad, len(lens)
    n_states = R if n_states is None else n_states
    x = _randn(torch, (T, C), dt, seed)
    weight = _randn(torch, (C, taps), dt, seed + 1, 0.6)
    b = _randn(torch, (C,), dt, seed + 2) if bias else None
    state = _randn(torch, (n_states, taps - 1, C), dt, seed + 3)
    print("conv", dtype, lens[:5], C, taps, heads, dim, flush=True)
    op = vq.ShortConv(weight.cuda(), None if b is None else b.cuda(), activation="silu" if silu else None,
                      unit_heads=heads, unit_dim=dim, eps=eps)
    sd = state.cuda()
    y, out = op.forward(x.cuda(), sd, _i(torch, cu), ctx_len=_i(torch, ctx), state_index=_i(torch, index),
                        state_out=sd if in_place else None)
    torch.cuda.synchronize()
    if not in_place:
        assert torch.equal(sd.cpu(), state)
    ry, tol, rs = _conv_ref(torch, x, weight, b, state, cu, ctx, index, silu, heads, dim, eps)
    n = cu[-1]
    _close(torch, y[:n], ry[:n], _u(torch, dt) * ry[:n].abs() + tol[:n] + 2.0 ** -25, "y")
    assert (y[n:] == 0).all()
    assert torch.equal(out.cpu(), rs)


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("taps", [2, 3, 4])
@pytest.mark.parametrize("C,heads,dim", [(8, 0, 0), (520, 0, 0), (1024, 8, 64), (600, 3, 96), (1240, 5, 136), (256, 1, 256),
                                         (200, 25, 8)])
def test_short_conv(vq, torch_dev, dtype, taps, C, heads, dim):
    _conv_check(vq, torch_dev, dtype, [1, 70, 0, 2, 33, 3], C, taps, heads, dim, bias=True, ctx=[1, 0, 5, 0, 2, 7])
    _conv_check(vq, torch_dev, dtype, [5], C, taps, heads, dim, silu=False, pad=40, in_place=True)


@pytest.mark.parametrize("in_place", [False, True])
def test_short_conv_states(vq, torch_dev, in_place):
    """Requests shorter than the filter keep part of their state; slots in any order, one outside."""
    for taps in (2, 4):
        _conv_check(vq, torch_dev, "f16", [1, 2, 0, 3, 9, 150], 72, taps, in_place=in_place, ctx=[1, 1, 1, 0, 0, 4])
        _conv_check(vq, torch_dev, "bf16", [1, 0, 2, 100], 72, taps, index=[4, 2, 9, 0], n_states=6, pad=1, in_place=in_place)


def test_short_conv_many_requests(vq, torch_dev):
    lens = np.random.default_rng(3).integers(0, 4, 4500).tolist()
    _conv_check(vq, torch_dev, "f16", lens, 16, 4)
    _conv_check(vq, torch_dev, "f16", [31, 32, 33, 64, 65, 500, 1] * 10, 40, 3)


@pytest.mark.parametrize("dtype,taps", [("f16", 2), ("bf16", 3), ("f16", 4), ("bf16", 4)])
@pytest.mark.parametrize("scale", [1, 3])
def test_short_conv_many_tokens(vq, torch_dev, dtype, taps, scale):
    """Units of several rounds of rows, ends inside a round and a unit."""
    lens = [683 * scale + 1, 0, 342 * scale, 15, 16, 17, 341 * scale + 3]
    _conv_check(vq, torch_dev, dtype, lens, 4104, taps, 4, 128, ctx=[1, 1, 0, 2, 0, 3, 1], in_place=True, pad=9)


def test_short_conv_large_inputs(vq, torch_dev):
    """SiLU of thousands, zero heads, and values that are not finite: they reach W tokens of their channel."""
    torch = torch_dev
    dt = torch.float16
    x = torch.zeros(9, 16, dtype=dt, device="cuda")
    x[:, 8:] = torch.tensor([3000.0, -3000.0, 1e-4, -1e-4, 20.0, -20.0, 88.0, -88.0], dtype=dt)
    w = torch.zeros(16, 4, dtype=dt, device="cuda")
    w[:, 3] = 1.0
    op = vq.ShortConv(w, unit_heads=1, unit_dim=8)
    y, _ = op.forward(x, op.state(1), _i(torch, [0, 9]))
    ref = x[:, 8:].double() * torch.sigmoid(x[:, 8:].double())
    assert (y[:, :8] == 0).all() and ((y[:, 8:].double() - ref).abs() <= 2.0 ** -11 * ref.abs() + 2.0 ** -24).all()
    w[:] = 0.5
    x[3, 9], x[4, 10] = math.inf, math.nan
    op = vq.ShortConv(w, activation=None)
    y, s = op.forward(x, op.state(1), _i(torch, [0, 9]))
    bad = ~y.isfinite()
    assert bad[3:7, 9].all() and bad[4:8, 10].all() and int(bad.sum()) == 8


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("W", [2, 3, 4])
def test_short_conv_few_tokens_in_place(vq, torch_dev, dtype, W):
    """A request's later tokens read its old state too, while its new one is written."""
    torch = torch_dev
    dt, C = _t(torch, dtype), 2048
    op = vq.ShortConv(_randn(torch, (C, W), dt, 1).cuda(), unit_heads=4, unit_dim=128)
    for lens in ([1], [2], [3], [5], [2, 3, 1, 8], [2] * 40, [3, 4] * 100):
        cu, T = _i(torch, _starts(lens)), sum(lens)
        x, state = _randn(torch, (T, C), dt, 2).cuda(), _randn(torch, (len(lens), W - 1, C), dt, 3).cuda()
        y, new = op.forward(x, state, cu)
        y1, same = op.forward(x, state, cu, state_out=state)
        assert same is state and torch.equal(y, y1) and torch.equal(state, new), lens


def test_short_conv_strides_streams_and_graphs(vq, torch_dev):
    torch = torch_dev
    lens, other, C = [40, 3, 90], [90, 0, 43], 640
    T = sum(lens)
    wide = _randn(torch, (T, C + 72), torch.bfloat16, 1).cuda()
    x = wide[:, 8:8 + C]
    weight = _randn(torch, (C, 4), torch.bfloat16, 2).cuda()
    op = vq.ShortConv(weight, unit_heads=2, unit_dim=128)
    state = _randn(torch, (3, 3, C), torch.bfloat16, 3).cuda()
    cu = _i(torch, _starts(lens))
    y, s = op.forward(x.contiguous(), state, cu)
    y2, s2 = op.forward(x, state, cu)
    assert torch.equal(y, y2) and torch.equal(s, s2)
    out = torch.full((T, C + 16), 3.0, dtype=torch.bfloat16, device="cuda")
    op.forward(x, state, cu, y=out[:, 8:8 + C])
    assert torch.equal(out[:, 8:8 + C], y) and (out[:, :8] == 3).all() and (out[:, 8 + C:] == 3).all()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    y3, s3 = op.forward(x, state, cu, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(y, y3) and torch.equal(s, s3)
    sout, graph = torch.empty_like(s), torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        op.forward(x, state, cu, y=y2, state_out=sout)
    for ls in (lens, other, lens):
        cu.copy_(_i(torch, _starts(ls)))
        graph.replay()
        torch.cuda.synchronize()
        y4, s4 = op.forward(x, state, cu)
        assert torch.equal(y2, y4) and torch.equal(sout, s4), ls


# ------------------------------------------------------------------ together


def test_mixer_ops_trace(vq, torch_dev, capfd, monkeypatch):
    torch = torch_dev
    monkeypatch.setenv("VQMLP_TRACE", "1")
    capfd.readouterr()
    h = torch.float16
    z = torch.zeros(2, 1, 64, dtype=h, device="cuda")
    cu = _i(torch, [0, 2])
    op = vq.ShortConv(torch.ones(64, 4, dtype=h, device="cuda"))
    op.forward(z.view(2, 64), op.state(1), cu)
    op = vq.DeltaRule(1, 1, 64, 64)
    f = torch.zeros(2, 1, device="cuda")
    op.forward(z, z, z, f, f, op.state(1), cu)
    cache = vq.PagedCache.empty(1, 1, 16, 64, h)
    cache.append(z, z, z, _i(torch, [0, 1]), _i(torch, [0, 1]), vq.Rotary(torch.ones(32, device="cuda")))
    torch.cuda.synchronize()
    lines = [x for x in capfd.readouterr().err.splitlines() if x.startswith("vqmlp: ")]
    assert len(lines) == 3 and "short_conv T=2" in lines[0] and "recurrence" in lines[1], lines
    assert "paged_append T=2 heads=1/1" in lines[2], lines
