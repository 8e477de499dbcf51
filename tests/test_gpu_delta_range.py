"""GPU: the gated delta rule at the ends of its ranges, token by token (max_q 16) and in chunks (300).

Tolerances.  u = eps / 2 of the 16-bit type is one rounding, W = 2^-24 one of FP32.  A token adds to a column of
the state at most C W (|S'| + a), a = |k| beta (|v| + |k| |S'|): its own sums and, in chunks, those of the
triangular system, C = 2 (Dk + 64).  Z sums that up with the decays, B the lengths |k| |u| that a column is made of.
Chunks of 64 tokens have one unit for all updates of a column: their largest is at least 2^5 2^-4 in it, and a binary16 part's
last bit is 2^-24, so where tokens of a chunk differ a is the largest |k| beta times the largest |v| + |k| |S'|.
An output adds C W scale |q| (B + Z) and its one rounding.
"""
import math

import pytest

from test_gpu_block_ops import _close, _randn, _t, _u, torch_dev, vq  # noqa: F401
from test_gpu_mixer_ops import W, _delta_inputs, _i, _starts

pytestmark = pytest.mark.gpu

TINY = {"f16": 2.0 ** -25, "bf16": 2.0 ** -134}  # half a step of the smallest outputs


def _ref(torch, q, k, v, g, beta, state, cu, scale, chunks=False):
    """Outputs, their bounds B and Z, states and theirs, in 64 bits."""
    T, hk, dk = q.shape
    hv, dv = v.shape[1:]
    y, yb = torch.zeros(T, hv, dv).double(), torch.zeros(T, hv, dv).double()
    out, sb = torch.zeros(state.shape).double(), torch.zeros(state.shape).double()
    kd, qd = (x.double().repeat_interleave(hv // hk, 1) for x in (k, q))
    vd, e, bd = v.double(), torch.exp(g.double().clamp(min=-80.0))[..., None], beta.double()[..., None]
    for r in range(len(cu) - 1):
        S = state[r].double().clone()
        B = S.norm(dim=1)
        Z = torch.zeros_like(B)
        for t in range(cu[r], cu[r + 1]):
            if chunks and (t - cu[r]) % 64 == 0:
                c = slice(t, min(t + 64, cu[r + 1]))
                lengths = kd[c].norm(dim=2)[..., None]
                most = (lengths * bd[c]).amax(0) * (vd[c].abs().amax(0) + lengths.amax(0) * S.norm(dim=1))
            S = e[t][..., None] * S
            length = kd[t].norm(dim=1)[:, None]
            u = bd[t] * (vd[t] - (S * kd[t][..., None]).sum(1))
            s = S.norm(dim=1)
            Z = e[t] * Z + s + (most if chunks else length * bd[t] * (vd[t].abs() + length * s))
            B = e[t] * B + length * u.abs()
            S = S + kd[t][:, :, None] * u[:, None, :]
            y[t] = scale * (S * qd[t][..., None]).sum(1)
            yb[t] = abs(scale) * qd[t].norm(dim=1)[:, None] * (B + Z)
        out[r], sb[r] = S, Z[:, None].expand_as(S)
    return y, yb, out, sb


def _check(vq, torch, dtype, lens, args, max_q, state=None, scale=None, work=None, chunks=False):
    q, k, v, g, beta = args
    hk, dk, hv, dv = q.shape[1], q.shape[2], v.shape[1], v.shape[2]
    cu = _starts(lens)
    if state is None:
        state = torch.zeros(len(lens), hv, dk, dv)
    op = vq.DeltaRule(hk, hv, dk, dv, scale)
    print("delta", dtype, lens, hk, hv, dk, dv, max_q, flush=True)
    y, out = op.forward(*(x.cuda() for x in args), state.cuda(), _i(torch, cu), max_q=max_q, workspace=work)
    torch.cuda.synchronize()
    ry, yb, rs, sb = _ref(torch, *args, state, cu, op.scale, chunks)
    c = 2 * (dk + 64) * W
    _close(torch, y, ry, _u(torch, _t(torch, dtype)) * ry.abs() + c * yb + TINY[dtype], "y")
    _close(torch, out, rs, c * sb + 2.0 ** -148, "state")
    return y, out, ry


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("lens,hk,hv,dk,dv,max_q", [
    ([150, 201], 2, 4, 64, 64, 16), ([150, 201], 2, 4, 64, 64, 300), ([400], 1, 3, 128, 128, 400), ([333, 64], 2, 2, 96, 72, 333),
    ([2600], 1, 1, 64, 64, 2600),
])
def test_outputs_are_rounded_once(vq, torch_dev, dtype, lens, hk, hv, dk, dv, max_q):
    """Many outputs are as far from the exact ones as those are from their own rounding; what the sums in front add is
    independent of it, and its root mean square grows with the root of the number of terms: 4 sqrt(Dk + 64) W of
    scale |q| |S|, so much for each of the tokens that a state of these decays remembers."""
    torch = torch_dev
    dt = _t(torch, dtype)
    args = _delta_inputs(torch, dt, sum(lens), hk, hv, dk, dv, 21)
    state = _randn(torch, (len(lens), hv, dk, dv), torch.float32, 22, 0.5)
    y, _, ry = _check(vq, torch, dtype, lens, args, max_q, state)
    own = (ry.to(dt).double() - ry).norm()
    # |S| of a column from |y|: queries point anywhere, so |y| = scale |q| |S| / sqrt(Dk) in the mean
    added = 4 * math.sqrt(dk + 64) * W * math.sqrt(dk) * ry.norm()
    err = (y.cpu().double() - ry).norm()
    print("%.4e of %.4e, %.1e" % (err / ry.norm(), own / ry.norm(), added / ry.norm()), flush=True)
    assert err <= (own * own + added * added).sqrt()


@pytest.mark.parametrize("max_q", [16, 300])
@pytest.mark.parametrize("power", [-120, -90, -30, 30, 80, 120])
def test_bfloat16_queries_of_any_length(vq, torch_dev, power, max_q):
    torch = torch_dev
    q, k, v, g, beta = _delta_inputs(torch, torch.bfloat16, 170, 2, 2, 64, 64, 34)
    q = (q.double() * 2.0 ** power).to(torch.bfloat16)
    state = _randn(torch, (1, 2, 64, 64), torch.float32, 35)
    _check(vq, torch, "bf16", [170], (q, k, v, g, beta), max_q, state)


@pytest.mark.parametrize("max_q", [16, 300])
def test_bfloat16_queries_of_the_largest_elements(vq, torch_dev, max_q):
    torch = torch_dev
    # v and the state below 2^-1, so that a row of the state times 1.5 2^127 is an FP32 number
    q, k, v, g, beta = _delta_inputs(torch, torch.bfloat16, 100, 1, 1, 64, 64, 36, 2.0 ** -4)
    q = torch.zeros_like(q)
    t = torch.arange(100)
    q[t, 0, t % 64] = 1.5 * 2.0 ** 127
    _check(vq, torch, "bf16", [100], (q, k, v, g, beta), max_q, _randn(torch, (1, 1, 64, 64), torch.float32, 37, 2.0 ** -4), scale=2.0 ** -8)


@pytest.mark.parametrize("max_q", [16, 300])
@pytest.mark.parametrize("apart", [20, 26])
def test_bfloat16_query_elements_far_apart(vq, torch_dev, apart, max_q):
    """Each query's largest element meets a row of the state that is zero; the others are 2^-apart of it.  What is left
    of an element is off by at most 2^-40 of the largest."""
    torch = torch_dev
    q, k, v, g, beta = _delta_inputs(torch, torch.bfloat16, 150, 1, 2, 64, 64, 38)
    k[:, :, 0] = 0.0
    q *= 2.0 ** -apart
    q[:, :, 0] = 0.0
    state = _randn(torch, (1, 2, 64, 64), torch.float32, 39)
    state[:, :, 0] = 0.0
    ry, yb, _, _ = _ref(torch, q, k, v, g, beta, state, [0, 150], 1.0)
    q[:, :, 0] = 1.0
    y, _ = vq.DeltaRule(1, 2, 64, 64, 1.0).forward(*(x.cuda() for x in (q, k, v, g, beta)), state.cuda(), _i(torch, [0, 150]),
                                                   max_q=max_q)
    # the sum of a column's magnitudes is at most sqrt(64) times its length, and B is no less than that
    length = q[:, :, 1:].double().norm(dim=2)[..., None]
    _close(torch, y, ry, 2.0 ** -8 * ry.abs() + 2 * 128 * W * yb + 2.0 ** -40 * 8 * yb / length + TINY["bf16"], "y")


def _updates(torch, dtype, what, seed):
    """Inputs whose updates |k| beta are small or whose keys are long, from a state of zeros."""
    dt = _t(torch, dtype)
    q, k, v, g, beta = _delta_inputs(torch, dt, 150, 1, 2, 128, 72, seed)
    if what[0] == "k":
        k = (k.double() * 2.0 ** what[1]).to(dt)
    elif what[0] == "beta":
        beta = beta * 2.0 ** what[1]
    elif what[0] == "long":  # each key orthogonal to the others, so that nothing grows
        k = torch.zeros_like(k)
        t = torch.arange(128)
        k[t, 0, (37 * t) % 128] = 2.0 ** what[1]
        beta = (beta * 2.0 ** what[2]).clone()
        beta[128:] = 0
    return q, k, v, g, beta


@pytest.mark.parametrize("max_q", [16, 300])
@pytest.mark.parametrize("dtype,what", [
    ("bf16", ("k", -15)), ("bf16", ("k", -25)), ("bf16", ("k", -36)), ("bf16", ("k", -60)), ("f16", ("k", -9)),
    ("bf16", ("beta", -12)), ("bf16", ("beta", -28)), ("f16", ("beta", -28)), ("f16", ("beta", -50)),
    ("bf16", ("long", 6, 0)), ("bf16", ("long", 30, 0)), ("bf16", ("long", 100, -95)), ("bf16", ("long", 127, -120)),
    ("f16", ("long", 6, 0)), ("f16", ("long", 12, 0)),
])
def test_updates_of_any_size(vq, torch_dev, dtype, what, max_q):
    """From a state of zeros the updates are all that the state holds.  binary16 outputs of small ones are lifted by
    the scale."""
    small = min(0, what[1]) if dtype == "f16" else 0
    _check(vq, torch_dev, dtype, [150], _updates(torch_dev, dtype, what, 31), max_q, scale=2.0 ** (-small - 4))


@pytest.mark.parametrize("max_q", [16, 300])
@pytest.mark.parametrize("dtype", ["f16", "bf16"])
def test_chunks_of_other_sizes(vq, torch_dev, dtype, max_q):
    """Chunks of ordinary, small and no updates by turns, and keys of zero between short ones."""
    torch = torch_dev
    q, k, v, g, beta = _delta_inputs(torch, _t(torch, dtype), 500, 1, 2, 64, 64, 32)
    beta[64:140] *= 2.0 ** -20
    beta[200:270] = 0.0
    beta[330:400, 0] *= 2.0 ** -40
    beta[330:400, 1] *= 1e-37
    if dtype == "bf16":
        k[64:100] *= 2.0 ** -12
        k[270:300] *= 2.0 ** -20
        k[405:470] *= 2.0 ** -33
    k[::5] = 0.0
    state = _randn(torch, (2, 2, 64, 64), torch.float32, 33)
    state[1] = 0.0
    _check(vq, torch, dtype, [280, 220], (q, k, v, g, beta), max_q, state)


@pytest.mark.parametrize("max_q", [16, 300])
@pytest.mark.parametrize("apart", [20, 26])
def test_bfloat16_key_elements_far_apart(vq, torch_dev, apart, max_q):
    """The elements of a key that are 2^-apart of its largest meet rows of the state 2^apart times the others'."""
    torch = torch_dev
    q, k, v, g, beta = _delta_inputs(torch, torch.bfloat16, 150, 1, 2, 64, 64, 40)
    state = _randn(torch, (1, 2, 64, 64), torch.float32, 41)
    k[:, :, 32:] *= 2.0 ** -apart
    state[:, :, 32:] *= 2.0 ** apart
    _check(vq, torch, "bf16", [150], (q, k, v, g, beta), max_q, state)


@pytest.mark.parametrize("max_q", [16, 300])
@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("what", ["k", "v", "beta", "state"])
@pytest.mark.parametrize("bad", [math.nan, math.inf, -math.inf])
def test_what_is_not_finite_gives_nan(vq, torch_dev, dtype, max_q, what, bad):
    torch = torch_dev
    args = [x.cuda() for x in _delta_inputs(torch, _t(torch, dtype), 150, 1, 2, 64, 72, 7)]
    op = vq.DeltaRule(1, 2, 64, 72)
    state = _randn(torch, (2, 2, 64, 72), torch.float32, 9).cuda()
    cu = _i(torch, [0, 110, 150])
    y0, s0 = op.forward(*args, state, cu, max_q=max_q)
    for t in (0, 5, 63, 64, 109):
        new, start = [x.clone() for x in args], state.clone()
        hit, lost = torch.zeros_like(y0, dtype=torch.bool), torch.zeros_like(s0, dtype=torch.bool)
        if what == "v":
            new[2][t, 1, 20] = bad
            hit[t:110, 1, 20] = lost[0, 1, :, 20] = True
        elif what == "k":
            new[1][t, 0, 9] = bad
            hit[t:110] = lost[0] = True
        elif what == "beta":
            new[4][t, 1] = bad
            hit[t:110, 1] = lost[0, 1] = True
        else:
            start[0, 1, t % 64, 20] = bad
            hit[:110, 1, 20] = lost[0, 1, :, 20] = True
        y, s = op.forward(*new, start, cu, max_q=max_q)
        assert torch.equal(y[~hit], y0[~hit]) and y[hit].isnan().all(), t
        assert torch.equal(s[~lost], s0[~lost]) and s[lost].isnan().all(), t


@pytest.mark.parametrize("max_q", [16, 300])
@pytest.mark.parametrize("dtype", ["f16", "bf16"])
def test_closed_gates(vq, torch_dev, dtype, max_q):
    """A state that only decays, while the values go on: its outputs are measured by it alone."""
    torch = torch_dev
    q, k, v, g, beta = _delta_inputs(torch, _t(torch, dtype), 280, 1, 2, 64, 64, 44)
    beta[70:, 0] = 0.0
    beta[:, 1] = 0.0
    g[:, 1] *= 0.1
    state = _randn(torch, (1, 2, 64, 64), torch.float32, 45)
    state[:, 1] *= 2.0 ** -30
    for h, scale in ((0, None), (1, 2.0 ** 20)):  # of each within binary16
        _check(vq, torch, dtype, [280], (q, k, *(x[:, h:h + 1].clone() for x in (v, g, beta))), max_q, state[:, h:h + 1].clone(),
               scale=scale)


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
def test_segments_of_other_sizes(vq, torch_dev, dtype):
    """Units that change from chunk to chunk inside segments and at their ends, from a state of zeros and from another."""
    torch = torch_dev
    T = 4000
    q, k, v, g, beta = _delta_inputs(torch, _t(torch, dtype), T, 1, 2, 64, 64, 42)
    for at in range(0, T, 500):
        beta[at:at + 130] *= 2.0 ** -(at // 100)
        if dtype == "bf16":
            k[at + 200:at + 330] *= 2.0 ** -(at // 100)
    beta[700:1400, 1] = 0.0
    assert vq.DeltaRule(1, 2, 64, 64).workspace_bytes(T, 1, T) > (T // 64 + 2) * (26624 * 2 + 16384)
    for state in (None, _randn(torch, (1, 2, 64, 64), torch.float32, 43)):
        _check(vq, torch, dtype, [T], (q, k, v, g, beta), T, state, chunks=True)


# ------------------------------------------------------------------ workspaces


def _trace(capfd):
    return [x for x in capfd.readouterr().err.splitlines() if "delta_rule" in x]


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
def test_one_workspace_for_smaller_calls(vq, torch_dev, dtype, capfd, monkeypatch):
    """The size for the most tokens, requests and max_q holds for every call with no more of each, also where that
    call by itself would ask for more."""
    torch = torch_dev
    monkeypatch.setenv("VQMLP_TRACE", "1")
    op = vq.DeltaRule(2, 6, 64, 64)
    for most, lens, max_q in (((4000, 4, 4000), [2000, 2000], 2000), ((900, 4, 900), [130, 70], 130),
                              ((1280, 64, 32), [32, 32], 32), ((1280, 64, 32), [20, 32, 1], 25)):
        work = torch.full((op.workspace_bytes(*most),), 255, dtype=torch.uint8, device="cuda")
        args = _delta_inputs(torch, _t(torch, dtype), sum(lens), 2, 6, 64, 64, 51)
        capfd.readouterr()
        _check(vq, torch, dtype, lens, args, max_q, _randn(torch, (len(lens), 6, 64, 64), torch.float32, 52), work=work)
        print(most, lens, op.workspace_bytes(sum(lens), len(lens), max_q), len(work), _trace(capfd), flush=True)


def test_sizes_of_smaller_calls_are_accepted(vq, torch_dev):
    """Sizes drawn over the whole range, each called with the workspace of a description that is no smaller in anything.
    Nothing but zeros: no request has a token."""
    import random

    torch = torch_dev
    rng = random.Random(5)
    for _ in range(60):
        hk, rep = rng.choice([1, 2, 4]), rng.choice([1, 2, 3])
        op = vq.DeltaRule(hk, hk * rep, 8, 8)
        T, R, m = rng.randint(1, 6000), rng.randint(1, 300), rng.randint(1, 6000)
        need = op.workspace_bytes(T, R, m)
        t, r, n = rng.randint(1, T), rng.randint(1, R), rng.randint(1, m)
        q, v, g = (torch.zeros(s, device="cuda", dtype=d) for s, d in (
            ((t, hk, 8), torch.bfloat16), ((t, hk * rep, 8), torch.bfloat16), ((t, hk * rep), torch.float32)))
        print("delta", hk, rep, (T, R, m), (t, r, n), need, flush=True)
        y, s = op.forward(q, q, v, g, g, torch.ones(r, hk * rep, 8, 8, device="cuda"), _i(torch, [0] * (r + 1)), max_q=n,
                          workspace=torch.empty(max(1, need), dtype=torch.uint8, device="cuda"))
        assert (y == 0).all() and (s == 1).all()


def test_a_small_workspace_is_refused(vq, torch_dev):
    torch = torch_dev
    op = vq.DeltaRule(1, 2, 64, 64)
    args = [x.cuda() for x in _delta_inputs(torch, torch.bfloat16, 300, 1, 2, 64, 64, 53)]  # the larger of both types' sizes
    cu, state = _i(torch, [0, 300]), torch.zeros(1, 2, 64, 64, device="cuda")
    need = op.workspace_bytes(300, 1, 300)
    assert need > 0
    with pytest.raises(vq.VqmlpError, match="needs"):
        op.forward(*args, state, cu, max_q=300, workspace=torch.empty(need - 256, dtype=torch.uint8, device="cuda"))
    y, s = op.forward(*args, state, cu, max_q=300, workspace=torch.empty(need, dtype=torch.uint8, device="cuda"))
    assert all(torch.equal(a, b) for a, b in zip((y, s), op.forward(*args, state, cu, max_q=300)))


@pytest.mark.parametrize("lens,hk,hv,dk,dv", [([4000], 1, 1, 128, 128), ([3001, 0, 1700, 1], 1, 2, 128, 72), ([2560, 2560], 2, 2, 64, 64),
                                              ([64, 5000, 130], 1, 1, 40, 16), ([2113, 2049, 3071], 1, 2, 96, 104)])
def test_which_calls_take_segments(vq, torch_dev, lens, hk, hv, dk, dv, capfd, monkeypatch):
    """Few heads and long requests do, with a workspace that holds them; a workspace for the chunks alone is enough."""
    torch = torch_dev
    monkeypatch.setenv("VQMLP_TRACE", "1")
    T, R = sum(lens), len(lens)
    args = [x.cuda() for x in _delta_inputs(torch, torch.bfloat16, T, hk, hv, dk, dv, 54)]
    op, cu, state = vq.DeltaRule(hk, hv, dk, dv), _i(torch, _starts(lens)), torch.zeros(R, hv, dk, dv, device="cuda")
    chunks = (T // 64 + R + 1) * (26624 * hv + 8192 * (1 if dk <= 64 else 2) * 2 * hk)
    assert op.workspace_bytes(T, R, max(lens)) > chunks
    capfd.readouterr()
    got = [op.forward(*args, state, cu, max_q=max(lens), workspace=w) for w in (
        None, torch.full((chunks,), 255, dtype=torch.uint8, device="cuda"))]
    torch.cuda.synchronize()
    assert ["join" in x for x in _trace(capfd)] == [True, False]
    # both within a rounding of the same values
    (y, s), (y1, s1) = got
    assert (s - s1).norm() <= 1e-5 * s.norm() and (y.float() - y1.float()).norm() <= 2.0 ** -8 * y.float().norm()
