"""GPU: linear attention where its sizes, decays and values lie far apart.

Tolerances.  u = 2^-11 (binary16) or 2^-8 (bfloat16) is one rounding, W = 2^-24 one of FP32.  z is the
output of the recurrence with absolute values.  An output is rounded once (u |y|); scores times decay
and the state as an operand are rounded once each (2 u z at most); FP32 sums and exponentials count 100 W
of z and a chunk's worth more for each 64 tokens (W / 16 a token).  2^-25 is half a step of the
smallest binary16.  The state is FP32: 100 W and W / 8 a token of its recurrence of absolute values.
"""
import math

import pytest

from test_gpu_block_ops import W, _close, _linear_ref, _randn, _t, _u, torch_dev, vq  # noqa: F401

pytestmark = pytest.mark.gpu


def _run(vq, torch, q, k, v, g, state, lens, max_q, scale=None):
    """The operator's outputs and state, checked against the 64-bit recurrence."""
    hk, dk, hv, dv = q.shape[1], q.shape[2], v.shape[1], v.shape[2]
    cu = [sum(lens[:i]) for i in range(len(lens) + 1)]
    op = vq.LinearAttention(hk, hv, dk, dv, scale)
    print("linear", q.dtype, lens, hk, hv, dk, dv, max_q, flush=True)
    y, out = op.forward(q.cuda(), k.cuda(), v.cuda(), g.cuda(), state.cuda(),
                        torch.tensor(cu, dtype=torch.int32, device="cuda"), max_q=max_q)
    torch.cuda.synchronize()
    ry, z, rs, size = _linear_ref(torch, q, k, v, g, state, cu, None, None, op.scale, len(lens))
    u, n = _u(torch, q.dtype), max(lens)
    _close(torch, y, ry, u * ry.abs() + (2 * u + (100 + n / 16) * W) * z + 2.0 ** -25, "y")
    _close(torch, out, rs, (100 + n / 8) * W * size + 2.0 ** -100, "state")
    return y, out


def _decays(torch, T, hv, seed):
    return -torch.rand((T, hv), generator=torch.Generator().manual_seed(seed)) * 0.1


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("max_q", [16, 200])
@pytest.mark.parametrize("std,vstd,scale", [(1e-3, 1000.0, None), (3e-3, 1000.0, None), (1e-4, 30000.0, 1.0),
                                            (30.0, 1.0, None), (150.0, 0.01, None), (1.0, 1.0, 1e-6),
                                            (0.1, 1.0, -1000.0)])
def test_scores_of_any_size(vq, torch_dev, dtype, max_q, std, vstd, scale):
    """Queries and keys from 1e-4 to 150: scores far below and above 1 keep the outputs' accuracy."""
    torch, dt, T = torch_dev, _t(torch_dev, dtype), 200
    q, k = _randn(torch, (T, 2, 128), dt, 1, std), _randn(torch, (T, 2, 128), dt, 2, std)
    v = _randn(torch, (T, 4, 64), dt, 3, vstd).clamp(-6e4, 6e4)
    state = _randn(torch, (2, 4, 128, 64), torch.float32, 4, 0.1 * std * vstd)
    _run(vq, torch, q, k, v, _decays(torch, T, 4, 5), state, [137, 63], max_q, scale)


@pytest.mark.parametrize("max_q", [16, 700])
@pytest.mark.parametrize("dk,dv", [(64, 64), (128, 128)])
def test_scores_that_change_size(vq, torch_dev, max_q, dk, dv):
    """Queries of one token in three 2^-12 of the others', and keys that go from 2^-10 to 2^5 and back
    from chunk to chunk, in segments too; values go the other way."""
    torch, dt, T = torch_dev, torch_dev.float16, 700
    q, k = _randn(torch, (T, 1, dk), dt, 1, dk ** -0.5), _randn(torch, (T, 1, dk), dt, 2, dk ** -0.5)
    v = _randn(torch, (T, 2, dv), dt, 3)
    q[::3] *= 2.0 ** -12
    for a, e in zip(range(0, T, 64), [0, -10, 5, 5, -10, -10, 0, 5, 0, -10, 0]):
        k[a:a + 64] *= 2.0 ** e
        v[a:a + 64] *= 2.0 ** -e
    _run(vq, torch, q, k, v, _decays(torch, T, 2, 5), torch.zeros(1, 2, dk, dv), [T], max_q, 64.0)


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("max_q", [16, 300])
@pytest.mark.parametrize("dv", [40, 64, 128])
@pytest.mark.parametrize("apart", [14, 20, 24])
def test_value_columns_far_apart(vq, torch_dev, dtype, max_q, dv, apart):
    """Columns 2^14 to 2^24 larger than their neighbours: each keeps its own accuracy, outputs and state."""
    torch, dt, T = torch_dev, _t(torch_dev, dtype), 300
    q, k = _randn(torch, (T, 1, 128), dt, 1, 1.0), _randn(torch, (T, 1, 128), dt, 2, 128 ** -0.5)
    v = _randn(torch, (T, 2, dv), dt, 3, 2.0 ** (12 - apart))
    state = _randn(torch, (1, 2, 128, dv), torch.float32, 4, 2.0 ** (10 - apart))
    for c in (3, dv // 2 + 1, dv - 1):
        v[:, :, c] *= 2.0 ** apart
        state[:, :, :, c] *= 2.0 ** apart
    _run(vq, torch, q, k, v, _decays(torch, T, 2, 5), state, [T], max_q, 1.0)


@pytest.mark.parametrize("max_q", [16, 1300])
def test_large_values_that_decay_at_once(vq, torch_dev, max_q):
    """A token of large values with strong decay behind it, once a chunk, leaves the small ones' accuracy."""
    torch, dt, T = torch_dev, torch_dev.float16, 1300
    q, k = _randn(torch, (T, 1, 64), dt, 1, 1.0), _randn(torch, (T, 1, 64), dt, 2, 0.125)
    v, g = _randn(torch, (T, 2, 64), dt, 3, 0.01), _decays(torch, T, 2, 5)
    v[10::64] *= 2.0 ** 20
    g[11::64] = -30.0
    _run(vq, torch, q, k, v, g, torch.zeros(1, 2, 64, 64), [T], max_q, 1.0)


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("lens,max_q", [([9, 30, 5], 16), ([9, 130, 70], 130), ([700, 900, 20], 900)])
def test_nan_decays_stay_nan(vq, torch_dev, dtype, lens, max_q):
    """A NaN decay: NaN in its head from that token on and in its state, nothing else changes."""
    torch, dt, T = torch_dev, _t(torch_dev, dtype), sum(lens)
    q, k = _randn(torch, (T, 2, 64), dt, 1, 0.125).cuda(), _randn(torch, (T, 2, 64), dt, 2, 0.125).cuda()
    v, g = _randn(torch, (T, 4, 64), dt, 3).cuda(), _decays(torch, T, 4, 5).cuda()
    state = _randn(torch, (3, 4, 64, 64), torch.float32, 4).cuda()
    cu = torch.tensor([sum(lens[:i]) for i in range(4)], dtype=torch.int32, device="cuda")
    op = vq.LinearAttention(2, 4, 64, 64)
    y, out = op.forward(q, k, v, g, state, cu, max_q=max_q)
    at = lens[0] + 2 * lens[1] // 3
    g[at, 2] = float("nan")
    y2, out2 = op.forward(q, k, v, g, state, cu, max_q=max_q)
    end = lens[0] + lens[1]
    assert y2[at:end, 2].isnan().all() and out2[1, 2].isnan().all()
    y2[at:end, 2], out2[1, 2] = y[at:end, 2], out[1, 2]
    assert torch.equal(y2, y) and torch.equal(out2, out)


@pytest.mark.parametrize("max_q", [16, 200])
@pytest.mark.parametrize("strong", [-math.inf, -79.37, -33.3])
def test_decays_behind_strong_ones(vq, torch_dev, max_q, strong):
    """Forty tokens that forget nearly everything, then weak decays: with one-hot keys and values each
    output is one score times its decay, rounded once, and 20 W for scale and exponential."""
    torch, T, n = torch_dev, 104, 64
    g = torch.full((T, 1), strong)
    g[40:, 0] = -0.02 * torch.rand(T - 40, generator=torch.Generator().manual_seed(3))
    q = torch.ones(T, 1, n, dtype=torch.float16)
    k, v = torch.zeros(T, 1, n, dtype=torch.float16), torch.zeros(T, 1, n, dtype=torch.float16)
    for j in range(n):
        k[40 + j, 0, j] = v[40 + j, 0, j] = 1.0
    i = lambda a: torch.tensor(a, dtype=torch.int32, device="cuda")  # noqa: E731
    # 64 tokens are one chunk: no state of a chunk before plays a part
    op = vq.LinearAttention(1, 1, n, n, 1.0)
    y, _ = op.forward(q[:64].cuda(), k[:64].cuda(), v[:64].cuda(), g[:64].cuda(), op.state(1), i([0, 64]), max_q=max_q)
    b = g[40:64, 0].double().cumsum(0)
    ref = torch.exp(b[:, None] - b[None, :]).tril()
    got = y[40:, 0, :24].double().cpu()
    _close(torch, got, ref, (2.0 ** -11 + 20 * W) * ref, "y")


@pytest.mark.parametrize("heads,dk,dv", [(48, 64, 128), (48, 64, 64), (4, 128, 128), (16, 40, 96)])
def test_workspaces_hold_for_both_types(vq, torch_dev, heads, dk, dv):
    """A workspace of workspace_bytes is large enough whichever 16-bit type the call has."""
    import ctypes as C

    torch = torch_dev
    torch.cuda.init()
    op = vq.LinearAttention(heads, heads, dk, dv)
    for T in list(range(100, 4000, 100)) + [5000, 8000, 12000, 20000, 40000]:
        for R in (1, 2, 5):
            have = op.workspace_bytes(T, R, T)
            for dtype in (0, 1):
                n = C.c_size_t()
                assert vq.lib().vqmlp_linear_attn_workspace(C.byref(op._desc(dtype, T, R, 0, T)), C.byref(n)) == 0
                assert n.value <= have, (T, R, dtype)


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("what", ["nan", "inf"])
@pytest.mark.parametrize("lens,max_q", [([9, 30, 5], 16), ([9, 130, 70], 130), ([700, 900, 20], 900)])
@pytest.mark.parametrize("dk,dv", [(64, 64), (128, 72)])
def test_values_that_are_not_finite_stay_behind_their_token(vq, torch_dev, dtype, what, lens, max_q, dk, dv):
    """A NaN or infinity in v: in its column no number from that token on and in the state; nothing else
    changes.  The same for a whole key, in every column of the heads that read it."""
    torch, dt, T = torch_dev, _t(torch_dev, dtype), sum(lens)
    q, k = _randn(torch, (T, 2, dk), dt, 1, 0.125).cuda(), _randn(torch, (T, 2, dk), dt, 2, 0.125).cuda()
    v, g = _randn(torch, (T, 4, dv), dt, 3).cuda(), _decays(torch, T, 4, 5).cuda()
    state = _randn(torch, (3, 4, dk, dv), torch.float32, 4).cuda()
    cu = torch.tensor([sum(lens[:i]) for i in range(4)], dtype=torch.int32, device="cuda")
    op = vq.LinearAttention(2, 4, dk, dv)
    y, out = op.forward(q, k, v, g, state, cu, max_q=max_q)
    end = lens[0] + lens[1]
    for at in (lens[0], lens[0] + 1, lens[0] + 2 * lens[1] // 3, end - 2, end - 1):
        print("linear", dtype, lens, max_q, what, at, flush=True)
        for col in (0, 5, dv - 1):
            w = v.clone()
            w[at, 2, col] = float(what)
            y2, out2 = op.forward(q, k, w, g, state, cu, max_q=max_q)
            assert not y2[at:end, 2, col].isfinite().any() and not out2[1, 2, :, col].isfinite().any()
            y2[at:end, 2, col], out2[1, 2, :, col] = y[at:end, 2, col], out[1, 2, :, col]
            assert torch.equal(y2, y) and torch.equal(out2, out)
        w = k.clone()
        w[at, 1] = float(what)
        y2, out2 = op.forward(q, w, v, g, state, cu, max_q=max_q)
        assert not y2[at:end, 2:].isfinite().any() and not out2[1, 2:].isfinite().any()
        y2[at:end, 2:], out2[1, 2:] = y[at:end, 2:], out[1, 2:]
        assert torch.equal(y2, y) and torch.equal(out2, out)
