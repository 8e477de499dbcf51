"""CPU tests of the operators in front of and inside the mixers: every refusal that the host half makes,
through the C ABI, before any device call; and the binding's own checks."""
import ctypes as C

import pytest

BUF = C.create_string_buffer(4096 + 256)
PTR = (C.addressof(BUF) + 255) // 256 * 256  # never dereferenced: every call here is refused first


@pytest.fixture(scope="module")
def vq():
    from bit_vector_lut_amd import vqmlp

    vqmlp.lib()
    return vqmlp


def _refused(vq, status, text, want=1):
    assert status == want, (status, vq.lib().vqmlp_last_error())
    assert text in vq.lib().vqmlp_last_error().decode(), vq.lib().vqmlp_last_error()


def _delta(vq, **kw):
    d = dict(dtype=0, T=20, R=2, k_heads=2, v_heads=4, Dk=64, Dv=32, n_states=2, max_q=20, scale=0.125, ld_q=128,
             ld_k=128, ld_v=128, ld_y=128, ld_g=4, ld_beta=4, q=PTR, k=PTR, v=PTR, g=PTR, beta=PTR, y=PTR,
             state_in=PTR, state_out=PTR, cu_q=PTR)
    d.update(kw)
    return vq._DeltaDesc(**d)


@pytest.mark.parametrize("kw,text,want", [
    (dict(dtype=2), "dtype", 1), (dict(T=-1), "out of range", 1), (dict(R=0), "out of range", 1),
    (dict(max_q=-1), "out of range", 1), (dict(v_heads=5), "no multiple", 1), (dict(Dk=136), "Dk=136", 1),
    (dict(Dk=12), "Dk=12", 1), (dict(Dv=4), "Dv=4", 1), (dict(R=65536), "65535", 2), (dict(T=1 << 30), "2^30", 2),
    (dict(scale=float("nan")), "scale", 1), (dict(scale=float("inf")), "scale", 1), (dict(cu_q=None), "cu_q", 1),
    (dict(state_in=None), "null state", 1), (dict(state_out=None), "null state", 1), (dict(state_out=PTR + 4), "16-byte", 1),
    (dict(g=None), "null", 1), (dict(beta=None), "null", 1), (dict(v=PTR + 8), "16-byte", 1), (dict(beta=PTR + 2), "4-byte", 1),
    (dict(ld_k=120), "strides", 1), (dict(ld_q=132), "strides", 1), (dict(ld_g=3), "strides", 1),
    (dict(ld_beta=3), "strides", 1), (dict(ld_v=(1 << 24) + 8), "2^24", 1), (dict(ld_beta=(1 << 24) + 1), "2^24", 1),
])
def test_delta_rule_refusals(vq, kw, text, want):
    _refused(vq, vq.lib().vqmlp_delta_rule(C.byref(_delta(vq, **kw)), None, 0, None), text, want)


def _conv(vq, **kw):
    d = dict(dtype=0, T=5, R=2, C=64, W=4, silu=1, unit_heads=2, unit_dim=16, n_states=2, eps=1e-6, ld_x=64, ld_y=64, x=PTR,
             weight=PTR, y=PTR + 256, state_in=PTR, state_out=PTR, cu_q=PTR)
    d.update(kw)
    return vq._ConvDesc(**d)


@pytest.mark.parametrize("kw,text,want", [
    (dict(dtype=2), "dtype", 1), (dict(T=-1), "out of range", 1), (dict(R=0), "out of range", 1), (dict(C=60), "C=60", 1),
    (dict(C=0), "C=0", 1), (dict(W=1), "W=1", 1), (dict(W=5), "W=5", 1), (dict(R=65536), "65535", 2), (dict(T=1 << 30), "2^30", 2),
    (dict(C=(1 << 20) + 8), "2^20", 2), (dict(unit_dim=12), "unit_dim=12", 1), (dict(unit_dim=264), "unit_dim=264", 1),
    (dict(unit_heads=5), "pass C", 1), (dict(unit_heads=-1), "out of range", 1), (dict(unit_heads=1 << 28), "pass C", 1),
    (dict(eps=-1.0), "eps", 1), (dict(eps=float("nan")), "eps", 1), (dict(cu_q=None), "cu_q", 1), (dict(cu_q=PTR + 2), "cu_q", 1),
    (dict(state_in=None), "null state", 1), (dict(state_out=PTR + 8), "16-byte", 1), (dict(weight=None), "weight", 1),
    (dict(bias=PTR + 2), "bias", 1), (dict(x=None), "null", 1), (dict(y=PTR), "y is x", 1), (dict(x=PTR + 8), "16-byte", 1),
    (dict(ld_x=56), "strides", 1), (dict(ld_y=68), "strides", 1), (dict(ld_x=(1 << 24) + 8), "2^24", 1),
])
def test_short_conv_refusals(vq, kw, text, want):
    _refused(vq, vq.lib().vqmlp_short_conv(C.byref(_conv(vq, **kw)), None), text, want)


def _append(vq, **kw):
    d = dict(dtype=0, T=3, heads=4, kv_heads=2, D=64, rot=32, pairs=0, page_size=16, n_pages=4, eps=1e-6, w_offset=0.0, q=PTR,
             ld_q=256, hs_q=64, k=PTR, ld_k=128, hs_k=64, v=PTR, ld_v=128, hs_v=64, q_out=PTR + 1024, ld_q_out=256,
             inv_freq=PTR, position=PTR, slot=PTR, k_cache=PTR, v_cache=PTR)
    d.update(kw)
    return vq._AppendDesc(**d)


@pytest.mark.parametrize("kw,text,want", [
    (dict(dtype=2), "dtype", 1), (dict(page_size=12), "page_size", 1), (dict(page_size=4), "page_size", 1),
    (dict(page_size=2048), "page_size", 1), (dict(T=-1), "T=-1", 1), (dict(heads=-1), "heads=-1", 1),
    (dict(heads=65536), "heads=65536", 1), (dict(kv_heads=0), "kv_heads=0", 1), (dict(D=12), "D=12", 1), (dict(D=264), "D=264", 1),
    (dict(n_pages=0), "n_pages=0", 1), (dict(n_pages=1 << 28), "2^31", 1), (dict(rot=72), "rot=72", 1), (dict(rot=12), "rot=12", 1),
    (dict(rot=-8), "rot=-8", 1), (dict(pairs=2), "pairs", 1), (dict(T=1 << 30), "2^30", 2), (dict(q_w=PTR, eps=-1.0), "eps", 1),
    (dict(k_w=PTR, w_offset=float("inf")), "w_offset", 1), (dict(k=None), "null", 1), (dict(q=None), "null", 1),
    (dict(q_out=None), "null", 1), (dict(inv_freq=None), "null", 1), (dict(position=None), "null", 1), (dict(slot=None), "null", 1),
    (dict(v_cache=None), "null", 1), (dict(ld_k=132), "multiples of 8", 1), (dict(ld_v=-8), "multiples of 8", 1),
    (dict(hs_q=60), "multiples of 8", 1), (dict(hs_v=(1 << 24) + 8), "2^24", 1), (dict(ld_q_out=248), "q_out", 1),
    (dict(ld_q_out=260), "q_out", 1), (dict(q_out=PTR, ld_q=512), "other strides", 1), (dict(q_out=PTR, hs_q=128), "other strides", 1),
    (dict(k=PTR + 8), "16-byte", 1), (dict(q_out=PTR + 8), "16-byte", 1), (dict(q_w=PTR + 8), "16-byte", 1),
    (dict(slot=PTR + 2), "4-byte", 1), (dict(inv_freq=PTR + 1), "4-byte", 1),
])
def test_paged_append_refusals(vq, kw, text, want):
    _refused(vq, vq.lib().vqmlp_paged_append(C.byref(_append(vq, **kw)), None), text, want)


def test_null_descriptions_and_empty_calls(vq):
    L = vq.lib()
    for f in (lambda: L.vqmlp_delta_rule(None, None, 0, None), lambda: L.vqmlp_short_conv(None, None),
              lambda: L.vqmlp_paged_append(None, None)):
        _refused(vq, f(), "null description")
    _refused(vq, L.vqmlp_delta_rule_workspace(C.byref(_delta(vq)), None), "null pointer")
    assert L.vqmlp_paged_append(C.byref(_append(vq, T=0, q=None, k=None, v=None)), None) == 0


def test_binding_refuses_what_does_not_fit(vq):
    import torch

    h, b, f, i = torch.float16, torch.bfloat16, torch.float32, torch.int32
    E = vq.VqmlpError
    z = lambda *s, t=h: torch.zeros(s, dtype=t)  # noqa: E731
    cu = z(2, t=i)
    rule = vq.DeltaRule(2, 4, 64, 32)
    q, v, g = z(3, 2, 64), z(3, 4, 32), z(3, 4, t=f)
    for args, text in (((q, q, v.float(), g, g), "differ"), ((q, q, v, g, g.half()), "beta"), ((q, q, v, g.half(), g), "beta")):
        with pytest.raises(E, match=text):
            rule.forward(*args, rule.state(1, "cpu"), cu)
    with pytest.raises(E, match="GPU"):
        rule.forward(q, q, v, g, g, rule.state(1, "cpu"), cu)
    for name in ("k_heads", "v_heads", "Dk", "Dv", "scale"):
        with pytest.raises(AttributeError):
            setattr(rule, name, 8)
    with pytest.raises(E, match="activation"):
        vq.ShortConv(z(16, 4), activation="relu")
    with pytest.raises(E, match="bias"):
        vq.ShortConv(z(16, 4), z(8))
    conv = vq.ShortConv(z(16, 4))
    for x, s, text in ((z(3, 24), conv.state(1), "shape"), (z(3, 16, t=b), conv.state(1), "differ"),
                       (z(3, 16), z(1, 3, 16, t=b), "differ"), (z(3, 1, 16), conv.state(1), "T, C")):
        with pytest.raises(E, match=text):
            conv.forward(x, s, cu)
    with pytest.raises(E, match="neither"):
        vq.Rotary()
    with pytest.raises(E, match="float32"):
        vq.Rotary(z(8))
    with pytest.raises(E, match="k_w"):
        vq.Rotary(q_weight=z(64), k_weight=z(32))
    cache = vq.PagedCache.empty(4, 2, 16, 64, h, "cpu")
    kv, at = z(3, 2, 64), z(3, t=i)
    turn = vq.Rotary(z(32, t=f))
    for call, text in ((lambda: cache.append(kv, kv, kv, at, at, vq.Rotary(z(40, t=f))), "fit"),
                       (lambda: cache.append(kv, kv, kv, at, at, vq.Rotary(q_weight=z(64, t=b))), "fit"),
                       (lambda: cache.append(kv, kv, kv, at, at, vq.Rotary(q_weight=z(32))), "32 elements"),
                       (lambda: cache.append(kv, kv.float(), kv, at, at, turn), "differ"),
                       (lambda: cache.append(kv, kv, z(3, 2, 128)[..., ::2], at, at, turn), "one after another"),
                       (lambda: cache.append(kv, kv, kv, at[:2], at, turn), "entries"),
                       (lambda: cache.append(kv, kv, kv, at, at.long(), turn), "int32"),
                       (lambda: cache.append(None, kv, kv, at, at, turn, q_out=kv), "without q"),
                       (lambda: cache.append(kv, kv, kv, at, at, turn), "GPU")):
        with pytest.raises(E, match=text):
            call()


@pytest.mark.parametrize("size", [2 ** 31, 2 ** 32 + 5, -1, -2 ** 32 + 5])
def test_sizes_beyond_32_bits_are_not_cut(vq, size):
    import torch

    rule = vq.DeltaRule(2, 2, 64, 64)
    w = torch.zeros(16, 4, dtype=torch.float16)
    for call in (lambda: rule.workspace_bytes(3, 1, size), lambda: rule.workspace_bytes(3, size, 3),
                 lambda: rule.workspace_bytes(size, 1, 3), lambda: vq.DeltaRule(size, 2, 64, 64),
                 lambda: vq.ShortConv(w, unit_heads=size, unit_dim=8), lambda: vq.ShortConv(w, unit_heads=1, unit_dim=size)):
        with pytest.raises(vq.VqmlpError, match="2\\^31"):
            call()
