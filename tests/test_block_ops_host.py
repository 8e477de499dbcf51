"""CPU tests of the operators around the MLP: every refusal that the host half makes, through the C
ABI, before any device call; and the binding's own checks of shapes, types and strides."""
import ctypes as C

import pytest


@pytest.fixture(scope="module")
def vq():
    from bit_vector_lut_amd import vqmlp

    vqmlp.lib()
    return vqmlp


BUF = C.create_string_buffer(4096 + 256)
PTR = (C.addressof(BUF) + 255) // 256 * 256  # never dereferenced: every call here is refused first


def _refused(vq, status, text, want=1):
    assert status == want, (status, vq.lib().vqmlp_last_error())
    assert text in vq.lib().vqmlp_last_error().decode(), vq.lib().vqmlp_last_error()


def _norm(vq, **kw):
    d = dict(dtype=0, res_dtype=0, kind=0, T=2, H=16, eps=1e-6, res_scale=1.0, w_offset=0.0, y=PTR,
             ld_y=16, res=PTR, ld_res=16, pre_w=PTR, res_out=PTR, ld_res_out=16, x=PTR, ld_x=16)
    d.update(kw)
    return vq._NormDesc(**d)


@pytest.mark.parametrize("kw,text", [
    (dict(dtype=2), "dtype"), (dict(res_dtype=1), "res_dtype"), (dict(kind=2), "kind"),
    (dict(T=-1), "out of range"), (dict(H=0), "out of range"), (dict(H=(1 << 20) + 1), "out of range"),
    (dict(y=None, res=None), "neither y nor res"), (dict(x=None, res_out=None), "neither x nor res_out"),
    (dict(pre_w=None), "needs pre_w"), (dict(y=None, post_w=PTR), "without y"),
    (dict(y=None, gate=PTR, ld_gate=16), "without y"), (dict(eps=-1.0), "eps"),
    (dict(eps=float("nan")), "eps"), (dict(ld_y=15), "row stride of y"), (dict(ld_x=8), "row stride of x"),
    (dict(gate=PTR, ld_gate=8), "row stride of gate"), (dict(y=PTR + 1), "aligned"),
    (dict(res_dtype=2, res=PTR + 2), "aligned"), (dict(pre_w=PTR + 1), "aligned"),
])
def test_block_norm_refusals(vq, kw, text):
    _refused(vq, vq.lib().vqmlp_block_norm(C.byref(_norm(vq, **kw)), None), text)


def test_null_descriptions_and_empty_calls(vq):
    L = vq.lib()
    for f in (lambda: L.vqmlp_block_norm(None, None), lambda: L.vqmlp_page_plan(None, None),
              lambda: L.vqmlp_paged_attn(None, None, 0, None),
              lambda: L.vqmlp_linear_attn(None, None, 0, None)):
        _refused(vq, f(), "null description")
    assert L.vqmlp_block_norm(C.byref(_norm(vq, T=0)), None) == 0
    assert L.vqmlp_paged_store(0, 0, 2, 64, 16, 4, None, 0, None, 0, None, None, None, None) == 0
    assert L.vqmlp_paged_attn(C.byref(_attn(vq, T=0)), None, 0, None) == 0


def _pages(vq, **kw):
    d = dict(R=4, max_tokens=32, page_size=16, n_pages=64, n_free=8, table_width=8, ld_table=8,
             ctx_len=PTR, q_len=PTR + 64, free_pages=PTR, table=PTR, seq_len=PTR + 128, cu_q=PTR,
             slot=PTR, position=PTR, status=PTR)
    d.update(kw)
    return vq._PagesDesc(**d)


@pytest.mark.parametrize("kw,text,want", [
    (dict(page_size=12), "page_size", 1), (dict(page_size=4), "page_size", 1),
    (dict(page_size=2048), "page_size", 1), (dict(R=0), "out of range", 1),
    (dict(max_tokens=-1), "out of range", 1), (dict(n_pages=0), "out of range", 1),
    (dict(n_free=-1), "out of range", 1), (dict(table_width=0), "out of range", 1),
    (dict(R=4097), "above 4096", 2), (dict(n_pages=1 << 28), "2^31", 1),
    (dict(table_width=1 << 28, ld_table=1 << 28), "2^31", 1), (dict(ld_table=7), "ld_table", 1),
    (dict(ctx_len=None), "null", 1), (dict(status=None), "null", 1), (dict(slot=None), "null", 1),
    (dict(free_pages=None), "free list", 1), (dict(free_head=PTR, free_head_out=PTR), "free_head", 1),
    (dict(seq_len=PTR), "input array", 1), (dict(cu_q=PTR + 2), "aligned", 1),
])
def test_page_plan_refusals(vq, kw, text, want):
    _refused(vq, vq.lib().vqmlp_page_plan(C.byref(_pages(vq, **kw)), None), text, want)


@pytest.mark.parametrize("at,value,text", [
    (0, 2, "dtype"), (4, 12, "page_size"), (1, -1, "T=-1"), (2, 0, "kv_heads=0"), (3, 12, "D=12"),
    (3, 264, "D=264"), (5, 0, "n_pages=0"), (5, 1 << 28, "2^31"), (6, None, "null"), (7, 120, "stride"),
    (7, 132, "multiples of 8"), (9, 64, "stride"), (6, PTR + 8, "aligned"), (11, PTR + 2, "aligned"),
    (10, PTR + 2, "aligned"), (12, None, "null"),
], ids=lambda v: "PTR+%d" % (v - PTR) if isinstance(v, int) and v >= PTR else None)
def test_paged_store_refusals(vq, at, value, text):
    args = [0, 3, 2, 64, 16, 4, PTR, 128, PTR, 128, PTR, PTR, PTR, None]
    args[at] = value
    _refused(vq, vq.lib().vqmlp_paged_store(*args), text)


def _attn(vq, **kw):
    d = dict(dtype=1, T=3, R=2, heads=6, kv_heads=2, D=64, page_size=16, n_pages=9, window=0, max_kv=64,
             scale=0.125, table_width=4, ld_table=4, ld_q=384, ld_y=384, q=PTR, y=PTR, k_cache=PTR,
             v_cache=PTR, table=PTR, cu_q=PTR, kv_len=PTR)
    d.update(kw)
    return vq._AttnDesc(**d)


@pytest.mark.parametrize("kw,text,want", [
    (dict(dtype=2), "dtype", 1), (dict(page_size=24), "page_size", 1), (dict(T=-1), "out of range", 1),
    (dict(R=0), "out of range", 1), (dict(window=-1), "out of range", 1), (dict(max_kv=-1), "out of range", 1),
    (dict(D=260), "D=260", 1), (dict(D=12), "D=12", 1), (dict(heads=7), "no multiple", 1),
    (dict(heads=130, ld_q=130 * 64, ld_y=130 * 64), "above 64", 2), (dict(R=65537), "65536", 2),
    (dict(T=1 << 28), "2^30", 2), (dict(n_pages=1 << 28), "2^31", 1), (dict(scale=0.0), "scale", 1),
    (dict(scale=-1.0), "scale", 1), (dict(scale=float("nan")), "scale", 1),
    (dict(scale=float("inf")), "scale", 1), (dict(q=None), "null", 1), (dict(kv_len=None), "null", 1),
    (dict(ld_q=376), "at least", 1), (dict(ld_y=388), "multiples of 8", 1), (dict(ld_table=3), "ld_table", 1),
    (dict(q=PTR + 8), "aligned", 1), (dict(lse=PTR + 2), "aligned", 1),
    (dict(R=65536, heads=600, kv_heads=300), "2^24", 2),
])
def test_paged_attn_refusals(vq, kw, text, want):
    _refused(vq, vq.lib().vqmlp_paged_attn(C.byref(_attn(vq, **kw)), None, 0, None), text, want)


def _linear(vq, **kw):
    d = dict(dtype=0, T=20, R=2, k_heads=2, v_heads=4, Dk=64, Dv=32, n_states=2, max_q=20, scale=0.125,
             ld_q=128, ld_k=128, ld_v=128, ld_y=128, ld_g=4, q=PTR, k=PTR, v=PTR, g=PTR, y=PTR,
             state_in=PTR, state_out=PTR, cu_q=PTR)
    d.update(kw)
    return vq._LinearDesc(**d)


@pytest.mark.parametrize("kw,text,want", [
    (dict(dtype=2), "dtype", 1), (dict(T=-1), "out of range", 1), (dict(R=0), "out of range", 1),
    (dict(max_q=-1), "out of range", 1), (dict(v_heads=5), "no multiple", 1), (dict(Dk=136), "Dk=136", 1),
    (dict(Dv=4), "Dv=4", 1), (dict(R=65536), "65535", 2), (dict(scale=float("nan")), "scale", 1),
    (dict(scale=float("inf")), "scale", 1), (dict(cu_q=None), "cu_q", 1), (dict(state_in=None), "null state", 1),
    (dict(state_out=PTR + 4), "16-byte", 1), (dict(g=None), "null", 1), (dict(v=PTR + 8), "16-byte", 1),
    (dict(ld_k=120), "strides", 1), (dict(ld_q=132), "strides", 1), (dict(ld_g=3), "strides", 1),
    (dict(ld_v=(1 << 24) + 8), "2^24", 1), (dict(ld_g=(1 << 24) + 1), "2^24", 1),
])
def test_linear_attn_refusals(vq, kw, text, want):
    _refused(vq, vq.lib().vqmlp_linear_attn(C.byref(_linear(vq, **kw)), None, 0, None), text, want)


def test_binding_refuses_what_does_not_fit(vq):
    """Shapes, types and strides that the C ABI cannot see are refused by the binding."""
    import torch

    h, f, i = torch.float16, torch.float32, torch.int32
    E = vq.VqmlpError
    with pytest.raises(E, match="norm kind"):
        vq.BlockNorm(kind="max")
    with pytest.raises(E, match="bias"):
        vq.BlockNorm(None, torch.zeros(8, dtype=h))
    norm = vq.BlockNorm(torch.ones(16, dtype=h))
    cases = [(torch.zeros(2, 24, dtype=h), None), (torch.zeros(2, 16, dtype=torch.bfloat16), None)]
    for y, r in cases:
        with pytest.raises(E, match="weights"):
            norm.forward(y, r)
    with pytest.raises(E):
        norm.forward(None, None)
    cache = vq.PagedCache.empty(4, 2, 16, 64, h, "cpu")
    with pytest.raises(E, match="shape"):
        vq.PagedCache(cache.k, cache.k)
    slot = torch.zeros(3, dtype=i)
    kv = torch.zeros(3, 2, 64, dtype=h)
    with pytest.raises(E, match="type"):
        cache.store(kv.float(), kv, slot)
    with pytest.raises(E, match="one after another"):
        cache.store(kv.transpose(1, 2).contiguous().transpose(1, 2), kv, slot)
    with pytest.raises(E, match="entries"):
        cache.store(kv, kv, slot[:2])
    with pytest.raises(E, match="int32"):
        cache.store(kv, kv, slot.long())
    planner = vq.PagePlanner(torch.zeros(2, 4, dtype=i), torch.zeros(3, dtype=i), 16, 8, 10)
    with pytest.raises(E, match="ctx_len"):
        planner.forward(slot, slot)
    lin = vq.LinearAttention(2, 4, 64, 32)
    q, v, g = torch.zeros(3, 2, 64, dtype=h), torch.zeros(3, 4, 32, dtype=h), torch.zeros(3, 4)
    with pytest.raises(E, match="differ"):
        lin.forward(q, q, v.float(), g, lin.state(1, "cpu"), slot[:2])


def test_sizes_that_pass_32_bit_workgroup_numbers_are_refused(vq):
    """Sizes whose launch would hold 2^32 threads or more, or whose rounding up passes 2^31."""
    L, top = vq.lib(), 2 ** 31 - 1
    for n in (top, 2 ** 30):
        _refused(vq, L.vqmlp_page_plan(C.byref(_pages(vq, max_tokens=n)), None), "max_tokens above", 2)
        _refused(vq, L.vqmlp_paged_store(0, n, 2, 64, 16, 4, PTR, 128, PTR, 128, PTR, PTR, PTR, None), "T above", 2)
    for kw in (dict(R=65535, v_heads=65534), dict(T=2 ** 30 - 1, v_heads=2048, ld_v=1 << 16, ld_y=1 << 16, ld_g=2048)):
        d = _linear(vq, **dict(dict(ld_v=65534 * 32, ld_y=65534 * 32, ld_g=65534), **kw))
        _refused(vq, L.vqmlp_linear_attn(C.byref(d), None, 0, None), "2^31 - 1", 2)


def test_tensors_that_the_library_points_to_are_not_replaced(vq):
    """A planner's and a cache's tensors and sizes are given to the library once: assigning others is refused,
    where a call would have gone on with the old memory."""
    import torch

    i = torch.int32
    planner = vq.PagePlanner(torch.zeros(2, 4, dtype=i), torch.zeros(3, dtype=i), 16, 8, 10, torch.zeros(1, dtype=i))
    cache = vq.PagedCache.empty(4, 2, 16, 64, torch.float16, "cpu")
    for what, names in ((planner, ("table", "free_pages", "free_head", "R", "max_tokens", "page_size", "n_pages", "device")),
                        (cache, ("k", "v", "n_pages", "kv_heads", "page_size", "D", "dtype", "device"))):
        for name in names:
            value = getattr(what, name)
            with pytest.raises(AttributeError):
                setattr(what, name, value)
            assert getattr(what, name) is value


@pytest.mark.parametrize("size", [2 ** 31, 2 ** 32 + 5, -1, -2 ** 32 + 5])
def test_sizes_beyond_32_bits_are_not_cut(vq, size):
    """A window of 2^32 + 5 is refused, not taken for one of 5; and so for every size that is passed on."""
    import torch

    i, h = torch.int32, torch.float16
    z = lambda *s, t=i: torch.zeros(s, dtype=t)  # noqa: E731
    cache, lin = vq.PagedCache.empty(4, 2, 16, 64, h, "cpu"), vq.LinearAttention(2, 2, 64, 64)
    q = z(3, 2, 64, t=h)
    for call in (lambda: cache.attention(q, z(1, 4), z(2), z(1), window=size),
                 lambda: cache.attention(q, z(1, 4), z(2), z(1), max_kv=size),
                 lambda: cache.workspace_bytes(3, 1, 2, 4, size), lambda: cache.workspace_bytes(size, 1, 2, 4),
                 lambda: lin.workspace_bytes(3, 1, size), lambda: lin.workspace_bytes(3, size, 3),
                 lambda: lin._desc(0, 3, 1, size, 3),
                 lambda: vq.PagePlanner(z(2, 4), z(3), 16, size, 10), lambda: vq.PagePlanner(z(2, 4), z(3), 16, 8, size),
                 lambda: vq.PagePlanner(z(2, 4), z(3), size, 8, 10),
                 lambda: vq.BlockNorm(torch.ones(1, dtype=h)).forward(z(1, 1, t=h).expand(2 ** 32 + 5, 1))):
        with pytest.raises(vq.VqmlpError, match="2\\^31"):
            call()
