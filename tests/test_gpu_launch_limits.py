"""GPU: sizes at the limit of a launch (fewer than 2^32 threads).  Asks for workspace sizes only; nothing is launched."""
import ctypes as C

import pytest

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("R,T,heads,kv_heads,max_kv", [
    (65536, 65536, 8, 8, 2 ** 30 - 1), (65536, 65536, 8, 8, 2 ** 29), (65536, 131072, 16, 16, 2 ** 30 - 1),
    (4096, 2 ** 21, 32, 2, 2 ** 30 - 1), (8, 64, 8, 8, 2 ** 30 - 1),
])
def test_attention_splits_fit_a_launch(R, T, heads, kv_heads, max_kv):
    """The workspace holds D sums and two words for each row and split: what it says of the splits."""
    import torch

    from bit_vector_lut_amd import vqmlp

    torch.cuda.init()
    D = 64
    d = vqmlp._AttnDesc(dtype=0, T=T, R=R, heads=heads, kv_heads=kv_heads, D=D, page_size=16, n_pages=64,
                        window=0, max_kv=max_kv, scale=0.125, table_width=64)
    n = C.c_size_t()
    assert vqmlp.lib().vqmlp_paged_attn_workspace(C.byref(d), C.byref(n)) == 0
    splits = max(1, n.value // (T * heads * (4 * D + 8)))
    places = splits | 1 if R > 1 else splits  # an odd number for each tile of several requests
    tiles = T * (heads // kv_heads) // 128 + R + 1
    print("splits", splits, flush=True)
    assert tiles * kv_heads * places * 256 < 2 ** 32
    assert splits == 1 or (T * heads + 3) // 4 * 256 < 2 ** 32  # the join


@pytest.mark.parametrize("T,H", [(2 ** 26 + 5, 8), (2 ** 24 + 9, 3)])
def test_norms_of_more_rows_than_a_launch_holds(T, H):
    """Rows in front of, around and behind the end of the first launch give what a call of their own gives."""
    import torch

    from bit_vector_lut_amd import vqmlp

    h = dict(dtype=torch.float16, device="cuda")
    g = torch.Generator(device="cuda").manual_seed(1)
    y, res = torch.empty(T, H, **h).normal_(generator=g), torch.empty(T, H, dtype=torch.float32, device="cuda").normal_(generator=g)
    gate = torch.empty(T, H, **h).normal_(generator=g)
    op = vqmlp.BlockNorm(torch.rand(H, generator=g, **h), post_weight=torch.rand(H, generator=g, **h))
    print("norm", T, H, flush=True)
    r, x = op.forward(y, res, gate)
    torch.cuda.synchronize()
    for a in (0, T // 2, T - 5 - 16, T - 8):
        rows = slice(a, min(T, a + 16))
        r2, x2 = op.forward(y[rows], res[rows], gate[rows])
        assert torch.equal(r[rows], r2) and torch.equal(x[rows], x2)
