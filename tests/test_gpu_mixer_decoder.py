"""GPU: the example decoder with the delta rule, the short convolution and turned heads, served step by step.

Tolerance, as of the decoder's other mixers: both sides round to binary16 (2^-11) at the same places, in a
layer into, convolution, y, out (of an attention layer qkv, q and k, y, out), two norms and the MLP's six; a
sum in another order may land one rounding apart, all of them in one direction: 4 layers x 12 x 2^-11 =
2.3e-2 of the norm.
"""
import pytest

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("options", [dict(mixer="delta"), dict(rotary=128), dict(mixer="delta", rotary=32, conv_width=3)])
def test_steps_equal_one_pass(options):
    import torch

    from bit_vector_lut_amd import decoder

    lens, chunks, steps = [37, 5, 150], ([20, 5, 70], [17, 0, 80]), 3
    g = torch.Generator().manual_seed(1)
    prompts = [torch.randint(0, 4096, (n,), generator=g) for n in lens]
    model = decoder.Decoder(seed=3, **options)
    at = [0, 0, 0]
    for part in chunks:
        tokens = torch.cat([p[a:a + n] for p, a, n in zip(prompts, at, part)]).cuda()
        x, plan = model.step(tokens, part)
        at = [a + n for a, n in zip(at, part)]
    seqs, last = [p.tolist() for p in prompts], [None] * 3
    tokens = torch.randint(0, 4096, (3,), generator=g).cuda()
    for _ in range(steps):
        x, plan = model.step(tokens, [1, 1, 1])
        for r in range(3):
            seqs[r].append(int(tokens[r]))
            last[r] = x[r].float().cpu()
        tokens = model.next_tokens(x, plan).long()
        assert ((tokens >= 0) & (tokens < 4096)).all()
    assert model.errors.item() == 0 and plan.seq_len.tolist() == [n + steps for n in lens]

    whole = decoder.Decoder(seed=3, **options)
    x, plan = whole.step(torch.tensor(sum(seqs, [])).cuda(), [len(s) for s in seqs])
    for r in range(3):
        ref = x[plan.cu_q[r + 1].item() - 1].float().cpu()
        err = ((last[r] - ref).norm() / ref.norm()).item()
        print("request %d: %.3e" % (r, err), flush=True)
        assert err <= 2.3e-2


def test_a_failed_plan_leaves_the_requests_as_they_are():
    import torch

    from bit_vector_lut_amd import decoder

    tokens = torch.randint(0, 4096, (40,), generator=torch.Generator().manual_seed(2)).cuda()
    got = []
    for fail in (False, True):
        model = decoder.Decoder(layers=4, max_len=32, seed=2, mixer="delta", rotary=64)
        model.step(tokens[:9], [4, 1, 4])
        if fail:
            x, plan = model.step(tokens[:29], [29, 0, 0])  # 33 of 32 positions
            assert plan.status[0].item() == 1 and model.next_tokens(x, plan).tolist() == [-1, -1, -1]
        x, plan = model.step(tokens[9:13], [1, 2, 1])
        assert plan.status[0].item() == 0 and x.isfinite().all()
        got.append(x)
    assert torch.equal(*got)


def test_an_unknown_mixer_is_refused():
    from bit_vector_lut_amd import decoder

    with pytest.raises(ValueError):
        decoder.Decoder(mixer="other")
