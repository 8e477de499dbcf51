"""GPU: the example decoder.  Serving step by step gives what one step over the whole sequences gives.

Tolerance.  Both sides round to binary16 (2^-11) at the same places, about a dozen a layer; where a
different kernel sums in another order, a value may land one rounding apart, and each such step passes
on to the layers behind it.  All of them in one direction: 4 layers x 12 x 2^-11 = 2.3e-2 of the norm.
"""
import pytest

pytestmark = pytest.mark.gpu


def test_steps_equal_one_pass():
    import torch

    from bit_vector_lut_amd import decoder

    lens, chunks, steps = [37, 5, 70], ([20, 5, 33], [17, 0, 37]), 3
    g = torch.Generator().manual_seed(1)
    prompts = [torch.randint(0, 4096, (n,), generator=g) for n in lens]
    model = decoder.Decoder(seed=3)
    at = [0, 0, 0]
    for part in chunks:  # the prompts in two chunks, one request idle in the second
        tokens = torch.cat([p[a:a + n] for p, a, n in zip(prompts, at, part)]).cuda()
        x, plan = model.step(tokens, part)
        at = [a + n for a, n in zip(at, part)]
    # 20 -> 37 of 16-token pages: 2 -> 3; 5 stays in its first; 33 -> 70: 3 -> 5
    assert plan.status.tolist() == [0, 54, 3, 0]
    seqs, last = [p.tolist() for p in prompts], [None] * 3
    tokens = torch.randint(0, 4096, (3,), generator=g).cuda()
    for _ in range(steps):
        x, plan = model.step(tokens, [1, 1, 1])
        assert plan.status[0].item() == 0
        for r in range(3):
            seqs[r].append(int(tokens[r]))
            last[r] = x[r].float().cpu()
        tokens = model.next_tokens(x, plan).long()
        assert ((tokens >= 0) & (tokens < 4096)).all()
    assert plan.seq_len.tolist() == [n + steps for n in lens]

    whole = decoder.Decoder(seed=3)
    x, plan = whole.step(torch.tensor(sum(seqs, [])).cuda(), [len(s) for s in seqs])
    assert plan.status[0].item() == 0 and plan.seq_len.tolist() == [n + steps for n in lens]
    for r in range(3):
        ref = x[plan.cu_q[r + 1].item() - 1].float().cpu()
        err = ((last[r] - ref).norm() / ref.norm()).item()
        print("request %d: %.3e" % (r, err), flush=True)
        assert err <= 2.3e-2


def test_step_refuses_what_does_not_fit():
    import torch

    from bit_vector_lut_amd import decoder

    model = decoder.Decoder(layers=1, seed=0)
    with pytest.raises(ValueError):
        model.step(torch.zeros(4, dtype=torch.long, device="cuda"), [1, 1, 1])
    with pytest.raises(ValueError):
        model.step(torch.zeros(2, dtype=torch.long, device="cuda"), [1, 1])


def test_idle_requests_and_failed_plans_give_no_token():
    """A request without new tokens has no next token (-1), nor has any after a plan that failed."""
    import torch

    from bit_vector_lut_amd import decoder

    model = decoder.Decoder(layers=1, max_len=32, seed=2)
    tokens = torch.randint(0, 4096, (9,), generator=torch.Generator().manual_seed(2)).cuda()
    x, plan = model.step(tokens[:9], [4, 0, 5])
    got = model.next_tokens(x, plan)
    want = model.head.argmax(x[[3, 8]].contiguous())[0]
    assert got.tolist() == [want[0].item(), -1, want[1].item()]
    x, plan = model.step(tokens[:3], [0, 3, 0])
    got = model.next_tokens(x, plan).tolist()
    assert got[0] == -1 and got[2] == -1 and got[1] >= 0
    assert model.errors.item() == 0
    x, plan = model.step(torch.zeros(29, dtype=torch.long, device="cuda"), [29, 0, 0])  # 33 of 32 positions
    assert plan.status[0].item() == 1 and model.next_tokens(x, plan).tolist() == [-1, -1, -1]
    x, plan = model.step(tokens[:3], [1, 1, 1])  # the step after it works, and the error is remembered
    assert plan.status[0].item() == 0 and min(model.next_tokens(x, plan).tolist()) >= 0
    assert model.errors.item() == 1
