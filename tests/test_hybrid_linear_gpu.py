"""The serving example with layers of linear attention and rotary positions:
it runs, in pieces as in one, and what it calls gets what the plan says."""
import os
import sys

import pytest
import torch

pytestmark = pytest.mark.gpu
sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))


@pytest.fixture(scope="module", autouse=True)
def built():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    from gated_delta_rule_32_gb300 import build, kda
    build.build()
    kda.load()


def ints(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def test_it_runs():
    import hybrid_serving
    model, out = hybrid_serving.main(["--layers", "lkla", "--rotary", "--steps", "3"])
    assert out.shape == (53, model.width) and bool(out.isfinite().all())
    # the prompts, one step and three more, the last one; the second row's request is new
    assert model.lens.tolist() == [301 + 5, 50, 96 + 5, 640 + 5]


def test_prompt_in_one_step_and_token_by_token():
    # one layer: the residual stream before it is the same, so outputs differ only by the kernels'
    # roundings (weights and states to 16 bits, 2^-8 each) and the sums they end in
    import hybrid_serving
    gen = torch.Generator(device="cuda").manual_seed(3)
    x = torch.randn(2 * 9, 512, generator=gen, device="cuda").to(torch.bfloat16)
    whole = hybrid_serving.Hybrid("l", requests=2)
    a = whole.step(x, ints([9, 9]), 9)
    steps = hybrid_serving.Hybrid("l", requests=2)
    b = torch.stack([steps.step(x.view(2, 9, 512)[:, t].contiguous(), ints([1, 1]), 1) for t in range(9)], 1)
    whole.check(), steps.check()
    assert whole.lens.tolist() == steps.lens.tolist() == [9, 9]
    d = (a.view(2, 9, 512).double() - b.double()).norm() / b.double().norm()
    assert d <= 3 * 2.0 ** -8, d
    s, t = whole.state[0].double(), steps.state[0].double()
    assert (s - t).norm() <= 2.0 ** -16 * t.norm()
    whole.finish(ints([0, 1]))
    assert (whole.state[0][1] == 0).all() and torch.equal(whole.state[0][0].double(), s[0])


def test_rotary_changes_attention_and_nothing_is_left_out():
    import hybrid_serving
    gen = torch.Generator(device="cuda").manual_seed(4)
    x = torch.randn(40, 512, generator=gen, device="cuda").to(torch.bfloat16)
    outs = []
    for rotary in (False, True):
        m = hybrid_serving.Hybrid("a", requests=2, rotary=rotary)
        outs.append(m.step(x, ints([30, 10]), 30))
        m.check()
    # a request's first token sees only itself, whatever its position
    assert torch.equal(outs[0][[0, 30]], outs[1][[0, 30]])
    assert not torch.equal(outs[0], outs[1]) and bool(outs[1].isfinite().all())
