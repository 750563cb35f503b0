"""The hybrid serving example's request rows: what one request leaves does not
reach the next in its row, and a step that does not fit is noticed."""
import pytest
import torch

from tests.test_hybrid_example_gpu import example  # noqa: F401

pytestmark = pytest.mark.gpu
INTS = {"dtype": torch.int32, "device": "cuda"}


def tokens(n, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    return torch.randn(n, 256, generator=gen, device="cuda").to(torch.bfloat16)


def model(example, **kw):  # noqa: F811
    return example.Hybrid("ka", width=256, heads=2, q_heads=4, kv_heads=2, page=16, requests=2,
                          seed=3, **kw)


@pytest.mark.parametrize("left", [float("nan"), float("inf")])
def test_a_finished_request_leaves_a_clean_state(example, left):  # noqa: F811
    m = model(example)
    m.step(tokens(12, 1), torch.tensor([5, 7], **INTS), 7)
    keep = m.state[0][1].clone()
    m.state[0][0, 1, 3, 4] = left
    m.finish(torch.tensor([1, 0], **INTS))
    assert (m.state[0][0] == 0).all() and torch.equal(m.state[0][1], keep)
    out = m.step(tokens(4, 2), torch.tensor([4, 0], **INTS), 4)
    assert out.isfinite().all()


def test_a_step_that_does_not_fit_changes_nothing(example):  # noqa: F811
    from gated_delta_rule_32_gb300 import kda
    m = model(example, pages=4)
    m.step(tokens(12, 1), torch.tensor([5, 7], **INTS), 7)
    state = m.state[0].clone()
    with pytest.raises(kda.KdaError, match="NO_PAGES"):
        m.step(tokens(70, 2), torch.tensor([60, 10], **INTS), 60)     # five pages, two are left
    assert m.lens.tolist() == [5, 7] and m.left.item() == 2 and torch.equal(m.state[0], state)
    out = m.step(tokens(2, 3), torch.tensor([1, 1], **INTS), 1)
    m.check()
    assert out.isfinite().all() and m.lens.tolist() == [6, 8]


def test_more_tokens_than_announced_are_noticed(example):  # noqa: F811
    from gated_delta_rule_32_gb300 import kda
    for late in (False, True):
        m = model(example)
        m.step(tokens(9, 1), torch.tensor([4, 5], **INTS), 4)
        with pytest.raises(kda.KdaError, match="BAD_SEQLENS"):
            if late:                                                  # by the next step at the latest
                m.step(tokens(2, 2), torch.tensor([1, 1], **INTS), 1)
            else:
                m.check()
        m.check()                                                     # said once


def test_a_release_that_fails_changes_nothing(example):  # noqa: F811
    from gated_delta_rule_32_gb300 import kda
    m = model(example)
    m.step(tokens(12, 1), torch.tensor([5, 7], **INTS), 7)
    state, page = m.state[0].clone(), m.table[0, 0].item()
    m.table[0, 0] = 10 ** 6
    with pytest.raises(kda.KdaError, match="BAD_PAGES"):
        m.finish(torch.tensor([1, 0], **INTS))
    assert torch.equal(m.state[0], state) and m.lens.tolist() == [5, 7]
    m.table[0, 0] = page
    m.finish(torch.tensor([1, 0], **INTS))
    assert (m.state[0][0] == 0).all() and m.lens.tolist() == [0, 7]
