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
