"""The hybrid serving example: decoding after a prompt gives what one longer
prompt gives, and its bookkeeping adds up."""
import importlib.util
import os

import pytest
import torch

pytestmark = pytest.mark.gpu
PATH = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples",
                    "hybrid_serving.py")


@pytest.fixture(scope="module")
def example():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    from gated_delta_rule_32_gb300 import build
    build.build()
    spec = importlib.util.spec_from_file_location("hybrid_serving", PATH)
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


@pytest.mark.parametrize("code", ["int8", "e4m3"])
def test_prompt_then_decode_equals_one_prompt(example, code):
    # The two differ by roundings only: bf16 activations, the gated delta
    # rule's two paths (each within 1e-2 of the exact one), and codes rounded
    # once more where a page's scale grew between steps (1/254 of the scale for
    # int8, 1/32 of a value for e4m3).  Through one attention layer with its
    # residual that stays below 5% of the output's size.
    lens, more = [70, 1, 33], 5
    ints = {"dtype": torch.int32, "device": "cuda"}
    gen = torch.Generator(device="cuda").manual_seed(4)
    xs = [torch.randn(n + more, 256, generator=gen, device="cuda").to(torch.bfloat16) for n in lens]

    def model():
        return example.Hybrid("ka", width=256, heads=2, q_heads=4, kv_heads=2, page=16, requests=3,
                              code=code, seed=2)
    whole = model()
    full = whole.step(torch.cat(xs), torch.tensor([n + more for n in lens], **ints), max(lens) + more)
    parts = model()
    parts.step(torch.cat([x[:n] for x, n in zip(xs, lens)]), torch.tensor(lens, **ints), max(lens))
    at = 0
    for i in range(more):
        got = parts.step(torch.stack([x[n + i] for x, n in zip(xs, lens)]),
                         torch.ones(3, **ints), 1)
        at = 0
        for r, n in enumerate(lens):
            want = full[at + n + i].float()
            assert (got[r].float() - want).abs().max() <= 0.05 * want.abs().max()
            at += n + more
    assert torch.equal(whole.lens, parts.lens) and torch.equal(whole.left, parts.left)


def test_the_example_runs(example):
    model, out = example.main(["--steps", "3"])
    assert out.isfinite().all()
    held = sum(-(-n // model.page) for n in model.lens.tolist())
    assert model.left.item() == model.free.numel() - held
    assert (model.table >= 0).sum().item() == held
