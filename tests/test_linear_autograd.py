"""Linear attention and rotary positions have no gradient: a tensor that wants
one is refused, and what changes in place does so in autograd's eyes too."""
import pytest
import torch

import gated_delta_rule_32_gb300 as pkg


@pytest.mark.parametrize("which", range(5))
def test_refusals_without_a_gpu(which):
    x = [torch.zeros(1, 4, 2, 64) for _ in "qkv"] + [torch.zeros(2), torch.zeros(1, 2, 64, 64)]
    x[which].requires_grad_()
    for call in (pkg.linear_attend, pkg.linear_decode):
        with pytest.raises(ValueError, match="gradient"):
            call(*x)
        with torch.no_grad(), pytest.raises(ValueError, match="CUDA"):
            call(*x)
    y = [torch.zeros(4, 2, 64), torch.zeros(4, 2, 64), torch.zeros(4, dtype=torch.int32),
         torch.zeros(32, dtype=torch.float64)]
    if which < 2 or which == 3:
        y[which].requires_grad_()
        for inplace in (False, True):
            with pytest.raises(ValueError, match="gradient"):
                pkg.rotary_embed(*y, inplace=inplace)
        with torch.no_grad(), pytest.raises(ValueError, match="CUDA"):
            pkg.rotary_embed(*y)


@pytest.fixture
def built():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    from gated_delta_rule_32_gb300 import build, kda
    build.build()
    kda.load()


@pytest.mark.gpu
def test_changes_in_place_are_seen(built):
    q = torch.randn(4, 2, 64, device="cuda")
    k = torch.randn(4, 2, 64, device="cuda")
    w = torch.ones(4, 2, 64, device="cuda", requires_grad=True)
    pos = torch.arange(4, dtype=torch.int32, device="cuda")
    f, _ = pkg.rotary_frequencies(64)
    for x in (q, k):
        z = (x * w).sum()                      # (keeps x for w's gradient)
        pkg.rotary_embed(q, k, pos, f)
        z.backward(retain_graph=True)
        pkg.rotary_embed(q, k, pos, f, inplace=True)
        with pytest.raises(RuntimeError, match="inplace"):
            z.backward()
    state = torch.randn(4, 2, 64, 64, device="cuda")
    v = torch.ones_like(state, requires_grad=True)
    z = (state * v).sum()
    t = q[:, None]
    pkg.linear_decode(t, t, t, torch.zeros(2, device="cuda"), state)
    with pytest.raises(RuntimeError, match="inplace"):
        z.backward()
    # parameters of a model that serves: without gradients nothing is refused, tensors of
    # inference mode (which have no version) among them
    a = torch.nn.Parameter(torch.zeros(2, device="cuda"))
    with torch.no_grad():
        want = pkg.linear_decode(t, t, t, a, state.clone())
    with torch.inference_mode():
        got = pkg.linear_decode(t.clone(), t, t, a, state.clone())
        pkg.rotary_embed(q.clone(), None, pos, f, inplace=True)
    assert torch.equal(want, got)
