"""A token whose factor is 0 forgets the state before it, whatever that holds;
factors that only come to 0 together do not."""
import math

import pytest
import torch

import gated_delta_rule_32_gb300 as pkg
from gated_delta_rule_32_gb300 import kda
from tests import _linear_oracle as plain

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module", autouse=True)
def built():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    from gated_delta_rule_32_gb300 import build
    build.build()
    kda.load()


def made(B, T, H, dk, dv, dtype=BF, seed=0):
    g = torch.Generator(device="cuda").manual_seed(seed)

    def normal(*shape):
        return torch.randn(*shape, generator=g, device="cuda")
    q, k = (torch.nn.functional.normalize(normal(B, T, H, dk), dim=-1).to(dtype) for _ in "qk")
    return dict(q=q, k=k, v=normal(B, T, H, dv).to(dtype), log_decay=-normal(B, T, H).abs() / 20)


def nothing(N, H, dk, dv):
    """States of what nobody wrote (each third column is finite, but far out)."""
    s = torch.full((N, H, dk, dv), math.nan, device="cuda")
    s[..., ::3] = math.inf
    s[..., 1::3] = -3e38
    return s


def dead(x):
    """Nothing of the columns that began without numbers is finite."""
    return not any(x[..., c::3].isfinite().any() for c in (0, 2))


@pytest.mark.parametrize("dtype,dk,dv", [(BF, 128, 128), (BF, 64, 64), (BF, 64, 128), (BF, 16, 64), (F32, 64, 64)])
@pytest.mark.parametrize("T,at", [(1, 0), (5, 0), (5, 4), (40, 17), (128, 127), (129, 128), (300, 0), (300, 31),
                                  (300, 32), (300, 126), (300, 200), (300, 299)])
@pytest.mark.parametrize("low", [-math.inf, -105.0])
def test_a_state_that_holds_anything(dtype, dk, dv, T, at, low):
    # two heads of three forget at a token each, the second once more before; as if the state had been zero
    x = made(2, T, 3, dk, dv, dtype, seed=T + at)
    x["log_decay"][:, at, :2] = low
    x["log_decay"][:, at // 2, 1] = low
    out, state = pkg.linear_attend(**x, init_state=nothing(2, 3, dk, dv))
    zero = torch.zeros(2, 3, dk, dv, device="cuda")
    want, after = pkg.linear_attend(**x, init_state=zero)
    for h, t in ((0, at), (1, at // 2)):
        assert torch.equal(out[:, t:, h], want[:, t:, h]) and torch.equal(state[:, h], after[:, h])
    assert dead(out[:, :at, 0]) and dead(state[:, 2])
    o, s, om, sm = plain.attend(x["q"], x["k"], x["v"], x["log_decay"], zero, 1.0)
    assert ((state[:, :2].double() - s[:, :2]).abs() <= (2.0 ** -16 + T * 2.0 ** -24) * sm[:, :2]).all()


@pytest.mark.parametrize("at", [0, 700, 2559, 2560, 4000, 4999])
@pytest.mark.parametrize("packed", [False, True])
def test_over_segments(at, packed):
    H, T, d = 3, 5000, 128
    x = made(1, T, H, d, d, seed=at)
    x["log_decay"][:, at, 0] = -math.inf
    x["log_decay"][:, 3500, 1] = -math.inf
    cu = torch.tensor([0, 100, T], dtype=torch.int32, device="cuda") if packed else None
    N = 2 if packed else 1
    assert kda.kda_linear_workspace_bytes(N, T, H, d, d, packed=packed) > 0
    out, state = pkg.linear_attend(**x, init_state=nothing(N, H, d, d), cu_seqlens=cu)
    want, after = pkg.linear_attend(**x, init_state=torch.zeros(N, H, d, d, device="cuda"), cu_seqlens=cu)
    last = at if not packed or at >= 100 else T          # (the second sequence begins at 100)
    assert torch.equal(out[:, last:, 0], want[:, last:, 0]) and torch.equal(out[:, 3500:, 1], want[:, 3500:, 1])
    if last < T:
        assert torch.equal(state[-1, 0], after[-1, 0])
    assert torch.equal(state[-1, 1], after[-1, 1])
    assert dead(out[:, 100:last, 0]) and dead(out[:, 100:3500, 1]) and dead(state[-1, 2])


@pytest.mark.parametrize("T", [60, 300, 5000])
def test_factors_that_come_to_0_together(T):
    # each of its own is not 0: what they multiply stays
    x = made(1, T, 2, 64, 64, seed=T)
    x["log_decay"][:] = -60.0
    s = torch.full((1, 2, 64, 64), math.nan, device="cuda")
    out, state = pkg.linear_attend(**x, init_state=s)
    assert out.isnan().all() and state.isnan().all()
    if T == 60:
        out, state = pkg.linear_attend(**{n: t.float() for n, t in x.items()}, init_state=s)
        assert out.isnan().all() and state.isnan().all()


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("dk,dv", [(128, 128), (64, 128), (16, 16)])
@pytest.mark.parametrize("T,at", [(1, 0), (4, 2), (19, 9)])
def test_single_tokens(dtype, dk, dv, T, at):
    x = made(5, T, 4, dk, dv, dtype, seed=T)
    x["log_decay"][1, at] = -math.inf
    x["log_decay"][3, at, 2] = -200.0
    state, after = nothing(5, 4, dk, dv), torch.zeros(5, 4, dk, dv, device="cuda")
    out, want = (pkg.linear_decode(**x, state=s) for s in (state, after))
    assert torch.equal(out[1, at:], want[1, at:]) and torch.equal(state[1], after[1])
    assert torch.equal(out[3, at:, 2], want[3, at:, 2]) and torch.equal(state[3, 2], after[3, 2])
    for n in (0, 2, 4):
        assert dead(out[n])
    assert dead(out[1, :at]) and dead(out[3, :, [0, 1, 3]])


def test_what_a_later_chunk_forgets():
    # values and a decay that are no numbers, in one chunk; a token of a later one forgets them
    x = made(1, 500, 3, 128, 128, seed=3)
    x["v"][0, 30, 0], x["k"][0, 30, 1], x["log_decay"][0, 30, 2] = math.inf, math.nan, math.nan
    x["log_decay"][0, 200] = -math.inf
    out, state = pkg.linear_attend(**x)
    y = {n: t.clone() for n, t in x.items()}
    for n in y:
        y[n][:, :128] = 0
    want, after = pkg.linear_attend(**y)
    assert torch.equal(out[:, 200:], want[:, 200:]) and torch.equal(state, after)
    assert not out[0, 128:200].isfinite().any()
