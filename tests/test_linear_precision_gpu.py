"""The state that prompts leave on the tensor cores is a 32-bit one: against the
64-bit recurrence, by norm."""
import pytest
import torch

import gated_delta_rule_32_gb300 as pkg
from tests import _linear_oracle as plain
from tests.test_linear_gpu import made

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    from gated_delta_rule_32_gb300 import build, kda
    build.build()
    kda.load()


@pytest.mark.parametrize("dk,dv", [(128, 128), (64, 64), (64, 128), (128, 64)])
@pytest.mark.parametrize("T,H,rate", [(1, 8, -4.0), (77, 8, -4.0), (128, 4, -1.0), (300, 4, 0.0), (1000, 4, -9.0),
                                      (5000, 2, -4.0), (5000, 2, -9.0)])
def test_states(T, H, rate, dk, dv):
    # a weighted value is the product of two exponentials (2^-22 each at most, uniform: 2^-22.8) and
    # a 16-bit value, in three parts that keep its 24 bits; a chunk's 128 products are summed in
    # fp32, and so is one update a chunk, their roundings uniform and independent: 2^-24 each of
    # sums whose squares add up to some log2(128) = 7 times the last one's (2^-23.4), and of the
    # chunks that count.  In all below 2^-21 of the norm (two parts of a value leave 2^-18.7)
    x = made(2 if T < 1000 else 1, T, H, H, dk, dv, seed=T + dk, rate=rate)
    out, state = pkg.linear_attend(**x, scale=0.3)
    o, s, om, sm = plain.attend(x["q"], x["k"], x["v"], x["log_decay"], x["init_state"], 0.3)
    assert (state.double() - s).norm() <= 2.0 ** -21 * s.norm()
    again = {n: x[n] for n in ("q", "k", "v", "log_decay")}
    _, state = pkg.linear_attend(**again, scale=0.3)
    _, s, _, sm = plain.attend(*again.values(), None, 0.3)
    assert (state.double() - s).norm() <= 2.0 ** -21 * s.norm()


def test_a_value_of_many_magnitudes():
    # single products: no sum hides what a part leaves out (k picks a row of the state each)
    x = made(1, 64, 2, 2, 64, 64, init=False, seed=3)
    x["k"] = torch.eye(64, device="cuda", dtype=torch.bfloat16)[None, :, None].expand(1, 64, 2, 64).contiguous()
    x["v"] = (x["v"].float() * torch.exp2(torch.randint(-60, 60, x["v"].shape, device="cuda").float())).bfloat16()
    _, state = pkg.linear_attend(**x)
    _, s, _, _ = plain.attend(x["q"], x["k"], x["v"], x["log_decay"], None, 1.0)
    # each exponential 2^-22 and the rounding of what it is taken of (sums of log2-decays: up to
    # 2^-24 of them, times ln 2), products 2^-24, parts 2^-24
    g = x["log_decay"].double().flip(1).cumsum(1).flip(1).abs()[0] / 0.693          # [T, H], at least each sum
    tol = (2 * 2.0 ** -22 + 4 * 2.0 ** -24 + 0.7 * 2.0 ** -24 * 2 * g).T[:, :, None] * s[0].abs()
    assert ((state[0].double() - s[0]).abs() <= tol).all()
