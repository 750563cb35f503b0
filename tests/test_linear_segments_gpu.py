"""Packed batches whose token axis is cut into segments, against the 64-bit
recurrence: columns, entry states, the scan, and what passes through segments'
factors.  Each case asks for scratch first, which only cut ones need."""
import math

import pytest
import torch

import gated_delta_rule_32_gb300 as pkg
from gated_delta_rule_32_gb300 import kda
from tests import _linear_oracle as plain
from tests.test_linear_gpu import check, made, status

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module", autouse=True)
def built():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    from gated_delta_rule_32_gb300 import build
    build.build()
    kda.load()


def is_cut(lens, H, dk, dv):
    return kda.kda_linear_workspace_bytes(len(lens), sum(lens), H, dk, dv, packed=1) > 0


def offsets(lens):
    return torch.tensor([sum(lens[:i]) for i in range(len(lens) + 1)], dtype=torch.int32, device="cuda")


CASES = [
    ([4000, 0, 1000], 3, 128, 128), ([700, 64, 1900], 3, 128, 128),
    ([2560, 1280, 1280], 2, 128, 128),          # borders on multiples of 128, segments' own among them
    ([1280] * 4, 1, 64, 128), ([768, 0, 0, 1536, 384, 2304], 3, 128, 64),
    ([3000, 2000], 1, 128, 64), ([1, 4998, 1], 1, 64, 64),
    ([9000, 1, 1, 1, 1, 1], 4, 64, 64), ([1] * 10 + [8000], 2, 128, 128), ([0, 0, 5000], 3, 64, 64),
    ([129, 255, 257, 127, 6000, 0, 385], 1, 128, 128), ([5120], 2, 128, 64),
]


@pytest.mark.parametrize("lens,H,dk,dv", CASES)
def test_against_64_bits(lens, H, dk, dv):
    assert is_cut(lens, H, dk, dv)
    T = sum(lens)
    check(made(1, T, H, 1, dk, dv, N=len(lens), seed=T, views=True), lens)
    # slow decays: what a segment starts from counts in all of its tokens
    check(made(1, T, H, H, dk, dv, N=len(lens), init=H > 1, decay="token" if H > 1 else "head", seed=T + 2,
               rate=-9.0), lens)


@pytest.mark.parametrize("lens,H,dk,dv", CASES[:5])
def test_in_place_and_rows_behind_the_last(lens, H, dk, dv):
    T = sum(lens)
    x = made(1, T + 300, H, H, dk, dv, N=len(lens), seed=T)
    assert kda.kda_linear_workspace_bytes(len(lens), T + 300, H, dk, dv, packed=1) > 0
    for name in ("q", "k", "v", "log_decay"):
        x[name][:, T:] = math.nan
    out = torch.full((T + 300, H, dv), 3.0, dtype=BF, device="cuda")
    state, st = x["init_state"].clone(), status()
    rc = kda.kda_linear_fwd(x["q"], H * dk, x["k"], H * dk, x["v"], H * dv, x["log_decay"], H, state, out, state,
                            len(lens), T + 300, H, H, dk, dv, offsets(lens), scale=0.3, dev_status=st,
                            stream=torch.cuda.current_stream())
    assert rc == 0 and st.item() == 0 and bool((out[T:] == 3.0).all())
    o, s, om, sm = plain.attend(*(x[n][:, :T] for n in ("q", "k", "v", "log_decay")), x["init_state"], 0.3, lens)
    # (one rounding to 16 bits of each weight or state element, and the output's: see test_linear_gpu)
    tol = (plain.BF16 + 2.0 ** -14) * om[0]
    tol = tol + plain.BF16 * (o[0].abs() + tol)
    assert ((out[:T].double() - o[0]).abs() <= tol).all()
    assert ((state.double() - s).abs() <= 2.0 ** -16 * sm).all()


@pytest.mark.parametrize("lens,H", [([4000, 0, 1000], 3), ([5000], 3), ([1280] * 4, 2)])
def test_decays_at_the_ends(lens, H):
    # all that is before forgotten at single tokens, at and around multiples of 128, factors that vanish
    T = sum(lens)
    assert is_cut(lens, H, 128, 128)
    x = made(1, T, H, H, 128, 128, N=len(lens), seed=9)
    a = x["log_decay"]
    for t in (0, 127, 128, 383, 384, 1279, 1280, 1281, 2559, 2560, 4001, T - 1):
        a[:, t, t % H] = -math.inf
    a[:, 1500:1700, 0] = -90.0 * torch.rand(200, device="cuda")
    a[:, 2000:2200:3, 1] = -1e30
    a[:, 600:900, 0] = 2.0
    check(x, lens)


@pytest.mark.parametrize("at", [0, 383, 384, 2000, 3999, 4000, 4999])
def test_a_decay_that_is_nan(at):
    lens, H = [4000, 0, 1000], 3
    x = made(1, 5000, H, H, 128, 128, N=3, seed=5)
    assert is_cut(lens, H, 128, 128)
    cu = offsets(lens)
    want, ws = pkg.linear_attend(**x, cu_seqlens=cu)
    x["log_decay"][0, at, 1] = math.nan
    out, state = pkg.linear_attend(**x, cu_seqlens=cu)
    n, end = (0, 4000) if at < 4000 else (2, 5000)
    assert out[0, at:end, 1].isnan().all() and state[n, 1].isnan().all()
    for t in (out, want):
        t[0, at:end, 1] = 0
    for s in (state, ws):
        s[n, 1] = 0
    assert torch.equal(out, want) and torch.equal(state, ws)


def test_a_sequence_of_nan_stays_alone():
    lens, H = [1500, 2000, 1500], 2
    x = made(1, 5000, H, H, 128, 128, N=3, seed=5)
    assert is_cut(lens, H, 128, 128)
    cu = offsets(lens)
    want, ws = pkg.linear_attend(**x, cu_seqlens=cu)
    for name in ("q", "k", "v", "log_decay"):
        x[name][:, 1500:3500] = math.nan
    x["init_state"][1] = math.inf
    out, state = pkg.linear_attend(**x, cu_seqlens=cu)
    assert out[:, 1500:3500].isnan().all() and state[1].isnan().all()
    for part in (slice(0, 1500), slice(3500, 5000)):
        assert torch.equal(out[:, part], want[:, part])
    assert torch.equal(state[::2], ws[::2])


@pytest.mark.parametrize("cu", [[0, 3000, 1000, 5000], [5, 2500, 5000], [0, 2500, 5001], [0, -1, 5000],
                                [0, 9000, 5000], [0, 2 ** 31 - 1, 5000], [0, 5000, 5000, 60],
                                [0, -2 ** 31, 5000], [0, 100, 50, 5000, 4000, 5000]])
def test_malformed_offsets(cu):
    # reported, whatever the search over them makes of it; nothing outside the rows is touched
    H, N = 2, len(cu) - 1
    x = made(1, 5000, H, H, 64, 64, N=N, seed=3)
    nb = kda.kda_linear_workspace_bytes(N, 5000, H, 64, 64, packed=1)
    assert nb > 0
    room = torch.full((5000 * H * 64 + 128,), 7.0, dtype=BF, device="cuda")
    ws = torch.full((nb + 512,), 9, dtype=torch.uint8, device="cuda")
    final = torch.full((N * H * 64 * 64 + 64,), 5.0, device="cuda")
    st = status()
    rc = kda.kda_linear_fwd(x["q"], H * 64, x["k"], H * 64, x["v"], H * 64, x["log_decay"], H, x["init_state"],
                            room[64:], final[32:], N, 5000, H, H, 64, 64,
                            torch.tensor(cu, dtype=torch.int32, device="cuda"), workspace=ws[256:],
                            workspace_bytes=nb, dev_status=st, stream=torch.cuda.current_stream())
    assert rc == 0 and st.item() == kda.KDA_ERR_BAD_SEQLENS
    assert (room[:64] == 7).all() and (room[-64:] == 7).all()
    assert (ws[:256] == 9).all() and (ws[-256:] == 9).all()
    assert (final[:32] == 5).all() and (final[-32:] == 5).all()
