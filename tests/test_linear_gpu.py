"""Linear attention with a decay for each head on the GPU against the 64-bit
recurrence (_linear_oracle), by bounds that follow what each result sums."""
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


def made(B, T, H, Hk, dk, dv, dtype=BF, decay="token", init=True, views=False, N=None, seed=0, rate=-4.0):
    g = torch.Generator(device="cuda").manual_seed(seed)

    def normal(*shape):
        return torch.randn(*shape, generator=g, device="cuda")
    q, k = (torch.nn.functional.normalize(normal(B, T, Hk, dk), dim=-1).to(dtype) for _ in "qk")
    v = normal(B, T, H, dv).to(dtype)
    if views:
        x = torch.cat([y.flatten(2) for y in (q, k, v)] + [normal(B, T, 8).to(dtype)], 2)
        q, k, v = (y.unflatten(2, shape) for y, shape in zip(x.split([Hk * dk, Hk * dk, H * dv, 8], 2),
                                                             ((Hk, dk), (Hk, dk), (H, dv))))
    a = -torch.exp(normal(H) * 1.5 + rate)
    if decay == "token":
        a = a * torch.nn.functional.softplus(normal(B, T, H) + 1.0)
    s = normal(N or B, H, dk, dv) if init else None
    return dict(q=q, k=k, v=v, log_decay=a, init_state=s)


def status():
    return torch.full((1,), 77, dtype=torch.int32, device="cuda")


def check(x, lens=None, scale=0.3, call=None, rows=None):
    """Runs a case and compares it.  Per token and element, results may err
    beside the output's own rounding
      on the tensor cores: by one rounding to 16 bits of each weight (within a
      chunk) or element of the state, and 2^-16 in what a token adds to the
      state (two 16-bit parts of it, 2^-9 of 2^-8 each, and fp32 sums);
      token by token: by an fp32 rounding for each token that still counts."""
    st = status()
    cu = None if lens is None else torch.tensor([sum(lens[:i]) for i in range(len(lens) + 1)],
                                                dtype=torch.int32, device="cuda")
    if call is None:
        out, state = pkg.linear_attend(**x, cu_seqlens=cu, scale=scale, dev_status=st)
        assert st.item() == 0
    else:
        out, state = call(cu)
    o, s, om, sm = plain.attend(x["q"], x["k"], x["v"], x["log_decay"], x["init_state"], scale, lens)
    live = ~o.isnan()
    assert out.dtype == x["v"].dtype and out.shape == o.shape and state.dtype is F32
    wide = x["q"].dtype is BF and min(x["q"].shape[-1], x["v"].shape[-1]) >= 64 and call is None
    T = x["q"].shape[1]
    if wide:
        tol_o, tol_s = (plain.BF16 + 2.0 ** -14) * om, 2.0 ** -16 * sm
    else:
        tol_o, tol_s = ((T + 300) * 2.0 ** -24) * om, ((T + 4) * 2.0 ** -24) * sm
    if out.dtype is BF:
        tol_o = tol_o + plain.BF16 * (o.abs() + tol_o)
    else:
        tol_o = tol_o + 2.0 ** -24 * o.abs()
    err = (out.double() - o).abs()
    assert (err <= tol_o + 1e-37)[live].all(), (err / (tol_o + 1e-37))[live].max()
    err_s = (state.double() - s).abs()
    assert (err_s <= tol_s + 1e-37).all(), (err_s / (tol_s + 1e-37)).max()
    # roundings of different elements are independent, uniform within their bound at most
    # (variance a third of its square): weights and states, then the output, each at most
    # BF16 / sqrt 3 of the norm of what they make up
    if wide and live.sum() > 4000:
        assert (out.double() - o)[live].norm() <= plain.BF16 * o[live].norm()
        assert (state.double() - s).norm() <= 2.0 ** -16 * s.norm()
    return out, state


@pytest.mark.parametrize("T", [0, 1, 2, 15, 17, 63, 64, 65, 127, 128, 129, 300])
@pytest.mark.parametrize("dk,dv", [(128, 128), (64, 64), (64, 128), (128, 64)])
def test_lengths(T, dk, dv):
    check(made(2, T, 3, 3, dk, dv, seed=T + dk))


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("dk,dv", [(16, 16), (16, 128), (32, 64), (128, 32), (64, 16), (128, 128)])
def test_head_sizes_token_by_token(dtype, dk, dv):
    check(made(2, 37, 2, 1, dk, dv, dtype, seed=dk + dv))


@pytest.mark.parametrize("decay", ["token", "head"])
@pytest.mark.parametrize("init", [True, False])
@pytest.mark.parametrize("H,Hk", [(1, 1), (6, 2), (8, 1), (5, 5)])
def test_heads_and_views(H, Hk, init, decay):
    check(made(3, 200, H, Hk, 128, 64, decay=decay, init=init, views=True, seed=H))


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("lens", [
    [0], [1], [0, 0, 5], [130, 0, 1, 128, 127, 129, 0, 64], [1] * 70, [i % 5 for i in range(300)],
    [700, 3, 256], [0, 384, 0, 0],
])
def test_packed(lens, dtype):
    T = sum(lens)
    check(made(1, T, 2, 2, 128, 128, dtype, N=len(lens), seed=T), lens)
    check(made(1, T, 4, 2, 64, 64, dtype, N=len(lens), views=True, init=False, seed=T), lens)


@pytest.mark.parametrize("n", [1023, 1024, 1025, 3000])
def test_many_sequences(n):
    # put in order up to 1024, as they come beyond
    lens = [(i * 37) % 4 for i in range(n)]
    check(made(1, sum(lens), 1, 1, 64, 64, N=n, seed=n), lens)


def test_one_token_rows_and_strided_decays():
    x = made(5, 1, 3, 3, 128, 64, views=True, seed=6)
    wide = torch.zeros(5, 1, 8, device="cuda")
    wide[..., 2:5] = x["log_decay"]
    x["log_decay"] = wide[..., 2:5]
    check(x)
    x = made(2, 300, 3, 3, 64, 64, seed=7)
    wide = torch.zeros(2, 300, 8, device="cuda")
    wide[..., 4:7] = x["log_decay"]
    x["log_decay"] = wide[..., 4:7]
    check(x)


def test_an_output_between_sectors():
    # 16-byte aligned is enough
    x = made(1, 260, 2, 2, 128, 128, seed=8)
    want, _ = pkg.linear_attend(**x)
    room = torch.full((260 * 256 + 16,), 7.0, dtype=BF, device="cuda")
    out = room[8:8 + 260 * 256]
    assert out.data_ptr() % 32 == 16
    rc = kda.kda_linear_fwd(x["q"], 256, x["k"], 256, x["v"], 256, x["log_decay"], 2, x["init_state"], out,
                            None, 1, 260, 2, 2, 128, 128, stream=torch.cuda.current_stream())
    assert rc == 0 and torch.equal(out.view(want.shape), want)
    assert (room[:8] == 7).all() and (room[-8:] == 7).all()


def test_tensor_calls_refuse_what_does_not_fit():
    x = made(2, 10, 4, 2, 64, 64, seed=1)
    cu = torch.tensor([0, 10], dtype=torch.int32, device="cuda")
    for over in (dict(k=x["k"][:, :5]), dict(v=x["v"].float()), dict(q=x["q"].half()), dict(v=x["v"][:, :, :3]),
                 dict(log_decay=x["log_decay"][:, :, :2]), dict(log_decay=x["log_decay"].to(BF)),
                 dict(init_state=x["init_state"][:1]), dict(init_state=x["init_state"].to(BF)),
                 dict(q=x["q"].transpose(1, 2)), dict(k=x["k"].cpu()), dict(cu_seqlens=cu),
                 dict(cu_seqlens=cu.long()), dict(q=x["q"][..., ::2], k=x["k"][..., ::2])):
        with pytest.raises((ValueError, kda.KdaError)):
            pkg.linear_attend(**(x | over))
    s = x["init_state"]
    d = {n: x[n] for n in ("q", "k", "v", "log_decay")}
    for bad in (s[:, :2], s.transpose(2, 3), s.double(), s[:1]):
        with pytest.raises(ValueError):
            pkg.linear_decode(**d, state=bad)


def test_rows_behind_the_last_sequence_stay():
    x = made(1, 400, 2, 2, 128, 128, N=2, seed=1)
    cu = torch.tensor([0, 130, 257], dtype=torch.int32, device="cuda")
    for name in "qkv":
        x[name][:, 257:] = math.nan         # what nobody wrote
    x["log_decay"][:, 257:] = math.nan
    out = torch.full((400, 2, 128), 3.0, dtype=BF, device="cuda")
    state = torch.empty(2, 2, 128, 128, device="cuda")
    st = status()
    rc = kda.kda_linear_fwd(x["q"], 256, x["k"], 256, x["v"], 256, x["log_decay"], 2, x["init_state"],
                            out, state, 2, 400, 2, 2, 128, 128, cu, scale=0.3, dev_status=st,
                            stream=torch.cuda.current_stream())
    assert rc == 0 and st.item() == 0
    assert (out[257:] == 3.0).all()
    o, s, om, sm = plain.attend(x["q"], x["k"], x["v"], x["log_decay"], x["init_state"], 0.3, [130, 127])
    tol = (2.2 * plain.BF16) * om[0, :257] + plain.BF16 * o[0, :257].abs()
    assert ((out[:257].double() - o[0, :257]).abs() <= tol).all()
    assert ((state.double() - s).abs() <= 2.0 ** -16 * sm).all()


def test_a_sequence_of_nan_stays_alone():
    lens = [100, 60, 200]
    x = made(1, 360, 2, 2, 128, 128, N=3, seed=5)
    for name in "qkv":
        x[name][:, 100:160] = math.nan
    x["init_state"][1] = math.inf
    st = status()
    cu = torch.tensor([0, 100, 160, 360], dtype=torch.int32, device="cuda")
    out, state = pkg.linear_attend(**x, cu_seqlens=cu, scale=0.3, dev_status=st)
    clean = {n: torch.where(t.isfinite(), t, 0.0).to(t.dtype) for n, t in x.items()}
    want, ws = pkg.linear_attend(**clean, cu_seqlens=cu, scale=0.3)
    assert out[:, 100:160].isnan().all()
    for part in (slice(0, 100), slice(160, 360)):
        assert torch.equal(out[:, part], want[:, part])
    assert torch.equal(state[::2], ws[::2]) and not state[1].isfinite().any()


@pytest.mark.parametrize("dk,dv", [(128, 128), (64, 64)])
def test_short_and_ragged_ones_in_turn(dk, dv):
    # hundreds of sequences that end inside a chunk, many on each SM, whatever the warps' pace
    lens = [1 + (i * 7919) % 301 for i in range(100)]
    x = made(1, sum(lens), 8, 2, dk, dv, N=len(lens), seed=3)
    out, state = check(x, lens)
    cu = torch.tensor([0] + lens, device="cuda").cumsum(0).to(torch.int32)
    for _ in range(30):
        torch.cuda.synchronize()
        again = pkg.linear_attend(**x, cu_seqlens=cu, scale=0.3)
        assert torch.equal(again[0], out) and torch.equal(again[1], state)


@pytest.mark.parametrize("dtype", [BF, F32])
def test_decays_at_the_ends(dtype):
    # nothing forgotten, everything forgotten at single tokens, factors that vanish in 32 bits, values above 0
    x = made(1, 333, 4, 4, 64, 64, dtype, seed=9)
    a = torch.zeros(1, 333, 4, device="cuda")
    a[:, 40, 1] = -math.inf
    a[:, 128, 1] = -math.inf
    a[:, 255, 1] = -math.inf
    a[:, :, 2] = -90.0 * torch.rand(333, device="cuda")
    a[:, ::3, 2] = -1e30
    a[:, :, 3] = torch.where(torch.rand(333, device="cuda") < 0.5, 2.0, -0.3)
    x["log_decay"] = a
    check(x)


def test_long_windows_keep_their_sums():
    # a decay so slow that thousands of tokens count, over many chunks and segments of the token axis
    x = made(1, 20000, 1, 1, 128, 128, decay="head", init=True, seed=2)
    x["log_decay"] = torch.full((1,), -1e-4, device="cuda")
    check(x)


@pytest.mark.parametrize("T,H", [(5000, 2), (3333, 7)])
def test_few_heads_long_rows(T, H):
    check(made(1, T, H, 1, 128, 64, seed=T, views=True))
    check(made(1, T, H, H, 64, 128, decay="head", init=False, seed=T))


def test_packed_long_and_short():
    lens = [2500, 1, 40, 0, 1300, 128]
    check(made(1, sum(lens), 2, 2, 128, 128, N=len(lens), seed=4), lens)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("T", [1, 2, 8, 9, 20])
@pytest.mark.parametrize("N,H,Hk,dk,dv", [(1, 1, 1, 128, 128), (5, 6, 3, 128, 64), (3, 4, 4, 16, 32), (70, 8, 2, 64, 128)])
def test_decode(N, H, Hk, dk, dv, T, dtype):
    x = made(N, T, H, Hk, dk, dv, dtype, views=T % 2 == 0, seed=N + T)

    def call(_):
        state = x["init_state"].clone()
        return pkg.linear_decode(x["q"], x["k"], x["v"], x["log_decay"], state, scale=0.3), state
    check(x, call=call)


def test_state_in_place_and_in_pieces():
    # a prompt in one call, and in three with the state handed over in place
    x = made(2, 300, 4, 2, 128, 128, seed=8)
    _, whole = check(x)
    state = x["init_state"].clone()
    outs = []
    for a, b in ((0, 130), (130, 131), (131, 300)):
        piece = {n: x[n][:, a:b].contiguous() for n in ("q", "k", "v", "log_decay")}
        out = torch.empty(2, b - a, 4, 128, dtype=BF, device="cuda")
        rc = kda.kda_linear_fwd(piece["q"], 256, piece["k"], 256, piece["v"], 512, piece["log_decay"], 4,
                                state, out, state, 2, b - a, 4, 2, 128, 128, scale=0.3,
                                stream=torch.cuda.current_stream())
        assert rc == 0
        outs.append(out)
    o, s, om, sm = plain.attend(x["q"], x["k"], x["v"], x["log_decay"], x["init_state"], 0.3)
    tol = (2.2 * plain.BF16) * om + plain.BF16 * o.abs()
    assert ((torch.cat(outs, 1).double() - o).abs() <= tol).all()
    assert ((state.double() - s).abs() <= 2.0 ** -15 * sm).all()
    assert ((whole.double() - s).abs() <= 2.0 ** -16 * sm).all()


@pytest.mark.parametrize("T,H,lens", [(6000, 2, None), (40000, 4, None), (5000, 3, [4000, 0, 1000])])
def test_state_in_place_over_segments(T, H, lens):
    # one buffer for the states before and after, long rows of few heads: segments read the one
    # while others write the other
    N = 1 if lens is None else len(lens)
    x = made(1, T, H, H, 128, 128, N=N, seed=T)
    cu = None if lens is None else torch.tensor([0, 4000, 4000, 5000], dtype=torch.int32, device="cuda")
    want, after = pkg.linear_attend(**x, cu_seqlens=cu, scale=0.3)
    for _ in range(10):
        state = x["init_state"].clone()
        out = torch.empty_like(want)
        rc = kda.kda_linear_fwd(x["q"], H * 128, x["k"], H * 128, x["v"], H * 128, x["log_decay"], H, state,
                                out, state, N, T, H, H, 128, 128, cu, scale=0.3,
                                stream=torch.cuda.current_stream())
        assert rc == 0
        assert torch.equal(out, want) and torch.equal(state, after)


def test_a_decay_that_is_nan():
    # what follows it in its head and sequence is NaN, nothing else
    lens = [300, 200]
    x = made(1, 500, 3, 3, 128, 64, N=2, seed=5)
    cu = torch.tensor([0, 300, 500], dtype=torch.int32, device="cuda")
    want, ws = pkg.linear_attend(**x, cu_seqlens=cu)
    x["log_decay"][0, 142, 1] = math.nan
    out, state = pkg.linear_attend(**x, cu_seqlens=cu)
    assert out[0, 142:300, 1].isnan().all() and state[0, 1].isnan().all()
    for t in (out, want):
        t[0, 142:300, 1] = 0
    assert torch.equal(out, want)
    assert torch.equal(state[1], ws[1]) and torch.equal(state[0, ::2], ws[0, ::2])


@pytest.mark.parametrize("cu", [[0, 50, 30, 100], [5, 50, 100], [0, 50, 101], [0, -1, 100], [0, 200, 100],
                                [0, 2 ** 31 - 1, 100], [0, 100, 100, 60]])
@pytest.mark.parametrize("dtype", [BF, F32])
def test_malformed_offsets(cu, dtype):
    x = made(1, 100, 2, 2, 64, 64, dtype, N=len(cu) - 1, seed=3)
    st = status()
    pkg.linear_attend(**x, cu_seqlens=torch.tensor(cu, dtype=torch.int32, device="cuda"), dev_status=st)
    assert st.item() == kda.KDA_ERR_BAD_SEQLENS


def test_the_same_bits_each_time_and_in_a_graph():
    lens = [700, 64, 1900]
    x = made(1, sum(lens), 3, 3, 128, 128, N=3, seed=6)
    cu = torch.tensor([0, 700, 764, 2664], dtype=torch.int32, device="cuda")
    a = pkg.linear_attend(**x, cu_seqlens=cu)
    b = pkg.linear_attend(**x, cu_seqlens=cu)
    assert all(torch.equal(s, t) for s, t in zip(a, b))
    y = made(4, 1, 3, 3, 128, 128, seed=7)
    other = torch.cuda.Stream()
    with torch.cuda.stream(other):          # (warm-up)
        pkg.linear_attend(**x, cu_seqlens=cu)
        pkg.linear_decode(y["q"], y["k"], y["v"], y["log_decay"], y["init_state"].clone())
    torch.cuda.synchronize()
    state = y["init_state"].clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        c = pkg.linear_attend(**x, cu_seqlens=cu)
        d = pkg.linear_decode(y["q"], y["k"], y["v"], y["log_decay"], state)
    for _ in range(2):
        state.copy_(y["init_state"])
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(s, t) for s, t in zip(a, c))
    want = y["init_state"].clone()
    assert torch.equal(d, pkg.linear_decode(y["q"], y["k"], y["v"], y["log_decay"], want))
    assert torch.equal(state, want)
    # other inputs in the same buffers
    x["v"].mul_(2.0)
    graph.replay()
    torch.cuda.synchronize()
    e = pkg.linear_attend(**x, cu_seqlens=cu)
    assert all(torch.equal(s, t) for s, t in zip(e, c))


def test_two_streams_at_once():
    xs = [made(1, 6000, 4, 4, 128, 128, seed=s) for s in (1, 2)]
    want = [pkg.linear_attend(**x) for x in xs]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in xs]
    for _ in range(3):
        got = [pkg.linear_attend(**x, stream=s) for x, s in zip(xs, streams)]
        torch.cuda.synchronize()
        for g, w in zip(got, want):
            assert torch.equal(g[0], w[0]) and torch.equal(g[1], w[1])


def test_the_librarys_own_workspace():
    x = made(1, 5000, 2, 2, 128, 128, seed=3)
    want = pkg.linear_attend(**x)
    out = torch.empty_like(want[0])
    state = torch.empty_like(want[1])
    rc = kda.kda_linear_fwd(x["q"], 256, x["k"], 256, x["v"], 256, x["log_decay"], 2, x["init_state"],
                            out, state, 1, 5000, 2, 2, 128, 128, stream=torch.cuda.current_stream())
    assert rc == 0
    assert torch.equal(out, want[0]) and torch.equal(state, want[1])


def test_no_final_state():
    x = made(2, 150, 2, 2, 128, 128, seed=3)
    want, _ = pkg.linear_attend(**x)
    out = torch.empty_like(want)
    rc = kda.kda_linear_fwd(x["q"], 256, x["k"], 256, x["v"], 256, x["log_decay"], 2, x["init_state"],
                            out, None, 2, 150, 2, 2, 128, 128, stream=torch.cuda.current_stream())
    assert rc == 0 and torch.equal(out, want)
