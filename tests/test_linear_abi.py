"""Linear attention and rotary positions: bad host-visible arguments are
refused before anything is queued, and the plain forms that the GPU tests
compare with are pinned.  CPU only."""
import math

import pytest
import torch

import gated_delta_rule_32_gb300 as pkg
from gated_delta_rule_32_gb300 import kda
from tests import _linear_oracle as plain

A = 1 << 28   # fake, aligned addresses far apart: never dereferenced on the host


@pytest.fixture(scope="module", autouse=True)
def lib():
    from gated_delta_rule_32_gb300 import build
    build.build()
    return kda.load()


def _fwd(**over):
    a = dict(q=A, q_stride=512, k=2 * A, k_stride=512, v=3 * A, v_stride=1024, log_decay=4 * A,
             decay_stride=8, init_state=5 * A, out=6 * A, final_state=7 * A, B=2, T=50, H=8, Hk=4,
             dk=128, dv=128)
    a.update(over)
    return kda.kda_linear_fwd(**a)


def _decode(**over):
    a = dict(q=A, q_stride=512, k=2 * A, k_stride=512, v=3 * A, v_stride=1024, log_decay=4 * A,
             decay_stride=8, state=5 * A, out=6 * A, N=2, T=1, H=8, Hk=4, dk=128, dv=128)
    a.update(over)
    return kda.kda_linear_decode(**a)


def _rotary(**over):
    a = dict(q=A, q_stride=1024, q_out=2 * A, q_out_stride=512, k=A + 1024, k_stride=1024,
             k_out=3 * A, k_out_stride=256, positions=4 * A, frequencies=5 * A, T=20, Hq=8, Hk=4,
             d=64, part=64)
    a.update(over)
    return kda.kda_rotary(**a)


INV, UNS, MIS = kda.KDA_ERR_INVALID_ARG, kda.KDA_ERR_UNSUPPORTED, kda.KDA_ERR_MISALIGNED


@pytest.mark.parametrize("call,name", [
    (c, n) for c, ns in ((_fwd, "q k v log_decay out"), (_decode, "q k v log_decay state out"),
                         (_rotary, "q q_out k k_out positions frequencies")) for n in ns.split()])
def test_null_pointers(call, name):
    assert call(**{name: None}) == INV


@pytest.mark.parametrize("call,name", [
    (c, n) for c, ns in ((_fwd, "q k v log_decay init_state out final_state cu_seqlens dev_status"),
                         (_decode, "q k v log_decay state out"),
                         (_rotary, "q q_out k k_out positions frequencies")) for n in ns.split()])
@pytest.mark.parametrize("off", [1, 2])
def test_misaligned_pointers(call, name, off):
    assert call(**{name: 40 * A + off}) == MIS


@pytest.mark.parametrize("call,over,code", [
    (_fwd, dict(B=0), INV), (_fwd, dict(T=-1), INV), (_fwd, dict(H=0), INV), (_fwd, dict(Hk=0), INV),
    (_fwd, dict(Hk=3), INV), (_fwd, dict(Hk=16), INV), (_fwd, dict(dk=96), UNS), (_fwd, dict(dv=256), UNS),
    (_fwd, dict(dtype=2), UNS), (_fwd, dict(H=65544, v_stride=65544 * 128, decay_stride=65544), UNS),
    (_fwd, dict(B=1 << 26), UNS), (_fwd, dict(q_stride=504), INV), (_fwd, dict(k_stride=0), INV),
    (_fwd, dict(v_stride=1016), INV), (_fwd, dict(q_stride=516), MIS), (_fwd, dict(v_stride=1028), MIS),
    (_fwd, dict(decay_stride=7), INV), (_fwd, dict(decay_stride=-8), INV),
    (_fwd, dict(q_stride=1 << 31), UNS),
    (_fwd, dict(out=A), INV), (_fwd, dict(out=3 * A + 2048), INV), (_fwd, dict(out=4 * A), INV),
    (_fwd, dict(out=5 * A), INV), (_fwd, dict(final_state=6 * A), INV),
    (_fwd, dict(final_state=5 * A + 65536), INV), (_fwd, dict(final_state=2 * A), INV),
    (_fwd, dict(cu_seqlens=6 * A + 4), INV),
    (_fwd, dict(workspace=8 * A + 128, workspace_bytes=1 << 30), MIS),
    (_decode, dict(N=0), INV), (_decode, dict(T=-1), INV), (_decode, dict(dk=8), UNS),
    (_decode, dict(out=5 * A), INV), (_decode, dict(state=A), INV), (_decode, dict(v_stride=8), INV),
    (_rotary, dict(T=-1), INV), (_rotary, dict(Hq=0, Hk=0), INV), (_rotary, dict(Hq=-1), INV),
    (_rotary, dict(d=0), INV), (_rotary, dict(part=0), INV), (_rotary, dict(part=80), INV),
    (_rotary, dict(part=24), UNS), (_rotary, dict(d=72, q_out_stride=576, k_out_stride=288), UNS),
    (_rotary, dict(d=528, q_stride=8448, q_out_stride=4224, k_stride=8448, k_out_stride=2112), UNS),
    (_rotary, dict(dtype=3), UNS), (_rotary, dict(q_stride=500), INV), (_rotary, dict(k_out_stride=248), INV),
    (_rotary, dict(q_stride=1028), MIS), (_rotary, dict(q_out_stride=516), MIS),
    (_rotary, dict(q_out=A), INV),              # over the input, at another distance
    (_rotary, dict(q_out=A + 1024, q_out_stride=1024), INV),            # over the keys
    (_rotary, dict(k_out=2 * A), INV), (_rotary, dict(k_out=2 * A + 512, k_out_stride=512), INV),
    (_rotary, dict(q_out=4 * A), INV), (_rotary, dict(k_out=5 * A), INV),
    (_rotary, dict(q_stride=1 << 31), UNS),
])
def test_refusals(call, over, code):
    assert call(**over) == code


def test_nothing_to_do():
    assert _rotary(T=0) == kda.KDA_OK
    assert _decode(T=0) == kda.KDA_OK


def test_workspace_query():
    f = kda.kda_linear_workspace_bytes
    assert f(0, 5, 1, 64, 64) == 0 and f(1, -1, 1, 64, 64) == 0 and f(1, 5, 0, 64, 64) == 0
    assert f(1, 5, 1, 48, 64) == 0 and f(1, 5, 1, 64, 64, 7) == 0
    assert f(1, 5000, 2, 16, 16) == 0 and f(1, 5000, 2, 64, 64, kda.KDA_F32) == 0


def test_tensor_calls_refuse_cpu_tensors():
    x = torch.zeros(1, 4, 2, 64)
    with pytest.raises(ValueError, match="CUDA"):
        pkg.linear_attend(x, x, x, torch.zeros(2))
    with pytest.raises(ValueError, match="CUDA"):
        pkg.linear_decode(x, x, x, torch.zeros(2), torch.zeros(1, 2, 64, 64))
    with pytest.raises(ValueError, match="CUDA"):
        pkg.rotary_embed(x[0], x[0], torch.zeros(4, dtype=torch.int32), torch.zeros(32, dtype=torch.float64))


# ---- frequencies

def test_frequencies():
    f, amp = pkg.rotary_frequencies(8, device="cpu")
    assert amp == 1.0 and torch.allclose(f, torch.tensor([1.0, 0.1, 0.01, 0.001], dtype=torch.float64), rtol=1e-14)
    g, amp = pkg.rotary_frequencies(8, scaling="linear", factor=4.0, device="cpu")
    assert amp == 1.0 and torch.allclose(g, f / 4, rtol=1e-14)
    g, amp = pkg.rotary_frequencies(8, scaling="ntk", factor=4.0, device="cpu")
    assert amp == 1.0 and g[0] == 1.0 and math.isclose(g[-1], f[-1] / 4, rel_tol=1e-12)
    f, _ = pkg.rotary_frequencies(128, device="cpu")
    g, amp = pkg.rotary_frequencies(128, scaling="yarn", factor=8.0, trained=4096, device="cpu")
    assert math.isclose(amp, 0.1 * math.log(8) + 1)
    turns = 4096 * f / (2 * math.pi)
    assert torch.equal(g[turns > 36], f[turns > 36]) and torch.allclose(g[turns < 0.9], f[turns < 0.9] / 8, rtol=1e-14)
    r = g / f
    assert (r.diff() <= 1e-15).all() and ((r > 0.126) & (r < 0.999)).sum() > 10
    for bad in (dict(part=7), dict(part=8, scaling="other"), dict(part=8, factor=0.5), dict(part=2, scaling="ntk"),
                dict(part=8, scaling="yarn", fast=1.0)):
        with pytest.raises(ValueError):
            pkg.rotary_frequencies(**bad, device="cpu")


# ---- pins of the plain forms

def test_plain_attention_by_sums():
    # o_t = scale sum_j e^(a_(j+1) + .. + a_t) (q_t . k_j) v_j + the initial state's part
    g = torch.Generator().manual_seed(1)
    q, k = (torch.randn(1, 9, 2, 3, generator=g, dtype=torch.float64) for _ in "qk")
    v = torch.randn(1, 9, 4, 5, generator=g, dtype=torch.float64)
    a = -torch.rand(1, 9, 4, generator=g, dtype=torch.float64)
    a[0, 4, 1], a[0, 2, 0] = -math.inf, 3.0
    s0 = torch.randn(2, 4, 3, 5, generator=g, dtype=torch.float64)
    lens = [3, 6]
    out, s, om, sm = plain.attend(q, k, v, a, s0, 0.7, lens)
    for n, (x, y) in enumerate(((0, 3), (3, 9))):
        for h in range(4):
            for t in range(x, y):
                w = [math.exp(sum(min(a[0, i, h].item(), 0.0) for i in range(j + 1, t + 1))) for j in range(x - 1, t + 1)]
                o = w[0] * (q[0, t, h // 2] @ s0[n, h]) + sum(
                    w[j - x + 1] * (q[0, t, h // 2] @ k[0, j, h // 2]) * v[0, j, h] for j in range(x, t + 1))
                assert torch.allclose(out[0, t, h], 0.7 * o, atol=1e-12)
                assert (om[0, t, h] >= out[0, t, h].abs() - 1e-12).all()
    assert (sm >= s.abs() - 1e-12).all()


def test_plain_turn_by_complex_numbers():
    g = torch.Generator().manual_seed(2)
    x = torch.randn(4, 2, 8, generator=g, dtype=torch.float64)
    f = torch.tensor([1.0, 0.01], dtype=torch.float64)
    pos = torch.tensor([0, 3, -1, 100000])
    for inter in (False, True):
        y = plain.turn(x, pos, f, interleaved=inter, amplitude=1.5)
        a, b = (x[..., 0:4:2], x[..., 1:4:2]) if inter else (x[..., :2], x[..., 2:4])
        z = torch.complex(a, b) * 1.5 * torch.exp(1j * pos.double()[:, None] * f)[:, None]
        c = torch.complex(*((y[..., 0:4:2], y[..., 1:4:2]) if inter else (y[..., :2], y[..., 2:4])))
        on = pos >= 0
        assert torch.allclose(c[on], z[on], atol=1e-9) and torch.equal(y[on][..., 4:], x[on][..., 4:])
        assert y[2].isnan().all()
