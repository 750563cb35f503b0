"""The paged 8-bit cache's entry points refuse bad host-visible arguments
before touching the GPU, and the plain forms its GPU tests compare with are
pinned.  CPU only."""
import math

import pytest
import torch

import gated_delta_rule_32_gb300 as pkg
from gated_delta_rule_32_gb300 import kda
from tests import _cache_oracle as plain

A = 1 << 24   # fake, aligned addresses far apart: never dereferenced on the host


@pytest.fixture(scope="module", autouse=True)
def lib():
    from gated_delta_rule_32_gb300 import build
    build.build()
    return kda.load()


def _plan(**over):
    a = dict(new_lens=A, ctx_lens=2 * A, R=3, T=40, page=16, block_table=3 * A, max_pages=8,
             free_pages=4 * A, free_count=5 * A, num_pages=64, cu_seqlens=6 * A, kv_lens=7 * A,
             slots=8 * A, positions=9 * A, runs=10 * A, free_count_out=11 * A)
    a.update(over)
    return kda.kda_page_plan(**a)


def _release(**over):
    a = dict(release=A, R=3, page=16, kv_lens=2 * A, block_table=3 * A, max_pages=8,
             free_pages=4 * A, free_count=5 * A, num_pages=64)
    a.update(over)
    return kda.kda_page_release(**a)


def _append(**over):
    a = dict(k=A, v=2 * A, k_stride=512, v_stride=512, T=40, runs=3 * A, num_runs=8,
             k_codes=4 * A, v_codes=5 * A, k_scale=6 * A, v_scale=7 * A, num_pages=64, page=16,
             Hkv=4, d=128)
    a.update(over)
    return kda.kda_cache_append(**a)


def _attn(**over):
    a = dict(q=A, q_stride=1024, cu_seqlens=2 * A, kv_lens=3 * A, block_table=4 * A, max_pages=8,
             k_codes=5 * A, v_codes=6 * A, k_scale=7 * A, v_scale=8 * A, out=9 * A, lse=10 * A,
             R=3, T=40, max_new=20, Hq=8, Hkv=4, d=128, num_pages=64, page=16)
    a.update(over)
    return kda.kda_cache_attn(**a)


INV, UNS, MIS = kda.KDA_ERR_INVALID_ARG, kda.KDA_ERR_UNSUPPORTED, kda.KDA_ERR_MISALIGNED


@pytest.mark.parametrize("call,name", [
    (c, n) for c, ns in (
        (_plan, "new_lens ctx_lens block_table free_pages free_count cu_seqlens kv_lens slots "
                "positions runs free_count_out"),
        (_release, "release kv_lens block_table free_pages free_count"),
        (_append, "k v runs k_codes v_codes k_scale v_scale"),
        (_attn, "q cu_seqlens kv_lens block_table k_codes v_codes k_scale v_scale out"))
    for n in ns.split()])
def test_null_pointers(call, name):
    assert call(**{name: None}) == INV


@pytest.mark.parametrize("call,over,code", [
    (_plan, dict(R=0), INV), (_plan, dict(T=-1), INV), (_plan, dict(max_pages=0), INV),
    (_plan, dict(num_pages=0), INV), (_plan, dict(page=48), UNS), (_plan, dict(R=16385), UNS),
    (_plan, dict(num_pages=1 << 28), UNS), (_plan, dict(runs=10 * A + 8), MIS),
    (_plan, dict(kv_lens=2 * A), INV),          # lengths out over lengths in
    (_plan, dict(free_count_out=5 * A), INV),
    (_plan, dict(slots=3 * A + 4), INV),        # inside the table
    (_plan, dict(free_pages=3 * A), INV),       # the stack is the table
    (_release, dict(R=0), INV), (_release, dict(page=8), UNS), (_release, dict(max_pages=0), INV),
    (_append, dict(T=-1), INV), (_append, dict(Hkv=0), INV), (_append, dict(num_pages=0), INV),
    (_append, dict(d=96), UNS), (_append, dict(page=256), UNS), (_append, dict(code=2), UNS),
    (_append, dict(Hkv=4097, k_stride=4097 * 128, v_stride=4097 * 128), UNS),
    (_append, dict(T=(1 << 26) + 1), UNS),
    (_plan, dict(T=(1 << 26) + 1), UNS), (_plan, dict(max_pages=1 << 27), UNS),
    (_attn, dict(T=(1 << 26) + 1), UNS), (_attn, dict(max_pages=1 << 27), UNS),
    (_attn, dict(Hkv=4097, Hq=4097, q_stride=4097 * 128), UNS),
    (_append, dict(k_stride=504), INV), (_append, dict(v_stride=516), MIS),
    (_append, dict(k=A + 2), MIS), (_append, dict(v_codes=5 * A + 8), MIS),
    (_append, dict(runs=3 * A + 4), MIS), (_append, dict(k_scale=6 * A + 2), MIS),
    (_append, dict(v_codes=4 * A), INV),        # one pool for both
    (_append, dict(k_codes=A), INV),            # codes over the keys
    (_append, dict(v_scale=6 * A), INV),
    (_attn, dict(R=0), INV), (_attn, dict(T=-1), INV), (_attn, dict(max_new=-1), INV),
    (_attn, dict(Hq=6), INV), (_attn, dict(Hkv=0), INV), (_attn, dict(d=256), UNS),
    (_attn, dict(page=20), UNS), (_attn, dict(code=7), UNS), (_attn, dict(R=20000), UNS),
    (_attn, dict(Hq=520, Hkv=8, q_stride=520 * 128), UNS), (_attn, dict(q_stride=1016), INV),
    (_attn, dict(q_stride=1028), MIS), (_attn, dict(q=A + 8), MIS), (_attn, dict(out=9 * A + 4), MIS),
    (_attn, dict(out=A), INV),                  # out over q
    (_attn, dict(lse=9 * A), INV),              # lse over out
    (_attn, dict(out=5 * A), INV),              # out over the codes
])
def test_refusals(call, over, code):
    assert call(**over) == code


def test_runs_bound():
    f = kda.kda_page_runs
    assert f(64, 64, 64) == 64 and f(17, 40000, 64) == 40000 // 64 + 34
    assert f(1, 0, 16) == 1 and f(0, 5, 16) == 0 and f(1, -1, 16) == 0 and f(1, 5, 24) == 0


def test_status_names():
    assert kda.status_string(kda.KDA_ERR_BAD_PAGES).startswith("KDA_ERR_BAD_PAGES")
    assert kda.status_string(kda.KDA_ERR_NO_PAGES).startswith("KDA_ERR_NO_PAGES")


def test_tensor_calls_refuse_cpu_tensors():
    x = torch.zeros(4, dtype=torch.int32)
    with pytest.raises(ValueError, match="CUDA"):
        pkg.page_plan(x, x, x[:, None], x, x, 4, 16)
    with pytest.raises(ValueError, match="CUDA"):
        pkg.page_release(x, x, x[:, None], x, x, 16)
    c = torch.zeros(2, 1, 16, 64, dtype=torch.int8)
    s = torch.zeros(2, 1)
    with pytest.raises(ValueError, match="CUDA"):
        pkg.cache_append(x, x, x, c, c, s, s)
    with pytest.raises(ValueError, match="CUDA"):
        pkg.cache_attend(x, x, x, x, c, c, s, s)


# ---- pins of the plain forms

def test_plain_plan_by_hand():
    cu, kv, slots, pos, runs, left, table = plain.plan(
        [3, 0, 18], [15, 4, 0], [[9, -1], [2, -1], [-1, -1]], [5, 7, 1], 24, 16, 10)
    assert cu == [0, 3, 3, 21] and kv == [18, 4, 18] and left == 0
    assert table == [[9, 1], [2, -1], [7, 5]]
    assert slots[:3] == [9 * 16 + 15, 16, 17] and slots[3] == 7 * 16 and slots[19:] == [80, 81, -1, -1, -1]
    assert pos[:4] == [15, 16, 17, 0]
    assert runs[:4] == [[0, 1, 9, 15], [1, 2, 1, 0], [3, 16, 7, 0], [19, 2, 5, 0]]
    assert runs[4:] == [[0, 0, 0, 0]] * 3


def test_plain_grid_is_the_types():
    # every e4m3 value is its own nearest code, midpoints go to the even one
    b = torch.arange(256, dtype=torch.uint8).view(torch.float8_e4m3fn).double()
    b = b[b.isfinite()]
    assert torch.equal(plain.to_grid(b, torch.float8_e4m3fn), b)
    pos = b[b >= 0].unique()
    mid = (pos[1:] + pos[:-1]) / 2
    got = plain.to_grid(mid, torch.float8_e4m3fn)
    assert torch.equal(got, mid.float().to(torch.float8_e4m3fn).double())


def test_plain_attention_of_equal_scores_is_the_mean():
    H, D, page, L = 2, 64, 16, 21
    kc = torch.zeros(3, H, page, D, dtype=torch.int8)
    vc = torch.randint(-127, 128, kc.shape, dtype=torch.int8)
    ks, vs = torch.rand(3, H), torch.rand(3, H) + 0.5
    q = torch.randn(2, H, D).to(torch.bfloat16)
    out, lse, _, _ = plain.attend(q, [0, 2], [L], [[2, 0]], kc, vc, ks, vs, 0.3)
    v = (vc.double() * (vs.double() / 127)[:, :, None, None])
    rows = torch.cat([v[2], v[0]], 1)
    for i in range(2):
        assert torch.allclose(out[i], rows[:, :L - 1 + i].mean(1), atol=1e-12)
        assert torch.allclose(lse[i], torch.full((H,), math.log(L - 1 + i), dtype=torch.float64))
    # rows before the cache's start see nothing
    out, lse, _, _ = plain.attend(q, [0, 2], [1], [[2, 0]], kc, vc, ks, vs, 0.3)
    assert (out[0] == 0).all() and lse[0].max() == -math.inf and lse[1].isfinite().all()
