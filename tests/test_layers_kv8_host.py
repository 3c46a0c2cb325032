"""Host logic of layers with positions and an 8-bit cache (no GPU): the calls that one layer's
attention issues, with the library calls replaced by recorders."""
import pytest

import verify_step_b200 as sd
from verify_step_b200 import drafter as VD
from verify_step_b200 import target as VT

NAMES = ("sd_rope", "sd_append_kv", "sd_verify_attn", "sd_verify_attn_q8", "sd_draft_xattn",
         "sd_draft_xattn_q8")


@pytest.fixture
def calls(monkeypatch):
    out = []
    for mod in (VT, VD):
        for n in NAMES:
            if hasattr(mod, n):
                monkeypatch.setattr(mod, n, lambda *a, n=n, **kw: out.append((n, a, kw)))
    return out


def cache(q8, rot, n_q):
    desc = sd.AttnDesc(batch=3, n_q=n_q, h_q=8, h_kv=2, head_dim=128, block_size=32,
                       max_blocks_per_seq=7, num_blocks=40, q_offset=2 if n_q == 1 else 0)
    c = dict(desc=desc, k="kc", v="vc", table="t")
    if rot:
        c["rot"] = "rot"
    if q8:
        c.update(k_scale="ks", v_scale="vs")
    return c


@pytest.mark.parametrize("rot", [False, True])
@pytest.mark.parametrize("q8", [False, True])
def test_target_attention(calls, q8, rot):
    shape = VT.TargetShape(batch=3, n_q=4, d=512, ff=64, h_q=8, h_kv=2, layers=((128, 0),))
    c = cache(q8, rot, 4)
    VT.attend(shape, 128, c, "q", "kn", "vn", "ctx", "o", "ws", stream=5)
    assert all(kw["stream"] == 5 for _, _, kw in calls)
    if not q8:
        assert [n for n, _, _ in calls] == ["sd_rope", "sd_rope"] * rot + ["sd_verify_attn"]
        assert calls[-1][1] == (c["desc"], "q", "kn", "vn", "kc", "vc", "t", "ctx", "o", "ws")
        for (_, a, _), x, h in zip(calls, ("q", "kn"), (8, 2)) if rot else ():
            d = a[0]
            assert (d.rows, d.heads, d.head_dim, d.ld_x, d.ld_out, d.dtype, d.rows_per_seq,
                    d.q_offset) == (12, h, 128, h * 128, h * 128, sd.SD_BF16, 4, 0)
            assert a[1:] == ("rot", x, None, "ctx", x)
        return
    (n0, a0, k0), (n1, a1, _) = calls
    assert (n0, n1) == ("sd_append_kv", "sd_verify_attn_q8")
    d = a0[0]
    assert (d.batch, d.n_new, d.n_rows, d.h_q, d.h_kv, d.head_dim) == (3, 4, 12, 8 * rot, 2, 128)
    assert (d.block_size, d.max_blocks_per_seq, d.num_blocks) == (32, 7, 40)
    assert (d.ld_k, d.ld_v, d.ld_q, d.ld_q_out) == (256, 256, 1024, 1024)
    assert (d.dtype, d.cache_dtype) == (sd.SD_BF16, sd.SD_E4M3)
    q = "q" if rot else None
    assert a0[1:] == ("rot" if rot else None, "kn", "vn", q, "kc", "vc", "ks", "vs", "t", "ctx")
    assert k0["q_out"] == q
    assert a1 == (c["desc"], "q", "kc", "vc", "ks", "vs", "t", "ctx", "o", "ws")


@pytest.mark.parametrize("q_pos", [None, "pos"])
@pytest.mark.parametrize("rot", [False, True])
@pytest.mark.parametrize("q8", [False, True])
def test_drafter_attention(calls, q8, rot, q_pos):
    shape = VD.DrafterShape(batch=3, d=64, d_target=128, ff=64, h_q=8, head_dims=(64, 128),
                            vocab=100)
    c = cache(q8, rot, 1)
    VD.cross_attention(shape, [None, c], "ctx", "ws", q_pos=q_pos, stream=5)(1, "q", "o")
    assert [n for n, _, _ in calls] == ["sd_rope"] * rot + [
        "sd_draft_xattn_q8" if q8 else "sd_draft_xattn"]
    if rot:
        d, *rest = calls[0][1]
        assert (d.rows, d.heads, d.head_dim, d.ld_x, d.rows_per_seq, d.q_offset) == (
            3, 8, 128, 1024, 1, 2)
        assert rest == ["rot", "q", q_pos, "ctx" if q_pos is None else None, "q"]
    scales = ("ks", "vs") if q8 else ()
    assert calls[-1][1] == (c["desc"], "q", "kc", "vc", *scales, "t", "ctx", q_pos, "o", "ws")
