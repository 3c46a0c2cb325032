"""sd_append_kv where test_gpu_rope_append does not go: every e4m3 code held to the border it lies at,
prompts that do not begin at the first row, rows that are views of a fused projection.

A code of a turned K row is the one nearest to the float64 value x / s, or the other one of a pair
whose border, the midpoint times s, lies within the float32 error of x (pair_bound there; the float32
product with 1 / s, a power of two, is exact).  Everything else is compared exactly: V, unturned
rows, rows that moved to a larger scale, and all that was not written.
"""
import numpy as np
import pytest
import torch

import verify_step_b200 as sd
from oracle import kv8, rotary as OR
from tests.gpu_util import DEV, status_ok
from tests.test_gpu_rope_append import Cache, check_turned, f64, make_rotary, pair_bound

pytestmark = pytest.mark.gpu


def check_codes(got, got_scales, codes, scales, exact, bound, where):
    """exact, bound [n, h, D]: float64 rows and their float32 error; where: their block and row."""
    assert np.array_equal(got_scales.double().numpy(), scales)
    a = got.numpy().transpose(0, 2, 1, 3)
    b = codes.transpose(0, 2, 1, 3)
    blk, off = where
    rest = np.ones(a.shape[:2], bool)
    rest[blk, off] = False
    assert np.array_equal(a[rest], b[rest])
    a, b, s = a[blk, off], b[blk, off], scales[blk][..., None]
    diff = a != b
    va, vb = kv8.decode(a), kv8.decode(b)
    assert np.all(np.abs(exact - (va + vb) / 2 * s)[diff] <= bound[diff])
    # neighbours only: no code lies between the two
    mags = np.abs(kv8.DECODE[:127])
    assert np.all(np.abs(np.searchsorted(mags, np.abs(va[diff])) -
                         np.searchsorted(mags, np.abs(vb[diff]))) <= 1)


def expect(c, ctx, counts, rows, old, olds):
    codes, scales = old.numpy().copy(), olds.double().numpy().copy()
    kv8.append(codes, scales, np.split(rows, np.cumsum(counts)[:-1]), c.table.numpy(), ctx, counts, c.bs)
    return codes, scales


def places(c, counts):
    pos = c.positions()
    seq = np.repeat(np.arange(len(counts)), counts)
    return pos, (c.table.numpy()[seq, pos // c.bs], pos % c.bs)


@pytest.mark.parametrize("kind,bs", [("e4m3", 16), ("e4m3", 32), ("bf16", 16)])
@pytest.mark.parametrize("front", [1, 15, 33, 65])
def test_prompts_behind_rows_of_no_sequence(kind, bs, front):
    """cu_new may begin anywhere: rows in front of the first sequence are not read, and their query
    rows not written; nothing is recorded."""
    ctx, counts, hkv, D, hq, back = [20, 0, 7], [30, 0, 50], 2, 128, 4, 2
    c = Cache(21, ctx, counts, hkv, D, bs, kind)
    m = sum(counts)
    n = front + m + back
    g = torch.Generator().manual_seed(22)
    k, v = (torch.randn((n, hkv, D), generator=g).bfloat16() for _ in range(2))
    q = torch.randn((n, hq, D), generator=g).bfloat16()
    k[:front] = v[:front] = k[front + m:] = v[front + m:] = float("nan")
    r, f, amp = make_rotary(D, 0)
    cu = torch.tensor([front, front + 30, front + 30, front + m], dtype=torch.int32, device=DEV)
    d = sd.AppendDesc(batch=3, n_rows=n, h_q=hq, h_kv=hkv, head_dim=D, block_size=bs,
                      max_blocks_per_seq=c.table.shape[1], num_blocks=c.nb, ld_k=hkv * D, ld_v=hkv * D,
                      ld_q=hq * D, ld_q_out=hq * D, dtype=sd.SD_BF16,
                      cache_dtype=sd.SD_E4M3 if kind == "e4m3" else sd.SD_BF16)
    on = lambda t: None if t is None else t.to(DEV)
    got = [on(t) for t in (c.k, c.v, c.ks, c.vs)]
    qo = torch.full((n, hq, D), 7.0, dtype=torch.bfloat16, device=DEV)
    sd.sd_append_kv(d, r, on(k), on(v), on(q), *got, on(c.table), on(c.ctx), cu, qo)
    torch.cuda.synchronize()
    assert status_ok()
    kc, vc, ks, vs = [None if t is None else t.cpu() for t in got]
    pos, where = places(c, counts)
    live = slice(front, front + m)
    kr, vr = f64(k[live]), f64(v[live])
    if kind == "e4m3":
        turned, e = OR.rotate(kr, pos, f, amp, 0), pair_bound(kr, pos, f, amp, 0)
        check_codes(kc, ks, *expect(c, ctx, counts, turned, c.k, c.ks), turned, e, where)
        check_codes(vc, vs, *expect(c, ctx, counts, vr, c.v, c.vs), vr, 0 * e, where)
    else:
        check_turned(f64(kc[where[0], :, where[1]]), kr, pos, f, amp, 0, 2.0 ** -8)
        assert torch.equal(vc[where[0], :, where[1]], v[live])
    check_turned(f64(qo[live]), f64(q[live]), pos, f, amp, 0, 2.0 ** -8)
    assert torch.all(qo[:front] == 7.0) and torch.all(qo[front + m:] == 7.0)
