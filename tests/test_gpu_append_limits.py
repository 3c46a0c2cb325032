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
from tests.test_gpu_rope_append import (Q8, TYPES, Cache, append, check_turned, f64, make_rotary,
                                        pair_bound)

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


@pytest.mark.parametrize("ctx,counts,ragged,hq,hkv,D,bs,rot,layout,dtype", Q8 + [
    ([10 ** 6 + 3, 77777], [20, 33], True, 0, 2, 128, 16, 128, 0, "bf16")])
def test_every_code_is_the_nearest_or_at_its_border(ctx, counts, ragged, hq, hkv, D, bs, rot, layout,
                                                    dtype):
    dt = TYPES[dtype][0]
    if max(ctx) > 10 ** 5:  # a far position without the memory before it: the table's blocks are shared
        c = Cache(3, [c % (4 * bs) for c in ctx], counts, hkv, D, bs, "e4m3")
        near, table = c.table, torch.zeros((len(ctx), max(ctx) // bs + 8), dtype=torch.int32)
        for b, x in enumerate(ctx):
            first = x // bs - x % (4 * bs) // bs
            table[b, first:first + near.shape[1]] = near[b]
        c.table, c.ctx = table, torch.tensor(ctx, dtype=torch.int32)
    else:
        c = Cache(3, ctx, counts, hkv, D, bs, "e4m3")
    g = torch.Generator().manual_seed(4)
    n = sum(counts)
    size = torch.exp2(torch.randint(-6, 6, (n, 1, 1), generator=g).float())
    k = (torch.randn((n, hkv, D), generator=g) * size).to(dt)
    v = (torch.randn((n, hkv, D), generator=g) * size).to(dt)
    q = torch.randn((n, hq, D), generator=g).to(dt) if hq else None
    r, f, amp = make_rotary(rot, layout) if rot else (None, np.zeros(0), 1.0)
    kc, vc, ks, vs, _ = append(c, k, v, q, r, dtype, ragged)
    pos, where = places(c, counts)
    turned = OR.rotate(f64(k), pos, f, amp, layout) if rot else f64(k)
    bound = pair_bound(f64(k), pos, f, amp, layout)
    for got, gs, old, olds, rows, e in ((kc, ks, c.k, c.ks, turned, bound),
                                        (vc, vs, c.v, c.vs, f64(v), 0 * bound)):
        codes, scales = expect(c, ctx, counts, rows, old, olds)
        check_codes(got, gs, codes, scales, rows, e, where)
    assert status_ok()


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


@pytest.mark.parametrize("kind", ["e4m3", "rows"])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("pad", [0, 16])
def test_rows_that_are_views_of_one_fused_projection(kind, dtype, pad):
    """q, k and v are column ranges of one buffer (row strides above their widths); the queries are
    turned in place there, and the buffer's other elements stay."""
    dt, code, half = TYPES[dtype]
    ctx, counts, hq, hkv, D, bs = [45, 130, 16], [5] * 3, 4, 2, 64, 16
    c = Cache(23, ctx, counts, hkv, D, bs, "e4m3" if kind == "e4m3" else dtype)
    n, w = 15, (hq + 2 * hkv) * D + pad
    g = torch.Generator().manual_seed(24)
    host = torch.randn((n, w), generator=g).to(dt)
    buf = host.to(DEV)
    cut = [0, hq * D, (hq + hkv) * D, (hq + 2 * hkv) * D]
    part = lambda x, i: x[:, cut[i]:cut[i + 1]]
    r, f, amp = make_rotary(32, 1)
    d = sd.AppendDesc(batch=3, n_new=5, n_rows=n, h_q=hq, h_kv=hkv, head_dim=D, block_size=bs,
                      max_blocks_per_seq=c.table.shape[1], num_blocks=c.nb, ld_k=w, ld_v=w, ld_q=w,
                      ld_q_out=w, dtype=code, cache_dtype=sd.SD_E4M3 if kind == "e4m3" else code)
    on = lambda t: None if t is None else t.to(DEV)
    got = [on(t) for t in (c.k, c.v, c.ks, c.vs)]
    sd.sd_append_kv(d, r, part(buf, 1), part(buf, 2), part(buf, 0), *got, on(c.table), on(c.ctx), None,
                    part(buf, 0))
    torch.cuda.synchronize()
    assert status_ok()
    kc, vc, ks, vs = [None if t is None else t.cpu() for t in got]
    pos, where = places(c, counts)
    q, k, v = (f64(part(host, i)).reshape(n, -1, D) for i in range(3))
    if kind == "e4m3":
        turned, e = OR.rotate(k, pos, f, amp, 1), pair_bound(k, pos, f, amp, 1)
        check_codes(kc, ks, *expect(c, ctx, counts, turned, c.k, c.ks), turned, e, where)
        check_codes(vc, vs, *expect(c, ctx, counts, v, c.v, c.vs), v, 0 * e, where)
    else:
        check_turned(f64(kc[where[0], :, where[1]]), k, pos, f, amp, 1, half)
        assert np.array_equal(f64(vc[where[0], :, where[1]]), v)
    check_turned(f64(part(buf, 0)).reshape(n, hq, D), q, pos, f, amp, 1, half)
    assert torch.equal(buf[:, cut[1]:].cpu(), host[:, cut[1]:])
