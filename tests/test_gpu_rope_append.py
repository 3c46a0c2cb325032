"""GPU parity of sd_rope_freqs, sd_rope and sd_append_kv against the float64 oracle.

Tolerance of a turned element (a, b the pair, A the amplitude), in float32: cos and sin are off by at
most 2^-23 (one unit of the last place of 1 each from the function and from the reduced angle),
times A rounded once more (2^-24); the product that is rounded alone and the fused sum add 2^-24
each, all relative to at most A (|a| + |b|): below 3 * 2^-23 A (|a| + |b|).  The angle t f itself is
off by |t| f (2^-51 of the table's power in float64 + 2^-53 of the oracle's frequency + 2^-53 of its
product) < |t| f 2^-50 radians, which matters at positions of 2^27 and more only.  A bf16 result is
off by half a step, 2^-8 of it, on top.  What is not turned is a copy: bit-exact.

e4m3 codes and scales are compared with the oracle's on the GPU's own terms: V rows (never turned)
and unturned K rows exactly; turned K rows may differ by one code where the float64 value lies within
the float32 tolerance of the border between two codes.
"""
import numpy as np
import pytest
import torch

import verify_step_b200 as sd
from oracle import kv8, rotary as OR
from tests.gpu_util import DEV, status_ok

pytestmark = pytest.mark.gpu

TYPES = {"f32": (torch.float32, sd.SD_F32, 0.0), "bf16": (torch.bfloat16, sd.SD_BF16, 2.0 ** -8)}


def freq_desc(rot, scaling=0, base=10000.0):
    return sd.RopeFreqDesc(rot_dim=rot, base=base, scaling=scaling, factor=8.0, orig_ctx=2048,
                           beta_fast=32.0, beta_slow=1.0)


def make_rotary(rot, layout, scaling=0, base=10000.0):
    table = torch.empty(rot // 2, dtype=torch.int64, device=DEV)
    amp = sd.sd_rope_freqs(freq_desc(rot, scaling, base), table)
    f, want = OR.frequencies(rot, base, scaling, 8.0, 2048)
    assert amp == np.float32(want)
    return sd.rotary(table, layout, amp), f, float(np.float32(want))


def f64(t):
    return t.detach().cpu().double().numpy()


def pair_bound(x, pos, f, amp, layout):
    """(3 * 2^-23 + |t| f 2^-50) A (|a| + |b|) of every element, 0 behind the turning part."""
    n = len(f)
    ia = np.arange(n) if layout == OR.HALF else 2 * np.arange(n)
    ib = ia + (n if layout == OR.HALF else 1)
    e = np.zeros(x.shape)
    rel = 3 * 2.0 ** -23 + np.abs(np.asarray(pos, float))[:, None, None] * f * 2.0 ** -50
    e[..., ia] = e[..., ib] = rel * abs(amp) * (np.abs(x[..., ia]) + np.abs(x[..., ib]))
    return e


def check_turned(got, x, pos, f, amp, layout, half_step):
    want = OR.rotate(x, pos, f, amp, layout)
    e = pair_bound(x, pos, f, amp, layout)
    tol = e + half_step * (np.abs(want) + e)
    n = 2 * len(f)
    assert np.all(np.abs(got - want) <= tol + 1e-38)
    assert np.array_equal(got[..., n:], x[..., n:])


@pytest.mark.parametrize("scaling", [0, 1, 2])
def test_frequencies_are_fractions_of_a_turn(scaling):
    rot = 256
    table = torch.empty(rot // 2, dtype=torch.int64, device=DEV)
    sd.sd_rope_freqs(freq_desc(rot, scaling), table)
    got = table.cpu().numpy().view(np.uint64).astype(np.float64) / 2.0 ** 64 * 2 * np.pi
    f, _ = OR.frequencies(rot, 10000.0, scaling, 8.0, 2048)
    # a few units of the last place of pow and the ramp, and half a fixed-point step of 2^-64 turns:
    # pi 2^-64 < 2^-62 radians whatever the frequency
    assert np.all(np.abs(got - f) <= 2.0 ** -48 * f + 2.0 ** -62)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("layout", [0, 1])
@pytest.mark.parametrize("rows,heads,D,rot,scaling", [
    (1, 1, 64, 64, 0), (24, 16, 512, 512, 0), (3, 5, 256, 64, 2), (130, 3, 128, 32, 1),
    (7, 2, 80, 80, 0), (5, 3, 10, 6, 0), (9, 1, 2, 2, 0), (33, 33, 96, 40, 2), (2, 70, 64, 64, 0)])
def test_rope_matches_the_oracle(rows, heads, D, rot, scaling, layout, dtype):
    dt, code, half = TYPES[dtype]
    r, f, amp = make_rotary(rot, layout, scaling)
    g = torch.Generator().manual_seed(rows * 1000 + D)
    x = torch.randn((rows, heads, D), generator=g).to(dt)
    pos = torch.randint(0, 200000, (rows,), generator=g, dtype=torch.int32)
    pos[0] = 2 ** 31 - 1
    if rows > 2:
        pos[1], pos[2] = 0, -12345  # positions behind the start are turns the other way
    out = torch.full_like(x, float("nan"), device=DEV)
    d = sd.RopeDesc(rows=rows, heads=heads, head_dim=D, ld_x=heads * D, ld_out=heads * D, dtype=code)
    sd.sd_rope(d, r, x.to(DEV), pos.to(DEV), None, out)
    check_turned(f64(out), f64(x), pos.numpy(), f, amp, layout, half)
    assert status_ok()


@pytest.mark.parametrize("ld,shift", [(640, 0), (528, 0), (515, 1)])
def test_rope_of_strided_rows_and_in_place(ld, shift):
    """Rows inside a wider buffer (16-byte aligned or not); the rest of the buffer is left alone;
    positions from ctx_len and an offset."""
    rows, heads, D, rot = 10, 4, 128, 96
    r, f, amp = make_rotary(rot, 0)
    buf = torch.randn((rows, ld), device=DEV).bfloat16()
    before = buf.clone()
    x = buf[:, shift:shift + heads * D]
    ctx = torch.tensor([100, 7], dtype=torch.int32, device=DEV)
    d = sd.RopeDesc(rows=rows, heads=heads, head_dim=D, ld_x=ld, ld_out=ld, dtype=sd.SD_BF16,
                    rows_per_seq=5, q_offset=3)
    sd.sd_rope(d, r, x, None, ctx, x)
    pos = np.concatenate([100 + 3 + np.arange(5), 7 + 3 + np.arange(5)])
    x0 = f64(before[:, shift:shift + heads * D]).reshape(rows, heads, D)
    check_turned(f64(buf[:, shift:shift + heads * D]).reshape(rows, heads, D), x0, pos, f, amp, 0,
                 2.0 ** -8)
    assert torch.equal(buf[:, :shift], before[:, :shift])
    assert torch.equal(buf[:, shift + heads * D:], before[:, shift + heads * D:])


# ---------------------------------------------------------------------------------- append

class Cache:
    """Random paged cache, block table and lengths on the host."""

    def __init__(self, seed, ctx, counts, hkv, D, bs, kind):
        g = torch.Generator().manual_seed(seed)
        need = [-(-(c + n) // bs) for c, n in zip(ctx, counts)]
        self.nb = sum(need) + 2
        perm = torch.randperm(self.nb, generator=g).int()
        self.table = torch.zeros((len(ctx), max(1, max(need)) + 1), dtype=torch.int32)
        at = 0
        for b, n in enumerate(need):
            self.table[b, :n] = perm[at:at + n]
            at += n
        self.ctx = torch.tensor(ctx, dtype=torch.int32)
        self.counts, self.bs, self.hkv, self.D, self.kind = counts, bs, hkv, D, kind
        shape = (self.nb, hkv, bs, D)
        if kind == "e4m3":
            code = lambda: torch.randint(0, 256, shape, generator=g, dtype=torch.uint8)
            fix = lambda c: torch.where((c & 0x7F) == 0x7F, torch.zeros_like(c), c)
            self.k, self.v = fix(code()), fix(code())
            sc = lambda: torch.exp2(torch.randint(-12, -5, (self.nb, hkv), generator=g).float())
            self.ks, self.vs = sc(), sc()
        else:
            dt = TYPES[kind][0]
            self.k, self.v = torch.randn(shape, generator=g).to(dt), torch.randn(shape, generator=g).to(dt)
            self.ks = self.vs = None

    def positions(self):
        return np.concatenate([np.arange(c, c + n) for c, n in zip(self.ctx.tolist(), self.counts)]
                              + [np.zeros(0, int)]).astype(np.int64)


def append(c, k, v, q, rot, dtype, ragged, q_out=None, extra=0):
    """One sd_append_kv; returns the updated caches, scales and turned queries."""
    on = lambda t: None if t is None else t.to(DEV)
    rows = k.shape[0]
    hq = q.shape[1] if q is not None else 0
    D = c.D
    cu = None
    if ragged:
        cu = torch.tensor([0] + list(np.cumsum(c.counts)), dtype=torch.int32, device=DEV)
    code = TYPES[dtype][1]
    d = sd.AppendDesc(batch=len(c.counts), n_new=0 if ragged else c.counts[0], n_rows=rows, h_q=hq,
                      h_kv=c.hkv, head_dim=D, block_size=c.bs, max_blocks_per_seq=c.table.shape[1],
                      num_blocks=c.nb, ld_k=c.hkv * D, ld_v=c.hkv * D, ld_q=hq * D, ld_q_out=hq * D,
                      dtype=code, cache_dtype=sd.SD_E4M3 if c.kind == "e4m3" else code)
    got = [on(c.k), on(c.v), on(c.ks), on(c.vs)]
    qd = on(q)
    qo = qd if q_out == "in place" else (torch.full_like(qd, 7.0) if q is not None else None)
    sd.sd_append_kv(d, rot, on(k), on(v), qd, got[0], got[1], got[2], got[3], on(c.table),
                    on(c.ctx), cu, qo)
    torch.cuda.synchronize()
    return [None if t is None else t.cpu() for t in got + [qo]]


def check_q8(got_codes, got_scales, codes, scales, turned_bound=None):
    """Codes and scales against the oracle's; where turned_bound is given, a code may be the
    neighbour whose border the exact value is that close to."""
    assert np.array_equal(got_scales.double().numpy(), scales)
    a, b = got_codes.numpy(), codes
    if turned_bound is None:
        assert np.array_equal(a, b)
        return
    diff = a != b
    # far below one in a thousand elements lies within 2^-21 of a border
    assert diff.mean() <= 1e-3
    va, vb = kv8.decode(a[diff]), kv8.decode(b[diff])
    assert np.all(np.abs(va - vb) <= np.maximum(np.abs(vb) / 8, 2.0 ** -9) * 1.0001)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("ctx,counts,ragged,hq,hkv,D,bs,rot,layout", [
    ([45, 130], [3, 3], False, 8, 2, 256, 16, 256, 0),
    ([0, 7, 100], [40, 0, 25], True, 4, 1, 64, 16, 32, 1),
    ([5], [70], True, 0, 3, 48, 10, 48, 0),       # block size of the float types: any
    ([3, 3], [1, 1], False, 3, 1, 10, 7, 6, 1),   # odd widths: scalar path
    ([0] * 5, [0, 17, 0, 1, 0], True, 2, 2, 128, 32, 0, 0)])
def test_append_in_the_rows_type(ctx, counts, ragged, hq, hkv, D, bs, rot, layout, dtype):
    dt, _, half = TYPES[dtype]
    c = Cache(1, ctx, counts, hkv, D, bs, dtype)
    g = torch.Generator().manual_seed(2)
    extra = 3 if ragged else 0  # rows behind the last sequence
    n = sum(counts) + extra
    k, v = torch.randn((n, hkv, D), generator=g).to(dt), torch.randn((n, hkv, D), generator=g).to(dt)
    q = torch.randn((n, hq, D), generator=g).to(dt) if hq else None
    r, f, amp = make_rotary(rot, layout) if rot else (None, np.zeros(0), 1.0)
    kc, vc, _, _, qo = append(c, k, v, q, r, dtype, ragged)
    pos, m = c.positions(), sum(counts)
    seq = np.repeat(np.arange(len(counts)), counts)
    blk, off = c.table.numpy()[seq, pos // bs], pos % bs
    check_turned(f64(kc[blk, :, off]), f64(k[:m]), pos, f, amp, layout, half)
    assert torch.equal(vc[blk, :, off], v[:m])
    rest = torch.ones((c.nb, bs), dtype=torch.bool)
    rest[blk, off] = False
    for got, old in ((kc, c.k), (vc, c.v)):  # every other row as it was
        assert torch.equal(got.transpose(1, 2)[rest], old.transpose(1, 2)[rest])
    if hq:
        check_turned(f64(qo[:m]), f64(q[:m]), pos, f, amp, layout, half)
        assert torch.all(qo[m:] == 7.0)
    assert status_ok()


Q8 = [
    # verify step, k = 2: blocks go on, begin, and are crossed
    ([45, 130, 16, 31, 15], [3] * 5, False, 8, 2, 256, 16, 256, 0, "bf16"),
    ([14, 16384], [3, 3], False, 16, 4, 512, 16, 512, 0, "bf16"),
    ([0, 7, 100, 33], [40, 0, 25, 1], True, 4, 1, 64, 16, 32, 1, "bf16"),
    ([3, 0, 60], [200, 64, 5], True, 0, 4, 512, 64, 256, 0, "bf16"),   # rows read twice
    ([0, 100], [300, 100], True, 2, 3, 512, 128, 512, 1, "bf16"),      # rows read twice
    ([9, 48], [7, 7], False, 2, 8, 128, 48, 128, 0, "f32"),
    ([0] * 40, [33] * 40, True, 1, 5, 128, 32, 0, 0, "bf16"),          # several heads a CTA
    ([1] * 40, [20] * 40, True, 0, 4, 512, 16, 512, 0, "f32"),
    ([3] * 40, [100] * 40, True, 0, 10, 64, 32, 64, 1, "bf16"),        # 8 heads a CTA, 2 left
    ([7] * 20, [130] * 20, True, 0, 3, 512, 64, 512, 0, "bf16"),       # read twice, 2 heads, 1 left
    ([9] * 30, [70] * 30, True, 2, 4, 512, 32, 512, 0, "bf16"),        # two units a thread
]


@pytest.mark.parametrize("ctx,counts,ragged,hq,hkv,D,bs,rot,layout,dtype", Q8)
def test_append_to_e4m3(ctx, counts, ragged, hq, hkv, D, bs, rot, layout, dtype):
    dt, _, half = TYPES[dtype]
    c = Cache(3, ctx, counts, hkv, D, bs, "e4m3")
    g = torch.Generator().manual_seed(4)
    n = sum(counts)
    # rows of very different size, so that some blocks grow and some do not
    size = torch.exp2(torch.randint(-6, 6, (n, 1, 1), generator=g).float())
    k = (torch.randn((n, hkv, D), generator=g) * size).to(dt)
    v = (torch.randn((n, hkv, D), generator=g) * size).to(dt)
    q = torch.randn((n, hq, D), generator=g).to(dt) if hq else None
    r, f, amp = make_rotary(rot, layout) if rot else (None, np.zeros(0), 1.0)
    kc, vc, ks, vs, qo = append(c, k, v, q, r, dtype, ragged)
    pos = c.positions()
    turned = OR.rotate(f64(k), pos, f, amp, layout) if rot else f64(k)
    cuts = np.cumsum(counts)[:-1]
    for got, gs, old, olds, rows, t in ((kc, ks, c.k, c.ks, turned, rot or None),
                                        (vc, vs, c.v, c.vs, f64(v), None)):
        codes, scales = old.numpy().copy(), olds.double().numpy().copy()
        kv8.append(codes, scales, np.split(rows, cuts), c.table.numpy(), ctx, counts, bs)
        check_q8(got, gs, codes, scales, t)
    if hq:
        check_turned(f64(qo), f64(q), pos, f, amp, layout, half)
    assert status_ok()


def test_scale_borders_zeros_and_values_that_are_not_finite():
    """Exactly 448 2^e keeps e, the next bf16 above takes e + 1; zero rows take the smallest scale;
    NaN and infinities do not count, infinities become +-448 s."""
    D, bs = 64, 16
    tops = [448.0, 450.0, 1.75 * 2.0 ** -30, 3.0e38, 0.0, 2.0 ** -100]
    c = Cache(5, [0] * len(tops), [2] * len(tops), 1, D, bs, "e4m3")
    c.k, c.ks = c.v.clone(), c.vs.clone()  # K and V get the same rows below
    v = torch.zeros((2 * len(tops), 1, D))
    for i, t in enumerate(tops):
        v[2 * i, 0, 0], v[2 * i + 1, 0, 1] = t, -t / 2
    v[0, 0, 5], v[0, 0, 6], v[1, 0, 7] = float("nan"), float("inf"), float("-inf")
    v = v.bfloat16()
    kc, vc, ks, vs, _ = append(c, v, v, None, None, "bf16", False)
    codes, scales = c.v.numpy().copy(), c.vs.double().numpy().copy()
    kv8.append(codes, scales, np.split(f64(v), len(tops)), c.table.numpy(), [0] * len(tops),
               [2] * len(tops), bs)
    mask = (codes & 0x7F) == 0x7F
    assert np.array_equal((vc.numpy() & 0x7F) == 0x7F, mask)
    assert np.array_equal(vc.numpy()[~mask], codes[~mask]) and torch.equal(kc, vc)
    assert np.array_equal(vs.double().numpy(), scales) and torch.equal(ks, vs)
    blk = c.table.numpy()[:, 0]
    assert [int(np.log2(s)) for s in scales[blk, 0]] == [0, 1, -38, 120, -64, -64]
    assert status_ok()


def test_append_twice_is_the_same_and_a_new_first_row_begins_the_block():
    c = Cache(6, [20], [3], 2, 128, 16, "e4m3")
    g = torch.Generator().manual_seed(7)
    k, v = torch.randn((3, 2, 128), generator=g).bfloat16(), torch.randn((3, 2, 128), generator=g).bfloat16()
    one = append(c, k, v, None, None, "bf16", False)
    c.k, c.v, c.ks, c.vs = one[:4]
    two = append(c, k, v, None, None, "bf16", False)
    assert all(torch.equal(a, b) for a, b in zip(one[:4], two[:4]))
    # the block's first row is written again: its scale is that of the new rows alone
    c.ctx = torch.tensor([16], dtype=torch.int32)
    three = append(c, k * 2.0 ** -10, v * 2.0 ** -10, None, None, "bf16", False)
    blk = int(c.table[0, 1])
    assert torch.all(three[3][blk] < two[3][blk])
    assert status_ok()


@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
def test_bad_pages_are_skipped_and_recorded(kind):
    """A block id out of range, a position beyond the table and a negative length: recorded, and
    every other sequence is served.  (The kernels check before they touch memory.)"""
    ctx, counts = [20, 20, 20, 20], [3] * 4
    c = Cache(8, ctx, counts, 1, 64, 16, kind)
    good_blk = int(c.table[3, 1])
    c.table[0, 1] = c.nb
    c.table[1, 1] = -1
    c.ctx[2] = c.table.shape[1] * 16 - 1  # its second and third row are beyond the table
    g = torch.Generator().manual_seed(9)
    k = torch.randn((12, 1, 64), generator=g).bfloat16()
    got = append(c, k, k, None, None, "bf16", False)
    assert sd.sd_device_status_read() == sd.SD_ERR_DEVICE
    sd.sd_device_status_clear()
    rows = got[0][good_blk, 0, 4:7]
    if kind == "bf16":
        assert torch.equal(rows, k[9:, 0])
    else:
        want = kv8.decode(rows.numpy()) * float(got[2][good_blk, 0])
        assert np.allclose(want, f64(k[9:, 0]), rtol=2.0 ** -4, atol=2.0 ** -9)
    c.ctx[:] = -5
    got = append(c, k, k, None, None, "bf16", False)
    assert sd.sd_device_status_read() == sd.SD_ERR_DEVICE
    sd.sd_device_status_clear()
    assert torch.equal(got[0], c.k) and torch.equal(got[1], c.v)


def test_queries_in_place_and_replayed_from_a_graph_on_another_stream():
    ctx, counts = [45, 130], [3, 3]
    c = Cache(10, ctx, counts, 2, 256, 16, "e4m3")
    r, f, amp = make_rotary(256, 0)
    g = torch.Generator().manual_seed(11)
    k = torch.randn((6, 2, 256), generator=g).bfloat16()
    q = torch.randn((6, 8, 256), generator=g).bfloat16()
    plain = append(c, k, k, q, r, "bf16", False)
    inplace = append(c, k, k, q, r, "bf16", False, q_out="in place")
    assert all(torch.equal(a, b) for a, b in zip(plain, inplace))
    dev = [t.to(DEV) for t in (k, k, q, c.k, c.v, c.ks, c.vs, c.table, c.ctx)]
    qo = torch.empty_like(dev[2])
    d = sd.AppendDesc(batch=2, n_new=3, n_rows=6, h_q=8, h_kv=2, head_dim=256, block_size=16,
                      max_blocks_per_seq=c.table.shape[1], num_blocks=c.nb, ld_k=512, ld_v=512,
                      ld_q=2048, ld_q_out=2048, dtype=sd.SD_BF16, cache_dtype=sd.SD_E4M3)
    s = torch.cuda.Stream()
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph, stream=s):
        sd.sd_append_kv(d, r, dev[0], dev[1], dev[2], dev[3], dev[4], dev[5], dev[6], dev[7],
                        dev[8], None, qo)
    for _ in range(2):
        graph.replay()
    torch.cuda.synchronize()
    for a, b in zip(plain, [dev[3], dev[4], dev[5], dev[6], qo]):
        assert torch.equal(a, b.cpu())
    assert status_ok()
