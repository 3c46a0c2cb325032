"""GPU parity of sd_verify_attn_q8 / sd_draft_xattn_q8 against the float64 oracle on the decoded cache.

Tolerance of an output element, p its softmax weights: a weight enters the product as two e4m3
parts, off by at most half a step of each, 2^-4 * 2^-4 = 2^-8 of it; below 2^-14 of 2^8 (the tile's
largest is scaled to 2^8) the second part's fixed step leaves 2^-22 of the largest weight, at most
2^-22 sum |v|.  Scores: products are exact, the float32 sum over D adds 2^-24 D of sum |q k| scale,
which for these inputs (|score| < 64) stays below 2^-10 relative in a weight.  So
    |err| <= (2^-8 + 2^-10) sum p |v| + 2^-22 n max p max |v| + 2^-8 |out|   (the bf16 result).
"""
import math

import numpy as np
import pytest
import torch

import verify_step_b200 as sd
from oracle import kv8
from tests.gpu_util import DEV, attn_desc, status_ok, workspace

pytestmark = pytest.mark.gpu


class Case:
    def __init__(self, seed, L, n_q, hq, hkv, D, bs, window=0, draft=False, scales="pow2", q_pos=None,
                 q_gain=1.0):
        g = torch.Generator().manual_seed(seed)
        self.L, self.n_q, self.window, self.draft, self.bs = list(L), n_q, window, draft, bs
        self.q_pos = q_pos
        need = [max(1, -(-(n + n_q) // bs)) for n in L]
        nb = sum(need) + 2
        perm = torch.randperm(nb, generator=g).int()
        self.table = torch.zeros((len(L), max(need)), dtype=torch.int32)
        at = 0
        for b, n in enumerate(need):
            self.table[b, :n] = perm[at:at + n]
            at += n
        x = lambda: (torch.randn((nb, hkv, bs, D), generator=g) * 100).clamp(-448, 448)
        self.kc = x().to(torch.float8_e4m3fn).view(torch.uint8)
        self.vc = x().to(torch.float8_e4m3fn).view(torch.uint8)
        if scales == "pow2":
            sc = lambda: torch.exp2(torch.randint(-9, -5, (nb, hkv), generator=g).float())
        else:  # any positive scales, some blocks far below the others
            sc = lambda: torch.rand((nb, hkv), generator=g) * 0.01 * torch.exp2(
                -20.0 * (torch.rand((nb, hkv), generator=g) < 0.2))
        self.ks, self.vs = sc(), sc()
        self.q = (torch.randn((len(L), n_q, hq, D), generator=g) * q_gain).bfloat16()
        self.desc = attn_desc(len(L), n_q, hq, hkv, D, bs, self.table.shape[1], nb, window)

    def on_gpu(self):
        qp = None if self.q_pos is None else torch.tensor(self.q_pos, dtype=torch.int32)
        self.dev = [t.to(DEV) if t is not None else None for t in
                    (self.q, self.kc, self.vc, self.ks, self.vs, self.table,
                     torch.tensor(self.L, dtype=torch.int32), qp)]
        size = sd.sd_draft_xattn_q8_workspace_size if self.draft else sd.sd_verify_attn_q8_workspace_size
        self.ws = workspace(size(self.desc))
        self.out = torch.full(self.q.shape, 9.0, dtype=torch.bfloat16, device=DEV)

    def launch(self):
        q, kc, vc, ks, vs, table, ctx, qp = self.dev
        if self.draft:
            sd.sd_draft_xattn_q8(self.desc, q, kc, vc, ks, vs, table, ctx, qp, self.out, self.ws)
        else:
            sd.sd_verify_attn_q8(self.desc, q, kc, vc, ks, vs, table, ctx, self.out, self.ws)

    def run(self):
        self.on_gpu()
        self.launch()
        torch.cuda.synchronize()
        return self.out.double().cpu().numpy()

    def reference(self):
        """(out, bound) of every element."""
        q = self.q.double().numpy()
        B, n_q, hq, D = q.shape
        hkv = self.kc.shape[1]
        K = kv8.decode(self.kc.numpy()) * self.ks.double().numpy()[..., None, None]
        V = kv8.decode(self.vc.numpy()) * self.vs.double().numpy()[..., None, None]
        out, tol = np.zeros_like(q), np.zeros_like(q)
        for b, L in enumerate(self.L):
            for j in range(n_q):
                t = (self.q_pos[b] if self.q_pos is not None else L + self.desc.q_offset) if self.draft else L + j
                lo = max(0, t - self.window + 1) if self.window else 0
                pos = np.arange(lo, min(t, L - 1 if self.draft else t) + 1)
                if not len(pos):
                    continue
                blk, off = self.table.numpy()[b, pos // self.bs], pos % self.bs
                for h in range(hq):
                    g = h // (hq // hkv)
                    k, v = K[blk, g, off], V[blk, g, off]
                    s = self.desc.scale * (k @ q[b, j, h])
                    w = np.exp(s - s.max())
                    w /= w.sum()
                    out[b, j, h] = w @ v
                    tol[b, j, h] = ((2.0 ** -8 + 2.0 ** -10) * (w @ np.abs(v)) +
                                    2.0 ** -22 * len(pos) * w.max() * np.abs(v).max())
        return out, tol + 2.0 ** -8 * np.abs(out) + 2.0 ** -8 * tol + 1e-30

    def check(self):
        got = self.run()
        want, tol = self.reference()
        assert np.all(np.isfinite(got))
        assert np.all(np.abs(got - want) <= tol), float((np.abs(got - want) / tol).max())
        assert status_ok()


@pytest.mark.parametrize("L,n_q,hq,hkv,D,bs,window", [
    ([0], 1, 1, 1, 64, 16, 0),                      # the first token of all
    ([0, 1, 2], 3, 8, 2, 128, 16, 0),
    ([40], 1, 4, 1, 512, 16, 0),
    ([127, 128, 129], 1, 4, 2, 256, 16, 0),         # around one tile
    ([125, 126, 253], 3, 4, 1, 64, 32, 0),          # new rows across a tile's end
    ([300, 17, 1500], 3, 16, 4, 512, 16, 0),
    ([700, 31], 7, 16, 4, 512, 48, 0),              # 28 rows: two row groups
    ([700, 31], 7, 9, 1, 256, 64, 0),               # 63 rows: two row groups, one row of padding
    ([200], 4, 16, 1, 512, 16, 0),                  # 64 rows: three groups of 22, 22 and 20
    ([90, 600], 1, 32, 1, 64, 128, 0),              # 32 rows, one TMA box a tile
    ([90, 600], 2, 12, 1, 128, 256, 0),             # 24 rows, blocks larger than a tile
    ([4096], 3, 8, 2, 256, 16, 512),                # sliding
    ([1000, 5, 511, 512], 3, 4, 2, 128, 16, 512),
    ([500, 40], 5, 4, 1, 512, 48, 33),              # window of about two blocks
    ([300], 3, 2, 1, 64, 16, 1),                    # each query reads its own key only
    ([50] * 70, 2, 4, 2, 64, 16, 0),                # several items a CTA
    ([3] * 200, 1, 2, 2, 512, 16, 0),
    ([9000, 100], 2, 4, 1, 128, 16, 0)])            # an item over many CTAs
def test_verify_matches_the_oracle(L, n_q, hq, hkv, D, bs, window):
    Case(len(L) * 100 + D, L, n_q, hq, hkv, D, bs, window).check()


@pytest.mark.parametrize("L,q_pos,hq,hkv,D,window", [
    ([100, 0, 33], None, 4, 2, 256, 0),             # an empty cache gives zeros
    ([100, 50, 33], [3, 60, 500], 4, 1, 512, 0),    # inside, at and behind the committed keys
    ([600, 600], [605, 1200], 8, 2, 128, 64),       # the second window holds no committed key
    ([2000], None, 16, 4, 512, 512)])
def test_drafter_matches_the_oracle(L, q_pos, hq, hkv, D, window):
    c = Case(7 + D, L, 1, hq, hkv, D, 16, window, draft=True, q_pos=q_pos)
    if q_pos is None:
        c.desc.q_offset = 2
    c.check()


def test_any_scales_and_large_scores():
    Case(11, [700, 90], 3, 8, 2, 256, 16, scales="any").check()
    Case(12, [700, 90], 2, 4, 2, 512, 16, q_gain=8.0).check()


def test_zero_scales_and_zero_queries():
    c = Case(13, [100, 260], 2, 4, 1, 128, 16)
    c.ks[:] = 0.0
    c.vs[c.table[0, 1]] = 0.0
    c.q[1] = 0
    c.check()


def test_query_elements_of_unlike_size():
    """Elements down to 2^-30 of their row's largest: what the split rounds, 2^-21 of the largest an
    element, moves a score by at most scale 2^-21 max |q| sum |k| < 2^-16, which the 2^-10 of the bound
    for scores covers."""
    c = Case(31, [300, 17], 3, 8, 2, 128, 16)
    g = torch.Generator().manual_seed(32)
    c.q = (c.q.float() * torch.exp2(-30 * torch.rand(c.q.shape, generator=g))).bfloat16()
    c.q[0, 0, 0] = 0
    c.check()
    c.q[0, 1, 1, 5] = math.inf
    got = c.run()
    assert np.isnan(got[0, 1, 1]).all() and np.isfinite(np.delete(got[0, 1], 1, axis=0)).all()


def test_a_heavy_first_key_leaves_the_others_their_weight():
    """One key holds half of the weight, 12000 others share the rest: 4e-5 each, below the last
    step of an 8-bit weight relative to the heavy one, and all of them point one way."""
    D, L = 128, 12000
    c = Case(14, [L], 1, 1, 1, D, 16)
    one = torch.tensor([1.0]).to(torch.float8_e4m3fn).view(torch.uint8)[0]
    c.kc[:] = 0
    c.kc[c.table[0, 0], 0, 0, 0] = one
    c.vc[:] = one
    c.vc[c.table[0, 0], 0, 0] = one | 0x80
    c.ks[:] = 1.0
    c.vs[:] = 1.0
    c.q[:] = 0
    c.q[0, 0, 0, 0] = math.log(L) / c.desc.scale
    got, (want, tol) = c.run(), c.reference()
    assert np.all(np.abs(got - want) <= 2.0 ** -7)  # weights of both signs cancel: 2^-8 of either half


def test_codes_outside_every_range_do_not_matter():
    """NaN codes in unwritten rows, in other blocks, behind the last key and before the window; the
    table's tail names blocks that do not exist."""
    for window in (0, 100):
        c = Case(15, [300, 77], 3, 4, 2, 256, 16, window)
        want, tol = c.reference()
        live = torch.zeros(c.kc.shape[0], 16, dtype=torch.bool)
        for b, L in enumerate(c.L):
            for p in range(max(0, L - window + 1) if window else 0, L + 3):
                live[c.table[b, p // 16], p % 16] = True
        for t in (c.kc, c.vc):
            t.transpose(1, 2)[~live] = 0x7F
        c.table = torch.cat([c.table, torch.full((2, 4), 1 << 20, dtype=torch.int32)], dim=1)
        c.desc.max_blocks_per_seq = c.table.shape[1]
        got = c.run()
        assert np.all(np.abs(got - want) <= tol)
        assert status_ok()


def test_nan_reaches_only_the_queries_that_attend_to_it():
    c = Case(16, [200], 3, 4, 2, 128, 16)
    want, tol = c.reference()
    blk, off = int(c.table[0, 201 // 16]), 201 % 16
    c.vc[blk, 0, off, 5] = 0xFF    # V of the second new position, kv head 0
    c.kc[blk, 1, off, 7] = 0x7F    # its K, kv head 1
    got = c.run()
    assert np.all(np.abs(got[0, 0] - want[0, 0]) <= tol[0, 0])
    assert np.all(np.isnan(got[0, 1:]))
    c = Case(17, [200], 3, 4, 2, 128, 16)
    want, tol = c.reference()
    c.q[0, 1, 2, 3] = float("nan")
    c.q[0, 2, 1, 3] = float("inf")
    got = c.run()
    bad = np.isnan(got).all(-1)
    assert np.array_equal(np.argwhere(bad[0]), [[1, 2], [2, 1]])
    assert np.all(np.abs(got - want)[~bad] <= tol[~bad])
    assert status_ok()


def test_bad_pages_and_lengths_are_recorded():
    """A block id out of range: its keys are left out; a position beyond the table and a negative
    length: a zero output.  All are checked before any access."""
    c = Case(18, [100, 100, 100, 60], 2, 4, 2, 64, 16)
    want, tol = c.reference()
    c.table[0, 2] = c.desc.num_blocks
    c.table[1, 0] = -3
    c.L[2] = c.table.shape[1] * 16
    got = c.run()
    assert sd.sd_device_status_read() == sd.SD_ERR_DEVICE
    sd.sd_device_status_clear()
    assert np.all(np.isfinite(got)) and np.all(got[2] == 0)
    assert np.all(np.abs(got - want)[3] <= tol[3])
    c.L = [-1] * 4
    got = c.run()
    assert sd.sd_device_status_read() == sd.SD_ERR_DEVICE
    sd.sd_device_status_clear()
    assert np.all(got == 0)


def test_runs_are_repeatable_in_graphs_and_on_two_streams():
    """The same call twice gives the same bits; two calls with a workspace each run at once on two
    streams; a captured call replays on new lengths."""
    a = Case(19, [3000, 500, 1], 3, 8, 2, 256, 16)
    b = Case(20, [40] * 30, 2, 4, 2, 512, 16, window=32)
    first = [a.run(), b.run()]
    a.out.zero_(), b.out.zero_()
    s = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    for _ in range(3):
        for c, st in zip((a, b), s):
            with torch.cuda.stream(st):
                c.launch()
    torch.cuda.synchronize()
    assert np.array_equal(a.out.double().cpu().numpy(), first[0])
    assert np.array_equal(b.out.double().cpu().numpy(), first[1])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        a.launch()
    a.L = [2500, 0, 130]
    a.dev[6].copy_(torch.tensor(a.L, dtype=torch.int32))
    a.ws.fill_(255)
    graph.replay()
    torch.cuda.synchronize()
    want, tol = a.reference()
    assert np.all(np.abs(a.out.double().cpu().numpy() - want) <= tol)
    assert status_ok()
