"""Layers with rotary positions and an 8-bit cache on the GPU, and one serving run of the operators
together: prompts appended, drafter and target layers, head, acceptance, log probabilities, commit.

Tolerances.  Projections and the residual stream: the bf16 bar of the layer tests, per-row max-abs
error / max-abs reference <= 2e-2; the 8-bit softmax weights add at most 2^-8 + 2^-10 < 1e-2 of an
attention output's largest value, so layers over the 8-bit cache have 3e-2.  What one call makes of
its own inputs (codes, scales, attention) is held to the bounds of that call's own tests.
"""
import math

import numpy as np
import pytest
import torch

import synthetic as S
import verify_step_b200 as sd
from oracle import attention as A
from oracle import drafter as DR
from oracle import kv8
from oracle import rotary as R
from tests.gpu_util import DEV, attn_desc, rel_err, status_ok, to_dev, workspace
from tests.test_gpu_logprobs import check as check_logprobs
from tests.test_gpu_rope_append import check_q8
from verify_step_b200 import drafter as VD
from verify_step_b200 import target as VT

pytestmark = pytest.mark.gpu

BF16_TOL, KV8_TOL = 2e-2, 3e-2
BASE = 1e6


def f64(t):
    return t.detach().cpu().double().numpy()


def make_rot(D, layout):
    freqs = torch.zeros(D // 2, dtype=torch.int64, device=DEV)
    amp = sd.sd_rope_freqs(sd.RopeFreqDesc(rot_dim=D, base=BASE), freqs)
    return sd.rotary(freqs, layout, amp)


def turned(x, pos, D, layout):
    f, amp = R.frequencies(D, BASE)
    return R.rotate(x, pos, f, amp, layout)


class Kv8:
    """One layer's 8-bit cache filled with prompts of L rows (appended by the call under test)."""
    def __init__(self, seed, L, room, n_q, hq, hkv, D, bs, window, layout):
        table, nb = S.block_table(seed, np.asarray(L, np.int32), room, bs, True)
        self.L, self.D, self.bs, self.hkv, self.layout = L, D, bs, hkv, layout
        self.table_h = table
        B, n = len(L), int(sum(L))
        kc = torch.zeros((nb, hkv, bs, D), dtype=torch.uint8, device=DEV)
        sc = torch.zeros((nb, hkv), device=DEV)
        self.rot = make_rot(D, layout)
        self.c = dict(desc=attn_desc(B, n_q, hq, hkv, D, bs, table.shape[1], nb, window), k=kc,
                      v=kc.clone(), k_scale=sc, v_scale=sc.clone(), table=to_dev(
                          torch.from_numpy(table)), rot=self.rot)
        self.xdesc = attn_desc(B, 1, hq, hkv, D, bs, table.shape[1], nb, window)
        g = torch.Generator().manual_seed(seed)
        k, v = (torch.randn((n, hkv, D), generator=g).bfloat16().to(DEV) for _ in range(2))
        cu = torch.tensor([0] + list(np.cumsum(L)), dtype=torch.int32, device=DEV)
        sd.sd_append_kv(sd.AppendDesc(
            batch=B, n_rows=n, h_kv=hkv, head_dim=D, block_size=bs,
            max_blocks_per_seq=table.shape[1], num_blocks=nb, ld_k=hkv * D, ld_v=hkv * D,
            dtype=sd.SD_BF16, cache_dtype=sd.SD_E4M3), self.rot, k, v, None, kc, self.c["v"],
            sc, self.c["v_scale"], self.c["table"],
            torch.zeros(B, dtype=torch.int32, device=DEV), cu)

    def host(self):
        return [self.c[n].cpu() for n in ("k", "v", "k_scale", "v_scale")]

    def decoded(self):
        k, v, ks, vs = [t.numpy() for t in self.host()]
        return (kv8.decode(k) * ks.astype(np.float64)[..., None, None],
                kv8.decode(v) * vs.astype(np.float64)[..., None, None])


@pytest.mark.parametrize("B,k,layout", [(3, 2, 0), (2, 6, 1), (1, 0, 0)])
def test_target_layers_over_the_8_bit_cache(B, k, layout):
    n_q, hq, hkv, bs, d, ff = k + 1, 8, 2, 16, 1024, 512
    layers = ((64, 40), (128, 0))
    L = [37, 150, 16][:B]
    host = S.make_target_weights(B + k, d, ff, hq, hkv, layers)
    x0 = torch.from_numpy(S.normal(17 + B, (B * n_q, d), 1.0))
    shape = VT.TargetShape(batch=B, n_q=n_q, d=d, ff=ff, h_q=hq, h_kv=hkv, layers=layers)
    kv = [Kv8(5 * i + B, L, n_q + 2, n_q, hq, hkv, D, bs, W, layout)
          for i, (D, W) in enumerate(layers)]
    before = [c.host() for c in kv]
    wts, buf = VT.device_weights(host), VT.buffers(shape)
    buf["x"].copy_(x0.to(DEV))
    ctx = torch.tensor(L, dtype=torch.int32, device=DEV)
    caches = [c.c for c in kv]
    ws = workspace(max(sd.sd_verify_attn_q8_workspace_size(c["desc"]) for c in caches))
    VT.verify_layers(shape, wts, buf, caches, ctx, ws)
    torch.cuda.synchronize()
    assert status_ok()

    x = f64(x0)
    pos = (np.asarray(L)[:, None] + np.arange(n_q)).reshape(-1)
    for i, ((D, W), c) in enumerate(zip(layers, kv)):
        lw = {n: f64(t) for n, t in host[i].items() if isinstance(t, torch.Tensor)}
        a = DR.rmsnorm(x, lw["g_attn"])
        q = turned(DR.linear(a, lw["Wq"]).reshape(-1, hq, D), pos, D, layout)
        assert rel_err(f64(buf["q"][i]).reshape(q.shape), q) <= BF16_TOL, i
        # the append of the kernel's own rows
        kn = f64(buf["k"][i]).reshape(-1, hkv, D)
        vn = f64(buf["v"][i]).reshape(-1, hkv, D)
        assert rel_err(kn, DR.linear(a, lw["Wk"]).reshape(kn.shape)) <= BF16_TOL, i
        codes = [t.numpy().copy() for t in before[i][:2]]
        scales = [t.double().numpy().copy() for t in before[i][2:]]
        after = c.host()
        for w, rows in enumerate((turned(kn, pos, D, layout), vn)):
            kv8.append(codes[w], scales[w], rows.reshape(B, n_q, hkv, D), c.table_h, L, [n_q] * B,
                       bs)
            check_q8(after[w], after[2 + w], codes[w], scales[w],
                     turned_bound=0 if w == 0 else None)
        # attention over the cache as it stands, with the oracle's queries
        K, V = c.decoded()
        o = np.zeros((B, n_q, hq, D))
        for b in range(B):
            for j in range(n_q):
                for h in range(hq):
                    lo, t = A.key_range(L[b] + j, W, L[b] + j)
                    p = np.arange(lo, t + 1)
                    blk, off = c.table_h[b, p // bs], p % bs
                    g = h // (hq // hkv)
                    o[b, j, h] = A.softmax_attend(q.reshape(B, n_q, hq, D)[b, j, h],
                                                  K[blk, g, off], V[blk, g, off],
                                                  1.0 / math.sqrt(D))
        o = o.reshape(B * n_q, hq * D)
        assert rel_err(f64(buf["o"][i]), o) <= KV8_TOL, i
        x = x + DR.linear(o, lw["Wo"])
        m = DR.rmsnorm(x, lw["g_mlp"])
        x = x + DR.linear(DR.geglu(m, lw["Wg"], lw["Wu"]), lw["Wd"])
    assert rel_err(f64(buf["x"]), x) <= KV8_TOL
    assert ctx.tolist() == L  # the verify does not commit


def test_bf16_layers_with_positions_hold_the_turned_keys():
    B, n_q, hq, hkv, bs, d, ff, D, layout = 2, 3, 4, 2, 16, 512, 256, 256, 0
    L, layers = [20, 5], ((D, 0),)
    host = S.make_target_weights(3, d, ff, hq, hkv, layers)
    table, nb = S.block_table(1, np.asarray(L, np.int32), n_q, bs, True)
    kc = torch.zeros((nb, hkv, bs, D), dtype=torch.bfloat16, device=DEV)
    c = dict(desc=attn_desc(B, n_q, hq, hkv, D, bs, table.shape[1], nb, 0), k=kc, v=kc.clone(),
             table=to_dev(torch.from_numpy(table)), rot=make_rot(D, layout))
    shape = VT.TargetShape(batch=B, n_q=n_q, d=d, ff=ff, h_q=hq, h_kv=hkv, layers=layers)
    wts, buf = VT.device_weights(host), VT.buffers(shape)
    x0 = torch.from_numpy(S.normal(2, (B * n_q, d), 1.0))
    buf["x"].copy_(x0.to(DEV))
    VT.verify_layers(shape, wts, buf, [c], torch.tensor(L, dtype=torch.int32, device=DEV),
                     workspace(sd.sd_verify_attn_workspace_size(c["desc"])))
    torch.cuda.synchronize()
    pos = (np.asarray(L)[:, None] + np.arange(n_q)).reshape(-1)
    a = DR.rmsnorm(f64(x0), f64(host[0]["g_attn"]))
    for name, W, h in (("q", "Wq", hq), ("k", "Wk", hkv)):
        want = turned(DR.linear(a, f64(host[0][W])).reshape(-1, h, D), pos, D, layout)
        assert rel_err(f64(buf[name][0]).reshape(want.shape), want) <= BF16_TOL
    rows = buf["k"][0].view(B, n_q, hkv, D)
    for b in range(B):
        for j in range(n_q):
            p = L[b] + j
            assert torch.equal(kc[table[b, p // bs], :, p % bs], rows[b, j])
    assert status_ok()


class Run:
    """A serving run: per step one drafter link for each draft, the target's layers over k + 1
    positions, the dense head, acceptance, log probabilities of what was emitted, the commit."""
    def __init__(self, seed):
        self.B, self.k, hq, hkv, bs, d, ff, V = 3, 2, 8, 2, 16, 512, 256, 1000
        self.V, n_q = V, self.k + 1
        self.layers = ((64, 40), (128, 0))
        L = [30, 47, 1]
        self.shape = VT.TargetShape(batch=self.B, n_q=n_q, d=d, ff=ff, h_q=hq, h_kv=hkv,
                                    layers=self.layers)
        self.wts = VT.device_weights(S.make_target_weights(seed, d, ff, hq, hkv, self.layers))
        self.buf = VT.buffers(self.shape)
        self.kv = [Kv8(seed + i, L, 4 * n_q, n_q, hq, hkv, D, bs, W, i) for i, (D, W) in
                   enumerate(self.layers)]
        self.ctx = torch.tensor(L, dtype=torch.int32, device=DEV)
        dd = 256
        self.dshape = VD.DrafterShape(batch=self.B, d=dd, d_target=d, ff=ff, h_q=hq,
                                      head_dims=tuple(D for D, _ in self.layers), vocab=V)
        w = lambda i, *s: S.bf16(S.normal(900 + i, s, 1 / math.sqrt(s[-1])))
        one = lambda n: torch.ones(n)
        host = dict(E=w(0, V, dd), W_in=w(1, dd, d + dd), g_final=one(dd), W_back=w(2, d, dd),
                    layers=[dict(g_attn=one(dd), Wq=w(10 + 9 * i, hq * D, dd),
                                 Wo=w(11 + 9 * i, dd, hq * D), g_mlp=one(dd),
                                 Wg=w(12 + 9 * i, ff, dd), Wu=w(13 + 9 * i, ff, dd),
                                 Wd=w(14 + 9 * i, dd, ff)) for i, (D, _) in enumerate(self.layers)])
        self.dwts, self.dbuf = VD.device_weights(host), VD.buffers(self.dshape)
        self.emb = to_dev(torch.from_numpy(S.normal(77, (V, d), 1.0)))
        self.head_d, self.head = to_dev(w(3, V, dd)), to_dev(w(4, V, d))
        i32 = lambda *s: torch.zeros(s, dtype=torch.int32, device=DEV)
        f32 = lambda *s: torch.zeros(s, dtype=torch.float32, device=DEV)
        self.drafts, self.n_acc, self.out = i32(self.B, self.k), i32(self.B), i32(self.B, n_q)
        self.last = torch.tensor([[3], [500], [999]], dtype=torch.int32, device=DEV)
        self.hid = torch.zeros((self.B, d), dtype=torch.bfloat16, device=DEV)
        self.zd, self.z = f32(self.k, self.B, V), f32(self.B * n_q, V)
        self.yd = f32(self.B, self.k, V)
        self.slots = i32(self.B, n_q)
        self.lp, self.H = f32(self.B * n_q), f32(self.B * n_q)
        self.ids, self.tops = i32(self.B * n_q, 5), f32(self.B * n_q, 5)
        self.ldesc = sd.LogprobsDesc(rows=self.B * n_q, vocab=V, ld_logits=V, temperature=1.0,
                                     top_n=5)
        self.adesc = sd.AcceptDesc(batch=self.B, k=self.k, vocab=V, temperature=0.0, seed=1, step=0,
                                   purpose=1)
        self.draw = sd.AcceptDesc(batch=self.B, k=0, vocab=V, temperature=0.0, seed=1, step=0,
                                  purpose=2, ld_out=self.k)
        sizes = [sd.sd_logprobs_workspace_size(self.ldesc), sd.sd_accept_workspace_size(self.adesc),
                 sd.sd_accept_workspace_size(self.draw)]
        for c in self.kv:
            sizes += [sd.sd_verify_attn_q8_workspace_size(c.c["desc"]),
                      sd.sd_draft_xattn_q8_workspace_size(c.xdesc)]
        self.ws = workspace(max(sizes))

    def step(self):
        B, k, n_q, V = self.B, self.k, self.k + 1, self.V
        hd = lambda m, d: sd.HeadDesc(m=m, d=d, vocab=V, dtype=sd.SD_BF16)
        h_prev, toks, ld = self.hid, self.last, 1
        for j in range(k):
            caches = []
            for c in self.kv:
                x = sd.AttnDesc.from_buffer_copy(c.xdesc)
                x.q_offset = j
                caches.append(dict(c.c, desc=x))
            VD.link(self.dshape, self.dwts, self.dbuf, h_prev, toks, ld,
                    VD.cross_attention(self.dshape, caches, self.ctx, self.ws))
            sd.sd_lm_head(hd(B, self.dshape.d), self.dbuf["h"], self.head_d, self.zd[j])
            sd.sd_accept(self.draw, self.zd[j], None, None, self.n_acc, self.drafts[:, j].data_ptr(),
                         None, self.ws)
            h_prev, toks, ld = self.dbuf["h_back"], self.drafts[:, j:].data_ptr(), k
        self.yd.copy_(self.zd.transpose(0, 1))
        rows = torch.cat([self.last, self.drafts], 1).reshape(-1).long()
        self.buf["x"].copy_(self.emb[rows])
        VT.verify_layers(self.shape, self.wts, self.buf, [c.c for c in self.kv], self.ctx, self.ws)
        hidden = self.buf["x"].bfloat16()
        sd.sd_lm_head(hd(B * n_q, self.shape.d), hidden, self.head, self.z)
        sd.sd_accept(self.adesc, self.z, self.yd, self.drafts, self.n_acc, self.out, None, self.ws)
        sd.sd_logprobs(self.ldesc, self.z, self.out, self.lp, self.H, self.ids, self.tops, self.ws)
        c = self.kv[0].c
        cd = sd.CommitDesc(batch=B, k=k, block_size=16, max_blocks_per_seq=c["table"].shape[1],
                           num_blocks=c["k"].shape[0])
        sd.sd_commit(cd, c["table"], self.ctx, self.n_acc, self.slots)
        self.last.copy_(self.out.gather(1, self.n_acc.long()[:, None]))

    def state(self):
        t = [self.ctx, self.drafts, self.n_acc, self.out, self.lp, self.H, self.ids, self.tops,
             self.z, self.last]
        for c in self.kv:
            t += [c.c["k"], c.c["v"], c.c["k_scale"], c.c["v_scale"]]
        return [x.clone() for x in t]


def test_a_serving_run_of_the_operators_together():
    run = Run(11)
    for _ in range(3):
        L = run.ctx.tolist()
        run.step()
        torch.cuda.synchronize()
        z, out, n = f64(run.z), run.out.cpu().numpy(), run.n_acc.cpu().numpy()
        # greedy: the emitted tokens are the target's own choices, the drafts they confirm first
        best = z.argmax(1).reshape(run.B, -1)
        for b in range(run.B):
            assert np.array_equal(out[b, :n[b] + 1], best[b, :n[b] + 1])
            assert np.array_equal(run.drafts.cpu().numpy()[b, :n[b]], out[b, :n[b]])
        assert run.ctx.tolist() == [l + int(m) + 1 for l, m in zip(L, n)]
        check_logprobs(run.z.cpu(), run.out.reshape(-1).cpu(),
                       [x.cpu().numpy() for x in (run.lp, run.H, run.ids, run.tops)], 1.0, 5)
    assert status_ok()


def test_a_captured_serving_step_is_the_eager_one():
    eager, run = Run(23), Run(23)
    for _ in range(3):
        eager.step()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        run.step()  # loads the kernels
    torch.cuda.current_stream().wait_stream(s)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        run.step()
    for _ in range(2):
        g.replay()
    torch.cuda.synchronize()
    for a, b in zip(eager.state(), run.state()):
        assert torch.equal(a, b) or torch.equal(a.nan_to_num(), b.nan_to_num())
    assert status_ok()
