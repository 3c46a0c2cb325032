"""Cases of the rotary, cache-append, 8-bit cache attention and log-probability operators.

Each case names its operator in "op":

  rope      sd_rope: rotary positions of query (or key) rows
  append    sd_append_kv: new K / V rows into the paged cache, K and Q rotated on the way; the cache in
            the rows' own type or in e4m3 with a power-of-two scale per (block, kv head)
  attn      sd_verify_attn_q8 / sd_draft_xattn_q8: attention over the e4m3 cache
  logprobs  sd_logprobs: log p(token), entropy and the top alternatives of logit rows

``run`` computes them in elementary torch operations, or with ``own`` through verify_step_b200.
"""
import math
import random

import numpy as np
import torch

own = False

E4M3_MAX = 448.0
E_MIN = -64  # smallest exponent of a block's scale


# ------------------------------------------------------------------------------------- cases

def listed():
    f = dict
    return [
        # the k + 1 = 3 queries of 8 sequences of a global layer: a latency-bound call
        f(name="rope verify", op="rope", rows=24, heads=16, D=512, rot=512, layout=0, dtype="bf16",
          scaling=0, per_seq=3, ctx=16384),
        # the queries of a whole 16384-token prompt, a quarter of each head turned, context
        # stretched by 4 (by parts): bandwidth
        f(name="rope prompt", op="rope", rows=16384, heads=16, D=256, rot=64, layout=1,
          dtype="bf16", scaling=2, per_seq=1, ctx=0),
        # append of one verify step (8 x 3 rows, global layer), queries turned in the same call
        f(name="append verify e4m3", op="append", B=8, n=3, lo=0, ctx=16384, ragged=0, hq=16, hkv=4,
          D=512, bs=16, rot=512, layout=0, dtype="bf16", cache="e4m3", lens=1),
        # prompts of 64 to 4096 tokens packed into one call, some going on from a cached prefix
        f(name="append prompts e4m3", op="append", B=16, n=4096, lo=64, ctx=1000, ragged=1, hq=0,
          hkv=4, D=512, bs=16, rot=512, layout=0, dtype="bf16", cache="e4m3", lens=2),
        # the same of a sliding layer kept in bf16, with its queries
        f(name="append prompts bf16", op="append", B=16, n=2048, lo=16, ctx=777, ragged=1, hq=16,
          hkv=4, D=256, bs=16, rot=256, layout=0, dtype="bf16", cache="bf16", lens=3),
        # one sequence on a sliding layer of an edge model: the smallest attention call
        f(name="attn edge sliding", op="attn", B=1, nq=3, hq=8, hkv=2, D=256, bs=16, window=512,
          lo=4096, ctx=4096, draft=0, lens=4),
        # the drafter's query over the target's global cache
        f(name="attn drafter", op="attn", B=8, nq=1, hq=16, hkv=4, D=512, bs=16, window=0,
          lo=16384, ctx=16384, draft=1, lens=5),
        # the verify step's global layer, k = 2
        f(name="attn verify global", op="attn", B=8, nq=3, hq=16, hkv=4, D=512, bs=16, window=0,
          lo=16384, ctx=16384, draft=0, lens=6),
        # 64 ragged sequences of 1024 to 16384 tokens on a head_dim 256 global layer
        f(name="attn serving", op="attn", B=64, nq=3, hq=16, hkv=4, D=256, bs=16, window=0,
          lo=1024, ctx=16384, draft=0, lens=7),
        # one token's log probability over a small vocabulary: launch latency
        f(name="logprobs small", op="logprobs", rows=3, V=1024, top=0, T=1.0),
        # the 24 rows of a verify step at the full vocabulary, 5 alternatives
        f(name="logprobs verify", op="logprobs", rows=24, V=262144, top=5, T=1.0),
        # 64 sequences, 20 alternatives
        f(name="logprobs serving", op="logprobs", rows=192, V=262144, top=20, T=0.7),
    ]


def _log(rng, a, b):
    return int(round(math.exp(rng.uniform(math.log(a), math.log(b)))))


def draw(rng):
    op = rng.choice(["rope", "append", "attn", "logprobs"])
    if op == "rope":
        D = rng.choice([64, 80, 128, 256, 512])
        heads = _log(rng, 1, 32)
        dtype = rng.choice(["bf16", "bf16", "f32"])
        rows = _log(rng, 1, max(1, (16384 * 16 * 256 // (heads * D)) // (2 if dtype == "f32" else 1)))
        return dict(op=op, rows=rows, heads=heads, D=D, rot=rng.choice([D, D // 2, D // 4]),
                    layout=rng.randrange(2), dtype=dtype, scaling=rng.randrange(3),
                    per_seq=rng.randint(1, 7), ctx=_log(rng, 1, 100000))
    if op == "append":
        D = rng.choice([64, 128, 256, 512])
        ragged = rng.randrange(2)
        B = _log(rng, 1, 64) if not ragged else _log(rng, 1, 16)
        hkv = rng.choice([1, 2, 4, 8])
        n = rng.randint(1, 7) if not ragged else _log(rng, 8, max(8, 2048 * 16 * 2048 // (B * hkv * D)))
        dtype = rng.choice(["bf16", "bf16", "f32"])
        n = min(n, 8192) if dtype == "bf16" else (min(n, 8192) + 1) // 2
        cache = rng.choice(["e4m3", dtype])
        return dict(op=op, B=B, n=n, lo=1, ctx=_log(rng, 1, 4096), ragged=ragged,
                    hq=rng.choice([0, hkv * 4]), hkv=hkv, D=D, bs=rng.choice([16, 32, 48, 64]),
                    rot=rng.choice([D, D // 2]), layout=rng.randrange(2), dtype=dtype, cache=cache,
                    lens=rng.randrange(1 << 20))
    if op == "attn":
        D = rng.choice([64, 128, 256, 512])
        draft = int(rng.random() < 0.3)
        nq = 1 if draft else rng.randint(1, 7)
        G = rng.choice([g for g in (1, 2, 4, 8, 16) if g * nq <= 64])
        hkv = rng.choice([1, 2, 4, 8])
        B = _log(rng, 1, 64)
        ctx = _log(rng, 1, max(64, min(32768, 64 * 9000 * 4 * 256 // (B * hkv * D))))
        return dict(op=op, B=B, nq=nq, hq=G * hkv, hkv=hkv, D=D, bs=rng.choice([16, 32, 48, 64]),
                    window=rng.choice([0, 0, _log(rng, 64, 1024)]), lo=max(1, ctx // rng.choice([1, 4])),
                    ctx=ctx, draft=draft, lens=rng.randrange(1 << 20))
    V = _log(rng, 64, 262144)
    return dict(op=op, rows=_log(rng, 1, max(1, min(1000, 192 * 262144 // V))), V=V,
                top=rng.choice([0, 1, 5, 20, 32]), T=rng.choice([1.0, 0.7, 1.3]))


def _lens(case, lo, hi):
    """Lengths of the case's sequences, part of the case itself."""
    r = random.Random(case["lens"])
    return [r.randint(lo, hi) for _ in range(case["B"])]


def _esize(name):
    return {"f32": 4, "bf16": 2, "e4m3": 1}[name]


def _append_counts(case):
    """(committed tokens, new tokens) of every sequence."""
    ctx = _lens(case, case["ctx"] // 2, case["ctx"])
    if not case["ragged"]:
        return ctx, [case["n"]] * case["B"]
    r = random.Random(case["lens"] + 1)
    lo, hi = math.log(max(1, case["lo"])), math.log(case["n"])
    new = [int(round(math.exp(lo + (hi - lo) * (i + 0.5) / case["B"]))) for i in range(case["B"])]
    r.shuffle(new)
    ctx = [c if i % 2 else 0 for i, c in enumerate(ctx)]  # every second one starts from nothing
    return ctx, new


def _attn_range(case, L):
    """First and last key of the union of a sequence's queries."""
    if case["draft"]:
        lo = max(0, L - case["window"] + 1) if case["window"] else 0
        return lo, L - 1
    return (max(0, L - case["window"] + 1) if case["window"] else 0), L + case["nq"] - 1


def work(case):
    op = case["op"]
    if op == "rope":
        n = case["rows"] * case["heads"] * case["D"]
        return {"bytes": 2 * n * _esize(case["dtype"]) + 4 * case["rows"],
                "flops": 3 * case["rows"] * case["heads"] * case["rot"]}
    if op == "append":
        rows = sum(_append_counts(case)[1])
        kv = rows * case["hkv"] * case["D"]
        q = rows * case["hq"] * case["D"]
        e = _esize(case["dtype"])
        return {"bytes": 2 * kv * (e + _esize(case["cache"])) + 2 * q * e,
                "flops": 3 * rows * (case["hq"] + case["hkv"]) * case["rot"]}
    if op == "attn":
        by = fl = 0
        for L in _lens(case, case["lo"], case["ctx"]):
            lo, hi = _attn_range(case, L)
            keys = max(0, hi - lo + 1)
            by += keys * case["hkv"] * (case["D"] * 2 + 8.0 / case["bs"])
            fl += 4 * keys * case["hq"] * case["nq"] * case["D"]
        by += 4 * case["B"] * case["nq"] * case["hq"] * case["D"]
        return {"bytes": by, "flops": fl}
    return {"bytes": case["rows"] * (4 * case["V"] + 12 + 8 * case["top"]),
            "flops": 6 * case["rows"] * case["V"]}


# ------------------------------------------------------------------------------------ inputs

_DT = {"f32": torch.float32, "bf16": torch.bfloat16}
BASE = 1000000.0
FACTOR, ORIG_CTX, BETA_FAST, BETA_SLOW = 4.0, 8192, 32.0, 1.0


def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed) & 0x7FFFFFFF)
    return g


def _randn(shape, g, dtype=torch.float32):
    return torch.randn(shape, device="cuda", generator=g, dtype=torch.float32).to(dtype)


def _tables(need, bs, seed):
    """Shuffled block table for sequences that need ``need`` token slots each."""
    blocks = [(n + bs - 1) // bs for n in need]
    nb = sum(blocks) + 3
    perm = np.random.RandomState(int(seed) & 0x7FFFFFFF).permutation(nb).astype(np.int32)
    table = np.zeros((len(need), max(1, max(blocks))), np.int32)
    at = 0
    for b, n in enumerate(blocks):
        table[b, :n] = perm[at:at + n]
        at += n
    return torch.from_numpy(table).cuda(), nb


def _codes(shape, g):
    """e4m3 codes of a cache whose rows were quantised block by block."""
    x = torch.randn(shape, device="cuda", generator=g, dtype=torch.float32)
    return x.mul_(112.0).clamp_(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn)


def _scales(nb, hkv, g):
    e = torch.randint(-9, -6, (nb, hkv), device="cuda", generator=g)
    return torch.exp2(e.float())


def prepare(case, seed):
    op = case["op"]
    g = _gen(seed)
    s = {"case": case}
    if op == "rope":
        rows, n = case["rows"], case["per_seq"]
        B = (rows + n - 1) // n
        s["x"] = _randn((rows, case["heads"], case["D"]), g, _DT[case["dtype"]])
        if n == 1 and case["ctx"] == 0:  # a prompt: positions 0 .. rows - 1
            s["pos"] = torch.arange(rows, device="cuda", dtype=torch.int32)
        else:
            ctx = torch.randint(case["ctx"] // 2, case["ctx"] + 1, (B,), device="cuda", generator=g)
            s["pos"] = (ctx[:, None] + torch.arange(n, device="cuda")).reshape(-1)[:rows].to(torch.int32)
        return s
    if op == "append":
        ctx, new = _append_counts(case)
        rows, hkv, D, bs = sum(new), case["hkv"], case["D"], case["bs"]
        s["table"], nb = _tables([a + b for a, b in zip(ctx, new)], bs, seed)
        s["ctx"] = torch.tensor(ctx, dtype=torch.int32, device="cuda")
        cu = np.zeros(len(new) + 1, np.int32)
        cu[1:] = np.cumsum(new)
        s["cu"] = torch.from_numpy(cu).cuda() if case["ragged"] else None
        dt = _DT[case["dtype"]]
        gain = torch.exp(_randn((hkv, D), g) * 0.5)  # channels of unlike size, as keys have
        s["k"] = (_randn((rows, hkv, D), g) * gain).to(dt)
        s["v"] = _randn((rows, hkv, D), g, dt)
        s["q"] = _randn((rows, case["hq"], D), g, dt) if case["hq"] else None
        if case["cache"] == "e4m3":
            s["kc"], s["vc"] = _codes((nb, hkv, bs, D), g), _codes((nb, hkv, bs, D), g)
            s["ks"], s["vs"] = _scales(nb, hkv, g), _scales(nb, hkv, g)
        else:
            s["kc"], s["vc"] = _randn((nb, hkv, bs, D), g, dt), _randn((nb, hkv, bs, D), g, dt)
            s["ks"] = s["vs"] = None
        return s
    if op == "attn":
        lens = _lens(case, case["lo"], case["ctx"])
        hkv, D, bs = case["hkv"], case["D"], case["bs"]
        s["table"], nb = _tables([n + case["nq"] for n in lens], bs, seed)
        s["ctx"] = torch.tensor(lens, dtype=torch.int32, device="cuda")
        s["q"] = _randn((case["B"], case["nq"], case["hq"], D), g, torch.bfloat16)
        s["kc"], s["vc"] = _codes((nb, hkv, bs, D), g), _codes((nb, hkv, bs, D), g)
        s["ks"], s["vs"] = _scales(nb, hkv, g), _scales(nb, hkv, g)
        return s
    s["z"] = _randn((case["rows"], case["V"]), g) * 2.5
    pick = torch.randn((case["rows"], case["V"]), device="cuda", generator=g) * 2.5
    s["tok"] = torch.argmax(s["z"] + pick, dim=1).to(torch.int32)  # likely tokens, not always the first
    return s


# ------------------------------------------------------------------------------- plain forms

def _inv_freq(rot, scaling):
    i = torch.arange(rot // 2, device="cuda", dtype=torch.float64)
    f = torch.pow(torch.tensor(BASE, device="cuda", dtype=torch.float64), -2.0 * i / rot)
    if scaling == 1:
        return f / FACTOR, 1.0
    if scaling == 2:
        turns = ORIG_CTX * f / (2 * math.pi)
        keep = ((turns - BETA_SLOW) / (BETA_FAST - BETA_SLOW)).clamp(0.0, 1.0)
        return f * keep + f / FACTOR * (1 - keep), 0.1 * math.log(FACTOR) + 1.0
    return f, 1.0


def _rotate(x, pos, rot, layout, scaling):
    """x [rows, heads, D] in float32, turned by its rows' positions (angles in 64 bits)."""
    f, amp = _inv_freq(rot, scaling)
    th = pos.double()[:, None] * f
    c, s = (th.cos() * amp).float()[:, None], (th.sin() * amp).float()[:, None]
    x = x.float()
    r, rest = x[..., :rot], x[..., rot:]
    if layout == 0:
        a, b = r[..., :rot // 2], r[..., rot // 2:]
        r = torch.cat((a * c - b * s, b * c + a * s), dim=-1)
    else:
        a, b = r[..., 0::2], r[..., 1::2]
        r = torch.stack((a * c - b * s, b * c + a * s), dim=-1).flatten(-2)
    return torch.cat((r, rest), dim=-1)


def _row_places(s):
    """Sequence and position of every new row."""
    case, B = s["case"], s["ctx"].numel()
    if s["cu"] is None:
        seq = torch.arange(B, device="cuda").repeat_interleave(case["n"])
        j = torch.arange(B * case["n"], device="cuda") % case["n"]
    else:
        n = (s["cu"][1:] - s["cu"][:-1]).long()
        seq = torch.repeat_interleave(torch.arange(B, device="cuda"), n, output_size=s["k"].shape[0])
        j = torch.arange(s["k"].shape[0], device="cuda") - s["cu"][:-1].long()[seq]
    return seq, s["ctx"].long()[seq] + j


def _exponent(amax):
    """Smallest e >= E_MIN with amax <= 448 * 2^e (448 = 0.875 * 2^9)."""
    m, x = torch.frexp(amax)
    e = x - 9 + (m > 0.875).int()
    return torch.where(amax > 0, e, torch.full_like(e, E_MIN)).clamp(min=E_MIN)


def _append_q8(s, x, codes, scales, blk, off, seq, pos):
    """Quantises the rows x [rows, h, D] (float32) into their blocks, in place."""
    nb, h, bs, D = codes.shape
    amax = torch.zeros((nb, h), device="cuda").index_reduce_(0, blk, x.abs().amax(-1), "amax")
    first = torch.full((nb,), bs, device="cuda").scatter_reduce_(0, blk, off, "amin")
    touched, goes_on = first < bs, (first > 0) & (first < bs)
    need = torch.exp2(_exponent(amax).float())
    new = torch.where(goes_on[:, None], torch.maximum(need, scales), need)
    # live rows of blocks that go on, in the new scale
    b = torch.nonzero(goes_on).flatten()
    live = torch.arange(bs, device="cuda")[None, :] < first[b][:, None]
    old = codes.view(torch.uint8)[b].view(torch.float8_e4m3fn)
    moved = (old.float() * (scales[b] / new[b])[..., None, None]).to(torch.float8_e4m3fn)
    codes.view(torch.uint8)[b] = torch.where(live[:, None, :, None], moved.view(torch.uint8), old.view(torch.uint8))
    scales.copy_(torch.where(touched[:, None], new, scales))
    q = (x / new[blk][..., None]).to(torch.float8_e4m3fn)
    codes.view(torch.uint8)[blk, :, off] = q.view(torch.uint8)


def _plain_append(s):
    case, bs = s["case"], s["case"]["bs"]
    seq, pos = _row_places(s)
    blk, off = s["table"].long()[seq, pos // bs], pos % bs
    k = _rotate(s["k"], pos, case["rot"], case["layout"], 0)
    if case["cache"] == "e4m3":
        _append_q8(s, k, s["kc"], s["ks"], blk, off, seq, pos)
        _append_q8(s, s["v"].float(), s["vc"], s["vs"], blk, off, seq, pos)
    else:
        s["kc"][blk, :, off] = k.to(s["kc"].dtype)
        s["vc"][blk, :, off] = s["v"]
    q = _rotate(s["q"], pos, case["rot"], case["layout"], 0).to(s["q"].dtype) if s["q"] is not None else None
    return {"k": s["kc"], "v": s["vc"], "ks": s["ks"], "vs": s["vs"], "q": q}


def _plain_attn(s):
    case = s["case"]
    B, nq, hq, hkv, D, bs, W = (case[x] for x in ("B", "nq", "hq", "hkv", "D", "bs", "window"))
    L = s["ctx"].long()
    first = (L - W + 1).clamp(min=0) if W else torch.zeros_like(L)
    most = min(W + nq, case["ctx"] + nq) if W else case["ctx"] + nq
    pos = first[:, None] + torch.arange(most, device="cuda")  # keys that some query may read
    last = L - 1 if case["draft"] else L + nq - 1
    inside = pos <= last[:, None]
    at = torch.where(inside, pos, torch.zeros_like(pos))
    blk, off = torch.gather(s["table"].long(), 1, at // bs), at % bs
    K = s["kc"].view(torch.uint8)[blk, :, off].view(torch.float8_e4m3fn).float() * s["ks"][blk][..., None]
    V = s["vc"].view(torch.uint8)[blk, :, off].view(torch.float8_e4m3fn).float() * s["vs"][blk][..., None]
    q = s["q"].float().view(B, nq, hkv, hq // hkv, D).permute(0, 2, 3, 1, 4).reshape(B, hkv, -1, D)
    S = torch.matmul(q, K.permute(0, 2, 3, 1)) / math.sqrt(D)  # [B, hkv, G * nq, keys]
    t = L[:, None] + torch.arange(nq, device="cuda")
    ok = inside[:, None] & (pos[:, None] <= t[..., None])
    if W:
        ok = ok & (pos[:, None] > t[..., None] - W)
    S = S.view(B, hkv, -1, nq, most).masked_fill(~ok[:, None, None], -math.inf)
    m = S.amax(-1, keepdim=True)
    e = torch.exp(S - torch.where(m == -math.inf, torch.zeros_like(m), m))
    d = e.sum(-1, keepdim=True)
    p = (e / torch.where(d > 0, d, torch.ones_like(d))).view(B, hkv, -1, most)
    o = torch.matmul(p, V.permute(0, 2, 1, 3)).view(B, hkv, hq // hkv, nq, D)
    return o.permute(0, 3, 1, 2, 4).reshape(B, nq, hq, D).to(torch.bfloat16)


def _plain_logprobs(s):
    case = s["case"]
    x = s["z"] / case["T"]
    m = x.amax(1, keepdim=True)
    e = torch.exp(x - m)
    S = e.sum(1, keepdim=True)
    logS = torch.log(S)
    lp = torch.gather(x, 1, s["tok"].long()[:, None]) - m - logS
    H = logS - ((x - m) * e).sum(1, keepdim=True) / S
    out = {"logprob": lp[:, 0], "entropy": H[:, 0]}
    if case["top"]:
        # equal logits in the order of their ids
        ids = torch.sort(s["z"], dim=1, descending=True, stable=True)[1][:, :case["top"]]
        out["ids"] = ids.to(torch.int32)
        out["top"] = torch.gather(x, 1, ids) - m - logS
    return out


# --------------------------------------------------------------------- the framework's calls

def _plan(s):
    """Descriptors, tables, workspaces and output buffers that a program keeps beside its inputs."""
    import verify_step_b200 as sd
    case, p = s["case"], {}
    dev = "cuda"
    code = {"f32": sd.SD_F32, "bf16": sd.SD_BF16, "e4m3": sd.SD_E4M3}
    p["sd"] = sd
    if case["op"] in ("rope", "append"):
        scaling = case.get("scaling", 0)
        p["freqs"] = torch.empty(case["rot"] // 2, dtype=torch.int64, device=dev)
        amp = sd.sd_rope_freqs(sd.RopeFreqDesc(rot_dim=case["rot"], base=BASE, scaling=scaling,
                                               factor=FACTOR, orig_ctx=ORIG_CTX, beta_fast=BETA_FAST,
                                               beta_slow=BETA_SLOW), p["freqs"])
        p["rot"] = sd.rotary(p["freqs"], case["layout"], amp)
    if case["op"] == "rope":
        ld = case["heads"] * case["D"]
        p["desc"] = sd.RopeDesc(rows=case["rows"], heads=case["heads"], head_dim=case["D"], ld_x=ld,
                                ld_out=ld, dtype=code[case["dtype"]])
        p["out"] = torch.empty_like(s["x"])
    elif case["op"] == "append":
        hkv, hq, D = case["hkv"], case["hq"], case["D"]
        p["desc"] = sd.AppendDesc(batch=case["B"], n_new=0 if case["ragged"] else case["n"],
                                  n_rows=s["k"].shape[0], h_q=hq, h_kv=hkv, head_dim=D,
                                  block_size=case["bs"], max_blocks_per_seq=s["table"].shape[1],
                                  num_blocks=s["kc"].shape[0], ld_k=hkv * D, ld_v=hkv * D, ld_q=hq * D,
                                  ld_q_out=hq * D, dtype=code[case["dtype"]],
                                  cache_dtype=code[case["cache"]])
        p["q"] = torch.empty_like(s["q"]) if s["q"] is not None else None
    elif case["op"] == "attn":
        p["desc"] = sd.AttnDesc(batch=case["B"], n_q=case["nq"], h_q=case["hq"], h_kv=case["hkv"],
                                head_dim=case["D"], block_size=case["bs"],
                                max_blocks_per_seq=s["table"].shape[1], num_blocks=s["kc"].shape[0],
                                window=case["window"], scale=1.0 / math.sqrt(case["D"]),
                                dtype=sd.SD_BF16)
        size = sd.sd_draft_xattn_q8_workspace_size if case["draft"] else sd.sd_verify_attn_q8_workspace_size
        p["ws"] = torch.empty(max(16, size(p["desc"])), dtype=torch.uint8, device=dev)
        p["out"] = torch.empty_like(s["q"])
    else:
        rows, top = case["rows"], case["top"]
        p["desc"] = sd.LogprobsDesc(rows=rows, vocab=case["V"], temperature=case["T"], top_n=top)
        p["ws"] = torch.empty(max(16, sd.sd_logprobs_workspace_size(p["desc"])), dtype=torch.uint8, device=dev)
        p["out"] = {"logprob": torch.empty(rows, device=dev), "entropy": torch.empty(rows, device=dev)}
        if top:
            p["out"]["ids"] = torch.empty((rows, top), dtype=torch.int32, device=dev)
            p["out"]["top"] = torch.empty((rows, top), device=dev)
    return p


def _own(s):
    p = s.get("plan")
    if p is None:
        p = s["plan"] = _plan(s)
    sd, case = p["sd"], s["case"]
    if case["op"] == "rope":
        sd.sd_rope(p["desc"], p["rot"], s["x"], s["pos"], None, p["out"])
        return p["out"]
    if case["op"] == "append":
        sd.sd_append_kv(p["desc"], p["rot"], s["k"], s["v"], s["q"], s["kc"], s["vc"], s["ks"], s["vs"],
                        s["table"], s["ctx"], s["cu"], p["q"])
        return {"k": s["kc"], "v": s["vc"], "ks": s["ks"], "vs": s["vs"], "q": p["q"]}
    if case["op"] == "attn":
        if case["draft"]:
            sd.sd_draft_xattn_q8(p["desc"], s["q"], s["kc"], s["vc"], s["ks"], s["vs"], s["table"],
                                 s["ctx"], None, p["out"], p["ws"])
        else:
            sd.sd_verify_attn_q8(p["desc"], s["q"], s["kc"], s["vc"], s["ks"], s["vs"], s["table"],
                                 s["ctx"], p["out"], p["ws"])
        return p["out"]
    o = p["out"]
    sd.sd_logprobs(p["desc"], s["z"], s["tok"], o["logprob"], o["entropy"], o.get("ids"), o.get("top"), p["ws"])
    return o


def run(state):
    if own:
        return _own(state)
    op = state["case"]["op"]
    if op == "rope":
        c = state["case"]
        return _rotate(state["x"], state["pos"], c["rot"], c["layout"], c["scaling"]).to(state["x"].dtype)
    if op == "append":
        return _plain_append(state)
    return _plain_attn(state) if op == "attn" else _plain_logprobs(state)


# ----------------------------------------------------------------------- from the definitions

def _turned(x, pos, rot, layout, scaling):
    """Complex multiplication by A exp(i theta), 64 bits."""
    freq, amp = [], 1.0
    for i in range(rot // 2):
        f = BASE ** (-2.0 * i / rot)
        if scaling == 1:
            f /= FACTOR
        elif scaling == 2:
            g = min(1.0, max(0.0, (ORIG_CTX * f / (2 * math.pi) - BETA_SLOW) / (BETA_FAST - BETA_SLOW)))
            f, amp = f * (g + (1.0 - g) / FACTOR), 1.0 + 0.1 * math.log(FACTOR)
        freq.append(f)
    th = torch.outer(pos.double(), torch.tensor(freq, dtype=torch.float64, device=x.device))
    y = x.double().clone()
    re, im = ((slice(0, rot // 2), slice(rot // 2, rot)) if layout == 0 else
              (slice(0, rot, 2), slice(1, rot, 2)))
    z = torch.complex(y[..., re].contiguous(), y[..., im].contiguous())
    z = z * torch.polar(torch.full_like(th, amp), th)[:, None]
    y[..., re], y[..., im] = z.real, z.imag
    return y


def _nearest_e4m3(x):
    """Nearest e4m3 value (ties to even) of float64 x, |x| <= 448: 3 fraction bits, exponent >= -6."""
    a = x.abs()
    step = torch.exp2(torch.floor(torch.log2(a.clamp(min=2.0 ** -6))) - 3)
    return torch.sign(x) * torch.round(a / step) * step


def _exact_append(s):
    case = s["case"]
    bs, B = case["bs"], case["B"]
    ctx, new = _append_counts(case)
    table = s["table"].cpu().numpy()
    kc, vc = s["kc"].to(torch.float64), s["vc"].to(torch.float64)
    ks, vs = (None, None) if s["ks"] is None else (s["ks"].double(), s["vs"].double())
    pos = torch.cat([torch.arange(c, c + n) for c, n in zip(ctx, new)]).cuda()
    k = _turned(s["k"], pos, case["rot"], case["layout"], 0)
    q = _turned(s["q"], pos, case["rot"], case["layout"], 0) if s["q"] is not None else None
    row = 0
    for b in range(B):
        p, end = ctx[b], ctx[b] + new[b]
        while p < end:  # one block at a time
            i, o = int(table[b, p // bs]), p % bs
            n = min(bs - o, end - p)
            for src, c, sc in ((k, kc, ks), (s["v"].double(), vc, vs)) if case["cache"] == "e4m3" else ((k, kc, None), (s["v"].double(), vc, None)):
                x = src[row:row + n].transpose(0, 1)  # [hkv, n, D]
                if sc is None:
                    c[i, :, o:o + n] = x
                    continue
                top = x.abs().amax((1, 2)).clamp(min=E4M3_MAX * 2.0 ** E_MIN)
                need = torch.exp2(torch.ceil(torch.log2(top / E4M3_MAX)))
                if o:
                    need = torch.maximum(need, sc[i])
                    c[i, :, :o] = _nearest_e4m3(c[i, :, :o] * (sc[i] / need)[:, None, None])
                sc[i] = need
                c[i, :, o:o + n] = _nearest_e4m3(x / need[:, None, None])
            p += n
            row += n
    return {"k": kc, "v": vc, "ks": ks, "vs": vs, "q": q}


def _exact_attn(s):
    case = s["case"]
    nq, hkv, D, bs, W = (case[x] for x in ("nq", "hkv", "D", "bs", "window"))
    G = case["hq"] // hkv
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda")
    for b, L in enumerate(_lens(case, case["lo"], case["ctx"])):
        n = L if case["draft"] else L + nq
        blocks = s["table"][b, :(n + bs - 1) // bs].long()
        kv = []
        for c, sc in ((s["kc"], s["ks"]), (s["vc"], s["vs"])):
            x = c.view(torch.uint8)[blocks].view(torch.float8_e4m3fn).double() * sc[blocks].double()[..., None, None]
            kv.append(x.transpose(0, 1).reshape(hkv, -1, D)[:, :n])
        for j in range(nq):
            t = L + j
            lo, hi = (max(0, t - W + 1) if W else 0), min(t, n - 1)
            if hi < lo:
                continue
            q = s["q"][b, j].double().view(hkv, G, D)
            w = torch.softmax(torch.bmm(q, kv[0][:, lo:hi + 1].transpose(1, 2)) / math.sqrt(D), dim=-1)
            out[b, j] = torch.bmm(w, kv[1][:, lo:hi + 1]).reshape(-1, D)
    return out


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "rope":
        return _turned(s["x"], s["pos"], case["rot"], case["layout"], case["scaling"])
    if case["op"] == "append":
        return _exact_append(s)
    if case["op"] == "attn":
        return _exact_attn(s)
    lp = torch.log_softmax(s["z"].double() / case["T"], dim=1)
    out = {"logprob": lp[torch.arange(case["rows"]), s["tok"].long()],
           "entropy": -(lp.exp() * lp).sum(1)}
    if case["top"]:
        z = s["z"].cpu().numpy()
        ids = np.stack([np.lexsort((np.arange(case["V"]), -r))[:case["top"]] for r in z])
        out["ids"] = torch.from_numpy(ids.astype(np.int32))
        out["top"] = torch.gather(lp, 1, torch.from_numpy(ids).cuda())
    return out
