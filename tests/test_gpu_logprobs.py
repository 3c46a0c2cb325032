"""GPU parity of sd_logprobs against the float64 oracle.

Ids are exact (equal logits in the order of their ids).  Tolerance of the float outputs, in float32
with x = z / T relative to the row's largest:
  - a weight 2^t is off by 2^-22 relative (the hardware's exp2) plus ln 2 |t| 2^-23 (t is a rounded
    difference times a rounded constant), a partial sum adds at most 60 roundings of 2^-24 (32 of a
    thread, the trees, the chunks): the sum S is off by at most
        dS = 2^-22 + 60 * 2^-24 + 2^-23 ln2 sum(w |t|) / S                          (relative)
  - log p = x - ln S: |x| 2^-23 + dS + 2^-23 |ln S|
  - entropy = ln S - (sum w t) ln 2 / S: dS (1 + |sum w t| ln 2 / S) for both sums, the same again
    for the weighted one, and 2^-22 of the result.
"""
import numpy as np
import pytest
import torch

import verify_step_b200 as sd
from oracle import logprobs as OL
from tests.gpu_util import DEV, status_ok, workspace

pytestmark = pytest.mark.gpu


def run(z, tokens, T=1.0, top=0, V=None, entropy=True, ws=None):
    R, ld = z.shape
    V = ld if V is None else V
    d = sd.LogprobsDesc(rows=R, vocab=V, ld_logits=ld, temperature=T, top_n=top)
    lp = torch.full((R,), 5.0, device=DEV)
    H = torch.full((R,), 5.0, device=DEV) if entropy else None
    ids = torch.full((R, top), -7, dtype=torch.int32, device=DEV) if top else None
    lt = torch.full((R, top), 5.0, device=DEV) if top else None
    ws = workspace(sd.sd_logprobs_workspace_size(d)) if ws is None else ws
    sd.sd_logprobs(d, z.to(DEV), tokens.to(DEV), lp, H, ids, lt, ws)
    torch.cuda.synchronize()
    return [None if t is None else t.cpu().numpy() for t in (lp, H, ids, lt)]


def check(z, tokens, got, T, top):
    zz, tok = z.double().numpy(), tokens.numpy()
    lp, H, ids, lt = OL.logprobs(zz, tok, T, top)
    for r in range(len(tok)):
        if not (0 <= tok[r] < zz.shape[1]) or np.isnan(lp[r]):
            assert np.array_equal(got[0][r], lp[r], equal_nan=True)
            if got[1] is not None:
                assert np.array_equal(got[1][r], H[r], equal_nan=True)
            if top:
                assert np.array_equal(got[2][r], ids[r])
                assert np.array_equal(got[3][r], lt[r], equal_nan=True)
            continue
        x = zz[r] / T - zz[r].max() / T
        w = np.exp(x)
        S = w.sum()
        wt = (w[w > 0] * -x[w > 0]).sum() / S  # sum w |t| ln 2 / S
        dS = 2.0 ** -22 + 60 * 2.0 ** -24 + 2.0 ** -23 * wt
        tol = lambda l: 2.0 ** -23 * np.abs(l + np.log(S)) + dS + 2.0 ** -23 * np.log(S) + 1e-7
        if np.isneginf(lp[r]):
            assert np.isneginf(got[0][r])
        else:
            assert abs(got[0][r] - lp[r]) <= tol(lp[r])
        if got[1] is not None:
            assert abs(got[1][r] - H[r]) <= 2 * dS * (1 + wt) + 2.0 ** -22 * H[r] + 2.0 ** -23 * np.log(S) + 1e-7
        if top:
            assert np.array_equal(got[2][r], ids[r])
            fin = np.isfinite(lt[r])
            assert np.array_equal(np.isneginf(got[3][r]), ~fin)
            assert np.all(np.abs(got[3][r][fin] - lt[r][fin]) <= tol(lt[r][fin]))


@pytest.mark.parametrize("R,V,top,T", [
    (1, 1, 1, 1.0), (3, 1024, 0, 1.0), (2, 7, 7, 0.5), (5, 100, 32, 1.0), (4, 2049, 20, 1.3),
    (3, 8193, 5, 0.7), (1, 262144, 20, 1.0), (24, 262144, 5, 1.0), (2, 100001, 32, 1.0),
    (300, 4099, 8, 1.0), (40, 50000, 1, 2.0)])
def test_matches_the_oracle(R, V, top, T):
    g = torch.Generator().manual_seed(R + V)
    z = torch.randn((R, V), generator=g) * 3
    tok = torch.randint(0, V, (R,), generator=g, dtype=torch.int32)
    check(z, tok, run(z, tok, T, top), T, top)
    assert status_ok()


def test_rows_with_a_stride_and_without_entropy():
    g = torch.Generator().manual_seed(1)
    for ld in (5000, 4999):  # 16-byte aligned rows, and not
        z = torch.full((6, ld), float("nan"))
        z[:, :4321] = torch.randn((6, 4321), generator=g)
        tok = torch.randint(0, 4321, (6,), generator=g, dtype=torch.int32)
        got = run(z, tok, 1.0, 3, V=4321, entropy=False)
        check(z[:, :4321], tok, got, 1.0, 3)


@pytest.mark.parametrize("V", [900, 60000])
def test_masked_padded_and_odd_rows(V):
    g = torch.Generator().manual_seed(2)
    z = torch.randn((12, V), generator=g)
    z[1, : V - 3] = -float("inf")          # three tokens left
    z[2] = -float("inf")                   # none
    z[3, 17] = float("nan")
    z[4, V - 1] = float("inf")
    z[5, ::2] = -float("inf")
    z[6] = -3.4e38                         # the type's lowest value everywhere
    z[7, 5] = 3.4e38
    z[8, 3], z[8, 9] = 0.0, -0.0
    z[8, 10:] = -1.0
    tok = torch.tensor([-1, V - 1, 0, 0, 0, 1, 4, 6, 3, V, 8, -2 ** 31], dtype=torch.int32)
    tok[5] = 0                             # a masked token
    got = run(z, tok, 1.0, 8)
    check(z, tok, got, 1.0, 8)
    assert sd.sd_device_status_read() == sd.SD_ERR_DEVICE  # the token V
    sd.sd_device_status_clear()


@pytest.mark.parametrize("V", [3000, 8192, 262144])
def test_alternatives_of_equal_and_ordered_logits(V):
    """Equal logits (every key ties but for its id), rising and falling rows, two values, and a row
    whose large logits all lie where one warp of a chunk has none: these take the search by bits."""
    r = torch.arange(V, dtype=torch.float32)
    z = torch.stack([torch.zeros(V), r, -r, (r % 2), torch.where((r % 1024) < 896, r % 7, -50.0),
                     torch.where((r.long() // 32) % 8 == 7, -float("inf"), 1.0),
                     torch.where(r < V - 40, -float("inf"), 2.0)])
    tok = torch.tensor([0, V - 1, 0, 1, 3, 0, V - 1], dtype=torch.int32)
    for top in (1, 20, 32):
        got = run(z, tok, 1.0, top)
        ids = OL.logprobs(z.double().numpy(), tok.numpy(), 1.0, top)[2]
        assert np.array_equal(got[2], ids)
    assert status_ok()


def test_workspace_is_not_kept_and_a_graph_replays():
    g = torch.Generator().manual_seed(3)
    V = 30000
    z = [torch.randn((4, V), generator=g).to(DEV) for _ in range(2)]
    tok = torch.randint(0, V, (4,), generator=g, dtype=torch.int32).to(DEV)
    d = sd.LogprobsDesc(rows=4, vocab=V, temperature=1.0, top_n=4)
    ws = workspace(sd.sd_logprobs_workspace_size(d))
    x = z[0].clone()
    out = [torch.empty(4, device=DEV), torch.empty(4, device=DEV),
           torch.empty((4, 4), dtype=torch.int32, device=DEV), torch.empty((4, 4), device=DEV)]
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        sd.sd_logprobs(d, x, tok, *out, ws)
    for i in (0, 1, 0):
        x.copy_(z[i])
        ws.fill_(255)
        graph.replay()
        torch.cuda.synchronize()
        check(z[i].cpu(), tok.cpu(), [t.cpu().numpy() for t in out], 1.0, 4)
    with pytest.raises(sd.SdError) as e:
        sd.sd_logprobs(d, x, tok, *out, ws[:-1].clone())
    assert e.value.status == sd.SD_ERR_WORKSPACE
