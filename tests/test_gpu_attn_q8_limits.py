"""sd_verify_attn_q8 / sd_draft_xattn_q8 at the ends of what the header allows.  Tolerances are
those of test_gpu_attn_q8, without its constant 1e-30 where outputs are small; a bf16 output below
2^-126 is off by half its fixed step, 2^-134.
"""
import math

import numpy as np
import pytest
import torch

import verify_step_b200 as sd
from tests.gpu_util import status_ok
from tests.test_gpu_attn_q8 import Case

pytestmark = pytest.mark.gpu

INT_MAX = 2 ** 31 - 1


def held(c, got=None):
    """Every output within the bound of its own size."""
    got = c.run() if got is None else got
    want, tol = c.reference()
    tol = tol - 1e-30 + 2.0 ** -134
    assert np.all(np.isfinite(got))
    assert np.all(np.abs(got - want) <= tol), float((np.abs(got - want) / tol).max())
    assert status_ok()
    return got


# ------------------------------------------------------------------------------- windows

@pytest.mark.parametrize("n_q", [3, 7])
@pytest.mark.parametrize("window", [INT_MAX, INT_MAX - 1, INT_MAX - 200, 2 ** 30])
def test_a_window_longer_than_every_sequence_hides_nothing(window, n_q):
    c = Case(1, [300, 17, 126, 0], n_q, 4, 2, 128, 16)
    plain = c.run()
    c.desc.window = c.window = window
    got = held(c)
    assert np.array_equal(got, plain)


@pytest.mark.parametrize("window,q_pos", [(INT_MAX, INT_MAX), (INT_MAX, 5), (INT_MAX - 99, INT_MAX),
                                          (INT_MAX - 400, INT_MAX - 1)])
def test_drafter_windows_and_positions_near_the_integer_limit(window, q_pos):
    held(Case(2, [300, 90], 1, 4, 2, 256, 16, window, draft=True, q_pos=[q_pos] * 2))


# -------------------------------------------------------------------------------- scales

@pytest.mark.parametrize("e", [-30, -79, -81, -100, -120, -126, -131, -140, 30, 100])
@pytest.mark.parametrize("L,D", [([200, 40], 128), ([5000], 256)])
def test_v_scales_of_any_size(L, D, e):
    """The output scales with them; the second length is joined from many CTAs."""
    c = Case(3, L, 3, 4, 1, D, 16)
    c.vs[:] = 2.0 ** e
    held(c)


@pytest.mark.parametrize("L,D", [([200, 40], 128), ([5000], 512)])
def test_v_scales_all_zero_give_zeros(L, D):
    c = Case(4, L, 2, 4, 2, D, 16)
    c.vs[:] = 0
    got = c.run()
    assert np.all(got == 0) and status_ok()


@pytest.mark.parametrize("low,high", [(0.0, 1.0), (2.0 ** -100, 1.0), (2.0 ** -140, 2.0 ** -100),
                                      (2.0 ** -60, 2.0 ** 60), (2.0 ** -20, 2.0 ** 110), (0.0, 2.0 ** -120)])
@pytest.mark.parametrize("L", [[200, 40], [6000]])
def test_v_scales_far_apart(L, low, high):
    """The keys of a tiny scale still take their share of the softmax."""
    c = Case(5, L, 3, 4, 1, 128, 16)
    g = torch.Generator().manual_seed(6)
    few = torch.rand(c.vs.shape, generator=g) < 0.1
    c.vs[:] = torch.where(few, high, low)
    held(c)
    c.vs[:] = torch.where(few, low, high)
    held(c)


@pytest.mark.parametrize("eq,ek", [(-110, 104), (-100, 94), (-126, 120), (-90, 84), (60, -66),
                                   (100, -106), (0, -6)])
def test_queries_and_k_scales_of_any_size(eq, ek):
    """Scores are about one, made of tiny queries and large scales or the other way round."""
    c = Case(7, [300, 60], 3, 8, 2, 128, 16)
    c.q = (c.q.double() * 2.0 ** eq).bfloat16()
    c.ks[:] = 2.0 ** ek
    held(c)


def test_keys_of_zeros_under_large_scales():
    """Their scores are 0, however large the query and the scale: the output is the values' mean."""
    c = Case(13, [100, 20], 2, 4, 2, 128, 16)
    c.q = (c.q.double() * 2.0 ** 120).bfloat16()
    c.kc[:] = 0
    c.ks[:] = 2.0 ** 60
    held(c)


def test_a_key_of_nearly_all_weight_whose_value_is_zero():
    """What is left of the output are the light keys of its tile, 2^-12 to 2^-20 of it each: a weight is
    off by the larger of 2^-8 of it and 2^-22 of the tile's largest."""
    D, L = 128, 120
    c = Case(8, [L], 1, 1, 1, D, 16)
    one = torch.tensor([1.0]).to(torch.float8_e4m3fn).view(torch.uint8)[0]
    light = np.exp2(-12 - 8 * np.arange(L + 1) / L)
    c.kc[:] = 0
    c.vc[:] = one
    c.ks[:] = c.vs[:] = 1.0
    c.q[:] = 0
    # key 0 scores 0, the others -12 ln 2: their scale spreads them down to -20 ln 2
    c.q[0, 0, 0, 0] = 12 * math.log(2) / c.desc.scale
    for p in range(1, L + 1):
        c.kc[c.table[0, p // 16], 0, p % 16, 0] = one | 0x80
        c.ks[c.table[0, p // 16]] = 1 + (p // 16) / 12
    c.vc[c.table[0, 0], 0, 0] = 0
    held(c)


# ------------------------------------------------------------------------------- lengths

@pytest.mark.parametrize("L", [INT_MAX, INT_MAX - 1, INT_MAX - 130])
def test_a_length_near_the_integer_limit_is_recorded(L):
    c = Case(9, [40, 40], 3, 4, 2, 64, 16)
    want, tol = c.reference()
    c.L[0] = L
    got = c.run()
    assert sd.sd_device_status_read() == sd.SD_ERR_DEVICE
    sd.sd_device_status_clear()
    assert np.all(got[0] == 0) and np.all(np.abs(got - want)[1] <= tol[1])


# ---------------------------------------------------------------------------- row groups

@pytest.mark.parametrize("L,n_q,hq,hkv,D,bs,window", [
    ([700, 31, 0], 7, 8, 2, 512, 16, 40),      # 28 rows: groups of 14
    ([513], 16, 4, 1, 512, 48, 3),             # 64 rows: three groups, a window inside a group's own
    ([300, 2], 9, 5, 1, 256, 16, 130),         # 45 rows
    ([129, 1000], 33, 1, 1, 64, 32, 20),       # 33 rows: 17 and 16
    ([90], 64, 1, 1, 128, 16, 0)])
def test_row_groups_with_windows(L, n_q, hq, hkv, D, bs, window):
    held(Case(10 + D, L, n_q, hq, hkv, D, bs, window))


@pytest.mark.parametrize("hq,hkv,D,window", [(40, 1, 512, 0), (50, 1, 128, 33), (64, 1, 64, 200),
                                             (66, 2, 256, 16)])
def test_row_groups_of_drafter_calls(hq, hkv, D, window):
    held(Case(11, [700, 3, 0], 1, hq, hkv, D, 16, window, draft=True, q_pos=[705, 3, 1]))


@pytest.mark.parametrize("n_q,hq,D,window", [(7, 4, 512, 0), (16, 4, 128, 0), (16, 4, 512, 20),
                                             (9, 4, 256, 300)])
def test_nan_with_several_row_groups(n_q, hq, D, window):
    """A NaN in V makes its column NaN for every query that attends to the key, and nothing for the
    others, whichever group a query is in."""
    L = 200
    for at in (L + n_q - 2, L + 2, L, max(0, L - window + 3) if window else 5):
        c = Case(12, [L], n_q, hq, 1, D, 16, window)
        want, tol = c.reference()
        c.vc[c.table[0, at // 16], 0, at % 16, 5] = 0x7F
        got = c.run()
        for j in range(n_q):
            t = L + j
            sees = at <= t and (not window or at >= t - window + 1)
            if sees:
                assert np.all(np.isnan(got[0, j, :, 5])), (at, j)
            else:
                assert np.all(np.abs(got[0, j] - want[0, j]) <= tol[0, j]), (at, j)
        assert status_ok()
