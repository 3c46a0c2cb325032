"""sd_verify_attn_q8 / sd_draft_xattn_q8 at the ends of what the header allows.  Tolerances are
those of test_gpu_attn_q8, without its constant 1e-30 where outputs are small; a bf16 output below
2^-126 is off by half its fixed step, 2^-134.
"""
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
