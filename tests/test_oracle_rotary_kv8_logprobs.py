"""Pins of the float64 oracle of rotary positions, the e4m3 cache and the log probabilities: closed
forms, invariants and library routines."""
import numpy as np
import pytest
import torch

from oracle import kv8, logprobs as OL, rotary as OR


@pytest.mark.parametrize("layout", [OR.HALF, OR.INTERLEAVED])
def test_rotation_keeps_lengths_and_depends_on_distance_only(layout):
    rng = np.random.default_rng(0)
    q, k = rng.standard_normal((1, 1, 16)), rng.standard_normal((1, 1, 16))
    f, _ = OR.frequencies(12, 10000.0)
    dots = []
    for t in (0, 5, 100000):
        a = OR.rotate(q, [t + 3], f, layout=layout)
        b = OR.rotate(k, [t], f, layout=layout)
        assert np.allclose(np.linalg.norm(a), np.linalg.norm(q))
        assert np.array_equal(a[..., 12:], q[..., 12:])  # behind the rotating part
        dots.append(float((a * b).sum()))
    assert np.allclose(dots, dots[0])
    assert np.array_equal(OR.rotate(q, [0], f, layout=layout), q)


def test_rotation_is_multiplication_by_a_unit_number():
    rng = np.random.default_rng(1)
    x = rng.standard_normal((3, 2, 8))
    f, _ = OR.frequencies(8, 100.0)
    t = np.array([1, 7, 50])
    z = (x[..., 0::2] + 1j * x[..., 1::2]) * np.exp(1j * t[:, None, None] * f)
    y = OR.rotate(x, t, f, layout=OR.INTERLEAVED)
    assert np.allclose(y[..., 0::2], z.real) and np.allclose(y[..., 1::2], z.imag)
    # the half layout is the same turn of permuted elements
    perm = np.concatenate([np.arange(0, 8, 2), np.arange(1, 8, 2)])
    assert np.allclose(OR.rotate(x[..., perm], t, f, layout=OR.HALF), y[..., perm])


def test_stretched_frequencies():
    f, a = OR.frequencies(64, 10000.0)
    assert f[0] == 1.0 and a == 1.0
    g, a = OR.frequencies(64, 10000.0, OR.LINEAR, 4.0)
    assert np.allclose(g, f / 4) and a == 1.0
    h, a = OR.frequencies(64, 10000.0, OR.BY_PARTS, 4.0, 4096, 32.0, 1.0)
    turns = 4096 * f / (2 * np.pi)
    assert np.allclose(h[turns >= 32], f[turns >= 32])
    assert np.allclose(h[turns <= 1], f[turns <= 1] / 4)
    assert np.all((h <= f) & (h >= f / 4)) and np.isclose(a, 1 + 0.1 * np.log(4))


def test_e4m3_codes_match_the_library():
    codes = torch.arange(256, dtype=torch.uint8)
    want = codes.view(torch.float8_e4m3fn).double().numpy()
    assert np.array_equal(kv8.DECODE, want, equal_nan=True)
    rng = np.random.default_rng(2)
    x = np.concatenate([rng.standard_normal(4000) * 100, rng.standard_normal(2000) * 2.0 ** -8,
                        kv8.DECODE[:127], (kv8.DECODE[:126] + kv8.DECODE[1:127]) / 2,  # ties
                        [448.0, -448.0, 0.0, -0.0]])
    x = np.clip(x, -448, 448).astype(np.float32)
    want = torch.from_numpy(x).to(torch.float8_e4m3fn).view(torch.uint8).numpy()
    assert np.array_equal(kv8.encode(x), want)
    assert kv8.encode(np.array([1e9]))[0] == 0x7E and kv8.encode(np.array([np.nan]))[0] == 0x7F


def test_exponent_is_the_smallest():
    for a in (448.0, 448.0001, 1.0, 3e38, 1e-30, 0.875 * 2.0 ** -20):
        e = kv8.exponent(a)
        assert a <= 448 * 2.0 ** e and (e == kv8.E_MIN or a > 448 * 2.0 ** (e - 1))
    assert kv8.exponent(0.0) == kv8.E_MIN


def test_append_in_parts_equals_append_at_once_up_to_subnormals():
    rng = np.random.default_rng(3)
    x = rng.standard_normal((20, 2, 16)) * np.exp2(rng.integers(0, 3, (20, 1, 1)))
    table = np.array([[1, 0]])
    got = []
    for parts in ([20], [3, 1, 16], [7, 13]):
        c, s = np.zeros((2, 2, 16, 16), np.uint8), np.full((2, 2), np.nan)
        at = 0
        for n in parts:
            kv8.append(c, s, [x[at:at + n]], table, [at], [n], 16)
            at += n
        got.append((c, s))
    for c, s in got[1:]:
        assert np.array_equal(s, got[0][1])
        # values this far above the subnormals are rounded once
        a = kv8.decode(got[0][0])
        big = np.abs(a) >= 2.0 ** -3
        assert np.array_equal(kv8.decode(c)[big], a[big])


def test_logprobs_against_the_library():
    rng = np.random.default_rng(4)
    z = rng.standard_normal((5, 40)) * 3
    z[1, 3:20] = -np.inf
    tok = np.array([0, 25, 39, -1, 40])
    lp, H, ids, top = OL.logprobs(z, tok, 0.8, 6)
    want = torch.log_softmax(torch.from_numpy(z) / 0.8, dim=1)
    for r in range(3):
        assert np.isclose(lp[r], want[r, tok[r]])
        d = torch.distributions.Categorical(logits=torch.from_numpy(z[r]) / 0.8)
        if r != 1:
            assert np.isclose(H[r], float(d.entropy()))
        v, i = torch.topk(want[r], 6)
        assert np.array_equal(ids[r], i.numpy()) and np.allclose(top[r], v.numpy())
    assert lp[3] == lp[4] == 0 and np.all(ids[3:] == -1) and np.all(np.isneginf(top[3:]))
    # equal logits in the order of their ids
    assert np.array_equal(OL.logprobs(np.zeros((1, 9)), [0], 1.0, 4)[2], [[0, 1, 2, 3]])
