"""Pins of the oracle's rotary positions and 8-bit cache: enumerations, closed forms, differences
and torch's own conversions (no GPU)."""
import math

import numpy as np
import pytest
import torch

import oracle
from block_masked_token_gb300 import packed


def codes():
    """Every finite e4m3 value, from its bits: sign, four bits of exponent, three of fraction."""
    out = []
    for b in range(256):
        e, m = (b >> 3) & 15, b & 7
        if e == 15 and m == 7:
            continue
        v = m / 8 * 2.0 ** -6 if e == 0 else (1 + m / 8) * 2.0 ** (e - 7)
        out.append(-v if b & 128 else v)
    return np.array(out)


def test_e4m3_is_the_nearest_of_all_codes():
    c = codes()
    x = np.concatenate([np.random.default_rng(0).normal(size=500) * 10.0 ** np.linspace(-4, 2.5, 500),
                        c, [0.0, 448.0, 464.0, 1e9, 2.0 ** -10, 2.0 ** -11]])
    got = oracle.e4m3(x)
    assert np.isin(got, c).all()
    assert (np.abs(got - x) == np.abs(c[None] - x[:, None]).min(axis=1)).all()
    assert (oracle.e4m3(c) == c).all()
    # halfway: the code with an even fraction
    for low, high, even in ((1.0, 1.125, 1.0), (1.125, 1.25, 1.25), (0.0, 2.0 ** -9, 0.0)):
        assert oracle.e4m3((low + high) / 2) == even
    assert np.isnan(oracle.e4m3([np.nan, np.inf, -np.inf])).all()
    # within the range it is torch's conversion
    y = torch.from_numpy(np.clip(x, -448, 448))
    assert (y.float().to(torch.float8_e4m3fn).double().numpy() == oracle.e4m3(y.float().numpy())).all()


def test_scales():
    for top, byte in ((448.0, 127), (448.0001, 128), (449.0, 128), (224.0, 126), (3.5, 120),
                      (3.51, 121), (0.0, 87), (1e-30, 87), (1e30, 167)):
        assert oracle.q8_scale(np.array([[-top, top / 2]])) == byte
    assert oracle.q8_scale(np.array([np.inf, np.nan, 1.0])) == oracle.q8_scale(np.array([1.0]))


def appended(n=40, P=21, seed=1, counts=None):
    rng = np.random.default_rng(seed)
    k, v = rng.normal(size=(2, n, 2, 8))
    pool = oracle.e4m3(rng.normal(size=(2, 6, 2, 16, 8)) * 100)
    scale = rng.integers(118, 124, size=(2, 6, 2))
    table = np.array([[3, 1, 4, 0, -1]])
    args = (k, v, [0, n], [P], table, *pool, *scale, 16)
    return args, oracle.kv_append_q8(*args, counts=counts)


def test_append_stands_for_its_rows():
    """Every row comes back within half a step of its page's codes, and so do the tokens held."""
    (k, v, _, _, table, kp, vp, ks, vs, _), (kp2, vp2, ks2, vs2, lens, slots) = appended()
    assert lens.tolist() == [61] and slots.tolist() == [int(table[0, p // 16]) * 16 + p % 16 for p in range(21, 61)]
    for x, pool, scale, old, old_scale in ((k, kp2, ks2, kp, ks), (v, vp2, vs2, vp, vs)):
        value = oracle.q8_values(pool, scale)
        got = np.array([value[s // 16, :, s % 16] for s in slots])
        room = 448 * np.exp2(scale[slots // 16] - 127.0)[..., None]
        # half a step: 2^-4 of the value, or of the smallest normal code, 2^-6 of 448 = 1.75 * 2^8
        assert (np.abs(got - x) <= np.maximum(2.0 ** -4 * np.abs(x), 2.0 ** -10 / 448 * room)).all()
        assert (np.abs(x) <= room).all()
        held, was = value[1, :, :5], oracle.q8_values(old, old_scale)[1, :, :5]
        assert (np.abs(held - was) <= np.maximum(2.0 ** -4 * np.abs(was), 2.0 ** -10 / 448 * room[0][:, None])).all()
        same = [p for p in range(6) if p not in (0, 1, 4)]
        assert (pool[same] == old[same]).all() and (scale[same] == old_scale[same]).all()
        assert (pool[0, :, 13:] == old[0, :, 13:]).all()         # free slots of the last page


def test_append_of_counts_and_in_parts():
    (k, v, cu, _, table, kp, vp, ks, vs, ps), whole = appended(P=16)
    _, some = appended(P=16, counts=[7])
    assert some[4].tolist() == [23] and (some[5][7:] == -1).all()
    # row by row: the same scales, and codes that agree unless a page grew on the way
    state = [kp, vp, ks, vs]
    for i in range(40):
        *state, _, _ = oracle.kv_append_q8(k[i:i + 1], v[i:i + 1], [0, 1], [16 + i], table, *state, ps)
    assert (state[2][[1, 4, 0]] == whole[2][[1, 4, 0]]).all()
    for a, b, s in ((state[0], whole[0], whole[2]), (state[1], whole[1], whole[3])):
        # only the smallest codes are rounded twice: off by at most a code's step, 2^-9
        assert np.abs(a[[1, 4]] - b[[1, 4]]).max() <= 2.0 ** -9


@pytest.mark.parametrize("interleaved", [False, True])
def test_rotary_is_a_complex_product(interleaved):
    rng = np.random.default_rng(2)
    x, f = rng.normal(size=(7, 3, 16)), np.array([1.0, 0.3, 0.01, 2.5])
    y = oracle.rotary(x, [0, 4, 7], [10, 0], f, interleaved, factor=1.5)
    pos = np.array([10, 11, 12, 13, 0, 1, 2])
    a, b = (x[..., 0:8:2], x[..., 1:8:2]) if interleaved else (x[..., :4], x[..., 4:8])
    z = 1.5 * (a + 1j * b) * np.exp(1j * pos[:, None] * f)[:, None]
    c, d = (y[..., 0:8:2], y[..., 1:8:2]) if interleaved else (y[..., :4], y[..., 4:8])
    np.testing.assert_allclose(c + 1j * d, z, atol=1e-12)
    assert (y[..., 8:] == x[..., 8:]).all()


@pytest.mark.parametrize("interleaved", [False, True])
def test_rotary_inverse_is_the_gradient(interleaved):
    """d<rotary(x), g>/dx by central differences, entry by entry."""
    rng = np.random.default_rng(3)
    x, g = rng.normal(size=(2, 3, 2, 8))
    f, args = np.array([0.7, 0.05]), ([0, 1, 3], [5, 100])
    got = oracle.rotary(g, *args, f, interleaved, factor=1.3, inverse=True)
    for at in np.ndindex(*x.shape):
        e = np.zeros_like(x)
        e[at] = 0.5
        diff = sum(s * (oracle.rotary(x + s * e, *args, f, interleaved, factor=1.3) * g).sum() for s in (1, -1))
        assert abs(diff - got[at]) < 1e-9


def test_frequencies():
    f, factor = packed.rotary_frequencies(8, 10000.0)
    np.testing.assert_allclose(f.numpy(), [1.0, 0.1, 0.01, 0.001], rtol=1e-7)
    assert factor == 1.0 and f.dtype == torch.float32 and f.shape == (4,)
    np.testing.assert_allclose(packed.rotary_frequencies(8, 1e4, "linear", 4.0)[0], f / 4, rtol=1e-7)
    by_base, one = packed.rotary_frequencies(8, 1e4, "base", 4.0)
    np.testing.assert_allclose(by_base[[0, -1]], [1.0, 0.001 / 4], rtol=1e-6)
    assert one == 1.0
    # over 2 pi 1000 positions the pairs turn 1000, 100, 10 and 1 times
    parts, factor = packed.rotary_frequencies(8, 1e4, "parts", 4.0, trained=6283, low=2, high=50)
    share = (6283 * 0.01 / (2 * math.pi) - 2) / 48
    np.testing.assert_allclose(parts, [1.0, 0.1, 0.01 * (share + (1 - share) / 4), 0.001 / 4], rtol=1e-6)
    assert factor == 1 + 0.1 * math.log(4)
    for bad in (dict(rot=7), dict(rot=0), dict(rot=8, base=0.0), dict(rot=8, stretch=0.5),
                dict(rot=8, scaling="other"), dict(rot=2, scaling="base"),
                dict(rot=8, scaling="parts"), dict(rot=8, scaling="parts", trained=9, low=3, high=3)):
        with pytest.raises(ValueError):
            packed.rotary_frequencies(**bad)
