"""Pins of the int4 oracle to facts other than itself (CPU)."""

from fractions import Fraction

import numpy as np
import pytest

import oracle


def _cases(seed, n, group):
    rng = np.random.default_rng(seed)
    w = (rng.standard_normal((n, 2 * group)) * 0.02).astype(np.float32)
    w[0, :group] = 0.0                       # an all-zero group
    w[1, :group] = np.abs(w[1, :group])      # no negative weight
    w[2, :group] = -np.abs(w[2, :group])     # no positive weight
    w[3, :group] = 1e-42                     # subnormal
    w[4, :group] *= np.float32(1e37)
    return w


@pytest.mark.parametrize("zero_points", [False, True])
@pytest.mark.parametrize("scale_dtype", ["f32", "bf16"])
def test_codes_are_the_nearest_level_in_exact_arithmetic(zero_points, scale_dtype):
    group = 32
    w = _cases(1, 6, group)
    packed, s, z = oracle.ref_int4_pack(w, group, zero_points, scale_dtype)
    for n in range(w.shape[0]):
        for k in range(w.shape[1]):
            sc = Fraction(float(s[n, k // group]))
            zp = 8 if z is None else int(z[n, k // group])
            byte = int(packed[n, k // 2])
            code = byte >> 4 if k % 2 == 0 else byte & 15
            if sc == 0:
                assert code == zp
                continue
            err = [abs(Fraction(float(w[n, k])) - (c - zp) * sc) for c in range(16)]
            assert code == err.index(min(err))   # index: the lowest of equal ones


def test_ties_go_to_the_lower_code():
    w = np.zeros((1, 32), dtype=np.float32)
    w[0, 0] = 7.0                            # s = 1 exactly
    w[0, 1:6] = [0.5, -0.5, 1.5, -6.5, 6.5]
    packed, s, _ = oracle.ref_int4_pack(w, 32, False, "f32")
    assert s[0, 0] == 1.0
    v = oracle.ref_int4_unpack(packed, s)[0]
    assert v[:6].tolist() == [7.0, 0.0, -1.0, 1.0, -7.0, 6.0]


@pytest.mark.parametrize("zero_points", [False, True])
def test_whole_multiples_of_the_scale_come_back_exactly(zero_points):
    q = np.tile(np.arange(-7, 8, dtype=np.float32), 9)[:128].reshape(1, 128) * np.float32(0.25)
    packed, s, z = oracle.ref_int4_pack(q, 128, zero_points, "f32")
    if not zero_points:                      # s = 7 * 0.25 / 7: every weight is a level
        assert np.array_equal(oracle.ref_int4_unpack(packed, s, z), q.astype(np.float64))
    err = np.abs(oracle.ref_int4_unpack(packed, s, z) - q)
    assert err.max() <= 0.5 * float(s.max()) * (1 + 1e-6)


def test_linear_is_a_sum_over_exact_fractions():
    rng = np.random.default_rng(3)
    w = (rng.standard_normal((3, 64)) * 0.1).astype(np.float32)
    packed, s, z = oracle.ref_int4_pack(w, 32, True, "f32")
    x = rng.standard_normal((2, 64)).astype(np.float32)
    y = oracle.ref_int4_linear(x, packed, s, z, bias=np.array([1.0, -2.0, 0.5]))
    for m in range(2):
        for n in range(3):
            t = Fraction([1.0, -2.0, 0.5][n])
            for k in range(64):
                b = int(packed[n, k // 2])
                c = b >> 4 if k % 2 == 0 else b & 15
                t += Fraction(float(x[m, k])) * (c - int(z[n, k // 32])) * Fraction(float(s[n, k // 32]))
            assert abs(float(t) - y[m, n]) <= 1e-13
