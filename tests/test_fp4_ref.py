"""The numpy 4-bit reference itself, on the CPU: round trips and the e4m3 table against torch."""
import numpy as np
import torch

from tests import fp4_ref


def test_scale_table_is_e4m3():
    t = torch.arange(127, dtype=torch.uint8).view(torch.float8_e4m3fn).double().numpy()
    assert np.array_equal(t, fp4_ref.E4M3)


def test_values_survive_a_second_rounding():
    rng = np.random.default_rng(0)
    v = fp4_ref.values(*fp4_ref.quantize(rng.standard_normal((64, 512))))
    again = fp4_ref.values(*fp4_ref.quantize(v))
    # a group whose largest code is 6 keeps its scale and so all its codes
    six = np.abs(v.reshape(64, -1, 16)).max(-1) == np.repeat(6.0, 32) * fp4_ref.E4M3[fp4_ref.quantize(v)[1]]
    assert six.any()
    assert np.array_equal(v.reshape(64, -1, 16)[six], again.reshape(64, -1, 16)[six])


def test_error_bound():
    # the largest magnitude in a group is at most 6.4 steps of s (s is within 1/16 of max/6), so a value is off
    # by at most half the widest gap (1 of 4..6, times s) or by the saturation 0.4 s: s <= max/6 * 17/16
    rng = np.random.default_rng(1)
    x = rng.standard_normal((256, 512)) * rng.uniform(0.1, 10, (256, 1))
    top = np.abs(x.reshape(256, -1, 16)).max(-1, keepdims=True)
    err = np.abs(fp4_ref.values(*fp4_ref.quantize(x)) - x).reshape(256, -1, 16)
    assert np.all(err <= top / 6 * 17 / 16 * 1.0 + 1e-12)


def test_ties_zero_and_nan():
    row = np.zeros((1, 64))
    row[0, :16] = [6, 0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5, -0.25, -0.75, -5, 0, -0.0, 0.26, -0.2, np.nan]
    c, s = fp4_ref.quantize(row)
    assert fp4_ref.E4M3[s[0, 0]] == 1.0
    got = fp4_ref.values(c, s)[0, :16]
    assert got.tolist() == [6, 0, 1, 1, 2, 2, 4, 4, 0, -1, -4, 0, 0, 0.5, 0, 0]
    assert not np.signbit(got[[8, 12, 14]]).any()
    assert np.all(fp4_ref.values(c, s)[0, 16:] == 0)
