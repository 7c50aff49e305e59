"""Pins for the oracle's 4-bit rows.

The format is tied to things other than the oracle's own formula: codes and
values worked out by hand, PyTorch's bfloat16 rounding, the error bound of a
step's half, exact zeros, and the layout of a word read back bit by bit.
Planted mistakes (a step rounded up to a power of two, a zero point left out
on read) must fail the bound.
"""

import numpy as np
import pytest
import torch

import oracle.ref as ref


def _bf16(x):
    return torch.as_tensor(x, dtype=torch.float32).to(torch.bfloat16).double().numpy()


def test_hand_values():
    # range -7 .. 8: step 1, zero point 7, every integer its own code
    x = np.arange(-7.0, 9.0)
    c, s, z = ref.q4_quantize(x)
    assert s == 1.0 and z == 7 and np.array_equal(c, np.arange(16))
    assert np.array_equal(ref.q4_values(c, s, z), x)
    # one sign only: the range starts at 0
    c, s, z = ref.q4_quantize(np.array([15.0, 30.0, 0.0, 8.0]))
    assert s == 2.0 and z == 0 and list(c) == [8, 15, 0, 4]  # 7.5 -> 8 (ties to even), 8 / 2 = 4
    c, s, z = ref.q4_quantize(np.array([-15.0, -30.0, 0.0, -5.0]))
    assert s == 2.0 and z == 15 and list(c) == [7, 0, 15, 13]  # -7.5 -> -8, -2.5 -> -2


def test_bf16_rounding_matches_the_library():
    rng = np.random.default_rng(0)
    x = (rng.standard_normal(20000) * 10.0 ** rng.integers(-30, 30, 20000)).astype(np.float32)
    x = np.concatenate([x, np.array([1.00390625, 1.01171875, 0.0, -0.0], dtype=np.float32)])
    assert np.array_equal(ref.bf16_round(x), torch.from_numpy(x).to(torch.bfloat16).double().numpy())


@pytest.mark.parametrize("spread", [0.0, 1.0, 20.0])
def test_error_is_half_a_step(spread):
    rng = np.random.default_rng(3)
    x = _bf16(rng.standard_normal((4000, 64)) + spread * rng.standard_normal((4000, 1)))
    c, s, z = ref.q4_quantize(x)
    assert c.min() >= 0 and c.max() <= 15 and z.min() >= 0 and z.max() <= 15
    err = np.abs(ref.q4_values(c, s, z) - x) / s[:, None]
    # half a step; at the upper end, where the step was rounded down (by half a
    # unit in bf16's last place, 2^-8, at most), the range is up to
    # 15 / (1 - 2^-8) steps long and the code stops at 15: with -lo / s = z - 1/2
    # the end lies 15 / (1 - 2^-8) - 15 + 1/2 steps past it.  (1e-5: the float32
    # product, 16 * 2^-24 steps, and this division.)
    assert err.max() <= 0.5 + 15 / (1 - 2.0 ** -8) - 15 + 1e-5
    # planted: a zero point left out on read is off by whole steps
    assert (np.abs(s[:, None] * c - x) / s[:, None]).max() > 1.0


def test_zero_is_exact_and_rows_of_zeros():
    rng = np.random.default_rng(5)
    x = _bf16(rng.standard_normal((500, 32)) * 3)
    x[:, 7] = 0.0
    assert np.all(ref.q4_store(x)[:, 7] == 0.0)
    c, s, z = ref.q4_quantize(np.zeros((2, 32)))
    assert np.all(c == 0) and np.all(s == 0) and np.all(z == 0)
    tiny = np.full((1, 32), 2.0 ** -130)
    assert np.all(ref.q4_store(tiny) == 0.0)


def test_rows_that_are_not_finite():
    for bad in (np.nan, np.inf, -np.inf):
        x = np.ones((1, 32))
        x[0, 3] = bad
        assert np.all(np.isnan(ref.q4_store(x)))
    big = np.zeros((1, 32))
    big[0, 0], big[0, 1] = 3.0e38, -3.0e38  # the range passes float32
    assert np.all(np.isnan(ref.q4_store(_bf16(big))))


def test_word_layout():
    c = np.arange(8)
    assert ref.q4_pack(c)[0] == 0x75316420
    w = ref.q4_scale_words(np.array([1.0]), np.array([9]))
    assert w[0] == 0x3F800009
    assert ref.q4_scale_words(np.array([np.nan]), np.array([0]))[0] == 0x7FC00000
