"""The oracle of the 8-bit cache against definitions it does not share: torch's own e4m3
conversion, brute force over all codes, hand-worked blocks and invariants."""
import numpy as np
import pytest
import torch

from oracle import cache_q8 as oc


def test_e4m3_numbers_are_torchs():
    codes = torch.arange(127, dtype=torch.uint8).view(torch.float8_e4m3fn).double().numpy()
    assert np.array_equal(oc.numbers("e4m3"), codes)


def test_e4m3_nearest_is_torchs_rounding():
    g = torch.Generator().manual_seed(1)
    y = torch.cat([torch.randn(20000, generator=g) * 2.0 ** torch.randint(-12, 8, (20000,), generator=g),
                   torch.tensor([0.0, 448.0, -448.0, 2.0 ** -9, 2.0 ** -10, 3 * 2.0 ** -10, 0.5 + 1 / 32, 17.0, 19.0])])
    y = y.clamp(-448, 448)
    want = y.to(torch.float8_e4m3fn).double().numpy()
    assert np.array_equal(oc.nearest(y.double().numpy(), "e4m3"), want)


@pytest.mark.parametrize("fmt", ["e4m3", "int8"])
def test_nearest_by_brute_force(fmt):
    t = oc.numbers(fmt)
    y = np.random.default_rng(2).uniform(-1.1 * t[-1], 1.1 * t[-1], 500)
    got = oc.nearest(y, fmt)
    allv = np.concatenate([-t, t])
    for a, b in zip(y, got):
        assert abs(b) in t and abs(a - b) == np.abs(allv - a).min()


def test_int8_ties_go_to_even():
    assert oc.nearest(np.array([0.5, 1.5, 2.5, -0.5, -1.5, 126.5]), "int8").tolist() == [0, 2, 2, -0.0, -2, 126]


@pytest.mark.parametrize("fmt,qmax", [("e4m3", 448.0), ("int8", 127.0)])
def test_block_scale_is_the_smallest_power_that_fits(fmt, qmax):
    for amax in [qmax, qmax * (1 + 2 ** -20), qmax / 2, 1.0, 3.1e38, 1e-20, 0.99, 2.0 ** -93]:
        s = oc.block_scale(amax, fmt)
        assert np.log2(s) == int(np.log2(s)) and amax <= qmax * s
        assert s == 2.0 ** -100 or amax > qmax * s / 2
    assert oc.block_scale(0.0, fmt) == oc.block_scale(1e-45, fmt) == 2.0 ** -100


def test_a_block_by_hand():
    # int8, block 16: rows 1.0, then 127 (scale stays 1), then 128 (scale 2: older rows halve)
    codes, scale = np.zeros((32, 1, 1)), np.zeros((2, 1))
    oc.write(codes, scale, np.array([[[1.0]]]), 0, 16, "int8")
    assert scale[0, 0] == 2.0 ** -6 and codes[0, 0, 0] == 64                  # 1.0 = 64 / 64
    oc.write(codes, scale, np.array([[[127.0]]]), 1, 16, "int8")
    assert scale[0, 0] == 1.0 and codes[:2, 0, 0].tolist() == [1, 127]
    oc.write(codes, scale, np.array([[[128.0]]]), 2, 16, "int8")
    assert scale[0, 0] == 2.0 and codes[:3, 0, 0].tolist() == [0, 64, 64]     # 0.5 and 63.5 tie to even
    oc.write(codes, scale, np.array([[[3.0]]]), 3, 16, "int8")
    assert scale[0, 0] == 2.0 and codes[3, 0, 0] == 2                         # 1.5 ties to even
    assert scale[1, 0] == 0.0 and not codes[4:].any()


@pytest.mark.parametrize("fmt", ["e4m3", "int8"])
def test_one_write_equals_block_by_block_and_errors_stay_in_a_step(fmt):
    rng = np.random.default_rng(3)
    x = rng.normal(size=(50, 2, 8)) * np.exp(rng.normal(size=(50, 2, 1)))
    a, b = [(np.zeros((64, 2, 8)), np.zeros((4, 2))) for _ in range(2)]
    oc.write(*a, x, 0, 16, fmt)
    for r in range(0, 50, 16):
        oc.write(*b, x[r:r + 16], r, 16, fmt)
    assert np.array_equal(a[0], b[0]) and np.array_equal(a[1], b[1])
    got = oc.read(*a, range(50), 16)
    s = np.repeat(a[1], 16, axis=0)[:50, :, None]
    step = s / 2 if fmt == "int8" else np.maximum(np.abs(x) * 2.0 ** -4, s * 2.0 ** -10)
    assert (np.abs(got - x) <= step * (1 + 1e-12)).all()


def test_growing_scale_is_exact_for_e4m3_normals():
    codes, scale = np.zeros((16, 1, 4)), np.zeros((1, 1))
    oc.write(codes, scale, np.array([[[100.0, 50.0, 3.0, 1.75]]]), 0, 16, "e4m3")
    before = oc.read(codes, scale, [0], 16)
    oc.write(codes, scale, np.full((1, 1, 4), 900.0), 1, 16, "e4m3")
    assert scale[0, 0] == 4.0 and np.array_equal(oc.read(codes, scale, [0], 16), before)


def test_read_outside_the_cache_is_zero():
    codes, scale = np.ones((16, 1, 2)), np.full((1, 1), 3.0)
    assert oc.read(codes, scale, [-1, 0, 16, 15], 16)[:, 0, 0].tolist() == [0, 3, 0, 3]
