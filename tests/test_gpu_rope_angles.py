"""The angles of the pass from the projections to the cache: small ones to the
accuracy of fp32, far and negative positions, and frequencies on both sides of
16, where their reduction changes form."""
import numpy as np
import pytest
import torch

from tests import serving_helpers as S
from tests.test_gpu_rope import ARITH

pytestmark = pytest.mark.gpu

PI_200 = 0x3243f6a8885a308d313198a2e03707344a4093822299f31d008   # pi 2^200, rounded down


def turned(q, pos, freq, interleaved=False, **kw):
    """q [T, H, D] fp32 after the rotation alone."""
    b = S.lib()
    t, h, d = q.shape
    kc = torch.zeros(-(-t // 16), 1, 16, d, device="cuda")
    kv = torch.zeros(t, 1, d, device="cuda")
    out = torch.empty_like(q)
    b.qk_norm_rope_append(out, q, kv, kv, torch.from_numpy(np.asarray(pos, dtype=np.int64)).cuda(),
                          torch.from_numpy(np.asarray(freq, dtype=np.float32)).cuda(), torch.arange(t, device="cuda"), kc,
                          kc.clone(), interleaved=interleaved, **kw)
    assert b.device_error() == 0
    return S.f64(out)


@pytest.mark.parametrize("interleaved", [False, True])
def test_small_angles_keep_their_bits(interleaved):
    """(a, b) = (0, 1) turns to (-sin, cos): the sine of an angle of 1e-6 is as good as any other's. The reduced angle
    r, at most half a turn of either sign, is rounded once, to fp32: off by 2^-24 |r|, which moves the sine by that
    much at most (as much as |sine| 2^-24 where r is small, more near half a turn). The sine itself and the products
    behind it cost 5 roundings of 2^-24 of it, the integer fraction |pos| 2^-64 of a turn."""
    d, half = 64, 32
    pos = np.array([1, -1, 2, 3, 1000, -77, 123456])
    freq = np.float32(10.0) ** -np.linspace(0.5, 9.5, half).astype(np.float32)
    q = torch.zeros(len(pos), 1, d, device="cuda")
    q[..., 1::2] = 1.0 if interleaved else q[..., 1::2]
    if not interleaved:
        q[..., half:] = 1.0
    got = turned(q, pos, freq, interleaved)
    got = got[:, 0, 0::2] if interleaved else got[:, 0, :half]
    angle = np.longdouble(pos)[:, None] * np.longdouble(freq.astype(np.float64))
    want = -np.sin(angle).astype(np.float64)
    fraction = np.abs(pos)[:, None] * 2.0 ** -64 * 2 * np.pi
    turn = 2 * np.longdouble("3.14159265358979323846264338327950288")
    reduced = np.abs(angle - np.rint(angle / turn) * turn).astype(np.float64)
    assert np.all(np.abs(got - want) <= 2.0 ** -24 * (reduced + 5 * np.abs(want)) + fraction)


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("lo,hi", [(-2 ** 31, 2 ** 31), (-5000, 0), (0, 40)])
def test_high_frequencies_and_negative_positions(lo, hi, interleaved):
    """Frequencies on both sides of 16, up to 2^39, at positions of either sign. Exact angles from whole numbers: a
    frequency is m 2^-e, so position times frequency is a fraction of integers, reduced by 2 pi to 200 bits."""
    rng = np.random.default_rng(hi % 1000)
    d, half, t = 128, 64, 9
    pos = rng.integers(lo, hi, size=t)
    freq = (2.0 ** rng.uniform(-3, 39, size=half)).astype(np.float32) * np.where(np.arange(half) % 5 == 4, -1, 1).astype(np.float32)
    freq[:4] = [16.0, 15.999999, 17.5, 1024.0]
    x = rng.standard_normal((t, 2, d)).astype(np.float32)
    got = turned(torch.from_numpy(x).cuda(), pos, freq, interleaved)
    angle = np.zeros((t, half))
    for i in range(t):
        for j in range(half):
            num, den = float(freq[j]).as_integer_ratio()
            angle[i, j] = (int(pos[i]) * num << 200) // den % (2 * PI_200) / 2 ** 200
    i = np.arange(half)
    ia, ib = (2 * i, 2 * i + 1) if interleaved else (i, i + half)
    a, b = x[..., ia].astype(np.float64), x[..., ib].astype(np.float64)
    c, s = np.cos(angle)[:, None], np.sin(angle)[:, None]
    want, mag = np.zeros(x.shape), np.zeros(x.shape)
    want[..., ia], want[..., ib] = a * c - b * s, b * c + a * s
    mag[..., ia] = mag[..., ib] = np.abs(a) + np.abs(b)
    S.close(got, want, 2.0 ** -24 * np.abs(want) + ARITH * mag)


def test_frequencies_that_are_not_finite_give_nan():
    x = torch.ones(2, 1, 64, device="cuda")
    freq = np.array([np.inf, np.nan, -np.inf] + [1.0] * 29)
    got = turned(x, [0, 5], freq)
    assert np.isnan(got[:, 0, [0, 1, 2, 32, 33, 34]]).all() and np.isfinite(got[:, 0, 3:32]).all()
