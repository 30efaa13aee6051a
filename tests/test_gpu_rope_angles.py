"""The angles of the pass from the projections to the cache: small ones to the
accuracy of fp32, at positions of either sign."""
import numpy as np
import pytest
import torch

from tests import serving_helpers as S

pytestmark = pytest.mark.gpu


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
