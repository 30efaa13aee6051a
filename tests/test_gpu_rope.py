"""The pass from the projections to the cache against a 64-bit form: norm,
rotation on one or several axes, query output, cache writes."""
import numpy as np
import pytest
import torch

from tests import serving_helpers as S

pytestmark = pytest.mark.gpu

# An fp32 result before its rounding is off by at most 20 u (|a| + |b|), u = 2^-24, (a, b) the pair it came from:
# the norm's sum of squares (12 additions, halved by the root), root, division and two products 10.5 u, sine and
# cosine 2 u, the fp32 angle 3.1 u (half a turn's rounding), the rotation's products and sum 2 u.
ARITH = 20 * 2.0 ** -24
ROUND = {torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}


def reference(x, w, eps, pos, freq, axes, interleaved):
    """x [T, H, D] in 64 bits -> (result, |a| + |b| of each element's pair)."""
    t, _, d = x.shape
    if w is not None:
        x = x / np.sqrt((x * x).mean(-1, keepdims=True) + eps) * w
    half = 0 if freq is None else len(freq)
    out, mag = x.copy(), np.abs(x)
    if half:
        i = np.arange(half)
        ia, ib = (2 * i, 2 * i + 1) if interleaved else (i, i + half)
        # whole turns removed exactly: extended precision holds position times frequency
        ang = np.longdouble(pos[axes].T) * np.longdouble(freq)[None]                 # [T, half]
        ang = np.remainder(ang, 2 * np.longdouble("3.14159265358979323846264338327950288")).astype(np.float64)
        c, s = np.cos(ang)[:, None], np.sin(ang)[:, None]
        a, b = x[..., ia], x[..., ib]
        out[..., ia], out[..., ib] = a * c - b * s, b * c + a * s
        mag[..., ia] = mag[..., ib] = np.abs(a) + np.abs(b)
    return out, mag


def run(t, hq, hkv, d, dtype, rot, axes_n=1, interleaved=False, norm=True, e4m3=False, fused=True, pos_hi=5000, seed=0,
        in_place=False):
    b = S.lib()
    rng = np.random.default_rng(seed + t + hq + d + rot)
    nb = -(-t // 16) + 2
    total = hq + 2 * hkv
    qkv = torch.from_numpy(rng.standard_normal((t, total + (1 if fused else 0), d)).astype(np.float32)).to(dtype).cuda()
    q, k, v = qkv[:, :hq], qkv[:, hq:hq + hkv], qkv[:, hq + hkv:total]
    if not fused:
        q, k, v = q.contiguous(), k.contiguous(), v.contiguous()
    q0, k0, v0 = S.f64(q), S.f64(k), S.f64(v)
    wq, wk = (torch.from_numpy((1 + 0.2 * rng.standard_normal(d)).astype(np.float32)).to(dtype).cuda() for _ in range(2))
    half = rot // 2
    freq = torch.from_numpy((1e4 ** (-np.arange(half) / max(1, half))).astype(np.float32)).cuda() if rot else None
    pos = rng.integers(0, pos_hi, size=(axes_n, t))
    pos[:, 0] = 0
    axes = rng.integers(0, axes_n, size=half).astype(np.int32)
    slots = rng.permutation(nb * 16)[:t]
    if t > 3:
        slots[1] = -5
    q_out = q if in_place else torch.full((t, hq, d), float("nan"), dtype=dtype, device="cuda")
    if e4m3:
        kc, vc = b.e4m3_cache(nb, hkv, d), b.e4m3_cache(nb, hkv, d)
    else:
        kc = torch.full((nb, hkv, 16, d), 3.0, dtype=dtype, device="cuda")
        vc = kc.clone()
    b.qk_norm_rope_append(q_out, q, k, v, torch.from_numpy(pos if axes_n > 1 else pos[0]).cuda() if rot else None, freq,
                          torch.from_numpy(slots).cuda(), kc, vc, q_weight=wq if norm else None,
                          k_weight=wk if norm else None, eps=1e-5,
                          axes=torch.from_numpy(axes).cuda() if rot and axes_n > 1 else None, interleaved=interleaved)
    assert b.device_error() == 0
    eps = float(np.float32(1e-5))
    fr = S.f64(freq) if rot else None
    if axes_n == 1:
        axes[:] = 0
    want_q, mag_q = reference(q0, S.f64(wq) if norm else None, eps, pos, fr, axes, interleaved)
    want_k, mag_k = reference(k0, S.f64(wk) if norm else None, eps, pos, fr, axes, interleaved)
    # a norm's or rotation's arithmetic moves a value by ARITH of its pair; untouched rows not at all
    S.close(q_out, want_q, ROUND[dtype] * (np.abs(want_q) + ARITH * mag_q) + ARITH * mag_q, "q")
    live = slots >= 0
    at = (slots[live] // 16, slice(None), slots[live] % 16)
    rest = np.ones((nb, 16), bool)
    rest[slots[live] // 16, slots[live] % 16] = False
    if not e4m3:
        S.close(S.f64(kc)[at], want_k[live], (ROUND[dtype] * (np.abs(want_k) + ARITH * mag_k) + ARITH * mag_k)[live], "k")
        assert np.array_equal(S.f64(vc)[at], v0[live])
        for c in (kc, vc):
            assert np.all(S.f64(c).transpose(0, 2, 1, 3)[rest] == 3.0)
        return
    codes, scales = S.tile_parts(vc)
    vcodes, vscales = S.e4m3_rows(v0)
    assert S.same_codes(codes[at], vcodes[live]) and np.array_equal(scales[at], vscales[live])
    codes, scales = S.tile_parts(kc)
    got, e = S.tile_values(kc)[at], scales[at].astype(np.int64) - 127
    top = np.abs(want_k[live]).max(-1)
    slack = ARITH * mag_k[live].max(-1)
    assert np.all(top - slack <= 448 * 2.0 ** e) and np.all(top + slack > 448 * 2.0 ** (e - 1))
    # half a step of e4m3: 2^-4 of the value, or 2^-10 of the scale below its normal range
    step = np.maximum(2.0 ** -4 * (np.abs(want_k) + ARITH * mag_k)[live], 2.0 ** -10 * 2.0 ** e[..., None])
    S.close(got, want_k[live], step + ARITH * mag_k[live], "k in e4m3")
    assert not codes.transpose(0, 2, 1, 3)[rest].any() and not scales.transpose(0, 2, 1)[rest].any()


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("d,rot", [(64, 64), (64, 16), (64, 48), (128, 128), (128, 64), (128, 112), (128, 0)])
@pytest.mark.parametrize("t,hq,hkv", [(1, 1, 1), (7, 4, 2), (33, 15, 5), (18, 40, 40)])
def test_norm_and_rotation(t, hq, hkv, d, rot, dtype, interleaved):
    run(t, hq, hkv, d, dtype, rot, interleaved=interleaved)


@pytest.mark.parametrize("axes_n", [1, 2, 3, 4])
@pytest.mark.parametrize("norm", [False, True])
@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("d", [64, 128])
def test_axes_norms_and_caches(axes_n, norm, e4m3, dtype, d):
    run(21, 8, 3, d, dtype, d, axes_n=axes_n, norm=norm, e4m3=e4m3, seed=axes_n, interleaved=axes_n == 2)


def test_far_positions():
    """The angle of position 2^31 is as good as that of position 1."""
    run(40, 4, 2, 128, torch.float32, 128, pos_hi=2 ** 31, seed=3)
    run(40, 4, 2, 64, torch.float32, 64, pos_hi=2 ** 31, interleaved=True, seed=4)


def test_contiguous_inputs_and_in_place_queries():
    run(50, 12, 4, 128, torch.bfloat16, 128, fused=False)
    run(50, 12, 4, 128, torch.bfloat16, 128, fused=False, in_place=True)
    run(50, 12, 4, 64, torch.float32, 32, fused=False, in_place=True, interleaved=True)


def test_many_tokens():
    run(5000, 3, 1, 128, torch.bfloat16, 128, pos_hi=131072)


def test_zero_rows_stay_zero():
    b = S.lib()
    q = torch.zeros(2, 2, 64, dtype=torch.bfloat16, device="cuda")
    w = torch.ones(64, dtype=torch.bfloat16, device="cuda")
    out, kc = torch.full_like(q, 5.0), torch.full((1, 2, 16, 64), 5.0, dtype=torch.bfloat16, device="cuda")
    vc = kc.clone()
    b.qk_norm_rope_append(out, q, q, q, torch.tensor([3, 4], device="cuda"), torch.ones(32, device="cuda"),
                          torch.tensor([0, 5], device="cuda"), kc, vc, q_weight=w, k_weight=w)
    assert not out.any() and not kc[0, :, [0, 5]].any() and bool((kc[0, :, 1] == 5).all())


def test_bad_slots_and_axes_are_flagged():
    b = S.lib()
    x = torch.randn(3, 2, 64, device="cuda")
    out, kc, vc = torch.zeros_like(x), torch.zeros(1, 2, 16, 64, device="cuda"), torch.zeros(1, 2, 16, 64, device="cuda")
    freq = torch.ones(16, device="cuda")
    axes = torch.zeros(16, dtype=torch.int32, device="cuda")
    pos = torch.tensor([[1, 2, 3]], device="cuda")
    b.qk_norm_rope_append(out, x, x, x, pos, freq, torch.tensor([0, 16, 1], device="cuda"), kc, vc, axes=axes)
    assert b.device_error() == b.DEVERR_SLOT
    assert bool(vc[0, :, 0].any()) and not vc[0, :, 2:].any() and bool(out[1].any())
    axes[3] = 1
    b.qk_norm_rope_append(out, x, x, x, pos, freq, torch.tensor([0, 2, 1], device="cuda"), kc, vc, axes=axes)
    assert b.device_error() == b.DEVERR_INDEX
    assert torch.equal(out[:, :, [3, 19]], x[:, :, [3, 19]]) and not torch.equal(out[:, :, 2], x[:, :, 2])


def test_replayed_from_a_graph_on_another_stream():
    b = S.lib()
    x = torch.randn(9, 4, 128, device="cuda").bfloat16()
    w = torch.ones(128, device="cuda").bfloat16()
    pos, freq = torch.arange(9, device="cuda"), torch.rand(64, device="cuda")
    slots = torch.arange(9, device="cuda")

    def call(out, kc, vc, stream=None):
        b.qk_norm_rope_append(out, x, x, x, pos, freq, slots, kc, vc, q_weight=w, k_weight=w, stream=stream)

    mk = lambda: (torch.zeros_like(x), torch.zeros(1, 4, 16, 128, dtype=x.dtype, device="cuda"),  # noqa: E731
                  torch.zeros(1, 4, 16, 128, dtype=x.dtype, device="cuda"))
    one, two, side = mk(), mk(), torch.cuda.Stream()
    torch.cuda.synchronize()
    call(*one, stream=side)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        call(*two)
    g.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(p, q) for p, q in zip(one, two))
    x.mul_(2)
    pos.add_(1)
    g.replay()
    call(*one)
    torch.cuda.synchronize()
    assert all(torch.equal(p, q) for p, q in zip(one, two))
