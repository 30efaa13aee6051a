"""Attention with transformed scores in 64 bits (numpy), its error bound, and
paged caches whose unseen parts are poisoned."""
import numpy as np
import torch

from tests import serving_helpers as S

BLOCK = 16
STEP = {torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}      # half a step of a rounding


def visible(pos, length, window=0, prefix=0):
    """bool [n, L]: key t of the row at position pos."""
    t, pos = np.arange(length)[None], np.asarray(pos)[:, None]
    see = (t <= pos) | (t < prefix)
    return see & (np.abs(pos - t) < window) if window else see


def attend(q, k, v, scale, pos, cap=0.0, slopes=None, window=0, prefix=0, dtype=torch.bfloat16, weight_step=None):
    """q [n, Hq, D] at positions pos, k, v [L, Hkv, D] -> (out, bound) [n, Hq, D].

    The bound: the output's rounding; one of the weights (``weight_step``, of sums of p |v|, once in the product and once
    in the sum that divides it); and of the scores, an error d of which changes a weight by d and so the output by at
    most 2 d sums of p |v|: fp32 sums of D products (in the tf32 form each off by 2^-20 too), the cap's formula (2^-20 of
    the score, or 2^-22 of the cap where it bends), and the bias' product and difference in 32 bits."""
    n, hq, d = q.shape
    length, hkv, _ = k.shape
    out, bound = np.zeros((n, hq, d)), np.zeros((n, hq, d))
    if length == 0 or n == 0:
        return out, bound
    g = hq // hkv
    if weight_step is None:
        weight_step = 2.0 ** -8 if dtype == torch.bfloat16 else 2.0 ** -19
    see = visible(pos, length, window, prefix)
    dist = np.abs(np.asarray(pos)[:, None] - np.arange(length)[None])
    for h in range(hq):
        kh, vh = k[:, h // g], v[:, h // g]
        used = see.any(0)
        kh, vh = np.where(used[:, None], kh, 0.0), np.where(used[:, None], vh, 0.0)
        s = q[:, h] @ kh.T * scale
        err = np.abs(q[:, h]) @ np.abs(kh).T * abs(scale) * ((d + 8) * 2.0 ** -24 + (0 if dtype == torch.bfloat16 else 2.0 ** -19))
        if cap:
            s = cap * np.tanh(s / cap)
            err = err + np.abs(s) * 2.0 ** -19
        if slopes is not None:
            s = s - slopes[h] * dist
            err = err + np.abs(slopes[h]) * dist * 2.0 ** -22
        err = err + np.abs(s) * 2.0 ** -22
        s = np.where(see, s, -np.inf)
        p = np.exp(s - s.max(1, keepdims=True))
        p /= p.sum(1, keepdims=True)
        out[:, h] = p @ vh
        spread = p @ np.abs(vh)
        # (an error far down the row has no weight: it counts with p)
        drift = (p * err) @ np.abs(vh) + (p * err).sum(1, keepdims=True) * spread
        bound[:, h] = STEP[dtype] * np.abs(out[:, h]) + 2 * weight_step * spread + 1.05 * drift + length * 2.0 ** -24 * spread + 1e-30
    return out, bound


def paged(seed, lens, hkv, d, dtype, window=0, first_seen=None, gain=1.0):
    """Caches and tables for contexts of these lengths.  What a call must not read is poisoned: rows that nothing sees
    (before first_seen[s]; of a decode call with this window if that is None) are NaN or infinite, table entries of
    blocks before them out of range.  Returns (k_cache, v_cache, tables, k rows by sequence, v rows by sequence); the rows hold 0 where poisoned."""
    rng = np.random.default_rng(seed)
    tables, nb = S.layout(rng, lens)
    t = lambda x: torch.from_numpy(x).to(dtype)
    k = t(rng.standard_normal((nb, hkv, BLOCK, d)).astype(np.float32) * gain)
    v = t(rng.standard_normal((nb, hkv, BLOCK, d)).astype(np.float32))
    kr, vr = [], []
    dead = np.ones((nb, BLOCK), dtype=bool)
    for s, n in enumerate(lens):
        kr.append(S.gather(S.f64(k), tables[s], n, nb))
        vr.append(S.gather(S.f64(v), tables[s], n, nb))
        first = first_seen[s] if first_seen else max(0, n - window) if window else 0
        for i in range(first, n):
            dead[tables[s, i // BLOCK], i % BLOCK] = False
        kr[-1][:first] = vr[-1][:first] = 0.0
    poison = torch.tensor([float("nan"), float("inf"), -float("inf")])
    where = torch.from_numpy(dead)[:, None, :, None].expand_as(k)
    pick = torch.from_numpy(rng.integers(0, 3, size=k.shape))
    k, v = torch.where(where, poison[pick].to(dtype), k), torch.where(where, poison[pick.flip(0)].to(dtype), v)
    for s, n in enumerate(lens):
        first = first_seen[s] if first_seen else max(0, n - window) if window else 0
        tables[s, :first // BLOCK] = -5
    return k.cuda(), v.cuda(), torch.from_numpy(tables).cuda(), kr, vr


def alibi(hq):
    return (2.0 ** (-8.0 * np.arange(1, hq + 1) / hq)).astype(np.float32)
