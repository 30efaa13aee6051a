"""Plain 64-bit forms of the serving calls (numpy), and small inputs for
their tests: e4m3 rows and tiles, attention over a paged cache with any mask,
shuffled block tables."""
import numpy as np
import torch

BLOCK = 16


def lib():
    from paged_kv_cache_177_gb300 import build
    build.build_library()
    from paged_kv_cache_177_gb300 import binding
    return binding


def bf16(x):
    """A bf16 CPU tensor from a numpy array."""
    return torch.from_numpy(np.asarray(x, dtype=np.float32)).to(torch.bfloat16)


def f64(t):
    return t.detach().double().cpu().numpy()


# ---- e4m3 -----------------------------------------------------------------------
def e4m3_values():
    """The value of every code 0..255 (NaN for 0x7f and 0xff)."""
    v = np.empty(256)
    for c in range(128):
        e, m = c >> 3, c & 7
        v[c] = m * 2.0 ** -9 if e == 0 else (8 + m) * 2.0 ** (e - 10)
    v[127] = np.nan
    v[128:] = -v[:128]
    return v


VALUES = e4m3_values()


def e4m3_rows(x):
    """(codes uint8, scale bytes uint8) of rows x [..., D]: the least e in
    [-50, 50] with max|x| 2^-e <= 448 over the finite elements, codes to
    nearest, ties to even, past 448 saturated, non-finite elements NaN."""
    x = np.asarray(x, dtype=np.float64)
    fin = np.isfinite(x)
    top = np.where(fin, np.abs(x), 0.0).max(-1)
    e = np.full(top.shape, 50, dtype=np.int64)
    for k in range(50, -51, -1):
        e = np.where(top <= 448 * 2.0 ** k, k, e)
    e = np.where(top == 0, 0, e)
    y = np.minimum(np.where(fin, np.abs(x), 0.0) * 2.0 ** (-e[..., None].astype(np.float64)), 448.0)
    table = VALUES[:127]
    mid = (table[1:] + table[:-1]) / 2
    lo, hi = np.searchsorted(mid, y, "left"), np.searchsorted(mid, y, "right")
    code = np.where(lo % 2 == 0, lo, hi).astype(np.uint8)
    code = np.where(np.signbit(x), code | 128, code).astype(np.uint8)
    return np.where(fin, code, np.uint8(127)), (e + 127).astype(np.uint8)


def same_codes(got, want):
    """Equal codes, NaN of either sign alike."""
    return np.array_equal(np.where((got & 127) == 127, 127, got), np.where((want & 127) == 127, 127, want))


def tile_parts(cache):
    """uint8 tiles [NB, Hkv, 16 (D + 1)] -> codes [NB, Hkv, 16, D], scales [NB, Hkv, 16]."""
    c = cache.cpu().numpy() if isinstance(cache, torch.Tensor) else cache
    d = c.shape[2] // BLOCK - 1
    return c[:, :, :BLOCK * d].reshape(*c.shape[:2], BLOCK, d), c[:, :, BLOCK * d:]


def tile_values(cache):
    codes, scales = tile_parts(cache)
    return VALUES[codes] * np.where(scales == 0, 0.0, 2.0 ** (scales.astype(np.float64) - 127))[..., None]


def make_tiles(x):
    """Tiles of an array [NB, Hkv, 16, D] of rows."""
    codes, scales = e4m3_rows(x)
    return torch.from_numpy(np.concatenate([codes.reshape(*codes.shape[:2], -1), scales], -1).copy())


# ---- paged caches ------------------------------------------------------------------
def layout(rng, lens, spare=3):
    """Shuffled tables int32 [S, maxB] (entries past a sequence's blocks out of
    range, so that reading one shows) and the pool's blocks."""
    need = [-(-n // BLOCK) for n in lens]
    nb = sum(need) + spare
    perm = rng.permutation(nb)
    tables = np.full((len(lens), max(1, max(need, default=1))), 1 << 30, dtype=np.int32)
    at = 0
    for s, k in enumerate(need):
        tables[s, :k] = perm[at:at + k]
        at += k
    return tables, nb


def live_slots(tables, lens, nb):
    """bool [NB, 16]: slots that belong to some sequence's context."""
    live = np.zeros((nb, BLOCK), dtype=bool)
    for s, n in enumerate(lens):
        for t in range(n):
            live[tables[s, t // BLOCK], t % BLOCK] = True
    return live


def gather(cache, table, n, nb):
    """Rows 0..n-1 of one sequence from [NB, Hkv, 16, D] (numpy): [n, Hkv, D]; bad blocks read as zeros."""
    t = np.arange(n)
    blk = table[t // BLOCK]
    ok = (blk >= 0) & (blk < nb)
    rows = cache[np.where(ok, blk, 0), :, t % BLOCK]
    return np.where(ok[:, None, None], rows, 0.0)


def attend(q, k, v, scale, see=None):
    """q [n, Hq, D], k, v [L, Hkv, D], see [n, L] -> (out [n, Hq, D], sum of p |v|), zeros where nothing is seen."""
    n, hq, d = q.shape
    length, hkv, _ = k.shape
    out, spread = np.zeros((n, hq, d)), np.zeros((n, hq, d))
    if length == 0:
        return out, spread
    g = hq // hkv
    for h in range(hq):
        s = q[:, h] @ k[:, h // g].T * scale
        if see is not None:
            s = np.where(see, s, -np.inf)
        top = s.max(1, keepdims=True)
        p = np.exp(s - np.where(np.isfinite(top), top, 0.0))
        total = p.sum(1, keepdims=True)
        p = p / np.where(total > 0, total, 1.0)
        # a value that nobody weighs may be anything
        vv = v[:, h // g]
        out[:, h] = np.where(p[:, :, None] > 0, p[:, :, None] * vv[None], 0.0).sum(1)
        spread[:, h] = np.where(p[:, :, None] > 0, p[:, :, None] * np.abs(vv)[None], 0.0).sum(1)
    return out, spread


def close(got, want, bound, what=""):
    got = got if isinstance(got, np.ndarray) else f64(got)
    assert np.all(np.isfinite(got)), f"{what}: non-finite output"
    err = np.abs(got - want)
    worst = np.unravel_index(np.argmax(err - bound), err.shape) if err.size else None
    assert np.all(err <= bound), f"{what}: {err[worst]:.3e} off at {worst}, bound {bound[worst]:.3e}"
