"""The 8-bit cache on the GPU: codes and scales byte for byte against the
definition, blocks read back exactly, whole-block moves, and decode attention
against a 64-bit softmax over the values the tiles stand for."""
import numpy as np
import pytest
import torch

from tests import serving_helpers as S

pytestmark = pytest.mark.gpu

# Bound of a decode output: its rounding (bf16 2^-8 of the value, fp32 2^-24) plus sum p |v| times
#   2^-11  the weights' rounding to f16 for the tensor cores,
#   2^-12  the scores: 128 terms accumulated in fp32, 128 * 2^-24 * sum |q k| scale, with sum |q k| scale
#          below 32 for these inputs, moves a weight by at most that share.
WEIGHTS = 2.0 ** -11 + 2.0 ** -12
ROUND = {torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}


def special_rows(rng, n, d):
    """Rows that a quantiser can get wrong: zeros, one element, exact powers, the border 448 * 2^k, denormals,
    far magnitudes, infinities and NaN, then ordinary ones."""
    x = rng.standard_normal((n, d)) * 2.0 ** rng.integers(-6, 7, size=(n, 1))
    fixed = [np.zeros(d), np.eye(1, d, 3)[0] * -5.0, np.full(d, 448.0), np.full(d, 448.0 * 2 ** 7),
             np.linspace(-450, 450, d), np.full(d, 1e-41), np.full(d, 3e38), np.linspace(-1e-20, 1e-20, d),
             np.where(np.arange(d) == 1, np.inf, 2.0), np.where(np.arange(d) == 2, np.nan, np.arange(d) - 9.0),
             np.full(d, -np.inf), np.linspace(0, 2 ** -9, d), 2.0 ** -np.arange(d).clip(0, 40)]
    for i, r in enumerate(fixed[:n]):
        x[i] = r
    return x


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("tokens,hkv", [(1, 1), (5, 3), (37, 8), (130, 5)])
def test_append_writes_the_defined_bytes(tokens, hkv, d, dtype):
    b = S.lib()
    rng = np.random.default_rng(tokens * 100 + hkv + d)
    nb = -(-tokens // 16) + 3
    k = torch.from_numpy(special_rows(rng, tokens * hkv, d).reshape(tokens, hkv, d)).float().to(dtype).cuda()
    v = torch.from_numpy(special_rows(rng, tokens * hkv, d)[::-1].copy().reshape(tokens, hkv, d)).float().to(dtype).cuda()
    slots = rng.permutation(nb * 16)[:tokens]
    if tokens > 4:
        slots[2] = -1
    before = torch.from_numpy(rng.integers(0, 256, size=(nb, hkv, 16 * (d + 1)), dtype=np.uint8)).cuda()
    kc, vc = before.clone(), before.clone()
    b.kv_append_e4m3(k, v, torch.from_numpy(slots).cuda(), kc, vc)
    assert b.device_error() == 0
    for rows, cache in ((k, kc), (v, vc)):
        codes, scales = S.e4m3_rows(S.f64(rows))
        want_c, want_s = (a.copy() for a in S.tile_parts(before))
        for t, slot in enumerate(slots):
            if slot >= 0:
                want_c[slot // 16, :, slot % 16] = codes[t]
                want_s[slot // 16, :, slot % 16] = scales[t]
        got_c, got_s = S.tile_parts(cache)
        written = np.zeros((nb, 16), bool)
        for slot in slots[slots >= 0]:
            written[slot // 16, slot % 16] = True
        written = np.broadcast_to(written[:, None, :, None], got_c.shape)
        assert S.same_codes(got_c[written], want_c[written])
        assert np.array_equal(got_c[~written], want_c[~written])
        assert np.array_equal(got_s, want_s)


def test_append_from_pinned_memory_and_bad_slots():
    b = S.lib()
    rng = np.random.default_rng(5)
    k = S.bf16(rng.standard_normal((3, 2, 64))).pin_memory()
    slots = torch.tensor([7, 99999, 20]).pin_memory()
    kc, vc = b.e4m3_cache(2, 2, 64), b.e4m3_cache(2, 2, 64)
    b.kv_append_e4m3(k, k, slots, kc, vc)
    torch.cuda.synchronize()
    assert b.device_error() == b.DEVERR_SLOT
    codes, scales = S.e4m3_rows(S.f64(k))
    got, gs = S.tile_parts(vc)
    assert np.array_equal(got[0, :, 7], codes[0]) and np.array_equal(got[1, :, 4], codes[2])
    assert np.array_equal(gs[0, :, 7], scales[0]) and int((kc != 0).sum()) == int((vc != 0).sum())


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("hkv", [1, 5])
def test_blocks_read_back_exactly(d, dtype, hkv):
    b = S.lib()
    rng = np.random.default_rng(d + hkv)
    nb = 9
    tiles = rng.integers(0, 256, size=(nb, hkv, 16 * (d + 1)), dtype=np.uint8)
    tiles[:, :, 16 * d:] = rng.integers(77, 178, size=(nb, hkv, 16))          # a quantiser's scales
    tiles[0, 0, 16 * d:] = 0                                                  # a fresh cache's
    kc, vc = torch.from_numpy(tiles).cuda(), torch.from_numpy(tiles[::-1].copy()).cuda()
    pairs = np.array([[0, 3], [8, 0], [4, 5], [0, 1]])
    out = [torch.full((6, hkv, 16, d), 7.0, dtype=dtype, device="cuda") for _ in range(2)]
    b.dequantize_blocks(*out, kc, vc, torch.from_numpy(pairs).cuda())
    assert b.device_error() == 0
    for got, cache in zip(out, (kc, vc)):
        want = np.full((6, hkv, 16, d), 7.0)
        for s, t in pairs:
            want[t] = S.tile_values(cache)[s]
        assert np.array_equal(S.f64(got), want, equal_nan=True)


def test_read_back_flags_pairs_out_of_range():
    b = S.lib()
    kc = b.e4m3_cache(3, 2, 64)
    out = [torch.full((2, 2, 16, 64), 7.0, device="cuda") for _ in range(2)]
    b.dequantize_blocks(*out, kc, kc, torch.tensor([[3, 0], [0, 2], [-1, 1], [1, 1]], device="cuda"), check=False)
    assert b.device_error() == b.DEVERR_PAIR
    assert bool((out[0][0] == 7).all()) and bool((out[1][1] == 0).all())
    with pytest.raises(b.PagedKVError):
        b.dequantize_blocks(*out, kc, kc, torch.tensor([[0, 1], [1, 1]], device="cuda"))


def test_whole_tiles_move():
    """copy_blocks, copy_blocks_layers and a swap through a pinned pool carry codes and scales together."""
    b = S.lib()
    rng = np.random.default_rng(8)
    mk = lambda n: torch.from_numpy(rng.integers(0, 256, size=(n, 3, 16 * 65), dtype=np.uint8))  # noqa: E731
    kc, vc = mk(8).cuda(), mk(8).cuda()
    k0, v0 = kc.clone(), vc.clone()
    pairs = torch.tensor([[1, 6], [1, 2], [4, 0]], device="cuda")
    b.copy_blocks(kc, vc, pairs)
    for c, c0 in ((kc, k0), (vc, v0)):
        want = c0.clone()
        want[[6, 2, 0]] = c0[[1, 1, 4]]
        assert torch.equal(c, want)
    layers_k, layers_v = [k0.clone(), v0.clone()], [v0.clone(), k0.clone()]
    b.copy_blocks_layers(layers_k, layers_v, pairs)
    assert torch.equal(layers_k[0], kc) and torch.equal(layers_v[1], kc) and torch.equal(layers_k[1], vc)
    hk, hv = mk(4).pin_memory(), mk(4).pin_memory()
    out = torch.tensor([[6, 1], [0, 3]], device="cuda")
    b.swap_blocks(hk, hv, kc, vc, out)
    torch.cuda.synchronize()
    assert torch.equal(hk[[1, 3]], kc[[6, 0]].cpu()) and torch.equal(hv[[1, 3]], vc[[6, 0]].cpu())
    b.swap_blocks(kc, vc, hk, hv, torch.tensor([[2, 5]], device="cuda"))
    assert torch.equal(kc[5].cpu(), hk[2]) and torch.equal(vc[5].cpu(), hv[2])
    assert b.device_error() == 0


class Case:
    """A decode batch over e4m3 caches, its tails and unused blocks poisoned (NaN codes, scale byte 255)."""

    def __init__(self, seed, lens, hkv, g, d, spread=2, gain=1.0):
        rng = np.random.default_rng(seed)
        self.lens, self.scale = lens, d ** -0.5
        self.tables, self.nb = S.layout(rng, lens)
        shape = (self.nb, hkv, 16, d)
        rows = lambda: rng.standard_normal(shape) * 2.0 ** rng.integers(-spread, spread + 1, size=shape[:3] + (1,))  # noqa: E731
        self.k, self.v = S.make_tiles(rows() * gain), S.make_tiles(rows())
        self.q = S.bf16(rng.standard_normal((len(lens), hkv * g, d)))
        dead = ~S.live_slots(self.tables, lens, self.nb)
        for c in (self.k, self.v):
            codes, scales = S.tile_parts(c.numpy())
            codes = np.where(dead[:, None, :, None], 127, codes)
            scales = np.where(dead[:, None], 255, scales)
            c.copy_(torch.from_numpy(np.concatenate([codes.reshape(*codes.shape[:2], -1), scales], -1)))

    def want(self):
        kv, vv, q = S.tile_values(self.k), S.tile_values(self.v), S.f64(self.q)
        res = [S.attend(q[s:s + 1], S.gather(kv, self.tables[s], n, self.nb), S.gather(vv, self.tables[s], n, self.nb),
                        self.scale) for s, n in enumerate(self.lens)]
        return np.concatenate([r[0] for r in res]), np.concatenate([r[1] for r in res])

    def cuda(self):
        return [t.cuda() for t in (self.q, self.k, self.v, torch.from_numpy(self.tables),
                                   torch.tensor(self.lens, dtype=torch.int32))]

    def check(self, out, what=""):
        want, spread = self.want()
        S.close(out, want, ROUND[out.dtype] * np.abs(want) + WEIGHTS * spread + 1e-30, what)


EDGES = [0, 1, 15, 16, 17, 31, 33, 64, 100, 255, 300, 513, 2, 777]


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("hkv,g", [(1, 1), (3, 1), (2, 2), (2, 4), (1, 5), (2, 8), (1, 9), (1, 16)])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_decode(hkv, g, d, dtype):
    b = S.lib()
    c = Case(hkv * 10 + g + d, EDGES, hkv, g, d)
    q, k, v, t, n = c.cuda()
    out = torch.full(q.shape, float("nan"), dtype=dtype, device="cuda")
    b.paged_decode_attention_e4m3(out, q, k, v, t, n, c.scale)
    assert b.device_error() == 0
    c.check(out)


@pytest.mark.parametrize("lens", [[1], [16], [5000, 3], [4096, 4097, 40, 9000], [20000]])
@pytest.mark.parametrize("hkv,g,d", [(2, 4, 128), (3, 1, 64), (1, 16, 128)])
def test_decode_long_contexts(lens, hkv, g, d):
    b = S.lib()
    c = Case(len(lens) + d, lens, hkv, g, d)
    q, k, v, t, n = c.cuda()
    out = torch.full_like(q, float("nan"))
    # garbage in the workspace must not matter
    need = b.e4m3_workspace_bytes(len(lens), hkv * g, hkv, d, max(lens))
    ws = torch.full((max(need, 16),), 255, dtype=torch.uint8, device="cuda")
    b.paged_decode_attention_e4m3(out, q, k, v, t, n, c.scale, max_context_len=max(lens), workspace=ws)
    assert b.device_error() == 0
    c.check(out)


def test_decode_many_sequences():
    b = S.lib()
    rng = np.random.default_rng(77)
    lens = [int(x) for x in rng.integers(0, 200, size=300)]
    c = Case(78, lens, 4, 4, 128)
    q, k, v, t, n = c.cuda()
    out = torch.full_like(q, float("nan"))
    b.paged_decode_attention_e4m3(out, q, k, v, t, n, c.scale, max_context_len=4096)
    assert b.device_error() == 0
    c.check(out)


def test_decode_more_sequences_than_one_launch_takes():
    """4100 sequences of one and two tokens, and a few longer ones: the batch goes in two launches."""
    b = S.lib()
    rng = np.random.default_rng(79)
    lens = [int(x) for x in rng.integers(0, 3, size=4100)]
    lens[5], lens[4095], lens[4096], lens[4099] = 40, 33, 70, 300
    c = Case(80, lens, 1, 2, 64)
    q, k, v, t, n = c.cuda()
    for most in (300, 512):
        out = torch.full_like(q, float("nan"))
        b.paged_decode_attention_e4m3(out, q, k, v, t, n, c.scale, max_context_len=most)
        assert b.device_error() == 0
        c.check(out)


def test_decode_one_long_context_among_many_short_ones():
    """A unit of many segments beside units of one or two: both ways the merge works in one call."""
    b = S.lib()
    lens = [3] * 700 + [30000] + [17] * 20
    c = Case(81, lens, 1, 4, 64)
    q, k, v, t, n = c.cuda()
    out = torch.full_like(q, float("nan"))
    b.paged_decode_attention_e4m3(out, q, k, v, t, n, c.scale)
    assert b.device_error() == 0
    c.check(out)


def test_decode_far_scales():
    """Rows whose scales lie far apart: the weight of a tiny value still counts in the sum, and a huge value with a
    small weight is not lost."""
    b = S.lib()
    c = Case(3, [200, 90, 17], 2, 4, 64, spread=12)
    c.v[:, :, 16 * 64 + 3] = 127 - 30
    c.v[:, :, 16 * 64 + 5] = 127 + 30
    q, k, v, t, n = c.cuda()
    out = torch.zeros(q.shape, dtype=torch.float32, device="cuda")
    c.scale = 0.01                                   # keys differ by powers of two as well
    b.paged_decode_attention_e4m3(out, q, k, v, t, n, c.scale)
    assert b.device_error() == 0
    c.check(out)


def test_decode_far_queries_zero_keys_and_scales():
    b = S.lib()
    c = Case(4, [70, 33], 2, 4, 128)
    c.q[0] *= 2.0 ** 60                              # outside f16 whatever the head
    c.q[1, :4] *= 2.0 ** -60
    q, k, v, t, n = c.cuda()
    for scale in (2.0 ** -60 * 0.08, 0.0, -2.0 ** -60 * 0.08):
        out = torch.zeros(q.shape, dtype=torch.float32, device="cuda")
        c.scale = float(np.float32(scale))
        b.paged_decode_attention_e4m3(out, q, k, v, t, n, c.scale)
        c.check(out, f"scale {scale}")
    zero = torch.zeros_like(q)
    c.q, c.scale = zero.cpu(), 0.1
    out = torch.zeros(q.shape, dtype=torch.float32, device="cuda")
    b.paged_decode_attention_e4m3(out, zero, k, v, t, n, c.scale)
    c.check(out, "zero queries")
    assert b.device_error() == 0


def test_decode_bad_blocks_and_lengths():
    """A table entry out of range reads as zeros and is flagged; lengths past the bounds are clamped and flagged."""
    b = S.lib()
    c = Case(6, [100, 50, 40], 2, 4, 64)
    c.tables[0, 2], c.tables[1, 0] = -7, c.nb
    q, k, v, t, n = c.cuda()
    out = torch.zeros(q.shape, dtype=torch.float32, device="cuda")
    b.paged_decode_attention_e4m3(out, q, k, v, t, n, c.scale)
    assert b.device_error() == b.DEVERR_BLOCK_ID
    c.check(out)
    c = Case(7, [100, 50, 40], 2, 4, 64)
    q, k, v, t, n = c.cuda()
    n[1] = -3
    c.lens = [64, 0, 40]
    b.paged_decode_attention_e4m3(out, q, k, v, t, n, c.scale, max_context_len=64)
    assert b.device_error() == b.DEVERR_LENGTH
    c.check(out)


def test_decode_in_graphs_streams_and_from_pinned_memory():
    b = S.lib()
    a, c = Case(11, [3000, 40, 700], 2, 4, 128), Case(12, [64, 5000], 1, 8, 64)
    side = torch.cuda.Stream()
    runs = []
    for case, stream in ((a, None), (c, side)):
        q, k, v, t, n = case.cuda()
        out = torch.zeros_like(q)
        need = b.e4m3_workspace_bytes(len(case.lens), q.shape[1], k.shape[1], q.shape[2], max(case.lens))
        runs.append((case, q, k, v, t, n, out, torch.empty(max(16, need), dtype=torch.uint8, device="cuda"), stream))
    torch.cuda.synchronize()
    for case, q, k, v, t, n, out, ws, stream in runs:          # two calls at once
        b.paged_decode_attention_e4m3(out, q, k, v, t, n, case.scale, max_context_len=max(case.lens), workspace=ws,
                                      stream=stream)
    torch.cuda.synchronize()
    for case, *_, out, ws, stream in runs:
        case.check(out)
    # one workspace behind two graphs, replayed in turn; their inputs changed in place
    case, q, k, v, t, n, out, ws, _ = runs[0]
    graphs = []
    for _ in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            b.paged_decode_attention_e4m3(out, q, k, v, t, n, case.scale, max_context_len=max(case.lens), workspace=ws)
        graphs.append(g)
    q.mul_(0.5)
    case.q = q.cpu()
    for g in graphs:
        out.zero_()
        g.replay()
        torch.cuda.synchronize()
        case.check(out)
    hq, ho = q.cpu().pin_memory(), torch.zeros(q.shape, dtype=q.dtype).pin_memory()
    b.paged_decode_attention_e4m3(ho, hq, k, v, t.cpu().pin_memory(), n.cpu().pin_memory(), case.scale,
                                  max_context_len=max(case.lens))
    torch.cuda.synchronize()
    case.check(ho)
    assert b.device_error() == 0
