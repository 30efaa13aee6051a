"""paged_decode_attention_scored against the formula in 64 bits: capped
scores, a bias by distance, a window, over poisoned caches."""
import numpy as np
import pytest
import torch

from tests import score_helpers as H
from tests import serving_helpers as S

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def seeded():
    torch.manual_seed(1)


BF, F32 = torch.bfloat16, torch.float32


def run(seed, lens, hq, hkv, d, dtype, cap=0.0, window=0, slopes=None, scale=None, q_gain=1.0, workspace=None, **kw):
    B = S.lib()
    B.device_error()
    k, v, tables, kr, vr = H.paged(seed, lens, hkv, d, dtype, window)
    rng = np.random.default_rng(seed + 1)
    q = torch.from_numpy((rng.standard_normal((len(lens), hq, d)) * q_gain).astype(np.float32)).to(dtype).cuda()
    out = torch.full_like(q, float("nan"))
    scale = d ** -0.5 if scale is None else scale
    t = None if slopes is None else torch.from_numpy(slopes).cuda()
    B.paged_decode_attention_scored(out, q, k, v, tables, torch.tensor(lens, dtype=torch.int32, device="cuda"), scale,
                                    softcap=cap, window=window, slopes=t, workspace=workspace, **kw)
    qf = S.f64(q)
    got = S.f64(out)
    for s, n in enumerate(lens):
        want, bound = H.attend(qf[s:s + 1], kr[s], vr[s], scale, [n - 1], cap, slopes, window, dtype=dtype)
        S.close(got[s:s + 1], want, bound, f"sequence {s} of {n}")
    assert B.device_error() == 0
    return out


LENS = [1, 15, 16, 17, 40, 64, 65, 127, 130, 0, 257, 513]


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("hq,hkv", [(8, 8), (8, 4), (9, 3), (12, 4), (8, 1), (32, 2), (7, 1)])
@pytest.mark.parametrize("cap,window,bias", [(30.0, 0, False), (0.0, 37, False), (0.0, 0, True), (5.0, 100, True)])
def test_every_shape(dtype, d, hq, hkv, cap, window, bias):
    for parts in (0, 48) + ((-1,) if dtype == BF else ()):
        run(d + hq, LENS, hq, hkv, d, dtype, cap, window, H.alibi(hq) if bias else None, q_gain=4.0, partition_tokens=parts)


@pytest.mark.parametrize("window", [1, 2, 15, 16, 17, 31, 32, 33, 512, 100000])
@pytest.mark.parametrize("dtype,hq", [(BF, 8), (BF, 2), (F32, 8), (F32, 32)])
def test_window_edges(window, dtype, hq):
    """Every place of the window's start in a block; a window longer than any context."""
    lens = list(range(1, 36)) + [512, 513, 528, 530, 1041]
    run(window, lens, hq, 2, 64, dtype, window=window, partition_tokens=-1 if dtype == BF else 0)
    run(window, lens, hq, 2, 64, dtype, window=window, partition_tokens=16)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("cap", [1e-3, 0.5, 20.0, 1e4, 1e15])
def test_caps_of_every_size(cap, dtype):
    """Scores far above the cap, around it and far below."""
    run(3, [5, 70, 200], 8, 2, 128, dtype, cap=cap, q_gain=10.0)
    run(4, [5, 70, 200], 4, 4, 64, dtype, cap=cap, q_gain=0.05)


@pytest.mark.parametrize("dtype", [BF, F32])
def test_slopes_of_every_kind(dtype):
    """Steep, flat, zero and negative slopes (a bias towards far tokens), and a negative scale."""
    slopes = np.array([8.0, 0.5, 0.0, -0.01, 1e-4, -2.0, 100.0, 0.03], dtype=np.float32)
    run(5, [1, 3, 66, 300, 1000], 8, 2, 64, dtype, slopes=slopes)
    run(6, [1, 3, 66, 300, 1000], 8, 8, 128, dtype, slopes=slopes, scale=-0.2, cap=7.0, window=150)


def test_far_positions():
    """Distances of tens of thousands, in partitions and cut into workers' ranges."""
    run(7, [40000, 33], 8, 2, 64, BF, slopes=H.alibi(8) * 0.01)
    run(8, [40000, 20001], 8, 2, 64, BF, cap=20.0, window=20000, partition_tokens=-1)
    run(9, [20000], 4, 4, 64, F32, slopes=H.alibi(4) * 0.01)


def test_no_transformation_is_plain_decode():
    """Without cap, bias or window both calls compute the same formula.  (Not bit for bit: plain decode loads a
    sequence's last block shifted, so its sums take the tokens in another order.)"""
    B = S.lib()
    lens = [3, 90, 400]
    for hq, dtype in ((2, BF), (8, BF), (4, F32), (16, F32)):
        k, v, tables, kr, vr = H.paged(10, lens, 2, 128, dtype)
        q = torch.randn(3, hq, 128, device="cuda").to(dtype)
        lt = torch.tensor(lens, dtype=torch.int32, device="cuda")
        for call in (B.paged_decode_attention_scored, B.paged_decode_attention):
            out = call(torch.empty_like(q), q, k, v, tables, lt, 0.1)
            for s, n in enumerate(lens):
                want, bound = H.attend(S.f64(q[s:s + 1]), kr[s], vr[s], 0.1, [n - 1], dtype=dtype)
                S.close(out[s:s + 1], want, bound)


def test_many_sequences_share_a_workspace_with_other_calls():
    """A batch that the persistent kernel takes, then plain decode and a batch in partitions, on one workspace."""
    B = S.lib()
    rng = np.random.default_rng(11)
    lens = list(rng.integers(1, 400, 90))
    ws = torch.zeros(B.workspace_bytes(90, 8, 2, 128, 2000, 0), dtype=torch.uint8, device="cuda")
    for _ in range(2):
        run(12, lens, 8, 2, 128, BF, cap=25.0, window=111, workspace=ws, partition_tokens=-1)
        k, v, tables, _, _ = H.paged(13, lens, 2, 128, BF)
        q = torch.randn(90, 8, 128, device="cuda").to(BF)
        lt = torch.tensor(lens, dtype=torch.int32, device="cuda")
        a = B.paged_decode_attention(torch.empty_like(q), q, k, v, tables, lt, 0.1, workspace=ws)
        assert torch.equal(a, B.paged_decode_attention(torch.empty_like(q), q, k, v, tables, lt, 0.1))
        run(14, [2000, 1], 8, 2, 128, BF, slopes=H.alibi(8), workspace=ws)


@pytest.mark.parametrize("window", [1, 16, 17, 200])
def test_a_windows_workspace_is_that_of_what_it_reads(window):
    """A long context's window in as much workspace as the description says, and not a byte less."""
    B = S.lib()
    read = 16 * ((window - 1) // 16 + 2)
    need = B.workspace_bytes(2, 8, 2, 64, min(read, 3000), 16)
    ws = torch.zeros(need, dtype=torch.uint8, device="cuda")
    for n in (3000, 2991, 2990):
        run(window, [n, 40], 8, 2, 64, BF, window=window, workspace=ws, partition_tokens=16)
    with pytest.raises(B.PagedKVError):
        run(window, [3000, 40], 8, 2, 64, BF, window=window, workspace=ws[:need - 16], partition_tokens=16)


def test_bad_pages_in_the_window_read_as_zeros():
    B = S.lib()
    k, v, tables, kr, vr = H.paged(15, [100, 100], 2, 64, BF, window=50)
    tables[1, 4] = 1 << 20
    q = torch.randn(2, 4, 64, device="cuda").to(BF)
    out = torch.empty_like(q)
    for parts in (-1, 16):
        B.device_error()
        B.paged_decode_attention_scored(out, q, k, v, tables, torch.tensor([100, 100], dtype=torch.int32, device="cuda"),
                                        0.125, window=50, softcap=9.0, partition_tokens=parts)
        kr[1][64:80] = vr[1][64:80] = 0.0
        for s in range(2):
            want, bound = H.attend(S.f64(q[s:s + 1]), kr[s], vr[s], 0.125, [99], 9.0, None, 50)
            S.close(out[s:s + 1], want, bound)
        assert B.device_error() == B.DEVERR_BLOCK_ID


def test_captured_and_on_another_stream():
    B = S.lib()
    lens = [77, 300, 16, 1]
    k, v, tables, kr, vr = H.paged(16, lens, 2, 64, BF, window=90)
    lt = torch.tensor(lens, dtype=torch.int32, device="cuda")
    slopes = torch.from_numpy(H.alibi(4)).cuda()
    q = torch.randn(4, 4, 64, device="cuda").to(BF)
    out = torch.empty_like(q)
    ws = torch.zeros(B.workspace_bytes(4, 4, 2, 64, 300, -1), dtype=torch.uint8, device="cuda")
    call = lambda **kw: B.paged_decode_attention_scored(out, q, k, v, tables, lt, 0.125, softcap=8.0, window=90,
                                                        slopes=slopes, max_context_len=300, partition_tokens=-1, **kw)

    def check():
        for s, n in enumerate(lens):
            want, bound = H.attend(S.f64(q[s:s + 1]), kr[s], vr[s], 0.125, [n - 1], 8.0, H.alibi(4), 90)
            S.close(out[s:s + 1], want, bound)
    call(workspace=ws)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call(workspace=ws)
    for _ in range(2):
        q.copy_(torch.randn_like(q))
        graph.replay()
        check()
    side = torch.cuda.Stream()
    q.copy_(torch.randn_like(q))
    out.fill_(float("nan"))
    side.wait_stream(torch.cuda.current_stream())
    call(stream=side)
    side.synchronize()
    check()
