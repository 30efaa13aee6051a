"""paged_decode_attention_common_prefix with few sequences whose own contexts
are long: units cut into many segments, whose states one warp merges."""
import numpy as np
import pytest
import torch

from tests import serving_helpers as S
from tests.test_gpu_common_prefix import compare, i32, make, run

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def seeded():
    torch.manual_seed(1)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("hq,hkv", [(1, 1), (4, 1), (7, 1), (8, 1), (9, 1), (16, 1), (10, 2), (15, 5)])
def test_long_own_contexts(d, hq, hkv):
    run(hq, [0, 3], [2100, 160, 900], [9], hq, hkv, d)
    run(hq + 1, [0, 1, 3], [5000, 33, 35], [2, 2], hq, hkv, d, gain=3.0)
    run(hq + 2, [0, 4], [16, 17, 1000, 16], [1], hq, hkv, d, gain=6.0)


@pytest.mark.parametrize("blocks", list(range(1, 14)) + [31, 32, 33, 64, 65])
def test_every_number_of_segments(blocks):
    run(blocks, [0, 2], [32 + 16 * blocks, 32 + 16 * blocks - 5], [2], 8, 1, 64)
    run(blocks, [0, 2], [32 + 16 * blocks, 33], [2], 3, 1, 128)


def test_values_that_are_not_finite_show_wherever_they_lie():
    B = S.lib()
    B.device_error()
    lens = [1500, 1400, 70]
    q, k, v, tables, rows = make(5, [0, 3], lens, [4], 8, 2, 64)
    tb = tables.cpu().numpy()
    k[tb[0, 50], 1] = float("nan")                     # a whole block, own: heads 4 to 7 of sequence 0
    k[tb[1, 87], 0, 7] = float("nan")                  # a single key, in the last block: heads 0 to 3 of sequence 1
    v[tb[1, 30], 1, 3, 9] = float("inf")               # an element: heads 4 to 7 of sequence 1
    for s, b, h in ((0, 50, 1), (1, 87, 0)):
        rows[s][0][16 * b:16 * b + 16, h] = 0.0
    out = torch.empty_like(q)
    B.paged_decode_attention_common_prefix(out, q, k, v, tables, i32(lens), 0.125, i32([0, 3]), i32([4]))
    got = out.float().cpu().numpy()
    assert np.isnan(got[0, 4:]).all() and np.isnan(got[1, :4]).all()
    assert (got[1, 4:, 9] == np.inf).all()
    rest = np.isfinite(got)
    assert rest[0, :4].all() and np.delete(rest[1, 4:], 9, 1).all() and rest[2].all()
    compare(out[2:], q[2:], rows[2:], lens[2:], 0.125)
    assert B.device_error() == 0


def test_again_and_again_the_same():
    B = S.lib()
    lens = [3001, 130, 2777, 64]
    q, k, v, tables, rows = make(6, [0, 4], lens, [4], 14, 2, 128)
    ws = torch.zeros(B.common_prefix_workspace_bytes(4, 14, 2, 128), dtype=torch.uint8, device="cuda")
    outs = []
    for _ in range(20):
        outs.append(torch.empty_like(q))
        B.paged_decode_attention_common_prefix(outs[-1], q, k, v, tables, i32(lens), 0.09, i32([0, 4]), i32([4]), workspace=ws)
    compare(outs[0], q, rows, lens, 0.09)
    assert all(torch.equal(outs[0], o) for o in outs)
