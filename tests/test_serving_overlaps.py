"""Outputs of the serving calls over their inputs are refused on the host (no
GPU here: a call that is not refused must not be made with these addresses)."""
import ctypes

import pytest

from tests.test_serving_abi import A, CF, CI, I64, OK, OVERLAP, VP, caller
from paged_kv_cache_177_gb300.build import build_library


@pytest.fixture(scope="module")
def lib():
    return ctypes.CDLL(build_library())


@pytest.mark.parametrize("name,size", [("qw", 128), ("kw", 128), ("pos", 2 * 4 * 8), ("freq", 32 * 4), ("axes", 32 * 4),
                                       ("slots", 4 * 8), ("kc", 8 * 2 * 16 * 64 * 2), ("vc", 8 * 2 * 16 * 64 * 2)])
def test_queries_go_over_no_other_tensor_of_the_call(lib, name, size):
    """T = 4 tokens of 8 heads of 64 bf16: q_out is the 4 KiB at 256 A."""
    f = caller(lib, "qk_norm_rope_append", [
        ("qo", VP, 256 * A), ("q", VP, 8 * A), ("k", VP, 12 * A), ("v", VP, 13 * A), ("qs", I64, 8 * 64), ("ks", I64, 2 * 64),
        ("vs", I64, 2 * 64), ("qw", VP, 14 * A), ("kw", VP, 15 * A), ("eps", CF, 1e-6), ("pos", VP, 16 * A), ("axes_n", CI, 2),
        ("freq", VP, 17 * A), ("axes", VP, 18 * A), ("rot", CI, 64), ("inter", CI, 0), ("slots", VP, 19 * A), ("kc", VP, 32 * A),
        ("vc", VP, 64 * A), ("T", CI, 4), ("hq", CI, 8), ("hkv", CI, 2), ("d", CI, 64), ("nb", CI, 8), ("dt", CI, 1),
        ("cdt", CI, 1), ("st", VP, None)])
    for at in (256 * A, 257 * A - 16, 256 * A - size + 16):
        assert f(**{name: at}) == OVERLAP, hex(at)
    if name in ("kc", "vc"):                     # tiles are smaller: 16 * 65 bytes each
        assert f(cdt=4, **{name: 256 * A - 8 * 2 * 16 * 65 + 16}) == OVERLAP


def test_blocks_are_read_back_into_other_memory(lib):
    """8 blocks of 2 heads of 64: 16640 bytes of tiles, 32 KiB in bf16, 64 KiB in fp32."""
    f = caller(lib, "dequantize_blocks", [("dk", VP, 256 * A), ("dv", VP, 512 * A), ("dnb", CI, 8), ("sk", VP, 8 * A),
                                          ("sv", VP, 16 * A), ("snb", CI, 8), ("pairs", VP, A), ("n", CI, 2), ("hkv", CI, 2),
                                          ("d", CI, 64), ("dt", CI, 1), ("st", VP, None)])
    for name in ("sk", "sv"):
        for base in (256 * A, 512 * A):
            for at in (base, base + 8 * A - 16, base - 16640 + 16):
                assert f(**{name: at}) == OVERLAP
            assert f(dt=0, **{name: base + 16 * A - 16}) == OVERLAP
    assert f(dv=256 * A) == OVERLAP and f(dv=264 * A - 16) == OVERLAP
    assert f(n=0, dv=256 * A) == OK                                  # nothing to do, nothing to refuse


def test_masks_go_over_no_input(lib):
    """9 drafts of two sequences, one word each."""
    f = caller(lib, "tree_masks", [("mask", VP, 4 * A), ("parents", VP, A), ("qs", VP, 2 * A), ("S", CI, 2), ("T", CI, 9),
                                   ("maxq", CI, 5), ("st", VP, None)])
    assert f(parents=4 * A) == OVERLAP and f(parents=4 * A + 68) == OVERLAP and f(parents=4 * A - 32) == OVERLAP
    assert f(qs=4 * A) == OVERLAP and f(qs=4 * A - 8) == OVERLAP and f(qs=4 * A + 68) == OVERLAP
