"""The serving calls refuse bad arguments on the host, before any launch (no
GPU here), the binding refuses bad tensors, and the 64-bit forms their GPU
tests use are pinned."""
import ctypes
import re

import numpy as np
import pytest
import torch

from tests import serving_helpers as S
from paged_kv_cache_177_gb300.build import INCLUDE, build_library

A = 1 << 12                                   # an aligned address that nothing reads
VP, CI, CF, SZ, I64 = ctypes.c_void_p, ctypes.c_int, ctypes.c_float, ctypes.c_size_t, ctypes.c_int64
OK, ARG, UNSUPPORTED, OVERLAP, WORKSPACE, ALIGN = 0, -1, -2, -4, -6, -7


@pytest.fixture(scope="module")
def lib():
    return ctypes.CDLL(build_library())


def caller(lib, name, spec):
    """spec: [(argument, type, default)] -> a function of keyword overrides."""
    fn = getattr(lib, name)
    fn.restype = CI
    fn.argtypes = [t for _, t, _ in spec]

    def call(**kw):
        assert not set(kw) - {n for n, _, _ in spec}
        return fn(*(kw.get(n, d) for n, _, d in spec))
    return call


def test_append_refusals(lib):
    f = caller(lib, "kv_append_e4m3", [("k", VP, A), ("v", VP, A), ("slots", VP, A), ("kc", VP, A), ("vc", VP, A),
                                       ("T", CI, 4), ("hkv", CI, 8), ("d", CI, 64), ("nb", CI, 32), ("dt", CI, 1),
                                       ("st", VP, None)])
    assert f(T=-1) == ARG and f(hkv=0) == ARG and f(nb=0) == ARG and f(k=None) == ARG and f(slots=None) == ARG
    assert f(d=96) == UNSUPPORTED and f(dt=2) == UNSUPPORTED and f(dt=4) == UNSUPPORTED
    assert f(nb=1 << 28) == UNSUPPORTED          # tile rows past 2^31
    assert f(kc=A + 8) == ALIGN and f(v=A + 2) == ALIGN
    assert f(T=0) == OK


def test_read_back_refusals(lib):
    f = caller(lib, "dequantize_blocks", [("dk", VP, A), ("dv", VP, A), ("dnb", CI, 8), ("sk", VP, A), ("sv", VP, A),
                                          ("snb", CI, 8), ("pairs", VP, A), ("n", CI, 2), ("hkv", CI, 8),
                                          ("d", CI, 128), ("dt", CI, 1), ("st", VP, None)])
    assert f(n=-1) == ARG and f(dnb=0) == ARG and f(snb=0) == ARG and f(hkv=0) == ARG and f(pairs=None) == ARG
    assert f(d=32) == UNSUPPORTED and f(dt=4) == UNSUPPORTED and f(hkv=65536) == UNSUPPORTED
    assert f(dk=A + 8) == ALIGN
    assert f(n=0) == OK


def test_moves_take_tiles(lib):
    """The block moves accept PKV_E4M3; append and attention over [16][D] rows do not."""
    f = caller(lib, "copy_blocks", [("k", VP, A), ("v", VP, A), ("p", VP, A), ("n", CI, 0), ("hkv", CI, 8), ("d", CI, 64),
                                    ("nb", CI, 32), ("dt", CI, 4), ("st", VP, None)])
    assert f() == OK and f(d=96) == UNSUPPORTED and f(dt=3) == UNSUPPORTED and f(dt=5) == UNSUPPORTED
    g = caller(lib, "kv_append", [("k", VP, A), ("v", VP, A), ("s", VP, A), ("kc", VP, A), ("vc", VP, A), ("T", CI, 0),
                                  ("hkv", CI, 8), ("d", CI, 64), ("nb", CI, 32), ("dt", CI, 4), ("st", VP, None)])
    assert g() == UNSUPPORTED


def test_decode_refusals(lib):
    f = caller(lib, "paged_decode_attention_e4m3", [
        ("out", VP, A), ("q", VP, A), ("kc", VP, A), ("vc", VP, A), ("bt", VP, A), ("cl", VP, A), ("scale", CF, 0.1),
        ("hkv", CI, 8), ("S", CI, 4), ("hq", CI, 32), ("d", CI, 128), ("maxb", CI, 8), ("nb", CI, 64), ("maxlen", CI, 128),
        ("dt", CI, 1), ("ws", VP, None), ("wsb", SZ, 0), ("st", VP, None)])
    assert f(S=-1) == ARG and f(hkv=0) == ARG and f(hq=33) == ARG and f(maxb=0) == ARG and f(maxlen=-1) == ARG
    assert f(scale=float("nan")) == ARG and f(scale=float("inf")) == ARG and f(out=None) == ARG and f(cl=None) == ARG
    assert f(d=80) == UNSUPPORTED and f(hq=8 * 17) == UNSUPPORTED and f(dt=0) == UNSUPPORTED and f(dt=4) == UNSUPPORTED
    assert f(S=65536) == UNSUPPORTED and f(nb=1 << 28) == UNSUPPORTED and f(maxb=1 << 28) == UNSUPPORTED
    assert f(S=4096, maxb=1 << 19, maxlen=1 << 30) == UNSUPPORTED      # 2^31 blocks in a launch
    assert f(hkv=1024, hq=1024, maxb=1 << 21, maxlen=1 << 30) == UNSUPPORTED
    assert f(q=A + 8) == ALIGN
    assert f(S=0) == OK


def test_rope_refusals(lib):
    f = caller(lib, "qk_norm_rope_append", [
        ("qo", VP, A), ("q", VP, 2 * A), ("k", VP, A), ("v", VP, A), ("qs", I64, 8 * 64), ("ks", I64, 2 * 64),
        ("vs", I64, 2 * 64), ("qw", VP, A), ("kw", VP, A), ("eps", CF, 1e-6), ("pos", VP, A), ("axes_n", CI, 1),
        ("freq", VP, A), ("axes", VP, None), ("rot", CI, 64), ("inter", CI, 0), ("slots", VP, A), ("kc", VP, A),
        ("vc", VP, A), ("T", CI, 4), ("hq", CI, 8), ("hkv", CI, 2), ("d", CI, 64), ("nb", CI, 8), ("dt", CI, 1),
        ("cdt", CI, 1), ("st", VP, None)])
    assert f(T=-1) == ARG and f(hq=0) == ARG and f(hkv=0) == ARG and f(rot=-16) == ARG and f(qw=None) == ARG
    assert f(qs=8 * 64 - 8) == ARG and f(vs=0) == ARG and f(pos=None) == ARG and f(freq=None) == ARG
    assert f(axes_n=0) == ARG and f(eps=-1.0) == ARG and f(eps=float("nan")) == ARG and f(slots=None) == ARG
    assert f(d=96) == UNSUPPORTED and f(rot=72) == UNSUPPORTED and f(rot=80) == UNSUPPORTED
    assert f(dt=2) == UNSUPPORTED and f(cdt=0) == UNSUPPORTED and f(dt=4, cdt=4) == UNSUPPORTED
    assert f(qs=8 * 64 + 4) == ALIGN and f(kc=A + 8) == ALIGN and f(kw=A + 8) == ALIGN
    assert f(qo=2 * A, qs=9 * 64) == OVERLAP
    assert f(T=0) == OK


def test_rope_refuses_outputs_over_its_inputs(lib):
    """q_out over k, v or a part of q; T = 4 tokens of 8 heads of 64 bf16 (4 KiB), k and v 1 KiB."""
    f = caller(lib, "qk_norm_rope_append", [
        ("qo", VP, 16 * A), ("q", VP, 8 * A), ("k", VP, 32 * A), ("v", VP, 33 * A), ("qs", I64, 8 * 64), ("ks", I64, 2 * 64),
        ("vs", I64, 2 * 64), ("qw", VP, None), ("kw", VP, None), ("eps", CF, 1e-6), ("pos", VP, None), ("axes_n", CI, 0),
        ("freq", VP, None), ("axes", VP, None), ("rot", CI, 0), ("inter", CI, 0), ("slots", VP, A), ("kc", VP, A),
        ("vc", VP, A), ("T", CI, 4), ("hq", CI, 8), ("hkv", CI, 2), ("d", CI, 64), ("nb", CI, 8), ("dt", CI, 1),
        ("cdt", CI, 1), ("st", VP, None)])
    assert f(k=16 * A) == OVERLAP and f(v=17 * A - 16) == OVERLAP and f(k=16 * A - 1024 + 16) == OVERLAP
    assert f(q=16 * A + 16) == OVERLAP and f(q=15 * A + 16) == OVERLAP
    assert f(q=13 * A, qs=4 * 8 * 64) == OVERLAP            # the last token's row reaches into q_out
    assert f(k=14 * A, ks=4 * 8 * 64) == OVERLAP


def test_tree_refusals(lib):
    f = caller(lib, "paged_tree_attention", [
        ("out", VP, A), ("q", VP, A), ("kc", VP, A), ("vc", VP, A), ("bt", VP, A), ("cl", VP, A), ("qs", VP, A),
        ("mask", VP, A), ("words", CI, 1), ("scale", CF, 0.1), ("hkv", CI, 8), ("S", CI, 4), ("hq", CI, 32), ("d", CI, 128),
        ("maxb", CI, 8), ("nb", CI, 64), ("T", CI, 40), ("maxq", CI, 16), ("maxlen", CI, 128), ("dt", CI, 1),
        ("ws", VP, None), ("wsb", SZ, 0), ("st", VP, None)])
    assert f(S=-1) == ARG and f(hq=33) == ARG and f(T=-1) == ARG and f(maxq=-1) == ARG and f(mask=None) == ARG
    assert f(maxq=65, words=1) == ARG and f(qs=None) == ARG and f(scale=float("inf")) == ARG
    assert f(dt=0) == UNSUPPORTED and f(d=32) == UNSUPPORTED and f(hq=8 * 65) == UNSUPPORTED
    assert f(maxq=1025, words=17) == UNSUPPORTED
    assert f(q=A + 2) == ALIGN and f(mask=A + 4) == ALIGN
    assert f(S=0) == OK and f(maxq=0) == OK and f(T=0) == OK
    m = caller(lib, "tree_masks", [("mask", VP, A), ("parents", VP, A), ("qs", VP, A), ("S", CI, 2), ("T", CI, 9),
                                   ("maxq", CI, 5), ("st", VP, None)])
    assert m(S=-1) == ARG and m(T=-1) == ARG and m(maxq=-1) == ARG and m(parents=None) == ARG
    assert m(maxq=1025) == UNSUPPORTED and m(mask=A + 4) == ALIGN and m(S=0) == OK and m(T=0) == OK


def test_acceptance_refusals(lib):
    f = caller(lib, "kv_accept_layers", [
        ("kcs", VP, A), ("vcs", VP, A), ("L", CI, 2), ("bt", VP, A), ("cl", VP, A), ("qs", VP, A), ("acc", VP, A),
        ("M", CI, 4), ("num", VP, A), ("new", VP, 2 * A), ("S", CI, 3), ("hkv", CI, 2), ("d", CI, 64), ("maxb", CI, 4),
        ("nb", CI, 8), ("dt", CI, 1), ("st", VP, None)])
    assert f(L=-1) == ARG and f(S=-1) == ARG and f(M=-1) == ARG and f(maxb=0) == ARG and f(acc=None) == ARG
    assert f(kcs=None) == ARG and f(new=None) == ARG
    assert f(d=96) == UNSUPPORTED and f(dt=4) == UNSUPPORTED and f(M=65) == UNSUPPORTED and f(S=65536) == UNSUPPORTED
    assert f(new=A) == OVERLAP and f(new=A + 8) == OVERLAP and f(new=A - 8) == OVERLAP
    assert f(L=0) == OK and f(S=0) == OK
    for other in ("num", "qs", "acc", "bt"):                # every CTA reads these after some have written
        assert f(new=2 * A, **{other: 2 * A}) == OVERLAP and f(new=2 * A + 8, **{other: 2 * A}) == OVERLAP
    assert f(new=2 * A - 12, qs=2 * A - 24) == OVERLAP      # S + 1 entries


def test_constants_match_the_header():
    from paged_kv_cache_177_gb300 import binding as b
    text = open(f"{INCLUDE}/pagedkv.h").read()
    for name, value in (("PKV_TREE_MAX_DRAFTS", b.TREE_MAX_DRAFTS), ("PKV_MAX_ACCEPTED", b.MAX_ACCEPTED)):
        assert int(re.search(rf"#define\s+{name}\s+(\d+)", text).group(1)) == value
    assert int(re.search(r"#define\s+PKV_DEVERR_INDEX\s+(0x\w+)u", text).group(1), 16) == b.DEVERR_INDEX
    assert int(re.search(r"PKV_E4M3 = (\d+)", text).group(1)) == b.PKV_E4M3


def test_workspace_sizes_are_whole_and_grow_with_the_batch():
    from paged_kv_cache_177_gb300 import binding as b
    for fn, args in ((b.e4m3_workspace_bytes, (8, 64, 8, 128, 131072)),
                     (b.tree_workspace_bytes, (8, 64, 8, 128, 16, 131072))):
        n = fn(*args)
        assert n >= 0 and n % 4 == 0 and fn(0, *args[1:]) == 0


def test_binding_refuses_bad_tensors():
    from paged_kv_cache_177_gb300 import binding as b
    z = torch.zeros
    kc = z(2, 1, 16 * 65, dtype=torch.uint8)
    with pytest.raises(ValueError):                                   # not on a GPU
        b.kv_append_e4m3(z(1, 1, 64), z(1, 1, 64), z(1, dtype=torch.int64), kc, kc)
    with pytest.raises(ValueError):
        b.paged_decode_attention_e4m3(z(1, 1, 64), z(1, 1, 64), kc, kc, z(1, 1, dtype=torch.int32),
                                      z(1, dtype=torch.int32), 0.1)
    with pytest.raises(ValueError):
        b.tree_masks(z(1, dtype=torch.int32), z(2, dtype=torch.int32), 1)
    with pytest.raises(ValueError):
        b.e4m3_cache(1, 1, 96, device="cpu")
    with pytest.raises(ValueError):
        b._pool_shape(z(2, 1, 17, dtype=torch.uint8))
    assert b._pool_shape(kc) == (2, 1, 64, b.PKV_E4M3)
    assert b.e4m3_cache(2, 3, 128, device="cpu").shape == (2, 3, 16 * 129)
    with pytest.raises(ValueError):                                   # heads apart
        b._token_rows(z(4, 3, 64)[:, ::2], "q")
    assert b._token_rows(z(4, 3, 64)[:, 1:], "q") == ((4, 2, 64), 192)


def test_the_64_bit_forms():
    """Codes against torch's own e4m3 cast, the scale's border, and attention against torch's softmax."""
    x = np.random.default_rng(0).standard_normal((50, 64)) * 100
    codes, scales = S.e4m3_rows(x)
    t = torch.from_numpy(x * 2.0 ** -(scales.astype(np.float64) - 127)[:, None]).float()
    assert np.array_equal(t.to(torch.float8_e4m3fn).view(torch.uint8).numpy(), codes)
    assert np.all(np.abs(t.numpy()).max(1) <= 448) and np.all(np.abs(t.numpy()).max(1) > 224)
    ref = torch.arange(256, dtype=torch.uint8).view(torch.float8_e4m3fn).double().numpy()
    assert np.array_equal(ref, S.VALUES, equal_nan=True)
    border = np.zeros((3, 64))
    border[:, 5] = [448, np.nextafter(448, 1e9), 449]
    assert S.e4m3_rows(border)[1].tolist() == [127, 128, 128]
    q, k, v = (torch.randn(3, 4, 64, dtype=torch.float64) for _ in range(3))
    got, spread = S.attend(q.numpy(), k[:, :2].numpy(), v[:, :2].numpy(), 0.3)
    for h in range(4):
        w = torch.softmax(q[:, h] @ k[:, h // 2].T * 0.3, -1)
        assert np.allclose(got[:, h], (w @ v[:, h // 2]).numpy(), atol=1e-14)
        assert np.allclose(spread[:, h], (w @ v[:, h // 2].abs()).numpy(), atol=1e-14)
