"""Host-side refusals of the 4-bit cache, norm + rotation and block calls: each
returns before anything is launched (CPU only; the pointers are never read)."""

import ctypes
import os

import pytest
import torch

import paged_kv_cache_304_gb300 as pkv
from paged_kv_cache_304_gb300 import q4, rope

NULL, SHAPE, UNSUPPORTED, WORKSPACE, ALIGN = -1, -2, -3, -4, -6
F = 0x10000  # stands for an aligned device pointer


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(pkv.LIB_PATH):
        from paged_kv_cache_304_gb300 import build
        build.build()
    return pkv.load()


def cache(**kw):
    a = dict(k_data=F, k_scales=F, v_data=F, v_scales=F, k_scale=1.0, v_scale=1.0, num_blocks=4, block_size=256,
             num_kv_heads=8, head_dim=128)
    c = q4._Struct(**{**a, **kw})
    cache.keep = c
    return ctypes.addressof(c)


BAD_CACHES = [(dict(num_blocks=0), SHAPE), (dict(block_size=16), UNSUPPORTED), (dict(head_dim=64), UNSUPPORTED),
              (dict(num_kv_heads=9), UNSUPPORTED), (dict(num_kv_heads=0), SHAPE), (dict(num_blocks=1 << 23), UNSUPPORTED),
              (dict(k_scale=0.0), SHAPE), (dict(v_scale=float("nan")), SHAPE), (dict(v_scale=float("inf")), SHAPE),
              (dict(k_scale=-1.0), SHAPE), (dict(k_scale=1e-45), SHAPE)]


@pytest.mark.parametrize("bad,status", BAD_CACHES)
def test_cache_refused_by_every_call(lib, bad, status):
    c = cache(**bad)
    nr = norm()
    assert lib.pkv_kv_cache_write_q4(F, 1024, F, 1024, F, 2, c, None) == status
    assert lib.pkv_kv_cache_read_q4(c, F, 2, F, F, None) == status
    assert lib.pkv_paged_attn_decode_q4(F, c, F, F, 4, 2, 16, 512, 0.1, F, F, 1 << 30, None) == status
    assert lib.pkv_paged_attn_prefill_q4(F, c, F, F, F, 4, 1, 8, 8, 8, 16, 0.1, F, F, 1 << 30, None) == status
    assert lib.pkv_qk_norm_rope_write_q4(F, 4096, F, 4096, F, 4096, 2, 16, nr, F, c, F, 2048, None) == status


def test_null_and_misaligned_cache_pointers(lib):
    for name in ("k_data", "k_scales", "v_data", "v_scales"):
        assert lib.pkv_kv_cache_write_q4(F, 1024, F, 1024, F, 2, cache(**{name: None}), None) == NULL
        assert lib.pkv_kv_cache_write_q4(F, 1024, F, 1024, F, 2, cache(**{name: F + 8}), None) == ALIGN
    assert lib.pkv_kv_cache_write_q4(F, 1024, F, 1024, F, 2, None, None) == NULL


def test_write_and_read_arguments(lib):
    c = cache()
    w = lib.pkv_kv_cache_write_q4
    assert w(F, 1024, F, 1024, F, -1, c, None) == SHAPE
    assert w(F, 1016, F, 1024, F, 2, c, None) == SHAPE
    assert w(F, 1028, F, 1024, F, 2, c, None) == ALIGN
    assert w(F + 2, 1024, F, 1024, F, 2, c, None) == ALIGN
    assert w(None, 1024, F, 1024, F, 2, c, None) == NULL
    assert w(F, 1024, F, 1024, None, 2, c, None) == NULL
    assert w(None, 1024, None, 1024, None, 0, c, None) == 0
    r = lib.pkv_kv_cache_read_q4
    assert r(c, F, -1, F, F, None) == SHAPE
    assert r(c, None, 2, F, F, None) == NULL
    assert r(c, F, 2, F + 8, F, None) == ALIGN
    assert r(c, None, 0, None, None, None) == 0


def test_decode_arguments(lib):
    c = cache()

    def call(q=F, hq=16, maxb=4, b=2, maxlen=512, scale=0.1, out=F, ctx=F):
        return lib.pkv_paged_attn_decode_q4(q, c, ctx, F, maxb, b, hq, maxlen, scale, out, F, 1 << 30, None)

    assert call(hq=12) == SHAPE and call(hq=0) == SHAPE
    assert call(hq=72) == UNSUPPORTED
    assert call(maxb=0) == SHAPE and call(b=-1) == SHAPE and call(maxlen=-1) == SHAPE
    assert call(maxlen=1 << 26) == UNSUPPORTED
    for s in (0.0, -1.0, float("nan"), float("inf")):
        assert call(scale=s) == SHAPE
    assert call(q=None) == NULL and call(ctx=None) == NULL
    assert call(q=F + 8) == ALIGN and call(out=F + 2) == ALIGN
    assert call(b=0) == 0


def test_group_above_sixteen_refused(lib):
    assert lib.pkv_paged_attn_decode_q4(F, cache(num_kv_heads=1), F, F, 4, 2, 32, 512, 0.1, F, F, 1 << 30,
                                        None) == UNSUPPORTED


def test_prefill_arguments(lib):
    c = cache()

    def call(hq=16, maxb=4, s=1, t=8, mq=8, mk=8, scale=0.1, q=F, cu=F):
        return lib.pkv_paged_attn_prefill_q4(q, c, cu, F, F, maxb, s, t, mq, mk, hq, scale, F, F, 1 << 30, None)

    assert call(mq=9) == SHAPE and call(s=-1) == SHAPE and call(t=-1) == SHAPE and call(hq=10) == SHAPE
    assert call(s=65536) == UNSUPPORTED and call(mk=1 << 26) == UNSUPPORTED
    assert call(q=None) == NULL and call(cu=None) == NULL and call(q=F + 4) == ALIGN
    assert call(t=0) == 0 and call(s=0) == 0 and call(mq=0) == 0


def norm(**kw):
    """A pkv_norm_rope description (bytes, read on the host)."""
    a = dict(q_weight=F, k_weight=F, freqs=F, positions=F, position_axis_stride=0, eps=1e-6, rope_dim=128,
             interleaved=0, num_axes=1, sections=(64, 0, 0))
    *fields, sections = ({**a, **kw}).values()
    return rope._PACK(*(f or 0 for f in fields), *sections)


@pytest.mark.parametrize("bad,status", [
    (dict(eps=-1.0), SHAPE), (dict(eps=float("nan")), SHAPE), (dict(rope_dim=130), SHAPE), (dict(rope_dim=-2), SHAPE),
    (dict(rope_dim=33), SHAPE), (dict(rope_dim=48), UNSUPPORTED), (dict(sections=(63, 0, 0)), SHAPE),
    (dict(num_axes=0), SHAPE), (dict(num_axes=4), UNSUPPORTED), (dict(num_axes=2, sections=(32, 31, 0)), SHAPE),
    (dict(num_axes=3, sections=(65, -1, 0)), SHAPE), (dict(num_axes=2, sections=(32, 32, 0), position_axis_stride=-1),
                                                      SHAPE),
    (dict(freqs=None), NULL), (dict(positions=None), NULL), (dict(freqs=F + 4), ALIGN), (dict(q_weight=F + 8), ALIGN)])
def test_norm_rope_description_refused(lib, bad, status):
    assert lib.pkv_qk_norm_rope(F, 2048, F, 1024, 2, 16, 8, 128, norm(**bad), F, 2048, F, 1024, None) == status
    assert lib.pkv_qk_norm_rope_write(F, 2048, F, 1024, F, 1024, 2, 16, norm(**bad), F, F, F, 4, 256, 8, 128, F, 2048,
                                      None) == status
    assert lib.pkv_qk_norm_rope_write_q4(F, 2048, F, 1024, F, 1024, 2, 16, norm(**bad), F, cache(), F, 2048,
                                         None) == status


def test_norm_rope_arguments(lib):
    f = lib.pkv_qk_norm_rope
    nr = norm()
    assert f(F, 2048, F, 1024, -1, 16, 8, 128, nr, F, 2048, F, 1024, None) == SHAPE
    assert f(F, 2040, F, 1024, 2, 16, 8, 128, nr, F, 2048, F, 1024, None) == SHAPE
    assert f(F, 2048, F, 1024, 2, 16, 8, 64, nr, F, 2048, F, 1024, None) == UNSUPPORTED
    assert f(F, 2048, F, 1024, 2, 65, 8, 128, nr, F, 2048, F, 1024, None) == UNSUPPORTED
    assert f(F, 2048, F, 1028, 2, 16, 8, 128, nr, F, 2048, F, 1024, None) == ALIGN
    assert f(F, 2048, F, 1024, 2, 16, 8, 128, nr, F + 8, 2048, F, 1024, None) == ALIGN
    assert f(F, 2048, F, 1024, 2, 16, 8, 128, nr, F, 2048, None, 1024, None) == NULL
    assert f(F, 2048, F, 1024, 2, 16, 8, 128, None, F, 2048, F, 1024, None) == NULL
    assert f(None, 2048, None, 1024, 0, 16, 8, 128, nr, None, 2048, None, 1024, None) == 0
    w = lib.pkv_qk_norm_rope_write
    assert w(F, 2048, F, 1024, None, 1024, 2, 16, nr, F, F, F, 4, 256, 8, 128, F, 2048, None) == NULL
    assert w(F, 2048, F, 1024, F, 1024, 2, 16, nr, F, F, F, 4, 128, 8, 128, F, 2048, None) == UNSUPPORTED
    assert w(F, 2048, F, 1024, F, 1000, 2, 16, nr, F, F, F, 4, 256, 8, 128, F, 2048, None) == SHAPE


def test_block_call_arguments(lib):
    fork, free, comp, copy = lib.pkv_fork_blocks, lib.pkv_free_blocks, lib.pkv_compact_blocks, lib.pkv_copy_blocks
    assert fork(F, F, 2, 0, F, 2, F, 8, F, F, F, F, None) == SHAPE
    assert fork(F, F, 2, 4, F, -1, F, 8, F, F, F, F, None) == SHAPE
    assert fork(F, F, 2, 4, F, 8193, F, 8, F, F, F, F, None) == UNSUPPORTED
    assert fork(F, F, 2, 4, F, 2, F, 1 << 23, F, F, F, F, None) == UNSUPPORTED
    assert fork(F, F, 2, 4, None, 2, F, 8, F, F, F, F, None) == NULL
    assert fork(None, None, 0, 4, None, 0, None, 8, None, None, None, None, None) == 0
    assert free(F, F, -1, 4, F, 8, None) == SHAPE
    assert free(F, F, 2, 4, None, 8, None) == NULL
    assert free(None, None, 0, 4, None, 8, None) == 0
    assert comp(F, F, 2, 4, F, 0, F, F, F, F, F, None) == SHAPE
    assert comp(F, F, 2, 4, F, 8, F, F, None, F, F, None) == NULL
    assert comp(F, F, 2, 4, F, 8, F, F, F, F, None, None) == NULL
    assert copy(F, 2, 1024, 8, 256, F, F, 3, None) == SHAPE       # planes overlap
    assert copy(F, 1, 0, 8, 24, F, F, 3, None) == ALIGN
    assert copy(F + 8, 1, 0, 8, 32, F, F, 3, None) == ALIGN
    assert copy(F, -1, 0, 8, 32, F, F, 3, None) == SHAPE
    assert copy(None, 1, 0, 8, 32, F, F, 3, None) == NULL
    assert copy(None, 1, 0, 8, 32, None, None, 0, None) == 0


def test_binding_refuses_host_tensors_and_bad_frequencies():
    t = torch.zeros(2, 256, 8, 64, dtype=torch.uint8)
    with pytest.raises(TypeError):
        pkv.Q4Cache(t, t, t, t)
    with pytest.raises(TypeError):
        pkv.kv_cache_write_q4(t, t, t, "cache")
    with pytest.raises(TypeError):
        pkv.copy_blocks(t, t, t)
    with pytest.raises(ValueError):
        pkv.rope_frequencies(3, device="cpu")
    with pytest.raises(ValueError):
        pkv.rope_frequencies(4, device="cpu", inv_freq=[1.0])
    with pytest.raises(ValueError):
        pkv.rope_frequencies(4, device="cpu", inv_freq=[1.0, float("inf")])


def test_frequencies_are_turns():
    f = pkv.rope_frequencies(4, 100.0, device="cpu")
    import math
    assert f.dtype == torch.int64 and list(f) == [round(x / (2 * math.pi) * 2**64) for x in (1.0, 0.1)]
    # a quarter turn backwards and one and a half turns
    g = pkv.rope_frequencies(4, device="cpu", inv_freq=[-math.pi / 2, 3 * math.pi])
    assert list(g) == [-(2**62), -(2**63)]
