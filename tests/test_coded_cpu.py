"""The operators around a cache in 8 bits without a GPU: refusals of the C entry points, before anything is enqueued."""
import ctypes
import math

import pytest

torch = pytest.importorskip("torch")

from transformer_head_scaled_fwd_gb300 import binding as bnd  # noqa: E402
from transformer_head_scaled_fwd_gb300 import build as B  # noqa: E402

INV, UNS = bnd.MHA_ERR_INVALID_ARG, bnd.MHA_ERR_UNSUPPORTED
P = ctypes.c_void_p(4096)


def at(n):
    return ctypes.c_void_p(n)


@pytest.fixture(scope="module")
def lib():
    B.build()
    return bnd.load()


def st(b=4096, l=512, h=64):
    return ctypes.byref(bnd.StridesT(b, l, h))


def rotary_t(**kw):
    return ctypes.byref(bnd.RotaryT(**(dict(inv_freq=4096, rot_dim=64, interleaved=0, scale=1.0) | kw)))


def cache_t(code=0, block=8, k_scales=4096, v_scales=4096, **kw):
    f = dict(k_pages=4096, v_pages=4096, page_stride=4096, slot_stride=256, head_stride=64, n_pages=10, page_size=16,
             block_table=4096, table_stride=4, max_pages=4) | kw
    return ctypes.byref(bnd.CodedCacheT(bnd.PagedCacheT(**f), code, block, k_scales, v_scales))


BAD_CACHES = [dict(k_pages=None), dict(v_pages=None), dict(block_table=None), dict(page_size=0), dict(n_pages=0), dict(max_pages=-1),
              dict(slot_stride=-16), dict(k_pages=4104), dict(v_pages=4097), dict(page_stride=4104), dict(slot_stride=257),
              dict(head_stride=72), dict(code=2), dict(code=-1), dict(block=0), dict(block=-8), dict(block=3), dict(block=32),
              dict(k_scales=None), dict(v_scales=None), dict(k_scales=4098)]


def test_append_refusals(lib):
    def call(dt=1, k=P, v=P, B_=2, T=3, h=8, hk=4, d=64, start=P, cache=None, rot=None, q=P, qo=P, ko=None, qs=None, ks=None, vs=None):
        return lib.mha_coded_append(dt, q, qs or st(), qo, st(), k, ks or st(), ko, st(), v, vs or st(), B_, T, h, hk, d, start, None,
                                    rot, cache or cache_t(), None)
    assert call(dt=2) == INV
    assert call(B_=0) == INV and call(T=0) == INV and call(hk=0) == INV and call(h=0) == INV
    assert call(start=None) == INV and call(k=None) == INV and call(v=None) == INV and call(qo=None) == INV
    assert call(d=80) == UNS and b"64 and 128" in lib.mha_last_error()
    assert call(B_=1 << 20, T=1 << 12) == UNS and call(B_=1 << 14, T=1 << 13, hk=8) == UNS
    for bad in BAD_CACHES:
        assert call(cache=cache_t(**bad)) == INV, bad
    assert call(cache=cache_t(page_size=512, block=512)) == UNS and b"256" in lib.mha_last_error()
    assert call(rot=rotary_t(rot_dim=66)) == INV and call(rot=rotary_t(rot_dim=63)) == INV and call(rot=rotary_t(scale=math.inf)) == INV
    # 16-byte alignment of every tensor
    for kw in (dict(k=at(4104)), dict(v=at(4098)), dict(q=at(4104)), dict(qo=at(4104)), dict(ko=at(4104))):
        assert call(**kw) == INV, kw
    assert call(ks=st(h=68)) == INV and call(vs=st(l=516)) == INV and call(qs=st(b=4100)) == INV and b"16 bytes" in lib.mha_last_error()
    assert call(ks=st(b=-8)) == INV and b"negative" in lib.mha_last_error()
    assert lib.mha_coded_append(1, None, None, None, None, P, st(), None, None, P, st(), 2, 3, 0, 4, 64, P, None, None, None, None) == INV


def test_attention_refusals(lib):
    def call(dt=1, q=P, out=P, B_=2, h=8, hk=4, d=64, lens=P, cache=None, ws=P, size=1 << 30, scores=None, qs=None):
        return lib.mha_coded_attention(dt, q, qs or st(), out, st(), B_, h, hk, d, lens, scores, cache or cache_t(), ws, size, None)
    assert call(dt=7) == INV and call(B_=0) == INV and call(h=9) == INV and call(h=0) == INV and call(hk=-1) == INV
    assert call(d=96) == UNS and call(B_=70000) == UNS and call(h=65536, hk=1) == UNS
    assert call(q=None) == INV and call(out=None) == INV and call(lens=None) == INV
    for bad in BAD_CACHES:
        assert call(cache=cache_t(**bad)) == INV, bad
    assert lib.mha_coded_attention(1, P, st(), P, st(), 2, 8, 4, 64, P, None, None, P, 1 << 30, None) == INV
    assert call(ws=None) == INV and call(ws=at(4097)) == INV
    need = lib.mha_coded_attention_workspace_size(1, 2, 8, 4, 64)
    assert need > 0 and call(size=need - 1) == INV and b"too small" in lib.mha_last_error()
    assert call(scores=ctypes.byref(bnd.ScoresT(math.nan, 0.0, None))) == INV
    assert call(scores=ctypes.byref(bnd.ScoresT(0.0, -1.0, None))) == INV
    assert call(dt=0, q=at(4098)) == INV and call(qs=st(b=-1)) == INV
    for args in ((3, 2, 8, 4, 64), (1, 0, 8, 4, 64), (1, 2, 9, 4, 64), (1, 2, 8, 4, 80), (1, 2, 8, 0, 64)):
        assert lib.mha_coded_attention_workspace_size(*args) == 0


def test_pages_of_too_many_scales_are_refused(lib):
    big = cache_t(page_size=1 << 30, block=1, slot_stride=256)
    assert lib.mha_coded_attention(1, P, st(), P, st(), 2, 8, 4, 64, P, None, big, P, 1 << 30, None) == UNS and b"scales" in lib.mha_last_error()
    assert lib.mha_coded_append(1, None, None, None, None, P, st(), None, None, P, st(), 2, 3, 0, 4, 64, P, None, None, big, None) == UNS


def test_resize_refusals(lib):
    def call(held=P, want=at(8192), B_=4, page=16, table=at(1 << 16), stride=8, most=8, free=at(1 << 17), n=100, count=at(1 << 18),
             lens=at(1 << 19), new=at(1 << 20), T=4, slots=at(1 << 21)):
        return lib.mha_paged_resize(held, want, B_, page, table, stride, most, free, n, count, lens, new, T, slots, None)
    for name in ("held", "want", "table", "free", "count", "lens"):
        assert call(**{name: None}) == INV, name
        assert call(**{name: at(4098)}) == INV, name
    assert call(new=at(4098)) == INV and call(slots=at(4100)) == INV
    assert call(B_=0) == INV and call(page=0) == INV and call(most=0) == INV and call(n=0) == INV and call(T=0) == INV
    assert call(stride=7) == INV and call(stride=-1) == INV and b"overlap" in lib.mha_last_error()
    assert call(B_=1 << 20, T=1 << 12) == UNS
    assert call(lens=P) == INV and call(lens=at(8192)) == INV and call(new=P) == INV and call(new=at(8192)) == INV
    assert call(new=at(1 << 19)) == INV


def test_resize_refuses_arrays_that_overlap_and_too_many_sequences(lib):
    def call(held, want, lens, new, B_=4):
        return lib.mha_paged_resize(held, want, B_, 16, at(1 << 28), 8, 8, at(1 << 17), 100, at(1 << 18), lens, new, 0, None, None)
    base = 1 << 19
    for off in (4, 12):
        for sign in (1, -1):
            near = at(base + sign * off)
            assert call(at(base), at(8192), near, None) == INV and b"of their own" in lib.mha_last_error(), (off, sign)
            assert call(at(8192), at(base), near, None) == INV
            assert call(at(base), at(8192), at(1 << 20), near) == INV
            assert call(at(8192), at(16384), at(base), near) == INV
    assert call(at(1 << 29), at(1 << 30), at(1 << 31), None, B_=(1 << 24) + 1) == UNS


def test_native_front_declines_what_is_no_call():
    if B.build_front() is None:
        pytest.skip("the headers of Python or torch are missing")
    from transformer_head_scaled_fwd_gb300 import _front as front
    x = torch.zeros(2, 3, 4, 64)
    for name, n in (("paged_resize", 10), ("coded_append", 10), ("coded_attention", 7)):
        f = getattr(front, name)
        assert f() is False and f(*[None] * n) is False and f(*[x] * n) is False and f(*[1.5] * n) is False
        assert f(*[x] * (n + 1)) is False


def test_binding_wants_cuda_tensors():
    x = torch.zeros(4, 16, 2, 64, dtype=torch.int8)
    s, t = torch.ones(4, 1, 2), torch.zeros(2, 2, dtype=torch.int32)
    with pytest.raises(ValueError):
        bnd.make_coded_cache(x, x, s, s, t)
    i = torch.zeros(2, dtype=torch.int32)
    with pytest.raises(ValueError):
        bnd.mha_paged_resize(i, i, block_table=t, page_size=16, free_pages=i, free_count=i[:1], lens=i)
