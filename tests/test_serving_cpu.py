"""Serving operators without a GPU: refusals of the C entry points (before anything is enqueued) and of
the binding, and the frequency tables of scaled rotary positions against their definitions."""
import ctypes
import math
import os
import shutil
import subprocess

import pytest

torch = pytest.importorskip("torch")

from transformer_head_scaled_fwd_gb300 import binding as bnd  # noqa: E402
from transformer_head_scaled_fwd_gb300 import build as B  # noqa: E402

INV, UNS = bnd.MHA_ERR_INVALID_ARG, bnd.MHA_ERR_UNSUPPORTED
P = ctypes.c_void_p(4096)


@pytest.fixture(scope="module")
def lib():
    B.build()
    return bnd.load()


def st(b=4096, l=512, h=64):
    return ctypes.byref(bnd.StridesT(b, l, h))


def rotary_t(**kw):
    f = dict(inv_freq=4096, rot_dim=64, interleaved=0, scale=1.0) | kw
    return ctypes.byref(bnd.RotaryT(**f))


def cache_t(**kw):
    f = dict(k_pages=4096, v_pages=4096, page_stride=8192, slot_stride=512, head_stride=64, n_pages=10, page_size=16,
             block_table=4096, table_stride=4, max_pages=4) | kw
    return ctypes.byref(bnd.PagedCacheT(**f))


def scores_t(**kw):
    return ctypes.byref(bnd.ScoresT(**(dict(scale=0.0, cap=0.0, slopes=None) | kw)))


def test_rotary_refusals(lib):
    def call(dt=0, q=P, qs=None, qo=P, k=P, ks=None, ko=P, kos=None, B_=2, T=3, h=8, hk=4, d=64, rot=None):
        return lib.mha_rotary(dt, q, qs or st(), qo, st(), k, ks or st(), ko, kos or st(), B_, T, h, hk, d, None,
                              rot or rotary_t(), None)
    assert call(dt=5) == INV
    assert call(B_=0) == INV and call(T=-1) == INV and call(h=0) == INV and call(hk=0) == INV
    assert call(d=2048) == UNS
    assert call(B_=1 << 20, T=1 << 12) == UNS
    assert call(q=None) == INV and call(qo=None) == INV and call(ko=None) == INV
    assert call(rot=rotary_t(rot_dim=63)) == INV
    assert call(rot=rotary_t(rot_dim=66)) == INV      # beyond d_k
    assert call(rot=rotary_t(rot_dim=0)) == INV
    assert call(rot=rotary_t(interleaved=2)) == INV
    assert call(rot=rotary_t(scale=math.nan)) == INV
    assert call(rot=rotary_t(inv_freq=None)) == INV
    assert call(qs=st(b=-1)) == INV and b"negative" in lib.mha_last_error()
    assert call(q=ctypes.c_void_p(4098)) == INV       # fp32 at an odd half word


def test_append_refusals(lib):
    def call(dt=1, k=P, v=P, B_=2, T=3, h=8, hk=4, d=64, start=P, cache=None, rot=None, q=P, qo=P):
        return lib.mha_paged_append(dt, q, st(), qo, st(), k, st(), None, None, v, st(), B_, T, h, hk, d, start, None,
                                    rot, cache or cache_t(), None)
    assert call(dt=2) == INV
    assert call(start=None) == INV and call(k=None) == INV and call(v=None) == INV and call(qo=None) == INV
    assert call(hk=0) == INV
    assert call(cache=cache_t(k_pages=None)) == INV
    assert call(cache=cache_t(page_size=0)) == INV and call(cache=cache_t(n_pages=0)) == INV
    assert call(cache=cache_t(max_pages=-1)) == INV and call(cache=cache_t(slot_stride=-8)) == INV
    assert call(cache=cache_t(k_pages=4097)) == INV
    assert call(rot=rotary_t(rot_dim=128)) == INV
    assert lib.mha_paged_append(1, None, None, None, None, P, st(), None, None, P, st(), 2, 3, 0, 4, 64, P, None, None,
                                None, None) == INV   # no cache


def test_paged_attention_refusals(lib):
    def call(dt=1, q=P, out=P, B_=2, h=8, hk=4, d=64, lens=P, sc=None, cache=None, ws=ctypes.c_void_p(4096), n=1 << 30):
        return lib.mha_paged_attention(dt, q, st(), out, st(), B_, h, hk, d, lens, sc, cache or cache_t(), ws, n, None)
    assert call(dt=9) == INV
    assert call(h=9) == INV and b"h_kv" in lib.mha_last_error()
    assert call(d=96) == UNS
    assert call(B_=0) == INV and call(B_=70000) == UNS
    assert call(lens=None) == INV and call(q=None) == INV and call(out=None) == INV
    assert call(sc=scores_t(cap=-1.0)) == INV and call(sc=scores_t(scale=math.inf)) == INV
    assert call(cache=cache_t(slot_stride=65)) == INV          # not 16 bytes
    assert call(cache=cache_t(v_pages=4104)) == INV
    assert call(dt=0, cache=cache_t(head_stride=66)) == INV and call(dt=0, cache=cache_t(k_pages=4100)) == INV
    assert call(ws=None) == INV and call(ws=ctypes.c_void_p(4100)) == INV and call(n=0) == INV
    assert bnd.paged_attention_workspace_size(1, 2, 9, 4, 64) == 0
    assert bnd.paged_attention_workspace_size(1, 2, 8, 4, 80) == 0
    assert bnd.paged_attention_workspace_size(0, 2, 8, 4, 64) > 0


def test_attention_refusals(lib):
    def call(dt=1, q=P, k=P, v=P, out=P, B_=2, Lq=8, Lk=8, h=8, hk=4, d=64, sc=None, qs=None, mask=None):
        return lib.mha_attention(dt, q, qs or st(), k, st(), v, st(), out, st(), B_, Lq, Lk, h, hk, d, sc,
                                 ctypes.byref(mask) if mask is not None else None, None)
    assert call(dt=3) == INV and call(dt=0, qs=st(l=66)) == INV and call(dt=0, q=ctypes.c_void_p(4100)) == INV
    assert call(Lk=0x7fffff01) == UNS and call(Lq=0x7fffff01) == UNS
    assert call(d=32) == UNS and call(h=6) == INV and call(Lk=0) == INV
    assert call(q=None) == INV and call(out=None) == INV
    assert call(qs=st(l=65)) == INV and call(q=ctypes.c_void_p(4104)) == INV
    assert call(sc=scores_t(cap=math.nan)) == INV
    assert call(B_=1 << 20, Lq=1 << 20) == UNS
    assert call(qs=st(l=0)) == INV
    m = bnd.SpanMaskT(1, -1, None, None, None)
    assert call(mask=m) == INV
    m = bnd.SpanMaskT(1, 0, None, None, 4100)
    assert call(mask=m) == INV
    assert lib.mha_document_spans(None, 1, 1, P, None) == INV
    assert lib.mha_document_spans(P, 0, 1, P, None) == INV
    assert lib.mha_document_spans(P, 1, 1, ctypes.c_void_p(4100), None) == INV
    assert lib.mha_document_spans(P, 70000, 1, P, None) == UNS


def test_prefix_lens_reach_no_kernel_unless_causal(tmp_path):
    """The kernels' parameters from a mask, as mha_attention fills them: prefix_lens is read only if causal, so a pointer that
    is left there otherwise is not passed on."""
    if shutil.which("g++") is None:
        pytest.skip("no g++")
    src, exe = tmp_path / "mask.cpp", tmp_path / "mask"
    src.write_text('''
#include "mha.h"
#include "serve.h"
int main() {
    static const int32_t lens[2] = {1, 2};
    for (int causal = 0; causal < 2; ++causal) {
        mha_span_mask_t m{causal, 7, lens, lens + 1, lens};
        mha::SpanAttnParams p{};
        mha::set_mask(m, &p);
        if (p.causal != causal || p.q_offset != 7 || p.valid_lens != lens || p.spans != lens) return 1;
        if (p.prefix_lens != (causal ? lens + 1 : nullptr)) return 2;
    }
    return 0;
}
''')
    cuda = os.path.join(os.path.dirname(os.path.dirname(os.path.realpath(B._nvcc()))), "include")
    subprocess.run(["g++", "-std=c++17", "-I", os.path.join(B.ROOT, "include"), "-I", B.CSRC, "-I", cuda, str(src), "-o", str(exe)],
                   check=True)
    assert subprocess.run([str(exe)]).returncode == 0


def test_scale_over_cap_must_be_finite(lib):
    sc = scores_t(scale=1e30, cap=1e-30)
    assert lib.mha_attention(1, P, st(), P, st(), P, st(), P, st(), 2, 8, 8, 8, 4, 64, sc, None, None) == INV
    assert b"scale / cap" in lib.mha_last_error()
    assert lib.mha_paged_attention(1, P, st(), P, st(), 2, 8, 4, 64, P, sc, cache_t(), P, 1 << 30, None) == INV
    assert b"scale / cap" in lib.mha_last_error()


def test_rmsnorm_refusals(lib):
    def call(dt=1, x=P, r=P, s=P, y=P, rows=4, d=256, eps=1e-6, scales=None, group=0, ys=256, ss=256, xs=256):
        return lib.mha_rmsnorm(dt, x, xs, r, 256, s, ss, None, eps, rows, d, y, ys, scales, group, None)
    assert call(dt=3) == INV
    assert call(rows=-1) == INV and call(d=0) == INV and call(rows=1 << 31) == UNS and call(d=(1 << 30) + 1) == UNS
    assert call(eps=-1.0) == INV and call(eps=math.nan) == INV
    assert call(x=None) == INV and call(y=None) == INV
    assert call(x=ctypes.c_void_p(4097)) == INV
    assert call(ys=255) == INV and call(ss=10) == INV and call(xs=-256) == INV
    assert call(scales=P, group=48) == INV and call(scales=P, group=128, d=200, ys=200) == INV
    assert call(rows=0) == bnd.MHA_OK          # nothing to do, nothing enqueued


def test_rmsnorm_ignores_the_sum_without_a_residual(lib):
    """Its address and stride are not looked at: what is refused is the overlap of y's rows, which comes later."""
    odd = ctypes.c_void_p(4097)
    args = (1, P, 256, None, -5, odd, -7, None, 1e-6, 4, 256, P, 255, None, 0, None)
    assert lib.mha_rmsnorm(*args) == INV and b"must not overlap" in lib.mha_last_error()


def test_binding_refuses_cpu_tensors_and_wrong_shapes(lib):
    q = torch.zeros(1, 2, 4, 64)
    for f in (lambda: bnd.mha_rotary(q, rotary=None, q_out=q), lambda: bnd.mha_attention(q, q, q, out=q),
              lambda: bnd.make_paged_cache(q, q, q), lambda: bnd.make_rotary(torch.zeros(4)),
              lambda: bnd.mha_rmsnorm(q[0, 0], None, 1e-6, y=q[0, 0]),
              lambda: bnd.mha_document_spans(torch.zeros(1, 4, dtype=torch.int32), spans=None)):
        with pytest.raises((ValueError, TypeError, RuntimeError, AssertionError)):
            f()


def _plain(r, base):
    return [base ** (-2.0 * i / r) for i in range(r // 2)]


@pytest.mark.parametrize("r,base", [(2, 10000.0), (64, 10000.0), (128, 500000.0)])
def test_frequencies_plain_linear_and_stretched_base(lib, r, base):
    """Each entry is the definition in fp64 rounded once: half a step of fp32, and pow's last digits."""
    plain = _plain(r, base)
    f, s = bnd.rotary_frequencies(r, base)
    assert s == 1.0 and f.shape == (r // 2,)
    for got, want in zip(f.tolist(), plain):
        assert abs(got - want) <= 2.0 ** -23 * want
    f, s = bnd.rotary_frequencies(r, base, bnd.ROPE_LINEAR, 4.0)
    for got, want in zip(f.tolist(), plain):
        assert abs(got - want / 4) <= 2.0 ** -23 * want
    if r > 2:
        f, s = bnd.rotary_frequencies(r, base, bnd.ROPE_BASE, 8.0)
        for got, want in zip(f.tolist(), _plain(r, base * 8.0 ** (r / (r - 2)))):
            assert abs(got - want) <= 2.0 ** -23 * want
        # the slowest pair turns 8 times slower, the fastest as before
        assert f[0] == 1.0 and abs(f[-1].item() * 8 / plain[-1] - 1) <= 2.0 ** -20


def test_frequencies_banded_and_ramp(lib):
    r, base, factor, length, low, high = 128, 10000.0, 8.0, 8192.0, 1.0, 4.0
    plain = _plain(r, base)
    f, s = bnd.rotary_frequencies(r, base, bnd.ROPE_BANDED, factor, length, low, high)
    assert s == 1.0
    kinds = set()
    for got, want in zip(f.tolist(), plain):
        w = 2 * math.pi / want
        if w < length / high:
            ref, kind = want, "kept"
        elif w > length / low:
            ref, kind = want / factor, "divided"
        else:
            t = (length / w - low) / (high - low)
            ref, kind = (1 - t) * want / factor + t * want, "blend"
        kinds.add(kind)
        assert abs(got - ref) <= 2.0 ** -22 * ref
    assert kinds == {"kept", "divided", "blend"}
    low, high = 1.0, 32.0
    f, s = bnd.rotary_frequencies(r, base, bnd.ROPE_RAMP, factor, length, low, high)
    assert abs(s - (0.1 * math.log(factor) + 1)) <= 1e-6
    at = lambda n: r * math.log(length / (n * 2 * math.pi)) / (2 * math.log(base))
    i0, i1 = max(math.floor(at(high)), 0), min(math.ceil(at(low)), r // 2 - 1)
    assert 0 < i0 < i1 < r // 2 - 1
    for i, (got, want) in enumerate(zip(f.tolist(), plain)):
        t = min(max((i - i0) / (i1 - i0), 0.0), 1.0)
        ref = (1 - t) * want + t * want / factor
        assert abs(got - ref) <= 2.0 ** -22 * ref


@pytest.mark.parametrize("r,base,factor,length,low,high", [
    (64, 10000.0, 8.0, 131072.0, 1.0, 32.0), (64, 10000.0, 4.0, 65536.0, 1.0, 32.0), (128, 10000.0, 4.0, 131072.0, 1.0, 32.0),
    (64, 10000.0, 4.0, 1e9, 1.0, 32.0), (64, 10000.0, 4.0, 1e12, 1.0, 32.0), (32, 500000.0, 16.0, 8192.0, 1.0, 32.0),
    (64, 10000.0, 2.0, 20.0, 1.0, 4.0)])
def test_ramp_ends_where_the_slowest_pair_still_turns(lib, r, base, factor, length, low, high):
    """The pairs that turn `high` and `low` times over the length, rounded outwards and limited to 0 .. r - 1: beyond the table
    (which ends at r / 2 - 1) where its slowest pair turns more often than `low` times."""
    f, s = bnd.rotary_frequencies(r, base, bnd.ROPE_RAMP, factor, length, low, high)
    at = lambda n: r * math.log(length / (n * 2 * math.pi)) / (2 * math.log(base))
    i0, i1 = max(math.floor(at(high)), 0), min(math.ceil(at(low)), r - 1)
    for i, (got, want) in enumerate(zip(f.tolist(), _plain(r, base))):
        t = min(max((i - i0) / max(i1 - i0, 1e-3), 0.0), 1.0)
        ref = (1 - t) * want + t * want / factor
        assert abs(got - ref) <= 2.0 ** -22 * ref


def test_frequencies_refusals(lib):
    for args in ((63,), (0,), (64, 1.0), (64, math.nan), (64, 1e4, 7), (64, 1e4, bnd.ROPE_LINEAR, 0.5),
                 (2, 1e4, bnd.ROPE_BASE, 2.0), (64, 1e4, bnd.ROPE_BANDED, 2.0, 0.0),
                 (64, 1e4, bnd.ROPE_RAMP, 2.0, 4096.0, 4.0, 1.0)):
        with pytest.raises(bnd.MHAError) as e:
            bnd.rotary_frequencies(*args)
        assert e.value.status == INV


def test_native_front_declines_what_is_no_call():
    """The native front on CPU tensors and other objects: False, and nothing done; bad addresses are refused."""
    torch = pytest.importorskip("torch")
    from transformer_head_scaled_fwd_gb300 import build as B
    if B.build_front() is None:
        pytest.skip("the headers of Python or torch are missing")
    from transformer_head_scaled_fwd_gb300 import _front as front
    x = torch.zeros(2, 3, 4, 64)
    for name, n in (("rotary", 7), ("paged_append", 10), ("paged_attention", 7), ("document_spans", 3), ("attention", 7),
                    ("rmsnorm", 8)):
        f = getattr(front, name)
        assert f() is False and f(*[None] * n) is False and f(*[x] * n) is False and f(*[1.5] * n) is False
        assert f(*[x] * (n + 1)) is False
    with pytest.raises(TypeError):
        front.set_library(1)
    with pytest.raises(ValueError):
        front.set_library(0, 0, 0, 0, 0, 0)
    with pytest.raises(TypeError):
        front.set_library(*["x"] * 6)


def test_a_front_that_does_not_compile_is_left_out(tmp_path, monkeypatch, capsys):
    """_front.so is optional: where g++ fails on it (a torch without CUDA, say) there is a message, no exception, and no
    module of an earlier build."""
    torch = pytest.importorskip("torch")
    if B.build_front() is None:
        pytest.skip("the headers of Python or torch are missing")
    bad = tmp_path / "front.cpp"
    bad.write_text("#include <c10/no_such_header.h>\n")
    for name, path in (("FRONT_SRC", bad), ("FRONT", tmp_path / "_front.so"), ("BUILD", tmp_path / "_build")):
        monkeypatch.setattr(B, name, str(path))
    (tmp_path / "_front.so").write_bytes(b"of an earlier build")
    assert B.build_front() is None
    assert "no_such_header" in capsys.readouterr().err
    assert not (tmp_path / "_front.so").exists()
    lib = B.LIB
    assert B.build() == lib and os.path.exists(lib)
