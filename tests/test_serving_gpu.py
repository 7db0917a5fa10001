"""Serving operators on the GPU against plain 64-bit forms (tests/serving_ref.py)."""
import math
import random
import struct

import pytest

torch = pytest.importorskip("torch")

import serving_ref as R  # noqa: E402

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32
E4M3 = torch.float8_e4m3fn


@pytest.fixture(scope="module")
def bnd():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from transformer_head_scaled_fwd_gb300 import build as B
    B.build()
    from transformer_head_scaled_fwd_gb300 import binding
    binding.load()
    binding.mha_check_device_status(reset=True)
    return binding


@pytest.fixture(autouse=True)
def clean_status(request):
    yield
    if torch.cuda.is_available():
        from transformer_head_scaled_fwd_gb300 import binding
        assert binding.mha_check_device_status(reset=True) == 0


def randn(seed, *shape, dtype=F32):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return torch.randn(shape, generator=g, device="cuda").to(dtype)


def ints(values):
    return torch.tensor(values, dtype=torch.int32, device="cuda")


def freqs(r, base=10000.0):
    return (base ** (-torch.arange(0, r, 2, dtype=torch.float64) / r)).float().cuda()


# ------------------------------------------------------------------------------------------ rotary
ROTARY = [
    # dtype, B, T, h, h_kv, d, rot, interleaved, first position
    (BF, 1, 1, 1, 1, 64, 64, False, 0),
    (BF, 2, 37, 4, 2, 64, 64, False, 5),
    (BF, 2, 37, 4, 2, 64, 64, True, 5),
    (BF, 1, 130, 3, 1, 128, 32, False, 100000),
    (BF, 1, 130, 3, 1, 128, 32, True, 100000),
    (BF, 3, 5, 5, 5, 80, 20, False, 17),         # halves of 10: no 16-byte chunks
    (BF, 3, 5, 2, 1, 72, 72, True, 17),
    (BF, 1, 9, 2, 2, 33, 6, False, 3),           # odd head width
    (F32, 2, 19, 4, 4, 64, 64, False, 1500000),
    (F32, 2, 19, 4, 2, 64, 64, True, 1500000),
    (F32, 1, 7, 1, 3, 128, 96, False, 123456789),
    (F32, 1, 7, 2, 1, 5, 2, True, 9),
    (F32, 1, 3, 2, 1, 256, 256, False, 0),
    # halves of odd length beside wide heads
    (BF, 2, 37, 5, 2, 64, 14, False, 9), (BF, 2, 19, 6, 2, 128, 126, False, 500), (BF, 1, 301, 3, 1, 512, 510, False, 3),
    (F32, 1, 21, 3, 3, 64, 10, False, 4), (F32, 3, 50, 2, 1, 256, 250, False, 100000), (BF, 1, 9, 4, 1, 16, 2, False, 7),
]


@pytest.mark.parametrize("dtype,B,T,h,hk,d,rot,inter,first", ROTARY)
def test_rotary(bnd, dtype, B, T, h, hk, d, rot, inter, first):
    qkv = randn(1, B, T, h + 2 * hk, d, dtype=dtype)
    q, k = qkv[:, :, :h], qkv[:, :, h:h + hk]                                 # slices of one projection
    pos = (first + torch.arange(B * T, device="cuda").view(B, T) * 3).int()
    f = freqs(rot)
    qo, ko = torch.empty(B, h, T, d, device="cuda", dtype=dtype).transpose(1, 2), torch.empty_like(k)   # another order
    bnd.mha_rotary(q, k=k, q_out=qo, k_out=ko, positions=pos, rotary=bnd.make_rotary(f, inter, 1.25))
    for x, got in ((q, qo), (k, ko)):
        ref = R.rotate(x, pos, f, inter, 1.25)
        R.check(got, ref, R.rotate_tol(x, ref, f, inter, dtype, 1.25), "rotary")
        assert torch.equal(got[..., rot:], x[..., rot:])


def test_rotary_in_place_default_and_negative_positions(bnd):
    B, T, h, d = 2, 11, 3, 64
    f = freqs(64)
    x = randn(2, B, T, h, d, dtype=BF)
    y = x.clone()
    bnd.mha_rotary(y, q_out=y, rotary=bnd.make_rotary(f))                     # positions 0 .. T-1
    ref = R.rotate(x, torch.arange(T, device="cuda").expand(B, T), f)
    R.check(y, ref, R.rotate_tol(x, ref, f, False, BF), "in place")
    assert torch.equal(y[:, 0], x[:, 0])                                      # position 0 turns nothing
    pos = ints([[-3 - t for t in range(T)]] * B)
    z = torch.empty_like(x)
    bnd.mha_rotary(x, q_out=z, positions=pos, rotary=bnd.make_rotary(f))
    ref = R.rotate(x, pos, f)
    R.check(z, ref, R.rotate_tol(x, ref, f, False, BF), "negative positions")


@pytest.mark.parametrize("dtype,d,rot", [(BF, 64, 22), (BF, 128, 126), (F32, 64, 6)])
def test_rotary_in_place_with_odd_halves(bnd, dtype, d, rot):
    x = randn(3, 3, 200, 6, d, dtype=dtype)
    y, z = x.clone(), torch.empty_like(x)
    r = bnd.make_rotary(freqs(rot))
    bnd.mha_rotary(y, q_out=y, rotary=r)
    bnd.mha_rotary(x, q_out=z, rotary=r)
    assert torch.equal(y, z) and not torch.equal(x, z)
    narrow = torch.empty(3, 200, 6, d + 1, device="cuda", dtype=dtype)[..., 1:]      # the same bits an element an access
    bnd.mha_rotary(x, q_out=narrow, rotary=r)
    assert torch.equal(narrow, z)


def test_rotary_unaligned_views(bnd):
    """Heads that start at an odd element (no 16-byte access) and a broadcast query."""
    B, T, h, d = 2, 6, 2, 64
    f = freqs(64)
    base = randn(3, B, T, h, d + 1, dtype=BF)
    x = base[..., 1:]
    y = torch.zeros(B, T, h, d + 3, device="cuda", dtype=BF)[..., 2:-1]
    bnd.mha_rotary(x, q_out=y, rotary=bnd.make_rotary(f))
    pos = torch.arange(T, device="cuda").expand(B, T)
    ref = R.rotate(x, pos, f)
    R.check(y, ref, R.rotate_tol(x, ref, f, False, BF), "odd start")
    one = randn(4, 1, 1, 1, d, dtype=BF).expand(B, T, h, d)
    out = torch.empty(B, T, h, d, device="cuda", dtype=BF)
    bnd.mha_rotary(one, q_out=out, rotary=bnd.make_rotary(f))
    ref = R.rotate(one, pos, f)
    R.check(out, ref, R.rotate_tol(one, ref, f, False, BF), "broadcast")


# ------------------------------------------------------------------------------------------ paged cache
def pages_of(seed, n_pages, page, hk, d, dtype, order="slots"):
    """Pages [n_pages, page, hk, d]; order "heads": stored head by head inside a page."""
    if order == "slots":
        return randn(seed, n_pages, page, hk, d, dtype=dtype), randn(seed + 1, n_pages, page, hk, d, dtype=dtype)
    return (randn(seed, n_pages, hk, page, d, dtype=dtype).transpose(1, 2),
            randn(seed + 1, n_pages, hk, page, d, dtype=dtype).transpose(1, 2))


def table_of(seed, B, per, extra=3):
    ids = list(range(B * per + extra))
    random.Random(seed).shuffle(ids)
    return ints([ids[b * per:(b + 1) * per] for b in range(B)]), B * per + extra


APPEND = [
    # dtype, T, h, h_kv, d, rot, interleaved, page, order, starts, new_lens
    (BF, 1, 4, 2, 64, 64, False, 16, "slots", [0, 15, 16], None),
    (BF, 1, 8, 1, 128, 64, True, 1, "slots", [3, 0, 7], [1, 0, 1]),
    (BF, 40, 4, 4, 64, 32, False, 24, "heads", [0, 23, 50], [40, 0, 17]),
    (BF, 33, 2, 2, 128, 128, True, 64, "heads", [60, 64, 1], None),
    (F32, 21, 3, 1, 64, 64, False, 8, "slots", [5, 0, 90], [21, 1, 20]),
    (F32, 5, 2, 2, 20, 6, True, 7, "slots", [5, 0, 9], [5, -2, 9]),      # lengths beyond T and below 0
    (BF, 33, 5, 2, 64, 22, False, 8, "heads", [0, 23, 50], [33, 0, 17]),
    (F32, 33, 5, 2, 64, 62, False, 8, "slots", [0, 23, 50], [33, 0, 17]),
]


@pytest.mark.parametrize("dtype,T,h,hk,d,rot,inter,page,order,start,lens", APPEND)
def test_paged_append(bnd, dtype, T, h, hk, d, rot, inter, page, order, start, lens):
    B = len(start)
    per = -(-(max(start) + T) // page)
    table, n_pages = table_of(5, B, per)
    kp, vp = pages_of(6, n_pages, page, hk, d, dtype, order)
    want_k, want_v = kp.double().clone(), vp.double().clone()
    tol = torch.zeros_like(want_k)
    qkv = randn(8, B, T, h + 2 * hk, d, dtype=dtype)
    q, k, v = qkv[:, :, :h], qkv[:, :, h:h + hk], qkv[:, :, h + hk:]
    qo, ko = randn(9, B, T, h, d, dtype=dtype), randn(10, B, T, hk, d, dtype=dtype)
    q0, k0 = qo.clone(), ko.clone()
    f = freqs(rot)
    bnd.mha_paged_append(k, v, ints(start), cache=bnd.make_paged_cache(kp, vp, table), q=q, q_out=qo, k_out=ko,
                         new_lens=None if lens is None else ints(lens), rotary=bnd.make_rotary(f, inter))
    pos = ints(start)[:, None] + torch.arange(T, device="cuda")
    qr, kr = R.rotate(q, pos, f, inter), R.rotate(k, pos, f, inter)
    kt = R.rotate_tol(k, kr, f, inter, dtype)
    for b in range(B):
        n = T if lens is None else min(max(lens[b], 0), T)
        for t in range(n):
            at = start[b] + t
            pg, slot = table[b, at // page].item(), at % page
            want_k[pg, slot], want_v[pg, slot], tol[pg, slot] = kr[b, t], v[b, t].double(), kt[b, t]
        R.check(qo[b, :n], qr[b, :n], R.rotate_tol(q, qr, f, inter, dtype)[b, :n], "q")
        R.check(ko[b, :n], kr[b, :n], kt[b, :n], "k")
        assert torch.equal(qo[b, n:], q0[b, n:]) and torch.equal(ko[b, n:], k0[b, n:])   # left as they were
    R.check(kp, want_k, tol, "k pages")              # zero tolerance where nothing was written
    assert torch.equal(vp.double(), want_v)


def test_append_without_queries_or_rotation(bnd):
    B, T, hk, d, page = 2, 9, 2, 64, 4
    table, n_pages = table_of(1, B, 3)
    kp, vp = pages_of(2, n_pages, page, hk, d, BF)
    k, v = randn(3, B, T, hk, d, dtype=BF), randn(4, B, T, hk, d, dtype=BF)
    bnd.mha_paged_append(k, v, ints([0, 3]), cache=bnd.make_paged_cache(kp, vp, table))
    for b, s in enumerate([0, 3]):
        rows = table[b].long()
        assert torch.equal(kp[rows].flatten(0, 1)[s:s + T], k[b]) and torch.equal(vp[rows].flatten(0, 1)[s:s + T], v[b])


def test_append_never_follows_a_bad_page(bnd):
    """Page numbers outside the pool, and positions beyond the table or below 0: skipped and reported."""
    B, T, hk, d, page = 4, 4, 1, 64, 4
    table = ints([[0, 1], [-1, 2], [99, 3], [4, 5]])
    kp, vp = pages_of(2, 6, page, hk, d, BF)
    k0, v0 = kp.clone(), vp.clone()
    k, v = randn(3, B, T, hk, d, dtype=BF), randn(4, B, T, hk, d, dtype=BF)
    bnd.mha_paged_append(k, v, ints([6, 0, 2, -2]), cache=bnd.make_paged_cache(kp, vp, table))
    assert bnd.mha_check_device_status(reset=True) == bnd.MHA_PAGED_BAD_PAGE
    k0[1, 2:], v0[1, 2:] = k[0, :2, :], v[0, :2, :]            # positions 6, 7; 8, 9 lie beyond the table
    k0[3, :2], v0[3, :2] = k[2, 2:, :], v[2, 2:, :]            # positions 4, 5; 2, 3 are on page 99
    k0[4, :2], v0[4, :2] = k[3, 2:, :], v[3, 2:, :]            # positions 0, 1; -2, -1 do not exist
    assert torch.equal(kp, k0) and torch.equal(vp, v0)


# ------------------------------------------------------------------------------------------ paged attention
def paged_ref(q, kp, vp, table, lens, hk, *, cap=0.0, slopes=None, scale=None, bad=()):
    """(reference, tolerance); positions in `bad` (sequence, position) are left out."""
    B, h, d = q.shape
    page = kp.shape[1]
    ref = torch.zeros(B, h, d, dtype=torch.float64, device="cuda")
    tol = torch.full_like(ref, 1e-30)
    for b in range(B):
        n = max(lens[b], 0)
        if n == 0:
            continue
        rows = table[b, : -(-n // page)].long().clamp(0, kp.shape[0] - 1)
        pos = torch.arange(n, device="cuda")
        ok = torch.ones(1, n, dtype=torch.bool, device="cuda")
        for bb, j in bad:
            if bb == b and j < n:
                ok[0, j] = False
        for i in range(h):
            k = kp[rows, :, i // (h // hk)].flatten(0, 1)[:n]
            v = vp[rows, :, i // (h // hk)].flatten(0, 1)[:n]
            slope = slopes[i].item() if slopes is not None else 0.0
            o, mag, size = R.attend(q[b, i:i + 1], k, v, ok, (n - 1 - pos)[None].double(),
                                    scale=d ** -0.5 if scale is None else scale, cap=cap, slope=slope)
            ref[b, i] = o[0]
            tol[b, i] = R.attend_tol(o, mag, size, n, d, q.dtype, cap=cap, far=abs(slope) * n)[0]
    return ref, tol


def slopes_of(h):
    return torch.tensor([2.0 ** (-8.0 * (i + 1) / h) for i in range(h)], device="cuda")


def run_paged(bnd, q, kp, vp, table, lens, hk, out=None, **scores):
    B, h, d = q.shape
    dt = bnd.MHA_BF16 if q.dtype == BF else bnd.MHA_F32
    ws = torch.full((bnd.paged_attention_workspace_size(dt, B, h, hk, d),), 0xff, dtype=torch.uint8, device="cuda")   # NaN
    out = torch.full_like(q, float("nan")) if out is None else out
    bnd.mha_paged_attention(q, ints(lens), cache=bnd.make_paged_cache(kp, vp, table), out=out, workspace=ws,
                            scores=bnd.make_scores(**scores) if scores else None)
    return out


def poison(kp, vp, table, lens):
    """NaN and infinities in every slot that no sequence holds."""
    page = kp.shape[1]
    keep = torch.zeros(kp.shape[0], page, dtype=torch.bool, device="cuda")
    for b, n in enumerate(lens):
        for j in range(max(n, 0)):
            keep[table[b, j // page], j % page] = True
    kp[~keep] = float("nan")
    vp[~keep] = float("inf")


PAGED = [
    # dtype, h, h_kv, d, page, order, lens, scores
    (BF, 4, 4, 64, 16, "slots", [1, 0, 15, 16, 17, 100], {}),
    (BF, 8, 2, 64, 16, "heads", [33, 1, 0, 640], {}),
    (BF, 8, 1, 128, 64, "slots", [63, 64, 65, 500], dict(cap=20.0)),
    (BF, 6, 2, 128, 24, "slots", [777, 24, 25], dict(slopes=True)),
    (BF, 10, 2, 64, 1, "slots", [130, 5], dict(cap=5.0, slopes=True)),
    (BF, 16, 1, 128, 7, "heads", [300, 29], dict(scale=0.3)),
    (BF, 20, 1, 64, 32, "slots", [257, 31, 1], dict(slopes=True)),        # more than 16 heads share a key head
    (BF, 64, 1, 128, 128, "slots", [129], {}),
    (BF, 33, 11, 64, 100, "slots", [201, 99, 100, 0], {}),
    (BF, 7, 7, 128, 16, "slots", [2000, 3], {}),
    (BF, 8, 2, 64, 16, "slots", [300, 0, 256, 257, 1, 700, 512, 768, 513, 2, 900], {}),      # units of 0 to 4 blocks
    (BF, 12, 12, 128, 32, "slots", [448, 129, 128, 127] * 20, {}),                              # more units than SMs
    (F32, 4, 4, 64, 16, "slots", [1, 0, 15, 16, 17, 100], {}),
    (F32, 8, 2, 128, 24, "heads", [333, 1, 48], dict(cap=15.0)),
    (F32, 9, 3, 64, 1, "slots", [66, 2], dict(slopes=True)),
    (F32, 20, 1, 128, 32, "slots", [257, 1], dict(scale=-0.2)),
]


@pytest.mark.parametrize("dtype,h,hk,d,page,order,lens,sc", PAGED)
def test_paged_attention(bnd, dtype, h, hk, d, page, order, lens, sc):
    B = len(lens)
    per = -(-max(lens) // page) + 1
    table, n_pages = table_of(11, B, per)
    kp, vp = pages_of(12, n_pages, page, hk, d, dtype, order)
    poison(kp, vp, table, lens)
    q = randn(14, h, B, d, dtype=dtype).transpose(0, 1) * 2.0           # strides of [h, B, d]
    sc = dict(sc)
    if sc.get("slopes"):
        sc["slopes"] = slopes_of(h)
    got = run_paged(bnd, q, kp, vp, table, lens, hk, **sc)
    ref, tol = paged_ref(q, kp, vp, table, lens, hk, **sc)
    R.check(got, ref, tol, "paged attention")
    again = run_paged(bnd, q, kp, vp, table, lens, hk, **sc)
    assert torch.equal(got, again)                                      # does not depend on timing
    for b, n in enumerate(lens):
        if n <= 0:
            assert torch.equal(got[b], torch.zeros_like(got[b]))


@pytest.mark.parametrize("dtype,B,h,hk,d,n", [(BF, 1, 16, 2, 128, 70001), (BF, 2, 4, 4, 64, 30000),
                                              (F32, 1, 4, 1, 64, 40001), (BF, 70, 4, 2, 64, 900)])
def test_paged_attention_long_and_many(bnd, dtype, B, h, hk, d, n):
    """Lengths that are split over the GPU and joined, and a batch of very different ones."""
    rng = random.Random(3)
    lens = [n] + [rng.choice([0, 1, n // 100, n // 3, n]) for _ in range(B - 1)]
    table, n_pages = table_of(15, B, -(-n // 64))
    kp, vp = pages_of(16, n_pages, 64, hk, d, dtype)
    q = randn(18, B, h, d, dtype=dtype) * 3.0
    got = run_paged(bnd, q, kp, vp, table, lens, hk)
    ref, tol = paged_ref(q, kp, vp, table, lens, hk)
    R.check(got, ref, tol, "long")


def test_paged_attention_large_scores_and_shared_pages(bnd):
    """Scores in the thousands (one key carries everything, the running maximum moves), and sequences that
    share their first pages."""
    h, hk, d, page = 4, 2, 64, 16
    table = ints([[0, 1, 2, 3], [0, 1, 4, 5], [0, 1, 2, 6]])
    kp, vp = pages_of(20, 7, page, hk, d, BF)
    q = randn(22, 3, h, d, dtype=BF) * 100.0
    lens = [64, 50, 33]
    got = run_paged(bnd, q, kp, vp, table, lens, hk)
    ref, tol = paged_ref(q, kp, vp, table, lens, hk)
    R.check(got, ref, tol, "large scores")


@pytest.mark.parametrize("dtype", [BF, F32])
def test_paged_attention_never_follows_a_bad_page(bnd, dtype):
    """A page outside the pool is left out; a length beyond the table is cut to it. Both are reported."""
    h, hk, d, page = 4, 2, 64, 8
    table = ints([[0, -1, 2], [3, 1, 1 << 30], [4, 5, 6]])
    kp, vp = pages_of(24, 7, page, hk, d, dtype)
    q = randn(26, 3, h, d, dtype=dtype)
    got = run_paged(bnd, q, kp, vp, table, [20, 24, 1000], hk)
    assert bnd.mha_check_device_status(reset=True) == bnd.MHA_PAGED_BAD_PAGE
    bad = [(0, j) for j in range(8, 16)] + [(1, j) for j in range(16, 24)]
    ref, tol = paged_ref(q, kp, vp, table, [20, 24, 24], hk, bad=bad)
    R.check(got, ref, tol, "bad pages")


def test_paged_attention_offsets_beyond_32_bits(bnd):
    """Pages whose element offsets pass 2^31 and 2^32."""
    hk, d, page = 8, 128, 64
    per_page = page * hk * d
    n_pages = (1 << 32) // per_page + 8
    kp = torch.zeros(n_pages, page, hk, d, device="cuda", dtype=BF)
    vp = torch.zeros(n_pages, page, hk, d, device="cuda", dtype=BF)
    far = [n_pages - 1, (1 << 31) // per_page, 1, (1 << 32) // per_page]
    for i, pg in enumerate(far):
        kp[pg], vp[pg] = randn(30 + i, page, hk, d, dtype=BF), randn(40 + i, page, hk, d, dtype=BF)
    table = ints([far])
    q = randn(50, 1, 16, d, dtype=BF)
    got = run_paged(bnd, q, kp, vp, table, [250], hk)
    ref, tol = paged_ref(q, kp, vp, table, [250], hk)
    R.check(got, ref, tol, "far pages")
    k, v = randn(51, 1, 2, hk, d, dtype=BF), randn(52, 1, 2, hk, d, dtype=BF)
    bnd.mha_paged_append(k, v, ints([254]), cache=bnd.make_paged_cache(kp, vp, table))
    assert torch.equal(kp[far[3], 62:], k[0]) and torch.equal(vp[far[3], 62:], v[0])


# ------------------------------------------------------------------------------------------ attention
def attention_ref(q, k, v, *, scale=None, cap=0.0, slopes=None, causal=False, q_offset=0, valid=None, prefix=None,
                  docs=None, spans=None):
    B, Lq, h, d = q.shape
    Lk, hk = k.shape[1], k.shape[2]
    ref = torch.zeros(B, Lq, h, d, dtype=torch.float64, device="cuda")
    tol = torch.full_like(ref, 1e-30)
    i, j = torch.arange(Lq, device="cuda")[:, None] + q_offset, torch.arange(Lk, device="cuda")[None]
    for b in range(B):
        ok = torch.ones(Lq, Lk, dtype=torch.bool, device="cuda")
        if causal:
            ok &= (j <= i) | (j < (prefix[b] if prefix is not None else 0))
        if valid is not None:
            ok &= j < valid[b]
        if docs is not None:
            ok &= (docs[b][:, None] == docs[b][None]) & (docs[b] >= 0)[:, None]
        if spans is not None:
            ok &= (j >= spans[b, :, :1]) & (j < spans[b, :, 1:])
        for n in range(h):
            slope = slopes[n].item() if slopes is not None else 0.0
            o, mag, size = R.attend(q[b, :, n], k[b, :, n // (h // hk)], v[b, :, n // (h // hk)], ok, (i - j).abs().double(),
                                    scale=d ** -0.5 if scale is None else scale, cap=cap, slope=slope)
            ref[b, :, n] = o
            tol[b, :, n] = R.attend_tol(o, mag, size, Lk, d, q.dtype, cap=cap, far=abs(slope) * (Lk + q_offset + Lq))
    return ref, tol


def docs_of(seed, B, L, mean, pad=0):
    rng, rows = random.Random(seed), []
    for _ in range(B):
        row, n = [], 0
        while len(row) < L:
            row += [n] * max(1, int(rng.expovariate(1.0 / mean)))
            n += 1
        row = row[:L]
        for t in range(pad):
            row[L - 1 - t] = -1
        rows.append(row)
    return ints(rows)


ATT = [
    # B, Lq, Lk, h, h_kv, d, options
    (1, 1, 1, 1, 1, 64, {}),
    (2, 1, 300, 4, 2, 128, dict(causal=True, q_offset=299)),
    (2, 77, 77, 4, 4, 64, dict(causal=True)),
    (2, 130, 130, 6, 2, 128, dict(causal=True, cap=8.0)),
    (1, 257, 257, 2, 1, 64, dict(slopes=True)),
    (1, 200, 333, 3, 1, 128, dict(causal=True, q_offset=133, slopes=True, cap=30.0)),
    (3, 255, 333, 4, 4, 64, dict(causal=True, q_offset=78, prefix=[0, 100, 333], valid=[333, 90, 0])),
    (2, 300, 300, 2, 2, 128, dict(docs=40, causal=True)),
    (2, 300, 300, 2, 2, 64, dict(docs=40)),
    (2, 513, 513, 2, 1, 128, dict(docs=150, causal=True, prefix=[64, 400], pad=70)),
    (2, 512, 512, 2, 2, 64, dict(valid=[1, 129])),
    (1, 128, 1000, 2, 1, 128, dict(scale=0.02)),
    (2, 640, 640, 5, 5, 64, dict(causal=True, cap=50.0, valid=[640, 320])),
    (1, 100, 40, 2, 2, 64, dict(causal=True)),            # more queries than keys: the last rows see all
    (1, 65, 129, 16, 2, 128, dict(causal=True, q_offset=500)),     # all queries behind all keys
    (1, 130, 700, 4, 2, 128, dict(causal=True, q_offset=570, cap=10.0, valid=[650])),
    (2, 600, 600, 2, 1, 128, dict(docs=20, causal=True, cap=30.0)),
    (1, 600, 600, 2, 1, 64, dict(cap=59.0)),
    (2, 700, 700, 3, 3, 64, dict(docs=60, pad=300)),                # whole query tiles without a key
    (60, 300, 300, 8, 4, 64, dict(valid=[0, 300, 0, 0] * 15, causal=True)),     # many units without a key
    (3, 128, 4000, 2, 2, 64, dict(causal=True, q_offset=100, valid=[4000, 77, 0])),
    # long key ranges of d_k = 64
    (1, 1, 2000, 2, 1, 64, {}),
    (2, 300, 1800, 4, 2, 64, dict(causal=True, q_offset=1500, slopes=True)),
    (2, 1700, 1700, 2, 2, 64, dict(docs=300, causal=True, pad=500)),
    (2, 1700, 1700, 2, 1, 64, dict(docs=90, cap=20.0)),
    (1, 257, 2500, 2, 2, 64, dict(cap=100.0, slopes=True)),
    (30, 200, 1600, 4, 4, 64, dict(causal=True, q_offset=1400, valid=[0, 1600, 0, 0, 1, 1401] * 5)),
    (2, 1600, 1600, 2, 2, 64, dict(causal=True, prefix=[900, 0], valid=[1600, 1000])),
    (1, 600, 600, 2, 1, 64, dict(cap=300.0, causal=True)),
    # ... with more tiles of 128 queries than SMs
    (3, 300, 1800, 18, 6, 64, dict(causal=True, q_offset=1500, slopes=True)),
    (2, 1700, 1700, 6, 2, 64, dict(docs=300, causal=True, pad=500)),
    (2, 1700, 1700, 6, 3, 64, dict(docs=90, cap=20.0)),
    (4, 257, 1537, 13, 1, 64, dict(cap=100.0, slopes=True, valid=[1537, 0, 700, 1536])),
    (2, 1600, 1600, 6, 6, 64, dict(causal=True, prefix=[900, 0], valid=[1600, 1000])),
    # few queries, long keys: several CTAs share a query tile
    (1, 1, 8192, 4, 1, 128, dict(causal=True, q_offset=8191)),
    (2, 3, 4100, 2, 2, 64, dict(causal=True, q_offset=4097, slopes=True)),
    (1, 130, 5000, 3, 1, 128, dict(causal=True, q_offset=4870, cap=30.0)),
    (3, 40, 3000, 2, 1, 64, dict(valid=[0, 100, 3000], cap=50.0)),       # pieces, and whole units, without a key
    (2, 129, 2100, 4, 2, 128, dict(causal=True, q_offset=60, valid=[2100, 70], prefix=[0, 1500])),
    (1, 1100, 1100, 2, 1, 64, dict(docs=300, causal=True, pad=200)),
    (1, 2048, 2048, 1, 1, 128, dict(causal=True, slopes=True, cap=100.0)),
    (20, 17, 1030, 2, 1, 128, dict(causal=True, q_offset=900, valid=[0, 1, 128, 129, 512, 513, 900, 917, 918, 1030] * 2)),
]


def run_attention(bnd, q, k, v, out=None, **o):
    scores = {n: o[n] for n in ("scale", "cap", "slopes") if n in o}
    spans = o.get("spans")
    if o.get("docs") is not None:
        spans = torch.empty(*o["docs"].shape, 2, dtype=torch.int32, device="cuda")
        bnd.mha_document_spans(o["docs"], spans=spans)
    mask = bnd.make_span_mask(causal=o.get("causal", False), q_offset=o.get("q_offset", 0),
                              key_valid_lens=None if o.get("valid") is None else ints(o["valid"]),
                              prefix_lens=None if o.get("prefix") is None else ints(o["prefix"]), doc_spans=spans)
    out = torch.full(q.shape, float("nan"), dtype=q.dtype, device="cuda") if out is None else out
    bnd.mha_attention(q, k, v, out=out, mask=mask, scores=bnd.make_scores(**scores) if scores else None)
    return out


@pytest.mark.parametrize("B,Lq,Lk,h,hk,d,opt", ATT)
def test_attention(bnd, B, Lq, Lk, h, hk, d, opt):
    opt = dict(opt)
    pad = opt.pop("pad", 0)
    if opt.get("slopes"):
        opt["slopes"] = slopes_of(h)
    if opt.get("docs"):
        opt["docs"] = docs_of(60, B, Lk, opt["docs"], pad)
    q, kv = randn(61, B, Lq, h, d, dtype=BF) * 1.5, randn(62, B, Lk, 2 * hk, d, dtype=BF)
    k, v = kv[:, :, :hk], kv[:, :, hk:]
    if opt.get("valid"):
        for b, n in enumerate(opt["valid"]):
            k[b, n:], v[b, n:] = float("nan"), float("inf")        # padding holds anything
    got = run_attention(bnd, q, k, v, **opt)
    ref, tol = attention_ref(q, k, v, **opt)
    R.check(got, ref, tol, "attention")
    assert torch.equal(got, run_attention(bnd, q, k, v, **opt))


@pytest.mark.parametrize("B,Lq,Lk,h,hk,d,opt", ATT)
def test_attention_fp32(bnd, B, Lq, Lk, h, hk, d, opt):
    opt = dict(opt)
    pad = opt.pop("pad", 0)
    if opt.get("slopes"):
        opt["slopes"] = slopes_of(h)
    if opt.get("docs"):
        opt["docs"] = docs_of(64, B, Lk, opt["docs"], pad)
    q, kv = randn(65, B, Lq, h, d) * 1.5, randn(66, B, Lk, 2 * hk, d)
    k, v = kv[:, :, :hk], kv[:, :, hk:]
    if opt.get("valid"):
        for b, n in enumerate(opt["valid"]):
            k[b, n:], v[b, n:] = float("nan"), float("inf")
    got = run_attention(bnd, q, k, v, **opt)
    ref, tol = attention_ref(q, k, v, **opt)
    R.check(got, ref, tol, "attention, fp32")
    assert torch.equal(got, run_attention(bnd, q, k, v, **opt))


@pytest.mark.parametrize("d", [64, 128])
def test_attention_fp32_strides_and_spans(bnd, d):
    """Head-major storage, a shared query (stride 0), a key at a 16-byte start inside wider rows, an output inside a wider
    tensor, arbitrary spans."""
    B, L, h, hk = 2, 150, 4, 2
    q = randn(67, B, L, 1, d).expand(B, L, h, d)
    k = randn(68, B, L, hk, d + 8)[..., 4:d + 4]
    v = randn(69, 1, hk, L, d).transpose(1, 2).expand(B, L, hk, d)
    rng = random.Random(9)
    spans = ints([[[rng.randint(-20, L), rng.randint(-20, L + 20)] for _ in range(L)] for _ in range(B)])
    wide = torch.full((B, L, h + 3, d), 7.0, device="cuda")
    got = run_attention(bnd, q, k, v, out=wide[:, :, 1:h + 1], spans=spans, scale=0.3)
    ref, tol = attention_ref(q, k, v, spans=spans, scale=0.3)
    R.check(got, ref, tol, "spans")
    assert (wide[:, :, 0] == 7).all() and (wide[:, :, h + 1:] == 7).all()
    empty = spans[..., 0].clamp(min=0) >= spans[..., 1].clamp(max=L)
    assert empty.any() and (got[empty] == 0).all()


@pytest.mark.parametrize("d,L,h", [(64, 200, 4), (128, 200, 4), (64, 1650, 4), (64, 1650, 6)])
def test_attention_head_major_strides_and_spans(bnd, d, L, h):
    """[B, h, L, d] storage (the workspace's order), an output inside a wider tensor, arbitrary spans with
    empty and inverted rows."""
    B, hk = 2, 2
    q = randn(70, B, h, L, d, dtype=BF).transpose(1, 2)
    k, v = randn(71, B, hk, L, d, dtype=BF).transpose(1, 2), randn(72, B, hk, L, d, dtype=BF).transpose(1, 2)
    rng = random.Random(7)
    spans = ints([[[rng.randint(-20, L), rng.randint(-20, L + 20)] for _ in range(L)] for _ in range(B)])
    wide = torch.full((B, L, h + 3, d), 7.0, dtype=BF, device="cuda")
    got = run_attention(bnd, q, k, v, out=wide[:, :, 1:h + 1], spans=spans)
    ref, tol = attention_ref(q, k, v, spans=spans)
    R.check(got, ref, tol, "spans")
    assert (wide[:, :, 0] == 7).all() and (wide[:, :, h + 1:] == 7).all()
    empty = spans[..., 0].clamp(min=0) >= spans[..., 1].clamp(max=L)
    assert empty.any() and (got[empty] == 0).all()


@pytest.mark.parametrize("d,L,cap", [(64, 700, 50.0), (128, 700, 20.0), (128, 130, 50.0), (64, 1600, 0.0), (64, 2500, 0.0)])
def test_attention_rows_of_one_key_are_its_value(bnd, d, L, cap):
    """One weight divided by itself is 1 whatever it was rounded to, so the only rounding is of a bf16 value to bf16."""
    q, k, v = (randn(73 + i, 2, L, n, d, dtype=BF) for i, n in enumerate((4, 2, 2)))
    got = run_attention(bnd, q * 2, k, v, causal=True, cap=cap)
    assert torch.equal(got[:, 0], v[:, 0].repeat_interleave(2, dim=1))
    last = run_attention(bnd, q[:, :1] * 2, k, v, causal=True, cap=cap, q_offset=L, valid=[1, 1])
    assert torch.equal(last[:, 0], v[:, 0].repeat_interleave(2, dim=1))


def test_attention_broadcast_inputs(bnd):
    """Keys and values shared by all sequences, a query shared by all heads (strides of 0)."""
    B, L, h, hk, d = 3, 140, 4, 2, 64
    k, v = (randn(75 + i, 1, L, hk, d, dtype=BF).expand(B, L, hk, d) for i in range(2))
    q = randn(77, B, L, 1, d, dtype=BF).expand(B, L, h, d)
    got = run_attention(bnd, q, k, v, out=torch.empty(B, L, h, d, dtype=BF, device="cuda"), causal=True)
    ref, tol = attention_ref(q, k, v, causal=True)
    R.check(got, ref, tol, "broadcast")


def test_attention_long_causal(bnd):
    """Rows sampled from a long sequence, grouped heads, cap and bias."""
    for d, sc in ((64, dict(slopes=True)), (128, dict(cap=50.0))):
        B, L, h, hk = 1, 5000, 4, 2
        sc = {n: slopes_of(h) if n == "slopes" else x for n, x in sc.items()}
        q, k, v = (randn(80 + i, B, L, n, d, dtype=BF) for i, n in enumerate((h, hk, hk)))
        got = run_attention(bnd, q * 3, k, v, causal=True, **sc)
        for r in (0, 1, 127, 128, 129, 2500, 4095, 4096, 4999):
            ref, tol = attention_ref((q * 3)[:, r:r + 1], k[:, :r + 1], v[:, :r + 1], causal=True, q_offset=r, **sc)
            R.check(got[:, r:r + 1], ref, tol, f"row {r}")


@pytest.mark.parametrize("B,L,mean,pad", [(1, 1, 5, 0), (3, 1000, 30, 100), (2, 5003, 700, 0), (1, 1024, 1, 1), (2, 4096, 5000, 0),
                                         (1, 2048, 1024, 1024), (3, 33, 9, 2), (1, 9000, 4000, 0)])
def test_document_spans(bnd, B, L, mean, pad):
    ids = docs_of(90, B, L, mean, pad)
    spans = torch.full((B, L, 2), -5, dtype=torch.int32, device="cuda")
    bnd.mha_document_spans(ids, spans=spans)
    for b in range(B):
        row, got = ids[b].tolist(), spans[b].tolist()
        i = 0
        while i < L:
            e = i
            while e < L and row[e] == row[i]:
                e += 1
            want = [0, 0] if row[i] < 0 else [i, e]
            assert all(got[t] == want for t in range(i, e))
            i = e


# ------------------------------------------------------------------------------------------ RMS norm
def norm_ref(x, r, gain, eps):
    z = x.double() + (r.double() if r is not None else 0.0)
    y = z / torch.sqrt((z * z).mean(dim=1, keepdim=True) + eps)
    return z, y * gain.double() if gain is not None else y


def norm_tol(z, y, d, dtype):
    """Half a step; d squares summed in fp32 (d 2^-24 at most, halved by the root), sum, product and rsqrt."""
    return R.HALF[dtype] * y.abs() + (d / 2 + 8) * 2.0 ** -24 * y.abs() + 2.0 ** -24 * y.abs().amax(dim=1, keepdim=True) + 1e-38


NORM = [
    # dtype, rows, d, residual, gain
    (BF, 1, 1, False, False), (BF, 3, 7, True, True), (BF, 5, 64, True, False), (BF, 33, 1024, True, True),
    (BF, 2, 1000, False, True), (BF, 9, 4096, True, True), (BF, 4, 8192, True, True), (BF, 3, 20000, True, True),
    (BF, 3, 16384, False, True), (BF, 1, 65536, True, True), (BF, 300, 520, True, True), (BF, 700, 1024, True, True), (BF, 611, 4096, False, True), (BF, 650, 2040, True, False),
    (BF, 9, 255, True, True), (BF, 4, 2047, True, True), (BF, 3, 4095, True, True), (BF, 2, 8191, True, True),
    (F32, 1, 1, True, True), (F32, 17, 1000, True, True), (F32, 4, 2048, False, False), (F32, 3, 12292, True, True),
    (F32, 2, 4099, True, True),
    # several rows a warp
    (BF, 131, 64, True, True), (BF, 67, 128, False, True), (BF, 35, 24, True, True), (BF, 1000, 96, True, False), (F32, 77, 32, True, True),
    (F32, 41, 64, False, True), (F32, 1, 16, True, True), (BF, 77, 33, True, True), (F32, 45, 63, True, True), (BF, 9, 123, False, True),
]


@pytest.mark.parametrize("dtype,rows,d,res,gain", NORM)
def test_rmsnorm(bnd, dtype, rows, d, res, gain):
    x, r = randn(100, rows, d, dtype=dtype), randn(101, rows, d, dtype=dtype) * 2 if res else None
    g = (randn(102, d) * 0.3 + 1).to(dtype) if gain else None
    y, s = torch.full_like(x, float("nan")), torch.full_like(x, float("nan")) if res else None
    bnd.mha_rmsnorm(x, g, 1e-5, y=y, residual=r, sum_out=s)
    z, ref = norm_ref(x, r, g, 1e-5)
    R.check(y, ref, norm_tol(z, ref, d, dtype), "y")
    if res:
        R.check(s, z, R.HALF[dtype] * z.abs(), "sum")
        s2, y2 = x.clone(), torch.empty_like(x)
        bnd.mha_rmsnorm(s2, g, 1e-5, y=y2, residual=r, sum_out=s2)           # the sum over x
        assert torch.equal(y2, y) and torch.equal(s2, s)
        s3 = r.clone()
        bnd.mha_rmsnorm(x, g, 1e-5, y=y2, residual=s3, sum_out=s3)           # the sum over the residual
        assert torch.equal(y2, y) and torch.equal(s3, s)
        bnd.mha_rmsnorm(x, g, 1e-5, y=y2, residual=r)                        # no sum wanted
        assert torch.equal(y2, y)
    y3 = x.clone()
    bnd.mha_rmsnorm(y3, g, 1e-5, y=y3, residual=r)                           # y over x
    assert torch.equal(y3, y)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("rows,d,group", [(1, 64, 0), (5, 999, 0), (7, 1024, 128), (3, 4096, 64), (2, 160, 32),
                                          (40, 4096, 0), (3, 8192, 128), (2, 20000, 32), (3, 16384, 0), (2, 30000, 0),
                                          (620, 1024, 32), (615, 4096, 128), (5, 255, 0), (2, 3999, 0), (700, 64, 64),
                                          (77, 64, 32), (41, 128, 32), (99, 128, 64), (33, 128, 0), (19, 96, 32), (50, 48, 0), (77, 123, 0),
                                          (23, 256, 128), (23, 256, 64), (50, 192, 64), (13, 512, 128), (21, 384, 128)])
def test_rmsnorm_e4m3(bnd, dtype, rows, d, group):
    """The scale to fp32 rounding; each value within half a step of e4m3 (2^-4 relative; 2^-10 below the
    smallest normal, 2^-6) of y / scale, where y / scale itself is off by the fp32 error of y and the scale."""
    x, r, g = randn(110, rows, d, dtype=dtype), randn(111, rows, d, dtype=dtype), (randn(112, d) * 0.3 + 1).to(dtype)
    groups = 1 if group == 0 else d // group
    y, sc, s = torch.empty(rows, d, device="cuda", dtype=E4M3), torch.empty(rows, groups, device="cuda"), torch.empty_like(x)
    bnd.mha_rmsnorm(x, g, 1e-6, y=y, residual=r, sum_out=s, scales=sc)
    z, ref = norm_ref(x, r, g, 1e-6)
    R.check(s, z, R.HALF[dtype] * z.abs(), "sum")
    want = ref.view(rows, groups, -1).abs().amax(dim=2) / 448
    err = (d / 2 + 12) * 2.0 ** -24
    R.check(sc, want, 4 * err * want, "scales")
    v = ref / want.repeat_interleave(d // groups, dim=1)
    R.check(y.float(), v, 2.0 ** -4 * v.abs() * (1 + 16 * err) + 2.0 ** -10 + 16 * err * v.abs(), "y")
    assert y.float().abs().amax().item() == 448.0


def test_rmsnorm_strides_and_zero_rows(bnd):
    rows, d = 6, 512
    base = randn(120, rows, 3, d, dtype=BF)
    x, r = base[:, 0], base[:, 2]                                     # rows 3 d apart
    g = randn(121, d, dtype=BF)
    wide = torch.full((rows, 2, d), 3.0, dtype=BF, device="cuda")
    bnd.mha_rmsnorm(x, g, 1e-6, y=wide[:, 1], residual=r, sum_out=None)
    z, ref = norm_ref(x, r, g, 1e-6)
    R.check(wide[:, 1], ref, norm_tol(z, ref, d, BF), "strided")
    assert (wide[:, 0] == 3).all()
    odd = randn(122, rows * (d + 1) + 1, dtype=BF)[1:].view(rows, d + 1)[:, :d]      # rows start anywhere
    y = torch.empty(rows, d, dtype=BF, device="cuda")
    bnd.mha_rmsnorm(odd, g, 1e-6, y=y)
    z, ref = norm_ref(odd, None, g, 1e-6)
    R.check(y, ref, norm_tol(z, ref, d, BF), "unaligned")
    for dt in (BF, F32):                                              # every start within a 16-byte piece, odd lengths
        for first in range(9):
            for n in (1, 3, 9, 700, 1023, 5001):
                a = randn(500 + first, 3 * n + first, dtype=dt)[first:].view(3, n)
                b = randn(510 + first, 3 * n + first, dtype=dt)[first:].view(3, n)
                outs = [torch.full((3 * n + first + 9,), 5.0, dtype=dt, device="cuda") for _ in range(2)]
                yy, ss = (o[first:first + 3 * n].view(3, n) for o in outs)
                gg = randn(520, n, dtype=dt)
                bnd.mha_rmsnorm(a, gg, 1e-6, y=yy, residual=b, sum_out=ss)
                z, ref = norm_ref(a, b, gg, 1e-6)
                R.check(yy, ref, norm_tol(z, ref, n, dt), f"start {first}")
                R.check(ss, z, R.HALF[dt] * z.abs(), "sum")
                for o in outs:
                    assert (o[:first] == 5).all() and (o[first + 3 * n:] == 5).all()
                y8 = torch.full((3 * n + first + 9,), 3.0, device="cuda").to(E4M3)
                sc = torch.empty(3, 1, device="cuda")
                bnd.mha_rmsnorm(a, gg, 1e-6, y=y8[first:first + 3 * n].view(3, n), residual=b, scales=sc)
                v = ref / (ref.abs().amax(dim=1, keepdim=True) / 448)
                R.check(y8.float()[first:first + 3 * n].view(3, n), v, 2.0 ** -4 * v.abs() * 1.01 + 2.0 ** -10 + 448 * n * 2.0 ** -23, "e4m3")
                assert (y8.float()[:first] == 3).all() and (y8.float()[first + 3 * n:] == 3).all()
    one = randn(123, 1, d, dtype=BF).expand(rows, d)                  # one residual for all rows
    bnd.mha_rmsnorm(x, g, 1e-6, y=y, residual=one)
    z, ref = norm_ref(x, one, g, 1e-6)
    R.check(y, ref, norm_tol(z, ref, d, BF), "broadcast residual")
    none = torch.empty(0, d, dtype=BF, device="cuda")
    bnd.mha_rmsnorm(none, g, 1e-6, y=none.clone())
    zero = torch.zeros(2, d, dtype=BF, device="cuda")
    y8, sc = torch.empty(2, d, device="cuda", dtype=E4M3), torch.empty(2, 4, device="cuda")
    bnd.mha_rmsnorm(zero, g, 1e-6, y=y8, scales=sc)
    assert (y8.float() == 0).all() and (sc == 1).all()


def test_rmsnorm_e4m3_of_tiny_values(bnd):
    """Groups below fp32's normal range keep their digits (448 / max would overflow)."""
    for d, group in ((256, 128), (77, 0)):
        x = randn(125, 3, d)
        g = torch.full((d,), 1e-38, device="cuda")
        groups = 1 if group == 0 else d // group
        y, sc = torch.empty(3, d, device="cuda", dtype=E4M3), torch.empty(3, groups, device="cuda")
        bnd.mha_rmsnorm(x, g, 1e-6, y=y, scales=sc)
        z, ref = norm_ref(x, None, g, 1e-6)
        v = ref / (ref.view(3, groups, -1).abs().amax(dim=2) / 448).repeat_interleave(d // groups, dim=1)
        # y itself is rounded to steps of 2^-149, 2^-23 of the largest values here; the scale too: 2^-14 of it
        R.check(y.float(), v, 2.0 ** -4 * v.abs() + 2.0 ** -10 + 2.0 ** -12 * 448, "tiny")


def test_rmsnorm_nan_stays_in_its_row(bnd):
    x = randn(130, 4, 1024, dtype=BF)
    x[1, 5] = float("nan")
    y8, sc = torch.empty(4, 1024, device="cuda", dtype=E4M3), torch.empty(4, 8, device="cuda")
    bnd.mha_rmsnorm(x, None, 1e-6, y=y8, scales=sc)
    bad = torch.isnan(y8.float()).all(dim=1)
    assert bad.tolist() == [False, True, False, False]
    assert not torch.isnan(y8.float()[[0, 2, 3]]).any()
    big = torch.full((1, 256), 1e18, device="cuda")                   # squares of 1e36: their mean is finite
    y = torch.empty_like(big)
    bnd.mha_rmsnorm(big, None, 1e-6, y=y)
    assert (y - 1).abs().max() <= 2.0 ** -16


# ------------------------------------------------------------------------------------------ together
@pytest.mark.parametrize("dtype,h,hk,d,sc", [(BF, 4, 2, 64, dict(cap=30.0)), (BF, 4, 1, 128, dict(slopes=True)),
                                             (F32, 4, 2, 64, dict(slopes=True)), (F32, 4, 1, 128, dict(cap=30.0))])
def test_prompt_and_steps_together(bnd, dtype, h, hk, d, sc):
    """Norm, projection, rotary and append, attention over the prompt, then single tokens over the cache: every
    step's output equals the row that attention over the whole sequence gives, in 64 bits from the same
    projected tensors."""
    B, L, T0, width, page = 3, 150, 121, 256, 16
    lens = [121, 64, 1]
    sc = {n: slopes_of(h) if n == "slopes" else x for n, x in sc.items()}
    x, gain = randn(140, B, L, width, dtype=dtype), (randn(141, width) * 0.2 + 1).to(dtype)
    w = randn(142, (h + 2 * hk) * d, width, dtype=dtype) * width ** -0.5
    normed = torch.empty_like(x)
    bnd.mha_rmsnorm(x.view(B * L, width), gain, 1e-6, y=normed.view(B * L, width))
    qkv = (normed @ w.T).view(B, L, h + 2 * hk, d)
    q, k, v = qkv[:, :, :h], qkv[:, :, h:h + hk], qkv[:, :, h + hk:]
    f, s = bnd.rotary_frequencies(d, 10000.0, bnd.ROPE_RAMP, 4.0, 64.0, 1.0, 8.0)
    rot = bnd.make_rotary(f.cuda(), scale=s)
    pos = torch.arange(L, device="cuda").expand(B, L)
    qr, kr = torch.empty_like(q), torch.empty_like(k)
    bnd.mha_rotary(q, k=k, q_out=qr, k_out=kr, rotary=rot)
    table, n_pages = table_of(143, B, -(-L // page))
    kp, vp = pages_of(144, n_pages, page, hk, d, dtype)
    kp.fill_(float("nan")), vp.fill_(float("nan"))
    cache = bnd.make_paged_cache(kp, vp, table)
    scores = bnd.make_scores(**sc)
    q0, k0 = torch.empty(B, T0, h, d, dtype=dtype, device="cuda"), torch.empty(B, T0, hk, d, dtype=dtype, device="cuda")
    held = ints([0] * B)
    bnd.mha_paged_append(k[:, :T0], v[:, :T0], held, cache=cache, q=q[:, :T0], q_out=q0, k_out=k0, new_lens=ints(lens), rotary=rot)
    held += ints(lens)
    for b, n in enumerate(lens):
        assert torch.equal(q0[b, :n], qr[b, :n]) and torch.equal(k0[b, :n], kr[b, :n])
    out = torch.empty_like(q0)
    bnd.mha_attention(q0, k0, v[:, :T0], out=out, scores=scores, mask=bnd.make_span_mask(causal=True, key_valid_lens=ints(lens)))
    ref, tol = attention_ref(qr, kr, v, causal=True, **sc)
    for b, n in enumerate(lens):
        R.check(out[b, :n], ref[b, :n], tol[b, :n], "prompt")
    ws = torch.empty(bnd.paged_attention_workspace_size(bnd.MHA_BF16 if dtype == BF else bnd.MHA_F32, B, h, hk, d), dtype=torch.uint8, device="cuda")
    q1, o1 = torch.empty(B, 1, h, d, dtype=dtype, device="cuda"), torch.empty(B, h, d, dtype=dtype, device="cuda")
    for step in range(20):
        at = [n + step for n in lens]
        pick = lambda t: torch.stack([t[b, at[b]:at[b] + 1] for b in range(B)])
        bnd.mha_paged_append(pick(k), pick(v), held, cache=cache, q=pick(q), q_out=q1, rotary=rot)
        held += 1
        bnd.mha_paged_attention(q1[:, 0], held, cache=cache, out=o1, workspace=ws, scores=scores)
        for b in range(B):
            R.check(o1[b], ref[b, at[b]], tol[b, at[b]], f"step {step}")


def test_captured_step_replays_with_new_lengths(bnd):
    """One decoding step captured into a graph and replayed: lengths, pages and inputs are read on the device. Two
    graphs with a workspace each replay on two streams at once."""
    B, h, hk, d, page, cap = 2, 8, 2, 64, 16, 400
    table, n_pages = table_of(150, B, cap // page)
    kp, vp = pages_of(151, n_pages, page, hk, d, BF)
    cache = bnd.make_paged_cache(kp, vp, table)
    rot = bnd.make_rotary(freqs(64))
    graphs = []
    for _ in range(2):
        st = dict(q=randn(152, B, 1, h, d, dtype=BF), k=randn(153, B, 1, hk, d, dtype=BF), v=randn(154, B, 1, hk, d, dtype=BF),
                  held=ints([0, 0]), n=ints([0, 0]), q1=torch.empty(B, 1, h, d, dtype=BF, device="cuda"),
                  out=torch.empty(B, h, d, dtype=BF, device="cuda"),
                  ws=torch.empty(bnd.paged_attention_workspace_size(bnd.MHA_BF16, B, h, hk, d), dtype=torch.uint8, device="cuda"))

        def step(st=st):
            bnd.mha_paged_append(st["k"], st["v"], st["held"], cache=cache, q=st["q"], q_out=st["q1"], rotary=rot)
            torch.add(st["held"], 1, out=st["n"])
            bnd.mha_paged_attention(st["q1"][:, 0], st["n"], cache=cache, out=st["out"], workspace=st["ws"])
        s = torch.cuda.Stream()
        s.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(s):
            step()
        s.synchronize()
        st["g"], st["s"] = torch.cuda.CUDAGraph(), s
        with torch.cuda.graph(st["g"]):
            step()
        graphs.append(st)
    torch.cuda.synchronize()
    for lens in ([5, 399], [130, 0]):
        for st in graphs:
            st["held"].copy_(ints(lens))
            st["out"].fill_(float("nan"))
        torch.cuda.synchronize()
        for st in graphs:                 # both append the same token to the same place
            with torch.cuda.stream(st["s"]):
                st["g"].replay()
        torch.cuda.synchronize()
        for st in graphs:
            ref, tol = paged_ref(st["q1"][:, 0], kp, vp, table, [n + 1 for n in lens], hk)
            R.check(st["out"], ref, tol, "replay")


def test_attention_and_norm_captured(bnd):
    B, L, h, d = 2, 260, 4, 128
    q, k, v = (randn(160 + i, B, L, h, d, dtype=BF) for i in range(3))
    valid = ints([L, L])
    out, y = torch.empty_like(q), torch.empty(B * L, h * d, dtype=BF, device="cuda")
    mask = bnd.make_span_mask(causal=True, key_valid_lens=valid)

    def step():
        bnd.mha_attention(q, k, v, out=out, mask=mask)
        bnd.mha_rmsnorm(out.view(B * L, h * d), None, 1e-6, y=y)
    step()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step()
    for n in (L, 100):
        valid.copy_(ints([n, 7]))
        q.copy_(randn(170 + n, B, L, h, d, dtype=BF))
        for _ in range(2):
            g.replay()
        torch.cuda.synchronize()
        ref, tol = attention_ref(q, k, v, causal=True, valid=[n, 7])
        R.check(out, ref, tol, "captured attention")
        z, want = norm_ref(out.view(B * L, h * d), None, None, 1e-6)
        R.check(y, want, norm_tol(z, want, h * d, BF), "captured norm")


def _step(bnd, seed, stream=None):
    """One call of each operator on its own tensors; the outputs."""
    B, h, hk, d, page = 2, 8, 2, 64, 16
    table, n_pages = table_of(seed, B, 20)
    kp, vp = pages_of(seed + 1, n_pages, page, hk, d, BF)
    cache = bnd.make_paged_cache(kp, vp, table)
    q, k, v = randn(seed + 3, B, 70, h, d, dtype=BF), randn(seed + 4, B, 70, hk, d, dtype=BF), randn(seed + 5, B, 70, hk, d, dtype=BF)
    q1, k1, att, dec = torch.empty_like(q), torch.empty_like(k), torch.empty_like(q), torch.empty(B, h, d, dtype=BF, device="cuda")
    ws = torch.empty(bnd.paged_attention_workspace_size(bnd.MHA_BF16, B, h, hk, d), dtype=torch.uint8, device="cuda")
    y = torch.empty(B * 70, h * d, dtype=BF, device="cuda")
    ids = docs_of(seed + 6, B, 70, 20)
    spans = torch.empty(B, 70, 2, dtype=torch.int32, device="cuda")
    rot, zero, held = bnd.make_rotary(freqs(d)), ints([0] * B), ints([300, 70])
    torch.cuda.synchronize()

    def call():
        bnd.mha_paged_append(k, v, zero, cache=cache, q=q, q_out=q1, k_out=k1, rotary=rot, stream=stream)
        bnd.mha_document_spans(ids, spans=spans, stream=stream)
        bnd.mha_attention(q1, k1, v, out=att, mask=bnd.make_span_mask(causal=True, doc_spans=spans), stream=stream)
        bnd.mha_rmsnorm(att.view(B * 70, h * d), None, 1e-6, y=y, stream=stream)
        bnd.mha_paged_attention(q1[:, 69], held, cache=cache, out=dec, workspace=ws, stream=stream)
    return call, (q1, k1, att, dec, y, kp, vp)


def test_explicit_streams_from_two_host_threads(bnd):
    """Two host threads, a stream each, call after call at once: the same results as one after the other."""
    import threading
    want = []
    for seed in (300, 320):
        call, outs = _step(bnd, seed)
        call()
        torch.cuda.synchronize()
        want.append([o.clone() for o in outs])
    jobs, errors = [], []
    for seed in (300, 320):
        s = torch.cuda.Stream()
        jobs.append(_step(bnd, seed, s) + (s,))

    def work(job):
        try:
            for _ in range(50):
                job[0]()
            job[2].synchronize()
        except Exception as e:
            errors.append(e)
    threads = [threading.Thread(target=work, args=(j,)) for j in jobs]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not errors
    for job, ref in zip(jobs, want):
        for got, o in zip(job[1], ref):
            assert torch.equal(got, o)


def test_first_call_may_be_captured():
    """A fresh process whose first calls are captured into a graph: nothing has to be set up before."""
    import os
    import subprocess
    import sys
    here = os.path.dirname(os.path.abspath(__file__))
    code = """
import sys
sys.path[:0] = [%r, %r]
import torch
import test_serving_gpu as T
from transformer_head_scaled_fwd_gb300 import binding as bnd
call, outs = T._step(bnd, 340)
g = torch.cuda.CUDAGraph()
with torch.cuda.graph(g):
    call()
g.replay()
torch.cuda.synchronize()
got = [o.clone() for o in outs]
for o in outs[:5]:
    o.zero_()
call()
torch.cuda.synchronize()
assert all(torch.equal(a, b) for a, b in zip(got, outs))
assert bnd.mha_check_device_status() == 0
print("captured first")
""" % (os.path.dirname(here), here)
    r = subprocess.run([sys.executable, "-c", code], capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and "captured first" in r.stdout, r.stdout + r.stderr


def _few_queries(bnd, seed, d):
    q, k, v = randn(seed, 2, 3, 4, d, dtype=BF), randn(seed + 1, 2, 2500, 2, d, dtype=BF), randn(seed + 2, 2, 2500, 2, d, dtype=BF)
    out = torch.zeros_like(q)
    mask = bnd.make_span_mask(causal=True, q_offset=2400, key_valid_lens=ints([2500, 900]))
    return lambda stream=None: bnd.mha_attention(q, k, v, out=out, mask=mask, stream=stream), out


def test_shared_units_captured_first():
    """A fresh process that captures attention of few queries over long keys as its first call."""
    import os
    import subprocess
    import sys
    here = os.path.dirname(os.path.abspath(__file__))
    code = """
import sys
sys.path[:0] = [%r, %r]
import torch
import test_serving_gpu as T
from transformer_head_scaled_fwd_gb300 import binding as bnd
call, out = T._few_queries(bnd, 360, 128)
torch.cuda.synchronize()
g = torch.cuda.CUDAGraph()
with torch.cuda.graph(g):
    call()
    call()
g.replay()
torch.cuda.synchronize()
got = out.clone()
out.zero_()
call()
torch.cuda.synchronize()
assert got.any() and torch.equal(got, out)
assert bnd.mha_check_device_status() == 0
print("captured first")
""" % (os.path.dirname(here), here)
    r = subprocess.run([sys.executable, "-c", code], capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and "captured first" in r.stdout, r.stdout + r.stderr


def test_shared_units_on_two_streams(bnd):
    """Two streams of calls whose clusters want the same SMs: the results of one after the other."""
    jobs = [_few_queries(bnd, 370 + 10 * i, d) + (torch.cuda.Stream(),) for i, d in enumerate((64, 128))]
    want = []
    for call, out, s in jobs:
        call()
        torch.cuda.synchronize()
        want.append(out.clone())
        out.zero_()
    torch.cuda.synchronize()
    for _ in range(100):
        for call, out, s in jobs:
            call(stream=s)
    torch.cuda.synchronize()
    assert all(torch.equal(j[1], w) for j, w in zip(jobs, want))


# ------------------------------------------------------------------------------------------ the binding's two ways
def one_of_each(bnd, dtype=BF):
    """A dict of calls with their outputs: {name: (call(**changes), [outputs])}."""
    B, T, h, hk, d, page, N = 2, 5, 4, 2, 64, 8, 6
    qkv = randn(170, B, T, h + 2 * hk, d, dtype=dtype)
    q, k, v = qkv[:, :, :h], qkv[:, :, h:h + hk], qkv[:, :, h + hk:]
    rot = bnd.make_rotary(freqs(32), interleaved=True, scale=1.1)
    kp, vp = (torch.zeros(N, page, hk, d, dtype=dtype, device="cuda") for _ in range(2))
    cache = bnd.make_paged_cache(kp, vp, ints([[3, 1], [0, 5]]))
    dt = bnd.MHA_BF16 if dtype == BF else bnd.MHA_F32
    ws = torch.empty(bnd.paged_attention_workspace_size(dt, B, h, hk, d), dtype=torch.uint8, device="cuda")
    scores = bnd.make_scores(cap=20.0, slopes=slopes_of(h))
    ids, spans = ints([[0, 0, 1, 1, -1], [4, 4, 4, 4, 4]]), torch.zeros(B, T, 2, dtype=torch.int32, device="cuda")
    q_out, k_out = torch.zeros(B, T, h, d, dtype=dtype, device="cuda"), torch.zeros(B, T, hk, d, dtype=dtype, device="cuda")
    a_out, d_out = torch.zeros_like(q_out), torch.zeros(B, h, d, dtype=dtype, device="cuda")
    x, r, gain = randn(171, 3, 256, dtype=dtype), randn(172, 3, 256, dtype=dtype), randn(173, 256, dtype=dtype)
    z, y8, sc = torch.zeros_like(x), torch.zeros(3, 256, device="cuda", dtype=E4M3), torch.zeros(3, 2, device="cuda")
    mask = bnd.make_span_mask(causal=True, q_offset=1, key_valid_lens=ints([5, 3]), prefix_lens=ints([2, 0]), doc_spans=spans)
    mk = lambda f, kw: lambda **ch: f(**{**kw, **ch})
    return {
        "rotary": (mk(bnd.mha_rotary, dict(q=q, k=k, q_out=q_out, k_out=k_out, rotary=rot, positions=ints([[9, 8, 7, 6, 5]] * 2))),
                   [q_out, k_out]),
        "append": (mk(bnd.mha_paged_append, dict(k=k, v=v, start=ints([0, 6]), cache=cache, q=q, q_out=q_out, k_out=k_out,
                                                 new_lens=ints([5, 2]), rotary=rot)), [q_out, k_out, kp, vp]),
        "decode": (mk(bnd.mha_paged_attention, dict(q=q[:, 0], kv_lens=ints([5, 8]), cache=cache, out=d_out, workspace=ws,
                                                    scores=scores)), [d_out]),
        "spans": (mk(bnd.mha_document_spans, dict(doc_ids=ids, spans=spans)), [spans]),
        "attention": (mk(bnd.mha_attention, dict(q=q, k=k, v=v, out=a_out, scores=scores, mask=mask)), [a_out]),
        "rmsnorm": (mk(bnd.mha_rmsnorm, dict(x=x, gain=gain, eps=1e-5, y=y8, residual=r, sum_out=z, scales=sc)), [y8, z, sc]),
    }


@pytest.mark.parametrize("dtype", [BF, F32])
def test_native_and_ctypes_calls_are_the_same(bnd, monkeypatch, dtype):
    """Every call once through the native front and once through ctypes: the same bits, on the current stream and on a
    given one, with optional arguments and without."""
    calls = one_of_each(bnd, dtype)
    calls["rotary"][0]()
    assert bnd._front is not None, "the native front is not built"
    optional = {"rotary": [{}, dict(k=None, k_out=None), dict(positions=None)],
                "append": [{}, dict(q=None, q_out=None), dict(k_out=None), dict(new_lens=None), dict(rotary=None)],
                "decode": [{}, dict(scores=None)], "spans": [{}],
                "attention": [{}, dict(scores=None), dict(mask=None), dict(mask=bnd.make_span_mask()), dict(mask=bnd.make_span_mask(causal=True))],
                "rmsnorm": [{}, dict(gain=None), dict(sum_out=None), dict(sum_out=None, residual=None)]}
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    for name, (call, outs) in calls.items():
        for change in optional[name]:
            got = []
            for front in (bnd._front, None):
                with monkeypatch.context() as m:
                    m.setattr(bnd, "_front", front)
                    for o in outs:
                        o.view(torch.uint8).zero_()
                    torch.cuda.synchronize()
                    with torch.cuda.stream(side) if front is None else torch.cuda.stream(torch.cuda.default_stream()):
                        call(**change, stream=side if front is not None else None)
                    torch.cuda.synchronize()
                    got.append([o.view(torch.uint8).clone() for o in outs])
            assert all(torch.equal(a, b) for a, b in zip(*got)), (name, change)
            assert any(a.any() for a in got[0]), (name, change)
    calls["spans"][0](), calls["attention"][0](), torch.cuda.synchronize()


def test_native_calls_leave_faults_to_python(bnd):
    """What is not in order: the native front declines without doing anything, and the error names the argument."""
    calls = one_of_each(bnd)
    calls["spans"][0]()
    half = lambda *s: torch.zeros(*s, device="cuda", dtype=torch.float16)
    fp = lambda *s: torch.zeros(*s, device="cuda")
    bf = lambda *s: torch.zeros(*s, device="cuda", dtype=BF)
    cpu = torch.zeros(2, 5, 4, 64, dtype=BF)
    other = bnd.make_paged_cache(bf(6, 8, 4, 64), bf(6, 8, 4, 64), ints([[3, 1], [0, 5]]))
    bad = {
        "rotary": [dict(q=half(2, 5, 4, 64)), dict(q_out=bf(2, 5, 4, 32)), dict(k_out=fp(2, 5, 2, 64)), dict(q=cpu), dict(rotary=None),
                   dict(positions=ints([1, 2])), dict(positions=torch.zeros(2, 5, dtype=torch.int64, device="cuda")), dict(k_out=None),
                   dict(q=bf(2, 5, 64, 4).transpose(2, 3)), dict(q=3)],
        "append": [dict(cache=other), dict(v=bf(2, 4, 2, 64)), dict(start=None), dict(start=ints([1])), dict(new_lens=fp(2)),
                   dict(q_out=None), dict(k=cpu), dict(cache=None)],
        "decode": [dict(out=fp(2, 4, 64)), dict(kv_lens=None), dict(workspace=bf(1)), dict(scores=bnd.make_scores(slopes=slopes_of(8))),
                   dict(q=bf(3, 4, 64)), dict(q=bf(2, 3, 64), out=bf(2, 3, 64))],
        "spans": [dict(spans=ints([[1]])), dict(doc_ids=fp(2, 5))],
        "attention": [dict(v=bf(2, 4, 2, 64)), dict(q=half(2, 5, 4, 64)), dict(out=bf(2, 5, 4, 128)), dict(mask=bnd.make_span_mask(q_offset=-1)),
                      dict(mask=bnd.make_span_mask(key_valid_lens=ints([1]))), dict(mask=bnd.make_span_mask(q_offset=1 << 40)),
                      dict(k=bf(2, 5, 3, 64), v=bf(2, 5, 3, 64))],
        "rmsnorm": [dict(y=bf(3, 256)), dict(scales=fp(3, 3)), dict(scales=fp(3, 128)), dict(residual=None), dict(gain=bf(255)), dict(eps=-1.0),
                    dict(x=bf(256, 3).t()), dict(x=bf(768))],
    }
    for name, changes in bad.items():
        call, outs = calls[name]
        for o in outs:
            o.view(torch.uint8).fill_(7)
        for change in changes:
            with pytest.raises((ValueError, TypeError, AttributeError, bnd.MHAError, struct.error)):
                call(**change)
        torch.cuda.synchronize()
        for o in outs:
            assert (o.view(torch.uint8) == 7).all(), name


def test_native_call_of_a_changed_description(bnd):
    """A description's fields may be changed between calls: both ways read them at the call."""
    q = randn(175, 1, 3, 2, 64)
    out, want = torch.empty_like(q), torch.empty_like(q)
    rot = bnd.make_rotary(freqs(64))
    bnd.mha_rotary(q, q_out=want, rotary=bnd.make_rotary(freqs(64), scale=2.0))
    bnd.mha_rotary(q, q_out=out, rotary=rot)
    rot.scale = 2.0
    bnd.mha_rotary(q, q_out=out, rotary=rot)
    assert torch.equal(out, want)
