"""Serving operators at the ends of their ranges (caps, values, empty and NaN rows, rounding of codes) and where a step
lost or doubled would show, against plain 64-bit forms."""
import math

import pytest

torch = pytest.importorskip("torch")

import serving_ref as R  # noqa: E402
import test_serving_gpu as S  # noqa: E402
from test_serving_gpu import BF, E4M3, F32, bnd, clean_status, ints, randn  # noqa: E402, F401

pytestmark = pytest.mark.gpu


def attend_fine(q, k, v, allowed, distance, *, scale, cap=0.0, slope=0.0):
    """One head in fp64 with a bound of |kernel - o| from the error of each key's own score: d products summed in fp32
    (d 2^-24 of sum |q k|), four roundings, and with a cap 2^-19 of min(cap, sum |q k|): tanh by its polynomials is within
    2^-19.7 of its value, its three fp32 roundings within 2^-22.4; beyond |x| = 0.7 an error of 2^-22 of the cap is below
    2^-21 of the score. A weight is then off by a relative d_j = e^(2 error_j) - 1, and o by sum p_j (d_j + sum p d) |v_j|;
    exp2 2^-20, weights to bf16 half a step, n sums in fp32 as in serving_ref.attend_tol."""
    dtype, (n, d) = v.dtype, v.shape
    q, k, v = q.double(), k.double(), v.double()
    s = (q @ k.T) * scale
    size = (q.abs() @ k.abs().T) * abs(scale)
    err = (d + 4) * 2.0 ** -24 * size + 4 * 2.0 ** -24 * abs(slope) * distance
    if cap:
        s = cap * torch.tanh(s / cap)
        err = err.clamp(max=2 * cap) + 2.0 ** -19 * size.clamp(max=cap)
    s = torch.where(allowed, s - slope * distance, -math.inf)
    p = torch.softmax(s, dim=1)
    dj = torch.expm1(2 * torch.where(allowed, err, 0.0).clamp(max=300))
    dj = torch.where(p > 0, dj, 0.0)
    o = p @ v
    rel = (p * dj) @ v.abs() + (p * dj).sum(dim=1, keepdim=True) * (p @ v.abs())
    tol = rel + (2.0 ** -20 + (R.HALF[dtype] if dtype == BF else 0.0) + 2 * (n + 16) * 2.0 ** -24) * (p @ v.abs())
    return o, tol + R.HALF[dtype] * o.abs() + 2.0 ** -120


def paged_fine(q, kp, vp, table, lens, hk, **sc):
    B, h, d = q.shape
    ref, tol = torch.zeros(B, h, d, dtype=torch.float64, device="cuda"), torch.zeros(B, h, d, dtype=torch.float64, device="cuda")
    slopes, sc = sc.get("slopes"), dict(scale=sc.get("scale", d ** -0.5), cap=sc.get("cap", 0.0))
    for b, n in enumerate(lens):
        rows = table[b, : -(-n // kp.shape[1])].long()
        ok, away = torch.ones(1, n, dtype=torch.bool, device="cuda"), (n - 1 - torch.arange(n, device="cuda"))[None].double()
        for i in range(h):
            k, v = (x[rows, :, i // (h // hk)].flatten(0, 1)[:n] for x in (kp, vp))
            ref[b, i], tol[b, i] = (x[0] for x in attend_fine(q[b, i:i + 1], k, v, ok, away, slope=0.0 if slopes is None else
                                                               slopes[i].item(), **sc))
    return ref, tol


def attention_fine(q, k, v, *, causal=False, q_offset=0, docs=None, slopes=None, **sc):
    B, Lq, h, d = q.shape
    Lk, hk = k.shape[1], k.shape[2]
    ref, tol = torch.zeros(q.shape, dtype=torch.float64, device="cuda"), torch.zeros(q.shape, dtype=torch.float64, device="cuda")
    sc = dict(scale=sc.get("scale", d ** -0.5), cap=sc.get("cap", 0.0))
    i, j = torch.arange(Lq, device="cuda")[:, None] + q_offset, torch.arange(Lk, device="cuda")[None]
    for b in range(B):
        ok = j <= i if causal else torch.ones(Lq, Lk, dtype=torch.bool, device="cuda")
        if docs is not None:
            ok = ok & (docs[b][:, None] == docs[b][None])
        for n in range(h):
            ref[b, :, n], tol[b, :, n] = attend_fine(q[b, :, n], k[b, :, n // (h // hk)], v[b, :, n // (h // hk)], ok,
                                                     (i - j).abs().double(), slope=0.0 if slopes is None else slopes[n].item(), **sc)
    return ref, tol


# ------------------------------------------------------------------------------------------ caps
CAPS = [1e-3, 2.0, 70.0, 1e3, 1e4, 1e6, 1e30]


def far_keys(q, k, every, score, scale):
    """Every `every`-th key along -q of each head's first query, so that its score with that query is `score`."""
    B, Lk, hk, d = k.shape
    g = q.shape[2] // hk
    for b in range(B):
        for n in range(hk):
            x = q[b, 0, n * g].double()
            k[b, 3::every, n] = (x * (score / (scale * (x @ x)))).to(k.dtype)


@pytest.mark.parametrize("dtype,h,hk,d", [(BF, 4, 2, 64), (BF, 12, 1, 128), (F32, 4, 1, 128)])
@pytest.mark.parametrize("cap", CAPS)
def test_paged_attention_caps_of_every_size(bnd, dtype, h, hk, d, cap):
    """cap tanh(s / cap) keeps a score's own digits however large or small the cap is; far above the scores it changes
    nothing."""
    lens = [300, 17, 2500]
    table, n_pages = S.table_of(1, 3, -(-2500 // 16))
    kp, vp = S.pages_of(2, n_pages, 16, hk, d, dtype)
    for gain in (2.0, 20.0):
        q = randn(4, 3, h, d, dtype=dtype) * gain
        got = S.run_paged(bnd, q, kp, vp, table, lens, hk, cap=cap)
        ref, tol = paged_fine(q, kp, vp, table, lens, hk, cap=cap)
        R.check(got, ref, tol, f"cap {cap}, scores up to about {4 * gain}")


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("cap", [1e3, 1e6])
def test_paged_attention_far_scores_beside_near_ones(bnd, dtype, cap):
    h, hk, d, n = 2, 2, 64, 700
    table, n_pages = S.table_of(3, 1, -(-n // 32))
    kp, vp = S.pages_of(4, n_pages, 32, hk, d, dtype)
    q = randn(6, 1, h, d, dtype=dtype)
    k = kp[table[0].long()].flatten(0, 1)[None].contiguous()
    far_keys(q[:, None], k, 16, -0.9 * cap, d ** -0.5)
    kp[table[0].long()] = k[0].view(-1, 32, hk, d)
    got = S.run_paged(bnd, q, kp, vp, table, [n], hk, cap=cap)
    ref, tol = paged_fine(q, kp, vp, table, [n], hk, cap=cap)
    R.check(got, ref, tol, "near scores")


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("cap,scale", [(3.4e38, None), (1e35, 1e-10), (1e-44, None), (1e-30, 1e3)])
def test_caps_at_the_ends_of_fp32(bnd, dtype, cap, scale):
    """Caps whose product with log2 e, or whose quotient with the scale, leaves fp32's range: no cap, or no score at all."""
    h, hk, d, n = 4, 2, 64, 200
    sc = dict(cap=cap) if scale is None else dict(cap=cap, scale=scale)
    table, n_pages = S.table_of(50, 1, -(-n // 16))
    kp, vp = S.pages_of(51, n_pages, 16, hk, d, dtype)
    q = randn(53, 1, h, d, dtype=dtype)
    q[0, 0] = 0.0
    got = S.run_paged(bnd, q, kp, vp, table, [n], hk, **sc)
    ref, tol = paged_fine(q, kp, vp, table, [n], hk, **sc)
    R.check(got, ref, tol, "paged")
    rows = table[0].long()
    k, v = (x[rows].flatten(0, 1)[None, :n].contiguous() for x in (kp, vp))
    got = S.run_attention(bnd, q[:, None].contiguous(), k, v, **sc)
    ref, tol = attention_fine(q[:, None], k, v, **sc)
    R.check(got, ref, tol, "attention")


SPANS = [
    # B, Lq, Lk, h, h_kv, d, options
    (1, 130, 130, 2, 1, 128, dict(causal=True)),
    (2, 300, 700, 4, 2, 64, dict(causal=True, q_offset=400)),
    (1, 600, 600, 2, 2, 64, dict(docs=150)),
    (1, 257, 513, 2, 1, 128, dict(slopes=True)),
    (1, 3, 4096, 2, 1, 128, dict()),                              # several CTAs share a query tile
    (2, 1600, 1600, 6, 6, 64, dict(causal=True, slopes=True)),    # two query tiles a unit
]


@pytest.mark.parametrize("B,Lq,Lk,h,hk,d,opt", SPANS)
@pytest.mark.parametrize("cap", CAPS)
@pytest.mark.parametrize("dtype", [BF, F32])
def test_attention_caps_of_every_size(bnd, dtype, cap, B, Lq, Lk, h, hk, d, opt):
    opt = dict(opt, cap=cap)
    if opt.get("slopes"):
        opt["slopes"] = S.slopes_of(h)
    if opt.get("docs"):
        opt["docs"] = S.docs_of(7, B, Lk, opt["docs"])
    q, k, v = randn(8, B, Lq, h, d, dtype=dtype) * 4.0, randn(9, B, Lk, hk, d, dtype=dtype), randn(10, B, Lk, hk, d, dtype=dtype)
    got = S.run_attention(bnd, q, k, v, **opt)
    ref, tol = attention_fine(q, k, v, **opt)
    R.check(got, ref, tol, f"cap {cap}")


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("Lq,Lk,h,d", [(1, 200, 2, 64), (1, 900, 2, 128), (2, 4096, 1, 64)])
@pytest.mark.parametrize("cap", [1e3, 1e6])
def test_attention_far_scores_beside_near_ones(bnd, dtype, Lq, Lk, h, d, cap):
    q, k, v = randn(11, 1, Lq, h, d, dtype=dtype), randn(12, 1, Lk, h, d, dtype=dtype), randn(13, 1, Lk, h, d, dtype=dtype)
    q[:, 1:] = q[:, :1]
    far_keys(q, k, 16, -0.9 * cap, d ** -0.5)
    got = S.run_attention(bnd, q, k, v, cap=cap)
    ref, tol = attention_fine(q, k, v, cap=cap)
    R.check(got, ref, tol, "near scores")


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("sc", [dict(cap=59.0), dict(cap=59.0, scale=-0.11), dict(cap=300.0), dict(cap=5000.0), {}, dict(cap=59.0, slopes=True)])
@pytest.mark.parametrize("B,Lq,Lk,h,d,opt", [(1, 200, 1500, 2, 128, {}), (1, 1300, 1300, 2, 64, dict(causal=True)),
                                             (1, 4, 5000, 2, 64, {}), (2, 900, 900, 1, 128, dict(docs=200))])
@pytest.mark.parametrize("way", ["rising", "falling", "deep"])
def test_scores_that_move_the_maximum_all_along(bnd, dtype, sc, B, Lq, Lk, h, d, opt, way):
    """Scores that grow (fall) steadily over the keys, by about 130 in all before the cap, or lie at about -100 throughout: the reference
    of every row moves tile after tile, or starts far below zero."""
    sc, opt = dict(sc), dict(opt)
    if sc.get("slopes"):
        sc["slopes"] = S.slopes_of(h)
    if opt.get("docs"):
        opt["docs"] = S.docs_of(60, B, Lk, opt["docs"])
    scale = sc.get("scale", d ** -0.5)
    q, k, v = randn(61, B, Lq, h, d), randn(62, B, Lk, h, d) * 0.3, randn(63, B, Lk, h, d, dtype=dtype)
    q[..., 0] = 8.0                                          # one feature carries the slow part of the scores
    t = torch.arange(Lk, device="cuda") / Lk
    k[..., 0] = ((dict(rising=130 * t - 65, falling=65 - 130 * t, deep=-100 + 5 * t)[way]) / (8.0 * scale))[None, :, None]
    q, k = q.to(dtype), k.to(dtype)
    got = S.run_attention(bnd, q, k, v, **sc, **opt)
    ref, tol = attention_fine(q, k, v, **sc, **opt)
    R.check(got, ref, tol, way)


# ------------------------------------------------------------------------------------------ values
@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("B,Lq,Lk,h,d,opt", [(1, 200, 600, 2, 128, {}), (1, 600, 600, 2, 64, dict(causal=True)),
                                             (1, 2, 4096, 2, 128, {}), (1, 512, 512, 1, 128, dict(valid=[300]))])
@pytest.mark.parametrize("cap,sign", [(59.0, 1), (59.0, -1), (30.0, -1)])
@pytest.mark.parametrize("size", [2.0 ** 100, 2.0 ** -100])
def test_capped_attention_of_large_and_tiny_values(bnd, dtype, B, Lq, Lk, h, d, opt, cap, sign, size):
    """All scores at one end of the cap: weights are equal whatever the values' size is. The fp32 sum of 4096 weighted values
    of 2^100 stays below 2^127, and a product of 2^-100 with a weight of 1 above fp32's smallest normal number."""
    q = torch.ones(B, Lq, h, d, device="cuda", dtype=dtype) * 40.0
    k = torch.ones(B, Lk, h, d, device="cuda", dtype=dtype) * sign * 40.0
    v = (randn(14, B, Lk, h, d).abs() + 0.5).to(dtype)
    got = S.run_attention(bnd, q, k, v * size, cap=cap, **opt)
    # equal scores, in fp32 too: the reference of scores of 0, and only the values' part of its bound
    ref, tol = S.attention_ref(torch.zeros_like(q), k, v, **opt)
    R.check(got.double() / size, ref, tol, "values")


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("n", [40, 4000])
@pytest.mark.parametrize("size", [2.0 ** 100, 2.0 ** -100])
def test_capped_paged_attention_of_large_and_tiny_values(bnd, dtype, n, size):
    h, hk, d = 4, 2, 64
    table, n_pages = S.table_of(15, 1, -(-n // 16))
    kp, vp = S.pages_of(16, n_pages, 16, hk, d, dtype)
    kp.fill_(-40.0)
    vp = (vp.float().abs() + 0.5).to(dtype)
    q = torch.ones(1, h, d, device="cuda", dtype=dtype) * 40.0
    got = S.run_paged(bnd, q, kp, vp * size, table, [n], hk, cap=59.0)
    ref, tol = S.paged_ref(torch.zeros_like(q), kp, vp, table, [n], hk)
    R.check(got.double() / size, ref, tol, "values")


# ------------------------------------------------------------------------------------------ rows without a key, NaN rows
@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
@pytest.mark.parametrize("sc", [{}, dict(cap=30.0), dict(slopes=True)])
@pytest.mark.parametrize("B,L,h,d", [(2, 200, 2, 64), (2, 200, 2, 128), (1, 700, 1, 128), (3, 1700, 6, 64)])
def test_rows_without_a_key_are_zeros_whatever_the_values(bnd, dtype, bad, sc, B, L, h, d):
    """Padding in front of the documents, between and behind them, with values that are not finite: its own rows are zeros."""
    sc = dict(sc, slopes=S.slopes_of(h)) if sc.get("slopes") else sc
    ids = torch.arange(L, device="cuda").div(90, rounding_mode="floor").int().expand(B, L).clone()
    ids[:, :70], ids[:, 100:103], ids[:, L - 5:] = -1, -1, -1
    pad = ids < 0
    q, k, v = (randn(17 + i, B, L, h, d, dtype=dtype) for i in range(3))
    v[pad] = bad
    got = S.run_attention(bnd, q, k, v, docs=ids, **sc)
    assert torch.equal(got[pad], torch.zeros_like(got[pad]))


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("sc", [{}, dict(cap=30.0), dict(slopes=True)])
@pytest.mark.parametrize("d", [64, 128])
def test_shared_units_rows_without_a_key(bnd, dtype, sc, d):
    B, Lq, Lk, h = 1, 4, 4096, 2
    sc = dict(sc, slopes=S.slopes_of(h)) if sc.get("slopes") else sc
    q, k, v = randn(20, B, Lq, h, d, dtype=dtype), randn(21, B, Lk, h, d, dtype=dtype), randn(22, B, Lk, h, d, dtype=dtype)
    v[:, ::97] = float("nan")
    spans = ints([[[0, 0], [0, Lk], [500, 500], [3000, 2000]]])
    got = S.run_attention(bnd, q, k, v, spans=spans, **sc)
    assert torch.equal(got[:, [0, 2, 3]], torch.zeros_like(got[:, [0, 2, 3]]))


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("sc", [{}, dict(cap=30.0), dict(slopes=True)])
@pytest.mark.parametrize("Lq,Lk,h,d", [(4, 100, 2, 64), (4, 4096, 2, 64), (4, 4096, 2, 128), (130, 2048, 2, 128)])
def test_nan_queries_give_nan_rows(bnd, dtype, sc, Lq, Lk, h, d):
    """A query that is NaN has NaN scores with all keys: so is its row, alone, however many CTAs share its keys."""
    sc = dict(sc, slopes=S.slopes_of(h)) if sc.get("slopes") else sc
    q, k, v = randn(23, 1, Lq, h, d, dtype=dtype), randn(24, 1, Lk, h, d, dtype=dtype), randn(25, 1, Lk, h, d, dtype=dtype)
    q[0, 2, 1, 5] = float("nan")
    got = S.run_attention(bnd, q, k, v, **sc)
    assert torch.isnan(got[0, 2, 1]).all()
    keep = torch.ones(Lq, h, dtype=torch.bool, device="cuda")
    keep[2, 1] = False
    assert torch.isfinite(got[0][keep]).all()


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("n", [40, 5000])
def test_nan_queries_give_nan_rows_over_the_paged_cache(bnd, dtype, n):
    h, hk, d = 4, 2, 64
    table, n_pages = S.table_of(26, 1, -(-n // 16))
    kp, vp = S.pages_of(27, n_pages, 16, hk, d, dtype)
    q = randn(29, 1, h, d, dtype=dtype)
    q[0, 1, 7] = float("nan")
    got = S.run_paged(bnd, q, kp, vp, table, [n], hk)
    assert torch.isnan(got[0, 1]).all() and torch.isfinite(got[0, [0, 2, 3]]).all()


# ------------------------------------------------------------------------------------------ e4m3 codes
def check_codes(y, y8, sc):
    """The codes are fp32 y over the stored scale by IEEE fp32 divisions; the scale is the largest value over 448, to within
    a product's two roundings."""
    rows, d = y.shape
    groups = sc.shape[1]
    top = y.double().abs().view(rows, groups, -1).amax(dim=2)
    assert ((sc.double() - top / 448).abs() <= 2.0 ** -23 * top / 448).all()
    want = (y / sc.repeat_interleave(d // groups, dim=1)).to(E4M3)
    diff = y8.view(torch.uint8) != want.view(torch.uint8)
    assert not diff.any(), f"{int(diff.sum())} codes of {diff.numel()}"


@pytest.mark.parametrize("rows,d,group", [(3, 256, 128), (2000, 512, 64), (700, 4096, 0), (700, 4096, 128), (64, 1001, 0), (5, 40000, 32)])
def test_rmsnorm_codes_are_the_quotients(bnd, rows, d, group):
    """Against the row in fp32 by the same call."""
    x, g = randn(30, rows, d), randn(31, d) + 1.5
    y, y8 = torch.empty(rows, d, device="cuda"), torch.empty(rows, d, device="cuda", dtype=E4M3)
    groups = 1 if group == 0 else d // group
    sc = torch.empty(rows, groups, device="cuda")
    bnd.mha_rmsnorm(x, g, 1e-6, y=y)
    bnd.mha_rmsnorm(x, g, 1e-6, y=y8, scales=sc)
    check_codes(y, y8, sc)


@pytest.mark.parametrize("top", [448.0, 1344.0, 448.0 / 3, 2.0 ** -120, 2.0 ** 120])
def test_rmsnorm_codes_at_ties(bnd, top):
    """Quotients half way between two codes, or next to it where top / 448 is not a power of two."""
    d = 128
    mids = torch.tensor([17, 19, 21, 23, 25, 27, 29, 31, 34, 38, 8.5, 9.5, 1.0625, 1.1875, 0.53125, 432, 400, 208] * 7 + [448.0, 448.0], device="cuda")
    g = (mids * (top / 448)).float()
    x = torch.ones(2, d, device="cuda")
    x[1] = -1
    y, y8, sc = torch.empty(2, d, device="cuda"), torch.empty(2, d, device="cuda", dtype=E4M3), torch.empty(2, 1, device="cuda")
    bnd.mha_rmsnorm(x, g, 0.0, y=y)
    bnd.mha_rmsnorm(x, g, 0.0, y=y8, scales=sc)
    assert torch.equal(y[0], g) and torch.equal(y[1], -g)
    check_codes(y, y8, sc)


def test_rmsnorm_scale_that_would_be_zero(bnd):
    """A largest value whose 448th part is below fp32's smallest number: a scale of 1, as for a row of zeros."""
    x = torch.ones(2, 64, device="cuda")
    g = torch.full((64,), 2.0 ** -145, device="cuda")
    g[::2] = 0.0
    y8, sc = torch.empty(2, 64, device="cuda", dtype=E4M3), torch.empty(2, 1, device="cuda")
    bnd.mha_rmsnorm(x, g, 0.0, y=y8, scales=sc)
    assert (sc == 1).all() and (y8.float() == 0).all()


# ------------------------------------------------------------------------------------------ nothing lost, nothing doubled
def norm_error(got, ref):
    return ((got.double() - ref).norm() / ref.norm()).item()


# Rounding normally distributed values to bf16: an error uniform over each value's step, sqrt(E step^2 / 12 / E x^2) = 1.66e-3
# of the norm wherever the distribution's width lies between two powers of two. Weights rounded to bf16 add as much again,
# independently: 2.35e-3. A twentieth on top for the spread of samples. fp32: products over d_k = 128 of scores up to 4 put
# weights off by 128 * 2^-24 * 4 * 2 = 6e-5 at most.
NORM = {("paged", BF): 1.75e-3, ("span", BF): 2.45e-3, ("paged", F32): 6e-5, ("span", F32): 6e-5}


@pytest.mark.parametrize("dtype,B,h,hk,d,n,sc", [
    (BF, 1, 16, 2, 128, 70001, {}), (BF, 2, 4, 4, 64, 30000, {}), (BF, 16, 8, 8, 64, 1000, dict(cap=30.0)),
    (BF, 64, 16, 4, 64, 200, {}), (BF, 3, 20, 1, 128, 5000, dict(slopes=True)),
    (F32, 1, 4, 1, 64, 40001, {}), (F32, 8, 8, 2, 128, 700, dict(cap=30.0))])
def test_paged_attention_error_of_the_norm(bnd, dtype, B, h, hk, d, n, sc):
    sc = dict(sc, slopes=S.slopes_of(h)) if sc.get("slopes") else sc
    lens = [n - 7 * b for b in range(B)]
    table, n_pages = S.table_of(32, B, -(-n // 64))
    kp, vp = S.pages_of(33, n_pages, 64, hk, d, dtype)
    q = randn(35, B, h, d, dtype=dtype)
    got = S.run_paged(bnd, q, kp, vp, table, lens, hk, **sc)
    ref, _ = S.paged_ref(q, kp, vp, table, lens, hk, **sc)
    assert norm_error(got, ref) <= NORM["paged", dtype]


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("B,Lq,Lk,h,hk,d,opt", [
    (1, 600, 600, 2, 1, 128, dict(causal=True)), (1, 600, 600, 2, 2, 64, dict(causal=True, cap=50.0)),
    (1, 1100, 1100, 2, 2, 128, dict(causal=True, cap=20.0)), (2, 700, 700, 2, 1, 128, dict(docs=60)),
    (1, 700, 700, 2, 1, 64, dict(causal=True, slopes=True)),
    (2, 1600, 1600, 6, 6, 64, dict(causal=True)), (2, 1600, 1600, 6, 6, 64, dict(docs=90, cap=20.0)),
    (1, 16, 8192, 4, 1, 128, dict(causal=True, q_offset=8176)), (2, 16, 4100, 4, 2, 64, dict(causal=True, q_offset=4084, cap=30.0))])
def test_attention_error_of_the_norm(bnd, dtype, B, Lq, Lk, h, hk, d, opt):
    opt = dict(opt)
    if opt.get("slopes"):
        opt["slopes"] = S.slopes_of(h)
    if opt.get("docs"):
        opt["docs"] = S.docs_of(36, B, Lk, opt["docs"])
    q, k, v = randn(37, B, Lq, h, d, dtype=dtype), randn(38, B, Lk, hk, d, dtype=dtype), randn(39, B, Lk, hk, d, dtype=dtype)
    got = S.run_attention(bnd, q, k, v, **opt)
    ref, _ = S.attention_ref(q, k, v, **opt)
    assert norm_error(got, ref) <= NORM["span", dtype]


def borders(n, *steps):
    """Positions around the multiples of each step in 0 .. n - 1, the first and the last ones among them."""
    at = {0, 1, n - 1, n - 2}
    for s in steps:
        for m in range(0, n + 1, s):
            at |= {m - 1, m, m + 1}
    return sorted(x for x in at if 0 <= x < n)


@pytest.mark.parametrize("dtype,h,hk,d,lens,page", [
    (BF, 4, 2, 64, [70001], 64), (BF, 16, 2, 128, [30000, 5], 128), (BF, 2, 2, 64, [1000] * 3, 16),
    (F32, 4, 1, 64, [20001], 64), (F32, 2, 2, 128, [513, 8000, 64], 24)])
def test_paged_attention_takes_every_key_once(bnd, dtype, h, hk, d, lens, page):
    """Equal scores, values that are zero but at keys around the borders of steps, blocks, pages and pieces, each with a
    feature of its own: that feature of the output is 1 / n, and 0 or 2 / n if the key is left out or taken twice. Half
    a step of the output's type, and fp32 sums of up to 70001 ones."""
    B, per = len(lens), -(-max(lens) // page)
    table, n_pages = S.table_of(40, B, per)
    kp, vp = S.pages_of(41, n_pages, page, hk, d, dtype)
    q = torch.zeros(B, h, d, device="cuda", dtype=dtype)
    step = max(lens) // 152 + 1                      # pieces of the line end about here, whatever the device
    todo = [borders(n, 64, step) if n < 3000 else borders(n, 128 * 16, step) for n in lens]
    for first in range(0, max(len(t) for t in todo), d):
        vp.zero_()
        want = torch.zeros(B, h, d, dtype=torch.float64, device="cuda")
        for b, n in enumerate(lens):
            keys = todo[b][first:first + d]
            at = torch.tensor(keys, device="cuda", dtype=torch.long)
            if len(keys):
                f = torch.arange(len(keys), device="cuda")
                vp[table[b].long()[at // page], at % page, :, f] = 1.0
                want[b, :, :len(keys)] = 1.0 / n
        got = S.run_paged(bnd, q, kp, vp, table, lens, hk)
        R.check(got, want, want * (R.HALF[dtype] + 2.0 ** -8 * (dtype == F32) + 2.0 ** -10) + 0.0, "every key once")


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("B,Lq,Lk,h,d,causal,cap", [
    (1, 130, 130, 2, 64, True, 0.0), (1, 3, 8192, 2, 128, False, 0.0), (1, 129, 3000, 2, 64, True, 20.0),
    (1, 300, 1000, 1, 128, True, 0.0), (2, 1600, 1600, 6, 64, True, 0.0), (1, 1, 5000, 4, 64, False, 0.0)])
def test_attention_takes_every_key_once(bnd, dtype, B, Lq, Lk, h, d, causal, cap):
    q, k = torch.zeros(B, Lq, h, d, device="cuda", dtype=dtype), randn(43, B, Lk, h, d, dtype=dtype)
    off = Lk - Lq
    seen = (torch.arange(Lq, device="cuda") + off + 1 if causal else torch.full((Lq,), Lk, device="cuda")).double()
    todo = borders(Lk, 64, Lk // 8 + 1)
    for first in range(0, len(todo), d):
        at = torch.tensor(todo[first:first + d], device="cuda")
        f = torch.arange(len(at), device="cuda")
        v = torch.zeros(B, Lk, h, d, device="cuda", dtype=dtype)
        v[:, at, :, f] = 1.0
        want = torch.zeros(B, Lq, h, d, dtype=torch.float64, device="cuda")
        want[:, :, :, :len(at)] = torch.where(at[None] < seen[:, None], 1.0 / seen[:, None], 0.0)[:, None]
        got = S.run_attention(bnd, q, k, v, causal=causal, q_offset=off if causal else 0, cap=cap)
        R.check(got, want, want * (R.HALF[dtype] + 2.0 ** -8 * (dtype == F32) + 2.0 ** -10) + 0.0, "every key once")
