"""The operators around a cache in 8 bits on the GPU, against plain forms (tests/coded_ref.py)."""
import math
import random

import pytest

torch = pytest.importorskip("torch")

import coded_ref as C  # noqa: E402
import serving_ref as R  # noqa: E402

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32
E4, I8 = torch.float8_e4m3fn, torch.int8


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


def freqs(r):
    return (10000.0 ** (-torch.arange(0, r, 2, dtype=torch.float64) / r)).float().cuda()


def table_of(seed, B, per, extra=3):
    ids = list(range(B * per + extra))
    random.Random(seed).shuffle(ids)
    return ints([ids[b * per:(b + 1) * per] for b in range(B)]), B * per + extra


def pages_of(seed, n_pages, page, block, hk, d, code, order="slots"):
    """Pages of normal values, a size for each block and head, as codes, and their scales."""
    shape = (n_pages, page, hk, d) if order == "slots" else (n_pages, hk, page, d)
    x = randn(seed, *shape) * (100.0 if code == E4 else 40.0)
    x = x.clamp(-C.TOP[code], C.TOP[code])
    pages = torch.round(x).to(I8) if code == I8 else x.to(E4)
    g = torch.Generator(device="cuda").manual_seed(seed + 7)
    scales = torch.exp2(torch.randint(-9, -4, (n_pages, page // block, hk), generator=g, device="cuda").float())
    return (pages if order == "slots" else pages.transpose(1, 2)), scales


def same(a, b):
    """Bits, for types that have no comparison."""
    return torch.equal(a.contiguous().view(torch.uint8), b.contiguous().view(torch.uint8))


# ------------------------------------------------------------------------------------------ append
APPEND = [
    # dtype, code, T, h, h_kv, d, rot, interleaved, page, block, order, starts, new_lens
    (BF, E4, 1, 4, 2, 64, 64, False, 16, 16, "slots", [0, 15, 16], None),
    (BF, I8, 1, 8, 1, 128, 64, True, 16, 4, "slots", [3, 0, 7], [1, 0, 1]),
    (BF, E4, 40, 4, 4, 64, 32, False, 24, 8, "heads", [0, 23, 50], [40, 0, 17]),
    (BF, I8, 33, 2, 2, 128, 128, True, 64, 64, "heads", [60, 64, 1], None),
    (BF, E4, 33, 5, 3, 64, 22, False, 8, 8, "slots", [0, 23, 50], [33, 1, 17]),         # halves of 11: through shared memory
    (BF, I8, 300, 3, 1, 128, 126, False, 256, 256, "slots", [0, 100, 255], [300, 157, 299]),
    (BF, E4, 520, 2, 2, 128, 128, False, 256, 256, "slots", [3, 250], None),            # rows read twice
    (BF, E4, 130, 1, 5, 64, 64, False, 128, 128, "heads", [0, 64], None),
    (BF, I8, 50, 2, 2, 64, 0, False, 1, 1, "slots", [0, 7], None),                      # a scale a token
    (BF, E4, 70, 6, 2, 128, 16, False, 100, 25, "slots", [99, 0], [70, 69]),
    (F32, E4, 21, 3, 1, 64, 64, False, 8, 4, "slots", [5, 0, 90], [21, 1, 20]),
    (F32, I8, 5, 2, 2, 128, 6, True, 7, 7, "slots", [5, 0, 9], [5, -2, 9]),             # lengths beyond T and below 0
    (F32, E4, 257, 2, 2, 128, 100, False, 256, 256, "heads", [1, 255], None),
    (F32, I8, 100, 1, 3, 64, 62, False, 32, 16, "slots", [17], None),
    (F32, E4, 1, 9, 3, 128, 128, False, 32, 32, "slots", list(range(40)), None),
    # numbers of heads that do not divide among CTAs
    (BF, E4, 363, 15, 5, 128, 50, False, 128, 64, "slots", [1, 0, 70], None),
    (F32, I8, 300, 7, 3, 64, 64, True, 64, 64, "slots", [5], None),
    (BF, I8, 200, 11, 1, 128, 64, False, 32, 16, "slots", [3, 40], [200, 133]),
    (F32, E4, 513, 32, 8, 128, 64, False, 64, 64, "heads", [2], None),
    (BF, E4, 2, 64, 16, 64, 20, False, 256, 256, "slots", [254, 255, 256, 0, 13], None),
]
# blocks of one pass of rows and of two, in few and in many tiles; each way of turning
for _i, (_dt, _d, _b) in enumerate([(BF, 128, 4), (BF, 64, 8), (F32, 128, 2), (F32, 64, 4), (BF, 128, 8), (BF, 64, 16), (F32, 128, 4), (F32, 64, 8)]):
    for _j, (_rot, _inter) in enumerate([(0, False), (24, True), (_d // 2, False), (22, False)]):
        _rng, _n = random.Random(4 * _i + _j), 80 if _j == _i % 4 else 9
        APPEND.append((_dt, (E4, I8)[(_i + _j) % 2], 33 + _i, 3 + _j, 1 + _j % 2, _d, _rot, _inter, 16, _b, ("slots", "heads")[_j % 2],
                       [_rng.randint(0, 40) for _ in range(_n)], [_rng.randint(0, 33 + _i) for _ in range(_n)] if _j > 1 else None))


def run_append(bnd, dtype, code, T, h, hk, d, rot, inter, page, block, order, start, lens, big=4.0, first=8):
    B = len(start)
    per = -(-(max(start) + T) // page)
    table, n_pages = table_of(5, B, per)
    kp, ks = pages_of(6, n_pages, page, block, hk, d, code, order)
    vp, vs = pages_of(7, n_pages, page, block, hk, d, code, order)
    qkv = randn(first, B, T, h + 2 * hk, d, dtype=dtype) * big
    q, k, v = qkv[:, :, :h], qkv[:, :, h:h + hk], qkv[:, :, h + hk:]
    qo, ko = randn(9, B, T, h, d, dtype=dtype), randn(10, B, T, hk, d, dtype=dtype)
    q0, k0 = qo.clone(), ko.clone()
    f = freqs(rot) if rot else None
    pos = ints(start)[:, None] + torch.arange(T, device="cuda")
    turned = R.rotate(k, pos, f, inter, 1.25) if rot else k.double()
    ktol = R.rotate_tol(k, turned, f, inter, F32, 1.25) if rot else torch.zeros_like(turned)
    kw, kt, ksw, kn = C.append(kp, ks, turned, ktol, table, start, lens, page, block)
    vw, vt, vsw, vn = C.append(vp, vs, v.double(), torch.zeros_like(turned), table, start, lens, page, block)
    cache = bnd.make_coded_cache(kp, vp, ks, vs, table)
    rotary = bnd.make_rotary(f, inter, 1.25) if rot else None
    bnd.mha_coded_append(k, v, ints(start), cache=cache, q=q, q_out=qo, k_out=ko, new_lens=None if lens is None else ints(lens), rotary=rotary)
    qr = R.rotate(q, pos, f, inter, 1.25) if rot else q.double()
    for b in range(B):
        n = T if lens is None else min(max(lens[b], 0), T)
        if rot:
            R.check(qo[b, :n], qr[b, :n], R.rotate_tol(q, qr, f, inter, dtype, 1.25)[b, :n], "q")
            R.check(ko[b, :n], turned[b, :n], R.rotate_tol(k, turned, f, inter, dtype, 1.25)[b, :n], "k")
        else:
            assert torch.equal(qo[b, :n], q[b, :n]) and torch.equal(ko[b, :n], k[b, :n])
        assert torch.equal(qo[b, n:], q0[b, n:]) and torch.equal(ko[b, n:], k0[b, n:])   # left as they were
    assert torch.equal(torch.where(kn, 0.0, ks.double()), torch.where(kn, 0.0, ksw)) and torch.equal(vs.double(), vsw) and not vn.any()
    R.check(C.values(kp, ks), kw, kt, "keys")               # zero tolerance where nothing was written
    R.check(C.values(vp, vs), vw, vt, "values")
    return kp, ks, vp, vs


@pytest.mark.parametrize("case", APPEND)
def test_append(bnd, case):
    run_append(bnd, *case)


@pytest.mark.parametrize("code", [E4, I8])
@pytest.mark.parametrize("dtype", [BF, F32])
def test_append_rounds_to_the_nearest_code(bnd, dtype, code):
    """Without rotation every code is the value over its scale as torch rounds it (nearest even), ties among them."""
    B, T, hk, d, page = 1, 64, 2, 64, 64
    x = (torch.arange(T * hk * d, device="cuda").view(B, T, hk, d) % 1021 - 510).float() / 4       # quarters: ties of int8
    x[..., 0] = 100.0
    x = x.to(dtype)
    kp, ks = torch.zeros(2, page, hk, d, device="cuda", dtype=F32).to(code), torch.zeros(2, 1, hk, device="cuda")
    vp, vs = kp.clone(), ks.clone()
    bnd.mha_coded_append(x, -x, ints([0]), cache=bnd.make_coded_cache(kp, vp, ks, vs, ints([[1]])))
    s = torch.tensor([C.scale_for(x[0, :, i].float().abs().max().item(), code) for i in range(hk)], device="cuda")
    assert torch.equal(ks[1, 0], s) and torch.equal(vs[1, 0], s) and not ks[0].any()
    y = x[0].float() / s[:, None]
    want = torch.round(y).to(I8) if code == I8 else y.to(E4)
    assert same(kp[1], want)
    back = torch.round(-y).to(I8) if code == I8 else (-y).to(E4)
    assert same(vp[1], back)


def test_a_block_grows_token_by_token(bnd):
    """Tokens that enter one by one, ever larger: e4m3 codes stay what they stand for (but for subnormals), the scale follows, and a
    token at the first slot begins the block anew."""
    page = block = 16
    hk, d = 2, 64
    for code in (E4, I8):
        kp, ks = torch.zeros(3, page, hk, d, device="cuda").to(code), torch.full((3, 1, hk), 777.0, device="cuda")
        vp, vs = kp.clone(), ks.clone()
        cache = bnd.make_coded_cache(kp, vp, ks, vs, ints([[2, 0]]))
        x = randn(1, 1, 20, hk, d, dtype=BF) * torch.exp2(torch.arange(20, device="cuda").float() % 16 / 2)[None, :, None, None].to(BF)
        for t in range(20):
            bnd.mha_coded_append(x[:, t:t + 1], x[:, t:t + 1], ints([t]), cache=cache)
            top = x[0, t - t % 16:t + 1].float().abs().amax(dim=(0, 2)).tolist()
            assert ks[2 if t < 16 else 0, 0].tolist() == [C.scale_for(v, code) for v in top]
        got = C.values(kp, ks)[ints([2, 0]).long()].flatten(0, 1)[:20]
        # every growth of a scale rounds once more; int8: half a step of every scale on the way, together less than one of the last
        step = (ks if code == I8 else ks * 2.0 ** -9)[ints([2, 0]).long()].double().repeat_interleave(16, dim=1).flatten(0, 1)[:20, :, None]
        R.check(got, x[0].double(), step + (0 if code == I8 else x[0].double().abs() * 2.0 ** -4), "grown")
        assert torch.equal(ks, vs) and same(kp, vp)


def test_append_keeps_a_larger_scale_of_any_mantissa(bnd):
    page = block = 8
    kp, ks = pages_of(3, 2, page, block, 1, 64, E4)
    vp, vs = kp.clone(), ks.clone()
    ks.fill_(3.3)
    vs.fill_(0.0)
    before = kp.clone()
    x = randn(4, 1, 2, 1, 64, dtype=F32) * 50
    bnd.mha_coded_append(x, x, ints([3]), cache=bnd.make_coded_cache(kp, vp, ks, vs, ints([[1]])))
    assert (ks == torch.tensor(3.3)).all() and same(kp[1, :3], before[1, :3]) and same(kp[0], before[0])
    assert same(kp[1, 3:5], (x[0] / ks[1, 0, 0]).to(E4))
    R.check(C.values(kp, ks)[1, 3:5], x[0].double(), C.half_step(x[0].double(), 3.300001, E4) * (1 + 1e-6), "kept scale")
    assert vs[1, 0, 0].item() == C.scale_for(x.abs().max().item(), E4) and not vp[1, :3].float().any()     # codes of scale 0


@pytest.mark.parametrize("code", [E4, I8])
def test_append_shows_what_is_not_finite(bnd, code):
    """A NaN or an infinity makes its block's scale NaN, other blocks and heads are as without it; the next owner begins anew."""
    page, block, hk, d, T = 8, 4, 2, 64, 16
    table = ints([[1, 0]])
    x = randn(1, 1, T, hk, d, dtype=BF)
    y = x.clone()
    y[0, 5, 1, 7] = math.nan
    y[0, 13, 0, 0] = -math.inf
    kept = []
    for z in (x, y, x):
        if not kept:
            kp, ks = torch.zeros(2, page, hk, d, device="cuda").to(code), torch.zeros(2, 2, hk, device="cuda")
            vp, vs = kp.clone(), ks.clone()
            cache = bnd.make_coded_cache(kp, vp, ks, vs, table)
        bnd.mha_coded_append(z, z, ints([0]), cache=cache)
        kept.append((kp.clone(), ks.clone()))
        assert same(kp, vp) and torch.equal(torch.nan_to_num(ks, 5.0), torch.nan_to_num(vs, 5.0))
    bad = torch.zeros(2, 2, hk, dtype=torch.bool, device="cuda")
    bad[1, 1, 1] = bad[0, 1, 0] = True
    assert torch.equal(torch.isnan(kept[1][1]), bad) and torch.equal(kept[1][1][~bad], kept[0][1][~bad])
    rows = ~bad.repeat_interleave(block, dim=1)
    assert same(kept[1][0].view(torch.uint8)[rows], kept[0][0].view(torch.uint8)[rows])
    assert same(kept[2][0], kept[0][0]) and torch.equal(kept[2][1], kept[0][1])
    # a finite token behind a NaN leaves it
    bnd.mha_coded_append(y[:, 5:6], y[:, 5:6], ints([5]), cache=cache)
    bnd.mha_coded_append(x[:, 6:7], x[:, 6:7], ints([6]), cache=cache)
    assert math.isnan(ks[1, 1, 1].item()) and ks[1, 1, 0].item() > 0


@pytest.mark.parametrize("dtype,d,rot,interleaved", [(BF, 64, 22, True), (BF, 128, 36, True), (F32, 64, 6, True), (F32, 128, 70, True),
                                                     (BF, 64, 22, False), (F32, 128, 64, False), (F32, 64, 6, False)])
def test_append_leaves_what_does_not_turn(bnd, dtype, d, rot, interleaved):
    """Elements behind rot_dim come out bit for bit, infinities, negative zeros and their neighbours too; a NaN is one."""
    T, h, hk = 5, 3, 2
    q, k = randn(1, 1, T, h, d, dtype=dtype), randn(2, 1, T, hk, d, dtype=dtype)
    for x in (q, k):
        for i, odd in enumerate((math.inf, -math.inf, math.nan, -0.0)):
            x[0, i, :, rot + i] = odd
            x[0, i, :, d - 1] = odd
    kp, ks = torch.zeros(1, 8, hk, d, device="cuda").to(E4), torch.zeros(1, 2, hk, device="cuda")
    vp, vs = kp.clone(), ks.clone()
    qo, ko = torch.zeros_like(q), torch.zeros_like(k)
    bnd.mha_coded_append(k, k, ints([1]), cache=bnd.make_coded_cache(kp, vp, ks, vs, ints([[0]])), q=q, q_out=qo, k_out=ko,
                         rotary=bnd.make_rotary(freqs(rot), interleaved))
    for got, x in ((qo[..., rot:], q[..., rot:]), (ko[..., rot:], k[..., rot:])):
        assert torch.equal(torch.isnan(got), torch.isnan(x))        # bf16: of whatever bits, conversions write their own
        assert same(torch.nan_to_num(got, 0.0, math.inf, -math.inf), torch.nan_to_num(x, 0.0, math.inf, -math.inf))
    assert torch.isfinite(qo[..., :rot]).all() and torch.isfinite(ko[..., :rot]).all()


def test_append_of_extreme_sizes(bnd):
    """Values at the ends of fp32's range, and nothing but zeros."""
    page = block = 4
    for top in (3.0e38, 1e30, 1e-30, 1e-38, 0.0):
        x = torch.zeros(1, 4, 1, 64, device="cuda")
        x[..., 3], x[..., 5] = top, -top / 3
        for code in (E4, I8):
            kp, ks = torch.zeros(1, page, 1, 64, device="cuda").to(code), torch.zeros(1, 1, 1, device="cuda")
            vp, vs = kp.clone(), ks.clone()
            bnd.mha_coded_append(x, x, ints([0]), cache=bnd.make_coded_cache(kp, vp, ks, vs, ints([[0]])))
            assert ks.item() == C.scale_for(x.abs().max().item(), code)
            R.check(C.values(kp, ks)[0], x[0].double(), C.half_step(x[0].double(), ks.item(), code), str((top, code)))


def test_append_never_follows_a_bad_page(bnd):
    B, T, hk, d, page = 4, 4, 1, 64, 4
    table = ints([[0, 1], [-1, 2], [99, 3], [4, 5]])
    kp, ks = pages_of(2, 6, page, 2, hk, d, E4)
    vp, vs = pages_of(3, 6, page, 2, hk, d, E4)
    k0, s0 = kp.clone(), ks.clone()
    k = randn(3, B, T, hk, d, dtype=BF)
    q, qo, ko = randn(4, B, T, 2, d, dtype=BF), torch.zeros(B, T, 2, d, device="cuda", dtype=BF), torch.zeros_like(k)
    bnd.mha_coded_append(k, k, ints([6, 0, 2, -2]), cache=bnd.make_coded_cache(kp, vp, ks, vs, table), q=q, q_out=qo, k_out=ko)
    assert bnd.mha_check_device_status(reset=True) == bnd.MHA_PAGED_BAD_PAGE
    assert torch.equal(qo, q) and torch.equal(ko, k)                 # queries and keys are turned all the same
    written = torch.zeros(6, page, dtype=torch.bool, device="cuda")
    written[1, 2:] = written[3, :2] = written[4, :2] = True          # positions 6, 7; 4, 5; 0, 1
    assert same(kp.view(torch.uint8)[~written], k0.view(torch.uint8)[~written])
    blocks = written.view(6, 2, 2).any(dim=2)
    assert torch.equal(ks[~blocks], s0[~blocks])
    for pg, sl, b, t in ((1, 2, 0, 0), (3, 0, 2, 2), (4, 0, 3, 2)):
        got = C.values(kp, ks)[pg, sl:sl + 2]
        x = k[b, t:t + 2].double()
        R.check(got, x, C.half_step(x, ks[pg, sl // 2, 0].item(), E4), "good pages")


def test_append_in_place_and_broadcast(bnd):
    """Keys and queries turned in place (blocks that are read twice too), a broadcast value, no queries."""
    for dtype, block in ((BF, 16), (BF, 256), (F32, 256)):
        T, h, hk, d = 300, 3, 2, 128
        table, n_pages = table_of(1, 1, -(-T // 256) + 1)
        new = lambda: (torch.zeros(n_pages, 256, hk, d, device="cuda").to(I8), torch.ones(n_pages, 256 // block, hk, device="cuda"))  # noqa: E731
        q, k = randn(1, 1, T, h, d, dtype=dtype), randn(2, 1, T, hk, d, dtype=dtype)
        v = randn(3, 1, 1, 1, d, dtype=dtype).expand(1, T, hk, d)
        r = bnd.make_rotary(freqs(128))
        (kp, ks), (vp, vs) = new(), new()
        qo, ko = torch.empty_like(q), torch.empty_like(k)
        bnd.mha_coded_append(k, v, ints([9]), cache=bnd.make_coded_cache(kp, vp, ks, vs, table), q=q, q_out=qo, k_out=ko, rotary=r)
        (kp2, ks2), (vp2, vs2) = new(), new()
        bnd.mha_coded_append(k, v, ints([9]), cache=bnd.make_coded_cache(kp2, vp2, ks2, vs2, table), q=q, q_out=q, k_out=k, rotary=r)
        assert torch.equal(q, qo) and torch.equal(k, ko) and same(kp, kp2) and same(vp, vp2)
        assert torch.equal(ks, ks2) and torch.equal(vs, vs2)
        (kp3, ks3), (vp3, vs3) = new(), new()
        bnd.mha_coded_append(k, v, ints([9]), cache=bnd.make_coded_cache(kp3, vp3, ks3, vs3, table))       # as they are
        assert same(vp, vp3) and torch.equal(vs, vs3)


# ------------------------------------------------------------------------------------------ attention
def slopes_of(h):
    return torch.tensor([2.0 ** (-8.0 * (i + 1) / h) for i in range(h)], device="cuda")


def run_attention(bnd, q, kp, ks, vp, vs, table, lens, hk, out=None, **scores):
    B, h, d = q.shape
    dt = bnd.MHA_BF16 if q.dtype == BF else bnd.MHA_F32
    ws = torch.full((bnd.coded_attention_workspace_size(dt, B, h, hk, d),), 0xff, dtype=torch.uint8, device="cuda")   # NaN
    out = torch.full_like(q, float("nan")) if out is None else out
    bnd.mha_coded_attention(q, ints(lens), cache=bnd.make_coded_cache(kp, vp, ks, vs, table), out=out, workspace=ws,
                            scores=bnd.make_scores(**scores) if scores else None)
    return out


def poison(kp, ks, vp, vs, table, lens, block):
    """NaN codes in every slot that no sequence holds, NaN scales of every block without such a slot."""
    page = kp.shape[1]
    keep = torch.zeros(kp.shape[0], page, dtype=torch.bool, device="cuda")
    for b, n in enumerate(lens):
        for j in range(max(n, 0)):
            keep[table[b, j // page], j % page] = True
    if kp.dtype == E4:
        for x in (kp, vp):
            x.view(torch.uint8)[~keep] = 0x7f
    blocks = keep.view(kp.shape[0], page // block, block).any(dim=2)
    ks[~blocks] = float("nan")
    vs[~blocks] = float("inf")


ATTEND = [
    # dtype, code, h, h_kv, d, page, block, order, lens, scores
    (BF, E4, 4, 4, 64, 16, 16, "slots", [1, 0, 15, 16, 17, 100], {}),
    (BF, I8, 8, 2, 64, 16, 8, "heads", [33, 1, 0, 640], {}),
    (BF, E4, 8, 1, 128, 64, 64, "slots", [63, 64, 65, 500], dict(cap=20.0)),
    (BF, I8, 6, 2, 128, 24, 24, "slots", [777, 24, 25], dict(slopes=True)),
    (BF, E4, 10, 2, 64, 1, 1, "slots", [130, 5], dict(cap=5.0, slopes=True)),
    (BF, I8, 16, 1, 128, 7, 7, "heads", [300, 29], dict(scale=0.3)),
    (BF, E4, 20, 1, 64, 32, 4, "slots", [257, 31, 1], dict(slopes=True)),        # more than 16 heads share a key head
    (BF, E4, 20, 1, 128, 32, 32, "slots", [1025, 31, 1], {}),
    (BF, I8, 64, 1, 128, 128, 32, "slots", [129], {}),
    (BF, E4, 33, 11, 64, 100, 25, "slots", [201, 99, 100, 0], {}),
    (BF, I8, 7, 7, 128, 16, 16, "slots", [2000, 3], {}),
    (BF, E4, 8, 2, 64, 16, 16, "slots", [300, 0, 256, 257, 1, 700, 512, 768, 513, 2, 900, 1024, 1025], {}),    # units of 0 to 5 blocks
    (BF, I8, 12, 12, 128, 32, 16, "slots", [448, 129, 128, 127] * 20, {}),            # more units than SMs
    (BF, E4, 18, 2, 64, 16, 16, "heads", [1300, 40], dict(cap=30.0)),
    (F32, E4, 4, 4, 64, 16, 16, "slots", [1, 0, 15, 16, 17, 100], {}),
    (F32, I8, 8, 2, 128, 24, 8, "heads", [333, 1, 48], dict(cap=15.0)),
    (F32, E4, 9, 3, 64, 1, 1, "slots", [66, 2], dict(slopes=True)),
    (F32, I8, 20, 1, 128, 32, 32, "slots", [257, 1], dict(scale=-0.2)),
    (F32, E4, 16, 1, 64, 256, 256, "slots", [3000, 256, 255], {}),
    # two key heads of 64 at a time: a tile of query columns for both, or one each; pages stored head by head
    (BF, I8, 8, 4, 64, 16, 16, "slots", [700, 33], dict(slopes=True, cap=8.0)),
    (BF, E4, 16, 4, 64, 32, 8, "heads", [513, 1, 260], dict(slopes=True)),
    (BF, E4, 14, 2, 64, 16, 16, "heads", [300, 77], dict(cap=12.0)),
    (F32, E4, 6, 2, 64, 16, 16, "heads", [300, 77], dict(slopes=True)),
    (F32, I8, 12, 2, 64, 32, 16, "slots", [900, 2], dict(cap=10.0)),
    # many units, split and whole: two CTAs an SM
    (BF, E4, 16, 16, 64, 32, 32, "slots", [random.Random(5).randint(0, 3000) for _ in range(30)], {}),
    (F32, I8, 32, 8, 64, 32, 32, "slots", [random.Random(6).randint(0, 2500) for _ in range(45)], {}),
    (F32, E4, 8, 8, 128, 64, 64, "heads", [random.Random(7).randint(0, 900) for _ in range(25)], {}),
    (BF, I8, 16, 8, 128, 16, 16, "slots", [random.Random(8).randint(0, 1500) for _ in range(60)], dict(cap=25.0, slopes=True)),
]


@pytest.mark.parametrize("dtype,code,h,hk,d,page,block,order,lens,sc", ATTEND)
def test_attention(bnd, dtype, code, h, hk, d, page, block, order, lens, sc):
    B = len(lens)
    per = -(-max(lens) // page) + 1
    table, n_pages = table_of(11, B, per)
    kp, ks = pages_of(12, n_pages, page, block, hk, d, code, order)
    vp, vs = pages_of(13, n_pages, page, block, hk, d, code, order)
    poison(kp, ks, vp, vs, table, lens, block)
    q = randn(14, h, B, d, dtype=dtype).transpose(0, 1) * 2.0           # strides of [h, B, d]
    sc = dict(sc)
    if sc.get("slopes"):
        sc["slopes"] = slopes_of(h)
    got = run_attention(bnd, q, kp, ks, vp, vs, table, lens, hk, **sc)
    ref, tol = C.attention(q, kp, ks, vp, vs, table, lens, hk, **sc)
    R.check(got, ref, tol, "attention")
    assert torch.equal(got, run_attention(bnd, q, kp, ks, vp, vs, table, lens, hk, **sc))    # does not depend on timing
    for b, n in enumerate(lens):
        if n <= 0:
            assert torch.equal(got[b], torch.zeros_like(got[b]))


@pytest.mark.parametrize("dtype,code,B,h,hk,d,n", [(BF, E4, 1, 16, 2, 128, 70001), (BF, I8, 2, 4, 4, 64, 30000), (F32, E4, 1, 4, 1, 64, 40001),
                                                   (F32, I8, 2, 8, 1, 128, 20000), (BF, E4, 70, 4, 2, 64, 900), (BF, I8, 3, 16, 1, 128, 9000)])
def test_attention_long_and_many(bnd, dtype, code, B, h, hk, d, n):
    rng = random.Random(3)
    lens = [n] + [rng.choice([0, 1, n // 100, n // 3, n]) for _ in range(B - 1)]
    table, n_pages = table_of(15, B, -(-n // 64))
    kp, ks = pages_of(16, n_pages, 64, 16, hk, d, code)
    vp, vs = pages_of(17, n_pages, 64, 16, hk, d, code)
    q = randn(18, B, h, d, dtype=dtype) * 3.0
    got = run_attention(bnd, q, kp, ks, vp, vs, table, lens, hk)
    ref, tol = C.attention(q, kp, ks, vp, vs, table, lens, hk)
    R.check(got, ref, tol, "long")


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("code", [E4, I8])
@pytest.mark.parametrize("seed", [1, 2])
def test_attention_scales_of_any_size(bnd, dtype, code, seed):
    """Scales of values from 2^-60 to 2^60 within a sequence, keys' of any mantissa, blocks of scale 0: the running maximum of the
    weights follows score and scale."""
    h, hk, d, page, block, n = 6, 2, 64, 32, 8, 3000
    g = torch.Generator(device="cuda").manual_seed(seed)
    table, n_pages = table_of(seed, 1, -(-n // page))
    kp, ks = pages_of(20, n_pages, page, block, hk, d, code)
    vp, vs = pages_of(21, n_pages, page, block, hk, d, code)
    ks.mul_(1.0 + torch.rand(ks.shape, generator=g, device="cuda"))
    vs.copy_(torch.exp2(torch.rand(vs.shape, generator=g, device="cuda") * 120 - 60))
    vs[torch.rand(vs.shape, generator=g, device="cuda") < 0.1] = 0.0
    if seed == 2:                      # scores that outweigh the scales: the largest scale belongs to what nobody looks at
        vs.mul_(torch.where(vs > 2.0 ** 30, 2.0 ** -80, 1.0))
    q = randn(22, 1, h, d, dtype=dtype) * (2.0 if seed == 1 else 60.0)
    got = run_attention(bnd, q, kp, ks, vp, vs, table, [n], hk)
    ref, tol = C.attention(q, kp, ks, vp, vs, table, [n], hk)
    R.check(got, ref, tol, "scales")


@pytest.mark.parametrize("dtype", [BF, F32])
def test_attention_tiny_and_zero_value_scales(bnd, dtype):
    """All values tiny (2^-118), all of scale 0, and one block of scale 2^-120 among ordinary ones that its score dwarfs."""
    h, hk, d, page, n = 4, 1, 128, 16, 500
    table, n_pages = table_of(1, 1, -(-n // page))
    kp, ks = pages_of(30, n_pages, page, 16, hk, d, E4)
    vp, vs = pages_of(31, n_pages, page, 16, hk, d, E4)
    q = randn(32, 1, h, d, dtype=dtype)
    for fill in (2.0 ** -118, 0.0, 2.0 ** 100):
        vs.fill_(fill)
        got = run_attention(bnd, q, kp, ks, vp, vs, table, [n], hk)
        ref, tol = C.attention(q, kp, ks, vp, vs, table, [n], hk)
        R.check(got, ref, tol * 1.0 if fill != 2.0 ** -118 else tol - 1e-30 + 2.0 ** -126, str(fill))
    vs.fill_(0.25)
    vs[table[0, 3].long()] = 2.0 ** -120
    ks[table[0, 3].long()] *= 8.0
    got = run_attention(bnd, q, kp, ks, vp, vs, table, [n], hk)
    ref, tol = C.attention(q, kp, ks, vp, vs, table, [n], hk)
    R.check(got, ref, tol, "one tiny block")


@pytest.mark.parametrize("dtype,d,hk", [(BF, 128, 1), (F32, 64, 2)])
@pytest.mark.parametrize("cap", [1e-38, 1e-6, 1e6, 1e25, 3e38])
def test_attention_caps_of_any_size(bnd, dtype, d, hk, cap):
    """A cap far above the scores changes nothing, far below it leaves the mean; small and large scales of keys under it."""
    h, page, n = 4, 16, 900
    table, n_pages = table_of(2, 1, -(-n // page))
    kp, ks = pages_of(44, n_pages, page, 16, hk, d, E4)
    vp, vs = pages_of(45, n_pages, page, 16, hk, d, E4)
    for up in (1.0, 2.0 ** -40, 2.0 ** 40):
        q = (randn(46, 1, h, d, dtype=F32) * 3.0 / up).to(dtype)
        k2 = ks * up
        got = run_attention(bnd, q, kp, k2, vp, vs, table, [n], hk, cap=cap)
        # caps beyond 2^100 are taken as 2^100, below 2^-100 as that
        kept = min(max(cap, 2.0 ** -100), 2.0 ** 100)
        plain = kept > 1e20      # fp64 itself loses cap * tanh(s / cap) = s far above s
        ref, tol = C.attention(q, kp, k2, vp, vs, table, [n], hk, cap=0.0 if plain else kept)
        if cap >= 1e6:           # off by 2^-20 of the score, not of the cap
            ref2, tol = C.attention(q, kp, k2, vp, vs, table, [n], hk)
            assert (ref2 - ref).abs().max() <= 1e-9
            tol = tol + 2.0 ** -19 * 60.0 * vs.max().item() * 448.0
        R.check(got, ref, tol, str((cap, up)))


def test_attention_key_codes_that_are_nan(bnd):
    """A NaN code of a key reaches its key head's queries only, whichever heads share a tile."""
    for h, hk in ((4, 4), (8, 2), (12, 2), (2, 1)):
        d, page, n = 64, 16, 300
        table, n_pages = table_of(1, 1, -(-n // page))
        kp, ks = pages_of(64, n_pages, page, 16, hk, d, E4)
        vp, vs = pages_of(65, n_pages, page, 16, hk, d, E4)
        q = randn(66, 1, h, d, dtype=BF)
        clean = run_attention(bnd, q, kp, ks, vp, vs, table, [n], hk)
        kp.view(torch.uint8)[table[0, 2].long(), 5, 0, 3] = 0x7f
        got = run_attention(bnd, q, kp, ks, vp, vs, table, [n], hk)
        g = h // hk
        assert torch.isnan(got[:, :g]).all() and torch.equal(got[:, g:], clean[:, g:])


@pytest.mark.parametrize("dtype", [BF, F32])
def test_attention_queries_of_any_size(bnd, dtype):
    """Queries of 1e30 beside keys of 1e-30 and the other way round, a query of zeros (the mean of the values), one element far
    above the others."""
    h, hk, d, page, n = 4, 2, 64, 16, 300
    table, n_pages = table_of(1, 1, -(-n // page))
    kp, ks = pages_of(40, n_pages, page, 16, hk, d, I8)
    vp, vs = pages_of(41, n_pages, page, 16, hk, d, I8)
    ks.fill_(2.0 ** -5)
    for up in (2.0 ** 90, 2.0 ** -90, 1.0):
        q = randn(42, 1, h, d, dtype=dtype)
        if up == 1.0:
            q[0, 0] = 0.0
            q[0, 1, 5] = 2000.0
        else:
            q = q * up
        k2 = ks / up
        got = run_attention(bnd, q, kp, k2, vp, vs, table, [n], hk)
        ref, tol = C.attention(q, kp, k2, vp, vs, table, [n], hk)
        R.check(got, ref, tol, str(up))


@pytest.mark.parametrize("dtype,h,hk,d", [(BF, 4, 2, 64), (F32, 3, 1, 128)])
def test_attention_codes_and_scales_of_other_origin(bnd, dtype, h, hk, d):
    """The code -128, key scales of 0 (equal scores) beside others, lengths below 0, another stream."""
    page, n = 16, 200
    table, n_pages = table_of(3, 3, -(-n // page))
    kp, ks = pages_of(47, n_pages, page, 16, hk, d, I8)
    vp, vs = pages_of(48, n_pages, page, 16, hk, d, I8)
    kp[kp > 60] = -128
    vp[vp > 60] = -128
    ks[::3] = 0.0
    q = randn(49, 3, h, d, dtype=dtype)
    lens = [n, -7, 33]
    got = run_attention(bnd, q, kp, ks, vp, vs, table, lens, hk)
    ref, tol = C.attention(q, kp, ks, vp, vs, table, lens, hk)
    R.check(got, ref, tol, "other origin")
    assert not got[1].any()
    side, out = torch.cuda.Stream(), torch.full_like(q, float("nan"))
    dt = bnd.MHA_BF16 if dtype == BF else bnd.MHA_F32
    ws = torch.zeros(bnd.coded_attention_workspace_size(dt, 3, h, hk, d), dtype=torch.uint8, device="cuda")
    cache, kv_lens = bnd.make_coded_cache(kp, vp, ks, vs, table), ints(lens)
    torch.cuda.synchronize()
    bnd.mha_coded_attention(q, kv_lens, cache=cache, out=out, workspace=ws, stream=side)
    side.synchronize()
    assert torch.equal(out, got)
    # appended to: codes rounded again from -128
    x = randn(50, 3, 1, hk, d, dtype=dtype) * 1e4
    before = C.values(kp, ks)
    held = [199, 0, 33]
    bnd.mha_coded_append(x, x, ints(held), cache=cache, new_lens=ints([1, 0, 1]), stream=side)
    side.synchronize()
    for b in (0, 2):
        pg, sl = table[b, held[b] // page].item(), held[b] % page
        now = C.values(kp, ks)[pg]
        R.check(now[:sl], before[pg, :sl], (ks[pg].double() / 2)[..., None].expand(sl, hk, d), "rounded again")
        R.check(now[sl], x[b, 0].double(), C.half_step(x[b, 0].double(), ks[pg, 0].double()[:, None], I8), "appended")


def test_two_calls_at_once(bnd):
    """Attention and append of two batches on two streams, a workspace each: as one after the other."""
    B, h, hk, d, page, n = 6, 8, 2, 128, 16, 3000
    sets = []
    for i in range(2):
        table, n_pages = table_of(i, B, -(-n // page) + 1)
        kp, ks = pages_of(60 + i, n_pages, page, 16, hk, d, E4)
        vp, vs = pages_of(70 + i, n_pages, page, 16, hk, d, E4)
        ws = torch.zeros(bnd.coded_attention_workspace_size(bnd.MHA_BF16, B, h, hk, d), dtype=torch.uint8, device="cuda")
        q, x = randn(80 + i, B, h, d, dtype=BF), randn(90 + i, B, 1, hk, d, dtype=BF)
        sets.append((bnd.make_coded_cache(kp, vp, ks, vs, table), q, x, ints([n - 37 * b for b in range(B)]), ws, torch.zeros_like(q)))
    def both(streams):
        for (cache, q, x, lens, ws, out), s in zip(sets, streams):
            bnd.mha_coded_append(x, x, lens, cache=cache, stream=s)
            bnd.mha_coded_attention(q, lens, cache=cache, out=out, workspace=ws, stream=s)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    both(streams)
    torch.cuda.synchronize()
    first = [s[5].clone() for s in sets]
    for _ in range(5):
        both(streams)
    torch.cuda.synchronize()
    assert all(torch.equal(a, s[5]) for a, s in zip(first, sets))
    for (cache, q, x, lens, ws, out), f in zip(sets, first):
        bnd.mha_coded_attention(q, lens, cache=cache, out=out, workspace=ws)
        assert torch.equal(out, f)


def test_attention_large_scores_and_shared_pages(bnd):
    h, hk, d, page = 4, 2, 64, 16
    kp, ks = pages_of(50, 40, page, 16, hk, d, E4)
    vp, vs = pages_of(51, 40, page, 16, hk, d, E4)
    table = ints([[0, 1, 2, 3 + b] for b in range(8)])
    lens = [64, 63, 49, 48, 33, 17, 16, 1]
    q = randn(52, 8, h, d, dtype=BF) * 100.0
    got = run_attention(bnd, q, kp, ks, vp, vs, table, lens, hk)
    ref, tol = C.attention(q, kp, ks, vp, vs, table, lens, hk)
    R.check(got, ref, tol, "large scores")


def test_attention_not_finite(bnd):
    """A NaN scale of keys, a NaN query, a NaN code of a value: what depends on it is NaN, and nothing else."""
    h, hk, d, page, n = 4, 2, 64, 16, 700
    table, n_pages = table_of(1, 3, -(-n // page))
    kp, ks = pages_of(60, n_pages, page, 16, hk, d, E4)
    vp, vs = pages_of(61, n_pages, page, 16, hk, d, E4)
    q = randn(62, 3, h, d, dtype=BF)
    clean = run_attention(bnd, q, kp, ks, vp, vs, table, [n] * 3, hk)
    ks[table[0, 20].long(), 0, 1] = math.nan                       # sequence 0, key head 1
    q[1, 2, 9] = math.nan                                          # sequence 1, head 2
    vp.view(torch.uint8)[table[2, 0].long(), 3, 0, 11] = 0xff      # sequence 2, key head 0, feature 11
    got = run_attention(bnd, q, kp, ks, vp, vs, table, [n] * 3, hk)
    bad = torch.zeros_like(got, dtype=torch.bool)
    bad[0, 2:] = bad[1, 2] = bad[2, :2, 11] = True
    assert torch.equal(torch.isnan(got), bad) and torch.equal(got[~bad], clean[~bad])


def test_attention_never_follows_a_bad_page(bnd):
    h, hk, d, page = 2, 1, 64, 16
    table = ints([[0, -1, 1], [2, 99, 3], [-5, -5, -5]])
    kp, ks = pages_of(70, 4, page, 16, hk, d, I8)
    vp, vs = pages_of(71, 4, page, 16, hk, d, I8)
    q = randn(72, 3, h, d, dtype=BF)
    lens = [40, 48, 20]
    got = run_attention(bnd, q, kp, ks, vp, vs, table, lens, hk)
    assert bnd.mha_check_device_status(reset=True) == bnd.MHA_PAGED_BAD_PAGE
    bad = [(0, j) for j in range(16, 32)] + [(1, j) for j in range(16, 32)] + [(2, j) for j in range(20)]
    ref, tol = C.attention(q, kp, ks, vp, vs, table, lens, hk, bad=bad)
    R.check(got, ref, tol, "bad pages left out")
    out = torch.full((1, h, d), math.nan, device="cuda", dtype=BF)
    t1 = ints([[2]])
    got = run_attention(bnd, q[:1], kp, ks, vp, vs, t1, [500], hk, out=out)
    assert bnd.mha_check_device_status(reset=True) == bnd.MHA_PAGED_BAD_PAGE
    ref, tol = C.attention(q[:1], kp, ks, vp, vs, t1, [16], hk)
    R.check(got, ref, tol, "cut to the table")


MANY = [
    # dtype, code, B, h, h_kv, d, page, pages of a sequence, scores: many units, a table with little room
    (BF, E4, 50, 32, 8, 128, 32, 1, {}),
    (BF, I8, 200, 6, 2, 128, 24, 4, dict(cap=20.0)),
    (F32, E4, 90, 8, 4, 128, 64, 2, dict(slopes=True)),
    (F32, I8, 60, 16, 16, 128, 32, 16, {}),                   # room for 512
    (BF, I8, 130, 36, 3, 128, 128, 1, dict(slopes=True)),     # twelve query heads a key head
    (F32, E4, 100, 24, 2, 128, 16, 8, dict(cap=10.0)),
    (BF, E4, 70, 24, 8, 64, 256, 1, {}),                      # pairs of heads, one tile
    (F32, I8, 120, 12, 12, 64, 8, 12, dict(slopes=True, cap=9.0)),
    (BF, I8, 60, 64, 8, 64, 32, 3, {}),                       # pairs of heads, a tile each
    (F32, E4, 160, 32, 4, 64, 1, 77, {}),
    (BF, E4, 50, 35, 5, 64, 100, 2, dict(cap=30.0)),          # an odd number of key heads
    (F32, E4, 180, 5, 1, 64, 16, 2, dict(scale=0.4)),
    (BF, I8, 100, 36, 3, 64, 64, 2, dict(slopes=True)),
    (BF, E4, 1000, 10, 1, 64, 16, 32, {}),
    (BF, E4, 300, 30, 10, 128, 16, 1, {}),                    # more units than run at a time, many times over
]


@pytest.mark.parametrize("dtype,code,B,h,hk,d,page,per,sc,order", [c + ("heads" if i % 2 else "slots",) for i, c in enumerate(MANY)])
def test_attention_many_short(bnd, dtype, code, B, h, hk, d, page, per, sc, order):
    room = page * per
    rng = random.Random(B + d)
    lens = [rng.choice([0, 1, room, rng.randint(0, room), rng.randint(0, room)]) for _ in range(B)]
    block = next(b for b in (16, 8, 25, 4, 1) if page % b == 0)
    table, n_pages = table_of(61, B, per)
    kp, ks = pages_of(62, n_pages, page, block, hk, d, code, order)
    vp, vs = pages_of(63, n_pages, page, block, hk, d, code, order)
    poison(kp, ks, vp, vs, table, lens, block)
    q = randn(64, h, B, d, dtype=dtype).transpose(0, 1) * 2.0
    sc = dict(sc)
    if sc.get("slopes"):
        sc["slopes"] = slopes_of(h)
    got = run_attention(bnd, q, kp, ks, vp, vs, table, lens, hk, **sc)
    ref, tol = C.attention(q, kp, ks, vp, vs, table, lens, hk, **sc)
    R.check(got, ref, tol, "attention")
    assert torch.equal(got, run_attention(bnd, q, kp, ks, vp, vs, table, lens, hk, **sc))
    empty = [b for b, n in enumerate(lens) if n == 0]
    assert not got[empty].any()
    assert bnd.mha_check_device_status() == 0


def test_attention_many_short_and_bad_pages(bnd):
    """Bad pages, lengths beyond the table and below 0, among more units than SMs hold."""
    B, h, hk, d, page = 400, 3, 1, 128, 16
    rows = [[0, -1, 1], [2, 99, 3], [-5, -5, -5], [1, 2, 0]]
    lens = [40, 48, 20, 3]
    table = ints([rows[b % 4] for b in range(B)])
    kp, ks = pages_of(70, 4, page, 16, hk, d, I8)
    vp, vs = pages_of(71, 4, page, 16, hk, d, I8)
    q = randn(72, B, h, d, dtype=BF)
    n = [lens[b % 4] for b in range(B)]
    bad = [(b, j) for b in range(B) for j in (range(16, 32) if b % 4 < 2 else range(20) if b % 4 == 2 else ())]
    got = run_attention(bnd, q, kp, ks, vp, vs, table, n, hk)
    assert bnd.mha_check_device_status(reset=True) == bnd.MHA_PAGED_BAD_PAGE
    ref, tol = C.attention(q, kp, ks, vp, vs, table, n, hk, bad=bad)
    R.check(got, ref, tol, "bad pages left out")
    good = ints([rows[3]] * B)
    got = run_attention(bnd, q, kp, ks, vp, vs, good, [49 if b % 2 else -7 for b in range(B)], hk)
    assert bnd.mha_check_device_status(reset=True) == bnd.MHA_PAGED_BAD_PAGE
    ref, tol = C.attention(q, kp, ks, vp, vs, good, [48 if b % 2 else 0 for b in range(B)], hk)
    R.check(got, ref, tol, "cut to the table")


def test_attention_strided_query_and_output(bnd):
    """q a slice of a projection, a broadcast q, an output between other data, which stays."""
    B, h, hk, d, page, n = 3, 4, 2, 64, 16, 90
    table, n_pages = table_of(1, B, 6)
    kp, ks = pages_of(80, n_pages, page, 8, hk, d, E4)
    vp, vs = pages_of(81, n_pages, page, 8, hk, d, E4)
    qkv = randn(82, B, h + 2 * hk, d + 1, dtype=BF)[..., 1:]                   # heads that start at odd elements
    q = qkv[:, :h]
    big = torch.full((B, 2 * h, d + 3), 7.0, device="cuda", dtype=BF)
    out = big[:, ::2, 1:d + 1]
    got = run_attention(bnd, q, kp, ks, vp, vs, table, [n] * B, hk, out=out)
    ref, tol = C.attention(q, kp, ks, vp, vs, table, [n] * B, hk)
    R.check(got, ref, tol, "strided")
    out.fill_(7.0)
    assert (big == 7.0).all()
    one = randn(83, 1, 1, d, dtype=BF).expand(B, h, d)
    got = run_attention(bnd, one, kp, ks, vp, vs, table, [n] * B, hk, out=torch.empty(B, h, d, device="cuda", dtype=BF))
    ref, tol = C.attention(one, kp, ks, vp, vs, table, [n] * B, hk)
    R.check(got, ref, tol, "broadcast")


def test_attention_offsets_beyond_32_bits(bnd):
    """Pages more than 2^31 bytes (and 2^32) apart, and a scale index there."""
    h, hk, d, page, block = 2, 1, 64, 16, 16
    n_pages = (5 << 30) // (page * hk * d)
    kp = torch.zeros(n_pages, page, hk, d, device="cuda", dtype=I8)
    vp = torch.zeros(n_pages, page, hk, d, device="cuda", dtype=I8)
    ks, vs = torch.ones(n_pages, 1, hk, device="cuda"), torch.ones(n_pages, 1, hk, device="cuda")
    ids = [n_pages - 1, 0, (1 << 31) // (page * d) + 1, (1 << 32) // (page * d) + 5]
    small_k, sk = pages_of(90, 4, page, block, hk, d, I8)
    small_v, sv = pages_of(91, 4, page, block, hk, d, I8)
    at = torch.tensor(ids, device="cuda")
    kp[at], vp[at], ks[at], vs[at] = small_k, small_v, sk, sv
    q = randn(92, 1, h, d, dtype=BF)
    got = run_attention(bnd, q, kp, ks, vp, vs, ints([ids]), [60], hk)
    ref, tol = C.attention(q, small_k, sk, small_v, sv, ints([[0, 1, 2, 3]]), [60], hk)
    R.check(got, ref, tol, "far pages")
    x = randn(93, 1, 4, hk, d, dtype=BF)
    bnd.mha_coded_append(x, x, ints([60]), cache=bnd.make_coded_cache(kp, vp, ks, vs, ints([ids])))
    want = C.values(kp[at[3:]], ks[at[3:]])[0, 12:]
    R.check(want, x[0].double(), C.half_step(x[0].double(), ks[ids[3], 0, 0].item(), I8), "far append")


# ------------------------------------------------------------------------------------------ pages granted and returned
class Pool:
    def __init__(self, bnd, B, room, n_pages, page, seed=0, free=None, stride=None):
        self.bnd, self.page = bnd, page
        ids = list(range(n_pages))
        random.Random(seed).shuffle(ids)
        whole = torch.full((B, stride or room), -1, dtype=torch.int32, device="cuda")
        self.table = whole[:, :room]
        self.stack = ints(ids)
        self.count = ints([n_pages if free is None else free])
        self.lens, self.new = ints([0] * B), ints([0] * B)

    def step(self, held, want, T=0):
        """The call against the plain form, everything equal."""
        slots = torch.full((len(held), T), -7, dtype=torch.int64, device="cuda") if T else None
        ref = C.resize(held, want, self.page, self.table.tolist(), self.stack.tolist(), self.count.item(), T)
        self.bnd.mha_paged_resize(ints(held), ints(want), block_table=self.table, page_size=self.page, free_pages=self.stack,
                                  free_count=self.count, lens=self.lens, new_lens=self.new, slots=slots)
        got = (self.lens.tolist(), self.new.tolist(), slots.tolist() if T else [[]] * len(held), self.table.tolist(), self.stack.tolist(),
               self.count.item())
        for g, w, name in zip(got, ref, ("lens", "new_lens", "slots", "table", "stack", "count")):
            assert g == w, name
        return got[0]


RESIZE = [
    # B, room, pages, page size, T, most new, steps
    (1, 1, 1, 1, 1, 1, 6), (1, 40, 30, 16, 1, 1, 40), (3, 8, 11, 4, 5, 9, 30), (16, 70, 400, 16, 1, 1, 25), (5, 100, 300, 7, 33, 300, 20),
    (512, 9, 2000, 8, 2, 20, 6), (513, 9, 2000, 8, 3, 20, 6), (1500, 5, 4000, 24, 1, 60, 6), (64, 300, 9000, 16, 700, 3000, 4), (2, 5000, 9000, 1, 4000, 4500, 5),
    (40, 300, 6000, 16, 3500, 3400, 3), (1, 3000, 2900, 64, 140000, 150000, 3), (700, 12, 5000, 16, 190, 200, 3),       # slots by a kernel of their own
]


@pytest.mark.parametrize("B,room,n_pages,page,T,most,steps", RESIZE)
def test_resize(bnd, B, room, n_pages, page, T, most, steps):
    """Random steps: growth, ends, partial returns, a pool that runs dry, wishes beyond the table and below 0."""
    rng = random.Random(B * room + T)
    pool = Pool(bnd, B, room, n_pages, page, stride=room + 3)
    held = [0] * B
    for _ in range(steps):
        want = []
        for h in held:
            what = rng.random()
            want.append(h + rng.randint(0, most) if what < 0.6 else h if what < 0.7 else 0 if what < 0.8 else rng.randint(0, h) if what < 0.95 else
                        -3 if what < 0.97 else room * page + rng.randint(0, 2))
        held = pool.step(held, want, T if rng.random() < 0.8 else 0)
    pool.step(held, [0] * B)
    assert pool.count.item() == n_pages and sorted(pool.stack.tolist()) == list(range(n_pages)) and (pool.table == -1).all()


def test_resize_step_and_return(bnd):
    """A step, and the step back with held and want exchanged: table, stack and count are what they were."""
    B, room, page = 300, 40, 16
    pool = Pool(bnd, B, room, 9000, page)
    rng = random.Random(1)
    held = pool.step([0] * B, [rng.randint(0, 300) for _ in range(B)])
    before = (pool.table.clone(), pool.stack.clone(), pool.count.clone())
    want = [0 if rng.random() < 0.3 else min(h + rng.randint(0, 300), room * page) for h in held]
    lens = pool.step(held, want, 7)
    assert lens == want
    pool.step(lens, held)
    n = before[2].item()
    assert torch.equal(pool.table, before[0]) and pool.count.item() == n and torch.equal(pool.stack[:n], before[1][:n])


def test_resize_the_pool_runs_dry_in_order(bnd):
    """Sequences that need no page are served whatever is left; the first that does not fit, and those behind it that need pages, are not."""
    pool = Pool(bnd, 5, 8, 4, 4)
    assert pool.step([0] * 5, [4, 8, 8, 1, 0], 9) == [4, 8, 0, 0, 0]        # one page is left: two are wanted, then one
    assert pool.step([4, 8, 0, 0, 0], [4, 7, 0, 4, 0], 4) == [4, 7, 0, 4, 0]
    assert pool.step([4, 7, 0, 4, 0], [0, 8, 4, 4, 5], 4) == [0, 8, 4, 4, 0]   # the page given back serves; two more do not fit


def test_resize_many_slots_with_a_bad_page(bnd):
    """The slots of many tokens are a second kernel's: a page number outside the pool gives none there either."""
    pool = Pool(bnd, 3, 400, 1200, 128, free=1100)
    pool.table[1, 0] = 5000
    pool.step([0, 100, 0], [51200, 51000, 1], 51200)
    assert bnd.mha_check_device_status(reset=True) == bnd.MHA_PAGED_BAD_PAGE


def test_resize_on_another_stream(bnd):
    """The same step in the default stream and, by the stream argument, in another; held and want may be one array."""
    got = []
    for stream in (None, torch.cuda.Stream()):
        pool = Pool(bnd, 4, 8, 20, 4)
        want, slots = ints([3, 9, 0, 31]), torch.zeros(4, 5, dtype=torch.int64, device="cuda")
        torch.cuda.synchronize()
        for held in (ints([0, 0, 0, 0]), want):
            bnd.mha_paged_resize(held, want, block_table=pool.table, page_size=4, free_pages=pool.stack, free_count=pool.count, lens=pool.lens,
                                 new_lens=pool.new, slots=slots if held is not want else None, stream=stream)
        torch.cuda.synchronize()
        got.append((pool.table.tolist(), pool.count.item(), pool.lens.tolist(), pool.new.tolist(), slots.tolist()))
    assert got[0] == got[1] and got[0][1:4] == (8, [3, 9, 0, 31], [0, 0, 0, 0])


def test_resize_reports_what_is_out_of_range(bnd):
    """Pages returned twice overflow the stack: dropped and reported. A page number outside the pool gives no slot, and a count
    outside 0 .. n_pages is taken as the nearer end."""
    pool = Pool(bnd, 2, 4, 6, 4, free=5)
    pool.table.copy_(ints([[1, 2, -1, -1], [3, -1, -1, -1]]))
    pool.step([8, 4], [0, 0])
    assert pool.bnd.mha_check_device_status(reset=True) == bnd.MHA_PAGED_BAD_PAGE and pool.count.item() == 6
    pool = Pool(bnd, 2, 4, 6, 4, free=2)
    pool.table[0, 0] = 77
    pool.step([2, 0], [4, 4], 4)
    assert bnd.mha_check_device_status(reset=True) == bnd.MHA_PAGED_BAD_PAGE
    pool = Pool(bnd, 2, 4, 6, 4)
    pool.stack[5] = -1
    pool.step([0, 0], [4, 4], 4)
    assert bnd.mha_check_device_status(reset=True) == bnd.MHA_PAGED_BAD_PAGE
    for free, reach in ((99, [16, 8]), (-4, [0, 0])):
        pool = Pool(bnd, 2, 4, 6, 4, free=free)
        assert pool.step([0, 0], [16, 8], 3) == reach
    pool = Pool(bnd, 1, 3, 6, 4)
    assert pool.step([0], [2147483647], 2) == [0] and pool.step([2147483647], [5], 2) == [5]      # 3 pages held by the table
    assert bnd.mha_check_device_status(reset=True) == bnd.MHA_PAGED_BAD_PAGE                       # they were -1


# ------------------------------------------------------------------------------------------ together
@pytest.mark.parametrize("code", [E4, I8])
def test_serving_with_a_cache_in_8_bits(bnd, code):
    """Requests come, are answered token by token and end, over a pool that their pages return to: every step's table, appended values and
    attention against plain forms, with the values that the cache stands for."""
    rng = random.Random(4)
    B, h, hk, d, page, block, T, room, n_pages = 4, 6, 2, 64, 8, 8, 21, 12, 22
    kp, vp = (torch.zeros(n_pages, page, hk, d, device="cuda").to(code) for _ in range(2))
    ks, vs = (torch.full((n_pages, page // block, hk), math.nan, device="cuda") for _ in range(2))
    pool = Pool(bnd, B, room, n_pages, page)
    cache = bnd.make_coded_cache(kp, vp, ks, vs, pool.table)
    rotary, f = bnd.make_rotary(freqs(32)), freqs(32)
    kept = [torch.zeros(0, 2, hk, d, dtype=torch.float64, device="cuda") for _ in range(B)]      # turned keys and values
    held = [0] * B
    for it in range(30):
        want = []
        for b in range(B):
            if held[b] == 0:
                want.append(rng.randint(0, T) if rng.random() < 0.6 else 0)
            else:
                want.append(0 if rng.random() < 0.12 else min(held[b] + 1, room * page))
        lens = pool.step(held, want, T)
        start = [min(a, c) for a, c in zip(held, lens)]
        qkv = randn(100 + it, B, T, h + 2 * hk, d, dtype=BF) * math.exp(rng.uniform(-1, 1))
        q, k, v = qkv[:, :, :h], qkv[:, :, h:h + hk], qkv[:, :, h + hk:]
        q1 = torch.zeros(B, T, h, d, device="cuda", dtype=BF)
        bnd.mha_coded_append(k, v, ints(start), cache=cache, q=q, q_out=q1, new_lens=pool.new, rotary=rotary)
        kr = R.rotate(k, ints(start)[:, None] + torch.arange(T, device="cuda"), f)
        last = torch.zeros(B, h, d, device="cuda", dtype=BF)
        for b in range(B):
            n = lens[b] - start[b]
            kept[b] = torch.cat((kept[b][:start[b]], torch.stack((kr[b, :n], v[b, :n].double()), dim=1))) if lens[b] else kept[b][:0]
            if n:
                last[b] = q1[b, n - 1]
            rows = pool.table[b].long()
            m = lens[b]
            for i, (p, s) in enumerate(((kp, ks), (vp, vs))):
                if m:
                    got = C.values(p[rows[:-(-m // page)]], s[rows[:-(-m // page)]]).flatten(0, 1)[:m]
                    x = kept[b][:, i]
                    step = s[rows[:-(-m // page)]].double().repeat_interleave(block, dim=1).flatten(0, 1)[:m, :, None]
                    # a block that grows is rounded again: int8 half a step of each scale, less than one step together; e4m3 below 2^-6
                    tol = step if code == I8 else x.abs() * 2.0 ** -4 + step * 2.0 ** -9
                    R.check(got, x, tol + x.abs() * 2.0 ** -18 + 2.0 ** -18, "what the cache stands for")
        got = run_attention(bnd, last, kp, ks, vp, vs, pool.table, lens, hk)
        ref, tol = C.attention(last, kp, ks, vp, vs, pool.table, lens, hk)
        R.check(got, ref, tol, "attention")
        held = lens


def test_captured_steps_and_streams(bnd):
    """A step of the three operators captured into a graph and replayed while lengths move on the device, on a side stream; two graphs
    that share a workspace, one after the other."""
    B, h, hk, d, page, n_pages, room = 3, 4, 2, 64, 16, 40, 8
    kp, vp = (torch.zeros(n_pages, page, hk, d, device="cuda").to(E4) for _ in range(2))
    ks, vs = (torch.ones(n_pages, 1, hk, device="cuda") for _ in range(2))
    pool = Pool(bnd, B, room, n_pages, page)
    cache = bnd.make_coded_cache(kp, vp, ks, vs, pool.table)
    held, want = ints([0, 5, 30]), ints([1, 6, 31])
    pool.step([0, 0, 0], [0, 5, 30])
    x = randn(1, B, 1, h + 2 * hk, d, dtype=BF)
    q1, out = torch.zeros(B, 1, h, d, device="cuda", dtype=BF), torch.zeros(B, h, d, device="cuda", dtype=BF)
    ws = torch.zeros(bnd.coded_attention_workspace_size(bnd.MHA_BF16, B, h, hk, d), dtype=torch.uint8, device="cuda")
    slots = torch.zeros(B, 1, dtype=torch.int64, device="cuda")

    def step():
        bnd.mha_paged_resize(held, want, block_table=pool.table, page_size=page, free_pages=pool.stack, free_count=pool.count, lens=pool.lens,
                             new_lens=pool.new, slots=slots)
        bnd.mha_coded_append(x[:, :, h:h + hk], x[:, :, h + hk:], held, cache=cache, q=x[:, :, :h], q_out=q1, new_lens=pool.new)
        bnd.mha_coded_attention(q1[:, 0], pool.lens, cache=cache, out=out, workspace=ws)
        held.copy_(pool.lens)
        want.copy_(pool.lens + 1)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graphs = []
    with torch.cuda.stream(side):
        step()
        for _ in range(2):
            g = torch.cuda.CUDAGraph()
            with torch.cuda.graph(g, stream=side):
                step()
            graphs.append(g)
        for i in range(40):
            x.copy_(randn(200 + i, B, 1, h + 2 * hk, d, dtype=BF))
            graphs[i % 2].replay()
    side.synchronize()
    assert held.tolist() == [41, 46, 71] and pool.count.item() == n_pages - 3 - 3 - 5
    ref, tol = C.attention(q1[:, 0], kp, ks, vp, vs, pool.table, [41, 46, 71], hk)
    R.check(out, ref, tol, "replayed")
    assert slots[:, 0].tolist() == [pool.table[b, (n - 1) // page].item() * page + (n - 1) % page for b, n in enumerate([41, 46, 71])]


def test_binding_refusals(bnd):
    B, hk, d, page, n_pages = 2, 2, 64, 16, 8
    kp, ks = pages_of(1, n_pages, page, 16, hk, d, E4)
    vp, vs = pages_of(2, n_pages, page, 16, hk, d, E4)
    t = ints([[0, 1], [2, 3]])
    make = bnd.make_coded_cache
    with pytest.raises(TypeError):
        make(kp.float(), vp.float(), ks, vs, t)
    with pytest.raises(TypeError):
        make(kp, vp.view(I8), ks, vs, t)
    with pytest.raises(TypeError):
        make(kp, vp, ks.double(), vs, t)
    for bad in ((ks[:, :, :1], vs), (ks[:4], vs), (ks, vs.expand(n_pages, 2, hk)), (ks.expand(n_pages, 3, hk), vs),
                (torch.ones(n_pages, hk, 1, device="cuda").transpose(1, 2).expand(n_pages, 2, hk), torch.ones(n_pages, 2, hk, device="cuda"))):
        with pytest.raises(ValueError):
            make(kp, vp, *bad, t)
    cache = make(kp, vp, ks, vs, t)
    plain = bnd.make_paged_cache(torch.zeros(n_pages, page, hk, d, device="cuda", dtype=BF), torch.zeros(n_pages, page, hk, d, device="cuda", dtype=BF), t)
    x, one = randn(1, B, 1, hk, d, dtype=BF), ints([0, 0])
    ws = torch.zeros(1 << 22, dtype=torch.uint8, device="cuda")
    q, out = randn(2, B, 4, d, dtype=BF), torch.zeros(B, 4, d, device="cuda", dtype=BF)
    # the two kinds of cache do not mix
    for call in (lambda: bnd.mha_coded_append(x, x, one, cache=plain), lambda: bnd.mha_paged_append(x, x, one, cache=cache),
                 lambda: bnd.mha_coded_attention(q, one, cache=plain, out=out, workspace=ws),
                 lambda: bnd.mha_paged_attention(q, one, cache=cache, out=out, workspace=ws),
                 lambda: bnd.mha_coded_append(x[:1], x[:1], one[:1], cache=cache), lambda: bnd.mha_coded_append(x, x, None, cache=cache),
                 lambda: bnd.mha_coded_append(x, x, one[:1], cache=cache), lambda: bnd.mha_coded_attention(q, None, cache=cache, out=out, workspace=ws),
                 lambda: bnd.mha_coded_attention(q[:, :, :32], one, cache=cache, out=out[:, :, :32], workspace=ws)):
        with pytest.raises(ValueError):
            call()
    with pytest.raises(TypeError):
        bnd.mha_coded_append(x.half(), x.half(), one, cache=cache)
    with pytest.raises(TypeError):
        bnd.mha_coded_attention(q, one.long(), cache=cache, out=out, workspace=ws)
    with pytest.raises(bnd.MHAError):
        bnd.mha_coded_attention(q, one, cache=cache, out=out, workspace=ws[:256])
    with pytest.raises(bnd.MHAError):
        bnd.mha_coded_append(randn(1, B, 1, hk, d + 1, dtype=BF)[..., 1:], x, one, cache=cache)     # keys at an odd element
    pool = dict(block_table=t, page_size=16, free_pages=ints([4, 5, 6, 7]), free_count=ints([4]), lens=ints([0, 0]))
    with pytest.raises(bnd.MHAError):
        bnd.mha_paged_resize(one, one, **(pool | dict(lens=one)))
    with pytest.raises(bnd.MHAError):
        bnd.mha_paged_resize(one, one, **(pool | dict(page_size=0)))
    for bad in (dict(block_table=t[:1]), dict(block_table=t[0]), dict(lens=ints([0])), dict(free_count=ints([1, 2])),
                dict(slots=torch.zeros(1, 3, device="cuda", dtype=torch.int64))):
        with pytest.raises(ValueError):
            bnd.mha_paged_resize(one, one, **(pool | bad))
    for bad in (dict(slots=torch.zeros(2, 3, device="cuda", dtype=torch.int32)), dict(free_pages=torch.zeros(4, device="cuda"))):
        with pytest.raises(TypeError):
            bnd.mha_paged_resize(one, one, **(pool | bad))
    assert same(kp, pages_of(1, n_pages, page, 16, hk, d, E4)[0])          # nothing was written
