"""The operators around a cache in 8 bits on the GPU: calls from several host threads, weights of very different sizes, nothing lost
and nothing doubled, calls captured first."""
import math
import os
import subprocess
import sys
import threading

import pytest

torch = pytest.importorskip("torch")

import coded_ref as C  # noqa: E402
import serving_ref as R  # noqa: E402
from test_coded_gpu import (BF, E4, F32, I8, bnd, clean_status, freqs, ints, pages_of, randn, run_attention, same,  # noqa: E402, F401
                            slopes_of, table_of)

pytestmark = pytest.mark.gpu


# ------------------------------------------------------------------------------------------ append
def test_appends_from_two_host_threads(bnd):
    """Blocks of 64 and of 256 tokens through one kernel, which need different amounts of shared memory, call after call from
    two host threads at once: every call is taken, with the results of calls one after the other."""
    h, hk, d, T = 4, 2, 128, 256
    jobs = []
    for i, block in enumerate((64, 256)):
        table, n_pages = table_of(i, 2, 2)
        kp, ks = pages_of(6 + i, n_pages, 256, block, hk, d, E4)
        vp, vs = pages_of(8 + i, n_pages, 256, block, hk, d, E4)
        q, k, v = (randn(10 + i + 3 * j, 2, T, (h, hk, hk)[j], d, dtype=BF) for j in range(3))
        cache, rotary = bnd.make_coded_cache(kp, vp, ks, vs, table), bnd.make_rotary(freqs(128 if block == 256 else 16))
        start, out = ints([0, 256]), torch.zeros_like(q)
        outs = (kp, vp, ks, vs, out)

        def call(stream=None, a=(k, v, start), kw=dict(cache=cache, q=q, q_out=out, rotary=rotary)):
            bnd.mha_coded_append(*a, stream=stream, **kw)

        def clear(cleared=(kp, vp, out)):        # pages that no call writes are zeros before and after
            for o in cleared:
                o.view(torch.uint8).zero_()
        clear()
        call()
        torch.cuda.synchronize()
        jobs.append((call, outs, [o.clone() for o in outs], torch.cuda.Stream()))
        clear()
    torch.cuda.synchronize()
    errors, begin = [], threading.Barrier(2)

    def work(call, stream):
        try:
            begin.wait(30)
            for _ in range(3000):
                call(stream)
            stream.synchronize()
        except Exception as e:
            errors.append(e)
    threads = [threading.Thread(target=work, args=(j[0], j[3])) for j in jobs]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not errors, errors
    for _, outs, want, _ in jobs:
        assert all(same(a, b) for a, b in zip(outs, want))


# ------------------------------------------------------------------------------------------ attention
def norm_error(got, ref):
    return ((got.double() - ref).norm() / ref.norm()).item()


# A first key of nearly all of the weight and of no value, scores of one product each. fp32: a weight is off by 2^-22 of itself, its score
# of up to 20 by four roundings, twice as it also enters the sum (2 * 20 * 4 * 2^-24 = 1e-5), exp2 and the factors of the running maximum by
# 4 * 2^-21 = 2e-6; the sum of values takes a product of 16 of a warp's n / 8 keys after the other, each cut at 2^-23 of what the sum came
# to, the sum of weights one of 32 of them, rounded. bf16: what rounding the exact result gives, r, and twice the error e in front of the
# rounding: |round(x + e) - x| is |round(x) - x| unless a border lies between x and x + e, where the first is at most half a step + e and
# the second at least half a step - e. (Of r itself no more than 1.66e-3 of the norm in the mean is known, and 128 values do not keep to
# that within a twentieth.) e: weights rounded to 2^-11 (2^-11 / sqrt 3 = 2.8e-4), or to 2^-25 where the largest is 2^10 or more, of which
# the others have share / (1 - share) / n in the mean and e^(1/2) of that in the root mean square: 2^-35 / sqrt 3 of the largest each, for
# the warp with the first key, which has every eighth step (4.7e-4 at 131071 keys and a share of 1 / 1000); a twentieth for samples.
@pytest.mark.parametrize("code", [E4, I8])
@pytest.mark.parametrize("dtype,hk,d,group", [(BF, 1, 128, 1), (F32, 1, 128, 3), (F32, 2, 64, 1), (F32, 2, 64, 5), (F32, 1, 64, 2)])
@pytest.mark.parametrize("n,share", [(400, 0.001), (8192, 0.1), (8192, 0.001), (32768, 0.01), (131071, 0.001)])
def test_attention_beside_a_key_of_nearly_all_the_weight(bnd, dtype, code, hk, d, group, n, share):
    """Sequences of the same pages, as many as keep each in one CTA, where a warp has every eighth step of it."""
    B, page, h = 400 // hk, 16, hk * group
    per = -(-n // page)
    table = torch.arange(per, device="cuda", dtype=torch.int32).repeat(B, 1)
    vp, vs = pages_of(47, per, page, 1, hk, d, code)
    kp, ks = pages_of(48, per, page, 1, hk, d, code)
    vs.fill_(2.0 ** -5)
    vp[0, 0] = 0
    one = 64.0
    first = torch.randn(per, page, hk, generator=torch.Generator(device="cuda").manual_seed(49), device="cuda") * one
    kp[..., 0] = first.round().clamp(-127, 127).to(kp.dtype)
    kp[0, 0, :, 0] = torch.tensor(one, device="cuda").to(kp.dtype)
    ks.fill_(1.0 / one)
    for g in range(hk):
        s = kp[..., g, 0].double().flatten()[1:n] / one
        ks[0, 0, g] = (torch.logsumexp(s, 0) + math.log((1 - share) / share)).item() / one
    q = torch.zeros(B, h, d, device="cuda", dtype=dtype)
    q[..., 0] = 1.0
    got = run_attention(bnd, q, kp, ks, vp, vs, table, [n] * B, hk, scale=1.0)
    want = torch.zeros(h, d, dtype=torch.float64, device="cuda")
    kv, vv = C.values(kp, ks).flatten(0, 1)[:n], C.values(vp, vs).flatten(0, 1)[:n]
    for i in range(h):
        want[i] = torch.softmax(kv[:, i // group, 0], 0) @ vv[:, i // group]
    bound = 1.3e-5 + n / 8 / 16 * 2.0 ** -23 + n / 8 / 32 * 2.0 ** -24
    if dtype == BF:
        small = (1 - share) / share * n * 2.0 ** -35 / math.sqrt(3) / math.exp(0.5) / math.sqrt(8)
        bound = norm_error(want.to(BF), want) + 2 * 1.05 * math.hypot(2.8e-4, small)
    worst = max(norm_error(got[b], want) for b in (0, B // 3, B - 1))
    assert worst <= bound, (worst, bound)
    assert all(norm_error(got[b], want) <= bound for b in range(B))


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("code", [E4, I8])
@pytest.mark.parametrize("n,far", [(20, 9), (300, 40), (300, 299), (20000, 3), (20000, 19000)])
@pytest.mark.parametrize("below", [90, 110, 125])
def test_attention_value_scales_that_outweigh_the_softmax(bnd, dtype, code, n, far, below):
    """A first key with nearly all of the softmax and values of scale 2^-120, one whose numerator is 2^-below of its and whose values, of scale 2^110
    (448 times that is 2^118.9: the sums' limit is 2^120), are the result: in one warp, in two, in two CTAs. The other keys lie in between and add nothing. Below 2^-126 the key may
    count as none: the result is then the exact one or that without it."""
    h, hk, d, page = 4, 2, 64, 16
    table, n_pages = table_of(1, 1, -(-n // page))
    kp, ks = pages_of(52, n_pages, page, 1, hk, d, code)
    vp, vs = pages_of(53, n_pages, page, 1, hk, d, code)
    where = table[0].long().repeat_interleave(page)[:n], torch.arange(n, device="cuda") % page
    kp[..., 0] = torch.tensor(1.0, device="cuda").to(code)
    score = torch.full((n,), -100.0, device="cuda")
    score[0] = 0.0
    vs[where] = 2.0 ** -120
    q = torch.zeros(1, h, d, device="cuda", dtype=dtype)
    q[..., 0] = 1.0
    for gap in (below, 126 + below):
        score[far] = -gap
        ks[where] = -score[:, None].expand(n, hk)           # codes of 1 and a scale of scores, which are powers of two's logarithms
        vs[where[0][far], where[1][far]] = 2.0 ** 110
        got = run_attention(bnd, -q, kp, ks, vp, vs, table, [n], hk, scale=math.log(2.0))
        ref, tol = C.attention(-q, kp, ks, vp, vs, table, [n], hk, scale=math.log(2.0))
        if gap > 126:
            vs[where[0][far], where[1][far]] = 0.0
            none, none_tol = C.attention(-q, kp, ks, vp, vs, table, [n], hk, scale=math.log(2.0))
            assert torch.isfinite(got).all()
            assert (((got.double() - ref).abs() <= tol) | ((got.double() - none).abs() <= none_tol)).all()
        else:
            assert (ref.abs() > 2.0 ** (105 - gap)).any()
            R.check(got, ref, tol, "outweighed")


@pytest.mark.parametrize("dtype", [BF, F32])
def test_attention_values_of_the_largest_scale(bnd, dtype):
    """Scales of 2^122, the largest that an append makes, with codes small enough for the sums."""
    h, hk, d, page, n = 4, 2, 128, 16, 8
    table, n_pages = table_of(1, 1, 1)
    kp, ks = pages_of(54, n_pages, page, 16, hk, d, E4)
    vp, vs = pages_of(55, n_pages, page, 16, hk, d, E4)
    vp = (vp.float().sign() * 2.0 ** -6).to(E4)
    vs.fill_(2.0 ** 122)
    q = randn(56, 1, h, d, dtype=dtype)
    got = run_attention(bnd, q, kp, ks, vp, vs, table, [n], hk)
    ref, tol = C.attention(q, kp, ks, vp, vs, table, [n], hk)
    R.check(got, ref, tol, "2^122")


# fp32: scores of up to 16 (16 sums in the matrix instruction, each cut at 2^-23, and four roundings, twice as they also enter the sum of
# weights: 2 (16 2^-23 + 4 2^-24) 16 = 6.9e-5), sums of at most 5000 keys a warp-wise 32 at a time (1e-5); the cap's tanh to 2^-20 of it, twice. bf16: what
# rounding the exact result gives and twice the error in front of it, weights rounded to 2^-11 (2^-11 / sqrt 3 = 2.8e-4) and the same of scores.
@pytest.mark.parametrize("dtype,code,B,h,hk,d,n,page,block,sc", [
    (BF, E4, 1, 16, 2, 128, 70001, 64, 16, {}), (BF, I8, 2, 4, 4, 64, 30000, 128, 128, {}), (BF, E4, 16, 8, 8, 64, 1000, 16, 16, dict(cap=30.0)),
    (BF, I8, 64, 16, 4, 64, 200, 16, 8, {}), (BF, E4, 3, 20, 1, 128, 5000, 100, 25, dict(slopes=True)), (BF, I8, 12, 32, 8, 128, 3000, 32, 32, {}),
    (BF, E4, 30, 48, 8, 64, 2000, 64, 64, {}), (BF, E4, 200, 32, 8, 128, 90, 32, 16, {}),
    (F32, E4, 1, 4, 1, 64, 40001, 64, 16, {}), (F32, I8, 8, 8, 2, 128, 700, 16, 16, dict(cap=30.0)), (F32, E4, 9, 24, 8, 128, 5000, 64, 32, {}),
    (F32, I8, 3, 16, 16, 64, 4000, 64, 64, dict(slopes=True)), (F32, E4, 5, 10, 2, 64, 3000, 24, 24, {}), (F32, I8, 130, 12, 4, 64, 100, 16, 16, {})])
def test_attention_error_of_the_norm(bnd, dtype, code, B, h, hk, d, n, page, block, sc):
    sc = dict(sc, slopes=slopes_of(h)) if sc.get("slopes") else sc
    lens = [max(n - 7 * b, 1) for b in range(B)]
    table, n_pages = table_of(32, B, -(-n // page))
    kp, ks = pages_of(33, n_pages, page, block, hk, d, code)
    vp, vs = pages_of(34, n_pages, page, block, hk, d, code)
    q = randn(35, B, h, d, dtype=dtype)
    got = run_attention(bnd, q, kp, ks, vp, vs, table, lens, hk, **sc)
    ref, _ = C.attention(q, kp, ks, vp, vs, table, lens, hk, **sc)
    off = 8e-5 + 2 * 2.0 ** -20 * sc.get("cap", 0.0)
    bound = off if dtype == F32 else norm_error(ref.to(BF), ref) + 2 * 1.05 * math.hypot(2.8e-4, off)
    assert norm_error(got, ref) <= bound


@pytest.mark.parametrize("dtype,code,h,hk,d,lens,page", [
    (BF, E4, 4, 2, 64, [40001], 64), (BF, I8, 16, 2, 128, [30000, 5], 128), (BF, E4, 16, 8, 128, [9000, 12000, 1], 64),
    (BF, I8, 6, 3, 64, [5000] * 3, 16), (BF, E4, 2, 2, 64, [1000] * 3, 16), (BF, E4, 8, 8, 128, [4000, 0, 3999] * 8, 32),
    (BF, I8, 24, 1, 128, [3000, 7], 104), (BF, E4, 48, 8, 64, [2500, 40], 64), (BF, I8, 8, 4, 64, [100, 33, 1, 97] * 40, 16),
    (F32, E4, 4, 1, 64, [20001], 64), (F32, I8, 2, 2, 128, [513, 8000, 64], 24), (F32, E4, 16, 16, 64, [3000, 2999], 64),
    (F32, I8, 12, 2, 64, [4097], 16), (F32, E4, 4, 4, 128, [250, 3] * 60, 16)])
def test_attention_takes_every_key_once(bnd, dtype, code, h, hk, d, lens, page):
    """Equal scores, values that are zero but at d keys at a time, each with a feature of its own: that feature of the output is 1 / n, and 0 or 2 / n
    if the key is left out or taken twice. Every key is looked at. Codes of 1, 2, 4 under scales of 1, 1/2, 1/4: weights are powers of two
    and sums whole numbers of the least of them, exact in fp32 up to 2^24; left are the quotient and the output's rounding."""
    B, n = len(lens), max(lens)
    table, n_pages = table_of(40, B, -(-n // page))
    kp, ks = pages_of(41, n_pages, page, 8, hk, d, code)
    vp, _ = pages_of(42, n_pages, page, 8, hk, d, code)
    down = torch.randint(0, 3, (n_pages, page // 8, hk), generator=torch.Generator(device="cuda").manual_seed(43), device="cuda")
    vs = torch.exp2(-down.float())
    ones = torch.exp2(down.float()).repeat_interleave(8, dim=1)               # codes that stand for 1, [n_pages, page, hk]
    q = torch.zeros(B, h, d, device="cuda", dtype=dtype)
    at = torch.arange(n, device="cuda")
    held = torch.tensor(lens, device="cuda")[:, None] > at                    # [B, n]
    pages, slots = table.long()[:, at // page], (at % page).expand(B, n)
    whole = torch.zeros(vp.shape, device="cuda")
    for first in range(0, n, d):
        live = held[:, first:first + d]
        f = torch.arange(d, device="cuda").expand(B, d)[:, :live.shape[1]][live]
        pg, sl = pages[:, first:first + d][live], slots[:, first:first + d][live]
        whole.zero_()
        whole[pg, sl, :, f] = ones[pg, sl]
        vp.copy_(whole.to(code))
        want = torch.zeros(B, h, d, dtype=torch.float64, device="cuda")
        want[:, :, :live.shape[1]] = (live.double() / torch.tensor(lens, device="cuda").clamp_min(1)[:, None])[:, None]
        got = run_attention(bnd, q, kp, ks, vp, vs, table, lens, hk)
        R.check(got, want, want * (R.HALF[dtype] + 2.0 ** -22), "every key once")


# ------------------------------------------------------------------------------------------ pages granted
def test_resize_behind_a_shared_prefix(bnd):
    """Three sequences whose first two pages are the same: the call gets the table's columns behind those, so that they are neither given
    back nor granted when the sequences end."""
    B, page, room, n_pages, shared = 3, 4, 8, 20, 2
    table = torch.full((B, room), -1, dtype=torch.int32, device="cuda")
    table[:, 0], table[:, 1] = 18, 7
    free = [p for p in range(n_pages) if p not in (18, 7)]
    stack, count = ints(free + [-1] * shared), ints([len(free)])
    at = [shared * page + x for x in (5, 0, 9)]                  # of the whole sequence
    lens, new_lens = (torch.zeros(B, dtype=torch.int32, device="cuda") for _ in range(2))
    slots = torch.zeros(B, 9, dtype=torch.int64, device="cuda")
    zero, behind = ints([0] * B), ints([x - shared * page for x in at])
    kw = dict(block_table=table[:, shared:], page_size=page, free_pages=stack, free_count=count, lens=lens, new_lens=new_lens)
    bnd.mha_paged_resize(zero, behind, slots=slots, **kw)
    want = C.resize([0] * B, [5, 0, 9], page, [[-1] * (room - shared)] * B, free + [-1] * shared, len(free), 9)
    assert lens.tolist() == want[0] and new_lens.tolist() == want[1] and slots.tolist() == want[2]
    assert table[:, shared:].tolist() == want[3] and stack.tolist() == want[4] and count.item() == want[5]
    granted = [p for row in table[:, shared:].tolist() for p in row if p >= 0]
    assert not {18, 7} & set(granted) and table[:, :shared].tolist() == [[18, 7]] * B
    bnd.mha_paged_resize(behind, zero, **kw)
    assert count.item() == len(free) and sorted(stack.tolist()[:len(free)]) == free and table[:, :shared].tolist() == [[18, 7]] * B


# ------------------------------------------------------------------------------------------ a run of them
def serving_step(bnd, B=5, T=3, h=8, hk=2, d=128, page=16, room=6):
    """Pages granted, T new tokens appended and the last one attending, from empty rows; what the step writes."""
    n_pages = B * room + 2
    table = torch.full((B, room), -1, dtype=torch.int32, device="cuda")
    stack, count = ints(list(range(n_pages))), ints([n_pages])
    kp, ks = pages_of(60, n_pages, page, 8, hk, d, E4)
    vp, vs = pages_of(61, n_pages, page, 8, hk, d, E4)
    q, k, v = (randn(62 + i, B, T, (h, hk, hk)[i], d, dtype=BF) for i in range(3))
    held, want, lens, new_lens = ints([0] * B), ints([T, 1, 0, 2, T]), ints([0] * B), ints([0] * B)
    slots, q1, out = torch.zeros(B, T, dtype=torch.int64, device="cuda"), torch.zeros_like(q), torch.zeros(B, h, d, device="cuda", dtype=BF)
    cache, rotary = bnd.make_coded_cache(kp, vp, ks, vs, table), bnd.make_rotary(freqs(64))
    ws = torch.zeros(bnd.coded_attention_workspace_size(bnd.MHA_BF16, B, h, hk, d), dtype=torch.uint8, device="cuda")
    state = (table, stack, count, kp, vp, ks, vs, lens, new_lens, slots, q1, out)
    begin = [t.clone() for t in state]

    def restart():
        for t, b in zip(state, begin):
            t.copy_(b)

    def step():
        bnd.mha_paged_resize(held, want, block_table=table, page_size=page, free_pages=stack, free_count=count, lens=lens, new_lens=new_lens,
                             slots=slots)
        bnd.mha_coded_append(k, v, held, cache=cache, q=q, q_out=q1, new_lens=new_lens, rotary=rotary)
        bnd.mha_coded_attention(q1[:, 0], lens, cache=cache, out=out, workspace=ws)
    return step, restart, state


def test_first_step_may_be_captured():
    """A fresh process whose first calls are captured into a graph: what a device has room for may be asked for there."""
    here = os.path.dirname(os.path.abspath(__file__))
    code = """
import sys
sys.path[:0] = [%r, %r]
import torch
import test_coded_ranges_gpu as T
from transformer_head_scaled_fwd_gb300 import binding as bnd
step, restart, state = T.serving_step(bnd)
torch.cuda.synchronize()
g = torch.cuda.CUDAGraph()
with torch.cuda.graph(g):
    step()
g.replay()
torch.cuda.synchronize()
got = [t.clone() for t in state]
assert got[2].item() == 32 - 4 and got[11].float().abs().sum() > 0
restart()
step()
torch.cuda.synchronize()
assert all(T.same(a, b) for a, b in zip(got, state))
assert bnd.mha_check_device_status() == 0
print("captured first")
""" % (os.path.dirname(here), here)
    r = subprocess.run([sys.executable, "-c", code], capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and "captured first" in r.stdout, r.stdout + r.stderr
