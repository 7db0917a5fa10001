"""Plain forms of the operators around a cache in 8 bits, from their definitions, and the tolerances of their comparisons."""
import math

import torch

import serving_ref as R

TOP = {torch.float8_e4m3fn: 448.0, torch.int8: 127.0}
LEAST = 2.0 ** -120


def scale_for(top, code):
    """Least power of two s >= 2^-120 with top <= TOP s (a Python float)."""
    if not math.isfinite(top):
        return math.nan
    s = LEAST
    if top > 0:
        s = max(LEAST, 2.0 ** (math.frexp(top / TOP[code])[1] - 2))
    while top > TOP[code] * s:
        s *= 2
    return s


def half_step(x, scale, code):
    """Largest |code * scale - x| of a code rounded to nearest."""
    if code == torch.int8:
        return torch.full_like(x, 0.5) * scale
    return torch.maximum(x.abs() * 2.0 ** -4, torch.full_like(x, 2.0 ** -10) * scale)


def values(pages, scales):
    """[n_pages, page, h_kv, d] in fp64."""
    n, page, hk, d = pages.shape
    blocks = scales.shape[1]
    x = pages.to(torch.float32).double().reshape(n, blocks, page // blocks, hk, d)
    return (x * scales.double()[:, :, None, :, None]).reshape(n, page, hk, d)


def append(pages, scales, x, tol, table, start, lens, page, block):
    """What the pages then stand for, the tolerance, and the scales that may differ: (values, tolerance, scales, near). x [B, T, hk, d] in
    fp64, tol the error of the turned x. Scales are compared where the block's maximum is not within tol of a power of two's border."""
    code = pages.dtype
    codes = pages.to(torch.float32).double()
    want, wtol = values(pages, scales), torch.zeros(pages.shape, dtype=torch.float64, device=pages.device)
    s_want, near = scales.double().clone(), torch.zeros(scales.shape, dtype=torch.bool, device=scales.device)
    B, T, hk, _ = x.shape
    for b in range(B):
        n = min(max(lens[b], 0), T) if lens is not None else T
        t = 0
        while t < n:
            p = start[b] + t
            m = min(n - t, block - p % block)
            pg, sl = table[b, p // page].item(), p % page
            blk = sl // block
            for h in range(hk):
                v, e = x[b, t:t + m, h], tol[b, t:t + m, h]
                top = v.abs().max().item()
                need = scale_for(top, code)
                err = e.max().item()
                if math.isfinite(top):
                    near[pg, blk, h] = scale_for(top + err, code) != scale_for(max(top - err, 0.0), code)
                old = s_want[pg, blk, h].item()
                new = need if p % block == 0 else (math.nan if math.isnan(need) or math.isnan(old) else max(old, need))
                s_want[pg, blk, h] = new
                rows = slice(sl - sl % block, sl)
                step = 2 * new if near[pg, blk, h] else new
                if p % block != 0 and new > old:
                    wtol[pg, rows, h] = half_step(want[pg, rows, h], step, code)
                # slots behind the last token keep their codes under the block's scale
                behind = slice(sl + m, sl - sl % block + block)
                want[pg, behind, h] = codes[pg, behind, h] * new
                wtol[pg, behind, h] = math.inf if near[pg, blk, h] else 0.0
                want[pg, sl:sl + m, h] = v if not math.isnan(new) else math.nan
                if math.isnan(new):
                    want[pg, rows, h] = math.nan
                # the turned key is off by e, and then rounded
                wtol[pg, sl:sl + m, h] = half_step(v.abs() + e, step, code) + e
            t += m
    return want, wtol, s_want, near


def attend(q, k, vc, vs, n, *, scale, cap=0.0, slope=0.0, drop=()):
    """One head in fp64: q [d], k [n, d] values, vc [n, d] codes, vs [n] scales. (o, tolerance's parts)."""
    pos = torch.arange(n, device=q.device, dtype=torch.float64)
    ok = torch.ones(1, n, dtype=torch.bool, device=q.device)
    for j in drop:
        ok[0, j] = False
    away = (n - 1 - pos)[None]
    o, mag, size = R.attend(q[None], k, vc * vs[:, None], ok, away, scale=scale, cap=cap, slope=slope)
    s = (k @ q.double()) * scale
    if cap:
        s = cap * torch.tanh(s / cap)
    s = torch.where(ok[0], s - slope * away[0], -math.inf)
    p = torch.softmax(s, 0) if ok.any() else torch.zeros_like(s)
    most = (p * vs).max().item() * TOP[torch.float8_e4m3fn] if n else 0.0
    return o[0], mag[0], size[0], most


def attend_tol(o, mag, size, most, n, d, dtype, *, cap=0.0, far=0.0):
    """Bound of |kernel - o|: the output's half step; every weight off by a relative e^delta - 1, delta twice the error of a score: d
    products summed by the matrix instruction in fp32, whose sums may be cut where additions round (2 d 2^-24 of sum |q k|), six roundings of
    the score itself, an fp32 query as two fp16 terms (2^-22 of it), the cap's tanh to 2^-20; exp2 to 2^-21, the scale and the running maximum's factors (2^-21 each); the weight rounded
    to fp16 (bf16 result: 2^-11, since fp16 keeps ten bits behind the leading one: its steps in [2^e, 2^(e + 1)) are 2^(e - 10), a rounding is
    off by half of one, 2^(e - 11), and the weight is at least 2^e; fp32: a second term holds what the first left, 2^-11 of it, and is off by
    2^-11 of that, 2^-22), or, where it is subnormal there, off by 2^-25 while the largest is at least
    2^6 (2^-31 of `most` a key); n weights and products summed in fp32, cut or rounded (2 n 2^-24 each)."""
    delta = 2 * ((2 * d + 10) * 2.0 ** -24 * size + 6 * 2.0 ** -24 * far + cap * 2.0 ** -20)
    weight = 2.0 ** -11 if dtype == torch.bfloat16 else 2.0 ** -22
    rel = torch.expm1(delta) + 3 * 2.0 ** -20 + weight + 4 * (n + 16) * 2.0 ** -24
    return R.HALF[dtype] * o.abs() + rel * mag + n * 2.0 ** -31 * most + 1e-30


def attention(q, kp, ks, vp, vs, table, lens, hk, *, cap=0.0, slopes=None, scale=None, bad=()):
    """(reference, tolerance) of q [B, h, d]; positions in `bad` (sequence, position) are left out."""
    B, h, d = q.shape
    page, blocks = kp.shape[1], ks.shape[1]
    kv = values(kp, ks)
    codes, steps = vp.to(torch.float32).double(), vs.double().repeat_interleave(page // blocks, dim=1)
    ref = torch.zeros(B, h, d, dtype=torch.float64, device=q.device)
    tol = torch.full_like(ref, 1e-30)
    for b in range(B):
        n = max(lens[b], 0)
        if n == 0:
            continue
        rows = table[b, : -(-n // page)].long().clamp(0, kp.shape[0] - 1)
        drop = [j for bb, j in bad if bb == b and j < n]
        for i in range(h):
            g = i // (h // hk)
            slope = slopes[i].item() if slopes is not None else 0.0
            k = kv[rows, :, g].flatten(0, 1)[:n]
            o, mag, size, most = attend(q[b, i].double(), k, codes[rows, :, g].flatten(0, 1)[:n], steps[rows, :, g].flatten(0, 1)[:n],
                                        n, scale=d ** -0.5 if scale is None else scale, cap=cap, slope=slope, drop=drop)
            ref[b, i] = o
            tol[b, i] = attend_tol(o, mag, size, most, n, d, q.dtype, cap=cap, far=abs(slope) * n)
    return ref, tol


def resize(held, want, page, table, stack, count, T):
    """One step on Python lists, sequence by sequence: (lens, new_lens, slots, table, stack, count)."""
    n_pages, room = len(stack), len(table[0])
    table, stack = [list(r) for r in table], list(stack)
    count = min(max(count, 0), n_pages)
    pages = lambda n: -(-n // page)  # noqa: E731
    held, want = [max(x, 0) for x in held], [max(x, 0) for x in want]
    asked = [h if w > h and pages(w) > room else w for h, w in zip(held, want)]
    have, then = [min(pages(x), room) for x in held], [min(pages(x), room) for x in asked]
    for b in reversed(range(len(held))):
        for i in reversed(range(then[b], have[b])):
            if count < n_pages:
                stack[count] = table[b][i]
                count += 1
            table[b][i] = -1
    lens, slots, sums, limit = [], [], 0, count
    for b in range(len(held)):
        up = max(then[b] - have[b], 0)
        sums += up
        ok = up == 0 or sums <= limit
        for i in range(have[b], have[b] + (up if ok else 0)):
            count -= 1
            table[b][i] = stack[count]
        lens.append(asked[b] if ok else held[b])
        new = max(lens[b] - held[b], 0)
        row = []
        for t in range(T):
            pg = table[b][(held[b] + t) // page] if t < new else -1
            row.append(pg * page + (held[b] + t) % page if 0 <= pg < n_pages else -1)
        slots.append(row)
    return lens, [max(a - h, 0) for a, h in zip(lens, held)], slots, table, stack, count
