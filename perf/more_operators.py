"""Cases of the operators around a key/value cache in 8 bits: pages granted and returned as sequences grow and end, the
append that turns keys and stores codes with a scale for each block of tokens and key head, and the attention of one new
token over such a cache. Each case runs in a plain form (elementary torch operations, fp32 with fp64 angles) or, where
``own`` is set, through the library's entry points."""
import math
import random

import numpy as np
import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
CODES = {"e4m3": torch.float8_e4m3fn, "int8": torch.int8}
TOP = {"e4m3": (0.875, 9, 448.0), "int8": (0.9921875, 7, 127.0)}     # largest code: m 2^e, 1/2 <= m < 1
LEAST = 2.0 ** -120                                                  # least scale


def listed():
    return [
        # a decoding step's tables: every sequence gets one more position, a few of them a page
        dict(name="resize one token", op="resize", batch=16, tokens=1, length=8192, page=16, ragged=False, ended=False, short=False),
        # admission: prompts of the long workload's length enter empty rows
        dict(name="resize prompts", op="resize", batch=64, tokens=8192, length=0, page=16, ragged=True, ended=False, short=False),
        # a mixed step: some sequences end, others get a chunk of a prompt, and the pool does not reach for all
        dict(name="resize mixed", op="resize", batch=509, tokens=333, length=4000, page=24, ragged=True, ended=True, short=True),
        # one new token of one sequence: the latency of the step's smallest call
        dict(name="append one token", op="append", dtype="bf16", code="e4m3", batch=1, tokens=1, start=700, heads=16,
             kv_heads=4, dim=64, page=16, block=16, rot=64, interleaved=False, ragged=False),
        # a decoding batch without rotation, int8 codes, a scale for half a page
        dict(name="append batch int8", op="append", dtype="bf16", code="int8", batch=61, tokens=1, start=3000, heads=32,
             kv_heads=8, dim=128, page=64, block=32, rot=0, interleaved=False, ragged=False),
        # a batch of prompts of the long workload's size enters the cache; heads of 128, half of each rotated
        dict(name="append prompts", op="append", dtype="bf16", code="e4m3", batch=4, tokens=8192, start=64, heads=32,
             kv_heads=8, dim=128, page=64, block=64, rot=64, interleaved=False, ragged=True),
        # chunks of prompts in fp32, interleaved pairs, small blocks
        dict(name="append chunks fp32", op="append", dtype="f32", code="e4m3", batch=7, tokens=333, start=900, heads=8,
             kv_heads=4, dim=64, page=24, block=8, rot=32, interleaved=True, ragged=True),
        # the decoding benchmark's cache (16 sequences of 8192 tokens, 16 heads of 64), in pages
        dict(name="decode 16 x 8192", op="decode", dtype="bf16", code="e4m3", batch=16, length=8192, ragged=False, heads=16,
             kv_heads=16, dim=64, page=64, block=64, cap=0.0, slopes=False),
        # many sequences of different lengths, grouped heads of 128, capped scores, int8 codes
        dict(name="decode ragged grouped", op="decode", dtype="bf16", code="int8", batch=48, length=15000, ragged=True,
             heads=32, kv_heads=8, dim=128, page=16, block=16, cap=30.0, slopes=False),
        # one sequence with a long history: the split over the length has to fill the GPU
        dict(name="decode one long", op="decode", dtype="bf16", code="e4m3", batch=1, length=131071, ragged=False, heads=16,
             kv_heads=2, dim=128, page=32, block=32, cap=0.0, slopes=True),
        # fp32 queries over a long cache in 8 bits
        dict(name="decode fp32", op="decode", dtype="f32", code="e4m3", batch=9, length=5000, ragged=True, heads=24,
             kv_heads=8, dim=128, page=64, block=32, cap=0.0, slopes=False),
        # a few short sequences: latency
        dict(name="decode short", op="decode", dtype="bf16", code="int8", batch=4, length=333, ragged=True, heads=8,
             kv_heads=4, dim=64, page=16, block=16, cap=0.0, slopes=False),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["resize", "append", "append", "decode", "decode", "decode"])
    page = rng.choice([8, 16, 24, 32, 64, 100, 128, 256])
    if op == "resize":
        batch = _log(rng, 1, 1024)
        return dict(op=op, batch=batch, tokens=_log(rng, 1, max(1, min(8192, 500_000 // batch))),
                    length=_log(rng, 1, max(1, min(32768, 4_000_000 // batch))), page=page, ragged=rng.random() < 0.6,
                    ended=rng.random() < 0.4, short=rng.random() < 0.3)
    block = rng.choice([b for b in (4, 8, 16, 25, 32, 64, 128, 256) if page % b == 0])
    dtype = "bf16" if rng.random() < 0.7 else "f32"
    code = rng.choice(["e4m3", "int8"])
    dim = rng.choice([64, 128])
    kv_heads = rng.choice([1, 2, 3, 4, 5, 8, 16])
    heads = kv_heads * rng.choice([1, 1, 2, 3, 4, 5, 7, 8])
    batch = _log(rng, 1, 64)
    if op == "append":
        tokens = _log(rng, 1, max(1, min(8192, 30_000_000 // (batch * (heads + 2 * kv_heads) * dim))))
        # int8 codes are whole numbers, compared as such: keys enter as they are
        return dict(op=op, dtype=dtype, code=code, batch=batch, tokens=tokens, start=_log(rng, 1, 4000), heads=heads,
                    kv_heads=kv_heads, dim=dim, page=page, block=block, rot=0 if code == "int8" else 2 * _log(rng, 4, dim // 2),
                    interleaved=rng.random() < 0.5, ragged=rng.random() < 0.5)
    most = 370_000_000 // (batch * kv_heads * dim)
    return dict(op=op, dtype=dtype, code=code, batch=batch, length=_log(rng, 1, min(131072, max(1, most))),
                ragged=rng.random() < 0.6, heads=heads, kv_heads=kv_heads, dim=dim, page=page, block=block,
                cap=rng.choice([0.0, 0.0, 15.0, 30.0, 50.0]), slopes=rng.random() < 0.3)


# ------------------------------------------------------------------------------------------ inputs
def _generators(seed):
    return torch.Generator(device="cuda").manual_seed(seed), random.Random(seed)


def _normal(g, *shape, dtype):
    return torch.randn(shape, generator=g, device="cuda", dtype=torch.float32).to(dtype)


def _ints(values):
    return torch.tensor(values, dtype=torch.int32, device="cuda")


def _scale_for(top, code):
    """The least power of two s with top <= s * (largest code)."""
    m, e = torch.frexp(top)
    limit, exponent, _ = TOP[code]
    s = torch.ldexp(torch.ones_like(top), e - exponent + (m > limit).to(e.dtype))
    return torch.where(top == 0, torch.full_like(s, LEAST), s.clamp_min(LEAST))


def _to_code(x, code):
    return torch.round(x).to(torch.int8) if code == "int8" else x.to(torch.float8_e4m3fn)


def _coded(c, g, total):
    """One array of pages of normal values, their sizes different by head, as codes, and their scales."""
    hk, per = c["kv_heads"], c["page"] // c["block"]
    x = _normal(g, total, per, c["block"], hk, c["dim"], dtype=torch.float32)
    x = x * torch.exp2(torch.randint(-2, 2, (hk, 1), generator=g, device="cuda").float())
    scale = _scale_for(x.abs().amax(dim=(2, 4)), c["code"])
    pages = _to_code(x / scale[:, :, None, :, None], c["code"]).view(total, c["page"], hk, c["dim"])
    return pages, scale


def _paged(c, g, rng, longest):
    """Pages of every sequence in a random order, with a few unused ones."""
    per = -(-longest // c["page"])
    total = c["batch"] * per + 3
    order = list(range(total))
    rng.shuffle(order)
    table = _ints(order[: c["batch"] * per]).view(c["batch"], per)
    k, ks = _coded(c, g, total)
    v, vs = _coded(c, g, total)
    return {"k_pages": k, "v_pages": v, "k_scales": ks, "v_scales": vs, "table": table}


def prepare(case, seed):
    c = case
    g, rng = _generators(seed)
    s = {"case": c}
    if c["op"] == "resize":
        B, T, page = c["batch"], c["tokens"], c["page"]
        r = np.random.RandomState(seed % (1 << 32))
        held = r.randint(c["length"] // 2, c["length"] + 1, B)
        add = r.randint(0, T + 1, B) if c["ragged"] else np.full(B, T)
        want = held + add
        if c["ended"]:
            want[r.random_sample(B) < 0.3] = 0
        have, then = -(-held // page), -(-want // page)
        room = -(-(c["length"] + T) // page)
        needed = int(np.maximum(then - have, 0).sum())
        freed = int(np.maximum(have - then, 0).sum())
        free = max(0, needed - freed) + 5 if not c["short"] else int(0.7 * max(0, needed - freed))
        total = B * room + 6                                         # the others are somebody else's
        order = r.permutation(total).astype(np.int32)
        table = np.full((B, room), -1, dtype=np.int32)
        column = np.arange(room)[None]
        owned = column < have[:, None]
        table[owned] = order[: int(have.sum())]
        stack = np.full(total, -1, dtype=np.int32)
        stack[:free] = order[int(have.sum()):][:free]
        s["held"], s["want"] = _ints(held.tolist()), _ints(want.tolist())
        s["table"], s["free_pages"] = torch.from_numpy(table).cuda(), torch.from_numpy(stack).cuda()
        s["free_count"] = _ints([free])
        s["lens"], s["new_lens"], s["back"] = (torch.zeros(B, dtype=torch.int32, device="cuda") for _ in range(3))
        s["slots"] = torch.empty(B, T, dtype=torch.int64, device="cuda")
        return s
    t = DTYPES[c["dtype"]]
    B, h, hk, d = c["batch"], c["heads"], c["kv_heads"], c["dim"]
    if c["op"] == "append":
        T = c["tokens"]
        # queries, keys and values as one projection leaves them
        qkv = _normal(g, B, T, h + 2 * hk, d, dtype=t)
        s["q"], s["k"], s["v"] = qkv[:, :, :h], qkv[:, :, h:h + hk], qkv[:, :, h + hk:]
        s["q_out"], s["k_out"] = torch.zeros(B, T, h, d, device="cuda", dtype=t), torch.zeros(B, T, hk, d, device="cuda", dtype=t)
        i = torch.arange(0, c["rot"], 2, device="cuda", dtype=torch.float64)
        s["inv_freq"] = (10000.0 ** (-i / max(c["rot"], 1))).float()
        s["start"] = _ints([rng.randint(0, c["start"]) for _ in range(B)])
        s["new_lens"] = _ints([rng.randint(0, T) if c["ragged"] else T for _ in range(B)])
        s.update(_paged(c, g, rng, c["start"] + T))
    else:
        s["q"] = _normal(g, B, h, d, dtype=t)
        lens = [rng.randint(0, c["length"]) if c["ragged"] else c["length"] for _ in range(B)]
        lens[0] = c["length"]
        s["lens"] = _ints(lens)
        s.update(_paged(c, g, rng, c["length"]))
        s["slopes"] = None
        if c["slopes"]:
            s["slopes"] = torch.tensor([2.0 ** (-8.0 * (i + 1) / h) for i in range(h)], device="cuda", dtype=torch.float32)
        s["out"] = torch.empty_like(s["q"])
    if own:
        _handles(s)
    return s


def _handles(s):
    """What a program builds once for a model and its cache: descriptions of the cache, the frequencies and the scores,
    and the workspace of the split attention."""
    from transformer_head_scaled_fwd_gb300 import binding as mha
    c = s["case"]
    s["cache"] = mha.make_coded_cache(s["k_pages"], s["v_pages"], s["k_scales"], s["v_scales"], s["table"])
    if c["op"] == "append":
        s["rotary"] = mha.make_rotary(s["inv_freq"], interleaved=c["interleaved"]) if c["rot"] else None
    else:
        s["scores"] = mha.make_scores(cap=c["cap"], slopes=s["slopes"])
        size = mha.coded_attention_workspace_size(mha.MHA_BF16 if c["dtype"] == "bf16" else mha.MHA_F32, c["batch"],
                                                  c["heads"], c["kv_heads"], c["dim"])
        s["workspace"] = torch.empty(size, dtype=torch.uint8, device="cuda")


# ------------------------------------------------------------------------------------------ plain forms
def _plain_resize(held, want, s, slots):
    """One step from held to want positions on s's table and stack; (lens, new_lens), and the slots written."""
    c = s["case"]
    page, room = c["page"], s["table"].shape[1]
    total = s["free_pages"].numel()
    held, want = held.long(), want.long()
    have, then = (held + page - 1) // page, (want + page - 1) // page
    down, up = (have - then).clamp_min(0), (then - have).clamp_min(0)
    column = torch.arange(room, device="cuda")[None]
    # pages of the sequences that shrink go on top of the stack, the first sequence's first page last
    rank = (torch.cumsum(down, 0) - down)[:, None] + column - then[:, None]
    gone = (column >= then[:, None]) & (column < have[:, None])
    count = s["free_count"].long() + down.sum()
    stack = torch.cat((s["free_pages"], s["free_pages"].new_zeros(1)))
    stack[torch.where(gone, count - 1 - rank, total)] = s["table"]
    stack = stack[:total]
    table = torch.where(gone, -1, s["table"])
    # pages for those that grow, while they last
    sums = torch.cumsum(up, 0)
    served = (up == 0) | (sums <= count)
    grown = torch.where(served, up, 0)
    rank = (torch.cumsum(grown, 0) - grown)[:, None] + column - have[:, None]
    new = (column >= have[:, None]) & (column < (have + grown)[:, None])
    table = torch.where(new, stack[(count - 1 - rank).clamp(0, max(total - 1, 0))], table)
    lens = torch.where(served, want, held)
    new_lens = (lens - held).clamp_min(0)
    s["table"].copy_(table)
    s["free_pages"].copy_(stack)
    s["free_count"].copy_(count - grown.sum())
    if slots:
        step = torch.arange(c["tokens"], device="cuda")[None]
        at = held[:, None] + step
        where = table.long().gather(1, (at // page).clamp_max(room - 1)) * page + at % page
        s["slots"].copy_(torch.where(step < new_lens[:, None], where, -1))
    return lens.int(), new_lens.int()


def _rotate(x, positions, inv_freq, interleaved):
    """x [B, T, H, d] in fp32; positions [B, T]; the first 2 len(inv_freq) columns of each head are rotated."""
    x = x.float()
    n = inv_freq.numel()
    if n == 0:
        return x
    angle = positions.to(torch.float64)[:, :, None, None] * inv_freq.to(torch.float64)
    cos, sin = torch.cos(angle).float(), torch.sin(angle).float()
    head, rest = x[..., : 2 * n], x[..., 2 * n:]
    if interleaved:
        a, b = head[..., 0::2], head[..., 1::2]
        turned = torch.stack((a * cos - b * sin, b * cos + a * sin), dim=-1).flatten(-2)
    else:
        a, b = head[..., :n], head[..., n:]
        turned = torch.cat((a * cos - b * sin, b * cos + a * sin), dim=-1)
    return torch.cat((turned, rest), dim=-1)


def _places(s):
    """Of each token: whether it exists, its page, slot, and block (of all blocks)."""
    c = s["case"]
    step = torch.arange(c["tokens"], device="cuda")
    at = s["start"].long()[:, None] + step
    live = step < s["new_lens"].long()[:, None]
    page = s["table"].long().gather(1, at // c["page"])
    slot = at % c["page"]
    return at, live, page, slot, page * (c["page"] // c["block"]) + slot // c["block"]


def _store(s, pages, scales, x, where):
    """x [B, T, hk, d] fp32 into the pages as codes: a block's scale is the larger of what it has and what its new values
    need; what it has held so far is rounded again where the scale grows."""
    c = s["case"]
    _, live, page, slot, block = where
    blocks, hk = scales.shape[0] * scales.shape[1], c["kv_heads"]
    old = scales.view(blocks, hk)
    index = torch.where(live, block, blocks).flatten()
    top = torch.full((blocks + 1, hk), -1.0, device="cuda")
    top = top.scatter_reduce(0, index[:, None].expand(-1, hk), x.abs().amax(dim=-1).flatten(0, 1), "amax")[:blocks]
    within = slot % c["block"]
    fresh = torch.zeros(blocks + 1, device="cuda").scatter_reduce(0, index, (within == 0).float().flatten(), "amax")[:blocks]
    # slots of a block that were filled before: those in front of the first new token
    first = torch.full((blocks + 1,), c["block"], device="cuda").scatter_reduce(0, index, within.flatten(), "amin")[:blocks]
    need = _scale_for(top.clamp_min(0), c["code"])
    new = torch.where(top < 0, old, torch.where(fresh[:, None] > 0, need, torch.maximum(old, need)))
    held = torch.arange(c["block"], device="cuda")[None] < first[:, None]
    again = (top >= 0) & (fresh[:, None] == 0) & (new > old)
    codes = pages.view(blocks, c["block"], hk, c["dim"])
    rounded = _to_code(codes.float() * (old / new)[:, None, :, None], c["code"])
    kept = torch.where((held[:, :, None] & again[:, None])[..., None], rounded.view(torch.uint8), codes.view(torch.uint8))
    pages.copy_(kept.view(CODES[c["code"]]).view_as(pages))
    scales.copy_(new.view_as(scales))
    fit = _to_code(x[live] / new[block[live]][..., None], c["code"])
    pages.view(torch.uint8)[page[live], slot[live]] = fit.view(torch.uint8)


def _plain_append(s):
    c = s["case"]
    t = s["q"].dtype
    where = _places(s)
    at, live = where[:2]
    k = _rotate(s["k"], at, s["inv_freq"], c["interleaved"])
    q = _rotate(s["q"], at, s["inv_freq"], c["interleaved"]).to(t)
    _store(s, s["k_pages"], s["k_scales"], k, where)
    _store(s, s["v_pages"], s["v_scales"], s["v"].float(), where)
    keep = live[:, :, None, None]
    return {"q": torch.where(keep, q, s["q_out"]), "k": torch.where(keep, k.to(t), s["k_out"]),
            **{n: s[n] for n in ("k_pages", "v_pages", "k_scales", "v_scales")}}


def _values(s, name):
    """The cached values of every sequence, [B, positions, hk, d] fp32."""
    c = s["case"]
    table = s["table"].long()
    x = s[name + "_pages"].view(torch.uint8)[table].view(CODES[c["code"]]).float()
    B, P = table.shape
    x = x.view(B, P, -1, c["block"], c["kv_heads"], c["dim"]) * s[name + "_scales"][table][:, :, :, None, :, None]
    return x.view(B, P * c["page"], c["kv_heads"], c["dim"])


def _plain_decode(s):
    c = s["case"]
    B, hk, d = c["batch"], c["kv_heads"], c["dim"]
    group = c["heads"] // hk
    k = _values(s, "k").permute(0, 2, 3, 1)
    v = _values(s, "v").permute(0, 2, 1, 3)
    q = s["q"].float().view(B, hk, group, d)
    x = torch.matmul(q, k) / math.sqrt(d)
    if c["cap"]:
        x = c["cap"] * torch.tanh(x / c["cap"])
    j = torch.arange(x.shape[-1], device="cuda")
    n = s["lens"].long()[:, None, None, None]
    if s["slopes"] is not None:
        x = x - s["slopes"].view(1, hk, group, 1) * (n - 1 - j).float()
    x = x.masked_fill(j >= n, -math.inf)
    top = x.amax(dim=-1, keepdim=True)
    p = torch.exp(x - torch.where(top == -math.inf, torch.zeros_like(top), top))
    total = p.sum(dim=-1, keepdim=True)
    p = p / torch.where(total == 0, torch.ones_like(total), total)
    return torch.matmul(p, v).view(B, c["heads"], d).to(s["q"].dtype)


# ------------------------------------------------------------------------------------------ the library's calls
def _own(s):
    from transformer_head_scaled_fwd_gb300 import binding as mha
    c = s["case"]
    if c["op"] == "resize":
        pool = dict(block_table=s["table"], page_size=c["page"], free_pages=s["free_pages"], free_count=s["free_count"])
        mha.mha_paged_resize(s["held"], s["want"], lens=s["lens"], new_lens=s["new_lens"], slots=s["slots"], **pool)
        mha.mha_paged_resize(s["lens"], s["held"], lens=s["back"], **pool)
        return {n: s[n] for n in ("lens", "new_lens", "slots", "back", "table", "free_pages", "free_count")}
    if c["op"] == "append":
        mha.mha_coded_append(s["k"], s["v"], s["start"], cache=s["cache"], q=s["q"], q_out=s["q_out"], k_out=s["k_out"],
                             new_lens=s["new_lens"], rotary=s["rotary"])
        return {"q": s["q_out"], "k": s["k_out"], **{n: s[n] for n in ("k_pages", "v_pages", "k_scales", "v_scales")}}
    mha.mha_coded_attention(s["q"], s["lens"], cache=s["cache"], out=s["out"], workspace=s["workspace"], scores=s["scores"])
    return s["out"]


def run(state):
    """One pass. A resize pass is a step and its return: the sequences go from held to want positions, and back, so the
    state is what it was; the slots hold the pages that the step granted."""
    if own:
        return _own(state)
    s = state
    if s["case"]["op"] == "resize":
        lens, new_lens = _plain_resize(s["held"], s["want"], s, True)
        back, _ = _plain_resize(lens, s["held"], s, False)
        return {"lens": lens, "new_lens": new_lens, "back": back, **{n: s[n] for n in ("slots", "table", "free_pages", "free_count")}}
    return {"append": _plain_append, "decode": _plain_decode}[s["case"]["op"]](s)


# ------------------------------------------------------------------------------------------ work and 64-bit results
def work(case):
    c = case
    if c["op"] == "resize":
        grown = c["batch"] * c["tokens"] * (0.5 if c["ragged"] else 1.0) / c["page"]
        ended = 0.3 * c["batch"] * 0.75 * c["length"] / c["page"] if c["ended"] else 0.0
        # lengths in, lengths out, slots; a page goes between the stack and the table, there and back
        return {"bytes": c["batch"] * (8.0 + 8.0 + 8.0 + 4.0) + 8.0 * c["batch"] * c["tokens"] + 2 * 8.0 * (grown + ended), "flops": 0.0}
    es = 4 if c["dtype"] == "f32" else 2
    if c["op"] == "append":
        tokens = (0.5 if c["ragged"] else 1.0) * c["batch"] * c["tokens"] * c["dim"]
        # q and k in and out, v in, codes out
        return {"bytes": tokens * (es * (2 * c["heads"] + 3 * c["kv_heads"]) + 2 * c["kv_heads"]),
                "flops": tokens * (3.0 * (c["heads"] + c["kv_heads"]) * c["rot"] / c["dim"] + 4.0 * c["kv_heads"])}
    keys = c["length"] + (c["batch"] - 1) * c["length"] * (0.5 if c["ragged"] else 1.0)
    return {"bytes": 2.0 * keys * c["kv_heads"] * (c["dim"] + 4.0 / c["block"]) + es * 2.0 * c["batch"] * c["heads"] * c["dim"],
            "flops": 4.0 * keys * c["heads"] * c["dim"]}


def _exact_append(c, s):
    where = _places(s)
    at, live, page, slot, block = where
    # rotation as a product of complex numbers
    turn = torch.polar(torch.ones((), dtype=torch.float64, device="cuda"), at.double()[:, :, None, None] * s["inv_freq"].double())
    n = s["inv_freq"].numel()
    done = {}
    for name in ("q", "k"):
        x = s[name].double().clone()
        if c["interleaved"]:
            z = torch.complex(x[..., 0:2 * n:2], x[..., 1:2 * n:2]) * turn
            x[..., 0:2 * n:2], x[..., 1:2 * n:2] = z.real, z.imag
        else:
            z = torch.complex(x[..., :n], x[..., n:2 * n]) * turn
            x[..., :n], x[..., n:2 * n] = z.real, z.imag
        done[name] = x
    got = {"q": done["q"].clone(), "k": done["k"].clone()}
    for b, m in enumerate(s["new_lens"].tolist()):
        got["q"][b, m:] = 0
        got["k"][b, m:] = 0
    size, per = c["block"], c["page"] // c["block"]
    starts, counts, table = s["start"].tolist(), s["new_lens"].tolist(), s["table"].tolist()
    for name, x in (("k", done["k"]), ("v", s["v"].double())):
        codes, scales = s[name + "_pages"].double(), s[name + "_scales"].double()
        for b, m in enumerate(counts):
            t = 0
            while t < m:
                p = starts[b] + t
                n_here = min(m - t, size - p % size)
                pg, sl = table[b][p // c["page"]], p % c["page"]
                values = x[b, t:t + n_here]
                most = values.abs().amax(dim=(0, 2)).clamp_min(1e-300) / TOP[c["code"]][2]
                e = torch.round(torch.log2(most))            # the least with most <= 2^e is this or the next, whatever log2 rounds
                e = e + (torch.exp2(e) < most)
                need = torch.exp2(e).clamp_min(LEAST)
                before = scales[pg, sl // size].clone()
                now = need if p % size == 0 else torch.maximum(before, need)
                codes[pg, sl - sl % size:sl] *= (before / now)[None, :, None]
                codes[pg, sl:sl + n_here] = values / now[None, :, None]
                scales[pg, sl // size] = now
                t += n_here
        # whole numbers have no value between them
        got[name + "_pages"] = codes if c["code"] == "e4m3" else None
        got[name + "_scales"] = scales
    return got


def exact(case, seed):
    c = case
    if c["op"] == "resize":
        return None
    s = prepare(case, seed)
    if c["op"] == "append":
        blocks = 2 * c["batch"] * (c["tokens"] // c["block"] + 2)
        return _exact_append(c, s) if blocks < 12000 else None
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda")
    group = c["heads"] // c["kv_heads"]
    for b, n in enumerate(s["lens"].tolist()):
        if n == 0:
            continue
        pages = s["table"][b, : -(-n // c["page"])].long()
        kv = []
        for name in ("k", "v"):
            step = s[name + "_scales"][pages].double().repeat_interleave(c["block"], dim=1)
            codes = s[name + "_pages"].view(torch.uint8)[pages].view(CODES[c["code"]])
            kv.append((codes.double() * step[..., None]).flatten(0, 1)[:n])
        away = n - 1 - torch.arange(n, device="cuda", dtype=torch.float64)
        for i in range(c["heads"]):
            x = kv[0][:, i // group] @ s["q"][b, i].double() * c["dim"] ** -0.5
            if c["cap"]:
                x = torch.tanh(x / c["cap"]) * c["cap"]
            if s["slopes"] is not None:
                x = x - s["slopes"][i].double() * away
            w = torch.exp(x - x.max())
            out[b, i] = (w @ kv[1][:, i // group]) / w.sum()
    return out
