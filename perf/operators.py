"""Cases of the serving operators around multi-head attention: rotary positions and the append to a paged key/value
cache, attention of one new token over that cache, attention with capped and biased scores under span masks, and the
RMS norm with residual addition and 8-bit output. Each case runs in a plain form (elementary torch operations, fp32
with fp64 angles) or, where ``own`` is set, through the library's entry points."""
import math
import random

import numpy as np
import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
E4M3_MAX = 448.0
EPS = 1e-6


def listed():
    return [
        # one new token of one sequence: the latency of the step's smallest call
        dict(name="append one token", op="append", dtype="bf16", batch=1, tokens=1, start=700, heads=16, kv_heads=4,
             dim=64, page=16, rot=64, interleaved=False, ragged=False),
        # a batch of prompts of the long workload's size enters the cache; heads of 128, half of each rotated
        dict(name="append prompts", op="append", dtype="bf16", batch=4, tokens=8192, start=64, heads=32, kv_heads=8,
             dim=128, page=64, rot=64, interleaved=False, ragged=True),
        # queries and keys far into a long context, interleaved pairs, fp32, no cache
        dict(name="rotary far fp32", op="rotary", dtype="f32", batch=3, tokens=2501, start=900000, heads=16,
             kv_heads=16, dim=64, rot=64, interleaved=True),
        # the decoding benchmark's cache (16 sequences of 8192 tokens, 16 heads of 64), in pages
        dict(name="decode 16 x 8192", op="decode", dtype="bf16", batch=16, length=8192, ragged=False, heads=16,
             kv_heads=16, dim=64, page=64, cap=0.0, slopes=False),
        # many sequences of different lengths, grouped heads of 128, capped scores
        dict(name="decode ragged grouped", op="decode", dtype="bf16", batch=48, length=15000, ragged=True, heads=32,
             kv_heads=8, dim=128, page=16, cap=30.0, slopes=False),
        # one sequence with a long history: the split over the length has to fill the GPU
        dict(name="decode one long", op="decode", dtype="bf16", batch=1, length=131071, ragged=False, heads=16,
             kv_heads=2, dim=128, page=32, cap=0.0, slopes=True),
        # a few short fp32 sequences: latency
        dict(name="decode short fp32", op="decode", dtype="f32", batch=4, length=333, ragged=True, heads=8,
             kv_heads=4, dim=64, page=16, cap=0.0, slopes=False),
        # the long workload (4 x 8192, 16 heads of 64) packed with documents
        dict(name="attention documents", op="attention", dtype="bf16", batch=4, lq=8192, lk=8192, heads=16,
             kv_heads=16, dim=64, causal=True, cap=0.0, slopes=False, docs=1500, prefix=False, padded=False),
        # the long workload with heads of 128, grouped, scores capped
        dict(name="attention capped", op="attention", dtype="bf16", batch=4, lq=8192, lk=8192, heads=8,
             kv_heads=2, dim=128, causal=True, cap=50.0, slopes=False, docs=0, prefix=False, padded=False),
        # the decoder workload's length behind a bidirectional prefix, distance bias, padded, odd sizes
        dict(name="attention prefix bias", op="attention", dtype="bf16", batch=5, lq=255, lk=333, heads=8,
             kv_heads=4, dim=64, causal=True, cap=0.0, slopes=True, docs=0, prefix=True, padded=True),
        # a decoding batch's rows: latency
        dict(name="norm few rows", op="norm", dtype="bf16", rows=16, width=1024, residual=True, quant="group"),
        # every token of the long workload at four times its width, one scale a row
        dict(name="norm long", op="norm", dtype="bf16", rows=32768, width=4096, residual=True, quant="row"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["append", "rotary", "decode", "decode", "attention", "attention", "norm"])
    dtype = "bf16" if rng.random() < 0.7 else "f32"
    dim = rng.choice([64, 128])
    kv_heads = rng.choice([1, 2, 3, 4, 5, 8, 16])
    group = rng.choice([1, 1, 2, 3, 4, 5, 7, 8])
    heads = kv_heads * group
    if op in ("append", "rotary"):
        batch = _log(rng, 1, 64)
        tokens = _log(rng, 1, max(1, min(8192, 30_000_000 // (batch * (heads + 2 * kv_heads) * dim))))
        c = dict(op=op, dtype=dtype, batch=batch, tokens=tokens, start=_log(rng, 1, 1_500_000 if op == "rotary" else 4000),
                 heads=heads, kv_heads=kv_heads, dim=dim, rot=2 * _log(rng, 4, dim // 2), interleaved=rng.random() < 0.5)
        if op == "append":
            c.update(page=rng.choice([1, 8, 16, 24, 32, 64, 100, 128, 256]), ragged=rng.random() < 0.5)
        return c
    if op == "decode":
        batch = _log(rng, 1, 64)
        most = 370_000_000 // (batch * kv_heads * dim * (2 if dtype == "f32" else 1))
        return dict(op=op, dtype=dtype, batch=batch, length=_log(rng, 1, min(131072, max(1, most))),
                    ragged=rng.random() < 0.6, heads=heads, kv_heads=kv_heads, dim=dim,
                    page=rng.choice([1, 8, 16, 24, 32, 64, 100, 128, 256]), cap=rng.choice([0.0, 0.0, 15.0, 30.0, 50.0]),
                    slopes=rng.random() < 0.3)
    if op == "attention":
        heads = min(heads, 16) // kv_heads * kv_heads
        batch = _log(rng, 1, 8)
        area = 1.28e11 / dim / (batch * heads)
        lk = _log(rng, 1, min(8192, int(math.sqrt(area))))
        lq = lk if rng.random() < 0.6 else _log(rng, 1, lk)
        causal = rng.random() < 0.7
        return dict(op=op, dtype="bf16", batch=batch, lq=lq, lk=lk, heads=heads, kv_heads=kv_heads, dim=dim,
                    causal=causal, cap=rng.choice([0.0, 0.0, 20.0, 50.0]), slopes=rng.random() < 0.3,
                    docs=_log(rng, 16, 2000) if lq == lk and rng.random() < 0.4 else 0,
                    prefix=causal and rng.random() < 0.3, padded=rng.random() < 0.4)
    quant = rng.choice(["none", "row", "group"])
    width = _log(rng, 1, 64) * 128 if quant == "group" else _log(rng, 64, 8192)
    return dict(op="norm", dtype=dtype, rows=_log(rng, 1, 130_000_000 // width // (2 if dtype == "f32" else 1)),
                width=width, residual=rng.random() < 0.7, quant=quant)


# ------------------------------------------------------------------------------------------ inputs
def _generators(seed):
    return torch.Generator(device="cuda").manual_seed(seed), random.Random(seed)


def _normal(g, *shape, dtype):
    return torch.randn(shape, generator=g, device="cuda", dtype=torch.float32).to(dtype)


def _ints(values):
    return torch.tensor(values, dtype=torch.int32, device="cuda")


def _frequencies(c):
    i = torch.arange(0, c["rot"], 2, device="cuda", dtype=torch.float64)
    return (10000.0 ** (-i / c["rot"])).float()


def _paged(c, g, rng, longest, dtype):
    """Pages of every sequence in a random order, with a few unused ones."""
    per = -(-longest // c["page"])
    total = c["batch"] * per + 3
    order = list(range(total))
    rng.shuffle(order)
    table = _ints(order[: c["batch"] * per]).view(c["batch"], per)
    k = _normal(g, total, c["page"], c["kv_heads"], c["dim"], dtype=dtype)
    v = _normal(g, total, c["page"], c["kv_heads"], c["dim"], dtype=dtype)
    return k, v, table


def _slopes(heads):
    return torch.tensor([2.0 ** (-8.0 * (i + 1) / heads) for i in range(heads)], device="cuda", dtype=torch.float32)


def prepare(case, seed):
    c = case
    g, rng = _generators(seed)
    s = {"case": c}
    if c["op"] in ("append", "rotary"):
        t = DTYPES[c["dtype"]]
        B, T, h, hk, d = c["batch"], c["tokens"], c["heads"], c["kv_heads"], c["dim"]
        # queries, keys and values as one projection leaves them
        qkv = _normal(g, B, T, h + 2 * hk, d, dtype=t)
        s["q"], s["k"], s["v"] = qkv[:, :, :h], qkv[:, :, h:h + hk], qkv[:, :, h + hk:]
        s["q_out"], s["k_out"] = torch.zeros(B, T, h, d, device="cuda", dtype=t), torch.zeros(B, T, hk, d, device="cuda", dtype=t)
        s["inv_freq"] = _frequencies(c)
        if c["op"] == "rotary":
            first = torch.tensor([rng.randint(0, c["start"]) for _ in range(B)], device="cuda")
            s["positions"] = (first[:, None] + torch.arange(T, device="cuda")).to(torch.int32)
        else:
            s["start"] = _ints([rng.randint(0, c["start"]) for _ in range(B)])
            s["new_lens"] = _ints([rng.randint(0, T) if c["ragged"] else T for _ in range(B)])
            s["k_pages"], s["v_pages"], s["table"] = _paged(c, g, rng, c["start"] + T, t)
    elif c["op"] == "decode":
        t = DTYPES[c["dtype"]]
        s["q"] = _normal(g, c["batch"], c["heads"], c["dim"], dtype=t)
        lens = [rng.randint(0, c["length"]) if c["ragged"] else c["length"] for _ in range(c["batch"])]
        lens[0] = c["length"]
        s["lens"] = _ints(lens)
        s["k_pages"], s["v_pages"], s["table"] = _paged(c, g, rng, c["length"], t)
        s["slopes"] = _slopes(c["heads"]) if c["slopes"] else None
        s["out"] = torch.empty_like(s["q"])
    elif c["op"] == "attention":
        t = DTYPES[c["dtype"]]
        B, h, hk, d = c["batch"], c["heads"], c["kv_heads"], c["dim"]
        if c["lq"] == c["lk"]:
            qkv = _normal(g, B, c["lk"], h + 2 * hk, d, dtype=t)
            s["q"], s["k"], s["v"] = qkv[:, :, :h], qkv[:, :, h:h + hk], qkv[:, :, h + hk:]
        else:
            s["q"] = _normal(g, B, c["lq"], h, d, dtype=t)
            kv = _normal(g, B, c["lk"], 2 * hk, d, dtype=t)
            s["k"], s["v"] = kv[:, :, :hk], kv[:, :, hk:]
        s["out"] = torch.empty(B, c["lq"], h, d, device="cuda", dtype=t)
        s["slopes"] = _slopes(h) if c["slopes"] else None
        s["valid"] = _ints([rng.randint(c["lk"] // 2, c["lk"]) for _ in range(B)]) if c["padded"] else None
        s["prefix"] = _ints([rng.randint(0, c["lk"] // 2) for _ in range(B)]) if c["prefix"] else None
        s["docs"] = None
        if c["docs"]:
            rows = np.zeros((B, c["lk"]), dtype=np.int32)
            for b in range(B):
                at, n = 0, 0
                while at < c["lk"]:
                    end = at + max(1, int(rng.expovariate(1.0 / c["docs"])))
                    rows[b, at:end] = n
                    at, n = end, n + 1
            s["docs"] = torch.from_numpy(rows).cuda()
            s["spans"] = torch.empty(B, c["lk"], 2, device="cuda", dtype=torch.int32)
    else:
        t = DTYPES[c["dtype"]]
        n, d = c["rows"], c["width"]
        s["x"] = _normal(g, n, d, dtype=t)
        s["residual"] = _normal(g, n, d, dtype=t) if c["residual"] else None
        s["gain"] = (1.0 + 0.2 * torch.randn(d, generator=g, device="cuda")).to(t)
        s["sum"] = torch.empty_like(s["x"]) if c["residual"] else None
        s["y"] = torch.empty(n, d, device="cuda", dtype=t if c["quant"] == "none" else torch.float8_e4m3fn)
        s["scales"] = None
        if c["quant"] != "none":
            s["scales"] = torch.empty(n, 1 if c["quant"] == "row" else d // 128, device="cuda", dtype=torch.float32)
    if own:
        _handles(s)
    return s


def _handles(s):
    """What a program builds once for a model and its cache: descriptions of the cache, the frequencies and the scores,
    and the workspace of the split attention."""
    from transformer_head_scaled_fwd_gb300 import binding as mha
    c = s["case"]
    if c["op"] in ("append", "rotary"):
        s["rotary"] = mha.make_rotary(s["inv_freq"], interleaved=c["interleaved"])
    if c["op"] in ("append", "decode"):
        s["cache"] = mha.make_paged_cache(s["k_pages"], s["v_pages"], s["table"])
    if c["op"] in ("decode", "attention"):
        s["scores"] = mha.make_scores(cap=c["cap"], slopes=s["slopes"])
    if c["op"] == "decode":
        size = mha.paged_attention_workspace_size(mha.MHA_BF16 if c["dtype"] == "bf16" else mha.MHA_F32, c["batch"],
                                                  c["heads"], c["kv_heads"], c["dim"])
        s["workspace"] = torch.empty(size, dtype=torch.uint8, device="cuda")


# ------------------------------------------------------------------------------------------ plain forms
def _rotate(x, positions, inv_freq, interleaved, real):
    """x [B, T, H, d]; positions [B, T]; the first 2 len(inv_freq) columns of each head are rotated."""
    angle = positions.to(torch.float64)[:, :, None, None] * inv_freq.to(torch.float64)
    cos, sin = torch.cos(angle).to(real), torch.sin(angle).to(real)
    n = inv_freq.numel()
    x = x.to(real)
    head, rest = x[..., : 2 * n], x[..., 2 * n:]
    if interleaved:
        a, b = head[..., 0::2], head[..., 1::2]
        turned = torch.stack((a * cos - b * sin, b * cos + a * sin), dim=-1).flatten(-2)
    else:
        a, b = head[..., :n], head[..., n:]
        turned = torch.cat((a * cos - b * sin, b * cos + a * sin), dim=-1)
    return torch.cat((turned, rest), dim=-1)


def _softmax_rows(s, allowed):
    """exp(s - max) over the allowed keys and its sum; rows that allow nothing give zeros."""
    s = s.masked_fill(~allowed, -math.inf)
    top = s.amax(dim=-1, keepdim=True)
    p = torch.exp(s - torch.where(top == -math.inf, torch.zeros_like(top), top))
    total = p.sum(dim=-1, keepdim=True)
    return p / torch.where(total == 0, torch.ones_like(total), total)


def _plain_append(s):
    c = s["case"]
    t = s["q"].dtype
    B, T = c["batch"], c["tokens"]
    step = torch.arange(T, device="cuda")
    at = s["start"].long()[:, None] + step
    live = step < s["new_lens"].long()[:, None]
    q = _rotate(s["q"], at, s["inv_freq"], c["interleaved"], torch.float32).to(t)
    k = _rotate(s["k"], at, s["inv_freq"], c["interleaved"], torch.float32).to(t)
    page = s["table"].long().gather(1, at // c["page"])[live]
    slot = (at % c["page"])[live]
    s["k_pages"][page, slot] = k[live]
    s["v_pages"][page, slot] = s["v"][live]
    keep = live[:, :, None, None]
    return {"q": torch.where(keep, q, s["q_out"]), "k": torch.where(keep, k, s["k_out"]), "k_pages": s["k_pages"], "v_pages": s["v_pages"]}


def _plain_decode(s):
    c = s["case"]
    B, hk, d = c["batch"], c["kv_heads"], c["dim"]
    group = c["heads"] // hk
    k = s["k_pages"][s["table"].long()].flatten(1, 2).float().permute(0, 2, 3, 1)
    v = s["v_pages"][s["table"].long()].flatten(1, 2).float().permute(0, 2, 1, 3)
    q = s["q"].float().view(B, hk, group, d)
    x = torch.matmul(q, k) / math.sqrt(d)
    if c["cap"]:
        x = c["cap"] * torch.tanh(x / c["cap"])
    j = torch.arange(x.shape[-1], device="cuda")
    n = s["lens"].long()[:, None, None, None]
    if s["slopes"] is not None:
        x = x - s["slopes"].view(1, hk, group, 1) * (n - 1 - j).float()
    p = _softmax_rows(x, (j < n).expand_as(x))
    # slots behind a sequence's end hold what an earlier owner left there
    v = torch.where((j < n[:, 0])[..., None], v, torch.zeros_like(v))
    return torch.matmul(p, v).view(B, c["heads"], d).to(s["q"].dtype)


def _allowed(s, lo=0, hi=None):
    """[B, rows lo:hi, L_k]: the keys that each query may attend to."""
    c = s["case"]
    i = torch.arange(c["lq"], device="cuda")[lo:hi, None] + (c["lk"] - c["lq"])
    j = torch.arange(c["lk"], device="cuda")[None]
    ok = torch.ones(c["batch"], i.shape[0], c["lk"], dtype=torch.bool, device="cuda")
    if c["causal"]:
        seen = (j <= i)[None]
        if s["prefix"] is not None:
            seen = seen | (j[None] < s["prefix"].long()[:, None, None])
        ok = ok & seen
    if s["docs"] is not None:
        ok = ok & (s["docs"][:, lo:hi, None] == s["docs"][:, None, :])
    if s["valid"] is not None:
        ok = ok & (j[None] < s["valid"].long()[:, None, None])
    return ok


def _plain_attention(s):
    c = s["case"]
    B, hk, d = c["batch"], c["kv_heads"], c["dim"]
    group = c["heads"] // hk
    q = s["q"].float().view(B, c["lq"], hk, group, d).permute(0, 2, 3, 1, 4).reshape(B, hk, group * c["lq"], d)
    k = s["k"].float().permute(0, 2, 3, 1)
    v = s["v"].float().permute(0, 2, 1, 3)
    x = (torch.matmul(q, k) / math.sqrt(d)).view(B, hk, group, c["lq"], c["lk"])
    if c["cap"]:
        x = c["cap"] * torch.tanh(x / c["cap"])
    if s["slopes"] is not None:
        i = torch.arange(c["lq"], device="cuda")[:, None] + (c["lk"] - c["lq"])
        away = (i - torch.arange(c["lk"], device="cuda")).abs().float()
        x = x - s["slopes"].view(1, hk, group, 1, 1) * away
    p = _softmax_rows(x, _allowed(s)[:, None, None])
    o = torch.matmul(p.view(B, hk, group * c["lq"], c["lk"]), v).view(B, hk, group, c["lq"], d)
    return o.permute(0, 3, 1, 2, 4).reshape(B, c["lq"], c["heads"], d).to(s["q"].dtype)


def _plain_norm(s):
    c = s["case"]
    z = s["x"].float()
    if s["residual"] is not None:
        z = z + s["residual"].float()
    y = z * torch.rsqrt((z * z).mean(dim=-1, keepdim=True) + EPS) * s["gain"].float()
    out = {}
    if s["residual"] is not None:
        out["sum"] = z.to(s["x"].dtype)
    if c["quant"] == "none":
        out["y"] = y.to(s["x"].dtype)
        return out
    blocks = y.view(c["rows"], s["scales"].shape[1], -1)
    top = blocks.abs().amax(dim=-1, keepdim=True)
    scale = torch.where(top == 0, torch.ones_like(top), top / E4M3_MAX)
    out["y"] = (blocks / scale).clamp(-E4M3_MAX, E4M3_MAX).view_as(y).to(torch.float8_e4m3fn)
    out["scales"] = scale.squeeze(-1)
    return out


# ------------------------------------------------------------------------------------------ the library's calls
def _own(s):
    from transformer_head_scaled_fwd_gb300 import binding as mha
    c = s["case"]
    if c["op"] == "rotary":
        mha.mha_rotary(s["q"], k=s["k"], q_out=s["q_out"], k_out=s["k_out"], positions=s["positions"], rotary=s["rotary"])
        return {"q": s["q_out"], "k": s["k_out"]}
    if c["op"] == "append":
        mha.mha_paged_append(s["k"], s["v"], s["start"], cache=s["cache"], q=s["q"], q_out=s["q_out"], k_out=s["k_out"],
                             new_lens=s["new_lens"], rotary=s["rotary"])
        return {"q": s["q_out"], "k": s["k_out"], "k_pages": s["k_pages"], "v_pages": s["v_pages"]}
    if c["op"] == "decode":
        mha.mha_paged_attention(s["q"], s["lens"], cache=s["cache"], out=s["out"], workspace=s["workspace"], scores=s["scores"])
        return s["out"]
    if c["op"] == "attention":
        spans = None
        if s["docs"] is not None:
            spans = s["spans"]
            mha.mha_document_spans(s["docs"], spans=spans)
        mask = mha.make_span_mask(causal=c["causal"], q_offset=c["lk"] - c["lq"], key_valid_lens=s["valid"],
                                  prefix_lens=s["prefix"], doc_spans=spans)
        mha.mha_attention(s["q"], s["k"], s["v"], out=s["out"], mask=mask, scores=s["scores"])
        return s["out"]
    mha.mha_rmsnorm(s["x"], s["gain"], EPS, y=s["y"], residual=s["residual"], sum_out=s["sum"], scales=s["scales"])
    return {k: s[k] for k in ("sum", "y", "scales") if s[k] is not None}


def run(state):
    if own:
        return _own(state)
    c = state["case"]
    if c["op"] == "rotary":
        return {"q": _rotate(state["q"], state["positions"], state["inv_freq"], c["interleaved"], torch.float32).to(state["q"].dtype),
                "k": _rotate(state["k"], state["positions"], state["inv_freq"], c["interleaved"], torch.float32).to(state["q"].dtype)}
    return {"append": _plain_append, "decode": _plain_decode, "attention": _plain_attention, "norm": _plain_norm}[c["op"]](state)


# ------------------------------------------------------------------------------------------ work and 64-bit results
def work(case):
    c = case
    es = 4 if c["dtype"] == "f32" else 2
    if c["op"] in ("append", "rotary"):
        live = 0.5 if c.get("ragged") else 1.0
        tokens = live * c["batch"] * c["tokens"] * c["dim"]
        turned = c["heads"] + c["kv_heads"]
        moved = 2 * turned if c["op"] == "rotary" else 2 * turned + 3 * c["kv_heads"]   # q, k in and out; k, v to the pages
        return {"bytes": es * tokens * moved, "flops": 3.0 * tokens * turned * c["rot"] / c["dim"]}
    if c["op"] == "decode":
        keys = c["length"] + (c["batch"] - 1) * c["length"] * (0.5 if c["ragged"] else 1.0)
        return {"bytes": es * (2.0 * keys * c["kv_heads"] * c["dim"] + 2 * c["batch"] * c["heads"] * c["dim"]),
                "flops": 4.0 * keys * c["heads"] * c["dim"]}
    if c["op"] == "attention":
        lq, lk = c["lq"], c["lk"]
        keys = lk * (0.75 if c["padded"] else 1.0)
        pairs = lq * keys if not c["causal"] else max(1.0, lq * keys - lq * lq / 2.0 * (0.6 if c["padded"] else 1.0))
        if c["docs"]:
            pairs = lq * min(keys, c["docs"]) * (1.0 if c["causal"] else 2.0)   # lengths spread exponentially about their mean
        return {"bytes": es * c["batch"] * c["dim"] * (2.0 * lq * c["heads"] + 2.0 * lk * c["kv_heads"]),
                "flops": 4.0 * c["batch"] * c["heads"] * c["dim"] * pairs}
    n = float(c["rows"]) * c["width"]
    out = es if c["quant"] == "none" else 1
    return {"bytes": n * (es * (3 if c["residual"] else 1) + out), "flops": 5.0 * n}


def _exact_heads(q, k, v, c, allowed, slopes, offset):
    """One sequence in fp64: q [rows, h, d], k, v [L_k, h_kv, d], allowed [rows, L_k]."""
    out = torch.zeros(q.shape, dtype=torch.float64, device="cuda")
    group = c["heads"] // c["kv_heads"]
    i = torch.arange(q.shape[0], device="cuda", dtype=torch.float64)[:, None] + offset
    away = (i - torch.arange(k.shape[0], device="cuda", dtype=torch.float64)[None]).abs()
    for n in range(c["heads"]):
        x = q[:, n].double() @ k[:, n // group].double().T * c["dim"] ** -0.5
        if c["cap"]:
            x = torch.tanh(x / c["cap"]) * c["cap"]
        if slopes is not None:
            x = x - slopes[n].double() * away
        x = torch.where(allowed, x, torch.full_like(x, -1e300))
        w = torch.exp(x - x.max(dim=1, keepdim=True).values) * allowed
        out[:, n] = (w @ v[:, n // group].double()) / w.sum(dim=1, keepdim=True).clamp_min(1e-300)
    return out


def exact(case, seed):
    c = case
    s = prepare(case, seed)
    if c["op"] in ("append", "rotary"):
        if c["op"] == "rotary":
            at = s["positions"].long()
        else:
            at = s["start"].long()[:, None] + torch.arange(c["tokens"], device="cuda")
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
        if c["op"] == "rotary":
            return done
        pages = {"k": s["k_pages"].double(), "v": s["v_pages"].double()}
        counts, table = s["new_lens"].tolist(), s["table"].long()
        for b, n in enumerate(counts):
            where = at[b, :n]
            page, slot = table[b, where // c["page"]], where % c["page"]
            pages["k"][page, slot] = done["k"][b, :n]
            pages["v"][page, slot] = s["v"][b, :n].double()
            done["q"][b, n:] = 0
            done["k"][b, n:] = 0
        return {"q": done["q"], "k": done["k"], "k_pages": pages["k"], "v_pages": pages["v"]}
    if c["op"] == "decode":
        out = torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda")
        for b, n in enumerate(s["lens"].tolist()):
            if n:
                pages = s["table"][b, : -(-n // c["page"])].long()
                k = s["k_pages"][pages].flatten(0, 1)[:n]
                v = s["v_pages"][pages].flatten(0, 1)[:n]
                out[b] = _exact_heads(s["q"][b:b + 1], k, v, c, torch.ones(1, n, dtype=torch.bool, device="cuda"), s["slopes"], n - 1)[0]
        return out
    if c["op"] == "attention":
        ok = _allowed(s)
        return torch.stack([_exact_heads(s["q"][b], s["k"][b], s["v"][b], c, ok[b], s["slopes"], c["lk"] - c["lq"])
                            for b in range(c["batch"])])
    z = s["x"].double() + (s["residual"].double() if s["residual"] is not None else 0.0)
    y = z / torch.sqrt((z ** 2).sum(dim=1, keepdim=True) / c["width"] + EPS) * s["gain"].double()
    got = {"sum": z} if s["residual"] is not None else {}
    if c["quant"] == "none":
        return {**got, "y": y}
    scale = y.view(c["rows"], s["scales"].shape[1], -1).abs().amax(dim=-1) / E4M3_MAX
    got["scales"] = torch.where(scale == 0, torch.ones_like(scale), scale)
    got["y"] = y / got["scales"].repeat_interleave(c["width"] // scale.shape[1], dim=1)
    return got
