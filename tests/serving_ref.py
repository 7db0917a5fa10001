"""Plain 64-bit forms of the serving operators, from their definitions, and the tolerances of their
comparisons (torch, any device; loops over sequences and heads)."""
import math

import torch

HALF = {torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}   # half a rounding step, relative


def rotate(x, positions, inv_freq, interleaved=False, scale=1.0):
    """x [B, T, H, d] turned at positions [B, T], in fp64."""
    x = x.double().clone()
    n = inv_freq.numel()
    for i in range(n):
        c0, c1 = (2 * i, 2 * i + 1) if interleaved else (i, i + n)
        angle = positions.double()[:, :, None] * inv_freq[i].double()
        a, b = x[..., c0].clone(), x[..., c1].clone()
        x[..., c0] = scale * (a * torch.cos(angle) - b * torch.sin(angle))
        x[..., c1] = scale * (b * torch.cos(angle) + a * torch.sin(angle))
    return x


def rotate_tol(x, ref, inv_freq, interleaved, dtype, scale=1.0):
    """Half a step of the result; cos and sin off by 2^-21 (half-turn angle rounded to 2^-25, the
    double-float product, two ulp of the function) and three fp32 roundings on |a| + |b|."""
    n = inv_freq.numel()
    size = x.double().abs()
    pair = torch.zeros_like(size)
    for i in range(n):
        c0, c1 = (2 * i, 2 * i + 1) if interleaved else (i, i + n)
        pair[..., c0] = pair[..., c1] = size[..., c0] + size[..., c1]
    return HALF[dtype] * ref.abs() + 2.0 ** -20 * abs(scale) * pair


def attend(q, k, v, allowed, distance, *, scale, cap=0.0, slope=0.0):
    """One head in fp64: q [R, d], k, v [N, d], allowed [R, N], distance [R, N]. Rows without a key give
    zeros. Returns (o, sum of p |v|, largest scale * sum |q k| of the row's allowed keys)."""
    q, k, v = q.double(), k.double(), v.double()
    ok = allowed.any(dim=1)
    o = torch.zeros(q.shape[0], v.shape[1], dtype=torch.float64, device=q.device)
    mag, size = torch.zeros_like(o), torch.zeros(q.shape[0], 1, dtype=torch.float64, device=q.device)
    if not ok.any():
        return o, mag, size
    used = allowed.any(dim=0)
    k, v = torch.where(used[:, None], k, 0.0), torch.where(used[:, None], v, 0.0)   # what nobody sees may be anything
    s = (q @ k.T) * scale
    if cap:
        s = cap * torch.tanh(s / cap)
    s = s - slope * distance
    s = torch.where(allowed, s, -math.inf)
    p = torch.softmax(s[ok], dim=1)
    o[ok], mag[ok] = p @ v, p @ v.abs()
    size[ok] = torch.where(allowed, (q.abs() @ k.abs().T) * abs(scale), 0.0).amax(dim=1, keepdim=True)[ok]
    return o, mag, size


def attend_tol(o, mag, size, n, d, dtype, *, cap=0.0, far=0.0):
    """Bound of |kernel - o|: the output's half step; every weight off by a relative e^delta - 1, delta
    twice the error of a score: d products summed in fp32 (d 2^-24 of sum |q k|, which the cap does not
    enlarge), four roundings of the score itself (size + far, far = the largest bias), the cap's tanh to
    2^-20; exp2 to 2^-21; weights rounded to the values' type (half a step); n weights and products summed
    in fp32 (n 2^-24, at most: they are partial sums of a tree)."""
    delta = 2 * ((d + 4) * 2.0 ** -24 * size + 4 * 2.0 ** -24 * far + cap * 2.0 ** -20)
    rel = torch.expm1(delta) + 2.0 ** -20 + (HALF[dtype] if dtype == torch.bfloat16 else 0.0) + 2 * (n + 16) * 2.0 ** -24
    return HALF[dtype] * o.abs() + rel * mag + 1e-30


def check(got, ref, tol, what=""):
    got = got.double()
    assert got.shape == ref.shape, (got.shape, ref.shape)
    assert torch.isfinite(got).all(), f"{what}: not finite"
    over = (got - ref).abs() - tol
    worst = over.max().item() if over.numel() else -1.0
    assert worst <= 0, f"{what}: {int((over > 0).sum())} of {over.numel()} outside; worst by {worst:.3e} " \
                       f"(largest error {(got - ref).abs().max().item():.3e})"
