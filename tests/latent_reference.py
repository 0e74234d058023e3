"""Latent attention by its definition in float64, and the error bounds of a rounded computation.

Bounds.  u is half a step of the type (bf16 2^-8, fp32 2^-24).  With A = sum_j p_j |v_j|:

 bf16   the weights p_j enter a bf16 product, each off by at most u of itself: u A.  The output is
        rounded once: u |o|.  Scores, sums and exponentials are fp32; a quarter of u (2^-10) covers
        them: a score's error is at most 36 accumulation steps x 2^-23 x E with E = scale sum |q k|
        (26 for unit-normal rows, at most 100 here), 4e-4 at E = 100, and a weight's relative error is
        twice that at most.  Together 1.25 u (A + |o|).
 fp32   a score is a sum of 576 (192) products in at most 80 (48) sequential steps; with independent
        roundings the error of the sum is below 8 sqrt(80) u E < 72 u E, doubled in the normalised
        weight; 200 u covers the sums over the keys (n < 1e5, the same argument: 8 sqrt(n / 32) u)
        and the exponential (2 u).  Together u (144 E + 200) A, and u |o| for the output.
 lse    u32 (72 E + 200) + 2 u32 |lse| with u32 = 2^-24, whatever the type.
"""
import math

import torch

U = {torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}
U32 = 2.0 ** -24
R, P, N = 512, 64, 128


def attend(q, k, v, scale, seen=None):
    """q [H, M, C], k [H, L, C], v [H, L, D] float64; seen [M, L] or None.  Returns o [H, M, D], lse,
    A (sum p |v|) and E [H, M] (the largest scale sum |q k| of a seen key)."""
    H, M, _ = q.shape
    L = k.shape[1]
    if L == 0:
        z = torch.zeros(H, M, v.shape[2], dtype=q.dtype, device=q.device)
        lse = torch.full((H, M), -math.inf, dtype=q.dtype, device=q.device)
        return z, lse, z.clone(), torch.zeros_like(lse)
    s = torch.matmul(q, k.transpose(1, 2)) * scale
    e = torch.matmul(q.abs(), k.abs().transpose(1, 2)) * abs(scale)
    if seen is not None:
        s = s.masked_fill(~seen, -math.inf)
        e = e.masked_fill(~seen, 0.0)
    m = s.amax(-1, keepdim=True)
    p = torch.exp(s - torch.where(m == -math.inf, torch.zeros_like(m), m))
    total = p.sum(-1, keepdim=True)
    p = torch.where(total > 0, p / total.clamp_min(1e-300), torch.zeros_like(p))
    lse = torch.where(m == -math.inf, m, m + torch.log(total.clamp_min(1e-300)))[..., 0]
    return torch.matmul(p, v), lse, torch.matmul(p, v.abs()), e.amax(-1)


def decode(q, cache, table, lens, scale):
    """As kda.latent_decode; returns o [B, H, 512], lse, A, E in float64."""
    page = cache.shape[1]
    outs = []
    for b, n in enumerate(lens):
        pages = table[b, :-(-n // page)].long()
        kv = cache[pages].reshape(-1, R + P)[:n].double()
        H = q.shape[1]
        o, lse, a, e = attend(q[b].double()[None], kv[None], kv[None, :, :R], scale)
        outs.append((o[0], lse[0], a[0], e[0]))
    return [torch.stack(x) for x in zip(*outs)]


def prefill(q, k_nope, k_pe, v, scale, lq, lk, causal):
    """As kda.latent_prefill, the lengths on the host; returns o [Tq, H, 128], lse [Tq, H], A, E."""
    H = q.shape[1]
    a = b = 0
    outs = []
    for n, m in zip(lq, lk):
        qs = q[a:a + n].double().transpose(0, 1)
        ks = torch.cat([k_nope[b:b + m].double(), k_pe[b:b + m].double()[:, None].expand(m, H, P)], -1).transpose(0, 1)
        seen = None
        if causal:
            i, j = torch.arange(n, device=q.device)[:, None], torch.arange(m, device=q.device)[None]
            seen = j <= i + m - n
        o, lse, aa, e = attend(qs, ks, v[b:b + m].double().transpose(0, 1), scale, seen)
        outs.append((o.transpose(0, 1), lse.T, aa.transpose(0, 1), e.T))
        a, b = a + n, b + m
    return [torch.cat(x) for x in zip(*outs)]


def check(o, lse, ref, label=""):
    """Asserts o and lse within the bounds of the module's text."""
    ro, rl, A, E = ref
    u = U[o.dtype]
    o, lse = o.double(), lse.double()
    if u == U32:
        tol = u * ((144 * E[..., None] + 200) * A + ro.abs())
    else:
        tol = 1.25 * u * (A + ro.abs())
    tol = tol + 1e-30
    assert torch.isfinite(o).all(), f"{label}: not finite"
    worst = ((o - ro).abs() / tol).max().item() if o.numel() else 0.0
    empty = rl == -math.inf
    assert torch.equal(lse == -math.inf, empty), f"{label}: rows without keys"
    far = ((lse - rl).abs() / (U32 * (72 * E + 200 + 2 * rl.abs())))[~empty]
    wl = far.max().item() if far.numel() else 0.0
    print(f"[latent] {label}: o at {worst:.3f} of its bound, lse at {wl:.3f}")
    assert worst <= 1.0, f"{label}: o off by {worst:.2f} of its bound"
    assert wl <= 1.0, f"{label}: lse off by {wl:.2f} of its bound"


def rotate(x, cos, sin, interleaved):
    """x [..., 64] float64 rotated by cos, sin [..., 32]."""
    a, b = (x[..., 0::2], x[..., 1::2]) if interleaved else (x[..., :32], x[..., 32:])
    c, d = a * cos - b * sin, b * cos + a * sin
    return torch.stack([c, d], -1).flatten(-2) if interleaved else torch.cat([c, d], -1)
