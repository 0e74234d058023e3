"""The projections, the short convolution and the selective scan by their definitions in float64, with the
error bounds of a rounded computation.

Bounds.  u is half a step of the output's type (bf16 2^-8, fp32 2^-24), u32 = 2^-24.

 linear  A partial sum of K products of random signs stays below P = 5 sqrt(sum (x w)^2) (five standard
         deviations).  On the CUDA cores each of K fp32 steps is off by at most u32 P, independently: 8 sqrt(K) u32 P.
         The tensor cores add 16 products at a time and may cut off instead of rounding: K / 16 steps of 2^-22 P,
         all of one sign.  The bias adds u32 (P + |b|).
 conv    at most five fp32 steps: 5 u32 (|b| + sum |w x|).
 act     no activation's slope is above 1.13.  Its own error: expf, division, erfcf and log1pf are good to
         a few units, 16 u32 of the result in all (the inner product v / sqrt 2 of gelu moves erfc's tail by
         v^2 u32 of itself at most: |v| <= 12 here, 144 u32); for bf16 outputs the approximations of exponential
         and quotient are good to (2 + 1.2 |v|) 2^-23 and 2^-22 of themselves: 2^-16 of the result for |v| <= 100.  Results
         below 1e-30 may be flushed.
 scan    The state follows  h = a h + b  with a = exp(d A), b = d B x.  d carries 8 u32 of itself (a sum, expf,
         log1pf), so a carries 9 |d A| u32 + 2^-21 (the hardware's exponential) of itself and b 11 u32.  With
         H = a H + |b| the error obeys  e = a e + ea a H + 11 u32 |b| + u32 H.  The sum over n states adds
         (n / 4 + 8) u32 sum |C| H.  dt + dt_bias carries u32 (|dt| + |dt_bias|) before the softplus, whose slope
         against its value is below 1, so in units of d that is (|dt| + |dt_bias|) u32 of itself.
         A state that grows (d A > 0) until its magnitude H, or the factor a alone, passes 2^127 has no value in
         fp32: from there on nothing is asked of what hangs on it (an infinite error, which check passes over).
"""
import math

import torch

U = {torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}
U32 = 2.0 ** -24
D = torch.float64


def softplus(v):
    return torch.logaddexp(v, torch.zeros((), dtype=v.dtype, device=v.device))


ACT = {None: lambda v: v, "silu": lambda v: v * torch.sigmoid(v), "sigmoid": torch.sigmoid,
       "gelu": lambda v: 0.5 * v * torch.special.erfc(-v * math.sqrt(0.5)), "softplus": softplus}


def own_error(act, y, dtype):
    if act is None:
        return torch.zeros_like(y)
    return (2.0 ** -16 if dtype == torch.bfloat16 else 160 * U32) * y.abs() + 1e-30


def check(got, want, err, label=""):
    """got within err (before the last rounding) and the rounding of want."""
    bound = err * (1 + U[got.dtype]) + U[got.dtype] * want.abs() + 1e-37
    beyond = torch.isinf(err).expand_as(want)
    assert not beyond.all() or not beyond.numel(), f"{label}: nothing to compare"
    nan = want.isnan() | beyond
    assert torch.equal(got.isnan() | beyond, nan), f"{label}: NaN in other places"
    far = ((got.to(D) - want).abs() / bound)[~nan]
    far = torch.where(got.to(D)[~nan] == want[~nan], torch.zeros_like(far), far)  # (infinities)
    worst = far.max().item() if far.numel() else 0.0
    print(f"[layer] {label}: {worst:.3f} of the bound")
    assert worst <= 1.0, f"{label}: off by {worst:.2f} of the bound"


def linear(x, w, bias, act, residual, out_dtype, tensor_cores):
    """As kda.linear, and its error before the last rounding."""
    K = x.shape[1]
    v = x.to(D) @ w.to(D).T
    P = 5 * torch.sqrt(x.to(D) ** 2 @ (w.to(D) ** 2).T)
    err = (2.0 ** -22 * max(1, K / 16) if tensor_cores else 8 * math.sqrt(K) * U32) * P
    if bias is not None:
        v = v + bias.to(D)
        err = err + U32 * (P + bias.to(D).abs())
    y = ACT[act](v)
    err = 1.13 * err + own_error(act, y, out_dtype)
    if residual is not None:
        y = y + residual.to(D)
        err = err + U32 * y.abs()
    return y, err


def conv(x, weight, bias, lens, state, act, parts=1):
    """As kda.short_conv on packed sequences (state [N, W - 1, C] or None); y, its error, the new state."""
    W, C = weight.shape[1], x.shape[1]
    y, err, new, first = [], [], [], 0
    for i, n in enumerate(lens):
        old = torch.zeros(W - 1, C, dtype=x.dtype, device=x.device) if state is None else state[i]
        rows = torch.cat([old, x[first:first + n]])
        new.append(rows[n:])
        v = torch.zeros(n, C, dtype=D, device=x.device) + (0 if bias is None else bias.to(D))
        size = v.abs()
        for j in range(W):
            p = rows[j:j + n].to(D) * weight[:, j].to(D)
            v, size = v + p, size + p.abs()
        a = ACT[act](v)
        y.append(a)
        err.append(1.13 * 5 * U32 * size + own_error(act, a, x.dtype))
        first += n
    y, err = torch.cat(y), torch.cat(err)
    if parts > 1:
        y, err = (t.view(t.shape[0], parts, C // parts).transpose(0, 1) for t in (y, err))
    return y, err, torch.stack(new)


def scan(x, dt, A, B, C, skip, z, dt_bias, lens, state, sp):
    """As kda.selective_scan on packed sequences, B and C [T, G, n]; y, its error, the new state and its error."""
    T, ch = x.shape
    n, G = A.shape[1], B.shape[1]
    raw = dt.to(D) + (0 if dt_bias is None else dt_bias.to(D))
    d = softplus(raw) if sp else raw
    moved = dt.to(D).abs() + (0 if dt_bias is None else dt_bias.to(D).abs())
    # relative to d; without softplus the sum's own
    rel = (8 + (moved if sp else moved / raw.abs().clamp_min(1e-300))) * U32
    A, xs = A.to(D), x.to(D)
    Bc = B.to(D).repeat_interleave(ch // G, 1)
    Cc = C.to(D).repeat_interleave(ch // G, 1)
    y, err = torch.zeros(T, ch, dtype=D, device=x.device), torch.zeros(T, ch, dtype=D, device=x.device)
    news, nerr, first = [], [], 0
    for i, m in enumerate(lens):
        h = torch.zeros(ch, n, dtype=D, device=x.device) if state is None else state[i].to(D)
        H, e = h.abs(), torch.zeros_like(h)
        for t in range(first, first + m):
            arg = d[t][:, None] * A
            a, b = torch.exp(arg), (d[t] * xs[t])[:, None] * Bc[t]
            ea = (rel[t][:, None] + U32) * arg.abs() + 2.0 ** -21
            e = a * e + ea * a * H + (rel[t][:, None] + 3 * U32) * b.abs()
            h, H = a * h + b, a * H + b.abs()
            e = torch.where((H > 2.0 ** 127) | (a > 2.0 ** 127), math.inf, e + U32 * H)
            y[t] = (Cc[t] * h).sum(1)
            err[t] = (Cc[t].abs() * (e + (n / 4 + 8) * U32 * H)).sum(1)
        news.append(h)
        nerr.append(e)
        first += m
    if skip is not None:
        y = y + skip.to(D) * xs
        err = err + 2 * U32 * ((skip.to(D) * xs).abs() + y.abs())
    if z is not None:
        g = ACT["silu"](z.to(D))
        err = torch.where(torch.isinf(err), err, err * g.abs()) + y.abs() * own_error("silu", g, x.dtype) + U32 * (y * g).abs()
        y = y * g
    return y, err, torch.stack(news), torch.stack(nerr)
