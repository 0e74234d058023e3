"""Timed cases of what stands around the recurrence in a recurrent layer: the projections (a matrix
product with bias, activation and residual in its epilogue), the short causal convolution, and the
selective scan, the sibling recurrence with a diagonal transition.

``run`` makes one pass through one operator.  With ``own`` it calls the library
(kda_gated_delta_04_gb300.kda); without, it computes the same thing in elementary torch
operations, in fp32, rounded once at the end.  ``exact`` gives the definition in fp64.

linear   y_mn = act(sum_k x_mk w_nk + b_n) + r_mn.
conv     y_tc = act(b_c + sum_{j<W} w_cj x_(t-W+1+j)c), rows before a sequence's first one from its
         state of W - 1 rows; the new state is the last W - 1 rows of [state; x].
scan     d = softplus(dt + dt_bias);  h_cn <- exp(d_c A_cn) h_cn + d_c B_n x_c;
         y_c = (sum_n C_n h_cn + D_c x_c) silu(z_c), from each sequence's state h, which is kept.
"""
import math
import random

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
WIDTH = 4  # taps of the convolution


def _kda():
    from kda_gated_delta_04_gb300 import kda
    return kda


# ---------------------------------------------------------------------------- cases
def listed():
    return [
        # a few conversations, the output projection (32 heads of 128) added to the residual stream: latency
        {"name": "linear_step_4", "op": "linear", "dtype": "bf16", "rows": 4, "inner": 4096, "outer": 4096,
         "bias": False, "act": None, "residual": True, "out": "bf16"},
        # the decode batch of the recurrence's benchmark (256), q, k and v of 32 heads in one projection
        {"name": "linear_step_256", "op": "linear", "dtype": "bf16", "rows": 256, "inner": 4096, "outer": 12288,
         "bias": False, "act": None, "residual": False, "out": "bf16"},
        # the same projection of the benchmark's prompt (T = 4096), with a bias and SiLU
        {"name": "linear_prompt_4096", "op": "linear", "dtype": "bf16", "rows": 4096, "inner": 4096, "outer": 12288,
         "bias": True, "act": "silu", "residual": False, "out": "bf16"},
        # the write strengths of 32 heads over packed prompts, fp32 for the recurrence: few columns
        {"name": "linear_beta_16411", "op": "linear", "dtype": "bf16", "rows": 16411, "inner": 4096, "outer": 32,
         "bias": True, "act": "sigmoid", "residual": False, "out": "f32"},
        # fp32 run (debugging, evaluation) with everything in the epilogue, odd sizes
        {"name": "linear_f32_1027", "op": "linear", "dtype": "f32", "rows": 1027, "inner": 1025, "outer": 1003,
         "bias": True, "act": "gelu", "residual": True, "out": "f32"},
        # one token of 256 sequences, q, k and v as separate outputs, states in a pool
        {"name": "conv_step_256", "op": "conv", "dtype": "bf16", "seqs": 256, "min_len": 1, "max_len": 1,
         "channels": 12288, "parts": 3, "bias": False, "lens": 21},
        # the benchmark's prompt
        {"name": "conv_prompt_4096", "op": "conv", "dtype": "bf16", "seqs": 1, "min_len": 4096, "max_len": 4096,
         "channels": 12288, "parts": 3, "bias": False, "lens": 22},
        # ragged prompts packed into one call, the scan's input, fp32
        {"name": "conv_packed_f32_16", "op": "conv", "dtype": "f32", "seqs": 16, "min_len": 1, "max_len": 1024,
         "channels": 2048, "parts": 1, "bias": True, "lens": 23},
        # one token of 256 sequences, states in a pool: the bytes of the states
        {"name": "scan_step_256", "op": "scan", "dtype": "bf16", "seqs": 256, "min_len": 1, "max_len": 1,
         "channels": 4096, "states": 16, "lens": 24},
        # the benchmark's prompt
        {"name": "scan_prompt_4096", "op": "scan", "dtype": "bf16", "seqs": 1, "min_len": 4096, "max_len": 4096,
         "channels": 4096, "states": 16, "lens": 25},
        # a long document in a narrow model: few channels, the work is along the sequence
        {"name": "scan_long_16384", "op": "scan", "dtype": "bf16", "seqs": 1, "min_len": 16384, "max_len": 16384,
         "channels": 1024, "states": 16, "lens": 26},
        # ragged prompts with larger states, fp32
        {"name": "scan_packed_f32_8", "op": "scan", "dtype": "f32", "seqs": 8, "min_len": 1, "max_len": 700,
         "channels": 520, "states": 64, "lens": 27},
    ]


def _log_uniform(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.5)))))))


def draw(rng):
    op = rng.choice(["linear", "linear", "conv", "scan", "scan"])
    f32 = rng.random() < 0.25
    if op == "linear":
        # rows of a bf16 operand start on 16 bytes, as every model's do; of an fp32 one anywhere
        inner = _log_uniform(rng, 64, 2048) if f32 else 8 * _log_uniform(rng, 8, 512)
        outer = _log_uniform(rng, 1, 2048 if f32 else 12288)
        # at most the products and the bytes of the largest listed case of the type
        top = (1027 * 1025 * 1003 if f32 else 4096 * 4096 * 12288) // (inner * outer)
        top = min(top, (1027 if f32 else 4096) * 4096 * 4 // (inner + 4 * outer))
        return {"op": op, "dtype": "f32" if f32 else "bf16", "rows": _log_uniform(rng, 1, max(1, min(16384, top))),
                "inner": inner, "outer": outer, "bias": rng.random() < 0.5,
                "act": rng.choice([None, "silu", "gelu", "sigmoid", "softplus"]), "residual": rng.random() < 0.4,
                "out": "f32" if f32 or rng.random() < 0.25 else "bf16"}
    step = rng.random() < 0.35
    seqs = _log_uniform(rng, 1, 256) if step else rng.choice([1, 1, 2, 3, 8, 16])
    if op == "conv":
        parts = rng.choice([1, 3])
        channels = 8 * parts * _log_uniform(rng, 1, (512 if f32 else 1536) // parts)
        max_len = 1 if step else _log_uniform(rng, 1, max(1, min(16384, 4096 * 12288 // (4 if f32 else 1) // (channels * seqs))))
        return {"op": op, "dtype": "f32" if f32 else "bf16", "seqs": seqs,
                "min_len": max_len if step else rng.choice([0, 1, max_len]), "max_len": max_len, "channels": channels,
                "parts": parts, "bias": rng.random() < 0.5, "lens": rng.randrange(1 << 20)}
    states = rng.choice([8, 16, 16, 32, 64])
    channels = 8 * _log_uniform(rng, 1, 1024 if step else 512)
    if step:
        seqs = max(1, min(seqs, 200 * 4096 * 16 // (channels * max(16, states))))
    top = 4096 * 4096 * 16 // (channels * max(16, states) * seqs)
    max_len = 1 if step else _log_uniform(rng, 1, max(1, min(4096, top // (4 if f32 else 1))))
    return {"op": op, "dtype": "f32" if f32 else "bf16", "seqs": seqs,
            "min_len": max_len if step else rng.choice([0, 1, max_len]), "max_len": max_len, "channels": channels,
            "states": states, "lens": rng.randrange(1 << 20)}


def _lengths(case):
    """The sequences' lengths: a case's own, the same for every seed of its values."""
    rng = random.Random(case["lens"])
    lens = [rng.randint(case["min_len"], case["max_len"]) for _ in range(case["seqs"])]
    lens[rng.randrange(case["seqs"])] = case["max_len"]
    return lens


def _step(case):
    """One token of every sequence: the call that a generated token makes."""
    return case["min_len"] == case["max_len"] == 1 and case["seqs"] > 1


# ---------------------------------------------------------------------------- inputs
def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    dt = DTYPES[case["dtype"]]

    def normal(*shape, scale=1.0, dtype=dt):
        return (torch.randn(*shape, generator=g, device="cuda") * scale).to(dtype)

    def uniform(*shape):
        return torch.rand(*shape, generator=g, device="cuda")

    if case["op"] == "linear":
        m, n, k = case["rows"], case["outer"], case["inner"]
        out = DTYPES[case["out"]]
        return {"case": case, "x": normal(m, k), "w": normal(n, k, scale=k ** -0.5),
                "bias": normal(n) if case["bias"] else None,
                "residual": normal(m, n, dtype=out) if case["residual"] else None,
                "out": torch.empty(m, n, dtype=out, device="cuda")}
    lens = _lengths(case)
    t, s, c = sum(lens), len(lens), case["channels"]
    state = {"case": case, "lens": lens}
    if _step(case):
        # a pool with more states than the batch; the step writes the new states to another pool, as a
        # program does that may have to take a token back
        state["slots"] = torch.randperm(s + s // 8 + 1, generator=g, device="cuda")[:s].to(torch.int32)
        pool = s + s // 8 + 1
    else:
        state["cu"] = torch.tensor([sum(lens[:i]) for i in range(s + 1)], dtype=torch.int32, device="cuda")
        pool = s
    if case["op"] == "conv":
        # the joint projection's rows, of which the convolution takes a part
        x = normal(t, c + 64)
        parts = case["parts"]
        state.update({"x": x[:, :c], "weight": normal(c, WIDTH, scale=0.5), "bias": normal(c) if case["bias"] else None,
                      "old": normal(pool, WIDTH - 1, c), "new": torch.zeros(pool, WIDTH - 1, c, dtype=dt, device="cuda"),
                      "y": torch.empty(*((t, c) if parts == 1 else (parts, t, c // parts)), dtype=dt, device="cuda")})
        return state
    n = case["states"]
    bc = normal(t, 2 * n)
    step = torch.exp(uniform(c) * math.log(100.0) + math.log(1e-3))  # what the layer's steps start from
    state.update({"x": normal(t, c), "dt": normal(t, c), "z": normal(t, c), "B": bc[:, :n], "C": bc[:, n:],
                  "A": -(torch.arange(1, n + 1, device="cuda").float() * torch.exp(0.2 * normal(c, n, dtype=torch.float32))),
                  "D": 1.0 + 0.1 * normal(c, dtype=torch.float32), "dt_bias": step + torch.log(-torch.expm1(-step)),
                  "old": normal(pool, c, n, dtype=torch.float32),
                  "new": torch.zeros(pool, c, n, dtype=torch.float32, device="cuda"),
                  "y": torch.empty(t, c, dtype=dt, device="cuda")})
    return state


# ---------------------------------------------------------------------------- one pass
def run(state):
    op = state["case"]["op"]
    if own:
        return {"linear": _own_linear, "conv": _own_conv, "scan": _own_scan}[op](state)
    return {"linear": _plain_linear, "conv": _plain_conv, "scan": _plain_scan}[op](state)


def _own_linear(s):
    return _kda().linear(s["x"], s["w"], s["bias"], activation=s["case"]["act"], residual=s["residual"], out=s["out"])


def _own_conv(s):
    if _step(s["case"]):
        y = _kda().short_conv_step(s["x"], s["weight"], s["old"], s["bias"], slots=s["slots"], new_state=s["new"],
                                   parts=s["case"]["parts"], out=s["y"])
        return {"y": y, "state": s["new"]}
    y, new = _kda().short_conv(s["x"], s["weight"], s["bias"], s["cu"], s["old"], parts=s["case"]["parts"], out=s["y"],
                               final_state=s["new"])
    return {"y": y, "state": new}


def _own_scan(s):
    if _step(s["case"]):
        y = _kda().selective_scan_step(s["x"], s["dt"], s["A"], s["B"], s["C"], s["old"], s["D"], s["z"], s["dt_bias"],
                                       slots=s["slots"], new_state=s["new"], out=s["y"])
        return {"y": y, "state": s["new"]}
    y, new = _kda().selective_scan(s["x"], s["dt"], s["A"], s["B"], s["C"], s["D"], s["z"], s["dt_bias"], s["cu"], s["old"],
                                   out=s["y"], final_state=s["new"])
    return {"y": y, "state": new}


def _softplus(x):
    return x.clamp_min(0) + torch.log1p(torch.exp(-x.abs()))


ACTIVATIONS = {None: lambda v: v, "silu": lambda v: v / (1 + torch.exp(-v)), "sigmoid": lambda v: 1 / (1 + torch.exp(-v)),
               "gelu": lambda v: 0.5 * v * (1 + torch.erf(v * math.sqrt(0.5))), "softplus": _softplus}


def _plain_linear(s):
    v = torch.matmul(s["x"].float(), s["w"].float().T)
    if s["bias"] is not None:
        v += s["bias"].float()
    v = ACTIVATIONS[s["case"]["act"]](v)
    if s["residual"] is not None:
        v += s["residual"].float()
    return v.to(s["out"].dtype)


def _rows(s):
    """Of each sequence its first row, its length and its state's place in the pool."""
    at = s["slots"].tolist() if _step(s["case"]) else range(len(s["lens"]))
    first = 0
    for n, slot in zip(s["lens"], at):
        yield first, n, slot
        first += n


def _split(y, parts):
    return y if parts == 1 else y.view(y.shape[0], parts, -1).transpose(0, 1).contiguous()


def _plain_conv(s):
    w, dt = s["weight"].float(), s["x"].dtype
    if _step(s["case"]):  # the sequences at once
        slots = s["slots"].long()
        rows = torch.cat([s["old"][slots], s["x"][:, None]], 1)
        s["new"][slots] = rows[:, 1:]
        v = (rows.float() * w.T).sum(1)
    else:
        v = torch.empty(s["x"].shape, device="cuda")
        for first, n, slot in _rows(s):
            rows = torch.cat([s["old"][slot], s["x"][first:first + n]])
            s["new"][slot] = rows[n:]
            rows = rows.float()
            v[first:first + n] = sum(rows[j:j + n] * w[:, j] for j in range(WIDTH))
    if s["bias"] is not None:
        v += s["bias"].float()
    return {"y": _split((v / (1 + torch.exp(-v))).to(dt), s["case"]["parts"]), "state": s["new"]}


def _plain_scan(s):
    x, b, c = s["x"].float(), s["B"].float(), s["C"].float()
    d = _softplus(s["dt"].float() + s["dt_bias"])
    dx = d * x
    if _step(s["case"]):
        slots = s["slots"].long()
        h = torch.exp(d[:, :, None] * s["A"]) * s["old"][slots] + dx[:, :, None] * b[:, None]
        s["new"][slots] = h
        y = (h * c[:, None]).sum(-1)
    else:
        y = torch.empty_like(x)
        for first, n, slot in _rows(s):
            h = s["old"][slot]
            for t in range(first, first + n, 64):  # what does not hang on the state for 64 tokens at once
                at = slice(t, min(t + 64, first + n))
                decay = torch.exp(d[at][:, :, None] * s["A"])
                states = dx[at][:, :, None] * b[at][:, None]
                for keep, new in zip(decay, states):
                    h = new.addcmul_(keep, h)
                y[at] = (states * c[at][:, None]).sum(-1)
            s["new"][slot] = h
    z = s["z"].float()
    return {"y": ((y + s["D"] * x) * (z / (1 + torch.exp(-z)))).to(s["x"].dtype), "state": s["new"]}


# ---------------------------------------------------------------------------- what cannot be done without
def work(case):
    es = 2 if case["dtype"] == "bf16" else 4
    if case["op"] == "linear":
        m, n, k = case["rows"], case["outer"], case["inner"]
        eo = 2 if case["out"] == "bf16" else 4
        return {"bytes": (m * k + n * k + (n if case["bias"] else 0)) * es + m * n * eo * (2 if case["residual"] else 1),
                "flops": 2 * m * n * k}
    t, s, c = sum(_lengths(case)), case["seqs"], case["channels"]
    if case["op"] == "conv":
        return {"bytes": (2 * t * c + 2 * s * (WIDTH - 1) * c + c * (WIDTH + (1 if case["bias"] else 0))) * es + 4 * (s + 1),
                "flops": t * c * (2 * WIDTH + 4)}
    n = case["states"]
    return {"bytes": t * (4 * c + 2 * n) * es + 2 * s * c * n * 4 + c * (n + 2) * 4 + 4 * (s + 1),
            "flops": t * c * (7 * n + 12)}


# ---------------------------------------------------------------------------- the definition, in 64 bits
def exact(case, seed):
    s = prepare(case, seed)
    d = torch.float64
    f = torch.nn.functional
    if case["op"] == "linear":
        y = f.linear(s["x"].to(d), s["w"].to(d), None if s["bias"] is None else s["bias"].to(d))
        act = {None: lambda v: v, "silu": f.silu, "gelu": f.gelu, "sigmoid": torch.sigmoid,
               "softplus": lambda v: torch.logaddexp(v, torch.zeros_like(v))}[case["act"]]
        y = act(y)
        return y if s["residual"] is None else y + s["residual"].to(d)
    new = s["new"].to(d)
    if case["op"] == "conv":
        taps = s["weight"].to(d)[:, None]
        bias = None if s["bias"] is None else s["bias"].to(d)
        pieces = []
        for first, n, slot in _rows(s):
            rows = torch.cat([s["old"][slot].to(d), s["x"][first:first + n].to(d)])
            new[slot] = rows[rows.shape[0] - (WIDTH - 1):]
            if n:
                pieces.append(f.silu(f.conv1d(rows.T[None], taps, bias, groups=taps.shape[0]))[0].T)
        return {"y": _split(torch.cat(pieces), case["parts"]), "state": new}
    x, z, a = s["x"].to(d), s["z"].to(d), s["A"].to(d)
    step = torch.logaddexp(s["dt"].to(d) + s["dt_bias"].to(d), torch.zeros((), dtype=d, device="cuda"))
    y = torch.zeros_like(x)
    b, c = s["B"].to(d), s["C"].to(d)
    for first, n, slot in _rows(s):
        h = s["old"][slot].to(d)
        for t in range(first, first + n):
            h = torch.addcmul(torch.outer(step[t] * x[t], b[t]), torch.exp(step[t][:, None] * a), h)
            y[t] = h @ c[t]
        new[slot] = h
    return {"y": f.silu(z) * torch.addcmul(y, s["D"].to(d), x), "state": new}
