"""Timed cases of the latent-attention operators: the cache append, the absorbed decode and the
expanded prefill that a hybrid of KDA and latent-attention layers runs next to the recurrence.

``run`` makes one pass through one operator.  With ``own`` it calls the library
(kda_gated_delta_04_gb300.kda); without, it computes the same thing in elementary torch
operations, in fp32, rounded once at the end.  ``exact`` gives the definition in fp64.

The operators (r = 512 latent channels, p = 64 position channels, n = v = 128 per head):

append   y_t = w * x_t / sqrt(mean(x_t^2) + eps);  cache[slot_t] = [y_t, R(pos_t) kpe_t];
         q'_th = R(pos_t) qpe_th.  R rotates the 32 channel pairs by the table's angles.
decode   s_bhj = scale * q_bh . cache_bj (all 576 channels), j < len_b;
         o_bh = sum_j softmax_j(s_bh) cache_bj[:512];  lse_bh = log sum_j exp(s_bhj).
prefill  s_thj = scale * q_th . [knope_jh, kpe_j], j in t's sequence and, counted from the end of
         both, not after t;  o_th = sum_j softmax_j(s_th) v_jh;  lse as above.
A row without keys has o = 0 and lse = -inf.
"""
import math
import random

import torch

own = False

R, P, N, V = 512, 64, 128, 128
SCALE = 1.0 / math.sqrt(N + P)
EPS = 1e-6
DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


def _kda():
    from kda_gated_delta_04_gb300 import kda
    return kda


# ---------------------------------------------------------------------------- cases
def listed():
    return [
        # one decode step of 64 sequences: the append is a handful of rows, latency is all
        {"name": "append_step_64", "op": "append", "dtype": "bf16", "tokens": 64, "heads": 32,
         "slots": 64 * 1024, "page": 64, "interleaved": False},
        # a packed prompt batch on its way into the cache
        {"name": "append_prompt_32768", "op": "append", "dtype": "bf16", "tokens": 32768, "heads": 32,
         "slots": 64 * 1024, "page": 64, "interleaved": False},
        # fp32 run (debugging, evaluation), pairs next to one another, an odd token count
        {"name": "append_f32_4097", "op": "append", "dtype": "f32", "tokens": 4097, "heads": 4,
         "slots": 8192, "page": 32, "interleaved": True},
        # a few short conversations: the smallest attention call
        {"name": "decode_short_4", "op": "decode", "dtype": "bf16", "batch": 4, "heads": 16,
         "min_len": 1, "max_len": 300, "page": 16, "lens": 11},
        # the decode batch of the recurrence's benchmark (256 x 32 heads), ragged contexts
        {"name": "decode_batch_256", "op": "decode", "dtype": "bf16", "batch": 256, "heads": 32,
         "min_len": 1, "max_len": 8192, "page": 64, "lens": 12},
        # two long documents: few rows, the work is along the cache
        {"name": "decode_long_2", "op": "decode", "dtype": "bf16", "batch": 2, "heads": 32,
         "min_len": 120000, "max_len": 131072, "page": 64, "lens": 13},
        # many heads on one latent: arithmetic weighs as much as the cache's bytes
        {"name": "decode_heads_128", "op": "decode", "dtype": "bf16", "batch": 48, "heads": 128,
         "min_len": 2000, "max_len": 8192, "page": 128, "lens": 14},
        # fp32 cache
        {"name": "decode_f32_16", "op": "decode", "dtype": "f32", "batch": 16, "heads": 8,
         "min_len": 1, "max_len": 2048, "page": 32, "lens": 15},
        # the prompt of the recurrence's benchmark (T = 4096, 32 heads)
        {"name": "prefill_4096", "op": "prefill", "dtype": "bf16", "seqs": 1, "heads": 32,
         "min_len": 4096, "max_len": 4096, "past": 0, "causal": True, "lens": 16},
        # ragged prompts packed into one call
        {"name": "prefill_packed_16", "op": "prefill", "dtype": "bf16", "seqs": 16, "heads": 16,
         "min_len": 1, "max_len": 1024, "past": 0, "causal": True, "lens": 17},
        # a chunk of a long prompt against what is cached already
        {"name": "prefill_chunk_1024", "op": "prefill", "dtype": "bf16", "seqs": 1, "heads": 32,
         "min_len": 1024, "max_len": 1024, "past": 15000, "causal": True, "lens": 18},
        # fp32 prompt, odd length
        {"name": "prefill_f32_1027", "op": "prefill", "dtype": "f32", "seqs": 1, "heads": 4,
         "min_len": 1027, "max_len": 1027, "past": 0, "causal": True, "lens": 19},
    ]


def _log_uniform(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.5)))))))


def draw(rng):
    op = rng.choice(["append", "decode", "decode", "prefill", "prefill"])
    f32 = rng.random() < 0.25
    if op == "append":
        return {"op": op, "dtype": "f32" if f32 else "bf16",
                "tokens": _log_uniform(rng, 1, 8192 if f32 else 32768),
                "heads": rng.choice([1, 4, 8, 16, 31, 32]), "slots": 64 * 1024, "page": rng.choice([16, 64, 128]),
                "interleaved": rng.random() < 0.5}
    if op == "decode":
        batch = _log_uniform(rng, 1, 32 if f32 else 256)
        heads = rng.choice([1, 4, 8] if f32 else [4, 8, 16, 20, 32, 64, 128])
        # at most the cache rows of the largest listed case, and its head-rows
        top = min(40000 if f32 else 1000000, (320000 if f32 else 32000000) // heads)
        max_len = _log_uniform(rng, 1, max(1, min(131072, top // batch)))
        return {"op": op, "dtype": "f32" if f32 else "bf16", "batch": batch, "heads": heads,
                "min_len": rng.choice([0, 1, max_len]), "max_len": max_len, "page": rng.choice([16, 32, 48, 64, 128]),
                "lens": rng.randrange(1 << 20)}
    heads = rng.choice([1, 2, 4] if f32 else [1, 4, 8, 16, 32])
    seqs = rng.choice([1, 1, 2, 3, 8, 16])
    # total rows and keys such that heads * rows * keys stays below the largest listed case of the type
    rows = int(math.sqrt((4200000 if f32 else 500000000) / heads))
    max_len = _log_uniform(rng, 1, max(1, min(8192, rows // seqs)))
    past = rng.choice([0, 0, _log_uniform(rng, 1, max(1, min(8192, rows // seqs - max_len)))])
    return {"op": op, "dtype": "f32" if f32 else "bf16", "seqs": seqs, "heads": heads,
            "min_len": rng.choice([0, 1, max_len]), "max_len": max_len, "past": past,
            "causal": rng.random() < 0.8, "lens": rng.randrange(1 << 20)}


def _lengths(case, count):
    """The sequences' lengths: a case's own, the same for every seed of its values."""
    rng = random.Random(case["lens"])
    lens = [rng.randint(case["min_len"], case["max_len"]) for _ in range(count)]
    lens[rng.randrange(count)] = case["max_len"]
    return lens


def _prefill_lengths(case):
    q = _lengths(case, case["seqs"])
    rng = random.Random(case["lens"] + 1)
    past = [0 if case["past"] == 0 else rng.randint((case["past"] + 1) // 2, case["past"]) for _ in q]
    return q, [a + b for a, b in zip(q, past)]


# ---------------------------------------------------------------------------- inputs
def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    dt = DTYPES[case["dtype"]]

    def normal(*shape, scale=1.0):
        return (torch.randn(*shape, generator=g, device="cuda") * scale).to(dt)

    if case["op"] == "append":
        t, h = case["tokens"], case["heads"]
        # the joint projection's rows [latent | position key], and queries [nope | position]
        kv = normal(t, R + P)
        q = normal(t, h, N + P)
        slots = torch.randperm(case["slots"], generator=g, device="cuda")[:t].to(torch.int32)
        positions = torch.randint(0, 131072, (t,), generator=g, device="cuda", dtype=torch.int32)
        angle = torch.arange(131072, device="cuda", dtype=torch.float64)[:, None] * (
            10000.0 ** (-torch.arange(0, P, 2, device="cuda", dtype=torch.float64) / P))
        return {"case": case, "latent": kv[:, :R], "k_pe": kv[:, R:], "q_pe": q[..., N:],
                "weight": (1.0 + 0.1 * torch.randn(R, generator=g, device="cuda")).to(dt),
                "cos_sin": torch.cat([angle.cos(), angle.sin()], 1).float(), "positions": positions, "slots": slots,
                "cache": normal(case["slots"] // case["page"], case["page"], R + P),
                "q_pe_out": torch.empty(t, h, P, dtype=dt, device="cuda"),
                "latent_out": torch.empty(t, R, dtype=dt, device="cuda")}
    if case["op"] == "decode":
        b, h, page = case["batch"], case["heads"], case["page"]
        lens = _lengths(case, b)
        pages = [-(-n // page) for n in lens]
        width = max(1, max(pages))
        total = max(1, sum(pages))
        order = torch.randperm(total, generator=g, device="cuda").to(torch.int32)
        table = torch.zeros(b, width, dtype=torch.int32, device="cuda")
        held = torch.arange(width, device="cuda")[None] < torch.tensor(pages, device="cuda")[:, None]
        table[held] = order[:sum(pages)]
        return {"case": case, "q": normal(b, h, R + P), "cache": normal(total, page, R + P), "table": table,
                "lens": torch.tensor(lens, dtype=torch.int32, device="cuda"),
                "o": torch.empty(b, h, R, dtype=dt, device="cuda"), "lse": torch.empty(b, h, device="cuda"),
                # the serving loop's scratch buffer, shared by every call
                "workspace": torch.empty(48 << 20, dtype=torch.uint8, device="cuda")}
    lq, lk = _prefill_lengths(case)
    h, tq, tk = case["heads"], sum(lq), sum(lk)
    kv = normal(tk, h, N + V)  # the up-projection's rows [nope key | value] of each head

    def offsets(lens):
        return torch.tensor([sum(lens[:i]) for i in range(len(lens) + 1)], dtype=torch.int32, device="cuda")

    return {"case": case, "q": normal(tq, h, N + P), "k_nope": kv[..., :N], "k_pe": normal(tk, P), "v": kv[..., N:],
            "cu_q": offsets(lq), "cu_k": offsets(lk), "o": torch.empty(tq, h, V, dtype=dt, device="cuda"),
            "lse": torch.empty(tq, h, device="cuda")}


# ---------------------------------------------------------------------------- one pass
def run(state):
    op = state["case"]["op"]
    if own:
        return {"append": _own_append, "decode": _own_decode, "prefill": _own_prefill}[op](state)
    return {"append": _plain_append, "decode": _plain_decode, "prefill": _plain_prefill}[op](state)


def _own_append(s):
    _kda().latent_append(s["latent"], s["k_pe"], s["cache"], s["slots"], norm_weight=s["weight"], norm_eps=EPS,
                         cos_sin=s["cos_sin"], positions=s["positions"], interleaved=s["case"]["interleaved"],
                         q_pe=s["q_pe"], q_pe_out=s["q_pe_out"], latent_out=s["latent_out"])
    return {"cache": s["cache"], "q_pe": s["q_pe_out"], "latent": s["latent_out"]}


def _own_decode(s):
    o, lse = _kda().latent_decode(s["q"], s["cache"], s["table"], s["lens"], SCALE, o=s["o"], lse=s["lse"],
                                  workspace=s["workspace"])
    return {"o": o, "lse": lse}


def _own_prefill(s):
    o, lse = _kda().latent_prefill(s["q"], s["k_nope"], s["k_pe"], s["v"], SCALE, s["cu_q"], s["cu_k"],
                                   causal=s["case"]["causal"], o=s["o"], lse=s["lse"])
    return {"o": o, "lse": lse}


def _rotate(x, cos, sin, interleaved):
    if interleaved:
        a, b = x[..., 0::2], x[..., 1::2]
        return torch.stack([a * cos - b * sin, b * cos + a * sin], -1).flatten(-2)
    a, b = x[..., :P // 2], x[..., P // 2:]
    return torch.cat([a * cos - b * sin, b * cos + a * sin], -1)


def _plain_append(s):
    dt, inter = s["latent"].dtype, s["case"]["interleaved"]
    x = s["latent"].float()
    y = (x * torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS) * s["weight"].float()).to(dt)
    cs = s["cos_sin"][s["positions"]]
    cos, sin = cs[:, :P // 2], cs[:, P // 2:]
    k = _rotate(s["k_pe"].float(), cos, sin, inter).to(dt)
    q = _rotate(s["q_pe"].float(), cos[:, None], sin[:, None], inter).to(dt)
    s["cache"].view(-1, R + P)[s["slots"].long()] = torch.cat([y, k], 1)
    return {"cache": s["cache"], "q_pe": q, "latent": y}


def _plain_decode(s):
    page, width = s["case"]["page"], s["table"].shape[1]
    at = torch.arange(width * page, device="cuda")
    rows = s["table"].long()[:, at // page] * page + at % page
    kv = s["cache"].view(-1, R + P)[rows].float()
    x = torch.matmul(s["q"].float(), kv.transpose(1, 2)) * SCALE
    x = x.masked_fill((at[None] >= s["lens"][:, None])[:, None], -math.inf)
    m = x.amax(-1, keepdim=True).clamp_min(torch.finfo(torch.float32).min)
    p = torch.exp(x - m)
    total = p.sum(-1, keepdim=True)
    o = torch.matmul(p, kv[..., :R]) / total.clamp_min(1e-30)
    return {"o": o.to(s["q"].dtype), "lse": (m + torch.log(total))[..., 0]}


def _plain_prefill(s):
    q, h = s["q"], s["q"].shape[1]
    tq, tk = q.shape[0], s["v"].shape[0]
    iq, ik = torch.arange(tq, device="cuda"), torch.arange(tk, device="cuda")
    nq = torch.searchsorted(s["cu_q"], iq, right=True, out_int32=True) - 1
    nk = torch.searchsorted(s["cu_k"], ik, right=True, out_int32=True) - 1
    seen = nq[:, None] == nk[None]
    if s["case"]["causal"]:  # counted from the end of both
        seen &= (s["cu_k"][nk + 1] - ik)[None] >= (s["cu_q"][nq + 1] - iq)[:, None]
    k = torch.cat([s["k_nope"].float(), s["k_pe"].float()[:, None].expand(-1, h, -1)], -1)
    x = torch.matmul(q.float().transpose(0, 1), k.permute(1, 2, 0)) * SCALE
    x = x.masked_fill_(~seen, -math.inf)
    m = x.amax(-1, keepdim=True).clamp_min(torch.finfo(torch.float32).min)
    p = x.sub_(m).exp_()
    total = p.sum(-1, keepdim=True)
    o = torch.matmul(p, s["v"].float().transpose(0, 1)) / total.clamp_min(1e-30)
    return {"o": o.transpose(0, 1).to(q.dtype), "lse": (m + torch.log(total))[..., 0].T}


# ---------------------------------------------------------------------------- what cannot be done without
def work(case):
    es = 2 if case["dtype"] == "bf16" else 4
    if case["op"] == "append":
        t, h = case["tokens"], case["heads"]
        # rows in, cache rows and normalised latent out, queries in and out, a table row, two indices
        return {"bytes": t * ((R + P) * 2 * es + R * es + 2 * h * P * es + P * 4 + 8) + R * es,
                "flops": t * (4 * R + 3 * P * (h + 1))}
    if case["op"] == "decode":
        lens, h = _lengths(case, case["batch"]), case["heads"]
        rows = case["batch"] * h
        return {"bytes": sum(lens) * (R + P) * es + rows * ((R + P + R) * es + 4)
                + sum(-(-n // case["page"]) for n in lens) * 4 + case["batch"] * 4,
                "flops": sum(lens) * h * 2 * (R + P + R)}
    lq, lk = _prefill_lengths(case)
    h, tq, tk = case["heads"], sum(lq), sum(lk)
    # the last query sees every key, each one before it a key less
    pairs = sum(a * b - (a * (a - 1) // 2 if case["causal"] else 0) for a, b in zip(lq, lk))
    return {"bytes": tq * h * ((N + P + V) * es + 4) + tk * (h * (N + V) + P) * es + 8 * (len(lq) + 1),
            "flops": pairs * h * 2 * (N + P + V)}


# ---------------------------------------------------------------------------- the definition, in 64 bits
def exact(case, seed):
    s = prepare(case, seed)
    d = torch.float64
    if case["op"] == "append":
        x = s["latent"].to(d)
        y = s["weight"].to(d) * x / torch.sqrt((x ** 2).sum(1, keepdim=True) / R + EPS)
        table = s["cos_sin"].to(d)[s["positions"].long()]
        turn = torch.complex(table[:, :P // 2], table[:, P // 2:])

        def rotated(z, by):
            pairs = z.unflatten(-1, (P // 2, 2)) if case["interleaved"] else z.unflatten(-1, (2, P // 2)).transpose(-1, -2)
            out = torch.view_as_real(torch.view_as_complex(pairs.contiguous()) * by)
            return (out if case["interleaved"] else out.transpose(-1, -2)).flatten(-2)

        cache = s["cache"].to(d).reshape(-1, R + P)
        cache.index_copy_(0, s["slots"].long(), torch.cat([y, rotated(s["k_pe"].to(d), turn)], 1))
        return {"cache": cache.view(s["cache"].shape), "q_pe": rotated(s["q_pe"].to(d), turn[:, None]), "latent": y}
    if case["op"] == "decode":
        b, h, page = case["batch"], case["heads"], case["page"]
        o = torch.zeros(b, h, R, dtype=d, device="cuda")
        lse = torch.full((b, h), -math.inf, dtype=d, device="cuda")
        for i, n in enumerate(_lengths(case, b)):
            if n:
                kv = s["cache"][s["table"][i, :-(-n // page)].long()].reshape(-1, R + P)[:n].to(d)
                x = SCALE * (s["q"][i].to(d) @ kv.T)
                lse[i] = torch.logsumexp(x, 1)
                o[i] = torch.softmax(x, 1) @ kv[:, :R]
        return {"o": o, "lse": lse}
    lq, lk = _prefill_lengths(case)
    o = torch.zeros(sum(lq), case["heads"], V, dtype=d, device="cuda")
    lse = torch.full((sum(lq), case["heads"]), -math.inf, dtype=d, device="cuda")
    a = b = 0
    for n, m in zip(lq, lk):
        for i in range(case["heads"] if n and m else 0):
            k = torch.cat([s["k_nope"][b:b + m, i], s["k_pe"][b:b + m]], 1).to(d)
            x = SCALE * (s["q"][a:a + n, i].to(d) @ k.T)
            if case["causal"]:
                x += torch.full_like(x, -math.inf).triu(m - n + 1)
            lse[a:a + n, i] = torch.logsumexp(x, 1)
            o[a:a + n, i] = torch.softmax(x, 1) @ s["v"][b:b + m, i].to(d)
        a, b = a + n, b + m
    return {"o": o, "lse": lse}
