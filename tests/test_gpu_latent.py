"""Latent attention on the GPU against its definition in float64 (latent_reference.py derives the
bounds), at the sizes, strides and contents where such kernels go wrong."""
import math
import random

import pytest
import torch

import latent_reference as ref
from kda_gated_delta_04_gb300 import kda

pytestmark = pytest.mark.gpu
SCALE = 192 ** -0.5
DT = {"bf16": torch.bfloat16, "f32": torch.float32}


def gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def normal(g, *shape, dtype=torch.bfloat16, scale=1.0):
    return (torch.randn(*shape, generator=g, device="cuda") * scale).to(dtype)


def errors():
    return torch.zeros(1, dtype=torch.int32, device="cuda")


# ------------------------------------------------------------------ append
def table_of(n, base=10000.0):
    angle = torch.arange(n, device="cuda", dtype=torch.float64)[:, None] * (
        base ** (-torch.arange(0, 64, 2, device="cuda", dtype=torch.float64) / 64))
    return torch.cat([angle.cos(), angle.sin()], 1).float()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("tokens,heads,page,interleaved", [
    (1, 1, 8, False), (1, 32, 16, True), (3, 7, 64, False), (33, 8, 64, True), (257, 9, 48, False), (1000, 16, 128, True)])
def test_append(dtype, tokens, heads, page, interleaved):
    """Normalised latent, rotated keys and queries, every row's slot; rows that are not written keep
    their contents.  Each output is one rounding (u) of an fp32 expression of at most 600 operations
    whose own error is far below u in bf16; in fp32 the mean of 512 squares is summed in 16 sequential
    and 5 tree steps (21 u at most), the root, the division and two products add 4 u: 16 u of the
    result in its square root; a rotation's two products and sum: 3 u (|a| + |b|)."""
    dt = DT[dtype]
    g = gen(tokens * 7 + heads)
    joint, q = normal(g, tokens, 576, dtype=dt), normal(g, tokens, heads, 192, dtype=dt)
    w = normal(g, 512, dtype=dt)
    pages = -(-tokens // page) + 2
    cache = normal(g, pages, page, 576, dtype=dt)
    before = cache.clone()
    slots = torch.randperm(pages * page, generator=g, device="cuda")[:tokens].int()
    if tokens > 2:
        slots[1] = -1
    cs = table_of(5000)
    pos = torch.randint(0, 5000, (tokens,), generator=g, device="cuda", dtype=torch.int32)
    pos[-1] = 4999
    lat, kpe = joint[:, :512], joint[:, 512:]
    q_out = torch.full((tokens, heads, 576), 7.0, dtype=dt, device="cuda")
    lat_out, kpe_out = torch.empty(tokens, 512, dtype=dt, device="cuda"), torch.empty(tokens, 64, dtype=dt, device="cuda")
    err = errors()
    kda.latent_append(lat, kpe, cache, slots, norm_weight=w, norm_eps=1e-5, cos_sin=cs, positions=pos,
                      interleaved=interleaved, q_pe=q[..., 128:], q_pe_out=q_out[..., 512:], latent_out=lat_out,
                      k_pe_out=kpe_out, errors=err)
    assert err.item() == 0
    x = lat.double()
    y = w.double() * x / torch.sqrt((x * x).mean(1, keepdim=True) + 1e-5)
    cos, sin = cs[pos.long()].double().split(32, 1)
    rk = ref.rotate(kpe.double(), cos, sin, interleaved)
    rq = ref.rotate(q[..., 128:].double(), cos[:, None], sin[:, None], interleaved)
    u = ref.U[dt]
    # a rotated pair is bounded by twice its larger member
    near = lambda a, b, k: ((a.double() - b).abs() <= k * u * b.abs() + 3 * ref.U32 * 2 * 6.0).all()
    k = 20 if dtype == "f32" else 1.01
    assert near(lat_out, y, k) and near(kpe_out, rk, k) and near(q_out[..., 512:], rq, k)
    assert (q_out[..., :512] == 7).all()
    want = before.view(-1, 576).clone()
    keep = slots >= 0
    want[slots[keep].long()] = torch.cat([lat_out, kpe_out], 1)[keep]
    assert torch.equal(cache.view(-1, 576), want)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_append_plain_and_in_place(dtype):
    """Without weight and table the rows are copied bit for bit; queries rotated in place are those
    rotated elsewhere; -0, infinity and NaN pass through an unrotated row."""
    dt = DT[dtype]
    g = gen(5)
    joint = normal(g, 40, 576, dtype=dt)
    joint[3, :4] = torch.tensor([math.inf, -math.inf, math.nan, -0.0])
    cache = torch.zeros(2, 32, 576, dtype=dt, device="cuda")
    slots = torch.arange(40, device="cuda", dtype=torch.int32)
    kda.latent_append(joint[:, :512], joint[:, 512:], cache, slots)
    bits = lambda t: t.contiguous().view(torch.int16 if dt == torch.bfloat16 else torch.int32)
    assert torch.equal(bits(cache.view(-1, 576)[:40]), bits(joint))
    q = normal(g, 40, 5, 64, dtype=dt)
    cs, pos = table_of(64), torch.arange(40, device="cuda", dtype=torch.int32)
    out = torch.empty_like(q)
    kda.latent_append(joint[:, :512], joint[:, 512:], cache, slots, cos_sin=cs, positions=pos, q_pe=q, q_pe_out=out)
    kda.latent_append(joint[:, :512], joint[:, 512:], cache, slots, cos_sin=cs, positions=pos, q_pe=q)
    assert torch.equal(q, out)


def test_append_reports_bad_slots_and_positions():
    """A slot out of range is not cached, a position out of range leaves the token out; both are
    reported and every other token is written."""
    g = gen(6)
    joint = normal(g, 6, 576)
    cache = torch.zeros(1, 8, 576, dtype=torch.bfloat16, device="cuda")
    slots = torch.tensor([0, 8, -2, 3, 4, 5], dtype=torch.int32, device="cuda")
    pos = torch.tensor([0, 1, 2, -1, 64, 63], dtype=torch.int32, device="cuda")
    q = normal(g, 6, 2, 64)
    out = torch.zeros_like(q)
    err = errors()
    kda.latent_append(joint[:, :512], joint[:, 512:], cache, slots, cos_sin=table_of(64), positions=pos, q_pe=q,
                      q_pe_out=out, errors=err)
    assert err.item() == 16 | 32
    assert cache[0].abs().sum(1).ne(0).tolist() == [True, False, False, False, False, True, False, False]
    assert out.abs().sum((1, 2)).ne(0).tolist() == [True, True, True, False, False, True]


def test_append_last_row_of_a_cache_past_32_bit_offsets():
    """A cache of 2^32 + bytes (element offsets past 2^31): the last slot's row is the one written."""
    rows = 3800000 // 8 * 8
    cache = torch.zeros(rows // 8, 8, 576, dtype=torch.bfloat16, device="cuda")
    assert cache.numel() > 2 ** 31
    joint = normal(gen(7), 1, 576)
    kda.latent_append(joint[:, :512], joint[:, 512:], cache, torch.tensor([rows - 1], dtype=torch.int32, device="cuda"))
    assert torch.equal(cache.view(-1, 576)[rows - 1], joint[0])
    assert cache.view(-1, 576)[:rows - 1].any().item() is False


# ------------------------------------------------------------------ decode
def paged(g, lens, page, dtype, width=None, extra=3, scale=1.0):
    """A shuffled paged cache for the lengths; table entries past a sequence's end are out of range
    and rows past it are NaN (neither may matter)."""
    pages = [-(-n // page) for n in lens]
    width = max([1] + pages) if width is None else width
    total = sum(pages) + extra
    cache = normal(g, total, page, 576, dtype=dtype, scale=scale)
    order = torch.randperm(total, generator=g, device="cuda").int().tolist()
    table = torch.full((len(lens), width), 2 ** 31 - 1, dtype=torch.int32)
    at = 0
    for b, k in enumerate(pages):
        table[b, :k] = torch.tensor(order[at:at + k], dtype=torch.int32)
        at += k
        if lens[b] % page:
            cache[order[at - 1], lens[b] % page:] = math.nan
    return cache, table.cuda()


DECODE = [
    ("one_token", 1, 1, 64, [1]), ("sixteen_heads", 4, 16, 16, [1, 63, 64, 65]), ("empty_rows", 5, 8, 32, [0, 7, 0, 129, 0]),
    ("all_empty", 3, 4, 16, [0, 0, 0]), ("odd_heads", 3, 5, 8, [31, 32, 33]), ("page_48", 3, 20, 48, [47, 48, 500]),
    ("page_8", 2, 32, 8, [1000, 77]), ("heads_33", 2, 33, 64, [300, 5]), ("heads_64", 3, 64, 64, [64, 1, 700]),
    ("heads_128", 2, 128, 128, [1500, 129]), ("heads_100", 2, 100, 64, [100, 400]), ("long", 1, 32, 64, [20001]),
    ("many", 200, 16, 16, [(37 * i) % 300 for i in range(200)]), ("page_256", 2, 32, 256, [257, 1023]),
    ("page_96", 2, 16, 96, [95, 1000]), ("a_thousand", 1000, 8, 8, [(53 * i) % 90 for i in range(1000)]),
    ("many_parts", 24, 32, 64, [3000 + 17 * i for i in range(24)]), ("long_short", 6, 64, 16, [5000, 1, 0, 3, 4000, 64]),
]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("name,batch,heads,page,lens", DECODE, ids=[c[0] for c in DECODE])
def test_decode(dtype, name, batch, heads, page, lens):
    g = gen(len(name) + batch)
    dt = DT[dtype]
    cache, table = paged(g, lens, page, dt)
    q = normal(g, batch, heads, 576, dtype=dt)
    err = errors()
    o, lse = kda.latent_decode(q, cache, table, torch.tensor(lens, dtype=torch.int32, device="cuda"), SCALE, errors=err)
    ref.check(o, lse, ref.decode(q, cache, table, lens, SCALE), name)
    assert err.item() == 0


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_decode_rising_and_falling_scores(dtype):
    """Scores that rise along the cache (every tile raises the maximum), that fall, and one key far
    above the rest in the middle: the running maximum is moved, kept and jumped."""
    g = gen(20)
    dt = DT[dtype]
    n, heads = 1500, 16
    cache, table = paged(g, [n] * 3, 64, dt)
    q = normal(g, 3, heads, 576, dtype=dt, scale=0.1)
    q[:, :, 0] = 4.0
    ramp = torch.linspace(-30, 30, n, device="cuda")
    for b, r in enumerate([ramp, -ramp, torch.where(torch.arange(n, device="cuda") == 700, 50.0, 0.0)]):
        at = torch.arange(n, device="cuda")
        cache.view(-1, 576)[table[b].long()[at // 64] * 64 + at % 64, 0] = (r / (4 * SCALE)).to(dt)
    o, lse = kda.latent_decode(q, cache, table, torch.tensor([n] * 3, dtype=torch.int32, device="cuda"), SCALE)
    ref.check(o, lse, ref.decode(q, cache, table, [n] * 3, SCALE), "ramps")


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_decode_strided_inputs_and_shared_table(dtype):
    """Queries as a part of wider rows, heads in front of the batch, a page table that is a slice of
    a wider one, and one table row for all sequences (stride 0)."""
    g = gen(21)
    dt = DT[dtype]
    lens = [130, 64, 200]
    cache, table = paged(g, lens, 64, dt)
    wide = torch.full((3, 50), -5, dtype=torch.int32, device="cuda")
    wide[:, 7:7 + table.shape[1]] = table
    base = normal(g, 8, 3, 640, dtype=dt)
    q = base.transpose(0, 1)[..., 64:]
    ln = torch.tensor(lens, dtype=torch.int32, device="cuda")
    o, lse = kda.latent_decode(q, cache, wide[:, 7:7 + table.shape[1]], ln, SCALE)
    ref.check(o, lse, ref.decode(q, cache, table, lens, SCALE), "strided")
    shared = table[2:3].expand(3, -1)
    lens = [200, 1, 131]
    o, lse = kda.latent_decode(q, cache, shared, torch.tensor(lens, dtype=torch.int32, device="cuda"), SCALE)
    ref.check(o, lse, ref.decode(q, cache, shared, lens, SCALE), "shared table")


def test_decode_is_deterministic_and_ignores_the_workspace():
    g = gen(22)
    lens = [3000, 1, 0, 777, 2049]
    cache, table = paged(g, lens, 64, torch.bfloat16)
    q = normal(g, 5, 32, 576)
    ln = torch.tensor(lens, dtype=torch.int32, device="cuda")
    ws = kda.latent_decode_workspace_for(32, kda.KDA_DTYPE_BF16, "cuda")
    a = [t.clone() for t in kda.latent_decode(q, cache, table, ln, SCALE, workspace=ws)]
    ws.fill_(255)
    b = kda.latent_decode(q, cache, table, ln, SCALE, workspace=ws)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_decode_reports_bad_pages_and_lengths(dtype):
    """A page out of range reads as zero rows, a length out of range is held to the table; both are
    reported, and the other sequences are as ever."""
    g = gen(23)
    dt = DT[dtype]
    lens = [100, 100, 100]
    cache, table = paged(g, lens, 64, dt)
    q = normal(g, 3, 8, 576, dtype=dt)
    bad = table.clone()
    bad[1, 0] = cache.shape[0]
    err = errors()
    o, lse = kda.latent_decode(q, cache, bad, torch.tensor(lens, dtype=torch.int32, device="cuda"), SCALE, errors=err)
    assert err.item() == 64
    want = ref.decode(q, cache, table, lens, SCALE)
    for b in (0, 2):
        ref.check(o[b], lse[b], [x[b] for x in want], f"sequence {b}")
    zero = torch.cat([cache, torch.zeros_like(cache[:1])])
    ref.check(o[1], lse[1], [x[0] for x in ref.decode(q[1:2], zero, bad[1:2], [100], SCALE)], "zero rows")
    cache2, table2 = paged(g, [128, 128, 128], 64, dt)
    err = errors()
    o, lse = kda.latent_decode(q, cache2, table2, torch.tensor([-1, 128, 129], dtype=torch.int32, device="cuda"), SCALE,
                               errors=err)
    assert err.item() == 1
    ref.check(o, lse, ref.decode(q, cache2, table2, [0, 128, 128], SCALE), "held lengths")


def test_decode_in_a_graph_with_new_lengths():
    """A captured call replays with other lengths, pages and queries, on a side stream."""
    g = gen(24)
    cache, table = paged(g, [500, 500], 64, torch.bfloat16)
    q = normal(g, 2, 32, 576)
    ln = torch.tensor([3, 400], dtype=torch.int32, device="cuda")
    ws = kda.latent_decode_workspace_for(32, kda.KDA_DTYPE_BF16, "cuda")
    o, lse = kda.latent_decode(q, cache, table, ln, SCALE, workspace=ws)
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        kda.latent_decode(q, cache, table, ln, SCALE, o=o, lse=lse, workspace=ws)
    for lens in ([500, 0], [64, 65], [1, 499]):
        ln.copy_(torch.tensor(lens, dtype=torch.int32))
        q.copy_(normal(g, 2, 32, 576))
        graph.replay()
        torch.cuda.synchronize()
        ref.check(o, lse, ref.decode(q, cache, table, lens, SCALE), str(lens))


def test_decode_offsets_past_32_bits():
    """Pages at the far end of a cache of more than 2^31 elements."""
    pages = 60000
    cache = torch.zeros(pages, 64, 576, dtype=torch.bfloat16, device="cuda")
    assert cache.numel() > 2 ** 31
    g = gen(25)
    cache[pages - 3:] = normal(g, 3, 64, 576)
    table = torch.tensor([[pages - 1, pages - 3, pages - 2]], dtype=torch.int32, device="cuda")
    q = normal(g, 1, 32, 576)
    o, lse = kda.latent_decode(q, cache, table, torch.tensor([190], dtype=torch.int32, device="cuda"), SCALE)
    ref.check(o, lse, ref.decode(q, cache, table, [190], SCALE), "far pages")


# ------------------------------------------------------------------ prefill
PREFILL = [
    ("one", 1, [1], [1]), ("tile", 2, [64], [64]), ("odd", 3, [65], [65]), ("two_tiles", 1, [128], [128]),
    ("past_a_tile", 2, [257], [257]), ("long", 2, [1100], [1100]), ("packed", 4, [5, 0, 130, 1, 300, 64], None),
    ("chunk", 3, [70], [1000]), ("chunks", 2, [1, 17, 256], [513, 17, 300]), ("fewer_keys", 2, [100, 40], [37, 0]),
    ("no_keys", 1, [9], [0]), ("step", 16, [1] * 20, [3 * i for i in range(20)]), ("tail", 1, [383], [385]),
]


def prefill_inputs(g, heads, lq, lk, dt, kscale=1.0):
    q, kv = normal(g, sum(lq), heads, 192, dtype=dt), normal(g, sum(lk), heads, 256, dtype=dt, scale=kscale)
    k_pe = normal(g, sum(lk), 576, dtype=dt)[:, 512:]
    cu = lambda l: torch.tensor([sum(l[:i]) for i in range(len(l) + 1)], dtype=torch.int32, device="cuda")
    return q, kv[..., :128], k_pe, kv[..., 128:], cu(lq), cu(lk)


@pytest.mark.parametrize("causal", [True, False], ids=["causal", "full"])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("name,heads,lq,lk", PREFILL, ids=[c[0] for c in PREFILL])
def test_prefill(dtype, causal, name, heads, lq, lk):
    lk = lq if lk is None else lk
    q, kn, kp, v, cu_q, cu_k = prefill_inputs(gen(len(name) + heads), heads, lq, lk, DT[dtype])
    err = errors()
    o, lse = kda.latent_prefill(q, kn, kp, v, SCALE, cu_q, cu_k, causal=causal, errors=err)
    ref.check(o, lse, ref.prefill(q, kn, kp, v, SCALE, lq, lk, causal), name)
    assert err.item() == 0


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_prefill_without_offsets_and_other_layouts(dtype):
    """One sequence without offsets; heads in front ([H, T, d] storage); a key shared by the heads
    (stride 0); outputs given."""
    g = gen(40)
    dt = DT[dtype]
    q = normal(g, 3, 150, 192, dtype=dt).transpose(0, 1)
    kn = normal(g, 150, 1, 128, dtype=dt).expand(150, 3, 128)
    v = normal(g, 3, 150, 128, dtype=dt).transpose(0, 1)
    kp = normal(g, 150, 64, dtype=dt)
    o = torch.empty(150, 3, 128, dtype=dt, device="cuda")
    o2, lse = kda.latent_prefill(q, kn, kp, v, SCALE, o=o)
    assert o2 is o
    ref.check(o, lse, ref.prefill(q, kn, kp, v, SCALE, [150], [150], True), "layouts")


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_prefill_peaked_scores(dtype):
    """Weights near one-hot, the peak at a random key of each row, and scores rising along the keys."""
    g = gen(41)
    q, kn, kp, v, cu, _ = prefill_inputs(g, 2, [520], [520], DT[dtype], kscale=3.0)
    ref.check(*kda.latent_prefill(q, kn, kp, v, SCALE), ref.prefill(q, kn, kp, v, SCALE, [520], [520], True), "peaked")
    kn[:, :, 0] = torch.linspace(-40, 40, 520, device="cuda").to(DT[dtype])[:, None]
    q[:, :, 0] = 5.0
    ref.check(*kda.latent_prefill(q, kn, kp, v, SCALE), ref.prefill(q, kn, kp, v, SCALE, [520], [520], True), "rising")


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("causal", [True, False], ids=["causal", "full"])
def test_prefill_rows_of_other_sequences_do_not_matter(dtype, causal):
    """The neighbours in the packing are NaN and infinite: the sequence between them is as alone."""
    g = gen(42)
    lens = [50, 91, 70]
    q, kn, kp, v, cu, _ = prefill_inputs(g, 2, lens, lens, DT[dtype])
    want = ref.prefill(q[50:141], kn[50:141], kp[50:141], v[50:141], SCALE, [91], [91], causal)
    for t in (q, kn, kp, v):
        t[:50] = math.nan
        t[141:] = math.inf
    o, lse = kda.latent_prefill(q, kn, kp, v, SCALE, cu, causal=causal)
    ref.check(o[50:141], lse[50:141], want, "between")


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_prefill_reports_malformed_offsets(dtype):
    g = gen(43)
    q, kn, kp, v, cu, _ = prefill_inputs(g, 1, [64, 64], [64, 64], DT[dtype])
    for bad in ([0, 100, 90], [0, 64, 200], [3, 64, 128], [0, -5, 128], [-7, 64, 128]):
        err = errors()
        kda.latent_prefill(q, kn, kp, v, SCALE, torch.tensor(bad, dtype=torch.int32, device="cuda"), errors=err)
        assert err.item() == 1, bad


def test_prefill_is_deterministic():
    """The pairs of CTAs take work over as they get done, in another order on every call: the same bits."""
    g = gen(46)
    lens = [700, 3, 1300, 0, 513, 64, 256]
    q, kn, kp, v, cu, _ = prefill_inputs(g, 16, lens, lens, torch.bfloat16)
    a = [t.clone() for t in kda.latent_prefill(q, kn, kp, v, SCALE, cu)]
    for _ in range(5):
        b = kda.latent_prefill(q, kn, kp, v, SCALE, cu)
        assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


@pytest.mark.parametrize("heads", [1, 24])
def test_prefill_many_sequences(heads):
    """More sequences than one round of the tile search holds (32 x 32), with empty ones between."""
    g = gen(47)
    lens = [(7 * i) % 13 for i in range(1500)]
    q, kn, kp, v, cu, _ = prefill_inputs(g, heads, lens, lens, torch.bfloat16)
    o, lse = kda.latent_prefill(q, kn, kp, v, SCALE, cu)
    ref.check(o, lse, ref.prefill(q, kn, kp, v, SCALE, lens, lens, True), "1500 sequences")


@pytest.mark.parametrize("causal", [True, False], ids=["causal", "full"])
def test_prefill_short_sequences_side_by_side(causal):
    """More query tiles than run at once, most of them the only one of their sequence: two such are worked
    on in turn, with key tiles of their own, whose tails may meet in one buffer."""
    rnd = random.Random(5)
    lq = [rnd.choice([0, 1, 17, 64, 200, 256, 300, 512, 700]) for _ in range(70)]
    lk = [l + rnd.choice([-3, 0, 0, 1, 63, 127, 128, 384, 500, 900]) if l else 0 for l in lq]
    lk = [max(0, l) for l in lk]
    q, kn, kp, v, cu_q, cu_k = prefill_inputs(gen(47), 3, lq, lk, torch.bfloat16)
    err = errors()
    o, lse = kda.latent_prefill(q, kn, kp, v, SCALE, cu_q, cu_k, causal=causal, errors=err)
    ref.check(o, lse, ref.prefill(q, kn, kp, v, SCALE, lq, lk, causal), "side by side")
    assert err.item() == 0


@pytest.mark.parametrize("causal", [True, False], ids=["causal", "full"])
@pytest.mark.parametrize("heads", [5, 6, 11, 12])
def test_prefill_f32_tiles_shared_by_four_two_or_one(heads, causal):
    """13 query tiles a head: 65 are shared by four CTAs each, 78 and 143 by two, 156 by none."""
    lq, lk = [5, 0, 130, 1, 300, 64], [5, 7, 200, 0, 310, 60]
    q, kn, kp, v, cu_q, cu_k = prefill_inputs(gen(48 + heads), heads, lq, lk, torch.float32)
    o, lse = kda.latent_prefill(q, kn, kp, v, SCALE, cu_q, cu_k, causal=causal)
    ref.check(o, lse, ref.prefill(q, kn, kp, v, SCALE, lq, lk, causal), "shared tiles")


# few queries behind many keys: the keys of a query tile are shared by several pairs of CTAs
SPLIT = [
    ("one_query", 1, [1], [1100]), ("chunk", 2, [300], [2000]), ("two_tiles", 3, [700], [1500]),
    ("ragged", 2, [1, 600, 0, 40], [1500, 3001, 900, 5]), ("no_keys", 2, [9, 70, 3], [0, 6000, 2]),
    ("fewer_keys", 2, [2100], [1700]), ("half_as_many", 20, [40], [1300]), ("thirty", 30, [513], [1409]),
    ("all_in_one_tile", 1, [64, 64], [2100, 60]), ("ragged_two", 4, [1, 600, 0, 40], [1500, 3001, 900, 5]),
    ("two_by_two", 17, [513], [1409]),
]


@pytest.mark.parametrize("causal", [True, False], ids=["causal", "full"])
@pytest.mark.parametrize("name,heads,lq,lk", SPLIT, ids=[c[0] for c in SPLIT])
def test_prefill_shared_keys(causal, name, heads, lq, lk):
    q, kn, kp, v, cu_q, cu_k = prefill_inputs(gen(60 + heads), heads, lq, lk, torch.bfloat16)
    err = errors()
    o, lse = kda.latent_prefill(q, kn, kp, v, SCALE, cu_q, cu_k, causal=causal, errors=err)
    ref.check(o, lse, ref.prefill(q, kn, kp, v, SCALE, lq, lk, causal), name)
    assert err.item() == 0
    for _ in range(3):
        again, lse2 = kda.latent_prefill(q, kn, kp, v, SCALE, cu_q, cu_k, causal=causal)
        assert torch.equal(o.view(torch.int16), again.view(torch.int16)) and torch.equal(lse, lse2)


def test_prefill_shared_keys_next_to_nan():
    """Sequences of NaN and infinity on both sides: the shares of the one between them see none of it."""
    lq, lk = [50, 91, 70], [1000, 1301, 1200]
    q, kn, kp, v, cu_q, cu_k = prefill_inputs(gen(59), 2, lq, lk, torch.bfloat16)
    qs, ks = slice(50, 141), slice(1000, 2301)
    want = ref.prefill(q[qs], kn[ks], kp[ks], v[ks], SCALE, [91], [1301], True)
    for t, at in ((q, qs), (kn, ks), (kp, ks), (v, ks)):
        t[:at.start], t[at.stop:] = math.nan, math.inf
    o, lse = kda.latent_prefill(q, kn, kp, v, SCALE, cu_q, cu_k)
    ref.check(o[qs], lse[qs], want, "between")


@pytest.mark.parametrize("name,heads,lq,lk", [
    ("shared_keys", 2, [200], [2000]), ("one_at_a_time", 40, [200], [900]),
    ("side_by_side", 12, [250, 100, 30, 256, 180, 1, 220, 90], [300, 1500, 30, 900, 181, 700, 1300, 89]),
    ("second_tile", 40, [512], [700]),
], ids=lambda x: x if isinstance(x, str) else "")
@pytest.mark.parametrize("causal", [True, False], ids=["causal", "full"])
def test_prefill_rising_scores_of_a_tile_alone(causal, name, heads, lq, lk):
    """Scores that rise along the keys, so that the maximum is moved again and again while a query tile's
    next scores are computed ahead."""
    q, kn, kp, v, cu_q, cu_k = prefill_inputs(gen(70), heads, lq, lk, torch.bfloat16)
    q[:, :, 0] = 5.0
    kn[:, :, 0] = torch.cat([torch.linspace(-40, 40, n, device="cuda") for n in lk]).to(torch.bfloat16)[:, None]
    err = errors()
    o, lse = kda.latent_prefill(q, kn, kp, v, SCALE, cu_q, cu_k, causal=causal, errors=err)
    ref.check(o, lse, ref.prefill(q, kn, kp, v, SCALE, lq, lk, causal), name)
    assert err.item() == 0


def test_prefill_output_aligned_to_16_bytes_only():
    g = gen(48)
    q, kn, kp, v, cu, _ = prefill_inputs(g, 3, [300], [300], torch.bfloat16)
    o = torch.empty(300 * 3 * 128 + 8, dtype=torch.bfloat16, device="cuda")[8:].view(300, 3, 128)
    assert o.data_ptr() % 32 == 16
    o, lse = kda.latent_prefill(q, kn, kp, v, SCALE, o=o)
    ref.check(o, lse, ref.prefill(q, kn, kp, v, SCALE, [300], [300], True), "unaligned output")


def test_prefill_on_another_stream_and_in_a_graph():
    g = gen(44)
    q, kn, kp, v, cu, _ = prefill_inputs(g, 4, [200, 100], [200, 100], torch.bfloat16)
    want = ref.prefill(q, kn, kp, v, SCALE, [200, 100], [200, 100], True)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    o, lse = kda.latent_prefill(q, kn, kp, v, SCALE, cu, stream=side)
    side.synchronize()
    ref.check(o, lse, want, "side stream")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        kda.latent_prefill(q, kn, kp, v, SCALE, cu, o=o, lse=lse)
    o.zero_()
    lse.zero_()
    graph.replay()
    torch.cuda.synchronize()
    ref.check(o, lse, want, "graph")


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("scale", [0.0, -0.07, 1e-3, 1.5])
def test_other_scales(dtype, scale):
    """A scale of 0 (the mean of the seen values), a negative one, a tiny and a large one."""
    g = gen(45)
    dt = DT[dtype]
    q, kn, kp, v, cu, _ = prefill_inputs(g, 2, [130, 31], [130, 31], dt, kscale=0.3)
    ref.check(*kda.latent_prefill(q, kn, kp, v, scale, cu), ref.prefill(q, kn, kp, v, scale, [130, 31], [130, 31], True),
              "prefill")
    cache, table = paged(g, [130, 31], 16, dt, scale=0.3)
    qd = normal(g, 2, 16, 576, dtype=dt)
    o, lse = kda.latent_decode(qd, cache, table, torch.tensor([130, 31], dtype=torch.int32, device="cuda"), scale)
    ref.check(o, lse, ref.decode(qd, cache, table, [130, 31], scale), "decode")


# ------------------------------------------------------------------ together
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_the_two_forms_agree(dtype):
    """The absorbed decode over the cache that the append wrote gives the expanded prefill's last
    row: q' = W_k^T q against the latent, W_v applied after.  In float64 both forms are the same;
    here the absorbed query, the latent and both outputs are rounded to the type: the bound is 8 u of
    the output's largest value (a weight moves by 2 u of its score, |score| < 2 here, and there are
    four roundings)."""
    dt = DT[dtype]
    g = gen(50)
    T, H, page = 77, 4, 16
    joint, q = normal(g, T, 576, dtype=dt), normal(g, T, H, 192, dtype=dt, scale=0.5)
    wk, wv = (normal(g, H, 128, 512, dtype=dt, scale=512 ** -0.5) for _ in range(2))
    cs, pos = table_of(T), torch.arange(T, device="cuda", dtype=torch.int32)
    cache = torch.zeros(-(-T // page), page, 576, dtype=dt, device="cuda")
    lat, kpe = torch.empty(T, 512, dtype=dt, device="cuda"), torch.empty(T, 64, dtype=dt, device="cuda")
    kda.latent_append(joint[:, :512], joint[:, 512:], cache, pos, norm_weight=torch.ones(512, dtype=dt, device="cuda"),
                      cos_sin=cs, positions=pos, q_pe=q[..., 128:], latent_out=lat, k_pe_out=kpe)
    up = lambda w: torch.einsum("tr,hnr->thn", lat.double(), w.double()).to(dt)
    o, _ = kda.latent_prefill(q, up(wk), kpe, up(wv), SCALE)
    qa = torch.empty(1, H, 576, dtype=dt, device="cuda")
    qa[0, :, :512] = torch.einsum("hn,hnr->hr", q[-1, :, :128].double(), wk.double()).to(dt)
    qa[0, :, 512:] = q[-1, :, 128:]
    table = torch.arange(cache.shape[0], dtype=torch.int32, device="cuda")[None]
    ol, _ = kda.latent_decode(qa, cache, table, torch.tensor([T], dtype=torch.int32, device="cuda"), SCALE)
    absorbed = torch.einsum("hr,hnr->hn", ol[0].double(), wv.double())
    u = ref.U[dt] if dtype == "bf16" else ref.U32 * 64
    assert (absorbed - o[-1].double()).abs().max() <= 8 * u * o[-1].double().abs().max()


@pytest.mark.parametrize("dtype,bound", [("bf16", 0.05), ("f32", 1e-4)])
def test_hybrid_example(dtype, bound):
    """The example's block: KDA and latent attention from packed prompts to generated tokens.  The two
    forms of the latent layer differ by the roundings of four matrix products and of the latent path
    between them: up to a dozen roundings of 2^-8 (bf16) of values no larger than the largest output."""
    import os
    import sys
    sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))
    import hybrid_block
    assert hybrid_block.run(dtype=DT[dtype]) <= bound
