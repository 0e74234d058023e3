"""Latent attention on the paths that the header promises and the other tests leave out: queries shared by a
batch, no log-sum-exp asked for, a cache without pages, a page table without columns, bad pages inside a
tile; and long caches whose outputs show every tile."""
import math

import pytest
import torch

import latent_reference as ref
from kda_gated_delta_04_gb300 import kda
from test_gpu_latent import DT, SCALE, errors, gen, normal, paged, prefill_inputs

pytestmark = pytest.mark.gpu
PAGE_ERROR = 64  # KDA_DEVICE_ERR_PAGE


def ints(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("heads", [1, 5, 16, 33, 100])
def test_decode_with_the_queries_shared_by_the_batch(dtype, heads):
    """A batch stride of 0: one set of queries for all sequences."""
    g = gen(80 + heads)
    lens = [130, 0, 64, 300, 1]
    cache, table = paged(g, lens, 16, DT[dtype])
    q = normal(g, 1, heads, 576, dtype=DT[dtype]).expand(5, -1, -1)
    err = errors()
    o, lse = kda.latent_decode(q, cache, table, ints(lens), SCALE, errors=err)
    ref.check(o, lse, ref.decode(q, cache, table, lens, SCALE), "shared queries")
    assert err.item() == 0


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("name,heads,lens", [("whole", 16, [64, 1, 0, 30]), ("split_by_unit", 32, [20001, 7000]),
                                             ("split_by_boundary", 8, [500 + 7 * i for i in range(400)])],
                         ids=lambda x: x if isinstance(x, str) else "")
def test_decode_without_lse(dtype, name, heads, lens):
    """lse NULL: the same outputs, bit for bit."""
    g = gen(81)
    dt, B = DT[dtype], len(lens)
    cache, table = paged(g, lens, 64, dt)
    q, ln = normal(g, B, heads, 576, dtype=dt), ints(lens)
    want, _ = kda.latent_decode(q, cache, table, ln, SCALE)
    o = torch.full_like(want, 3.0)
    code = kda.KDA_DTYPE_BF16 if dt == torch.bfloat16 else kda.KDA_DTYPE_F32
    ws = kda.latent_decode_workspace_for(heads, code, "cuda")
    st = kda.kda_latent_decode(q.data_ptr(), q.stride(0), q.stride(1), cache.data_ptr(), cache.shape[0], 64,
                               table.data_ptr(), table.stride(0), table.shape[1], ln.data_ptr(), B, heads, 512, 64, code,
                               SCALE, o.data_ptr(), None, ws.data_ptr(), ws.numel(), None,
                               torch.cuda.current_stream().cuda_stream)
    assert st == kda.KDA_OK
    assert torch.equal(o, want)


@pytest.mark.parametrize("dtype,name,heads,lq,lk", [
    ("bf16", "one_pair", 40, [300, 5], [300, 5]), ("bf16", "four_pairs", 2, [300], [2000]),
    ("bf16", "two_pairs", 20, [40], [1300]), ("bf16", "no_keys", 2, [70], [0]),
    ("f32", "one", 12, [300, 200, 300], [310, 200, 300]), ("f32", "two", 12, [300, 200], [310, 200]),
    ("f32", "four", 2, [300], [700]), ("f32", "no_keys", 2, [70], [0]),
], ids=lambda x: x if isinstance(x, str) else "")
def test_prefill_without_lse(dtype, name, heads, lq, lk):
    dt = DT[dtype]
    q, kn, kp, v, cu_q, cu_k = prefill_inputs(gen(82), heads, lq, lk, dt)
    want, _ = kda.latent_prefill(q, kn, kp, v, SCALE, cu_q, cu_k)
    o = torch.full_like(want, 3.0)
    st = kda.kda_latent_prefill(q.data_ptr(), q.stride(0), q.stride(1), kn.data_ptr(), kn.stride(0), kn.stride(1),
                                kp.data_ptr(), kp.stride(0), v.data_ptr(), v.stride(0), v.stride(1), cu_q.data_ptr(),
                                cu_k.data_ptr(), len(lq), sum(lq), sum(lk), heads, 128, 64, 128,
                                kda.KDA_DTYPE_BF16 if dt == torch.bfloat16 else kda.KDA_DTYPE_F32, SCALE, o.data_ptr(), None,
                                None, torch.cuda.current_stream().cuda_stream, 0)
    assert st == kda.KDA_OK
    assert torch.equal(o, want)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_decode_of_a_cache_without_pages(dtype):
    """Every page is out of range: zero rows, whose mean is 0 and whose log-sum-exp is log(len), within the
    rounding of a logarithm (2 units of 2^-24 of it) and of its conversion from base 2."""
    dt = DT[dtype]
    cache = torch.empty(0, 64, 576, dtype=dt, device="cuda")
    lens = [1, 0, 200, 128]
    q = normal(gen(83), 4, 16, 576, dtype=dt)
    err = errors()
    o, lse = kda.latent_decode(q, cache, ints([[0, 1, 2, 3]] * 4), ints(lens), SCALE, errors=err)
    assert err.item() == PAGE_ERROR
    assert not o.any()
    want = torch.tensor([math.log(n) if n else -math.inf for n in lens], dtype=torch.float64, device="cuda")[:, None]
    empty = want.expand_as(lse) == -math.inf
    assert torch.equal(lse == -math.inf, empty)
    assert ((lse.double() - want).abs()[~empty] <= 4 * ref.U32 * math.log(200)).all()



@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_decode_with_a_table_without_columns(dtype):
    """Nothing can be held: sequences of length 0, and longer ones are held to that and reported."""
    dt = DT[dtype]
    cache = normal(gen(84), 2, 64, 576, dtype=dt)
    table = torch.empty(3, 0, dtype=torch.int32, device="cuda")
    q = normal(gen(85), 3, 20, 576, dtype=dt)
    for lens, want in (([0, 0, 0], 0), ([0, 5, 1], 1)):
        err = errors()
        o, lse = kda.latent_decode(q, cache, table, ints(lens), SCALE, o=torch.full((3, 20, 512), 3.0, dtype=dt, device="cuda"),
                                   errors=err)
        assert err.item() == want
        assert not o.any() and (lse == -math.inf).all()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("page", [8, 16, 48])
def test_decode_with_bad_pages_inside_a_tile(dtype, page):
    """Pages below 0 and past the cache among good ones, several to a tile: their rows are zero rows."""
    g = gen(86)
    dt, lens = DT[dtype], [200, 333, 64]
    cache, table = paged(g, lens, page, dt)
    bad = table.clone()
    bad[0, 1], bad[0, 3], bad[1, 4], bad[2, 0] = -1, cache.shape[0], 2 ** 30, -(2 ** 31)
    q = normal(g, 3, 16, 576, dtype=dt)
    err = errors()
    o, lse = kda.latent_decode(q, cache, bad, ints(lens), SCALE, errors=err)
    assert err.item() == PAGE_ERROR
    zero = torch.cat([cache, torch.zeros_like(cache[:1])])
    held = torch.where((bad >= 0) & (bad < cache.shape[0]), bad, cache.shape[0])
    ref.check(o, lse, ref.decode(q, zero, held, lens, SCALE), "bad pages")


# Rows of a tile are 1 in a channel of the tile's own and 0 elsewhere: an output channel is the weight of a
# few tiles, so that a tile left out, taken twice or exchanged changes it by a quarter and more, where the
# bound (|o| = sum p |v|) allows a hundredth in bf16.
@pytest.mark.parametrize("dtype,heads,lens,page", [
    ("bf16", 32, [131072, 120001], 64), ("bf16", 16, [100003], 16), ("bf16", 128, [60001, 33000], 128),
    ("bf16", 8, [9000 + 64 * i for i in range(24)], 8), ("f32", 8, [99999, 5], 64)])
def test_decode_of_a_long_cache_tile_by_tile(dtype, heads, lens, page):
    """fp32: below 1e5 rows, for which the bound is derived.  bf16: a row's share of the sum goes through at
    most 27 tiles, 6 steps of a reduction and 152 parts, which the bound's 200 steps cover."""
    g = gen(87)
    dt = DT[dtype]
    cache, table = paged(g, lens, page, dt)
    at = torch.arange(max(lens), device="cuda")
    rows = cache.view(-1, 576)
    for b, n in enumerate(lens):
        j = at[:n]
        row = table[b].long()[j // page] * page + j % page
        rows[row, :512] = torch.nn.functional.one_hot((j // 64) % 512, 512).to(dt)
    q = normal(g, len(lens), heads, 576, dtype=dt)
    err = errors()
    o, lse = kda.latent_decode(q, cache, table, ints(lens), SCALE, errors=err)
    for b, n in enumerate(lens):  # (one at a time: the reference's rows are 8 bytes a channel)
        ref.check(o[b:b + 1], lse[b:b + 1], ref.decode(q[b:b + 1], cache, table[b:b + 1], [n], SCALE), f"{n} rows")
    assert err.item() == 0


@pytest.mark.parametrize("dtype,heads,lq,lk", [
    ("bf16", 4, 600, 15600), ("bf16", 12, 600, 15600), ("bf16", 40, 600, 15600), ("bf16", 40, 200, 16001),
    ("bf16", 20, 4096, 4096), ("f32", 2, 70, 15600), ("f32", 3, 4096, 4096)])
def test_prefill_of_many_keys_tile_by_tile(dtype, heads, lq, lk):
    dt = DT[dtype]
    q, kn, kp, v, _, _ = prefill_inputs(gen(88), heads, [lq], [lk], dt)
    wide = 128 if dtype == "bf16" else 64  # a key tile
    v[:] = torch.nn.functional.one_hot((torch.arange(lk, device="cuda") // wide) % 128, 128).to(dt)[:, None]
    err = errors()
    o, lse = kda.latent_prefill(q, kn, kp, v, SCALE, ints([0, lq]), ints([0, lk]), errors=err)
    for h in range(heads):
        one = slice(h, h + 1)
        want = ref.prefill(q[:, one], kn[:, one], kp, v[:, one], SCALE, [lq], [lk], True)
        ref.check(o[:, one], lse[:, one], want, f"{lk} keys, head {h}")
    assert err.item() == 0
