"""The projections, the short convolution and the selective scan on the GPU against their definitions in float64
(layer_reference.py derives the bounds), at the sizes, strides and contents where such kernels go wrong."""
import math

import pytest
import torch

import layer_reference as ref
from kda_gated_delta_04_gb300 import kda

pytestmark = pytest.mark.gpu
DT = {"bf16": torch.bfloat16, "f32": torch.float32}


def gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def normal(g, *shape, dtype=torch.bfloat16, scale=1.0):
    return (torch.randn(*shape, generator=g, device="cuda") * scale).to(dtype)


def errors():
    return torch.zeros(1, dtype=torch.int32, device="cuda")


def ints(*x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def offsets(lens):
    return ints(*[sum(lens[:i]) for i in range(len(lens) + 1)])


# ------------------------------------------------------------------ linear
SHAPES = [(1, 1, 1), (1, 8, 8), (1, 4096, 128), (3, 33, 72), (5, 1000, 264), (16, 128, 64), (17, 129, 1024), (64, 64, 64),
          (100, 32, 512), (128, 256, 128), (129, 257, 200), (255, 511, 136), (256, 4096, 256), (300, 4104, 96),
          (513, 1, 640), (300, 72, 64), (700, 100, 256), (1000, 128, 512), (5000, 96, 72), (1000, 40, 2048), (40, 4096, 512),
          (33, 100, 64), (128, 5000, 256), (12, 9000, 64), (4200, 4300, 192), (9000, 3900, 72), (1024, 1024, 1024), (2049, 384, 64), (2500, 777, 320)]


@pytest.mark.parametrize("dtype,out", [("bf16", "bf16"), ("bf16", "f32"), ("f32", "f32")])
@pytest.mark.parametrize("m,n,k", SHAPES)
def test_linear(m, n, k, dtype, out):
    dt, odt = DT[dtype], DT[out]
    g = gen(m * 31 + n * 7 + k)
    x, w = normal(g, m, k, dtype=dt), normal(g, n, k, dtype=dt, scale=k ** -0.5)
    bias, r = normal(g, n, dtype=dt), normal(g, m, n, dtype=odt)
    tc = dtype == "bf16" and k % 8 == 0
    for act, b, res in [(None, None, None), ("silu", bias, None), ("gelu", bias, r), ("sigmoid", None, r), ("softplus", bias, None)]:
        y = kda.linear(x, w, b, activation=act, residual=res, out_dtype=odt)
        ref.check(y, *ref.linear(x, w, b, act, res, odt, tc), f"{m}x{n}x{k} {act}")


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("m", [2, 40, 300])
def test_linear_strides_and_alignment(m, dtype):
    """Rows that are parts of wider ones, on any alignment and of any width; what lies around the output's rows stays."""
    dt = DT[dtype]
    g = gen(m)
    for k, xo, wo, yo, n in [(64, 8, 16, 8, 72), (64, 1, 0, 3, 65), (65, 0, 7, 1, 72), (128, 0, 1, 0, 33), (72, 4, 4, 4, 130)]:
        xs, ws = normal(g, m, k + 24, dtype=dt), normal(g, n, k + 16, dtype=dt, scale=k ** -0.5)
        ys = torch.full((m, n + 13), 7.0, dtype=dt, device="cuda")
        rs = normal(g, m, n + 5, dtype=dt)
        x, w, y, r = xs[:, xo:xo + k], ws[:, wo:wo + k], ys[:, yo:yo + n], rs[:, 1:1 + n]
        bias = normal(g, n + 1, dtype=dt)[1:]
        kda.linear(x, w, bias, activation="silu", residual=r, out=y)
        ref.check(y, *ref.linear(x, w, bias, "silu", r, dt, dtype == "bf16"), f"{m} {k} {xo} {wo} {yo} {n}")
        assert (ys[:, :yo] == 7).all() and (ys[:, yo + n:] == 7).all()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_linear_shared_rows_and_in_place(dtype):
    """One input row for all (a stride of 0), rows that overlap; a residual that the output replaces."""
    dt = DT[dtype]
    g = gen(3)
    w = normal(g, 96, 64, dtype=dt, scale=0.1)
    one = normal(g, 1, 64, dtype=dt).expand(50, 64)
    ref.check(kda.linear(one, w), *ref.linear(one, w, None, None, None, dt, True), "one row")
    over = normal(g, 8 * 50 + 64, dtype=dt).as_strided((50, 64), (8, 1))
    ref.check(kda.linear(over, w), *ref.linear(over, w, None, None, None, dt, True), "overlapping rows")
    for m in (3, 50, 700):
        x, r = normal(g, m, 64, dtype=dt), normal(g, m, 96, dtype=dt)
        want = kda.linear(x, w, activation="gelu", residual=r.clone())
        got = kda.linear(x, w, activation="gelu", residual=r, out=r)
        assert got is r and torch.equal(r, want)


@pytest.mark.parametrize("m", [1, 33, 520])
def test_linear_special_values(m):
    """Infinities and NaN stay in the rows and columns that they stand in; nothing past a row's end is read into it."""
    g = gen(m)
    for dtype in ("bf16", "f32"):
        dt = DT[dtype]
        xs, ws = normal(g, m + 1, 72, dtype=dt), normal(g, 48, 72, dtype=dt)
        xs[:, 64:] = math.nan  # beside the rows
        xs[m:] = math.nan      # behind them
        ws[:, 64:] = math.inf
        x, w = xs[:m, :64], ws[:47, :64]
        x[0, 3] = math.inf
        w[5, 7] = math.nan
        w[6] = 0
        y = kda.linear(x, w)
        want = x.to(torch.float64) @ w.to(torch.float64).T
        assert torch.equal(y.isnan(), want.isnan()) and torch.equal(y.isinf(), want.isinf())
        fine = want.isfinite()
        assert ((y.double() - want).abs()[fine] <= 2.0 ** -8 * want.abs()[fine] + 1e-3).all()


def test_linear_nothing_to_do():
    x, w = torch.zeros(0, 16, device="cuda"), torch.zeros(8, 16, device="cuda")
    assert kda.linear(x, w).shape == (0, 8)
    assert kda.linear(w, torch.zeros(0, 16, device="cuda")).shape == (8, 0)


# ------------------------------------------------------------------ short convolution
LENS = [[1], [2], [5], [0], [64], [1, 1, 1], [0, 3, 0, 0, 1], [2, 0, 7, 16, 17, 1, 0], [15, 16, 33, 3, 100], [300, 1, 2, 0, 257]]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("width", [2, 3, 4])
@pytest.mark.parametrize("lens", LENS, ids=str)
def test_short_conv(lens, width, dtype):
    dt = DT[dtype]
    g = gen(sum(lens) + width)
    T = sum(lens)
    for channels, parts, act, has_bias, has_state, pad in [(8, 1, "silu", True, True, 0), (48, 3, None, False, True, 3),
                                                         (1040, 1, "silu", False, False, 20), (1048, 1, None, True, True, 0)]:
        wide = normal(g, T + pad, channels + 16, dtype=dt)
        x = wide[:, 8:8 + channels]
        w = normal(g, channels, width, dtype=dt)
        bias = normal(g, channels, dtype=dt) if has_bias else None
        state = normal(g, len(lens), width - 1, channels, dtype=dt) if has_state else None
        y = torch.full((parts, T + pad, channels // parts) if parts > 1 else (T + pad, channels), 7.0, dtype=dt, device="cuda")
        err = errors()
        out, new = kda.short_conv(x, w, bias, offsets(lens), state, activation=act, parts=parts, out=y, errors=err)
        assert out is y and err.item() == 0
        want, e, wn = ref.conv(x[:T], w, bias, lens, state, act, parts)
        ref.check(y[..., :T, :], want, e, f"{lens} {channels}")
        assert torch.equal(new, wn)
        assert (y[..., T:, :] == 7).all()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("batch,channels,parts", [(1, 8, 1), (3, 48, 3), (64, 1032, 1), (257, 96, 3)])
def test_short_conv_step(batch, channels, parts, dtype):
    """One token of every sequence, the states in a pool; in place and elsewhere; entries of others stay."""
    dt = DT[dtype]
    g = gen(batch)
    x, w, bias = normal(g, batch, channels, dtype=dt), normal(g, channels, 4, dtype=dt), normal(g, channels, dtype=dt)
    pool = normal(g, batch + 5, 3, channels, dtype=dt)
    slots = torch.randperm(batch + 5, generator=g, device="cuda")[:batch].int()
    want, e, wn = ref.conv(x, w, bias, [1] * batch, pool[slots.long()], "silu", parts)
    other = torch.full_like(pool, 7.0)
    y = kda.short_conv_step(x, w, pool, bias, slots=slots, new_state=other, parts=parts)
    ref.check(y, want, e, f"step {batch}")
    assert torch.equal(other[slots.long()], wn)
    rest = torch.ones(batch + 5, dtype=torch.bool, device="cuda")
    rest[slots.long()] = False
    assert (other[rest] == 7).all()
    before = pool.clone()
    assert torch.equal(kda.short_conv_step(x, w, pool, bias, slots=slots, parts=parts), y)
    assert torch.equal(pool[slots.long()], wn) and torch.equal(pool[rest], before[rest])
    dense = before[slots.long()]
    assert torch.equal(kda.short_conv_step(x, w, dense, bias, parts=parts), y) and torch.equal(dense, wn)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_short_conv_in_pieces(dtype):
    """A prompt in pieces of any lengths, the state in place between them, is the prompt in one: the same bits."""
    dt = DT[dtype]
    g = gen(8)
    x, w = normal(g, 200, 64, dtype=dt), normal(g, 64, 4, dtype=dt)
    whole, end = kda.short_conv(x, w)
    state = torch.zeros(1, 3, 64, dtype=dt, device="cuda")
    out, at = [], 0
    for n in (1, 1, 2, 0, 3, 5, 18, 70, 100):
        out.append(kda.short_conv(x[at:at + n], w, None, ints(0, n), state, final_state=state)[0])
        at += n
    assert at == 200 and torch.equal(torch.cat(out), whole) and torch.equal(state, end)


def test_equal_sequences_and_slots():
    """No offsets: sequences of one length (through the C entry point); an entry of -1 starts from zero or is not kept;
    an entry out of range is reported, starts from zero and is not kept, and the others run."""
    g = gen(9)
    x, w = normal(g, 24, 16), normal(g, 16, 4)
    a, _ = kda.short_conv(x, w, None, ints(0, 6, 12, 18, 24))
    b = torch.empty_like(x)
    st = kda.kda_short_conv(x.data_ptr(), 16, w.data_ptr(), None, 4, None, 4, 24, 16, 1, 0, kda.KDA_ACT_SILU, None, None, 0,
                            None, None, 0, b.data_ptr(), 0, 16, None, torch.cuda.current_stream().cuda_stream)
    assert st == 0 and torch.equal(a, b)
    pool = normal(g, 3, 3, 16)
    keep = pool.clone()
    for bad, code in [(-1, 0), (3, 16), (-2, 16)]:
        pool.copy_(keep)
        err = errors()
        y, _ = kda.short_conv(x, w, None, ints(0, 6, 12, 18, 24), pool, init_slots=ints(2, bad, 0, 1), final_state=pool,
                              final_slots=ints(2, bad, 0, 1), errors=err)
        assert err.item() == code
        want = [2, None, 0, 1]
        state = torch.stack([torch.zeros_like(keep[0]) if i is None else keep[i] for i in want])
        wy, e, wn = ref.conv(x, w, None, [6] * 4, state, "silu")
        ref.check(y, wy, e, "slots")
        assert torch.equal(pool[2], wn[0]) and torch.equal(pool[0], wn[2]) and torch.equal(pool[1], wn[3])


def test_malformed_offsets_are_reported():
    """They stay in the buffers (shown on the CPU by the clamp in packed_range); later calls run."""
    g = gen(10)
    x, w = normal(g, 32, 16), normal(g, 16, 4)
    s = scan_inputs(g, 32, 16, 8, torch.bfloat16)
    for cu in (ints(0, 40), ints(3, 32), ints(0, 20, 10, 32), ints(-5, 32), ints(0, 2 ** 31 - 1, 32)):
        err = errors()
        y = torch.full((40, 16), 7.0, dtype=torch.bfloat16, device="cuda")
        kda.short_conv(x, w, None, cu, out=y[:32], errors=err)
        assert err.item() == 1 and (y[32:] == 7).all()
        err.zero_()
        kda.selective_scan(**s, cu_seqlens=cu, out=y[:32], errors=err)
        assert err.item() == 1 and (y[32:] == 7).all()


# ------------------------------------------------------------------ selective scan
def scan_inputs(g, T, ch, n, dt, groups=None):
    bc = normal(g, T, 2 * (groups or 1) * n + 8, dtype=dt)
    m = (groups or 1) * n
    B, C = bc[:, :m], bc[:, m:2 * m]
    if groups:
        B, C = B.unflatten(1, (groups, n)), C.unflatten(1, (groups, n))
    wide = normal(g, T, 3 * ch + 8, dtype=dt)
    step = torch.exp(torch.rand(ch, generator=g, device="cuda") * 5 - 6)
    return dict(x=wide[:, :ch], dt=wide[:, ch:2 * ch], z=wide[:, 2 * ch:3 * ch], B=B, C=C,
                A=-torch.exp(normal(g, ch, n, dtype=torch.float32)) * 3, D=normal(g, ch, dtype=torch.float32),
                dt_bias=step + torch.log(-torch.expm1(-step)))


def grouped(t):
    return t if t.dim() == 3 else t[:, None]


def reference(s, lens, state, sp=True):
    return ref.scan(s["x"], s["dt"], s["A"], grouped(s["B"]), grouped(s["C"]), s["D"], s["z"], s["dt_bias"], lens, state, sp)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("n", [8, 16, 32, 64])
@pytest.mark.parametrize("lens", LENS + [[31, 32, 33, 65]], ids=str)
def test_scan(lens, n, dtype):
    dt = DT[dtype]
    g = gen(sum(lens) + n)
    T = sum(lens)
    for channels, groups, has, sp, pad in [(8, None, True, True, 0), (72, None, False, True, 5), (48, 2, True, False, 0),
                                          (136, 1, True, True, 0)]:
        s = scan_inputs(g, T + pad, channels, n, dt, groups)
        if not has:
            s["z"] = s["D"] = s["dt_bias"] = None
        if not sp:
            s["dt"] = s["dt"].abs()
        state = normal(g, len(lens), channels, n, dtype=torch.float32) if has else None
        y = torch.full((T + pad, channels + 8), 7.0, dtype=dt, device="cuda")
        err = errors()
        out, new = kda.selective_scan(**s, cu_seqlens=offsets(lens), init_state=state, softplus=sp, out=y[:, :channels], errors=err)
        assert err.item() == 0
        cut = {k: v[:T] if v is not None and k in ("x", "dt", "z", "B", "C") else v for k, v in s.items()}
        wy, e, wn, ne = reference(cut, lens, state, sp)
        ref.check(y[:T, :channels], wy, e, f"{lens} {channels}")
        ref.check(new, wn, ne, f"{lens} {channels} state")
        assert (y[T:] == 7).all() and (y[:, channels:] == 7).all()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("n", [8, 16, 32, 64])
@pytest.mark.parametrize("batch,channels,groups", [(1, 8, None), (3, 72, 3), (5, 1032, None), (130, 40, None)])
def test_scan_step(batch, channels, groups, n, dtype):
    dt = DT[dtype]
    g = gen(batch + n)
    s = scan_inputs(g, batch, channels, n, dt, groups)
    pool = normal(g, batch + 3, channels, n, dtype=torch.float32)
    slots = torch.randperm(batch + 3, generator=g, device="cuda")[:batch].int()
    wy, e, wn, ne = reference(s, [1] * batch, pool[slots.long()])
    other = torch.full_like(pool, 7.0)
    y = kda.selective_scan_step(**s, state=pool, slots=slots, new_state=other)
    ref.check(y, wy, e, f"step {batch}")
    ref.check(other[slots.long()], wn, ne, f"step {batch} state")
    rest = torch.ones(batch + 3, dtype=torch.bool, device="cuda")
    rest[slots.long()] = False
    assert (other[rest] == 7).all()
    before = pool.clone()
    assert torch.equal(kda.selective_scan_step(**s, state=pool, slots=slots), y)
    assert torch.equal(pool[slots.long()], other[slots.long()]) and torch.equal(pool[rest], before[rest])
    dense = before[slots.long()]
    assert torch.equal(kda.selective_scan_step(**s, state=dense), y)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("n,channels,lens", [
    (8, 24, [700]), (8, 200, [900, 3, 0, 640]), (16, 8, [1100]), (16, 64, [520]), (16, 136, [1000, 1, 0, 1010]), (16, 264, [2000]),
    (32, 16, [700]), (32, 72, [650, 0, 900]), (64, 8, [800]), (64, 40, [513, 600])], ids=str)
def test_scan_in_parts(n, channels, lens, dtype):
    """Few channels and long sequences, of which several CTAs have a part each (parts without tokens among them); states
    in place, a sequence that starts from zero, another that is not kept; the same bits again."""
    dt = DT[dtype]
    g = gen(sum(lens) + channels)
    s = scan_inputs(g, sum(lens) + 7, channels, n, dt)
    s["A"] = s["A"] * torch.where(torch.arange(channels, device="cuda")[:, None] % 3 == 0, 0.01, 1.0)  # long memories too
    first = normal(g, len(lens) + 1, channels, n, dtype=torch.float32)
    at = torch.arange(len(lens), dtype=torch.int32, device="cuda")
    start, keep = at.clone(), at.clone()
    if len(lens) > 1:
        start[-1], keep[0] = -1, -1
    state = torch.stack([first[i] if i >= 0 else torch.zeros_like(first[0]) for i in start.tolist()])
    cut = {k: v[:sum(lens)] if v is not None and k in ("x", "dt", "z", "B", "C") else v for k, v in s.items()}
    wy, e, wn, ne = reference(cut, lens, state)
    results = []
    for _ in range(2):
        pool, err = first.clone(), errors()
        y = torch.full((sum(lens) + 7, channels), 7.0, dtype=dt, device="cuda")
        kda.selective_scan(**s, cu_seqlens=offsets(lens), init_state=pool, init_slots=start, final_state=pool, final_slots=keep,
                           out=y, errors=err)
        assert err.item() == 0 and (y[sum(lens):] == 7).all() and torch.equal(pool[-1], first[-1])
        ref.check(y[:sum(lens)], wy, e, f"{lens} {channels}")
        for i, k in enumerate(keep.tolist()):
            if k >= 0:
                ref.check(pool[k], wn[i], ne[i], f"{lens} {channels} state {i}")
            else:
                assert torch.equal(pool[i], first[i])
        results.append((y, pool))
    assert all(torch.equal(a, b) for a, b in zip(*results))


def test_scan_slots():
    """-1: from zero, not kept; out of range: reported, from zero, not kept."""
    g = gen(12)
    s = scan_inputs(g, 40, 24, 16, torch.float32)
    pool = normal(g, 3, 24, 16, dtype=torch.float32)
    keep = pool.clone()
    for bad, code in [(-1, 0), (3, 16), (-2, 16)]:
        for lens in ([10] * 4, [1] * 4):
            pool.copy_(keep)
            T = sum(lens)
            cut = {k: v[:T] if k in ("x", "dt", "z", "B", "C") else v for k, v in s.items()}
            err, at = errors(), ints(2, bad, 0, 1)
            if T == 4:
                y = kda.selective_scan_step(**cut, state=pool, slots=at, errors=err)
            else:
                y, _ = kda.selective_scan(**cut, cu_seqlens=offsets(lens), init_state=pool, init_slots=at, final_state=pool,
                                          final_slots=at, errors=err)
            assert err.item() == code
            state = torch.stack([torch.zeros_like(keep[0]) if i is None else keep[i] for i in (2, None, 0, 1)])
            wy, e, wn, ne = reference(cut, lens, state)
            ref.check(y, wy, e, "slots")
            ref.check(pool[ints(2, 0, 1).long()], wn[[0, 2, 3]], ne[[0, 2, 3]], "slots state")


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_scan_in_pieces(dtype):
    """A prompt in pieces of any lengths, prefills and steps, the state in place between them."""
    dt = DT[dtype]
    g = gen(13)
    s = scan_inputs(g, 230, 40, 16, dt)
    wy, e, wn, ne = reference(s, [230], None)
    state = torch.zeros(1, 40, 16, device="cuda")
    out, at = [], 0
    for n in (1, 30, 1, 2, 0, 32, 64, 100):
        cut = {k: v[at:at + n] if k in ("x", "dt", "z", "B", "C") else v for k, v in s.items()}
        if n == 1:
            out.append(kda.selective_scan_step(**cut, state=state))
        else:
            out.append(kda.selective_scan(**cut, cu_seqlens=ints(0, n), init_state=state, final_state=state)[0])
        at += n
    assert at == 230
    ref.check(torch.cat(out), wy, e, "pieces")
    ref.check(state, wn, ne, "pieces state")


def test_scan_extreme_steps():
    """Steps that forget everything (d A far below the exponential's range), steps of almost nothing, NaN in
    one channel and sequence."""
    g = gen(14)
    s = scan_inputs(g, 96, 32, 16, torch.float32)
    s["dt"] = s["dt"].clone()
    s["dt"][5] = 300.0
    s["dt"][6] = -90.0
    s["x"] = s["x"].clone()
    s["x"][70, 3] = math.nan
    wy, e, wn, ne = reference(s, [48, 40, 8], None)
    y, new = kda.selective_scan(**s, cu_seqlens=ints(0, 48, 88, 96))
    ref.check(y, wy, e, "extreme")
    ref.check(new, wn, ne, "extreme state")


# ------------------------------------------------------------------ streams, graphs, order
def test_streams_graphs_and_repeats():
    """On another stream, captured and replayed with new contents and lengths, and again: the same bits."""
    g = gen(15)
    x, w = normal(g, 96, 64), normal(g, 192, 64, scale=0.125)
    cw, A = normal(g, 192, 4), -torch.rand(64, 16, generator=g, device="cuda") - 0.1
    cu = ints(0, 40, 41, 90)
    dtw = normal(g, 96, 64)
    conv_state, scan_state = torch.zeros(3, 3, 192, dtype=torch.bfloat16, device="cuda"), torch.zeros(3, 64, 16, device="cuda")

    def layer(stream=None):
        p = kda.linear(x, w, activation="silu", stream=stream)
        q, _ = kda.short_conv(p, cw, None, cu, conv_state, parts=3, final_state=conv_state, stream=stream)
        return kda.selective_scan(q[0], dtw, A, q[1][:, :16], q[2][:, :16], None, q[1], None, cu, scan_state,
                                  final_state=scan_state, stream=stream)[0]

    def fresh():
        conv_state.zero_()
        scan_state.zero_()

    a = layer()
    want = [t.clone() for t in (a[:90], conv_state, scan_state)]
    side = torch.cuda.Stream()
    fresh()
    side.wait_stream(torch.cuda.current_stream())
    b = layer(side)
    torch.cuda.current_stream().wait_stream(side)
    assert all(torch.equal(p, q) for p, q in zip((b[:90], conv_state, scan_state), want))
    fresh()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        c = layer()
    graph.replay()
    assert all(torch.equal(p, q) for p, q in zip((c[:90], conv_state, scan_state), want))
    x.copy_(normal(g, 96, 64))
    cu.copy_(ints(0, 3, 96, 96))
    fresh()
    graph.replay()
    got = [t.clone() for t in (c, conv_state, scan_state)]
    fresh()
    d = layer()
    assert all(torch.equal(p, q) for p, q in zip((d, conv_state, scan_state), got))


@pytest.mark.parametrize("m", [1, 4, 12, 64, 300])
def test_weights_written_by_the_call_before(m):
    """A call whose weights (and rows) the call before it wrote in place, with the ends and beginnings of all of them
    overlapping in a replayed graph: as with a synchronisation between any two."""
    g = gen(100 + m)
    a, b, x = normal(g, 512, 64, scale=0.1), normal(g, 256, 64, scale=0.1), normal(g, m, 256)
    first = normal(g, 512, 256)
    w, y = first.clone(), torch.zeros(m, 512, dtype=torch.bfloat16, device="cuda")

    def run(between):
        for _ in range(8):
            kda.linear(a, b, residual=w, out=w)
            between()
            kda.linear(x, w, residual=y, out=y)
            between()

    run(torch.cuda.synchronize)
    want = [w.clone(), y.clone()]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        run(lambda: None)
    for _ in range(3):
        w.copy_(first)
        y.zero_()
        graph.replay()
        assert torch.equal(w, want[0]) and torch.equal(y, want[1])


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_offsets_past_32_bits(dtype):
    """Rows and entries of pools more than 2^32 elements apart: the bits of the same calls on compact tensors."""
    dt, rows, stride = DT[dtype], 65, (1 << 26) + 64
    g = gen(16)
    try:
        wide = torch.empty(rows * stride, dtype=dt, device="cuda")
    except torch.cuda.OutOfMemoryError:
        pytest.skip("not enough memory")

    def far(t, column):
        view = wide.as_strided((t.shape[0], t.shape[1]), (stride, 1), column)
        view.copy_(t)
        return view

    x, w, r = normal(g, rows, 64, dtype=dt), normal(g, 40, 64, dtype=dt, scale=0.125), normal(g, rows, 40, dtype=dt)
    out = torch.zeros(rows, 40, dtype=dt, device="cuda")
    for m in (4, rows):  # (few rows, many)
        y = far(out[:m], 1024)
        kda.linear(far(x[:m], 0), far(w, 128), residual=far(r[:m], 256), out=y)
        assert torch.equal(y, kda.linear(x[:m], w, residual=r[:m]))
    conv_w, cu = normal(g, 64, 4, dtype=dt), ints(0, 20, 21, rows)
    z, b, c = normal(g, rows, 64, dtype=dt), normal(g, rows, 8, dtype=dt), normal(g, rows, 8, dtype=dt)
    dts = normal(g, rows, 64, dtype=dt)
    A = -torch.rand(64, 8, generator=g, device="cuda") - 0.1
    for offsets, step in ((cu, False), (None, True)):
        y = far(torch.zeros_like(x), 1024)
        if step:
            kda.short_conv_step(far(x, 0), conv_w, torch.zeros(rows, 3, 64, dtype=dt, device="cuda"), out=y)
            want = kda.short_conv_step(x, conv_w, torch.zeros(rows, 3, 64, dtype=dt, device="cuda"))
        else:
            kda.short_conv(far(x, 0), conv_w, None, offsets, out=y)
            want = kda.short_conv(x, conv_w, None, offsets)[0]
        assert torch.equal(y, want)
        y = far(torch.zeros_like(x), 1024)
        f = [far(t, 128 * i) for i, t in enumerate((x, dts, b, c, z))]
        if step:
            kda.selective_scan_step(f[0], f[1], A, f[2], f[3], torch.zeros(rows, 64, 8, device="cuda"), z=f[4], out=y)
            want = kda.selective_scan_step(x, dts, A, b, c, torch.zeros(rows, 64, 8, device="cuda"), z=z)
        else:
            kda.selective_scan(f[0], f[1], A, f[2], f[3], None, f[4], None, offsets, out=y)
            want = kda.selective_scan(x, dts, A, b, c, None, z, None, offsets)[0]
        assert torch.equal(y, want)
    del wide, y, f
    # the last entries of pools
    n, ch = 9000, 4096 * 8
    x, dts = normal(g, 2, ch, dtype=dt), normal(g, 2, ch, dtype=dt)
    slots = ints(n - 1, 7)
    pool, few = torch.empty(n, ch, 8, device="cuda"), torch.zeros(2, ch, 8, device="cuda")
    pool[n - 1] = pool[7] = 0
    A = -torch.rand(ch, 8, generator=g, device="cuda") - 0.1
    for _ in range(2):
        got = kda.selective_scan_step(x, dts, A, b[:2], c[:2], pool, slots=slots)
        assert torch.equal(got, kda.selective_scan_step(x, dts, A, b[:2], c[:2], few))
        kda.selective_scan(x, dts, A, b[:2], c[:2], None, None, None, ints(0, 1, 2), pool, init_slots=slots, final_state=pool,
                           final_slots=slots)
        kda.selective_scan(x, dts, A, b[:2], c[:2], None, None, None, ints(0, 1, 2), few, final_state=few)
        assert torch.equal(pool[n - 1], few[0]) and torch.equal(pool[7], few[1])
    del pool, few
    n = 24000
    conv_w = normal(g, ch, 4, dtype=dt)
    slots = ints(n - 1, 7)
    pool, few = torch.empty(n, 3, ch, dtype=dt, device="cuda"), torch.zeros(2, 3, ch, dtype=dt, device="cuda")
    pool[n - 1] = pool[7] = 0
    for _ in range(2):
        got = kda.short_conv_step(x, conv_w, pool, slots=slots)
        assert torch.equal(got, kda.short_conv_step(x, conv_w, few))
        kda.short_conv(x, conv_w, None, ints(0, 1, 2), pool, init_slots=slots, final_state=pool, final_slots=slots)
        kda.short_conv(x, conv_w, None, ints(0, 1, 2), few, final_state=few)
        assert torch.equal(pool[n - 1], few[0]) and torch.equal(pool[7], few[1])


def test_calls_on_streams_at_once():
    """Calls of all forms (pairs, split inputs, single CTAs, few rows, fp32) on four streams at once, and the convolution
    and the scan in parts beside them: as one after the other."""
    g = gen(17)
    w = normal(g, 1024, 1024, scale=1 / 32)
    xs = [normal(g, m, 1024) for m in (4, 64, 128, 300, 1500)]
    wf, xf = w[:100].float(), xs[2].float()
    cw, A = normal(g, 1024, 4), -torch.rand(1024, 16, generator=g, device="cuda") - 0.1
    bc = normal(g, 1500, 32)

    def run(stream):
        out = [kda.linear(x, w, activation="silu", stream=stream) for x in xs]
        out += [kda.linear(xs[3], w, out_dtype=torch.float32, stream=stream), kda.linear(xf, wf, stream=stream)]
        out += [kda.short_conv(xs[4], cw, stream=stream)[0]]
        return out + [kda.selective_scan(xs[4], xs[4], A, bc[:, :16], bc[:, 16:], stream=stream)[0]]

    want = run(None)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(4)]
    got = []
    for _ in range(5):
        for s in streams:
            with torch.cuda.stream(s):
                got.append(run(s))
    torch.cuda.synchronize()
    for out in got:
        assert all(torch.equal(a, b) for a, b in zip(out, want))
