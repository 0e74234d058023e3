"""The two ways that the arguments of the calls around the recurrence take from tensors to the C entry points (the
native one and ctypes) accept and refuse the same calls, with the same errors and the same results."""
import pytest
import torch

from kda_gated_delta_04_gb300 import kda

pytestmark = pytest.mark.gpu


def calls():
    """(name, function, arguments, keywords, the tensors that the call writes) of good and bad calls."""
    g = torch.Generator(device="cuda").manual_seed(1)
    r = lambda *s, dt=torch.bfloat16: torch.randn(*s, generator=g, device="cuda").to(dt)
    f = lambda *s: r(*s, dt=torch.float32)
    i = lambda *x: torch.tensor(x, dtype=torch.int32, device="cuda")
    x, w = r(6, 64), r(48, 64)
    good = dict(activation="silu", residual=r(6, 48), out=r(6, 50)[:, :48], errors=i(0))
    yield "linear", kda.linear, (x, w, r(48)), good
    yield "linear plain", kda.linear, (x, w), {}
    yield "linear to fp32", kda.linear, (x, w), dict(out_dtype=torch.float32, residual=f(6, 48))
    for name, args, kw in [
            ("inner sizes", (x, r(48, 63)), {}), ("weight type", (x, w.float()), {}), ("bias shape", (x, w, r(47)), {}),
            ("residual type", (x, w), dict(residual=f(6, 48))), ("out shape", (x, w), dict(out=r(6, 47))),
            ("out type", (x, w), dict(out=r(6, 48).half())), ("out_dtype", (x, w), dict(out=r(6, 48), out_dtype=torch.float32)),
            ("activation", (x, w), dict(activation="relu")), ("last stride", (x, r(64, 48).T), {}), ("on the CPU", (x, w.cpu()), {}),
            ("shared output rows", (x, w), dict(out=r(1, 48).expand(6, 48))), ("fp32 to bf16", (x.float(), w.float()), dict(out_dtype=torch.bfloat16)),
            ("one dimension", (x[0], w), {}), ("no weight", (x, None), {}), ("weight of one dimension", (x, w[0]), {}), ("half", (x.half(), w.half()), {})]:
        yield "linear, " + name, kda.linear, args, kw
    c, t, b = r(10, 56)[:, :48], r(48, 4), r(48)
    yield "conv", kda.short_conv, (c, t, b, i(0, 3, 10), r(2, 3, 48)), dict(parts=3, out=r(3, 10, 16), final_state=r(2, 3, 48))
    yield "conv slots", kda.short_conv, (c, t, None, i(0, 3, 10), r(5, 3, 48)), dict(
        init_slots=i(4, -1), final_state=r(5, 3, 48), final_slots=i(0, 2), activation=None, errors=i(0))
    yield "conv step", kda.short_conv_step, (c, t, r(10, 3, 48), b), {}
    for name, args, kw in [
            ("taps", (c, r(48, 5)), {}), ("channels", (r(10, 44), r(44, 4)), {}), ("parts", (c, t), dict(parts=5)),
            ("narrow parts", (c, t), dict(parts=12)), ("offsets type", (c, t, None, i(0, 10).long()), {}), ("no offsets", (c, t, None, i()), {}), ("taps of one dimension", (c, t[:, 0]), {}), ("state", (c, t, None, None, r(1, 4, 48)), {}),
            ("states", (c, t, None, i(0, 3, 10), r(1, 3, 48)), {}), ("state type", (c, t, None, None, f(1, 3, 48)), {}),
            ("slots alone", (c, t), dict(init_slots=i(0))), ("slots shape", (c, t, None, None, r(4, 3, 48)), dict(init_slots=i(0, 1))),
            ("activation", (c, t), dict(activation="gelu")), ("misaligned", (r(10, 57)[:, 1:49], t), {}), ("bias type", (c, t, b.float()), {})]:
        yield "conv, " + name, kda.short_conv, args, kw
    s, A, bc = (r(10, 48), r(10, 48)), -f(48, 16).abs(), r(10, 72)
    B, C = bc[:, :16], bc[:, 16:32]
    yield "scan", kda.selective_scan, (*s, A, B, C, f(48), r(10, 48), f(48), i(0, 3, 10), f(2, 48, 16)), dict(
        final_state=f(2, 48, 16), errors=i(0))
    yield "scan groups", kda.selective_scan, (*s, A, bc[:, :32].unflatten(1, (2, 16)), bc[:, 32:64].unflatten(1, (2, 16))), dict(softplus=False)
    yield "scan step", kda.selective_scan_step, (*s, A, B, C, f(12, 48, 16)), dict(slots=i(*range(10)), new_state=f(12, 48, 16))
    for name, args, kw in [
            ("states", (*s, f(48, 24), r(10, 24), r(10, 24)), {}), ("A type", (*s, A.bfloat16(), B, C), {}), ("A of one dimension", (*s, A[:, 0], B, C), {}), ("offsets of two", (*s, A, B, C, None, None, None, i(0, 10)[None]), {}), ("B type", (*s, A, B.float(), C), {}),
            ("groups apart", (*s, A, r(10, 4, 16)[:, ::2], r(10, 4, 16)[:, ::2]), {}), ("groups differ", (*s, A, r(10, 2, 16), C), {}),
            ("D shape", (*s, A, B, C, f(47)), {}), ("z type", (*s, A, B, C, None, f(10, 48)), {}), ("dt rows", (s[0], r(9, 48), A, B, C), {}),
            ("state type", (*s, A, B, C, None, None, None, None, r(1, 48, 16)), {}), ("errors", (*s, A, B, C), dict(errors=i(0, 0))),
            ("narrow groups", (*s, A, r(10, 12, 16), r(10, 12, 16)), {}), ("slots without a state", (*s, A, B, C), dict(init_slots=i(0)))]:
        yield "scan, " + name, kda.selective_scan, args, kw


def outcome(f, args, kw):
    args = [a.clone() if isinstance(a, torch.Tensor) and a.dim() == 3 and a.is_contiguous() else a for a in args]  # states
    kw = {k: v.clone() if k in ("final_state", "new_state", "errors") else v for k, v in kw.items()}
    try:
        out = f(*args, **kw)
    except (TypeError, ValueError, RuntimeError) as e:
        return type(e).__name__, str(e)
    torch.cuda.synchronize()
    out = out if isinstance(out, tuple) else (out,)
    return [t.clone() for t in (*out, *args, *kw.values()) if isinstance(t, torch.Tensor)]


def test_native_and_ctypes_agree(monkeypatch):
    kda._load_torch()
    if kda._native is None:
        pytest.skip("latent_args.cpp was left out of the build")
    good = 0
    for name, f, args, kw in calls():
        native = outcome(f, args, kw)
        with monkeypatch.context() as m:
            m.setattr(kda, "_native", None)
            plain = outcome(f, args, kw)
        if isinstance(plain, tuple):
            assert native == plain, name
            assert "," in name, (name, plain)
        else:
            good += 1
            assert not isinstance(native, tuple) and len(native) == len(plain), (name, native)
            assert all(torch.equal(a.isnan(), b.isnan()) and torch.equal(a.nan_to_num(), b.nan_to_num()) for a, b in zip(native, plain)), name
    assert good == 9


def test_native_is_the_way_taken():
    """Good calls do not go through ctypes where the native way is built."""
    kda._load_torch()
    if kda._native is None:
        pytest.skip("latent_args.cpp was left out of the build")
    made = list(calls())
    real, kda._lib = kda._lib, None
    try:
        for name, f, args, kw in made:
            if "," not in name:
                f(*args, **kw)
                assert kda._lib is None, name
    finally:
        kda._lib = real
