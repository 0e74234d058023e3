"""The two ways the latent calls' arguments take from tensors to the C entry points (the native one and
ctypes) accept and refuse the same calls, with the same errors and the same results."""
import pytest
import torch

from kda_gated_delta_04_gb300 import kda

pytestmark = pytest.mark.gpu


def calls():
    """(name, function, arguments, keywords) of good and bad calls."""
    g = torch.Generator(device="cuda").manual_seed(1)
    r = lambda *s, dt=torch.bfloat16: torch.randn(*s, generator=g, device="cuda").to(dt)
    i = lambda *s: torch.zeros(*s, dtype=torch.int32, device="cuda")
    kv, q, cache = r(4, 576), r(4, 3, 192), r(2, 8, 576)
    slots = torch.arange(4, dtype=torch.int32, device="cuda")
    cs = r(16, 64, dt=torch.float32)
    A = (kv[:, :512], kv[:, 512:], cache, slots)
    ok = dict(norm_weight=r(512), cos_sin=cs, positions=slots, q_pe=q[..., 128:], q_pe_out=r(4, 3, 64))
    yield "append", kda.latent_append, A, ok
    yield "append plain", kda.latent_append, A, {}
    for name, bad in [("norm shape", dict(norm_weight=r(511))), ("norm type", dict(norm_weight=r(512, dt=torch.float32))),
                      ("table type", dict(cos_sin=cs.double())), ("positions missing", dict(positions=None)),
                      ("positions length", dict(positions=i(5))), ("query rows", dict(q_pe=q[:3, :, 128:])),
                      ("query last stride", dict(q_pe=q[..., ::3])), ("out on the CPU", dict(q_pe_out=q[..., 128:].cpu())),
                      ("out not a tensor", dict(latent_out=3)), ("errors shape", dict(errors=i(2))),
                      ("misaligned", dict(q_pe=q[..., 127:191])), ("eps", dict(norm_eps=-1.0))]:
        yield "append, " + name, kda.latent_append, A, {**ok, **bad}
    yield "append, cache strided", kda.latent_append, (*A[:2], r(2, 16, 576)[:, ::2], slots), ok
    qa, table, lens = r(2, 3, 576), i(2, 1), torch.tensor([3, 8], dtype=torch.int32, device="cuda")
    D = (qa, cache, table, lens, 0.1)
    yield "decode", kda.latent_decode, D, {}
    yield "decode, given", kda.latent_decode, D, dict(o=torch.empty_like(qa[..., :512]), lse=r(2, 3, dt=torch.float32),
                                                     workspace=kda.latent_decode_workspace_for(3, 0, "cuda"))
    for name, args, kw in [("lengths type", (qa, cache, table, lens.long(), 0.1), {}), ("table rows", (qa, cache, i(3, 1), lens, 0.1), {}),
                           ("output shape", D, dict(o=r(2, 3, 511))), ("small workspace", D, dict(workspace=i(64))),
                           ("cache type", (qa, cache.float(), table, lens, 0.1), {}), ("scale", (qa, cache, table, lens, float("nan")), {}),
                           ("page of 4", (qa, cache.view(4, 4, 576), table, lens, 0.1), {})]:
        yield "decode, " + name, kda.latent_decode, args, kw
    qp, kvp, kpe = r(5, 3, 192), r(6, 3, 256), r(6, 64)
    cu = lambda *x: torch.tensor(x, dtype=torch.int32, device="cuda")
    P = (qp, kvp[..., :128], kpe, kvp[..., 128:], 0.1)
    yield "prefill", kda.latent_prefill, (*P, cu(0, 2, 5), cu(0, 2, 6)), {}
    yield "prefill, full", kda.latent_prefill, P, dict(causal=False)
    for name, args, kw in [("keys missing", (*P, cu(0, 2, 5)), {}), ("offsets type", (*P, cu(0, 2, 5).long(), cu(0, 2, 6)), {}),
                           ("offsets length", (*P, cu(0, 2, 5), cu(0, 6)), {}), ("values", (*P[:3], kvp[:5, :, 128:], 0.1), {}),
                           ("offsets of keys alone", P, dict(cu_k=cu(0, 6))), ("lse type", P, dict(lse=r(5, 3)))]:
        yield "prefill, " + name, kda.latent_prefill, args, kw


def outcome(f, args, kw):
    try:
        out = f(*args, **kw)
    except (TypeError, ValueError, RuntimeError) as e:
        return type(e).__name__, str(e)
    torch.cuda.synchronize()
    given = [t for t in (kw.get("q_pe_out"), args[2] if f is kda.latent_append else None) if t is not None]
    return [t.clone() for t in (out or [])] + [t.clone() for t in given]


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
        else:
            good += 1
            assert len(native) == len(plain) and all(torch.equal(a, b) for a, b in zip(native, plain)), name
    assert good == 6


def test_native_is_the_way_taken():
    """Good calls do not go through ctypes where the native way is built."""
    kda._load_torch()
    if kda._native is None:
        pytest.skip("latent_args.cpp was left out of the build")
    made = list(calls())  # (making the arguments uses the library too)
    real, kda._lib = kda._lib, None
    try:
        for name, f, args, kw in made:
            if name in ("append", "decode, given"):
                f(*args, **kw)
                assert kda._lib is None, name
    finally:
        kda._lib = real
