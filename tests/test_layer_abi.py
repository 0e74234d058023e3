"""The host side of the projections, the short convolution and the selective scan: every refusal before
anything touches a GPU."""
import importlib.machinery
import importlib.util
import os
import subprocess

import pytest
import torch

from test_latent_abi import FAKE, INVALID, OK, UNSUPPORTED, kda  # noqa: F401 (a fixture)
from test_latent_host import Claimed, Recorded, Stream

BIG = 2 ** 31 - 1


def linear_args(**over):
    a = dict(x=FAKE, x_stride=64, w=FAKE, w_stride=64, bias=FAKE, residual=2 * FAKE, residual_stride=32, y=FAKE, y_stride=32,
             rows=4, out_features=32, in_features=64, dtype=0, out_dtype=0, activation=1, errors=FAKE, stream=None)
    assert set(over) <= set(a)
    a.update(over)
    return a.values()


@pytest.mark.parametrize("over,expected", [
    (dict(x=None), INVALID), (dict(w=None), INVALID), (dict(y=None), INVALID), (dict(x=FAKE + 1), INVALID),
    (dict(w=FAKE + 2, dtype=1, out_dtype=1), INVALID), (dict(bias=FAKE + 1), INVALID), (dict(residual=FAKE + 2, out_dtype=1), INVALID),
    (dict(y=FAKE + 1), INVALID), (dict(errors=FAKE + 2), INVALID), (dict(x_stride=-1), INVALID), (dict(w_stride=-64), INVALID), (dict(y_stride=31), INVALID),
    (dict(y_stride=0), INVALID), (dict(residual_stride=-1), INVALID), (dict(residual=FAKE, residual_stride=40), INVALID),
    (dict(y_stride=2 ** 39), INVALID), (dict(rows=-1), INVALID), (dict(out_features=-1), INVALID), (dict(in_features=0), INVALID),
    (dict(dtype=2), INVALID), (dict(out_dtype=-1), INVALID), (dict(activation=5), INVALID), (dict(activation=-1), INVALID),
    (dict(dtype=1, out_dtype=0), UNSUPPORTED), (dict(rows=BIG), UNSUPPORTED), (dict(in_features=BIG), UNSUPPORTED),
    (dict(out_features=BIG), UNSUPPORTED), (dict(rows=2 ** 30, out_features=2 ** 14, y_stride=2 ** 14, residual=None), UNSUPPORTED),
    (dict(rows=0, x=None, y=None), OK), (dict(out_features=0, w=None, y=None), OK),
])
def test_linear_refusals(kda, over, expected):  # noqa: F811
    assert kda.kda_linear(*linear_args(**over)) == expected


def conv_args(**over):
    a = dict(x=FAKE, x_stride=64, weight=FAKE, bias=FAKE, width=4, cu_seqlens=FAKE, num_seqs=2, total_tokens=10, channels=48,
             parts=3, dtype=0, activation=1, init_state=FAKE, init_slots=FAKE, num_init=5, final_state=FAKE, final_slots=FAKE,
             num_final=5, y=FAKE, y_part_stride=160, y_stride=16, errors=FAKE, stream=None)
    assert set(over) <= set(a)
    a.update(over)
    return a.values()


SEQUENCES = [
    (dict(num_seqs=-1), INVALID), (dict(total_tokens=-1), INVALID), (dict(num_seqs=0), INVALID), (dict(cu_seqlens=None, num_seqs=3), INVALID),
    (dict(cu_seqlens=FAKE + 2), INVALID), (dict(init_state=None), INVALID), (dict(final_state=None), INVALID),
    (dict(init_state=FAKE + 8), INVALID), (dict(final_state=FAKE + 4), INVALID), (dict(init_slots=FAKE + 1), INVALID),
    (dict(final_slots=FAKE + 2), INVALID), (dict(num_init=-1), INVALID), (dict(num_final=-1), INVALID),
    (dict(init_slots=None, num_init=1), INVALID), (dict(final_slots=None, num_final=1), INVALID), (dict(errors=FAKE + 1), INVALID),
    (dict(total_tokens=BIG, num_seqs=1), UNSUPPORTED), (dict(dtype=2), INVALID),
    (dict(num_seqs=0, total_tokens=0), OK),
]


@pytest.mark.parametrize("over,expected", SEQUENCES + [
    (dict(x=None), INVALID), (dict(weight=None), INVALID), (dict(y=None), INVALID), (dict(x=FAKE + 8), INVALID),
    (dict(weight=FAKE + 2), INVALID), (dict(bias=FAKE + 2), INVALID), (dict(y=FAKE + 8), INVALID), (dict(x_stride=60), INVALID),
    (dict(x_stride=-8), INVALID), (dict(y_stride=8), INVALID), (dict(y_stride=20), INVALID), (dict(y_part_stride=0), INVALID),
    (dict(y_part_stride=152), INVALID), (dict(y_stride=48, y_part_stride=8), INVALID), (dict(y_stride=40, y_part_stride=16), INVALID),
    (dict(parts=1, y_stride=40), INVALID), (dict(width=0), INVALID), (dict(channels=0), INVALID), (dict(parts=0), INVALID),
    (dict(activation=9), INVALID), (dict(width=1), UNSUPPORTED), (dict(width=5), UNSUPPORTED), (dict(channels=36), UNSUPPORTED),
    (dict(parts=5), UNSUPPORTED), (dict(parts=4), UNSUPPORTED), (dict(activation=3), UNSUPPORTED),
])
def test_conv_refusals(kda, over, expected):  # noqa: F811
    assert kda.kda_short_conv(*conv_args(**over)) == expected


def scan_args(**over):
    a = dict(x=FAKE, x_stride=64, dt=FAKE, dt_stride=64, A=FAKE, B=FAKE, b_stride=32, C=FAKE, c_stride=32, D=FAKE, z=FAKE,
             z_stride=64, dt_bias=FAKE, cu_seqlens=FAKE, num_seqs=2, total_tokens=10, channels=64, num_groups=2, d_state=16,
             dtype=0, init_state=FAKE, init_slots=FAKE, num_init=5, final_state=FAKE, final_slots=FAKE, num_final=5, y=FAKE,
             y_stride=64, errors=FAKE, stream=None, flags=1)
    assert set(over) <= set(a)
    a.update(over)
    return a.values()


@pytest.mark.parametrize("over,expected", SEQUENCES + [
    (dict(x=None), INVALID), (dict(dt=None), INVALID), (dict(A=None), INVALID), (dict(B=None), INVALID), (dict(C=None), INVALID),
    (dict(y=None), INVALID), (dict(x=FAKE + 8), INVALID), (dict(A=FAKE + 4), INVALID), (dict(D=FAKE + 4), INVALID),
    (dict(z=FAKE + 2), INVALID), (dict(dt_bias=FAKE + 8), INVALID), (dict(y=FAKE + 8), INVALID), (dict(b_stride=17), INVALID),
    (dict(c_stride=-8), INVALID), (dict(z_stride=4), INVALID), (dict(y_stride=56), INVALID), (dict(y_stride=0), INVALID),
    (dict(flags=2), INVALID), (dict(channels=0), INVALID), (dict(num_groups=0), INVALID), (dict(d_state=0), INVALID),
    (dict(d_state=24), UNSUPPORTED), (dict(d_state=128), UNSUPPORTED), (dict(num_groups=3), UNSUPPORTED),
    (dict(num_groups=16), UNSUPPORTED), (dict(channels=36, num_groups=1), UNSUPPORTED),
])
def test_scan_refusals(kda, over, expected):  # noqa: F811
    assert kda.kda_selective_scan(*scan_args(**over)) == expected


# ------------------------------------------------------------------ the binding
def calls():
    t, f32, i32 = Claimed, torch.float32, torch.int32
    yield "linear", (t(4, 64), t(32, 64)), dict(out=t(4, 32))
    yield "short_conv", (t(10, 48), t(48, 4)), dict(parts=3, out=t(3, 10, 16), final_state=t(1, 3, 48))
    yield "short_conv_step", (t(10, 48), t(48, 4), t(12, 3, 48)), dict(slots=t(10, dtype=i32), out=t(10, 48))
    scan = (t(10, 48), t(10, 48), t(48, 16, dtype=f32), t(10, 16), t(10, 16))
    yield "selective_scan", scan, dict(out=t(10, 48), final_state=t(1, 48, 16, dtype=f32))
    yield "selective_scan_step", (*scan, t(10, 48, 16, dtype=f32)), dict(out=t(10, 48))


@pytest.mark.parametrize("name,args,kw", list(calls()), ids=lambda x: x if isinstance(x, str) else "")
def test_tensors_of_another_gpu_are_refused(kda, monkeypatch, name, args, kw):  # noqa: F811
    fake = Recorded()
    monkeypatch.setattr(kda, "_lib", fake)
    monkeypatch.setattr(kda, "_native", None)
    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: 0, raising=False)
    with pytest.raises(ValueError, match="cuda:1.*cuda:0"):
        getattr(kda, name)(*args, stream=Stream(), **kw)
    assert not fake.called
    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: 1)  # made current: taken
    getattr(kda, name)(*args, stream=Stream(), **kw)
    assert fake.called == ["kda_" + name.removesuffix("_step")]


# ------------------------------------------------------------------ the native way
STUB = """
int PyGILState_Check(void);
int kda_latent_append() { return 0; }
int kda_latent_decode() { return 0; }
int kda_latent_prefill() { return 0; }
int kda_linear() { return 100 + PyGILState_Check(); }
int kda_short_conv() { return 100 + PyGILState_Check(); }
int kda_selective_scan() { return 100 + PyGILState_Check(); }
"""


@pytest.fixture(scope="module")
def stubbed(kda, tmp_path_factory):  # noqa: F811
    """The native module over a library whose entry points do nothing but say whether the calling thread
    holds the interpreter's lock (101) or not (100)."""
    from kda_gated_delta_04_gb300 import build
    if not os.path.exists(build.ARGS_PATH):
        pytest.skip("latent_args.cpp was left out of the build")
    where = str(tmp_path_factory.mktemp("stub"))
    with open(os.path.join(where, "stub.c"), "w") as f:
        f.write(STUB)
    run = lambda *cmd: subprocess.run(cmd, check=True, capture_output=True)
    run("gcc", "-shared", "-fPIC", "-o", os.path.join(where, "liblayerstub.so"), os.path.join(where, "stub.c"))
    path = os.path.join(where, "_latent_args.so")
    run("g++", "-shared", "-o", path, os.path.join(build.BUILD_DIR, "latent_args.o"), "-L", where, "-llayerstub",
        f"-Wl,-rpath,{where}", "-Wl,-Bsymbolic", "-L", os.path.join(os.path.dirname(torch.__file__), "lib"),
        "-ltorch_python", "-ltorch_cpu", "-lc10", "-lc10_cuda")
    loader = importlib.machinery.ExtensionFileLoader("_latent_args", path)
    return importlib.util.module_from_spec(importlib.util.spec_from_loader("_latent_args", loader))


def native_calls():
    """Each call's arguments without the stream; where its numbers are, and its flag."""
    t, f32, i32 = Claimed, torch.float32, torch.int32
    yield "linear", [t(4, 64), t(32, 64), None, None, 1, t(4, 32), None], [4], None
    yield "conv", [t(10, 48), t(48, 4), None, None, 1, None, None, t(1, 3, 48), None, 1, 3, t(3, 10, 16), None], [4, 9, 10], None
    yield "scan", [t(10, 48), t(10, 48), t(48, 16, dtype=f32), t(10, 16), t(10, 16), None, None, None, t(3, dtype=i32), 2, None, None,
                   t(2, 48, 16, dtype=f32), None, True, t(10, 48), None], [9], 14


class Unclear:
    def __bool__(self):
        raise RuntimeError("neither true nor false")


@pytest.mark.skipif(torch.cuda.is_available(), reason="with a device the tensors' own is compared first")
@pytest.mark.parametrize("name,args,numbers,flag", list(native_calls()), ids=lambda x: x if isinstance(x, str) else "")
def test_the_native_way(stubbed, name, args, numbers, flag):
    """The lock is let go during the entry point; what is no number, or a flag without a truth value, is handed back
    like any other bad argument, and leaves no error set."""
    call = getattr(stubbed, name)
    assert call(*args, 0) == 100
    for at, bad in [(n, b) for n in numbers for b in (None, 1.5, "1", 2 ** 70, -1)] + ([] if flag is None else [(flag, Unclear())]):
        st, after = call(*args[:at], bad, *args[at + 1:], 0), [i for i in range(3)]
        assert st == -1 and after == [0, 1, 2], (at, bad)
    assert call(*args) == -1 and call(*args, 0, 0) == -1
    for at in range(len(args)):  # a tensor where none belongs, and none where one does
        if isinstance(args[at], torch.Tensor) and at not in (7, 8, 12):
            assert call(*args[:at], None, *args[at + 1:], 0) == -1, at
        assert call(*args[:at], object(), *args[at + 1:], 0) in (-1, 100 if at == flag else -1), at
