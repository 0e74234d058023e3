"""More of the latent calls' host side, without a GPU: calls whose outputs' rows overlap."""
import importlib.machinery
import importlib.util
import os
import subprocess

import pytest
import torch

from test_latent_abi import FAKE, INVALID, append_args, kda  # noqa: F401 (a fixture)


@pytest.mark.parametrize("over", [
    dict(out_head_stride=0), dict(out_token_stride=0), dict(out_token_stride=0, out_head_stride=0),
    dict(out_head_stride=56), dict(out_head_stride=8),            # a row reaches into the next head's
    dict(out_token_stride=56, out_head_stride=1024),              # ... the next token's
    dict(out_token_stride=248), dict(out_token_stride=192),       # the heads of two tokens meet
    dict(out_token_stride=64, out_head_stride=248),               # heads outermost, the tokens of two heads meet
    dict(q_token_stride=0, q_head_stride=0, out_token_stride=384, out_head_stride=0),
    dict(num_heads=1, out_token_stride=0), dict(num_heads=1, out_token_stride=56),
    dict(num_tokens=1, out_head_stride=0), dict(num_tokens=1, out_head_stride=56),
    dict(latent_out_stride=0), dict(latent_out_stride=504), dict(k_pe_out_stride=0), dict(k_pe_out_stride=56),
    dict(out_token_stride=2 ** 37, out_head_stride=2 ** 38, num_tokens=2 ** 29),  # (products past 64 bits)
])
@pytest.mark.parametrize("dtype", [0, 1])
def test_append_refuses_outputs_that_overlap(kda, over, dtype):  # noqa: F811
    """Rows written by several warps: the result would hang on their order (in place, on how often a shared
    row had been rotated when it was read)."""
    assert kda.kda_latent_append(*append_args(**over, dtype=dtype)) == INVALID


@pytest.mark.skipif(torch.cuda.is_available(), reason="passes every check, and the addresses are no one's")
@pytest.mark.parametrize("over", [
    dict(), dict(out_token_stride=64, out_head_stride=256), dict(out_token_stride=128, out_head_stride=64),
    dict(out_token_stride=256, out_head_stride=192), dict(num_tokens=1, out_token_stride=0, latent_out_stride=0, k_pe_out_stride=0),
    dict(num_heads=1, out_head_stride=0), dict(num_tokens=1, num_heads=1, out_token_stride=0, out_head_stride=0),
    dict(q_token_stride=0, q_head_stride=0), dict(latent_stride=0, k_pe_stride=0),  # inputs may be shared
    dict(latent_out=None, latent_out_stride=0), dict(k_pe_out=None, k_pe_out_stride=0),
    dict(q_pe=None, q_pe_out=None, out_token_stride=0, out_head_stride=0),
    dict(latent_out_stride=512, k_pe_out_stride=64),
])
def test_append_takes_outputs_that_do_not(kda, over):  # noqa: F811
    """Past the checks of the arguments the entry point finds that there is no device."""
    assert kda.kda_latent_append(*append_args(**over)) == kda.KDA_ERR_CUDA


# ------------------------------------------------------------------ the device
class Claimed(torch.Tensor):
    """A tensor that says it is on the second GPU.  It holds nothing, and its address is no one's."""

    @staticmethod
    def __new__(cls, *size, dtype=torch.bfloat16):
        return torch.Tensor._make_wrapper_subclass(cls, size, dtype=dtype, device="cuda:1")

    def data_ptr(self):
        return FAKE

    @classmethod
    def __torch_dispatch__(cls, func, types, args=(), kwargs=None):
        raise AssertionError(f"{func} on a tensor without contents")


class Recorded:
    """Stands in for the loaded library: what is called, and nothing happens."""

    def __init__(self):
        self.called = []

    def __getattr__(self, name):
        return lambda *args: self.called.append(name) or 0


class Stream:
    cuda_stream = 0


def claimed_calls():
    """(name, positional arguments, keywords, the native module's arguments without the stream)."""
    t, i32, f32 = Claimed, torch.int32, torch.float32
    a = (t(4, 512), t(4, 64), t(2, 8, 576), t(4, dtype=i32))
    yield "latent_append", a, {}, (*a, None, 1e-6, None, None, False, None, None, None, None, None)
    d = (t(2, 3, 576), t(2, 8, 576), t(2, 1, dtype=i32), t(2, dtype=i32), 0.1)
    out = dict(o=t(2, 3, 512), lse=t(2, 3, dtype=f32))
    ws = t(50331648, dtype=torch.uint8)
    yield "latent_decode", d, dict(**out, workspace=ws), (*d, *out.values(), ws, None)
    p = (t(5, 3, 192), t(5, 3, 128), t(5, 64), t(5, 3, 128), 0.1)
    out = dict(o=t(5, 3, 128), lse=t(5, 3, dtype=f32))
    yield "latent_prefill", p, out, (*p, None, None, True, *out.values(), None)


@pytest.mark.parametrize("stream", [None, Stream()], ids=["current_stream", "given_stream"])
@pytest.mark.parametrize("name,args,kw,native", list(claimed_calls()), ids=lambda x: x if isinstance(x, str) else "")
def test_tensors_of_another_gpu_are_refused(kda, monkeypatch, name, args, kw, native, stream):  # noqa: F811
    """The entry points launch on the current device: with another GPU's tensors the kernel would run on the
    wrong one, on addresses that are not its own."""
    fake = Recorded()
    monkeypatch.setattr(kda, "_lib", fake)
    monkeypatch.setattr(kda, "_native", None)
    monkeypatch.setattr(kda, "_torch_module", torch)
    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: 0)
    monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda dev: 0)
    with pytest.raises(ValueError, match="cuda:1.*cuda:0"):
        getattr(kda, name)(*args, stream=stream, **kw)
    assert not fake.called
    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: 1)  # made current: taken
    getattr(kda, name)(*args, stream=stream, **kw)
    assert fake.called == ["kda_" + name]


# ------------------------------------------------------------------ the native way
STUB = """
#include <stddef.h>
int PyGILState_Check(void);
int kda_latent_append() { return 100 + PyGILState_Check(); }
int kda_latent_decode() { return 100 + PyGILState_Check(); }
int kda_latent_prefill() { return 100 + PyGILState_Check(); }
"""


@pytest.fixture(scope="module")
def stubbed(kda, tmp_path_factory):  # noqa: F811
    """The native module over a library whose entry points do nothing but say whether the calling thread
    holds the interpreter's lock (101) or not (100)."""
    from kda_gated_delta_04_gb300 import build
    obj = os.path.join(build.BUILD_DIR, "latent_args.o")
    if not os.path.exists(build.ARGS_PATH):
        pytest.skip("latent_args.cpp was left out of the build")
    where = str(tmp_path_factory.mktemp("stub"))
    with open(os.path.join(where, "stub.c"), "w") as f:
        f.write(STUB)
    run = lambda *cmd: subprocess.run(cmd, check=True, capture_output=True)
    run("gcc", "-shared", "-fPIC", "-o", os.path.join(where, "libstub.so"), os.path.join(where, "stub.c"))
    path = os.path.join(where, "_latent_args.so")
    run("g++", "-shared", "-o", path, obj, "-L", where, "-lstub", f"-Wl,-rpath,{where}", "-Wl,-Bsymbolic", "-L",
        os.path.join(os.path.dirname(torch.__file__), "lib"), "-ltorch_python", "-ltorch_cpu", "-lc10", "-lc10_cuda")
    loader = importlib.machinery.ExtensionFileLoader("_latent_args", path)
    return importlib.util.module_from_spec(importlib.util.spec_from_loader("_latent_args", loader))


@pytest.mark.skipif(torch.cuda.is_available(), reason="with a device the tensors' own is compared first")
@pytest.mark.parametrize("name,native", [(c[0], c[3]) for c in claimed_calls()], ids=lambda x: x if isinstance(x, str) else "")
def test_the_native_way_lets_other_threads_run(stubbed, name, native):
    """A launch waits where the GPU's queue is full, maybe for a host function that needs the interpreter:
    as in a call through ctypes, the lock is not held meanwhile."""
    assert getattr(stubbed, name.removeprefix("latent_"))(*native, 0) == 100


class Unclear:
    def __bool__(self):
        raise RuntimeError("neither true nor false")


@pytest.mark.parametrize("name,native", [(c[0], c[3]) for c in claimed_calls() if c[0] != "latent_decode"],
                         ids=lambda x: x if isinstance(x, str) else "")
def test_the_native_way_leaves_no_error_behind(stubbed, name, native):
    """A flag without a truth value is handed back like any other bad argument; the error that asking for it
    raised does not stay set, to come up at some later call."""
    args = list(native)
    args[8 if name == "latent_append" else 7] = Unclear()
    call = getattr(stubbed, name.removeprefix("latent_"))
    st, after = call(*args, None), [i for i in range(3)]
    assert st == -1 and after == [0, 1, 2]
