"""The latent calls' native argument passing where a device is there to ask about."""
import pytest
import torch

from kda_gated_delta_04_gb300 import kda
from test_latent_host import Claimed

pytestmark = pytest.mark.gpu


def test_native_refuses_tensors_of_another_gpu():
    """Calls without tokens, which launch nothing: with another GPU's tensors they are handed back (-1) to the
    checks that name the fault, before the entry point."""
    kda._load_torch()
    if kda._native is None:
        pytest.skip("latent_args.cpp was left out of the build")
    assert torch.cuda.current_device() == 0
    t, i32, f32 = Claimed, torch.int32, torch.float32
    a = (t(0, 512), t(0, 64), t(2, 8, 576), t(0, dtype=i32))
    assert kda._native.append(*a, None, 1e-6, None, None, False, None, None, None, None, None, 0) == -1
    d = (t(0, 3, 576), t(2, 8, 576), t(0, 1, dtype=i32), t(0, dtype=i32), 0.1, t(0, 3, 512), t(0, 3, dtype=f32))
    assert kda._native.decode(*d, t(512, dtype=torch.uint8), None, 0) == -1
    p = (t(0, 3, 192), t(0, 3, 128), t(0, 64), t(0, 3, 128), 0.1, None, None, True, t(0, 3, 128), t(0, 3, dtype=f32))
    assert kda._native.prefill(*p, None, 0) == -1


def test_native_takes_the_same_calls_here():
    kda._load_torch()
    if kda._native is None:
        pytest.skip("latent_args.cpp was left out of the build")
    t = lambda *size, dtype=torch.bfloat16: torch.empty(size, dtype=dtype, device="cuda")
    i32, f32 = torch.int32, torch.float32
    a = (t(0, 512), t(0, 64), t(2, 8, 576), t(0, dtype=i32))
    assert kda._native.append(*a, None, 1e-6, None, None, False, None, None, None, None, None, 0) == kda.KDA_OK
    d = (t(0, 3, 576), t(2, 8, 576), t(0, 1, dtype=i32), t(0, dtype=i32), 0.1, t(0, 3, 512), t(0, 3, dtype=f32))
    assert kda._native.decode(*d, t(512, dtype=torch.uint8), None, 0) == kda.KDA_OK
    p = (t(0, 3, 192), t(0, 3, 128), t(0, 64), t(0, 3, 128), 0.1, None, None, True, t(0, 3, 128), t(0, 3, dtype=f32))
    assert kda._native.prefill(*p, None, 0) == kda.KDA_OK
