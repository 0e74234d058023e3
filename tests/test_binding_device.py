"""The binding's calls launch on the current device: tensors of another GPU are refused before anything runs."""
import pytest
import torch

from test_abi import kda  # noqa: F401 (a fixture)
from test_latent_host import Claimed, Recorded, Stream


def calls():
    t, f32, i32 = Claimed, torch.float32, torch.int32
    x = (t(8, 2, 128), t(8, 2, 128), t(8, 2, 128), t(8, 2, 128, dtype=f32), t(8, 2, dtype=f32))
    state, ws = t(1, 2, 128, 128, dtype=f32), t(4096, dtype=torch.uint8)
    yield "prefill", x, dict(o=t(8, 2, 128), final_state=state, workspace=ws)
    yield "prefill_slots", (*x, None, state, t(1, dtype=i32)), dict(o=t(8, 2, 128), workspace=ws)
    many = t(8, 2, 128, 128, dtype=f32)
    yield "decode_step", (*x, many), dict(o=t(8, 2, 128))
    yield "decode_step_slots", (*x, many, t(8, dtype=i32)), dict(o=t(8, 2, 128))
    yield "diag_tensor_phases", (0, 1, ws), {}


@pytest.mark.parametrize("stream", [None, Stream()], ids=["current_stream", "given_stream"])
@pytest.mark.parametrize("name,args,kw", list(calls()), ids=lambda x: x if isinstance(x, str) else "")
def test_tensors_of_another_gpu_are_refused(kda, monkeypatch, name, args, kw, stream):  # noqa: F811
    fake = Recorded()
    monkeypatch.setattr(kda, "_lib", fake)
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda device=None: Stream())
    with pytest.raises(ValueError, match="cuda:1.*cuda:0"):
        getattr(kda, name)(*args, stream=stream, **kw)
    assert not fake.called
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 1)  # made current: taken
    getattr(kda, name)(*args, stream=stream, **kw)
    assert len(fake.called) == 1 and fake.called[0].startswith("kda_" + name)
