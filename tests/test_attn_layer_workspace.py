"""The workspace that an attention call makes for itself: allocated for the stream that
the call runs on, and alive until the call is made.  Host side alone: tensors that
say they are on a device, and stand-ins for torch's streams (no device needed)."""
import contextlib
import gc
import weakref

import pytest

import attention_decode_megakernel_b200 as mk

torch = pytest.importorskip("torch")


class OnDevice(torch.Tensor):
    """A CPU tensor that says it is on device 0."""

    def get_device(self):
        return 0


def _on_device(*shape, dtype=torch.bfloat16):
    return torch.zeros(*shape, dtype=dtype).as_subclass(OnDevice)


@pytest.fixture
def record(monkeypatch):
    """What happens during a call: ("made", stream) of every workspace and ("call",
    stream, whether its workspace is alive)."""
    seen, current, made = [], ["current"], []

    @contextlib.contextmanager
    def on_stream(s):
        current.append(s)
        yield
        current.pop()

    def workspace(head_dim, device="cuda"):
        seen.append(("made", current[-1]))
        w = _on_device(4096, dtype=torch.uint8)
        made.append(weakref.ref(w))
        return w

    def call(device, stream, *args):
        gc.collect()
        w = made[-1]() if made else None
        seen.append(("call", stream, w is not None and w.data_ptr() in args))

    monkeypatch.setattr(torch.cuda, "stream", on_stream)
    monkeypatch.setattr(torch.cuda, "ExternalStream", lambda s, device=None: ("external", s))
    monkeypatch.setattr(torch.cuda, "default_stream", lambda device=None: "default")
    monkeypatch.setattr(mk, "attn_workspace", workspace)
    monkeypatch.setattr(mk._paged_call, "slow", call)
    monkeypatch.setattr(mk._packed_call, "slow", call)
    return seen


def _calls(**given):
    q, k = _on_device(3, 4, 64), _on_device(3, 2, 64)
    i32 = dict(dtype=torch.int32)
    cu, out = _on_device(2, **i32), _on_device(3, 4, 64)
    cache = mk.KvCache(_on_device(2, 2, 16, 64), _on_device(2, 2, 16, 64))
    mk.attn_packed(q, k, k, cu, out, **given)
    mk.attn_paged(q, cache, _on_device(1, 2, **i32), _on_device(1, **i32), cu, out, **given)


@pytest.mark.parametrize("stream,made_on", [
    (None, "current"), (0x5550, ("external", 0x5550)), (0, "default"), (1, "default"),
    (2, ("external", 2))])
def test_workspace_of_a_call(record, stream, made_on):
    """Without a workspace of the caller's: one in the call's own stream (0 and 1 are the
    names of the default one)."""
    _calls(stream=stream)
    assert record == [("made", made_on), ("call", stream, True)] * 2


def test_workspace_of_the_caller(record):
    ws = _on_device(4096, dtype=torch.uint8)
    _calls(stream=0x5550, workspace=ws)
    assert [r[:2] for r in record] == [("call", 0x5550)] * 2
