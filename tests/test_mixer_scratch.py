"""Whose memory the packed prefill's scratch is, without a GPU: the binding with
a library that only records its calls."""
import gc
import types
import weakref

import pytest
import torch


class Dev(torch.Tensor):
    is_cuda = True


class RecordingLibrary:
    def __init__(self):
        self.calls = []

    def replayssm_prefill_packed_workspace(self, desc, total):
        return 10 * total

    def replayssm_prefill_packed(self, *args):
        self.calls.append(args)
        return 0


@pytest.fixture
def calls(monkeypatch):
    """call(total) -> (scratch address, bytes) as the library got them, and the allocations behind the calls."""
    import state_space_recurrence_amd as rs
    from state_space_recurrence_amd import mixer
    L, allocated = RecordingLibrary(), []

    def empty(shape, dtype, device, stream):
        t = torch.empty(shape, dtype=dtype)
        if dtype == torch.uint8:
            allocated.append((t.data_ptr(), t.numel(), weakref.ref(t)))
        return t.as_subclass(Dev)

    monkeypatch.setattr(mixer, "_lib", lambda: L)
    monkeypatch.setattr(mixer, "_empty", empty)
    monkeypatch.setattr(mixer, "_raw_stream", lambda stream, t: 0)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda *a: types.SimpleNamespace(cuda_stream=0))
    ls = rs.LayerState(2, 4, 1, -torch.ones(4), torch.ones(4), device="cpu")
    dev = lambda *s, dt=torch.bfloat16: torch.zeros(*s, dtype=dt).as_subclass(Dev)  # noqa: E731

    def call(total):
        mixer.prefill_packed(ls, dev(total, 4, 64), dev(total, 1, 128), dev(total, 1, 128), dev(total, 4),
                             dev(3, dt=torch.int32))
        return L.calls[-1][-3:-1]

    return call, allocated


def test_each_call_has_its_own_scratch(calls):
    """A later call, larger or not, neither takes over nor drops the memory of an earlier one: a captured graph may
    still write there, and a call on another stream may be running."""
    call, allocated = calls
    for n, total in enumerate((8, 16, 8, 4)):
        at, size = call(total)
        assert len(allocated) == n + 1
        assert (at, size) == allocated[n][:2] and size == 10 * total


def test_no_scratch_is_kept_between_calls(calls):
    call, allocated = calls
    call(16)
    gc.collect()
    assert [ref() for _, _, ref in allocated] == [None]
