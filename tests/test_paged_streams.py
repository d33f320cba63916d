"""Where the paged calls allocate when they are given a stream, with stand-ins for CUDA and the
library (no GPU): a workspace that is dropped, and results, have to be memory of the stream that the
kernels run on."""
import contextlib

import pytest
import torch

from kimi_delta_attention_03_gb300 import paged

E4M3 = torch.float8_e4m3fn


class Stream:
    def __init__(self, handle):
        self.cuda_stream, self.device = handle, torch.device("cpu")


class Library:
    """Answers every call with success and notes the stream it was given."""

    def __init__(self, seen):
        self.seen = seen

    def kda_paged_attention_workspace_bytes(self, *_):
        return 4096

    def __getattr__(self, name):
        return lambda *a: self.seen.append((name, a[-1])) or 0


@pytest.fixture
def world(monkeypatch):
    here, seen, allocated = [Stream(1)], [], []
    monkeypatch.setattr(paged, "_lib", lambda: Library(seen))
    monkeypatch.setattr(paged, "_cuda", lambda name, t: -1)
    monkeypatch.setattr(paged, "_stream", lambda s, dev: (s or here[-1]).cuda_stream)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda *_: here[-1])

    @contextlib.contextmanager
    def on(stream):
        here.append(stream)
        yield
        here.pop()

    monkeypatch.setattr(torch.cuda, "stream", on)
    empty, empty_like = torch.empty, torch.empty_like
    monkeypatch.setattr(torch, "empty", lambda *a, **k: allocated.append(here[-1].cuda_stream) or empty(*a, **k))
    monkeypatch.setattr(paged, "empty_like",
                        lambda *a, **k: allocated.append(here[-1].cuda_stream) or empty_like(*a, **k))
    return seen, allocated


def calls():
    i = torch.zeros(2, dtype=torch.int32)
    x = torch.zeros(3, 2, 128, dtype=torch.bfloat16)
    c, s = torch.zeros(3, 2, 16, 128).to(E4M3), torch.ones(3, 2)
    cu, one, p = torch.tensor([0, 1, 3], dtype=torch.int32), torch.zeros(1, dtype=torch.int32), torch.zeros(3, 8)
    t = torch.zeros(3, dtype=torch.int32)
    return {
        "plan": (5, lambda **k: paged.paged_plan(i, cu, torch.zeros(2, 4, dtype=torch.int32), i, t, one, 16, 3, **k)),
        "append": (0, lambda **k: paged.paged_append(x, x, t, c, c, s, s, **k)),
        "attention": (2, lambda **k: paged.paged_attention(x, cu, torch.zeros(2, 4, dtype=torch.int32), i, c, c, s, s, 2, **k)),
        "verify": (3, lambda **k: paged.verify_draft(p, t, cu, torch.zeros(3), torch.zeros(2, 8), **k)),
    }


@pytest.mark.parametrize("name", ["plan", "append", "attention", "verify"])
def test_memory_belongs_to_the_stream_of_the_kernels(world, name):
    seen, allocated = world
    count, call = calls()[name]
    seen.clear(), allocated.clear()
    call()
    assert allocated == [1] * count and [h for _, h in seen] == [1]
    seen.clear(), allocated.clear()
    call(stream=Stream(7))
    assert [h for _, h in seen] == [7]
    assert allocated == [7] * count


def test_given_buffers_are_used_as_they_are(world):
    _, allocated = world
    out, ws = torch.zeros(3, 2, 128, dtype=torch.bfloat16), torch.zeros(4096, dtype=torch.uint8)
    call = calls()["attention"][1]
    allocated.clear()
    assert call(out=out, workspace=ws, stream=Stream(7)) is out and not allocated
