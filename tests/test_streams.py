"""Calls given a stream: what they allocate belongs to it.  On the CPU with stand-ins for CUDA's
streams, on the GPU beside allocations of the workspace's size on the current stream."""
import contextlib
import inspect

import pytest
import torch

from kimi_delta_attention_03_gb300 import binding

ALLOCATING = ["fwd_chunked", "fwd_chunked_prologue", "fwd_chunked_checkpoints", "prologue", "prologue_conv",
              "decode_step", "decode_step_prologue", "decode_window", "decode_window_prologue", "bwd"]


class Stream:
    device = torch.device("cpu")


@pytest.fixture
def current(monkeypatch):
    stack = ["caller's"]

    @contextlib.contextmanager
    def on(stream):
        stack.append(stream)
        try:
            yield
        finally:
            stack.pop()

    monkeypatch.setattr(torch.cuda, "stream", on)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda *_: stack[-1])
    return stack


@pytest.mark.parametrize("name", ALLOCATING)
def test_calls_run_with_the_given_stream_as_the_current_one(name, current, monkeypatch):
    call = getattr(binding, name)
    seen = []

    def probe(lib=None):  # the first thing that each call does
        seen.append(current[-1])
        raise InterruptedError

    monkeypatch.setattr(binding, "load_library", probe)
    side = Stream()
    params = inspect.signature(call).parameters
    given = {p: None for p, v in params.items() if v.default is inspect.Parameter.empty}
    for kw, want in (({}, "caller's"), (dict(stream=None), "caller's"), (dict(stream=side), side)):
        with contextlib.suppress(InterruptedError):
            call(**given, **kw)
        assert seen.pop() is want
    assert list(params)[-1] == "stream"
    positional = [p.default if p.default is not inspect.Parameter.empty else None for p in params.values()]
    with contextlib.suppress(InterruptedError):
        call(*positional[:-1], side)
    assert seen.pop() is side and current == ["caller's"]


def test_every_call_that_allocates_is_listed():
    """A call that takes a stream and makes tensors of its own."""
    made = [n for n, f in inspect.getmembers(binding, inspect.isfunction)
            if f.__module__ == binding.__name__ and "stream" in inspect.signature(f).parameters
            and "torch.empty(" in inspect.getsource(inspect.unwrap(f))]
    assert sorted(made) == sorted(ALLOCATING)


@pytest.mark.gpu
@pytest.mark.parametrize("name", ["fwd_chunked", "bwd"])
def test_workspaces_stay_out_of_the_current_streams_hands(name):
    import kimi_delta_attention_03_gb300 as kda
    g = torch.Generator(device="cuda").manual_seed(1)
    lens, heads = [700, 64, 1500], 4
    t = sum(lens)
    q, k, v = (torch.nn.functional.normalize(torch.randn(t, heads, 128, device="cuda", generator=g), dim=-1)
               .to(torch.bfloat16) for _ in range(3))
    la = (-torch.rand(t, heads, 128, device="cuda", generator=g) * 0.1).to(torch.bfloat16)
    beta = torch.rand(t, heads, device="cuda", generator=g).to(torch.bfloat16)
    cu = torch.tensor([0, 700, 764, 2264], dtype=torch.int32, device="cuda")
    args = [q, k, v, la, beta, cu, lens]
    if name == "bwd":
        args.append(torch.randn(t, heads, 128, device="cuda", generator=g))
    call = getattr(kda, name)
    want = call(*args)
    side = torch.cuda.Stream()
    sizes = [1 << p for p in range(16, 27)]
    torch.cuda.synchronize()
    got = []
    for _ in range(6):
        got.append(call(*args, stream=side))
        for size in sizes:
            torch.full((size,), 255, dtype=torch.uint8, device="cuda")
    torch.cuda.synchronize()
    for one in got:
        assert all(torch.equal(a, b) for a, b in zip(one, want))
    assert kda.read_device_status() == 0
