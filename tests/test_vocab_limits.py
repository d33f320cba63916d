"""Sizes that the C ABI's 32-bit integers do not hold, and devices: what the Python calls of the vocabulary
rows refuse.  No GPU needed: stand-ins for CUDA, and every call is refused or answered on the host."""
import pytest
import torch

from kimi_delta_attention_03_gb300 import KdaError, vocab

WIDE = 2 ** 32 + 8  # its low 32 bits are 8
I32, F32 = torch.int32, torch.float32


@pytest.fixture
def host(monkeypatch):
    from kimi_delta_attention_03_gb300 import build
    build.build()
    monkeypatch.setattr(vocab, "_cuda", lambda name, t: -1)
    monkeypatch.setattr(vocab, "_stream", lambda s, dev: None)


def calls(v, k, t=0):
    x, ids, val = torch.empty(t, v), torch.empty(t, k, dtype=I32), torch.empty(t, k)
    w, stats = torch.empty(t), torch.empty(t, 4)
    return {
        "logprobs": lambda: vocab.token_logprobs(x, top_k=1),
        "loss": lambda: vocab.distill_topk(x, ids, val),
        "bwd": lambda: vocab.distill_topk_bwd(w, x, ids, val, stats),
        "grad": lambda: vocab.distill_topk_grad(x, ids, val, w),
    }


@pytest.mark.parametrize("name", ["logprobs", "loss", "bwd", "grad"])
def test_vocabularies_beyond_31_bits_are_refused(host, name):
    calls(8, 3)[name]()
    for v in (WIDE, 2 ** 31 + 8, 2 ** 32):
        with pytest.raises(KdaError) as e:
            calls(v, 3)[name]()
        assert e.value.status == -2


@pytest.mark.parametrize("name", ["loss", "bwd", "grad"])
def test_entries_beyond_31_bits_are_refused(host, name):
    for k in (WIDE, 2 ** 31 + 8):
        with pytest.raises(KdaError) as e:
            calls(9000, k)[name]()
        assert e.value.status == -2


class On:
    """A tensor on a device, as far as a call looks before it refuses."""
    is_cuda = True

    def __init__(self, index):
        self.index = index

    def get_device(self):
        return self.index


def test_tensors_of_another_device_than_the_current_one_are_refused(monkeypatch):
    """The kernels would run on the current device, with the other's memory."""
    from kimi_delta_attention_03_gb300 import paged
    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: 0)
    there, i = On(1), torch.zeros(1, 1, dtype=I32)
    for call in (lambda: vocab.token_logprobs(there), lambda: vocab.distill_topk(there, i, i),
                 lambda: vocab.distill_topk_bwd(i, there, i, i, i), lambda: vocab.distill_topk_grad(there, i, i, i),
                 lambda: paged.verify_draft(there, i, i, i, i), lambda: paged.paged_append(there, i, i, i, i, i, i),
                 lambda: paged.paged_plan(there, i, i, i, i, i, 16, 1),
                 lambda: paged.paged_attention(there, i, i, i, i, i, i, i, 1)):
        with pytest.raises(ValueError, match="current device"):
            call()
    assert paged._cuda("a call", On(0)) == 0
