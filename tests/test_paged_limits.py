"""Sizes near the ends of 31 bits that the kernels' integers would pass.  No GPU needed: refused on
the host."""
import pytest

from tests.test_paged_abi import UNSUPPORTED, attend, lib, verify  # noqa: F401

TOP = 2 ** 31 - 1


@pytest.mark.parametrize("kw", [
    dict(width=TOP // 16), dict(bs=64, width=TOP // 64),  # keys, rounded up to tiles of 128
    dict(t=TOP // 4), dict(t=(TOP - 200) // 4)])            # rows, rounded up to tiles of 256
def test_attention_refuses_what_rounds_past_31_bits(lib, kw):  # noqa: F811
    assert attend(lib, **kw) == UNSUPPORTED


@pytest.mark.parametrize("vocab", [2 ** 30 + 1, TOP])
def test_verification_refuses_a_vocabulary_whose_strides_pass_31_bits(lib, vocab):  # noqa: F811
    assert verify(lib, vocab=vocab) == UNSUPPORTED
