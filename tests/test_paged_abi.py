"""Host-side refusals of the paged serving calls, and pins of the plain implementations the GPU
tests compare with.  No GPU needed: every call below is rejected or answered on the host."""
import numpy as np
import pytest
import torch

from tests import paged_reference as ref

OK, INVALID, UNSUPPORTED, WORKSPACE = 0, -1, -2, -3
P = 1 << 20  # a made-up device address: nothing is launched with it


@pytest.fixture(scope="module")
def lib():
    from kimi_delta_attention_03_gb300 import build, binding
    build.build()
    return binding.load_library()


def plan(lib, **kw):
    a = dict(n=4, width=8, bs=16, t=10, cap=5, cached=P, cu=P + 64, release=None, held=P + 128,
             tables=P + 192, free=P + 256, count=P + 320, context=P + 384, held_out=P + 448,
             count_out=P + 512, positions=P + 576, slots=P + 640) | kw
    return lib.kda_paged_plan(*a.values(), None)


@pytest.mark.parametrize("want,kw", [
    (INVALID, dict(n=0)), (INVALID, dict(width=-1)), (INVALID, dict(t=-1)), (INVALID, dict(cap=-1)),
    (UNSUPPORTED, dict(bs=0)), (UNSUPPORTED, dict(bs=24)), (UNSUPPORTED, dict(bs=256)),
    (UNSUPPORTED, dict(n=8193)), (UNSUPPORTED, dict(t=2 ** 31)), (UNSUPPORTED, dict(width=2 ** 27)),
    (INVALID, dict(cached=None)), (INVALID, dict(cu=None)), (INVALID, dict(held=None)),
    (INVALID, dict(tables=None)), (INVALID, dict(free=None)), (INVALID, dict(count=None)),
    (INVALID, dict(context=None)), (INVALID, dict(held_out=None)), (INVALID, dict(count_out=None)),
    (INVALID, dict(positions=None)), (INVALID, dict(slots=None)),
    (INVALID, dict(held_out=P + 128)), (INVALID, dict(count_out=P + 320))])
def test_plan_refuses(lib, want, kw):
    assert plan(lib, **kw) == want


def append(lib, **kw):
    a = dict(t=10, heads=2, bs=16, pages=9, k=P, ks=256, v=P + 64, vs=256, slots=P, kc=P, vc=P + 64,
             kscale=P, vscale=P + 64) | kw
    return lib.kda_paged_append(*a.values(), None)


@pytest.mark.parametrize("want,kw", [
    (OK, dict(t=0)), (INVALID, dict(t=-1)), (INVALID, dict(heads=0)), (INVALID, dict(pages=-1)),
    (UNSUPPORTED, dict(bs=17)), (UNSUPPORTED, dict(pages=2 ** 27)), (UNSUPPORTED, dict(heads=65536, ks=2 ** 24, vs=2 ** 24)),
    (INVALID, dict(k=None)), (INVALID, dict(v=None)), (INVALID, dict(slots=None)),
    (INVALID, dict(kc=None)), (INVALID, dict(vc=None)), (INVALID, dict(kscale=None)),
    (INVALID, dict(vscale=None)), (INVALID, dict(k=P + 8)), (INVALID, dict(kc=P + 8)),
    (INVALID, dict(ks=255)), (INVALID, dict(ks=252)), (INVALID, dict(vs=128)),
    (INVALID, dict(vc=P)), (INVALID, dict(vscale=P))])
def test_append_refuses(lib, want, kw):
    assert append(lib, **kw) == want


def attend(lib, **kw):
    a = dict(n=2, t=3, heads=4, kv=2, bs=16, pages=9, width=4, max_run=2, scale=0.1, q=P, qs=512,
             cu=P, tables=P, ctx=P, kc=P, vc=P, ks=P, vs=P, out=P + 1024, ws=P,
             size=lib.kda_paged_attention_workspace_bytes(4, 2, 2)) | kw
    return lib.kda_paged_attention(*a.values(), None)


@pytest.mark.parametrize("want,kw", [
    (OK, dict(t=0)), (INVALID, dict(n=0)), (INVALID, dict(t=-1)), (INVALID, dict(heads=0)),
    (INVALID, dict(heads=5)), (INVALID, dict(kv=0)), (INVALID, dict(pages=-1)),
    (INVALID, dict(width=-1)), (INVALID, dict(max_run=-1)), (INVALID, dict(scale=0.0)),
    (INVALID, dict(scale=-1.0)), (INVALID, dict(scale=float("inf"))), (INVALID, dict(scale=float("nan"))),
    (UNSUPPORTED, dict(bs=48)), (UNSUPPORTED, dict(t=2 ** 31)), (UNSUPPORTED, dict(pages=2 ** 27)),
    (UNSUPPORTED, dict(width=2 ** 27)), (INVALID, dict(q=None)), (INVALID, dict(cu=None)),
    (INVALID, dict(tables=None)), (INVALID, dict(ctx=None)), (INVALID, dict(kc=None)),
    (INVALID, dict(vc=None)), (INVALID, dict(ks=None)), (INVALID, dict(vs=None)),
    (INVALID, dict(out=None)), (INVALID, dict(out=P)), (INVALID, dict(q=P + 8)),
    (INVALID, dict(out=P + 8)), (INVALID, dict(kc=P + 4)), (INVALID, dict(qs=500)),
    (INVALID, dict(qs=256))])
def test_attention_refuses(lib, want, kw):
    assert attend(lib, **kw) == want


def test_attention_refuses_a_missing_workspace(lib):
    need = lib.kda_paged_attention_workspace_bytes(4, 2, 2)
    if need:
        assert attend(lib, ws=None) == WORKSPACE
        assert attend(lib, ws=P + 128) == WORKSPACE
        assert attend(lib, size=need - 1) == WORKSPACE
    for bad in ((0, 1, 1), (1, 0, 1), (3, 2, 1), (2, 1, -1)):
        assert lib.kda_paged_attention_workspace_bytes(*bad) == 0


def verify(lib, **kw):
    a = dict(n=2, t=5, vocab=10, dt=1, p=P, q=P, tokens=P, cu=P, u=P, e=P, commit=P, nxt=P,
             out=P + 64) | kw
    return lib.kda_verify_draft(*a.values(), None)


@pytest.mark.parametrize("want,kw", [
    (UNSUPPORTED, dict(dt=2)), (UNSUPPORTED, dict(n=65536)), (UNSUPPORTED, dict(t=2 ** 31)),
    (INVALID, dict(n=0)), (INVALID, dict(t=-1)), (INVALID, dict(vocab=0)), (INVALID, dict(p=None)),
    (INVALID, dict(tokens=None)), (INVALID, dict(cu=None)), (INVALID, dict(u=None)),
    (INVALID, dict(e=None)), (INVALID, dict(commit=None)), (INVALID, dict(nxt=None)),
    (INVALID, dict(out=None)), (INVALID, dict(out=P))])
def test_verify_refuses(lib, want, kw):
    assert verify(lib, **kw) == want


def test_python_calls_need_cuda_tensors():
    import kimi_delta_attention_03_gb300 as kda
    i = torch.zeros(2, dtype=torch.int32)
    x = torch.zeros(2, 2, 128, dtype=torch.bfloat16)
    c, s = torch.zeros(3, 2, 16, 128, dtype=torch.float8_e4m3fn), torch.ones(3, 2)
    with pytest.raises(ValueError, match="CUDA"):
        kda.paged_plan(i, i, i[:, None], i, i, i, 16, 2)
    with pytest.raises(ValueError, match="CUDA"):
        kda.paged_append(x, x, i, c, c, s, s)
    with pytest.raises(ValueError, match="CUDA"):
        kda.paged_attention(x, i, i[:1, None], i[:1], c, c, s, s, 1)
    with pytest.raises(ValueError, match="CUDA"):
        kda.verify_draft(s, i, i, s[0], s)


# ------------------------------------------------------------- pins of the plain implementations
def test_nearest_e4m3_is_torchs_conversion():
    """Every bf16 in the format's range, and the 64-bit midpoints between neighbours."""
    x = torch.arange(0, 1 << 16, dtype=torch.int32).to(torch.int16).view(torch.bfloat16).float()
    x = x[x.isfinite() & (x.abs() <= 464)]
    want = x.to(torch.float8_e4m3fn).float()
    keep = want.isfinite()
    np.testing.assert_array_equal(ref.nearest_e4m3(x[keep].numpy()), want[keep].numpy())


def test_scale_is_the_smallest_power_of_two():
    for amax in (448.0, 449.0, 447.9, 1.0, 1.75, 1.7500001, 1e-20, 3e38):
        s = ref.scale_for(amax)
        assert amax <= 448 * s and (s == 2.0 ** -100 or amax > 448 * s / 2)


def test_plan_by_hand():
    """bs 4.  Request 0 (5 cached, 2 pages, run 3) needs none; 1 gives pages 8, 9 back; 2 (new, run
    5) needs two: the end of the list, 9 then 8; 3 (4 cached, run 1) one more: 1."""
    got = ref.plan([5, 7, 0, 4], [0, 3, 3, 8, 9], [[2, 3, 0], [8, 9, 0], [0, 0, 0], [7, 0, 0]],
                   [2, 2, 0, 1], [0, 1, 0, 0], 2, 4, 9, [0, 1, 0, 0])
    assert got[0] == [8, 0, 5, 5] and got[1] == [2, 0, 2, 2] and got[2] == 1
    assert got[3] == [5, 6, 7, 0, 1, 2, 3, 4, 4]
    assert got[4] == [13, 14, 15, 36, 37, 38, 39, 32, 4]


def test_attention_by_hand():
    """Two keys, scores 0 and ln 3: weights 1/4 and 3/4; the first run token sees one key."""
    q = torch.zeros(2, 1, 128, dtype=torch.bfloat16)
    q[:, 0, 0] = 1.0
    kc = torch.zeros(1, 1, 16, 128)
    kc[0, 0, 1, 0] = 2.0
    vc = torch.zeros(1, 1, 16, 128)
    vc[0, 0, 0, 5], vc[0, 0, 1, 5] = 1.0, 3.0
    one = torch.ones(1, 1)
    out, spread, _, _ = ref.attention(q, [0, 2], [[0]], [2], kc, vc, one, 2 * one, sm_scale=np.log(3) / 2)
    assert np.allclose(out[:, 0, 5], [2.0, 5.0]) and np.allclose(spread, out)


def test_verify_by_hand():
    p = np.array([[.5, .5, 0], [.2, .2, .6], [1, 0, 0]], dtype=np.float32)
    q = np.array([[.2, .8, 0], [.9, .05, .05], [0, 0, 0]], dtype=np.float32)
    e = np.array([[1, 1, 4]], dtype=np.float32)
    u = np.array([.6, .3, 0], dtype=np.float32)
    # draft 1: .6 * .8 < .5 holds; draft 0: .3 * .9 < .2 does not; w = (0, .15, .55) / e -> 1
    assert ref.verify(p, q, [7, 1, 0], [0, 3], u, e) == ([2], [1], [1, 1, -1])
    # certain drafts: .6 * 1 < .5 does not; w = (.5, 0, 0)
    assert ref.verify(p, None, [7, 1, 0], [0, 3], u, e) == ([1], [0], [0, -1, -1])
