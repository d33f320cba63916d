"""Paged calls on a stream that is not the current one, with memory of their own."""
import pytest
import torch

from tests.test_gpu_paged import (DEV, attend_case, cu_of, i32, kda, plan_case, verify_case)

pytestmark = pytest.mark.gpu


def test_attention_keeps_its_workspace_from_the_current_stream():
    """While the current stream allocates and fills memory of the workspace's size, and results of
    earlier calls are dropped, every call gives the same bits."""
    c = attend_case(15, [2, 1, 4], [9000, 70, 5150], 8, 2, 64)
    d = [c[k].to(DEV) for k in ("kc", "vc", "ks", "vs")]
    args = (c["q"].to(DEV), i32(c["cu"]), i32(c["tables"]), i32(c["ctx"]), *d, 4)
    want = kda().paged_attention(*args)
    need = kda().paged_attention_workspace_bytes(8, 2, 4)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    outs = []
    for _ in range(50):
        outs.append(kda().paged_attention(*args, stream=side))
        for _ in range(3):
            torch.full((need,), 255, dtype=torch.uint8, device=DEV)
        if len(outs) > 3:
            del outs[0]
    torch.cuda.synchronize()
    assert all(torch.equal(out, want) for out in outs)
    assert kda().read_device_status() == 0


def test_plan_and_verification_on_another_stream():
    side = torch.cuda.Stream()
    c = plan_case(3, 70, 40, 16, 300)
    args = [i32(c[k]) for k in ("cached", "cu", "tables", "held", "free")] + [i32([c["count"]]), 16, c["t"]]
    want = kda().paged_plan(*args)
    v = verify_case(4, [4, 1, 3], 5000, torch.float32)
    vargs = (v["p"].to(DEV), v["tokens"].to(DEV), i32(cu_of([4, 1, 3])), v["u"].to(DEV), v["e"].to(DEV))
    judged = kda().verify_draft(*vargs, draft_probs=v["q"].to(DEV))
    torch.cuda.synchronize()
    got = [kda().paged_plan(*args, stream=side) for _ in range(20)]
    gone = [kda().verify_draft(*vargs, draft_probs=v["q"].to(DEV), stream=torch.cuda.current_stream())
            for _ in range(3)]
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for g in got for a, b in zip(g, want))
    assert all(torch.equal(a, b) for g in gone for a, b in zip(g, judged))
    assert kda().read_device_status() == 0
