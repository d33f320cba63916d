"""Cache appends to pages whose scale says nothing."""
import pytest
import torch

from tests.test_gpu_paged import DEV, i32, kda, pool

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("m", [1, 9, 60])
def test_append_to_a_page_whose_scale_is_nan(m):
    """A begun page without a scale (never written, so NaN) stays NaN: what is added does not give
    its held codes a meaning."""
    g = torch.Generator().manual_seed(m)
    k = torch.randn(m, 2, 128, generator=g).to(torch.bfloat16)
    kc, ks = pool(1, 3, 2, 64)
    ks[1, 0] = float("nan")
    dev = [x.to(DEV) for x in (kc, kc, ks, ks)]
    kda().paged_append(k.to(DEV), k.to(DEV), i32([64 + 3 + i for i in range(m)]), *dev)
    for codes, scale in ((dev[0], dev[2]), (dev[1], dev[3])):
        codes, scale = codes.float().cpu(), scale.cpu()
        assert scale[1, 0].isnan() and codes[1, 0, 3:3 + m].isnan().all()
        assert torch.equal(codes[1, 0, :3], kc.float()[1, 0, :3])
        assert scale[1, 1].isfinite() and codes[1, 1, 3:3 + m].isfinite().all()
    assert kda().read_device_status() == 0
