"""Plans from several host threads at once."""
import threading

import pytest
import torch

from tests.test_gpu_paged import DEV, i32, kda, plan_case

pytestmark = pytest.mark.gpu


def test_plans_of_different_sizes_do_not_take_each_others_shared_memory():
    """Plans of 2,200 to 8,192 requests need 50 to 200 KB of shared memory a block; each thread has
    its stream and calls the library as fast as it can."""
    from kimi_delta_attention_03_gb300 import binding
    lib = binding.load_library()
    failed = []

    def serve(c, stream):
        n, t = len(c["cached"]), c["t"]
        keep = [i32(c[k]) for k in ("cached", "cu", "held", "tables", "free")] + [i32([c["count"]])]
        cached, cu, held, tables, free, count = (x.data_ptr() for x in keep)
        outs = [torch.empty(m, dtype=torch.int32, device=DEV) for m in (n, n, 1, t, t)]
        args = (n, len(c["tables"][0]), c["bs"], t, len(c["free"]), cached, cu, None, held, tables, free,
                count, *(x.data_ptr() for x in outs), stream.cuda_stream)
        for _ in range(4000):
            st = lib.kda_paged_plan(*args)
            if st:
                failed.append((n, st))
                break
        stream.synchronize()

    cases = [plan_case(k, n, 1, 16, 40) for k, n in enumerate((8192, 2200, 8000, 3000))]
    torch.cuda.synchronize()
    threads = [threading.Thread(target=serve, args=(c, torch.cuda.Stream())) for c in cases]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not failed
    assert kda().read_device_status() == 0
