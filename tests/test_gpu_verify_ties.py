"""Draft verification where the races of w / e say nothing."""
import pytest
import torch

from tests.test_gpu_paged import check_verify, kda, verify_case

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("drafted", [True, False])
@pytest.mark.parametrize("vocab", [64, 1001, 8000])
@pytest.mark.parametrize("n", [3, 40])
def test_verify_a_residual_whose_races_are_all_zero(dtype, drafted, vocab, n):
    """Something is left of p - q, but w / e is zero wherever it is (infinite noise; w / e below the
    smallest number): all races tie and token 0 is next, as the definition has it, not the target's
    best."""
    c = verify_case(vocab, [2] * n, vocab, dtype, drafted)
    c["u"][:] = 0.999
    first = torch.arange(0, 2 * n, 2)
    c["tokens"][first + 1] = 7
    c["p"][:] = 0.0
    c["p"][first, 7], c["p"][first, 20], c["p"][first, vocab - 3] = 0.25, 0.125, 2.0 ** -100
    if drafted:
        c["q"][:] = 0.0
        c["q"][first, 7] = 0.5
        c["q"][first, 20] = 0.125
    c["e"][:] = 1.0
    c["e"][:, vocab - 3] = 2.0 ** 80
    c["e"][0, vocab - 3] = float("inf")
    if not drafted:
        c["e"][:, 20] = float("inf")
    c["e"][n - 1, vocab - 3] = 1.0  # and one request whose residual does win
    want = check_verify(c)
    assert want[0] == [1] * n and want[1] == [0] * (n - 1) + [vocab - 3]
    assert kda().read_device_status() == 0


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("n", [35, 36, 37, 38])
def test_verify_where_the_block_size_changes(dtype, n):
    check_verify(verify_case(n, [k % 5 for k in range(n)], 3001, dtype))
    check_verify(verify_case(n, [1 + k % 3 for k in range(n)], 4096, dtype, drafted=False))
    assert kda().read_device_status() == 0
