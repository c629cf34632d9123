"""The device-side error word keeps every kind of error until it is reported."""
import pytest
import torch

from exact_io_aware_20_gb300 import binding

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


def test_an_expired_wait_does_not_hide_a_bad_length():
    lib = binding.load()
    assert binding.fa_get_device_status() == binding.FA_OK
    codes = [torch.zeros(2, 1, 16, 64, dtype=torch.uint8, device=DEV) for _ in range(2)]
    one = torch.ones(2, 1, device=DEV)
    cache = binding.Cache(*codes, one, one.clone(), torch.zeros(1, 2, dtype=torch.int32, device=DEV))
    q = torch.zeros(1, 1, 1, 64, dtype=torch.float16, device=DEV)
    for first in (0, 1):
        for which in (first, 1 - first):
            if which:      # 33 tokens where the table has room for 32
                binding.forward_cache(q, cache, torch.tensor([33], dtype=torch.int32, device=DEV), True, 0.1)
            else:
                assert lib.fa_selftest_expired_wait(20000, torch.cuda.current_stream().cuda_stream or None) == binding.FA_OK
        got = [binding.fa_get_device_status() for _ in range(3)]
        assert got == [binding.FA_ERR_TIMEOUT, binding.FA_ERR_CACHE, binding.FA_OK]
