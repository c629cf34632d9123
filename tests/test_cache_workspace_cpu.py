"""forward_cache takes a workspace's size from its element count, so it has to
be contiguous: an expanded or strided tensor counts memory that is not its
own.  On the CPU; the library is never reached."""
import pytest
import torch

from exact_io_aware_20_gb300 import binding


class Reached(Exception):
    pass


class Library:
    def fa_fwd_cache_workspace_size(self, *args):
        return 1 << 16

    def fa_fwd_cache(self, *args):
        raise Reached


class Cache:
    key, device, device_index, _ref = (1, 2, 64, -1), torch.device("cpu"), -1, 0


def call(workspace):
    q = torch.zeros(1, 4, 1, 64, dtype=torch.float16)
    lens = torch.ones(1, dtype=torch.int32)
    binding._forward_cache(q, Cache, lens, True, 0.1, None, None, None, workspace, None)


def test_a_workspace_that_is_not_contiguous_is_refused(monkeypatch):
    monkeypatch.setattr(binding, "load", lambda: Library())
    for bad in (torch.zeros(1, dtype=torch.uint8).expand(1 << 16), torch.zeros(1 << 17, dtype=torch.uint8)[::2],
                torch.zeros(256, 512, dtype=torch.uint8)[:, :256]):
        with pytest.raises(ValueError):
            call(bad)
    for good in (None, torch.zeros(1 << 16, dtype=torch.uint8), torch.zeros(1 << 14, dtype=torch.float32)):
        with pytest.raises(Reached):
            call(good)
