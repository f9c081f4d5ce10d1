"""Host-only: the scan's workspace is asked for with the tensors' device current, for each device apart."""
import contextlib

import pytest
import torch

from gated_deltanet_linear_03_gb300 import ssm


@pytest.fixture
def devices(monkeypatch):
    """Two devices of different sizes, and the one that is current."""
    now = [0]

    @contextlib.contextmanager
    def device(index):
        before, now[0] = now[0], index
        yield
        now[0] = before

    class Library:
        @staticmethod
        def gdn_ssm_scan_workspace_size(n, T, C, N, G, max_len, st):
            return 1000 * (now[0] + 1) + T

    monkeypatch.setattr(torch.cuda, "device", device)
    monkeypatch.setattr(torch.cuda, "current_device", lambda: now[0])
    monkeypatch.setattr(torch.cuda, "is_available", lambda: True)
    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: now[0], raising=False)
    monkeypatch.setattr(ssm, "load_library", lambda: Library)
    ssm._workspace_size.cache_clear()
    yield now
    ssm._workspace_size.cache_clear()


def test_by_device(devices):
    for turn in range(2):
        for current in (0, 1):
            devices[0] = current
            assert ssm.scan_workspace_size(1, 7, 64, 16, 1) == 1000 * (current + 1) + 7
            for index in (0, 1):
                assert ssm._workspace_size(index, 1, 9, 64, 16, 1, 0) == 1000 * (index + 1) + 9
            assert devices[0] == current
