"""A pytest plugin (-p device_status): after every test the device status word is
read, so that one access which a checking build skipped fails the test that made it."""

import pytest


@pytest.fixture(autouse=True)
def device_status_stays_ok(lib):
    import torch
    yield
    torch.cuda.synchronize()
    assert lib.last_device_status() == 0
