"""Which workspaces the Softmax branch's calls take, without a GPU."""

import pytest

torch = pytest.importorskip("torch")

from frame_wise_delta_vda_b200 import api


class OnDevice:
    """What the check looks at, of a tensor on device 1."""

    def __init__(self, t):
        self.t = t

    def get_device(self):
        return 1

    def __getattr__(self, name):
        return getattr(self.t, name)


def test_workspace_address_and_bytes():
    t = torch.empty(64, dtype=torch.float32)
    assert api._workspace(None, 1) == (0, 0)
    assert api._workspace(OnDevice(t), 1) == (t.data_ptr(), 256)


@pytest.mark.parametrize("t,index", [
    (torch.empty(64, dtype=torch.uint8), 1),                            # on the CPU
    (OnDevice(torch.empty(64, dtype=torch.uint8)), 0),                  # on another device
    (OnDevice(torch.empty(1, dtype=torch.uint8).expand(1 << 30)), 1),   # fewer bytes than elements
    (OnDevice(torch.empty(64, dtype=torch.uint8)[::2]), 1),
])
def test_workspaces_that_are_refused(t, index):
    with pytest.raises(ValueError):
        api._workspace(t, index)
