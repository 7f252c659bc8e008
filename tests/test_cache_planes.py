"""A cache's planes are on one device (no GPU needed)."""
import pytest

from tests.test_abi import K  # noqa: F401


class Plane:
    is_cuda = True

    def __init__(self, device):
        self.device = device

    def is_contiguous(self):
        return True

    def get_device(self):
        return self.device

    def data_ptr(self):
        return 4096


def test_planes_of_two_devices_are_refused(K):
    c = K.Cache.__new__(K.Cache)
    c.fmt, c.Hk, c.D, c.rope, c.page_size, c.num_pages, c.signs = K.FMT_Q4_HAD32, 2, 256, 0, 16, 4, None
    c.k, c.v, c.k_scale, c.v_scale = (Plane(1) for _ in range(4))
    c.refresh()
    assert c.handle[1] == 1
    c.v = Plane(0)
    with pytest.raises(ValueError, match="one device"):
        c.refresh()
